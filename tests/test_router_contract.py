"""What the router's training calls say about slots without an expert: the balance loss counts
them in K, and the renormalized weights are those over the slots that are left, which is
another function than router_topk's weights with a slot left out."""
import numpy as np
import pytest

from oracle import train as ot
from oracle.layer import router_topk

F32 = np.float32
T, E, K = 12, 9, 4


def _case():
    rng = np.random.default_rng(31)
    logits = rng.standard_normal((T, E)).astype(F32)
    ids, _ = router_topk(logits, K, True)
    dropped = np.zeros((T, K), bool)
    dropped[::2, 1] = dropped[3, :3] = True
    return logits, ids, dropped, rng.standard_normal((T, K)).astype(F32)


def _differences(f, a, h=1e-5):
    g = np.zeros(a.shape)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + h
        up = f()
        a[i] = keep - h
        g[i] = (up - f()) / (2 * h)
        a[i] = keep
    return g


def test_even_load_with_dropped_slots():
    """Every expert in one slot of two: 1 with all slots, 1/2 where every other slot has no expert."""
    ids = np.array([[0, 1], [1, 0]])
    assert np.isclose(ot.router_balance(np.zeros((2, 2)), ids)[3][0], 1.0)
    assert np.isclose(ot.router_balance(np.zeros((2, 2)), [[0, -1], [1, -1]])[3][0], 0.5)


def _wanted(logits, ids, dropped, dw):
    """Gradients by differences: of the weights over the slots that are left, and of router_topk's
    weights (over all K slots) of which the dropped ones are not used."""
    l = logits.astype(np.float64)
    kept = np.where(dropped, 0.0, dw.astype(np.float64))
    left = np.where(dropped, -1, ids)
    return (_differences(lambda: np.sum(kept * ot.topk_weights(l, left, True)), l),
            _differences(lambda: np.sum(kept * ot.topk_weights(l, ids, True)), l))


def test_the_two_ways_to_drop_a_slot():
    logits, ids, dropped, dw = _case()
    over_left, over_all = _wanted(logits, ids, dropped, dw)
    kept = np.where(dropped, 0.0, dw)
    np.testing.assert_allclose(ot.router_backward(logits, np.where(dropped, -1, ids), d_w=dw, renormalize=True)[0],
                               over_left, atol=1e-7)
    np.testing.assert_allclose(ot.router_backward(logits, ids, d_w=kept, renormalize=True)[0], over_all, atol=1e-7)
    assert np.abs(over_left - over_all).max() > 1e-2


@pytest.mark.gpu
def test_the_two_ways_to_drop_a_slot_on_the_gpu():
    """64 u (u = 2^-24) of terms that add up to 16 at most, and 1e-7 of the differences."""
    import torch
    import precision_moe_amd as pm
    from helpers import dev
    logits, ids, dropped, dw = _case()
    over_left, over_all = _wanted(logits, ids, dropped, dw)
    assert np.abs(dw).sum(axis=1).max() < 8
    kept, left = np.where(dropped, F32(0), dw), np.where(dropped, -1, ids).astype(np.int32)
    for i, d, want in ((left, dw, over_left), (ids.astype(np.int32), kept, over_all)):
        got = pm.router_backward(dev(logits), dev(i), d_topk_w=dev(d), renormalize=True)
        torch.cuda.synchronize()
        assert np.abs(got.cpu().numpy() - want).max() < 64 * 16 * 2.0 ** -24 + 1e-7
    even = pm.router_balance(torch.zeros(2, 2, device="cuda"), dev(np.array([[0, -1], [1, -1]], np.int32)))
    assert even.balance.item() == 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("E", [40, 64, 256, 700])
def test_one_expert_in_many_slots_repeats(E):
    """32 slots of a token on two experts: the gradient is the oracle's to 64 u of the sizes and 31
    additions, and has the same bits every time."""
    import torch
    import precision_moe_amd as pm
    from helpers import dev
    rng = np.random.default_rng(E)
    logits, dw = rng.standard_normal((300, E)).astype(F32), rng.standard_normal((300, 32)).astype(F32)
    ids = rng.choice(np.array([3, E - 1], np.int32), (300, 32))
    for renorm in (False, True):
        want, size = ot.router_backward(logits, ids, d_w=dw, renormalize=renorm)
        args = dev(logits), dev(ids)
        first = pm.router_backward(*args, d_topk_w=dev(dw), renormalize=renorm)
        assert np.all(np.abs(first.cpu().numpy() - want) <= (64 + 31) * 2.0 ** -24 * size + 1e-36)
        for _ in range(5):
            assert torch.equal(pm.router_backward(*args, d_topk_w=dev(dw), renormalize=renorm), first)
