"""The adapter calls at the edges of what they accept: arguments that only some outputs need."""
import pytest

from helpers import dev, dev_bf16
from test_gpu_adapter import Case, pm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_down_has_to_be_on_the_device_without_dx_too(pm):  # noqa: F811
    import torch
    c = Case(20, 2, 64, 64, 8)
    down, up, scale = c.weights()
    x, ids, dy, v = c.d("x"), c.d("ids"), c.d("dy"), torch.zeros(20, 8, device="cuda")
    with pytest.raises(pm.PmoeError, match="down is not"):
        pm.adapter_backward(dy, x, v, ids, down.cpu(), up, scale, need_dx=False)
    _, d_down, d_up = pm.adapter_backward(dy, x, v, ids, down, up, scale, need_dx=False)
    assert d_down.shape == down.shape and d_up.shape == up.shape


def test_layer_adapters_that_are_refused_leave_out_alone(pm):  # noqa: F811
    """`out` is not written by the layer either; views and int64 ids that are accepted give the layer
    followed by the adapter call."""
    import torch
    import synth
    w = synth.WORKLOADS["tiny"]
    P = pm.prepare_weights(*synth.all_weights(w, device="cuda"))
    x, (tk, wt) = dev_bf16(synth.activations(w)), (dev(a) for a in synth.router(w))
    c = Case(w.T, 3, w.H, w.H, 8)
    down, up, scale = c.weights()
    ids = c.d("ids").long()
    out = torch.full((w.T, w.H), 7.0, dtype=torch.bfloat16, device="cuda")
    shifted = torch.empty(down.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(down.shape)
    for adapters in ((shifted, up, scale), (down.cpu(), up, scale)):
        with pytest.raises(ValueError, match="aligned|on the device of x"):
            pm.moe_forward(x, tk, wt, P, out=out, adapters=adapters, adapter_ids=ids)
    ws = torch.empty(pm.adapter_workspace_bytes(w.T, 3, w.H, w.H, 8) + 8, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="aligned"):
        pm.moe_forward(x, tk, wt, P, out=out, adapters=(down, up, scale), adapter_ids=ids, adapter_workspace=ws[8:])
    torch.cuda.synchronize()
    assert bool((out == 7).all())
    want, _ = pm.adapter_forward(x, ids, down, up, scale, base=pm.moe_forward(x, tk, wt, P))
    wide = torch.zeros(3, 8, 2 * w.H, dtype=torch.bfloat16, device="cuda")
    wide[:, :, ::2] = down
    far = torch.stack((ids, ids), 1)[:, 0]
    side = torch.cuda.Stream()
    for stream in (None, side):
        got = pm.moe_forward(x, tk, wt, P, out=out, adapters=(wide[:, :, ::2], up, scale), adapter_ids=far, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        assert got is out and torch.equal(got.view(torch.int16), want.view(torch.int16))
        out.fill_(7)


@pytest.mark.parametrize("R", [8, 24, 64, 128])
def test_low_rank_values_at_the_end_of_the_range(pm, R):  # noqa: F811
    """scale * v and scale * du between BF16's largest value and FP32's (2^128 (1 - 2^-10), whose
    nearest BF16 value would be infinite) enter the second product as finite values; infinite
    ones give infinite results. Few bits are set in any value, so the results are exact."""
    import torch

    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")
    H, N = 32, 48
    ids, r = torch.zeros(3, dtype=torch.int32, device="cuda"), R - 1
    scale = torch.full((1,), 2.0 ** 28 * (1 - 2.0 ** -10), device="cuda")
    x, down, up = zeros(3, H), zeros(1, R, H), zeros(1, N, R)
    x[:, 5], down[0, r, 5], up[0, :, r] = 2.0 ** 100, 1.0, 2.0 ** -120
    out, v = pm.adapter_forward(x, ids, down, up, scale)
    assert bool((v[:, r] == 2.0 ** 100).all()) and bool((out == 256).all())      # 255.75 in BF16
    x[1, 5], down[0, :, 5], up[0, :, :] = float("inf"), 1.0, 2.0 ** -120         # without inf * 0
    out, _ = pm.adapter_forward(x, ids, down, up, scale)
    assert bool((out[[0, 2]] == 256 * R).all()) and bool((out[1] == float("inf")).all())
    dy, down, up = zeros(3, N), zeros(1, R, H), zeros(1, N, R)
    dy[:, 7], up[0, 7, r], down[0, r, :] = -2.0 ** 100, 1.0, 2.0 ** -120
    dx, _, _ = pm.adapter_backward(dy, None, None, ids, down, up, scale, need_weights=False)
    assert bool((dx == -256).all())


@pytest.mark.parametrize("R", [16, 40])
def test_infinite_entries_stay_where_they_enter(pm, R):  # noqa: F811
    """An infinite entry of a matrix, x or dy makes every result that it enters infinite or NaN, and
    changes no bit of the others."""
    import torch
    c = Case(50, 3, 64, 96, R)
    down, up, scale = c.weights()
    x, dy, ids = c.d("x"), c.d("dy"), c.d("ids")
    out, v = pm.adapter_forward(x, ids, down, up, scale)
    dx, d_down, d_up = pm.adapter_backward(dy, x, v, ids, down, up, scale)

    def check(got, want, *hit):
        touched = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
        touched[hit] = True
        assert touched.any() and not torch.isfinite(got[touched]).any()
        assert torch.equal(got[~touched], want[~touched])
    mine, t = (ids == 1).nonzero()[:, 0], int((ids == 1).nonzero()[2])
    inf = float("inf")
    bad_up, bad_down, bad_x, bad_dy = up.clone(), down.clone(), x.clone(), dy.clone()
    bad_up[1, 5, 3], bad_down[1, 2, 7], bad_x[t, 9], bad_dy[t, 11] = inf, -inf, inf, -inf
    check(pm.adapter_forward(x, ids, down, bad_up, scale)[0], out, mine, 5)
    got = pm.adapter_backward(dy, x, v, ids, bad_down, up, scale)
    check(got[0], dx, mine, 7)
    assert torch.equal(got[1], d_down) and torch.equal(got[2], d_up)
    got = pm.adapter_backward(dy, bad_x, v, ids, down, up, scale)
    check(got[1], d_down, 1, slice(None), 9)
    assert torch.equal(got[0], dx) and torch.equal(got[2], d_up)
    check(pm.adapter_backward(bad_dy, x, v, ids, down, up, scale)[2], d_up, 1, 11)


def test_one_workspace_for_the_layer_and_its_adapters(pm):  # noqa: F811
    """The adapters run after the layer, so both may use one workspace; no tokens are a call too; and
    captured, the whole call replays to the eager bits."""
    import torch
    import synth
    w = synth.WORKLOADS["tiny"]
    P = pm.prepare_weights(*synth.all_weights(w, device="cuda"))
    x, (tk, wt) = dev_bf16(synth.activations(w)), (dev(a) for a in synth.router(w))
    c = Case(w.T, 3, w.H, w.H, 8)
    adapters, ids = c.weights(), c.d("ids")
    want = pm.moe_forward(x, tk, wt, P, adapters=adapters, adapter_ids=ids)
    need = max(pm.moe_workspace_bytes(w.T, w.K, w.E, w.H, w.I, P.act), pm.adapter_workspace_bytes(w.T, 3, w.H, w.H, 8))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)

    def call():
        out.fill_(7)
        pm.moe_forward(x, tk, wt, P, adapters=adapters, adapter_ids=ids, workspace=ws, adapter_workspace=ws, out=out)
    call()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    none = pm.moe_forward(x[:0], tk[:0], wt[:0], P, adapters=adapters, adapter_ids=ids[:0])
    assert none.shape == (0, w.H)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        out.fill_(i)
        ws.fill_(i)
        assert torch.equal(pm.adapter_forward(x, ids, *adapters)[0], pm.adapter_forward(x, ids, *adapters)[0])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), i
    del g
    torch.cuda.synchronize()
