"""GPU parity of the router's training side with the float64 oracle.

Counts and token numbers are exact. Tolerances, with u = 2^-24 (half a step of FP32):
  softmax  exp's argument l - m is rounded (at most |l - m| u; where |l - m| > 16 the value
           is below 2^-23 of the row's largest, so 16 u covers what is seen), exp and log within
           2 u, the sum over at most 1024 logits in 16 + 6 additions: 64 u in all;
  prob     one sum of positive terms: of the rows of a workgroup a wave adds an eighth at most, then
           4 lanes and 8 waves are added, then the slots of the sequence: rows / 8 + 10 + slots
           additions, below 64 + T / 16 at every size here (rows and slots are about sqrt(T));
  balance  the same and 20 more for the sum over experts and the scaling;
  z        lse enters squared (twice its error), lse itself with 64 u of max(|m|, 1) + log E;
  gradient every term within 64 u of its size, the sizes added up by the oracle.
"""
import numpy as np
import pytest

from helpers import dev
from oracle import train as ot

pytestmark = pytest.mark.gpu
F32 = np.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def pm():
    import torch
    import precision_moe_amd as pm
    assert torch.cuda.is_available()
    return pm


def _case(seed, T, E, K, S=None, pad=False, masked=False, spread=1.5):
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((T, E)) * spread).astype(F32)
    if masked:
        off = rng.random((T, E)) < 0.2
        off[:, rng.permutation(E)[:K]] = False
        logits[off] = -np.inf
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :K].astype(np.int32)
    if pad:
        ids[rng.random(T) < 0.2] = -1
        ids[rng.random((T, K)) < 0.1] = E + 3
    offsets = None
    if S is not None:
        offsets = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)   # the ends stay outside, some are empty
    return rng, logits, ids, offsets


SHAPES = [(1, 4, 1, None), (1, 1, 1, None), (3, 5, 2, 2), (17, 64, 6, None), (64, 65, 8, 1), (250, 33, 4, 40),
          (777, 96, 6, 5), (1000, 256, 8, 300), (300, 1000, 32, 3), (65, 1024, 1, None), (5000, 130, 3, 7)]


def _args(logits, ids, offsets):
    return dev(logits), dev(ids), None if offsets is None else dev(offsets)


@pytest.mark.parametrize("T,E,K,S", SHAPES)
@pytest.mark.parametrize("hard", [False, True])
def test_balance(pm, T, E, K, S, hard):
    import torch
    _, logits, ids, off = _case(T + E, T, E, K, S, pad=hard, masked=hard)
    if hard and T > 2:
        logits[T // 2] = -np.inf                     # a row that the mask leaves empty
    r = pm.router_balance(*_args(logits, ids, off))
    torch.cuda.synchronize()
    counts, tokens, prob, balance, z = ot.router_balance(logits, ids, off)
    assert np.array_equal(r.counts.cpu().numpy(), counts) and np.array_equal(r.tokens.cpu().numpy(), tokens)
    tol = (64 + 64 + T / 16) * U
    np.testing.assert_allclose(r.prob.cpu().numpy(), prob, rtol=tol, atol=1e-30)
    np.testing.assert_allclose(r.balance.cpu().numpy(), balance, rtol=tol + 20 * U)
    top = np.abs(np.where(np.isfinite(logits), logits, 0)).max() + np.log(E) + 1
    np.testing.assert_allclose(r.z.cpu().numpy(), z, rtol=tol, atol=2 * 64 * U * top * top)


@pytest.mark.parametrize("T,E,K,S", SHAPES)
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("parts", ["all", "balance", "z", "w"])
def test_gradient(pm, T, E, K, S, renorm, parts):
    import torch
    rng, logits, ids, off = _case(T + 3 * E, T, E, K, S, pad=True, masked=True)
    if T > 2:
        logits[T // 2] = -np.inf
    n_seq = 1 if off is None else off.size - 1
    counts, tokens, *_ = ot.router_balance(logits, ids, off)
    db, dz = rng.standard_normal(n_seq).astype(F32), rng.standard_normal(n_seq).astype(F32)
    dw = rng.standard_normal((T, K)).astype(F32)
    db, dz, dw = (a if parts in ("all", name) else None for a, name in ((db, "balance"), (dz, "z"), (dw, "w")))
    want, size = ot.router_backward(logits, ids, counts, tokens, db, dz, dw, renorm, off)
    lg, tk, o = _args(logits, ids, off)
    got = pm.router_backward(lg, tk, counts=dev(counts.astype(np.int32)), tokens=dev(tokens.astype(np.int32)),
                             d_balance=None if db is None else dev(db), d_z=None if dz is None else dev(dz),
                             d_topk_w=None if dw is None else dev(dw), renormalize=renorm, seq_offsets=o)
    torch.cuda.synchronize()
    err = np.abs(got.cpu().numpy() - want)
    assert np.all(err <= 64 * U * size + 1e-36), (err - 64 * U * size).max()


def test_gradient_matches_differences_of_the_losses(pm):
    """The GPU gradient against central differences of the oracle's losses (counts held)."""
    import torch
    rng, logits, ids, _ = _case(5, 6, 9, 3)
    counts, tokens, *_ = ot.router_balance(logits, ids)
    dw, h = rng.standard_normal(ids.shape).astype(F32), 1e-5
    got = pm.router_backward(dev(logits), dev(ids), counts=dev(counts.astype(np.int32)),
                             tokens=dev(tokens.astype(np.int32)), d_balance=dev(np.ones(1, F32)),
                             d_z=dev(np.full(1, 0.5, F32)), d_topk_w=dev(dw), renormalize=True)
    torch.cuda.synchronize()
    l = logits.astype(np.float64)

    def loss():
        _, n, P, _, z = ot.router_balance(l, ids)
        return (9 * np.sum(counts / (n * 3) * P / n) + 0.5 * z[0] +
                np.sum(dw.astype(np.float64) * ot.topk_weights(l, ids, True)))

    for t in range(6):
        for e in range(9):
            keep = l[t, e]
            l[t, e] = keep + h
            up = loss()
            l[t, e] = keep - h
            down = loss()
            l[t, e] = keep
            # the difference itself is good to 1e-9; FP32 adds 64 u of terms of size 10
            assert abs(got[t, e].item() - (up - down) / (2 * h)) < 1e-8 + 640 * U


def test_lowest_values_and_nan(pm):
    """Logits masked by FP32's lowest value behave as numbers (probability 0 beside ordinary ones);
    a NaN or +inf logit shows in its own token's results and in its own sequence only."""
    import torch
    _, logits, ids, _ = _case(11, 40, 70, 4)
    low = logits.copy()
    low[:, 60:] = np.finfo(F32).min
    ids = np.argsort(-low, axis=1, kind="stable")[:, :4].astype(np.int32)
    off = np.array([0, 20, 40], np.int32)
    r = pm.router_balance(*_args(low, ids, off))
    assert torch.isfinite(r.balance).all() and not r.prob[:, 60:].any()
    clean = pm.router_backward(dev(low), dev(ids), counts=r.counts, tokens=r.tokens,
                               d_balance=torch.ones(2, device="cuda"), seq_offsets=dev(off))
    for bad in (np.nan, np.inf):
        l = low.copy()
        l[25, 3] = bad
        q = pm.router_balance(*_args(l, ids, off))
        assert torch.isnan(q.balance[1]) and torch.equal(q.balance[:1], r.balance[:1])
        assert torch.equal(q.prob[0], r.prob[0]) and torch.equal(q.counts, r.counts)
        g = pm.router_backward(dev(l), dev(ids), counts=r.counts, tokens=r.tokens,
                               d_balance=torch.ones(2, device="cuda"), seq_offsets=dev(off))
        assert torch.isnan(g[25]).any()
        rest = [t for t in range(40) if t != 25]
        assert torch.equal(g[rest], clean[rest])


@pytest.mark.parametrize("E", [5, 64, 200, 1024])
def test_padding_tokens_may_hold_anything(pm, E):
    """Logits of tokens without a valid id do not reach any result, whatever they are."""
    import torch
    rng, logits, ids, off = _case(29, 150, E, 3, 4)
    pad = rng.random(150) < 0.3
    ids[pad] = -1
    zero, wild = logits.copy(), logits.copy()
    zero[pad] = 0.0
    wild[pad] = rng.choice(np.array([np.nan, np.inf, -np.inf, 3e38, 700.0], F32), (int(pad.sum()), E))
    dw = dev(rng.standard_normal(ids.shape).astype(F32))
    a, b = pm.router_balance(*_args(zero, ids, off)), pm.router_balance(*_args(wild, ids, off))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    one = torch.ones(4, device="cuda")
    for renorm in (False, True):
        g, h = (pm.router_backward(dev(l), dev(ids), counts=a.counts, tokens=a.tokens, d_balance=one, d_z=one,
                                   d_topk_w=dw, renormalize=renorm, seq_offsets=dev(off)) for l in (zero, wild))
        assert torch.equal(g, h) and not g[dev(pad)].any()


def test_int64_ids_repeats_views_and_empty_batch(pm):
    import torch
    _, logits, ids, off = _case(13, 333, 100, 5, 6, pad=True)
    lg, tk, o = _args(logits, ids, off)
    r = pm.router_balance(lg, tk, o)
    far = ids.astype(np.int64)
    far[ids < 0] = -(1 << 40)
    far[ids >= 100] = 1 << 40
    for again in (pm.router_balance(lg, dev(far), o), pm.router_balance(lg, tk, o)):
        assert all(torch.equal(a, b) for a, b in zip(r, again))       # the same bits every time
    wide = torch.zeros(333, 200, device="cuda")
    wide[:, ::2] = lg
    assert all(torch.equal(a, b) for a, b in zip(r, pm.router_balance(wide[:, ::2], tk.t().contiguous().t(), o)))
    twice = ids.copy()
    twice[:, 1] = twice[:, 0]                                         # one expert in two slots
    got = pm.router_balance(lg, dev(twice), o)
    assert np.array_equal(got.counts.cpu().numpy(), ot.router_balance(logits, twice, off)[0])
    dw = np.random.default_rng(1).standard_normal(ids.shape).astype(F32)
    for renorm in (False, True):
        want, size = ot.router_backward(logits, twice, d_w=dw, renormalize=renorm)
        g = pm.router_backward(lg, dev(twice), d_topk_w=dev(dw), renormalize=renorm).cpu().numpy()
        assert np.all(np.abs(g - want) <= 64 * U * size + 1e-36)
    none = pm.router_balance(lg[:0], tk[:0], torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert not any(t.any() for t in none) and none.counts.shape == (3, 100)
    assert pm.router_backward(lg[:0], tk[:0], d_topk_w=torch.zeros(0, 5, device="cuda")).shape == (0, 100)
    buf = lg.clone()                                                  # in place
    dwt = dev(dw)
    want = pm.router_backward(lg, tk, d_topk_w=dwt)
    pm.router_backward(buf, tk, d_topk_w=dwt, out=buf)
    assert torch.equal(buf, want)


def test_counts_of_several_ranks(pm):
    """Counts, tokens and probability sums of two halves add up to those of the whole batch."""
    import torch
    _, logits, ids, _ = _case(17, 600, 48, 4, pad=True)
    lg, tk, _ = _args(logits, ids, None)
    whole, a, b = pm.router_balance(lg, tk), pm.router_balance(lg[:250], tk[:250]), pm.router_balance(lg[250:], tk[250:])
    assert torch.equal(a.counts + b.counts, whole.counts) and torch.equal(a.tokens + b.tokens, whole.tokens)
    torch.testing.assert_close(a.prob + b.prob, whole.prob, rtol=(64 + 600 / 16) * U, atol=0)
    g = torch.ones(1, device="cuda")
    full = pm.router_backward(lg, tk, counts=whole.counts, tokens=whole.tokens, d_balance=g, d_z=g)
    part = pm.router_backward(lg[250:], tk[250:], counts=whole.counts, tokens=whole.tokens, d_balance=g, d_z=g)
    assert torch.equal(part, full[250:])


def test_refusals(pm):
    import torch
    _, logits, ids, _ = _case(19, 40, 16, 2)
    lg, tk, _ = _args(logits, ids, None)
    out = pm.router_balance(lg, tk)
    for t in out:
        t.fill_(7)
    with pytest.raises(pm.PmoeError, match="workspace too small"):
        pm.router_balance(lg, tk, out=out, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pm.PmoeError, match="not a HIP device pointer|not device memory"):
        pm.router_balance(lg, tk.cpu(), out=out)
    with pytest.raises(pm.PmoeError, match="not a HIP device pointer|not device memory"):
        pm.router_backward(lg, tk, d_topk_w=torch.zeros(40, 2))
    E = lg.shape[1]
    rows = torch.zeros(41, E, device="cuda")
    with pytest.raises(pm.PmoeError, match="overlaps"):
        pm.router_backward(rows[:40], tk, d_topk_w=torch.zeros(40, tk.shape[1], device="cuda"), out=rows[1:])
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in out)


def test_graph_and_side_stream(pm):
    """Captured, the calls replay to the eager bits, with eager calls and overwritten outputs in
    between; on a side stream they give them too."""
    import torch
    _, logits, ids, off = _case(23, 2000, 96, 6, 9, pad=True)
    lg, tk, o = _args(logits, ids, off)
    one = torch.ones(9, device="cuda")
    eager = pm.router_balance(lg, tk, o)
    grad = pm.router_backward(lg, tk, counts=eager.counts, tokens=eager.tokens, d_balance=one, d_z=one, seq_offsets=o)
    side = torch.cuda.Stream()
    got = pm.router_balance(lg, tk, o, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    ws = torch.empty(pm.router_balance_workspace_bytes(2000, 6, 96, 9), dtype=torch.uint8, device="cuda")
    out = pm.RouterBalance(*(torch.empty_like(t) for t in eager))
    dl = torch.empty_like(grad)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pm.router_balance(lg, tk, o, out=out, workspace=ws)
        pm.router_backward(lg, tk, counts=out.counts, tokens=out.tokens, d_balance=one, d_z=one, seq_offsets=o, out=dl)
    for i in range(4):
        for t in (*out, dl):
            t.fill_(i + 3)
        ws.fill_(0xA5)
        assert torch.equal(pm.router_balance(lg, tk, o).prob, eager.prob)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)) and torch.equal(dl, grad), i
    del g
    torch.cuda.synchronize()


def test_most_tokens(pm):
    import torch
    # one expert: p = 1, lse = the logit 0.5, so every sum is exact in FP32
    T, S, each = (1 << 30) - 1, 65536, 1 << 14
    lg = torch.full((T, 1), 0.5, device="cuda")
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    off = (torch.arange(S + 1, device="cuda", dtype=torch.int64) * each).clamp(max=T).to(torch.int32)
    r = pm.router_balance(lg, ids, seq_offsets=off)
    n = off[1:] - off[:-1]
    assert torch.equal(r.tokens, n) and torch.equal(r.counts[:, 0], n) and torch.equal(r.prob[:, 0], n.float())
    assert torch.equal(r.balance, torch.ones(S, device="cuda")) and torch.equal(r.z, torch.full_like(r.z, 0.25))
    d = pm.router_backward(lg, ids, tokens=r.tokens, d_z=torch.ones(S, device="cuda"), seq_offsets=off, out=lg)
    assert bool((d[:(S - 1) * each] == 1.0 / each).all())
    assert bool(((d[(S - 1) * each:] * (each - 1) - 1).abs() <= 4 * 2.0 ** -24).all())
