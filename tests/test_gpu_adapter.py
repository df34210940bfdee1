"""GPU parity of the adapters with the float64 oracle.

Tolerances, u = 2^-24. A sum over H (or N) of products of BF16 values (exact in FP32) is taken by
waves over at most 256 elements each, then over 8 waves and at most 8 parts, or 4 and 16 (below 528):
  v, du    528 u of the sum of the sizes;
  out, dx  the FP32 result rounded to BF16 (half a step, 2^-8 of its size) plus the error of the low-rank
           term: that of v (du), two BF16 values for scale * v (rest below 2^-16 of it) and at most 256 + 2
           additions: (528 + 260) u + 2^-16 of the sum of the sizes |scale| |up| |down| |x|;
  d_down, d_up  sums over the adapter's tokens (three BF16 values hold all of du and v): tokens + 16
           additions and the error of du: (tokens + 16 + 528) u of the sum of the sizes.
"""
import numpy as np
import pytest

from helpers import bf16_bits, dev, dev_bf16
from oracle import train as ot
from oracle.formats import bf16_to_f32, f32_to_bf16_rne

pytestmark = pytest.mark.gpu
F32 = np.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def pm():
    import torch
    import precision_moe_amd as pm
    assert torch.cuda.is_available()
    return pm


def _bf(rng, *shape, std=1.0):
    return f32_to_bf16_rne((rng.standard_normal(shape) * std).astype(F32))


class Case:
    def __init__(self, T, n, H, N, R, order="mixed", seed=0):
        rng = self.rng = np.random.default_rng(seed + 7 * T + n + H + N + R)
        self.T, self.n, self.H, self.N, self.R = T, n, H, N, R
        ids = rng.integers(-1, n, T)
        if order == "runs":
            ids = np.sort(ids)[::-1]
        elif order == "one":
            ids = np.full(T, n - 1)
        elif order == "none":
            ids = np.full(T, -1)
        self.ids = np.ascontiguousarray(ids).astype(np.int32)
        self.x, self.dy = _bf(rng, T, H), _bf(rng, T, N)
        self.base, self.dx_base = _bf(rng, T, N), _bf(rng, T, H)
        self.down, self.up = _bf(rng, n, R, H, std=H ** -0.5), _bf(rng, n, N, R, std=R ** -0.5)
        self.scale = rng.uniform(-2, 2, n).astype(F32)

    def f(self, name):
        a = getattr(self, name)
        return bf16_to_f32(a).astype(np.float64) if a.dtype == np.uint16 else a.astype(np.float64)

    def d(self, name):
        a = getattr(self, name)
        return dev_bf16(a) if a.dtype == np.uint16 else dev(a)

    def weights(self):
        return self.d("down"), self.d("up"), self.d("scale")

    def forward_want(self, base="base"):
        b = self.f(base) if base else None
        out, v = ot.adapter_forward(self.f("x"), self.ids, self.f("down"), self.f("up"), self.f("scale"), b)
        abs_ = [np.abs(self.f(k)) for k in ("x", "down", "up", "scale")]
        size, v_size = ot.adapter_forward(abs_[0], self.ids, *abs_[1:])
        return out, v, size, v_size


def _close_bf16(got, want, size, what):
    got = bf16_to_f32(bf16_bits(got)).astype(np.float64)
    extra = ((528 + 260) * U + 2.0 ** -16) * size
    err = np.abs(got - want)
    tol = 2.0 ** -8 * (np.abs(want) + extra) + extra + 1e-38
    assert np.all(err <= tol), f"{what}: {(err - tol).max()} at {np.unravel_index((err - tol).argmax(), err.shape)}"


def _check_forward(c, out, v, base="base"):
    want, want_v, size, v_size = c.forward_want(base)
    _close_bf16(out, want, size, "out")
    assert np.all(np.abs(v.cpu().numpy() - want_v) <= 528 * U * v_size)
    plain = c.ids < 0
    if base and plain.any():                       # tokens without an adapter: the bits of base
        assert np.array_equal(bf16_bits(out)[plain], getattr(c, base)[plain])


SIZES = [(1, 1, 16, 16, 8, "one"), (1, 3, 4096, 16, 16, "one"), (2, 1, 16, 4096, 128, "mixed"),
         (16, 16, 512, 272, 16, "mixed"), (63, 5, 1040, 2064, 24, "mixed"), (64, 2, 2064, 1040, 8, "runs"),
         (65, 70, 256, 256, 32, "mixed"), (129, 1, 7168, 528, 64, "one"), (200, 8, 528, 7168, 40, "runs"),
         (257, 300, 320, 336, 72, "mixed"), (300, 4, 2688, 640, 128, "runs"), (130, 2, 16384, 64, 16, "mixed"),
         (70, 3, 48, 16384, 56, "runs"), (77, 4, 128, 128, 104, "none"), (1030, 6, 640, 272, 16, "runs")]


@pytest.mark.parametrize("T,n,H,N,R,order", SIZES)
def test_forward(pm, T, n, H, N, R, order):
    import torch
    c = Case(T, n, H, N, R, order)
    out, v = pm.adapter_forward(c.d("x"), c.d("ids"), *c.weights(), base=c.d("base"))
    torch.cuda.synchronize()
    _check_forward(c, out, v)


@pytest.mark.parametrize("T,n,H,N,R,order", SIZES)
def test_backward(pm, T, n, H, N, R, order):
    import torch
    c = Case(T, n, H, N, R, order)
    v = ot.adapter_forward(c.f("x"), c.ids, c.f("down"), c.f("up"), c.f("scale"))[1].astype(F32)
    dx, d_down, d_up = pm.adapter_backward(c.d("dy"), c.d("x"), dev(v), c.d("ids"), *c.weights(), base=c.d("dx_base"))
    torch.cuda.synchronize()
    dy, x, down, up, scale = (c.f(k) for k in ("dy", "x", "down", "up", "scale"))
    want = ot.adapter_backward(dy, x, v, c.ids, down, up, scale, c.f("dx_base"))
    size = ot.adapter_backward(np.abs(dy), np.abs(x), np.abs(v), c.ids, np.abs(down), np.abs(up), np.abs(scale))
    _close_bf16(dx, want[0], size[0], "dx")
    tokens = np.bincount(c.ids[c.ids >= 0], minlength=n)[:, None, None]
    for got, i in ((d_down, 1), (d_up, 2)):
        assert np.all(np.abs(got.cpu().numpy() - want[i]) <= (tokens + 16 + 528) * U * size[i]), i
    assert not d_down[dev(tokens[:, 0, 0] == 0)].any() and not d_up[dev(tokens[:, 0, 0] == 0)].any()
    plain = c.ids < 0
    assert np.array_equal(bf16_bits(dx)[plain], c.dx_base[plain])


@pytest.mark.parametrize("n,R,order", [(1, 16, "one"), (2, 16, "runs"), (3, 16, "mixed"), (300, 16, "mixed"),
                                       (700, 24, "runs"), (1, 40, "one"), (3, 72, "mixed"), (600, 64, "mixed")])
def test_long_batches(pm, n, R, order):
    """Tokens past one window of the matrices' gradients: with few adapters, whose windows are shared
    by several workgroups, and with many, where one workgroup goes through several windows."""
    import torch
    c = Case(9001, n, 64, 48, R, order)
    v = ot.adapter_forward(c.f("x"), c.ids, c.f("down"), c.f("up"), c.f("scale"))[1].astype(F32)
    _, d_down, d_up = pm.adapter_backward(c.d("dy"), c.d("x"), dev(v), c.d("ids"), *c.weights(), need_dx=False)
    torch.cuda.synchronize()
    args = [c.f(k) for k in ("dy", "x")] + [v, c.ids] + [c.f(k) for k in ("down", "up", "scale")]
    want = ot.adapter_backward(*args)
    size = ot.adapter_backward(*[a if a is c.ids else np.abs(a) for a in args])
    for got, i in ((d_down, 1), (d_up, 2)):
        assert np.all(np.abs(got.cpu().numpy() - want[i]) <= (9001 + 16 + 528) * U * size[i]), (n, i)


def test_gradient_matches_differences(pm):
    """d_down and d_up against central differences of the oracle's loss. The loss is linear in each
    entry, so the difference is exact up to float64; FP32 leaves (T + 544) u of the sizes."""
    import torch
    c = Case(9, 2, 16, 16, 8)
    down, up, dy = c.f("down"), c.f("up"), c.f("dy")
    v = ot.adapter_forward(c.f("x"), c.ids, down, up, c.f("scale"))[1].astype(F32)
    _, d_down, d_up = pm.adapter_backward(c.d("dy"), c.d("x"), dev(v), c.d("ids"), *c.weights())
    torch.cuda.synchronize()
    for got, a in ((d_down, down), (d_up, up)):
        for i in list(np.ndindex(a.shape))[::7]:
            keep, vals = a[i], []
            for step in (0.5, -0.5):
                a[i] = keep + step
                vals.append(np.sum(ot.adapter_forward(c.f("x"), c.ids, down, up, c.f("scale"))[0] * dy))
            a[i] = keep
            assert abs(got[i].item() - (vals[0] - vals[1])) < 1e-3, i


@pytest.mark.parametrize("R", [8, 16, 40, 128])
def test_bits_of_a_token_do_not_depend_on_the_batch(pm, R):
    import torch
    c = Case(700, 9, 1040, 784, R)
    w = c.weights()
    x, ids, base, dy = c.d("x"), c.d("ids"), c.d("base"), c.d("dy")
    out, v = pm.adapter_forward(x, ids, *w, base=base)
    dx, _, _ = pm.adapter_backward(dy, x, v, ids, *w)
    for pick in (torch.arange(333, 334), torch.arange(100, 164), torch.randperm(700)[:257]):
        p = pick.cuda()
        o, vv = pm.adapter_forward(x[p], ids[p], *w, base=base[p])
        d, _, _ = pm.adapter_backward(dy[p], x[p], vv, ids[p], *w)
        assert torch.equal(vv, v[p])
        assert torch.equal(o.view(torch.int16), out[p].view(torch.int16))
        assert torch.equal(d.view(torch.int16), dx[p].view(torch.int16))


def test_forms_of_the_call(pm):
    """base itself as out, no base, int64 ids, views, a side stream, no v, T = 0, repeats."""
    import torch
    c = Case(150, 4, 272, 272, 16)
    w, x, ids, base = c.weights(), c.d("x"), c.d("ids"), c.d("base")
    out, v = pm.adapter_forward(x, ids, *w, base=base)
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))     # noqa: E731
    buf = base.clone()
    got, none = pm.adapter_forward(x, ids, *w, base=buf, out=buf, need_v=False)
    assert none is None and got.data_ptr() == buf.data_ptr() and same(buf, out)
    far = ids.long()
    far[ids < 0] = 1 << 40
    assert same(pm.adapter_forward(x, far, *w, base=base)[0], out)
    xt = x.t().contiguous().t()
    wide = torch.zeros(150, 544, dtype=torch.bfloat16, device="cuda")
    wide[:, ::2] = base
    assert same(pm.adapter_forward(xt, ids, *w, base=wide[:, ::2])[0], out)
    delta, _ = pm.adapter_forward(x, ids, *w)
    _check_forward(c, delta, v, base=None)
    assert not delta[ids < 0].any()
    side = torch.cuda.Stream()
    so, sv = pm.adapter_forward(x, ids, *w, base=base, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert same(so, out) and torch.equal(sv, v)
    dy = c.d("dy")
    full = pm.adapter_backward(dy, x, v, ids, *w)
    again = pm.adapter_backward(dy, x, v, ids, *w)
    assert same(full[0], again[0]) and torch.equal(full[1], again[1]) and torch.equal(full[2], again[2])
    only_dx = pm.adapter_backward(dy, None, None, ids, *w, need_weights=False)
    assert same(only_dx[0], full[0]) and only_dx[1] is None and only_dx[2] is None
    only_w = pm.adapter_backward(dy, x, v, ids, *w, need_dx=False)
    assert only_w[0] is None and torch.equal(only_w[1], full[1]) and torch.equal(only_w[2], full[2])
    acc = c.d("dx_base")
    want = pm.adapter_backward(dy, x, v, ids, *w, base=acc)[0]
    pm.adapter_backward(dy, x, v, ids, *w, base=acc, out=(acc, None, None))
    assert same(acc, want)
    o, vv = pm.adapter_forward(x[:0], ids[:0], *w)
    assert o.shape == (0, 272) and vv.shape == (0, 16)
    dx, dd, du = pm.adapter_backward(dy[:0], x[:0], vv, ids[:0], *w)
    assert dx.shape == (0, 272) and not dd.any() and not du.any()


def test_nan_and_inf_stay_with_their_token_and_adapter(pm):
    import torch
    c = Case(90, 3, 256, 256, 16)
    w, x, ids, base, dy = c.weights(), c.d("x"), c.d("ids"), c.d("base"), c.d("dy")
    out, v = pm.adapter_forward(x, ids, *w, base=base)
    clean = pm.adapter_backward(dy, x, v, ids, *w)
    t = int((ids == 1).nonzero()[0])
    rest = torch.arange(90, device="cuda") != t
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[t, 5] = bad
        o, vv = pm.adapter_forward(y, ids, *w, base=base)
        assert not torch.isfinite(o[t]).all() and torch.equal(o[rest].view(torch.int16), out[rest].view(torch.int16))
        g = pm.adapter_backward(dy, y, vv, ids, *w)
        for i in (1, 2):
            assert torch.equal(g[i][[0, 2]], clean[i][[0, 2]]) and not torch.isfinite(g[i][1]).all()
    broken = w[0].clone(), w[1].clone(), w[2]
    broken[0][2], broken[1][2] = float("nan"), float("inf")           # an adapter that is loaded but broken
    o, _ = pm.adapter_forward(x, ids, *broken, base=base)
    keep = ids != 2
    assert torch.equal(o[keep].view(torch.int16), out[keep].view(torch.int16))
    quiet = x.clone()
    quiet[ids < 0] = float("nan")                                     # tokens without an adapter are not read
    assert torch.equal(pm.adapter_forward(quiet, ids, *w, base=base)[0].view(torch.int16), out.view(torch.int16))


def test_offsets_past_32_bits(pm):
    """T * N above 2^31 elements: the last tokens against the oracle."""
    import torch
    T, N, H, R = (1 << 31) // 16384 + 70, 16384, 16, 8
    c = Case(64, 2, H, N, R)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    x[-64:], ids[-64:] = c.d("x"), c.d("ids")
    out, v = pm.adapter_forward(x, ids, *c.weights())
    torch.cuda.synchronize()
    _check_forward(c, out[-64:].clone(), v[-64:], base=None)
    assert not out[:4].any() and not out[T // 2].any()
    dy = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    dy[-64:] = c.d("dy")
    dx, d_down, _ = pm.adapter_backward(dy, x, v, ids, *c.weights())
    small = pm.adapter_backward(c.d("dy"), c.d("x"), v[-64:].contiguous(), c.d("ids"), *c.weights())
    assert torch.equal(dx[-64:].view(torch.int16), small[0].view(torch.int16))
    torch.testing.assert_close(d_down, small[1], rtol=1e-4, atol=1e-4)
    del out, dy, x
    torch.cuda.empty_cache()


def test_two_captured_calls_and_replays(pm):
    """Two calls that share one workspace, captured one after the other with their backward calls:
    every replay gives the eager bits, with eager work and overwritten buffers in between."""
    import torch
    cs = [Case(200, 3, 256, 512, 16), Case(90, 3, 512, 256, 32)]
    need = max(pm.adapter_workspace_bytes(c.T, c.n, c.H, c.N, c.R, b) for c in cs for b in (False, True))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    eager, args, outs = [], [], []
    for c in cs:
        a = dict(w=c.weights(), x=c.d("x"), ids=c.d("ids"), base=c.d("base"), dy=c.d("dy"))
        o, v = pm.adapter_forward(a["x"], a["ids"], *a["w"], base=a["base"])
        eager.append((o, v, *pm.adapter_backward(a["dy"], a["x"], v, a["ids"], *a["w"])))
        outs.append([torch.empty_like(t) for t in eager[-1]])
        args.append(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for a, o in zip(args, outs):
            pm.adapter_forward(a["x"], a["ids"], *a["w"], base=a["base"], out=o[0], v=o[1], workspace=ws)
            pm.adapter_backward(a["dy"], a["x"], o[1], a["ids"], *a["w"], out=o[2:], workspace=ws)
    for i in range(4):
        for o in outs:
            for t in o:
                t.fill_(i + 2)
        ws.fill_(0xA5 if i % 2 else 0)
        a = args[0]
        assert torch.equal(pm.adapter_forward(a["x"], a["ids"], *a["w"], base=a["base"])[1], eager[0][1])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, eager):
            assert all(torch.equal(p, q) for p, q in zip(got, want)), i
    del g
    torch.cuda.synchronize()


def test_beside_the_layer(pm):
    """moe_forward with adapters is the layer followed by the adapter call, token by token; tokens
    without an adapter keep the layer's bits."""
    import torch
    import synth
    w = synth.WORKLOADS["swiglu"]
    P = pm.prepare_weights(*synth.all_weights(w, device="cuda"))
    x, (tk, wt) = dev_bf16(synth.activations(w)), (dev(a) for a in synth.router(w))
    c = Case(w.T, 5, w.H, w.H, 16)
    plain = pm.moe_forward(x, tk, wt, P)
    want, _ = pm.adapter_forward(x, c.d("ids"), *c.weights(), base=plain)
    got = pm.moe_forward(x, tk, wt, P, adapters=c.weights(), adapter_ids=c.d("ids"))
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    none = dev(c.ids < 0)
    assert torch.equal(got[none].view(torch.int16), plain[none].view(torch.int16))
    assert not torch.equal(got.view(torch.int16), plain.view(torch.int16))


def test_refusals(pm):
    import torch
    c = Case(20, 2, 64, 64, 8)
    w, x, ids, base = c.weights(), c.d("x"), c.d("ids"), c.d("base")
    out = torch.full((20, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pm.PmoeError, match="workspace too small"):
        pm.adapter_forward(x, ids, *w, out=out, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pm.PmoeError, match="not a HIP device pointer|not device memory"):
        pm.adapter_forward(x, ids.cpu(), *w, out=out)
    with pytest.raises(pm.PmoeError, match="overlaps"):
        pm.adapter_forward(x, ids, *w, out=x)
    both = torch.zeros(21, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pm.PmoeError, match="overlaps"):
        pm.adapter_forward(x, ids, *w, base=both[:20], out=both[1:])
    odd = torch.zeros(20 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(20, 64)
    with pytest.raises(pm.PmoeError, match="aligned"):
        pm.adapter_forward(odd, ids, *w, out=out)
    dy, v = c.d("dy"), torch.zeros(20, 8, device="cuda")
    with pytest.raises(pm.PmoeError, match="overlaps"):
        pm.adapter_backward(dy, x, v, ids, *w, out=(dy, None, None))
    with pytest.raises(pm.PmoeError, match="workspace too small"):
        pm.adapter_backward(dy, x, v, ids, *w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pm.PmoeError, match="v overlaps"):
        pm.adapter_forward(x, ids, *w, out=out, v=out.view(torch.float32).view(-1)[:160].view(20, 8))
    grads = torch.zeros(2 * 8 * 64 + 4, device="cuda")
    with pytest.raises(pm.PmoeError, match="d_down or d_up overlaps"):
        pm.adapter_backward(dy, x, v, ids, *w, out=(None, grads[:1024].view(2, 8, 64), grads[4:].view(2, 64, 8)))
    torch.cuda.synchronize()
    assert bool((out == 7).all())


@pytest.mark.parametrize("R,order", [(8, "runs"), (24, "mixed"), (40, "mixed"), (128, "runs")])
def test_long_batches_of_wide_rows(pm, R, order):
    """From T * N (T * H) = 2^24 on a workgroup writes 512 columns: right at a width that is no
    multiple of them, for tokens with and without an adapter, and with the bits of a short call."""
    import torch
    c = Case(1100, 5, 64, 15888, R, order)
    w, x, ids, base = c.weights(), c.d("x"), c.d("ids"), c.d("base")
    out, v = pm.adapter_forward(x, ids, *w, base=base)
    some, _ = pm.adapter_forward(x[7:90], ids[7:90], *w, base=base[7:90])
    none, _ = pm.adapter_forward(x, torch.full_like(ids, -1), *w)
    torch.cuda.synchronize()
    _check_forward(c, out, v)
    assert torch.equal(some.view(torch.int16), out[7:90].view(torch.int16))
    assert not none.any()
    c = Case(1100, 5, 15888, 64, R, order)
    w, ids, dy, dx_base = c.weights(), c.d("ids"), c.d("dy"), c.d("dx_base")
    dx, _, _ = pm.adapter_backward(dy, None, None, ids, *w, base=dx_base, need_weights=False)
    some, _, _ = pm.adapter_backward(dy[7:90], None, None, ids[7:90], *w, base=dx_base[7:90], need_weights=False)
    torch.cuda.synchronize()
    v0 = np.zeros((1100, R), F32)
    args = [c.f(k) for k in ("dy", "x")] + [v0, c.ids] + [c.f(k) for k in ("down", "up", "scale")]
    want = ot.adapter_backward(*args, c.f("dx_base"))[0]
    size = ot.adapter_backward(*[a if a is c.ids else np.abs(a) for a in args])[0]
    _close_bf16(dx, want, size, "dx")
    assert torch.equal(some.view(torch.int16), dx[7:90].view(torch.int16))


@pytest.mark.parametrize("T,n,H,N,R", [(2000, 300, 1040, 784, 72), (1500, 400, 272, 528, 16), (4200, 3, 528, 784, 40)])
def test_runs_repeat(pm, T, n, H, N, R):
    """The same inputs give the same bits, with many workgroups to a CU and with shared windows."""
    import torch
    c = Case(T, n, H, N, R)
    w, x, ids, dy = c.weights(), c.d("x"), c.d("ids"), c.d("dy")

    def call():
        out, v = pm.adapter_forward(x, ids, *w)
        return (out, v, *pm.adapter_backward(dy, x, v, ids, *w))
    first = call()
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(call(), first))
