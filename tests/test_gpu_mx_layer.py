"""An MXFP4 expert layer and its gradient, put together from the library's calls as a user would:
router front -> order of the routes -> quantized tokens -> gathered first product -> activation with
8-bit checkpoint -> second product -> finalize, and back to the tokens and the routing weights. Each
step is compared with the float64 oracle fed with the tensors that the GPU's own steps produced, within its
own call's tolerance (U = 2^-24, half a step of BF16 = 2^-8), so that the chain's wiring is what is tested.
The same layer is then captured in graphs, run on other streams and from strided tensors."""
import numpy as np
import pytest

from helpers import bf16_bits, dev
from oracle import mx
from oracle import train as ot
from oracle.formats import bf16_to_f32

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def pm():
    import torch
    import precision_moe_amd as pm
    assert torch.cuda.is_available()
    return pm


def _np(t):
    import torch
    if t.dtype == torch.bfloat16:
        return bf16_to_f32(bf16_bits(t.contiguous())).astype(np.float64)
    a = t.cpu().numpy()
    return a.astype(np.float64) if a.dtype == np.float32 else a


class Layer:
    """Weights, inputs and buffers of one layer; held = experts of this rank, the first of them `first`."""

    def __init__(self, pm, T, H, I, E, K, act, limit=0.0, first=0, held=None, seed=1):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
        self.pm, self.T, self.H, self.I, self.K, self.limit, self.first = pm, T, H, I, K, limit, first
        self.E = E if held is None else held
        self.act, self.name = (pm.ACT_SWIGLU, "swiglu") if act == "swiglu" else (pm.ACT_RELU2, "relu2")
        N1 = 2 * I if act == "swiglu" else I
        self.w1 = pm.mx_quantize(rand(self.E, N1, H, std=H ** -0.5))
        self.w2 = pm.mx_quantize(rand(self.E, H, I, std=I ** -0.5))
        self.x, self.dout = rand(T, H).bfloat16(), rand(T, H).bfloat16()
        self.ids, self.wt = pm.router_topk(rand(T, E), K)

    def forward(self, **kw):
        pm = self.pm
        o = pm.permute_tokens(None, self.ids, self.E, expert_offset=self.first, **kw)
        self.order, off = o, o.expert_offsets
        self.xq = pm.mx_quantize(self.x, **kw)
        self.y = pm.mx_grouped_gemm(*self.xq, *self.w1, off, route_of_row=o.route_of_row, topk=self.K, **kw)
        self.h = pm.mx_activation(self.y, self.act, swiglu_limit=self.limit, checkpoint=True, row_count=off[-1:], **kw)
        self.z = pm.mx_grouped_gemm(*self.h[:2], *self.w2, off, **kw)
        self.out = pm.finalize(self.z, o.row_of_route, self.wt, **kw)
        return self.out

    def backward(self, **kw):
        pm, o = self.pm, self.order
        off = o.expert_offsets
        self.dw, self.dz = pm.finalize_backward(self.dout, self.z, o.row_of_route, self.wt, **kw)
        self.dh = pm.mx_grouped_gemm_backward(self.dz, *self.w2, off, **kw)
        self.dy = pm.mx_activation_backward(self.dh, *self.h[2:], self.act, swiglu_limit=self.limit, row_count=off[-1:], **kw)
        self.drows = pm.mx_grouped_gemm_backward(self.dy, *self.w1, off, **kw)
        self.dx = pm.permute_tokens_backward(self.drows, o.row_of_route, self.K, **kw)
        return self.dx, self.dw


def _near(got, want, size, slack, half=HALF):
    s = slack * size
    assert np.all(np.abs(got - want) <= s + half * (np.abs(want) + s))


@pytest.mark.parametrize("T,H,I,E,K,act,limit,first,held", [
    (1, 64, 32, 4, 1, "relu2", 0.0, 0, None), (37, 256, 128, 16, 4, "swiglu", 2.5, 0, None),
    (300, 160, 96, 6, 3, "swiglu", 0.0, 0, None), (300, 512, 384, 32, 6, "swiglu", 1.0, 8, 8),
    (2048, 128, 256, 4, 2, "relu2", 0.0, 0, None), (9, 96, 64, 64, 2, "swiglu", 0.0, 63, 1), (500, 64, 64, 64, 8, "swiglu", 0.0, 60, 4)])
def test_layer_and_gradient(pm, T, H, I, E, K, act, limit, first, held):
    L = Layer(pm, T, H, I, E, K, act, limit, first, held)
    L.forward()
    L.backward()
    n = L.order.expert_offsets.cpu().numpy()
    row, route, off = mx.permute(_np(L.ids), L.E, first)
    R = off[-1]
    assert np.array_equal(n, off) and np.array_equal(_np(L.order.row_of_route), row)
    assert np.array_equal(_np(L.order.route_of_row)[:R], route)
    xq = [_np(t) for t in L.xq]
    for got, want in zip(xq, mx.quantize(_np(L.x))):
        assert np.array_equal(got, want)
    w1, w2 = mx.dequantize(*map(_np, L.w1)), mx.dequantize(*map(_np, L.w2))
    a = mx.dequantize(*xq)[route // K]
    y = _np(L.y)[:R]
    _near(y, mx.grouped_gemm(a, w1, off), mx.grouped_gemm(abs(a), abs(w1), off), 2 * H * U)
    hq, y8 = mx.quantize(mx.activation(y, L.name, limit)), mx.quantize(y, "e4m3")
    for got, want in zip(L.h, (*hq, *y8)):
        assert np.array_equal(_np(got)[:R], want)
    h = mx.dequantize(*hq)
    z = _np(L.z)[:R]
    _near(z, mx.grouped_gemm(h, w2, off), mx.grouped_gemm(abs(h), abs(w2), off), 2 * I * U)
    wt, dout = _np(L.wt), _np(L.dout)
    on = (row >= 0).reshape(T, K)
    zt = np.where(on[..., None], z[np.where(on, row.reshape(T, K), 0)] if R else 0, 0.0)
    _near(_np(L.out), (wt[..., None] * zt).sum(1), abs(wt[..., None] * zt).sum(1), 2 * K * U)
    dw, dz, size = ot.finalize_backward(dout, z, row, wt)
    assert np.all(np.abs(_np(L.dw) - dw) <= (H / 64 + 16) * U * size)
    got = _np(L.dz)[:R]
    assert np.all(np.abs(got - dz) <= (HALF + 2 * U) * np.abs(dz))
    dz, dh = got, _np(L.dh)[:R]
    _near(dh, mx.grouped_gemm_backward(dz, w2, off), mx.grouped_gemm_backward(abs(dz), abs(w2), off), 2 * H * U)
    v, dy = mx.dequantize(*y8, "e4m3"), _np(L.dy)[:R]
    want = mx.activation_backward(dh, v, L.name, limit)
    size = np.abs(want)
    if act == "swiglu":
        g, u = np.split(abs(v), 2, 1)
        g, u = (np.minimum(g, limit), np.minimum(u, limit)) if limit else (g, u)
        size = np.concatenate([abs(dh) * u * (1 + g), abs(dh) * g], 1)
    _near(dy, want, size, 32 * U)
    drows = _np(L.drows)[:R]
    _near(drows, mx.grouped_gemm_backward(dy, w1, off), mx.grouped_gemm_backward(abs(dy), abs(w1), off), 2 * w1.shape[1] * U)
    _near(_np(L.dx), mx.permute_backward(drows, row, K), mx.permute_backward(abs(drows), row, K), K * U)


def _bits(t):
    import torch
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def test_gradient_against_differences(pm):
    """d <dout, layer(y)> / dy of the second half, from the values of h before their codes: the difference over a
    step of 2^-10 of float64 y (the checkpoint's values) agrees with dy to the step's second-order term. Products are linear:
    their gradient is the transposed product, tested exactly elsewhere."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)
    y = torch.randn(40, 128, generator=g, device="cuda").bfloat16()
    dh = torch.randn(40, 64, generator=g, device="cuda").bfloat16()
    _, _, y8, y8_sf = pm.mx_activation(y, pm.ACT_SWIGLU, checkpoint=True)
    dy = _np(pm.mx_activation_backward(dh, y8, y8_sf, pm.ACT_SWIGLU))
    v, d, step = _np(pm.mx_dequantize(y8, y8_sf, "e4m3", dtype=torch.float32)), _np(dh), 2.0 ** -10
    for i in range(0, 128, 9):
        e = np.zeros_like(v)
        e[:, i] = step
        diff = (d * (mx.activation(v + e, "swiglu") - mx.activation(v - e, "swiglu"))).sum(1) / (2 * step)
        # |third derivative of silu| < 1, up and dh below 2^3 here: the difference is off by step^2 / 6 * 2^6;
        # the terms of dy are below 8 * 8 * (1 + 8)
        assert np.abs(v).max() < 8 and np.abs(d).max() < 8
        assert np.all(np.abs(dy[:, i] - diff) <= HALF * (np.abs(diff) + 2 ** -16) + step ** 2 * 64 / 6 + 576 * 32 * U)


# ----------------------------------------------------------------------------- graphs and streams
def _capture(fn):
    import torch
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = fn()
    torch.cuda.synchronize()
    return g, res


@pytest.mark.parametrize("T,H,I,E,K", [(16, 256, 128, 8, 2), (700, 256, 384, 16, 4), (5000, 1024, 768, 8, 4)])
def test_captured_layer(pm, T, H, I, E, K):
    """Forward and backward in one graph, with inputs that change between the replays: each is the eager result."""
    import torch
    L = Layer(pm, T, H, I, E, K, "swiglu", 2.0)
    g, res = _capture(lambda: (L.forward(), *L.backward()))
    keep = L.x, L.ids, L.wt, L.dout
    for i in range(4):
        fresh = Layer(pm, T, H, I, E, K, "swiglu", 2.0, seed=20 + i)
        fresh.w1, fresh.w2 = L.w1, L.w2
        want = fresh.forward(), *fresh.backward()          # eager work between the replays
        for a, b in zip(keep, (fresh.x, fresh.ids, fresh.wt, fresh.dout)):
            a.copy_(b)
        for t in res:
            t.fill_(float(i))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, want):
            assert torch.equal(_bits(a), _bits(b)), f"replay {i}"


def test_two_graphs_of_one_workspace(pm):
    """Two captured sorts that share their workspace and their outputs, replayed in turn."""
    import torch
    rng = np.random.default_rng(2)
    E, K, H = 24, 3, 64
    ids = [dev(rng.integers(-1, E, (T, K)).astype(np.int32)) for T in (50, 4000)]
    x = [torch.randn(len(t), H, device="cuda").bfloat16() for t in ids]
    ws = torch.empty(max(pm.permute_workspace_bytes(len(t), K, E) for t in ids), dtype=torch.uint8, device="cuda")
    want = [pm.permute_tokens(a, t, E) for a, t in zip(x, ids)]
    pair = [_capture(lambda a=a, t=t: pm.permute_tokens(a, t, E, workspace=ws)) for a, t in zip(x, ids)]
    for i in (0, 1, 0, 0, 1, 1, 0):
        g, got = pair[i]
        ws.fill_(0xA5)
        for t in got:
            t.fill_(-3)
        torch.cuda.synchronize()
        g.replay()
        R = int(want[i].expert_offsets[-1])
        for a, b in zip(got, want[i]):
            n = R if a is got.rows or a is got.route_of_row else len(a)
            assert torch.equal(a[:n], b[:n])


def test_other_streams(pm):
    """On a stream of the caller's, which waits for the current one, and two streams at once: the same bits."""
    import torch
    make = lambda: Layer(pm, 900, 512, 256, 16, 4, "swiglu", seed=6)
    L = make()
    want = L.forward(), *L.backward()
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:                                           # one after the other, inputs made just before on the current stream
        M = make()
        M.x = (M.x.float() * 1.0).bfloat16()
        M.forward(stream=s)
        got = M.out, *M.backward(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(got, want):
            assert torch.equal(_bits(a), _bits(b))
    pair = [make() for _ in side]
    torch.cuda.synchronize()
    for _ in range(3):
        for M, s in zip(pair, side):
            with torch.cuda.stream(s):
                M.got = M.forward(), *M.backward()
    torch.cuda.synchronize()
    for M in pair:
        for a, b in zip(M.got, want):
            assert torch.equal(_bits(a), _bits(b))


def test_strided_tensors(pm):
    """Inputs that are views (every second column, a transposed matrix, a slice of rows) give what their copies give;
    an output that is one is refused."""
    import torch
    L = Layer(pm, 130, 256, 128, 8, 2, "swiglu", seed=8)
    L.forward()
    L.backward()
    wide = lambda t: torch.stack([t, t], -1).flatten(-2)[..., ::2]
    turned = lambda t: t.transpose(-1, -2).contiguous().transpose(-1, -2)
    off = L.order.expert_offsets
    for view in (wide, turned):
        assert all(not view(t).is_contiguous() for t in (L.x, *L.w1))
        for a, b in zip(pm.mx_quantize(view(L.x)), L.xq):
            assert torch.equal(a, b)
        assert torch.equal(pm.mx_dequantize(*map(view, L.xq)), pm.mx_dequantize(*L.xq))
        y = pm.mx_grouped_gemm(*map(view, L.xq), *map(view, L.w1), off, route_of_row=L.order.route_of_row, topk=2)
        assert torch.equal(y, L.y)
        assert torch.equal(pm.mx_grouped_gemm_backward(view(L.dz), *map(view, L.w2), off), L.dh)
        assert torch.equal(pm.mx_activation(view(L.y), L.act)[0], L.h[0])
        assert torch.equal(pm.mx_activation_backward(view(L.dh), *map(view, L.h[2:]), L.act), L.dy)
        assert torch.equal(pm.permute_tokens_backward(view(L.drows), L.order.row_of_route, 2), L.dx)
        assert torch.equal(pm.permute_tokens(view(L.x), turned(L.ids), 8).rows, L.x[L.order.route_of_row.long() // 2])
    with pytest.raises(ValueError):
        pm.mx_grouped_gemm(*L.xq, *L.w1, off, route_of_row=L.order.route_of_row, topk=2, out=wide(L.y))
    with pytest.raises(pm.PmoeError):                       # what is written lies in what is read
        pm.mx_activation(L.y, L.act, out=(L.y.view(torch.uint8).view(-1)[:260 * 64].view(260, 64), None, None, None))
    with pytest.raises(pm.PmoeError):                       # 8 bytes past a 16-byte boundary
        flat = torch.empty(130 * 256 + 8, dtype=torch.bfloat16, device="cuda")
        pm.mx_quantize(flat[4:4 + 130 * 256].view(130, 256))


# ----------------------------------------------------------------------------- the permutation's paths
@pytest.mark.parametrize("T,K,H", [(4096, 2, 64), (4097, 2, 64), (8, 4, 2 ** 18), (5, 8, 2 ** 19), (32, 1, 2 ** 19),
                                   (4200, 3, 6144), (1200, 4, 16384)])
def test_permute_paths(pm, T, K, H):
    """One launch and two, below and above what the caches hold: the same rows, twice the same bits, and what
    lies behind the last row untouched."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    E = 11
    ids = torch.randint(-1, E + 2, (T, K), generator=g, device="cuda", dtype=torch.int32)    # some twice in a token
    x = torch.randint(-2 ** 15, 2 ** 15, (T, H), generator=g, device="cuda", dtype=torch.int16)
    got = pm.permute_tokens(x, ids, E, out=(torch.full((T * K, H), 77, dtype=torch.int16, device="cuda"), None, None, None))
    row, route, off = mx.permute(ids.cpu().numpy(), E)
    R = int(off[-1])
    assert R < T * K and np.array_equal(got.row_of_route.cpu().numpy(), row)
    assert np.array_equal(got.route_of_row[:R].cpu().numpy(), route)
    assert torch.equal(got.rows[:R], x[torch.from_numpy(route // K).cuda().long()]) and (got.rows[R:] == 77).all()
    again = pm.permute_tokens(x, ids, E)
    assert torch.equal(again.rows[:R], got.rows[:R]) and torch.equal(again.row_of_route, got.row_of_route)


def test_permute_ids_out_of_32_bits(pm):
    """Ids that would be an expert's after a cut to 32 bits, and offsets at the ends of the type: no rows."""
    import torch
    x = torch.arange(4 * 8, device="cuda").view(4, 8).bfloat16()
    ids = torch.tensor([[2 ** 32 + 1], [-2 ** 63], [1], [2 ** 63 - 1]], device="cuda")
    got = pm.permute_tokens(x, ids, 4)
    assert got.row_of_route.tolist() == [-1, -1, 0, -1] and got.expert_offsets.tolist() == [0, 0, 1, 1, 1]
    for offset in (-2 ** 31, 2 ** 31 - 1):
        got = pm.permute_tokens(x, ids.clamp(-5, 5).int(), 4, expert_offset=offset)
        assert got.row_of_route.tolist() == [-1] * 4 and got.expert_offsets.tolist() == [0] * 5


def test_activation_of_any_row_count(pm):
    """A count below 0 or above R is cut to it."""
    import torch
    y = torch.randn(50, 64, device="cuda").bfloat16()
    want = pm.mx_activation(y, pm.ACT_RELU2, checkpoint=True)
    for n in (-1, -2 ** 31, 0, 1, 49, 50, 51, 2 ** 31 - 1):
        count, m = torch.tensor([n], dtype=torch.int32, device="cuda"), min(max(n, 0), 50)
        out = [torch.full_like(t, 9) for t in want]
        pm.mx_activation(y, pm.ACT_RELU2, checkpoint=True, row_count=count, out=out)
        for a, b in zip(out, want):
            assert torch.equal(a[:m], b[:m]) and (a[m:] == 9).all()
        dy = torch.full_like(y, 9.0)
        pm.mx_activation_backward(y, *want[2:], pm.ACT_RELU2, row_count=count, out=dy)
        full = pm.mx_activation_backward(y, *want[2:], pm.ACT_RELU2)
        assert torch.equal(dy[:m], full[:m]) and (dy[m:] == 9).all()
