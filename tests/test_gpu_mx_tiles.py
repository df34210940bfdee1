"""The MXFP4 products' tiles: the persistent kernel with several tiles a workgroup and several pairs of
stages, bit for bit, and each tile's rows against the same rows in calls of one row, which another tile computes."""
import numpy as np
import pytest

from helpers import bf16_bits, dev, dev_bf16
from mx_tiles import backward_tile, forward_tile, persistent_tiles
from oracle import mx
from oracle.formats import bf16_to_f32, f32_to_bf16_rne

pytestmark = pytest.mark.gpu
F32 = np.float32


@pytest.fixture(scope="module")
def pm():
    import torch
    import precision_moe_amd as pm
    assert torch.cuda.is_available()
    return pm


def _f(t):
    import torch
    return bf16_to_f32(bf16_bits(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def _codes(rng, *shape):
    """Codes and scales whose products are multiples of 2^-4 below 36: sums of up to 2^14 of them are exact in FP32."""
    *lead, Kd = shape
    return (rng.integers(0, 256, (*lead, Kd // 2)).astype(np.uint8),
            rng.integers(126, 128, (*lead, Kd // 32)).astype(np.uint8))


def _offsets(rng, E, R, even):
    """Offsets of E experts over R rows: nearly alike, or some large, some empty."""
    if even:
        cuts = np.linspace(0, R, E + 1)[1:-1] + rng.integers(-9, 10, E - 1)
        return np.concatenate([[0], np.sort(np.clip(cuts, 0, R)), [R]]).astype(np.int32)
    share = np.exp(2 * rng.standard_normal(E)) * (rng.random(E) > 0.2)
    return np.round(np.concatenate([[0], np.cumsum(share) / share.sum()]) * R).astype(np.int32)


@pytest.mark.parametrize("E,R,N,Kd,even", [
    (64, 24000, 2064, 1280, True), (64, 24000, 2064, 1152, False), (40, 26000, 2064, 1792, False), (64, 24000, 1808, 2048, True),
    (64, 24000, 2064, 1312, True), (64, 24000, 2064, 1312, False), (48, 24000, 2064, 1824, False)])
def test_persistent_workgroups_take_several_tiles(pm, E, R, N, Kd, even):
    """Three tiles a workgroup at least, three or four pairs of stages, no row of zeros."""
    import torch
    rng = np.random.default_rng(E + N + Kd)
    off = _offsets(rng, E, R, even)
    assert forward_tile(R, E, N, Kd)[0] in (192, 256) and persistent_tiles(off, N, Kd) > 3 * 256 and Kd > 1024
    a, w = _codes(rng, R, Kd), _codes(rng, E, N, Kd)
    want = np.empty((R, N), F32)
    va = mx.dequantize(*a).astype(F32)
    for e in range(E):                                 # FP32 sums here are exact in any order
        rows = slice(off[e], off[e + 1])
        want[rows] = va[rows] @ mx.dequantize(w[0][e], w[1][e]).astype(F32).T
    args = [dev(t) for t in (*a, *w, off)]
    assert np.array_equal(_f(pm.mx_grouped_gemm(*args, dtype=torch.float32)), want)
    assert np.array_equal(_f(pm.mx_grouped_gemm(*args)), bf16_to_f32(f32_to_bf16_rne(want)))


@pytest.mark.parametrize("T,K,E,N,Kd", [(8000, 3, 64, 2064, 1280), (6500, 4, 40, 2064, 1824)])
def test_persistent_workgroups_gather(pm, T, K, E, N, Kd):
    """The same with tokens gathered by route, a part of the routes elsewhere, experts of unlike size."""
    import torch
    rng = np.random.default_rng(T + Kd)
    ids = np.minimum(rng.exponential(E / 2, (T, K)), E + 2).astype(np.int32)
    row, route, off = mx.permute(ids, E)
    R = int(off[-1])
    assert forward_tile(T * K, E, N, Kd)[0] in (192, 256) and persistent_tiles(off, N, Kd) > 3 * 256 and R < T * K
    a, w = _codes(rng, T, Kd), _codes(rng, E, N, Kd)
    want = np.full((T * K, N), -5.0, F32)
    va = mx.dequantize(*a).astype(F32)[route // K]
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        want[rows] = va[rows] @ mx.dequantize(w[0][e], w[1][e]).astype(F32).T
    order = pm.permute_tokens(None, dev(ids), E)
    out = torch.full((T * K, N), -5.0, dtype=torch.float32, device="cuda")
    pm.mx_grouped_gemm(*(dev(t) for t in (*a, *w)), order.expert_offsets, route_of_row=order.route_of_row, topk=K, out=out)
    assert np.array_equal(_f(out), want)


def _unlike(g, *shape):
    """Normal values whose blocks of 32 differ by powers of two up to 2^20, so that sums of their products round."""
    import torch
    *lead, Kd = shape
    size = torch.randint(-10, 11, (*lead, Kd // 32, 1), generator=g, device="cuda").float()
    return (torch.randn(*lead, Kd // 32, 32, generator=g, device="cuda") * torch.exp2(size)).reshape(shape)


def _some_rows(rng, off):
    """Rows to look at, with their experts: ends of experts and some between."""
    e = np.searchsorted(off[1:], np.arange(off[-1]), side="right")
    r = np.unique(np.concatenate([[0, off[-1] - 1], off[1:-1][:4], rng.integers(0, off[-1], 8)]))
    return [(int(i), int(e[i])) for i in r if i < off[-1]]


@pytest.mark.parametrize("E,R,N,Kd,tile", [
    (40, 9000, 1040, 1152, (256, 256)), (40, 20000, 2064, 1184, (192, 256)), (30, 3600, 1040, 1152, (128, 256)),
    (30, 3600, 1040, 1184, (128, 256)), (16, 1600, 1040, 1152, (128, 128)), (16, 1600, 1040, 1184, (128, 128)),
    (64, 300, 528, 1152, (32, 128)), (64, 300, 528, 1184, (32, 128))])
def test_rows_are_the_same_in_every_tile(pm, E, R, N, Kd, tile):
    """Sums that round (asserted): a row of a call that takes `tile` has the bits of that row alone (tiles of 32 x 64)."""
    import torch
    rng = np.random.default_rng(E + R + Kd)
    off = _offsets(rng, E, R, True)
    assert forward_tile(R, E, N, Kd) == tile and forward_tile(1, E, N, Kd) == (32, 64)
    g = torch.Generator(device="cuda").manual_seed(R + Kd)
    w = pm.mx_quantize(_unlike(g, E, N, Kd))
    a = pm.mx_quantize(_unlike(g, R, Kd))
    every = pm.mx_grouped_gemm(*a, *w, dev(off), dtype=torch.float32)
    for r, e in _some_rows(rng, off):
        one = pm.mx_grouped_gemm(a[0][r:r + 1], a[1][r:r + 1], *w, dev((np.arange(E + 1) > e).astype(np.int32)),
                                 dtype=torch.float32)
        assert torch.equal(one[0], every[r])
    # the sums do round: they differ from FP64's somewhere in the first row
    e = int(np.searchsorted(off[1:], 0, side="right"))
    exact = pm.mx_dequantize(*(t[:1] for t in a)).double() @ pm.mx_dequantize(*(t[e] for t in w)).double().T
    assert (exact[0] != every[0].double()).any()


@pytest.mark.parametrize("E,R,N,Kd,tile", [
    (70, 8400, 528, 1152, (128, 512)), (70, 8400, 528, 1184, (128, 512)), (26, 1950, 528, 1152, (64, 256)),
    (26, 1950, 528, 1184, (64, 256)), (100, 300, 528, 1152, (32, 512)), (100, 300, 528, 1184, (32, 512))])
def test_gradient_rows_are_the_same_in_every_tile(pm, E, R, N, Kd, tile):
    """As above for the gradient: a row alone takes tiles of 32 x 128."""
    import torch
    rng = np.random.default_rng(E + R + Kd)
    off = _offsets(rng, E, R, True)
    assert backward_tile(R, E, N, Kd) == tile and backward_tile(1, E, N, Kd) == (32, 128)
    g = torch.Generator(device="cuda").manual_seed(R + Kd)
    w = pm.mx_quantize(_unlike(g, E, N, Kd))
    dy = torch.randn(R, N, generator=g, device="cuda").bfloat16()
    every = pm.mx_grouped_gemm_backward(dy, *w, dev(off))
    for r, e in _some_rows(rng, off):
        one = pm.mx_grouped_gemm_backward(dy[r:r + 1], *w, dev((np.arange(E + 1) > e).astype(np.int32)))
        assert torch.equal(one[0], every[r])
