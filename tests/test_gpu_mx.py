"""GPU parity of the token permutation and the microscaled operators with the float64 oracle.

Codes, scales and rows are compared bit for bit. Tolerances, u = 2^-24:
  product   products of codes and powers of two are exact, a sum of Kd of them has at most Kd roundings, each
            of at most 2 u (an adder that truncates) of the sum of the sizes; the result rounded to BF16: half a
            step, 2^-8. Where every partial sum is a multiple of one power of two below 2^24 of it, nothing is rounded.
  gradient  the same with N in Kd's place.
  dx of the permutation  K additions in FP32, one rounding.
  activation gradient    the exponential within 3 units (2^-23), 1 + e, a reciprocal within 1 unit, 1 - s and at most
            6 more FP32 operations: 16 units of 2^-23 of the sum of the sizes of the terms (1 - s also loses u of 1,
            which gate multiplies), then half a step of BF16.
"""
import numpy as np
import pytest

from helpers import bf16_bits, dev, dev_bf16
from oracle import mx
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


def _f(t):
    import torch
    return bf16_to_f32(bf16_bits(t)).astype(np.float64) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


def _bf(rng, *shape, std=1.0):
    return f32_to_bf16_rne((rng.standard_normal(shape) * std).astype(F32))


def _bf64(bits):
    return bf16_to_f32(bits).astype(np.float64)


# ----------------------------------------------------------------------------- permutation
@pytest.mark.parametrize("T,K,E,H,offset,ids64", [
    (1, 1, 1, 8, 0, False), (0, 2, 5, 16, 0, False), (61, 6, 64, 4096, 0, False), (33, 4, 16, 264, 16, True),
    (700, 8, 96, 1040, 96, False), (2100, 5, 7, 40, 0, True), (3, 32, 1024, 520, 0, False), (40, 2, 4, 64, 1000, False)])
def test_permute(pm, T, K, E, H, offset, ids64):
    import torch
    rng = np.random.default_rng(T + K + E)
    ids = np.stack([rng.permutation(4 * E if offset else E)[:K] for _ in range(T)]).astype(np.int64) if T else \
        np.zeros((0, K), np.int64)
    ids[rng.random(ids.shape) < 0.1] = -1
    x = _bf(rng, T, H)
    got = pm.permute_tokens(dev_bf16(x), dev(ids if ids64 else ids.astype(np.int32)), E, expert_offset=offset,
                            out=(torch.full((T * K, H), 7.0, dtype=torch.bfloat16, device="cuda"), None,
                                 torch.full((T * K,), -9, dtype=torch.int32, device="cuda"), None))
    row, route, off = mx.permute(ids, E, offset)
    R = off[-1]
    assert np.array_equal(got.row_of_route.cpu().numpy(), row)
    assert np.array_equal(got.expert_offsets.cpu().numpy(), off)
    assert np.array_equal(got.route_of_row.cpu().numpy(), np.append(route, np.full(T * K - R, -9)))
    want = np.full((T * K, H), f32_to_bf16_rne(np.array([7.0], F32))[0], np.uint16)
    want[:R] = x[route // K]
    assert np.array_equal(bf16_bits(got.rows), want)
    only = pm.permute_tokens(None, dev(ids), E, expert_offset=offset)
    assert only.rows is None and torch.equal(only.row_of_route, got.row_of_route)


@pytest.mark.parametrize("dtype", ["uint8", "float32", "float64"])
def test_permute_moves_rows_of_any_type(pm, dtype):
    import torch
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((50, 48)) * 50).astype(dtype)
    ids = rng.integers(0, 9, (50, 3)).astype(np.int32)
    got = pm.permute_tokens(dev(x), dev(ids), 9)
    route = mx.permute(ids, 9)[1]
    assert got.rows.dtype == getattr(torch, dtype) and np.array_equal(got.rows.cpu().numpy(), x[route // 3])


@pytest.mark.parametrize("T,K,H,R,f32", [(1, 1, 8, 1, False), (130, 6, 4096, 780, False), (77, 4, 520, 200, False),
                                         (64, 32, 72, 2048, True), (50, 3, 4, 0, True), (2049, 8, 1032, 4000, False)])
def test_permute_backward(pm, T, K, H, R, f32):
    rng = np.random.default_rng(T * K + H)
    row = rng.permutation(max(R, T * K))[:T * K].astype(np.int32)      # at most R rows are named
    row[row >= R] = np.where(rng.random((row >= R).sum()) < 0.5, -1, R + 5)
    d = rng.standard_normal((R, H)).astype(F32) if f32 else _bf(rng, R, H)
    got = _f(pm.permute_tokens_backward(dev(d) if f32 else dev_bf16(d), dev(row), K))
    v = d.astype(np.float64) if f32 else _bf64(d)
    want, size = mx.permute_backward(v, row, K), mx.permute_backward(np.abs(v), row, K)
    assert np.all(np.abs(got - want) <= K * U * size + (0 if f32 else 2.0 ** -8) * (np.abs(want) + K * U * size))


# ----------------------------------------------------------------------------- formats
def _rows(rng, rows, n, kind):
    x = rng.standard_normal((rows, n)) * np.exp(rng.standard_normal((rows, 1)) * 3)
    if kind == "ties":                                 # borders between codes, and exact powers as amax
        x = rng.choice([0, .25, .5, .75, 1, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.5, 17, 19, 248, 464], (rows, n)) * \
            rng.choice([-1, 1], (rows, n)) * 2.0 ** rng.integers(-20, 20, (rows, 1))
    elif kind == "ends":                               # subnormals, the largest values, zeros of both signs
        x = rng.standard_normal((rows, n)) * 2.0 ** rng.choice([-148, -140, -130, -126, -120, 100, 120, 125], (rows, 1))
        x[:, ::7] = -0.0
        x[::5] = 0.0
    elif kind == "bad":
        x[rng.random((rows, n)) < 0.01] = np.nan
        x[rng.random((rows, n)) < 0.01] = np.inf
        x[rng.random((rows, n)) < 0.01] = -np.inf
    return x.astype(F32)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind,rows,n", [("normal", 1, 32), ("normal", 37, 7168), ("ties", 300, 96), ("ends", 300, 64),
                                         ("bad", 200, 224)])
def test_quantize(pm, kind, rows, n, f32, fmt):
    import torch
    x = _rows(np.random.default_rng(rows + n), rows, n, kind)
    if not f32:
        x = f32_to_bf16_rne(x)
    codes, scales = pm.mx_quantize(dev(x) if f32 else dev_bf16(x), format=fmt)
    want = mx.quantize(x.astype(np.float64) if f32 else _bf64(x), fmt)
    assert np.array_equal(scales.cpu().numpy(), want[1])
    assert np.array_equal(codes.cpu().numpy(), want[0])
    v = mx.dequantize(*want, fmt)
    for dtype in (torch.float32, torch.bfloat16):
        got = pm.mx_dequantize(codes, scales, format=fmt, dtype=dtype)
        assert got.dtype == dtype
        ref = v.astype(F32)
        if dtype == torch.bfloat16:
            ref = bf16_to_f32(f32_to_bf16_rne(ref))
        got = _f(got).astype(F32)
        bad = np.isnan(ref)
        assert np.array_equal(np.isnan(got), bad)
        assert np.array_equal(got[~bad].view(np.uint32), ref[~bad].view(np.uint32))


def test_dequantize_every_code_and_scale(pm):
    import torch
    codes = np.tile(np.arange(256, dtype=np.uint8)[None], (256, 1))
    for fmt, n in (("e2m1", 512), ("e4m3", 256)):
        if fmt == "e4m3":
            codes = np.where((codes & 127) == 127, 0, codes)           # NaN codes, which no block holds
        scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], n // 32, 1)
        with np.errstate(over="ignore"):
            want = mx.dequantize(codes, scales, fmt).astype(F32)
        got = _f(pm.mx_dequantize(dev(codes), dev(scales), format=fmt, dtype=torch.float32)).astype(F32)
        assert np.array_equal(got, want, equal_nan=True)


def test_quantize_more_than_32_bits_of_elements(pm):
    import torch
    rows, n = (1 << 32) // 16384 + 3, 16384
    x = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    tail = _bf(np.random.default_rng(8), 4, n)
    x[-4:] = dev_bf16(tail)
    codes, scales = pm.mx_quantize(x)
    want = mx.quantize(_bf64(tail))
    assert np.array_equal(codes[-4:].cpu().numpy(), want[0]) and np.array_equal(scales[-4:].cpu().numpy(), want[1])
    back = pm.mx_dequantize(codes, scales, out=x)
    assert np.array_equal(_f(back[-4:]), mx.dequantize(*want)) and not back[:8].any()


# ----------------------------------------------------------------------------- products
def _offsets(rng, E, R, spare, kind):
    """Ascending offsets of E experts over R - spare rows; "one": all in one expert; "gaps": empty ones."""
    n = R - spare
    if kind == "one":
        return np.where(np.arange(E + 1) > E // 2, n, 0).astype(np.int32)
    cuts = np.sort(rng.integers(0, n + 1, E - 1))
    if kind == "gaps":
        cuts = np.sort(rng.choice(cuts, E - 1)) if E > 1 else cuts
    return np.concatenate([[0], cuts, [n]]).astype(np.int32)


def _exact_codes(rng, rows, Kd):
    """Codes and scales whose products are multiples of 2^-8 below 2^8 of it, so that sums are exact."""
    return (rng.integers(0, 256, (rows, Kd // 2)).astype(np.uint8),
            rng.integers(124, 128, (rows, Kd // 32)).astype(np.uint8))


PRODUCTS = [  # E, R, spare, N, Kd, offsets
    (1, 1, 0, 16, 32, "cuts"), (1, 33, 0, 48, 256, "cuts"), (3, 70, 9, 272, 288, "gaps"), (8, 200, 0, 144, 2080, "cuts"),
    (5, 700, 13, 400, 384, "one"), (64, 96, 0, 512, 1024, "gaps"), (130, 50, 5, 80, 160, "cuts"),
    (2, 513, 0, 1040, 512, "cuts"), (1024, 1200, 7, 32, 64, "cuts"), (4, 900, 40, 128, 1184, "gaps")]


# shapes that reach every tile of the products, forward and back, with rows of scales that are whole dwords and not
TILES = [(40, 5300, 11, 1040, 640, "cuts"), (40, 5300, 0, 1040, 256, "gaps"), (64, 8100, 9, 2064, 544, "cuts"),
         (64, 8100, 0, 2064, 96, "gaps"), (16, 800, 5, 4112, 256, "cuts"), (16, 800, 5, 4112, 224, "gaps"),
         (8, 1000, 3, 2064, 512, "cuts"), (8, 1000, 3, 2064, 480, "one"), (100, 300, 0, 528, 256, "cuts"),
         (100, 300, 0, 528, 288, "gaps"), (3, 5, 0, 208, 1152, "cuts"), (3, 5, 0, 208, 1120, "cuts"),
         (24, 2000, 7, 96, 4608, "cuts"), (24, 2000, 0, 112, 4640, "gaps"), (40, 400, 5, 80, 3584, "cuts"),
         (40, 400, 0, 64, 3616, "cuts"), (16, 1200, 20, 144, 2176, "cuts"), (16, 1200, 0, 144, 2080, "cuts"),
         (32, 4400, 10, 1552, 160, "cuts"), (8, 2048, 0, 4112, 1056, "gaps"), (32, 6144, 0, 1552, 96, "cuts")]


@pytest.mark.parametrize("E,R,spare,N,Kd,kind", PRODUCTS + TILES)
def test_product_exact(pm, E, R, spare, N, Kd, kind):
    """Sums that FP32 holds exactly: every output is checked to the bit, in both types."""
    import torch
    rng = np.random.default_rng(E + R + N + Kd)
    off = _offsets(rng, E, R, spare, kind)
    a, w = _exact_codes(rng, R, Kd), _exact_codes(rng, E * N, Kd)
    w = (w[0].reshape(E, N, -1), w[1].reshape(E, N, -1))
    want = mx.grouped_gemm(mx.dequantize(*a), mx.dequantize(*w), off)
    args = [dev(t) for t in (*a, *w, off)]
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((R, N), 5.0, dtype=dtype, device="cuda")
        got = _f(pm.mx_grouped_gemm(*args, out=out))
        ref = np.where(np.isnan(want), 5.0, want).astype(F32)
        if dtype == torch.bfloat16:
            ref = bf16_to_f32(f32_to_bf16_rne(ref))
        assert np.array_equal(got, ref.astype(np.float64))


@pytest.mark.parametrize("T,K,E,N,Kd,offset", [(16, 6, 64, 512, 1024, 0), (300, 4, 8, 176, 544, 8), (1, 1, 1, 16, 96, 0),
                                               (513, 2, 5, 272, 256, 0), (1500, 4, 40, 1040, 640, 0),
                                               (1700, 5, 64, 2064, 288, 64), (3000, 3, 64, 2064, 544, 0)])
def test_product_gathers_tokens(pm, T, K, E, N, Kd, offset):
    import torch
    rng = np.random.default_rng(T + E)
    ids = np.stack([rng.permutation(4 * E if offset else E)[:K] for _ in range(T)]).astype(np.int32)
    order = pm.permute_tokens(None, dev(ids), E, expert_offset=offset)
    a, w = _exact_codes(rng, T, Kd), _exact_codes(rng, E * N, Kd)
    w = (w[0].reshape(E, N, -1), w[1].reshape(E, N, -1))
    out = torch.full((T * K, N), -3.0, dtype=torch.float32, device="cuda")
    got = _f(pm.mx_grouped_gemm(*(dev(t) for t in (*a, *w)), order.expert_offsets, route_of_row=order.route_of_row, topk=K,
                                out=out))
    _, route, off = mx.permute(ids, E, offset)
    want = np.full((T * K, N), -3.0)
    want[:off[-1]] = mx.grouped_gemm(mx.dequantize(*a)[route // K], mx.dequantize(*w), off)
    assert np.array_equal(got, want)
    # routes that name no token read as zeros
    bad = dev(np.where(np.arange(T * K) % 3 == 0, T * K + 5, -1).astype(np.int32))
    got = pm.mx_grouped_gemm(*(dev(t) for t in (*a, *w)), order.expert_offsets, route_of_row=bad, topk=K, out=out)
    assert not got[:off[-1]].any()


@pytest.mark.parametrize("E,R,spare,N,Kd,kind", [(4, 300, 0, 256, 1024, "cuts"), (9, 64, 3, 96, 416, "gaps"),
                                                 (2, 1000, 0, 512, 2048, "cuts")])
def test_product_of_normal_values(pm, E, R, spare, N, Kd, kind):
    import torch
    rng = np.random.default_rng(E + R)
    off = _offsets(rng, E, R, spare, kind)
    a = mx.quantize(rng.standard_normal((R, Kd)) * np.exp(rng.standard_normal((R, 1)) * 3))
    w = mx.quantize(rng.standard_normal((E, N, Kd)) * Kd ** -0.5)
    va, vw = mx.dequantize(*a), mx.dequantize(*w)
    want, size = mx.grouped_gemm(va, vw, off), mx.grouped_gemm(np.abs(va), np.abs(vw), off)
    on = ~np.isnan(want[:, 0])
    for dtype, half in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        got = _f(pm.mx_grouped_gemm(*(dev(t) for t in (*a, *w, off)), dtype=dtype))
        slack = 2 * Kd * U * size[on]
        assert np.all(np.abs(got - np.where(np.isnan(want), 0, want))[on] <= slack + half * (np.abs(want[on]) + slack))


def test_product_keeps_nan_blocks_to_what_they_enter(pm):
    rng = np.random.default_rng(0)
    E, R, N, Kd = 2, 40, 48, 320
    off = np.array([0, 25, 40], np.int32)
    a, w = _exact_codes(rng, R, Kd), _exact_codes(rng, E * N, Kd)
    w = (w[0].reshape(E, N, -1), w[1].reshape(E, N, -1))
    a[1][7, 9], w[1][1, 30, 0] = 255, 255
    want = mx.grouped_gemm(mx.dequantize(*a), mx.dequantize(*w), off)
    import torch
    got = _f(pm.mx_grouped_gemm(*(dev(t) for t in (*a, *w, off)), dtype=torch.float32))
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isnan(want[7]).all() and np.isnan(want[25:, 30]).all() and np.isnan(want).sum() == N + 15


def test_product_rows_do_not_depend_on_each_other(pm):
    import torch
    rng = np.random.default_rng(4)
    E, N, Kd = 6, 272, 1184
    w = [dev(t) for t in mx.quantize(rng.standard_normal((E, N, Kd)))]
    a = [dev(t) for t in mx.quantize(rng.standard_normal((1500, Kd)))]
    off = dev(np.array([0, 300, 300, 800, 801, 1200, 1500], np.int32))
    every = pm.mx_grouped_gemm(*a, *w, off, dtype=torch.float32)
    dy = dev_bf16(_bf(rng, 1500, N))
    every_dx = pm.mx_grouped_gemm_backward(dy, *w, off)
    for r, e in ((0, 0), (299, 0), (555, 2), (800, 3), (1499, 5)):
        o = dev((np.arange(E + 1) > e).astype(np.int32))
        one = pm.mx_grouped_gemm(a[0][r:r + 1], a[1][r:r + 1], *w, o, dtype=torch.float32)
        assert torch.equal(one[0], every[r])
        assert torch.equal(pm.mx_grouped_gemm_backward(dy[r:r + 1], *w, o)[0], every_dx[r])


def test_product_past_32_bits(pm):
    """An output and an operand of more than 2^32 bytes; only the last rows hold anything."""
    import torch
    R, N, Kd = (1 << 32) // 16384 + 130, 16384, 512
    rng = np.random.default_rng(6)
    a, w = _exact_codes(rng, 5, Kd), _exact_codes(rng, N, Kd)
    A = [torch.zeros(R, t.shape[1], dtype=torch.uint8, device="cuda") for t in a]
    for t, v in zip(A, a):
        t[-5:] = dev(v)
    off = dev(np.array([0, R], np.int32))
    W = [dev(t)[None] for t in w]
    got = pm.mx_grouped_gemm(*A, *W, off)
    want = mx.dequantize(*a) @ mx.dequantize(*w).T
    assert np.array_equal(_f(got[-5:]), bf16_to_f32(f32_to_bf16_rne(want.astype(F32))).astype(np.float64))
    assert not got[:-5].any()
    dx = pm.mx_grouped_gemm_backward(got, *W, off)
    v = _f(got[-5:])
    ref, size = v @ mx.dequantize(*w), np.abs(v) @ np.abs(mx.dequantize(*w))
    slack = 2 * N * U * size
    assert np.all(np.abs(_f(dx[-5:]) - ref) <= slack + 2.0 ** -8 * (np.abs(ref) + slack)) and not dx[:-5].any()


def test_product_with_offsets_that_are_none(pm):
    """Offsets outside [0, R] or descending: nothing outside the output is touched, and rows of
    proper ranges are right."""
    import torch
    rng = np.random.default_rng(2)
    E, R, N, Kd = 3, 40, 32, 64
    a, w = _exact_codes(rng, R, Kd), _exact_codes(rng, E * N, Kd)
    w = (w[0].reshape(E, N, -1), w[1].reshape(E, N, -1))
    want = mx.dequantize(*a)[:10] @ mx.dequantize(*w)[0].T
    for off in ([-5, 10, 7, 7], [0, 10, 10, 1 << 30]):
        buf = torch.full((R + 40, N), 9.0, dtype=torch.float32, device="cuda")
        got = pm.mx_grouped_gemm(*(dev(t) for t in (*a, *w, np.array(off, np.int32))), out=buf[20:20 + R])
        assert np.array_equal(_f(got[:7]), want[:7])
        assert (buf[:20] == 9).all() and (buf[20 + R:] == 9).all()


@pytest.mark.parametrize("E,R,spare,N,Kd,kind", PRODUCTS + TILES)
def test_product_gradient_exact(pm, E, R, spare, N, Kd, kind):
    """dy of small whole numbers: sums that FP32 holds exactly, rounded to BF16 once."""
    import torch
    rng = np.random.default_rng(E * R + N)
    off = _offsets(rng, E, R, spare, kind)
    w = _exact_codes(rng, E * N, Kd)
    w = (w[0].reshape(E, N, -1), w[1].reshape(E, N, -1))
    dy = rng.integers(-16, 17, (R, N)).astype(F32)
    want = mx.grouped_gemm_backward(dy, mx.dequantize(*w), off)
    out = torch.full((R, Kd), 5.0, dtype=torch.bfloat16, device="cuda")
    got = _f(pm.mx_grouped_gemm_backward(dev_bf16(f32_to_bf16_rne(dy)), *(dev(t) for t in (*w, off)), out=out))
    assert np.array_equal(got, bf16_to_f32(f32_to_bf16_rne(np.where(np.isnan(want), 5.0, want).astype(F32))).astype(np.float64))


@pytest.mark.parametrize("E,R,N,Kd", [(3, 400, 1040, 640), (7, 60, 528, 224)])
def test_product_gradient_of_normal_values(pm, E, R, N, Kd):
    rng = np.random.default_rng(E + R)
    off = _offsets(rng, E, R, 0, "cuts")
    w = mx.quantize(rng.standard_normal((E, N, Kd)))
    dy = _bf(rng, R, N, std=1e-3)
    vw = mx.dequantize(*w)
    want, size = mx.grouped_gemm_backward(_bf64(dy), vw, off), mx.grouped_gemm_backward(np.abs(_bf64(dy)), np.abs(vw), off)
    got = _f(pm.mx_grouped_gemm_backward(dev_bf16(dy), *(dev(t) for t in (*w, off))))
    slack = 2 * N * U * size
    assert np.all(np.abs(got - want) <= slack + 2.0 ** -8 * (np.abs(want) + slack))


def test_product_gradient_is_the_transpose(pm):
    """<dy, W a> = <W^T dy, a>, exactly, where both sides are whole sums."""
    import torch
    rng = np.random.default_rng(9)
    E, R, N, Kd = 3, 90, 64, 96
    off = dev(np.array([0, 30, 31, 90], np.int32))
    a, w = [dev(t) for t in _exact_codes(rng, R, Kd)], [dev(t) for t in _exact_codes(rng, E * N, Kd)]
    w = [w[0].view(E, N, -1), w[1].view(E, N, -1)]
    dy = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    dy[torch.arange(R), torch.arange(R) % N] = 1.0     # one row of W each: dx is exact in BF16
    y = pm.mx_grouped_gemm(*a, *w, off, dtype=torch.float32)
    dx = pm.mx_grouped_gemm_backward(dy, *w, off)
    left = (y.double() * dy.double()).sum(1)
    right = (dx.double() * pm.mx_dequantize(*a).double()).sum(1)
    assert torch.equal(left, right)


# ----------------------------------------------------------------------------- activation
@pytest.mark.parametrize("R,I", [(1, 32), (96, 2048), (333, 160)])
@pytest.mark.parametrize("act,limit", [("relu2", 0.0), ("swiglu", 0.0), ("swiglu", 1.25)])
def test_activation_and_gradient(pm, R, I, act, limit):
    rng = np.random.default_rng(R + I)
    a = pm.ACT_SWIGLU if act == "swiglu" else pm.ACT_RELU2
    y = _bf(rng, R, 2 * I if act == "swiglu" else I, std=2.0)
    hq, h_sf, y8, y8_sf = pm.mx_activation(dev_bf16(y), a, swiglu_limit=limit, checkpoint=True)
    want = mx.quantize(mx.activation(_bf64(y), act, limit))
    assert np.array_equal(h_sf.cpu().numpy(), want[1]) and np.array_equal(hq.cpu().numpy(), want[0])
    keep = mx.quantize(_bf64(y), "e4m3")
    assert np.array_equal(y8.cpu().numpy(), keep[0]) and np.array_equal(y8_sf.cpu().numpy(), keep[1])
    plain = pm.mx_activation(dev_bf16(y), a, swiglu_limit=limit)
    assert plain[2] is None and plain[3] is None and (plain[0] == hq).all() and (plain[1] == h_sf).all()
    dh = _bf(rng, R, I)
    got = _f(pm.mx_activation_backward(dev_bf16(dh), y8, y8_sf, a, swiglu_limit=limit))
    v = mx.dequantize(*keep, "e4m3")
    ref = mx.activation_backward(_bf64(dh), v, act, limit)
    if act == "relu2":
        size = np.abs(ref)
    else:
        g, u = np.split(np.abs(v), 2, 1)
        g, u = (np.minimum(g, limit), np.minimum(u, limit)) if limit else (g, u)
        d = np.abs(_bf64(dh))
        size = np.concatenate([d * u * (1 + g), d * g], 1)
    slack = 32 * U * size
    assert np.all(np.abs(got - ref) <= slack + 2.0 ** -8 * (np.abs(ref) + slack))


def test_activation_codes_are_those_of_the_exact_value(pm):
    """Many values, so that some lie within FP32's error of a border between codes: all are those of h in 64 bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(11)
    y = (torch.randn(4096, 2 * 1024, generator=g, device="cuda") * 3).bfloat16()
    hq, h_sf, _, _ = pm.mx_activation(y, pm.ACT_SWIGLU)
    for i in range(0, 4096, 512):
        want = mx.quantize(mx.activation(_f(y[i:i + 512]), "swiglu"))
        assert np.array_equal(h_sf[i:i + 512].cpu().numpy(), want[1])
        assert np.array_equal(hq[i:i + 512].cpu().numpy(), want[0])


def test_activation_at_the_ends_of_the_range(pm):
    """Gates whose exponential overflows or vanishes, and products below and near FP32's smallest and largest."""
    rng = np.random.default_rng(12)
    I = 64
    g = np.concatenate([rng.uniform(-95, -75, (40, I)), rng.uniform(-400, -80, (40, I)), rng.uniform(80, 400, (40, I)),
                        rng.choice([0.0, -0.0, 1e-38, -1e-38, 1e-30, 3.0], (40, I)), rng.uniform(-3, 3, (40, I)),
                        rng.uniform(1e37, 3e38, (40, I))])
    u = np.concatenate([rng.standard_normal((160, I)), rng.standard_normal((40, I)) * 2.0 ** rng.integers(-140, -90, (40, 1)),
                        rng.uniform(-1.0, 1.0, (40, I))])
    y = f32_to_bf16_rne(np.concatenate([g, u], 1).astype(F32))
    h = mx.activation(_bf64(y), "swiglu")
    assert np.abs(h).max() < 3.4e38
    hq, h_sf, _, _ = pm.mx_activation(dev_bf16(y), pm.ACT_SWIGLU)
    want = mx.quantize(h)
    assert np.array_equal(h_sf.cpu().numpy(), want[1]) and np.array_equal(hq.cpu().numpy(), want[0])
    y8 = mx.quantize(_bf64(y), "e4m3")
    dh = _bf(rng, 240, I)
    got = _f(pm.mx_activation_backward(dev_bf16(dh), dev(y8[0]), dev(y8[1]), pm.ACT_SWIGLU))
    v = mx.dequantize(*y8, "e4m3")
    ref = mx.activation_backward(_bf64(dh), v, "swiglu")
    gv, uv = np.split(np.abs(v), 2, 1)
    d = np.abs(_bf64(dh))
    # below 2^-126 of a sigmoid (gates under -87) the result is 0, BF16 keeps no more than 2^-133 of a step
    slack = 32 * U * np.concatenate([d * uv * (1 + gv), d * gv], 1) + 2.0 ** -125 * np.concatenate([d * uv, d], 1) * \
        np.concatenate([1 + gv, gv], 1) + 2.0 ** -134
    # d up = d h * gate passes BF16's largest, (2 - 2^-7) 2^127, for some of the gates near 3e38: infinite there
    top = (2.0 - 2.0 ** -7) * 2.0 ** 127
    over = np.abs(ref) >= 2.0 ** 128
    assert over.any() and np.array_equal(got[over], np.copysign(np.inf, ref[over]))
    fits = np.abs(ref) <= top
    assert np.all((np.abs(got - np.where(fits, ref, got)) <= slack + 2.0 ** -8 * (np.abs(ref) + slack))[fits])


@pytest.mark.parametrize("act", ["relu2", "swiglu"])
def test_activation_of_infinities_and_nan(pm, act):
    rng = np.random.default_rng(13)
    a = pm.ACT_SWIGLU if act == "swiglu" else pm.ACT_RELU2
    y = (rng.standard_normal((50, 256))).astype(F32)
    y[rng.random(y.shape) < 0.005] = np.inf
    y[rng.random(y.shape) < 0.005] = -np.inf
    y[rng.random(y.shape) < 0.005] = np.nan
    y = f32_to_bf16_rne(y)
    hq, h_sf, y8, y8_sf = pm.mx_activation(dev_bf16(y), a, checkpoint=True)
    h = mx.activation(_bf64(y), act)
    want = mx.quantize(h)
    assert (want[1] == 255).any() and np.array_equal(h_sf.cpu().numpy(), want[1]) and np.array_equal(hq.cpu().numpy(), want[0])
    keep = mx.quantize(_bf64(y), "e4m3")
    assert np.array_equal(y8.cpu().numpy(), keep[0]) and np.array_equal(y8_sf.cpu().numpy(), keep[1])
    got = _f(pm.mx_activation_backward(dev_bf16(_bf(rng, 50, h.shape[1])), y8, y8_sf, a))
    nan = np.isnan(mx.dequantize(*keep, "e4m3"))
    if act == "swiglu":                                # either of a pair that reads as NaN makes both gradients NaN
        both = nan[:, :128] | nan[:, 128:]
        # d up does not read up, so only the gate's block counts for it
        nan = np.concatenate([both, nan[:, :128]], 1)
    assert np.array_equal(np.isnan(got), nan)


def test_activation_rows_behind_the_count(pm):
    import torch
    rng = np.random.default_rng(14)
    R, I = 70, 96
    y, dh = dev_bf16(_bf(rng, R, 2 * I)), dev_bf16(_bf(rng, R, I))
    u8 = dict(dtype=torch.uint8, device="cuda")
    whole = pm.mx_activation(y, pm.ACT_SWIGLU, checkpoint=True)
    dy = pm.mx_activation_backward(dh, whole[2], whole[3], pm.ACT_SWIGLU)
    for n in (0, 1, 41, 70, 90, -3):
        count = torch.tensor([n], dtype=torch.int32, device="cuda")
        out = tuple(torch.full(t.shape, 77, **u8) for t in whole)
        pm.mx_activation(y, pm.ACT_SWIGLU, checkpoint=True, row_count=count, out=out)
        k = min(max(n, 0), R)
        for t, w in zip(out, whole):
            assert torch.equal(t[:k], w[:k]) and (t[k:] == 77).all()
        d = torch.full((R, 2 * I), 3.0, dtype=torch.bfloat16, device="cuda")
        pm.mx_activation_backward(dh, whole[2], whole[3], pm.ACT_SWIGLU, row_count=count, out=d)
        assert torch.equal(d[:k], dy[:k]) and (d[k:] == 3).all()
