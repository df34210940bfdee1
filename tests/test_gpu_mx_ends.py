"""The microscaled operators at the ends of their ranges, against the float64 oracle (U = 2^-24, half a
step of BF16 = 2^-8 of a normal value, 2^-134 of a subnormal one)."""
import numpy as np
import pytest

from helpers import bf16_bits, dev, dev_bf16
from mx_tiles import backward_tile, forward_tile
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


def _bf(x):
    return f32_to_bf16_rne(np.asarray(x).astype(F32))


def _f(t):
    import torch
    return bf16_to_f32(bf16_bits(t)).astype(np.float64) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


# ----------------------------------------------------------------------------- order of the routes
@pytest.mark.parametrize("blocks", [33, 36, 40, 41, 48, 49, 56, 57, 64, 65, 72, 80, 81, 96, 104, 113, 130])
@pytest.mark.parametrize("E", [3, 512, 513, 1024])
def test_order_of_any_number_of_blocks(pm, blocks, E):
    """Above 8192 routes the sort counts blocks of 256 and sums the counts in rounds of 8, 16 or 32: ends inside and at each."""
    rng = np.random.default_rng(blocks + E)
    ids = rng.integers(-1, E + 1, (blocks * 256 - int(rng.integers(0, 255)), 1)).astype(np.int32)
    got = pm.permute_tokens(None, dev(ids), E)
    key = np.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    route = np.argsort(key, kind="stable")[:(key < E).sum()]
    row = np.full(key.size, -1)
    row[route] = np.arange(len(route))
    assert np.array_equal(got.row_of_route.cpu().numpy(), row)
    assert np.array_equal(got.route_of_row.cpu().numpy()[:len(route)], route)
    assert np.array_equal(got.expert_offsets.cpu().numpy(), np.searchsorted(np.sort(key), np.arange(E + 1)))


# ----------------------------------------------------------------------------- activation
@pytest.mark.parametrize("limit,d_bits,up_bits", [(0.0, (-10, 30), (0, 90)), (7.0, (60, 110), (-2, 2))])
def test_activation_gradient_of_gates_far_below_zero(pm, limit, d_bits, up_bits):
    """Gates whose sigmoid is near or below FP32's smallest normal number (2^-126 at -87.3), with d h and up for which
    the gradients are ordinary numbers. There 1 + gate (1 - sigmoid) has no cancellation, so that the FP32 chain (the
    exponential within 3 units of 2^-23, 7 more roundings) is within 16 units of 2^-23 of the result; a power of
    two that is applied to a subnormal loses up to 2^-150, times the gate's 1000 at most, 2^-140."""
    rng = np.random.default_rng(21)
    R, I = 96, 64
    gate = -rng.choice([80.0, 88, 96, 104, 112, 128, 144, 160, 176, 208, 448, 896], (R, I))    # 4 bits each: E4M3 holds them
    gate[-8:] *= 1e30
    up = rng.standard_normal((R, I)) * 2.0 ** rng.integers(*up_bits, (R, 1))
    codes, scales = mx.quantize(np.concatenate([gate, up], 1), "e4m3")
    v = mx.dequantize(codes, scales, "e4m3")
    assert np.array_equal(v[:-8, :I], gate[:-8])
    dh = _bf(rng.standard_normal((R, I)) * 2.0 ** rng.integers(*d_bits, (R, 1)))
    ref = mx.activation_backward(bf16_to_f32(dh), v, "swiglu", limit)
    far = v[:, :I] < -87
    assert (np.abs(ref[:, :I][far]) > 2.0 ** -120).sum() > 300
    got = _f(pm.mx_activation_backward(dev_bf16(dh), dev(codes), dev(scales), pm.ACT_SWIGLU, swiglu_limit=limit))
    slack = 32 * U * np.abs(ref) + 2.0 ** -140
    assert np.all(np.abs(got - ref) <= slack + 2.0 ** -134 + 2.0 ** -8 * (np.abs(ref) + slack))


def test_relu2_gradient_of_the_largest_values(pm):
    """2 y is past FP32's largest number where y is at least 2^127, 2 y d h is not. The product of a value of 4 bits and
    one of 8 is exact, so the result is rounded to BF16 once."""
    rng = np.random.default_rng(22)
    y = rng.choice([1.0, -1.0, 1.125, 1.5, 1.75], (40, 64)) * 2.0 ** rng.choice([119, 126, 127, 127], (40, 64))
    codes, scales = mx.quantize(y, "e4m3")
    v = mx.dequantize(codes, scales, "e4m3")
    assert np.array_equal(v, y)
    dh = _bf(rng.standard_normal((40, 64)) * 2.0 ** rng.integers(-40, -4, (40, 1)))
    got = _f(pm.mx_activation_backward(dev_bf16(dh), dev(codes), dev(scales), pm.ACT_RELU2))
    assert np.array_equal(got, bf16_to_f32(_bf(mx.activation_backward(bf16_to_f32(dh), v, "relu2"))))


def test_activation_gradient_does_not_cut_off_a_nan(pm):
    """With a clamp, too, a block of up that reads as NaN makes d gate NaN and leaves d up what the gate says, and
    a NaN gate makes both NaN; other blocks are those of the row without it."""
    rng = np.random.default_rng(23)
    y = rng.standard_normal((6, 256)) * 3
    dh = dev_bf16(_bf(rng.standard_normal((6, 128))))
    codes, scales = mx.quantize(y, "e4m3")
    call = lambda s, limit: _f(pm.mx_activation_backward(dh, dev(codes), dev(s), pm.ACT_SWIGLU, swiglu_limit=limit))
    bad = scales.copy()
    bad[1, 5] = 255                                    # up 32 .. 63 of row 1
    bad[4, 2] = 255                                    # gate 64 .. 95 of row 4
    for limit in (0.0, 20.0):                          # 20: the values are below it
        got, want = call(bad, limit), call(scales, limit)
        want[1, 32:64] = want[4, 64:96] = want[4, 192:224] = np.nan
        assert np.array_equal(got, want, equal_nan=True)


# ----------------------------------------------------------------------------- products
# Experts of 255 or 256 rows, all alike, for which each tile is chosen: with N = 256 and Kd up to 512 (forward), with
# Kd up to 256 (backward). Every expert's output has to be the first one's.
FORWARD = [(E, Kd, tile) for Kd, wide in ((256, 160), (288, 256))
           for E, tile in ((1, (32, 64)), (16, (32, 128)), (32, (128, 128)), (64, (128, 256)),
                           (wide, (192 if Kd % 128 else 256, 256)))]
BACKWARD = [(E, Kd, tile) for Kd in (128, 160)
            for E, tile in ((1, (32, 128)), (32, (32, 512)), (64, (64, 256)), (100, (128, 512)))]


def _every(t, E):
    """E copies of the rows t, on the device."""
    return dev(t).repeat(E, *[1] * (t.ndim - 1))


def _first(t, E):
    """The rows of the first expert, after a check that the others' are the same bits."""
    import torch
    bits = t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).view(E, -1)
    assert (bits == bits[:1]).all()
    return _f(t.view(E, -1, t.shape[1])[0])


@pytest.mark.parametrize("E,Kd,tile", FORWARD)
def test_product_of_every_pair_of_scales(pm, E, Kd, tile):
    """One element of either operand, with every pair of the 255 scales and every magnitude: exact; products
    below 2^-126, which FP32 holds with fewer bits, within its smallest number, those past its largest infinite."""
    import torch
    rng = np.random.default_rng(E + Kd)
    N, R = 256, 255
    assert forward_tile(R * E, E, N, Kd) == tile
    off = dev((np.arange(E + 1) * R).astype(np.int32))
    for k in (0, Kd - 1):
        def side(rows):
            codes, scales = np.zeros((rows, Kd // 2), np.uint8), rng.integers(0, 255, (rows, Kd // 32)).astype(np.uint8)
            codes[:, k // 2] = rng.integers(0, 16, rows) << (4 if k % 2 else 0)
            scales[:, k // 32] = np.arange(rows) % 255
            return codes, scales
        a, w = side(R), side(N)
        got = _first(pm.mx_grouped_gemm(*(_every(t, E) for t in a), *(_every(t[None], E) for t in w), off,
                                        dtype=torch.float32), E)
        exact = np.outer(mx.dequantize(*a)[:, k], mx.dequantize(*w)[:, k])
        with np.errstate(over="ignore"):
            want = exact.astype(F32).astype(np.float64)
        small = np.abs(exact) < 2.0 ** -126
        assert np.array_equal(got[~small], want[~small]) and np.isinf(want).any()
        assert np.all(np.abs(got - exact)[small] <= 2.0 ** -149)


@pytest.mark.parametrize("E,Kd,tile", BACKWARD)
def test_product_gradient_of_every_code_and_scale(pm, E, Kd, tile):
    """dy with one power of two a row, so that dx is that times a row of the matrix: every code with every scale that
    the quantizer gives (0 .. 252: the largest magnitude, 6 * 2^125, is below BF16's), subnormal values and subnormal
    dy among them, rounded to BF16 once."""
    N = R = 256
    assert backward_tile(R * E, E, N, Kd) == tile
    off = dev((np.arange(E + 1) * R).astype(np.int32))
    codes = np.tile(np.arange(0, 16, 2) | np.arange(1, 16, 2) << 4, (N, Kd // 16)).astype(np.uint8)
    scales = np.tile((np.arange(N) % 253)[:, None], (1, Kd // 32)).astype(np.uint8)
    w = [_every(t[None], E) for t in (codes, scales)]
    v = mx.dequantize(codes, scales)
    for p in (-130, -100, -40, 0, 40, 127):
        dy = np.zeros((R, N))
        dy[np.arange(R), np.arange(N)] = 2.0 ** p
        got = _first(pm.mx_grouped_gemm_backward(dev_bf16(np.tile(_bf(dy), (E, 1))), *w, off), E)
        with np.errstate(over="ignore"):
            want = bf16_to_f32(_bf(v * 2.0 ** p)).astype(np.float64)
        assert np.array_equal(got, want)
        assert np.isinf(want).any() == (p > 0) and ((np.abs(want) < 2.0 ** -126) & (want != 0)).any() == (p <= 0)


def test_product_gradient_of_the_two_largest_scales(pm):
    """Scales 253 and 254, which the quantizer does not give: elements that BF16 holds are exact."""
    for byte, fit in ((253, [0, 1, 2, 3, 4, 5]), (254, [0, 1, 2, 3])):
        for code in fit:
            for Kd in (64, 128):
                codes = np.full((1, 16, Kd // 2), code | (code + 8) << 4, np.uint8)
                scales = np.full((1, 16, Kd // 32), byte, np.uint8)
                dy = np.zeros((3, 16))
                dy[[0, 1, 2], [3, 15, 0]] = 2.0 ** -100, -1.0, 2.0 ** -20
                got = _f(pm.mx_grouped_gemm_backward(dev_bf16(_bf(dy)), dev(codes), dev(scales), dev(np.array([0, 3], np.int32))))
                assert np.array_equal(got, dy @ mx.dequantize(codes[0], scales[0]))


def _codes(rng, *shape):
    """Codes and scales [..., Kd] whose products are whole multiples of 2^-4, below 2^20 of it in sum."""
    *lead, Kd = shape
    return (rng.integers(0, 256, (*lead, Kd // 2)).astype(np.uint8),
            rng.integers(126, 128, (*lead, Kd // 32)).astype(np.uint8))


@pytest.mark.parametrize("E,Kd,tile", FORWARD)
def test_product_keeps_nan_blocks_to_what_they_enter_in_every_tile(pm, E, Kd, tile):
    import torch
    rng = np.random.default_rng(E)
    N, R = 256, 255
    assert forward_tile(R * E, E, N, Kd) == tile
    a, w = _codes(rng, R, Kd), _codes(rng, N, Kd)
    a[1][[0, 77, 254], [0, Kd // 32 - 1, 3]] = 255
    w[1][[0, 130, 255], [2, Kd // 32 - 1, 0]] = 255
    off = dev((np.arange(E + 1) * R).astype(np.int32))
    got = _first(pm.mx_grouped_gemm(*(_every(t, E) for t in a), *(_every(t[None], E) for t in w), off, dtype=torch.float32), E)
    want = mx.dequantize(*a) @ mx.dequantize(*w).T
    nan = np.zeros((R, N), bool)
    nan[[0, 77, 254]] = True
    nan[:, [0, 130, 255]] = True
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("E,Kd,tile", BACKWARD)
def test_product_gradient_keeps_nan_to_what_it_enters(pm, E, Kd, tile):
    """A NaN block of the matrix reaches its 32 columns of every row, also where dy is 0; a NaN of dy its whole row."""
    rng = np.random.default_rng(E)
    N = R = 256
    assert backward_tile(R * E, E, N, Kd) == tile
    w, dy = _codes(rng, N, Kd), rng.integers(-16, 17, (R, N)).astype(np.float64)
    w[1][[7, 255], [1, 3]] = 255
    dy[:, 7] = 0.0
    dy[[0, 200], [9, 255]] = np.nan
    off = dev((np.arange(E + 1) * R).astype(np.int32))
    got = _first(pm.mx_grouped_gemm_backward(dev_bf16(np.tile(_bf(dy), (E, 1))), *(_every(t[None], E) for t in w), off), E)
    nan = np.zeros((R, Kd), bool)
    nan[[0, 200]] = True
    nan[:, 32:64] = True
    nan[:, 96:128] = True
    with np.errstate(invalid="ignore"):
        want = bf16_to_f32(_bf(np.where(nan, 0, dy @ mx.dequantize(*w)))).astype(np.float64)
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[~nan], want[~nan])
