"""The microscaled operators at the ends of their ranges, against the float64 oracle (U = 2^-24, half a
step of BF16 = 2^-8 of a normal value, 2^-134 of a subnormal one)."""
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


def _bf(x):
    return f32_to_bf16_rne(np.asarray(x).astype(F32))


def _f(t):
    import torch
    return bf16_to_f32(bf16_bits(t)).astype(np.float64) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


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
