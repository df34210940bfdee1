"""Pins of oracle/mx.py against hand enumerations, a library cast and differences."""
import numpy as np
import pytest
import torch

from oracle import mx


def _row(*head):
    return np.array([list(head) + [0.0] * (32 - len(head))])


def test_e2m1_by_hand():
    x = _row(4.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.9, -0.25, -0.5, -0.0)
    codes, scales = mx.quantize(x)
    assert scales[0, 0] == 127                         # amax 7.9: 2^2 / 2^2
    got = mx.dequantize(codes, scales)[0, :13]
    assert got.tolist() == [4, 0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, 0, -0.5]
    nib = [int(codes[0, i // 2] >> (4 * (i % 2)) & 15) for i in range(14)]
    assert nib == [6, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 8, 9, 8]


def test_e4m3_by_hand():
    x = _row(448.0, 464.0, 500.0, -2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 17.0, 19.0, 1.0)
    codes, scales = mx.quantize(x, "e4m3")
    assert scales[0, 0] == 127
    assert mx.dequantize(codes, scales, "e4m3")[0, :9].tolist() == \
        [448, 448, 448, -2.0 ** -9, 0, 2.0 ** -8, 16, 20, 1]


@pytest.mark.parametrize("fmt,emax", [("e2m1", 2), ("e4m3", 8)])
def test_scale_bytes_by_hand(fmt, emax):
    for amax, want in ((1.0, 127 - emax), (1.999, 127 - emax), (2.0, 128 - emax), (2.0 ** -200, 0), (0.0, 0),
                       (2.0 ** (emax - 127), 0), (2.0 ** (emax - 126), 1), (np.inf, 255), (np.nan, 255)):
        codes, scales = mx.quantize(_row(1e-300, -amax), fmt)
        assert scales[0, 0] == want, amax
        if want == 255:
            assert not codes.any() and np.isnan(mx.dequantize(codes, scales, fmt)).all()


def test_e4m3_grid_is_the_library_type():
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(every, mx.E4M3)
    v = np.random.default_rng(0).uniform(0, 448, 4096).astype(np.float32)
    assert np.array_equal(torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), mx.encode(v, "e4m3"))


@pytest.mark.parametrize("fmt,half", [("e2m1", 0.25), ("e4m3", 2.0 ** -4)])
def test_values_are_fixed_points_and_near(fmt, half):
    x = np.random.default_rng(1).standard_normal((40, 96)) * np.exp(np.random.default_rng(2).standard_normal((40, 1)) * 9)
    codes, scales = mx.quantize(x, fmt)
    v = mx.dequantize(codes, scales, fmt)
    again = mx.quantize(v, fmt)
    assert np.array_equal(mx.dequantize(*again, fmt), v)
    amax = np.repeat(np.abs(x).reshape(-1, 32).max(1), 32).reshape(x.shape)
    # half a step of the top binade, or what saturates: amax in [6 X, 8 X) or [448 X, 512 X)
    assert np.all(np.abs(v - x) <= amax * max(half, 0.25 if fmt == "e2m1" else 0.125))


def test_products_by_hand():
    w = np.arange(12.0).reshape(2, 3, 2)
    a = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    out = mx.grouped_gemm(a, w, [0, 1, 2])
    assert out[0].tolist() == [2, 8, 14] and out[1].tolist() == [46, 60, 74] and np.isnan(out[2]).all()
    dx = mx.grouped_gemm_backward(out[:2], w, [0, 1, 2])
    assert dx[0].tolist() == [72, 96]


@pytest.mark.parametrize("act,limit", [("relu2", 0.0), ("swiglu", 0.0), ("swiglu", 1.5)])
def test_activation_gradient_by_differences(act, limit):
    rng = np.random.default_rng(3)
    y, dh = rng.standard_normal((5, 12)) * 2, rng.standard_normal((5, 12 if act == "relu2" else 6))
    y = np.where(np.abs(np.abs(y) - limit) < 1e-3, y + 0.01, y)
    got = mx.activation_backward(dh, y, act, limit)
    for i in np.ndindex(*y.shape):
        d = np.zeros_like(y)
        d[i] = 1e-6
        want = (dh * (mx.activation(y + d, act, limit) - mx.activation(y - d, act, limit))).sum() / 2e-6
        assert abs(got[i] - want) <= 1e-6 * max(1.0, abs(want))
    t = torch.from_numpy(y)
    if act == "swiglu" and not limit:
        g, u = t.chunk(2, 1)
        assert np.allclose(mx.activation(y, act), (torch.nn.functional.silu(g) * u).numpy(), rtol=1e-14)


def test_permutation_by_hand():
    ids = [[2, 0], [0, 5], [1, 2], [-1, 0]]
    row, route, off = mx.permute(ids, 3)
    assert route.tolist() == [1, 2, 7, 4, 0, 5] and off.tolist() == [0, 3, 4, 6]
    assert row.tolist() == [4, 0, 1, -1, 3, 5, -1, 2]
    d = np.arange(6.0)[:, None]
    assert mx.permute_backward(d, row, 2)[:, 0].tolist() == [4, 1, 8, 2]
    row, route, off = mx.permute(ids, 2, expert_offset=4)
    assert route.tolist() == [3] and off.tolist() == [0, 0, 1]
