"""Microscaled formats and the operators of an MXFP4 expert layer, on the CPU in float64:
quantization and its inverse, the grouped product with its gradient, the activation with its
8-bit checkpoint, and tokens sorted by expert with the gradient of the copy.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py). The formats are those of the OCP Microscaling
Formats specification v1.0 (section 5.3.3: E2M1, 5.3.1: E4M3, 5.4: E8M0, 6.3: the conversion): a
block of 32 elements shares X = 2^(byte - 127), byte = max(floor(log2 amax) - emax, -127) + 127,
and its elements are x / X, to nearest, ties to the even code, saturated. A block with an infinity
or a NaN has byte 255 and zero codes.
"""
import numpy as np

F64 = np.float64
BLOCK = 32
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], F64)
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1], F64)
GRID = {"e2m1": E2M1, "e4m3": E4M3}
EMAX = {"e2m1": 2, "e4m3": 8}


def encode(a, fmt):
    """Codes (sign apart) of magnitudes: the borders passed, one that is met only towards an even code."""
    grid = GRID[fmt]
    mid = (grid[1:] + grid[:-1]) / 2
    below, upto = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
    return np.where(below % 2 == 0, below, upto)


def quantize(x, fmt="e2m1"):
    """(codes, scale bytes) of float64 rows [..., n]; E2M1 codes are packed, element 2i in the low nibble."""
    x = np.asarray(x, F64)
    b = x.reshape(-1, BLOCK)
    good = np.isfinite(b).all(1)
    b = np.where(good[:, None], b, 0.0)
    amax = np.abs(b).max(1)
    _, e = np.frexp(amax)                              # amax = m 2^e, 0.5 <= m < 1
    byte = np.where(amax > 0, np.maximum(e - 1 - EMAX[fmt], -127) + 127, 0)
    assert byte.max(initial=0) <= 254
    code = encode(np.abs(b) * np.ldexp(1.0, 127 - byte)[:, None], fmt)
    code = code + np.signbit(b) * (8 if fmt == "e2m1" else 128)
    code = np.where(good[:, None], code, 0).astype(np.uint8).reshape(x.shape)
    if fmt == "e2m1":
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    return code, np.where(good, byte, 255).astype(np.uint8).reshape(*x.shape[:-1], x.shape[-1] // BLOCK)


def dequantize(codes, scales, fmt="e2m1"):
    """The float64 values that codes and scales stand for."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    if fmt == "e2m1":
        c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
        v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    else:
        c = codes
        v = np.append(E4M3, np.nan)[c & 127] * np.where(c & 128, -1.0, 1.0)
    x = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(x, BLOCK, -1)


def experts_of_rows(offsets, R):
    """Expert of each row, -1 for rows of no expert."""
    e = np.full(R, -1)
    for i in range(len(offsets) - 1):
        e[offsets[i]:offsets[i + 1]] = i
    return e


def grouped_gemm(a, w, offsets):
    """out[r] = w[e(r)] a[r] of values a [R, Kd] and w [E, N, Kd]; NaN in rows of no expert."""
    e = experts_of_rows(offsets, len(a))
    out = np.full((len(a), w.shape[1]), np.nan)
    for i in np.unique(e[e >= 0]):
        out[e == i] = a[e == i] @ w[i].T
    return out


def grouped_gemm_backward(dy, w, offsets):
    return grouped_gemm(dy, w.transpose(0, 2, 1), offsets)


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def activation(y, act, limit=0.0):
    """h in float64: squared ReLU, or SwiGLU of gate and up halves."""
    y = np.asarray(y, F64)
    if act == "relu2":
        return np.where(y < 0, 0.0, y) ** 2
    g, u = np.split(y, 2, axis=-1)
    if limit > 0:
        g, u = np.where(g > limit, limit, g), np.clip(u, -limit, limit)
    with np.errstate(invalid="ignore"):
        return g * _sigmoid(g) * u


def activation_backward(dh, y, act, limit=0.0):
    dh, y = np.asarray(dh, F64), np.asarray(y, F64)
    if act == "relu2":
        return 2 * np.where(y < 0, 0.0, y) * dh
    g, u = np.split(y, 2, axis=-1)
    in_g, in_u = np.ones_like(g), np.ones_like(u)
    if limit > 0:
        in_g, in_u = (g <= limit).astype(F64), (np.abs(u) <= limit).astype(F64)
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    s = _sigmoid(g)
    return np.concatenate([dh * u * s * (1 + g * (1 - s)) * in_g, dh * g * s * in_u], -1)


def permute(ids, E, expert_offset=0):
    """(row_of_route, route_of_row of the valid rows, expert_offsets)."""
    flat = np.asarray(ids).reshape(-1).astype(np.int64) - expert_offset
    route = [f for e in range(E) for f in np.nonzero(flat == e)[0]]
    row = np.full(flat.size, -1, np.int32)
    row[route] = np.arange(len(route))
    counts = [int((flat == e).sum()) for e in range(E)]
    return row, np.array(route, np.int32), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def permute_backward(d_rows, row_of_route, K):
    """dx [T, H]: the sum of each token's rows."""
    d = np.asarray(d_rows, F64)
    row = np.asarray(row_of_route).reshape(-1, K)
    dx = np.zeros((row.shape[0], d.shape[1]))
    for j in range(K):
        on = (row[:, j] >= 0) & (row[:, j] < len(d))
        dx[on] += d[row[on, j]]
    return dx
