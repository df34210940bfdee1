"""What is trained, or chosen per request, around the frozen experts, on the CPU in
float64: the router's balance loss and z-loss, the gradients of the router and of
the finalize, and low-rank adapters with their gradients.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py). Plain formulas without any of
the library's blocking, rounded nowhere; the losses are written so that central
differences of them check the gradients.
"""
import numpy as np

F64 = np.float64


def _softmax(logits):
    """(p, lse) of float64 rows; rows of -inf only give p = 0, lse = -inf."""
    l = np.asarray(logits, F64)
    m = l.max(axis=1, keepdims=True)
    ex = np.exp(l - np.where(m > -np.inf, m, 0.0))
    den = ex.sum(axis=1, keepdims=True)
    p = ex / np.where(den > 0, den, 1.0)
    with np.errstate(divide="ignore"):
        lse = np.where(m > -np.inf, m, 0.0)[:, 0] + np.log(den[:, 0])
    return p, lse


def active_tokens(logits, ids):
    ids = np.asarray(ids)
    E = np.shape(logits)[1]
    return ((ids >= 0) & (ids < E)).any(axis=1) & (np.asarray(logits) > -np.inf).any(axis=1)


def router_balance(logits, ids, offsets=None):
    """(counts [S, E], tokens [S], prob [S, E], balance [S], z [S])."""
    logits, ids = np.asarray(logits, F64), np.asarray(ids)
    T, E = logits.shape
    K = ids.shape[1]
    offsets = np.array([0, T]) if offsets is None else np.asarray(offsets)
    S = offsets.size - 1
    p, lse = _softmax(logits)
    active = active_tokens(logits, ids)
    counts, tokens = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    prob, balance, z = np.zeros((S, E)), np.zeros(S), np.zeros(S)
    for s in range(S):
        for t in range(offsets[s], offsets[s + 1]):
            if active[t]:
                tokens[s] += 1
                prob[s] += p[t]
                z[s] += lse[t] ** 2
                for e in ids[t]:
                    if 0 <= e < E:
                        counts[s, e] += 1
        if tokens[s]:
            n = tokens[s]
            balance[s] = E * np.sum(counts[s] / (n * K) * prob[s] / n)
            z[s] /= n
    return counts, tokens, prob, balance, z


def topk_weights(logits, ids, renormalize=False):
    """The weights of given ids [T, K] (0 where an id is no expert or a token not active)."""
    logits, ids = np.asarray(logits, F64), np.asarray(ids).astype(np.int64)
    E = logits.shape[1]
    valid = (ids >= 0) & (ids < E) & active_tokens(logits, ids)[:, None]
    w = np.where(valid, np.take_along_axis(_softmax(logits)[0], np.where(valid, ids, 0), axis=1), 0.0)
    if renormalize:
        den = w.sum(axis=1, keepdims=True)
        w = w / np.where(den > 0, den, 1.0)
    return w


def router_backward(logits, ids, counts=None, tokens=None, d_balance=None, d_z=None, d_w=None,
                    renormalize=False, offsets=None):
    """(gradient of the logits, the same with every term taken positive: the size of what is added)."""
    logits, ids = np.asarray(logits, F64), np.asarray(ids)
    T, E = logits.shape
    K = ids.shape[1]
    offsets = np.array([0, T]) if offsets is None else np.asarray(offsets)
    p, lse = _softmax(logits)
    active = active_tokens(logits, ids)
    w = topk_weights(logits, ids, renormalize)
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if not active[t]:
            continue
        s = int(np.searchsorted(offsets, t, side="right")) - 1
        if 0 <= s < offsets.size - 1:
            n = max(int(tokens[s]), 1) if tokens is not None else 1
            if d_balance is not None:
                f = np.asarray(counts[s], F64) / (n * K)
                c = float(d_balance[s]) * E / n
                grad[t] += c * p[t] * (f - np.sum(f * p[t]))
                size[t] += abs(c) * p[t] * (f + np.sum(f * p[t]))
            if d_z is not None:
                c = 2.0 * float(d_z[s]) / n * lse[t]
                grad[t] += c * p[t]
                size[t] += abs(c) * p[t]
        if d_w is not None:
            valid = [j for j in range(K) if 0 <= ids[t, j] < E]
            dw = np.asarray(d_w[t], F64)
            mean = sum(dw[j] * w[t, j] for j in valid)
            mean_abs = sum(abs(dw[j]) * w[t, j] for j in valid)
            if not renormalize:
                grad[t] -= p[t] * mean
                size[t] += p[t] * mean_abs
            for j in valid:
                e = ids[t, j]
                grad[t, e] += w[t, j] * (dw[j] - mean) if renormalize else w[t, j] * dw[j]
                size[t, e] += w[t, j] * (abs(dw[j]) + (mean_abs if renormalize else 0.0))
    return grad, size


def finalize_backward(dout, z, row_of_route, w):
    """(d_w [T, K], d_z [R, H] with NaN in rows that no route names, the size of the sums in d_w)."""
    dout, z, w = (np.asarray(a, F64) for a in (dout, z, w))
    T, K = w.shape
    row = np.asarray(row_of_route).reshape(T, K)
    d_w, size, d_z = np.zeros((T, K)), np.zeros((T, K)), np.full(z.shape, np.nan)
    for t in range(T):
        for j in range(K):
            r = row[t, j]
            if 0 <= r < z.shape[0]:
                d_w[t, j] = np.sum(dout[t] * z[r])
                size[t, j] = np.sum(np.abs(dout[t] * z[r]))
                d_z[r] = w[t, j] * dout[t]
    return d_w, d_z, size


def adapter_forward(x, ids, down, up, scale, base=None):
    """(out [T, N], v [T, R]), not rounded."""
    x, down, up, scale = (np.asarray(a, F64) for a in (x, down, up, scale))
    n, R, _ = down.shape
    out = np.zeros((x.shape[0], up.shape[1])) if base is None else np.array(base, F64)
    v = np.zeros((x.shape[0], R))
    for a in range(n):
        t = np.nonzero(np.asarray(ids) == a)[0]
        v[t] = x[t] @ down[a].T
        out[t] += scale[a] * (v[t] @ up[a].T)
    return out, v


def adapter_backward(dy, x, v, ids, down, up, scale, base=None):
    """(dx [T, H], d_down [n, R, H], d_up [n, N, R], du [T, R]), not rounded."""
    dy, x, v, down, up, scale = (np.asarray(a, F64) for a in (dy, x, v, down, up, scale))
    dx = np.zeros(x.shape) if base is None else np.array(base, F64)
    d_down, d_up, du = np.zeros(down.shape), np.zeros(up.shape), np.zeros(v.shape)
    for a in range(down.shape[0]):
        t = np.nonzero(np.asarray(ids) == a)[0]
        du[t] = scale[a] * (dy[t] @ up[a])
        dx[t] += du[t] @ down[a]
        d_down[a] = du[t].T @ x[t]
        d_up[a] = scale[a] * (dy[t].T @ v[t])
    return dx, d_down, d_up, du
