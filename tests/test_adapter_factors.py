"""The gradients of the adapters' matrices hold all 24 bits of v and du.

Every column of x (dy) is zero but for one token, so an entry of d_down (d_up) is one product and
whatever else is added to it is zero. With u = 2^-24, half a step of FP32, it is off by the
rounding of scale * v (of scale * dy, where `up` has one 1 in each column: du is that product) and by
the sum of the three BF16 parts of that factor times the BF16 value: products of 8 and 8 bits are exact,
the two lower parts are below 2^-7 of the whole, and the additions may round or cut (u or 2 u):
(1 + 2 (1 + 2^-7)) u, below 4 u. Without the last part up to 2^-15 = 512 u of a product are missing."""
import numpy as np
import pytest

from helpers import dev, dev_bf16
from oracle.formats import bf16_to_f32, f32_to_bf16_rne

F32, F64 = np.float32, np.float64
BOUND = 4 * 2.0 ** -24
CASES = [(144, 3, 8), (144, 3, 24), (144, 3, 64), (144, 3, 128), (1200, 1, 16), (1200, 1, 72)]


def _bf16(rng, *shape):
    """Values of size 1 .. 2, either sign."""
    a = (rng.uniform(1, 2, shape) * rng.choice([-1.0, 1.0], shape)).astype(F32)
    return f32_to_bf16_rne(a)


class Case:
    def __init__(self, T, n, R):
        rng = np.random.default_rng(T + R)
        self.T, self.n, self.R = T, n, R
        self.ids = rng.integers(0, n, T).astype(np.int32)
        self.one = np.where(np.eye(T, dtype=bool), _bf16(rng, T, T), np.uint16(0))      # column t is token t's
        self.full = _bf16(rng, T, T)
        self.v = (rng.uniform(1, 2, (T, R)) * rng.choice([-1.0, 1.0], (T, R))).astype(F32)
        self.scale = rng.uniform(0.5, 2, n).astype(F32)
        self.down = _bf16(rng, n, R, T)
        self.up = np.zeros((n, T, R), np.uint16)
        self.up[:, rng.permutation(T)[:R], np.arange(R)] = f32_to_bf16_rne(np.ones(R, F32))

    def factors(self, which):
        """scale * v, or du = scale * dy at the rows of `up` that hold a 1: float64 [T, R], not rounded."""
        s = self.scale[self.ids].astype(F64)[:, None]
        if which == "up":
            return s * self.v
        row = np.array([np.nonzero(self.up[0, :, r])[0][0] for r in range(self.R)])
        return s * bf16_to_f32(self.full)[:, row]

    def want(self, which):
        """[n, R, T], 0 where the column's token uses another adapter."""
        mine = np.arange(self.n)[:, None, None] == self.ids
        return np.where(mine, (self.factors(which) * np.diag(bf16_to_f32(self.one)).astype(F64)[:, None]).T, 0.0)


def _parts(a, count):
    """The sum of the first `count` BF16 parts of FP32 values, each the upper half of what is left."""
    total, rest = np.zeros(a.shape, F64), a.astype(F32)
    for _ in range(count):
        part = (rest.view(np.uint32) & np.uint32(0xFFFF0000)).view(F32)
        total, rest = total + part, rest - part
    return total


@pytest.mark.parametrize("T,n,R", CASES)
@pytest.mark.parametrize("which", ["up", "down"])
def test_the_bound_tells_two_parts_from_three(T, n, R, which):
    c = Case(T, n, R)
    exact = c.factors(which)
    rounded = exact.astype(F32)
    assert np.array_equal(_parts(rounded, 3), rounded)
    assert np.all(np.abs(_parts(rounded, 3) - exact) <= BOUND * np.abs(exact))
    missing = np.abs(_parts(rounded, 2) - exact) > BOUND * np.abs(exact)
    assert missing.mean() > 0.9 and missing.any(axis=1).all() and missing.any(axis=0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,R", CASES)
def test_factors_are_held_whole(T, n, R):
    import torch
    import precision_moe_amd as pm
    c = Case(T, n, R)
    weights = dev_bf16(c.down), dev_bf16(c.up), dev(c.scale)
    one, full, v, ids = dev_bf16(c.one), dev_bf16(c.full), dev(c.v), dev(c.ids)
    _, _, d_up = pm.adapter_backward(one, full, v, ids, *weights, need_dx=False)
    _, d_down, _ = pm.adapter_backward(full, one, v, ids, *weights, need_dx=False)
    torch.cuda.synchronize()
    for got, which in ((d_up.cpu().numpy().transpose(0, 2, 1), "up"), (d_down.cpu().numpy(), "down")):
        want = c.want(which)
        assert np.all(np.abs(got - want) <= BOUND * np.abs(want)), which
