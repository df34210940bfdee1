"""GPU parity of the finalize's gradients with the float64 oracle. Tolerances: d_topk_w is a sum
of H products of BF16 values (exact in FP32 up to their rounding) taken in at most H / 64 + 8
fused steps per lane and 6 between lanes: (H / 64 + 16) 2^-24 of the sum of the sizes; d_z is a
product rounded to FP32 (2^-24) and to BF16 (half a step, 2^-8 of its size)."""
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


def _case(T, K, H, share=0.75, seed=0):
    rng = np.random.default_rng(seed + T * K + H)
    R = max(1, int(T * K * share))
    row = np.full(T * K, -1, np.int32)
    row[rng.permutation(T * K)[:R]] = rng.permutation(R)
    z = f32_to_bf16_rne(rng.standard_normal((R, H)).astype(F32))
    dout = f32_to_bf16_rne(rng.standard_normal((T, H)).astype(F32))
    return dout, z, row, rng.random((T, K)).astype(F32)


def _check(dw, dz, dout, z, row, w):
    H = z.shape[1]
    want_w, want_z, size = ot.finalize_backward(bf16_to_f32(dout), bf16_to_f32(z), row, w)
    assert np.all(np.abs(dw.cpu().numpy() - want_w) <= (H / 64 + 16) * U * size)
    named = ~np.isnan(want_z)
    got = bf16_to_f32(bf16_bits(dz)).astype(np.float64)
    assert np.all(np.abs(got - want_z)[named] <= 2.0 ** -8 * (1 + 2.0 ** -14) * np.abs(want_z)[named] + 1e-38)


@pytest.mark.parametrize("T,K,H", [(1, 1, 8), (1, 8, 7168), (3, 2, 24), (5, 32, 520), (64, 6, 2064), (130, 3, 512),
                                   (257, 17, 1000), (40, 4, 16384)])
def test_gradients(pm, T, K, H):
    import torch
    a = _case(T, K, H)
    dw, dz = pm.finalize_backward(dev_bf16(a[0]), dev_bf16(a[1]), dev(a[2]), dev(a[3]))
    torch.cuda.synchronize()
    _check(dw, dz, *a)


def test_rows_without_a_route_stay_and_bad_rows_are_no_routes(pm):
    import torch
    dout, z, row, w = _case(20, 4, 128)
    R = z.shape[0]
    bad = row.copy()
    bad[row == 3], bad[row == 5] = R, 1 << 30            # behind the last row: no route
    bad[row == 7] = -(1 << 30)
    dz = torch.full((R, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((20, 4), 5.0, device="cuda")
    pm.finalize_backward(dev_bf16(dout), dev_bf16(z), dev(bad), dev(w), out=(dw, dz))
    torch.cuda.synchronize()
    _check(dw, dz, dout, z, bad, w)
    assert bool((dz[[3, 5, 7]] == 5).all()) and not dw.reshape(-1)[dev(bad < 0)].any()
    only_w, none = pm.finalize_backward(dev_bf16(dout), dev_bf16(z), dev(row), dev(w), need_d_z=False)
    none_w, only_z = pm.finalize_backward(dev_bf16(dout), dev_bf16(z), dev(row), dev(w), need_d_topk_w=False)
    full = pm.finalize_backward(dev_bf16(dout), dev_bf16(z), dev(row), dev(w))
    assert none is None and none_w is None
    assert torch.equal(only_w, full[0]) and torch.equal(only_z.view(torch.int16), full[1].view(torch.int16))


def test_nan_stays_with_its_route(pm):
    import torch
    dout, z, row, w = _case(30, 3, 256, share=1.0)
    base = pm.finalize_backward(dev_bf16(dout), dev_bf16(z), dev(row), dev(w))
    zz = z.copy()
    zz[11, 100] = 0x7FC0
    dw, dz = pm.finalize_backward(dev_bf16(dout), dev_bf16(zz), dev(row), dev(w))
    hit = dev(row.reshape(30, 3) == 11)
    assert torch.isnan(dw[hit]).all() and torch.equal(dw[~hit], base[0][~hit])
    assert torch.equal(dz.view(torch.int16), base[1].view(torch.int16))


def test_after_the_layer(pm):
    """z and row_of_route straight from a layer's workspace; rows behind the last route stay."""
    import torch
    import synth
    w = synth.WORKLOADS["swiglu"]
    ids, wts = synth.router(w)
    ids[::5, 1] = -1
    P = pm.prepare_weights(*synth.all_weights(w, device="cuda"))
    ws = torch.empty(pm.moe_workspace_bytes(w.T, w.K, w.E, w.H, w.I, P.act), dtype=torch.uint8, device="cuda")
    pm.moe_forward(dev_bf16(synth.activations(w)), dev(ids), dev(wts), P, workspace=ws)
    v = pm.workspace_views(ws, w.T, w.K, w.E, w.H, w.I, P.act)
    z, row = v["z"].view(torch.bfloat16), v["row_of_route"]
    R = int(v["counters"][0])
    dout = _case(w.T, 1, w.H)[0]
    dz = torch.full((w.T * w.K, w.H), 3.0, dtype=torch.bfloat16, device="cuda")
    dw, _ = pm.finalize_backward(dev_bf16(dout), z, row, dev(wts), out=(None, dz))
    torch.cuda.synchronize()
    assert bool((dz[R:] == 3).all()) and R < w.T * w.K
    _check(dw, dz[:R], dout, bf16_bits(z[:R]), row.cpu().numpy(), wts)


def test_refusals(pm):
    import torch
    dout, z, row, w = _case(8, 2, 64)
    d, zz, r, ww = dev_bf16(dout), dev_bf16(z), dev(row), dev(w)
    with pytest.raises(pm.PmoeError, match="overlaps"):
        pm.finalize_backward(d, zz, r, ww, out=(None, zz))
    with pytest.raises(pm.PmoeError, match="not a HIP device pointer|not device memory"):
        pm.finalize_backward(d, zz, r.cpu(), ww)
    shifted = torch.empty(zz.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(zz.shape)
    with pytest.raises(pm.PmoeError, match="aligned"):
        pm.finalize_backward(d, shifted, r, ww)


def test_more_tokens_than_one_launch_has_threads_for(pm):
    import torch
    T, K, H = (1 << 22) + 3, 16, 8                       # a wave for each slot would be 2^32 threads
    rng = np.random.default_rng(5)
    at = np.array([0, 1, 17, (1 << 20) - 1, 1 << 20, (1 << 22) - 1, 1 << 22, T - 1])
    dout = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    some = f32_to_bf16_rne(rng.standard_normal((len(at), H)).astype(F32))
    dout[torch.from_numpy(at).cuda()] = dev_bf16(some)
    z = f32_to_bf16_rne(rng.standard_normal((len(at) * K, H)).astype(F32))
    row = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    names = rng.permutation(len(at) * K).astype(np.int32).reshape(len(at), K)
    row[torch.from_numpy(at).cuda()] = dev(names)
    w = torch.rand(T, K, device="cuda")
    dw, dz = pm.finalize_backward(dout, dev_bf16(z), row.reshape(-1), w)
    torch.cuda.synchronize()
    pick = torch.from_numpy(at).cuda()
    _check(dw[pick], dz, some, z, names.reshape(-1), w[pick].cpu().numpy())
    dw[pick] = 0
    assert not dw.any()
