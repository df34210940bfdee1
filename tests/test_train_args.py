"""Refusals of the router, finalize and adapter training calls that need no GPU: shapes and
arguments are checked before any device work (C ABI), dtypes and tensor shapes by the binding."""
import ctypes

import pytest
import torch

import precision_moe_amd as pm

SHAPE, ARG = 3, 7
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _rc(name, *args):
    return getattr(pm.lib(), name)(*args)


def _balance(T=4, K=2, E=8, off=None, S=1, ids_type=0):
    return _rc("pmoe_router_balance", None, None, ids_type, T, K, E, off, S, None, None, None, None, None,
               None, 0, None)


def _backward(T=4, K=2, E=8, renorm=0, off=None, S=1, counts=None, tokens=None, db=None, dz=None, dw=None,
              ids_type=0):
    return _rc("pmoe_router_backward", None, None, ids_type, T, K, E, renorm, off, S, counts, tokens, db, dz,
               dw, None, None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=9), dict(E=64, K=33),
                                dict(S=0, off=1), dict(S=65537, off=1), dict(T=1 << 29, K=2)])
def test_router_shapes(kw):
    assert _balance(**kw) == SHAPE
    assert _backward(dw=1, **kw) == SHAPE
    assert pm.lib().pmoe_last_error()
    if "off" not in kw:
        sizes = dict(T=4, K=2, E=8, S=1) | kw
        assert _rc("pmoe_router_balance_workspace_bytes", sizes["T"], sizes["E"], sizes["K"], sizes["S"]) == 0


def test_router_arguments():
    assert _balance(S=2) == ARG                        # several sequences need offsets
    assert _balance(ids_type=2) == ARG
    assert _backward() == ARG                          # no gradient given
    assert _backward(dw=1, ids_type=5) == ARG
    assert _backward(dw=1, renorm=2) == ARG
    assert _backward(db=1, tokens=1) == ARG            # counts missing
    assert _backward(db=1, counts=1) == ARG            # tokens missing
    assert _backward(dz=1) == ARG
    assert _backward(T=0) == 0                         # nothing to do
    with pytest.raises(pm.PmoeError):
        pm.router_balance_workspace_bytes(4, 9, 8)
    assert pm.router_balance_workspace_bytes(0, 2, 8) > 0


def test_finalize_backward_arguments():
    def call(T=4, K=2, H=64, R=8, dw=1, dz=None):
        return _rc("pmoe_finalize_backward", None, None, None, None, T, K, H, R, dw, dz, None)
    for kw in (dict(T=-1), dict(K=0), dict(K=33), dict(H=0), dict(H=60), dict(H=(1 << 30) + 8), dict(R=-1),
               dict(T=1 << 29, K=2)):
        assert call(**kw) == SHAPE, kw
    assert call(dw=None) == ARG
    assert call(T=0, dw=None) == 0 and call(R=0, dw=None) == 0         # nothing to do


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=(1 << 24) + 1), dict(n=0), dict(n=65536), dict(H=8),
                                dict(H=100), dict(H=16400), dict(N=0), dict(N=24), dict(R=0), dict(R=4),
                                dict(R=12), dict(R=136)])
def test_adapter_shapes(kw):
    d = dict(T=4, n=2, H=64, N=64, R=16) | kw
    sizes = (d["T"], d["n"], d["H"], d["N"], d["R"])
    assert _rc("pmoe_adapter_forward", None, None, 0, *sizes, None, None, None, None, None, None, None, 0,
               None) == SHAPE
    assert _rc("pmoe_adapter_backward", None, None, None, None, 0, *sizes, None, None, None, None, 1, 1, 1,
               None, 0, None) == SHAPE
    assert _rc("pmoe_adapter_workspace_bytes", *sizes, 0) == 0
    with pytest.raises(pm.PmoeError):
        pm.adapter_workspace_bytes(*sizes, backward=True)


def test_adapter_arguments():
    sizes = (4, 2, 64, 64, 16)

    def forward(sizes=sizes, ids_type=0):
        return _rc("pmoe_adapter_forward", None, None, ids_type, *sizes, None, None, None, None, None, None,
                   None, 0, None)

    def backward(base=None, dx=1, dd=1, du=1, sizes=sizes, ids_type=0):
        return _rc("pmoe_adapter_backward", None, None, None, None, ids_type, *sizes, None, None, None, base,
                   dx, dd, du, None, 0, None)

    assert forward(ids_type=3) == ARG and backward(ids_type=3) == ARG
    assert backward(dd=None) == ARG and backward(du=None) == ARG       # both or neither
    assert backward(dx=None, dd=None, du=None) == ARG                  # nothing wanted
    assert backward(base=1, dx=None) == ARG
    assert forward(sizes=(0, 2, 64, 64, 16)) == 0
    assert backward(sizes=(0, 2, 64, 64, 16), dd=None, du=None) == 0
    assert _rc("pmoe_adapter_workspace_bytes", *sizes, 2) == 0
    assert pm.adapter_workspace_bytes(*sizes) >= 256


def test_binding_dtypes_and_shapes():
    T, n, H, N, R = 4, 2, 64, 32, 16
    x, ids = torch.zeros(T, H, dtype=BF), torch.zeros(T, dtype=I32)
    down, up, scale = torch.zeros(n, R, H, dtype=BF), torch.zeros(n, N, R, dtype=BF), torch.zeros(n)
    good = dict(x=x, adapter_ids=ids, down=down, up=up, scale=scale)
    for bad, err in ((dict(x=x.half()), TypeError), (dict(x=x[:3]), ValueError), (dict(up=up.float()), TypeError),
                     (dict(up=up[:1]), ValueError), (dict(up=up[:, :, :8]), ValueError),
                     (dict(scale=scale[:1]), ValueError), (dict(scale=scale.double()), TypeError),
                     (dict(adapter_ids=ids.float()), TypeError), (dict(adapter_ids=ids[None]), ValueError),
                     (dict(base=torch.zeros(T, H, dtype=BF)), ValueError),
                     (dict(out=torch.zeros(N, T, dtype=BF).t()), ValueError),
                     (dict(v=torch.zeros(T, R + 8)), ValueError)):
        with pytest.raises(err):
            pm.adapter_forward(**(good | bad))
    dy, v = torch.zeros(T, N, dtype=BF), torch.zeros(T, R)
    for bad, err in ((dict(dy=dy.float()), TypeError), (dict(v=v[:, :8]), ValueError), (dict(v=v.to(BF)), TypeError),
                     (dict(out=(None, torch.zeros(n, H, R), None)), ValueError)):
        with pytest.raises(err):
            pm.adapter_backward(**(dict(dy=dy, v=v) | good | bad))
    lg, tk = torch.zeros(T, 8), torch.zeros(T, 2, dtype=I32)
    for args, kw, err in (((lg.double(), tk), {}, TypeError), ((lg, tk.float()), {}, TypeError),
                          ((lg, tk[:3]), {}, ValueError), ((lg[0], tk), {}, ValueError),
                          ((lg, tk), dict(seq_offsets=torch.zeros(1, dtype=I32)), ValueError),
                          ((lg, tk), dict(seq_offsets=torch.zeros(3)), TypeError)):
        with pytest.raises(err):
            pm.router_balance(*args, **kw)
        with pytest.raises(err):
            pm.router_backward(*args, d_topk_w=torch.zeros(T, 2), **kw)
    with pytest.raises(ValueError):
        pm.router_backward(lg, tk, d_topk_w=torch.zeros(T, 3))
    z, w = torch.zeros(8, H, dtype=BF), torch.zeros(T, 2)
    row = torch.zeros(T * 2, dtype=I32)
    for args, err in (((x.float(), z, row, w), TypeError), ((x, z.float(), row, w), TypeError),
                      ((x, z[:, :32], row, w), ValueError), ((x, z, row[:3], w), ValueError),
                      ((x, z, row.long(), w), TypeError)):
        with pytest.raises(err):
            pm.finalize_backward(*args)


def test_layer_adapters_are_refused_before_the_layer_runs():
    H, E, K, T = 64, 4, 2, 4
    P = pm.PreparedWeights(E, H, H, H, *([None] * 6))
    x, tk, w = torch.zeros(T, H, dtype=BF), torch.zeros(T, K, dtype=I32), torch.zeros(T, K)
    down, up, scale = torch.zeros(2, 8, H, dtype=BF), torch.zeros(2, 32, 8, dtype=BF), torch.zeros(2)
    ids = torch.zeros(T, dtype=I32)
    with pytest.raises(ValueError, match="both or neither"):
        pm.moe_forward(x, tk, w, P, adapters=(down, up, scale))
    with pytest.raises(ValueError, match="adapters of a layer"):
        pm.moe_forward(x, tk, w, P, adapters=(down, up, scale), adapter_ids=ids)
    up = torch.zeros(2, H, 8, dtype=BF)
    layer = dict(adapters=(down, up, scale), adapter_ids=ids)
    with pytest.raises(ValueError, match="overlaps x"):
        pm.moe_forward(x, tk, w, P, out=x, **layer)
    with pytest.raises(ValueError, match="overlaps x"):
        both = torch.zeros(T + 1, H, dtype=BF)
        pm.moe_forward(both[1:], tk, w, P, out=both[:T], **layer)
    with pytest.raises(ValueError, match="adapter_workspace too small"):
        pm.moe_forward(x, tk, w, P, adapter_workspace=torch.empty(16, dtype=torch.uint8), **layer)
    with pytest.raises(ValueError, match="on the device of x"):
        pm.moe_forward(x, tk, w, P, adapters=(down, up.to("meta"), scale), adapter_ids=ids)
    with pytest.raises(pm.PmoeError, match="multiple of 8"):
        pm.moe_forward(x, tk, w, P, adapters=(down[:, :4], up[:, :, :4], scale), adapter_ids=ids)
    assert ctypes.sizeof(pm.MoeOptions) == 48          # the options of the C ABI keep their layout
