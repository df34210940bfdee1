"""Refusals of the permutation and microscaled calls that need no GPU: shapes and arguments are
checked before any device work (C ABI), dtypes and tensor shapes by the binding."""
import pytest
import torch

import precision_moe_amd as pm

SHAPE, ACT, ARG = 3, 4, 7
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _rc(name, *args):
    return getattr(pm.lib(), name)(*args)


def _permute(T=4, K=2, E=8, ids_type=0, x=None, row_bytes=16, rows=None):
    return _rc("pmoe_permute_tokens", None, ids_type, T, K, E, 0, x, row_bytes, rows, None, None, None, None, 0, None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=33), dict(E=64, K=33),
                                dict(T=1 << 29, K=2), dict(x=16, rows=16, row_bytes=0),
                                dict(x=16, rows=16, row_bytes=24), dict(x=16, rows=16, row_bytes=(1 << 20) + 16)])
def test_permute_shapes(kw):
    assert _permute(**kw) == SHAPE
    if "x" not in kw:
        sizes = dict(T=4, K=2, E=8) | kw
        assert _rc("pmoe_permute_workspace_bytes", sizes["T"], sizes["K"], sizes["E"]) == 0


def test_permute_arguments():
    assert _permute(ids_type=2) == ARG
    assert _permute(x=16) == ARG and _permute(rows=16) == ARG          # both or neither
    with pytest.raises(pm.PmoeError):
        pm.permute_workspace_bytes(4, 33, 8)
    assert pm.permute_workspace_bytes(0, 2, 8) > 0 and pm.permute_workspace_bytes(4, 9, 8) > 0

    def back(type=0, T=4, K=2, R=8, H=64):
        return _rc("pmoe_permute_tokens_backward", None, type, None, T, K, R, H, None, None)
    for kw in (dict(T=-1), dict(K=0), dict(K=33), dict(R=-1), dict(H=0), dict(H=60), dict(H=62, type=1),
               dict(H=(1 << 18) + 8), dict(T=1 << 29)):
        assert back(**kw) == SHAPE, kw
    assert back(type=2) == ARG
    assert back(T=0) == 0


def test_quantize_arguments():
    def both(type=0, fmt=0, rows=4, n=64):
        a = _rc("pmoe_mx_quantize", None, type, fmt, rows, n, None, None, None)
        assert a == _rc("pmoe_mx_dequantize", None, None, fmt, rows, n, type, None, None)
        return a
    for kw in (dict(rows=-1), dict(n=0), dict(n=-32), dict(n=48), dict(rows=1 << 35), dict(rows=(1 << 63) - 1)):
        assert both(**kw) == SHAPE, kw
    assert both(type=2) == ARG and both(fmt=2) == ARG and both(fmt=-1) == ARG
    assert both(rows=0) == 0


def test_gemm_arguments():
    def forward(a_rows=8, route=None, topk=1, R=8, E=2, N=32, Kd=64, type=0):
        return _rc("pmoe_mx_grouped_gemm", None, None, a_rows, route, topk, None, R, E, None, None, N, Kd, None, type, None)

    def backward(R=8, E=2, N=32, Kd=64):
        return _rc("pmoe_mx_grouped_gemm_backward", None, None, R, E, None, None, N, Kd, None, None)
    for kw in (dict(R=-1), dict(R=(1 << 23) + 1), dict(E=0), dict(E=1025), dict(N=0), dict(N=24), dict(N=32784),
               dict(Kd=0), dict(Kd=48), dict(Kd=16416)):
        assert forward(**kw) == SHAPE and backward(**kw) == SHAPE, kw
    assert forward(a_rows=7) == SHAPE and forward(a_rows=-1, route=16) == SHAPE
    assert forward(a_rows=1 << 26, route=16) == SHAPE                  # 32-bit offsets of a gathered operand
    assert forward(topk=0) == ARG and forward(type=2) == ARG
    assert forward(R=0, a_rows=0) == 0 and backward(R=0) == 0


def test_activation_arguments():
    def forward(R=8, I=64, act=1, limit=0.0, y8=None, y8_sf=None):
        return _rc("pmoe_mx_activation", None, R, I, act, limit, None, None, None, y8, y8_sf, None)

    def backward(R=8, I=64, act=1, limit=0.0):
        return _rc("pmoe_mx_activation_backward", None, None, None, R, I, act, limit, None, None, None)
    for f in (forward, backward):
        for kw in (dict(R=-1), dict(R=(1 << 23) + 1), dict(I=0), dict(I=48), dict(I=16416)):
            assert f(**kw) == SHAPE, kw
        assert f(act=2) == ACT and f(limit=-1.0) == ARG and f(limit=float("nan")) == ARG
        assert f(act=0, limit=1.0) == ARG and f(R=0) == 0
    assert forward(y8=16) == ARG and forward(y8_sf=16) == ARG


def test_binding_dtypes_and_shapes():
    T, K, E, H = 4, 2, 8, 64
    x, ids = torch.zeros(T, H, dtype=BF), torch.zeros(T, K, dtype=I32)
    for args, kw, err in (((x, ids.float(), E), {}, TypeError), ((x[:3], ids, E), {}, ValueError),
                          ((x, ids[0], E), {}, ValueError), ((x[0], ids, E), {}, ValueError),
                          ((None, ids, E), dict(out=(x, None, None, None)), ValueError),
                          ((x, ids, E), dict(out=(x, None, None, None)), ValueError),
                          ((x, ids, E), dict(out=(None, None, None, torch.zeros(E, dtype=I32))), ValueError)):
        with pytest.raises(err):
            pm.permute_tokens(*args, **kw)
    row = torch.zeros(T * K, dtype=I32)
    for args, err in (((x.half(), row, K), TypeError), ((x, row.long(), K), TypeError), ((x, row, 3), ValueError),
                      ((x, row, 0), ValueError), ((x[0], row, K), ValueError)):
        with pytest.raises(err):
            pm.permute_tokens_backward(*args)
    for args, kw, err in (((x.half(),), {}, TypeError), ((x[:, :48],), {}, ValueError), ((x,), dict(format="e5m2"), ValueError),
                          ((x,), dict(out=(torch.zeros(T, H, dtype=U8), None)), ValueError)):
        with pytest.raises(err):
            pm.mx_quantize(*args, **kw)
    codes, sf = torch.zeros(T, H // 2, dtype=U8), torch.zeros(T, H // 32, dtype=U8)
    for args, kw, err in (((codes, sf[:, :1]), {}, ValueError), ((codes.int(), sf), {}, TypeError),
                          ((codes, sf), dict(dtype=torch.float16), TypeError), ((codes, sf), dict(format="e4m3"), ValueError)):
        with pytest.raises(err):
            pm.mx_dequantize(*args, **kw)
    w, w_sf, off = torch.zeros(E, 32, H // 2, dtype=U8), torch.zeros(E, 32, H // 32, dtype=U8), torch.zeros(E + 1, dtype=I32)
    for args, kw, err in (((codes, sf, w, w_sf, off[1:]), {}, ValueError), ((codes, sf, w, w_sf, off.long()), {}, TypeError),
                          ((codes[:, :16], sf, w, w_sf, off), {}, ValueError), ((codes, sf[:, :1], w, w_sf, off), {}, ValueError),
                          ((codes, sf, w[0], w_sf, off), {}, ValueError), ((codes, sf, w, w_sf[:, :16], off), {}, ValueError),
                          ((codes, sf, w, w_sf, off), dict(dtype=torch.float16), TypeError),
                          ((codes, sf, w, w_sf, off), dict(out=torch.zeros(T, 16, dtype=BF)), ValueError),
                          ((codes, sf, w, w_sf, off), dict(route_of_row=row.long()), TypeError)):
        with pytest.raises(err):
            pm.mx_grouped_gemm(*args, **kw)
    dy = torch.zeros(T, 32, dtype=BF)
    for args, err in (((dy.float(), w, w_sf, off), TypeError), ((dy[:, :16], w, w_sf, off), ValueError),
                      ((dy, w, w_sf, off[1:]), ValueError), ((dy[0], w, w_sf, off), ValueError)):
        with pytest.raises(err):
            pm.mx_grouped_gemm_backward(*args)
    for args, kw, err in (((x.float(), 1), {}, TypeError), ((x[:, :63], 1), {}, ValueError), ((x[0], 1), {}, ValueError),
                          ((x, 1), dict(row_count=off), ValueError), ((x, 1), dict(row_count=torch.zeros(1)), TypeError),
                          ((x, 1), dict(out=(codes, None, None, None)), ValueError)):
        with pytest.raises(err):
            pm.mx_activation(*args, **kw)
    y8, y8_sf = torch.zeros(T, H, dtype=U8), torch.zeros(T, H // 32, dtype=U8)
    for args, err in (((dy.float(), y8, y8_sf, 1), TypeError), ((dy, y8[:, :32], y8_sf, 1), ValueError),
                      ((dy, y8, y8_sf[:, :1], 1), ValueError), ((dy, y8, y8_sf, 0), ValueError)):
        with pytest.raises(err):
            pm.mx_activation_backward(*args)


def test_binding_refuses_what_an_int_would_cut():
    """Sizes past 32 bits, on tensors without memory: they reach the C interface as 32-bit ints."""
    def meta(*shape, dtype=BF):
        return torch.empty(shape, dtype=dtype, device="meta")
    big, ids, row = 2 ** 32 + 32, torch.zeros(4, 2, dtype=I32), torch.zeros(8, dtype=I32)
    w, w_sf, off = meta(1, 32, 32, dtype=U8), meta(1, 32, 2, dtype=U8), torch.zeros(2, dtype=I32)
    for call in (lambda: pm.permute_tokens(meta(4, big), ids, 8), lambda: pm.permute_tokens(None, ids, 8, expert_offset=2 ** 32),
                 lambda: pm.permute_tokens(None, ids, 2 ** 32 + 8), lambda: pm.permute_tokens(None, meta(big, 1, dtype=I32), 8),
                 lambda: pm.permute_workspace_bytes(big, 1, 8), lambda: pm.permute_tokens_backward(meta(8, big), row, 2),
                 lambda: pm.permute_tokens_backward(meta(big, 8), row, 2), lambda: pm.mx_quantize(meta(big)),
                 lambda: pm.mx_quantize(meta(2, big), format="e4m3"),
                 lambda: pm.mx_dequantize(meta(big // 2, dtype=U8), meta(big // 32, dtype=U8)),
                 lambda: pm.mx_grouped_gemm(meta(big, 32, dtype=U8), meta(big, 2, dtype=U8), w, w_sf, off),
                 lambda: pm.mx_grouped_gemm(meta(8, 32, dtype=U8), meta(8, 2, dtype=U8), w, w_sf, off, route_of_row=row, topk=big),
                 lambda: pm.mx_grouped_gemm_backward(meta(big, 32), w, w_sf, off), lambda: pm.mx_activation(meta(big, 64), 1),
                 lambda: pm.mx_activation_backward(meta(big, 32), None, None, 1)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    y8, y8_sf = torch.zeros(4, 64, dtype=U8), torch.zeros(4, 2, dtype=U8)
    for out in ((None, None, y8, None), (None, None, y8, y8_sf)):      # a checkpoint that would not be written
        with pytest.raises(ValueError, match="need checkpoint"):
            pm.mx_activation(torch.zeros(4, 64, dtype=BF), 1, out=out)
