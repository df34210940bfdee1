"""A tuning step around frozen 4-bit experts, put together from the library's calls as a user would:
gate projection -> router front -> layer with adapters -> losses, and back: adapters, routing
weights, router losses, gate. Its gradients are compared with the float64 oracle fed with the
FP32 and BF16 tensors that the GPU's own steps produced, each within its own call's tolerance, so that the
chain's wiring is what is tested."""
import numpy as np
import pytest

import synth
from helpers import bf16_bits, dev, dev_bf16
from oracle import train as ot
from oracle.formats import bf16_to_f32

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _np(t):
    import torch
    return bf16_to_f32(bf16_bits(t)).astype(np.float64) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("name", ["tiny", "swiglu"])
def test_tuning_step(name):
    import torch
    import precision_moe_amd as pm
    w = synth.WORKLOADS[name]
    T, H, E, K, n, R = w.T, w.H, w.E, w.K, 3, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    P = pm.prepare_weights(*synth.all_weights(w, device="cuda"))
    x = dev_bf16(synth.activations(w))
    gate = torch.randn(E, H, generator=g, device="cuda") * H ** -0.5
    down = (torch.randn(n, R, H, generator=g, device="cuda") * H ** -0.5).bfloat16()
    up = (torch.randn(n, H, R, generator=g, device="cuda") * 0.1).bfloat16()
    scale = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    dout = torch.randn(T, H, generator=g, device="cuda").bfloat16()      # d loss / d output

    # forward
    logits = x.float() @ gate.t()
    tk, wt = pm.router_topk(logits, K, w.renormalize)
    load = pm.router_balance(logits, tk)
    ws = torch.empty(pm.moe_workspace_bytes(T, K, E, H, w.I, P.act), dtype=torch.uint8, device="cuda")
    layer = pm.moe_forward(x, tk, wt, P, workspace=ws)
    out, v = pm.adapter_forward(x, ids, down, up, scale, base=layer)
    # backward
    view = pm.workspace_views(ws, T, K, E, H, w.I, P.act)
    z, row = view["z"].view(torch.bfloat16), view["row_of_route"]
    dw, _ = pm.finalize_backward(dout, z, row, wt, need_d_z=False)
    c_b, c_z = torch.full((1,), 0.01, device="cuda"), torch.full((1,), 0.001, device="cuda")
    dl = pm.router_backward(logits, tk, counts=load.counts, tokens=load.tokens, d_balance=c_b, d_z=c_z,
                            d_topk_w=dw, renormalize=w.renormalize)
    dx, d_down, d_up = pm.adapter_backward(dout, x, v, ids, down, up, scale)
    d_gate = dl.t() @ x.float()
    torch.cuda.synchronize()

    lg, tki = _np(logits), tk.cpu().numpy()
    counts, tokens, prob, balance, zl = ot.router_balance(lg, tki)
    assert np.array_equal(load.counts.cpu().numpy(), counts) and int(load.tokens) == T
    np.testing.assert_allclose(_np(load.balance), balance, rtol=(148 + T / 16) * U)
    want_w, _, size_w = ot.finalize_backward(_np(dout), _np(z), row.cpu().numpy(), _np(wt))
    assert np.all(np.abs(_np(dw) - want_w) <= (H / 64 + 16) * U * size_w)
    want_l, size_l = ot.router_backward(lg, tki, counts, tokens, [0.01], [0.001], _np(dw), w.renormalize)
    # 0.01 and 0.001 are not FP32 values: one rounding more
    assert np.all(np.abs(_np(dl) - want_l) <= 66 * U * size_l)
    ida = ids.cpu().numpy()
    want_out, want_v = ot.adapter_forward(_np(x), ida, _np(down), _np(up), _np(scale), _np(layer))
    size_out, size_v = ot.adapter_forward(*(np.abs(a) if a is not ida else a for a in
                                            (_np(x), ida, _np(down), _np(up), _np(scale))))
    extra = (788 * U + 2.0 ** -16) * size_out
    assert np.all(np.abs(_np(out) - want_out) <= 2.0 ** -8 * (np.abs(want_out) + extra) + extra)
    args = (_np(dout), _np(x), _np(v), ida, _np(down), _np(up), _np(scale))
    want = ot.adapter_backward(*args)
    size = ot.adapter_backward(*(a if a is ida else np.abs(a) for a in args))
    extra = (788 * U + 2.0 ** -16) * size[0]
    assert np.all(np.abs(_np(dx) - want[0]) <= 2.0 ** -8 * (np.abs(want[0]) + extra) + extra)
    for got, i in ((d_down, 1), (d_up, 2)):
        assert np.all(np.abs(_np(got) - want[i]) <= (T + 544) * U * size[i])
    assert torch.isfinite(d_gate).all() and d_gate.abs().max() > 0
