"""precision_moe_amd -- per-token NVFP4 routed-MoE expert path on AMD MI355X (gfx950).

Thin Python binding over the C ABI of libpmoe.so (include/pmoe.h): every
function here only marshals torch tensors (device memory) and the current HIP
stream into the C calls; all computation runs in the library's HIP kernels.
The library is loaded on first use and its absence raises an error -- there
is no fallback implementation.
"""
import ctypes
import os
from collections import namedtuple
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
# PMOE_LIB may point at another build of the same library (e.g. a tuning variant).
LIB_PATH = os.environ.get("PMOE_LIB") or os.path.join(_HERE, "_lib", "libpmoe.so")

ACT_RELU2, ACT_SWIGLU = 0, 1
IDS_INT32, IDS_INT64 = 0, 1
RECIPE_PER_TOKEN, RECIPE_PER_TENSOR, RECIPE_W4A16 = 0, 1, 2
FINALIZE_ORDERED, FINALIZE_FUSED = 0, 1
MX_E2M1, MX_E4M3 = 0, 1
_MX_FORMATS = {"e2m1": MX_E2M1, "e4m3": MX_E4M3}
_RECIPES = {"per_token": RECIPE_PER_TOKEN, "per_tensor": RECIPE_PER_TENSOR, "w4a16": RECIPE_W4A16}
_FINALIZE = {"ordered": FINALIZE_ORDERED, "fused": FINALIZE_FUSED}
WS_FIELDS = ("row_of_route", "route_of_row", "expert_offsets", "counters", "h", "hq", "h_sf",
             "h_scale", "z")

_c_size_p = ctypes.POINTER(ctypes.c_size_t)
_vp = ctypes.c_void_p
_i = ctypes.c_int


class MoeOptions(ctypes.Structure):
    """pmoe_moe_options (include/pmoe.h)."""
    _fields_ = [("recipe", ctypes.c_int), ("finalize", ctypes.c_int),
                ("swiglu_limit", ctypes.c_float), ("a2_scale", ctypes.c_void_p),
                ("streams", ctypes.c_int), ("a1_scale", ctypes.c_void_p),
                ("step_events", ctypes.c_void_p)]
STEP_EVENTS = 8
_SIGNATURES = {
    "pmoe_version": (_i, []),
    "pmoe_last_error": (ctypes.c_char_p, []),
    "pmoe_weight_bytes": (_i, [_i, _i, _i, _i, _c_size_p]),
    "pmoe_prepare_workspace_bytes": (ctypes.c_size_t, [_i, _i, _i, _i]),
    "pmoe_prepare_weights": (_i, [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  ctypes.c_size_t, _vp]),
    "pmoe_quantize_input_per_token": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp]),
    "pmoe_quantize_rows_f32": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp]),
    "pmoe_moe_workspace_bytes": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i]),
    "pmoe_moe_workspace_layout": (_i, [_i, _i, _i, _i, _i, _i, _c_size_p]),
    "pmoe_routed_moe": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp,
                             _vp, _vp, _vp, _vp, _i, _vp, ctypes.c_size_t, _vp, _vp]),
    "pmoe_routed_moe_static": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                    _vp, _vp, _vp, _vp, _i, _vp, _vp]),
    "pmoe_routed_moe_steps": (_i, [_i, _i, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _i,
                                   _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, ctypes.c_size_t, _vp, _vp]),
    "pmoe_finalize": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp]),
    "pmoe_prepare_weights_per_tensor": (_i, [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                             _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "pmoe_quantize_input_per_tensor": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp]),
    "pmoe_routed_moe_per_tensor": (_i, [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                        _vp, _vp, _vp, _vp, _vp, _i, _vp, ctypes.c_size_t, _vp, _vp]),
    "pmoe_routed_moe_w4a16": (_i, [_vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _i, _vp, ctypes.c_size_t, _vp, _vp]),
    "pmoe_routed_moe_ex": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                _vp, _vp, _vp, _vp, _i, ctypes.POINTER(MoeOptions), _vp,
                                ctypes.c_size_t, _vp, _vp]),
    "pmoe_router_topk": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp]),
    "pmoe_moe_forward": (_i, [_vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                              _vp, _i, ctypes.POINTER(MoeOptions), _vp, ctypes.c_size_t, _vp, _vp]),
    "pmoe_router_balance_workspace_bytes": (ctypes.c_size_t, [_i, _i, _i, _i]),
    "pmoe_router_balance": (_i, [_vp, _vp, _i, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                 ctypes.c_size_t, _vp]),
    "pmoe_router_backward": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp]),
    "pmoe_finalize_backward": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp]),
    "pmoe_adapter_workspace_bytes": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i]),
    "pmoe_adapter_forward": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  ctypes.c_size_t, _vp]),
    "pmoe_adapter_backward": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "pmoe_permute_workspace_bytes": (ctypes.c_size_t, [_i, _i, _i]),
    "pmoe_permute_tokens": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                 _vp]),
    "pmoe_permute_tokens_backward": (_i, [_vp, _i, _vp, _i, _i, _i, _i, _vp, _vp]),
    "pmoe_mx_quantize": (_i, [_vp, _i, _i, ctypes.c_longlong, _i, _vp, _vp, _vp]),
    "pmoe_mx_dequantize": (_i, [_vp, _vp, _i, ctypes.c_longlong, _i, _i, _vp, _vp]),
    "pmoe_mx_grouped_gemm": (_i, [_vp, _vp, _i, _vp, _i, _vp, _i, _i, _vp, _vp, _i, _i, _vp, _i, _vp]),
    "pmoe_mx_grouped_gemm_backward": (_i, [_vp, _vp, _i, _i, _vp, _vp, _i, _i, _vp, _vp]),
    "pmoe_mx_activation": (_i, [_vp, _i, _i, _i, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp]),
    "pmoe_mx_activation_backward": (_i, [_vp, _vp, _vp, _i, _i, _i, ctypes.c_float, _vp, _vp, _vp]),
}
STEP_ROUTE, STEP_FC1, STEP_REQUANT, STEP_FC2, STEP_FINALIZE = range(5)

_lib = None


class PmoeError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"pmoe error {code}: {message}")
        self.code = code


def lib():
    """Load libpmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with precision_moe_amd.build.build()")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _check(rc):
    if rc != 0:
        raise PmoeError(rc, lib().pmoe_last_error().decode())


def _ptr(t):
    return t.data_ptr() if t is not None else None      # ctypes turns an int or None into void*


def _stream(stream=None, *tensors):
    """The hipStream_t to enqueue on. A `stream` other than torch's current one first
    waits for the current stream (the inputs and the temporaries made here were produced
    there), and every tensor the call touches is recorded as used on `stream`, so the
    caching allocator does not hand its memory out again before that work is done."""
    import torch
    if stream is None:      # the raw handle alone: a quarter of the cost of a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    cur = torch.cuda.current_stream()
    if stream == cur:
        return ctypes.c_void_p(cur.cuda_stream)
    stream.wait_stream(cur)
    for t in tensors:
        if t is not None and torch.is_tensor(t) and t.is_cuda:
            t.record_stream(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _event_array(events):
    """ctypes array of the raw hipEvent_t handles of STEP_EVENTS torch.cuda.Events (or None)."""
    import torch
    if events is None:
        return None
    if len(events) != STEP_EVENTS:
        raise ValueError(f"step_events needs {STEP_EVENTS} events")
    handles = []
    for ev in events:
        if ev is None:
            handles.append(None)
            continue
        if ev.cuda_event == 0:          # torch creates the event on its first record
            ev.record(torch.cuda.current_stream())
        handles.append(ev.cuda_event)
    return (ctypes.c_void_p * STEP_EVENTS)(*handles)


def _bf16_storage(t):
    import torch
    if t.element_size() != 2:
        raise TypeError("expected a 2-byte (BF16) tensor")
    return t


# ----------------------------------------------------------------------------- weights
@dataclass
class PreparedWeights:
    """Prepared NVFP4 expert weights (layout in include/pmoe.h), all on one device."""
    E: int
    N1: int
    H: int
    I: int
    w1_codes: object
    w1_scales: object
    w1_alpha: object
    w2_codes: object
    w2_scales: object
    w2_alpha: object

    @property
    def act(self):
        return ACT_SWIGLU if self.N1 == 2 * self.I else ACT_RELU2


def weight_bytes(E, N1, H, I):
    sizes = (ctypes.c_size_t * 4)()
    _check(lib().pmoe_weight_bytes(E, N1, H, I, sizes))
    return tuple(int(s) for s in sizes)


def empty_weights(E, N1, H, I, device):
    import torch
    b = weight_bytes(E, N1, H, I)
    u8 = dict(dtype=torch.uint8, device=device)
    f32 = dict(dtype=torch.float32, device=device)
    return PreparedWeights(E, N1, H, I, torch.empty(b[0], **u8), torch.empty(b[1], **u8),
                           torch.empty(E, **f32), torch.empty(b[2], **u8), torch.empty(b[3], **u8),
                           torch.empty(E, **f32))


def prepare_weights(w1, w2, out=None, workspace=None, stream=None, input_scales=None):
    """BF16 FC1 [E, N1, H] and FC2 [E, H, I] -> PreparedWeights (in place into `out` if given).

    input_scales = (a1, a2), device float32 scalars, selects the per-tensor
    recipe: the static input scales are folded into the alphas.
    """
    import torch
    E, N1, H = w1.shape
    I = w2.shape[2]
    if tuple(w2.shape[:2]) != (E, H):
        raise ValueError("FC2 must be [E, H, I] with FC1's E and H")
    w1, w2 = _bf16_storage(w1.contiguous()), _bf16_storage(w2.contiguous())
    if out is None:
        out = empty_weights(E, N1, H, I, w1.device)
    elif (out.E, out.N1, out.H, out.I) != (E, N1, H, I):
        raise ValueError("`out` was prepared for other shapes")
    need = lib().pmoe_prepare_workspace_bytes(E, N1, H, I)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=w1.device)
    if input_scales is None:
        _check(lib().pmoe_prepare_weights(
            _ptr(w1), _ptr(w2), E, N1, H, I, _ptr(out.w1_codes), _ptr(out.w1_scales),
            _ptr(out.w1_alpha), _ptr(out.w2_codes), _ptr(out.w2_scales), _ptr(out.w2_alpha),
            _ptr(workspace), workspace.numel(), _stream(stream, w1, w2, workspace, out.w1_codes, out.w1_scales,
                                                          out.w1_alpha, out.w2_codes, out.w2_scales,
                                                          out.w2_alpha)))
    else:
        a1, a2 = (_f32_scalar(a) for a in input_scales)
        _check(lib().pmoe_prepare_weights_per_tensor(
            _ptr(w1), _ptr(w2), E, N1, H, I, _ptr(a1), _ptr(a2), _ptr(out.w1_codes),
            _ptr(out.w1_scales), _ptr(out.w1_alpha), _ptr(out.w2_codes), _ptr(out.w2_scales),
            _ptr(out.w2_alpha), _ptr(workspace), workspace.numel(),
            _stream(stream, w1, w2, a1, a2, workspace, out.w1_codes, out.w1_scales, out.w1_alpha,
                    out.w2_codes, out.w2_scales, out.w2_alpha)))
    return out


def _f32_scalar(a):
    import torch
    if not (torch.is_tensor(a) and a.dtype == torch.float32 and a.numel() == 1 and a.is_cuda):
        raise TypeError("static scales are device float32 tensors of one element")
    return a


# ----------------------------------------------------------------------------- quantizers
def quantize_input_per_token(x, out=None, stream=None):
    """BF16 [T, H] -> (xq uint8 [T, H/2], x_sf uint8 [T, H/16], x_scale float32 [T])."""
    import torch
    T, H = x.shape
    x = _bf16_storage(x.contiguous())
    if out is None:
        out = (torch.empty((T, H // 2), dtype=torch.uint8, device=x.device),
               torch.empty((T, H // 16), dtype=torch.uint8, device=x.device),
               torch.empty((T,), dtype=torch.float32, device=x.device))
    xq, xsf, xs = out
    _check(lib().pmoe_quantize_input_per_token(_ptr(x), T, H, _ptr(xq), _ptr(xsf), _ptr(xs),
                                               _stream(stream, x, xq, xsf, xs)))
    return xq, xsf, xs


def quantize_input_per_tensor(x, a1, out=None, stream=None):
    """BF16 [T, H] with a static scale a1 (device float32 scalar) -> (xq [T, H/2], x_sf [T, H/16])."""
    import torch
    T, H = x.shape
    x = _bf16_storage(x.contiguous())
    if out is None:
        out = (torch.empty((T, H // 2), dtype=torch.uint8, device=x.device),
               torch.empty((T, H // 16), dtype=torch.uint8, device=x.device))
    xq, xsf = out
    _check(lib().pmoe_quantize_input_per_tensor(_ptr(x), T, H, _ptr(_f32_scalar(a1)), _ptr(xq),
                                                _ptr(xsf), _stream(stream, x, a1, xq, xsf)))
    return xq, xsf


def quantize_rows_f32(h, out=None, stream=None):
    """float32 [R, L] -> (hq uint8 [R, L/2], h_sf uint8 [R, L/16], h_scale float32 [R])."""
    import torch
    R, L = h.shape
    h = h.contiguous()
    if h.dtype != torch.float32:
        raise TypeError("h must be float32")
    if out is None:
        out = (torch.empty((R, L // 2), dtype=torch.uint8, device=h.device),
               torch.empty((R, L // 16), dtype=torch.uint8, device=h.device),
               torch.empty((R,), dtype=torch.float32, device=h.device))
    hq, hsf, hs = out
    _check(lib().pmoe_quantize_rows_f32(_ptr(h), R, L, _ptr(hq), _ptr(hsf), _ptr(hs),
                                        _stream(stream, h, hq, hsf, hs)))
    return hq, hsf, hs


# ----------------------------------------------------------------------------- routed MoE
def moe_workspace_bytes(T, K, E, H, I, act):
    n = lib().pmoe_moe_workspace_bytes(T, K, E, H, I, act)
    if n == 0:
        _check(lib().pmoe_moe_workspace_layout(T, K, E, H, I, act, (ctypes.c_size_t * 9)()))
    return int(n)


def moe_workspace_layout(T, K, E, H, I, act):
    offs = (ctypes.c_size_t * len(WS_FIELDS))()
    _check(lib().pmoe_moe_workspace_layout(T, K, E, H, I, act, offs))
    return dict(zip(WS_FIELDS, (int(o) for o in offs)))


def workspace_views(ws, T, K, E, H, I, act):
    """Typed views of the routed_moe workspace fields. After moe_forward (ordered finalize) z (BF16
    bits) and row_of_route are what finalize_backward takes, until the workspace is used again; the
    other fields are for inspection in tests."""
    import torch
    off = moe_workspace_layout(T, K, E, H, I, act)
    TK = T * K
    Ip = -(-I // 64) * 64          # the intermediate's rows are padded to whole 64-element chunks

    def view(name, count, dtype):
        nbytes = count * torch.empty((), dtype=dtype).element_size()
        return ws[off[name]:off[name] + nbytes].view(dtype)

    return {
        "row_of_route": view("row_of_route", TK, torch.int32),
        "route_of_row": view("route_of_row", TK, torch.int32),
        "expert_offsets": view("expert_offsets", E + 1, torch.int32),
        "counters": view("counters", 4, torch.int32),
        "h": view("h", TK * I, torch.float32).view(TK, I),
        # W4A16: BF16 h in the same field, rows of Ip (zeros past I)
        "h_bf16": view("h", TK * Ip, torch.int16).view(TK, Ip)[:, :I],
        "hq": view("hq", TK * Ip // 2, torch.uint8).view(TK, Ip // 2)[:, :I // 2],
        "h_sf": view("h_sf", TK * Ip // 16, torch.uint8).view(TK, Ip // 16)[:, :I // 16],
        "hq_padded": view("hq", TK * Ip // 2, torch.uint8).view(TK, Ip // 2),
        "h_sf_padded": view("h_sf", TK * Ip // 16, torch.uint8).view(TK, Ip // 16),
        "h_scale": view("h_scale", TK, torch.float32),
        "z": view("z", TK * H, torch.int16).view(TK, H),
    }


def routed_moe(xq, x_sf, x_scale, topk_ids, topk_w, weights: PreparedWeights, act=None,
               expert_offset=0, workspace=None, out=None, stream=None, steps=None):
    """Routing, FC1 + activation, requantization, FC2 and the fixed-order finalize.

    Returns BF16 [T, H] (as torch.bfloat16 unless `out` is given). `steps`
    = (first, last) runs only that range of the five steps (STEP_*), reusing
    `workspace` and `out` from earlier calls.
    """
    import torch
    T, K = topk_ids.shape
    W = weights
    act = W.act if act is None else act
    if topk_ids.dtype == torch.int32:
        ids_type = IDS_INT32
    elif topk_ids.dtype == torch.int64:
        ids_type = IDS_INT64
    else:
        raise TypeError("topk_ids must be int32 or int64")
    topk_ids = topk_ids.contiguous()
    topk_w = topk_w.contiguous()
    if topk_w.dtype != torch.float32:
        raise TypeError("topk_w must be float32")
    if workspace is None:
        workspace = torch.empty(max(moe_workspace_bytes(T, K, W.E, W.H, W.I, act), 256),
                                dtype=torch.uint8, device=xq.device)
    if out is None:
        out = torch.empty((T, W.H), dtype=torch.bfloat16, device=xq.device)
    first, last = (STEP_ROUTE, STEP_FINALIZE) if steps is None else steps
    _check(lib().pmoe_routed_moe_steps(
        first, last, _ptr(xq), _ptr(x_sf), _ptr(x_scale), _ptr(topk_ids), ids_type, _ptr(topk_w), T, K,
        W.E, W.H, W.I, W.N1, expert_offset, _ptr(W.w1_codes), _ptr(W.w1_scales), _ptr(W.w1_alpha),
        _ptr(W.w2_codes), _ptr(W.w2_scales), _ptr(W.w2_alpha), act, _ptr(workspace),
        workspace.numel(), _ptr(out),
        _stream(stream, xq, x_sf, x_scale, topk_ids, topk_w, workspace, out, W.w1_codes, W.w1_scales, W.w1_alpha, W.w2_codes, W.w2_scales, W.w2_alpha)))
    return out


STATIC_SCRATCH_BYTES = 64 << 20


def routed_moe_static(xq, x_sf, x_scale, topk_ids, topk_w, weights: PreparedWeights, act=None,
                      expert_offset=0, out=None, stream=None):
    """routed_moe on the library's static scratch (pmoe_routed_moe_static): no workspace
    argument and no device allocation inside the call; `out` should be given by callers
    that cannot allocate (else one BF16 [T, H] tensor is allocated here)."""
    import torch
    T, K = topk_ids.shape
    W = weights
    act = W.act if act is None else act
    topk_ids, ids_type, topk_w = _routing_args(topk_ids, topk_w)
    if out is None:
        out = torch.empty((T, W.H), dtype=torch.bfloat16, device=xq.device)
    _check(lib().pmoe_routed_moe_static(
        _ptr(xq), _ptr(x_sf), _ptr(x_scale), _ptr(topk_ids), ids_type, _ptr(topk_w), T, K, W.E, W.H,
        W.I, W.N1, expert_offset, _ptr(W.w1_codes), _ptr(W.w1_scales), _ptr(W.w1_alpha),
        _ptr(W.w2_codes), _ptr(W.w2_scales), _ptr(W.w2_alpha), act, _ptr(out),
        _stream(stream, xq, x_sf, x_scale, topk_ids, topk_w, out, W.w1_codes, W.w1_scales,
                W.w1_alpha, W.w2_codes, W.w2_scales, W.w2_alpha)))
    return out


def _routing_args(topk_ids, topk_w):
    import torch
    if topk_ids.dtype == torch.int32:
        ids_type = IDS_INT32
    elif topk_ids.dtype == torch.int64:
        ids_type = IDS_INT64
    else:
        raise TypeError("topk_ids must be int32 or int64")
    if topk_w.dtype != torch.float32:
        raise TypeError("topk_w must be float32")
    return topk_ids.contiguous(), ids_type, topk_w.contiguous()


def _moe_buffers(T, K, W, act, device, workspace, out):
    import torch
    if workspace is None:
        workspace = torch.empty(max(moe_workspace_bytes(T, K, W.E, W.H, W.I, act), 256),
                                dtype=torch.uint8, device=device)
    if out is None:
        out = torch.empty((T, W.H), dtype=torch.bfloat16, device=device)
    return workspace, out


def routed_moe_per_tensor(xq, x_sf, topk_ids, topk_w, weights: PreparedWeights, a2, act=None,
                          expert_offset=0, workspace=None, out=None, stream=None):
    """Per-tensor NVFP4 recipe: (xq, x_sf) from quantize_input_per_tensor, weights prepared
    with input_scales=(a1, a2), a2 the static FC2 input scale (device float32 scalar)."""
    T, K = topk_ids.shape
    W = weights
    act = W.act if act is None else act
    topk_ids, ids_type, topk_w = _routing_args(topk_ids, topk_w)
    workspace, out = _moe_buffers(T, K, W, act, xq.device, workspace, out)
    _check(lib().pmoe_routed_moe_per_tensor(
        _ptr(xq), _ptr(x_sf), _ptr(topk_ids), ids_type, _ptr(topk_w), T, K, W.E, W.H, W.I, W.N1,
        expert_offset, _ptr(W.w1_codes), _ptr(W.w1_scales), _ptr(W.w1_alpha), _ptr(W.w2_codes),
        _ptr(W.w2_scales), _ptr(W.w2_alpha), _ptr(_f32_scalar(a2)), act, _ptr(workspace),
        workspace.numel(), _ptr(out),
        _stream(stream, xq, x_sf, topk_ids, topk_w, a2, workspace, out, W.w1_codes, W.w1_scales, W.w1_alpha, W.w2_codes, W.w2_scales, W.w2_alpha)))
    return out


def routed_moe_w4a16(x, topk_ids, topk_w, weights: PreparedWeights, act=None, expert_offset=0,
                     workspace=None, out=None, stream=None):
    """W4A16 (weight_only) recipe: BF16 activations x [T, H], NVFP4 weights from prepare_weights."""
    T, K = topk_ids.shape
    W = weights
    act = W.act if act is None else act
    x = _bf16_storage(x.contiguous())
    topk_ids, ids_type, topk_w = _routing_args(topk_ids, topk_w)
    workspace, out = _moe_buffers(T, K, W, act, x.device, workspace, out)
    _check(lib().pmoe_routed_moe_w4a16(
        _ptr(x), _ptr(topk_ids), ids_type, _ptr(topk_w), T, K, W.E, W.H, W.I, W.N1, expert_offset,
        _ptr(W.w1_codes), _ptr(W.w1_scales), _ptr(W.w1_alpha), _ptr(W.w2_codes), _ptr(W.w2_scales),
        _ptr(W.w2_alpha), act, _ptr(workspace), workspace.numel(), _ptr(out),
        _stream(stream, x, topk_ids, topk_w, workspace, out, W.w1_codes, W.w1_scales, W.w1_alpha, W.w2_codes, W.w2_scales, W.w2_alpha)))
    return out


def routed_moe_ex(x, x_sf, x_scale, topk_ids, topk_w, weights: PreparedWeights, recipe="per_token",
                  finalize="ordered", swiglu_limit=0.0, a2=None, act=None, expert_offset=0,
                  workspace=None, out=None, stream=None, streams=0, step_events=None):
    """The routed path with options (pmoe_routed_moe_ex): recipe "per_token" (x = xq, x_sf,
    x_scale), "per_tensor" (x = xq, x_sf; a2) or "w4a16" (x = BF16 activations; x_sf, x_scale
    None); finalize "ordered" or "fused"; swiglu_limit > 0 clamps SwiGLU; step_events: None
    or STEP_EVENTS torch.cuda.Events (timing enabled) recorded around the grouped GEMMs."""
    T, K = topk_ids.shape
    W = weights
    act = W.act if act is None else act
    topk_ids, ids_type, topk_w = _routing_args(topk_ids, topk_w)
    if recipe == "w4a16":
        x = _bf16_storage(x.contiguous())
    workspace, out = _moe_buffers(T, K, W, act, x.device, workspace, out)
    evs = _event_array(step_events)
    opt = MoeOptions(_RECIPES[recipe], _FINALIZE[finalize], float(swiglu_limit),
                     _f32_scalar(a2).data_ptr() if a2 is not None else None, int(streams), None,
                     ctypes.cast(evs, ctypes.c_void_p) if evs is not None else None)
    _check(lib().pmoe_routed_moe_ex(
        _ptr(x), _ptr(x_sf), _ptr(x_scale), _ptr(topk_ids), ids_type, _ptr(topk_w), T, K, W.E, W.H,
        W.I, W.N1, expert_offset, _ptr(W.w1_codes), _ptr(W.w1_scales), _ptr(W.w1_alpha),
        _ptr(W.w2_codes), _ptr(W.w2_scales), _ptr(W.w2_alpha), act, ctypes.byref(opt),
        _ptr(workspace), workspace.numel(), _ptr(out),
        _stream(stream, x, x_sf, x_scale, topk_ids, topk_w, a2, workspace, out, W.w1_codes, W.w1_scales, W.w1_alpha, W.w2_codes, W.w2_scales, W.w2_alpha)))
    return out


def _adapters_beside(x, out, adapters, workspace, need, layer_workspace):
    """Refuses what adapter_forward on x and the layer's `out` would refuse after the layer, and
    adapters that the layer would overwrite: layer_workspace is None or (tensor, bytes it uses)."""
    import torch
    given = {**adapters, "adapter_workspace": workspace} | ({} if out is None else {"out": out})
    for name, t in given.items():
        if t.device != x.device:
            raise ValueError(f"adapters and adapter_ids, out and adapter_workspace must be on the device of x: {name}")
    if x.is_cuda and x.device.index != torch.cuda.current_device():
        raise ValueError("x must be on the current device")
    if workspace.numel() < need:
        raise ValueError("adapter_workspace too small")
    written = [(k, given[k].data_ptr(), n) for k, n in (("out", 2 * x.numel()), ("adapter_workspace", need)) if k in given]
    read = [(k, t.data_ptr(), t.numel() * t.element_size()) for k, t in (("x", x), *adapters.items())]
    for i, (name, at, size) in enumerate(written):
        for other, start, length in written[i + 1:] + read:
            if size and length and at < start + length and start < at + size:
                raise ValueError(f"{name} overlaps {other}, which the adapters use after the layer")
    if layer_workspace is not None:     # it may be the adapters' workspace too, one after the other
        at, size = layer_workspace[0].data_ptr(), layer_workspace[1]
        for other, start, length in read[1:]:
            if length and at < start + length and start < at + size:
                raise ValueError(f"workspace overlaps {other}, which the adapters use after the layer")
    for name, align in (("down", 16), ("up", 16), ("adapter_workspace", 256)):
        if given[name].data_ptr() % align:
            raise ValueError(f"{name} is not {align}-byte aligned")


def moe_forward(x, topk_ids, topk_w, weights: PreparedWeights, recipe="per_token",
                finalize="ordered", swiglu_limit=0.0, a1=None, a2=None, act=None, expert_offset=0,
                workspace=None, out=None, stream=None, streams=0, step_events=None, adapters=None,
                adapter_ids=None, adapter_workspace=None):
    """The whole routed layer from BF16 activations x [T, H] (pmoe_moe_forward): the NVFP4
    recipes quantize x inside the call, overlapped with the routing. step_events: None or
    STEP_EVENTS torch.cuda.Events (timing enabled) recorded around the grouped GEMMs.
    adapters = (down, up, scale) with N = H adds, after the layer, each token's own adapter
    adapter_ids[t] beside it (adapter_forward on x with the layer's BF16 output as its base)."""
    import torch
    T, K = topk_ids.shape
    W = weights
    act = W.act if act is None else act
    x = _bf16_storage(x.contiguous())
    if (adapters is None) != (adapter_ids is None):
        raise ValueError("adapters and adapter_ids are wanted both or neither")
    if adapters is not None:            # refused before the layer is enqueued
        adapter_ids, _, aT, n, aH, aN, R, *adapters = _adapter_args(adapter_ids, *adapters)
        if (aT, aH, aN) != (T, W.H, W.H):
            raise ValueError("adapters of a layer must be [n, R, H] and [n, H, R], adapter_ids [T]")
        _bf16(x, "x", (T, W.H))
        if out is not None:
            _out(out, "out", torch.bfloat16, (T, W.H), x)
        need = adapter_workspace_bytes(T, n, aH, aN, R)
        adapter_workspace = _scratch(need, adapter_workspace, x)
        _adapters_beside(x, out, dict(zip(("adapter_ids", "down", "up", "scale"), (adapter_ids, *adapters))),
                         adapter_workspace, need,
                         None if workspace is None else (workspace, moe_workspace_bytes(T, K, W.E, W.H, W.I, act)))
    topk_ids, ids_type, topk_w = _routing_args(topk_ids, topk_w)
    workspace, out = _moe_buffers(T, K, W, act, x.device, workspace, out)
    evs = _event_array(step_events)
    opt = MoeOptions(_RECIPES[recipe], _FINALIZE[finalize], float(swiglu_limit),
                     _f32_scalar(a2).data_ptr() if a2 is not None else None, int(streams),
                     _f32_scalar(a1).data_ptr() if a1 is not None else None,
                     ctypes.cast(evs, ctypes.c_void_p) if evs is not None else None)
    _check(lib().pmoe_moe_forward(
        _ptr(x), _ptr(topk_ids), ids_type, _ptr(topk_w), T, K, W.E, W.H, W.I, W.N1, expert_offset,
        _ptr(W.w1_codes), _ptr(W.w1_scales), _ptr(W.w1_alpha), _ptr(W.w2_codes), _ptr(W.w2_scales),
        _ptr(W.w2_alpha), act, ctypes.byref(opt), _ptr(workspace), workspace.numel(), _ptr(out),
        _stream(stream, x, topk_ids, topk_w, a1, a2, workspace, out, W.w1_codes, W.w1_scales, W.w1_alpha, W.w2_codes, W.w2_scales, W.w2_alpha)))
    if adapters is not None:
        adapter_forward(x, adapter_ids, *adapters, base=out, out=out, need_v=False,
                        workspace=adapter_workspace, stream=stream)
    return out


def router_topk(logits, k, renormalize=False, out=None, stream=None):
    """FP32 logits [T, E] -> (topk_ids int32 [T, k], topk_w float32 [T, k])."""
    import torch
    T, E = logits.shape
    if logits.dtype != torch.float32:
        raise TypeError("logits must be float32")
    logits = logits.contiguous()
    if out is None:
        out = (torch.empty((T, k), dtype=torch.int32, device=logits.device),
               torch.empty((T, k), dtype=torch.float32, device=logits.device))
    ids, w = out
    _check(lib().pmoe_router_topk(_ptr(logits), T, E, k, int(bool(renormalize)), _ptr(ids), _ptr(w),
                                  _stream(stream, logits, ids, w)))
    return ids, w


def finalize(z, row_of_route, topk_w, out=None, stream=None):
    """Fixed-order finalize: z BF16 [R, H], row_of_route int32 [T*K], topk_w float32 [T, K]."""
    import torch
    T, K = topk_w.shape
    H = z.shape[1]
    z = _bf16_storage(z.contiguous())
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=z.device)
    row_of_route = row_of_route.contiguous()
    topk_w = topk_w.contiguous()
    _check(lib().pmoe_finalize(_ptr(z), _ptr(row_of_route), _ptr(topk_w), T, K, H, _ptr(out),
                               _stream(stream, z, row_of_route, topk_w, out)))
    return out


# ----------------------------------------------------------------------------- router, training side
RouterBalance = namedtuple("RouterBalance", "counts tokens prob balance z")


def _is(t, name, dtype, shape):
    """Checks the dtype and shape of a device tensor argument and returns it contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}".replace("torch.", ""))
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.contiguous()


def _out(t, name, dtype, shape, like):
    """An output: allocated on the device of `like` if None, else checked (it is written in place)."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _is(t, name, dtype, shape)


def _ids(t, name):
    import torch
    if t.dtype is torch.int32:
        return t.contiguous(), IDS_INT32
    if t.dtype is torch.int64:
        return t.contiguous(), IDS_INT64
    raise TypeError(f"{name} must be int32 or int64")


def _scratch(need, workspace, like):
    import torch
    if workspace is None:
        return like.new_empty((max(need, 256),), dtype=torch.uint8)
    return workspace


def _sequences(seq_offsets):
    import torch
    if seq_offsets is None:
        return None, 1
    if seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
        raise ValueError("seq_offsets must be a vector of S + 1 offsets")
    return _is(seq_offsets, "seq_offsets", torch.int32, seq_offsets.shape), seq_offsets.numel() - 1


def _router_args(logits, topk_ids):
    import torch
    if logits.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError("logits must be [T, E] and topk_ids [T, K]")
    T, E = logits.shape
    K = topk_ids.shape[1]
    if topk_ids.shape[0] != T:
        raise ValueError("logits and topk_ids must have the same number of tokens")
    ids, ids_type = _ids(topk_ids, "topk_ids")
    return _is(logits, "logits", torch.float32, (T, E)), ids, ids_type, T, K, E


def router_balance_workspace_bytes(T, K, E, S=1):
    size = lib().pmoe_router_balance_workspace_bytes(T, E, K, S)
    if size == 0:
        raise PmoeError(3, lib().pmoe_last_error().decode())
    return int(size)


def router_balance(logits, topk_ids, seq_offsets=None, out=None, workspace=None, stream=None):
    """Expert counts, balance loss and z-loss of each sequence (pmoe_router_balance).

    logits float32 [T, E], topk_ids [T, K] (ids outside [0, E) are no routes), seq_offsets
    int32 [S+1] on the device or None for one sequence. Returns RouterBalance(counts int32
    [S, E], tokens int32 [S], prob float32 [S, E], balance float32 [S], z float32 [S])."""
    import torch
    logits, ids, ids_type, T, K, E = _router_args(logits, topk_ids)
    off, S = _sequences(seq_offsets)
    i32, f32 = torch.int32, torch.float32
    counts, tokens, prob, balance, z = out if out is not None else (None,) * 5
    res = RouterBalance(_out(counts, "counts", i32, (S, E), logits), _out(tokens, "tokens", i32, (S,), logits),
                        _out(prob, "prob", f32, (S, E), logits), _out(balance, "balance", f32, (S,), logits),
                        _out(z, "z", f32, (S,), logits))
    ws = _scratch(lib().pmoe_router_balance_workspace_bytes(T, E, K, S), workspace, logits)
    _check(lib().pmoe_router_balance(
        _ptr(logits), _ptr(ids), ids_type, T, K, E, _ptr(off), S, *(_ptr(t) for t in res), _ptr(ws),
        ws.numel(), _stream(stream, logits, ids, off, ws, *res)))
    return res


def router_backward(logits, topk_ids, counts=None, tokens=None, d_balance=None, d_z=None, d_topk_w=None,
                    renormalize=False, seq_offsets=None, out=None, stream=None):
    """Gradient of the logits (pmoe_router_backward), float32 [T, E]: from the losses of
    router_balance (d_balance, d_z float32 [S], with its counts and tokens) and from the
    weights of router_topk (d_topk_w float32 [T, K]); at least one of the three. With renormalize
    the weights are those over the slots whose id is an expert's: a slot that was dropped after
    router_topk keeps its id here and gets a zero d_topk_w."""
    import torch
    logits, ids, ids_type, T, K, E = _router_args(logits, topk_ids)
    off, S = _sequences(seq_offsets)
    f32, i32 = torch.float32, torch.int32
    out = _out(out, "out", f32, (T, E), logits)
    opt = [None if t is None else _is(t, name, dt, shape)
           for t, name, dt, shape in ((counts, "counts", i32, (S, E)), (tokens, "tokens", i32, (S,)),
                                      (d_balance, "d_balance", f32, (S,)), (d_z, "d_z", f32, (S,)),
                                      (d_topk_w, "d_topk_w", f32, (T, K)))]
    _check(lib().pmoe_router_backward(
        _ptr(logits), _ptr(ids), ids_type, T, K, E, int(bool(renormalize)), _ptr(off), S,
        *(_ptr(t) for t in opt), _ptr(out), _stream(stream, logits, ids, off, out, *opt)))
    return out


def finalize_backward(dout, z, row_of_route, topk_w, need_d_topk_w=True, need_d_z=True, out=None,
                      stream=None):
    """Gradients of finalize (pmoe_finalize_backward): (d_topk_w float32 [T, K], d_z BF16 [R, H])
    from dout BF16 [T, H], z BF16 [R, H], row_of_route int32 [T*K] and topk_w float32 [T, K]; None
    in the place of one that is not needed. A fresh d_z is not initialised in rows that no route
    names. out = (d_topk_w, d_z), either of them None, is written in place."""
    import torch
    T, K = topk_w.shape
    R, H = z.shape
    dout = _bf16(dout, "dout", (T, H))
    z = _bf16(z, "z", (R, H))
    row = _is(row_of_route.reshape(-1), "row_of_route", torch.int32, (T * K,))
    topk_w = _is(topk_w, "topk_w", torch.float32, (T, K))
    given = out if out is not None else (None, None)
    dw = _out(given[0], "d_topk_w", torch.float32, (T, K), z) if need_d_topk_w else None
    dz = _out(given[1], "d_z", torch.bfloat16, (R, H), z) if need_d_z else None
    _check(lib().pmoe_finalize_backward(
        _ptr(dout), _ptr(z), _ptr(row), _ptr(topk_w), T, K, H, R, _ptr(dw), _ptr(dz),
        _stream(stream, dout, z, row, topk_w, dw, dz)))
    return dw, dz


# ----------------------------------------------------------------------------- adapters
def _bf16(t, name, shape):
    import torch
    return _is(t, name, torch.bfloat16, shape)


def _adapter_args(adapter_ids, down, up, scale):
    import torch
    if down.dim() != 3 or up.dim() != 3 or adapter_ids.dim() != 1:
        raise ValueError("adapter_ids must be [T], down [n, R, H] and up [n, N, R]")
    n, R, H = down.shape
    N = up.shape[1]
    ids, ids_type = _ids(adapter_ids, "adapter_ids")
    return (ids, ids_type, ids.shape[0], n, H, N, R, _bf16(down, "down", (n, R, H)),
            _bf16(up, "up", (n, N, R)), _is(scale, "scale", torch.float32, (n,)))


def adapter_workspace_bytes(T, n, H, N, R, backward=False):
    size = lib().pmoe_adapter_workspace_bytes(T, n, H, N, R, int(bool(backward)))
    if size == 0:
        raise PmoeError(3, lib().pmoe_last_error().decode())
    return int(size)


def adapter_forward(x, adapter_ids, down, up, scale, base=None, out=None, v=None, need_v=True,
                    workspace=None, stream=None):
    """Low-rank adapters of many requests (pmoe_adapter_forward): token t of x BF16 [T, H] uses
    adapter adapter_ids[t] (int32 or int64, outside [0, n): none) of down BF16 [n, R, H], up BF16
    [n, N, R] and scale float32 [n]. Returns (out, v): out BF16 [T, N] = base + scale * up(v), v
    float32 [T, R] = down(x), which adapter_backward wants (None with need_v False). base None
    means zeros; out may be base."""
    import torch
    ids, ids_type, T, n, H, N, R, down, up, scale = _adapter_args(adapter_ids, down, up, scale)
    x = _bf16(x, "x", (T, H))
    if base is not None:
        base = _bf16(base, "base", (T, N))
    out = _out(out, "out", torch.bfloat16, (T, N), x)
    v = _out(v, "v", torch.float32, (T, R), x) if need_v else None
    ws = _scratch(lib().pmoe_adapter_workspace_bytes(T, n, H, N, R, 0), workspace, x)
    _check(lib().pmoe_adapter_forward(
        _ptr(x), _ptr(ids), ids_type, T, n, H, N, R, _ptr(down), _ptr(up), _ptr(scale), _ptr(base),
        _ptr(out), _ptr(v), _ptr(ws), ws.numel(), _stream(stream, x, ids, down, up, scale, base, out, v, ws)))
    return out, v


def adapter_backward(dy, x, v, adapter_ids, down, up, scale, base=None, need_dx=True, need_weights=True,
                     out=None, workspace=None, stream=None):
    """Gradients of adapter_forward (pmoe_adapter_backward) for the gradient dy BF16 [T, N] of out:
    (dx BF16 [T, H] = base + down^T(scale * up^T(dy)), d_down float32 [n, R, H], d_up float32
    [n, N, R]), None in the place of what is not needed. base BF16 [T, H] is the gradient that dx
    adds to (None: zeros); out = (dx, d_down, d_up), any of them None, is written in place and
    its dx may be base."""
    import torch
    ids, ids_type, T, n, H, N, R, down, up, scale = _adapter_args(adapter_ids, down, up, scale)
    dy = _bf16(dy, "dy", (T, N))
    x = _bf16(x, "x", (T, H)) if need_weights else None
    v = _is(v, "v", torch.float32, (T, R)) if need_weights else None
    if base is not None:
        base = _bf16(base, "base", (T, H))
    dx, d_down, d_up = out if out is not None else (None, None, None)
    dx = _out(dx, "dx", torch.bfloat16, (T, H), dy) if need_dx else None
    d_down = _out(d_down, "d_down", torch.float32, (n, R, H), dy) if need_weights else None
    d_up = _out(d_up, "d_up", torch.float32, (n, N, R), dy) if need_weights else None
    ws = _scratch(lib().pmoe_adapter_workspace_bytes(T, n, H, N, R, 1), workspace, dy)
    _check(lib().pmoe_adapter_backward(
        _ptr(dy), _ptr(x), _ptr(v), _ptr(ids), ids_type, T, n, H, N, R, _ptr(down), _ptr(up), _ptr(scale),
        _ptr(base), _ptr(dx), _ptr(d_down), _ptr(d_up), _ptr(ws), ws.numel(),
        _stream(stream, dy, x, v, ids, down, up, scale, base, dx, d_down, d_up, ws)))
    return dx, d_down, d_up


# ----------------------------------------------------------------------------- tokens sorted by expert
PermutedTokens = namedtuple("PermutedTokens", "rows row_of_route route_of_row expert_offsets")


def _type(dtype, name):
    """PMOE_BF16 or PMOE_F32."""
    import torch
    if dtype is torch.bfloat16:
        return 0
    if dtype is torch.float32:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float32")


def _c_ints(*values):
    """Refuses what the C interface's int would cut."""
    if max(values) > 0x7FFFFFFF or min(values) < -0x80000000:
        raise ValueError(f"sizes and offsets must fit 32 bits: {values}")


def permute_workspace_bytes(T, K, E):
    _c_ints(T, K, E)
    size = lib().pmoe_permute_workspace_bytes(T, K, E)
    if size == 0:
        raise PmoeError(3, lib().pmoe_last_error().decode())
    return int(size)


def permute_tokens(x, topk_ids, E, expert_offset=0, out=None, workspace=None, stream=None):
    """Routes sorted by expert, and each token copied to its routes' rows (pmoe_permute_tokens).

    x [T, H], of any type whose rows are a multiple of 16 bytes, or None for the order alone;
    topk_ids [T, K] int32 or int64, ids outside [expert_offset, expert_offset + E) have no row.
    Returns PermutedTokens(rows [T*K, H] or None, row_of_route int32 [T*K] (-1: no row), route_of_row
    int32 [T*K], expert_offsets int32 [E+1]); rows and route_of_row behind row expert_offsets[E]
    are left as they were, in fresh tensors uninitialised. out, a PermutedTokens or 4-tuple, any of
    its entries None, is written in place."""
    import torch
    if topk_ids.dim() != 2 or (x is not None and (x.dim() != 2 or x.shape[0] != topk_ids.shape[0])):
        raise ValueError("topk_ids must be [T, K] and x [T, H]")
    T, K = topk_ids.shape
    row_bytes = 0 if x is None else x.shape[1] * x.element_size()
    _c_ints(T, K, E, expert_offset, row_bytes)
    ids, ids_type = _ids(topk_ids, "topk_ids")
    rows, row, route, offsets = out if out is not None else (None,) * 4
    if x is not None:
        x = x.contiguous()
        rows = _out(rows, "rows", x.dtype, (T * K, x.shape[1]), x)
    elif rows is not None:
        raise ValueError("rows needs x")
    i32 = torch.int32
    res = PermutedTokens(rows, _out(row, "row_of_route", i32, (T * K,), ids),
                         _out(route, "route_of_row", i32, (T * K,), ids),
                         _out(offsets, "expert_offsets", i32, (E + 1,), ids))
    ws = _scratch(lib().pmoe_permute_workspace_bytes(T, K, E), workspace, ids)
    _check(lib().pmoe_permute_tokens(
        _ptr(ids), ids_type, T, K, E, expert_offset, _ptr(x), row_bytes,
        *(_ptr(t) for t in res), _ptr(ws), ws.numel(), _stream(stream, ids, x, ws, *res)))
    return res


def permute_tokens_backward(d_rows, row_of_route, K, out=None, stream=None):
    """Gradient of permute_tokens (pmoe_permute_tokens_backward): dx [T, H], the FP32 sum of d_rows
    [R, H] (BF16 or FP32, dx too) over the K slots of each token; row_of_route int32 [T*K], values
    outside [0, R) are no rows."""
    import torch
    if d_rows.dim() != 2 or K < 1 or row_of_route.numel() % K:
        raise ValueError("d_rows must be [R, H] and row_of_route [T*K]")
    R, H = d_rows.shape
    T = row_of_route.numel() // K
    _c_ints(T, K, R, H)
    kind = _type(d_rows.dtype, "d_rows")
    d_rows = d_rows.contiguous()
    row = _is(row_of_route.reshape(-1), "row_of_route", torch.int32, (T * K,))
    out = _out(out, "out", d_rows.dtype, (T, H), d_rows)
    _check(lib().pmoe_permute_tokens_backward(_ptr(d_rows), kind, _ptr(row), T, K, R, H, _ptr(out),
                                              _stream(stream, d_rows, row, out)))
    return out


# ----------------------------------------------------------------------------- microscaled formats
def _mx_format(format):
    if format not in _MX_FORMATS:
        raise ValueError("format must be 'e2m1' or 'e4m3'")
    return _MX_FORMATS[format]


def _mx_pair(codes, scales, name, shape, fmt=MX_E2M1):
    """Codes and scales of a tensor of `shape`, checked."""
    import torch
    *lead, n = shape
    per = 2 if fmt == MX_E2M1 else 1
    return (_is(codes, f"codes of {name}", torch.uint8, (*lead, n // per)),
            _is(scales, f"scales of {name}", torch.uint8, (*lead, n // 32)))


def mx_quantize(x, format="e2m1", out=None, stream=None):
    """Microscaled quantization (pmoe_mx_quantize) of x BF16 or FP32 [..., n], n a multiple of 32:
    (codes uint8 [..., n/2] packed E2M1 or [..., n] E4M3, scales uint8 [..., n/32], E8M0)."""
    import torch
    fmt, kind = _mx_format(format), _type(x.dtype, "x")
    if x.dim() < 1 or x.shape[-1] % 32:
        raise ValueError("the last dimension of x must be a multiple of 32")
    _c_ints(x.shape[-1])
    x = x.contiguous()
    *lead, n = x.shape
    codes, scales = out if out is not None else (None, None)
    codes = _out(codes, "codes", torch.uint8, (*lead, n // 2 if fmt == MX_E2M1 else n), x)
    scales = _out(scales, "scales", torch.uint8, (*lead, n // 32), x)
    _check(lib().pmoe_mx_quantize(_ptr(x), kind, fmt, x.numel() // n if n else 0, n, _ptr(codes), _ptr(scales),
                                  _stream(stream, x, codes, scales)))
    return codes, scales


def mx_dequantize(codes, scales, format="e2m1", dtype=None, out=None, stream=None):
    """The values of microscaled codes and scales (pmoe_mx_dequantize), BF16 unless dtype is
    torch.float32."""
    import torch
    fmt = _mx_format(format)
    dtype = torch.bfloat16 if dtype is None else dtype
    kind = _type(dtype, "dtype")
    if codes.dim() < 1:
        raise ValueError("codes must be [..., n/2] (E4M3: [..., n])")
    n = codes.shape[-1] * (2 if fmt == MX_E2M1 else 1)
    _c_ints(n)
    shape = (*codes.shape[:-1], n)
    codes, scales = _mx_pair(codes, scales, "the input", shape, fmt)
    out = _out(out, "out", dtype, shape, codes)
    _check(lib().pmoe_mx_dequantize(_ptr(codes), _ptr(scales), fmt, out.numel() // n if n else 0, n, kind, _ptr(out),
                                    _stream(stream, codes, scales, out)))
    return out


def _mx_matrices(w, w_sf, expert_offsets):
    """(w, w_sf, offsets, E, N, Kd) of quantized expert matrices [E, N, Kd], checked."""
    import torch
    if w.dim() != 3:
        raise ValueError("w must be [E, N, Kd/2]")
    E, N, Kd = w.shape[0], w.shape[1], 2 * w.shape[2]
    w, w_sf = _mx_pair(w, w_sf, "w", (E, N, Kd))
    return w, w_sf, _is(expert_offsets, "expert_offsets", torch.int32, (E + 1,)), E, N, Kd


def mx_grouped_gemm(a, a_sf, w, w_sf, expert_offsets, route_of_row=None, topk=1, dtype=None, out=None, stream=None):
    """Grouped product of MXFP4 rows with MXFP4 expert matrices (pmoe_mx_grouped_gemm): out [R, N] BF16
    (or dtype torch.float32), row r of expert e (expert_offsets int32 [E+1]) times w[e].

    a uint8 [rows, Kd/2], a_sf uint8 [rows, Kd/32]: the rows themselves (R = rows), or, with
    route_of_row int32 [R] and topk, tokens, of which row r reads number route_of_row[r] // topk.
    w uint8 [E, N, Kd/2], w_sf uint8 [E, N, Kd/32], as mx_quantize gives them. Rows of no expert are
    left as they were (in a fresh out uninitialised)."""
    import torch
    w, w_sf, offsets, E, N, Kd = _mx_matrices(w, w_sf, expert_offsets)
    if a.dim() != 2:
        raise ValueError("a must be [rows, Kd/2]")
    a, a_sf = _mx_pair(a, a_sf, "a", (a.shape[0], Kd))
    if route_of_row is None:
        route, R = None, a.shape[0]
    else:
        route = _is(route_of_row, "route_of_row", torch.int32, (route_of_row.numel(),))
        R = route.shape[0]
    _c_ints(a.shape[0], topk, R, E, N, Kd)
    dtype = (out.dtype if out is not None else torch.bfloat16) if dtype is None else dtype
    kind = _type(dtype, "out")
    out = _out(out, "out", dtype, (R, N), a)
    _check(lib().pmoe_mx_grouped_gemm(
        _ptr(a), _ptr(a_sf), a.shape[0], _ptr(route), topk, _ptr(offsets), R, E, _ptr(w), _ptr(w_sf), N, Kd, _ptr(out),
        kind, _stream(stream, a, a_sf, route, offsets, w, w_sf, out)))
    return out


def mx_grouped_gemm_backward(dy, w, w_sf, expert_offsets, out=None, stream=None):
    """Gradient of the rows of mx_grouped_gemm (pmoe_mx_grouped_gemm_backward): dx BF16 [R, Kd] from dy
    BF16 [R, N]; rows of no expert are left as they were. For the tokens of a gathered product:
    permute_tokens_backward of dx."""
    import torch
    w, w_sf, offsets, E, N, Kd = _mx_matrices(w, w_sf, expert_offsets)
    if dy.dim() != 2:
        raise ValueError("dy must be [R, N]")
    R = dy.shape[0]
    _c_ints(R, E, N, Kd)
    dy = _bf16(dy, "dy", (R, N))
    out = _out(out, "out", torch.bfloat16, (R, Kd), dy)
    _check(lib().pmoe_mx_grouped_gemm_backward(_ptr(dy), _ptr(offsets), R, E, _ptr(w), _ptr(w_sf), N, Kd, _ptr(out),
                                               _stream(stream, dy, offsets, w, w_sf, out)))
    return out


def _row_count(t):
    import torch
    return None if t is None else _is(t.reshape(-1), "row_count", torch.int32, (1,))


def mx_activation(y, act, swiglu_limit=0.0, checkpoint=False, row_count=None, out=None, stream=None):
    """Squared ReLU or SwiGLU of y BF16 [R, I] (SwiGLU: [R, 2I], gate then up) into MXFP4, with an 8-bit
    checkpoint of y (pmoe_mx_activation): (hq uint8 [R, I/2], h_sf uint8 [R, I/32], y8 uint8 as y (E4M3),
    y8_sf uint8 [R, .../32]); the last two are None without `checkpoint`. row_count: a device int32
    (expert_offsets[-1:], say), only rows below it are read and written. out = (hq, h_sf, y8, y8_sf),
    any of them None, is written in place."""
    import torch
    if y.dim() != 2:
        raise ValueError("y must be [R, I] or [R, 2I]")
    R, W = y.shape
    if act == ACT_SWIGLU and W % 2:
        raise ValueError("SwiGLU needs y [R, 2I]")
    _c_ints(R, W)
    I = W // 2 if act == ACT_SWIGLU else W
    y = _bf16(y, "y", (R, W))
    count = _row_count(row_count)
    hq, h_sf, y8, y8_sf = out if out is not None else (None,) * 4
    if not checkpoint and (y8 is not None or y8_sf is not None):
        raise ValueError("y8 and y8_sf need checkpoint")
    u8 = torch.uint8
    hq, h_sf = _out(hq, "hq", u8, (R, I // 2), y), _out(h_sf, "h_sf", u8, (R, I // 32), y)
    y8 = _out(y8, "y8", u8, (R, W), y) if checkpoint else None
    y8_sf = _out(y8_sf, "y8_sf", u8, (R, W // 32), y) if checkpoint else None
    _check(lib().pmoe_mx_activation(_ptr(y), R, I, act, float(swiglu_limit), _ptr(count), _ptr(hq), _ptr(h_sf),
                                    _ptr(y8), _ptr(y8_sf), _stream(stream, y, count, hq, h_sf, y8, y8_sf)))
    return hq, h_sf, y8, y8_sf


def mx_activation_backward(dh, y8, y8_sf, act, swiglu_limit=0.0, row_count=None, out=None, stream=None):
    """Gradient dy BF16 [R, I or 2I] of mx_activation from dh BF16 [R, I] and the checkpoint
    (pmoe_mx_activation_backward)."""
    import torch
    if dh.dim() != 2:
        raise ValueError("dh must be [R, I]")
    R, I = dh.shape
    W = 2 * I if act == ACT_SWIGLU else I
    _c_ints(R, W)
    dh = _bf16(dh, "dh", (R, I))
    y8, y8_sf = _mx_pair(y8, y8_sf, "the checkpoint", (R, W), MX_E4M3)
    count = _row_count(row_count)
    out = _out(out, "out", torch.bfloat16, (R, W), dh)
    _check(lib().pmoe_mx_activation_backward(_ptr(dh), _ptr(y8), _ptr(y8_sf), R, I, act, float(swiglu_limit),
                                             _ptr(count), _ptr(out), _stream(stream, dh, y8, y8_sf, count, out)))
    return out
