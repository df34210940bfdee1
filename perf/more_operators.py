"""Workloads of the operators of an MXFP4 expert layer: tokens sorted by expert and back, the
microscaled formats, the grouped product with its gradient, and the activation with its 8-bit
checkpoint.

A case is one call of one operator ("op"):

  permute         the routes sorted by expert, and each route's token copied to its row
  permute_grad    gradient of the tokens: the sum of their rows' gradients
  quantize        rows to a microscaled format, and read back
  product         rows sorted by expert (or gathered from tokens) times their expert's matrix
  product_grad    gradient of the rows of such a product
  activation      squared ReLU or SwiGLU of a product's rows, quantized for the next product;
                  with "train", the checkpoint is kept and the gradient taken from it

A microscaled block is 32 values along a row with one power of two, 2^(floor(log2 amax) - emax),
and elements rounded to nearest even and saturated: E2M1 (emax 2, largest 6) or E4M3 (emax 8,
largest 448). `run` computes the operators in elementary torch operations, or, with `own` set, by
the calls of precision_moe_amd; `exact` computes the definitions in 64 bits, one expert, slot or
block row at a time. Codes are returned as the values that they stand for.
"""
import math

import torch

own = False

BLOCK = 32


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 61 requests: latency alone counts
        dict(name="permute_decode", op="permute", T=61, E=64, K=6, H=4096, ranks=1),
        # a prompt batch at the widest layer, every expert on this rank
        dict(name="permute_prefill", op="permute", T=4096, E=256, K=8, H=7168, ranks=1),
        # backward of a training batch on one of four ranks: most routes have no row here
        dict(name="permute_grad_share", op="permute_grad", T=4095, E=96, K=6, H=7168, ranks=4),
        # activations of a small decode step
        dict(name="quantize_decode", op="quantize", rows=16, n=7168, fmt="e2m1", dtype="bfloat16"),
        # a refresh of expert matrices from FP32 masters
        dict(name="quantize_weights", op="quantize", rows=65536, n=4096, fmt="e2m1", dtype="float32"),
        # one decode step: a few tokens meet most experts, whose weights are read once
        dict(name="product_decode", op="product", T=16, E=64, K=6, N=4096, Kd=4096, ranks=1, gather=True),
        # a small uneven batch on odd widths, rows already sorted
        dict(name="product_ragged", op="product", T=1100, E=32, K=4, N=1552, Kd=2080, ranks=1, gather=False),
        # a long prompt batch
        dict(name="product_prefill", op="product", T=8192, E=64, K=6, N=4096, Kd=4096, ranks=1, gather=True),
        # gradient of a small uneven batch on one of four ranks
        dict(name="product_grad_share", op="product_grad", T=777, E=16, K=4, N=1536, Kd=2048, ranks=4),
        # gradient of a training batch
        dict(name="product_grad_batch", op="product_grad", T=4096, E=64, K=6, N=4096, Kd=4096, ranks=1),
        # the activation of one decode step
        dict(name="activation_decode", op="activation", rows=96, I=2048, act="swiglu", limit=0.0, train=False),
        # the activation of a training batch, forward and backward
        dict(name="activation_train", op="activation", rows=32763, I=2048, act="swiglu", limit=7.0, train=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["permute", "permute_grad", "quantize", "product", "product_grad", "activation"])
    if op == "quantize":
        n = 32 * _log_int(rng, 1, 512)
        return dict(op=op, rows=_log_int(rng, 1, 65536 * 4096 // n), n=n, fmt=rng.choice(["e2m1", "e4m3"]),
                    dtype=rng.choice(["bfloat16", "float32"]))
    if op == "activation":
        I = 32 * _log_int(rng, 4, 256)
        act = rng.choice(["swiglu", "relu2"])
        return dict(op=op, rows=_log_int(rng, 1, 32763 * 2048 // I), I=I, act=act,
                    limit=rng.choice([0.0, 7.0]) if act == "swiglu" else 0.0, train=rng.random() < 0.5)
    E, ranks = _log_int(rng, 4, 256), rng.choice([1, 1, 4])
    K = rng.randint(1, min(8, E))
    if op in ("permute", "permute_grad"):
        H = 16 * _log_int(rng, 16, 448)
        return dict(op=op, T=_log_int(rng, 1, min(65536, 4096 * 8 * 7168 // (K * H))), E=E, K=K, H=H, ranks=ranks)
    N, Kd = 16 * _log_int(rng, 16, 448), 32 * _log_int(rng, 8, 224)
    E = min(E, 64 * 4096 * 4096 // (N * Kd))
    K = min(K, E)
    rows = 8192 * 6 if op == "product" else 4096 * 6
    case = dict(op=op, T=_log_int(rng, 1, min(8192, rows * 4096 * 4096 // (K * N * Kd))), E=E, K=K, N=N, Kd=Kd,
                ranks=ranks)
    if op == "product":
        case["gather"] = rng.random() < 0.5
    return case


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _ids(case, g):
    """Top-k experts of a router over all ranks' experts, some asked for more often: int32 [T, K]."""
    total = case["E"] * case["ranks"]
    logits = _normal(g, case["T"], total) + _normal(g, total, std=0.5)
    return torch.topk(logits, case["K"], dim=1).indices.to(torch.int32).contiguous()


def _sorted(case, ids):
    """Routes of this rank's experts in expert order: (row_of_route, route_of_row, offsets, valid rows)."""
    E, total = case["E"], ids.numel()
    local = ids.reshape(-1).long() - case["E"] * (case["ranks"] // 2)      # this rank: the middle one
    key = torch.where((local >= 0) & (local < E), local, E)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)])
    place = torch.arange(total, device=ids.device)
    row = torch.empty_like(order).scatter_(0, order, place)
    valid = place < offsets[E]
    row = torch.where(key < E, row, -1)
    return row.to(torch.int32), torch.where(valid, order, -1).to(torch.int32), offsets.to(torch.int32), valid


def _matrices(case, g):
    """Quantized expert matrices [E, N, Kd], one expert at a time."""
    E, N, Kd = case["E"], case["N"], case["Kd"]
    codes = torch.empty(E, N, Kd // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, Kd // BLOCK, dtype=torch.uint8, device="cuda")
    for e in range(E):
        codes[e], scales[e] = _pack(_normal(g, N, Kd, std=Kd ** -0.5))
    return codes, scales


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    bf16 = torch.bfloat16
    if op == "quantize":
        x = _normal(g, case["rows"], case["n"])
        spread = torch.exp(_normal(g, case["rows"], 1))                    # rows of unlike size
        return dict(case=case, x=(x * spread).to(getattr(torch, case["dtype"])))
    if op == "activation":
        R, I = case["rows"], case["I"]
        st = dict(case=case, y=_normal(g, R, 2 * I if case["act"] == "swiglu" else I, std=2.0, dtype=bf16))
        if case["train"]:
            st["dh"] = _normal(g, R, I, std=1e-2, dtype=bf16)
        return st
    ids = _ids(case, g)
    T, K = case["T"], case["K"]
    row, route, offsets, _ = _sorted(case, ids)
    if op == "permute":
        H, i32 = case["H"], dict(dtype=torch.int32, device="cuda")
        return dict(case=case, ids=ids, x=_normal(g, T, H, dtype=bf16),    # buffers that a program keeps
                    out=(torch.zeros(T * K, H, dtype=bf16, device="cuda"), torch.empty(T * K, **i32),
                         torch.full((T * K,), -1, **i32), torch.empty(case["E"] + 1, **i32)))
    if op == "permute_grad":
        return dict(case=case, row=row, d_rows=_normal(g, T * K, case["H"], std=1e-2, dtype=bf16))
    st = dict(case=case, offsets=offsets, route=route, most=max(1, int((offsets[1:] - offsets[:-1]).max())))
    st["w"], st["w_sf"] = _matrices(case, g)
    if op == "product":
        gather = case["gather"]
        st["a"], st["a_sf"] = _pack(_normal(g, T if gather else T * K, case["Kd"]))
        st["out"] = torch.zeros(T * K, case["N"], dtype=bf16, device="cuda")
    else:
        st["dy"] = _normal(g, T * K, case["N"], std=1e-2, dtype=bf16)
        st["out"] = torch.zeros(T * K, case["Kd"], dtype=bf16, device="cuda")
    return st


# ----------------------------------------------------------------------------- microscaled formats
def _power(s):
    """2^s in the 32-bit type, s whole and in [-126, 127]."""
    return ((s + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(x, fmt):
    """(|elements|, exponent of each block) of the rows x in format fmt, in the type of x."""
    emax, top = (2, 6.0) if fmt == "e2m1" else (8, 448.0)
    b = x.reshape(-1, BLOCK)
    amax = b.abs().amax(1, keepdim=True)
    s = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - emax, 0).clamp(-126, 127)
    a = b.abs() * _power(-s).to(x.dtype)
    if fmt == "e2m1":
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    else:
        step = _power((torch.frexp(a).exponent - 1).clamp(min=-6) - 3).to(x.dtype)
    return (torch.round(a / step) * step).clamp(max=top), s


def _rounded(x, fmt):
    """The values that the rows x stand for in format fmt, in 32 bits."""
    a, s = _blocks(x, fmt)
    return torch.copysign(a.float() * _power(s), x.reshape(-1, BLOCK).float()).reshape(x.shape)


def _pack(x):
    """E2M1 codes [..., n/2] (element 2i in the low four bits) and exponents [..., n/32] of x."""
    a, s = _blocks(x, "e2m1")
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(x.reshape(-1, BLOCK)).to(torch.uint8)).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] + 16 * code[..., 1], (s + 127).to(torch.uint8).reshape(*x.shape[:-1], -1)


def _unpack(codes, scales):
    """The values of packed E2M1 rows, in 32 bits."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    v = v.reshape(*scales.shape, BLOCK) * _power(scales.int() - 127)[..., None]
    return v.reshape(*codes.shape[:-1], -1)


# ----------------------------------------------------------------------------- plain forms
def _plain_permute(st):
    case = st["case"]
    row, route, offsets, valid = _sorted(case, st["ids"])
    rows = torch.where(valid[:, None], st["x"][(route // case["K"]).clamp(min=0).long()], 0)
    return dict(rows=rows, row_of_route=row, route_of_row=route, offsets=offsets)


def _plain_permute_grad(st):
    K = st["case"]["K"]
    row = st["row"].reshape(-1, K)
    d = st["d_rows"].float()[row.clamp(min=0).long()]
    return torch.where((row >= 0)[:, :, None], d, 0.0).sum(1).to(torch.bfloat16)


def _plain_quantize(st):
    return _rounded(st["x"].float(), st["case"]["fmt"]).to(torch.bfloat16)


def _by_expert(st, rows):
    """Where each sorted row stands among [E, most] places (the last place: rows of no expert)."""
    E, most = st["case"]["E"], st["most"]
    r = torch.arange(rows, device="cuda")
    e = torch.searchsorted(st["offsets"][1:].contiguous(), r.to(torch.int32), right=True)
    valid = e < E
    e = e.clamp(max=E - 1)
    return torch.where(valid, e * most + r - st["offsets"][e], E * most), valid


def _products(st, rows, matrices):
    """Each sorted row of `rows` times its expert's matrix; zero for rows of no expert."""
    E, most = st["case"]["E"], st["most"]
    place, valid = _by_expert(st, rows.shape[0])
    padded = rows.new_zeros(E * most + 1, rows.shape[1])
    padded[place] = torch.where(valid[:, None], rows, 0.0)
    y = torch.bmm(padded[:-1].reshape(E, most, -1), matrices).reshape(E * most, -1)
    return torch.where(valid[:, None], y[place.clamp(max=E * most - 1)], 0.0).to(torch.bfloat16)


def _plain_product(st):
    a = _unpack(st["a"], st["a_sf"])
    if st["case"]["gather"]:
        a = a[(st["route"] // st["case"]["K"]).clamp(min=0).long()]
    return _products(st, a, _unpack(st["w"], st["w_sf"]).transpose(1, 2))


def _plain_product_grad(st):
    return _products(st, st["dy"].float(), _unpack(st["w"], st["w_sf"]))


def _halves(y, case):
    """Gate and up, clamped, and where the clamp lets a gradient through."""
    g, u = y[:, :case["I"]], y[:, case["I"]:]
    L = case["limit"]
    if L == 0.0:
        return g, u, 1.0, 1.0
    return g.clamp(max=L), u.clamp(-L, L), (g <= L).to(y.dtype), (u.abs() <= L).to(y.dtype)


def _plain_activation(st):
    case = st["case"]
    y = st["y"].double()                              # an element next to a border goes to its own side
    if case["act"] == "swiglu":
        g, u, _, _ = _halves(y, case)
        h = g / (1 + torch.exp(-g)) * u
    else:
        h = y.clamp(min=0) ** 2
    out = dict(h=_rounded(h, "e2m1").to(torch.bfloat16))
    if case["train"]:
        y, dh = _rounded(st["y"].float(), "e4m3"), st["dh"].float()      # the checkpoint, read back
        if case["act"] == "swiglu":
            g, u, in_g, in_u = _halves(y, case)
            s = 1 / (1 + torch.exp(-g))
            dy = torch.cat([dh * u * s * (1 + g * (1 - s)) * in_g, dh * g * s * in_u], 1)
        else:
            dy = 2 * y.clamp(min=0) * dh
        out["dy"] = dy.to(torch.bfloat16)
    return out


# ----------------------------------------------------------------------------- the framework's calls
def _own(st):
    import precision_moe_amd as pm
    case, op = st["case"], st["case"]["op"]
    if op == "permute":
        rows, row, route, offsets = pm.permute_tokens(st["x"], st["ids"], case["E"], out=st["out"],
                                                      expert_offset=case["E"] * (case["ranks"] // 2))
        return dict(rows=rows, row_of_route=row, route_of_row=route, offsets=offsets)
    if op == "permute_grad":
        return pm.permute_tokens_backward(st["d_rows"], st["row"], case["K"])
    if op == "quantize":
        return pm.mx_dequantize(*pm.mx_quantize(st["x"], format=case["fmt"]), format=case["fmt"])
    if op == "product":
        gather = dict(route_of_row=st["route"], topk=case["K"]) if case["gather"] else {}
        return pm.mx_grouped_gemm(st["a"], st["a_sf"], st["w"], st["w_sf"], st["offsets"], out=st["out"], **gather)
    if op == "product_grad":
        return pm.mx_grouped_gemm_backward(st["dy"], st["w"], st["w_sf"], st["offsets"], out=st["out"])
    act = pm.ACT_SWIGLU if case["act"] == "swiglu" else pm.ACT_RELU2
    hq, h_sf, y8, y8_sf = pm.mx_activation(st["y"], act, swiglu_limit=case["limit"], checkpoint=case["train"])
    out = dict(h=pm.mx_dequantize(hq, h_sf))
    if case["train"]:
        out["dy"] = pm.mx_activation_backward(st["dh"], y8, y8_sf, act, swiglu_limit=case["limit"])
    return out


def run(state):
    if own:
        return _own(state)
    return dict(permute=_plain_permute, permute_grad=_plain_permute_grad, quantize=_plain_quantize,
                product=_plain_product, product_grad=_plain_product_grad,
                activation=_plain_activation)[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "quantize":
        size = 2 if case["dtype"] == "bfloat16" else 4
        kept = (0.5 if case["fmt"] == "e2m1" else 1.0) + 1 / BLOCK
        n = case["rows"] * case["n"]
        return dict(bytes=n * (size + 2 * kept + 2), flops=3 * n)       # written, read back
    if op == "activation":
        n = case["rows"] * case["I"]
        wide = 2 if case["act"] == "swiglu" else 1
        moved = 2 * wide + 2 * (0.5 + 1 / BLOCK) + 2
        if case["train"]:                              # checkpoint out and in, dh in, dy out
            moved += 2 * wide * (1 + 1 / BLOCK) + 2 + 2 * wide
        return dict(bytes=n * moved, flops=n * (30 if case["train"] else 12))
    T, K, E = case["T"], case["K"], case["E"]
    R = T * K / case["ranks"]                          # routes that have a row here
    if op == "permute":
        return dict(bytes=2 * case["H"] * (min(T, R) + R) + 12 * T * K, flops=4 * T * K)
    if op == "permute_grad":
        return dict(bytes=2 * case["H"] * (R + T) + 4 * T * K, flops=R * case["H"])
    N, Kd = case["N"], case["Kd"]
    used = E * (1 - (1 - 1 / E) ** R)                  # experts that have a row
    weights = used * N * Kd * (0.5 + 1 / BLOCK)
    if op == "product":
        rows = min(T, R) if case["gather"] else R
        return dict(bytes=weights + rows * Kd * (0.5 + 1 / BLOCK) + 2 * R * N, flops=2 * R * N * Kd)
    return dict(bytes=weights + 2 * R * (N + Kd), flops=2 * R * N * Kd)


# ----------------------------------------------------------------------------- 64 bits
def _exact_power(e):
    """2^e in 64 bits, e whole (in 64 bits): its exponent field, as a library's power may be an ulp off."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_element(a, fmt):
    """The nearest element to each a >= 0 (64 bits), ties to the even code, by counting the borders below it."""
    if fmt == "e2m1":
        grid = [0, .5, 1, 1.5, 2, 3, 4, 6]
    else:
        grid = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1]
    grid = torch.tensor(grid, dtype=torch.float64, device=a.device)
    borders = (grid[1:] + grid[:-1]) / 2
    low, high = torch.searchsorted(borders, a.contiguous()), torch.searchsorted(borders, a.contiguous(), right=True)
    return grid[torch.where(low % 2 == 0, low, high)]  # on a border, low = high - 1


def _exact_rounded(x, fmt):
    """x (64 bits) in format fmt, 4096 rows at a time."""
    emax = 2 if fmt == "e2m1" else 8
    out = torch.empty_like(x)
    for part, to in zip(x.split(4096), out.split(4096)):
        b = part.reshape(-1, BLOCK)
        amax = b.abs().amax(1, keepdim=True)
        e = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
        e = torch.where(_exact_power(e) > amax, e - 1, torch.where(_exact_power(e + 1) <= amax, e + 1, e))
        scale = torch.where(amax > 0, _exact_power(e - emax), 1.0)
        to.copy_((_exact_element(b.abs() / scale, fmt) * scale * torch.sign(b)).reshape(part.shape))
    return out


def _exact_matrix(codes, scales):
    """One packed matrix in 64 bits."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    v = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    for half, c in enumerate((codes & 15, codes >> 4)):
        v[:, half::2] = grid[(c & 7).long()] * (1 - 2 * (c >> 3).double())
    return v * _exact_power(scales.double() - 127).repeat_interleave(BLOCK, 1)


def _exact_products(st):
    case = st["case"]
    grad = case["op"] == "product_grad"
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    cuts = st["offsets"].tolist()
    for e in range(case["E"]):
        rows = torch.arange(cuts[e], cuts[e + 1], device="cuda")
        if not len(rows):
            continue
        m = _exact_matrix(st["w"][e], st["w_sf"][e])
        if grad:
            out[rows] = st["dy"][rows].double() @ m
        else:
            at = st["route"][rows].long() // case["K"] if case["gather"] else rows
            out[rows] = _exact_matrix(st["a"][at], st["a_sf"][at]) @ m.t()
    return out


def _exact_activation(st):
    case = st["case"]
    I, L, swiglu = case["I"], case["limit"] or math.inf, case["act"] == "swiglu"
    y = st["y"].double()
    if swiglu:
        gate = torch.minimum(y[:, :I], y.new_tensor(L))
        up = torch.maximum(torch.minimum(y[:, I:], y.new_tensor(L)), y.new_tensor(-L))
        h = gate * torch.sigmoid(gate) * up
    else:
        h = torch.relu(y).square()
    out = dict(h=_exact_rounded(h, "e2m1"))
    if not case["train"]:
        return out
    y, dh = _exact_rounded(y, "e4m3"), st["dh"].double()
    if not swiglu:
        return dict(out, dy=dh * 2 * torch.relu(y))
    gate, up = y[:, :I], y[:, I:]
    inside, between = gate <= L, (up <= L) & (up >= -L)
    gate = torch.where(inside, gate, L)
    up = torch.where(between, up, torch.sign(up) * min(L, 1e300))
    sig = torch.sigmoid(gate)
    slope = sig + gate * sig * torch.sigmoid(-gate)
    return dict(out, dy=torch.cat([torch.where(inside, dh * up * slope, 0.0),
                                   torch.where(between, dh * gate * sig, 0.0)], 1))


def exact(case, seed):
    op = case["op"]
    if op == "permute":                                # nothing is computed but places
        return None
    st = prepare(case, seed)
    if op == "quantize":
        return _exact_rounded(st["x"].double(), case["fmt"])
    if op == "activation":
        return _exact_activation(st)
    if op == "permute_grad":
        row, d = st["row"].reshape(case["T"], case["K"]).long(), st["d_rows"].double()
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        for j in range(case["K"]):
            on = row[:, j] >= 0
            out[on] += d[row[on, j]]
        return out
    return _exact_products(st)
