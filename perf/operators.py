"""Workloads of the operators around the frozen experts: the router's balance loss and
gradient, the gradient of the finalize, and low-rank adapters of many requests.

A case is one call of one operator ("op"):

  balance        expert counts, probability sums, balance loss and z-loss of each sequence
  router_grad    gradient of the logits from both losses and from the top-k weights
  finalize_grad  gradients of the routing weights and of the expert outputs
  adapter        out = base + scale * up(down(x)), the adapter chosen by each token
  adapter_grad   gradients of an adapter call: of its input and of both matrices

`run` computes them in elementary torch operations in 32 bits, or, with `own`
set, by the calls of precision_moe_amd; `exact` computes the definitions in
64 bits, one sequence, one slot or one adapter at a time.
"""
import math

import torch

own = False

INF = float("inf")


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # expert load of one decode step: latency alone counts
        dict(name="balance_decode", op="balance", T=64, E=64, K=6, S=1, pad=False, masked=False),
        # one training micro-batch, the loss over the whole batch
        dict(name="balance_batch", op="balance", T=4096, E=256, K=8, S=1, pad=False, masked=False),
        # packed sequences of unequal length with padding and disabled experts, a loss for each
        dict(name="balance_ragged", op="balance", T=32749, E=96, K=6, S=61, pad=True, masked=True),
        # gradient of a small micro-batch, renormalized weights
        dict(name="router_grad_step", op="router_grad", T=1024, E=64, K=6, S=1, renorm=True,
             pad=False, masked=False),
        # gradient of a long packed batch
        dict(name="router_grad_long", op="router_grad", T=65521, E=256, K=8, S=16, renorm=False,
             pad=True, masked=False),
        # gradient of the finalize in a small layer, a quarter of the routes on other ranks
        dict(name="finalize_grad_small", op="finalize_grad", T=256, H=2048, K=4, dropped=True),
        # gradient of the finalize at the widest layer and batch
        dict(name="finalize_grad_wide", op="finalize_grad", T=4096, H=7168, K=8, dropped=False),
        # a decode step of few requests, each with its own adapter
        dict(name="adapter_decode", op="adapter", T=16, n=16, H=4096, N=4096, R=16, runs=False),
        # a decode step of many requests that share 64 adapters
        dict(name="adapter_decode_many", op="adapter", T=257, n=64, H=7168, N=7168, R=32, runs=False),
        # prompts of a few requests, each a run of tokens
        dict(name="adapter_prefill", op="adapter", T=8192, n=6, H=7168, N=7168, R=16, runs=True),
        # training of small adapters on odd widths and an odd batch
        dict(name="adapter_grad_odd", op="adapter_grad", T=1100, n=6, H=2064, N=2688, R=8, runs=True),
        # training of large adapters at the widest layer
        dict(name="adapter_grad_wide", op="adapter_grad", T=4096, n=4, H=7168, N=7168, R=64, runs=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "router_grad", "finalize_grad", "adapter", "adapter_grad"])
    if op in ("balance", "router_grad"):
        T, E = _log_int(rng, 1, 65000), _log_int(rng, 4, 256)
        case = dict(op=op, T=T, E=E, K=rng.randint(1, min(8, E)), S=min(T, _log_int(rng, 1, 64)),
                    pad=rng.random() < 0.5, masked=rng.random() < 0.5)
        if op == "router_grad":
            case["renorm"] = rng.random() < 0.5
        return case
    H = 16 * _log_int(rng, 16, 448)
    if op == "finalize_grad":
        K = rng.randint(1, 8)
        T = _log_int(rng, 1, min(4096, 4096 * 8 * 7168 // (K * H)))
        return dict(op=op, T=T, H=H, K=K, dropped=rng.random() < 0.5)
    return dict(op=op, T=_log_int(rng, 1, 8192 if op == "adapter" else 4096), n=_log_int(rng, 1, 64), H=H,
                N=16 * _log_int(rng, 16, 448), R=rng.choice([8, 16, 32, 64]), runs=rng.random() < 0.5)


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _cuts(g, total, parts):
    """parts + 1 ascending offsets from 0 to total; parts may be empty."""
    inner = (_uniform(g, parts - 1) * total).to(torch.int32).sort().values
    ends = torch.tensor([0, total], dtype=torch.int32, device="cuda")
    return torch.cat([ends[:1], inner, ends[1:]])


def _prepare_router(case, g):
    T, E, K, S = case["T"], case["E"], case["K"], case["S"]
    hot = _normal(g, E, std=0.5)                      # some experts are asked for more often
    logits = _normal(g, T, E, std=1.5) + hot
    if case["masked"]:                                # experts that are switched off for a token
        off = _uniform(g, T, E) < 0.1
        off[:, :K] = False
        logits = logits.masked_fill(off, -INF)
    top, ids = torch.topk(logits, K, dim=1)
    ids = ids.to(torch.int32)
    if case["pad"]:                                   # padding tokens and slots without an expert
        ids[_uniform(g, T) < 0.1] = -1
        ids[_uniform(g, T, K) < 0.02] = -1
    st = dict(case=case, logits=logits.contiguous(), ids=ids.contiguous(), offsets=_cuts(g, T, S))
    if case["op"] == "router_grad":
        active, p, _, seq = _probabilities(st["logits"], st["ids"], st["offsets"])
        st["counts"], st["tokens"], _ = _sums(st, active, p, seq)
        st["d_balance"], st["d_z"] = _normal(g, S, std=1e-2), _normal(g, S, std=1e-3)
        st["d_w"] = _normal(g, T, K, std=1.0 / T)
    return st


def _prepare_finalize(case, g):
    T, H, K = case["T"], case["H"], case["K"]
    R = max(1, T * K * 3 // 4) if case["dropped"] else T * K
    routes = torch.randperm(T * K, generator=g, device="cuda").to(torch.int32)
    routes = torch.where(routes < R, routes, -1)      # routes of other ranks' experts have no row
    return dict(case=case, dout=_normal(g, T, H, std=1e-2, dtype=torch.bfloat16),
                z=_normal(g, R, H, dtype=torch.bfloat16), row=routes.contiguous(),
                w=torch.softmax(_normal(g, T, K), 1).contiguous())


def _adapter_ids(case, g):
    T, n = case["T"], case["n"]
    if not case["runs"]:
        ids = (_uniform(g, T) * n).to(torch.int32)
        ids[_uniform(g, T) < 0.1] = -1                # requests without an adapter
        return ids
    cuts = _cuts(g, T, min(T, n + 1))                 # one run for each adapter and one without
    run = torch.searchsorted(cuts[1:-1].contiguous(), torch.arange(T, device="cuda", dtype=torch.int32),
                             right=True)
    who = torch.randperm(n + 1, generator=g, device="cuda") - 1
    return who[run].to(torch.int32)


def _prepare_adapter(case, g):
    T, n, H, N, R = (case[k] for k in ("T", "n", "H", "N", "R"))
    bf16 = torch.bfloat16
    st = dict(case=case, x=_normal(g, T, H, dtype=bf16), ids=_adapter_ids(case, g),
              down=_normal(g, n, R, H, std=H ** -0.5, dtype=bf16),
              up=_normal(g, n, N, R, std=R ** -0.5, dtype=bf16), scale=0.5 + 1.5 * _uniform(g, n))
    if case["op"] == "adapter":
        st["base"] = _normal(g, T, N, dtype=bf16)     # the shared projection's output
    else:
        st["dy"] = _normal(g, T, N, std=1e-2, dtype=bf16)
        st["base"] = _normal(g, T, H, std=1e-2, dtype=bf16)   # the shared projection's gradient
        st["v"] = _low(st, torch.float32)             # kept by the forward call
    return st


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("balance", "router_grad"):
        return _prepare_router(case, g)
    if case["op"] == "finalize_grad":
        return _prepare_finalize(case, g)
    return _prepare_adapter(case, g)


# ----------------------------------------------------------------------------- plain forms
def _probabilities(logits, ids, offsets):
    """Active tokens, softmax rows (0 where inactive), log-sum-exp and the sequence of each token."""
    T, E = logits.shape
    m = logits.max(1, keepdim=True).values
    active = ((ids >= 0) & (ids < E)).any(1) & (m[:, 0] > -INF)
    m = torch.where(m > -INF, m, 0.0)
    ex = torch.exp(logits - m)
    den = ex.sum(1, keepdim=True)
    p = torch.where(active[:, None], ex / den, 0.0)
    lse = torch.where(active, m[:, 0] + torch.log(den[:, 0]), 0.0)
    seq = torch.searchsorted(offsets[1:-1].contiguous(),
                             torch.arange(T, device=logits.device, dtype=torch.int32), right=True)
    return active, p, lse, seq


def _sums(st, active, p, seq):
    """Routes per expert, active tokens and probability sums of each sequence."""
    E, S = st["case"]["E"], st["case"]["S"]
    ids = st["ids"].long()
    valid = (ids >= 0) & (ids < E) & active[:, None]
    slot = torch.where(valid, seq[:, None] * E + ids, S * E).reshape(-1)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=p.device)
    counts.index_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))
    tokens = torch.zeros(S, dtype=torch.int32, device=p.device)
    tokens.index_add_(0, seq, active.to(torch.int32))
    member = (seq[None, :] == torch.arange(S, device=p.device)[:, None]).to(p.dtype)
    return counts[:-1].reshape(S, E), tokens, member @ p


def _plain_balance(st):
    E, K = st["case"]["E"], st["case"]["K"]
    active, p, lse, seq = _probabilities(st["logits"], st["ids"], st["offsets"])
    counts, tokens, prob = _sums(st, active, p, seq)
    n = tokens.clamp(min=1).float()
    balance = E / K * (counts.float() * prob).sum(1) / (n * n)
    member = (seq[None, :] == torch.arange(st["case"]["S"], device=p.device)[:, None]).float()
    return dict(counts=counts, tokens=tokens, prob=prob, balance=balance, z=member @ (lse * lse) / n)


def _plain_router_grad(st):
    E, K = st["case"]["E"], st["case"]["K"]
    active, p, lse, seq = _probabilities(st["logits"], st["ids"], st["offsets"])
    n = st["tokens"].clamp(min=1).float()
    f = st["counts"].float() / (n * K)[:, None]
    fp = (f[seq] * p).sum(1, keepdim=True)
    g = (st["d_balance"] * E / n)[seq][:, None] * p * (f[seq] - fp)
    g = g + (2 * st["d_z"] / n)[seq][:, None] * lse[:, None] * p
    valid = (st["ids"] >= 0) & (st["ids"] < E) & active[:, None]
    ids = torch.where(valid, st["ids"], 0).long()
    dw = torch.where(valid, st["d_w"], 0.0)
    pj = torch.where(valid, torch.gather(p, 1, ids), 0.0)
    if st["case"]["renorm"]:
        q = pj / pj.sum(1, keepdim=True).clamp(min=1e-37)
        return g.scatter_add(1, ids, q * (dw - (dw * q).sum(1, keepdim=True)))
    direct = torch.zeros_like(p).scatter_add(1, ids, dw)
    return g + p * (direct - (dw * pj).sum(1, keepdim=True))


def _plain_finalize_grad(st):
    K = st["case"]["K"]
    row = st["row"].reshape(-1, K).long()
    valid = row >= 0
    R, H = st["z"].shape
    z = st["z"].float()[torch.where(valid, row, 0)]
    d = st["dout"].float()[:, None, :]
    dw = torch.where(valid, (z * d).sum(2), 0.0)
    dz = torch.empty(R + 1, H, dtype=torch.bfloat16, device=z.device)
    dz[torch.where(valid, row, R)] = (st["w"][:, :, None] * d).to(torch.bfloat16)
    return dict(d_topk_w=dw, d_z=dz[:R])


def _chosen(st, dtype):
    """[T, n, 1]: 1 where the token uses the adapter."""
    return (st["ids"][:, None] == torch.arange(st["case"]["n"], device="cuda")).to(dtype)[:, :, None]


def _low(st, dtype):
    """down(x) of each token's own adapter, [T, R]."""
    T, n, R = st["case"]["T"], st["case"]["n"], st["case"]["R"]
    every = st["x"].to(dtype) @ st["down"].to(dtype).reshape(n * R, -1).t()
    return (every.reshape(T, n, R) * _chosen(st, dtype)).sum(1)


def _plain_adapter(st):
    T, n, N, R = (st["case"][k] for k in ("T", "n", "N", "R"))
    v = _low(st, torch.float32)
    wide = (v[:, None, :] * _chosen(st, torch.float32) * st["scale"][None, :, None]).reshape(T, n * R)
    up = st["up"].float().transpose(1, 2).reshape(n * R, N)
    return dict(out=(st["base"].float() + wide @ up).to(torch.bfloat16), v=v)


def _plain_adapter_grad(st):
    T, n, H, N, R = (st["case"][k] for k in ("T", "n", "H", "N", "R"))
    mine = _chosen(st, torch.float32) * st["scale"][None, :, None]
    dy, x = st["dy"].float(), st["x"].float()
    up = st["up"].float().transpose(1, 2).reshape(n * R, N)
    du = ((dy @ up.t()).reshape(T, n, R) * mine).reshape(T, n * R)
    dx = st["base"].float() + du @ st["down"].float().reshape(n * R, H)
    v = (st["v"][:, None, :] * mine).reshape(T, n * R)
    d_up = (v.t() @ dy).reshape(n, R, N).transpose(1, 2).contiguous()
    return dict(dx=dx.to(torch.bfloat16), d_down=(du.t() @ x).reshape(n, R, H), d_up=d_up)


# ----------------------------------------------------------------------------- the framework's calls
def _own_balance(st):
    import precision_moe_amd as pm
    return pm.router_balance(st["logits"], st["ids"], st["offsets"])._asdict()


def _own_router_grad(st):
    import precision_moe_amd as pm
    return pm.router_backward(st["logits"], st["ids"], counts=st["counts"], tokens=st["tokens"],
                              d_balance=st["d_balance"], d_z=st["d_z"], d_topk_w=st["d_w"],
                              renormalize=st["case"]["renorm"], seq_offsets=st["offsets"])


def _own_finalize_grad(st):
    import precision_moe_amd as pm
    d_topk_w, d_z = pm.finalize_backward(st["dout"], st["z"], st["row"], st["w"])
    return dict(d_topk_w=d_topk_w, d_z=d_z)


def _own_adapter(st):
    import precision_moe_amd as pm
    out, v = pm.adapter_forward(st["x"], st["ids"], st["down"], st["up"], st["scale"], base=st["base"])
    return dict(out=out, v=v)


def _own_adapter_grad(st):
    import precision_moe_amd as pm
    dx, d_down, d_up = pm.adapter_backward(st["dy"], st["x"], st["v"], st["ids"], st["down"], st["up"],
                                           st["scale"], base=st["base"])
    return dict(dx=dx, d_down=d_down, d_up=d_up)


def run(state):
    op = state["case"]["op"]
    if own:
        if op == "balance":
            return _own_balance(state)
        if op == "router_grad":
            return _own_router_grad(state)
        if op == "finalize_grad":
            return _own_finalize_grad(state)
        return _own_adapter(state) if op == "adapter" else _own_adapter_grad(state)
    if op == "balance":
        return _plain_balance(state)
    if op == "router_grad":
        return _plain_router_grad(state)
    if op == "finalize_grad":
        return _plain_finalize_grad(state)
    return _plain_adapter(state) if op == "adapter" else _plain_adapter_grad(state)


# ----------------------------------------------------------------------------- work
def work(case):
    op, T = case["op"], case["T"]
    if op in ("balance", "router_grad"):
        E, K, S = case["E"], case["K"], case["S"]
        if op == "balance":
            return dict(bytes=4 * (T * E + T * K + 2 * S * E + 4 * S), flops=5 * T * E)
        return dict(bytes=4 * (2 * T * E + 2 * T * K + S * E + 4 * S), flops=12 * T * E)
    H = case["H"]
    if op == "finalize_grad":
        K = case["K"]
        R = max(1, T * K * 3 // 4) if case["dropped"] else T * K
        return dict(bytes=2 * T * H + 4 * R * H + 12 * T * K, flops=3 * R * H)
    n, N, R = case["n"], case["N"], case["R"]
    share = n / (n + 1) if case["runs"] else 0.9      # tokens that have an adapter
    used = n * (1 - (1 - 0.9 / n) ** T) if not case["runs"] else n * min(T, n + 1) / (n + 1)
    weights = 2 * used * R * (H + N)
    if op == "adapter":
        return dict(bytes=2 * (share * T * H + 2 * T * N) + weights + 4 * T * R,
                    flops=2 * share * T * R * (H + N))
    return dict(bytes=2 * (share * T * (H + N) + 2 * T * H) + weights + 4 * n * R * (H + N) + 4 * share * T * R,
                flops=4 * share * T * R * (H + N))


# ----------------------------------------------------------------------------- 64 bits
def _exact_router(st):
    """Softmax rows, log-sum-exp, active tokens and the slice of each sequence."""
    l = st["logits"].double()
    E = l.shape[1]
    lse = torch.logsumexp(l, 1)
    ids = st["ids"]
    active = ((ids >= 0) & (ids < E)).any(1) & (lse > -INF)
    cuts = st["offsets"].tolist()
    return l, lse, active, list(zip(cuts[:-1], cuts[1:]))


def _exact_balance(st):
    l, lse, active, spans = _exact_router(st)
    E, K = st["case"]["E"], st["case"]["K"]
    out = dict(counts=[], tokens=[], prob=[], balance=[], z=[])
    for a, b in spans:
        on = active[a:b]
        x, s, ids = l[a:b][on], lse[a:b][on], st["ids"][a:b][on].long()
        c = torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        P = torch.exp(x - s[:, None]).sum(0)
        n = max(1, x.shape[0])
        out["counts"].append(c.to(torch.int32))
        out["tokens"].append(on.sum().to(torch.int32))
        out["prob"].append(P)
        out["balance"].append(E * ((c.double() / (n * K)) * (P / n)).sum())
        out["z"].append((s * s).sum() / n)
    return {k: torch.stack(v) for k, v in out.items()}


def _exact_router_grad(st):
    l, lse, active, spans = _exact_router(st)
    E, K = st["case"]["E"], st["case"]["K"]
    grad = torch.zeros_like(l)
    for s, (a, b) in enumerate(spans):
        n = max(1, int(st["tokens"][s]))
        f = st["counts"][s].double() / (n * K)
        p = torch.where(active[a:b, None], torch.exp(l[a:b] - lse[a:b, None]), 0.0)
        mean_f = (p @ f)[:, None]
        grad[a:b] = float(st["d_balance"][s]) * E / n * p * (f - mean_f)
        grad[a:b] += float(st["d_z"][s]) * 2 / n * p * torch.where(active[a:b], lse[a:b], 0.0)[:, None]
    p = torch.where(active[:, None], torch.exp(l - lse[:, None]), 0.0)
    dw = st["d_w"].double()
    weight = torch.zeros_like(p)                      # d loss / d weight, and which experts were chosen
    picked = torch.zeros_like(p)
    t = torch.arange(l.shape[0], device=l.device)
    for j in range(K):
        e = st["ids"][:, j].long()
        on = active & (e >= 0) & (e < E)
        weight[t[on], e[on]] += dw[on, j]
        picked[t[on], e[on]] = 1.0
    if st["case"]["renorm"]:
        p = p * picked
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    return grad + p * (weight - (p * weight).sum(1, keepdim=True))


def _exact_finalize_grad(st):
    T, K = st["case"]["T"], st["case"]["K"]
    row = st["row"].reshape(T, K).long()
    dw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    dz = torch.zeros(st["z"].shape, dtype=torch.float64, device="cuda")
    d = st["dout"].double()
    for j in range(K):
        on = row[:, j] >= 0
        r = row[on, j]
        dw[on, j] = (d[on] * st["z"][r].double()).sum(1)
        dz[r] = st["w"][on, j].double()[:, None] * d[on]
    return dict(d_topk_w=dw, d_z=dz)


def _exact_adapter(st):
    T, R = st["case"]["T"], st["case"]["R"]
    out = st["base"].double()
    v = torch.zeros(T, R, dtype=torch.float64, device="cuda")
    for a in range(st["case"]["n"]):
        t = (st["ids"] == a).nonzero()[:, 0]
        v[t] = st["x"][t].double() @ st["down"][a].double().t()
        out[t] += float(st["scale"][a]) * (v[t] @ st["up"][a].double().t())
    return dict(out=out, v=v)


def _exact_adapter_grad(st):
    dx = st["base"].double()
    d_down = torch.zeros(st["down"].shape, dtype=torch.float64, device="cuda")
    d_up = torch.zeros(st["up"].shape, dtype=torch.float64, device="cuda")
    for a in range(st["case"]["n"]):
        t = (st["ids"] == a).nonzero()[:, 0]
        dy = float(st["scale"][a]) * st["dy"][t].double()
        du = dy @ st["up"][a].double()
        dx[t] += du @ st["down"][a].double()
        d_down[a] = du.t() @ st["x"][t].double()
        d_up[a] = dy.t() @ st["v"][t].double()
    return dict(dx=dx, d_down=d_down, d_up=d_up)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(st)
    if case["op"] == "router_grad":
        return _exact_router_grad(st)
    if case["op"] == "finalize_grad":
        return _exact_finalize_grad(st)
    return _exact_adapter(st) if case["op"] == "adapter" else _exact_adapter_grad(st)
