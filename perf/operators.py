"""The operators whose weights are chosen for each token, as a user calls them, with their plain forms.

Three operators of a decoder that is served on packed-int4 weights:

* ``moe_route``: the router's choice, the top k of a row of logits and their softmax weights;
* ``moe`` (``moe_awq_w4a16`` and ``moe_experts_awq_w4a16``): a whole mixture-of-experts layer for a few tokens,
  its experts in the AWQ W4A16 format of ``gemv_awq_w4a16``;
* ``lora`` (``lora_add``): the low-rank adapters of many requests, added to the output of a projection
  that all of them share.

``run`` computes the plain form in 32 bits, or with ``own`` calls the package's kernels.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of a batch: the choice among 128 experts
        dict(name="route decode", op="route", T=64, E=128, k=8, dtype="fp32", renorm=True),
        # a long prompt; bf16 logits meet many ties; the weights stay shares of all experts
        dict(name="route prompt", op="route", T=8192, E=64, k=6, dtype="bf16", renorm=False),
        # a single stream's decode step: eight small experts of 64
        dict(name="moe single token", op="moe", T=1, E=64, k=8, K=2048, I=1024, G=64, dtype="bf16", given=False, renorm=True),
        # odd sizes, the choice made elsewhere (a router with rules of its own), some slots without an expert
        dict(name="moe odd given", op="moe", T=5, E=20, k=3, K=1472, I=704, G=64, dtype="fp16", given=True, renorm=True),
        # a small batch's decode step: nearly every expert is met by a token or two
        dict(name="moe batch 16", op="moe", T=16, E=64, k=8, K=2048, I=1024, G=64, dtype="bf16", given=False, renorm=True),
        # few wide experts, a batch with several tokens for each of them
        dict(name="moe wide 32", op="moe", T=32, E=8, k=2, K=3840, I=10240, G=128, dtype="bf16", given=False, renorm=False),
        # a single stream's decode step beside a square projection
        dict(name="lora single token", op="lora", M=1, K=3840, N=3840, R=16, L=8, run=1, dtype="bf16", ydtype="bf16", scaled=True),
        # a decode step of 64 requests with adapters of their own beside a wide projection
        dict(name="lora decode 64", op="lora", M=64, K=4096, N=12288, R=32, L=48, run=1, dtype="bf16", ydtype="bf16", scaled=True),
        # several requests' prompts, packed, with the odd sizes of a small model
        dict(name="lora odd", op="lora", M=777, K=1480, N=1001, R=24, L=5, run=150, dtype="fp16", ydtype="bf16", scaled=False),
        # prompts beside the linear's own wide side
        dict(name="lora prompts wide", op="lora", M=2048, K=3840, N=10240, R=16, L=12, run=300, dtype="fp16", ydtype="fp16", scaled=True),
        # a full prefill batch
        dict(name="lora prompts 8192", op="lora", M=8192, K=3840, N=3840, R=64, L=8, run=1024, dtype="bf16", ydtype="bf16", scaled=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "lora", "lora"])
    if op == "route":
        E = rng.randint(2, 256)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 16)),
                    dtype=rng.choice(["fp32", "bf16", "fp16"]), renorm=rng.random() < 0.5)
    if op == "moe":
        G = rng.choice([64, 128])
        E = _log(rng, 4, 128)
        K, I = G * _log(rng, 4, 4096 // G), G * _log(rng, 2, 4096 // G)
        while E * K * I > 8 * 3840 * 10240:        # no more weights than the largest listed case
            E = (E + 1) // 2
        return dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(E, 8)), K=K, I=I, G=G,
                    dtype=rng.choice(["bf16", "fp16"]), given=rng.random() < 0.3, renorm=rng.random() < 0.5)
    M = _log(rng, 1, 8192)
    K, N, R = 8 * _log(rng, 16, 640), _log(rng, 100, 12288), 8 * _log(rng, 1, 16)
    L = _log(rng, 1, 64)
    while L > 1 and (L * R > 2048 or M * L * R * (K + N) > 8192 * 512 * 7680):
        L = (L + 1) // 2
    while M * R * (K + N) > 8192 * 64 * 7680 or M * (K + 2 * N) > 8192 * 3 * 3840:
        M = (M + 1) // 2
    dtype = rng.choice(["bf16", "fp16"])
    return dict(op="lora", M=M, K=K, N=N, R=R, L=L, run=_log(rng, 1, max(M, 2)), dtype=dtype,
                ydtype=rng.choice(["bf16", dtype]), scaled=rng.random() < 0.7)


# ------------------------------------------------------------------- inputs

def _experts(E, K, I, G, dt, g, dev):
    def q(rows, cols):
        return torch.randint(0, 256, (E, rows, cols // 2), generator=g, device=dev, dtype=torch.uint8)

    def s(rows, cols):
        return (torch.rand((E, cols // G, rows), generator=g, device=dev) * 0.009 + 0.001).to(dt)

    def z(rows, cols):
        return (torch.randn((E, cols // G, rows), generator=g, device=dev) * 0.01).to(dt)

    return (q(2 * I, K), s(2 * I, K), z(2 * I, K)), (q(K, I), s(K, I), z(K, I))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = dict(case)
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["op"] == "route":
        st["logits"] = (torch.randn((c["T"], c["E"]), generator=g, device=dev) * 2).to(dt)
    elif c["op"] == "moe":
        st["x"] = torch.randn((c["T"], c["K"]), generator=g, device=dev).to(dt)
        st["gate_up"], st["down"] = _experts(c["E"], c["K"], c["I"], c["G"], dt, g, dev)
        logits = torch.randn((c["T"], c["E"]), generator=g, device=dev) * 1.5
        if c["given"]:
            order = logits.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
            drop = torch.rand(order.shape, generator=g, device=dev) < 0.1      # slots over an expert's capacity
            st["ids"] = order.masked_fill(drop, -1).to(torch.int32)
            st["weights"] = torch.rand(order.shape, generator=g, device=dev)
        else:
            st["logits"] = logits
    else:
        M, K, N, R, L = c["M"], c["K"], c["N"], c["R"], c["L"]
        st["x"] = torch.randn((M, K), generator=g, device=dev).to(dt)
        st["y"] = torch.randn((M, N), generator=g, device=dev).to(DTYPES[c["ydtype"]])
        st["a"] = (torch.randn((L, R, K), generator=g, device=dev) / math.sqrt(K)).to(dt)
        st["b"] = (torch.randn((L, N, R), generator=g, device=dev) / math.sqrt(R)).to(dt)
        # requests of about `run` tokens each, an adapter or none (-1) for each request
        runs = -(-M // c["run"])
        ids = torch.randint(-1 if runs > 4 else 0, L, (runs,), generator=g, device=dev, dtype=torch.int32)
        st["ids"] = ids.repeat_interleave(c["run"])[:M].contiguous()
        st["scales"] = torch.rand((L,), generator=g, device=dev) + 0.5 if c["scaled"] else None
    return st


# -------------------------------------------------------------- plain forms

def _route(logits, k, renorm):
    v = logits.float()
    order = v.sort(dim=1, descending=True, stable=True)       # stable: the lowest index of a tie comes first
    top, ids = order.values[:, :k], order.indices[:, :k]
    live = top > -math.inf
    best = v.amax(dim=1, keepdim=True)
    p = torch.exp(top - best)
    total = p.sum(dim=1, keepdim=True) if renorm else torch.exp(v - best).sum(dim=1, keepdim=True)
    return torch.where(live, p / total, 0.0), torch.where(live, ids, -1).to(torch.int32)


def _dequantize(packed, scales, zeros):
    """(E, rows, cols/2) bytes, (E, cols/G, rows) scales and zeros -> (E, rows, cols) in 32 bits."""
    q = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(2).float() - 8
    E, rows, cols = q.shape
    q = q.view(E, rows, scales.shape[1], -1)
    w = q * scales.float().transpose(1, 2).unsqueeze(-1) + zeros.float().transpose(1, 2).unsqueeze(-1)
    return w.view(E, rows, cols)


def _experts_product(x, st, at):
    gu = torch.matmul(x, _dequantize(*(p[at] for p in st["gate_up"])).transpose(1, 2))
    gate, up = gu.chunk(2, dim=-1)
    h = gate / (1 + torch.exp(-gate)) * up
    return torch.matmul(h, _dequantize(*(p[at] for p in st["down"])).transpose(1, 2))


def _moe(st):
    c = st["case"]
    if c["given"]:
        weights, ids = st["weights"], st["ids"]
    else:
        weights, ids = _route(st["logits"], c["k"], c["renorm"])
    x = st["x"].float()
    if ids.numel() < c["E"]:                       # a slot at a time: fewer weights than all experts have
        share = torch.where(ids < 0, 0.0, weights)
        at = ids.flatten().clamp(min=0).long()
        y = _experts_product(x.repeat_interleave(c["k"], 0).unsqueeze(1), st, at)      # (T k, 1, K)
        out = (y.view(c["T"], c["k"], -1) * share.unsqueeze(-1)).sum(dim=1)
    else:                                          # all tokens through all experts, weighted
        share = torch.zeros((c["T"], c["E"] + 1), device=ids.device)
        share.scatter_add_(1, torch.where(ids < 0, c["E"], ids).long(), weights)       # the last column: no expert
        y = _experts_product(x, st, slice(None))                                       # (E, T, K)
        out = (y * share[:, :-1].t().unsqueeze(-1)).sum(dim=0)
    return out.to(st["x"].dtype)


def _lora(st):
    x, y, a, b, ids = st["x"].float(), st["y"].float(), st["a"].float(), st["b"].float(), st["ids"]
    L, R, K = a.shape
    N = b.shape[1]
    mine = (ids.unsqueeze(1) == torch.arange(L, device=ids.device)).float()
    if st["scales"] is not None:
        mine = mine * st["scales"]
    v = torch.matmul(x, a.view(L * R, K).t()).view(-1, L, R) * mine.unsqueeze(-1)
    d = torch.matmul(v.view(-1, L * R), b.transpose(1, 2).reshape(L * R, N))
    return (y + d).to(st["y"].dtype)


def run(st):
    c = st["case"]
    if own:
        from bit_quantized_linear_rotate_b200 import ck
        if c["op"] == "route":
            return ck.moe_route(st["logits"], c["k"], renormalize=c["renorm"])
        if c["op"] == "lora":
            return ck.lora_add(st["y"], st["x"], st["a"], st["b"], st["ids"], scales=st["scales"])
        if c["given"]:
            return ck.moe_experts_awq_w4a16(st["x"], st["ids"], st["weights"], *st["gate_up"], *st["down"],
                                            group_size=c["G"])
        return ck.moe_awq_w4a16(st["x"], st["logits"], c["k"], *st["gate_up"], *st["down"], group_size=c["G"],
                                renormalize=c["renorm"])
    if c["op"] == "route":
        return _route(st["logits"], c["k"], c["renorm"])
    return _moe(st) if c["op"] == "moe" else _lora(st)


# --------------------------------------------------------------------- work

def work(case):
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * size + 8 * T * k, "flops": 4 * T * E}
    if c["op"] == "moe":
        T, E, k, K, I, G = c["T"], c["E"], c["k"], c["K"], c["I"], c["G"]
        live = k * (0.9 if c["given"] else 1.0)
        met = E * (1 - (1 - live / E) ** T)        # experts that some token goes to, on average
        weights = 3 * K * I * (0.5 + 4 / G)        # nibbles, and a scale and a zero of 16 bits for each group
        route = 8 * T * k if c["given"] else 4 * T * E
        return {"bytes": met * weights + 4 * T * K + route, "flops": 2 * T * live * 3 * K * I}
    M, K, N, R, L = c["M"], c["K"], c["N"], c["R"], c["L"]
    runs = -(-M // c["run"])
    share = L / (L + 1) if runs > 4 else 1.0       # tokens with an adapter
    met = L * (1 - (1 - share / L) ** runs)
    return {"bytes": 2 * (share * M * K + 2 * M * N + met * R * (K + N)) + 4 * M, "flops": 2 * share * M * R * (K + N)}


# -------------------------------------------------------------------- exact

def _exact_route(logits, k, renorm):
    v = logits.double().cpu()
    T, E = v.shape
    w = torch.zeros((T, k), dtype=torch.float64)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    at = torch.arange(E, dtype=torch.float64)
    rest = v.clone()
    for j in range(k):
        best = rest.max(dim=1).values
        first = torch.where(rest == best[:, None], at, float(E)).min(dim=1).values.long()
        ok = best > -math.inf
        ids[:, j] = torch.where(ok, first, -1).int()
        w[:, j] = torch.where(ok, best, -math.inf)
        rest[torch.arange(T), first] = -math.inf
    total = torch.logsumexp(w, 1) if renorm else torch.logsumexp(v, 1)
    return torch.exp(w - total[:, None]), ids


def _exact_moe(st):
    c = st["case"]
    if c["given"]:
        w, ids = st["weights"].double().cpu(), st["ids"].cpu()
    else:
        w, ids = _exact_route(st["logits"], c["k"], c["renorm"])
    dev = st["x"].device
    x = st["x"].double()
    out = torch.zeros((c["T"], c["K"]), dtype=torch.float64, device=dev)

    def product(rows, expert, parts):
        packed, s, z = (p[expert] for p in parts)
        n, half = packed.shape
        w64 = torch.empty((n, 2 * half), dtype=torch.float64, device=dev)
        w64[:, 0::2] = (packed % 16).double() - 8.0
        w64[:, 1::2] = (packed // 16).double() - 8.0
        w64.mul_(s.double().repeat_interleave(c["G"], 0).t()).add_(z.double().repeat_interleave(c["G"], 0).t())
        return torch.einsum("tc,nc->tn", rows, w64)

    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = product(x[t.to(dev)], e, st["gate_up"])
        gate, up = gu[:, :c["I"]], gu[:, c["I"]:]
        y = product(gate * torch.sigmoid(gate) * up, e, st["down"])
        out.index_add_(0, t.to(dev), y * w[t, j].to(dev)[:, None])
    return out


def _exact_lora(st):
    out = st["y"].double()
    for i in sorted(set(st["ids"].tolist()) - {-1}):
        rows = torch.nonzero(st["ids"] == i).flatten()
        v = torch.einsum("mk,rk->mr", st["x"][rows].double(), st["a"][i].double())
        d = torch.einsum("mr,nr->mn", v, st["b"][i].double())
        out[rows] += d if st["scales"] is None else d * st["scales"][i].double()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        w, _ = _exact_route(st["logits"], case["k"], case["renorm"])
        return w, None
    return _exact_moe(st) if case["op"] == "moe" else _exact_lora(st)
