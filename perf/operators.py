"""Operators of mixture-of-experts and adapter serving beside the quantized linears: cases, inputs, plain forms and calls.

Kinds of cases (`op`):
  route    T token rows of E router logits -> top-k experts, weights, and the slots sorted by expert
  gate_up  h = silu(x G_e^T) * (x U_e^T) for the rows of each expert, BenQ 6-bit weights
  linear   y = x W_e^T for the rows of each expert, BenQ 6-bit weights
  combine  out[t] = residual[t] + sum_j w[t, j] y[t k + j]
  lora     y_s += scale (x A^T) B^T with each row's own adapter, for several layers of one input
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# output features of the layers that read one input, by name
_LAYERS = {"qkv": (5120, 1024, 1024), "up": (17408,), "o": (5120,), "gate_up": (17408, 17408), "kv": (1024, 1024)}


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 32 sequences: the router of one layer
        dict(name="route 32 of 64 bf16", op="route", T=32, E=64, k=8, dtype="bf16", normalize=True, masked=False),
        # a prompt of 8192 tokens; some experts are masked off
        dict(name="route 8192 of 128", op="route", T=8192, E=128, k=8, dtype="f32", normalize=True, masked=True),
        # one sequence decoding: latency of a small expert layer
        dict(name="gate_up 1 token", op="gate_up", T=1, E=64, k=8, K=2048, N=1024, dtype="bf16"),
        # 64 sequences decoding, experts of a sixteenth of the 17408-wide MLP of the 5120-wide model
        dict(name="gate_up 64 tokens", op="gate_up", T=64, E=64, k=8, K=5120, N=1088, dtype="bf16"),
        # a prompt of 4096 tokens through the same layer
        dict(name="gate_up 4096 tokens", op="gate_up", T=4096, E=64, k=8, K=5120, N=1088, dtype="bf16"),
        # the down projections of the same layer
        dict(name="linear 17 tokens f32", op="linear", T=17, E=64, k=8, K=1088, N=5120, dtype="f32"),
        dict(name="linear 4096 tokens", op="linear", T=4096, E=64, k=8, K=1088, N=5120, dtype="bf16"),
        # the end of an expert layer: one decode step, and a prompt
        dict(name="combine 16", op="combine", T=16, k=8, N=5120, dtype="bf16", out="bf16", residual=True),
        dict(name="combine 4096", op="combine", T=4096, k=8, N=5120, dtype="bf16", out="bf16", residual=True),
        # 32 requests with 16 adapters beside the q, k and v projections, the plan kept from the step's first layer
        dict(name="lora qkv 32 rows", op="lora", T=32, S=16, r=16, K=5120, layers="qkv", dtype="bf16", plan=False, runs=False),
        # a large decode batch with many adapters, the plan made in the pass
        dict(name="lora o 500 rows f32", op="lora", T=500, S=64, r=32, K=5120, layers="o", dtype="f32", plan=True, runs=False),
        # prompts of a few requests, each with its own adapter
        dict(name="lora up 4096 rows", op="lora", T=4096, S=8, r=64, K=5120, layers="up", dtype="bf16", plan=True, runs=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "gate_up", "linear", "combine", "lora"))
    dtype = rng.choice(("f32", "bf16"))
    if op == "route":
        E = _log(rng, 8, 128)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, 8), dtype=dtype, normalize=rng.random() < 0.7,
                    masked=rng.random() < 0.5)
    if op == "combine":
        return dict(op=op, T=_log(rng, 1, 4096), k=rng.randint(1, 8), N=_log(rng, 100, 5120), dtype=dtype,
                    out=rng.choice(("f32", "bf16")), residual=rng.random() < 0.5)
    if op == "lora":
        return dict(op=op, T=_log(rng, 1, 4096), S=_log(rng, 1, 64), r=rng.choice((4, 8, 16, 16, 24, 32, 64)),
                    K=64 * rng.randint(8, 80), layers=rng.choice(tuple(_LAYERS)), dtype=dtype,
                    plan=rng.random() < 0.5, runs=rng.random() < 0.5)
    E = _log(rng, 4, 64)
    wide, narrow = 64 * rng.randint(8, 80), rng.randint(64, 1088)
    K, N = (wide, narrow) if op == "gate_up" else (64 * rng.randint(2, 17), rng.randint(512, 5120))
    # an expert layer keeps its rows in bf16; fp32 rows are for small batches that are reduced further
    T = _log(rng, 1, 4096)
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), K=K, N=N, dtype=dtype if T <= 64 else "bf16")


# ------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _weights(E, N, K, g):
    """BenQ storage of E layers: codes uint8 [E, N, 3K/4], tables bf16 [E, N, 64] (31 .. 0 negated, then 0 .. 31)."""
    sigma = 0.01 + 0.02 * torch.rand(E, N, 1, device="cuda", generator=g)
    tiers = torch.arange(32, device="cuda") + 0.4 + 0.2 * torch.rand(E, N, 32, device="cuda", generator=g)
    levels = tiers * sigma * (4.0 / 32)          # equal-width shells of a range of about four sigma
    lut = torch.cat((-levels.flip(2), levels), 2).to(torch.bfloat16).contiguous()
    codes = torch.empty(E, N, K // 4, 3, dtype=torch.uint8, device="cuda")
    for e in range(0, E, 8):
        z = torch.randn(min(8, E - e), N, K // 4, 4, device="cuda", generator=g)
        c = (z * 8).floor().clamp_(-32, 31).to(torch.int32) + 32      # codes of normal weights
        v = c[..., 0] | (c[..., 1] << 6) | (c[..., 2] << 12) | (c[..., 3] << 18)
        codes[e:e + 8, ..., 0] = v & 255
        codes[e:e + 8, ..., 1] = (v >> 8) & 255
        codes[e:e + 8, ..., 2] = v >> 16
    return codes.view(E, N, 3 * K // 4), lut


def _logits(T, E, g):
    """Router logits: some experts are liked better than others."""
    return torch.randn(T, E, device="cuda", generator=g) + 0.7 * torch.randn(1, E, device="cuda", generator=g)


def _grouped(index, G):
    """Rows sorted by group (stable), group bounds; rows of no group (index outside [0, G)) come last, as -1."""
    key = torch.where((index >= 0) & (index < G), index, G).long()
    order = torch.argsort(key, stable=True)
    offsets = torch.zeros(G + 1, dtype=torch.int64, device=index.device)
    offsets[1:] = torch.zeros(G + 1, dtype=torch.int64, device=index.device).scatter_add_(0, key, torch.ones_like(key))[:G].cumsum(0)
    order = torch.where(torch.arange(order.numel(), device=index.device) < offsets[G], order, -1)
    return order.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], dict(case)
    bf = torch.bfloat16
    if op == "route":
        T, E, k = case["T"], case["E"], min(case["k"], case["E"])
        l = _logits(T, E, g)
        if case["masked"]:
            l = l.masked_fill(torch.rand(T, E, device="cuda", generator=g) < 0.2, -math.inf)
        s["logits"] = l.to(_DT[case["dtype"]])
        i32 = dict(dtype=torch.int32, device="cuda")
        s["experts"], s["weights"] = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
        s["order"], s["offsets"] = torch.empty(T * k, **i32), torch.empty(E + 1, **i32)
    elif op in ("gate_up", "linear"):
        T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
        experts = _logits(T, E, g).topk(k, 1).indices.to(torch.int32)
        s["order"], s["offsets"] = _grouped(experts.reshape(-1), E)
        if op == "gate_up":
            s["x"] = torch.randn(T, K, device="cuda", generator=g).to(bf)      # one row per token
            s["wg"], s["wu"] = _weights(E, N, K, g), _weights(E, N, K, g)
        else:
            s["x"] = (0.3 * torch.randn(T * k, K, device="cuda", generator=g)).to(bf)   # sorted rows of gate_up
            s["w"] = _weights(E, N, K, g)
        s["y"] = torch.zeros(T * k, N, dtype=_DT[case["dtype"]], device="cuda")
    elif op == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        s["rows"] = torch.randn(T * k, N, device="cuda", generator=g).to(_DT[case["dtype"]])
        s["weights"] = torch.softmax(torch.randn(T, k, device="cuda", generator=g), 1)
        s["experts"] = torch.randint(0, 64, (T, k), dtype=torch.int32, device="cuda", generator=g)
        s["add"] = torch.randn(T, N, device="cuda", generator=g).to(_DT[case["out"]]) if case["residual"] else None
        s["y"] = torch.empty(T, N, dtype=_DT[case["out"]], device="cuda")
    else:
        T, S, r, K = case["T"], case["S"], case["r"], case["K"]
        s["x"] = torch.randn(T, K, device="cuda", generator=g).to(bf)
        # each row's adapter: rows of one request follow one another in a prompt batch; -1 is a row without an adapter
        if case["runs"]:
            cuts = torch.randint(0, T + 1, (2 * S,), device="cuda", generator=g).sort().values
            which = torch.randint(-1, S, (2 * S + 1,), device="cuda", generator=g)
            s["index"] = which[torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)].to(torch.int32)
        else:
            s["index"] = torch.randint(-1 if S > 1 else 0, S, (T,), dtype=torch.int32, device="cuda", generator=g)
        s["scale"] = 0.5 + torch.rand(S, device="cuda", generator=g)
        s["layers"] = [((torch.randn(S, r, K, device="cuda", generator=g) / K ** 0.5).to(bf),
                        (torch.randn(S, n, r, device="cuda", generator=g) / r ** 0.5).to(bf),
                        torch.randn(T, n, device="cuda", generator=g).to(_DT[case["dtype"]])) for n in _LAYERS[case["layers"]]]
        s["order"], s["offsets"] = _grouped(s["index"], S)
    s["ws"] = None
    return s


# ------------------------------------------------------------------------------------------- plain forms

def _dequant(codes, lut):
    E, N, B = codes.shape
    b = codes.view(E, N, B // 3, 3).to(torch.int32)
    v = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
    c = torch.stack((v & 63, (v >> 6) & 63, (v >> 12) & 63, v >> 18), -1).view(E, N, B // 3 * 4)
    return lut.float().gather(2, c.long())


def _padded(offsets, rows):
    """Positions of every group's rows, padded to the longest group: [G, cap], and which of them exist."""
    o = offsets.long()
    count = o[1:] - o[:-1]
    at = torch.arange(max(1, int(count.max())), device=o.device)
    return (o[:-1, None] + at).clamp_(max=max(0, rows - 1)), at < count[:, None]


def _plain_route(s):
    l = s["logits"].float()
    T, E = l.shape
    k = s["experts"].shape[1]
    value, at = (v[:, :k] for v in torch.sort(l, dim=1, descending=True, stable=True))
    routed = value != -math.inf
    top = value[:, :1]
    e = torch.where(routed, torch.exp(value - top), 0.0)
    total = e.sum(1, keepdim=True) if s["normalize"] else torch.where(l == -math.inf, 0.0, torch.exp(l - top)).sum(1, keepdim=True)
    experts = torch.where(routed, at, -1).to(torch.int32)
    weights = torch.where(routed, e / total, 0.0)
    return experts, weights, *_grouped(experts.reshape(-1), E)


def _plain_gate_up(s):
    at, there = _padded(s["offsets"], s["order"].numel())
    x = s["x"][s["order"].long()[at].clamp_(min=0) // s["k"]].float()
    gate = torch.bmm(x, _dequant(*s["wg"]).transpose(1, 2))
    up = torch.bmm(x, _dequant(*s["wu"]).transpose(1, 2))
    s["y"][at[there]] = (gate / (1 + torch.exp(-gate)) * up)[there].to(s["y"].dtype)
    return s["y"]


def _plain_linear(s):
    at, there = _padded(s["offsets"], s["order"].numel())
    y = torch.bmm(s["x"][at].float(), _dequant(*s["w"]).transpose(1, 2))
    s["y"][s["order"].long()[at[there]]] = y[there].to(s["y"].dtype)
    return s["y"]


def _plain_combine(s):
    T, k = s["weights"].shape
    w = torch.where(s["experts"] >= 0, s["weights"], 0.0)
    y = (s["rows"].view(T, k, -1).float() * w[..., None]).sum(1)
    return (y if s["add"] is None else y + s["add"].float()).to(s["y"].dtype)


def _plain_lora(s):
    order, offsets = _grouped(s["index"], s["S"]) if s["plan"] else (s["order"], s["offsets"])
    at, there = _padded(offsets, order.numel())
    rows = order.long()[at[there]]
    x = s["x"][order.long()[at].clamp_(min=0)].float()
    return [_plain_adapter(x, a, b, y, s["scale"], rows, there) for a, b, y in s["layers"]]


def _plain_adapter(x, a, b, y, scale, rows, there):
    t = torch.bmm(x, a.float().transpose(1, 2)) * scale[:, None, None]
    y[rows] = (y[rows].float() + torch.bmm(t, b.float().transpose(1, 2))[there]).to(y.dtype)
    return y


# ------------------------------------------------------------------------------------------- one pass

def _room(s, n):
    """The workspace that a program keeps."""
    if s["ws"] is None:
        s["ws"] = torch.empty(max(256, n), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_route(s, ql):
    T, E = s["logits"].shape
    ws = s["ws"] if s["ws"] is not None else _room(s, ql.moe_route_workspace_bytes(T, E, s["experts"].shape[1]))
    ql.moe_route(s["logits"], s["experts"], s["weights"], s["order"], s["offsets"], normalize=s["normalize"], workspace=ws)
    return s["experts"], s["weights"], s["order"], s["offsets"]


def _own_gate_up(s, ql):
    return ql.benq_grouped_gate_up(*s["wg"], *s["wu"], s["x"], s["offsets"], s["y"], x_rows=s["order"], x_div=s["k"])


def _own_linear(s, ql):
    return ql.benq_grouped_linear(*s["w"], s["x"], s["offsets"], s["y"], y_rows=s["order"])


def _own_combine(s, ql):
    return ql.moe_combine(s["rows"], s["experts"], s["weights"], s["y"], residual=s["add"])


def _own_lora(s, ql):
    T, S = s["T"], s["S"]
    ws = s["ws"] if s["ws"] is not None else _room(s, max(ql.group_rows_workspace_bytes(T, S),
                                                          ql.lora_workspace_bytes(len(s["layers"]), T, s["r"])))
    if s["plan"]:
        ql.group_rows(s["index"], S, s["order"], s["offsets"], workspace=ws)
    return ql.lora_add(s["layers"], s["x"], s["order"], s["offsets"], scale=s["scale"], workspace=ws)


def run(state):
    if own:
        import quantized_linear_b200 as ql
        return _OWN[state["op"]](state, ql)
    return _PLAIN[state["op"]](state)


_PLAIN = dict(route=_plain_route, gate_up=_plain_gate_up, linear=_plain_linear, combine=_plain_combine, lora=_plain_lora)
_OWN = dict(route=_own_route, gate_up=_own_gate_up, linear=_own_linear, combine=_own_combine, lora=_own_lora)


# ------------------------------------------------------------------------------------------- floors

def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], min(case["k"], case["E"])
        return dict(bytes=T * E * _size(case["dtype"]) + 12 * T * k + 4 * (E + 1), flops=4 * T * E)
    if op == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        ob = _size(case["out"])
        return dict(bytes=T * k * (N * _size(case["dtype"]) + 8) + T * N * ob * (2 if case["residual"] else 1), flops=2 * T * k * N)
    if op == "lora":
        T, S, r, K = case["T"], case["S"], case["r"], case["K"]
        rows = T * S / (S + 1) if S > 1 else T                          # some rows have no adapter
        used = S * (1 - (1 - 1 / (S + 1)) ** T) if not case["runs"] else S * (1 - (1 - 1 / (S + 1)) ** min(T, 2 * S + 1))
        N = sum(_LAYERS[case["layers"]])
        L = len(_LAYERS[case["layers"]])
        return dict(bytes=used * 2 * r * (L * K + N) + rows * (2 * K + 2 * N * _size(case["dtype"])) + 8 * T,
                    flops=2 * rows * r * (L * K + N))
    T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
    mats = 2 if op == "gate_up" else 1
    used = E * (1 - (1 - k / E) ** T)                                   # experts that have rows
    x_rows = T if op == "gate_up" else T * k
    return dict(bytes=used * mats * N * (0.75 * K + 128) + 2 * x_rows * K + T * k * (N * _size(case["dtype"]) + 4),
                flops=2 * mats * T * k * N * K)


# ------------------------------------------------------------------------------------------- 64 bits

def _table_lookup(codes, lut):
    """One layer's W in 64 bits from its packed codes: bits [6j, 6j + 6) of a row's little-endian stream index its table."""
    N, B = codes.shape
    bits = (codes[:, :, None] >> torch.arange(8, device=codes.device, dtype=torch.uint8)) & 1
    place = (1 << torch.arange(6, device=codes.device)).to(torch.int64)
    c = (bits.view(N, B * 8 // 6, 6).to(torch.int64) * place).sum(2)
    return torch.take_along_dim(lut.double(), c, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        l = s["logits"].double()
        T, E = l.shape
        k = s["experts"].shape[1]
        experts = torch.full((T, k), -1, dtype=torch.int64, device="cuda")
        weights = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        p = torch.softmax(l, 1).nan_to_num(0.0)
        left = l.clone()
        for j in range(k):
            best = left.max(1, keepdim=True).values
            place = torch.where(left == best, torch.arange(E, device="cuda"), E).min(1, keepdim=True).values   # ties: the first
            live = best[:, 0] > -math.inf
            experts[live, j] = place[live, 0]
            weights[live, j] = p.gather(1, place)[live, 0]
            left.scatter_(1, place, -math.inf)
        if case["normalize"]:
            weights = (weights / weights.sum(1, keepdim=True)).nan_to_num(0.0)
        return None, weights, None, None
    if op == "combine":
        T, k = s["weights"].shape
        y = torch.zeros(T, case["N"], dtype=torch.float64, device="cuda")
        for j in range(k):
            y += s["weights"][:, j, None].double() * s["rows"][j::k].double()
        return y if s["add"] is None else y + s["add"].double()
    if op == "lora":
        index, outs = s["index"].tolist(), []
        rows = {a: torch.tensor([t for t, i in enumerate(index) if i == a], device="cuda") for a in sorted(set(index)) if a >= 0}
        for a_all, b_all, y in s["layers"]:
            out = y.double()
            for a, at in rows.items():
                out[at] += float(s["scale"][a]) * (s["x"][at].double() @ a_all[a].double().T @ b_all[a].double().T)
            outs.append(out)
        return outs
    out = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    bounds, order = s["offsets"].tolist(), s["order"].long()
    for e in range(case["E"]):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        if op == "gate_up":
            x = s["x"][order[a:b] // case["k"]].double()
            gate, up = (x @ _table_lookup(w[0][e], w[1][e]).T for w in (s["wg"], s["wu"]))
            out[a:b] = gate * torch.sigmoid(gate) * up
        else:
            out[order[a:b]] = s["x"][a:b].double() @ _table_lookup(s["w"][0][e], s["w"][1][e]).T
    return out
