"""The training and 8-bit operators of the layer, measured: tokens sorted by
expert and combined back (with their gradients), the router's gradient, and
the experts' products in 8-bit integers.

`run` computes a case in plain torch operations, or, where `own` is true, by
the calls of mixture_experts_ffn_token_b200.abi that a user makes.
"""
import math

import torch

own = False

BF16, F32 = "bfloat16", "float32"


# ------------------------------------------------------------------ the cases
def _rows(name, op, T, H, E, k, dtype=BF16, weighted=True, drop=0.0):
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "k": k, "dtype": dtype, "weighted": weighted,
            "drop": drop}


def _route(name, T, E, k, S=0, dtype=F32, std=1.0):
    return {"name": name, "op": "route_backward", "T": T, "E": E, "k": k, "S": S, "dtype": dtype, "std": std}


def _int8(name, part, T, H, D, E, k, act="silu", fmt="concatenated", bias=False, zipf=False):
    return {"name": name, "op": "int8", "part": part, "T": T, "H": H, "D": D, "E": E, "k": k, "act": act,
            "fmt": fmt, "bias": bias, "zipf": zipf}


def listed():
    return [
        # one generated token on its way to 8 of 64 experts: latency
        _rows("dispatch one token", "dispatch", 1, 4096, 64, 8, weighted=False),
        # the sigmoid-sink layer's tokens to their experts, scaled first
        _rows("dispatch sink layer", "dispatch", 8192, 2048, 128, 6),
        # the Mixtral-shaped layer's gradient on its way back to the tokens and the router weights
        _rows("dispatch backward mixtral", "dispatch_backward", 4096, 4096, 8, 2),
        # the GptOss-shaped layer's expert outputs summed per token
        _rows("combine gptoss", "combine", 2048, 2880, 128, 4),
        # the sigmoid-sink layer's gradient to the experts and the router weights
        _rows("combine backward sink", "combine_backward", 8192, 2048, 128, 6),
        # a ragged fp32 batch in which a tenth of the slots went to no expert
        _rows("combine backward fp32", "combine_backward", 1021, 2880, 128, 4, dtype=F32, drop=0.1),
        # gradients of the router: softmax over the selected, and the sigmoid gate with its sink lanes
        _route("router gradient gptoss", 2048, 128, 4, std=2.0),
        _route("router gradient sink", 8192, 128, 6, S=2),
        # 8-bit experts: one token and one decode batch through the down product (weights from HBM)
        _int8("int8 down one token", "down", 1, 4096, 1536, 64, 8),
        _int8("int8 down decode", "down", 32, 4096, 1536, 64, 8, zipf=True),
        # a GptOss-shaped prefill (many experts, bias, interleaved clamped activation) and a Mixtral-shaped one
        _int8("int8 gate_up gptoss", "gate_up", 2048, 2880, 2880, 128, 4, act="swigluoai", fmt="interleaved",
              bias=True),
        _int8("int8 gate_up mixtral", "gate_up", 4096, 4096, 14336, 8, 2),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_backward", "combine", "combine_backward", "route_backward", "int8", "int8"])
    E = _log(rng, 2, 256)
    if op == "route_backward":
        T, dtype = _log(rng, 1, 16384), rng.choice([F32, BF16])
        n = rng.choice([2, 4, 8, 16])
        if rng.random() < 0.5 and n <= E:
            k = rng.randint(1, n)
            c = _route("", T, E, k, n - k, dtype, 1.0) if n > k else _route("", T, E, k, 0, dtype, 2.0)
        else:
            c = _route("", T, E, rng.randint(2, min(E, 16)), 0, dtype, 2.0)  # (one selected expert has no gradient)
    elif op == "int8":
        k = rng.randint(1, min(E, 8))
        while True:
            T, H, D = _log(rng, 1, 4096), _log(rng, 64, 8192, 8), _log(rng, 64, 8192, 8)
            if T * k * H * D * 6 <= 1.9e12 and E * H * D <= 1.2e9 and E * min(T, 64 + 3 * T * k // E) * (H + 2 * D) <= 2e9:
                break
        c = _int8("", rng.choice(["gate_up", "down"]), T, H, D, E, k, rng.choice(["silu", "swigluoai", "gelu_tanh"]),
                  rng.choice(["concatenated", "interleaved"]), rng.random() < 0.5)
    else:
        k = rng.randint(1, min(E, 16))
        while True:
            T, H = _log(rng, 1, 16384), _log(rng, 64, 8192, 8)
            if T * k * H <= 2e8:
                break
        c = _rows("", op, T, H, E, k, rng.choice([BF16, BF16, F32]), rng.random() < 0.8, rng.choice([0.0, 0.0, 0.2]))
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs
def _normal(gen, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _routing(case, gen):
    """expert_indices [T, k], expert_offsets [E+1] and inverse [T*k] (-1: the slot goes to no expert)."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = _normal(gen, T, E)
    if case.get("zipf"):
        rank = torch.randperm(E, generator=gen, device="cuda") + 1.0
        gumbel = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-12, 1 - 1e-7)))
        logits = gumbel - 1.2 * torch.log(rank)
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    flat = idx.reshape(-1).long()
    if case.get("drop"):
        flat = torch.where(torch.rand(T * k, generator=gen, device="cuda") < case["drop"], E, flat)
    order = torch.argsort(flat, stable=True)
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(T * k, device="cuda")
    inverse = torch.where(flat < E, inverse, -1).to(torch.int32)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return idx, offsets, inverse, int(counts.max())


def _pitch(n):
    return (n + 15) // 16 * 16


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, E, k, op = case["T"], case["E"], case["k"], case["op"]
    s = {"case": case}
    if op == "route_backward":
        S, dtype = case["S"], getattr(torch, case["dtype"])
        s["logits"] = _normal(gen, T, E + S, std=case["std"], dtype=dtype)
        score = torch.sigmoid(s["logits"][:, :E].float()) + 0.2 * torch.rand(E, generator=gen, device="cuda") - 0.1
        s["idx"] = torch.topk(score if S else s["logits"][:, :E].float(), k, dim=1).indices.to(torch.int32)
        s["global_scale"] = torch.rand(1, generator=gen, device="cuda") + 0.5
        s["d_w"], s["d_sink"] = _normal(gen, T, k), _normal(gen, T, S)
        s["d_logits"], s["d_global_scale"] = torch.zeros_like(s["logits"]), torch.zeros(1, device="cuda")
        return s
    s["idx"], s["offsets"], s["inverse"], s["most"] = _routing(case, gen)
    R = T * k
    if op == "int8":
        gate_up = case["part"] == "gate_up"
        K, N = (case["H"], 2 * case["D"]) if gate_up else (case["D"], case["H"])
        # gate_up: the tokens; down: the activations of the sorted rows
        s["a"] = _normal(gen, T if gate_up else R, K, dtype=torch.bfloat16)
        s["w_q"] = torch.zeros(E, N, _pitch(K), dtype=torch.int8, device="cuda")
        for e in range(E):
            s["w_q"][e, :, :K] = _normal(gen, N, K, std=127 / 4).round_().clamp_(-127, 127).to(torch.int8)
        s["w_scales"] = (torch.rand(E, N, generator=gen, device="cuda") * 0.2 + 0.9) * (0.08 / 127)
        s["bias"] = _normal(gen, E, N, std=0.01, dtype=torch.bfloat16) if case["bias"] else None
        s["out"] = torch.zeros(R, case["D"] if gate_up else N, dtype=torch.bfloat16, device="cuda")
        s["rows_q"] = torch.zeros(R, _pitch(K), dtype=torch.int8, device="cuda")
        s["row_scales"] = torch.zeros(R, device="cuda")
        return s
    H, dtype = case["H"], getattr(torch, case["dtype"])
    w = torch.rand(T, k, generator=gen, device="cuda") + 0.05
    s["w"] = w / w.sum(1, keepdim=True) if case["weighted"] else None
    s["tokens"], s["rows"] = _normal(gen, T, H, dtype=dtype), _normal(gen, R, H, dtype=dtype)
    s["out_tokens"], s["out_rows"] = torch.zeros_like(s["tokens"]), torch.zeros_like(s["rows"])
    s["d_w"] = torch.zeros(T, k, device="cuda")
    return s


# --------------------------------------------------------------- one pass
_ALPHA, _LIMIT = 1.702, 7.0


def _act(kind, g, u):
    if kind == "silu":
        return g * torch.sigmoid(g) * u
    if kind == "swigluoai":
        g, u = g.clamp(max=_LIMIT), u.clamp(-_LIMIT, _LIMIT)
        return g * torch.sigmoid(_ALPHA * g) * (u + 1)
    return 0.5 * g * (1 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g))) * u


def _plain_rows(s):
    case, op = s["case"], s["case"]["op"]
    T, k, H = case["T"], case["k"], case["H"]
    live = (s["inverse"] >= 0).view(T, k, 1)
    pos = s["inverse"].clamp(min=0).long()
    w = s["w"].view(T, k, 1) if s["w"] is not None else 1.0
    if op in ("dispatch", "combine_backward"):
        scaled = (s["tokens"].float().view(T, 1, H) * w).expand(T, k, H).reshape(T * k, H)
        rows = torch.zeros(T * k + 1, H, dtype=s["rows"].dtype, device="cuda")
        rows[torch.where(live.view(-1), pos, T * k)] = scaled.to(rows.dtype)
        if op == "dispatch":
            return rows[:-1]
    picked = torch.where(live, s["rows"][pos].float().view(T, k, H), 0.0)
    d_w = (picked * s["tokens"].float().view(T, 1, H)).sum(2) if s["w"] is not None else None
    if op == "combine_backward":
        return (rows[:-1], d_w) if d_w is not None else rows[:-1]
    out = (picked * w).sum(1).to(s["rows"].dtype)
    return (out, d_w) if op == "dispatch_backward" and d_w is not None else out


def _plain_route(s):
    case = s["case"]
    T, E, S = case["T"], case["E"], case["S"]
    cols = torch.cat([s["idx"].long(), torch.arange(E, E + S, device="cuda").expand(T, S)], 1)
    z = s["logits"].float().gather(1, cols)
    d_w = torch.cat([s["d_w"], s["d_sink"]], 1)
    c = 2.5 * s["global_scale"] if S else 1.0
    p = torch.softmax(torch.nn.functional.logsigmoid(z) if S else z, 1)
    d_z = c * p * (d_w - (p * d_w).sum(1, keepdim=True))
    if S:
        d_z = d_z * torch.sigmoid(-z)
    d_logits = torch.zeros(T, E + S, device="cuda").scatter_(1, cols, d_z).to(s["logits"].dtype)
    return (d_logits, 2.5 * (p.double() * d_w.double()).sum().float().view(1)) if S else d_logits


def _plain_int8(s):
    case = s["case"]
    T, E, k, K = case["T"], case["E"], case["k"], s["a"].shape[1]
    gate_up = case["part"] == "gate_up"
    a = s["a"].float()
    top = a.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(a * 127 / top), 0.0)
    scale = top / 127
    if gate_up:  # tokens to their sorted rows
        rows = torch.empty(T * k, dtype=torch.long, device="cuda")
        rows[s["inverse"].long()] = torch.arange(T * k, device="cuda") // k
        q, scale = q[rows], scale[rows]
    # every expert's rows, padded to the longest segment
    pos = s["offsets"][:-1, None].long() + torch.arange(s["most"], device="cuda")
    live = pos < s["offsets"][1:, None]
    pos = torch.where(live, pos, T * k)
    acc = torch.bmm(q[pos.clamp(max=T * k - 1)], s["w_q"][:, :, :K].float().transpose(1, 2))
    y = acc * scale[pos.clamp(max=T * k - 1)] * s["w_scales"][:, None, :]
    if s["bias"] is not None:
        y = y + s["bias"][:, None, :].float()
    if gate_up:
        g, u = y.chunk(2, dim=2) if case["fmt"] == "concatenated" else (y[..., 0::2], y[..., 1::2])
        y = _act(case["act"], g, u)
    out = torch.zeros(T * k + 1, y.shape[2], dtype=torch.bfloat16, device="cuda")
    out[pos] = y.to(torch.bfloat16)
    return out[:-1]


def _config(s):
    """The layer's configuration, made once as a program keeps it."""
    from mixture_experts_ffn_token_b200 import abi
    if "cfg" not in s:
        c = s["case"]
        swiglu = c.get("act") == "swigluoai"
        s["cfg"] = abi.config(c["T"], c.get("H", 64), c["E"], c["k"], c.get("D", 64),
                              router="sigmoid_sink" if c.get("S") else "softmax_topk", num_sink=c.get("S", 0),
                              logits_dtype=getattr(torch, c.get("dtype", F32)) if c["op"] == "route_backward" else torch.float32,
                              route_scale=2.5 if c.get("S") else 1.0,
                              gate_up_format=c.get("fmt", "concatenated"), activation=c.get("act", "silu"),
                              alpha=_ALPHA if swiglu else 0.0, limit=_LIMIT if swiglu else 0.0,
                              has_bias=c.get("bias", False))
        s["ws"] = torch.empty(abi.moe_operator_workspace_size(s["cfg"]), dtype=torch.uint8, device="cuda")
    return abi, s["cfg"]


def _own_rows(s):
    abi, cfg = _config(s)
    op, w = s["case"]["op"], s["w"]
    d_w = s["d_w"] if w is not None else None
    if op == "dispatch":
        abi.moe_dispatch(cfg, s["tokens"], s["inverse"], s["out_rows"], expert_weights=w)
        return s["out_rows"]
    if op == "combine":
        abi.moe_combine(cfg, s["rows"], s["inverse"], s["out_tokens"], expert_weights=w)
        return s["out_tokens"]
    if op == "dispatch_backward":
        abi.moe_dispatch_backward(cfg, s["rows"], s["inverse"], s["out_tokens"], x=s["tokens"] if w is not None else None,
                                  expert_weights=w, d_expert_weights=d_w)
        return (s["out_tokens"], d_w) if w is not None else s["out_tokens"]
    abi.moe_combine_backward(cfg, s["tokens"], s["inverse"], s["out_rows"], rows=s["rows"] if w is not None else None,
                             expert_weights=w, d_expert_weights=d_w)
    return (s["out_rows"], d_w) if w is not None else s["out_rows"]


def _own_route(s):
    abi, cfg = _config(s)
    if s["case"]["S"]:
        abi.moe_route_backward(cfg, s["logits"], s["idx"], s["d_w"], s["d_logits"], d_sink_weights=s["d_sink"],
                               global_scale=s["global_scale"], d_global_scale=s["d_global_scale"], workspace=s["ws"])
        return s["d_logits"], s["d_global_scale"]
    abi.moe_route_backward(cfg, s["logits"], s["idx"], s["d_w"], s["d_logits"])
    return s["d_logits"]


def _own_int8(s):
    abi, cfg = _config(s)
    if s["case"]["part"] == "gate_up":
        abi.moe_dispatch_int8(cfg, s["a"], s["inverse"], s["rows_q"], s["row_scales"])
    else:
        abi.moe_quantize_rows(cfg, s["a"], s["offsets"], s["rows_q"], s["row_scales"])
    abi.moe_grouped_linear_int8(cfg, s["case"]["part"], s["rows_q"], s["row_scales"], s["w_q"], s["w_scales"],
                                s["offsets"], s["out"], s["ws"], bias=s["bias"])
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if op == "route_backward":
        return _own_route(state) if own else _plain_route(state)
    if op == "int8":
        return _own_int8(state) if own else _plain_int8(state)
    return _own_rows(state) if own else _plain_rows(state)


# ------------------------------------------------------------ work and truth
def work(case):
    T, E, k, op = case["T"], case["E"], case["k"], case["op"]
    R = T * k
    if op == "route_backward":
        S, size = case["S"], 2 if case["dtype"] == BF16 else 4
        n = k + S
        return {"bytes": T * (n * (size + 4) + k * 4 + (E + S) * size), "flops": T * n * 12}
    if op == "int8":
        gate_up = case["part"] == "gate_up"
        K, N = (case["H"], 2 * case["D"]) if gate_up else (case["D"], case["H"])
        # how many experts the batch reaches, on average: an expert's chance of
        # being among a token's k is min(1, c * popularity), where these sum to k
        p = [(r + 1.0) ** -1.2 if case["zipf"] else 1.0 for r in range(E)]
        lo, hi = 0.0, 1e6
        for _ in range(60):
            c = 0.5 * (lo + hi)
            lo, hi = (c, hi) if sum(min(1.0, c * q) for q in p) < k else (lo, c)
        used = sum(1 - (1 - min(1.0, hi * q)) ** T for q in p)
        weights = int(used * N * (K + 4 + (2 if case["bias"] else 0)))
        rows = (T if gate_up else R) * K * 2 + R * (case["D"] if gate_up else N) * 2 + (R * 4 if gate_up else 0)
        return {"bytes": weights + rows + 4 * (E + 1), "flops": 2 * R * K * N}
    H, size = case["H"], 2 if case["dtype"] == BF16 else 4
    n, w = T * H * size, R * 4 if case["weighted"] else 0
    rows = int(R * (1 - case["drop"])) * H * size
    moved = n + rows
    if case["weighted"] and op == "dispatch_backward":
        moved += n + R * 4
    if case["weighted"] and op == "combine_backward":
        moved += rows + R * 4
    return {"bytes": moved + w + R * 4, "flops": 4 * R * H}


def exact(case, seed):
    s = prepare(case, seed)
    T, E, k, op = case["T"], case["E"], case["k"], case["op"]
    f64 = torch.float64
    if op == "route_backward":
        S = case["S"]
        out = torch.zeros(T, E + S, dtype=f64, device="cuda")
        z = torch.stack([s["logits"][torch.arange(T, device="cuda"), s["idx"][:, j].long()] for j in range(k)]
                        + [s["logits"][:, E + i] for i in range(S)], 1).to(f64)
        d_w = torch.cat([s["d_w"], s["d_sink"]], 1).to(f64)
        e = 1 / (1 + torch.exp(-z)) if S else torch.exp(z)
        p = e / e.sum(1, keepdim=True)
        c = 2.5 * s["global_scale"].to(f64) if S else torch.ones(1, dtype=f64, device="cuda")
        for j in range(k + S):
            d_z = c * p[:, j] * (d_w[:, j] - (p * d_w).sum(1))
            if S:
                d_z = d_z * (1 - e[:, j])
            col = s["idx"][:, j].long() if j < k else torch.full((T,), E + j - k, device="cuda")
            out[torch.arange(T, device="cuda"), col] += d_z
        return (out, 2.5 * (p * d_w).sum().view(1)) if S else out
    if op == "int8":
        gate_up = case["part"] == "gate_up"
        K = s["a"].shape[1]
        out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
        if gate_up:
            token = torch.zeros(T * k, dtype=torch.long, device="cuda")
            token[s["inverse"].long()] = torch.arange(T * k, device="cuda") // k
        for e in range(E):
            lo, hi = int(s["offsets"][e]), int(s["offsets"][e + 1])
            if lo == hi:
                continue
            a = (s["a"][token[lo:hi]] if gate_up else s["a"][lo:hi]).to(f64)
            top = a.abs().max(1, keepdim=True).values
            y = torch.round(a * 127 / top) @ s["w_q"][e, :, :K].to(f64).T
            y = y * (top / 127) * s["w_scales"][e].to(f64)
            if s["bias"] is not None:
                y = y + s["bias"][e].to(f64)
            if gate_up:
                D = case["D"]
                g, u = (y[:, :D], y[:, D:]) if case["fmt"] == "concatenated" else (y[:, 0::2], y[:, 1::2])
                if case["act"] == "silu":
                    y = g / (1 + torch.exp(-g)) * u
                elif case["act"] == "swigluoai":
                    g, u = torch.minimum(g, torch.full_like(g, _LIMIT)), torch.clip(u, -_LIMIT, _LIMIT)
                    y = g / (1 + torch.exp(-_ALPHA * g)) * (1 + u)
                else:
                    y = g / (1 + torch.exp(-2 * 0.7978845608028654 * (g + 0.044715 * g ** 3))) * u
            out[lo:hi] = y
        return out
    tokens, rows = s["tokens"].to(f64), s["rows"].to(f64)
    out_tokens, out_rows = torch.zeros_like(tokens), torch.zeros_like(rows)
    d_w = torch.zeros(T, k, dtype=f64, device="cuda")
    for j in range(k):
        p = s["inverse"].view(T, k)[:, j].long()
        t = torch.nonzero(p >= 0).view(-1)
        p = p[t]
        w = s["w"][t, j].to(f64).unsqueeze(1) if s["w"] is not None else 1.0
        out_tokens[t] += w * rows[p]
        out_rows[p] = w * tokens[t]
        d_w[t, j] = torch.einsum("th,th->t", tokens[t], rows[p])
    if op == "dispatch":
        return out_rows
    if op == "combine":
        return out_tokens
    out = out_tokens if op == "dispatch_backward" else out_rows
    return (out, d_w) if s["w"] is not None else out
