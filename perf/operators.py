"""Cases and plain forms of the operators around the int8 linears of a decoder layer.

  norm     residual addition + root-mean-square norm + int8 codes with one scale per token (qa_rmsnorm_int8)
  route    a token's experts: scores, balance bias, groups, top-k, weights, and the pairs in expert order
           (qa_route_experts)
  experts  the gated feed-forward of the chosen experts on int8 codes, summed per token (qa_experts_int8)
  lora     a shared int8 projection with the low-rank adapters of many requests (qa_qlinear_int8_lora)

`run` computes a case in its plain form (elementary torch operations in 32 bits, one rounding at the end), or,
with `own` set, by the library's entry points.  `exact` computes it in 64 bits, apart from both.
"""
import math

import torch

own = False

DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
DTYPES = {"f16": F16, "bf16": BF16, "f32": F32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one request between two projections: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "K": 4096, "dtype": "f16", "residual": True, "y": True},
        # a 2048-token prompt at the hidden size 4096, the sum and the 16-bit norm kept for the next blocks
        {"name": "norm_prompt", "op": "norm", "rows": 2048, "K": 4096, "dtype": "f16", "residual": True, "y": True},
        # a full batch of packed prompts at the hidden size 8192, codes only
        {"name": "norm_batch", "op": "norm", "rows": 16384, "K": 8192, "dtype": "bf16", "residual": True, "y": False},
        # one decoding step of 32 requests
        {"name": "route_step", "op": "route", "T": 32, "E": 64, "k": 6, "dtype": "f32", "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renorm": False, "scale": 1.0},
        # prompts through many experts in groups, sigmoid scores with the balance bias
        {"name": "route_grouped", "op": "route", "T": 4096, "E": 256, "k": 8, "dtype": "f32", "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5},
        # a full batch of packed prompts, 16-bit logits, an odd number of tokens
        {"name": "route_batch", "op": "route", "T": 50001, "E": 128, "k": 8, "dtype": "bf16", "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renorm": True, "scale": 1.0},
        # one decoding step of 8 requests: every active expert's weights are read for a row or two
        {"name": "experts_step", "op": "experts", "T": 8, "E": 64, "k": 8, "K": 4096, "F": 1024, "dtype": "f16"},
        # a decoding step of many requests, or a short prompt: about 32 rows for each expert
        {"name": "experts_chunk", "op": "experts", "T": 256, "E": 64, "k": 8, "K": 4096, "F": 1024, "dtype": "bf16"},
        # packed prompts, an odd number of tokens: the products bound it
        {"name": "experts_prompt", "op": "experts", "T": 4099, "E": 32, "k": 4, "K": 4096, "F": 2048,
         "dtype": "f16"},
        # one decoding step of 16 requests, each with its adapter
        {"name": "lora_step", "op": "lora", "M": 16, "K": 4096, "N": 4096, "r": 16, "L": 16, "R": 16,
         "dtype": "f16"},
        # decoding requests beside chunks of prompts, ragged, many adapters of a high rank
        {"name": "lora_mixed", "op": "lora", "M": 777, "K": 4096, "N": 4096, "r": 64, "L": 32, "R": 48,
         "dtype": "bf16"},
        # 2048 tokens of a few prompts through the up projection of the prefill workload
        {"name": "lora_prompt", "op": "lora", "M": 2048, "K": 4096, "N": 11008, "r": 16, "L": 8, "R": 8,
         "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "experts", "lora"])
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 16384), "K": rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024)]),
                "dtype": rng.choice(["f16", "bf16", "f32"]), "residual": rng.random() < 0.7, "y": rng.random() < 0.5}
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, 8 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * top_groups))
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "T": _log(rng, 1, 50000), "E": E, "k": k, "dtype": rng.choice(["f16", "bf16", "f32"]),
                "score": score, "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups,
                "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5])}
    if op == "experts":
        K, F, E = 16 * _log(rng, 8, 256), 16 * _log(rng, 8, 128), _log(rng, 2, 64)
        k = rng.randint(1, min(8, E))
        return {"op": op, "T": _log(rng, 1, 16384 // k), "E": E, "k": k, "K": K, "F": F,
                "dtype": rng.choice(["f16", "bf16", "f32"])}
    R = _log(rng, 1, 64)
    return {"op": op, "M": _log(rng, 1, 2048), "K": 16 * _log(rng, 8, 256), "N": _log(rng, 64, 11008),
            "r": rng.choice([8, 16, 24, 32, 64, 128]), "L": _log(rng, 1, 32), "R": R,
            "dtype": rng.choice(["f16", "bf16"])}


def work(case):
    c, op = case, case["op"]
    if op == "norm":
        n, b = c["rows"] * c["K"], SIZE[c["dtype"]]
        reads = n * b * (2 if c["residual"] else 1) + c["K"] * b
        writes = n + 4 * c["rows"] + n * b * (int(c["residual"]) + int(c["y"]))
        return {"bytes": reads + writes, "flops": 6 * n}
    if op == "route":
        n, p = c["T"] * c["E"], c["T"] * c["k"]
        return {"bytes": n * SIZE[c["dtype"]] + 12 * p + 8 * c["E"], "flops": 4 * n}
    if op == "experts":
        pairs = c["T"] * c["k"]
        active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])
        rows = c["T"] * (c["K"] * (1 + SIZE[c["dtype"]]) + 4) + 8 * pairs
        return {"bytes": active * (3 * c["F"] * c["K"] + 4 * (2 * c["F"] + c["K"])) + rows,
                "flops": 6 * pairs * c["F"] * c["K"]}
    used = min(c["L"], c["R"])
    rows = c["M"] * (c["K"] * (1 + SIZE[c["dtype"]]) + 4 + c["N"] * SIZE[c["dtype"]])
    return {"bytes": rows + c["N"] * (c["K"] + 4) + used * c["r"] * (c["K"] + c["N"]) * SIZE[c["dtype"]],
            "flops": 2 * c["M"] * (c["N"] * c["K"] + c["r"] * (c["K"] + c["N"]))}


# ---------------------------------------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, device=DEV, generator=g) * std


def _uniform(g, *shape, lo=0.0, hi=1.0):
    return torch.rand(*shape, device=DEV, generator=g) * (hi - lo) + lo


def _codes(g, *shape):
    """int8 codes of normal values quantized by absmax: about 4 standard deviations reach 127."""
    return torch.randn(*shape, device=DEV, dtype=F16, generator=g).mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)


def prepare(case, seed):
    g = _gen(seed)
    return {"norm": _prepare_norm, "route": _prepare_route, "experts": _prepare_experts,
            "lora": _prepare_lora}[case["op"]](dict(case), g)


def _prepare_norm(c, g):
    rows, K, dt = c["rows"], c["K"], DTYPES[c["dtype"]]
    # activations with a few large feature dimensions, as they meet in front of a quantized linear
    dims = 1.0 + 20.0 * (_uniform(g, K) < 6.0 / K).float()
    c["X"] = (_normal(g, rows, K) * dims).to(dt)
    c["res"] = (_normal(g, rows, K, std=3.0) * dims).to(dt) if c["residual"] else None
    c["w"] = _uniform(g, K, lo=0.2, hi=1.8).to(dt)
    return c


def _choice_scores(logits, c, bias, to):
    """What experts are chosen by, [T x E] in `to`, masked experts at -inf; and whether it is the logits themselves."""
    x = logits.to(to)
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=torch.finfo(to).min))
        s = e / e.sum(1, keepdim=True)
    b = s if bias is None else s + bias.to(to)
    return s, b.masked_fill(torch.isneginf(x), -math.inf)


def _prepare_route(c, g):
    T, E, dt = c["T"], c["E"], DTYPES[c["dtype"]]
    bias = _normal(g, E, std=0.05) if c["bias"] else None
    spread = _normal(g, E, std=0.5)                          # some experts are liked more than others
    logits = (_normal(g, T, E, std=1.5) + spread).to(dt)
    # Two experts whose unequal scores lie within a few roundings of 32 bits can come in either order, and so can two
    # groups: such rows take another row's logits, so that the order is one that 32 bits can tell.
    tied = torch.zeros(T, dtype=torch.bool, device=DEV)
    _, ch = _choice_scores(logits, c, bias, torch.float64)
    group = ch.view(T, c["groups"], -1).sort(2).values[:, :, -c["group_top"]:].sum(2)
    for v in (ch, group):
        v = v.sort(1).values
        d = v[:, 1:] - v[:, :-1]
        tied |= ((d > 0) & (d < 2e-6 * v[:, 1:].abs().clamp(min=0.02))).any(1)
    good = torch.nonzero(~tied)[:, 0]
    if good.numel():
        pick = good[(torch.arange(T, device=DEV) * 7) % good.numel()]
        logits = torch.where(tied[:, None], logits[pick], logits)
    pad = _uniform(g, T) < 1.0 / 64                          # padding tokens: every expert masked
    pad[0] = False
    c["logits"] = logits.masked_fill(pad[:, None], -math.inf)
    c["b"] = bias
    return c


def _dispatch(ids, E):
    """The pairs t * k + j with an expert, ordered by expert and then by pair (-1 after them), and each expert's start."""
    flat = ids.reshape(-1).to(torch.int64)
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0) if key.numel() * E < 1 << 26 else \
        torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = torch.where(torch.arange(order.numel(), device=key.device) < offsets[E], order, -1)
    return order.to(torch.int32), offsets.to(torch.int32)


def _prepare_experts(c, g):
    T, E, k, K, F = c["T"], c["E"], c["k"], c["K"], c["F"]
    liked = _normal(g, T, E) + _normal(g, E, std=0.5)
    ids = liked.topk(k, 1).indices.to(torch.int32)
    pad = _uniform(g, T) < 1.0 / 64                          # padding tokens have no expert
    pad[0] = False
    ids = ids.masked_fill(pad[:, None], -1)
    w = _uniform(g, T, k, lo=0.2, hi=1.0)
    c["w"] = (w / w.sum(1, keepdim=True)).masked_fill(ids < 0, 0.0)
    c["order"], c["offsets"] = _dispatch(ids, E)
    c["Xq"], c["s_x"] = _codes(g, T, K), _uniform(g, T, lo=0.5, hi=1.5) / 32
    c["W13"] = torch.stack([_codes(g, 2 * F, K) for _ in range(E)])
    c["W2"] = torch.stack([_codes(g, K, F) for _ in range(E)])
    c["s13"] = _uniform(g, E, 2 * F, lo=0.5, hi=1.5) * (0.02 / 32)
    c["s2"] = _uniform(g, E, K, lo=0.5, hi=1.5) * (0.02 / 32)
    c["starts"] = c["offsets"].tolist()                      # for the plain form's loop over experts
    return c


def _prepare_lora(c, g):
    M, K, N, r, L, R, dt = c["M"], c["K"], c["N"], c["r"], c["L"], c["R"], DTYPES[c["dtype"]]
    X = _normal(g, M, K).to(dt)
    c["X"] = X
    c["s_x"] = X.float().abs().amax(1) / 127
    c["Xq"] = torch.round(X.float() / c["s_x"][:, None]).clamp(-127, 127).to(torch.int8)
    c["Wq"], c["s_w"] = _codes(g, N, K), _uniform(g, N, lo=0.5, hi=1.5) * (0.02 / 32)
    c["A"] = _normal(g, L, r, K, std=K ** -0.5).to(dt)
    c["B"] = _normal(g, L, N, r, std=0.05).to(dt)
    c["alpha"] = _uniform(g, L, lo=0.5, hi=2.0)
    # as many requests as tokens: one token each; else requests of all lengths, empty ones among them
    if M == R:
        cuts = torch.arange(R + 1, device=DEV)
    else:
        cuts = torch.cat([torch.zeros(1, device=DEV), _uniform(g, R).square().cumsum(0)])
        cuts = (cuts / cuts[-1] * M).round().long()
    c["seg"] = cuts.to(torch.int32)
    which = torch.randint(0, L, (R,), device=DEV, generator=g)
    none = _uniform(g, R) < 1.0 / 16                         # a request without an adapter
    none[0] = False
    c["which"] = which.masked_fill(none, -1).to(torch.int32)
    return c


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def _own_norm(c):
    import bit_quantized_linear_int8_amd as qa
    q, s, total, y = qa.qa_rmsnorm_int8(c["X"], c["w"], residual=c["res"], eps=EPS, want_y=c["y"])
    return {"x": _values(q, s), "s": s, "total": total, "y": y}


def _own_route(c):
    import bit_quantized_linear_int8_amd as qa
    score = qa.QA_SCORE_SIGMOID if c["score"] == "sigmoid" else qa.QA_SCORE_SOFTMAX
    ids, w, order, offsets = qa.qa_route_experts(
        c["logits"], c["k"], bias=c["b"], score=score, groups=c["groups"], top_groups=c["top_groups"],
        group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"])
    return {"ids": ids, "w": w, "order": order, "offsets": offsets}


def _own_experts(c):
    import bit_quantized_linear_int8_amd as qa
    return qa.qa_experts_int8(c["Xq"], c["s_x"], c["w"], c["order"], c["offsets"], c["W13"], c["s13"], c["W2"],
                              c["s2"], out_dtype=DTYPES[c["dtype"]])


def _own_lora(c):
    import bit_quantized_linear_int8_amd as qa
    return qa.qa_qlinear_int8_lora(c["Xq"], c["s_x"], c["X"], c["Wq"], c["s_w"], c["A"], c["B"], c["alpha"], c["seg"],
                                   c["which"], out_dtype=DTYPES[c["dtype"]])


def _values(q, s):
    """The values that int8 codes stand for, in fp16."""
    return torch.mul(q, s[:, None], out=torch.empty(q.shape, dtype=F16, device=q.device))


def _scale(a):
    """absmax / 127 per row, 1 for a row of zeros."""
    s = a.abs().amax(1) / 127
    return torch.where(s > 0, s, torch.ones_like(s))


def _plain_norm(c):
    dt = DTYPES[c["dtype"]]
    h = c["X"].float()
    if c["res"] is not None:
        h = h + c["res"].float()
    y = h * (1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)) * c["w"].float()
    s = _scale(y)
    q = torch.round(y / s[:, None]).clamp(-127, 127)
    return {"x": _values(q, s), "s": s, "total": h.to(dt) if c["res"] is not None else None,
            "y": y.to(dt) if c["y"] else None}


def _select(s, ch, c):
    """The chosen experts by `ch` (ties to the lower index, -1 where none is left) and their weights out of `s`."""
    T, E = ch.shape
    if c["groups"] > 1:
        by = ch.view(T, c["groups"], -1)
        top = by.sort(dim=2, descending=True).values[:, :, : c["group_top"]]
        # a masked expert adds nothing to its group, and a group of masked experts comes last
        value = top.masked_fill(torch.isneginf(top), 0.0).sum(2).masked_fill(torch.isneginf(top[:, :, 0]), -math.inf)
        rank = value.sort(dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=ch.device).scatter_(1, rank, True)
        ch = by.masked_fill(~keep[:, :, None], -math.inf).view(T, E)
    v, at = ch.sort(dim=1, descending=True, stable=True)
    v, at = v[:, : c["k"]], at[:, : c["k"]]
    none = torch.isneginf(v)
    w = s.gather(1, at).masked_fill(none, 0.0)
    if c["renorm"]:
        t = w.sum(1, keepdim=True)
        w = torch.where(t > 0, w / t, w)
    return at.masked_fill(none, -1).to(torch.int32), w * c["scale"]


def _plain_route(c):
    s, ch = _choice_scores(c["logits"], c, c["b"], F32)
    if c["score"] == "softmax" and c["b"] is None and (c["groups"] == 1 or c["group_top"] == 1):
        ch = c["logits"].float()                             # the same order, before rounding
    ids, w = _select(s, ch, c)
    order, offsets = _dispatch(ids, c["E"])
    return {"ids": ids, "w": w, "order": order, "offsets": offsets}


def _experts(c, to, out_dtype):
    T, k, K, F = c["T"], c["k"], c["K"], c["F"]
    y = torch.zeros(T * k, K, dtype=to, device=DEV)
    for e in range(c["E"]):
        a, b = c["starts"][e], c["starts"][e + 1]
        if a == b:
            continue
        pair = c["order"][a:b].long()
        x = c["Xq"][pair // k].to(to) * c["s_x"][pair // k].to(to)[:, None]
        gu = x @ (c["W13"][e].to(to) * c["s13"][e].to(to)[:, None]).t()
        h = gu[:, :F] / (1.0 + torch.exp(-gu[:, :F])) * gu[:, F:]
        s = _scale(h)
        hq = torch.round(h / s[:, None]).clamp(-127, 127) * s[:, None]
        y[pair] = hq @ (c["W2"][e].to(to) * c["s2"][e].to(to)[:, None]).t()
    return (y.view(T, k, K) * c["w"].to(to)[:, :, None]).sum(1).to(out_dtype)


def _plain_experts(c):
    return _experts(c, F32, DTYPES[c["dtype"]])


def _adapter_of_token(c):
    t = torch.arange(c["M"], device=DEV, dtype=torch.int32)
    at = torch.searchsorted(c["seg"], t, right=True) - 1     # the last request that starts at or before the token
    return torch.where(t < c["seg"][-1], c["which"][at.clamp(0, c["R"] - 1)], -1).long()


def _plain_lora(c):
    M, N, r, L = c["M"], c["N"], c["r"], c["L"]
    base = (c["Xq"].float() @ c["Wq"].float().t()) * c["s_x"][:, None] * c["s_w"]
    # every adapter on every token, and then each token's own alone
    h = (c["X"].float() @ c["A"].float().view(L * r, -1).t()).view(M, L, r)
    mine = _adapter_of_token(c)[:, None] == torch.arange(L, device=DEV)
    h = torch.where(mine[:, :, None], h * c["alpha"][:, None], torch.zeros_like(h)).view(M, L * r)
    return (base + h @ c["B"].float().transpose(1, 2).reshape(L * r, N)).to(DTYPES[c["dtype"]])


_OWN = {"norm": _own_norm, "route": _own_route, "experts": _own_experts, "lora": _own_lora}
_PLAIN = {"norm": _plain_norm, "route": _plain_route, "experts": _plain_experts, "lora": _plain_lora}


# ------------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = prepare(case, seed)
    D = torch.float64
    if c["op"] == "norm":
        h = c["X"].to(D) + (0.0 if c["res"] is None else c["res"].to(D))
        y = h * c["w"].to(D) / (h.pow(2).sum(1, keepdim=True) / c["K"] + EPS).sqrt()
        s = y.abs().max(1).values / 127
        s[s == 0] = 1.0
        x = (y / s[:, None]).round() * s[:, None]
        return {"x": x, "s": s, "total": h if c["residual"] else None, "y": y if c["y"] else None}
    if c["op"] == "route":
        return _exact_route(c, D)
    if c["op"] == "experts":
        return _exact_experts(c, D)
    out = torch.empty(c["M"], c["N"], dtype=D, device=DEV)
    for m0 in range(0, c["M"], 512):
        rows = slice(m0, m0 + 512)
        out[rows] = (c["Xq"][rows].to(D) @ c["Wq"].to(D).T) * (c["s_x"][rows].to(D)[:, None] * c["s_w"].to(D)[None])
    cuts, which = c["seg"].tolist(), c["which"].tolist()
    for i in range(c["R"]):
        if which[i] >= 0 and cuts[i + 1] > cuts[i]:
            rows, a = slice(cuts[i], cuts[i + 1]), which[i]
            out[rows] += float(c["alpha"][a]) * ((c["X"][rows].to(D) @ c["A"][a].to(D).T) @ c["B"][a].to(D).T)
    return out


def _exact_route(c, D):
    x = c["logits"].to(D)
    dead = x == -math.inf
    if c["score"] == "sigmoid":
        s = torch.sigmoid(x)
    else:
        s = torch.softmax(x, 1).masked_fill(dead, 0.0)
    ch = s + (0.0 if c["b"] is None else c["b"].to(D))
    low = -1e300
    ch = ch.masked_fill(dead, low)
    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        part = [ch[:, i * size:(i + 1) * size] for i in range(c["groups"])]
        value = []
        for p in part:
            best = p.sort(dim=1, descending=True).values[:, : c["group_top"]]
            value.append(torch.where(best > low, best, 0.0).sum(1).masked_fill(best[:, 0] <= low, low))
        value = torch.stack(value, 1)
        for i, p in enumerate(part):                         # groups that come before this one: larger, or as large and lower
            before = (value > value[:, i:i + 1]).sum(1) + (value[:, :i] == value[:, i:i + 1]).sum(1)
            p.masked_fill_((before >= c["top_groups"])[:, None], low)
    left, w = ch.clone(), []
    for _ in range(c["k"]):
        best = left.max(1).values
        at = (left == best[:, None]).int().argmax(1)
        w.append(torch.where(best > low, s.gather(1, at[:, None])[:, 0], 0.0))
        left.scatter_(1, at[:, None], low)
    w = torch.stack(w, 1)
    if c["renorm"]:
        t = w.sum(1, keepdim=True)
        w = w / torch.where(t > 0, t, 1.0)
    return {"ids": None, "w": w * c["scale"], "order": None, "offsets": None}


def _exact_experts(c, D):
    k, F = c["k"], c["F"]
    out = torch.zeros(c["T"], c["K"], dtype=D, device=DEV)
    for e in range(c["E"]):
        pair = c["order"][c["starts"][e]:c["starts"][e + 1]].long()
        t = pair // k
        if not t.numel():
            continue
        gu = (c["Xq"][t].to(D) @ c["W13"][e].to(D).T) * (c["s_x"][t].to(D)[:, None] * c["s13"][e].to(D)[None])
        h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        s = h.abs().max(1).values / 127
        s[s == 0] = 1.0
        v = ((h / s[:, None]).round() @ c["W2"][e].to(D).T) * (s[:, None] * c["s2"][e].to(D)[None])
        out.index_add_(0, t, v * c["w"].view(-1)[pair].to(D)[:, None])
    return out
