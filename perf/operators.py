"""What the 8-bit integer products and the routing to experts are measured on.

The operators are those of a layer of expert MLPs whose weights and
activations are held in 8-bit integers: a router picks k of E experts for each
token, a plan sorts the (token, choice) slots by expert, the activations are
quantized to int8 with one scale per token, the experts' products run over the
sorted rows against int8 weights with one scale per output channel, and the
experts' outputs are weighted and summed per token.  The dense product is the
same product with one expert.  Where ``own`` is false, run() computes them with
elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda:0"

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # ---- routing: scores, top-k, weights and the plan of the sorted slots
        # one token of a serving step
        {"name": "route_1_of_64", "op": "route", "tokens": 1, "experts": 64, "k": 4, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_top": 1, "type": "fp32"},
        # a prompt, sigmoid scores with a balance bias, experts in groups
        {"name": "route_16384_of_128_groups", "op": "route", "tokens": 16384, "experts": 128, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 4, "top_groups": 2, "group_top": 2, "type": "fp32"},
        # the router's gradient for an odd batch of training tokens
        {"name": "route_backward_8191", "op": "route_backward", "tokens": 8191, "experts": 128, "k": 8,
         "score": "softmax", "type": "bf16"},
        # ---- activations to int8 with a scale per token
        # the rows of a decode step
        {"name": "quantize_16x8192", "op": "quantize", "rows": 16, "K": 8192, "type": "bf16"},
        # a prompt's hidden layer, before the down projection
        {"name": "quantize_8192x14336", "op": "quantize", "rows": 8192, "K": 14336, "type": "bf16"},
        # ---- int8 product, scales per token and channel
        # a decode step of 16 tokens
        {"name": "product_16x28672x8192", "op": "product", "M": 16, "N": 28672, "K": 8192, "bias": False, "act": False,
         "type": "bf16"},
        # an odd number of tokens, ragged sizes, fp32 output
        {"name": "product_777x4100x2064", "op": "product", "M": 777, "N": 4100, "K": 2064, "bias": True, "act": False,
         "type": "fp32"},
        # a prompt's up projection with bias and GELU
        {"name": "product_8192x14336x4096", "op": "product", "M": 8192, "N": 14336, "K": 4096, "bias": True, "act": True,
         "type": "bf16"},
        # ---- experts' products over the sorted slots
        # 16 tokens of a serving step over 64 experts: about one row for each
        {"name": "experts_16_of_64_2048x4096", "op": "grouped", "tokens": 16, "k": 4, "experts": 64, "N": 2048, "K": 4096,
         "bias": False, "act": False, "type": "bf16"},
        # a prompt over 16 experts
        {"name": "experts_4096_of_16_4096x2048", "op": "grouped", "tokens": 4096, "k": 4, "experts": 16, "N": 4096,
         "K": 2048, "bias": True, "act": True, "type": "bf16"},
        # ---- experts' outputs weighted and summed per token, and its gradient
        {"name": "combine_8192x4096", "op": "combine", "tokens": 8192, "k": 4, "N": 4096, "type": "bf16"},
        {"name": "combine_backward_2047x4096", "op": "combine_backward", "tokens": 2047, "k": 8, "N": 4096, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _experts(rng):
    """Experts, choices per token and groups of a router."""
    groups = rng.choice([1, 1, 2, 4, 8])
    experts = groups * _log(rng, 4, 512 // groups)
    top_groups = rng.randint(1, groups)
    k = _log(rng, 1, min(16, experts // groups * top_groups))
    return experts, k, groups, top_groups


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "quantize", "product", "product", "grouped", "grouped", "combine",
                     "combine_backward"])
    kind = rng.choice(["fp32", "bf16", "fp16"])
    if op == "route":
        experts, k, groups, top_groups = _experts(rng)
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "k": k,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": top_groups, "group_top": rng.choice([1, 2]), "type": kind}
    if op == "route_backward":
        experts, k, _, _ = _experts(rng)
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "k": k,
                "score": rng.choice(["softmax", "sigmoid"]), "type": kind}
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "K": 16 * _log(rng, 4, 896), "type": kind}
    if op == "product":
        M, N, K = _log(rng, 1, 8192), _log(rng, 16, 14336), 16 * _log(rng, 4, 512)
        return {"op": op, "M": M, "N": N, "K": K if M * N * K <= 8192 * 14336 * 4096 else 4096, "bias": rng.random() < 0.5,
                "act": rng.random() < 0.5, "type": kind}
    if op == "grouped":
        experts = _log(rng, 2, 64)
        return {"op": op, "tokens": _log(rng, 1, 4096), "k": _log(rng, 1, min(8, experts)), "experts": experts,
                "N": _log(rng, 64, 4096), "K": 16 * _log(rng, 4, 256), "bias": rng.random() < 0.5, "act": rng.random() < 0.5,
                "type": kind}
    return {"op": op, "tokens": _log(rng, 1, 4096), "k": _log(rng, 1, 8), "N": _log(rng, 64, 8192), "type": kind}


# ---- inputs -----------------------------------------------------------------


def _codes(x):
    """Rows quantized to int8 with one scale each, as a user holds weights and activations."""
    s = (x.abs().amax(-1, keepdim=True).double() / 127.0).float()
    return torch.round(x / s).clamp_(-127, 127).to(torch.int8), s.squeeze(-1)


def _router_logits(g, tokens, experts, kind):
    """Logits with some experts more popular than others."""
    x = torch.randn(tokens, experts, generator=g, device=DEV)
    return (x + 0.3 * torch.randn(experts, generator=g, device=DEV)).to(kind)


def _plan(ids, experts):
    """Offsets of the experts' rows, slots in order of their expert, and each slot's row."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    edges = torch.arange(experts + 1, device=flat.device)
    offsets = (flat[None, :] < edges[:, None]).sum(1)
    position = torch.empty_like(order)
    position[order] = torch.arange(flat.numel(), device=flat.device)
    return offsets.int(), order.int(), position.int().view(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kind = TYPES[case["type"]]
    st = dict(case)
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        st["logits"] = _router_logits(g, T, E, kind)
        if op == "route":
            st["bias"] = 0.05 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        else:
            st["ids"] = torch.sort(st["logits"].float(), dim=-1, descending=True, stable=True).indices[:, :k].int().contiguous()
            st["d_weights"] = torch.randn(T, k, generator=g, device=DEV)
    elif op == "quantize":
        x = torch.randn(case["rows"], case["K"], generator=g, device=DEV)
        outlier = torch.rand(case["K"], generator=g, device=DEV) < 0.002
        st["x"] = (x * (1.0 + 19.0 * outlier)).to(kind)
    elif op in ("product", "grouped"):
        N, K = case["N"], case["K"]
        E = case["experts"] if op == "grouped" else 1
        rows = case["tokens"] if op == "grouped" else case["M"]
        st["a"], st["a_s"] = _codes(torch.randn(rows, K, generator=g, device=DEV))
        b, s = _codes(0.02 * torch.randn(E * N, K, generator=g, device=DEV))
        bias = 0.1 * torch.randn(E * N, generator=g, device=DEV) if case["bias"] else None
        if op == "grouped":
            ids = torch.sort(_router_logits(g, rows, E, torch.float32), dim=-1, descending=True).indices[:, :case["k"]]
            st["offsets"], st["order"], _ = _plan(ids, E)
            b, s = b.view(E, N, K), s.view(E, N)
            bias = None if bias is None else bias.view(E, N)
        st["b"], st["b_s"], st["bias"] = b, s, bias
    else:
        T, k, N = case["tokens"], case["k"], case["N"]
        st["y"] = torch.randn(T * k, N, generator=g, device=DEV).to(kind)
        # the rows of the slots, as a plan of random choices leaves them
        st["position"] = torch.randperm(T * k, generator=g, device=DEV).int().view(T, k)
        w = torch.rand(T, k, generator=g, device=DEV) + 0.05
        st["weights"] = w / w.sum(-1, keepdim=True)
        if op == "combine_backward":
            st["d_out"] = torch.randn(T, N, generator=g, device=DEV).to(kind)
            st["d_y"] = torch.empty_like(st["y"])
    return st


# ---- plain forms ------------------------------------------------------------


def _scores(x, score):
    if score == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True))
        return e / e.sum(-1, keepdim=True)
    return 1.0 / (1.0 + torch.exp(-x))


def _route_plain(st):
    logits = st["logits"]
    T, E = logits.shape
    k, G = st["k"], st["groups"]
    # the order of the experts in 64 bits: neighbouring scores can be closer
    # than 32 bits resolve
    key = _scores(logits.double(), st["score"])
    if st["bias"] is not None:
        key = key + st["bias"].double()
    if G > 1:
        best = torch.sort(key.view(T, G, E // G), dim=-1, descending=True, stable=True).values
        group = best[..., :st["group_top"]].sum(-1)
        kept = torch.sort(group, dim=-1, descending=True, stable=True).indices[:, :st["top_groups"]]
        allowed = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, kept, True)
        key = torch.where(allowed[:, :, None], key.view(T, G, E // G), -math.inf).view(T, E)
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k]
    w = _scores(logits.float(), st["score"]).gather(1, ids)
    w = w / w.sum(-1, keepdim=True)
    return (ids.int(), w) + _plan(ids, E)


def _route_backward_plain(st):
    x, ids, dw = st["logits"].float(), st["ids"].long(), st["d_weights"]
    s = _scores(x, st["score"])
    p = s.gather(1, ids)
    total = p.sum(-1, keepdim=True)
    dp = (dw - (dw * p / total).sum(-1, keepdim=True)) / total
    ds = torch.zeros_like(s).scatter_(1, ids, dp)
    dx = s * (ds - (ds * s).sum(-1, keepdim=True)) if st["score"] == "softmax" else ds * s * (1.0 - s)
    return dx.to(st["logits"].dtype)


def _quantize_plain(st):
    x = st["x"].float()
    s = (x.abs().amax(-1).double() / 127.0).float()
    # the codes in 64 bits: a quotient can lie next to the border of two codes
    q = torch.round(x.double() / s.double()[:, None])
    return q.to(torch.int8), s


def _finish(y, bias, act, kind):
    if bias is not None:
        y = y + bias
    if act:
        y = 0.5 * y * torch.special.erfc(y * -math.sqrt(0.5))
    return y.to(kind)


def _product_plain(st):
    y = st["a"].float() @ st["b"].float().t()
    return _finish(y * st["a_s"][:, None] * st["b_s"][None, :], st["bias"], st["act"], TYPES[st["type"]])


def _grouped_plain(st):
    order, offsets = st["order"].long(), st["offsets"].long()
    E, N, K = st["b"].shape
    rows = torch.arange(order.numel(), device=order.device)
    expert = (rows[:, None] >= offsets[None, 1:]).sum(1)
    place = rows - offsets[expert]
    # every expert's rows, padded to the longest
    a = torch.zeros(E, int(offsets.diff().max()), K, device=order.device)
    token = order // st["k"]
    a[expert, place] = st["a"].float()[token]
    y = torch.bmm(a, st["b"].float().transpose(1, 2).contiguous())[expert, place]
    y = y * st["a_s"][token][:, None] * st["b_s"][expert]
    return _finish(y, None if st["bias"] is None else st["bias"][expert], st["act"], TYPES[st["type"]])


def _combine_plain(st):
    y = st["y"].float()[st["position"].long()]
    return (st["weights"][..., None] * y).sum(1).to(TYPES[st["type"]])


def _combine_backward_plain(st):
    at = st["position"].long()
    d = st["d_out"].float()[:, None, :]
    st["d_y"][at] = (st["weights"][..., None] * d).to(st["d_y"].dtype)
    return st["d_y"], (d * st["y"].float()[at]).sum(-1)


def run(st):
    op = st["op"]
    if own:
        from block_scaled_precision_mxgemm_amd import mxgemm as mx

        out_type = {"fp32": mx.OUT_F32, "bf16": mx.OUT_BF16, "fp16": mx.OUT_F16}[st["type"]]
        score = mx.SCORE_SOFTMAX if st.get("score") == "softmax" else mx.SCORE_SIGMOID
        act = mx.ACT_GELU if st.get("act") else mx.ACT_NONE
        if op == "route":
            ids, weights = mx.expert_route(st["logits"], st["k"], score, bias=st["bias"], groups=st["groups"],
                                           top_groups=st["top_groups"], group_top=st["group_top"])
            return (ids, weights) + mx.expert_plan(ids, st["experts"])
        if op == "route_backward":
            return mx.expert_route_backward(st["logits"], st["ids"], st["d_weights"], score)
        if op == "quantize":
            return mx.int8gemm_quantize(st["x"])
        if op == "product":
            return mx.int8gemm_run(st["a"], st["a_s"], st["b"], st["b_s"], bias=st["bias"], act=act, out_type=out_type)
        if op == "grouped":
            return mx.int8gemm_run_grouped(st["a"], st["a_s"], st["b"], st["b_s"], st["offsets"], index=st["order"],
                                           index_div=st["k"], bias=st["bias"], act=act, out_type=out_type)
        if op == "combine":
            return mx.expert_combine(st["y"], st["position"], st["weights"], out_type=out_type)
        return mx.expert_combine_backward(st["d_out"], st["y"], st["position"], st["weights"], d_y=st["d_y"])
    return {"route": _route_plain, "route_backward": _route_backward_plain, "quantize": _quantize_plain,
            "product": _product_plain, "grouped": _grouped_plain, "combine": _combine_plain,
            "combine_backward": _combine_backward_plain}[op](st)


# ---- what a pass cannot do without ------------------------------------------


def work(case):
    op = case["op"]
    size = {"fp32": 4, "bf16": 2, "fp16": 2}[case["type"]]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        # logits in; ids, weights, order and position out, with the offsets
        return {"bytes": T * E * size + 4 * T * k * 4 + 4 * (E + 1) + (4 * E if case["bias"] else 0), "flops": 6 * T * E}
    if op == "route_backward":
        T, E, k = case["tokens"], case["experts"], case["k"]
        return {"bytes": 2 * T * E * size + 8 * T * k, "flops": 6 * T * E}
    if op == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": n * (size + 1) + 4 * case["rows"], "flops": 3 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + M * N * size + 4 * (M + N) + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "grouped":
        T, k, E, N, K = case["tokens"], case["k"], case["experts"], case["N"], case["K"]
        # the experts that get a row at all, were every choice as likely
        hit = E * (1.0 - (1.0 - k / E) ** T)
        return {"bytes": int(hit * N * (K + 4 + (4 if case["bias"] else 0))) + T * (K + 4) + T * k * (N * size + 4),
                "flops": 2 * T * k * N * K}
    T, k, N = case["tokens"], case["k"], case["N"]
    if op == "combine":
        return {"bytes": T * (k + 1) * N * size + 8 * T * k, "flops": 2 * T * k * N}
    return {"bytes": T * (2 * k + 1) * N * size + 12 * T * k, "flops": 3 * T * k * N}


# ---- the definitions in 64 bits ---------------------------------------------


def _first_of_largest(key):
    """The lowest index of each row's largest value."""
    top = key.max(-1, keepdim=True).values
    at = torch.arange(key.shape[-1], device=key.device).expand_as(key)
    return torch.where(key == top, at, key.shape[-1]).min(-1).values


def _exact_scores(x, score):
    return torch.exp(x - torch.logsumexp(x, -1, keepdim=True)) if score == "softmax" else torch.sigmoid(x)


def _exact_route(case, st):
    x = st["logits"].double()
    T, E = x.shape
    G = case["groups"]
    s = _exact_scores(x, case["score"])
    key = s + (0.0 if st["bias"] is None else st["bias"].double())
    if G > 1:
        rest, group = key.reshape(T, G, E // G).clone(), torch.zeros(T, G, dtype=torch.float64, device=x.device)
        for _ in range(min(case["group_top"], E // G)):
            at = _first_of_largest(rest)[..., None]
            group += rest.gather(-1, at)[..., 0]
            rest.scatter_(-1, at, -math.inf)
        out = torch.full_like(group, -math.inf)
        for _ in range(case["top_groups"]):
            at = _first_of_largest(group)[:, None]
            out.scatter_(1, at, 0.0)
            group.scatter_(1, at, -math.inf)
        key = key + out.repeat_interleave(E // G, dim=1)
    chosen = []
    for _ in range(case["k"]):
        at = _first_of_largest(key)
        chosen.append(at)
        key.scatter_(1, at[:, None], -math.inf)
    ids = torch.stack(chosen, 1)
    w = s.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    # a slot's row: the slots of lower experts, and those of its own before it
    flat = ids.reshape(-1)
    count = torch.bincount(flat, minlength=E)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    order = (flat * flat.numel() + torch.arange(flat.numel(), device=flat.device)).argsort()
    position = order.argsort().view(T, -1)
    return ids.int(), w, offsets.int(), order.int(), position.int()


def _exact_route_backward(case, st):
    x = st["logits"].double()
    ids, dw = st["ids"].long(), st["d_weights"].double()
    if case["score"] == "softmax":
        # the weights are the softmax over the chosen logits alone
        w = torch.softmax(x.gather(1, ids), -1)
        d = w * (dw - (w * dw).sum(-1, keepdim=True))
    else:
        p = torch.sigmoid(x.gather(1, ids))
        w = p / p.sum(-1, keepdim=True)
        d = w * (dw - (w * dw).sum(-1, keepdim=True)) * torch.sigmoid(-x.gather(1, ids))
    return torch.zeros_like(x).scatter_add_(1, ids, d)


def _exact_gelu(y):
    return y * torch.special.ndtr(y)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "route_backward":
        return _exact_route_backward(case, st)
    if op == "quantize":
        x = st["x"].double()
        s = x.abs().max(-1).values / 127.0
        # the codes are those of the scale as it is stored, in 32 bits
        step = s.float().double()[:, None]
        low = torch.floor(x / step)
        far = x / step - low
        up = (far > 0.5) | ((far == 0.5) & (low % 2 != 0))
        return (low + up).to(torch.int8), s
    if op in ("product", "grouped"):
        a = st["a"].double() * st["a_s"].double()[:, None]
        if op == "product":
            y = a @ (st["b"].double() * st["b_s"].double()[:, None]).t()
            y = y if st["bias"] is None else y + st["bias"].double()
        else:
            token = st["order"].long() // case["k"]
            edges = st["offsets"].tolist()
            parts = []
            for e in range(case["experts"]):
                mine = a[token[edges[e]:edges[e + 1]]]
                p = mine @ (st["b"][e].double() * st["b_s"][e].double()[:, None]).t()
                parts.append(p if st["bias"] is None else p + st["bias"][e].double())
            y = torch.cat(parts)
        return _exact_gelu(y) if case["act"] else y
    at, w = st["position"].long(), st["weights"].double()
    y = st["y"].double()
    if op == "combine":
        out = torch.zeros(case["tokens"], case["N"], dtype=torch.float64, device=y.device)
        for j in range(case["k"]):
            out += w[:, j, None] * y[at[:, j]]
        return out
    d = st["d_out"].double()
    d_y = torch.empty_like(y)
    d_w = torch.empty_like(w)
    for j in range(case["k"]):
        d_y[at[:, j]] = w[:, j, None] * d
        d_w[:, j] = (d * y[at[:, j]]).sum(-1)
    return d_y, d_w
