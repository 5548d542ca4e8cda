"""Workloads of the operators around an expert layer: routing to experts and
its gradient, the join of the experts' rows and its gradient, products with
4-bit weights (one weight, and grouped by expert), and the norm of many
gradients with clipping.

With ``own`` false, ``run`` computes them with elementary torch operations in
fp32 (scores that decide a choice, and long sums, in fp64); with ``own`` true it
calls the library (``dense_fp32_gemm_f32_amd.binding``).
"""
import math

import torch

own = False

# The library's constants: epilogue activation, scores, formats of 4-bit codes.
RELU = 1
SCORES = {"softmax": 0, "sigmoid": 1}
FORMATS = {"int": 0, "e2m1": 1}

# What the code of an e2m1 weight stands for (bit 3 is the sign).
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def listed():
    return [
        # one small decode batch through a softmax router: launch latency only
        {"name": "route_decode", "op": "route", "tokens": 16, "experts": 32, "top": 4,
         "score": "softmax", "bias": False, "groups": 1, "group_top": 1, "group_best": 1,
         "renorm": True, "masked": 0.0, "train": False},
        # a long prefill: sigmoid scores, a balance bias, groups of experts
        {"name": "route_prefill", "op": "route", "tokens": 16384, "experts": 256, "top": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "group_top": 4, "group_best": 2,
         "renorm": True, "masked": 0.0, "train": False},
        # training: choices, weights and the gradient of the logits; some rows are padding
        {"name": "route_train", "op": "route", "tokens": 8192, "experts": 64, "top": 4,
         "score": "softmax", "bias": False, "groups": 1, "group_top": 1, "group_best": 1,
         "renorm": False, "masked": 0.05, "train": True},
        # the experts' rows of a decode batch added up for each token
        {"name": "join_decode", "op": "join", "tokens": 48, "top": 4, "n": 1024, "drop": 0.0,
         "train": False},
        # training: the same for a long batch with dropped choices, and its gradients
        {"name": "join_train", "op": "join", "tokens": 8192, "top": 2, "n": 2048, "drop": 0.05,
         "train": True},
        # one token through a large projection in 4 bits: the read of the codes
        {"name": "q4_token", "op": "q4", "m": 1, "n": 8192, "k": 8192, "format": "int",
         "zeros": True, "group": 128, "scale": "float16", "act": 0},
        # a few requests, odd sizes, short groups
        {"name": "q4_ragged", "op": "q4", "m": 13, "n": 1001, "k": 2047, "format": "int",
         "zeros": False, "group": 32, "scale": "float32", "act": RELU},
        # a prefill through the same kind of projection: bound by the matrix cores
        {"name": "q4_prefill", "op": "q4", "m": 4096, "n": 4096, "k": 4096, "format": "int",
         "zeros": False, "group": 128, "scale": "bfloat16", "act": 0},
        # a decode batch through experts in 4 bits: every expert has a few rows
        {"name": "q4_experts_decode", "op": "q4_grouped", "tokens": 48, "top": 4, "groups": 32,
         "k": 1024, "n": 2048, "format": "e2m1", "zeros": False, "group": 32, "scale": "e8m0",
         "gather": True, "act": RELU, "drop": 0.0},
        # a prefill through the down projection of 4-bit experts, scattered to the choices' slots
        {"name": "q4_experts_prefill", "op": "q4_grouped", "tokens": 4096, "top": 2, "groups": 8,
         "k": 2048, "n": 1024, "format": "e2m1", "zeros": False, "group": 32, "scale": "e8m0",
         "gather": False, "act": 0, "drop": 0.0},
        # clipping the gradients of a few adapters: many small arrays
        {"name": "clip_adapters", "op": "clip", "arrays": 64, "smallest": 2048,
         "largest": 131072, "clips": True},
        # clipping the gradients of a whole model: some arrays hold most of them
        {"name": "clip_model", "op": "clip", "arrays": 120, "smallest": 1024,
         "largest": 16777216, "clips": True},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "join", "q4", "q4", "q4_grouped", "q4_grouped", "clip"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log(rng, 2, 256 // groups)
        experts = groups * size
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts,
                "top": rng.randint(1, min(8, experts)), "score": rng.choice(list(SCORES)),
                "bias": rng.random() < 0.5, "groups": groups,
                "group_top": rng.randint(1, groups), "group_best": rng.choice([1, 2]),
                "renorm": rng.random() < 0.5, "masked": rng.choice([0.0, 0.1]),
                "train": rng.random() < 0.4}

    # widths: whole multiples of 32 as models have them, or any number
    def width(lo, hi):
        w = _log(rng, lo, hi)
        return max(32, w // 32 * 32) if rng.random() < 0.6 else w
    if op == "join":
        top = rng.choice([1, 2, 3, 4, 6, 8])
        return {"op": op, "tokens": _log(rng, 1, 16384 // top), "top": top,
                "n": width(32, 2048), "drop": rng.choice([0.0, 0.1]), "train": rng.random() < 0.5}
    if op == "clip":
        arrays = _log(rng, 1, 400)
        return {"op": op, "arrays": arrays, "smallest": _log(rng, 1, 4096),
                "largest": _log(rng, 4096, 16777216), "clips": rng.random() < 0.7}
    kind = {"format": rng.choice(list(FORMATS)), "group": rng.choice([32, 64, 128, 65536]),
            "scale": rng.choice(["float32", "float16", "bfloat16", "e8m0"]),
            "act": rng.choice([0, RELU])}
    kind["zeros"] = kind["format"] == "int" and rng.random() < 0.5
    if op == "q4":
        return {"op": op, "m": rng.choice([1, _log(rng, 1, 64), _log(rng, 1, 2048)]),
                "n": width(32, 8192), "k": width(32, 4096), **kind}
    top = rng.choice([1, 2, 3, 4])
    return {"op": op, "tokens": _log(rng, 1, 8192 // top), "top": top,
            "groups": _log(rng, max(2, top), 64), "k": width(32, 1408), "n": width(32, 1408),
            "gather": rng.random() < 0.5, "drop": rng.choice([0.0, 0.1]), **kind}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def _choices(tokens, top, groups, drop, g):
    """Each token's `top` different experts, drawn from a skewed popularity as
    routers give; a dropped choice is -1.  int32, tokens * top entries."""
    popularity = torch.randn(groups, generator=g, device="cuda") * 0.5
    noise = torch.rand(tokens, groups, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    scores = popularity - torch.log(-torch.log(noise))
    choice = torch.topk(scores, top, dim=1).indices.to(torch.int32)
    if drop > 0:
        choice[torch.rand(tokens, top, generator=g, device="cuda") < drop] = -1
    return choice


def _order(index, groups):
    """offsets (groups + 1) and the entries sorted by (group, entry), int32,
    with -1 behind the last one."""
    i = index.to(torch.int64)
    kept = (i >= 0) & (i < groups)
    key = torch.where(kept, i, torch.full_like(i, groups))
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(groups, device=key.device)).sum(0)
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device=key.device)
    offsets[1:] = torch.cumsum(counts, 0)
    order = torch.where(torch.arange(order.numel(), device=key.device) < offsets[-1], order,
                        torch.full_like(order, -1))
    return offsets.to(torch.int32), order.to(torch.int32)


def _weights4(case, g, stack=()):
    """Codes (two to a byte along K, the even k in the low half), scales and zero
    points of weights whose products stay of order one."""
    n, k, group = case["n"], case["k"], case["group"]
    along = (k + group - 1) // group
    codes = torch.randint(0, 256, (*stack, n, (k + 1) // 2), generator=g, device="cuda",
                          dtype=torch.uint8)
    size = k ** -0.5 / (4.6 if case["format"] == "int" else 3.0)
    if case["scale"] == "e8m0":
        power = 127 + round(math.log2(size))
        scale = torch.randint(power - 1, power + 2, (*stack, n, along), generator=g,
                              device="cuda").to(torch.uint8)
    else:
        scale = size * (0.5 + torch.rand(*stack, n, along, generator=g, device="cuda"))
        scale = scale.to(getattr(torch, case["scale"]))
    zero = None
    if case["zeros"]:
        zero = torch.randint(5, 11, (*stack, n, along), generator=g, device="cuda").to(torch.uint8)
    return codes, scale, zero


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op == "route":
        t, e = case["tokens"], case["experts"]
        s["logits"] = _normal(g, t, e, scale=1.5) + _normal(g, e, scale=0.5)
        if case["masked"]:
            # experts that are switched off for a token, and rows of padding
            off = torch.rand(t, e, generator=g, device="cuda") < case["masked"]
            off |= torch.rand(t, 1, generator=g, device="cuda") < case["masked"]
            s["logits"].masked_fill_(off, -math.inf)
        s["bias"] = _normal(g, e, scale=0.05) if case["bias"] else None
        if case["train"]:
            s["dweight"] = _normal(g, t, case["top"])
        return s
    if op == "join":
        t, top, n = case["tokens"], case["top"], case["n"]
        s["h"] = _normal(g, t * top, n)
        s["weight"] = torch.rand(t, top, generator=g, device="cuda") + 0.05
        s["choice"] = None
        if case["drop"]:
            s["choice"] = _choices(t, top, 16, case["drop"], g)
        if case["train"]:
            s["dy"] = _normal(g, t, n)
        return s
    if op == "clip":
        # sizes spread over the logarithm of the range, the same for every seed
        lo, hi, n = case["smallest"], case["largest"], case["arrays"]
        sizes = [hi] + [int(lo * (hi / lo) ** ((i * 0.6180339887) % 1.0)) for i in range(1, n)]
        s["grads"] = [_normal(g, size, scale=1e-3) for size in sizes]
        # the clipped arrays lie in one buffer, each from a multiple of 64 floats on
        places = [(size + 63) // 64 * 64 for size in sizes]
        s["flat"] = torch.zeros(sum(places), device="cuda")
        s["out"] = [part[:size] for part, size in zip(s["flat"].split(places), sizes)]
        s["max_norm"] = 1e-3 * math.sqrt(sum(sizes)) * (0.25 if case["clips"] else 4.0)
        return s
    if op == "q4":
        s["a"] = _normal(g, case["m"], case["k"])
        s["codes"], s["scale"], s["zero"] = _weights4(case, g)
        s["bias"] = _normal(g, case["n"]) if case["act"] else None
        return s
    top = min(case["top"], case["groups"])
    index = _choices(case["tokens"], top, case["groups"], case["drop"], g).reshape(-1)
    s["offsets"], s["order"] = _order(index, case["groups"])
    s["tokens_of"] = torch.where(s["order"] >= 0,
                                 torch.div(s["order"], top, rounding_mode="floor"),
                                 s["order"]).to(torch.int32)
    # gather: tokens are read by choice; otherwise one row a choice, read and written by slot
    s["a"] = _normal(g, case["tokens"] if case["gather"] else index.numel(), case["k"])
    s["codes"], s["scale"], s["zero"] = _weights4(case, g, (case["groups"],))
    s["bias"] = _normal(g, case["groups"], case["n"]) if case["act"] else None
    return s


# ---- the plain forms -----------------------------------------------------------

def _plain_choose(s):
    """The experts chosen for each token (-1 for none), from scores in 64 bits."""
    case, logits = s["case"], s["logits"].double()
    t, e = logits.shape
    groups = case["groups"]
    if case["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        top = logits.max(1, keepdim=True).values
        score = torch.exp(logits - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        score = score / score.sum(1, keepdim=True).clamp_min(1e-300)
    # the order of scores without a bias is that of the logits
    value = score + s["bias"].double() if s["bias"] is not None else logits
    value = torch.where(logits > -math.inf, value, torch.full_like(value, -math.inf))
    if case["group_top"] < groups:
        if case["group_best"] == 2:
            two = torch.where(value > -math.inf, value if s["bias"] is not None else score,
                              torch.full_like(value, -math.inf)).view(t, groups, e // groups)
            two = torch.sort(two, dim=2, descending=True).values[:, :, :2]
            best = two[:, :, 0]
            if two.shape[2] > 1:
                best = best + torch.where(two[:, :, 1] > -math.inf, two[:, :, 1],
                                          torch.zeros_like(best))
        else:
            best = value.view(t, groups, e // groups).max(2).values
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["group_top"]]
        mask = torch.zeros(t, groups, dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        value = value.masked_fill(~mask.repeat_interleave(e // groups, 1), -math.inf)
    order = torch.sort(value, dim=1, descending=True, stable=True)
    choice, best = order.indices[:, :case["top"]], order.values[:, :case["top"]]
    return torch.where(best > -math.inf, choice, torch.full_like(choice, -1))


def _plain_route(s):
    case = s["case"]
    choice = _plain_choose(s)
    logits, there = s["logits"], choice >= 0
    if case["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        top = logits.max(1, keepdim=True).values
        score = torch.exp(logits - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        score = score / score.sum(1, keepdim=True).clamp_min(1e-30)
    at = choice.clamp_min(0)
    picked = torch.where(there, score.gather(1, at), torch.zeros_like(score[:, :1]))
    scale = 2.5 if case["renorm"] else 1.0
    total = picked.sum(1, keepdim=True).clamp_min(1e-30)
    weight = scale * (picked / total if case["renorm"] else picked)
    if not case["train"]:
        return choice.to(torch.int32), weight
    d = torch.where(there, s["dweight"], torch.zeros_like(s["dweight"])) * scale
    if case["renorm"]:
        share = picked / total
        d = (d - (share * d).sum(1, keepdim=True)) / total
    grad = torch.zeros_like(score).scatter_add_(1, at, d)
    if case["score"] == "sigmoid":
        grad = grad * score * (1 - score)
    else:
        grad = score * (grad - (grad * score).sum(1, keepdim=True))
    return choice.to(torch.int32), weight, grad


def _plain_join(s):
    case = s["case"]
    t, top, n = case["tokens"], case["top"], case["n"]
    w, h = s["weight"], s["h"].view(t, top, n)
    if s["choice"] is not None:
        there = s["choice"] >= 0
        w = torch.where(there, w, torch.zeros_like(w))
        h = torch.where(there[:, :, None], h, torch.zeros_like(h))
    y = (w[:, :, None] * h).sum(1)
    if not case["train"]:
        return y
    dh = (w[:, :, None] * s["dy"][:, None, :]).view(t * top, n)
    return y, dh, (h * s["dy"][:, None, :]).sum(2)


def _plain_weights(case, codes, scale, zero):
    """The weights (N x K) that codes, scales and zero points of one matrix stand for."""
    k, group = case["k"], case["group"]
    c = torch.stack((codes & 15, codes >> 4), dim=2).view(codes.shape[0], -1)[:, :k]
    at = torch.arange(k, device="cuda") // group
    if case["scale"] == "e8m0":
        by = torch.exp2(scale.float() - 127)
    else:
        by = scale.float()
    if case["format"] == "e2m1":
        value = torch.tensor(E2M1, device="cuda")[c.long()]
    elif zero is None:
        value = c.float() - 8
    else:
        value = c.float() - zero.float()[:, at]
    return value * by[:, at]


def _plain_q4(s):
    case = s["case"]
    y = s["a"] @ _plain_weights(case, s["codes"], s["scale"], s["zero"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return torch.clamp_min(y, 0) if case["act"] == RELU else y


def _plain_q4_grouped(s):
    case = s["case"]
    o, order = s["offsets"].tolist(), s["order"].long()
    read = s["tokens_of"].long() if case["gather"] else order
    c = torch.zeros(order.numel(), case["n"], device="cuda")
    for e in range(case["groups"]):
        if o[e] == o[e + 1]:
            continue
        w = _plain_weights(case, s["codes"][e], s["scale"][e],
                           None if s["zero"] is None else s["zero"][e])
        y = s["a"][read[o[e]:o[e + 1]]] @ w.t()
        if s["bias"] is not None:
            y = y + s["bias"][e]
        if case["act"] == RELU:
            y = torch.clamp_min(y, 0)
        if case["gather"]:
            c[o[e]:o[e + 1]] = y          # rows stay in expert order
        else:
            c[order[o[e]:o[e + 1]]] = y   # back to the choice's slot
    return c


def _plain_clip(s):
    total = torch.stack([(x.double() * x.double()).sum() for x in s["grads"]]).sum()
    norm = torch.sqrt(total)
    by = torch.clamp_max(s["max_norm"] / norm, 1.0).float()
    for x, y in zip(s["grads"], s["out"]):
        torch.mul(x, by, out=y)
    return norm.float().view(1), s["flat"]


# ---- the library's calls -------------------------------------------------------

def _own(s):
    from dense_fp32_gemm_f32_amd import binding
    case = s["case"]
    op = case["op"]
    if op == "route":
        how = {"score": SCORES[case["score"]], "renorm": case["renorm"],
               "scale": 2.5 if case["renorm"] else 1.0}
        choice, weight = binding.route(s["logits"], case["top"], bias=s["bias"],
                                       groups=case["groups"], group_top=case["group_top"],
                                       group_best=case["group_best"], **how)
        if not case["train"]:
            return choice, weight
        return choice, weight, binding.route_grad(s["dweight"], s["logits"], choice, **how)
    if op == "join":
        y = binding.join_rows(s["h"], s["weight"], s["choice"])
        if not case["train"]:
            return y
        dh, dweight = binding.join_rows_grad(s["dy"], s["h"], s["weight"], s["choice"])
        return y, dh, dweight
    if op == "clip":
        norm = binding.clip_norm(s["grads"], s["max_norm"], out=s["out"])
        return norm, s["flat"]
    kind = {"zero": s["zero"], "group": case["group"], "format": FORMATS[case["format"]],
            "bias": s["bias"], "act": case["act"]}
    if op == "q4":
        return binding.gemm_q4(s["a"], s["codes"], s["scale"], **kind)
    # rows that no expert takes are left as they are: cleared here
    c = torch.zeros(s["order"].numel(), case["n"], device="cuda") if case["drop"] else None
    if case["gather"]:
        return binding.gemm_q4_grouped(s["a"], s["codes"], s["scale"], s["offsets"], c,
                                       index_a=s["tokens_of"], **kind)
    return binding.gemm_q4_grouped(s["a"], s["codes"], s["scale"], s["offsets"], c,
                                   index_a=s["order"], index_c=s["order"], **kind)


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "join": _plain_join, "q4": _plain_q4,
            "q4_grouped": _plain_q4_grouped, "clip": _plain_clip}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "route":
        t, e, top = case["tokens"], case["experts"], case["top"]
        size, flops = 4 * (t * e + (e if case["bias"] else 0)) + 8 * t * top, 4 * t * e
        if case["train"]:
            size, flops = size + 4 * t * (e + top), flops + 4 * t * e
        return {"bytes": size, "flops": flops}
    if op == "join":
        t, top, n = case["tokens"], case["top"], case["n"]
        rows = t * top * (1 - case["drop"])   # the share that was not dropped
        size = 4 * (rows * n + t * n + t * top)
        if case["train"]:
            # the same rows of H, and dY, are read once; dH and the weights' gradient written
            size += 4 * (t * n + t * top * n + t * top)
        return {"bytes": int(size), "flops": int((6 if case["train"] else 2) * rows * n)}
    if op == "clip":
        lo, hi, n = case["smallest"], case["largest"], case["arrays"]
        total = hi + sum(int(lo * (hi / lo) ** ((i * 0.6180339887) % 1.0)) for i in range(1, n))
        return {"bytes": 8 * total, "flops": 3 * total}
    n, k = case["n"], case["k"]
    along = (k + case["group"] - 1) // case["group"]
    each = {"float32": 4, "float16": 2, "bfloat16": 2, "e8m0": 1}[case["scale"]]
    weights = n * ((k + 1) // 2 + along * (each + (1 if case["zeros"] else 0)))
    if op == "q4":
        m = case["m"]
        return {"bytes": weights + 4 * (m * k + m * n), "flops": 2 * m * n * k}
    rows = case["tokens"] * min(case["top"], case["groups"])
    a_rows = case["tokens"] if case["gather"] else rows
    return {"bytes": min(rows, case["groups"]) * weights + 4 * (a_rows * k + rows * n),
            "flops": 2 * rows * n * k}


# ---- the definitions, in 64 bits -------------------------------------------------

def _exact_route(case, s):
    """One expert at a time: the best value left, as the definition says it."""
    x = s["logits"].double()
    t, e, groups = case["tokens"], case["experts"], case["groups"]
    live = x > -math.inf
    z = torch.where(live, x, torch.zeros_like(x))
    if case["score"] == "sigmoid":
        p = torch.sigmoid(z) * live
    else:
        p = torch.exp(z - torch.logsumexp(x, 1, keepdim=True).nan_to_num(neginf=0.0)) * live
    value = z if s["bias"] is None else p + s["bias"].double()
    low = torch.full_like(value, -math.inf)
    value = torch.where(live, value, low)
    rows = torch.arange(t, device="cuda")
    if case["group_top"] < groups:
        base = value if s["bias"] is not None or case["group_best"] == 1 else torch.where(live, p,
                                                                                         low)
        base = base.reshape(t, groups, e // groups).clone()
        best = base.max(2).values
        if case["group_best"] == 2 and e // groups > 1:
            base.scatter_(2, base.argmax(2, keepdim=True), -math.inf)
            second = base.max(2).values
            best = best + torch.where(second > -math.inf, second, torch.zeros_like(second))
        open_ = torch.zeros(t, groups, dtype=torch.bool, device="cuda")
        for _ in range(case["group_top"]):
            top = best.max(1, keepdim=True).values
            first = (best == top).to(torch.int8).argmax(1)
            open_[rows, first] = True
            best[rows, first] = -math.inf
        value = torch.where(open_[:, torch.arange(e, device="cuda") // (e // groups)], value, low)
    choice = torch.empty(t, case["top"], dtype=torch.int64, device="cuda")
    for j in range(case["top"]):
        top = value.max(1, keepdim=True).values
        first = (value == top).to(torch.int8).argmax(1)
        choice[:, j] = torch.where(top[:, 0] > -math.inf, first, torch.full_like(first, -1))
        value[rows, first] = -math.inf
    mark = torch.zeros(t, e + 1, dtype=torch.float64, device="cuda")
    mark[rows[:, None], torch.where(choice >= 0, choice, torch.full_like(choice, e))] = 1
    mark = mark[:, :e]
    scale = 2.5 if case["renorm"] else 1.0
    total = (p * mark).sum(1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    q = p * mark / total if case["renorm"] else p * mark
    weight = torch.zeros(t, case["top"], dtype=torch.float64, device="cuda")
    up = torch.zeros(t, e, dtype=torch.float64, device="cuda")
    for j in range(case["top"]):
        there = choice[:, j] >= 0
        at = choice[:, j].clamp_min(0)
        weight[:, j] = scale * q[rows, at] * there
        if case["train"]:
            up[rows, at] += s["dweight"].double()[:, j] * there
    if not case["train"]:
        return None, weight
    if case["score"] == "sigmoid":
        slope = 1 - p
        grad = (q * slope * (up - (q * up).sum(1, keepdim=True)) if case["renorm"]
                else q * slope * up)
    elif case["renorm"]:
        grad = q * (up - (q * up).sum(1, keepdim=True))
    else:
        grad = p * (up - (p * up).sum(1, keepdim=True))
    return None, weight, scale * grad


def _exact_weights(case, codes, scale, zero):
    """K x N in 64 bits, by a table of the sixteen codes and one group of K at a time."""
    table = torch.tensor([float(c) for c in range(16)] if case["format"] == "int" else E2M1,
                         dtype=torch.float64, device="cuda")
    out = torch.empty(case["k"], case["n"], dtype=torch.float64, device="cuda")
    both = codes.t().long()
    out[0::2] = table[both % 16][:(case["k"] + 1) // 2]
    out[1::2] = table[both // 16][:case["k"] // 2]
    for i, begin in enumerate(range(0, case["k"], case["group"])):
        part = out[begin:begin + case["group"]]
        if case["format"] == "int":
            part -= 8.0 if zero is None else zero[:, i].double()
        by = scale[:, i].double()
        part *= torch.pow(torch.full_like(by, 2.0), by - 127) if case["scale"] == "e8m0" else by
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, s)
    if op == "join":
        t, top, n = case["tokens"], case["top"], case["n"]
        h = s["h"].double().view(t, top, n)
        w = s["weight"].double()
        if s["choice"] is not None:
            w = w * (s["choice"] >= 0)
            h = h * (s["choice"] >= 0)[:, :, None]
        y = torch.zeros(t, n, dtype=torch.float64, device="cuda")
        for j in range(top):
            y += w[:, j:j + 1] * h[:, j]
        if not case["train"]:
            return y
        dy = s["dy"].double()
        dh = torch.stack([w[:, j:j + 1] * dy for j in range(top)], 1).view(t * top, n)
        return y, dh, torch.stack([(dy * h[:, j]).sum(1) for j in range(top)], 1)
    if op == "clip":
        norm = math.sqrt(sum(float(torch.dot(x.double(), x.double())) for x in s["grads"]))
        by = s["max_norm"] / norm if norm > s["max_norm"] else 1.0
        flat = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda")
        at = 0
        for x in s["grads"]:
            flat[at:at + x.numel()] = x.double() * by
            at += (x.numel() + 63) // 64 * 64
        return torch.tensor([norm], dtype=torch.float64, device="cuda"), flat
    if op == "q4":
        y = torch.mm(s["a"].double(), _exact_weights(case, s["codes"], s["scale"], s["zero"]))
        if case["act"] == RELU:
            y = y + s["bias"].double()
            y = y * (y > 0)
        return y
    offsets, order = s["offsets"].cpu().tolist(), s["order"].cpu().long()
    top = min(case["top"], case["groups"])
    out = torch.zeros(order.numel(), case["n"], dtype=torch.float64, device="cuda")
    for e, (begin, end) in enumerate(zip(offsets, offsets[1:])):
        if end <= begin:
            continue
        slots = order[begin:end].cuda()
        w = _exact_weights(case, s["codes"][e], s["scale"][e],
                           None if s["zero"] is None else s["zero"][e])
        v = torch.mm(s["a"].double().index_select(0, slots // top if case["gather"] else slots), w)
        if case["act"] == RELU:
            v = v + s["bias"][e].double()
            v = v * (v > 0)
        at = torch.arange(begin, end, device="cuda") if case["gather"] else slots
        out.index_copy_(0, at, v)
    return out
