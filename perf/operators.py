"""Workloads of the operators whose rows belong to different weights: rows
ordered by group, products grouped by expert (forward, gradient of the rows,
gradient of the weights) and low-rank adapters beside a shared projection
(forward, and a training pass).

With ``own`` false, ``run`` computes them with elementary torch operations in
fp32; with ``own`` true it calls the library (``dense_fp32_gemm_f32_amd.binding``).
"""
import math

import torch

own = False

# The library's epilogue activation: 0 none, 1 ReLU.
RELU = 1


def listed():
    return [
        # the router's choices of one small decode batch: launch latency only
        {"name": "group_decode", "op": "group", "tokens": 16, "top": 4, "groups": 32, "drop": 0.0},
        # a long prefill routed to many experts, some choices dropped for capacity
        {"name": "group_prefill", "op": "group", "tokens": 16384, "top": 4, "groups": 64,
         "drop": 0.05},
        # one token through its eight experts, weights as checkpoints store
        # them (outputs x inputs): latency and the weights' read
        {"name": "experts_token", "op": "grouped", "tokens": 1, "top": 8, "groups": 64, "k": 2048,
         "n": 1024, "trans": True, "gather": True, "act": 0, "drop": 0.0},
        # a decode batch: every expert has a few rows, the weights' read bounds it
        {"name": "experts_decode", "op": "grouped", "tokens": 48, "top": 4, "groups": 32,
         "k": 1024, "n": 2048, "trans": False, "gather": True, "act": RELU, "drop": 0.0},
        # a prefill: the up projection of an expert layer, bias and ReLU fused
        {"name": "experts_prefill", "op": "grouped", "tokens": 4096, "top": 2, "groups": 8,
         "k": 1024, "n": 2048, "trans": False, "gather": True, "act": RELU, "drop": 0.0},
        # odd sizes that no 16-byte load fits, results scattered to their slots, dropped choices
        {"name": "experts_ragged", "op": "grouped", "tokens": 777, "top": 3, "groups": 13,
         "k": 769, "n": 1001, "trans": False, "gather": False, "act": 0, "drop": 0.1},
        # training: the gradient of the rows of experts_prefill's product
        {"name": "experts_dgrad", "op": "grouped", "tokens": 4096, "top": 2, "groups": 8,
         "k": 2048, "n": 1024, "trans": True, "gather": False, "act": 0, "drop": 0.0},
        # training: the gradient of its weights
        {"name": "experts_wgrad", "op": "wgrad", "tokens": 4096, "top": 2, "groups": 8, "m": 1024,
         "n": 2048, "drop": 0.0},
        # a short odd batch over many experts, some of them without a row
        {"name": "wgrad_ragged", "op": "wgrad", "tokens": 150, "top": 2, "groups": 40, "m": 513,
         "n": 257, "drop": 0.1},
        # serving: a decode batch of requests, each with its own adapter or none
        {"name": "adapters_decode", "op": "adapters", "requests": 32, "length": 1, "adapters": 8,
         "k": 2048, "n": 2048, "rank": 16, "trans": True, "train": False},
        # serving: prompts of several requests in one batch
        {"name": "adapters_prefill", "op": "adapters", "requests": 7, "length": 585,
         "adapters": 4, "k": 2048, "n": 2048, "rank": 32, "trans": True, "train": False},
        # training several adapters at once over a frozen projection
        {"name": "adapters_train", "op": "adapters", "requests": 8, "length": 256, "adapters": 3,
         "k": 1024, "n": 1536, "rank": 8, "trans": False, "train": True},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["group", "grouped", "grouped", "wgrad", "adapters"])
    if op == "group":
        return {"op": op, "tokens": _log(rng, 1, 16384), "top": rng.choice([1, 2, 3, 4]),
                "groups": _log(rng, 1, 256), "drop": rng.choice([0.0, 0.1])}

    # widths: whole multiples of 32 as models have them, or any number
    def width(lo, hi):
        w = _log(rng, lo, hi)
        return max(32, w // 32 * 32) if rng.random() < 0.6 else w
    if op == "adapters":
        train = rng.random() < 0.4
        widest = 1408 if train else 2048   # a training pass has two products of the projection's size
        return {"op": op, "requests": _log(rng, 1, 32),
                "length": rng.choice([1, 1, _log(rng, 2, 120)]), "adapters": _log(rng, 1, 16),
                "k": width(64, widest), "n": width(64, widest),
                "rank": rng.choice([1, 4, 8, 16, 24, 32, 64]), "trans": rng.random() < 0.5,
                "train": train}
    top = rng.choice([1, 2, 3, 4])
    groups = _log(rng, max(2, top), 64)
    if op == "wgrad":
        return {"op": op, "tokens": _log(rng, 1, 4096 // top), "top": top, "groups": groups,
                "m": width(32, 768), "n": width(32, 1024), "drop": rng.choice([0.0, 0.1])}
    return {"op": op, "tokens": _log(rng, 1, 8192 // top), "top": top, "groups": groups,
            "k": width(32, 1408), "n": width(32, 1408), "trans": rng.random() < 0.5,
            "gather": rng.random() < 0.5, "act": rng.choice([0, RELU]),
            "drop": rng.choice([0.0, 0.1])}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def _choices(case, g):
    """Each token's `top` different experts, drawn from a skewed popularity as
    routers give; a dropped choice is -1.  int32, tokens * top entries."""
    t, top, n = case["tokens"], min(case["top"], case["groups"]), case["groups"]
    popularity = torch.randn(n, generator=g, device="cuda") * 0.5
    noise = torch.rand(t, n, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    scores = popularity - torch.log(-torch.log(noise))
    choice = torch.topk(scores, top, dim=1).indices.to(torch.int32)
    if case["drop"] > 0:
        choice[torch.rand(t, top, generator=g, device="cuda") < case["drop"]] = -1
    return choice.reshape(-1).contiguous()


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


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op == "adapters":
        m = case["requests"] * case["length"]
        k, n, r, a = case["k"], case["n"], case["rank"], case["adapters"]
        # each request has one adapter, or none (the draw of `adapters` itself)
        of = torch.randint(0, a + 1, (case["requests"],), generator=g, device="cuda")
        of = torch.where(of == a, torch.full_like(of, -1), of)
        index = of.repeat_interleave(case["length"]).to(torch.int32)
        s["offsets"], s["order"] = _order(index, a)
        s["x"] = _normal(g, m, k)
        t = case["trans"]
        s["w"] = _normal(g, *((n, k) if t else (k, n)), scale=k ** -0.5)
        s["down"] = _normal(g, a, *((r, k) if t else (k, r)), scale=k ** -0.5)
        s["up"] = _normal(g, a, *((n, r) if t else (r, n)), scale=0.1)
        s["scale"] = torch.rand(a, generator=g, device="cuda") + 0.5
        s["bias"] = _normal(g, n)
        if case["train"]:
            s["dy"] = _normal(g, m, n)
        return s
    index = _choices(case, g)
    if op == "group":
        s["index"] = index
        return s
    top = min(case["top"], case["groups"])
    s["offsets"], s["order"] = _order(index, case["groups"])
    s["tokens_of"] = torch.where(s["order"] >= 0,
                                 torch.div(s["order"], top, rounding_mode="floor"),
                                 s["order"]).to(torch.int32)
    rows, groups = index.numel(), case["groups"]
    if op == "grouped":
        k, n = case["k"], case["n"]
        # gather: tokens are read by choice; otherwise one row a choice, read and written by slot
        s["a"] = _normal(g, case["tokens"] if case["gather"] else rows, k)
        s["b"] = _normal(g, groups, *((n, k) if case["trans"] else (k, n)), scale=k ** -0.5)
        s["bias"] = _normal(g, groups, n) if case["act"] else None
    else:
        s["a"] = _normal(g, case["tokens"], case["m"])
        s["b"] = _normal(g, rows, case["n"], scale=0.1)
    return s


# ---- the plain forms -----------------------------------------------------------

def _plain_group(s):
    case = s["case"]
    offsets, order = _order(s["index"], case["groups"])
    rows = torch.where(order >= 0, torch.div(order, min(case["top"], case["groups"]),
                                             rounding_mode="floor"), order)
    return offsets, order, rows.to(torch.int32)


def _plain_grouped(s):
    case = s["case"]
    o, order = s["offsets"].tolist(), s["order"].long()
    read = s["tokens_of"].long() if case["gather"] else order
    c = torch.zeros(order.numel(), case["n"], device="cuda")
    for e in range(case["groups"]):
        if o[e] == o[e + 1]:
            continue
        w = s["b"][e].t() if case["trans"] else s["b"][e]
        y = s["a"][read[o[e]:o[e + 1]]] @ w
        if s["bias"] is not None:
            y = y + s["bias"][e]
        if case["act"] == RELU:
            y = torch.clamp_min(y, 0)
        if case["gather"]:
            c[o[e]:o[e + 1]] = y          # rows stay in expert order
        else:
            c[order[o[e]:o[e + 1]]] = y   # back to the choice's slot
    return c


def _plain_wgrad(s):
    case = s["case"]
    o, order, tokens = s["offsets"].tolist(), s["order"].long(), s["tokens_of"].long()
    c = torch.zeros(case["groups"], case["m"], case["n"], device="cuda")
    for e in range(case["groups"]):
        if o[e] < o[e + 1]:
            c[e] = s["a"][tokens[o[e]:o[e + 1]]].t() @ s["b"][order[o[e]:o[e + 1]]]
    return c


def _plain_adapters(s):
    case = s["case"]
    t = case["trans"]
    o, order = s["offsets"].tolist(), s["order"].long()
    w = s["w"].t() if t else s["w"]
    y = s["x"] @ w + s["bias"]
    dx = s["dy"] @ w.t() if case["train"] else None
    d_down, d_up = torch.zeros_like(s["down"]), torch.zeros_like(s["up"])
    for e in range(case["adapters"]):
        if o[e] == o[e + 1]:
            continue
        rows = order[o[e]:o[e + 1]]
        down = s["down"][e].t() if t else s["down"][e]
        up = s["up"][e].t() if t else s["up"][e]
        x = s["x"][rows]
        h = (x @ down) * s["scale"][e]
        y[rows] += h @ up
        if case["train"]:
            dy = s["dy"][rows]
            gh = (dy @ up.t()) * s["scale"][e]
            dx[rows] += gh @ down.t()
            d_down[e] = gh.t() @ x if t else x.t() @ gh
            d_up[e] = dy.t() @ h if t else h.t() @ dy
    return (y, dx, d_down, d_up) if case["train"] else y


# ---- the library's calls -------------------------------------------------------

def _own(s):
    from dense_fp32_gemm_f32_amd import binding
    case = s["case"]
    op = case["op"]
    if op == "group":
        return binding.group_rows(s["index"], case["groups"],
                                  per_row=min(case["top"], case["groups"]))
    if op == "grouped":
        # rows that no expert takes are left as they are: cleared here
        c = torch.zeros(s["order"].numel(), case["n"], device="cuda") if case["drop"] else None
        if case["gather"]:
            return binding.gemm_grouped(s["a"], s["b"], s["offsets"], c, trans_b=case["trans"],
                                        bias=s["bias"], act=case["act"], index_a=s["tokens_of"])
        return binding.gemm_grouped(s["a"], s["b"], s["offsets"], c, trans_b=case["trans"],
                                    bias=s["bias"], act=case["act"], index_a=s["order"],
                                    index_c=s["order"])
    if op == "wgrad":
        return binding.gemm_grouped_wgrad(s["a"], s["b"], s["offsets"], index_a=s["tokens_of"],
                                          index_b=s["order"])
    y, h = binding.gemm_adapters(s["x"], s["w"], s["down"], s["up"], s["offsets"], s["order"],
                                 trans=case["trans"], scale=s["scale"], bias=s["bias"])
    if not case["train"]:
        return y
    dx, d_down, d_up = binding.gemm_adapters_grad(
        s["dy"], s["x"], s["w"], s["down"], s["up"], s["offsets"], s["order"], h,
        trans=case["trans"], scale=s["scale"])
    return y, dx, d_down, d_up


def run(state):
    if own:
        return _own(state)
    return {"group": _plain_group, "grouped": _plain_grouped, "wgrad": _plain_wgrad,
            "adapters": _plain_adapters}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "adapters":
        m = case["requests"] * case["length"]
        k, n, r = case["k"], case["n"], case["rank"]
        a = min(case["adapters"], case["requests"])
        flops = 2 * m * n * k + 2 * m * r * (k + n)
        size = m * k + k * n + a * r * (k + n) + m * n
        if case["train"]:
            flops += 2 * m * n * k + 4 * m * r * (k + n)
            size += m * n + m * k + case["adapters"] * r * (k + n)
        return {"bytes": 4 * size, "flops": flops}
    rows = case["tokens"] * min(case["top"], case["groups"])
    if op == "group":
        return {"bytes": 4 * (3 * rows + case["groups"] + 1), "flops": rows}
    if op == "grouped":
        k, n = case["k"], case["n"]
        a_rows = case["tokens"] if case["gather"] else rows
        busy = min(rows, case["groups"])
        return {"bytes": 4 * (a_rows * k + busy * k * n + rows * n), "flops": 2 * rows * k * n}
    m, n = case["m"], case["n"]
    return {"bytes": 4 * (case["tokens"] * m + rows * n + case["groups"] * m * n),
            "flops": 2 * rows * m * n}


# ---- the definitions, in 64 bits -------------------------------------------------

def exact(case, seed):
    if case["op"] == "group":
        return None
    s = prepare(case, seed)
    offsets = s["offsets"].cpu().tolist()
    order = s["order"].cpu().long()
    spans = [(g, order[b:e].cuda()) for g, (b, e) in enumerate(zip(offsets, offsets[1:])) if e > b]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if case["op"] == "grouped":
        top = min(case["top"], case["groups"])
        out = torch.zeros(order.numel(), case["n"], dtype=torch.float64, device="cuda")
        for g, slots in spans:
            w = d["b"][g].transpose(0, 1) if case["trans"] else d["b"][g]
            a = d["a"].index_select(0, slots // top if case["gather"] else slots)
            v = torch.mm(a, w)
            if case["act"] == RELU:
                v = v + d["bias"][g]
                v = v * (v > 0)
            at = (torch.arange(offsets[g], offsets[g + 1], device="cuda") if case["gather"]
                  else slots)
            out.index_copy_(0, at, v)
        return out
    if case["op"] == "wgrad":
        top = min(case["top"], case["groups"])
        out = torch.zeros(case["groups"], case["m"], case["n"], dtype=torch.float64, device="cuda")
        for g, slots in spans:
            a = d["a"].index_select(0, slots // top)
            out[g] = torch.mm(a.transpose(0, 1).contiguous(), d["b"].index_select(0, slots))
        return out
    t = case["trans"]
    flip = (lambda v: v.transpose(-2, -1).contiguous()) if t else (lambda v: v)
    w, down, up = flip(d["w"]), flip(d["down"]), flip(d["up"])
    # the weights that each row sees: the projection plus its adapter's product
    y = torch.mm(d["x"], w) + d["bias"]
    for g, rows in spans:
        seen = w + d["scale"][g] * torch.mm(down[g], up[g])
        y[rows] = torch.mm(d["x"][rows], seen) + d["bias"]
    if not case["train"]:
        return y
    dx = torch.mm(d["dy"], w.transpose(0, 1).contiguous())
    d_down, d_up = torch.zeros_like(down), torch.zeros_like(up)
    for g, rows in spans:
        seen = w + d["scale"][g] * torch.mm(down[g], up[g])
        dx[rows] = torch.mm(d["dy"][rows], seen.transpose(0, 1).contiguous())
        # the gradient of the row's whole weight, then of its two factors
        full = torch.mm(d["x"][rows].transpose(0, 1).contiguous(), d["dy"][rows])
        d_down[g] = d["scale"][g] * torch.mm(full, up[g].transpose(0, 1).contiguous())
        d_up[g] = d["scale"][g] * torch.mm(down[g].transpose(0, 1).contiguous(), full)
    return y, dx, flip(d_down), flip(d_up)
