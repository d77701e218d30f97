"""Cases that time the routing to experts, the expert products with 4-bit weights and
the gradients of the combine: `run` computes them with elementary torch operations,
or with this library's calls where `own` is true.

A case names one operator (`op`) and the share of an expert-parallel layer it works on:
`ranks` source ranks of `tokens` tokens each, `experts` in all, the first `local` of
them on this GPU, `top_k` picks a token."""
import math

import numpy as np
import torch

own = False

_LOGITS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_FLT_MAX = torch.finfo(torch.float32).max
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _route(op, name, **kw):
    case = dict(op=op, ranks=8, tokens=1024, experts=256, top_k=8, groups=1, kept=1,
                score="softmax", group_score="max", bias=False, renormalize=True, scale=1.0,
                dtype="f32", masked=False)
    case.update(kw)
    return dict(case, **({"name": name} if name else {}))


def _w4(op, name, **kw):
    case = dict(op=op, ranks=8, tokens=128, experts=256, local=32, top_k=8, hidden=7168,
                inter=2048, fmt="int4", group=128, scales="bf16", zipf=False)
    case.update(kw)
    return dict(case, **({"name": name} if name else {}))


def _cb(name, **kw):
    case = dict(op="combine_backward", ranks=8, tokens=128, experts=256, local=32, top_k=8,
                hidden=7168, zipf=False)
    case.update(kw)
    return dict(case, **({"name": name} if name else {}))


def listed():
    grouped = dict(groups=8, kept=4, score="sigmoid", group_score="top2", bias=True, scale=2.5)
    return [
        # the router of one decoded token: latency alone counts
        _route("route", "route_one_token", ranks=1, tokens=1, **grouped),
        # a prefill step of a 256-expert layer with grouped, bias-balanced sigmoid routing
        _route("route", "route_prefill_grouped", tokens=4096, **grouped),
        # a 128-expert layer with plain softmax routing, some experts out of service
        _route("route", "route_softmax_masked", experts=128, dtype="bf16", masked=True),
        # the training step of the same two kinds of router; the second with odd sizes
        _route("route_backward", "route_backward_prefill", tokens=4096, **grouped),
        _route("route_backward", "route_backward_odd", ranks=3, tokens=1111, experts=60, top_k=6,
               dtype="f16", renormalize=False, scale=16.0),
        # the combine's gradient at a training step's size, and at a small odd one
        _cb("combine_backward_prefill", tokens=4096),
        _cb("combine_backward_small", ranks=4, tokens=77, experts=64, local=16, hidden=4096),
        # up-projection of a decode step: about 32 rows an expert
        _w4("up_w4", "up_w4_decode"),
        # up-projection of a single token, every expert on this GPU
        _w4("up_w4", "up_w4_one_token", ranks=1, tokens=1, experts=32, scales="f16"),
        # down-projection into the receive buffers of a decode step, small groups of weights
        _w4("down_w4", "down_w4_decode", fmt="e2m1", group=32),
        # down-projection of a single token
        _w4("down_w4", "down_w4_one_token", ranks=1, tokens=1, experts=32, scales="f16"),
        # skewed routing: a few experts hold most of the rows
        _w4("down_w4", "down_w4_skewed", tokens=192, experts=128, local=16, hidden=4096,
            inter=1536, group=64, zipf=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine_backward", "up_w4", "down_w4"])
    ranks = rng.randint(1, 8)
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 4, 256 // groups)
        top_k = rng.randint(1, min(12, experts))
        return _route(op, None, ranks=ranks, tokens=_log(rng, 1, 4096), experts=experts,
                      top_k=top_k, groups=groups, kept=rng.randint(1, groups),
                      score=rng.choice(["softmax", "sigmoid"]),
                      group_score=rng.choice(["max", "top2"]), bias=rng.random() < 0.5,
                      renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                      dtype=rng.choice(["f32", "bf16", "f16"]), masked=rng.random() < 0.3)
    top_k = rng.randint(1, 8)
    if op == "combine_backward":
        local = rng.randint(top_k, 48)
        return _cb(None, ranks=ranks, tokens=_log(rng, 1, 1024), experts=local * ranks,
                   local=local, top_k=top_k, hidden=128 * _log(rng, 1, 56), zipf=rng.random() < 0.3)
    local = rng.randint(top_k, 32)
    return _w4(op, None, ranks=ranks, tokens=_log(rng, 1, 128), experts=local * ranks, local=local,
               top_k=top_k, hidden=128 * _log(rng, 2, 56), inter=128 * _log(rng, 1, 16),
               fmt=rng.choice(["int4", "e2m1"]), group=rng.choice([32, 64, 128]),
               scales=rng.choice(["bf16", "f16"]), zipf=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _router_inputs(case, g):
    R, T, E = case["ranks"], case["tokens"], case["experts"]
    # logits of a trained router: spread of about 1.5, one offset an expert
    logits = 1.5 * _randn(g, R, T, E) + 0.5 * _randn(g, E)
    if case["masked"]:
        # one expert in eight is out of service; one token in 64 (a padded one) has none
        perm = torch.randperm(E, generator=g, device="cuda")
        logits[..., perm[: (E - 1) // 8]] = -math.inf
        logits[torch.rand(R, T, generator=g, device="cuda") < 1 / 64] = -math.inf
    s = {"logits": logits.to(_LOGITS[case["dtype"]]),
         "bias": 0.1 * _randn(g, E) if case["bias"] else None}
    if case["op"] == "route_backward":
        # the picks of the forward pass (of a 32-bit sort: any distinct ids serve the
        # gradient), and the gradient that reaches the weights
        top = torch.sort(logits, dim=-1, descending=True, stable=True)
        ids = top.indices[..., : case["top_k"]].to(torch.int32)
        ids[top.values[..., : case["top_k"]] == -math.inf] = -1
        s["ids"] = ids
        s["grad_w"] = 0.01 * _randn(g, R, T, case["top_k"])
    return s


def _routing_inputs(case, g):
    """Picks, their weights and the grouped layout of the local ones: rows ordered by
    (expert, rank, token, pick)."""
    R, T, E, k = case["ranks"], case["tokens"], case["experts"], case["top_k"]
    u = torch.rand(R, T, E, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    keys = -torch.log(-torch.log(u))
    if case["zipf"]:
        rank = torch.randperm(E, generator=g, device="cuda")
        keys -= 1.2 * torch.log(rank + 1.0)
    ids = torch.topk(keys, k, dim=-1).indices.to(torch.int32)
    logit = _randn(g, R, T, k)
    flat = ids.reshape(-1).long()
    pick = torch.nonzero(flat < case["local"]).reshape(-1)  # (rk, t, k) order
    order = torch.sort(flat[pick], stable=True).indices
    pick = pick[order]
    rk, t, kk = pick // (T * k), pick // k % T, pick % k
    run = flat[pick] * R + rk
    counts = torch.bincount(run, minlength=case["local"] * R)
    offsets = torch.zeros(case["local"] * R + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return {"ids": ids, "w": torch.softmax(logit, -1), "offsets": offsets,
            "src_info": torch.stack([t, kk], 1).to(torch.int32).contiguous(),
            "m": int(pick.numel()), "rank": rk, "expert": flat[pick],
            "rows_max": int(counts.reshape(-1, R).sum(1).max())}


def _weights_4bit(case, g, n, k):
    """Codes [local][n][k/2] (even k in the low bits) and scales [local][n][k/group] of
    normally distributed weights of size 1/sqrt(k)."""
    E = case["local"]
    v = _randn(g, E, n, k, dtype=torch.bfloat16)
    if case["fmt"] == "int4":
        c = (v.mul_(2.7).round_() + 8).clamp_(0, 15).to(torch.uint8)
        step = 1 / 2.7
    else:
        a = v.abs().mul_(2.0)
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda",
                             dtype=torch.bfloat16)
        c = torch.bucketize(a, edges, out_int32=True).to(torch.uint8)
        c |= (v < 0).to(torch.uint8) << 3
        step = 0.5
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    scales = (step / math.sqrt(k)) * (0.75 + 0.5 * torch.rand(
        E, n, k // case["group"], generator=g, device="cuda"))
    return codes, scales.to(_LOGITS[case["scales"]])


def _inputs(case, seed):
    g = _generator(seed)
    if case["op"] in ("route", "route_backward"):
        return _router_inputs(case, g)
    s = _routing_inputs(case, g)
    N, I = case["hidden"], case["inter"] if "inter" in case else 0
    if case["op"] == "combine_backward":
        s["grad_out"] = _randn(g, case["ranks"], case["tokens"], N, dtype=torch.bfloat16)
        # what the forward pass left in the receive buffers: a row for each slot
        s["recv"] = _randn(g, case["ranks"], case["tokens"] * case["top_k"], N,
                           dtype=torch.bfloat16)
    elif case["op"] == "up_w4":
        s["x"] = _randn(g, s["m"], N, dtype=torch.bfloat16)
        s["codes"], s["scales"] = _weights_4bit(case, g, 2 * I, N)
    else:
        s["x"] = _randn(g, s["m"], I, dtype=torch.bfloat16)
        s["codes"], s["scales"] = _weights_4bit(case, g, N, I)
    return s


def _capacity(case):
    """Rows of the buffers that a program keeps for grouped rows: the expected number and
    a quarter, or every pick where the routing is skewed."""
    most = case["ranks"] * case["tokens"] * case["top_k"]
    return most if case["zipf"] else min(most, int(1.25 * _expected(case)[0]) + 256)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] in ("combine_backward", "up_w4"):
        s["out"] = torch.zeros(_capacity(case), case["inter" if case["op"] == "up_w4" else "hidden"],
                               dtype=torch.bfloat16, device="cuda")
    if own:
        # the handle that a program keeps for the layer, and the weights laid out once
        from grouped_gemm_scatter_amd import EpCombine
        router = case["op"] in ("route", "route_backward")
        s["ctx"] = ctx = EpCombine(
            n_ranks=case["ranks"], top_k=case["top_k"], max_tokens_per_rank=case["tokens"],
            n_experts_per_device=1 if router else case["local"],
            hidden_k=case.get("inter", 128), hidden_n=128 if router else case["hidden"],
            sentinel=0)
        if case["op"] == "combine_backward":
            for dst, rows in zip(ctx.recv, s.pop("recv")):
                dst.copy_(rows.view(-1).view(torch.uint8))
        if "codes" in s:
            s["w4"] = ctx.pack_weights_w4(s.pop("codes"), s.pop("scales"), codes=case["fmt"])
    elif case["op"] == "down_w4":
        s["recv"] = torch.zeros(case["ranks"], case["tokens"] * case["top_k"], case["hidden"],
                                dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](state, case, state["ctx"])
    return _PLAIN[case["op"]](state, case)


def _own_route(s, case, ctx):
    return ctx.route(s["logits"], bias=s["bias"], n_groups=case["groups"],
                     topk_groups=case["kept"], score=case["score"],
                     group_score=case["group_score"], renormalize=case["renormalize"],
                     scale=case["scale"])


def _own_route_backward(s, case, ctx):
    return ctx.route_backward(s["logits"], s["ids"], s["grad_w"], score=case["score"],
                              renormalize=case["renormalize"], scale=case["scale"])


def _own_combine_backward(s, case, ctx):
    return ctx.combine_backward(s["grad_out"], s["ids"], s["w"], s["offsets"], s["src_info"],
                                s["m"], grad_rows=s["out"])


def _own_up(s, case, ctx):
    ctx.up_swiglu_w4(s["x"], s["w4"], s["offsets"], s["m"], s["out"])
    return s["out"]


def _own_down(s, case, ctx):
    ctx.next_epoch()
    ctx.gemm_scatter_w4(s["x"], s["w4"], s["offsets"], s["src_info"], s["m"])
    return [r.view(torch.bfloat16).view(-1, case["hidden"]) for r in ctx.recv]


_OWN = {"route": _own_route, "route_backward": _own_route_backward,
        "combine_backward": _own_combine_backward, "up_w4": _own_up, "down_w4": _own_down}


def _clean(logits):
    """32-bit logits with +inf at the largest number and NaN, like -inf, a missing expert."""
    x = logits.float().clamp(max=_FLT_MAX)
    return torch.where(torch.isnan(x), -math.inf, x)


def _softmax(x):
    top = x.amax(-1, keepdim=True).clamp(min=-_FLT_MAX)
    e = torch.exp(x - top)
    return e / e.sum(-1, keepdim=True).clamp(min=torch.finfo(x.dtype).tiny)


def _plain_route(s, case):
    x = _clean(s["logits"])
    k, G = case["top_k"], case["groups"]
    # which experts: values next to a border decide, so in 64 bits
    x64 = x.double()
    score = _softmax(x64) if case["score"] == "softmax" else torch.sigmoid(x64)
    score = torch.where(x == -math.inf, -math.inf, score)
    if s["bias"] is not None:
        score = score + torch.nan_to_num(s["bias"].double(), nan=-math.inf, neginf=-math.inf,
                                         posinf=math.inf)
    choice = x64 if s["bias"] is None else score
    if G > 1:
        by = choice if case["group_score"] == "max" else score
        by = torch.sort(by.unflatten(-1, (G, -1)), dim=-1, descending=True).values
        value = by[..., 0]
        if case["group_score"] == "top2" and by.shape[-1] > 1:
            value = value + torch.where(by[..., 1] == -math.inf, 0.0, by[..., 1])
        order = torch.sort(value, dim=-1, descending=True, stable=True).indices
        keep = torch.zeros_like(value, dtype=torch.bool)
        keep.scatter_(-1, order[..., : case["kept"]], True)
        choice = torch.where(keep.repeat_interleave(choice.shape[-1] // G, -1), choice, -math.inf)
    top = torch.sort(choice, dim=-1, descending=True, stable=True)
    ids, there = top.indices[..., :k], top.values[..., :k] > -math.inf
    # how much of each: 32 bits
    if case["renormalize"]:
        w = _shares(torch.gather(x, -1, ids), there, case["score"])
    else:
        w = _softmax(x) if case["score"] == "softmax" else torch.sigmoid(x)
        w = torch.gather(w, -1, ids)
    w = torch.where(there, w * case["scale"], 0.0)
    return torch.where(there, ids, -1).to(torch.int32), w


def _shares(l, there, score):
    """Scores of the picks over their sum, free of 0/0 where all of them are tiny."""
    l = torch.where(there, l, -math.inf)
    if score == "softmax":
        return _softmax(l)
    low = l.clamp(max=0.0)
    top = low.amax(-1, keepdim=True).clamp(min=-_FLT_MAX)
    a = torch.exp(low - top) / (1 + torch.exp(-l.abs()))
    return a / a.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)


def _plain_route_backward(s, case):
    x = _clean(s["logits"])
    ids, there = s["ids"].clamp(min=0).long(), s["ids"] >= 0
    g = torch.where(there, s["grad_w"] * case["scale"], 0.0)
    dense = torch.zeros_like(x)
    if case["score"] == "softmax" and not case["renormalize"]:
        p = _softmax(x)
        dense.scatter_add_(-1, ids, g)
        dense = p * (dense - (dense * p).sum(-1, keepdim=True))
        return dense.to(s["logits"].dtype)
    l = torch.gather(x, -1, ids)
    if case["renormalize"]:
        p = _shares(l, there, case["score"])
        d = p * (g - (g * p).sum(-1, keepdim=True))
    else:
        d = g * torch.sigmoid(l)
    if case["score"] == "sigmoid":
        d = d * torch.sigmoid(-l)
    dense.scatter_add_(-1, ids, torch.where(there, d, 0.0))
    return dense.to(s["logits"].dtype)


def _plain_combine_backward(s, case):
    t, k = s["src_info"][:, 0].long(), s["src_info"][:, 1].long()
    slots = s["recv"][s["rank"], t * case["top_k"] + k]
    g = s["grad_out"][s["rank"], t].float()
    grad_w = torch.zeros_like(s["w"])
    grad_w[s["rank"], t, k] = (g * slots.float()).sum(-1)
    s["out"][: s["m"]] = s["w"][s["rank"], t, k].unsqueeze(-1) * g
    return grad_w, s["out"]


def _dequantized(s, case):
    """Weights [local][n][k] in 32 bits."""
    c = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten(-2)
    if case["fmt"] == "int4":
        v = c.float() - 8
    else:
        v = torch.tensor(_E2M1, device=c.device).index_select(0, c.flatten().int()).view(c.shape)
    v = v.unflatten(-1, (-1, case["group"])) * s["scales"].float().unsqueeze(-1)
    return v.flatten(-2)


def _grouped_product(s, case):
    """sum_k x[m][k] w[expert of m][n][k] for every row, in 32 bits."""
    group = s["offsets"][:: case["ranks"]].long()
    at = torch.arange(s["m"], device="cuda") - group[s["expert"]]
    x = torch.zeros(case["local"], s["x"].shape[1], max(1, s["rows_max"]), device="cuda")
    x[s["expert"], :, at] = s["x"].float()
    y = torch.bmm(_dequantized(s, case), x)
    return y[s["expert"], :, at]


def _plain_up(s, case):
    gate, up = _grouped_product(s, case).split(case["inter"], -1)
    s["out"][: s["m"]] = gate * torch.sigmoid(gate) * up
    return s["out"]


def _plain_down(s, case):
    y = _grouped_product(s, case).to(torch.bfloat16)
    slot = s["src_info"][:, 0].long() * case["top_k"] + s["src_info"][:, 1].long()
    s["recv"][s["rank"], slot] = y
    return list(s["recv"].unbind())


_PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward,
          "combine_backward": _plain_combine_backward, "up_w4": _plain_up, "down_w4": _plain_down}


# ---------------------------------------------------------------- bytes and operations


def _expected(case):
    """(rows, experts with rows, tokens with a local pick) of uniform routing."""
    R, T, E, L, k = (case[n] for n in ("ranks", "tokens", "experts", "local", "top_k"))
    none = 1.0
    for j in range(k):
        none *= max(0.0, (E - L - j) / (E - j))
    return R * T * k * L / E, L * (1 - (1 - k / E) ** (R * T)), R * T * (1 - none)


def work(case):
    tokens, k = case["ranks"] * case["tokens"], case["top_k"]
    if case["op"] in ("route", "route_backward"):
        values = tokens * case["experts"]
        size = 4 if case["dtype"] == "f32" else 2
        if case["op"] == "route":
            return {"bytes": values * size + tokens * k * 8 + 4 * case["experts"] * case["bias"],
                    "flops": 10 * values}
        # a renormalised or sigmoid gradient reads the picked logits alone
        dense = case["score"] == "softmax" and not case["renormalize"]
        read = values if dense else tokens * k
        return {"bytes": (read + values) * size + tokens * k * 8, "flops": 6 * read + 10 * tokens * k}
    rows, active, touched = _expected(case)
    N = case["hidden"]
    if case["op"] == "combine_backward":
        return {"bytes": 2 * N * (touched + 2 * rows) + tokens * k * 12 + rows * 8,
                "flops": 3 * rows * N}
    K = N if case["op"] == "up_w4" else case["inter"]
    n = 2 * case["inter"] if case["op"] == "up_w4" else N
    out = case["inter"] if case["op"] == "up_w4" else N
    return {"bytes": active * n * K * (0.5 + 2 / case["group"]) + 2 * rows * (K + out),
            "flops": 2 * rows * n * K}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = _inputs(case, seed)
    return _EXACT[case["op"]](s, case)


def _np(t):
    return t.double().cpu().numpy()


def _scores64(l, ok, score):
    """Scores of numpy logits; 0 where an expert is not eligible."""
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return np.where(ok, 1 / (1 + np.exp(-l)), 0.0)
        top = np.max(np.where(ok, l, -np.inf), -1, keepdims=True)
        e = np.where(ok, np.exp(l - top), 0.0)
        total = e.sum(-1, keepdims=True)
        return e / np.where(total > 0, total, 1.0)


def _exact_route(s, case):
    l = _np(s["logits"])
    E, k, G = case["experts"], case["top_k"], case["groups"]
    l = np.minimum(l.reshape(-1, E), _FLT_MAX)
    ok = l > -np.inf
    p = _scores64(l, ok, case["score"])
    if s["bias"] is not None:
        b = _np(s["bias"])
        ok = ok & (b > -np.inf)
    value = l if s["bias"] is None else p + b
    key = np.where(ok, value, -np.inf)
    rows = np.arange(len(l))[:, None]
    if G > 1:
        per = E // G
        if case["group_score"] == "max":
            by = key.reshape(-1, G, per).max(-1)
        else:
            summed = np.where(ok, p if s["bias"] is None else p + b, -np.inf)
            part = -np.sort(-summed.reshape(-1, G, per), -1)[..., :2]
            by = part[..., 0] + (np.where(np.isinf(part[..., 1]), 0.0, part[..., 1])
                                 if per > 1 else 0.0)
        first = np.argsort(-by, -1, kind="stable")[:, : case["kept"]]
        keep = np.zeros(by.shape, bool)
        keep[rows, first] = True
        key = np.where(np.repeat(keep, per, -1), key, -np.inf)
    ids = np.argsort(-key, -1, kind="stable")[:, :k]
    there = key[rows, ids] > -np.inf
    w = np.where(there, p[rows, ids], 0.0)
    if case["renormalize"]:
        total = w.sum(-1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    shape = (case["ranks"], case["tokens"], k)
    return [np.where(there, ids, -1).astype(np.int32).reshape(shape),
            (w * case["scale"]).reshape(shape)]


def _exact_route_backward(s, case):
    E, k = case["experts"], case["top_k"]
    l = np.minimum(_np(s["logits"]).reshape(-1, E), _FLT_MAX)
    ids = s["ids"].cpu().numpy().reshape(-1, k)
    g = case["scale"] * _np(s["grad_w"]).reshape(-1, k)
    rows = np.arange(len(l))[:, None]
    picked = np.zeros(l.shape, bool)
    dp = np.zeros(l.shape)
    for j in range(k):  # distinct picks
        at = ids[:, j] >= 0
        picked[rows[at, 0], ids[at, j]] = True
        dp[rows[at, 0], ids[at, j]] = g[at, j]
    p = _scores64(l, l > -np.inf, case["score"])
    if case["renormalize"]:
        q = np.where(picked, p, 0.0)
        total = q.sum(-1, keepdims=True)
        total = np.where(total > 0, total, 1.0)
        dp = np.where(picked, (dp - (dp * q).sum(-1, keepdims=True) / total) / total, 0.0)
    if case["score"] == "softmax":
        d = p * (dp - (dp * p).sum(-1, keepdims=True))
    else:
        d = dp * p * (1 - p)
    return d.reshape(case["ranks"], case["tokens"], E)


def _exact_combine_backward(s, case):
    T, k = case["tokens"], case["top_k"]
    pick = (s["rank"] * T + s["src_info"][:, 0]) * k + s["src_info"][:, 1]
    slots = s["recv"].view(-1, case["hidden"])[pick].double()
    g = s["grad_out"].view(-1, case["hidden"])[pick // k].double()
    grad_w = torch.zeros(case["ranks"] * T * k, dtype=torch.float64, device="cuda")
    grad_w[pick] = torch.mul(g, slots).sum(1)
    rows = torch.zeros(_capacity(case), case["hidden"], dtype=torch.float64, device="cuda")
    rows[: s["m"]] = g * s["w"].double().view(-1)[pick][:, None]
    return [grad_w.view(case["ranks"], T, k), rows]


def _exact_product(s, case):
    lo, hi = s["codes"] & 15, s["codes"] >> 4
    bounds = s["offsets"][:: case["ranks"]].tolist()
    table = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    if case["fmt"] == "int4":
        table = torch.arange(-8.0, 8.0, dtype=torch.float64, device="cuda")
    n = s["codes"].shape[1]
    y = torch.zeros(s["m"], n, dtype=torch.float64, device="cuda")
    for e in range(case["local"]):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        w = torch.empty(n, 2 * lo.shape[2], dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = table[lo[e].long()], table[hi[e].long()]
        w *= s["scales"][e].double().repeat_interleave(case["group"], 1)
        y[a:b] = torch.mm(s["x"][a:b].double(), w.t().contiguous())
    return y


def _exact_up(s, case):
    y = _exact_product(s, case)
    g, u = y[:, : case["inter"]], y[:, case["inter"]:]
    h = torch.zeros(_capacity(case), case["inter"], dtype=torch.float64, device="cuda")
    h[: s["m"]] = g / (1 + torch.exp(-g)) * u
    return h


def _exact_down(s, case):
    y = _exact_product(s, case)
    out = torch.zeros(case["ranks"], case["tokens"] * case["top_k"], case["hidden"],
                      dtype=torch.float64, device="cuda")
    out[s["rank"], s["src_info"][:, 0].long() * case["top_k"] + s["src_info"][:, 1].long()] = y
    return list(out)


_EXACT = {"route": _exact_route, "route_backward": _exact_route_backward,
          "combine_backward": _exact_combine_backward, "up_w4": _exact_up, "down_w4": _exact_down}
