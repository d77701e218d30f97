"""Cases that time the RMS norm in front of a mixture-of-experts layer, its gradient, and
the whole layer for a few tokens: `run` computes them with elementary torch operations,
or with this library's calls where `own` is true.

A case names one operator (`op`) and the share of an expert-parallel layer it works on:
`ranks` source ranks of `tokens` tokens each, rows of `hidden` values, and for the layer
`experts` in all, the first `local` of them on this GPU, `top_k` picks a token."""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
_EPS = 1e-6
_E4M3_MAX = 448.0


def _norm(op, name, **kw):
    case = dict(op=op, ranks=8, tokens=4096, hidden=7168, dtype="bf16", weight="bf16",
                residual="bf16", rows=True, fp8=False)
    case.update(kw)
    return dict(case, **({"name": name} if name else {}))


def _moe(name, **kw):
    case = dict(op="moe_layer", ranks=1, tokens=1, hidden=7168, inter=2048, experts=32, local=32,
                top_k=8, fmt="bf16", group=128, scales="bf16", zipf=False)
    case.update(kw)
    return dict(case, **({"name": name} if name else {}))


def listed():
    return [
        # the norm of one decoded token: rows for the router, codes for the experts; latency
        _norm("rms_norm", "norm_one_token", ranks=1, tokens=1, fp8=True),
        # the same of a prefill step
        _norm("rms_norm", "norm_prefill_fp8", fp8=True),
        # fp16 rows beside a residual stream in 32 bits, odd sizes
        _norm("rms_norm", "norm_odd", ranks=3, tokens=1111, hidden=3968, dtype="f16",
              weight="f32", residual="f32"),
        # the training step of the same norms; the second small, odd and without a residual
        _norm("rms_norm_backward", "norm_backward_prefill"),
        _norm("rms_norm_backward", "norm_backward_odd", ranks=3, tokens=77, hidden=2176,
              dtype="f32", weight="f32", residual="none"),
        # one token through a small layer: latency alone counts
        _moe("moe_small", hidden=1024, inter=256, experts=16, local=16, top_k=2),
        # one token, every expert on this GPU, in each kind of weights
        _moe("moe_bf16_one_token"),
        _moe("moe_fp8_one_token", fmt="fp8"),
        _moe("moe_int4_one_token", fmt="int4", scales="f16"),
        # the few tokens of a speculative step, five and not a power of two
        _moe("moe_fp8_five_tokens", fmt="fp8", tokens=5),
        # small decode batches from eight ranks on this GPU's share of the experts
        _moe("moe_bf16_batch", ranks=8, tokens=2, hidden=4096, inter=1024, experts=64, local=16),
        _moe("moe_e2m1_batch", ranks=8, tokens=8, experts=256, local=32, fmt="e2m1", group=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rms_norm", "rms_norm_backward", "moe_layer", "moe_layer"])
    ranks = rng.randint(1, 8)
    if op != "moe_layer":
        dtype = rng.choice(["f32", "bf16", "f16"])
        rows, fp8 = rng.choice([(True, False), (True, True), (False, True)])
        return _norm(op, None, ranks=ranks, tokens=_log(rng, 1, 2048),
                     hidden=128 * _log(rng, 1, 64), dtype=dtype,
                     weight=rng.choice([dtype, "f32"]),
                     residual=rng.choice(["none", dtype, "f32"]), rows=rows, fp8=fp8)
    top_k = rng.randint(1, 8)
    local = rng.randint(top_k, 32)
    return _moe(None, ranks=ranks, tokens=_log(rng, 1, 64 // ranks), hidden=128 * _log(rng, 2, 56),
                inter=128 * _log(rng, 1, 16), experts=local * rng.randint(1, 8), local=local,
                top_k=top_k, fmt=rng.choice(["bf16", "fp8", "int4", "e2m1"]),
                group=rng.choice([32, 64, 128]), scales=rng.choice(["bf16", "f16"]),
                zipf=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _norm_inputs(case, g):
    R, T, N = case["ranks"], case["tokens"], case["hidden"]
    D, W = _TYPES[case["dtype"]], _TYPES[case["weight"]]
    RD = None if case["residual"] == "none" else _TYPES[case["residual"]]
    # tokens of differing size, a few channels that stand out
    size = torch.exp(0.5 * _randn(g, R, T, 1)).to(D)
    channel = torch.where(_rand(g, N) < 0.005, 8.0, 1.0)
    s = {"weight": (0.8 + 0.4 * _rand(g, N)).to(W)}
    if case["op"] == "rms_norm":
        s["x"] = _randn(g, R, T, N, dtype=D).mul_(size)
        s["residual"] = None
        if RD is not None:
            s["residual"] = _randn(g, R, T, N, dtype=RD).mul_((2 * channel).to(RD))
    else:
        # the stored sums of the forward pass, and the gradients that reach its outputs
        s["sums"] = _randn(g, R, T, N, dtype=RD or D).mul_((2 * channel).to(RD or D))
        s["grad_out"] = _randn(g, R, T, N, dtype=D).mul_(0.01)
        s["grad_residual"] = None
        if RD is not None:
            s["grad_residual"] = _randn(g, R, T, N, dtype=RD).mul_(0.01)
    return s


def _codes_4bit(case, g, n, k):
    """Codes [local][n][k/2] (even k in the low bits) and scales [local][n][k/group] of
    normally distributed weights of size 1/sqrt(k)."""
    E = case["local"]
    v = _randn(g, E, n, k, dtype=torch.bfloat16)
    if case["fmt"] == "int4":
        c = (v.mul_(2.7).round_() + 8).clamp_(0, 15).to(torch.uint8)
        step = 1 / 2.7
    else:
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda",
                             dtype=torch.bfloat16)
        c = torch.bucketize(v.abs().mul_(2.0), edges, out_int32=True).to(torch.uint8)
        c |= (v < 0).to(torch.uint8) << 3
        step = 0.5
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    scales = (step / math.sqrt(k)) * (0.75 + 0.5 * _rand(g, E, n, k // case["group"]))
    return codes, scales.to(_TYPES[case["scales"]])


def _stack(case, g, n, k):
    """The weights [local][n][k] of one product and their scales (None for bf16)."""
    E = case["local"]
    if case["fmt"] == "bf16":
        return _randn(g, E, n, k, dtype=torch.bfloat16).mul_(1 / math.sqrt(k)), None
    if case["fmt"] == "fp8":
        # e4m3fn codes and a scale for 128 x 128 of them
        codes = _randn(g, E, n, k, dtype=torch.bfloat16).mul_(100.0).clamp_(-448, 448)
        scales = (0.01 / math.sqrt(k)) * (0.75 + 0.5 * _rand(g, E, n // 128, k // 128))
        return codes.to(torch.float8_e4m3fn), scales
    return _codes_4bit(case, g, n, k)


def _moe_inputs(case, g):
    R, T, E, k = case["ranks"], case["tokens"], case["experts"], case["top_k"]
    N, I = case["hidden"], case["inter"]
    u = _rand(g, R, T, E).clamp_(1e-7, 1 - 1e-7)
    keys = -torch.log(-torch.log(u))
    if case["zipf"]:
        keys -= 1.2 * torch.log(torch.randperm(E, generator=g, device="cuda") + 1.0)
    s = {"ids": torch.topk(keys, k, dim=-1).indices.to(torch.int32),
         "w": torch.softmax(_randn(g, R, T, k), -1)}
    # normalised rows, as the norm in front of the layer makes them
    x = _randn(g, R, T, N)
    s["x_scale"] = None
    if case["fmt"] == "fp8":
        blocks = x.view(R, T, N // 128, 128)
        s["x_scale"] = blocks.abs().amax(-1) / _E4M3_MAX
        x = (blocks / s["x_scale"].unsqueeze(-1)).view(R, T, N).to(torch.float8_e4m3fn)
    else:
        x = x.to(torch.bfloat16)
    s["x"] = x
    s["w1"], s["w1_scale"] = _stack(case, g, 2 * I, N)
    s["w2"], s["w2_scale"] = _stack(case, g, N, I)
    return s


def _inputs(case, seed):
    g = _generator(seed)
    return _moe_inputs(case, g) if case["op"] == "moe_layer" else _norm_inputs(case, g)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        # the handle that a program keeps for the layer, and the weights laid out once
        from grouped_gemm_scatter_amd import EpCombine
        moe = case["op"] == "moe_layer"
        s["ctx"] = ctx = EpCombine(
            n_ranks=case["ranks"], top_k=case.get("top_k", 1), max_tokens_per_rank=case["tokens"],
            n_experts_per_device=case.get("local", 1), hidden_k=case.get("inter", 128),
            hidden_n=case["hidden"], dtype="fp8" if case.get("fmt") == "fp8" else "bf16")
        if moe and case["fmt"] in ("int4", "e2m1"):
            for w in ("w1", "w2"):
                s[w] = ctx.pack_weights_w4(s[w], s.pop(w + "_scale"), codes=case["fmt"])
        elif moe and case["fmt"] == "fp8":
            for t in ("x", "w1", "w2"):  # the library takes codes as bytes
                s[t] = s[t].view(torch.uint8)
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](state, case, state["ctx"])
    return _PLAIN[case["op"]](state, case)


def _outputs(out, codes, scales, residual):
    got = {"out": out, "codes": codes, "scales": scales, "residual": residual}
    return {name: t for name, t in got.items() if t is not None}


def _own_norm(s, case, ctx):
    y = ctx.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=_EPS, rows=case["rows"],
                     fp8=case["fp8"])
    codes = None if y.codes is None else y.codes.view(torch.float8_e4m3fn)
    return _outputs(y.out, codes, y.scales, y.residual)


def _own_norm_backward(s, case, ctx):
    d = ctx.rms_norm_backward(s["grad_out"], s["sums"], s["weight"],
                              grad_residual=s["grad_residual"], eps=_EPS)
    return _gradients(case, d.x, d.residual, d.weight)


def _own_moe(s, case, ctx):
    if case["fmt"] != "fp8":
        return ctx.moe_layer(s["x"], s["w1"], s["w2"], s["ids"], s["w"])
    return ctx.moe_layer(s["x"], s["w1"], s["w2"], s["ids"], s["w"], x_scale=s["x_scale"],
                         w1_scale=s["w1_scale"], w2_scale=s["w2_scale"])


_OWN = {"rms_norm": _own_norm, "rms_norm_backward": _own_norm_backward, "moe_layer": _own_moe}


def _gradients(case, x, residual, weight):
    """The sum's gradient is that of both its terms: once where they have one type."""
    got = {"x": x, "weight": weight}
    if case["residual"] not in ("none", case["dtype"]):
        got["residual"] = residual
    return got


def _plain_norm(s, case):
    r = s["x"].float()
    kept = None
    if s["residual"] is not None:
        r = r + s["residual"].float()
        kept = r.to(s["residual"].dtype)
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS) * s["weight"].float()
    out = y.to(s["x"].dtype) if case["rows"] else None
    codes = scales = None
    if case["fp8"]:
        blocks = y.unflatten(-1, (-1, 128))
        scales = blocks.abs().amax(-1) / _E4M3_MAX
        scales = torch.where(scales > 0, scales, 1.0)
        codes = (blocks / scales.unsqueeze(-1)).flatten(-2).to(torch.float8_e4m3fn)
    return _outputs(out, codes, scales, kept)


def _plain_norm_backward(s, case):
    r, g = s["sums"].float(), s["grad_out"].float()
    inv = torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS)
    xh = r * inv
    gw = g * s["weight"].float()
    d = inv * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    if s["grad_residual"] is not None:
        d = d + s["grad_residual"].float()
    dw = (g * xh).sum((0, 1))
    return _gradients(case, d.to(s["grad_out"].dtype), d.to(s["sums"].dtype), dw)


def _values(w, scales, case):
    """Weights of some experts in 32 bits."""
    if case["fmt"] == "bf16":
        return w.float()
    if case["fmt"] == "fp8":
        v = w.float().unflatten(1, (-1, 128)).unflatten(3, (-1, 128))
        return (v * scales[:, :, None, :, None]).flatten(3).flatten(1, 2)
    c = torch.stack([w & 15, w >> 4], -1).flatten(-2)
    if case["fmt"] == "int4":
        v = c.float() - 8
    else:
        v = torch.tensor(_E2M1, device=c.device).index_select(0, c.flatten().int()).view(c.shape)
    return (v.unflatten(-1, (-1, case["group"])) * scales.float().unsqueeze(-1)).flatten(-2)


def _plain_moe(s, case):
    k, N = case["top_k"], case["hidden"]
    ids, w = s["ids"].view(-1, k).long(), s["w"].view(-1, k)
    x = s["x"].view(-1, N).float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].view(-1, N // 128).repeat_interleave(128, 1)
    # the experts with tokens, and each token's weight of each
    active = torch.unique(ids[ids < case["local"]])
    share = ((ids[None] == active[:, None, None]) * w[None]).sum(-1)
    some = [None if t is None else t[active] for t in (s["w1_scale"], s["w2_scale"])]
    gate, up = torch.matmul(_values(s["w1"][active], some[0], case),
                            x.t().contiguous()).split(case["inter"], 1)
    h = gate * torch.sigmoid(gate) * up * share[:, None, :]
    y = torch.bmm(_values(s["w2"][active], some[1], case), h).sum(0)
    return y.t().to(torch.bfloat16).view(case["ranks"], case["tokens"], N).contiguous()


_PLAIN = {"rms_norm": _plain_norm, "rms_norm_backward": _plain_norm_backward,
          "moe_layer": _plain_moe}


# ---------------------------------------------------------------- bytes and operations


def work(case):
    rows, N = case["ranks"] * case["tokens"], case["hidden"]
    size = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
    if case["op"] == "moe_layer":
        # uniform routing: picks on this GPU, and experts with at least one
        E, L, k, I = case["experts"], case["local"], case["top_k"], case["inter"]
        picks, active = rows * k * L / E, L * (1 - (1 - k / E) ** rows)
        one = {"bf16": 2, "fp8": 1 + 4 / 128 ** 2}.get(case["fmt"], 0.5 + 2 / case["group"])
        x = 1 + 4 / 128 if case["fmt"] == "fp8" else 2
        return {"bytes": active * 3 * I * N * one + rows * (N * (x + 2) + 8 * k),
                "flops": 6 * picks * I * N}
    d, res = size[case["dtype"]], size[case["residual"]]
    if case["op"] == "rms_norm":
        out = case["rows"] * d + case["fp8"] * (1 + 4 / 128)
        return {"bytes": rows * N * (d + 2 * res + out) + N * size[case["weight"]],
                "flops": (6 + 4 * case["fp8"]) * rows * N}
    # read: the gradient, the sums, the other gradient; written: one or two of the sum
    kept = res or d
    written = d + (res if res and case["residual"] != case["dtype"] else 0)
    return {"bytes": rows * N * (d + kept + res + written) + N * (4 + size[case["weight"]]),
            "flops": 12 * rows * N}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = _inputs(case, seed)
    return _EXACT[case["op"]](s, case)


def _exact_norm(s, case):
    total = s["x"].double()
    if s["residual"] is not None:
        total = total.add_(s["residual"])
    length = torch.linalg.vector_norm(total, dim=-1, keepdim=True)
    y = total / torch.sqrt(length * length / case["hidden"] + _EPS)
    y = y.mul_(s["weight"])
    codes = scales = None
    if case["fp8"]:
        scales = torch.stack([b.abs().amax(-1) for b in y.split(128, -1)], -1) / _E4M3_MAX
        scales[scales == 0] = 1.0
        codes = y / scales.repeat_interleave(128, -1)
    return _outputs(y if case["rows"] else None, codes, scales,
                    total if s["residual"] is not None else None)


def _exact_norm_backward(s, case):
    r, g = s["sums"].double(), s["grad_out"].double()
    n = case["hidden"]
    power = torch.linalg.vecdot(r, r).unsqueeze(-1) / n + _EPS
    g.div_(power.sqrt())
    dw = (g * r).sum((0, 1))
    g.mul_(s["weight"])
    g -= r * (torch.linalg.vecdot(g, r).unsqueeze(-1) / (n * power))
    if s["grad_residual"] is not None:
        g += s["grad_residual"]
    return _gradients(case, g, g, dw)


def _exact_stack(w, scale, case):
    """One expert's weights [n][k]."""
    if case["fmt"] == "bf16":
        return w.double()
    if case["fmt"] == "fp8":
        return w.double() * scale.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    table = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    if case["fmt"] == "int4":
        table = torch.arange(-8.0, 8.0, dtype=torch.float64, device="cuda")
    v = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device="cuda")
    v[:, 0::2], v[:, 1::2] = table[(w & 15).long()], table[(w >> 4).long()]
    return v * scale.double().repeat_interleave(case["group"], 1)


def _exact_moe(s, case):
    k, N, I = case["top_k"], case["hidden"], case["inter"]
    x = s["x"].view(-1, N).double()
    if s["x_scale"] is not None:
        x *= s["x_scale"].view(-1, N // 128).double().repeat_interleave(128, 1)
    out = torch.zeros_like(x)
    ids, w = s["ids"].view(-1, k), s["w"].view(-1, k).double()
    for e in range(case["local"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        one = [None if s[n] is None else s[n][e] for n in ("w1_scale", "w2_scale")]
        a = torch.mm(_exact_stack(s["w1"][e], one[0], case), x[t].t().contiguous())
        a = a[:I] / (1 + torch.exp(-a[:I])) * a[I:]
        y = torch.mm(_exact_stack(s["w2"][e], one[1], case), a)
        out.index_add_(0, t, y.t() * w[t, j, None])
    return out.view(case["ranks"], case["tokens"], N)


_EXACT = {"rms_norm": _exact_norm, "rms_norm_backward": _exact_norm_backward,
          "moe_layer": _exact_moe}
