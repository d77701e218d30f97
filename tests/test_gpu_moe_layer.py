"""The whole layer for a few tokens against float64, in every kind of weights; then with
the norms and the router around it, and against the path through the grouped layout.
Tolerances are the bound that oracle/operators.py derives for its sums, and half a bf16
step for the output."""
import numpy as np
import pytest
import torch

import oracle as O
from ep_synth import TINY
from grouped_gemm_scatter_amd import EpCombine, EpError
from grouped_gemm_scatter_amd import binding as B
from gpu_helpers import bits, make_ctx, to_dev
from oracle import operators as P

pytestmark = pytest.mark.gpu

SCALES = {"bf16": torch.bfloat16, "f16": torch.float16}
FORMATS = ["bf16", "bf16_sliced", "fp8"] + [
    (c, g, s) for c in ("int4", "e2m1") for g, s in ((32, "bf16"), (32, "f16"), (64, "f16"),
                                                    (64, "bf16"), (128, "bf16"), (128, "f16"))]


def _id(f):
    return f if isinstance(f, str) else "-".join(map(str, f))


class Layer:
    """A handle, random weights of every expert as the library takes them and as numbers."""

    def __init__(self, fmt, El, hidden, inter, R=1, T=1, top_k=2, my_rank=0, seed=0, **kw):
        rng = np.random.default_rng(seed)
        self.fp8 = fmt == "fp8"
        self.ctx = EpCombine(n_ranks=R, top_k=top_k, max_tokens_per_rank=T, my_rank=my_rank,
                             n_experts_per_device=El, hidden_k=inter, hidden_n=hidden,
                             dtype="fp8" if self.fp8 else "bf16",
                             w_slice_major=fmt == "bf16_sliced", **kw)
        self.lo = my_rank * El
        self.args, self.scales, self.values = [], {}, []
        for name, rows, k in (("w1", 2 * inter, hidden), ("w2", hidden, inter)):
            if isinstance(fmt, str) and not self.fp8:
                w = O.f64_to_bf16(rng.standard_normal((El, rows, k)) / np.sqrt(k))
                self.values.append(O.bf16_to_f64(w))
                d = to_dev(w, torch.bfloat16)
                if fmt == "bf16_sliced" and name == "w2":
                    d = self.ctx.pack_weights(d)
                self.args.append(d)
            elif self.fp8:
                c = rng.integers(0, 256, (El, rows, k), dtype=np.uint8)
                c[(c & 0x7F) == 0x7F] = 0                # no NaN
                s = ((0.5 + rng.random((El, rows // 128, k // 128))) /
                     (100 * np.sqrt(k))).astype(np.float32)
                self.values.append(O.e4m3fn_to_f64(c) *
                                   np.repeat(np.repeat(s.astype(np.float64), 128, 1), 128, 2))
                self.args.append(to_dev(c))
                self.scales[name + "_scale"] = to_dev(s)
            else:
                codes_are, group, st = fmt
                c = rng.integers(0, 256, (El, rows, k // 2), dtype=np.uint8)
                s = torch.from_numpy((0.5 + rng.random((El, rows, k // group))) /
                                     (5 * np.sqrt(k))).to(SCALES[st])
                self.values.append(P.weights_w4(c, s.double().numpy(), codes_are))
                self.args.append(self.ctx.pack_weights_w4(to_dev(c), s.cuda(), codes=codes_are))

    def rows(self, rng, R, T, hidden):
        """(arguments x and x_scale, the rows as numbers [R*T][hidden])."""
        x = rng.standard_normal((R * T, hidden))
        if not self.fp8:
            b = O.f64_to_bf16(x)
            return (to_dev(b, torch.bfloat16).view(R, T, hidden), {}), O.bf16_to_f64(b)
        c, s = O.quantize_rows_e4m3(x.astype(np.float32))
        return ((to_dev(c).view(R, T, hidden),
                 {"x_scale": to_dev(s).view(R, T, hidden // 128)}),
                O.e4m3fn_to_f64(c) * np.repeat(s.astype(np.float64), 128, axis=1))

    def __call__(self, x, ids, tw, **kw):
        return self.ctx.moe_layer(x[0], *self.args, ids, tw, **x[1], **self.scales, **kw)

    def check(self, got, values, ids, tw):
        N = values.shape[1]
        k = ids.shape[-1]
        want, bound = P.moe_layer(values, *self.values, ids.reshape(-1, k), tw.reshape(-1, k),
                                  self.lo)
        out = O.bf16_to_f64(bits(got)).reshape(-1, N)
        err = np.abs(out - want)
        tol = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 1e-38
        good = bool(np.all(err <= tol))
        assert good, float((err / tol).max())
        none = ~((ids >= self.lo) & (ids < self.lo + self.ctx.n_experts_per_device)).any(-1)
        assert np.all(bits(got).reshape(-1, N)[none.reshape(-1)] == 0)


def _picks(rng, R, T, k, E):
    ids = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k)
                    for _ in range(R * T)])
    return ids.reshape(R, T, k).astype(np.int32), rng.random((R, T, k)).astype(np.float32)


def _run(fmt, R, T, El, k, hidden, inter, E=None, my_rank=0, edit=None, seed=1):
    print(f"[case] moe {_id(fmt)} R={R} T={T} El={El} k={k} hidden={hidden} inter={inter}",
          flush=True)
    rng = np.random.default_rng(seed)
    layer = Layer(fmt, El, hidden, inter, R, T, k, my_rank, seed)
    ids, tw = _picks(rng, R, T, k, E or El)
    if edit is not None:
        edit(ids, tw)
    x, values = layer.rows(rng, R, T, hidden)
    got = layer(x, to_dev(ids), to_dev(tw))
    torch.cuda.synchronize()
    assert layer.ctx.query_error() == 0
    layer.check(got, values, ids, tw)
    return layer, x, ids, tw, got


@pytest.mark.parametrize("fmt", FORMATS, ids=_id)
@pytest.mark.parametrize("tokens", [1, 3, 16, 17, 64])
def test_every_kind_of_weights(fmt, tokens):
    _run(fmt, 1, tokens, 6, 2, 384, 256)


@pytest.mark.parametrize("fmt", ["bf16", "bf16_sliced", "fp8", ("int4", 128, "f16"),
                                 ("e2m1", 32, "bf16")], ids=_id)
@pytest.mark.parametrize("hidden,inter", [(128, 128), (256, 1152), (2176, 128), (1152, 640)])
def test_widths(fmt, hidden, inter):
    """Fewer steps than waves, as many, more and not a multiple; one to 72 column blocks."""
    _run(fmt, 1, 5, 4, 3, hidden, inter)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", ("int4", 64, "bf16")], ids=_id)
def test_a_rank_in_the_middle_with_dropped_picks(fmt):
    def edit(ids, tw):
        ids[0, 0] = -1                             # a token without picks
        ids[1, 1] = [0, 3, 23]                     # and one without local ones
        ids[2, 2, 1] = -7
        ids[3, 3, 0] = 1 << 30
        tw[0, 0] = np.nan                          # weights of dropped picks count nothing
    _run(fmt, 4, 9, 5, 3, 256, 256, E=20, my_rank=2, edit=edit)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", ("e2m1", 64, "f16")], ids=_id)
def test_no_local_picks_at_all(fmt):
    layer, x, ids, tw, got = _run(fmt, 2, 4, 3, 2, 128, 128, E=3, my_rank=1)
    assert torch.all(got == 0)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", ("int4", 32, "f16")], ids=_id)
@pytest.mark.parametrize("tokens", [13, 33, 64])
def test_all_tokens_on_one_expert_and_the_same_expert_twice(fmt, tokens):
    def edit(ids, tw):
        ids[...] = 2
        ids[0, ::3, 1] = 0
        tw[0, ::4, 0] *= -1
    _run(fmt, 1, tokens, 3, 4, 256, 128, edit=edit)


def test_many_experts_and_many_picks():
    _run("bf16", 1, 64, 256, 16, 128, 128)         # 1024 picks
    _run("fp8", 1, 16, 256, 64, 128, 128, E=300)   # 64 picks a token
    _run(("int4", 128, "bf16"), 8, 8, 256, 8, 128, 128)


def test_eight_ranks_are_one_batch():
    """The tokens of the ranks in order: the same as one rank's."""
    layer, x, ids, tw, got = _run("bf16", 8, 3, 8, 2, 256, 256)
    one = Layer("bf16", 8, 256, 256, 1, 24, 2, 0, 1)
    again = one((x[0].view(1, 24, 256), {}), to_dev(ids.reshape(1, 24, 2)),
                to_dev(tw.reshape(1, 24, 2)))
    assert torch.equal(got.view(24, 256), again.view(24, 256))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", ("e2m1", 32, "f16")], ids=_id)
@pytest.mark.parametrize("tokens", [9, 40])
def test_numbers_without_an_end_stay_with_their_token_and_expert(fmt, tokens):
    layer, x, ids, tw, got = _run(fmt, 1, tokens, 5, 2, 256, 256)
    bad = x[0].clone()
    if layer.fp8:
        bad[0, 2, 7] = 0x7F
    else:
        bad[0, 2, 7] = float("inf")
        bad[0, tokens - 1, 255] = float("nan")
    keep = torch.ones(tokens, dtype=torch.bool)
    keep[2] = False
    if not layer.fp8:
        keep[tokens - 1] = False
    out = layer((bad, x[1]), to_dev(ids), to_dev(tw))
    assert torch.equal(out[0, keep], got[0, keep])
    assert not torch.isfinite(out[0, ~keep]).all(-1).any()
    # an expert's weights: only the tokens that picked it
    without = torch.from_numpy(~(ids == 3).any(-1)[0])
    assert without.any() and not without.all()
    if isinstance(fmt, str):
        for w in layer.args:
            if layer.fp8:
                w[3, 5] = 0x7F
            else:
                w[3, 5] = float("nan")
    else:
        for w in layer.args:
            w.scales.view(5, -1)[3, :4] = float("nan")
    out = layer(x, to_dev(ids), to_dev(tw))
    assert torch.equal(out[0, without], got[0, without])
    assert not torch.isfinite(out[0, ~without].float()).all(-1).any()


def test_one_token_of_a_large_layer():
    """7168 x 2048 in bf16, every expert of a step picked once by one of the tokens."""
    torch.manual_seed(3)
    hidden, inter, El, T, k = 7168, 2048, 8, 3, 8
    ctx = EpCombine(n_ranks=1, top_k=k, max_tokens_per_rank=T, n_experts_per_device=El,
                    hidden_k=inter, hidden_n=hidden)
    w1 = (torch.randn(El, 2 * inter, hidden, device="cuda") / hidden ** 0.5).bfloat16()
    w2 = (torch.randn(El, hidden, inter, device="cuda") / inter ** 0.5).bfloat16()
    x = torch.randn(1, T, hidden, device="cuda").bfloat16()
    ids = torch.stack([torch.randperm(El) for _ in range(T)])[None].int().cuda()
    ids[0, 1, 5:] = -1
    tw = torch.rand(1, T, k, device="cuda")
    got = ctx.moe_layer(x, w1, w2, ids, tw)
    torch.cuda.synchronize()
    want, bound = P.moe_layer(_f64(x)[0], _f64(w1), _f64(w2), ids[0].cpu().numpy(),
                              _f64(tw)[0])
    err = np.abs(_f64(got)[0] - want)
    good = bool(np.all(err <= bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)))
    assert good, float(err.max())


def _f64(t):
    return t.double().cpu().numpy()


def test_a_stack_past_four_gib():
    """256 experts whose w1 in bf16 is over 4 GiB: the last one's offsets."""
    hidden, inter, El = 4096, 1024, 256
    ctx = EpCombine(n_ranks=1, top_k=2, max_tokens_per_rank=4, n_experts_per_device=El,
                    hidden_k=inter, hidden_n=hidden)
    w1 = torch.empty(El, 2 * inter, hidden, dtype=torch.bfloat16, device="cuda")
    w2 = torch.empty(El, hidden, inter, dtype=torch.bfloat16, device="cuda")
    for w in (w1, w2):
        w.normal_(std=w.shape[-1] ** -0.5)
    assert w1.numel() * 2 >= 1 << 32
    x = torch.randn(1, 4, hidden, device="cuda").bfloat16()
    ids = torch.tensor([[[255, 0], [254, 255], [3, 200], [-1, 255]]], dtype=torch.int32,
                       device="cuda")
    tw = torch.rand(1, 4, 2, device="cuda")
    got = ctx.moe_layer(x, w1, w2, ids, tw)
    torch.cuda.synchronize()
    used = sorted(set(ids.flatten().tolist()) - {-1})
    few = np.searchsorted(used, ids[0].cpu().numpy())
    few[ids[0].cpu().numpy() < 0] = -1
    want, bound = P.moe_layer(_f64(x)[0], _f64(w1[used]), _f64(w2[used]), few, _f64(tw)[0])
    err = np.abs(_f64(got)[0] - want)
    good = bool(np.all(err <= bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)))
    assert good, float(err.max())


@pytest.mark.parametrize("fmt", ["bf16", "bf16_sliced", "fp8", ("int4", 64, "bf16")], ids=_id)
def test_it_is_what_the_grouped_path_gives(fmt):
    """route, then the layer in one call against group, dispatch, both products and the
    combine, whose second product's rows (and H of the fp8 path) are rounded once more."""
    R, T, E, k, hidden, inter = 2, 7, 16, 4, 512, 384
    layer = Layer(fmt, 8, hidden, inter, R, T, k, 1, 4)
    ctx = layer.ctx
    rng = np.random.default_rng(5)
    logits = to_dev(rng.standard_normal((R, T, E)).astype(np.float32))
    ids, tw = ctx.route(logits, score="sigmoid", scale=2.0)
    x, values = layer.rows(rng, R, T, hidden)
    got = layer(x, ids, tw)
    off, src = ctx.group(ids)
    m = int(off[-1])
    out = torch.empty(R, T, hidden, dtype=torch.bfloat16, device="cuda")
    x1 = torch.empty(m, hidden, dtype=x[0].dtype, device="cuda")
    ctx.dispatch(x[0], off, src, m, x1)
    ctx.next_epoch()
    if layer.fp8:
        x1s = torch.empty(m, hidden // 128, device="cuda")
        ctx.dispatch(x[1]["x_scale"], off, src, m, x1s)
        h = torch.empty(m, inter, dtype=torch.uint8, device="cuda")
        hs = torch.empty(m, inter // 128, device="cuda")
        ctx.up_swiglu_fp8(x1, x1s, layer.args[0], layer.scales["w1_scale"], off, m, h, hs)
        ctx.gemm_scatter(h, layer.args[1], off, src, m, x_scale=hs,
                         w_scale=layer.scales["w2_scale"])
    else:
        h = torch.empty(m, inter, dtype=torch.bfloat16, device="cuda")
        if isinstance(fmt, str):
            ctx.up_swiglu(x1, layer.args[0], off, m, h)
            ctx.gemm_scatter(h, layer.args[1], off, src, m)
        else:
            ctx.up_swiglu_w4(x1, layer.args[0], off, m, h)
            ctx.gemm_scatter_w4(h, layer.args[1], off, src, m)
    ctx.combine(ids, tw, out)
    torch.cuda.synchronize()
    assert ctx.query_error() == 0
    ids_h, tw_h = ids.cpu().numpy(), _f64(tw)
    layer.check(got, values, ids_h, tw_h)
    want, bound = P.moe_layer(values, *layer.values, ids_h.reshape(-1, k), tw_h.reshape(-1, k),
                              layer.lo)
    # the path's own extra roundings: each pick's row to bf16, within 2^-8 of sizes whose
    # sum the absolute products bound; for fp8, H once more to half a step of e4m3
    a1, a2 = np.abs(layer.values[0]), np.abs(layer.values[1])
    extra = np.zeros_like(want)
    for t in range(R * T):
        for j in range(k):
            e = ids_h.reshape(-1, k)[t, j] - layer.lo
            if 0 <= e < 8:
                y = layer.values[0][e] @ values[t]
                hid = np.abs(y[:inter] / (1 + np.exp(-y[:inter])) * y[inter:])
                c = tw_h.reshape(-1, k)[t, j]
                extra[t] += c * 2.0 ** -8 * 1.1 * (a2[e] @ hid)
                if layer.fp8:
                    top = np.repeat(hid.reshape(-1, 128).max(-1), 128)
                    extra[t] += c * 1.1 * (a2[e] @ np.maximum(2.0 ** -4 * hid,
                                                              2.0 ** -10 * top / 448))
    err = np.abs(_f64(out).reshape(-1, hidden) - _f64(got).reshape(-1, hidden))
    assert np.all(err <= 2 * bound + extra + 2.0 ** -7 * np.abs(want) + 1e-30)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", ("e2m1", 128, "bf16")], ids=_id)
@pytest.mark.parametrize("tokens", [1, 6])
def test_norm_route_layer_norm(fmt, tokens):
    """As a decode step uses them: the norm with the residual, the router's logits from its
    rows, the layer on its rows or codes, the next norm with the layer's output.  Each stage
    against float64 on what the kernels left before it; captured and replayed."""
    R, E, k, hidden, inter = 2, 8, 2, 512, 256
    layer = Layer(fmt, E, hidden, inter, R, tokens, k, 0, 6)
    ctx = layer.ctx
    gen = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, res = rnd(R, tokens, hidden).bfloat16(), rnd(R, tokens, hidden)
    gain, router = (1 + 0.1 * rnd(hidden)).bfloat16(), (rnd(hidden, E) / hidden ** 0.5).bfloat16()

    def step(stream=None):
        y = ctx.rms_norm(x, gain, residual=res, fp8=layer.fp8)
        logits = (y.out.view(-1, hidden).float() @ router.float()).view(R, tokens, E)
        ids, tw = ctx.route(logits)
        rows = (y.codes, {"x_scale": y.scales}) if layer.fp8 else (y.out, {})
        z = layer(rows, ids, tw)
        n = ctx.rms_norm(z, gain, residual=y.residual)
        return y, ids, tw, rows, z, n

    def check(y, ids, tw, rows, z, n):
        if layer.fp8:
            values = (O.e4m3fn_to_f64(rows[0].cpu().numpy()) *
                      np.repeat(_f64(rows[1]["x_scale"]), 128, axis=-1))
        else:
            values = _f64(rows[0])
        layer.check(z, values.reshape(-1, hidden), ids.cpu().numpy(), _f64(tw))
        s, want = P.rms_norm(_f64(x), _f64(gain), residual=_f64(res))
        assert np.all(np.abs(_f64(y.out) - want) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(want))
        assert np.all(np.abs(_f64(y.residual) - s) <= 2.0 ** -23 * np.abs(s))
        _, want = P.rms_norm(_f64(z), _f64(gain), residual=_f64(y.residual))
        assert np.all(np.abs(_f64(n.out) - want) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(want))

    first = step()
    torch.cuda.synchronize()
    check(*first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        x.copy_(rnd(R, tokens, hidden))
        res.copy_(rnd(R, tokens, hidden))
        graph.replay()
        torch.cuda.synchronize()
        check(*got)
        eager = step()
        torch.cuda.synchronize()
        assert torch.equal(eager[-1].out, got[-1].out) and torch.equal(eager[-2], got[-2])


def test_two_streams_at_once_and_two_graphs():
    """One handle on two streams (the layer uses none of its buffers), late inputs, and two
    graphs replayed at the same time."""
    layer, x, ids, tw, want = _run(("int4", 128, "bf16"), 1, 7, 6, 2, 1024, 512)
    d_ids, d_tw = to_dev(ids), to_dev(tw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    late = [torch.zeros_like(x[0]) for _ in streams]
    for s, t in zip(streams, late):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
            t.copy_(x[0])
    outs = [layer((t, {}), d_ids, d_tw, stream=s) for s, t in zip(streams, late)]
    for s in streams:
        s.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    inputs, graphs = [x[0].clone() for _ in range(2)], []
    for t in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer((t, {}), d_ids, d_tw)
        graphs.append((g, out))
    for _ in range(3):
        for t in inputs:
            t.copy_(torch.randn(t.shape, device="cuda"))
        for s, (g, _) in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for t, (_, out) in zip(inputs, graphs):
            assert torch.equal(out, layer((t, {}), d_ids, d_tw))


def test_rows_behind_the_last_and_no_tokens():
    layer, x, ids, tw, got = _run("bf16", 1, 5, 4, 2, 256, 128)
    room = torch.full((1, 8, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    out = layer(x, to_dev(ids), to_dev(tw), out=room[:, :5])
    torch.cuda.synchronize()
    assert torch.equal(out, got) and torch.all(room[:, 5:] == 7.0)
    none = layer((x[0][:, :0], {}), to_dev(ids)[:, :0], to_dev(tw)[:, :0])
    assert none.shape == (1, 0, 256)
    fewer = layer((x[0][:, :3], {}), to_dev(ids)[:, :3].contiguous(),
                  to_dev(tw)[:, :3].contiguous())
    assert torch.equal(fewer, got[:, :3])


def test_refusals():
    layer, x, ids, tw, _ = _run("bf16", 1, 4, 2, 2, 256, 128)
    ctx, (w1, w2) = layer.ctx, layer.args
    ids, tw, x = to_dev(ids), to_dev(tw), x[0]
    codes = torch.zeros(2, 256, 128, dtype=torch.uint8, device="cuda")
    p1 = ctx.pack_weights_w4(codes, torch.ones(2, 256, 4, device="cuda").bfloat16())
    p2 = ctx.pack_weights_w4(codes[..., :64].contiguous(),
                             torch.ones(2, 256, 2, device="cuda").bfloat16())
    for call in (lambda: ctx.moe_layer(x.half(), w1, w2, ids, tw),
                 lambda: ctx.moe_layer(x, w1.half(), w2, ids, tw),
                 lambda: ctx.moe_layer(x, w1[:1], w2, ids, tw),
                 lambda: ctx.moe_layer(x, w1, w2.transpose(1, 2), ids, tw),
                 lambda: ctx.moe_layer(x, w1, w2, ids.long(), tw),
                 lambda: ctx.moe_layer(x, w1, w2, ids[:, :3], tw),
                 lambda: ctx.moe_layer(x, w1, w2, ids, tw.bfloat16()),
                 lambda: ctx.moe_layer(x, w1, w2, ids, tw, x_scale=tw),
                 lambda: ctx.moe_layer(x, w1, w2, ids, tw, out=x.float()),
                 lambda: ctx.moe_layer(x, p1, w2, ids, tw),
                 lambda: ctx.moe_layer(x, p2, p1, ids, tw),
                 lambda: ctx.moe_layer(x.cpu(), w1, w2, ids, tw)):
        with pytest.raises(ValueError):
            call()
    ctx.moe_layer(x, p1, p2, ids, tw)                      # formats may differ
    for call in (lambda: ctx.moe_layer(x, w1, w2, ids, tw, out=x),
                 lambda: ctx.moe_layer(x, w1, w2, ids, tw,
                                       out=w2.view(-1)[-4 * 256:].view(1, 4, 256))):
        with pytest.raises(EpError) as e:
            call()
        assert e.value.code == B.EP_ERR_INVALID_ARG
    need = B.ep_moe_layer_workspace(ctx.handle, 4)
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty_like(x)
    ok = [ctx.handle, None, None, x, None, w1, None, w2, None, ids, tw, 4, out, ws, need]
    B.ep_moe_layer(*ok)
    for at, value in ((3, None), (5, None), (7, None), (9, None), (10, None), (12, None),
                      (13, None), (14, need - 1), (11, -1), (11, 5), (3, x.data_ptr() + 2),
                      (1, p1.format), (2, p2.format), (13, x.data_ptr())):
        args = list(ok)
        args[at] = value
        with pytest.raises(EpError) as e:
            B.ep_moe_layer(*args)
        assert e.value.code == B.EP_ERR_INVALID_ARG
    for field, value in (("codes", 2), ("group", 16), ("scales", 2)):
        f = B.EpW4Format.from_buffer_copy(p1.format)
        setattr(f, field, value)
        with pytest.raises(EpError) as e:
            B.ep_moe_layer(ctx.handle, f, p2.format, x, None, p1.codes, p1.scales, p2.codes,
                           p2.scales, ids, tw, 4, out, ws, need)
        assert e.value.code == B.EP_ERR_INVALID_ARG
    torch.cuda.synchronize()


@pytest.mark.parametrize("over", [dict(R=8, T=9), dict(R=1, T=65), dict(R=1, T=17, top_k=64)])
def test_too_many_tokens_or_picks_are_refused(over):
    layer = Layer("bf16", 2, 128, 128, **over)
    R, T, k = over["R"], over["T"], over.get("top_k", 2)
    x = torch.zeros(R, T, 128, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(R, T, k, dtype=torch.int32, device="cuda")
    with pytest.raises(EpError) as e:
        layer.ctx.moe_layer(x, *layer.args, ids, ids.float())
    assert e.value.code == B.EP_ERR_UNSUPPORTED


def test_handles_that_cannot():
    fp8 = Layer("fp8", 2, 256, 128, 1, 4)
    w4 = Layer(("int4", 32, "bf16"), 2, 256, 128, 1, 4)
    x = torch.zeros(1, 4, 256, dtype=torch.uint8, device="cuda")
    ids = torch.zeros(1, 4, 2, dtype=torch.int32, device="cuda")
    s = torch.ones(1, 4, 2, device="cuda")
    with pytest.raises(EpError) as e:                      # 4-bit weights on an fp8 handle
        fp8.ctx.moe_layer(x, *w4.args, ids, s, x_scale=s, **fp8.scales)
    assert e.value.code == B.EP_ERR_UNSUPPORTED
    with pytest.raises(ValueError):                        # no scales
        fp8.ctx.moe_layer(x, *fp8.args, ids, s)
    odd = make_ctx(TINY.replace(k=64, n=128))              # I not a multiple of 128
    xb = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(2, 8, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(2, 128, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(EpError) as e:
        odd.moe_layer(xb, w, w, ids, ids.float())
    assert e.value.code == B.EP_ERR_UNSUPPORTED


@pytest.mark.parametrize("fmt", ["bf16", "bf16_sliced", "fp8", ("int4", 128, "bf16"),
                                 ("e2m1", 32, "f16")], ids=_id)
@pytest.mark.parametrize("counts", [[1, 4, 5, 8], [9, 16, 0, 2], [17, 32, 33, 64],
                                    [1, 0, 3, 40, 7, 12, 64, 31], [64], [8, 4, 0, 0, 0, 15]],
                         ids=lambda c: "-".join(map(str, c)))
def test_experts_of_few_and_of_many_tokens_together(fmt, counts):
    """Every number of rows that the products tell apart, alone and beside the others."""
    k = len(counts)

    def edit(ids, tw):
        # pick j of the first counts[j] tokens is expert j, in another order for each
        ids[...] = -1
        for j, n in enumerate(counts):
            ids[0, np.random.default_rng(j).permutation(64)[:n], j] = k - 1 - j
    _run(fmt, 1, 64, k, k, 256, 384, edit=edit)


@pytest.mark.parametrize("El", [65, 130, 256])
def test_few_and_many_tokens_among_many_experts(El):
    def edit(ids, tw):
        ids[0, :, 0] = El - 1                      # all tokens
        ids[0, ::3, 1] = 63                        # 22
        ids[0, 5::7, 1] = 64                       # 9
    _run(("e2m1", 64, "bf16"), 1, 64, El, 6, 128, 128, edit=edit)
