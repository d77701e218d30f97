"""Grouped products with 4-bit weights: the layout, the up-projection with SwiGLU and
the down-projection with the receive-buffer sink, against float64 products of the
decoded weights; then the whole path from router logits to gradients."""
import numpy as np
import pytest
import torch

import oracle as O
from ep_synth import TINY
from grouped_gemm_scatter_amd import EpError
from grouped_gemm_scatter_amd import binding as B
from gpu_helpers import SENTINEL, bits, make_ctx, to_dev
from oracle import operators as P

pytestmark = pytest.mark.gpu

SCALES = {"bf16": torch.bfloat16, "f16": torch.float16}
FORMATS = [("int4", 32, "bf16"), ("int4", 64, "f16"), ("int4", 128, "f16"), ("int4", 128, "bf16"),
           ("e2m1", 32, "bf16"), ("e2m1", 64, "bf16"), ("e2m1", 128, "f16")]


def _weights(rng, E, n, k, group, scale_type):
    codes = rng.integers(0, 256, (E, n, k // 2), dtype=np.uint8)
    s = torch.from_numpy((0.5 + rng.random((E, n, k // group))) / (5 * np.sqrt(k)))
    return codes, s.to(SCALES[scale_type])


def _layout(sizes, R, rng):
    """offsets [E*R + 1] of groups of these many rows, split over the ranks at random,
    and distinct (t, k) for the rows of a rank."""
    E = len(sizes)
    counts = np.stack([rng.multinomial(s, np.ones(R) / R) for s in sizes])     # [E][R]
    off = np.concatenate([[0], np.cumsum(counts.reshape(-1))]).astype(np.int32)
    src = np.zeros((int(off[-1]), 2), np.int32)
    nxt = np.zeros(R, np.int64)
    for e in range(E):
        for r in range(R):
            lo, hi = off[e * R + r], off[e * R + r + 1]
            at = nxt[r] + np.arange(hi - lo)
            src[lo:hi, 0], src[lo:hi, 1] = at // 2, at % 2
            nxt[r] += hi - lo
    return off, src, int(max(1, (nxt.max() + 1) // 2))


def _ctx(sizes, R, T, k, n, **kw):
    cfg = TINY.replace(n_ranks=R, n_experts_global=len(sizes) * R, n_experts_local=len(sizes),
                       tokens_per_rank=T, top_k=2, k=k, n=n)
    return make_ctx(cfg, **kw), cfg


def _sum_bound(a, k, group):
    """k exact products, each addition of the matrix unit within one step (2^-23) of a
    partial sum that a = sum |x w| bounds; then a product and an addition for every group."""
    return (k + 2 * k // group) * 2.0 ** -23 * a


SIZES = {
    "one_row": [1],
    "empty_and_one": [0, 1, 0, 0, 2, 0],
    "edges": [15, 16, 17, 0, 31, 32, 33, 47, 48, 49, 63, 64, 65],
    "no_rows": [0, 0, 0],
    "large_group": [5, 300, 0, 129],
    "many_experts": [(7 * i) % 5 for i in range(256)],
    # enough tiles for the 256-column tile, one to two row tiles of 0..70 rows an expert
    "decode_tile": [(11 * i) % 71 for i in range(256)],
}


@pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: "-".join(map(str, f)))
@pytest.mark.parametrize("k,n", [(128, 128), (640, 256), (2048, 384)])
def test_down_projection(fmt, k, n):
    _down("edges", fmt, k, n, R=3)


@pytest.mark.parametrize("name", sorted(SIZES))
@pytest.mark.parametrize("mode", ["flag", "per_expert", "system", "padded"])
def test_down_projection_groups_and_modes(name, mode):
    _down(name, ("int4", 64, "bf16"), 256, 256, R=8 if name == "edges" else 2, mode=mode)


@pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: "-".join(map(str, f)))
def test_down_projection_of_the_decode_tile(fmt):
    # 640 columns: the last tile of every expert is half empty
    _down("decode_tile", fmt, 384, 640, R=2)


def _down(name, fmt, k, n, R, mode="flag"):
    codes_are, group, st = fmt
    sizes = SIZES[name]
    print(f"[case] w4 down {name} {fmt} k={k} n={n} R={R} {mode}", flush=True)
    rng = np.random.default_rng(sum(map(ord, name)) + k)
    off, src, T = _layout(sizes, R, rng)
    M = int(off[-1])
    kw = {"per_expert": dict(per_expert_release=True), "system": dict(system_scope=True),
          "padded": dict(msg_bytes=2 * n + 32)}.get(mode, {})
    ctx, cfg = _ctx(sizes, R, T, k, n, **kw)
    codes, scales = _weights(rng, len(sizes), n, k, group, st)
    x = O.f64_to_bf16(rng.standard_normal((M, k)))
    w = ctx.pack_weights_w4(to_dev(codes), scales.cuda(), codes=codes_are)
    args = (to_dev(x, torch.bfloat16) if M else None, w, to_dev(off), to_dev(src) if M else None, M)
    y, a = P.grouped_product(O.bf16_to_f64(x), P.weights_w4(codes, scales.double().numpy(), codes_are),
                             off[::R])
    tol = _sum_bound(a, k, group) + 2.0 ** -8 * np.abs(y) + 1e-38
    # the sink off: a local product
    c = torch.full((M + 2, n), 7.0, dtype=torch.bfloat16, device="cuda")
    ctx.gemm_scatter_w4(*args, p3_control=-1, c_local=c)
    torch.cuda.synchronize()
    assert ctx.query_error() == 0 and torch.all(c[M:] == 7.0)
    assert torch.all(ctx.words == 0)
    got = O.bf16_to_f64(bits(c[:M]))
    assert np.all(np.abs(got - y) <= tol)
    # two steps through the sink
    for _ in range(2):
        ctx.next_epoch()
        ctx.gemm_scatter_w4(*args)
    torch.cuda.synchronize()
    assert ctx.query_error() == 0
    rank = (np.searchsorted(off, np.arange(M), side="right") - 1) % R
    for r in range(R):
        buf = ctx.recv[r].view(T * 2, ctx.msg_bytes).cpu()
        mine = np.nonzero(rank == r)[0]
        slot = src[mine, 0] * 2 + src[mine, 1]
        sent = torch.zeros(T * 2, dtype=torch.bool)
        sent[slot] = True
        assert torch.all(buf[~sent] == SENTINEL) and torch.all(buf[:, 2 * n:] == SENTINEL)
        assert torch.equal(buf[slot, : 2 * n].contiguous().view(torch.bfloat16), c.cpu()[mine])
    words = ctx.words.cpu().numpy().view(np.uint64)
    counts = np.diff(off).astype(np.uint64)
    if mode == "per_expert":
        assert np.array_equal(words[: len(counts)], (np.uint64(2) << np.uint64(32)) | counts)
    else:
        assert np.array_equal(words[: len(counts)], counts)
        assert np.all(words[len(counts):] == 2)
    assert torch.all(ctx.rank_counter == 0) and torch.all(ctx.tile_counter == 0)


@pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: "-".join(map(str, f)))
@pytest.mark.parametrize("name,inter,hidden", [
    ("edges", 128, 384), ("empty_and_one", 384, 7168), ("one_row", 2048, 256),
    ("large_group", 256, 128), ("no_rows", 128, 128), ("decode_tile", 256, 256)])
def test_up_projection(fmt, name, inter, hidden):
    codes_are, group, st = fmt
    sizes, R = SIZES[name], 2
    print(f"[case] w4 up {name} {fmt} inter={inter} hidden={hidden}", flush=True)
    rng = np.random.default_rng(inter + hidden)
    off, src, T = _layout(sizes, R, rng)
    M = int(off[-1])
    ctx, cfg = _ctx(sizes, R, T, inter, hidden)
    codes, scales = _weights(rng, len(sizes), 2 * inter, hidden, group, st)
    x = O.f64_to_bf16(rng.standard_normal((M, hidden)))
    w1 = ctx.pack_weights_w4(to_dev(codes), scales.cuda(), codes=codes_are)
    h = torch.full((M + 1, inter), 7.0, dtype=torch.bfloat16, device="cuda")
    ctx.up_swiglu_w4(to_dev(x, torch.bfloat16) if M else None, w1, to_dev(off), M, h)
    torch.cuda.synchronize()
    assert ctx.query_error() == 0 and torch.all(h[M:] == 7.0)
    y, a = P.grouped_product(O.bf16_to_f64(x), P.weights_w4(codes, scales.double().numpy(), codes_are),
                             off[::R])
    g, u = y[:, :inter], y[:, inter:]
    silu = g / (1 + np.exp(-g))
    bound = _sum_bound(a, hidden, group)
    # |silu'| <= 1.1; the activation's own roundings are within 2^-20 of its value
    tol = (1.1 * bound[:, :inter] * (np.abs(u) + bound[:, inter:]) + np.abs(silu) * bound[:, inter:] +
           (2.0 ** -8 + 2.0 ** -20) * np.abs(silu * u) + 1e-38)
    assert np.all(np.abs(O.bf16_to_f64(bits(h[:M])) - silu * u) <= tol)


@pytest.mark.parametrize("codes_are", ["int4", "e2m1"])
def test_every_code_at_every_place(codes_are):
    """Unit rows pick single weights: every result is one code times its scale, exactly,
    and the layout puts each at its place."""
    k, n, group = 256, 128, 32
    rng = np.random.default_rng(1)
    ctx, _ = _ctx([k], 1, k, k, n)
    codes, _ = _weights(rng, 1, n, k, group, "bf16")
    scales = torch.from_numpy(2.0 ** rng.integers(-8, 8, (1, n, k // group))).to(torch.bfloat16)
    w = ctx.pack_weights_w4(to_dev(codes), scales.cuda(), codes=codes_are)
    assert torch.equal(torch.sort(w.codes.flatten()).values,
                       torch.sort(to_dev(codes).flatten()).values) or codes_are == "int4"
    x = torch.eye(k, dtype=torch.bfloat16, device="cuda")
    c = torch.empty(k, n, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, k], dtype=torch.int32, device="cuda")
    src = torch.zeros(k, 2, dtype=torch.int32, device="cuda")
    ctx.gemm_scatter_w4(x, w, off, src, k, p3_control=-1, c_local=c)
    want = P.weights_w4(codes, scales.double().numpy(), codes_are)[0].T
    assert np.array_equal(c.double().cpu().numpy(), want)


@pytest.mark.parametrize("codes_are,zero", [("int4", 0x88), ("e2m1", 0x00), ("e2m1", 0x88)])
def test_weights_of_zero_give_zeros(codes_are, zero):
    k, n = 384, 128
    ctx, _ = _ctx([5, 40], 1, 45, k, n)
    codes = torch.full((2, n, k // 2), zero, dtype=torch.uint8, device="cuda")
    scales = torch.rand(2, n, k // 64, device="cuda").bfloat16()
    w = ctx.pack_weights_w4(codes, scales, codes=codes_are)
    off = torch.tensor([0, 5, 45], dtype=torch.int32, device="cuda")
    src = torch.zeros(45, 2, dtype=torch.int32, device="cuda")
    x = (100 * torch.randn(45, k, device="cuda")).to(torch.bfloat16)
    c = torch.full((45, n), 7.0, dtype=torch.bfloat16, device="cuda")
    ctx.gemm_scatter_w4(x, w, off, src, 45, p3_control=-1, c_local=c)
    assert torch.all(c == 0)


def test_numbers_without_an_end_stay_in_their_row():
    k, n = 256, 128
    rng = np.random.default_rng(2)
    ctx, _ = _ctx([20], 1, 20, k, n)
    codes, scales = _weights(rng, 1, n, k, 64, "bf16")
    w = ctx.pack_weights_w4(to_dev(codes), scales.cuda())
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    src = torch.zeros(20, 2, dtype=torch.int32, device="cuda")
    x = torch.randn(20, k, device="cuda").to(torch.bfloat16)
    c = torch.empty(20, n, dtype=torch.bfloat16, device="cuda")
    ctx.gemm_scatter_w4(x, w, off, src, 20, p3_control=-1, c_local=c)
    bad = x.clone()
    bad[3, 17] = float("inf")
    bad[19, 200] = float("nan")
    d = torch.empty_like(c)
    ctx.gemm_scatter_w4(bad, w, off, src, 20, p3_control=-1, c_local=d)
    keep = torch.ones(20, dtype=torch.bool)
    keep[3] = keep[19] = False
    assert torch.equal(c[keep], d[keep]) and not torch.isfinite(d[~keep]).any()


def test_slots_out_of_bounds_and_bad_offsets_are_latched():
    k, n, R = 128, 128, 2
    rng = np.random.default_rng(3)
    off, src, T = _layout([20, 0, 9], R, rng)
    ctx, _ = _ctx([20, 0, 9], R, T, k, n)
    codes, scales = _weights(rng, 3, n, k, 32, "bf16")
    w = ctx.pack_weights_w4(to_dev(codes), scales.cuda())
    x = torch.randn(29, k, device="cuda").to(torch.bfloat16)
    bad = src.copy()
    bad[4, 0], bad[5, 1] = T, 2
    ctx.next_epoch()
    ctx.gemm_scatter_w4(x, w, to_dev(off), to_dev(bad), 29)
    assert ctx.query_error() == B.EP_ERR_SLOT_OOB
    assert np.all(ctx.flags.cpu().numpy() == 1)
    before = ctx.words.clone()
    h = torch.full((29, k), 7.0, dtype=torch.bfloat16, device="cuda")
    w1 = ctx.pack_weights_w4(*(t.cuda() for t in (torch.zeros(3, 2 * k, n // 2, dtype=torch.uint8),
                                                  torch.ones(3, 2 * k, n // 32).bfloat16())))
    for wrong in (np.where(np.arange(7) == 3, 30, off), np.where(np.arange(7) == 6, 28, off),
                  np.where(np.arange(7) == 0, 1, off), np.where(np.arange(7) == 2, -1, off)):
        o = to_dev(wrong.astype(np.int32))
        ctx.next_epoch()
        ctx.gemm_scatter_w4(x, w, o, to_dev(src), 29)
        assert ctx.query_error() == B.EP_ERR_BAD_GROUP
        ctx.up_swiglu_w4(x, w1, o, 29, h)
        assert ctx.query_error() == B.EP_ERR_BAD_GROUP
    assert torch.equal(ctx.words, before) and torch.all(h == 7.0)


def test_on_another_stream_and_in_a_graph():
    """Two handles' steps in one graph, and a replay per new input."""
    k, n, R = 256, 128, 2
    rng = np.random.default_rng(4)
    off, src, T = _layout([20, 0, 70, 1], R, rng)
    M = int(off[-1])
    steps = []
    for _ in range(2):
        ctx, _ = _ctx([20, 0, 70, 1], R, T, k, n, device_epoch=True)
        codes, scales = _weights(rng, 4, n, k, 32, "bf16")
        c1, s1 = _weights(rng, 4, 2 * k, n, 128, "f16")
        steps.append((ctx, ctx.pack_weights_w4(to_dev(codes), scales.cuda(), codes="e2m1"),
                      ctx.pack_weights_w4(to_dev(c1), s1.cuda()),
                      torch.empty(M, k, dtype=torch.bfloat16, device="cuda")))
    x = torch.randn(M, n, device="cuda").to(torch.bfloat16)
    d_off, d_src = to_dev(off), to_dev(src)

    def run(stream=None):
        for ctx, w, w1, h in steps:
            ctx.next_epoch(stream)
            ctx.up_swiglu_w4(x, w1, d_off, M, h, stream=stream)
            ctx.gemm_scatter_w4(h, w, d_off, d_src, M, stream=stream)

    run()
    torch.cuda.synchronize()
    want = [[r.clone() for r in ctx.recv] for ctx, *_ in steps]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(s)
    s.synchronize()
    assert all(torch.equal(a, b) for (ctx, *_), ws in zip(steps, want)
               for a, b in zip(ctx.recv, ws))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(3):
        x.copy_(torch.randn(M, n, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [[r.clone() for r in ctx.recv] for ctx, *_ in steps]
        run()
        torch.cuda.synchronize()
        for (ctx, *_), gs in zip(steps, got):
            assert ctx.query_error() == 0
            assert all(torch.equal(a, b) for a, b in zip(ctx.recv, gs))


def test_refusals():
    k, n = 128, 128
    ctx, _ = _ctx([4, 4], 1, 8, k, n)
    codes = torch.zeros(2, n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.ones(2, n, k // 32, device="cuda").bfloat16()
    w = ctx.pack_weights_w4(codes, scales)
    x = torch.zeros(8, k, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    src = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    for bad in ((codes[:1], scales[:1]), (codes, scales.float()), (codes.char(), scales),
                (codes, scales[:, :64]), (codes.cpu(), scales), (codes[:, ::2], scales[:, ::2]),
                (codes, scales[..., :3])):
        with pytest.raises(ValueError):
            ctx.pack_weights_w4(*bad)
    with pytest.raises(ValueError):
        ctx.pack_weights_w4(codes, scales, codes="int8")
    for bad_scales in (scales.new_ones(2, n, 8), scales.new_ones(2, n, 128)):   # groups of 16, 1
        with pytest.raises(EpError) as e:
            ctx.pack_weights_w4(codes, bad_scales)
        assert e.value.code == B.EP_ERR_INVALID_ARG
    for rows, kk in ((24, 128), (16, 64)):
        with pytest.raises(EpError) as e:
            ctx.pack_weights_w4(codes.new_zeros(2, rows, kk // 2), scales.new_ones(2, rows, kk // 32))
        assert e.value.code == B.EP_ERR_UNSUPPORTED
    with pytest.raises(EpError):                       # in place
        B.ep_pack_weights_w4(ctx.handle, w.format, codes, scales, n, k, codes, w.scales)
    with pytest.raises(ValueError):                    # the up-projection's stack is 2 k rows
        ctx.up_swiglu_w4(x, w, off, 8, x)
    with pytest.raises(ValueError):
        ctx.gemm_scatter_w4(x, codes, off, src, 8, epoch=1)
    with pytest.raises(ValueError):
        ctx.gemm_scatter_w4(x[:7], w, off, src, 8, epoch=1)
    with pytest.raises(EpError):                       # no epoch yet
        ctx.gemm_scatter_w4(x, w, off, src, 8, epoch=0)
    with pytest.raises(EpError):                       # no output for the sink's off state
        B.ep_grouped_gemm_scatter_w4(ctx.handle, w.format, x, w.codes, w.scales, off, src, 8, -1)
    with pytest.raises(EpError):
        B.ep_grouped_gemm_scatter_w4(ctx.handle, w.format, x, w.codes, w.scales, off, None, 8)
    for field, value in (("codes", 2), ("group", 16), ("scales", 2)):
        f = B.EpW4Format.from_buffer_copy(w.format)
        setattr(f, field, value)
        with pytest.raises(EpError) as e:
            B.ep_grouped_gemm_scatter_w4(ctx.handle, f, x, w.codes, w.scales, off, src, 8)
        assert e.value.code == B.EP_ERR_INVALID_ARG
    cfg = TINY.replace(n_ranks=1, n_experts_global=2, n_experts_local=2, k=128, n=128)
    for other in (make_ctx(cfg.replace(dtype="fp8")), make_ctx(cfg, send_waves=4),
                  make_ctx(cfg, send_tile=True), make_ctx(cfg, trace_records=8),
                  make_ctx(cfg, epilogue_only=True), make_ctx(cfg.replace(k=192))):
        with pytest.raises(EpError) as e:
            B.ep_grouped_gemm_scatter_w4(other.handle, w.format, x, w.codes, w.scales, off, src, 8)
        assert e.value.code == B.EP_ERR_UNSUPPORTED


@pytest.mark.parametrize("tokens", [1, 40])
def test_from_router_logits_to_the_gradients(tokens):
    """route, group, dispatch, both 4-bit products, combine, then the combine's and the
    router's gradients, against float64 from the kernels' own stored intermediates."""
    R, E, k, hidden, inter = 4, 32, 4, 256, 128
    cfg = TINY.replace(n_ranks=R, n_experts_global=E, n_experts_local=16, tokens_per_rank=tokens,
                       top_k=k, k=inter, n=hidden)
    ctx = make_ctx(cfg)
    rng = np.random.default_rng(tokens)
    route = dict(n_groups=4, topk_groups=2, score="sigmoid", group_score="top2", scale=2.5)
    logits = to_dev(rng.standard_normal((R, tokens, E)).astype(np.float32))
    bias = to_dev((0.1 * rng.standard_normal(E)).astype(np.float32))
    toks = to_dev(O.f64_to_bf16(rng.standard_normal((R, tokens, hidden))), torch.bfloat16)
    c1, s1 = _weights(rng, 16, 2 * inter, hidden, 32, "bf16")
    c2, s2 = _weights(rng, 16, hidden, inter, 128, "bf16")
    w1 = ctx.pack_weights_w4(to_dev(c1), s1.cuda())
    w2 = ctx.pack_weights_w4(to_dev(c2), s2.cuda(), codes="e2m1")

    ids, tw = ctx.route(logits, bias=bias, **route)
    off, src = ctx.group(ids)
    m = int(off[-1])
    x1 = torch.empty(m, hidden, dtype=torch.bfloat16, device="cuda")
    h = torch.empty(m, inter, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(R, tokens, hidden, dtype=torch.bfloat16, device="cuda")
    ctx.dispatch(toks, off, src, m, x1)
    ctx.up_swiglu_w4(x1, w1, off, m, h)
    ctx.next_epoch()
    ctx.gemm_scatter_w4(h, w2, off, src, m)
    ctx.combine(ids, tw, out)
    go = to_dev(O.f64_to_bf16(rng.standard_normal((R, tokens, hidden))), torch.bfloat16)
    gw, gr = ctx.combine_backward(go, ids, tw, off, src, m)
    gl = ctx.route_backward(logits, ids, gw, score="sigmoid", scale=2.5)
    torch.cuda.synchronize()
    assert ctx.query_error() == 0

    want_ids, want_tw = P.route(logits.cpu().double().numpy().reshape(-1, E), k,
                                bias=bias.cpu().numpy(), **route)
    assert np.array_equal(ids.cpu().numpy().reshape(-1, k), want_ids)
    np.testing.assert_allclose(tw.cpu().numpy().reshape(-1, k), want_tw, rtol=40 * 2.0 ** -24)
    o_off, o_src = O.group_local_picks(ids.cpu().numpy(), 16, 0)
    picks = O.row_picks(o_off, o_src, R)
    assert len(picks) == m
    y, a = P.grouped_product(O.bf16_to_f64(bits(x1)),
                             P.weights_w4(c1, s1.double().numpy(), "int4"), o_off[::R])
    g, u = y[:, :inter], y[:, inter:]
    b = _sum_bound(a, hidden, 32)
    act = g / (1 + np.exp(-g)) * u
    tol = 1.1 * b[:, :inter] * (np.abs(u) + b[:, inter:]) + np.abs(g) * b[:, inter:]
    assert np.all(np.abs(O.bf16_to_f64(bits(h)) - act) <= tol + (2.0 ** -8 + 2.0 ** -20) * np.abs(act))
    y, a = P.grouped_product(O.bf16_to_f64(bits(h)), P.weights_w4(c2, s2.double().numpy(), "e2m1"),
                             o_off[::R])
    slots = np.stack([bits(ctx.recv[r].view(torch.bfloat16).view(-1, hidden)) for r in range(R)])
    sent = slots[picks[:, 0], picks[:, 1] * k + picks[:, 2]]
    assert np.all(np.abs(O.bf16_to_f64(sent) - y) <=
                  _sum_bound(a, inter, 128) + 2.0 ** -8 * np.abs(y) + 1e-38)
    total = np.zeros((R, tokens, hidden))
    tw64 = tw.cpu().double().numpy()
    for row, (rk, t, kk) in zip(O.bf16_to_f64(sent), picks):
        total[rk, t] += tw64[rk, t, kk] * row
    np.testing.assert_allclose(O.bf16_to_f64(bits(out)), total, rtol=2.0 ** -8 + 1e-6, atol=1e-5)
    want_gw, want_gr, bound = P.combine_backward(bits(go), tw64, picks, sent, ids.shape)
    assert np.all(np.abs(gw.cpu().double().numpy() - want_gw) <= 2 * hidden * 2.0 ** -24 * bound)
    np.testing.assert_allclose(O.bf16_to_f64(bits(gr)), want_gr, rtol=2.0 ** -8 + 1e-6)
    gw64 = gw.cpu().double().numpy().reshape(-1, k)
    want_gl = P.route_backward(logits.cpu().double().numpy().reshape(-1, E), want_ids, gw64,
                               score="sigmoid", scale=2.5)
    tol = 60 * 2.0 ** -24 * 2 * 2.5 * np.abs(gw64).max(1, keepdims=True)
    assert np.all(np.abs(gl.cpu().double().numpy().reshape(-1, E) - want_gl) <= tol)


def test_inputs_past_four_gib():
    """Rows whose byte offsets in x pass 32 bits."""
    inter, hidden, M = 128, 8192, 262144 + 81
    ctx, _ = _ctx([1, 1], 1, 1, inter, hidden)
    rng = np.random.default_rng(6)
    codes, scales = _weights(rng, 2, 2 * inter, hidden, 128, "bf16")
    w1 = ctx.pack_weights_w4(to_dev(codes), scales.cuda())
    x = torch.empty(M, hidden, dtype=torch.bfloat16, device="cuda")
    for piece in x.split(32768):
        piece.copy_(torch.randn(piece.shape, device="cuda"))
    h = torch.empty(M, inter, dtype=torch.bfloat16, device="cuda")
    ctx.up_swiglu_w4(x, w1, to_dev(np.array([0, 37, M], np.int32)), M, h)
    # the same rows by themselves
    last = x[M - 100:].clone()
    tail = torch.empty(100, inter, dtype=torch.bfloat16, device="cuda")
    ctx.up_swiglu_w4(last, w1, to_dev(np.array([0, 0, 100], np.int32)), 100, tail)
    torch.cuda.synchronize()
    assert ctx.query_error() == 0
    y, a = P.grouped_product(O.bf16_to_f64(bits(last)), P.weights_w4(
        codes, scales.double().numpy(), "int4"), np.array([0, 0, 100]))
    g, u = y[:, :inter], y[:, inter:]
    silu, bound = g / (1 + np.exp(-g)), _sum_bound(a, hidden, 128)
    tol = (1.1 * bound[:, :inter] * (np.abs(u) + bound[:, inter:]) + np.abs(silu) * bound[:, inter:] +
           (2.0 ** -8 + 2.0 ** -20) * np.abs(silu * u) + 1e-38)
    for got in (h[M - 100:], tail):
        assert np.all(np.abs(O.bf16_to_f64(bits(got)) - silu * u) <= tol)


def test_strides_types_and_overlaps_are_refused():
    k, n = 128, 128
    ctx, _ = _ctx([4, 4], 1, 8, k, n)
    w = ctx.pack_weights_w4(torch.zeros(2, n, k // 2, dtype=torch.uint8, device="cuda"),
                            torch.ones(2, n, k // 32, device="cuda").bfloat16())
    w1 = ctx.pack_weights_w4(torch.zeros(2, 2 * k, n // 2, dtype=torch.uint8, device="cuda"),
                             torch.ones(2, 2 * k, n // 32, device="cuda").bfloat16())
    x = torch.zeros(8, k, dtype=torch.bfloat16, device="cuda")
    h, c = torch.zeros_like(x), torch.zeros_like(x)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    src = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    for bad in ((x.half(), off, src, c), (x.cpu(), off, src, c), (x, off.cpu(), src, c),
                (x, off, src.cpu(), c), (x, off, src, c.cpu()), (x, off, src.float(), c),
                (torch.zeros(k, 8, dtype=torch.bfloat16, device="cuda").t(), off, src, c),
                (x, off, src, torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda").t())):
        with pytest.raises(ValueError):
            ctx.gemm_scatter_w4(bad[0], w, bad[1], bad[2], 8, p3_control=-1, c_local=bad[3])
    for bad in ((x.half(), off, h), (x, off.cpu(), h), (x, off, h.float()), (x, off, h.t())):
        with pytest.raises(ValueError):
            ctx.up_swiglu_w4(bad[0], w1, bad[1], 8, bad[2])
    with pytest.raises(EpError) as e:
        ctx.up_swiglu_w4(x, w1, off, 8, x)
    assert e.value.code == B.EP_ERR_INVALID_ARG
    with pytest.raises(EpError) as e:
        ctx.gemm_scatter_w4(x, w, off, src, 8, p3_control=-1, c_local=x)
    assert e.value.code == B.EP_ERR_INVALID_ARG
    ctx.up_swiglu_w4(x, w1, off, 8, h)
    ctx.gemm_scatter_w4(x, w, off, src, 8, p3_control=-1, c_local=c)
    torch.cuda.synchronize()
    assert ctx.query_error() == 0


@pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: "-".join(map(str, f)))
@pytest.mark.parametrize("name", ["edges", "large_group"])
def test_down_projection_of_the_narrow_tile(name, fmt):
    # too many 16-row tiles for the GPU, too few of 256 columns
    _down(name, fmt, 384, 2048 - 128 if name == "edges" else 4096, R=3)


@pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: "-".join(map(str, f)))
def test_up_projection_of_the_narrow_tile(fmt):
    test_up_projection(fmt, "edges", 1152, 256)


def test_outputs_over_what_is_read_are_refused():
    """The rows of both products over each input, in whole or by their last row."""
    k, n, m = 128, 256, 8
    ctx, _ = _ctx([4, 4], 1, m, k, n)
    rng = np.random.default_rng(9)
    packed = [ctx.pack_weights_w4(to_dev(c), s.cuda())
              for c, s in (_weights(rng, 2, 2 * k, n, 32, "bf16"),
                           _weights(rng, 2, n, k, 64, "f16"))]
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    src = torch.tensor([[i, 0] for i in range(m)], dtype=torch.int32, device="cuda")

    def up(x, codes, scales, offsets, out):
        B.ep_grouped_gemm_swiglu_w4(ctx.handle, packed[0].format, x, codes, scales, offsets, m, out)

    def down(x, codes, scales, offsets, out):
        B.ep_grouped_gemm_scatter_w4(ctx.handle, packed[1].format, x, codes, scales, offsets, src,
                                     m, -1, out)

    for call, w, width, out_width in ((up, packed[0], n, k), (down, packed[1], k, n)):
        x = torch.randn(m, width, device="cuda").bfloat16()
        inputs = (x, w.codes, w.scales, off)
        want = torch.empty(m, out_width, dtype=torch.bfloat16, device="cuda")
        call(*inputs, want)
        row = 2 * out_width
        for i, t in enumerate(inputs):
            size = (t.numel() * t.element_size() + 15) // 16 * 16
            # rows before the input, the input, rows behind it
            room = torch.zeros(2 * m * row + size, dtype=torch.uint8, device="cuda")
            moved = room[m * row:][: t.numel() * t.element_size()].view(t.dtype).view(t.shape)
            moved.copy_(t)
            call_inputs = inputs[:i] + (moved,) + inputs[i + 1:]
            for at in (16, m * row, m * row + (t.numel() * t.element_size() - 1) // 16 * 16):
                out = room[at: at + m * row].view(torch.bfloat16)
                with pytest.raises(EpError) as e:
                    call(*call_inputs, out)
                assert e.value.code == B.EP_ERR_INVALID_ARG
            for at in (0, m * row + size):
                out = room[at: at + m * row].view(torch.bfloat16).view(m, out_width)
                call(*call_inputs, out)
                assert torch.equal(out, want)
    assert ctx.query_error() == 0


@pytest.mark.parametrize("sizes", [
    {0: 3, 146: 1, 255: 2}, {e: 40 for e in range(3, 256, 23)},
    {e: 11 * e % 9 for e in range(256)}], ids=["few_rows", "few_experts", "every_expert"])
def test_a_whole_layer_of_256_experts(sizes):
    """Both products of a stack whose 2-byte weights would be 7.5 GB, in each tile; products
    of such weights are refused."""
    k, n, E, R = 2048, 7168, 256, 2
    rng = np.random.default_rng(len(sizes))
    off, src, T = _layout([sizes.get(e, 0) for e in range(E)], R, rng)
    M = int(off[-1])
    ctx, _ = _ctx([0] * E, R, T, k, n)
    gen = torch.Generator(device="cuda").manual_seed(M)
    stacks = []
    for rows, kk, group, st in ((2 * k, n, 128, "bf16"), (n, k, 32, "f16")):
        codes = torch.randint(0, 256, (E, rows, kk // 2), dtype=torch.uint8, device="cuda",
                              generator=gen)
        scales = ((0.5 + torch.rand(E, rows, kk // group, device="cuda", generator=gen)) /
                  (5 * kk ** 0.5)).to(SCALES[st])
        stacks.append((codes, scales, ctx.pack_weights_w4(codes, scales), group))
    x = torch.randn(M, n, device="cuda", generator=gen).bfloat16()
    h = torch.empty(M, k, dtype=torch.bfloat16, device="cuda")
    c = torch.empty(M, n, dtype=torch.bfloat16, device="cuda")
    d_off, d_src = to_dev(off), to_dev(src)
    ctx.up_swiglu_w4(x, stacks[0][2], d_off, M, h)
    ctx.gemm_scatter_w4(h, stacks[1][2], d_off, d_src, M, p3_control=-1, c_local=c)
    ctx.next_epoch()
    ctx.gemm_scatter_w4(h, stacks[1][2], d_off, d_src, M)
    torch.cuda.synchronize()
    assert ctx.query_error() == 0 and torch.all(ctx.flags == 1)
    rank = (np.searchsorted(off, np.arange(M), side="right") - 1) % R
    for m in range(M):
        slot = ctx.recv[rank[m]].view(-1, 2 * n)[int(src[m, 0]) * 2 + int(src[m, 1])]
        assert torch.equal(slot.view(torch.bfloat16), c[m])
    busy = [e for e in range(E) if sizes.get(e, 0)]
    for e in sorted({busy[0], busy[len(busy) // 2], busy[-2], busy[-1]}):
        at = slice(int(off[e * R]), int(off[(e + 1) * R]))
        for (codes, scales, _, group), inp, got in ((stacks[0], x, h), (stacks[1], h, c)):
            w = P.weights_w4(codes[e].cpu().numpy(), scales[e].double().cpu().numpy(), "int4")
            y, a = P.grouped_product(O.bf16_to_f64(bits(inp[at])), w[None], [0, at.stop - at.start])
            b = _sum_bound(a, w.shape[1], group)
            if got is h:
                (g, u), (bg, bu) = (y[:, :k], y[:, k:]), (b[:, :k], b[:, k:])
                silu = g / (1 + np.exp(-g))
                y = silu * u
                b = 1.1 * bg * (np.abs(u) + bu) + np.abs(silu) * bu + 2.0 ** -20 * np.abs(y)
            tol = b + 2.0 ** -8 * np.abs(y) + 1e-38
            assert np.all(np.abs(O.bf16_to_f64(bits(got[at])) - y) <= tol)
    w = stacks[0][0].data_ptr()
    for call in (lambda: B.ep_grouped_gemm_scatter(ctx.handle, h, w, None, None, d_off, d_src, M,
                                                   0, None, 2),
                 lambda: B.ep_grouped_gemm_swiglu(ctx.handle, x, w, d_off, M, h),
                 lambda: B.ep_pack_weights(ctx.handle, w, stacks[1][0].data_ptr())):
        with pytest.raises(EpError) as e:
            call()
        assert e.value.code == B.EP_ERR_UNSUPPORTED


def test_on_another_stream_everything_is_written_there():
    """A step on a stream whose earlier work it needs: the input arrives there, late, and what
    the step writes held something else before."""
    k, n, R = 256, 128, 2
    rng = np.random.default_rng(14)
    off, src, T = _layout([20, 0, 70, 1], R, rng)
    M = int(off[-1])
    ctx, _ = _ctx([20, 0, 70, 1], R, T, k, n)
    c, s = _weights(rng, 4, n, k, 32, "bf16")
    c1, s1 = _weights(rng, 4, 2 * k, n, 128, "f16")
    w = ctx.pack_weights_w4(to_dev(c), s.cuda(), codes="e2m1")
    w1 = ctx.pack_weights_w4(to_dev(c1), s1.cuda())
    old, new = (torch.randn(M, n, device="cuda").bfloat16() for _ in range(2))
    d_off, d_src = to_dev(off), to_dev(src)
    h = torch.empty(M, k, dtype=torch.bfloat16, device="cuda")

    def step(x, stream=None):
        ctx.next_epoch(stream)
        ctx.up_swiglu_w4(x, w1, d_off, M, h, stream=stream)
        ctx.gemm_scatter_w4(h, w, d_off, d_src, M, stream=stream)

    step(new)
    torch.cuda.synchronize()
    want, want_h, want_words = [r.clone() for r in ctx.recv], h.clone(), ctx.words.clone()
    for r in ctx.recv:
        r.fill_(SENTINEL)
    h.fill_(7.0)
    ctx.words.zero_()
    x = old.clone()
    late = torch.cuda.Stream()
    late.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(late):
        torch.cuda._sleep(20_000_000)
        x.copy_(new)
    step(x, late)
    late.synchronize()
    assert ctx.query_error() == 0
    assert torch.equal(h, want_h)
    assert all(torch.equal(a, b) for a, b in zip(ctx.recv, want))
    want_words[-R:] = 2                              # the second step's flags
    assert torch.equal(ctx.words, want_words)
    assert torch.all(ctx.rank_counter == 0) and torch.all(ctx.tile_counter == 0)
    # packed there as well, from codes that arrive late
    codes, scales = torch.zeros_like(to_dev(c1)), torch.zeros_like(s1).cuda()
    d_c1, d_s1 = to_dev(c1), s1.cuda()
    late.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(late):
        torch.cuda._sleep(20_000_000)
        codes.copy_(d_c1)
        scales.copy_(d_s1)
    there = ctx.pack_weights_w4(codes, scales, stream=late)
    late.synchronize()
    assert torch.equal(there.codes, w1.codes) and torch.equal(there.scales, w1.scales)
