"""Gradient of the combine (ep_combine_backward) against its float64 definition."""
import numpy as np
import pytest
import torch

import oracle as O
from ep_synth import TINY, make_inputs, make_routing
from grouped_gemm_scatter_amd import EpError
from grouped_gemm_scatter_amd import binding as B
from gpu_helpers import make_ctx, to_dev
from oracle import operators as P

pytestmark = pytest.mark.gpu

CASES = {
    "tiny": TINY,
    "one_token": TINY.replace(n_ranks=1, n_experts_global=4, n_experts_local=4,
                              tokens_per_rank=1, n=256),
    "several_local_picks": TINY.replace(n_ranks=3, n_experts_global=8, n_experts_local=6,
                                        tokens_per_rank=50, top_k=5, n=384, seed=2),
    "wide_rows": TINY.replace(n_ranks=2, n_experts_global=8, n_experts_local=4,
                              tokens_per_rank=37, top_k=4, n=7168, seed=3),
    "widest_rows": TINY.replace(n_ranks=2, n_experts_global=8, n_experts_local=2, my_rank=1,
                                tokens_per_rank=9, top_k=2, n=16384, seed=4),
    "empty_experts": TINY.replace(n_ranks=8, n_experts_global=64, n_experts_local=8,
                                  tokens_per_rank=60, top_k=6, n=256, routing="zipf",
                                  n_forced_empty=3, seed=5),
    "no_local_rows": TINY.replace(n_ranks=2, n_experts_global=8, n_experts_local=4,
                                  tokens_per_rank=16, routing="zipf", n_forced_empty=4, seed=6),
    "many_picks": TINY.replace(n_ranks=1, n_experts_global=128, n_experts_local=100,
                               tokens_per_rank=6, top_k=64, n=128, seed=7),
}


def _case(cfg, ids, pad=0):
    """(ctx, device arguments, oracle's results) with random receive buffers."""
    rng = np.random.default_rng(cfg.seed + 100)
    R, T, k, N = cfg.n_ranks, cfg.tokens_per_rank, cfg.top_k, cfg.n
    ctx = make_ctx(cfg, msg_bytes=2 * N + pad)
    _, tw = make_routing(cfg)
    go = O.f64_to_bf16(rng.standard_normal((R, T, N)))
    slots = O.f64_to_bf16(rng.standard_normal((R, T * k, N)))
    for r in range(R):
        v = ctx.recv[r].view(T * k, 2 * N + pad)
        v[:, : 2 * N] = to_dev(slots[r]).view(torch.uint8).view(T * k, 2 * N)
    d_ids = to_dev(ids.astype(np.int32))
    off, src = ctx.group(d_ids)
    m = int(off[-1])
    o_off, o_src = O.group_local_picks(ids, cfg.n_experts_local, cfg.my_rank)
    picks = O.row_picks(o_off, o_src, R)
    assert len(picks) == m
    want = P.combine_backward(go, tw, picks, slots[picks[:, 0], picks[:, 1] * k + picks[:, 2]],
                              (R, T, k))
    return ctx, (to_dev(go, torch.bfloat16), d_ids, to_dev(tw), off, src, m), want


def _check(got, want, N, m):
    gw, gr, bound = want
    # N products in some order: one rounding a product and an addition, each within
    # 2^-24 of a partial sum that sum |a b| bounds
    err = np.abs(got[0].cpu().double().numpy() - gw)
    assert np.all(err <= 2 * N * 2.0 ** -24 * bound)
    # one binary32 product, then half a step of bf16
    rows = got[1][:m].float().cpu().double().numpy()
    assert np.all(np.abs(rows - gr) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(gr) + 1e-38)


@pytest.mark.parametrize("name", sorted(CASES))
def test_combine_backward(name):
    cfg = CASES[name]
    print(f"[case] combine backward {name}", flush=True)
    ids, _ = make_routing(cfg)
    ctx, args, want = _case(cfg, ids)
    m = args[-1]
    rows = torch.full((m + 3, cfg.n), 7.0, dtype=torch.bfloat16, device="cuda")
    got = ctx.combine_backward(*args, grad_rows=rows,
                               grad_w=torch.full(ids.shape, float("nan"), device="cuda"))
    torch.cuda.synchronize()
    assert ctx.query_error() == 0
    _check(got, want, cfg.n, m)
    assert torch.all(rows[m:] == 7.0), "rows behind the last one changed"
    # the weights' gradient alone
    gw, none = ctx.combine_backward(*args[:3], None, None, m, rows=False)
    assert none is None and torch.equal(gw, got[0])
    # the same bits again
    again = ctx.combine_backward(*args)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1][:m])


def test_dropped_and_equal_picks_and_padded_slots():
    cfg = CASES["several_local_picks"]
    ids, _ = make_routing(cfg)
    rng = np.random.default_rng(9)
    ids = ids.copy()
    ids[rng.random(ids.shape) < 0.3] = -1
    ids[0, :, 3] = ids[0, :, 1]                      # the same expert twice
    ids[1, 4] = 2 ** 31 - 1                          # an id that no layer has
    ctx, args, want = _case(cfg, ids, pad=48)
    got = ctx.combine_backward(*args)
    assert ctx.query_error() == 0
    _check(got, want, cfg.n, args[-1])
    assert torch.all(got[0][args[1] < 0] == 0)


def test_fewer_tokens_than_the_buffers_hold_and_no_tokens():
    cfg = CASES["tiny"]
    ctx = make_ctx(cfg, max_tokens=cfg.tokens_per_rank + 5)
    ids, tw = make_routing(cfg)
    for r in ctx.recv:
        r.view(torch.bfloat16).fill_(1.0)
    d_ids = to_dev(ids.astype(np.int32))
    off, src = ctx.group(d_ids)
    m = int(off[-1])
    go = torch.ones(cfg.n_ranks, cfg.tokens_per_rank, cfg.n, dtype=torch.bfloat16, device="cuda")
    gw, gr = ctx.combine_backward(go, d_ids, to_dev(tw), off, src, m)
    local = torch.from_numpy((ids >= 0) & (ids < cfg.n_experts_local))
    assert torch.equal(gw.cpu(), local * float(cfg.n))
    assert torch.equal(gr[:, 0].float(), gr[:, -1].float())
    gw, gr = ctx.combine_backward(go[:, :0].contiguous(), d_ids[:, :0].contiguous(),
                                  to_dev(tw[:, :0]), off, src, 0)
    assert gw.numel() == 0 and gr.shape == (0, cfg.n)


def test_infinite_and_missing_numbers_stay_in_their_rows():
    cfg = CASES["several_local_picks"]
    ids, _ = make_routing(cfg)
    ctx, args, want = _case(cfg, ids)
    go = args[0].clone()
    go[0, 3, 5] = float("inf")
    go[1, 2, 0] = float("nan")
    clean = ctx.combine_backward(*args)
    got = ctx.combine_backward(go, *args[1:])
    same = torch.ones(ids.shape, dtype=torch.bool)
    same[0, 3] = same[1, 2] = False
    assert torch.equal(got[0].cpu()[same], clean[0].cpu()[same])
    local = torch.from_numpy((ids >= 0) & (ids < cfg.n_experts_local))
    assert not torch.isfinite(got[0].cpu()[~same & local]).any()
    assert torch.all(got[0].cpu()[~local] == 0)


def test_a_layout_of_other_picks_is_latched():
    """A local pick that has no row in the layout given: the error is latched and the
    weights' gradient is right all the same."""
    cfg = CASES["several_local_picks"]
    ids, _ = make_routing(cfg)
    ctx, args, want = _case(cfg, ids)
    src = args[4].clone()
    src[0, 0] = cfg.tokens_per_rank + 1
    got = ctx.combine_backward(*args[:4], src, args[5])
    assert ctx.query_error() == B.EP_ERR_BAD_GROUP
    assert torch.equal(got[0], ctx.combine_backward(*args)[0])
    assert ctx.query_error() == 0
    # offsets beyond the rows there are
    off = args[3].clone()
    off[1:] += 1000
    ctx.combine_backward(*args[:3], off, *args[4:])
    assert ctx.query_error() == B.EP_ERR_BAD_GROUP


def test_after_a_step_and_in_a_graph():
    """The gradient of a real step's combine, captured with it and replayed."""
    cfg = TINY.replace(n_ranks=4, n_experts_global=16, n_experts_local=4, tokens_per_rank=40,
                       top_k=4, k=128, n=256, seed=8)
    inp = make_inputs(cfg)
    ctx = make_ctx(cfg, device_epoch=True)
    d_ids, tw = to_dev(inp.topk_ids.astype(np.int32)), to_dev(inp.topk_w)
    off, src = ctx.group(d_ids)
    m = int(off[-1])
    x = torch.randn(m, cfg.k, device="cuda").to(torch.bfloat16)
    w = to_dev(inp.w, torch.bfloat16)
    out = torch.empty(cfg.n_ranks, cfg.tokens_per_rank, cfg.n, dtype=torch.bfloat16, device="cuda")
    go = torch.randn_like(out)
    gw = torch.empty(inp.topk_w.shape, device="cuda")
    gr = torch.empty(m, cfg.n, dtype=torch.bfloat16, device="cuda")

    def step():
        ctx.step(x, w, off, src, m, d_ids, tw, out)
        ctx.combine_backward(go, d_ids, tw, off, src, m, grad_rows=gr, grad_w=gw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(torch.randn(m, cfg.k, device="cuda"))
        go.copy_(torch.randn_like(out))
        graph.replay()
        torch.cuda.synchronize()
        a, b = gw.clone(), gr.clone()
        step()
        torch.cuda.synchronize()
        assert ctx.query_error() == 0
        assert torch.equal(a, gw) and torch.equal(b, gr)


def test_refusals():
    cfg = CASES["tiny"]
    ids, _ = make_routing(cfg)
    ctx, args, _ = _case(cfg, ids)
    go, d_ids, tw, off, src, m = args
    for bad in ((go.float(), d_ids, tw, off, src, m), (go[:, :7], d_ids, tw, off, src, m),
                (go, d_ids.long(), tw, off, src, m), (go, d_ids, tw.half(), off, src, m),
                (go, d_ids, tw, off[:-1], src, m), (go, d_ids, tw, off, src[: m - 1], m),
                (go.cpu(), d_ids, tw, off, src, m)):
        with pytest.raises(ValueError):
            ctx.combine_backward(*bad)
    with pytest.raises(ValueError):
        ctx.combine_backward(*args, grad_rows=torch.empty(m - 1, cfg.n, dtype=torch.bfloat16,
                                                          device="cuda"))
    with pytest.raises(ValueError):
        ctx.combine_backward(*args, rows=False, grad_rows=torch.empty_like(go))
    gw = torch.empty(ids.shape, device="cuda")
    gr = torch.empty(m * cfg.n + 8, dtype=torch.bfloat16, device="cuda")
    T = cfg.tokens_per_rank
    for bad in ((go, d_ids, tw, T, None, src, m, gr, gw), (go, d_ids, tw, T, off, None, m, gr, gw),
                (go, d_ids, tw, T + 1, off, src, m, gr, gw), (go, d_ids, tw, T, off, src, -1, gr, gw),
                (go, d_ids, tw, T, off, src, m, gr[1:], gw), (go, d_ids, tw, T, off, src, m, gr, None),
                (None, d_ids, tw, T, off, src, m, gr, gw), (go, None, tw, T, off, src, m, gr, gw)):
        with pytest.raises(EpError) as e:
            B.ep_combine_backward(ctx.handle, *bad)
        assert e.value.code == B.EP_ERR_INVALID_ARG


def test_rows_past_four_gib():
    """Tokens, slots and rows whose byte offsets pass 32 bits."""
    T, N = 262144 + 61, 8192
    cfg = TINY.replace(n_ranks=1, n_experts_global=2, n_experts_local=2, tokens_per_rank=T, top_k=1,
                       n=N, k=64)
    ctx = make_ctx(cfg)
    slots = ctx.recv[0].view(torch.bfloat16).view(T, N)
    go = torch.empty(1, T, N, dtype=torch.bfloat16, device="cuda")
    for t in (slots, go[0]):
        for piece in t.split(32768):
            piece.copy_(torch.randn(piece.shape, device="cuda"))
    ids = torch.randint(0, 2, (1, T, 1), dtype=torch.int32, device="cuda")
    tw = torch.rand(1, T, 1, device="cuda")
    off, src = ctx.group(ids)
    assert int(off[-1]) == T
    gw, gr = ctx.combine_backward(go, ids, tw, off, src, T)
    torch.cuda.synchronize()
    assert ctx.query_error() == 0
    row_of = torch.empty(T, dtype=torch.int64, device="cuda")
    row_of[src[:T, 0].long()] = torch.arange(T, device="cuda")
    for at in (slice(0, 300), slice(T // 2, T // 2 + 300), slice(T - 300, T)):
        a, s = go[0, at].cpu().double(), slots[at].cpu().double()
        err = (gw[0, at, 0].cpu().double() - (a * s).sum(1)).abs()
        assert torch.all(err <= 2 * N * 2.0 ** -24 * (a * s).abs().sum(1))
        want = (tw[0, at] * go[0, at].float()).bfloat16()
        assert torch.equal(gr[row_of[at]], want)


def test_strides_types_and_overlaps_are_refused():
    cfg = CASES["tiny"]
    ids, _ = make_routing(cfg)
    ctx, args, _ = _case(cfg, ids)
    go, d_ids, tw, off, src, m = args
    for bad in ((off.cpu(), src), (off.float(), src), (off, src.cpu()), (off, src.float()),
                (off, src.t())):
        with pytest.raises(ValueError):
            ctx.combine_backward(go, d_ids, tw, *bad, m)
    for rows in (torch.empty(m, cfg.n, dtype=torch.float16, device="cuda"),
                 torch.empty(m, cfg.n, dtype=torch.bfloat16),
                 torch.empty(cfg.n, m, dtype=torch.bfloat16, device="cuda").t()):
        with pytest.raises(ValueError):
            ctx.combine_backward(*args, grad_rows=rows)
    both = torch.zeros(go.numel() // cfg.n + m, cfg.n, dtype=torch.bfloat16, device="cuda")
    go = both[: go.numel() // cfg.n].view(go.shape)
    args = (go, *args[1:])
    for kw in (dict(grad_rows=both[both.shape[0] - m - 1:]), dict(grad_w=tw),
               dict(grad_w=d_ids.view(torch.float32)),
               dict(grad_w=go.view(-1)[: 2 * tw.numel()].view(torch.float32).view(tw.shape))):
        with pytest.raises(EpError) as e:
            ctx.combine_backward(*args, **kw)
        assert e.value.code == B.EP_ERR_INVALID_ARG


def test_outputs_over_anything_that_is_read_are_refused():
    """grad_rows and grad_w over each input and over the slots of a receive buffer, which
    workgroups read while others store; memory next to them is accepted."""
    cfg = TINY.replace(n_ranks=2, n_experts_global=16, n_experts_local=4, tokens_per_rank=50,
                       top_k=5, n=384, seed=8)
    ids, _ = make_routing(cfg)
    ctx, args, want = _case(cfg, ids)
    go, d_ids, tw, off, src, m = args
    N, slots = cfg.n, cfg.tokens_per_rank * cfg.top_k
    row = 2 * N
    # every tensor in one allocation, m rows of room behind its first byte
    for name in range(5):
        room = torch.zeros(max(args[name].numel() * 4, 4 * tw.numel()) + (m + 1) * row,
                           dtype=torch.uint8, device="cuda")
        t = args[name]
        moved = room[: t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        moved.copy_(t)
        call = args[:name] + (moved,) + args[name + 1:]
        rows = room[: m * row].view(torch.bfloat16).view(m, N)
        weights = room[: 4 * tw.numel()].view(torch.float32).view(tw.shape)
        for kw in (dict(grad_rows=rows), dict(grad_w=weights)):
            with pytest.raises(EpError) as e:
                ctx.combine_backward(*call, **kw)
            assert e.value.code == B.EP_ERR_INVALID_ARG
        if name >= 3:                 # not read without rows
            gw, _ = ctx.combine_backward(*call, rows=False, grad_w=weights)
            err = np.abs(gw.cpu().double().numpy() - want[0])
            assert np.all(err <= 2 * N * 2.0 ** -24 * want[2])
    for recv in ctx.recv:
        assert recv.numel() == slots * row and m <= slots
        for kw in (dict(grad_rows=recv[recv.numel() - m * row:].view(torch.bfloat16).view(m, N)),
                   dict(grad_w=recv[recv.numel() - 4 * tw.numel():].view(torch.float32).view(tw.shape))):
            with pytest.raises(EpError) as e:
                ctx.combine_backward(*args, **kw)
            assert e.value.code == B.EP_ERR_INVALID_ARG
    # slots of tokens that the call leaves out are not read
    T = cfg.tokens_per_rank - 1
    less = d_ids[:, :T].contiguous()
    off, src = ctx.group(less)
    free = ctx.recv[1][T * cfg.top_k * row:].view(torch.float32)
    n = cfg.n_ranks * T * cfg.top_k
    assert free.numel() >= n
    gw, gr = ctx.combine_backward(go[:, :T].contiguous(), less, tw[:, :T].contiguous(), off, src,
                                  int(off[-1]), grad_w=free[:n].view(cfg.n_ranks, T, cfg.top_k))
    err = np.abs(gw.cpu().double().numpy() - want[0][:, :T])
    assert np.all(err <= 2 * N * 2.0 ** -24 * want[2][:, :T])
    assert ctx.query_error() == 0
