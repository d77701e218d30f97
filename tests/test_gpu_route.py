"""Routing to experts (ep_route_topk) and its gradient against the float64
definitions: picks exactly, weights and gradients within the bounds of binary32."""
import numpy as np
import pytest
import torch

from grouped_gemm_scatter_amd import EpCombine, EpError
from grouped_gemm_scatter_amd import binding as B
from oracle import operators as P

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24                     # half a step of binary32, relative


def _ctx(R, T, top_k):
    return EpCombine(n_ranks=R, top_k=top_k, max_tokens_per_rank=T, n_experts_per_device=1,
                     hidden_k=64, hidden_n=128)


def _logits(seed, R, T, E, dtype, masked=False, spread=1.5):
    rng = np.random.default_rng(seed)
    l = torch.from_numpy(spread * rng.standard_normal((R, T, E)).astype(np.float32))
    if masked:
        l[torch.from_numpy(rng.random((R, T, E)) < 0.4)] = -float("inf")
        l[:, 0] = -float("inf")    # a token with no expert at all
    return l.to(DTYPES[dtype])


def _numpy(t):
    return t.cpu().double().numpy().reshape(-1, t.shape[-1])


def _weight_bound(l, E):
    """Relative error of a weight: numerator e^a with a = l - top rounded (|a| U) and expf
    within an ulp (2 U), the like in the terms of the sum, a sum of E terms over 64
    lanes (E/64 + 6 additions), the sigmoids' 1 + e^-|l| (3 U twice), a division and
    the scale."""
    x = P.clean_logits(l)
    spread = np.where(x > -np.inf, x.max(1, keepdims=True) - np.maximum(x, -1e4), 0.0)
    spread = np.maximum(spread, np.where(x > -np.inf, np.abs(np.maximum(x, -1e4)), 0.0))
    return (2 * np.minimum(spread.max(1, keepdims=True), 200.0) + 4 + E / 64 + 6 + 6 + 4) * U


CASES = {
    # R, T, E, top_k, options
    "one_token": (1, 1, 256, 8, dict(n_groups=8, topk_groups=4, score="sigmoid",
                                     group_score="top2", bias=True, scale=2.5)),
    "grouped_sigmoid": (4, 130, 256, 8, dict(n_groups=8, topk_groups=4, score="sigmoid",
                                             group_score="top2", bias=True, scale=2.5)),
    "softmax": (8, 65, 128, 8, dict()),
    "softmax_plain": (3, 77, 60, 6, dict(renormalize=False, scale=16.0)),
    "sigmoid_plain": (2, 33, 96, 4, dict(score="sigmoid", renormalize=False)),
    "softmax_bias": (2, 50, 72, 5, dict(bias=True)),
    "softmax_grouped_max": (2, 64, 160, 6, dict(n_groups=8, topk_groups=3, renormalize=False)),
    "softmax_grouped_top2": (2, 64, 160, 6, dict(n_groups=32, topk_groups=3, group_score="top2")),
    "groups_of_one": (1, 40, 16, 3, dict(n_groups=16, topk_groups=2, group_score="top2")),
    "more_groups_than_the_limit_keeps": (1, 40, 64, 3, dict(n_groups=64, topk_groups=64)),
    "one_expert": (2, 9, 1, 1, dict(score="sigmoid")),
    "all_experts": (1, 20, 7, 7, dict()),
    "many_picks": (1, 30, 200, 64, dict(score="sigmoid", bias=True)),
    "largest": (1, 25, 1024, 16, dict(n_groups=64, topk_groups=5, bias=True)),
    "odd": (5, 13, 333, 9, dict(n_groups=3, topk_groups=2, score="sigmoid")),
    # enough tokens for four of them a wave, with a count that is no multiple of four
    "many_grouped_sigmoid": (7, 601, 256, 8, dict(n_groups=8, topk_groups=4, score="sigmoid",
                                                  group_score="top2", bias=True, scale=2.5)),
    "many_odd_groups": (3, 1501, 130, 5, dict(n_groups=10, topk_groups=3, group_score="top2")),
    "many_groups_of_one_lane": (1, 4100, 64, 4, dict(n_groups=16, topk_groups=5, bias=True)),
    "many_plain": (8, 513, 33, 16, dict(renormalize=False, bias=True)),
    "many_softmax": (5, 900, 250, 11, dict()),
    "many_too_many_picks": (1, 4200, 96, 17, dict(score="sigmoid")),
    "many_too_many_experts": (1, 4200, 300, 4, dict(n_groups=4, topk_groups=2, bias=True)),
    "bias_alone_moves_the_picks": (1, 60, 40, 4, dict(bias=True, score="sigmoid", renormalize=False)),
}


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("name", sorted(CASES))
def test_route_and_gradient(name, dtype, masked):
    R, T, E, k, opt = CASES[name]
    print(f"[case] route {name} {dtype} masked={masked}", flush=True)
    opt = dict(opt)
    rng = np.random.default_rng(7)
    bias = None
    if opt.pop("bias", False):
        bias = (0.3 * rng.standard_normal(E)).astype(np.float32)
        if masked:
            bias[E // 2] = -np.inf
            bias[E // 3] = np.nan
    ctx = _ctx(R, T, k)
    l = _logits(11, R, T, E, dtype, masked)
    d_l = l.cuda()
    kw = dict(opt, bias=None if bias is None else torch.from_numpy(bias).cuda())
    ids, w = ctx.route(d_l, **kw)
    want_ids, want_w = P.route(_numpy(l), k, **dict(opt, bias=bias))
    got_ids, got_w = ids.cpu().numpy().reshape(-1, k), _numpy(w)
    assert np.array_equal(got_ids, want_ids), "picks differ"
    tol = _weight_bound(_numpy(l), E) * np.abs(want_w) + 1e-36
    assert np.all(np.abs(got_w - want_w) <= tol)
    assert np.all(got_w[want_ids < 0] == 0)

    g = torch.from_numpy(rng.standard_normal((R, T, k)).astype(np.float32))
    g[ids.cpu() < 0] = float("nan")          # the gradient of a dropped pick is not read
    bw = {n: opt[n] for n in ("score", "renormalize", "scale") if n in opt}
    d = ctx.route_backward(d_l, ids, g.cuda(), **bw)
    want = P.route_backward(_numpy(l), want_ids, np.nan_to_num(_numpy(g)), **bw)
    # |p (g - sum g p)|: the errors of p against |g| + sum |g p|, the sums' own, the
    # (1 - s) factor's, then the rounding to the logits' type
    gg = np.abs(np.nan_to_num(_numpy(g))).max(1, keepdims=True) * opt.get("scale", 1.0)
    p = np.abs(P.scores(_numpy(l), opt.get("score", "softmax")))
    if opt.get("renormalize", True):
        p = np.zeros_like(p)
        share = P.pick_shares(_numpy(l), want_ids, opt.get("score", "softmax"))
        r = np.broadcast_to(np.arange(len(p))[:, None], want_ids.shape)
        np.add.at(p, (r[want_ids >= 0], want_ids[want_ids >= 0]), share[want_ids >= 0])
    tol = (3 * _weight_bound(_numpy(l), E) * p * 2 * gg +
           torch.finfo(DTYPES[dtype]).eps / 2 * np.abs(want) * (1 + 2.0 ** -10) +
           (2.0 ** -25 if dtype == "f16" else 1e-36))     # half of fp16's smallest step
    assert np.all(np.abs(_numpy(d) - want) <= tol)
    assert d.dtype == l.dtype


def test_ties_go_to_the_lowest_index():
    ctx = _ctx(1, 3, 4)
    l = torch.zeros(1, 3, 64)
    l[0, 1, 10:20] = 1.0
    l[0, 2] = torch.arange(64).remainder(4)
    ids, w = ctx.route(l.cuda(), bias=torch.zeros(64, device="cuda"), score="sigmoid")
    assert ids.tolist() == [[[0, 1, 2, 3], [10, 11, 12, 13], [3, 7, 11, 15]]]
    ids, w = ctx.route(l.cuda(), n_groups=8, topk_groups=2, group_score="top2")
    assert ids.tolist() == [[[0, 1, 2, 3], [10, 11, 12, 13], [3, 7, 11, 15]]]
    assert torch.all(w == 0.25)


@pytest.mark.parametrize("T", [9, 4099])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choices_that_tie_or_nearly_tie(score, group_score, T):
    """Logits and biases of few values: most tokens hold choices and groups that are equal,
    or apart by less than binary32 can tell."""
    rng = np.random.default_rng(T)
    E, k = 64, 6
    steps = 2.0 ** -21 * np.arange(-3, 4)
    l = rng.choice([-1.0, 0.25, 0.5, 1.5], (1, T, E))
    l = (l + rng.choice(steps, l.shape) * (rng.random(l.shape) < 0.5)).astype(np.float32)
    bias = rng.choice([0.0, 0.125, 0.25], E).astype(np.float32)
    ctx = _ctx(1, T, k)
    kw = dict(n_groups=8, topk_groups=3, group_score=group_score, score=score)
    ids, w = ctx.route(torch.from_numpy(l).cuda(), bias=torch.from_numpy(bias).cuda(), **kw)
    want_ids, want_w = P.route(l.reshape(-1, E).astype(np.float64), k, bias=bias, **kw)
    # choices closer than binary64 itself can tell are left out: equal logits and biases
    # give equal choices on both sides, others differ by 2^-21 / 16 or more
    assert np.array_equal(ids.cpu().numpy().reshape(-1, k), want_ids)
    np.testing.assert_allclose(_numpy(w), want_w, rtol=60 * U)


def test_choices_a_binary32_step_apart_are_told_apart():
    """Choices whose difference binary32 cannot hold: the logits decide, in 64 bits."""
    ctx = _ctx(1, 1, 2)
    E = 64
    base = np.float32(0.3)
    l = np.full((1, E), -5.0, np.float32)
    l[0, 5] = base
    l[0, 9] = np.nextafter(base, np.float32(1))
    l[0, 40] = np.nextafter(l[0, 9], np.float32(1))
    bias = np.full(E, 100.0, np.float32)       # one step of the sum is 2^-17 in binary32
    for score in ("softmax", "sigmoid"):
        ids, _ = ctx.route(torch.from_numpy(l)[None].cuda(), bias=torch.from_numpy(bias).cuda(),
                           score=score)
        want, _ = P.route(l.astype(np.float64), 2, bias=bias, score=score)
        assert ids.tolist() == [want.tolist()] == [[[40, 9]]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_without_a_number(score):
    """NaN and -infinity are never picked, +infinity first; a bias of NaN or -infinity
    keeps its expert out."""
    ctx = _ctx(1, 4, 3)
    inf, nan = float("inf"), float("nan")
    l = torch.full((1, 4, 8), -2.0)
    l[0, 0, :3] = torch.tensor([nan, inf, inf])
    l[0, 1] = nan
    l[0, 2, 2:] = -inf
    l[0, 3] = -inf
    l[0, 3, 6] = 3e38
    for bias in (None, torch.tensor([0, 0, nan, 0, -inf, 0, 0, 0.5])):
        ids, w = ctx.route(l.cuda(), bias=None if bias is None else bias.cuda(), score=score)
        want_ids, want_w = P.route(_numpy(l), 3, bias=None if bias is None else bias.numpy(),
                                   score=score)
        assert np.array_equal(ids.cpu().numpy()[0], want_ids)
        np.testing.assert_allclose(_numpy(w), want_w, rtol=1e-6)
        d = ctx.route_backward(l.cuda(), ids, torch.ones_like(w), score=score)
        assert torch.isfinite(d).all()


def test_tiny_scores_keep_their_shares():
    """Sigmoids and exponentials that binary32 cannot hold, renormalised."""
    ctx = _ctx(1, 2, 3)
    l = torch.tensor([[[-300.0, -301.0, -302.0, -900.0], [-104.0, -1e30, -105.0, -110.0]]])
    for score in ("softmax", "sigmoid"):
        ids, w = ctx.route(l.cuda(), score=score)
        want_ids, want_w = P.route(_numpy(l), 3, score=score)
        assert np.array_equal(ids.cpu().numpy().reshape(-1, 3), want_ids)
        np.testing.assert_allclose(_numpy(w), want_w, rtol=300 * 2 * U + 20 * U)


def test_gradient_of_equal_and_bad_picks():
    ctx = _ctx(1, 1, 5)
    l = torch.tensor([[[0.1, 0.7, -0.3, 0.2, float("-inf"), 1.0]]])
    ids = torch.tensor([[[1, 1, 6, -5, 4]]], dtype=torch.int32)
    g = torch.tensor([[[1.0, 2.0, float("inf"), 8.0, float("nan")]]])
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            d = ctx.route_backward(l.cuda(), ids.cuda(), g.cuda(), score=score,
                                   renormalize=renormalize)
            want = P.route_backward(_numpy(l), ids.numpy()[0],
                                    np.array([[1.0, 2.0, 0.0, 0.0, 0.0]]), score=score,
                                    renormalize=renormalize)
            # terms of at most 3, twenty roundings
            np.testing.assert_allclose(_numpy(d), want, rtol=0, atol=3 * 20 * U)


def test_gradient_by_differences():
    """The gradient of sum(g w) against differences of the GPU's own weights, away from
    changes of picks; the step's error is O(h^2) = 1e-4, the weights' 1e-6 / h."""
    ctx = _ctx(1, 1, 3)
    l = torch.tensor([[[2.0, -1.0, 1.2, 0.4, -0.5, 1.7]]])
    g = torch.tensor([[[0.5, -1.0, 2.0]]])
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            kw = dict(score=score, renormalize=renormalize)
            ids, _ = ctx.route(l.cuda(), **kw)
            d = ctx.route_backward(l.cuda(), ids, g.cuda(), **kw).cpu()
            h = 0.01
            for i in range(6):
                up, down = l.clone(), l.clone()
                up[0, 0, i] += h
                down[0, 0, i] -= h
                a, wa = ctx.route(up.cuda(), **kw)
                b, wb = ctx.route(down.cuda(), **kw)
                assert torch.equal(a, ids) and torch.equal(b, ids)
                slope = ((wa - wb).cpu() * g).sum() / (2 * h)
                assert abs(slope - d[0, 0, i]) < 5e-4


def test_no_tokens():
    ctx = _ctx(2, 4, 2)
    l = torch.empty(2, 0, 16, device="cuda")
    ids, w = ctx.route(l)
    assert ids.shape == (2, 0, 2) and w.shape == (2, 0, 2)
    assert ctx.route_backward(l, ids, w).shape == (2, 0, 16)


def test_route_on_another_stream_and_in_a_graph():
    ctx = _ctx(2, 64, 4)
    l = _logits(3, 2, 64, 48, "f32").cuda()
    g = torch.randn(2, 64, 4, device="cuda")
    bias = torch.randn(48, device="cuda")
    want_ids, want_w = ctx.route(l, bias=bias, score="sigmoid")
    want_d = ctx.route_backward(l, want_ids, g, score="sigmoid")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids, w = ctx.route(l, bias=bias, score="sigmoid", stream=s)
    d = ctx.route_backward(l, ids, g, score="sigmoid", stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(ids, want_ids) and torch.equal(w, want_w) and torch.equal(d, want_d)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = ctx.route(l, bias=bias, score="sigmoid")
        d = ctx.route_backward(l, ids, g, score="sigmoid")
    for seed in (3, 4, 5, 6):
        l.copy_(_logits(seed, 2, 64, 48, "f32"))
        graph.replay()
        torch.cuda.synchronize()
        a, b = ctx.route(l, bias=bias, score="sigmoid")
        assert torch.equal(ids, a) and torch.equal(w, b)
        assert torch.equal(d, ctx.route_backward(l, a, g, score="sigmoid"))


def test_refusals():
    ctx = _ctx(2, 8, 4)
    l = torch.zeros(2, 8, 32, device="cuda")
    ids, w = ctx.route(l)
    for bad in (dict(n_groups=5), dict(n_groups=0), dict(n_groups=4, topk_groups=5),
                dict(topk_groups=0), dict(scale=float("inf")), dict(scale=float("nan"))):
        with pytest.raises(EpError) as e:
            ctx.route(l, **bad)
        assert e.value.code == B.EP_ERR_INVALID_ARG
    with pytest.raises(EpError) as e:                  # fewer experts than picks
        ctx.route(l[..., :3].contiguous())
    assert e.value.code == B.EP_ERR_INVALID_ARG
    with pytest.raises(EpError) as e:                  # more tokens than the handle's
        ctx.route(torch.zeros(2, 9, 32, device="cuda"))
    assert e.value.code == B.EP_ERR_INVALID_ARG
    with pytest.raises(EpError) as e:
        ctx.route(torch.zeros(2, 8, 1025, device="cuda"))
    assert e.value.code == B.EP_ERR_UNSUPPORTED
    with pytest.raises(EpError) as e:
        ctx.route(torch.zeros(2, 8, 130, device="cuda"), n_groups=65)
    assert e.value.code == B.EP_ERR_UNSUPPORTED
    for bad in (dict(score="tanh"), dict(group_score="mean"), dict(bias=torch.zeros(31).cuda()),
                dict(bias=torch.zeros(32)), dict(bias=torch.zeros(32).cuda().half()),
                dict(topk_ids=ids.long()), dict(topk_w=w[:, :7])):
        with pytest.raises(ValueError):
            ctx.route(l, **bad)
    for bad in (l.double(), l[:1], l.cpu(), torch.zeros(2, 8, 64, device="cuda")[..., ::2], l[0]):
        with pytest.raises(ValueError):
            ctx.route(bad)
    # a row that starts between 16-byte borders
    flat = torch.zeros(2 * 8 * 32 + 1, device="cuda")
    with pytest.raises(EpError) as e:
        ctx.route(flat[1:].view(2, 8, 32))
    assert e.value.code == B.EP_ERR_INVALID_ARG
    with pytest.raises(EpError):                       # a gradient over its own logits
        ctx.route_backward(l, ids, w, grad_logits=l)
    with pytest.raises(ValueError):
        ctx.route_backward(l, ids, w.half())
    with pytest.raises(ValueError):
        ctx.route_backward(l, ids[:, :4], w)
    # unknown flags at the C boundary
    p = B.make_route_params(n_experts=32, logits_dtype=torch.float32)
    for field, value in (("score", 2), ("group_score", -1), ("renormalize", 2),
                         ("logits_dtype", 3)):
        q = B.EpRouteParams.from_buffer_copy(p)
        setattr(q, field, value)
        with pytest.raises(EpError):
            B.ep_route_topk(ctx.handle, q, l, None, 8, ids, w)
    with pytest.raises(EpError):
        B.ep_route_topk(ctx.handle, p, l, None, 8, None, w)
    with pytest.raises(EpError):
        B.ep_route_topk(ctx.handle, p, l, None, -1, ids, w)


def test_logits_past_four_gib():
    """Tokens whose byte offsets in the logits pass 32 bits, forward and backward."""
    T, E = 2_097_152 + 37, 1024
    opts = dict(score="sigmoid", renormalize=True)
    ctx = _ctx(1, T, 2)
    l = torch.empty(1, T, E, dtype=torch.bfloat16, device="cuda")
    for piece in l[0].split(262144):
        piece.copy_(torch.randn(piece.shape, device="cuda"))
    bias = torch.randn(E, device="cuda")
    ids, w = ctx.route(l, bias=bias, **opts)
    gw = torch.randn(1, T, 2, device="cuda")
    grad = ctx.route_backward(l, ids, gw, **opts)
    dense = ctx.route_backward(l, ids, gw, renormalize=False)
    last = l[:, -101:].clone()
    ids2, w2 = ctx.route(last, bias=bias, **opts)
    assert torch.equal(ids[:, -101:], ids2) and torch.equal(w[:, -101:], w2)
    gw2 = gw[:, -101:].clone()
    assert torch.equal(grad[:, -101:], ctx.route_backward(last, ids2, gw2, **opts))
    assert torch.equal(dense[:, -101:], ctx.route_backward(last, ids2, gw2, renormalize=False))
    b = bias.cpu().double().numpy()
    want_ids, _ = P.route(_numpy(last), 2, bias=b, **opts)
    assert np.array_equal(ids2.cpu().numpy().reshape(-1, 2), want_ids)


def test_overlaps_are_refused():
    ctx = _ctx(1, 8, 4)
    l = torch.zeros(1, 8, 32, device="cuda")
    ids, w = ctx.route(l)
    as_ids = l.view(-1)[:32].view(1, 8, 4).view(torch.int32)
    as_w, other = l.view(-1)[:32].view(1, 8, 4), torch.zeros_like(l)
    for call in (lambda: ctx.route(l, topk_ids=as_ids), lambda: ctx.route(l, topk_w=as_w),
                 lambda: ctx.route(l, topk_ids=ids, topk_w=ids.view(torch.float32)),
                 lambda: ctx.route_backward(other, as_ids, w, grad_logits=l),
                 lambda: ctx.route_backward(other, ids, as_w, grad_logits=l)):
        with pytest.raises(EpError) as e:
            call()
        assert e.value.code == B.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("T", [5, 4100])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_signaling_nans_are_missing_experts(dtype, T):
    ctx = _ctx(1, T, 2)
    l = torch.randn(1, T, 16).to(DTYPES[dtype])
    bits = l.view(torch.int32 if dtype == "f32" else torch.int16)
    bits[..., 3] = 0x7f800001 if dtype == "f32" else 0x7f81
    bits[..., 8] = -0x7fffff if dtype == "f32" else -0x7f     # the same, negative
    for opts in (dict(), dict(score="sigmoid", n_groups=4, topk_groups=2, group_score="top2")):
        for bias in (None, torch.zeros(16)):
            ids, _ = ctx.route(l.cuda(), bias=None if bias is None else bias.cuda(), **opts)
            want, _ = P.route(_numpy(l), 2, bias=None if bias is None else bias.numpy(), **opts)
            assert np.array_equal(ids.cpu().numpy()[0], want)


@pytest.mark.parametrize("large", [0.0, 6.0, 9.0, 1e6])
@pytest.mark.parametrize("E,top_k", [(256, 8), (200, 16), (60, 9), (100, 3)])
def test_biases_of_any_size_over_many_tokens(large, E, top_k):
    """Biases that leave the range in which choices are compared as integers, on both
    sides, and groups whose experts are all one lane's."""
    T = 4099
    ctx = _ctx(1, T, top_k)
    l = _logits(E + top_k, 1, T, E, "f32", masked=True)
    bias = torch.linspace(-1, 1, E) * large + 0.1 * torch.randn(E)
    for opts in (dict(score="sigmoid"), dict(n_groups=E // 4 if E == 60 else 4, topk_groups=2,
                                             renormalize=False)):
        ids, _ = ctx.route(l.cuda(), bias=bias.cuda(), **opts)
        want, _ = P.route(_numpy(l), top_k, bias=bias.numpy(), **opts)
        assert np.array_equal(ids.cpu().numpy()[0], want)


@pytest.mark.parametrize("T", [7, 4101])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_single_pick_has_the_whole_weight_and_no_gradient(score, dtype, T):
    ctx = _ctx(1, T, 1)
    l = _logits(T, 1, T, 60, dtype, spread=4.0).cuda()
    ids, w = ctx.route(l, score=score, scale=2.5)
    assert torch.all(w == 2.5)
    d = ctx.route_backward(l, ids, torch.randn(1, T, 1, device="cuda"), score=score, scale=2.5)
    assert torch.all(d == 0)


def test_many_tokens_on_another_stream_and_in_a_graph():
    """The form with a second launch for near ties, captured once and replayed on new logits
    and biases, and two calls at once."""
    T, E = 4500, 250
    opts = dict(score="sigmoid", n_groups=10, topk_groups=4, group_score="top2")
    ctx = _ctx(1, T, 6)
    l, bias = _logits(1, 1, T, E, "bf16").cuda(), (0.1 * torch.randn(E)).cuda()
    l2 = _logits(2, 1, T, E, "bf16").cuda()
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ids1, w1 = ctx.route(l, bias=bias, stream=first, **opts)
    ids2, w2 = ctx.route(l2, bias=bias, stream=second, **opts)
    torch.cuda.synchronize()
    for x, ids, w in ((l, ids1, w1), (l2, ids2, w2)):
        want = ctx.route(x, bias=bias, **opts)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
        assert np.array_equal(ids.cpu().numpy()[0], P.route(
            _numpy(x), 6, bias=bias.cpu().numpy(), **opts)[0])
    ids, w = torch.empty_like(ids1), torch.empty_like(w1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.route(l, bias=bias, topk_ids=ids, topk_w=w, **opts)
        grad = ctx.route_backward(l, ids, w, score="sigmoid")
    for seed in range(3):
        l.copy_(_logits(10 + seed, 1, T, E, "bf16"))
        bias.copy_(0.1 * torch.randn(E))
        graph.replay()
        torch.cuda.synchronize()
        want = ctx.route(l, bias=bias, **opts)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
        assert torch.equal(grad, ctx.route_backward(l, ids, w, score="sigmoid"))


@pytest.mark.parametrize("T", [7, 4101])
@pytest.mark.parametrize("E,n_groups", [(8, 2), (12, 2), (64, 4)])
def test_group_sums_past_the_range_of_binary32(E, n_groups, T):
    """Finite biases whose sums of two overflow binary32, either way: such a group has experts
    to pick, unlike one whose logits are all missing, and its sum is compared in binary64."""
    per = E // n_groups
    ctx = _ctx(1, T, 2)
    l = _logits(E, 1, T, E, "f32")
    missing = l.clone()
    missing[..., :per] = -float("inf")
    low = torch.full((E,), -3e38)
    order = low.clone()
    order[per:2 * per] = -2e38                     # the second group's sum is the larger one
    tied = order.clone()
    tied[:per] = -2e38
    far = torch.full((E,), torch.finfo(torch.float32).min)
    for x, bias in ((missing, low), (l, low), (l, order), (l, tied), (missing, tied),
                    (missing, far), (l, far), (l, -order), (missing, -low)):
        for score in ("sigmoid", "softmax"):
            opts = dict(score=score, n_groups=n_groups, topk_groups=1, group_score="top2")
            ids, w = ctx.route(x.cuda(), bias=bias.cuda(), **opts)
            want_ids, want_w = P.route(_numpy(x), 2, bias=bias.numpy(), **opts)
            assert np.array_equal(ids.cpu().numpy()[0], want_ids)
            assert np.all(np.abs(_numpy(w) - want_w) <= _weight_bound(_numpy(x), E) * want_w)


def test_outputs_over_the_bias_are_refused():
    ctx = _ctx(1, 8, 4)
    l = _logits(5, 1, 8, 32, "f32").cuda()
    room = torch.zeros(64, device="cuda")          # 32 of bias, then 32 of output
    for at in (0, 8, 31):
        out = room[at: at + 32].view(1, 8, 4)
        for kw in (dict(topk_w=out), dict(topk_ids=out.view(torch.int32))):
            with pytest.raises(EpError) as e:
                ctx.route(l, bias=room[:32], **kw)
            assert e.value.code == B.EP_ERR_INVALID_ARG
    want_ids, want_w = ctx.route(l, bias=room[:32].clone())
    ids, w = ctx.route(l, bias=room[:32], topk_w=room[32:].view(1, 8, 4))
    assert torch.equal(ids, want_ids) and torch.equal(w, want_w)
