"""The RMS norm with the residual's addition, its 8-bit output and its gradient, against
float64.  Tolerances: the sum of squares and the mean of the gradient are binary32 sums of at
most 400 sequential operations in any order the kernels use, and a handful of products
follow; a rounding is half a step of the type."""
import numpy as np
import pytest
import torch

import oracle as O
from ep_synth import TINY
from grouped_gemm_scatter_amd import EpError
from grouped_gemm_scatter_amd import binding as B
from gpu_helpers import make_ctx
from oracle import operators as P

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS32 = 2.0 ** -24
# residual's type (None: no residual) and weight's type for each type of rows
KINDS = [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("bf16", None, "bf16"),
         ("f16", "f16", "f16"), ("f16", "f32", "f16"), ("f16", None, "f32"),
         ("f32", "f32", "f32"), ("f32", None, "f32")]
# 128 and 512 values: 16 lanes a row; to 2048 a wave; to 8192 256 threads; more 1024, the last
# with values that no thread can hold
WIDTHS = [128, 384, 512, 640, 2048, 2176, 7168, 8192, 8320, 32768, 33024, 40960]


def _half(t):
    return torch.finfo(t).eps / 2


def _tiny(t):
    """Half a step of the type's smallest numbers."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def _within(err, tol, what):
    assert err.shape == tol.shape
    good = bool(np.all(err <= tol))
    assert good, (what, float((err / tol).max()))


def _ctx(R, T, N, **kw):
    return make_ctx(TINY.replace(n_ranks=R, tokens_per_rank=T, n=N, **kw))


def _np(t):
    return t.double().cpu().numpy()


def _inputs(R, T, N, kind, seed, size=1.0):
    x_type, res_type, w_type = kind
    g = torch.Generator().manual_seed(seed)
    x = (size * torch.randn(R, T, N, generator=g)).to(TYPES[x_type]).cuda()
    res = None
    if res_type:
        res = (3 * size * torch.randn(R, T, N, generator=g)).to(TYPES[res_type]).cuda()
    w = (0.8 + 0.4 * torch.rand(N, generator=g)).to(TYPES[w_type]).cuda()
    return x, res, w


def _check_norm(got, x, res, w, eps, rows, fp8):
    s, y = P.rms_norm(_np(x), _np(w), residual=None if res is None else _np(res), eps=eps)
    sum_err = 2.0 ** -17 * np.abs(y)               # 128 steps of 2^-24
    assert (got.out is not None) == rows and (got.codes is not None) == fp8
    if res is not None:
        t = res.dtype
        assert got.residual.dtype == t
        bound = (_half(t) + EPS32) * np.abs(s) + _tiny(t)
        _within(np.abs(_np(got.residual) - s), bound, "sums")
    else:
        assert got.residual is None
    if rows:
        assert got.out.dtype == x.dtype
        _within(np.abs(_np(got.out) - y),
                sum_err + _half(x.dtype) * np.abs(y) * 1.01 + _tiny(x.dtype), "rows")
    if fp8:
        blocks = np.abs(y).reshape(*y.shape[:2], -1, 128).max(-1)
        want = np.where(blocks > 0, np.maximum(blocks / 448, 2.0 ** -126), 1.0)
        scales = _np(got.scales)
        _within(np.abs(scales - want), (2.0 ** -17 + EPS32) * want, "scales")
        sc = np.repeat(scales, 128, axis=-1)
        values = O.e4m3fn_to_f64(got.codes.cpu().numpy()) * sc
        half = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * sc)
        _within(np.abs(values - y), half * (1 + 2.0 ** -20) + 2 * sum_err, "codes")


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "-".join(map(str, k)))
def test_norm_of_every_width(N, kind):
    R, T = 2, 3 if N > 8192 else 19
    print(f"[case] norm N={N} {kind}", flush=True)
    x, res, w = _inputs(R, T, N, kind, N)
    ctx = _ctx(R, T, N)
    for rows, fp8 in ((True, False), (True, True), (False, True)):
        got = ctx.rms_norm(x, w, residual=res, eps=1e-5, rows=rows, fp8=fp8)
        torch.cuda.synchronize()
        _check_norm(got, x, res, w, 1e-5, rows, fp8)
    assert ctx.query_error() == 0


@pytest.mark.parametrize("R,T", [(1, 1), (8, 1), (3, 77), (8, 700)])
@pytest.mark.parametrize("N", [256, 1024, 4096])
def test_norm_of_few_and_many_rows(R, T, N):
    print(f"[case] norm rows {R}x{T} N={N}", flush=True)
    x, res, w = _inputs(R, T, N, ("bf16", "bf16", "bf16"), T)
    ctx = _ctx(R, T, N)
    got = ctx.rms_norm(x, w, residual=res, fp8=True)
    torch.cuda.synchronize()
    _check_norm(got, x, res, w, 1e-6, True, True)


@pytest.mark.parametrize("N", [128, 896, 7168])
def test_codes_are_those_of_the_rows_in_32_bits(N):
    """The rows that come out in 32 bits are what the codes are made of: codes and scales
    equal the oracle's quantisation of them bit for bit."""
    x, _, w = _inputs(1, 33, N, ("f32", None, "f32"), 5)
    x[0, 3] = 0                                    # a row of zeros
    x[0, 4, :128] = 0                              # a block of zeros
    x[0, 5] *= torch.exp(6 * torch.randn(N, device="cuda"))
    got = _ctx(1, 33, N).rms_norm(x, w, fp8=True)
    torch.cuda.synchronize()
    codes, scales = O.quantize_rows_e4m3(got.out[0].cpu().numpy())
    assert np.array_equal(got.codes[0].cpu().numpy(), codes)
    assert np.array_equal(got.scales[0].cpu().numpy(), scales)
    assert torch.all(got.out[0, 3] == 0) and torch.all(got.scales[0, 3] == 1)


def test_tiny_rows_have_finite_codes():
    """Norms of 1e-42: their scale stays a normal number and no code is NaN."""
    x = torch.full((1, 2, 128), 1e-38, device="cuda")
    x[0, 1, 5] = -2e-38
    w = torch.full((128,), 1e-7, device="cuda")
    got = _ctx(1, 2, 128).rms_norm(x, w, eps=1.0, fp8=True)
    torch.cuda.synchronize()
    assert torch.all(got.scales == 2.0 ** -126)
    assert torch.all((got.codes & 0x7F) <= 0x7E)


def test_numbers_without_an_end_stay_in_their_row():
    for N in (256, 1024, 7168):
        x, res, w = _inputs(1, 40, N, ("bf16", "bf16", "bf16"), 6)
        g = torch.randn(1, 40, N, device="cuda").bfloat16()
        ctx = _ctx(1, 40, N)
        want = ctx.rms_norm(x, w, residual=res, fp8=True)
        d = ctx.rms_norm_backward(g, want.residual, w)
        bad = x.clone()
        bad[0, 3, 17] = float("inf")
        bad[0, 39, N - 1] = float("nan")
        got = ctx.rms_norm(bad, w, residual=res, fp8=True)
        e = ctx.rms_norm_backward(g, got.residual, w)
        keep = torch.ones(40, dtype=torch.bool)
        keep[3] = keep[39] = False
        for a, b in ((want.out, got.out), (want.codes, got.codes), (want.scales, got.scales),
                     (want.residual, got.residual), (d.x, e.x)):
            assert torch.equal(a[0, keep], b[0, keep])
        assert torch.isnan(got.out[0, 39]).all() and not torch.isfinite(got.out[0, 3]).all()


def _check_backward(ctx, x_type, sums, w, g, q, eps=1e-5):
    d = ctx.rms_norm_backward(g, sums, w, grad_residual=q, eps=eps)
    torch.cuda.synchronize()
    N = sums.shape[-1]
    ds, dw, bs, bw = P.rms_norm_backward(
        _np(g).reshape(-1, N), _np(sums).reshape(-1, N), _np(w),
        grad_residual=None if q is None else _np(q).reshape(-1, N), eps=eps)
    rows = ds.shape[0]
    for got, t in ((d.x, g.dtype), (d.residual, sums.dtype)):
        assert got.dtype == t
        err = np.abs(_np(got).reshape(-1, N) - ds)
        _within(err, 450 * EPS32 * bs + _half(t) * np.abs(ds) * 1.01 + _tiny(t), "sums")
    assert d.weight.dtype == torch.float32
    _within(np.abs(_np(d.weight) - dw), (rows + 400) * EPS32 * bw + 1e-38, "weight")
    return d


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "-".join(map(str, k)))
def test_gradient_of_every_width(N, kind):
    R, T = 2, 3 if N > 8192 else 19
    print(f"[case] norm gradient N={N} {kind}", flush=True)
    x_type, res_type, _ = kind
    x, res, w = _inputs(R, T, N, kind, N + 1)
    sums = x if res is None else (x.float() + res.float()).to(res.dtype)
    gen = torch.Generator().manual_seed(N)
    g = torch.randn(R, T, N, generator=gen).to(x.dtype).cuda()
    q = None if res is None else torch.randn(R, T, N, generator=gen).to(res.dtype).cuda()
    _check_backward(_ctx(R, T, N), x_type, sums, w, g, q)
    _check_backward(_ctx(R, T, N), x_type, sums, w, g, None)


@pytest.mark.parametrize("R,T,N", [(1, 1, 7168), (8, 1, 128), (3, 411, 256), (8, 700, 1024),
                                   (7, 301, 2176), (1, 2100, 8320), (1, 300, 33024)])
def test_gradient_of_few_and_many_rows(R, T, N):
    """More rows than workgroups: each adds up the weights' gradient of several."""
    print(f"[case] norm gradient rows {R}x{T} N={N}", flush=True)
    x, _, w = _inputs(R, T, N, ("bf16", None, "bf16"), T)
    g = torch.randn(R, T, N, device="cuda").bfloat16()
    q = torch.randn(R, T, N, device="cuda").bfloat16()
    ctx = _ctx(R, T, N)
    d = _check_backward(ctx, "bf16", x, w, g, q)
    again = ctx.rms_norm_backward(g, x, w, grad_residual=q, eps=1e-5)
    assert torch.equal(d.x, again.x) and torch.equal(d.weight, again.weight)


def test_gradient_is_that_of_differences():
    """Along a random direction, from the kernel's own outputs in 32 bits.  The loss is
    summed in 64 bits; a central difference of step h is off by h^2/6 of the third
    derivative and by the outputs' rounding over h."""
    R, T, N, h = 1, 4, 256, 1e-2
    x, _, w = _inputs(R, T, N, ("f32", None, "f32"), 11)
    g = torch.randn(R, T, N, device="cuda")
    ctx = _ctx(R, T, N)
    d = ctx.rms_norm_backward(g, x, w)

    def loss(x, w):
        return (ctx.rms_norm(x, w).out.double() * g.double()).sum().item()

    v = torch.randn_like(x)
    u = torch.randn_like(w)
    size = (d.x.double().abs() * v.double().abs()).sum().item()
    for got, want in (((loss(x + h * v, w) - loss(x - h * v, w)) / (2 * h),
                       (d.x.double() * v.double()).sum().item()),
                      ((loss(x, w + h * u) - loss(x, w - h * u)) / (2 * h),
                       (d.weight.double() * u.double()).sum().item())):
        # values of size 1 over rows of size 1: the third derivative along v is within
        # 100 |v|^3 of a row's, the rounding 2^-22 of 1024 values over h
        assert abs(got - want) <= 100 * h * h * size + 1024 * 2.0 ** -22 * 4 / h


def test_in_place():
    """The sums over the residual, the rows over x, gradients over gradients."""
    for N in (384, 7168, 33024):
        for kind in (("bf16", "bf16", "bf16"), ("f16", "f32", "f32")):
            x, res, w = _inputs(2, 5, N, kind, 8)
            ctx = _ctx(2, 5, N)
            want = ctx.rms_norm(x, w, residual=res, fp8=True)
            x2, res2 = x.clone(), res.clone()
            got = ctx.rms_norm(x2, w, residual=res2, fp8=True, out=x2, residual_out=res2)
            assert got.out is x2 and got.residual is res2
            for a, b in zip(want, got):
                assert torch.equal(a, b)
            g, q = torch.randn_like(x), torch.randn_like(res)
            d = ctx.rms_norm_backward(g, want.residual, w, grad_residual=q)
            g2, q2 = g.clone(), q.clone()
            more = {} if kind[0] == kind[1] else {"grad_sums": q2}
            e = ctx.rms_norm_backward(g2, want.residual, w, grad_residual=q2, grad_x=g2, **more)
            for a, b in zip(d, e):
                assert torch.equal(a, b)


def test_a_residual_that_is_x():
    """s = 2 x, the rows over both."""
    x, _, w = _inputs(1, 5, 640, ("bf16", None, "bf16"), 13)
    ctx = _ctx(1, 5, 640)
    want = ctx.rms_norm(x, w, residual=x.clone())
    y = x.clone()
    got = ctx.rms_norm(y, w, residual=y, out=y)
    assert torch.equal(got.out, want.out) and torch.equal(got.residual, want.residual)


def test_sums_without_a_residual():
    """At the C boundary: the stored sums are x, in the residual's type."""
    x, _, w = _inputs(1, 7, 640, ("f16", None, "f16"), 14)
    ctx = _ctx(1, 7, 640)
    for t in (torch.float16, torch.float32):
        p = B.make_norm_params(dtype=torch.float16, residual_dtype=t)
        kept = torch.empty(1, 7, 640, dtype=t, device="cuda")
        out = torch.empty_like(x)
        B.ep_rms_norm(ctx.handle, p, x, None, w, 7, kept, out, None, None)
        assert torch.equal(kept, x.to(t))
        assert torch.equal(out, ctx.rms_norm(x, w, eps=1e-6).out)


def test_no_eps_and_values_out_of_range():
    """eps = 0 on a row of zeros, squares past binary32, an infinity, a NaN: as documented."""
    x = torch.ones(1, 5, 256, device="cuda")
    x[0, 0] = 0
    x[0, 1] = 3e19
    x[0, 2, 7] = float("inf")
    x[0, 3, 200] = float("nan")
    w = torch.full((256,), 2.0, device="cuda")
    y = _ctx(1, 5, 256).rms_norm(x, w, eps=0.0, fp8=True)
    torch.cuda.synchronize()
    assert torch.isnan(y.out[0, 0]).all() and torch.all(y.out[0, 1] == 0)
    assert torch.isnan(y.out[0, 2, 7]) and torch.all(y.out[0, 2, :7] == 0)
    assert torch.isnan(y.out[0, 3]).all() and torch.all(y.out[0, 4] == 2)
    assert torch.all((y.codes[0, 3] & 0x7F) == 0x7F) and torch.all((y.codes[0, 0] & 0x7F) == 0x7F)
    assert (y.codes[0, 2, 7] & 0x7F) == 0x7F and torch.all(y.codes[0, 2, 8:] == 0)
    assert torch.all(y.scales[0, :4] == 1) and torch.all(y.scales[0, 4] == np.float32(2) / 448)


def test_no_tokens():
    ctx = _ctx(2, 4, 256)
    x = torch.empty(2, 0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    got = ctx.rms_norm(x, w, residual=x, fp8=True)
    assert got.out.shape == x.shape and got.scales.shape == (2, 0, 2)
    d = ctx.rms_norm_backward(x, x, w, grad_weight=torch.full((256,), 7.0, device="cuda"))
    torch.cuda.synchronize()
    assert d.x.shape == x.shape and torch.all(d.weight == 0)


def test_rows_behind_the_last_are_left():
    """Buffers of more rows than the call has: nothing is written past its own."""
    for N in (128, 1024, 4096, 8320):
        R, T = 1, 5
        x, res, w = _inputs(R, T, N, ("bf16", "f32", "f32"), 9)
        ctx = _ctx(R, T, N)
        room = [torch.full((R, T + 3, N), 7, dtype=t, device="cuda")
                for t in (torch.bfloat16, torch.float32, torch.uint8)]
        scales = torch.full((R, T + 3, N // 128), 7.0, device="cuda")
        out, kept, codes = (t[:, :T] for t in room)
        got = ctx.rms_norm(x, w, residual=res, fp8=True, out=out, residual_out=kept, codes=codes,
                           scales=scales[:, :T])
        _check_norm(got, x, res, w, 1e-6, True, True)
        g = torch.randn(R, T, N, device="cuda").bfloat16()
        grads = [torch.full((R, T + 3, N), 7.0, dtype=t, device="cuda")
                 for t in (torch.bfloat16, torch.float32)]
        wide = torch.full((N + 64,), 7.0, device="cuda")
        ctx.rms_norm_backward(g, got.residual, w, grad_x=grads[0][:, :T], grad_sums=grads[1][:, :T],
                              grad_weight=wide[:N])
        torch.cuda.synchronize()
        for t in room + grads + [scales]:
            assert torch.all(t[:, T:] == 7)
        assert torch.all(wide[N:] == 7)


def test_rows_past_four_gib():
    """Rows whose byte offsets pass 32 bits (and whose values pass 2^31)."""
    R, T, N = 1, 300000, 7168
    ctx = _big_handle(T, N)
    x = torch.empty(R, T, N, dtype=torch.bfloat16, device="cuda")
    for piece in x[0].split(32768):
        piece.copy_(torch.randn(piece.shape, device="cuda"))
    w = torch.rand(N, device="cuda").bfloat16()
    got = ctx.rms_norm(x, w, fp8=True)
    d = ctx.rms_norm_backward(x, x, w, grad_x=got.out)
    tail = x[:, -40:].clone()
    small = _ctx(1, 40, N)
    want = small.rms_norm(tail, w, fp8=True)
    dt = small.rms_norm_backward(tail, tail, w)
    torch.cuda.synchronize()
    assert torch.equal(got.codes[:, -40:], want.codes)
    assert torch.equal(got.scales[:, -40:], want.scales)
    assert torch.equal(d.x[:, -40:], dt.x)
    _check_norm(want, tail, None, w, 1e-6, True, True)


def _big_handle(T, N):
    """A handle for many tokens whose receive slots no call of the norm touches: one pick, and
    one shared buffer."""
    from grouped_gemm_scatter_amd import EpCombine
    return EpCombine(n_ranks=1, top_k=1, max_tokens_per_rank=T, n_experts_per_device=1,
                     hidden_k=128, hidden_n=N)


def test_on_a_late_stream_and_in_graphs():
    R, T, N = 2, 9, 1024
    x, res, w = _inputs(R, T, N, ("bf16", "bf16", "bf16"), 10)
    g, q = torch.randn_like(x), torch.randn_like(x)
    ctx = _ctx(R, T, N)

    def run(x, stream=None):
        y = ctx.rms_norm(x, w, residual=res, fp8=True, stream=stream)
        d = ctx.rms_norm_backward(g, y.residual, w, grad_residual=q, stream=stream)
        return [*y, d.x, d.weight]

    want = [t.clone() for t in run(x)]
    torch.cuda.synchronize()
    late, stale = torch.cuda.Stream(), torch.zeros_like(x)
    late.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(late):
        torch.cuda._sleep(20_000_000)
        stale.copy_(x)
    got = run(stale, late)
    late.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # two graphs, replayed in turn beside eager calls
    inputs, graphs = [x.clone(), x.clone()], []
    for inp in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = run(inp)
        graphs.append((graph, outs))
    for seed in range(3):
        for inp, (graph, outs) in zip(inputs, graphs):
            inp.copy_(torch.randn(x.shape, device="cuda"))
            graph.replay()
        eager = [run(inp) for inp in inputs]
        torch.cuda.synchronize()
        for (_, outs), e in zip(graphs, eager):
            assert all(torch.equal(a, b) for a, b in zip(outs, e))


def test_refusals():
    R, T, N = 1, 6, 256
    x, res, w = _inputs(R, T, N, ("bf16", "bf16", "bf16"), 12)
    ctx = _ctx(R, T, N)
    g = torch.randn_like(x)
    wide = torch.zeros(R, T, 2 * N, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: ctx.rms_norm(wide[..., ::2], w), lambda: ctx.rms_norm(x.cpu(), w),
                 lambda: ctx.rms_norm(x, w[:-1]), lambda: ctx.rms_norm(x, w.half()),
                 lambda: ctx.rms_norm(x, w, residual=res.half()),
                 lambda: ctx.rms_norm(x, w, residual=res[:, :-1]),
                 lambda: ctx.rms_norm(x, w, rows=False),
                 lambda: ctx.rms_norm(x, w, out=x.float()),
                 lambda: ctx.rms_norm(x, w, rows=False, fp8=True, out=x),
                 lambda: ctx.rms_norm(x, w, residual_out=res),
                 lambda: ctx.rms_norm(x, w, codes=torch.zeros(R, T, N, device="cuda").byte()),
                 lambda: ctx.rms_norm_backward(g, x.half(), w),
                 lambda: ctx.rms_norm_backward(g, x, w, grad_residual=g.float()),
                 lambda: ctx.rms_norm_backward(g, x, w, grad_sums=res),
                 lambda: ctx.rms_norm_backward(g[..., :128], x, w)):
        with pytest.raises(ValueError):
            call()
    more = torch.zeros(R, T + 1, N, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: ctx.rms_norm(more, w),                  # more tokens than the handle
                 lambda: ctx.rms_norm_backward(more, more, w),
                 lambda: ctx.rms_norm(x, w, eps=-1.0), lambda: ctx.rms_norm(x, w, eps=float("nan")),
                 lambda: ctx.rms_norm(x, w, residual=res, out=res),
                 lambda: ctx.rms_norm(x, w, residual=res, residual_out=x),
                 lambda: ctx.rms_norm(x, w, residual=res, residual_out=more[:, :T], out=more[:, :T]),
                 lambda: ctx.rms_norm(x, w, fp8=True, out=more[:, :T], codes=more.view(
                     torch.uint8).view(-1)[N:][:R * T * N].view(R, T, N)),
                 lambda: ctx.rms_norm_backward(g, x, w, grad_x=x),
                 lambda: ctx.rms_norm_backward(g, x, w, grad_residual=res, grad_x=res)):
        with pytest.raises(EpError) as e:
            call()
        assert e.value.code == B.EP_ERR_INVALID_ARG
    p = B.make_norm_params(dtype=torch.bfloat16)
    for field, value in (("dtype", 3), ("dtype", -1), ("residual_dtype", 2), ("weight_dtype", 2)):
        f = B.EpNormParams.from_buffer_copy(p)
        setattr(f, field, value)
        with pytest.raises(EpError):
            B.ep_rms_norm(ctx.handle, f, x, None, w, T, None, torch.empty_like(x), None, None)
    out = torch.empty_like(x)
    for args in ((None, None, w, T, None, out, None, None), (x, None, w, T, None, None, None, None),
                 (x, None, w, T, None, out, torch.empty(R, T, N, dtype=torch.uint8, device="cuda"),
                  None),
                 (x.data_ptr() + 2, None, w, T, None, out, None, None)):
        with pytest.raises(EpError):
            B.ep_rms_norm(ctx.handle, p, *args)
    need = B.ep_rms_norm_backward_workspace(ctx.handle, T)
    ws, gw = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(N, device="cuda")
    for args in ((g, None, x, w, T, out, None, gw, ws, need - 1),
                 (g, None, x, w, T, None, None, gw, ws, need),
                 (g, None, x, w, T, out, None, gw, None, need),
                 (g, None, x, w, T, out, None, gw, out, need),
                 (None, None, x, w, T, out, None, gw, ws, need)):
        with pytest.raises(EpError):
            B.ep_rms_norm_backward(ctx.handle, p, *args)
    with pytest.raises(EpError):
        B.ep_rms_norm_backward_workspace(ctx.handle, T + 1)
