"""The norm and its gradient where their rows go past the caches' replacement (calls that
move over 134 MB do), against the same rows in small calls, and at the widths next to each
change of the threads a row takes: 16 lanes to 256 values, a wave to 1024, 256 threads to
4096, 512 to 8192, 1024 beyond, and values that are read again past 16384."""
import pytest
import torch

from test_gpu_norm import KINDS, TYPES, _check_backward, _check_norm, _ctx, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [256, 1024, 4096, 4224, 16384, 16512])
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "-".join(map(str, k)))
def test_widths_at_the_changes(N, kind):
    R, T = 2, 3 if N > 8192 else 19
    print(f"[case] norm and gradient N={N} {kind}", flush=True)
    x, res, w = _inputs(R, T, N, kind, N)
    ctx = _ctx(R, T, N)
    for rows, fp8 in ((True, False), (True, True), (False, True)):
        got = ctx.rms_norm(x, w, residual=res, eps=1e-5, rows=rows, fp8=fp8)
        torch.cuda.synchronize()
        _check_norm(got, x, res, w, 1e-5, rows, fp8)
    gen = torch.Generator().manual_seed(N)
    g = torch.randn(R, T, N, generator=gen).to(x.dtype).cuda()
    sums = x if res is None else got.residual
    q = None if res is None else torch.randn(R, T, N, generator=gen).to(res.dtype).cuda()
    _check_backward(ctx, kind[0], sums, w, g, q)


STREAMED = [("bf16", None, "bf16"), ("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"),
            ("f16", None, "f32"), ("f16", "f16", "f16"), ("f16", "f32", "f32")]


def _streamed_inputs(kind, N, T, seed):
    x_type, res_type, w_type = kind
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rnd(1, T, N).to(TYPES[x_type])
    res = None if res_type is None else (3 * rnd(1, T, N)).to(TYPES[res_type])
    w = (1 + 0.1 * rnd(N)).to(TYPES[w_type])
    go = rnd(1, T, N).to(x.dtype)
    q = None if res is None else rnd(1, T, N).to(res.dtype)
    return x, res, w, go, q


def _pieces(T, N):
    """Parts of the rows, each a call of a few MB."""
    step = max(1, (1 << 19) // N)
    return [slice(t, min(t + step, T)) for t in range(0, T, step)][:: max(1, T // step // 12)] + [
        slice(max(T - step, 0), T)]


# rows of a wave, of 512 threads, and of 1024 with values that are read again
@pytest.mark.parametrize("N", [640, 7168, 17408])
@pytest.mark.parametrize("kind", STREAMED, ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("in_place", [False, True], ids=["", "in_place"])
def test_streamed_rows_are_those_of_small_calls(kind, N, in_place):
    T = (160 << 20) // (4 * N) + 1          # 4 bytes a value at least, x and the rows
    print(f"[case] streamed norm {kind} N={N} T={T} in_place={in_place}", flush=True)
    x, res, w, go, q = _streamed_inputs(kind, N, T, N)
    pieces = _pieces(T, N)
    small = _ctx(1, max(p.stop - p.start for p in pieces), N)
    parts = [(p, small.rms_norm(x[:, p], w, residual=None if res is None else res[:, p], fp8=True))
             for p in pieces]
    ctx = _ctx(1, T, N)
    p0, part = pieces[0], parts[0][1]
    _check_norm(part, x[:, p0], None if res is None else res[:, p0], w, 1e-6, True, True)
    into = dict(out=x, **({} if res is None else {"residual_out": res})) if in_place else {}
    got = ctx.rms_norm(x, w, residual=res, fp8=True, **into)
    assert got.out is x or not in_place
    for p, want in parts:
        for a, b in zip(got, want):
            assert (a is None) == (b is None)
            assert a is None or torch.equal(a[:, p], b)


@pytest.mark.parametrize("N", [640, 7168, 17408])
@pytest.mark.parametrize("kind", STREAMED, ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("in_place", [False, True], ids=["", "in_place"])
def test_streamed_gradient_is_that_of_small_calls(kind, N, in_place):
    T = (160 << 20) // (6 * N) + 1          # 6 bytes a value at least
    print(f"[case] streamed norm gradient {kind} N={N} T={T} in_place={in_place}", flush=True)
    x, res, w, go, q = _streamed_inputs(kind, N, T, N + 1)
    sums = x if res is None else res
    pieces = _pieces(T, N)
    small = _ctx(1, max(p.stop - p.start for p in pieces), N)
    parts = [(p, small.rms_norm_backward(go[:, p], sums[:, p], w,
                                         grad_residual=None if q is None else q[:, p]))
             for p in pieces]
    p0 = pieces[0]
    _check_backward(small, kind[0], sums[:, p0], w, go[:, p0], None if q is None else q[:, p0])
    # the weight's gradient in 64 bits, some rows at a time, with the sum of its terms' sizes
    want, size = torch.zeros(2, N, dtype=torch.float64, device="cuda")
    for g, r in zip(go[0].split(2048), sums[0].split(2048)):
        r = r.double()
        each = g.double() * r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6)
        want += each.sum(0)
        size += each.abs().sum(0)
    ctx = _ctx(1, T, N)
    into = {}
    if in_place:
        into["grad_x"] = go
        if q is not None and q.dtype != go.dtype:
            into["grad_sums"] = q
    d = ctx.rms_norm_backward(go, sums, w, grad_residual=q, **into)
    assert d.x is go or not in_place
    for p, e in parts:
        assert torch.equal(d.x[:, p], e.x) and torch.equal(d.residual[:, p], e.residual)
    # 400 operations for 1 / rms; at most T additions, one after the other
    assert torch.all((d.weight - want).abs() <= (T + 400) * 2.0 ** -24 * size)
