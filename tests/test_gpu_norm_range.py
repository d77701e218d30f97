"""The norm and its gradient on rows so small that the square of 1 / rms is past binary32,
against float64.  Rows are signed powers of two, whose squares are whole multiples of
2^-149, binary32's smallest number, so their sum is exact; the mean's rounding is half of
that, 2^-150, for means of 2^-132 and more a relative 2^-18, of which 1 / rms has half and
the gradient's second term, in which it stands three times, 2^-16.4.  Sums of N terms take at
most 400 operations of 2^-24 in the kernels' order, as in the other tests of the norm."""
import numpy as np
import pytest
import torch

from ep_synth import TINY
from gpu_helpers import make_ctx
from oracle import operators as P

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _np(t):
    return t.double().cpu().numpy()


def _half(t):
    return torch.finfo(t).eps / 2


def _rows(R, T, N, t):
    """Signed powers of two, 2^-66 to 2^-64 within a row and between rows."""
    g = torch.Generator().manual_seed(N)
    e = torch.randint(-66, -63, (R, T, N), generator=g)
    e[:, 0] = -66
    sign = 2.0 * torch.randint(0, 2, (R, T, N), generator=g) - 1
    return (sign * torch.exp2(e.float())).to(t).cuda()


@pytest.mark.parametrize("kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")],
                         ids=lambda k: "-".join(k))
@pytest.mark.parametrize("N", [256, 2176, 33024])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -133])
def test_gradient_where_the_square_of_one_over_rms_is_past_the_range(N, kind, eps):
    print(f"[case] small rows N={N} {kind} eps={eps}", flush=True)
    x_type, sum_type = (TYPES[k] for k in kind)
    R, T = 2, 3
    sums = _rows(R, T, N, sum_type)
    gen = torch.Generator().manual_seed(N + 1)
    # a part along the rows, so that the gradient's second term counts
    along = (sums.cpu() * 2.0 ** 65).float()
    g = (torch.randn(R, T, N, generator=gen) + along).to(x_type).cuda()
    w = (0.8 + 0.4 * torch.rand(N, generator=gen)).cuda()
    ctx = make_ctx(TINY.replace(n_ranks=R, tokens_per_rank=T, n=N))
    d = ctx.rms_norm_backward(g, sums, w, eps=eps)
    torch.cuda.synchronize()
    ds, dw, bs, bw = P.rms_norm_backward(_np(g).reshape(-1, N), _np(sums).reshape(-1, N), _np(w),
                                         eps=eps)
    for got in (d.x, d.residual):
        err = np.abs(_np(got).reshape(-1, N) - ds)
        assert np.all(err <= (450 * 2.0 ** -24 + 2.0 ** -16) * bs +
                      _half(got.dtype) * 1.01 * np.abs(ds))
    assert np.all(np.abs(_np(d.weight) - dw) <= (406 * 2.0 ** -24 + 2.0 ** -19) * bw)


@pytest.mark.parametrize("kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")],
                         ids=lambda k: "-".join(k))
def test_norm_of_the_same_rows(kind):
    R, T, N = 2, 3, 2176
    x = _rows(R, T, N, TYPES[kind[0]])
    w = torch.ones(N, device="cuda")
    res = torch.zeros(R, T, N, dtype=TYPES[kind[1]], device="cuda")
    y = make_ctx(TINY.replace(n_ranks=R, tokens_per_rank=T, n=N)).rms_norm(
        x, w, residual=res, eps=0.0)
    _, want = P.rms_norm(_np(x), _np(w), eps=0.0)
    err = np.abs(_np(y.out) - want)
    assert np.all(err <= (2.0 ** -17 + 2.0 ** -19 + _half(x.dtype) * 1.01) * np.abs(want))
    assert torch.equal(y.residual, x.to(res.dtype))


def test_an_infinite_output_and_its_block():
    """An infinite weight: its own value infinite, the code NaN, the block's scale infinite;
    the other block as it was."""
    x, w = torch.ones(1, 3, 256, device="cuda"), torch.ones(256, device="cuda")
    ctx = make_ctx(TINY.replace(n_ranks=1, tokens_per_rank=3, n=256))
    want = ctx.rms_norm(x, w, fp8=True)
    w[3] = float("inf")
    y = ctx.rms_norm(x, w, fp8=True)
    assert torch.all(y.out[..., 3] == float("inf")) and torch.all((y.codes[..., 3] & 127) == 127)
    assert torch.all(y.scales[..., 0] == float("inf"))
    keep = torch.arange(256) != 3
    assert torch.equal(y.out[..., keep], want.out[..., keep])
    assert torch.equal(y.codes[..., 128:], want.codes[..., 128:])
    assert torch.equal(y.scales[..., 1], want.scales[..., 1])
