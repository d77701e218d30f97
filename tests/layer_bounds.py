"""Measures of error for the norm's gradient and the few-token layer that a wrong kernel
cannot meet: tests of the kernels and of the measures themselves share them."""
import numpy as np
import torch


def along_rows(norm, gradient, r, w, g, eps, h=2.0 ** -6):
    """(error, tolerance) of a gradient of the norm along the rows themselves: the derivative of
    sum(g y(u r)) by u at 1, from norm(x) -> y at u = 1 +- h, against sum(gradient r).

    With m = mean(r^2), y(u r) = r w u / sqrt(u^2 m + eps), whose derivative at 1 is
    r w eps / s^1.5, s = m + eps: the gradient's second term takes nearly all of the first
    away where eps is small beside m.  A central difference is off by h^2 / 6 of the third
    derivative, eps (15 u^2 m^2 / s^3.5 - 3 m / s^2.5) |r w| (s at u); outputs are off by at
    most 2^-17 (128 operations of 2^-24), and by 2^-22 for x's own rounding, over h; the
    gradient by 450 operations of the terms that make it."""
    m = (r * r).mean(-1, keepdims=True)
    top = np.abs(g * w * r)
    low = (1 - h) ** 2 * m + eps
    third = eps * (15 * (1 + h) ** 2 * m * m / low ** 3.5 + 3 * m / low ** 2.5)
    up, down = norm((1 + h) * r), norm((1 - h) * r)
    got = (g * up - g * down).sum() / (2 * h)
    want = (gradient(g, r) * r).sum()
    inv = 1 / np.sqrt(m + eps)
    terms = inv * (top + r * r * inv ** 2 * top.mean(-1, keepdims=True))
    tol = ((h * h / 6 * third * top).sum() +
           ((2.0 ** -17 + 2.0 ** -22) * top / np.sqrt(low)).sum() / h +
           450 * 2.0 ** -24 * terms.sum())
    return abs(got - want), tol


def gradient_inputs(rows, N, seed):
    """Rows of size 1, weights, and a gradient with a part along the outputs."""
    rng = np.random.default_rng(seed)
    r = rng.standard_normal((rows, N)).astype(np.float32).astype(np.float64)
    w = (0.8 + 0.4 * rng.random(N)).astype(np.float32).astype(np.float64)
    g = (r * w + rng.standard_normal((rows, N))).astype(np.float32).astype(np.float64)
    return r, w, g


def layer(x, w1, w2, ids, topk_w, expert_lo=0):
    """(out, spread) of the few-token layer in float64 torch tensors, on any device: tokens x
    [n][hidden] with picks ids and weights topk_w [n][k], lists (or functions) w1 and w2 of
    the local experts' weights.  spread [n][hidden] is the root of the sum of the squares of
    the terms c w2 h that make an output."""
    out, square = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(len(w1)):
        share = (topk_w * (ids == e + expert_lo)).sum(-1, dtype=torch.float64)
        t = torch.nonzero((ids == e + expert_lo).any(-1)).flatten()
        if t.numel() == 0:
            continue
        a, b = w1[e].double(), w2[e].double()
        y = torch.mm(a, x[t].t().contiguous())
        h = y[:len(y) // 2] / (1 + torch.exp(-y[:len(y) // 2])) * y[len(y) // 2:]
        out[t] += share[t, None] * torch.mm(b, h).t()
        square[t] += share[t, None] ** 2 * torch.mm(b * b, h * h).t()
    return out, square.sqrt()


def layer_error(got, want, spread):
    """How far `got` is off as a part of what is allowed (at most 1 is right).

    The hidden values are two bf16 parts, within 2^-17 of what they stand for.  Their
    roundings are independent, so their sum passes t times 2^-17 of the spread of an output's
    terms with a probability of 2 exp(-t^2 / 2) at most: for t = 8.2 once in 10^14.  The sums
    in binary32 are a few hundred additions within 2^-23 of a partial sum each, those of a
    hidden value and of an output alike, whose signs are as good as random: 2 (300)^(1/2)
    2^-23 is under 2^-17, of partial sums of up to a few spreads; 2^-13 is allowed for them.
    The output is rounded once: half a step of bf16."""
    delta = 8.2 * (2.0 ** -17 + 2.0 ** -13) * spread
    half = torch.exp2(torch.floor(torch.log2(want.abs() + delta + 1e-38)) - 8)
    return float(((got.double() - want).abs() / (half + delta + 1e-38)).max())
