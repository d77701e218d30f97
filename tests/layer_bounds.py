"""Measures of error for the norm's gradient and the few-token layer that a wrong kernel
cannot meet: tests of the kernels and of the measures themselves share them."""
import numpy as np


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
