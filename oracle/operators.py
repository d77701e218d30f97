"""Plain float64 definitions of the router, the 4-bit expert products and the gradients
of the combine.  TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no
code with the HIP path."""
from __future__ import annotations

import numpy as np

from . import bf16_to_f64

FLT_MAX = float(np.finfo(np.float32).max)
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def clean_logits(logits) -> np.ndarray:
    """Logits in float64: +infinity at the largest binary32 number, a missing expert
    (NaN or -infinity) at -infinity."""
    l = np.asarray(logits, dtype=np.float64)
    return np.where(np.isnan(l), -np.inf, np.minimum(l, FLT_MAX))


def scores(logits, score) -> np.ndarray:
    """Scores of cleaned logits [n][E]; 0 for a missing expert."""
    l = clean_logits(logits)
    here = l > -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return np.where(here, 1.0 / (1.0 + np.exp(-l)), 0.0)
        top = l.max(axis=-1, keepdims=True)
        e = np.where(here, np.exp(np.where(here, l - top, -np.inf)), 0.0)
    total = e.sum(axis=-1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def pick_shares(logits, ids, score) -> np.ndarray:
    """Scores of the picks ids [n][k] over their sum (0 for a pick that is not there),
    from the logarithms of the scores, so that tiny ones keep their shares."""
    l = clean_logits(logits)
    ids = np.asarray(ids)
    inside = (ids >= 0) & (ids < l.shape[1])
    x = np.take_along_axis(l, np.where(inside, ids, 0), axis=1)
    there = inside & (x > -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            x = np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))
        x = np.where(there, x, -np.inf)
        top = x.max(axis=1, keepdims=True)
        e = np.where(there, np.exp(np.where(there, x - top, -np.inf)), 0.0)
    total = e.sum(axis=1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def route(logits, top_k, *, bias=None, n_groups=1, topk_groups=1, score="softmax",
          group_score="max", renormalize=True, scale=1.0):
    """(ids int32 [n][top_k], weights float64 [n][top_k]) of logits [n][E]."""
    l = clean_logits(logits)
    n, E = l.shape
    s = scores(logits, score)
    can = l > -np.inf
    summed = s
    choice = l
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        can = can & (b > -np.inf)          # False for NaN
        summed = choice = s + np.where(b > -np.inf, b, 0.0)
    choice = np.where(can, choice, -np.inf)
    if n_groups > 1:
        per = E // n_groups
        if group_score == "max":
            value = choice.reshape(n, n_groups, per).max(axis=2)
        else:
            v = np.sort(np.where(can, summed, -np.inf).reshape(n, n_groups, per), axis=2)[..., ::-1]
            second = v[..., 1] if per > 1 else np.full(v.shape[:2], -np.inf)
            value = v[..., 0] + np.where(second > -np.inf, second, 0.0)
        order = np.argsort(-value, axis=1, kind="stable")[:, :topk_groups]
        kept = np.zeros((n, n_groups), dtype=bool)
        np.put_along_axis(kept, order, True, axis=1)
        choice = np.where(np.repeat(kept, per, axis=1), choice, -np.inf)
    ids = np.argsort(-choice, axis=1, kind="stable")[:, :top_k]
    there = np.take_along_axis(choice, ids, axis=1) > -np.inf
    ids = np.where(there, ids, -1)
    if renormalize:
        w = pick_shares(logits, ids, score)
    else:
        w = np.where(there, np.take_along_axis(s, np.maximum(ids, 0), axis=1), 0.0)
    return ids.astype(np.int32), scale * w


def route_backward(logits, ids, grad_w, *, score="softmax", renormalize=True, scale=1.0):
    """Gradient [n][E] of the weights with respect to the logits."""
    l = clean_logits(logits)
    ids = np.asarray(ids)
    n, E = l.shape
    inside = (ids >= 0) & (ids < E)
    x = np.take_along_axis(l, np.where(inside, ids, 0), axis=1)
    there = inside & (x > -np.inf)
    g = np.where(there, scale * np.asarray(grad_w, dtype=np.float64), 0.0)
    s = scores(logits, score)
    dense = np.zeros((n, E))
    rows = np.broadcast_to(np.arange(n)[:, None], ids.shape)
    if score == "softmax" and not renormalize:
        np.add.at(dense, (rows[there], ids[there]), g[there])
        return s * (dense - (dense * s).sum(axis=1, keepdims=True))
    if renormalize:
        p = pick_shares(logits, ids, score)
        d = p * (g - (g * p).sum(axis=1, keepdims=True))
    else:
        d = g * np.take_along_axis(s, np.where(inside, ids, 0), axis=1)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            d = d / (1.0 + np.exp(np.where(there, x, 0.0)))
    np.add.at(dense, (rows[there], ids[there]), d[there])
    return dense


def unpack_w4(codes, codes_are) -> np.ndarray:
    """Code values [..][k] of bytes [..][k/2], even k in the low half."""
    c = np.asarray(codes, dtype=np.uint8)
    c = np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], -1).astype(np.int64)
    if codes_are == "int4":
        return c - 8.0
    return np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]


def weights_w4(codes, scales, codes_are) -> np.ndarray:
    """Weights [..][k] in float64; scales [..][k/group] as numbers."""
    v = unpack_w4(codes, codes_are)
    s = np.asarray(scales, dtype=np.float64)
    return v * np.repeat(s, v.shape[-1] // s.shape[-1], axis=-1)


def grouped_product(x, w, group_starts):
    """(y, a): y[m] = x[m] . w[e]^T for the rows of every group, and the same with
    absolute values, which bounds rounding errors.  x [M][k], w [E][n][k] float64."""
    M, n = x.shape[0], w.shape[1]
    y, a = np.zeros((M, n)), np.zeros((M, n))
    for e in range(w.shape[0]):
        lo, hi = int(group_starts[e]), int(group_starts[e + 1])
        if hi > lo:
            y[lo:hi] = x[lo:hi] @ w[e].T
            a[lo:hi] = np.abs(x[lo:hi]) @ np.abs(w[e]).T
    return y, a


def combine_backward(grad_out_bits, topk_w, picks, slot_bits, shape):
    """(grad_w, grad_rows, bound) for the local picks [M][3] of (rk, t, k), in row
    order, and the bf16 bits [M][N] of their slots; bound holds sum |grad_out * slot|
    at each pick's place."""
    g = bf16_to_f64(grad_out_bits)[picks[:, 0], picks[:, 1]]
    s = bf16_to_f64(slot_bits)
    grad_w, bound = np.zeros(shape), np.zeros(shape)
    at = (picks[:, 0], picks[:, 1], picks[:, 2])
    grad_w[at] = (g * s).sum(axis=1)
    bound[at] = np.abs(g * s).sum(axis=1)
    return grad_w, np.asarray(topk_w, dtype=np.float64)[at][:, None] * g, bound


def rms_norm(x, weight, *, residual=None, eps=1e-6):
    """(s, y) of rows [n][N]: s = x + residual, y = s w / sqrt(mean(s^2) + eps)."""
    s = np.asarray(x, dtype=np.float64)
    if residual is not None:
        s = s + np.asarray(residual, dtype=np.float64)
    rms = np.sqrt((s * s).mean(axis=-1, keepdims=True) + eps)
    return s, s / rms * np.asarray(weight, dtype=np.float64)


def rms_norm_backward(grad_out, sums, weight, *, grad_residual=None, eps=1e-6):
    """(ds [n][N], dw [N], bound_ds, bound_dw): the gradients of the sums and the weight,
    and the sums of the absolute values of the terms that make them."""
    g, r = np.asarray(grad_out, dtype=np.float64), np.asarray(sums, dtype=np.float64)
    w = np.asarray(weight, dtype=np.float64)
    inv = 1.0 / np.sqrt((r * r).mean(axis=-1, keepdims=True) + eps)
    gw = g * w
    ds = inv * (gw - r * inv ** 2 * (gw * r).mean(axis=-1, keepdims=True))
    bound = inv * (np.abs(gw) + np.abs(r) * inv ** 2 * np.abs(gw * r).mean(axis=-1, keepdims=True))
    if grad_residual is not None:
        q = np.asarray(grad_residual, dtype=np.float64)
        ds, bound = ds + q, bound + np.abs(q)
    each = g * r * inv
    return ds, each.sum(axis=0), bound, np.abs(each).sum(axis=0)


def moe_layer(x, w1, w2, ids, topk_w, expert_lo=0):
    """The layer of tokens x [n][hidden] through the experts w1 [E][2I][hidden], w2
    [E][hidden][I] that their picks ids [n][k] name: out[t] = sum over local picks of
    topk_w * w2 (silu(g) u).  Returns (out, bound): bound [n][hidden] is what rounding may
    move it by where the products are summed in binary32 and silu(g) u is rounded to
    bf16 or finer.  Each product of K terms: the matrix unit's additions are within 2^-23 of a
    partial sum each, and scales and joins add at most K / 16 + 32 operations of 2^-24."""
    x, topk_w = np.asarray(x, dtype=np.float64), np.asarray(topk_w, dtype=np.float64)
    out, bound = np.zeros_like(x), np.zeros_like(x)

    def steps(k):
        return k * 2.0 ** -23 + (k / 16 + 32) * 2.0 ** -24

    for t in range(x.shape[0]):
        total, size = np.zeros(x.shape[1]), np.zeros(x.shape[1])
        for k, i in enumerate(np.asarray(ids)[t]):
            e = int(i) - expert_lo
            if not 0 <= e < w1.shape[0]:
                continue
            I = w1.shape[1] // 2
            y, a = w1[e] @ x[t], np.abs(w1[e]) @ np.abs(x[t])
            g, u, b = y[:I], y[I:], steps(x.shape[1]) * a
            with np.errstate(over="ignore"):
                silu = g / (1.0 + np.exp(-g))
            h = silu * u
            dh = (1.1 * b[:I] * (np.abs(u) + b[I:]) + np.abs(silu) * b[I:] +
                  (2.0 ** -8 + 2.0 ** -20) * np.abs(h) + 1e-38)
            z = w2[e] @ h
            mag = np.abs(w2[e]) @ (np.abs(h) + dh)
            total += topk_w[t, k] * z
            size += np.abs(topk_w[t, k]) * mag
            bound[t] += np.abs(topk_w[t, k]) * (np.abs(w2[e]) @ dh + steps(I) * mag)
        out[t] = total
        bound[t] += 128 * 2.0 ** -24 * size
    return out, bound
