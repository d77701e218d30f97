"""Pins of oracle/operators.py: the router, its gradient, the 4-bit weights and the
gradient of the combine against loops over single numbers, differences and torch."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from oracle import operators as P


def _brute_route(l, top_k, bias, n_groups, topk_groups, score, group_score, renormalize, scale):
    """One token, one number at a time, on finite or -inf logits."""
    E = len(l)
    here = [i for i in range(E) if l[i] > -math.inf]
    if score == "sigmoid":
        s = {i: 1 / (1 + math.exp(-l[i])) for i in here}
    else:
        z = math.fsum(math.exp(l[i]) for i in here)
        s = {i: math.exp(l[i]) / z for i in here}
    can = [i for i in here if bias is None or bias[i] > -math.inf]
    choice = {i: l[i] if bias is None else s[i] + bias[i] for i in can}
    per = E // n_groups
    value = []
    for g in range(n_groups):
        mine = [i for i in can if i // per == g]
        if not mine:
            continue
        if group_score == "max":
            v = max(choice[i] for i in mine)
        else:
            v = sum(sorted((s[i] + (0 if bias is None else bias[i]) for i in mine))[-2:])
        value.append((-v, g))
    kept = {g for _, g in sorted(value)[:topk_groups]} if n_groups > 1 else {0}
    order = sorted((i for i in can if i // per in kept), key=lambda i: (-choice[i], i))[:top_k]
    total = sum(s[i] for i in order) if renormalize else 1.0
    ids = order + [-1] * (top_k - len(order))
    return ids, [scale * s[i] / total if i >= 0 else 0.0 for i in ids]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_is_the_definition(score, group_score, with_bias, renormalize):
    rng = np.random.default_rng(3)
    for E, G, kept, k in ((12, 1, 1, 4), (12, 4, 2, 5), (8, 8, 3, 3), (6, 2, 1, 6)):
        l = rng.standard_normal((20, E))
        l[rng.random(l.shape) < 0.3] = -np.inf
        l[0] = -np.inf
        l[1] = 0.5                                   # all equal: lowest indices
        bias = np.round(rng.standard_normal(E), 1) if with_bias else None
        if with_bias:
            bias[1] = -np.inf
        ids, w = P.route(l, k, bias=bias, n_groups=G, topk_groups=kept, score=score,
                         group_score=group_score, renormalize=renormalize, scale=2.0)
        for r in range(l.shape[0]):
            want_ids, want_w = _brute_route(list(l[r]), k, bias, G, kept, score, group_score,
                                            renormalize, 2.0)
            assert list(ids[r]) == want_ids
            np.testing.assert_allclose(w[r], want_w, rtol=1e-12)


def test_route_special_logits():
    l = np.array([[np.nan, np.inf, 1.0, np.inf, -np.inf]])
    ids, w = P.route(l, 3, score="softmax")
    assert list(ids[0]) == [1, 3, 2] and list(w[0]) == [0.5, 0.5, 0.0]
    ids, w = P.route(np.full((1, 4), -1000.0), 2, score="sigmoid")
    assert list(ids[0]) == [0, 1] and np.allclose(w, 0.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_is_that_of_differences_and_of_torch(score, renormalize):
    rng = np.random.default_rng(4)
    l = rng.standard_normal((7, 10))
    l[:, 3] = -np.inf
    ids, _ = P.route(l, 4, score=score, renormalize=renormalize)
    ids[2, 3] = -1
    g = rng.standard_normal(ids.shape)
    d = P.route_backward(l, ids, g, score=score, renormalize=renormalize, scale=1.5)

    def loss(x):
        if renormalize:
            w = P.pick_shares(x, ids, score)
        else:
            w = np.where(ids >= 0, np.take_along_axis(P.scores(x, score), np.maximum(ids, 0), 1), 0)
        return 1.5 * (g * w).sum(axis=1)

    eps = 1e-6
    for i in range(l.shape[1]):
        up, down = l.copy(), l.copy()
        up[:, i] += eps
        down[:, i] -= eps
        np.testing.assert_allclose(d[:, i], (loss(up) - loss(down)) / (2 * eps), atol=1e-8)

    x = torch.tensor(l, requires_grad=True)
    s = torch.softmax(x, -1) if score == "softmax" else torch.sigmoid(x)
    keep = torch.tensor(ids >= 0)
    w = torch.gather(s, 1, torch.tensor(np.maximum(ids, 0)).long()) * keep
    if renormalize:
        w = w / w.sum(-1, keepdim=True)
    (1.5 * w * torch.tensor(g)).sum().backward()
    np.testing.assert_allclose(d, np.nan_to_num(x.grad.numpy()), atol=1e-12)


def test_route_gradient_adds_equal_picks_and_drops_bad_ones():
    l = np.array([[0.1, 0.7, -0.3]])
    ids = np.array([[1, 1, 7, -5]])
    d = P.route_backward(l, ids, np.array([[1.0, 2.0, 4.0, 8.0]]), score="sigmoid",
                         renormalize=False)
    s = 1 / (1 + math.exp(-0.7))
    np.testing.assert_allclose(d, [[0.0, 3 * s * (1 - s), 0.0]])


def test_weights_in_4_bits():
    codes = np.arange(256, dtype=np.uint8)[None]
    v = P.unpack_w4(codes, "int4").reshape(256, 2)
    assert all(tuple(v[b]) == ((b & 15) - 8, (b >> 4) - 8) for b in range(256))
    e = P.unpack_w4(codes, "e2m1").reshape(256, 2)

    def e2m1(c):
        exponent, mantissa = c >> 1 & 3, c & 1
        m = mantissa * 0.5 if exponent == 0 else (1 + 0.5 * mantissa) * 2.0 ** (exponent - 1)
        return -m if c & 8 else m

    assert all(tuple(e[b]) == (e2m1(b & 15), e2m1(b >> 4)) for b in range(256))
    w = P.weights_w4(np.full((1, 32), 0x9A, np.uint8), np.array([[2.0, 3.0]]), "int4")
    assert list(w[0, :4]) == [4.0, 2.0, 4.0, 2.0] and list(w[0, 32:34]) == [6.0, 3.0]


def test_combine_gradient_is_that_of_torch():
    rng = np.random.default_rng(5)
    R, T, k, N, lo, El = 2, 5, 3, 8, 2, 2
    ids = np.stack([[rng.choice(6, k, replace=False) for _ in range(T)] for _ in range(R)])
    w = rng.random((R, T, k))
    off, src = O.group_local_picks(ids, El, 1)
    picks = O.row_picks(off, src, R)
    y = O.f64_to_bf16(rng.standard_normal((len(picks), N)))
    go = O.f64_to_bf16(rng.standard_normal((R, T, N)))
    gw, gr, bound = P.combine_backward(go, w, picks, y, (R, T, k))
    tw = torch.tensor(w, requires_grad=True)
    ty = torch.tensor(O.bf16_to_f64(y), requires_grad=True)
    out = torch.zeros(R, T, N, dtype=torch.float64)
    for m, (rk, t, kk) in enumerate(picks):
        assert lo <= ids[rk, t, kk] < lo + El
        out[rk, t] = out[rk, t] + tw[rk, t, kk] * ty[m]
    (out * torch.tensor(O.bf16_to_f64(go))).sum().backward()
    np.testing.assert_allclose(gw, tw.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(gr, ty.grad.numpy(), atol=1e-12)
    assert np.all(bound >= np.abs(gw) - 1e-12)
