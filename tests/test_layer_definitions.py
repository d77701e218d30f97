"""Pins of the norm's and the few-token layer's definitions in oracle/operators.py: loops
over single numbers, differences and torch's gradients."""
import math

import numpy as np
import pytest
import torch

from oracle import operators as P


@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_is_the_definition(with_residual):
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((3, 8)), rng.standard_normal(8)
    res = rng.standard_normal((3, 8)) if with_residual else None
    s, y = P.rms_norm(x, w, residual=res, eps=0.01)
    for r in range(3):
        row = [x[r, i] + (res[r, i] if with_residual else 0.0) for i in range(8)]
        mean = math.fsum(v * v for v in row) / 8
        for i in range(8):
            assert s[r, i] == row[i]
            assert math.isclose(y[r, i], row[i] / math.sqrt(mean + 0.01) * w[i], rel_tol=1e-14)
    assert np.all(P.rms_norm(np.zeros((1, 8)), w)[1] == 0)


@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_gradient_is_that_of_differences_and_of_torch(with_residual):
    rng = np.random.default_rng(2)
    r, g, w = rng.standard_normal((4, 6)), rng.standard_normal((4, 6)), rng.standard_normal(6)
    q = rng.standard_normal((4, 6)) if with_residual else None
    ds, dw, bs, bw = P.rms_norm_backward(g, r, w, grad_residual=q, eps=0.03)

    def loss(r, w):
        s, y = P.rms_norm(r, w, eps=0.03)
        return (g * y).sum() + ((q * s).sum() if with_residual else 0.0)

    eps = 1e-6
    for i in np.ndindex(r.shape):
        up, down = r.copy(), r.copy()
        up[i] += eps
        down[i] -= eps
        assert abs(ds[i] - (loss(up, w) - loss(down, w)) / (2 * eps)) < 1e-7
    for i in range(6):
        up, down = w.copy(), w.copy()
        up[i] += eps
        down[i] -= eps
        assert abs(dw[i] - (loss(r, up) - loss(r, down)) / (2 * eps)) < 1e-7
    tr, tw = torch.tensor(r, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = tr * torch.rsqrt(tr.square().mean(-1, keepdim=True) + 0.03) * tw
    total = (y * torch.tensor(g)).sum()
    if with_residual:
        total = total + (tr * torch.tensor(q)).sum()
    total.backward()
    np.testing.assert_allclose(ds, tr.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-12)
    assert np.all(bs >= np.abs(ds) - 1e-12) and np.all(bw >= np.abs(dw) - 1e-12)


def test_layer_is_the_definition():
    rng = np.random.default_rng(3)
    E, N, I, k = 3, 5, 4, 3
    w1, w2 = rng.standard_normal((E, 2 * I, N)), rng.standard_normal((E, N, I))
    x = rng.standard_normal((4, N))
    # a dropped pick, experts below and above the local ones, one expert twice, none at all
    ids = np.array([[10, 12, -1], [9, 13, 11], [11, 11, 10], [0, 13, -1]])
    tw = rng.random((4, k))
    out, bound = P.moe_layer(x, w1, w2, ids, tw, expert_lo=10)
    for t in range(4):
        for n in range(N):
            v = 0.0
            for j in range(k):
                e = ids[t, j] - 10
                if e not in (0, 1, 2):
                    continue
                for i in range(I):
                    g = math.fsum(w1[e, i, c] * x[t, c] for c in range(N))
                    u = math.fsum(w1[e, I + i, c] * x[t, c] for c in range(N))
                    v += tw[t, j] * w2[e, n, i] * g / (1 + math.exp(-g)) * u
            assert math.isclose(out[t, n], v, rel_tol=1e-12, abs_tol=1e-14)
    assert np.all(out[3] == 0) and np.all(bound[3] == 0)
    assert np.all(bound[:3] > 0) and np.all(bound < 0.1 * (1 + np.abs(out)))
