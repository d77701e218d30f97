"""The measures of tests/layer_bounds.py themselves: they hold for the definitions, computed
in binary32 and rounded as the kernels round, and no planted mistake meets them."""
import numpy as np
import pytest
import torch

import layer_bounds as L
from oracle import operators as P


def _norm32(w, eps):
    """The definition in binary32."""
    def norm(x):
        x = x.astype(np.float32)
        inv = 1 / np.sqrt((x * x).mean(-1, keepdims=True, dtype=np.float32) + np.float32(eps))
        return (x * inv * w.astype(np.float32)).astype(np.float64)
    return norm


@pytest.mark.parametrize("eps", [1e-6, 0.25])
@pytest.mark.parametrize("N", [128, 2176])
def test_gradients_along_the_rows(N, eps):
    def gradient(g, r, *, part=1.0, of=eps, mean=True):
        gw = g * w
        inv = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + of)
        dot = (gw * r).mean(-1, keepdims=True) * (1 if mean else N)
        return inv * (gw - part * r * inv ** 2 * dot)

    for seed in range(20):
        r, w, g = L.gradient_inputs(4, N, seed)
        args = (r, w, g, eps)
        err, tol = L.along_rows(_norm32(w, eps),
                                lambda g, r: P.rms_norm_backward(g, r, w, eps=eps)[0], *args)
        assert err <= tol
        # without its second term, with half of it, with a sum in place of the mean, with
        # another eps, with the other sign
        for wrong in (dict(part=0.0), dict(part=0.5), dict(mean=False), dict(part=-1.0),
                      dict(part=1.01)) + ((dict(of=1e-6),) if eps > 0.1 else ()):
            err, tol = L.along_rows(_norm32(w, eps), lambda g, r: gradient(g, r, **wrong), *args)
            assert err > 2 * tol, wrong


class Planted:
    """The layer at the size of a large model, as the kernels round it, with a mistake."""
    hidden, inter, experts, tokens, k = 7168, 2048, 3, 2, 2

    def __init__(self):
        g = torch.Generator().manual_seed(1)
        self.w1 = torch.randn(self.experts, 2 * self.inter, self.hidden, generator=g)
        self.w2 = torch.randn(self.experts, self.hidden, self.inter, generator=g)
        self.w1 *= self.hidden ** -0.5
        self.w2 *= self.inter ** -0.5
        self.x = torch.randn(self.tokens, self.hidden, generator=g).double()
        self.ids = torch.tensor([[2, 0], [1, 2]])
        # weights as a router's softmax gives them, the smaller one a tenth
        self.topk_w = torch.tensor([[0.9, 0.1], [0.6, 0.4]])
        self.want, self.spread = L.layer(self.x, self.w1, self.w2, self.ids, self.topk_w)

    def out(self, *, up=None, down=None, swap=False, ids=None, topk_w=None, columns=None,
            parts=2):
        """up, down: slices of k that the products leave out; parts: of bf16 that a hidden
        value is held in."""
        ids = self.ids if ids is None else ids
        topk_w = self.topk_w if topk_w is None else topk_w
        out = torch.zeros_like(self.x)
        for t in range(self.tokens):
            for j in range(self.k):
                e, x = int(ids[t, j]), self.x[t].clone()
                if up is not None and j == 0:
                    x[up] = 0
                y = self.w1[e].double() @ x
                gate, up_ = y[:self.inter], y[self.inter:]
                if swap:
                    gate, up_ = up_, gate
                exact = gate / (1 + torch.exp(-gate)) * up_
                h = exact.bfloat16().double()
                if parts == 2:
                    h += (exact - h).bfloat16().double()
                if down is not None and j == 0:
                    h[down] = 0
                out[t] += topk_w[t, j] * (self.w2[e].double() @ h)
        if columns is not None:
            out[0, columns] = 0
        return out.bfloat16()

    def error(self, got):
        return L.layer_error(got, self.want, self.spread)


@pytest.fixture(scope="module")
def planted():
    return Planted()


def test_the_layer_as_it_is_meets_its_bound(planted):
    assert planted.error(planted.out()) <= 1


@pytest.mark.parametrize("mistake", [
    dict(up=slice(640, 768)), dict(up=slice(7136, 7168)), dict(down=slice(1920, 2048)),
    dict(down=slice(32, 64)), dict(parts=1), dict(swap=True), dict(columns=slice(7152, 7168)),
    dict(columns=slice(16, 17)), dict(ids=torch.tensor([[1, 0], [1, 2]])),
    dict(ids=torch.tensor([[2, 1], [1, 2]])), dict(topk_w=torch.tensor([[0.9, 0.0], [0.6, 0.4]])),
    dict(topk_w=torch.tensor([[0.9, 0.1], [0.4, 0.6]])),
    dict(topk_w=torch.tensor([[0.9, 0.1], [0.6, 0.42]]))], ids=str)
def test_no_planted_mistake_meets_the_layers_bound(planted, mistake):
    assert planted.error(planted.out(**mistake)) > 1.5


def test_zeros_and_another_tokens_rows_do_not_meet_it(planted):
    got = planted.out()
    assert planted.error(torch.zeros_like(got)) > 10
    assert planted.error(got.flip(0)) > 10
