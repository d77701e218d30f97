"""The measures of tests/layer_bounds.py themselves: they hold for the definitions, computed
in binary32 and rounded as the kernels round, and no planted mistake meets them."""
import numpy as np
import pytest

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
