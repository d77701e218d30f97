"""The norm's gradient against differences of the norm's own outputs, along the rows, where
its two terms nearly cancel (tests/layer_bounds.py; tests/test_layer_bounds.py shows that a
gradient without the second term, or with another amount of it, does not meet the bound)."""
import numpy as np
import pytest
import torch

import layer_bounds as L
from ep_synth import TINY
from gpu_helpers import make_ctx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-6, 0.25])
@pytest.mark.parametrize("N", [128, 384, 2176, 8320, 17408])
def test_gradient_along_the_rows(N, eps):
    print(f"[case] differences N={N} eps={eps}", flush=True)
    r, w, g = L.gradient_inputs(6, N, N)
    ctx = make_ctx(TINY.replace(n_ranks=2, tokens_per_rank=3, n=N))
    dev = lambda a: torch.from_numpy(a.astype(np.float32)).cuda().view(2, 3, N)  # noqa: E731
    weight = torch.from_numpy(w.astype(np.float32)).cuda()
    host = lambda t: t.double().cpu().numpy().reshape(6, N)  # noqa: E731
    norm = lambda x: host(ctx.rms_norm(dev(x), weight, eps=eps).out)  # noqa: E731
    for wide in (False, True):
        # alone, and with another gradient that is added to it
        q = torch.full((2, 3, N), 0.5, device="cuda") if wide else None

        def gradient(g, r):
            return host(ctx.rms_norm_backward(dev(g), dev(r), weight, grad_residual=q, eps=eps).x)
        err, tol = L.along_rows(norm, lambda g, r: gradient(g, r) - (0.5 if wide else 0.0),
                                r, w, g, eps)
        # that addition rounds each value once more
        tol += 2.0 ** -24 * (np.abs(r) * np.abs(gradient(g, r))).sum() if wide else 0.0
        assert err <= tol
