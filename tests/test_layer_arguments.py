"""Arguments of the norm, the routing and the few-token layer that need no GPU: what reaches
the C boundary, and refusals in the plumbing."""
import numpy as np
import pytest
import torch

from grouped_gemm_scatter_amd import binding as B
from grouped_gemm_scatter_amd.context import EpCombine


@pytest.fixture
def ctx(monkeypatch):
    """A context without a device whose calls end at the C boundary; `sent` holds the options
    that arrived there, copied."""
    c = EpCombine.__new__(EpCombine)
    c._device_index, c.handle, c._workspaces = 0, None, {}
    c.n_experts_per_device, c.n_ranks, c.top_k = 2, 1, 2
    c.hidden_n, c.hidden_k, c.dtype = 128, 128, "bf16"
    c.sent = []
    c._shape = lambda t, *a: 4096             # as if every tensor were on the device
    c._empty = lambda shape, dtype, stream: torch.empty(shape, dtype=dtype)
    for name in ("ep_rms_norm", "ep_rms_norm_backward", "ep_route_topk", "ep_route_topk_backward"):
        monkeypatch.setattr(B, name, lambda h, p, *a: c.sent.append(type(p).from_buffer_copy(p)))
    monkeypatch.setattr(B, "ep_rms_norm_backward_workspace", lambda h, t: 0)
    return c


def test_options_in_tensors_are_read_at_every_call(ctx):
    """A number in a tensor that changes between two calls: each call has the value of its
    time."""
    x, w = torch.zeros(1, 3, 128), torch.zeros(128)
    ids = torch.zeros(1, 3, 2, dtype=torch.int32)
    number = torch.tensor(0.25)
    calls = (("eps", lambda: ctx.rms_norm(x, w, eps=number)),
             ("eps", lambda: ctx.rms_norm_backward(x, x, w, eps=number)),
             ("scale", lambda: ctx.route(x, scale=number)),
             ("scale", lambda: ctx.route_backward(x, ids, x, scale=number)))
    for field, call in calls:
        for value in (0.25, 0.5, 2.0):
            number.fill_(value)
            call()
            assert getattr(ctx.sent[-1], field) == value
    groups, flag = torch.tensor(1), torch.tensor(True)
    for n, f in ((1, True), (4, False), (2, True)):
        groups.fill_(n)
        flag.fill_(f)
        ctx.route(x, n_groups=groups, topk_groups=groups, renormalize=flag)
        got = ctx.sent[-1]
        assert (got.n_groups, got.topk_groups, bool(got.renormalize)) == (n, n, f)


def test_options_of_any_number_type(ctx):
    x, w = torch.zeros(1, 3, 128), torch.zeros(128)
    for eps in (0, 1, 0.5, np.float32(0.5), np.float64(0.5), np.array(0.5)):
        ctx.rms_norm(x, w, eps=eps)
        assert ctx.sent[-1].eps == float(eps)
    for bad in (1.5, "2"):
        with pytest.raises(TypeError):
            ctx.route(x, n_groups=bad)


@pytest.mark.parametrize("shape", [(), (128,), (3, 128), (1, 1, 3, 128)])
def test_rows_of_other_than_three_dimensions(ctx, shape):
    t = torch.zeros(shape, dtype=torch.bfloat16)
    w, ids = torch.zeros(128), torch.zeros(1, 3, 2, dtype=torch.int32)
    for call, name in ((lambda: ctx.rms_norm(t, w), "x"),
                       (lambda: ctx.rms_norm_backward(t, t, w), "grad_out"),
                       (lambda: ctx.moe_layer(t, t, t, ids, w), "x"),
                       (lambda: ctx.combine_backward(t, ids, w, None, None, 0), "grad_out")):
        with pytest.raises(ValueError, match=rf"{name} must be \[1\]\[T\]\[128\]"):
            call()
