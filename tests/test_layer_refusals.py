"""Refusals of the norm and the few-token layer that need no GPU: null handles at the C
boundary, types, shapes and contradictions in the plumbing, and the limits of a handle."""
import ctypes
import os

import pytest
import torch

from grouped_gemm_scatter_amd import PackedW4
from grouped_gemm_scatter_amd import binding as B
from grouped_gemm_scatter_amd.context import EpCombine


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from grouped_gemm_scatter_amd.build import build
        build(jobs=4)
    return B.load_library()


def test_null_handles_are_rejected(lib):
    p = ctypes.byref(B.make_norm_params(dtype=torch.bfloat16))
    assert lib.ep_rms_norm(None, p, None, None, None, 0, None, None, None, None,
                           None) == B.EP_ERR_INVALID_ARG
    assert lib.ep_rms_norm_backward(None, p, None, None, None, None, 0, None, None, None, None, 0,
                                    None) == B.EP_ERR_INVALID_ARG
    assert lib.ep_rms_norm_backward_workspace(None, 1) == B.EP_ERR_INVALID_ARG
    assert lib.ep_moe_layer(None, None, None, None, None, None, None, None, None, None, None, 0,
                            None, None, 0, None) == B.EP_ERR_INVALID_ARG
    assert lib.ep_moe_layer_workspace(None, 1) == B.EP_ERR_INVALID_ARG


def test_types():
    for bad in (dict(dtype=torch.float64), dict(dtype=torch.float32, weight_dtype=torch.int32),
                dict(dtype=torch.bfloat16, residual_dtype=torch.float64)):
        with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
            B.make_norm_params(**bad)
    for bad in (dict(dtype=torch.bfloat16, residual_dtype=torch.float16),
                dict(dtype=torch.float32, weight_dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="or float32"):
            B.make_norm_params(**bad)


def _ctx(**over):
    ctx = EpCombine.__new__(EpCombine)       # no device: the checks come before it is used
    ctx._device_index = 0
    ctx.n_experts_per_device, ctx.n_ranks, ctx.top_k = 2, 1, 2
    ctx.hidden_n, ctx.hidden_k, ctx.dtype = 128, 128, "bf16"
    for k, v in over.items():
        setattr(ctx, k, v)
    return ctx


def test_norm_shapes_and_contradictions():
    ctx = _ctx()
    x = torch.zeros(1, 3, 128, dtype=torch.bfloat16)
    w = torch.zeros(128)
    for call, message in (
            (lambda: ctx.rms_norm(x[..., :64], w), "x must be"),
            (lambda: ctx.rms_norm(x, w), "handle's device"),
            (lambda: ctx.rms_norm(x, w.double()), "float32, bfloat16 or float16"),
            (lambda: ctx.rms_norm(x, w, residual=x.half()), "residual must be"),
            (lambda: ctx.rms_norm_backward(x, x.half(), w), "residual must be"),
            (lambda: ctx.rms_norm_backward(x[:, :, 1:], x, w), "grad_out must be")):
        with pytest.raises(ValueError, match=message):
            call()


def test_layer_shapes_and_contradictions():
    x = torch.zeros(1, 3, 128, dtype=torch.bfloat16)
    ids, tw = torch.zeros(1, 3, 2, dtype=torch.int32), torch.zeros(1, 3, 2)
    for call, message in (
            (lambda: _ctx().moe_layer(x[..., :64], x, x, ids, tw), "x must be"),
            (lambda: _ctx().moe_layer(x.half(), x, x, ids, tw), "x must be"),
            (lambda: _ctx(dtype="fp8").moe_layer(x, x, x, ids, tw), "x must be torch.uint8"),
            (lambda: _ctx().moe_layer(x, x, x, ids, tw), "handle's device")):
        with pytest.raises(ValueError, match=message):
            call()


def test_one_stack_of_4_bits_beside_one_of_16_is_refused():
    ctx = _ctx()
    ctx._shape = lambda *a: 4096              # as if the rows and picks were on the device
    fmt = B.make_w4_format(codes=0, group=32, scale_dtype=torch.bfloat16)
    w = PackedW4(torch.zeros(2, 256, 64, dtype=torch.uint8),
                 torch.zeros(2, 256, 4, dtype=torch.bfloat16), 256, 128, fmt)
    x = torch.zeros(1, 3, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="pack_weights_w4"):
        ctx.moe_layer(x, w, x, x, x)
    with pytest.raises(ValueError, match="pack_weights_w4"):
        ctx.moe_layer(x, x, w, x, x)


def test_limits_are_those_of_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "ep_combine.h")).read()
    for name in ("EP_MOE_MAX_TOKENS", "EP_MOE_MAX_PICKS", "EP_ROWS_F32", "EP_ROWS_BF16",
                 "EP_ROWS_F16"):
        assert f"#define {name} {getattr(B, name)}\n" in text
