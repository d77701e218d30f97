"""Refusals of the routing, 4-bit weight and combine-gradient calls that need no GPU: null
handles at the C boundary, unknown names and types in the plumbing."""
import ctypes
import os

import pytest
import torch

from grouped_gemm_scatter_amd import PackedW4
from grouped_gemm_scatter_amd import binding as B
from grouped_gemm_scatter_amd.context import EpCombine, _choice


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from grouped_gemm_scatter_amd.build import build
        build(jobs=4)
    return B.load_library()


def test_null_handles_are_rejected(lib):
    p = ctypes.byref(B.make_route_params(n_experts=8, logits_dtype=torch.float32))
    f = ctypes.byref(B.make_w4_format(codes=B.EP_W4_INT4, group=32, scale_dtype=torch.bfloat16))
    assert lib.ep_route_topk(None, p, None, None, 0, None, None, None) == B.EP_ERR_INVALID_ARG
    assert lib.ep_route_topk_backward(None, p, None, None, None, 0, None,
                                      None) == B.EP_ERR_INVALID_ARG
    assert lib.ep_combine_backward(None, None, None, None, 0, None, None, 0, None, None,
                                   None) == B.EP_ERR_INVALID_ARG
    assert lib.ep_pack_weights_w4(None, f, None, None, 16, 128, None, None,
                                  None) == B.EP_ERR_INVALID_ARG
    assert lib.ep_grouped_gemm_swiglu_w4(None, f, None, None, None, None, 0, None,
                                         None) == B.EP_ERR_INVALID_ARG
    assert lib.ep_grouped_gemm_scatter_w4(None, f, None, None, None, None, None, 0, 0, None, 1,
                                          None) == B.EP_ERR_INVALID_ARG


def test_types_and_names():
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        B.make_route_params(n_experts=8, logits_dtype=torch.float64)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        B.make_w4_format(codes=0, group=32, scale_dtype=torch.float32)
    with pytest.raises(ValueError, match="score must be one of"):
        _choice({"softmax": 0}, "tanh", "score")


def test_shapes_and_devices():
    t = torch.zeros(2, 3, 4)
    ctx = EpCombine.__new__(EpCombine)       # no device: the checks come before it is used
    ctx._device_index = 0
    for args, message in (((t, "x", (2, 3, 5), torch.float32), "must be"),
                          ((t, "x", (2, 3, 4), torch.int32), "must be torch.int32"),
                          ((t, "x", (2, 3, 4), torch.float32), "handle's device")):
        with pytest.raises(ValueError, match=message):
            ctx._shape(*args)


def test_packed_weights_of_another_shape():
    ctx = EpCombine.__new__(EpCombine)
    ctx.n_experts_per_device = 2
    fmt = B.make_w4_format(codes=0, group=32, scale_dtype=torch.bfloat16)
    w = PackedW4(torch.zeros(2, 16, 64, dtype=torch.uint8), torch.zeros(2, 16, 4), 16, 128, fmt)
    ctx._need_w4(w, 16, 128)
    for rows, k in ((32, 128), (16, 256)):
        with pytest.raises(ValueError, match="packed weights"):
            ctx._need_w4(w, rows, k)
    ctx.n_experts_per_device = 3
    with pytest.raises(ValueError, match="packed weights"):
        ctx._need_w4(w, 16, 128)
    with pytest.raises(ValueError, match="pack_weights_w4"):
        ctx._need_w4(torch.zeros(4), 16, 128)


def test_packed_weights_that_are_not_what_their_format_says():
    """A stack put together by hand: too few codes or scales, scales of the other type, or on
    another device, before anything is launched."""
    ctx = EpCombine.__new__(EpCombine)       # no device: the checks come before it is used
    ctx._device_index = 0
    ctx.n_experts_per_device, ctx.n_ranks = 2, 1
    ctx.hidden_n, ctx.hidden_k = 128, 128
    fmt = B.make_w4_format(codes=0, group=32, scale_dtype=torch.bfloat16)
    calls = ((256, lambda w: ctx.up_swiglu_w4(4096, w, 4096, 1, 4096)),
             (128, lambda w: ctx.gemm_scatter_w4(4096, w, 4096, 4096, 1, epoch=1)))
    for rows, call in calls:
        codes = torch.zeros(2, rows, 64, dtype=torch.uint8)
        scales = torch.zeros(2, rows, 4, dtype=torch.bfloat16)
        for c, s, message in ((codes[:, :, :63], scales, "codes: .* at least"),
                              (codes, scales, "codes must be on the handle's device"),
                              (codes.char(), scales, "codes must be torch.uint8"),
                              (codes, scales.half(), "scales must be torch.bfloat16"),
                              (codes, scales[:, :, :2], "scales: .* at least")):
            with pytest.raises(ValueError, match=message):
                call(PackedW4(c, s, rows, 128, fmt))


def _init(lib, **over):
    kw = dict(n_ranks=1, my_rank=0, top_k=2, max_tokens_per_rank=8, n_experts_per_device=1,
              hidden_k=64, hidden_n=128)
    kw.update(over)
    b = B.EpCombineBuffers()
    b.recv_buf[0] = 4096
    b.recv_count = b.rank_counter = b.tile_counter = b.error_word = 1 << 20
    h = ctypes.c_void_p()
    rc = lib.ep_combine_init(ctypes.byref(B.make_params(msg_bytes=2 * kw["hidden_n"], **kw)),
                             ctypes.byref(b), ctypes.byref(h))
    lib.ep_combine_destroy(h)
    return rc


@pytest.mark.parametrize("over", [dict(n_experts_per_device=256, hidden_k=2048, hidden_n=4096),
                                  dict(n_experts_per_device=256, hidden_k=2048, hidden_n=7168)])
def test_handles_of_stacks_that_only_4_bits_hold(lib, over):
    """4 GiB and more in 2-byte weights (without a GPU the call ends at the device's)."""
    assert _init(lib, **over) in (B.EP_OK, B.EP_ERR_HIP)


def test_one_expert_past_four_gib_is_refused(lib):
    assert _init(lib, hidden_k=1 << 24) == B.EP_ERR_UNSUPPORTED
    assert _init(lib, hidden_k=(1 << 24) - 64) in (B.EP_OK, B.EP_ERR_HIP)
