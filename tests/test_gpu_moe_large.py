"""The layer for a few tokens at the sizes of large models, in every kind of weights, within
an error that no dropped step, expert, pick or column meets (tests/layer_bounds.py,
tests/test_layer_bounds.py)."""
import pytest
import torch

import layer_bounds as L
from grouped_gemm_scatter_amd import EpCombine

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "bf16_sliced", "fp8", ("int4", 128, torch.float16), ("int4", 32, torch.bfloat16),
           ("e2m1", 32, torch.bfloat16), ("e2m1", 64, torch.float16)]
E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


def _id(f):
    return f if isinstance(f, str) else "-".join(map(str, f)).replace("torch.", "")


class Stack:
    """One product's weights [E][n][k] of size 1 / sqrt(k), as the library takes them (w,
    scale); [e]: an expert's values in float64."""

    def __init__(self, ctx, fmt, E, n, k, g, sliced):
        self.fmt, self.scale, self.shape = fmt, None, (n, k)
        size = k ** -0.5
        if fmt == "fp8":
            v = torch.randn(E, n, k, generator=g, device="cuda").mul_(100).clamp_(-448, 448)
            self.codes = v.to(torch.float8_e4m3fn)
            self.scale = size / 100 * (0.75 + 0.5 * torch.rand(E, n // 128, k // 128, generator=g,
                                                               device="cuda"))
            self.w = self.codes.view(torch.uint8)
        elif isinstance(fmt, str):
            self.codes = (torch.randn(E, n, k, generator=g, device="cuda") * size).bfloat16()
            self.w = ctx.pack_weights(self.codes) if sliced else self.codes
        else:
            kind, group, scale_type = fmt
            self.codes = torch.randint(0, 256, (E, n, k // 2), generator=g, device="cuda",
                                       dtype=torch.uint8)
            self.scales = (size / 4 * (0.75 + 0.5 * torch.rand(
                E, n, k // group, generator=g, device="cuda"))).to(scale_type)
            self.w = ctx.pack_weights_w4(self.codes, self.scales, codes=kind)

    def __len__(self):
        return len(self.codes)

    def __getitem__(self, e):
        c = self.codes[e]
        if self.fmt == "fp8":
            s = self.scale[e].double()
            return c.double() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)
        if isinstance(self.fmt, str):
            return c.double()
        values = torch.tensor(E2M1 if self.fmt[0] == "e2m1" else list(range(-8, 8)),
                              dtype=torch.float64, device="cuda")
        v = torch.stack([values[(c & 15).long()], values[(c >> 4).long()]], -1).view(self.shape)
        return v * self.scales[e].double().repeat_interleave(self.fmt[1], 1)


class Layer:
    def __init__(self, fmt, E, hidden, inter, T, k, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.fp8, self.shape, self.T, self.k = fmt == "fp8", (1, T, hidden), T, k
        sliced = fmt == "bf16_sliced"
        self.ctx = EpCombine(n_ranks=1, top_k=k, max_tokens_per_rank=T, n_experts_per_device=E,
                             hidden_k=inter, hidden_n=hidden, w_slice_major=sliced,
                             dtype="fp8" if self.fp8 else "bf16")
        self.w1 = Stack(self.ctx, fmt, E, 2 * inter, hidden, self.g, False)
        self.w2 = Stack(self.ctx, fmt, E, hidden, inter, self.g, sliced)

    def check(self, ids):
        x = torch.randn(self.shape, generator=self.g, device="cuda")
        tw = torch.softmax(torch.randn(1, self.T, self.k, generator=self.g, device="cuda"), -1)
        more = {}
        if self.fp8:
            # codes and scales as the norm makes them
            ones = torch.ones(self.shape[-1], device="cuda")
            y = self.ctx.rms_norm(x, ones, rows=False, fp8=True)
            more = dict(x_scale=y.scales, w1_scale=self.w1.scale, w2_scale=self.w2.scale)
            rows = y.codes
            x = (y.codes.view(torch.float8_e4m3fn).double() *
                 y.scales.double().repeat_interleave(128, -1))
        else:
            rows = x.bfloat16()
            x = rows.double()
        got = self.ctx.moe_layer(rows, self.w1.w, self.w2.w, ids, tw, **more)
        want, spread = L.layer(x[0], self.w1, self.w2, ids[0], tw[0].double())
        error = L.layer_error(got[0], want, spread)
        assert error <= 1, error
        assert self.ctx.query_error() == 0


# pairs an expert: up to 3, about 8, about 16 (both sides of the borders between the paths),
# 64
@pytest.mark.parametrize("E,T,k", [(4, 3, 3), (3, 12, 2), (2, 32, 1), (2, 64, 2)])
@pytest.mark.parametrize("fmt", FORMATS, ids=_id)
def test_seven_thousand_by_two_thousand(fmt, E, T, k):
    print(f"[case] large layer {_id(fmt)} E={E} T={T} k={k}", flush=True)
    layer = Layer(fmt, E, 7168, 2048, T, k)
    for _ in range(2):
        ids = torch.stack([torch.randperm(E)[:k] for _ in range(T)])[None].int().cuda()
        if T == 3:
            ids[0, 1, 2] = -1
        layer.check(ids)


@pytest.mark.parametrize("fmt", FORMATS, ids=_id)
def test_many_experts_of_a_narrow_layer(fmt):
    """Few column blocks, many experts: hidden 2048, the intermediate size 768."""
    print(f"[case] narrow layer {_id(fmt)}", flush=True)
    layer = Layer(fmt, 64, 2048, 768, 40, 8)
    layer.check(torch.stack([torch.randperm(64)[:8] for _ in range(40)])[None].int().cuda())


def test_experts_behind_four_gib():
    """A w1 of over 4 GiB: experts at both ends of it."""
    layer = Layer("bf16", 256, 4096, 1152, 4, 2)
    assert 255 * layer.w1.w[0].numel() * 2 > 1 << 32
    ids = torch.tensor([[[255, 0], [254, 255], [3, 200], [-1, 255]]], dtype=torch.int32)
    layer.check(ids.cuda())


@pytest.mark.parametrize("T", [1, 3, 7, 20])
def test_a_hidden_value_past_the_range(T):
    """silu(g) u of one hidden value is past binary32: infinite, with the sign of its weight;
    its second part adds nothing.  The other experts' tokens are as they were."""
    N = I = 128
    ctx = EpCombine(n_ranks=1, top_k=1, max_tokens_per_rank=T + 1, n_experts_per_device=2,
                    hidden_k=I, hidden_n=N)
    w1 = torch.zeros(2, 2 * I, N, device="cuda")
    w2 = torch.zeros(2, N, I, device="cuda")
    w1[:, :, 0] = 1.0
    w1[0, 0, 0] = w1[0, I, 0] = 1e20
    w2[:, :, :] = 0.5
    w2[0, :, 0] = torch.where(torch.arange(N, device="cuda") % 2 == 0, 2.0, -2.0)
    x = torch.zeros(1, T + 1, N, device="cuda").bfloat16()
    x[..., 0] = 4.0
    ids = torch.zeros(1, T + 1, 1, dtype=torch.int32, device="cuda")
    ids[0, T] = 1
    tw = torch.ones(1, T + 1, 1, device="cuda")
    out = ctx.moe_layer(x, w1.bfloat16(), w2.bfloat16(), ids, tw).float()
    assert torch.all(out[0, :T, ::2] == float("inf"))
    assert torch.all(out[0, :T, 1::2] == -float("inf"))
    four = torch.tensor(4.0, dtype=torch.float64)
    want = 0.5 * I * (four * four / (1 + torch.exp(-four))).item()
    assert torch.all((out[0, T] - want).abs() <= 2.0 ** -8 * want)
