// Gradient of the combine on one GPU's share.  For every local pick (rk, t, k):
//   grad_w = sum_n grad_out[rk][t][n] * slot(rk, t, k)[n],
//   grad_rows[m] = bf16(topk_w * grad_out[rk][t]) for the pick's grouped row m.
// One wave per token.  The lanes holding picks find the local ones, and each finds
// its pick's row by bisection of its (expert, rank) run, whose rows are in
// ascending (t, k); the wave then streams the pick's slot against the token's
// row of grad_out.  Products and sums are binary32, in an order that the shape
// alone fixes.
#include <algorithm>

#include "ep_kernels.h"

namespace ep {
namespace {

constexpr int kCombBwdThreads = 256;
constexpr int kCombBwdWaves = kCombBwdThreads / 64;

// Grouped row of pick (t, k) in run [lo, hi) of src_info (ascending (t, k)), or -1.
__device__ __forceinline__ int find_row(const int32_t* src_info, int lo, int hi, int t, int k) {
  const int end = hi;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    const int mt = src_info[2 * (size_t)mid], mk = src_info[2 * (size_t)mid + 1];
    if (mt < t || (mt == t && mk < k)) lo = mid + 1; else hi = mid;
  }
  if (lo >= end) return -1;
  return src_info[2 * (size_t)lo] == t && src_info[2 * (size_t)lo + 1] == k ? lo : -1;
}

__global__ __launch_bounds__(kCombBwdThreads) void combine_backward_kernel(CombineBackwardArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kCombBwdWaves + (threadIdx.x >> 6);
  const int64_t waves = (int64_t)gridDim.x * kCombBwdWaves;
  const int64_t total = (int64_t)a.n_ranks * a.tokens;
  const int chunks = a.N / 8;
  for (int64_t i = wave; i < total; i += waves) {
    const int rk = (int)(i / a.tokens), t = (int)(i % a.tokens);
    const uint8_t* recv = nullptr;
#pragma unroll
    for (int r = 0; r < kMaxRanks; ++r)
      if (r == rk) recv = a.recv[r];
    int g = -1, row = -1;
    float wk = 0.f;
    if (lane < a.top_k) {
      g = a.topk_ids[i * a.top_k + lane];
      wk = a.topk_w[i * a.top_k + lane];
    }
    const bool is_local = g >= a.expert_lo && g < a.expert_lo + a.n_experts;
    if (is_local && a.grad_rows) {
      const int run = count_index(g - a.expert_lo, rk, a.n_ranks);
      const int lo = min(max(a.offsets[run], 0), a.m_total);
      const int hi = min(max(a.offsets[run + 1], 0), a.m_total);
      row = find_row(a.src_info, lo, hi, t, lane);
      if (row < 0) latch_error(a.err, kErrBadGroup);
    }
    const uint8_t* go = a.grad_out + (size_t)i * a.N * 2;
    float gw = 0.f;                // lane k: the gradient of pick k's weight
    uint64_t mask = __ballot(is_local);
    while (mask) {
      const int k = __builtin_ctzll(mask);
      mask &= mask - 1;
      const float w = __shfl(wk, k);
      const int m = __shfl(row, k);
      const uint8_t* src = recv + slot_offset(t, k, a.top_k, a.msg_bytes);
      float dot = 0.f;
      for (int c = lane; c < chunks; c += 64) {
        const u32x4 v = load16(go + (size_t)c * 16), s = load16_nt(src + (size_t)c * 16);
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          dot = __builtin_fmaf(bf16_lo(v[q]), bf16_lo(s[q]), dot);
          dot = __builtin_fmaf(bf16_hi(v[q]), bf16_hi(s[q]), dot);
          o[q] = pack_bf16x2(w * bf16_lo(v[q]), w * bf16_hi(v[q]));
        }
        if (m >= 0) store16_nt(a.grad_rows + ((size_t)m * a.N + (size_t)c * 8) * 2, o);
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d);
      if (lane == k) gw = dot;
    }
    if (lane < a.top_k) a.grad_w[i * a.top_k + lane] = gw;
  }
}

}  // namespace

hipError_t launch_combine_backward(const CombineBackwardArgs& a, int num_cus, hipStream_t st) {
  const int64_t total = (int64_t)a.n_ranks * a.tokens;
  const int64_t grid = std::min<int64_t>((total + kCombBwdWaves - 1) / kCombBwdWaves,
                                         16 * (int64_t)num_cus);
  hipLaunchKernelGGL(combine_backward_kernel, dim3((int)grid), dim3(kCombBwdThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace ep
