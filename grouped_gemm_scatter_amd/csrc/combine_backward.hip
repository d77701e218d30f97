// Gradient of the combine on one GPU's share.  For every local pick (rk, t, k):
//   grad_w = sum_n grad_out[rk][t][n] * slot(rk, t, k)[n],
//   grad_rows[m] = bf16(topk_w * grad_out[rk][t]) for the pick's grouped row m.
// An HBM stream: the token's row of grad_out and each local pick's slot are read
// once, each grouped row is written once; a token without local picks reads nothing.
//
// `parts` waves share a token, a column range each, and add up their sums through LDS in
// the order of the columns.  A wave holds up to 4 chunks of 16 bytes a lane of grad_out
// while it goes through the token's local picks, with as many chunks of a slot in
// flight.  The row of a pick is found among its (expert, rank) run, whose rows are in
// ascending (t, k), by probing 64 places at a time: one load for runs of up to 64
// rows, two up to 4096, where a lane's bisection takes seven for 128 rows.
//
// What it measured: 32768 tokens of 7168 values, one pick in eight local, 1.25 GB:
// 265 us, 4.7 TB/s, 80% of the rate of a plain copy (293 us with one wave a token and
// bisection).  308 tokens of 4096 values, 12.4 MB: 9.7 us, of which three dependent reads (ids, run
// bounds, rows' places) are most; a copy of the bytes would take 2.1.
#include <algorithm>

#include "ep_kernels.h"

namespace ep {
namespace {

constexpr int kCombBwdThreads = 512;
constexpr int kCombBwdWaves = kCombBwdThreads / 64;
constexpr int kHeld = 4;           // chunks a lane holds

// Grouped row of pick (t, k) in run [lo, hi) of src_info (ascending (t, k)), or -1; all
// lanes take part, with the same arguments.
__device__ __forceinline__ int find_row(const int32_t* src_info, int lo, int hi, int t, int k,
                                        int lane) {
  const int64_t want = (int64_t)t << 6 | k;        // a handle has at most 64 picks
  auto at = [&](int m) -> int64_t {
    const u32x2 v = *reinterpret_cast<const u32x2*>(src_info + 2 * (size_t)m);
    return (int64_t)(int)v[0] << 6 | (int)v[1];
  };
  while (hi - lo > 64) {
    const int step = (hi - lo + 63) / 64, m = lo + lane * step;
    const int below = __popcll(__ballot(m < hi && at(min(m, hi - 1)) <= want));
    if (below == 0) return -1;
    lo += (below - 1) * step;
    hi = min(hi, lo + step);
  }
  const int m = lo + lane;
  const uint64_t found = __ballot(m < hi && at(min(m, hi - 1)) == want);
  return found ? lo + (int)__builtin_ctzll(found) : -1;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

__global__ __launch_bounds__(kCombBwdThreads) void combine_backward_kernel(CombineBackwardArgs a,
                                                                           int parts) {
  __shared__ float s_dot[kCombBwdWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per_wg = kCombBwdWaves / parts;
  const int64_t total = (int64_t)a.n_ranks * a.tokens;
  const int chunks = a.N / 8, range = (chunks + parts - 1) / parts;
  const int cbeg = (wave % parts) * range, cend = min(chunks, cbeg + range);
  for (int64_t first = (int64_t)blockIdx.x * per_wg; first < total;
       first += (int64_t)gridDim.x * per_wg) {
    const int64_t i = first + wave / parts;
    float gw = 0.f;                // lane k: the gradient of pick k's weight
    if (i < total) {
      const int rk = (int)(i / a.tokens), t = (int)(i % a.tokens);
      const uint8_t* recv = nullptr;
#pragma unroll
      for (int r = 0; r < kMaxRanks; ++r)
        if (r == rk) recv = a.recv[r];
      int g = -1, lo = 0, hi = 0;
      float wk = 0.f;
      if (lane < a.top_k) {
        g = a.topk_ids[i * a.top_k + lane];
        wk = a.topk_w[i * a.top_k + lane];
      }
      const bool is_local = g >= a.expert_lo && g < a.expert_lo + a.n_experts;
      if (is_local && a.grad_rows) {
        const int run = count_index(g - a.expert_lo, rk, a.n_ranks);
        lo = min(max(a.offsets[run], 0), a.m_total);
        hi = min(max(a.offsets[run + 1], 0), a.m_total);
      }
      const uint64_t local = __ballot(is_local);
      const uint8_t* go = a.grad_out + (size_t)i * a.N * 2;
      for (int c0 = cbeg; local && c0 < cend; c0 += 64 * kHeld) {
        u32x4 v[kHeld];
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
          const int c = c0 + u * 64 + lane;
          v[u] = c < cend ? load16_nt(go + (size_t)c * 16) : u32x4{0u, 0u, 0u, 0u};
        }
        for (uint64_t left = local; left; left &= left - 1) {
          const int k = __builtin_ctzll(left);
          const uint8_t* src = recv + slot_offset(t, k, a.top_k, a.msg_bytes);
          u32x4 s[kHeld];
#pragma unroll
          for (int u = 0; u < kHeld; ++u) {
            const int c = c0 + u * 64 + lane;
            s[u] = c < cend ? load16_nt(src + (size_t)c * 16) : u32x4{0u, 0u, 0u, 0u};
          }
          int m = -1;
          if (a.grad_rows) {
            m = find_row(a.src_info, __builtin_amdgcn_readlane(lo, k),
                         __builtin_amdgcn_readlane(hi, k), t, k, lane);
            if (m < 0 && lane == 0) latch_error(a.err, kErrBadGroup);
          }
          const float w = __shfl(wk, k);
          float dot = 0.f;
#pragma unroll
          for (int u = 0; u < kHeld; ++u) {
            const int c = c0 + u * 64 + lane;
            u32x4 o;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float x = bf16_lo(v[u][q]), y = bf16_hi(v[u][q]);
              dot = __builtin_fmaf(x, bf16_lo(s[u][q]), dot);
              dot = __builtin_fmaf(y, bf16_hi(s[u][q]), dot);
              o[q] = pack_bf16x2(w * x, w * y);
            }
            if (m >= 0 && c < cend)
              store16_nt(a.grad_rows + ((size_t)m * a.N + (size_t)c * 8) * 2, o);
          }
          dot = wave_sum(dot);
          if (lane == k) gw += dot;
        }
      }
    }
    if (parts > 1) {
      s_dot[wave][lane] = gw;
      __syncthreads();
      if (wave % parts == 0)
        for (int p = 1; p < parts; ++p) gw += s_dot[wave + p][lane];
      __syncthreads();
    }
    if (i < total && wave % parts == 0 && lane < a.top_k) a.grad_w[i * a.top_k + lane] = gw;
  }
}

}  // namespace

hipError_t launch_combine_backward(const CombineBackwardArgs& a, int num_cus, hipStream_t st) {
  const int64_t total = (int64_t)a.n_ranks * a.tokens;
  // waves a token: enough that each holds its range of the row at once, and all eight
  // where that leaves CUs without a token
  const int chunks = a.N / 8;
  int parts = 1;
  while (parts < kCombBwdWaves &&
         (chunks > parts * 64 * kHeld ||
          (chunks > parts * 64 && total * parts < 2 * (int64_t)num_cus * kCombBwdWaves)))
    parts *= 2;
  const int per_wg = kCombBwdWaves / parts;
  const int64_t grid = std::min<int64_t>((total + per_wg - 1) / per_wg, 16 * (int64_t)num_cus);
  hipLaunchKernelGGL(combine_backward_kernel, dim3((int)grid), dim3(kCombBwdThreads), 0, st, a,
                     parts);
  return hipGetLastError();
}

}  // namespace ep
