// A whole mixture-of-experts layer for at most 64 tokens, in two launches:
//
//   h[p] = bf16( silu(g) u ),  [g; u] = W1_e x[t]      for every pair p of a token t and a
//                                                      local expert e among its picks
//   out[t] = bf16( sum over the token's pairs of c_p W2_e h[p] ),  c_p the pick's weight
//
// What bounds it is streaming the weights of the experts that have tokens, once.  Every
// workgroup finds those experts and their pairs by itself from the picks (a few
// microseconds of LDS work in place of the grouping's launches and of a row count that
// the host would have to read), so the launches' sizes follow from the tokens alone.
//
// The products are 16 x 16 MFMAs with the tokens of an expert as the 16 rows of the first
// operand, 16 rows of the weights as the second.  A workgroup is 8 waves that split K (up) or
// experts and K (down) among them, and join their sums through LDS in the order of the waves.
#include <algorithm>

#include "ep_kernels.h"
#include "w4_device.h"

namespace ep {
namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kMaxSegments = kMaxLocalExperts + kMoeTokens;

// The pairs of a launch.  A segment is up to ROWS pairs of one expert; pairs are numbered by
// (expert, token).
struct Table {
  uint64_t tokens[kMaxLocalExperts];   // expert e: its tokens
  int first[kMaxLocalExperts];         // its first pair
  int seg_expert[kMaxSegments], seg_pair[kMaxSegments], seg_pairs[kMaxSegments];
  float weight[kMoePicks];             // pair: the sum of the token's weights of this expert
  int16_t pick[kMoePicks];             // local expert of a pick, or -1
  uint8_t token[kMoePicks];            // pair: its token
  int segments;
};

template <int ROWS, bool WEIGHTS>
__device__ __forceinline__ void build_table(const MoeArgs& a, Table& s) {
  const int tid = threadIdx.x, picks = a.tokens * a.top_k;
  for (int e = tid; e < a.n_experts; e += kThreads) s.tokens[e] = 0;
  __syncthreads();
  for (int p = tid; p < picks; p += kThreads) {
    const int e = a.topk_ids[p] - a.expert_lo;
    const bool local = e >= 0 && e < a.n_experts;
    s.pick[p] = (int16_t)(local ? e : -1);
    if (local)
      atomicOr(reinterpret_cast<unsigned long long*>(&s.tokens[e]), 1ull << (p / a.top_k));
  }
  __syncthreads();
  if (tid < 64) {
    // pairs and segments before each expert: scans over the lanes, 64 experts at a time
    int pair = 0, seg = 0;
    for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
      const int e = e0 + tid;
      const int n = e < a.n_experts ? __popcll(s.tokens[e]) : 0;
      const int m = (n + ROWS - 1) / ROWS;
      int pn = n, pm = m;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int un = __shfl_up(pn, d), um = __shfl_up(pm, d);
        if (tid >= d) {
          pn += un;
          pm += um;
        }
      }
      if (e < a.n_experts) s.first[e] = pair + pn - n;
      for (int i = 0; i < m; ++i) {
        const int at = seg + pm - m + i;
        s.seg_expert[at] = e;
        s.seg_pair[at] = pair + pn - n + i * ROWS;
        s.seg_pairs[at] = min(n - i * ROWS, ROWS);
      }
      pair += __shfl(pn, 63);
      seg += __shfl(pm, 63);
    }
    if (tid == 0) s.segments = seg;
  }
  __syncthreads();
  for (int p = tid; p < picks; p += kThreads) {
    const int e = s.pick[p], t = p / a.top_k;
    if (e < 0) continue;
    bool again = false;                 // an earlier pick of the same token and expert
    for (int q = t * a.top_k; q < p; ++q) again |= s.pick[q] == e;
    if (again) continue;
    const int pair = s.first[e] + __popcll(s.tokens[e] & ((1ull << t) - 1));
    s.token[pair] = (uint8_t)t;
    if constexpr (WEIGHTS) {
      float w = a.topk_w[p];
      for (int q = p + 1; q < (t + 1) * a.top_k; ++q)
        if (s.pick[q] == e) w += a.topk_w[q];
      s.weight[pair] = w;
    }
  }
  __syncthreads();
}

// Loads and uses of the steps stay where they are written: a wait for a step counts the
// loads behind it, which the compiler can only do where they are in one order on every path.
#define in_order(...)                    \
  do {                                   \
    __VA_ARGS__;                         \
    __builtin_amdgcn_sched_barrier(0);   \
  } while (0)

// ---- The three kinds of weights.  Block: 16 rows of them, one step of 128 k, as a wave
// holds it; Rows: the first operand's 16 rows of the same k.  Wave-uniform: where a
// block's rows start (`row0`), the step.

struct Bf16 {
  static constexpr int DEPTH = 2, DEPTH2 = 1;     // steps in flight, with one and two row blocks
  static constexpr bool PAIR_A_LANE = false;
  struct Source {
    const uint8_t* w;
    uint32_t slice, lane;               // bytes between 64-k slices; of this lane's row
  };
  struct Block { u32x4 v[4]; };
  struct Rows { u32x4 v[4]; };
  static __device__ __forceinline__ Source source(const MoeWeights& w, int e, int rows, int k,
                                                  int lane) {
    Source s;
    s.w = w.w + (size_t)e * rows * k * 2;
    const uint32_t pitch = w.slice_major ? 128 : k * 2;
    s.slice = w.slice_major ? (uint32_t)rows * 128 : 128;
    s.lane = (lane & 15) * pitch + (lane >> 4) * 16;
    return s;
  }
  static __device__ __forceinline__ uint32_t start(const MoeWeights& w, int row0, int k) {
    return (uint32_t)row0 * (w.slice_major ? 128 : k * 2);
  }
  static __device__ __forceinline__ void load(Block& b, const Source& s, uint32_t start, int kt,
                                              int length) {
    const buffer w = make_buffer(s.w, length);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      in_order(b.v[q] = buffer_load16(w, s.lane + (q & 1) * 64,
                                      start + (2 * kt + (q >> 1)) * s.slice));
  }
  // lane L: row L % 16 (at byte `row` of it), k = 32 q + 8 (L / 16) + 0..7
  static __device__ __forceinline__ uint32_t row_lane(int lane) { return (lane >> 4) * 16; }
  static __device__ __forceinline__ void load_rows(Rows& r, buffer x, uint32_t row, int kt) {
#pragma unroll
    for (int q = 0; q < 4; ++q) in_order(r.v[q] = buffer_load16(x, row + q * 64, kt * 256));
  }
  static __device__ __forceinline__ void multiply(f32x4& acc, const Rows& r, const Block& b) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, r.v[q]),
                                                    __builtin_bit_cast(bf16x8, b.v[q]), acc, 0, 0, 0);
  }
};

// e4m3fn codes with a scale for 128 x 128 of them.  A lane's 16 bytes are two operands of 8
// consecutive k, so MFMA 2 i + j takes k = 64 i + 16 (L / 16) + 8 j + 0..7 of both sides.
struct Fp8 {
  struct Source {
    const uint8_t* w;
    const float* s;
    uint32_t lane;
    int kb;                             // scale blocks a row
  };
  struct Block {
    u32x4 v[2];
    uint32_t s;
  };
  static __device__ __forceinline__ Source source(const MoeWeights& w, int e, int rows, int k,
                                                  int lane) {
    Source s;
    s.kb = k / 128;
    s.w = w.w + (size_t)e * rows * k;
    s.s = reinterpret_cast<const float*>(w.scales) + (size_t)e * (rows / 128) * s.kb;
    s.lane = (lane & 15) * k + (lane >> 4) * 16;
    return s;
  }
  static __device__ __forceinline__ uint32_t start(const MoeWeights&, int row0, int) {
    return row0;
  }
  static __device__ __forceinline__ void load(Block& b, const Source& s, uint32_t row0, int kt,
                                              int length) {
    const buffer w = make_buffer(s.w, length);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      in_order(b.v[i] = buffer_load16(w, s.lane + i * 64, (row0 * s.kb + kt) * 128));
    in_order(buffer_load_to(b.s, make_buffer(s.s, length), 0, ((row0 >> 7) * s.kb + kt) * 4));
  }
};

// Rows of codes with a scale for 128 of them: the up-projection.  The weights are the
// first operand, so that a lane's results are of one pair, whose scale it has loaded.
struct Fp8Up : Fp8 {
  static constexpr int DEPTH = 3, DEPTH2 = 2;
  static constexpr bool PAIR_A_LANE = true;
  struct Rows {
    u32x4 v[2];
    uint32_t s;
  };
  static __device__ __forceinline__ uint32_t row_lane(int lane) { return (lane >> 4) * 16; }
  static __device__ __forceinline__ void load_rows(Rows& r, buffer x, uint32_t row, int kt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) in_order(r.v[i] = buffer_load16(x, row + i * 64, kt * 128));
  }
  static __device__ __forceinline__ void multiply(f32x4& acc, const Rows& r, const Block& b) {
    f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const long xr = (long)r.v[i][2 * j] | (long)((uint64_t)r.v[i][2 * j + 1] << 32);
        const long wr = (long)b.v[i][2 * j] | (long)((uint64_t)b.v[i][2 * j + 1] << 32);
        part = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(wr, xr, part, 0, 0, 0);
      }
    const float sc = __builtin_bit_cast(float, r.s) * __builtin_bit_cast(float, b.s);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(part[i], sc, acc[i]);
  }
};

// Rows in bf16: the down-projection, the codes converted (exactly).
struct Fp8Down : Fp8 {
  static constexpr int DEPTH = 3;
  struct Rows { u32x4 v[4]; };
  static __device__ __forceinline__ uint32_t row_lane(int lane) { return (lane >> 4) * 32; }
  static __device__ __forceinline__ void load_rows(Rows& r, buffer x, uint32_t row, int kt) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      in_order(r.v[q] = buffer_load16(x, row + (q >> 1) * 128 + (q & 1) * 16, kt * 256));
  }
  static __device__ __forceinline__ bf16x8 values(uint32_t lo, uint32_t hi) {
    const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, 0);
    const bf16x2 q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, 1);
    const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, 0);
    const bf16x2 s = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, 1);
    return bf16x8{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
  }
  static __device__ __forceinline__ void multiply(f32x4& acc, const Rows& r, const Block& b) {
    f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          __builtin_bit_cast(bf16x8, r.v[q]),
          values(b.v[q >> 1][2 * (q & 1)], b.v[q >> 1][2 * (q & 1) + 1]), part, 0, 0, 0);
    const float ws = __builtin_bit_cast(float, b.s);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(part[i], ws, acc[i]);
  }
};

// Packed 4-bit codes: 16 rows x 128 k are one run of 1 KB.
template <class F>
struct W4 {
  static constexpr int DEPTH = 3, DEPTH2 = 1;
  static constexpr bool PAIR_A_LANE = false;
  static constexpr uint32_t SB = 16 * (128 / F::GROUP) * 2;   // scale bytes of a run
  struct Source {
    const uint8_t *w, *s;
    uint32_t lane, lane_s;
    int kt;                             // runs of a 16-row block
  };
  struct Block {
    u32x4 v;
    typename F::word s;
  };
  struct Rows { u32x4 v[4]; };
  static __device__ __forceinline__ Source source(const MoeWeights& w, int e, int rows, int k,
                                                  int lane) {
    Source s;
    s.kt = k / 128;
    const size_t run = (size_t)e * (rows / 16) * s.kt;
    s.w = w.w + run * 1024;
    s.s = reinterpret_cast<const uint8_t*>(w.scales) + run * SB;
    s.lane = lane * 16;
    s.lane_s = (lane & 15) * (SB / 16);
    return s;
  }
  static __device__ __forceinline__ uint32_t start(const MoeWeights&, int row0, int) {
    return row0 / 16;
  }
  static __device__ __forceinline__ void load(Block& b, const Source& s, uint32_t start, int kt,
                                              int length) {
    const uint32_t run = start * s.kt + kt;
    in_order(b.v = buffer_load16(make_buffer(s.w, length), s.lane, run * 1024));
    in_order(buffer_load_to(b.s, make_buffer(s.s, length), s.lane_s, run * SB));
  }
  static __device__ __forceinline__ uint32_t row_lane(int lane) { return (lane >> 4) * 16; }
  static __device__ __forceinline__ void load_rows(Rows& r, buffer x, uint32_t row, int kt) {
#pragma unroll
    for (int q = 0; q < 4; ++q) in_order(r.v[q] = buffer_load16(x, row + q * 64, kt * 256));
  }
  static __device__ __forceinline__ void multiply(f32x4& acc, const Rows& r, const Block& b) {
    constexpr int SPT = 128 / F::GROUP, QPS = 4 / SPT;
#pragma unroll
    for (int s = 0; s < SPT; ++s) {
      f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < QPS; ++q)
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, r.v[s * QPS + q]), decode8<F::CODES>(b.v[s * QPS + q]), part,
            0, 0, 0);
      const float sc = F::scale((uint16_t)(b.s >> (16 * s)));
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(sc, part[i], acc[i]);
    }
  }
};

// ---- Up-projection and SwiGLU.  An item is a segment and 16 outputs: 16 gate rows and the 16
// up rows of W1, whose K the waves split.
template <class P, int MT, int DEPTH>
__device__ __forceinline__ void up_item(const MoeArgs& a, const Table& s, f32x4 (*s_part)[2][2][64],
                                        int e, int b, int pair, int n, int wave, int lane) {
  const int KT = a.hidden / 128;
  const auto src = P::source(a.w1, e, 2 * a.inter, a.hidden, lane);
  const uint32_t gate = P::start(a.w1, b * 16, a.hidden);
  const uint32_t up = P::start(a.w1, a.inter + b * 16, a.hidden);
  // rows past the segment's last repeat it; their results are not stored
  uint32_t row[MT], scale_at[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int t = s.token[pair + min(j * 16 + (lane & 15), n - 1)];
    row[j] = (uint32_t)t * (uint32_t)a.hidden * (P::PAIR_A_LANE ? 1 : 2) + P::row_lane(lane);
    scale_at[j] = t * KT * 4;
  }
  struct Step {
    typename P::Block g, u;
    typename P::Rows r[MT];
  };
  auto load = [&](Step& st, int k) {
    const int length = buffer_length(k, KT);
    P::load(st.g, src, gate, k, length);
    P::load(st.u, src, up, k, length);
    const buffer x = make_buffer(a.x, length);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      P::load_rows(st.r[j], x, row[j], k);
      if constexpr (P::PAIR_A_LANE)
        in_order(buffer_load_to(st.r[j].s, make_buffer(a.x_scale, length), scale_at[j], k * 4));
    }
  };
  f32x4 ag[MT], au[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) ag[j] = au[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // A wave takes every eighth step, so that the workgroup's reads of a row are one run.
  // Loads ahead are unconditional, past the end of an empty buffer: with one under a
  // condition the compiler would wait for all that are in flight.
  Step st[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(st[d], wave + d * kWaves);
  for (int k = wave; k < KT;) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        P::multiply(ag[j], st[d].r[j], st[d].g);
        P::multiply(au[j], st[d].r[j], st[d].u);
      }
      __builtin_amdgcn_sched_barrier(0);
      load(st[d], k + DEPTH * kWaves);
      k += kWaves;
      if (k >= KT) break;
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    s_part[wave][0][j][lane] = ag[j];
    s_part[wave][1][j][lane] = au[j];
  }
}

template <class P>
__global__ __launch_bounds__(kThreads, 4) void moe_up_kernel(MoeArgs a) {
  __shared__ Table s;
  __shared__ f32x4 s_part[kWaves][2][2][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  build_table<32, false>(a, s);
  const int per = a.inter / 16;
  const int items = __builtin_amdgcn_readfirstlane(s.segments) * per;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int seg = item / per, b = item % per;
    const int e = __builtin_amdgcn_readfirstlane(s.seg_expert[seg]);
    const int pair = __builtin_amdgcn_readfirstlane(s.seg_pair[seg]);
    const int n = __builtin_amdgcn_readfirstlane(s.seg_pairs[seg]);
    if (n <= 16)
      up_item<P, 1, P::DEPTH>(a, s, s_part, e, b, pair, n, wave, lane);
    else
      up_item<P, 2, P::DEPTH2>(a, s, s_part, e, b, pair, n, wave, lane);
    __syncthreads();
    // one value a thread: a pair's row and an output
    {
      const int j = tid >> 8, l = (tid >> 2) & 63, i = tid & 3;
      const int r = j * 16 + (P::PAIR_A_LANE ? l & 15 : (l >> 4) * 4 + i);
      const int c = P::PAIR_A_LANE ? (l >> 4) * 4 + i : l & 15;
      if (r < n) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          g += s_part[w][0][j][l][i];
          u += s_part[w][1][j][l][i];
        }
        reinterpret_cast<__bf16*>(a.h)[(size_t)(pair + r) * a.inter + b * 16 + c] =
            (__bf16)(g / (1.f + expf(-g)) * u);
      }
    }
    __syncthreads();
  }
}

// ---- Down-projection and the weighted sum.  A workgroup takes 16 columns of the output; the
// steps of all segments are one run that the waves split evenly.  A wave adds what it has of
// a segment, times the pairs' weights, to its own sums of the tokens in LDS.
// The segments are of 16 pairs: an expert's weights are read again for its next 16, by the
// same workgroup and at once.
template <class P>
__global__ __launch_bounds__(kThreads, 4) void moe_down_kernel(MoeArgs a) {
  __shared__ Table s;
  __shared__ float s_out[kWaves][kMoeTokens][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = lane; i < a.tokens * 16; i += 64) s_out[wave][i >> 4][i & 15] = 0.f;
  build_table<16, true>(a, s);
  const int KT = a.inter / 128;
  const int b = blockIdx.x;
  const uint32_t start = P::start(a.w2, b * 16, a.inter);
  struct Step {
    typename P::Block w;
    typename P::Rows r;
  };
  // A step by its segment and its k; a wave takes every eighth.
  struct Place {
    int seg, k;
  };
  auto next = [&](Place p) {
    p.k += kWaves;
    while (p.k >= KT) {
      p.k -= KT;
      ++p.seg;
    }
    return p;
  };
  const int segments = __builtin_amdgcn_readfirstlane(s.segments);
  auto load = [&](Step& st, Place p) {
    const int length = buffer_length(p.seg, segments);
    const int seg = min(p.seg, kMaxSegments - 1);
    const int e = __builtin_amdgcn_readfirstlane(s.seg_expert[seg]);
    const int pair = __builtin_amdgcn_readfirstlane(s.seg_pair[seg]);
    const int n = __builtin_amdgcn_readfirstlane(s.seg_pairs[seg]);
    const auto src = P::source(a.w2, e, a.hidden, a.inter, lane);
    P::load(st.w, src, start, p.k, length);
    const buffer h = make_buffer(a.h, length);
    P::load_rows(st.r, h,
                 (uint32_t)(pair + min(lane & 15, n - 1)) * (uint32_t)a.inter * 2 +
                     P::row_lane(lane),
                 p.k);
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  Step st[P::DEPTH];
  Place now{0, wave - kWaves}, ahead;
  now = next(now);
  ahead = now;
#pragma unroll
  for (int d = 0; d < P::DEPTH; ++d) {
    load(st[d], ahead);
    ahead = next(ahead);
  }
  while (now.seg < segments) {
#pragma unroll
    for (int d = 0; d < P::DEPTH; ++d) {
      P::multiply(acc, st[d].r, st[d].w);
      __builtin_amdgcn_sched_barrier(0);
      load(st[d], ahead);
      ahead = next(ahead);
      const Place then = next(now);
      if (then.seg != now.seg) {
        const int pair = s.seg_pair[now.seg], n = s.seg_pairs[now.seg];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (lane >> 4) * 4 + i;
          if (r < n) s_out[wave][s.token[pair + r]][lane & 15] += s.weight[pair + r] * acc[i];
        }
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      now = then;
      if (now.seg >= segments) break;
    }
  }
  __syncthreads();
  for (int i = tid; i < a.tokens * 8; i += kThreads) {
    const int t = i >> 3, c = (i & 7) * 2;
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      lo += s_out[w][t][c];
      hi += s_out[w][t][c + 1];
    }
    reinterpret_cast<uint32_t*>(a.out)[((size_t)t * a.hidden + b * 16 + c) / 2] = pack_bf16x2(lo, hi);
  }
}

template <class P>
void launch_up(const MoeArgs& a, int num_cus, hipStream_t st) {
  // at most one segment a pair, and one an expert and every 32 pairs
  const int64_t picks = (int64_t)a.tokens * a.top_k;
  const int64_t segments = std::min<int64_t>(picks, a.n_experts + picks / 32);
  const int64_t grid = std::min<int64_t>(segments * (a.inter / 16), 2 * (int64_t)num_cus);
  hipLaunchKernelGGL((moe_up_kernel<P>), dim3((int)grid), dim3(kThreads), 0, st, a);
}

template <class P>
void launch_down(const MoeArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((moe_down_kernel<P>), dim3(a.hidden / 16), dim3(kThreads), 0, st, a);
}

template <class P>
void launch_product(const MoeArgs& a, bool up, int num_cus, hipStream_t st) {
  up ? launch_up<P>(a, num_cus, st) : launch_down<P>(a, st);
}

template <int CODES, int GROUP>
void launch_w4(const MoeArgs& a, bool up, bool f16, int num_cus, hipStream_t st) {
  if (f16)
    launch_product<W4<Format<CODES, GROUP, true>>>(a, up, num_cus, st);
  else
    launch_product<W4<Format<CODES, GROUP, false>>>(a, up, num_cus, st);
}

hipError_t launch_product_of(const MoeArgs& a, const MoeWeights& w, bool up, int num_cus,
                             hipStream_t st) {
  if (w.group == 0) {
    if (!a.fp8)
      launch_product<Bf16>(a, up, num_cus, st);
    else
      up ? launch_up<Fp8Up>(a, num_cus, st) : launch_down<Fp8Down>(a, st);
    return hipGetLastError();
  }
  switch (w.codes * 1000 + w.group) {
    case 32: launch_w4<EP_W4_INT4, 32>(a, up, w.scale_f16, num_cus, st); break;
    case 64: launch_w4<EP_W4_INT4, 64>(a, up, w.scale_f16, num_cus, st); break;
    case 128: launch_w4<EP_W4_INT4, 128>(a, up, w.scale_f16, num_cus, st); break;
    case 1032: launch_w4<EP_W4_E2M1, 32>(a, up, w.scale_f16, num_cus, st); break;
    case 1064: launch_w4<EP_W4_E2M1, 64>(a, up, w.scale_f16, num_cus, st); break;
    case 1128: launch_w4<EP_W4_E2M1, 128>(a, up, w.scale_f16, num_cus, st); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(const MoeArgs& a, int num_cus, hipStream_t st) {
  const hipError_t err = launch_product_of(a, a.w1, true, num_cus, st);
  return err != hipSuccess ? err : launch_product_of(a, a.w2, false, num_cus, st);
}

}  // namespace ep
