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

// ---- The three kinds of weights.  Block: 16 rows of them, one step of 128 k, as a wave
// holds it; Rows: the first operand's 16 rows of the same k.  Wave-uniform: where a
// block's rows start (`row0`), the step.

struct Bf16 {
  static constexpr int DEPTH = 2;
  struct Source {
    buffer w;
    uint32_t slice, lane;               // bytes between 64-k slices; of this lane's row
  };
  struct Block { u32x4 v[4]; };
  struct Rows { u32x4 v[4]; };
  static __device__ __forceinline__ Source source(const MoeWeights& w, int e, int rows, int k,
                                                  int lane) {
    Source s;
    s.w = make_buffer(w.w + (size_t)e * rows * k * 2);
    const uint32_t pitch = w.slice_major ? 128 : k * 2;
    s.slice = w.slice_major ? (uint32_t)rows * 128 : 128;
    s.lane = (lane & 15) * pitch + (lane >> 4) * 16;
    return s;
  }
  static __device__ __forceinline__ uint32_t start(const MoeWeights& w, int row0, int k) {
    return (uint32_t)row0 * (w.slice_major ? 128 : k * 2);
  }
  static __device__ __forceinline__ void load(Block& b, const Source& s, uint32_t start, int kt) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      b.v[q] = buffer_load16_nt(s.w, s.lane + (q & 1) * 64, start + (2 * kt + (q >> 1)) * s.slice);
  }
  // lane L: row L % 16 (at byte `row` of it), k = 32 q + 8 (L / 16) + 0..7
  static __device__ __forceinline__ uint32_t row_lane(int lane) { return (lane >> 4) * 16; }
  static __device__ __forceinline__ void load_rows(Rows& r, buffer x, uint32_t row, int kt) {
#pragma unroll
    for (int q = 0; q < 4; ++q) r.v[q] = buffer_load16(x, row + q * 64, kt * 256);
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
  static constexpr int DEPTH = 3;
  struct Source {
    buffer w, s;
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
    s.w = make_buffer(w.w + (size_t)e * rows * k);
    s.s = make_buffer(reinterpret_cast<const float*>(w.scales) + (size_t)e * (rows / 128) * s.kb);
    s.lane = (lane & 15) * k + (lane >> 4) * 16;
    return s;
  }
  static __device__ __forceinline__ uint32_t start(const MoeWeights&, int row0, int) {
    return row0;
  }
  static __device__ __forceinline__ void load(Block& b, const Source& s, uint32_t row0, int kt) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      b.v[i] = buffer_load16_nt(s.w, s.lane + i * 64, (row0 * s.kb + kt) * 128);
    buffer_load_to(b.s, s.s, 0, ((row0 >> 7) * s.kb + kt) * 4);
  }
};

// Rows of codes with a scale for 128 of them: the up-projection.
struct Fp8Up : Fp8 {
  struct Rows {
    u32x4 v[2];
    uint32_t s[4];                      // of rows 4 (L / 16) + 0..3, as the results have them
  };
  static __device__ __forceinline__ uint32_t row_lane(int lane) { return (lane >> 4) * 16; }
  static __device__ __forceinline__ void load_rows(Rows& r, buffer x, uint32_t row, int kt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) r.v[i] = buffer_load16(x, row + i * 64, kt * 128);
  }
  static __device__ __forceinline__ void multiply(f32x4& acc, const Rows& r, const Block& b) {
    f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const long xr = (long)r.v[i][2 * j] | (long)((uint64_t)r.v[i][2 * j + 1] << 32);
        const long wr = (long)b.v[i][2 * j] | (long)((uint64_t)b.v[i][2 * j + 1] << 32);
        part = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(xr, wr, part, 0, 0, 0);
      }
    const float ws = __builtin_bit_cast(float, b.s);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i] = __builtin_fmaf(part[i], __builtin_bit_cast(float, r.s[i]) * ws, acc[i]);
  }
};

// Rows in bf16: the down-projection, the codes converted (exactly).
struct Fp8Down : Fp8 {
  struct Rows { u32x4 v[4]; };
  static __device__ __forceinline__ uint32_t row_lane(int lane) { return (lane >> 4) * 32; }
  static __device__ __forceinline__ void load_rows(Rows& r, buffer x, uint32_t row, int kt) {
#pragma unroll
    for (int q = 0; q < 4; ++q) r.v[q] = buffer_load16(x, row + (q >> 1) * 128 + (q & 1) * 16, kt * 256);
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
  static constexpr int DEPTH = 3;
  static constexpr uint32_t SB = 16 * (128 / F::GROUP) * 2;   // scale bytes of a run
  struct Source {
    buffer w, s;
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
    s.w = make_buffer(w.w + run * 1024);
    s.s = make_buffer(reinterpret_cast<const uint8_t*>(w.scales) + run * SB);
    s.lane = lane * 16;
    s.lane_s = (lane & 15) * (SB / 16);
    return s;
  }
  static __device__ __forceinline__ uint32_t start(const MoeWeights&, int row0, int) {
    return row0 / 16;
  }
  static __device__ __forceinline__ void load(Block& b, const Source& s, uint32_t start, int kt) {
    const uint32_t run = start * s.kt + kt;
    b.v = buffer_load16_nt(s.w, s.lane, run * 1024);
    buffer_load_to(b.s, s.s, s.lane_s, run * SB);
  }
  static __device__ __forceinline__ uint32_t row_lane(int lane) { return (lane >> 4) * 16; }
  static __device__ __forceinline__ void load_rows(Rows& r, buffer x, uint32_t row, int kt) {
#pragma unroll
    for (int q = 0; q < 4; ++q) r.v[q] = buffer_load16(x, row + q * 64, kt * 256);
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

// Waves a SIMD: 128 registers hold the steps of one row block, two take up to 256.
template <int MT> constexpr int kPerSimd = MT == 1 ? 4 : 2;

template <class P> constexpr bool kCodedRows = false;
template <> constexpr bool kCodedRows<Fp8Up> = true;

// ---- Up-projection and SwiGLU.  An item is a segment and 16 outputs: 16 gate rows and the 16
// up rows of W1, whose K the waves split.
template <class P, int MT>
__global__ __launch_bounds__(kThreads, kPerSimd<MT>) void moe_up_kernel(MoeArgs a) {
  __shared__ Table s;
  __shared__ f32x4 s_part[kWaves][2][MT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  build_table<16 * MT, false>(a, s);
  const int KT = a.hidden / 128, per = a.inter / 16;
  const int k0 = wave * KT / kWaves, k1 = (wave + 1) * KT / kWaves;
  const int items = __builtin_amdgcn_readfirstlane(s.segments) * per;
  constexpr int XB = kCodedRows<P> ? 1 : 2;           // bytes a value of x
  const buffer x = make_buffer(a.x), xs = make_buffer(a.x_scale);
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int seg = item / per, b = item % per;
    const int e = __builtin_amdgcn_readfirstlane(s.seg_expert[seg]);
    const int pair = __builtin_amdgcn_readfirstlane(s.seg_pair[seg]);
    const int n = __builtin_amdgcn_readfirstlane(s.seg_pairs[seg]);
    const auto src = P::source(a.w1, e, 2 * a.inter, a.hidden, lane);
    const uint32_t gate = P::start(a.w1, b * 16, a.hidden);
    const uint32_t up = P::start(a.w1, a.inter + b * 16, a.hidden);
    // rows past the segment's last repeat it; their results are not stored
    uint32_t row[MT], scale_at[MT][4];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int t = s.token[pair + min(j * 16 + (lane & 15), n - 1)];
      row[j] = (uint32_t)t * (uint32_t)a.hidden * XB + P::row_lane(lane);
      if constexpr (kCodedRows<P>)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          scale_at[j][i] = s.token[pair + min(j * 16 + (lane >> 4) * 4 + i, n - 1)] * KT * 4;
    }
    struct Step {
      typename P::Block g, u;
      typename P::Rows r[MT];
    };
    auto load = [&](Step& st, int k) {
      P::load(st.g, src, gate, k);
      P::load(st.u, src, up, k);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        P::load_rows(st.r[j], x, row[j], k);
        if constexpr (kCodedRows<P>)
#pragma unroll
          for (int i = 0; i < 4; ++i) buffer_load_to(st.r[j].s[i], xs, scale_at[j][i], k * 4);
      }
    };
    f32x4 ag[MT], au[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) ag[j] = au[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (k0 < k1) {
      // Loads ahead are unconditional, past the end those of the last step again: with one
      // under a condition the compiler would wait for all that are in flight.
      Step st[P::DEPTH];
#pragma unroll
      for (int d = 0; d < P::DEPTH; ++d) load(st[d], min(k0 + d, k1 - 1));
      for (int k = k0; k < k1;) {
#pragma unroll
        for (int d = 0; d < P::DEPTH; ++d) {
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            P::multiply(ag[j], st[d].r[j], st[d].g);
            P::multiply(au[j], st[d].r[j], st[d].u);
          }
          load(st[d], min(k + P::DEPTH, k1 - 1));
          if (++k >= k1) break;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      s_part[wave][0][j][lane] = ag[j];
      s_part[wave][1][j][lane] = au[j];
    }
    __syncthreads();
    // one value a thread: a pair's row and an output
    if (tid < MT * 256) {
      const int j = tid >> 8, l = (tid >> 2) & 63, i = tid & 3;
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        g += s_part[w][0][j][l][i];
        u += s_part[w][1][j][l][i];
      }
      const int r = j * 16 + (l >> 4) * 4 + i;
      if (r < n)
        reinterpret_cast<__bf16*>(a.h)[(size_t)(pair + r) * a.inter + b * 16 + (l & 15)] =
            (__bf16)(g / (1.f + expf(-g)) * u);
    }
    __syncthreads();
  }
}

// ---- Down-projection and the weighted sum.  A workgroup takes 16 columns of the output; the
// steps of all segments are one run that the waves split evenly.  A wave adds what it has of
// a segment, times the pairs' weights, to its own sums of the tokens in LDS.
template <class P, int MT>
__global__ __launch_bounds__(kThreads, kPerSimd<MT>) void moe_down_kernel(MoeArgs a) {
  __shared__ Table s;
  __shared__ float s_out[kWaves][MT == 1 ? 16 : kMoeTokens][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = lane; i < a.tokens * 16; i += 64) s_out[wave][i >> 4][i & 15] = 0.f;
  build_table<16 * MT, true>(a, s);
  const int KT = a.inter / 128;
  const int steps = __builtin_amdgcn_readfirstlane(s.segments) * KT;
  const int s0 = wave * steps / kWaves, s1 = (wave + 1) * steps / kWaves;
  const int b = blockIdx.x;
  const buffer h = make_buffer(a.h);
  const uint32_t start = P::start(a.w2, b * 16, a.inter);
  if (s0 < s1) {
    struct Step {
      typename P::Block w;
      typename P::Rows r[MT];
    };
    auto load = [&](Step& st, int at) {
      const int seg = at / KT, k = at % KT;
      const int e = __builtin_amdgcn_readfirstlane(s.seg_expert[seg]);
      const int pair = __builtin_amdgcn_readfirstlane(s.seg_pair[seg]);
      const int n = __builtin_amdgcn_readfirstlane(s.seg_pairs[seg]);
      const auto src = P::source(a.w2, e, a.hidden, a.inter, lane);
      P::load(st.w, src, start, k);
#pragma unroll
      for (int j = 0; j < MT; ++j)
        P::load_rows(st.r[j], h,
                     (uint32_t)(pair + min(j * 16 + (lane & 15), n - 1)) * (uint32_t)a.inter * 2 +
                         P::row_lane(lane),
                     k);
    };
    f32x4 acc[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    Step st[P::DEPTH];
#pragma unroll
    for (int d = 0; d < P::DEPTH; ++d) load(st[d], min(s0 + d, s1 - 1));
    for (int at = s0; at < s1;) {
#pragma unroll
      for (int d = 0; d < P::DEPTH; ++d) {
#pragma unroll
        for (int j = 0; j < MT; ++j) P::multiply(acc[j], st[d].r[j], st[d].w);
        load(st[d], min(at + P::DEPTH, s1 - 1));
        ++at;
        if (at % KT == 0 || at >= s1) {
          const int seg = (at - 1) / KT, pair = s.seg_pair[seg], n = s.seg_pairs[seg];
#pragma unroll
          for (int j = 0; j < MT; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = j * 16 + (lane >> 4) * 4 + i;
              if (r < n) s_out[wave][s.token[pair + r]][lane & 15] += s.weight[pair + r] * acc[j][i];
            }
            acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
        }
        if (at >= s1) break;
      }
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

template <class P, int MT>
void launch_up(const MoeArgs& a, int num_cus, hipStream_t st) {
  // at most one segment a pair, and one an expert and every 16 MT pairs
  const int64_t picks = (int64_t)a.tokens * a.top_k;
  const int64_t segments = std::min<int64_t>(picks, a.n_experts + picks / (16 * MT));
  const int64_t grid = std::min<int64_t>(segments * (a.inter / 16), kPerSimd<MT> / 2 * (int64_t)num_cus);
  hipLaunchKernelGGL((moe_up_kernel<P, MT>), dim3((int)grid), dim3(kThreads), 0, st, a);
}

template <class P, int MT>
void launch_down(const MoeArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((moe_down_kernel<P, MT>), dim3(a.hidden / 16), dim3(kThreads), 0, st, a);
}

template <class P>
void launch_product(const MoeArgs& a, bool up, int num_cus, hipStream_t st) {
  if (a.tokens <= 16)
    up ? launch_up<P, 1>(a, num_cus, st) : launch_down<P, 1>(a, st);
  else
    up ? launch_up<P, 2>(a, num_cus, st) : launch_down<P, 2>(a, st);
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
    else if (up)
      a.tokens <= 16 ? launch_up<Fp8Up, 1>(a, num_cus, st) : launch_up<Fp8Up, 2>(a, num_cus, st);
    else
      a.tokens <= 16 ? launch_down<Fp8Down, 1>(a, st) : launch_down<Fp8Down, 2>(a, st);
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
