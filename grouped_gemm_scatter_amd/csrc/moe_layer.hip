// A whole mixture-of-experts layer for at most 64 tokens, in two launches:
//
//   h[p] = silu(g) u,  [g; u] = W1_e x[t]              for every pair p of a token t and a
//                                                      local expert e among its picks
//   out[t] = bf16( sum over the token's pairs of c_p W2_e h[p] ),  c_p the pick's weight
//
// What bounds it is streaming the weights of the experts that have tokens: once for up to 32
// tokens of an expert in the up-projection and up to 16 in the down-projection, then again for
// every further 32 and 16.  Every workgroup finds those experts and their pairs by itself
// from the picks (1.6 us of LDS work in place of the grouping's launches and of a row count
// that the host would have to read), so the launches' sizes follow from the tokens alone.
//
// The products are 16 x 16 MFMAs with the tokens of an expert as rows of the first operand, 16
// rows of the weights as the second.  A workgroup is 8 waves that split K (up) or experts and
// K (down) among them, and join their sums through LDS in the order of the waves.  h is
// held as two bf16 values, since the matrix instruction takes bf16: the second is what the
// first one's rounding leaves, together 2^-17 of the value.  (The first alone takes the
// output's error from the 0.0017 of its own rounding to 0.0024 of its length.)  They are two
// rows of the first operand, of which an expert of one or two tokens leaves most unused
// anyway; of more tokens they cost row loads, 10 to 15% of the down-projection for 2 tokens an
// expert on average, half of it for 16.  Its sums are rounded once, as the output.
//
// What it measured (kernels alone, us up and down; the bytes at the 5.95 TB/s of a plain copy):
//   one token, 8 experts of 7168 x 2048    bf16  80 + 45 (118)   fp8 44 + 27 (59)
//                                          int4, groups of 128   27 + 18 (31)
//   five tokens of the same in fp8, 25 experts             140 + 82 (185)
//   64 tokens, 28 of 32 experts, e2m1, groups of 32         74 + 61 (116)
//   16 tokens, 14 of 16 experts of 4096 x 1024, bf16        46 + 26 (60)
//   one token, 2 experts of 1024 x 256, bf16                 6 + 5: launches and latency
// Large up-projections run at 5.2 to 6.2 TB/s, down-projections at 3.8 to 5.3.  Without a local
// pick the two launches take 2.8 and 3.5 us (picks, table, zeros), and the first weights' trip
// to memory follows; there is no gap between the two.  Vector instructions, most of them code
// conversions, are 16 of the 27 us of one int4 token's up-projection.
// Beside the grouped calls (group, dispatch, both products, combine, in a graph with the row
// count known), us here and there, 32 experts of 7168 x 2048, eight picks a token:
//   tokens an expert       4            6            8            12           16
//   bf16                499 and 602  531 and 608  575 and 606  662 and 611  779 and 616
//   fp8                 289 and 367  325 and 369  372 and 369  459 and 372  554 and 373
//   int4, groups of 128 174 and 178  204 and 179  244 and 183  333 and 189  414 and 196
//   e2m1, groups of 32  178 and 179  216 and 181  253 and 180  404 and 186  491 and 195
// (the weights once: 474, 237, 122 and 133).  Many tokens cost here what their rows do, loaded
// again for every 16 outputs, and weights that are read again; with groups of 32, also 16
// registers that the up-projection's path of 32 rows spills.
#include <algorithm>

#include "ep_kernels.h"
#include "layer_kernels.h"
#include "w4_device.h"

namespace ep {
namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kMaxSegments = kMaxLocalExperts + kMoeTokens;

// The pairs of a launch, numbered by (expert, token).  A segment is up to ROWS pairs of one
// expert.  Up to FEW pairs, up to MID and more of them take different paths through the
// products, so that an expert of many tokens does not slow down those of few.
struct Table {
  uint64_t tokens[kMaxLocalExperts];   // expert e: its tokens
  int first[kMaxLocalExperts];         // its first pair
  int seg_expert[kMaxSegments], seg_pair[kMaxSegments], seg_pairs[kMaxSegments];
  int16_t pick[kMoePicks];             // local expert of a pick, or -1
  uint8_t token[kMoePicks];            // pair: its token
  int few, mid, segments;              // ends of the segments of few and of up to MID pairs
                                       // in the list, and of the list
  int over_half, over16;               // whether experts of FEW / 2 + 1..FEW pairs, and of
                                       // over 16, are there
};

// Lanes below this one in a mask of lanes.
__device__ __forceinline__ int lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// The picks' weights, and by pairs: the sum of the token's weights of this expert.
struct Weights {
  float pick[kMoePicks], pair[kMoePicks];
};

template <int ROWS, int FEW, int MID>
__device__ __forceinline__ void build_table(const MoeArgs& a, Table& s, Weights* w = nullptr) {
  const int tid = threadIdx.x, picks = a.tokens * a.top_k;
  for (int e = tid; e < a.n_experts; e += kThreads) s.tokens[e] = 0;
  __syncthreads();
  for (int p = tid; p < picks; p += kThreads) {
    const int e = a.topk_ids[p] - a.expert_lo;
    if (w) w->pick[p] = a.topk_w[p];
    const bool local = e >= 0 && e < a.n_experts;
    s.pick[p] = (int16_t)(local ? e : -1);
    if (local)
      atomicOr(reinterpret_cast<unsigned long long*>(&s.tokens[e]), 1ull << (p / a.top_k));
  }
  __syncthreads();
  if (tid < 64) {
    // pairs and segments before each expert, 64 experts at a time: counts by their bits, each
    // a ballot
    auto pairs_of = [&](int e) { return e < a.n_experts ? __popcll(s.tokens[e]) : 0; };
    auto is_few = [](int n) { return n > 0 && n <= FEW; };
    auto is_mid = [](int n) { return n > FEW && n <= MID; };
    int few = 0, mid = 0, pair = 0, over_half = 0, over16 = 0;
    for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
      const int n = pairs_of(e0 + tid);
      few += __popcll(__ballot(is_few(n)));
      if constexpr (MID > FEW) mid += __popcll(__ballot(is_mid(n)));
    }
    int few_seg = 0, mid_seg = few, seg = few + mid;
    for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
      const int e = e0 + tid, n = pairs_of(e);
      int pairs_before = pair;
      for (int bit = 0; a.tokens >> bit; ++bit) {
        const uint64_t m = __ballot(n >> bit & 1);
        pairs_before += lanes_below(m) << bit;
        pair += __popcll(m) << bit;
      }
      const uint64_t in_few = __ballot(is_few(n));
      int at = n > FEW ? seg : few_seg + lanes_below(in_few);
      few_seg += __popcll(in_few);
      if constexpr (MID > FEW) {
        const uint64_t in_mid = __ballot(is_mid(n));
        if (is_mid(n)) at = mid_seg + lanes_below(in_mid);
        mid_seg += __popcll(in_mid);
      }
      for (int i = 0; i * ROWS < a.tokens; ++i) {
        const uint64_t m = __ballot(n > MID && n > i * ROWS);
        if (n > MID) at += lanes_below(m);
        seg += __popcll(m);
      }
      over_half |= __ballot(n > FEW / 2 && n <= FEW) != 0;
      over16 |= __ballot(n > 16) != 0;
      if (e < a.n_experts) s.first[e] = pairs_before;
      for (int i = 0; i * ROWS < n; ++i) {
        s.seg_expert[at + i] = e;
        s.seg_pair[at + i] = pairs_before + i * ROWS;
        s.seg_pairs[at + i] = min(n - i * ROWS, ROWS);
      }
    }
    if (tid == 0) {
      s.few = few;
      s.mid = few + mid;
      s.segments = seg;
      s.over_half = over_half;
      s.over16 = over16;
    }
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
    if (w) {
      float sum = w->pick[p];
      for (int q = p + 1; q < (t + 1) * a.top_k; ++q)
        if (s.pick[q] == e) sum += w->pick[q];
      w->pair[pair] = sum;
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

// ---- The first operand's rows, RB of them: 4, 8, 16 or 32 for pairs of an expert (one a pair
// in the up-projection, two in the down-projection).
// An MFMA has 16 rows, and in a step's 128 k four of them follow (by quarters of k).
// Fewer than 16 rows would leave its lanes loading one row over and over, four loads a
// step that cost as much of the memory path as the weights (a stream of 4-bit weights by
// itself 6.1 TB/s, with these loads 4.4).  So lane L % 16 loads row L % 16 % RB, of a quarter
// of its own, and every quarter's MFMA takes the same register: its rows with another
// quarter's values come out wrong and are left out, which 16 / RB accumulators, one a
// quarter (or two quarters), make possible.
// JOINED: the row blocks are parts of the same pairs, and go into one accumulator.
template <int RB, bool JOINED = false>
struct RowsOf {
  static constexpr int ROWS = RB;
  static constexpr int BLOCKS = RB > 16 ? RB / 16 : 1;
  static constexpr int SUMS = JOINED ? 1 : BLOCKS;       // of one quarter's products
  static constexpr int ACCS = RB < 16 ? 16 / RB : SUMS;
  static constexpr int sum(int j) { return JOINED ? 0 : j; }
};

// The sums of all quarters of a lane's accumulators, RB rows in rows 0..RB - 1 of the result.
__device__ __forceinline__ float add_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_quarters(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Rows of the results by lane: 4 (L / 16) + i.
template <int RB>
__device__ __forceinline__ f32x4 add_row_parts(const f32x4 (&acc)[RowsOf<RB>::ACCS], int lane) {
  static_assert(RB <= 8, "rows in parts");
  const int g = lane >> 4;
  f32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (RB == 8) {
      v[i] = add_halves(g < 2 ? acc[0][i] : acc[1][i]);
    } else {
      const float lo = g == 0 ? acc[0][i] : acc[1][i], hi = g == 2 ? acc[2][i] : acc[3][i];
      v[i] = add_halves(add_quarters(g < 2 ? lo : hi));
    }
  }
  return v;
}

// Rows in bf16: 8 values a lane of each quarter of a step's 128 k (where they lie: at()).
template <int RB, bool JOINED = false>
struct Bf16Rows : RowsOf<RB, JOINED> {
  u32x4 v[RB < 16 ? RB / 4 : 4 * RowsOf<RB>::BLOCKS];
  // register of row block j and quarter q, and its accumulator
  static constexpr int reg(int j, int q) { return RB < 16 ? q & (RB / 4 - 1) : 4 * j + q; }
  static constexpr int acc(int j, int q) { return RB < 16 ? q / (RB / 4) : JOINED ? 0 : j; }
  // quarter that the lane loads first
  static __device__ __forceinline__ int quarter(int lane) {
    return RB < 16 ? (lane & 15) / RB * (RB / 4) : 0;
  }
};

// The blocks of a step of the up-projection: 16 gate rows and their 16 up rows.
template <class P>
struct TwoBlocks {
  typename P::Block g, u;
  __device__ __forceinline__ void load(const typename P::Source& s, uint32_t gate, uint32_t up,
                                       int kt, int length) {
    P::load(g, s, gate, kt, length);
    P::load(u, s, up, kt, length);
  }
  template <class Rows>
  __device__ __forceinline__ void multiply(f32x4 (&ag)[Rows::ACCS], f32x4 (&au)[Rows::ACCS],
                                           const Rows& r) const {
    P::multiply(ag, r, g);
    P::multiply(au, r, u);
  }
};

// ---- The three kinds of weights.  Block: 16 rows of them, one step of 128 k, as a wave
// holds it; Rows: the first operand's 16 rows of the same k.  Wave-uniform: where a
// block's rows start (`row0`), the step.

struct Bf16 {
  static constexpr int STEP = 128;                 // k of a step of the down-projection
  static constexpr bool SPREAD = true;             // its steps: every eighth, or a run
  // Steps on their way beside the one that is multiplied.  One serves where sixteen waves a CU
  // hold 2 to 8 KB each (two and three were as fast or up to 5% slower in every product,
  // 4-bit: 77 and 74 us up); in bf16 down, one took 48.9 us where two take 43.8 (one token
  // of 7168 x 2048; 16 of 4096 x 1024: 24.5 and 25.6).
  static constexpr int UP_DEPTH = 1, DOWN_DEPTH = 2;
  static constexpr bool PAIR_A_LANE = false;
  struct Source {
    const uint8_t* w;
    uint32_t slice, lane;               // bytes between 64-k slices; of this lane's row
  };
  struct Block { u32x4 v[4]; };
  template <int RB, bool JOINED = false> using Rows = Bf16Rows<RB, JOINED>;
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
  // byte of a lane's first values in its row's 256 of a step, and of the next quarter
  static __device__ __forceinline__ uint32_t at(int lane, int quarter) {
    return (lane >> 4) * 16 + quarter * 64;
  }
  template <int RB, bool JOINED>
  static __device__ __forceinline__ void load_rows(Bf16Rows<RB, JOINED>& r, const uint8_t* x0,
                                                   int length,
                                                   const uint32_t (&row)[RowsOf<RB>::BLOCKS],
                                                   int kt, int) {
    const buffer x = make_buffer(x0, length);
#pragma unroll
    for (int j = 0; j < RowsOf<RB>::BLOCKS; ++j)
#pragma unroll
      for (int q = 0; q < (RB < 16 ? RB / 4 : 4); ++q)
        in_order(r.v[4 * j + q] = buffer_load16(x, row[j] + q * 64, kt * 256));
  }
  template <class R>
  static __device__ __forceinline__ void multiply(f32x4 (&acc)[R::ACCS], const R& r,
                                                  const Block& b) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < R::BLOCKS; ++j) {
        f32x4& to = acc[r.acc(j, q)];
        to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, r.v[r.reg(j, q)]),
                                                     __builtin_bit_cast(bf16x8, b.v[q]), to, 0, 0, 0);
      }
  }
};

// One step of weights whose scale holds for QPS quarters: w(q) the values of quarter q,
// scale(q) its scale.
template <int QPS, class R, class W, class S>
__device__ __forceinline__ void scaled_multiply(f32x4 (&acc)[R::ACCS], const R& r, W w, S scale) {
  // quarters of one sum: of one scale and one accumulator
  constexpr int RUN = R::ROWS < 16 && R::ROWS / 4 < QPS ? R::ROWS / 4 : QPS;
#pragma unroll
  for (int q0 = 0; q0 < 4; q0 += RUN) {
    f32x4 part[R::SUMS] = {};
#pragma unroll
    for (int q = q0; q < q0 + RUN; ++q) {
      const bf16x8 wq = w(q);
#pragma unroll
      for (int j = 0; j < R::BLOCKS; ++j) {
        f32x4& to = part[R::sum(j)];
        to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, r.v[r.reg(j, q)]), wq, to, 0, 0, 0);
      }
    }
    const float sc = scale(q0);
#pragma unroll
    for (int j = 0; j < R::SUMS; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4& to = acc[r.acc(j, q0)];
        to[i] = __builtin_fmaf(sc, part[j][i], to[i]);
      }
  }
}

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
  static constexpr int UP_DEPTH = 1;
  static constexpr bool PAIR_A_LANE = true;
  // a row's 128 bytes of a step are two halves of k; with 8 rows a lane loads one of them
  template <int RB>
  struct Rows : RowsOf<RB> {
    static_assert(RB >= 8, "halves of k");
    u32x4 v[RB < 16 ? 1 : 2 * RowsOf<RB>::BLOCKS];
    uint32_t s[RowsOf<RB>::BLOCKS];
    static constexpr int reg(int j, int h) { return RB < 16 ? 0 : 2 * j + h; }
    static constexpr int acc(int j, int h) { return RB < 16 ? h : j; }
    static __device__ __forceinline__ int quarter(int lane) { return RB < 16 ? (lane & 15) / 8 : 0; }
  };
  static __device__ __forceinline__ uint32_t at(int lane, int half) {
    return (lane >> 4) * 16 + half * 64;
  }
  template <int RB>
  static __device__ __forceinline__ void load_rows(Rows<RB>& r, const uint8_t* x0, int length,
                                                   const uint32_t (&row)[RowsOf<RB>::BLOCKS],
                                                   int kt, int) {
    const buffer x = make_buffer(x0, length);
#pragma unroll
    for (int j = 0; j < RowsOf<RB>::BLOCKS; ++j)
#pragma unroll
      for (int h = 0; h < (RB < 16 ? 1 : 2); ++h)
        in_order(r.v[2 * j + h] = buffer_load16(x, row[j] + h * 64, kt * 128));
  }
  template <class R>
  static __device__ __forceinline__ void multiply(f32x4 (&acc)[R::ACCS], const R& r,
                                                  const Block& b) {
    const float ws = __builtin_bit_cast(float, b.s);
    constexpr int PARTS = R::ROWS < 16 ? 2 : 1;      // accumulators a step's halves go to
#pragma unroll
    for (int j = 0; j < R::BLOCKS; ++j) {
      const float sc = __builtin_bit_cast(float, r.s[j]) * ws;
      f32x4 part[PARTS] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const u32x4 x = r.v[r.reg(j, h)], w = b.v[h];
          const long xr = (long)x[2 * o] | (long)((uint64_t)x[2 * o + 1] << 32);
          const long wr = (long)w[2 * o] | (long)((uint64_t)w[2 * o + 1] << 32);
          f32x4& to = part[PARTS == 2 ? h : 0];
          to = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(wr, xr, to, 0, 0, 0);
        }
#pragma unroll
      for (int h = 0; h < PARTS; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4& to = acc[r.acc(j, h)];
          to[i] = __builtin_fmaf(part[h][i], sc, to[i]);
        }
    }
  }
};

// Rows in bf16: the down-projection, the codes converted (exactly).  A step is 256 k, whose
// two scales come with one load (as with the 4-bit weights below); the second 128 may lie
// past the end.
struct Fp8Down : Fp8 {
  static constexpr int STEP = 256;
  static constexpr bool SPREAD = true;
  static constexpr int DOWN_DEPTH = 1;
  struct Block {
    u32x4 v[2][2];
    uint32_t s;
  };
  template <int RB, bool JOINED>
  struct Rows : RowsOf<RB, JOINED> {
    Bf16Rows<RB, JOINED> r[2];
    static __device__ __forceinline__ int quarter(int lane) { return Bf16Rows<RB>::quarter(lane); }
  };
  static __device__ __forceinline__ void load(Block& b, const Source& s, uint32_t row0, int k,
                                              int length) {
    const int second = length & buffer_length(2 * k + 1, s.kb);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const buffer w = make_buffer(s.w, o ? second : length);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        in_order(b.v[o][i] = buffer_load16(w, s.lane + i * 64, (row0 * s.kb + 2 * k + o) * 128));
    }
    in_order(buffer_load_to(b.s, make_buffer(s.s, length), odd_lanes() & second & 4,
                            ((row0 >> 7) * s.kb + 2 * k) * 4));
  }
  static __device__ __forceinline__ int odd_lanes() { return -((int)(threadIdx.x >> 4) & 1); }
  static __device__ __forceinline__ uint32_t at(int lane, int quarter) {
    return (lane >> 4) * 32 + (quarter >> 1) * 128 + (quarter & 1) * 16;
  }
  template <int RB, bool JOINED>
  static __device__ __forceinline__ void load_rows(Rows<RB, JOINED>& r, const uint8_t* x0,
                                                   int length,
                                                   const uint32_t (&row)[RowsOf<RB>::BLOCKS],
                                                   int k, int inter) {
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const buffer x =
          make_buffer(x0, o ? length & buffer_length(2 * k + 1, inter / 128) : length);
#pragma unroll
      for (int j = 0; j < RowsOf<RB>::BLOCKS; ++j)
#pragma unroll
        for (int q = 0; q < (RB < 16 ? RB / 4 : 4); ++q)
          in_order(r.r[o].v[4 * j + q] = buffer_load16(x, row[j] + (q >> 1) * 128 + (q & 1) * 16,
                                                       (2 * k + o) * 256));
    }
  }
  static __device__ __forceinline__ bf16x8 values(uint32_t lo, uint32_t hi) {
    const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, 0);
    const bf16x2 q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, 1);
    const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, 0);
    const bf16x2 s = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, 1);
    return bf16x8{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
  }
  template <class R>
  static __device__ __forceinline__ void multiply(f32x4 (&acc)[R::ACCS], const R& r,
                                                  const Block& b) {
    const auto s = __builtin_amdgcn_permlane16_swap(b.s, b.s, false, false);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const float ws = __uint_as_float(s[o]);
      scaled_multiply<4>(
          acc, r.r[o],
          [&](int q) { return values(b.v[o][q >> 1][2 * (q & 1)], b.v[o][q >> 1][2 * (q & 1) + 1]); },
          [&](int) { return ws; });
    }
  }
};

// Packed 4-bit codes: 16 rows x 128 k are one run of 1 KB.  A wave's load is whole lines
// that no other takes, so it goes past the caches' replacement (6.7 TB/s against 6.1; where a
// line is two loads of 64 bytes a row, as with the other weights, it is the other way
// around, 4.3 and 5.5).  The vector memory path takes about 40 clocks a load of a wave,
// however few bytes it brings, and 1 KB of codes is 95 clocks of the memory's rate: so two
// blocks' scales come with one load, the even and the odd 16 lanes each one block's,
// exchanged in registers.
template <class F>
struct W4 {
  static constexpr uint32_t SB = 16 * (128 / F::GROUP) * 2;   // scale bytes of a run
  static constexpr bool PAIR_A_LANE = false;
  static constexpr int UP_DEPTH = 1;
  typedef typename F::word word;
  struct Source {
    const uint8_t *w, *s;
    uint32_t lane, lane_s;
    int odd;                            // all bits in the lanes of the second block
    int kt;                             // runs of a 16-row block
  };
  template <int RB, bool JOINED = false> using Rows = Bf16Rows<RB, JOINED>;
  static __device__ __forceinline__ Source source(const MoeWeights& w, int e, int rows, int k,
                                                  int lane) {
    Source s;
    s.kt = k / 128;
    const size_t run = (size_t)e * (rows / 16) * s.kt;
    s.w = w.w + run * 1024;
    s.s = reinterpret_cast<const uint8_t*>(w.scales) + run * SB;
    s.lane = lane * 16;
    s.lane_s = (lane & 15) * (SB / 16);
    s.odd = -((lane >> 4) & 1);
    return s;
  }
  static __device__ __forceinline__ uint32_t start(const MoeWeights&, int row0, int) {
    return row0 / 16;
  }
  // the scales of the even and of the odd lanes' block, in all lanes
  static __device__ __forceinline__ void both(word v, word& even, word& odd) {
    if constexpr (sizeof(word) == 8) {
      const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32),
                                                       false, false);
      even = (uint64_t)hi[0] << 32 | lo[0];
      odd = (uint64_t)hi[1] << 32 | lo[1];
    } else {
      const auto r = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
      even = (word)r[0];
      odd = (word)r[1];
    }
  }
  static __device__ __forceinline__ uint32_t at(int lane, int quarter) {
    return Bf16::at(lane, quarter);
  }
  template <int RB>
  static __device__ __forceinline__ void load_rows(Bf16Rows<RB>& r, const uint8_t* x, int length,
                                                   const uint32_t (&row)[RowsOf<RB>::BLOCKS],
                                                   int kt, int) {
    Bf16::load_rows(r, x, length, row, kt, 0);
  }
  template <class R>
  static __device__ __forceinline__ void multiply_block(f32x4 (&acc)[R::ACCS], const R& r,
                                                        const u32x4& v, word s) {
    constexpr int QPS = F::GROUP / 32;
    scaled_multiply<QPS>(
        acc, r, [&](int q) { return decode8<F::CODES>(v[q]); },
        [&](int q) { return F::scale((uint16_t)(s >> (16 * (q / QPS)))); });
  }
};

template <class F>
struct TwoBlocks<W4<F>> {
  typedef W4<F> P;
  u32x4 g, u;
  typename P::word s;
  __device__ __forceinline__ void load(const typename P::Source& src, uint32_t gate, uint32_t up,
                                       int kt, int length) {
    const uint32_t rg = gate * src.kt + kt, ru = up * src.kt + kt;
    in_order(g = buffer_load16_nt(make_buffer(src.w, length), src.lane, rg * 1024));
    in_order(u = buffer_load16_nt(make_buffer(src.w, length), src.lane, ru * 1024));
    in_order(buffer_load_to(s, make_buffer(src.s, length),
                            src.lane_s + (src.odd & (int)((ru - rg) * P::SB)), rg * P::SB));
  }
  template <class Rows>
  __device__ __forceinline__ void multiply(f32x4 (&ag)[Rows::ACCS], f32x4 (&au)[Rows::ACCS],
                                           const Rows& r) const {
    typename P::word sg, su;
    P::both(s, sg, su);
    P::multiply_block(ag, r, g, sg);
    P::multiply_block(au, r, u, su);
  }
};

// The same for the down-projection, where the two blocks are two consecutive 128 k of a row
// block, of which the second may lie past the end.
template <class F>
struct W4Down : W4<F> {
  typedef W4<F> P;
  typedef typename P::word word;
  typedef typename P::Source Source;
  static constexpr int DOWN_DEPTH = 1;
  static constexpr int STEP = 256;
  static constexpr bool SPREAD = false;
  struct Block {
    u32x4 v[2];
    word s;
  };
  template <int RB, bool JOINED>
  struct Rows : RowsOf<RB, JOINED> {
    Bf16Rows<RB, JOINED> r[2];
    static __device__ __forceinline__ int quarter(int lane) { return Bf16Rows<RB>::quarter(lane); }
  };
  static __device__ __forceinline__ void load(Block& b, const Source& s, uint32_t start, int k,
                                              int length) {
    const uint32_t run = start * s.kt + 2 * k;
    const int second = length & buffer_length(2 * k + 1, s.kt);
    in_order(b.v[0] = buffer_load16_nt(make_buffer(s.w, length), s.lane, run * 1024));
    in_order(b.v[1] = buffer_load16_nt(make_buffer(s.w, second), s.lane, run * 1024 + 1024));
    in_order(buffer_load_to(b.s, make_buffer(s.s, length),
                            s.lane_s + (s.odd & second & (int)P::SB), run * P::SB));
  }
  template <int RB, bool JOINED>
  static __device__ __forceinline__ void load_rows(Rows<RB, JOINED>& r, const uint8_t* x,
                                                   int length,
                                                   const uint32_t (&row)[RowsOf<RB>::BLOCKS],
                                                   int k, int inter) {
    Bf16::load_rows(r.r[0], x, length, row, 2 * k, 0);
    Bf16::load_rows(r.r[1], x, length & buffer_length(2 * k + 1, inter / 128), row, 2 * k + 1, 0);
  }
  template <class R>
  static __device__ __forceinline__ void multiply(f32x4 (&acc)[R::ACCS], const R& r,
                                                  const Block& b) {
    word s0, s1;
    P::both(b.s, s0, s1);
    P::multiply_block(acc, r.r[0], b.v[0], s0);
    P::multiply_block(acc, r.r[1], b.v[1], s1);
  }
};

// Waits for this wave's LDS accesses, then for the workgroup; loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);                // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A hidden value, as the down-projection multiplies it: in two bf16 parts, the second what
// the first's rounding leaves (off by 2^-17 of the value at most), in two rows of the
// workspace.  What is not finite has the first alone.
__device__ __forceinline__ void store_hidden(const MoeArgs& a, int pair, int n, float v) {
  const __bf16 hi = (__bf16)v;
  const float rest = __builtin_isfinite((float)hi) ? v - (float)hi : 0.f;
  __bf16* h = reinterpret_cast<__bf16*>(a.h) + (size_t)pair * 2 * a.inter + n;
  h[0] = hi;
  h[a.inter] = (__bf16)rest;
}

// ---- Up-projection and SwiGLU.  An item is a segment and 16 outputs: 16 gate rows and the 16
// up rows of W1, whose K the waves split: a wave takes every eighth step, so that the
// workgroup's reads of a row are one run.  The loads of the next item's first steps are
// on their way while an item's sums are joined.
template <class P, int RB>
__device__ __forceinline__ void up_items(const MoeArgs& a, const Table& s, int seg0, int seg1,
                                         f32x4 (*s_part)[kWaves][2][RowsOf<RB>::BLOCKS][64]) {
  constexpr int BLOCKS = RowsOf<RB>::BLOCKS, ACCS = RowsOf<RB>::ACCS, BUFS = 2 / BLOCKS;
  constexpr int DEPTH = P::UP_DEPTH;
  typedef typename P::template Rows<RB> Rows;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int KT = a.hidden / 128, per = a.inter / 16;
  const int items = (seg1 - seg0) * per;
  struct Step {
    TwoBlocks<P> w;
    Rows r;
  };
  struct Place {
    int item, k;
    decltype(P::source(a.w1, 0, 0, 0, 0)) src;
    uint32_t gate, up, row[BLOCKS], scale_at[BLOCKS];
  };
  auto enter = [&](Place& p) {
    const int item = min(p.item, items - 1), seg = seg0 + item / per, b = item % per;
    const int e = __builtin_amdgcn_readfirstlane(s.seg_expert[seg]);
    const int pair = __builtin_amdgcn_readfirstlane(s.seg_pair[seg]);
    const int n = __builtin_amdgcn_readfirstlane(s.seg_pairs[seg]);
    p.src = P::source(a.w1, e, 2 * a.inter, a.hidden, lane);
    p.gate = P::start(a.w1, b * 16, a.hidden);
    p.up = P::start(a.w1, a.inter + b * 16, a.hidden);
    // rows past the segment's last repeat it; their results are not stored
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j) {
      const int t = s.token[pair + min(j * 16 + (lane & 15) % RB, n - 1)];
      p.row[j] = (uint32_t)t * (uint32_t)a.hidden * (P::PAIR_A_LANE ? 1 : 2) +
                 P::at(lane, Rows::quarter(lane));
      p.scale_at[j] = t * KT * 4;
    }
  };
  // Loads ahead are unconditional, past the end of an empty buffer: with one under a
  // condition the compiler would wait for all that are in flight.
  auto load = [&](Step& st, Place& p) {
    const int length = buffer_length(p.item, items) & buffer_length(p.k, KT);
    st.w.load(p.src, p.gate, p.up, p.k, length);
    P::load_rows(st.r, a.x, length, p.row, p.k, a.hidden);
    if constexpr (P::PAIR_A_LANE)
#pragma unroll
      for (int j = 0; j < BLOCKS; ++j)
        in_order(buffer_load_to(st.r.s[j], make_buffer(a.x_scale, length), p.scale_at[j], p.k * 4));
    p.k += kWaves;
    if (p.k >= KT) {
      p.k = wave;
      p.item += gridDim.x;
      enter(p);
    }
  };
  int item = blockIdx.x, k = wave, buf = 0;
  if (item >= items) return;
  f32x4 ag[ACCS] = {}, au[ACCS] = {};
  Place ahead;
  ahead.item = item;
  ahead.k = k;
  enter(ahead);
  Step st[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(st[d], ahead);
  while (item < items) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      // (a wave without a step of its own multiplies the empty buffer's zeros)
      st[d].w.multiply(ag, au, st[d].r);
      __builtin_amdgcn_sched_barrier(0);
      load(st[d], ahead);
      k += kWaves;
      if (k >= KT) {
        auto& part = s_part[buf];
        if constexpr (RB >= 16) {
#pragma unroll
          for (int j = 0; j < BLOCKS; ++j) {
            part[wave][0][j][lane] = ag[j];
            part[wave][1][j][lane] = au[j];
          }
        } else if constexpr (P::PAIR_A_LANE) {
          // a pair's two halves of k lie eight lanes apart
          f32x4 g, u;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g[i] = (lane & 8) ? ag[1][i] : ag[0][i];
            u[i] = (lane & 8) ? au[1][i] : au[0][i];
            g[i] += __shfl_xor(g[i], 8);
            u[i] += __shfl_xor(u[i], 8);
          }
          part[wave][0][0][lane] = g;
          part[wave][1][0][lane] = u;
        } else {
          part[wave][0][0][lane] = add_row_parts<RB>(ag, lane);
          part[wave][1][0][lane] = add_row_parts<RB>(au, lane);
        }
#pragma unroll
        for (int j = 0; j < ACCS; ++j) ag[j] = au[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        lds_barrier();
        const int seg = seg0 + item / per, b = item % per;
        const int pair = s.seg_pair[seg], n = s.seg_pairs[seg];
        // one value a thread: a pair's row and an output
        const int j = tid >> 8, l = (tid >> 2) & 63, i = tid & 3;
        const int r = j * 16 + (P::PAIR_A_LANE ? l & 15 : (l >> 4) * 4 + i);
        const int c = P::PAIR_A_LANE ? (l >> 4) * 4 + i : l & 15;
        if (j < BLOCKS && r < n) {
          float g = 0.f, u = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            g += part[w][0][j][l][i];
            u += part[w][1][j][l][i];
          }
          store_hidden(a, pair + r, b * 16 + c, g / (1.f + expf(-g)) * u);
        }
        // one barrier an item: the next one's sums go to the other buffer, if there is one
        if constexpr (BUFS == 1) lds_barrier();
        buf ^= BUFS - 1;
        k = wave;
        item += gridDim.x;
      }
      if (item >= items) break;
    }
  }
}

template <class P>
__global__ __launch_bounds__(kThreads, 4) void moe_up_kernel(MoeArgs a) {
  __shared__ Table s;
  __shared__ f32x4 s_part[1][kWaves][2][2][64];
  build_table<32, 8, 8>(a, s);
  const int few = __builtin_amdgcn_readfirstlane(s.few);
  const int segments = __builtin_amdgcn_readfirstlane(s.segments);
  typedef f32x4 (*OneBlock)[kWaves][2][1][64];
  const OneBlock part = reinterpret_cast<OneBlock>(s_part);
  if (few > 0) {
    if (!P::PAIR_A_LANE && !__builtin_amdgcn_readfirstlane(s.over_half))
      up_items<P, P::PAIR_A_LANE ? 8 : 4>(a, s, 0, few, part);
    else
      up_items<P, 8>(a, s, 0, few, part);
  }
  if (few < segments) {
    __syncthreads();       // the sums of the last item are read
    if (!__builtin_amdgcn_readfirstlane(s.over16))
      up_items<P, 16>(a, s, few, segments, part);
    else
      up_items<P, 32>(a, s, few, segments, s_part);
  }
}

// ---- Down-projection and the weighted sum.  A workgroup takes 16 columns of the output; the
// steps of all segments are one run that the waves split evenly.  A wave adds what it has of
// a segment, times the pairs' weights, to its own sums of the tokens in LDS.
// A pair is two rows, the parts of its h: of RB rows the first half are the first parts, and
// with 32 rows a row block each, joined in one accumulator.  Three classes of experts, of up
// to 4 pairs (8 rows, or 4 where none has over 2), up to 8 (16) and more (32): us of the
// down-projection of 64 tokens in e2m1 and of 16 in bf16 (2 pairs an expert on average)
//   classes up to 4, 8 and more   61.4 and 26.3     up to 8 and more        67.9 and 26.3
//   up to 2, 8 and more           60.3 and 27.0     up to 2, 4, 8 and more  59.5 and 27.2
// (a class more is a start of the loads more, a class less are rows that most experts lack).
// The segments are of at most 16 pairs: an expert's weights are read again for its next 16,
// by the same workgroup (where its waves take runs of the steps, by another wave of it).
template <class P, int RB>
__device__ __forceinline__ void down_steps(const MoeArgs& a, const Table& s, int seg0, int seg1,
                                           const float* weight, float (*s_out)[16], int b, int wave,
                                           int lane) {
  constexpr bool JOINED = RB > 16;
  typedef typename P::template Rows<RB, JOINED> Rows;
  constexpr int BLOCKS = Rows::BLOCKS, PAIRS = RB / 2;
  const int KT = (a.inter + P::STEP - 1) / P::STEP;     // steps
  constexpr int DEPTH = P::DOWN_DEPTH;
  const uint32_t start = P::start(a.w2, b * 16, a.inter);
  struct Step {
    typename P::Block w;
    Rows r;
  };
  // A wave takes `count` of the steps of all segments, every eighth or a run of them.
  const int steps = (seg1 - seg0) * KT;
  const int begin = P::SPREAD ? wave : wave * steps / kWaves;
  const int count = P::SPREAD ? (steps - wave + kWaves - 1) / kWaves
                              : (wave + 1) * steps / kWaves - begin;
  constexpr int STRIDE = P::SPREAD ? kWaves : 1;
  const int whole = STRIDE / KT, rest = STRIDE % KT;
  // moves on; true if that left the segment
  auto move = [&](int& seg, int& k) {
    const int was = seg, over = k + rest >= KT;
    seg += whole + over;
    k += rest - over * KT;
    return seg != was;
  };
  // Where the loads are.  What belongs to the segment is looked up when it is entered.
  struct Place {
    int seg, k, at;
    decltype(P::source(a.w2, 0, 0, 0, 0)) src;
    uint32_t row[BLOCKS];
  };
  auto enter = [&](Place& p) {
    const int seg = min(p.seg, seg1 - 1);
    const int e = __builtin_amdgcn_readfirstlane(s.seg_expert[seg]);
    const int pair = __builtin_amdgcn_readfirstlane(s.seg_pair[seg]);
    const int n = __builtin_amdgcn_readfirstlane(s.seg_pairs[seg]);
    p.src = P::source(a.w2, e, a.hidden, a.inter, lane);
    const int r = (lane & 15) % RB;
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j)
      p.row[j] = (uint32_t)(2 * (pair + min(r % PAIRS, n - 1)) + (JOINED ? j : r / PAIRS)) *
                     (uint32_t)a.inter * 2 +
                 P::at(lane, Rows::quarter(lane));
  };
  auto load = [&](Step& st, Place& p) {
    const int length = buffer_length(p.at++, count);
    P::load(st.w, p.src, start, p.k, length);
    P::load_rows(st.r, a.h, length, p.row, p.k, a.inter);
    if (move(p.seg, p.k)) enter(p);
  };
  if (count <= 0) return;
  f32x4 acc[Rows::ACCS] = {};
  Step st[DEPTH];
  int seg = seg0 + begin / KT, k = begin % KT;
  Place ahead;
  ahead.seg = seg;
  ahead.k = k;
  ahead.at = 0;
  enter(ahead);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(st[d], ahead);
  for (int at = 0; at < count;) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      P::multiply(acc, st[d].r, st[d].w);
      __builtin_amdgcn_sched_barrier(0);
      load(st[d], ahead);
      const int was = seg;
      if (move(seg, k) || at + 1 >= count) {
        const int pair = s.seg_pair[was], n = s.seg_pairs[was];
        f32x4 v;
        if constexpr (RB < 16)
          v = add_row_parts<RB>(acc, lane);
        else
          v = acc[0];
        // the two parts' rows, 2, 4 or 8 apart
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (RB == 4) v[i] += v[(i + 2) & 3];
          if constexpr (RB == 8) v[i] = add_quarters(v[i]);
          if constexpr (RB == 16) v[i] = add_halves(v[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (lane >> 4) * 4 + i;
          if (r < n) s_out[s.token[pair + r]][lane & 15] += weight[pair + r] * v[i];
        }
#pragma unroll
        for (int j = 0; j < Rows::ACCS; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      if (++at >= count) break;
    }
  }
}

template <class P>
__global__ __launch_bounds__(kThreads, 4) void moe_down_kernel(MoeArgs a) {
  __shared__ Table s;
  __shared__ Weights weights;
  __shared__ float s_out[kWaves][kMoeTokens][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = lane; i < a.tokens * 16; i += 64) s_out[wave][i >> 4][i & 15] = 0.f;
  build_table<16, 4, 8>(a, s, &weights);
  const int b = blockIdx.x;
  const int few = __builtin_amdgcn_readfirstlane(s.few);
  const int segments = __builtin_amdgcn_readfirstlane(s.segments);
  const int mid = __builtin_amdgcn_readfirstlane(s.mid);
  float(*out)[16] = s_out[wave];
  if (few > 0) {
    if (!__builtin_amdgcn_readfirstlane(s.over_half))
      down_steps<P, 4>(a, s, 0, few, weights.pair, out, b, wave, lane);
    else
      down_steps<P, 8>(a, s, 0, few, weights.pair, out, b, wave, lane);
  }
  if (few < mid) down_steps<P, 16>(a, s, few, mid, weights.pair, out, b, wave, lane);
  if (mid < segments) down_steps<P, 32>(a, s, mid, segments, weights.pair, out, b, wave, lane);
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

template <int CODES, int GROUP>
void launch_w4(const MoeArgs& a, bool up, bool f16, int num_cus, hipStream_t st) {
  typedef Format<CODES, GROUP, true> Half;
  typedef Format<CODES, GROUP, false> Bf;
  if (f16)
    up ? launch_up<W4<Half>>(a, num_cus, st) : launch_down<W4Down<Half>>(a, st);
  else
    up ? launch_up<W4<Bf>>(a, num_cus, st) : launch_down<W4Down<Bf>>(a, st);
}

hipError_t launch_product_of(const MoeArgs& a, const MoeWeights& w, bool up, int num_cus,
                             hipStream_t st) {
  if (w.group == 0) {
    if (!a.fp8)
      up ? launch_up<Bf16>(a, num_cus, st) : launch_down<Bf16>(a, st);
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
