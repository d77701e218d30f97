// Routing to experts: scores, the group limit, top-k picks and their weights for
// every token, and the gradient of the weights with respect to the logits.
// LPT lanes per token, 64 or, where there are many tokens, 16 (four tokens a wave; up to
// 256 experts, 16 groups and 16 picks); lane L of them holds VPL consecutive experts from
// L * VPL, so that the lowest lane holds the lowest index of a tie.
//
// Which experts are picked is exact.  Without a bias the choice is the order of the
// logits themselves.  Where a score is compared (a bias, a sum of two) it is defined in
// binary64, but computed in binary32 first with a bound on the error: only a token in
// which two choices next to each other, or the groups at the limit, lie within that
// bound is chosen again in binary64: in the same kernel where tokens are few, in a second
// one where they are many, since the registers of the binary64 path would leave the first
// kernel two waves a SIMD.  That is a few tokens of a thousand where the biases are of the
// scores' size.  It is every token where one finite bias is huge, since the bound grows with
// the largest sum of the token, pickable or not (32768 tokens, one bias of -1e9: 125 us, of
// -infinity 28), and many where groups are ranked by sums without a bias: then picks, though
// by logits, must lie a score's bound apart as well (bf16 logits, of which many are equal:
// 89 us, binary32 32).
// A pick: the largest key of every lane, the largest of the token by cross-lane moves,
// the lowest lane that has it from a ballot's lowest bit.  That is about 85 vector
// instructions whatever LPT is, so four tokens share them where they fit; biased choices
// of many tokens come from sorted lists instead (take_heads).
//
// What it measured: 32768 tokens of 256 experts in 8 groups (sigmoid, bias, top-2 group sums,
// fp32 logits) 22 us and 7 us for the second kernel, where a copy of the same bytes takes
// 6.0: bound by vector instructions, 1030 a wave of four tokens (1770 and 31 us with
// pick() alone).  8192 tokens of 128 experts 6.2 us, one token 5.2 us, of which most is
// the latency of a launch.
//
// The weights are binary32.  Renormalised softmax weights are a softmax over the
// picked logits; renormalised sigmoid weights use
//   s_k = e^min(l_k, 0) / (1 + e^-|l_k|),
// whose numerators can be scaled by e^-max_j min(l_j, 0) before the division, so
// neither form divides 0 by 0 when all scores are tiny.
#include <cfloat>

#include "ep_combine.h"
#include "ep_kernels.h"

namespace ep {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;

// A missing expert (NaN, -infinity) is -infinity; +infinity the largest number: the median
// of those two and a logit, which for a quiet NaN is the least of the others (written
// out, because the compiler drops the -infinity).
__device__ __forceinline__ float clean(float v) {
  v = __builtin_canonicalizef(v);
  asm("v_med3_f32 %0, %0, %1, %2" : "+v"(v) : "s"(-INFINITY), "v"(FLT_MAX));
  return v;
}

// A lane's first expert, as a value that the compiler does not follow: bounds and
// quotients of rare paths would otherwise be computed for every token.
__device__ __forceinline__ int opaque(int first) {
  asm volatile("" : "+v"(first));
  return first;
}

__device__ __forceinline__ float f16_value(uint32_t v) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t i) {
  if (a.dtype == EP_LOGITS_F32) return clean(reinterpret_cast<const float*>(a.logits)[i]);
  const uint16_t h = reinterpret_cast<const uint16_t*>(a.logits)[i];
  return clean(a.dtype == EP_LOGITS_BF16 ? bf16_lo(h) : f16_value(h));
}

// Logits of experts lane * VPL + 0..VPL-1 of token t, -infinity past the last.  Rows of
// a multiple of VPL experts start where a lane's values can be loaded together.
template <int VPL>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t t, int lane, float (&x)[VPL]) {
  const int E = a.n_experts, first = lane * VPL;
  const int64_t at = t * E + first;
  if (E % VPL == 0) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = -INFINITY;
    if (first >= E) return;
    if (a.dtype == EP_LOGITS_F32) {
      const float* p = reinterpret_cast<const float*>(a.logits) + at;
#pragma unroll
      for (int j = 0; j < VPL / 4; ++j) {
        const u32x4 v = load16(p + 4 * j);
#pragma unroll
        for (int q = 0; q < 4; ++q) x[4 * j + q] = clean(__uint_as_float(v[q]));
      }
    } else {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(
          reinterpret_cast<const uint16_t*>(a.logits) + at);
      uint32_t v[VPL / 2];
#pragma unroll
      for (int j = 0; j < VPL / 2; ++j) v[j] = p[j];
      if (a.dtype == EP_LOGITS_BF16) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) x[j] = clean(j & 1 ? bf16_hi(v[j / 2]) : bf16_lo(v[j / 2]));
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) x[j] = clean(f16_value(v[j / 2] >> (16 * (j & 1)) & 0xffffu));
      }
    }
    return;
  }
  const int i = opaque(first);
#pragma unroll
  for (int j = 0; j < VPL; ++j) x[j] = i + j < E ? load_logit(a, at + j) : -INFINITY;
}

template <int VPL>
__device__ __forceinline__ void store_row(const RouteArgs& a, int64_t t, int lane,
                                          const float (&v)[VPL]) {
  const int E = a.n_experts, first = lane * VPL;
  const int64_t at = t * E + first;
  if (first >= E) return;
  if (E % VPL == 0) {
    if (a.dtype == EP_LOGITS_F32) {
      float* p = reinterpret_cast<float*>(a.grad_logits) + at;
#pragma unroll
      for (int j = 0; j < VPL / 4; ++j) {
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = __float_as_uint(v[4 * j + q]);
        store16_nt(p + 4 * j, o);
      }
    } else {
      uint32_t* p = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.grad_logits) + at);
#pragma unroll
      for (int j = 0; j < VPL / 2; ++j) {
        if (a.dtype == EP_LOGITS_BF16) {
          p[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        } else {
          const uint16_t lo = __builtin_bit_cast(uint16_t, (_Float16)v[2 * j]);
          const uint16_t hi = __builtin_bit_cast(uint16_t, (_Float16)v[2 * j + 1]);
          p[j] = (uint32_t)lo | (uint32_t)hi << 16;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (first + j < E) {
      if (a.dtype == EP_LOGITS_F32)
        reinterpret_cast<float*>(a.grad_logits)[at + j] = v[j];
      else if (a.dtype == EP_LOGITS_BF16)
        reinterpret_cast<__bf16*>(a.grad_logits)[at + j] = (__bf16)v[j];
      else
        reinterpret_cast<_Float16*>(a.grad_logits)[at + j] = (_Float16)v[j];
    }
}

// v from the lane that the data-parallel move CTRL names, `old` where there is none.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float lane_move(float old, float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v),
                                         CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float read_lane(float v, int lane) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Reductions over the LPT lanes of a token, the same result in each of them: 16 lanes are
// a row of the data-parallel moves, reduced by rotations; 64 by shifts within the rows,
// rows 0 and 2 into 1 and 3, the lower half into the upper, and its last lane.
// (The maxima are written out: fmaxf() of a moved value takes a move, a quieting of
// NaNs, which do not occur here, and the maximum; s_nop covers the wait that such a move
// needs after its operand is written.)
#define EP_MAX_MOVE(V, CTRL) \
  asm("s_nop 1\n\tv_max_f32_dpp %0, %0, %0 " CTRL " bank_mask:0xf" : "+v"(V))
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (LPT == 16) {
    EP_MAX_MOVE(v, "row_ror:8 row_mask:0xf");
    EP_MAX_MOVE(v, "row_ror:4 row_mask:0xf");
    EP_MAX_MOVE(v, "row_ror:2 row_mask:0xf");
    EP_MAX_MOVE(v, "row_ror:1 row_mask:0xf");
    return v;
  } else {
    EP_MAX_MOVE(v, "row_shr:1 row_mask:0xf");
    EP_MAX_MOVE(v, "row_shr:2 row_mask:0xf");
    EP_MAX_MOVE(v, "row_shr:4 row_mask:0xf");
    EP_MAX_MOVE(v, "row_shr:8 row_mask:0xf");
    EP_MAX_MOVE(v, "row_bcast:15 row_mask:0xa");
    EP_MAX_MOVE(v, "row_bcast:31 row_mask:0xc");
    return read_lane(v, 63);
  }
}
#undef EP_MAX_MOVE
template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LPT == 16) {
    v += lane_move<0x128>(0.f, v);
    v += lane_move<0x124>(0.f, v);
    v += lane_move<0x122>(0.f, v);
    return v + lane_move<0x121>(0.f, v);
  } else {
    v += lane_move<0x111>(0.f, v);
    v += lane_move<0x112>(0.f, v);
    v += lane_move<0x114>(0.f, v);
    v += lane_move<0x118>(0.f, v);
    v += lane_move<0x142, 0xa>(0.f, v);
    v += lane_move<0x143, 0xc>(0.f, v);
    return read_lane(v, 63);
  }
}
template <int LPT>
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int d = LPT / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
// Binary64 keys hold no NaN.
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return a < b ? a : b; }
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double max_move(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int lo = (int)u, hi = (int)(u >> 32);
  const uint32_t l = __builtin_amdgcn_update_dpp(lo, lo, CTRL, ROWS, 0xf, false);
  const uint32_t h = __builtin_amdgcn_update_dpp(hi, hi, CTRL, ROWS, 0xf, false);
  return larger(v, __builtin_bit_cast(double, (uint64_t)h << 32 | l));
}
__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t l = __builtin_amdgcn_readlane((int)u, lane);
  const uint32_t h = __builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}
template <int LPT>
__device__ __forceinline__ double lanes_max(double v) {
  static_assert(LPT == 64, "binary64 choices take a wave per token");
  v = max_move<0x111>(v);
  v = max_move<0x112>(v);
  v = max_move<0x114>(v);
  v = max_move<0x118>(v);
  v = max_move<0x142, 0xa>(v);
  v = max_move<0x143, 0xc>(v);
  return read_lane(v, 63);
}
// v of lane `from` of the token's lanes.
template <int LPT, class T>
__device__ __forceinline__ T of_lane(T v, int from) {
  if constexpr (LPT == 16) return __shfl(v, (int)(threadIdx.x & 48) + from);
  else return read_lane(v, from);
}
// Whether this is the lowest lane of its token for which `is` holds (it holds for one
// at least in each token of the wave).
template <int LPT>
__device__ __forceinline__ bool lowest_lane(bool is) {
  const uint64_t m = __ballot(is);
  // the lowest bit of each 16 (a nonzero field's ~m + 1 does not carry), or of all
  const uint64_t low = m & (~m + (LPT == 16 ? 0x0001000100010001ull : 1ull));
  return low >> (threadIdx.x & 63) & 1;
}

// e^x for x <= 88 within 2 * 2^-23 of itself (0 below 2^-126): 2^t for t = x log2(e)
// rounded, times 1 + the rounding's part.
__device__ __forceinline__ float exp_near(float x) {
  x = fmaxf(x, -200.f);
  const float t = x * 0x1.715476p0f;                       // log2(e) to 24 bits
  const float r = __builtin_fmaf(x, 0x1.4ae0cp-26f, __builtin_fmaf(x, 0x1.715476p0f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e * r, 0x1.62e43p-1f, e);          // ln 2
}

// Shares of the picks, lane k holding pick k's logit l (there: lane k has a pick):
// softmax over the picks, or their sigmoids over the sum.  The division is a rounded one, so
// that the share of a single pick is 1 and its gradient 0.
template <int LPT>
__device__ __forceinline__ float pick_share(float l, bool there, int score) {
  const float low = score == EP_SCORE_SIGMOID ? fminf(l, 0.f) : l;
  const float top = lanes_max<LPT>(there ? low : -FLT_MAX);
  float e = there ? exp_near(low - top) : 0.f;
  if (score == EP_SCORE_SIGMOID) e *= __builtin_amdgcn_rcpf(1.f + exp_near(-fabsf(l)));
  const float sum = lanes_sum<LPT>(e);
  return there ? e / sum : 0.f;
}

// Bias of the lane's experts, 0 without one (an expert that it keeps out: NaN or -infinity).
template <int VPL>
__device__ __forceinline__ void load_bias(const RouteArgs& a, int lane, float (&b)[VPL]) {
  const int first = lane * VPL;
#pragma unroll
  for (int j = 0; j < VPL; ++j) b[j] = 0.f;
  if (!a.bias) return;
  if (a.n_experts % VPL == 0 && (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0) {
    if (first < a.n_experts) {
#pragma unroll
      for (int j = 0; j < VPL / 4; ++j) {
        const u32x4 v = load16(a.bias + first + 4 * j);
#pragma unroll
        for (int q = 0; q < 4; ++q) b[4 * j + q] = __uint_as_float(v[q]);
      }
    }
  } else {
    const int i = opaque(first);
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (i + j < a.n_experts) b[j] = a.bias[i + j];
  }
}

// Bounds on the error of a binary32 score plus bias, over 1 + the largest such sum of the
// token.  The exponential's argument d, within 2.5 |d| 2^-24, is rounded, 2^d is within
// 2^-23 of itself: in a softmax score s that is within s (2.5 |d| + 2 + 25) 2^-24 <=
// 28 * 2^-24 (a sum of at most 16 + 6 additions and the division), in a sigmoid within
// s (1 - s) (2.5 |d| + 2) + 3 s <= 5 times 2^-24 (the addition, the reciprocal); the bias
// adds one rounding of the sum.
__device__ __forceinline__ float choice_error(int score) {
  return score == EP_SCORE_SOFTMAX ? 0x1p-19f : 0x1p-21f;
}

// Takes the experts outside the topk_groups best groups out of a token's choices `key`.
// score: scores plus bias; both -infinity for what cannot be picked, and each within
// `error` unless `exact`.  Returns whether the groups at the limit lie further apart than that.
// lanes: lanes of a group where that is a power of two of whole lanes, 0: no groups,
// -1: groups of any other size.
template <int LPT, int VPL, class T>
__device__ __forceinline__ bool limit_groups(const RouteArgs& a, int lane, T (&key)[VPL],
                                             const T (&score)[VPL], bool exact, float error,
                                             int lanes) {
  constexpr T none = -INFINITY;
  bool sure = true;
  if (lanes != 0) {
    const bool top2 = a.group_score == EP_GROUP_TOP2;
    const int per = a.n_experts / a.n_groups;
    // the two largest of this lane's group (lanes > 0), or of group `lane`
    T v1 = none, v2 = none, by[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) by[j] = top2 ? score[j] : key[j];
    if (lanes > 0) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        v2 = larger(v2, smaller(v1, by[j]));
        v1 = larger(v1, by[j]);
      }
      for (int d = 1; d < lanes; d <<= 1) {
        const T o1 = __shfl_xor(v1, d), o2 = __shfl_xor(v2, d);
        v2 = larger(smaller(v1, o1), larger(v2, o2));
        v1 = larger(v1, o1);
      }
    } else {
      const int first = opaque(lane * VPL);
      for (int g = 0; g < a.n_groups; ++g) {
        T w1 = none, w2 = none;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int i = first + j - g * per;
          const T y = i < 0 || i >= per ? none : by[j];
          w2 = larger(w2, smaller(w1, y));
          w1 = larger(w1, y);
        }
        const T m1 = lanes_max<LPT>(w1);
        T m2 = none;
        // the second: the lane that has the first gives its second, the others their first
        if (top2) m2 = lanes_max<LPT>(lowest_lane<LPT>(w1 == m1) ? w2 : w1);
        if (lane == g) {
          v1 = m1;
          v2 = m2;
        }
      }
    }
    T value = v1;
    if (top2 && v2 > none) {
      value += v2;
      // a binary32 sum past the range is not that of a group without experts: kept finite, it
      // lies within the error of the others past the range, which are told apart in binary64
      if (!exact) value = larger(value, (T)-FLT_MAX);
    }
    const int step = lanes > 0 ? lanes : 1, g = lane / step;
    int above = 0;                             // groups that come before this one
    for (int o = 0; o < a.n_groups; ++o) {
      const T v = of_lane<LPT>(value, o * step);
      above += v > value || (v == value && o < g);
    }
    const bool mine = g < a.n_groups;
    const bool keep = mine && above < a.topk_groups;
    if (!exact && a.topk_groups < a.n_groups) {
      const T in = -lanes_max<LPT>(keep ? -value : none);        // the last kept
      const T out = lanes_max<LPT>(mine && !keep ? value : none);
      // (infinite values: a group without experts, a bias of +infinity)
      if (!(in - out > 4.f * error)) sure = out == none;
    }
    if (lanes > 0) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = keep ? key[j] : none;
    } else {
      const uint64_t kept = __ballot(keep) >> (LPT == 16 ? threadIdx.x & 48 : 0);   // by group
      const int first = opaque(lane * VPL);
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = kept >> min((first + j) / per, 63) & 1 ? key[j] : none;
    }
  }
  return sure;
}

// The picks of one token, lane k's id (or -1) in lane k.  key: the choices, within `error`
// unless `exact`.  Returns whether none that decide lie within their error of each other.
template <int LPT, int VPL, class T>
__device__ __forceinline__ bool pick(const RouteArgs& a, int lane, T (&key)[VPL], bool exact,
                                     float error, int& id) {
  constexpr T none = -INFINITY;
  bool sure = true;
  T before = INFINITY;
  id = -1;
  // one more pick than asked for, to see how near it comes
  const int picks = a.top_k + (exact ? 0 : 1);
  for (int k = 0; k < picks; ++k) {
    T best = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = larger(best, key[j]);
    const T m = lanes_max<LPT>(best);
    if (!exact && k > 0 && m > none && !(before - m > 2.f * error)) sure = false;
    before = m;
    if (k == a.top_k) break;
    // the winning lane, and the first of its keys that is m
    const bool win = lowest_lane<LPT>(best == m);
    bool open = win;
    int at = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const bool is = open && key[j] == m;
      open = open && !is;
      at = is ? j : at;
      key[j] = is ? none : key[j];
    }
    // from the one lane that has it to lane k
    const float picked = lanes_max<LPT>(win ? (float)(lane * VPL + at) : -1.f);
    if (lane == k && m > none) id = (int)picked;
  }
  return sure;
}

// Batcher's odd-even merge sort of N values as a list of the pairs it compares.
template <int N>
struct SortingNetwork {
  int a[64] = {}, b[64] = {}, size = 0;
  constexpr SortingNetwork() {
    for (int p = 1; p < N; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < N; j += 2 * k)
          for (int i = j; i < j + k && i + k < N; ++i)
            if (i / (2 * p) == (i + k) / (2 * p)) {
              a[size] = i;
              b[size++] = i + k;
            }
  }
};

// pick() for biased scores, 16 lanes a token: choices as integers of 2^-24 with their place
// among the lane's VPL in the low four bits, sorted within the lane first, so that a
// pick is the largest head of 16 lists and a step of the list that had it, about 25
// vector instructions instead of 85.  The integers hold choices below 8 in magnitude,
// others are left to pick().  Equal ones of two lanes step together, which the count of
// steps shows.
// L: entries of a list that matter to so many picks.
constexpr float kSortedBelow = 7.9f;
template <int L, int VPL>
__device__ __forceinline__ bool take_heads(const int (&list)[VPL], int picks, int wanted, int lane,
                                           uint32_t apart, int* ids, int& found) {
  constexpr int none = -0x7fffffff - 1 + 16;   // below: no choice
  int head[L];
#pragma unroll
  for (int i = 0; i < L; ++i) head[i] = list[i];
  bool sure = true;
  int before = 0, steps = 0;
  found = 0;
  for (int k = 0; k < picks; ++k) {
    int m = head[0];
    asm("s_nop 1\n\tv_max_i32_dpp %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_i32_dpp %0, %0, %0 row_ror:4 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_i32_dpp %0, %0, %0 row_ror:2 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_i32_dpp %0, %0, %0 row_ror:1 row_mask:0xf bank_mask:0xf" : "+v"(m));
    const bool is = m >= none;
    if (k > 0 && is && !((uint32_t)before - (uint32_t)m > apart)) sure = false;
    before = m;
    found += is;
    const bool win = is && head[0] == m;
    if (k < wanted && win) ids[k] = lane * VPL + (m & 15);
    // by a mask: of a condition the compiler makes a variable index into the list
    const int step = win ? -1 : 0;
    steps -= step;
#pragma unroll
    for (int i = 0; i + 1 < L; ++i) head[i] = (step & head[i + 1]) | (~step & head[i]);
    head[L - 1] = (step & (none - 16)) | (~step & head[L - 1]);
  }
  return sure && (int)lanes_sum<16>((float)steps) == found;
}
template <int VPL>
__device__ __forceinline__ bool pick_sorted(const RouteArgs& a, int lane, const float (&key)[VPL],
                                            float error, int* ids, int& id) {
  int list[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    list[j] = (int)__builtin_amdgcn_fmed3f(key[j] * 0x1p24f, -0x1p27f, 0x1p27f - 16.f) * 16 + j;
  constexpr SortingNetwork<VPL> net;
#pragma unroll
  for (int c = 0; c < net.size; ++c) {
    const int x = list[net.a[c]], y = list[net.b[c]];
    list[net.a[c]] = max(x, y);
    list[net.b[c]] = min(x, y);
  }
  // one more pick than asked for; both conversions cut less than a unit off
  const int picks = a.top_k + 1;
  const uint32_t apart = (uint32_t)(2.f * error * 0x1p28f) + 32;
  bool sure;
  int found;
  if (picks <= 9)
    sure = take_heads<(VPL < 9 ? VPL : 9), VPL>(list, picks, a.top_k, lane, apart, ids, found);
  else
    sure = take_heads<VPL, VPL>(list, picks, a.top_k, lane, apart, ids, found);
  id = lane < min(a.top_k, found) ? ids[lane] : -1;
  return sure;
}

// Lanes of a group for limit_groups().
template <int VPL>
__device__ __forceinline__ int group_lanes(const RouteArgs& a) {
  const int per = a.n_experts / a.n_groups, span = per / VPL;
  return a.n_groups == 1 ? 0 : per % VPL == 0 && (span & (span - 1)) == 0 ? span : -1;
}

// The picks of one token in binary64.
template <int VPL>
__device__ __forceinline__ int pick_binary64(const RouteArgs& a, int lane, const float (&x)[VPL],
                                             float top) {
  double key[VPL], score[VPL], sum = 0.;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const double l = x[j];
    score[j] = a.score == EP_SCORE_SOFTMAX ? exp(l - top) : 1. / (1. + exp(-l));
    sum += score[j];
    // one at a time: this path is rare, and its registers are every token's
    asm volatile("" : "+v"(score[j]));
  }
  sum = a.score == EP_SCORE_SOFTMAX ? lanes_sum<64>(sum) : 1.;
  float b[VPL];
  load_bias<VPL>(a, lane, b);
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const bool there = x[j] > -INFINITY && b[j] > -INFINITY;
    score[j] = there ? score[j] / sum + b[j] : -INFINITY;
    key[j] = a.bias ? score[j] : x[j];
  }
  int id;
  limit_groups<64, VPL, double>(a, lane, key, score, true, 0.f, group_lanes<VPL>(a));
  pick<64, VPL, double>(a, lane, key, true, 0.f, id);
  return id;
}

// Largest logit of a token, at least the smallest finite number.
template <int LPT, int VPL>
__device__ __forceinline__ float largest(const float (&x)[VPL]) {
  float top = x[0];
#pragma unroll
  for (int j = 1; j < VPL; ++j) top = fmaxf(top, x[j]);
  return fmaxf(lanes_max<LPT>(top), -FLT_MAX);
}

// Weights and stores of one token, lane k with pick k's id.
template <int LPT, int VPL>
__device__ __forceinline__ void finish_token(const RouteArgs& a, int64_t t, bool token, int lane,
                                             const float (&x)[VPL], float top, int id) {
  const bool there = token && id >= 0;
  const float l = there ? load_logit(a, t * a.n_experts + id) : -INFINITY;
  float w;
  if (a.renormalize) {
    w = pick_share<LPT>(l, there, a.score);
  } else if (a.score == EP_SCORE_SIGMOID) {
    w = 1.f / (1.f + expf(-l));
  } else {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) sum += exp_near(x[j] - top);
    w = expf(l - top) / lanes_sum<LPT>(sum);
  }
  if (token && lane < a.top_k) {
    a.topk_ids[t * a.top_k + lane] = id;
    a.topk_w[t * a.top_k + lane] = there ? a.scale * w : 0.f;
  }
}

// First id of a token that is to be picked in binary64.
constexpr int kPickAgain = -0x7fffffff;

// HERE: tokens that binary32 cannot decide are picked in binary64 here; else they are
// marked for pick_again_kernel.
template <int LPT, int VPL, bool HERE>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
  constexpr int TPW = 64 / LPT;                // tokens of a wave
  const int lane = threadIdx.x & (LPT - 1), row = (threadIdx.x & 63) / LPT;
  const int64_t wave = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  const int64_t waves = (int64_t)gridDim.x * kRouteWaves;
  const int E = a.n_experts, lanes = group_lanes<VPL>(a);
  const bool exact = !a.bias && !(a.n_groups > 1 && a.group_score == EP_GROUP_TOP2);
  const bool biased = a.bias != nullptr;
  __shared__ int s_ids[HERE ? 1 : kRouteThreads / LPT][16];
  for (int64_t first = wave * TPW; first < a.tokens; first += waves * TPW) {
    const int64_t t = first + row;
    const bool token = t < a.tokens;           // the last wave's may be fewer
    float x[VPL];
    load_row<VPL>(a, t, token ? lane : E, x);
    const float top = largest<LPT>(x);
    float key[VPL], score[VPL], error = 0.f, size = 0.f;
    if (exact) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = x[j];
    } else {
      load_bias<VPL>(a, lane, key);
      float inv = 1.f;
      constexpr float log2e = 0x1.715476p0f;
      if (a.score == EP_SCORE_SOFTMAX) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          score[j] = __builtin_amdgcn_exp2f((x[j] - top) * log2e);
          sum += score[j];
        }
        sum = lanes_sum<LPT>(sum);
        inv = sum > 0.f ? 1.f / sum : 0.f;
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
          score[j] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x[j] * -log2e));
      }
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const float v = score[j] * inv + key[j];
        const bool there = x[j] > -INFINITY && v > -INFINITY;
        score[j] = there ? v : -INFINITY;
        key[j] = biased ? score[j] : x[j];
        size = fmaxf(size, there ? fabsf(v) : 0.f);
      }
      size = lanes_max<LPT>(size);
      error = choice_error(a.score) * (1.f + size);
    }
    int id;
    bool sure = limit_groups<LPT, VPL, float>(a, lane, key, score, exact, error, lanes);
    if (!HERE && biased && __ballot(size < kSortedBelow) == ~0ull)   // in every token of the wave
      sure &= pick_sorted<VPL>(a, lane, key, error, s_ids[HERE ? 0 : threadIdx.x / LPT], id);
    else
      sure &= pick<LPT, VPL, float>(a, lane, key, exact, error, id);
    if constexpr (HERE) {
      if (!sure) id = pick_binary64<VPL>(a, lane, x, top);
    } else if (token && !sure && lane == 0) {
      a.topk_ids[t * a.top_k] = kPickAgain;
    }
    finish_token<LPT, VPL>(a, t, token && (HERE || sure), lane, x, top, id);
  }
}

// The marked tokens, a wave each: every wave looks through runs of kRun tokens.
constexpr int kRun = 16;
template <int VPL>
__global__ __launch_bounds__(kRouteThreads) void pick_again_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  const int64_t waves = (int64_t)gridDim.x * kRouteWaves;
  for (int64_t first = wave * kRun; first < a.tokens; first += waves * kRun) {
    const int64_t mine = first + lane;
    uint64_t marked = __ballot(lane < kRun && mine < a.tokens && a.topk_ids[mine * a.top_k] == kPickAgain);
    while (marked) {
      const int64_t t = first + __builtin_ctzll(marked);
      marked &= marked - 1;
      float x[VPL];
      load_row<VPL>(a, t, lane, x);
      const float top = largest<64>(x);
      finish_token<64, VPL>(a, t, true, lane, x, top, pick_binary64<VPL>(a, lane, x, top));
    }
  }
}

// What pick k adds at its expert, lane k of the token's LPT lanes with its logit l and
// scaled gradient g; not for the plain softmax, whose gradient is dense.  The reciprocals are
// the hardware's, within a step (2^-23) of themselves where a division is within half
// of one, and the exponentials are exp_near()'s: a share is off by a few steps either way, which
// the difference g - sum g p multiplies in any form, and the kernel took 17 us instead of
// 20 with them (32768 tokens of 256 experts).
template <int LPT>
__device__ __forceinline__ float pick_gradient(const RouteArgs& a, float l, float g, bool there) {
  float d;
  if (a.renormalize) {
    const float p = pick_share<LPT>(l, there, a.score);
    d = p * (g - lanes_sum<LPT>(g * p));
  } else {
    d = g * __builtin_amdgcn_rcpf(1.f + exp_near(fminf(-l, 88.f)));
  }
  if (a.score == EP_SCORE_SIGMOID) d *= __builtin_amdgcn_rcpf(1.f + exp_near(fminf(l, 88.f)));
  return there ? d : 0.f;
}

// The gradient at the picks alone, four tokens a wave: their rows, which follow one
// another, are filled with zeros, and once those stores are acknowledged the lanes that
// hold picks store theirs.  At 32768 tokens of 256 experts it takes 12.1 us, the kernel
// below, in which every lane looks for its experts among the picks, took 16.6.  A line that
// holds a pick goes out twice, with a wait between: 48.7 MB written for a gradient of 33.6.
__global__ __launch_bounds__(kRouteThreads) void route_backward_picks_kernel(RouteArgs a) {
  const int wl = threadIdx.x & 63, lane = wl & 15, row = wl >> 4;
  const int64_t wave = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  const int64_t waves = (int64_t)gridDim.x * kRouteWaves;
  const int E = a.n_experts, size = a.dtype == EP_LOGITS_F32 ? 4 : 2;
  for (int64_t first = wave * 4; first < a.tokens; first += waves * 4) {
    const int64_t t = first + row;
    int id = -1;
    float l = -INFINITY, g = 0.f;
    if (t < a.tokens && lane < a.top_k) {
      id = a.topk_ids[t * a.top_k + lane];
      g = a.grad_w[t * a.top_k + lane];
      if (id >= 0 && id < E) l = load_logit(a, t * E + id);
    }
    // four rows start at a multiple of 8 bytes
    const int64_t left = a.tokens - first;
    const int bytes = (int)(left < 4 ? left : 4) * E * size;
    uint8_t* rows = a.grad_logits + first * E * size;
    for (int o = wl * 8; o + 8 <= bytes; o += 512) *reinterpret_cast<uint64_t*>(rows + o) = 0;
    const int rest = (bytes & ~7) + wl * 2;
    if (rest < bytes) *reinterpret_cast<uint16_t*>(rows + rest) = 0;

    const bool there = l > -INFINITY;
    const float mine = pick_gradient<16>(a, l, there ? a.scale * g : 0.f, there);
    float d = 0.f;                 // picks of one expert add up, the same in each of them
    for (int k = 0; k < a.top_k; ++k) {
      const int i = of_lane<16>(id, k);
      const float v = of_lane<16>(mine, k);
      d += i == id ? v : 0.f;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (there) {
      const int64_t at = t * E + id;
      if (a.dtype == EP_LOGITS_F32)
        reinterpret_cast<float*>(a.grad_logits)[at] = d;
      else if (a.dtype == EP_LOGITS_BF16)
        reinterpret_cast<__bf16*>(a.grad_logits)[at] = (__bf16)d;
      else
        reinterpret_cast<_Float16*>(a.grad_logits)[at] = (_Float16)d;
    }
  }
}

// Any gradient, a wave per token; the next token's picks and their logits are loaded
// before this one's row is computed and stored.
template <int VPL>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  const int64_t waves = (int64_t)gridDim.x * kRouteWaves;
  const int E = a.n_experts;
  const bool dense = a.score == EP_SCORE_SOFTMAX && !a.renormalize;
  // lane k: pick k's id (-1: none), logit and gradient
  auto load_pick = [&](int64_t t, int& id, float& l, float& g) {
    id = -1;
    l = -INFINITY;
    g = 0.f;
    if (t >= a.tokens || lane >= a.top_k) return;
    id = a.topk_ids[t * a.top_k + lane];
    g = a.grad_w[t * a.top_k + lane];
    if (id >= 0 && id < E) l = load_logit(a, t * E + id);
  };
  int id;
  float l, g;
  load_pick(wave, id, l, g);
  for (int64_t t = wave; t < a.tokens; t += waves) {
    const bool there = l > -INFINITY;
    const int at = there ? id : -1;
    const float mine = l, gk = there ? a.scale * g : 0.f;
    load_pick(t + waves, id, l, g);
    float out[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) out[j] = 0.f;
    // what pick k adds at its expert
    const float d = dense ? gk : pick_gradient<64>(a, mine, gk, there);
    for (int k = 0; k < a.top_k; ++k) {
      const int i = __builtin_amdgcn_readlane(at, k) - lane * VPL;
      const float v = read_lane(d, k);
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (i == j) out[j] += v;
    }
    if (dense) {
      float x[VPL], sum = 0.f, dot = 0.f;
      load_row<VPL>(a, t, lane, x);
      const float top = largest<64>(x);
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        x[j] = exp_near(x[j] - top);
        sum += x[j];
        dot += x[j] * out[j];
      }
      sum = lanes_sum<64>(sum);
      dot = lanes_sum<64>(dot);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      dot *= inv;
#pragma unroll
      for (int j = 0; j < VPL; ++j) out[j] = x[j] * inv * (out[j] - dot);
    }
    store_row<VPL>(a, t, lane, out);
  }
}

}  // namespace

// Workgroups for `tokens` tokens, `each` a workgroup at a time, at most `per_cu` a CU.
static int route_grid(int64_t tokens, int each, int num_cus, int per_cu) {
  const int64_t blocks = (tokens + each - 1) / each, most = (int64_t)per_cu * num_cus;
  return (int)(blocks < most ? blocks : most);
}

hipError_t launch_route(const RouteArgs& a, int num_cus, hipStream_t st) {
  const dim3 block(kRouteThreads);
  // four tokens a wave from 16 tokens a CU on: one token took 5.6 us with 64 lanes and
  // 10.4 with 16, 8192 tokens of 128 experts 11.5 and 7.9
  const bool many = a.tokens >= 16 * (int64_t)num_cus && a.n_experts <= 256 && a.n_groups <= 16 &&
                    a.top_k <= 16;
  if (many) {
    const dim3 grid(route_grid(a.tokens, 4 * kRouteWaves, num_cus, 16));
    const int vpl = (a.n_experts + 15) / 16;
    if (vpl <= 4)
      hipLaunchKernelGGL((route_kernel<16, 4, false>), grid, block, 0, st, a);
    else if (vpl <= 8)
      hipLaunchKernelGGL((route_kernel<16, 8, false>), grid, block, 0, st, a);
    else
      hipLaunchKernelGGL((route_kernel<16, 16, false>), grid, block, 0, st, a);
    const bool exact = !a.bias && !(a.n_groups > 1 && a.group_score == EP_GROUP_TOP2);
    if (!exact)
      hipLaunchKernelGGL(pick_again_kernel<4>,
                         dim3(route_grid(a.tokens, kRun * kRouteWaves, num_cus, 4)), block, 0, st, a);
  } else {
    const dim3 grid(route_grid(a.tokens, kRouteWaves, num_cus, 16));
    const int vpl = (a.n_experts + 63) / 64;
    if (vpl <= 4)
      hipLaunchKernelGGL((route_kernel<64, 4, true>), grid, block, 0, st, a);
    else if (vpl <= 8)
      hipLaunchKernelGGL((route_kernel<64, 8, true>), grid, block, 0, st, a);
    else
      hipLaunchKernelGGL((route_kernel<64, 16, true>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs& a, int num_cus, hipStream_t st) {
  const dim3 block(kRouteThreads);
  if (!(a.score == EP_SCORE_SOFTMAX && !a.renormalize) && a.top_k <= 16) {
    const dim3 grid(route_grid(a.tokens, 4 * kRouteWaves, num_cus, 16));
    hipLaunchKernelGGL(route_backward_picks_kernel, grid, block, 0, st, a);
    return hipGetLastError();
  }
  const dim3 grid(route_grid(a.tokens, kRouteWaves, num_cus, 16));
  const int vpl = (a.n_experts + 63) / 64;
  if (vpl <= 4) hipLaunchKernelGGL(route_backward_kernel<4>, grid, block, 0, st, a);
  else if (vpl <= 8) hipLaunchKernelGGL(route_backward_kernel<8>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(route_backward_kernel<16>, grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace ep
