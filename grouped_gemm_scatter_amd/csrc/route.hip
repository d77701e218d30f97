// Routing to experts: scores, the group limit, top-k picks and their weights for
// every token, and the gradient of the weights with respect to the logits.
// One wave per token; lane L holds VPL consecutive experts from L * VPL, so that the
// lowest lane holds the lowest index of a tie.
//
// Which experts are picked is exact.  Without a bias the choice is the order of the
// logits themselves.  Where a score is compared (a bias, a sum of two) it is defined in
// binary64, but computed in binary32 first with a bound on the error: only a token in
// which two choices next to each other, or the groups at the limit, lie within that
// bound is chosen again in binary64, in a few tokens of a thousand.
// A pick: the largest key of every lane, the largest of the wave by six cross-lane
// moves, the lowest lane that has it by a ballot.
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

// A missing expert (NaN, -infinity) is -infinity; +infinity the largest number.
__device__ __forceinline__ float clean(float v) { return v != v ? -INFINITY : fminf(v, FLT_MAX); }

__device__ __forceinline__ float f16_value(uint32_t v) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t i) {
  if (a.dtype == EP_LOGITS_F32) return clean(reinterpret_cast<const float*>(a.logits)[i]);
  const uint16_t h = reinterpret_cast<const uint16_t*>(a.logits)[i];
  return clean(a.dtype == EP_LOGITS_BF16 ? bf16_lo(h) : f16_value(h));
}

__device__ __forceinline__ float half_value(const RouteArgs& a, uint32_t h) {
  return clean(a.dtype == EP_LOGITS_BF16 ? bf16_lo(h & 0xffffu) : f16_value(h));
}

// Logits of experts lane * VPL + 0..VPL-1 of token t, -infinity past the last.  Rows of
// a multiple of VPL experts start where a lane's values can be loaded together.
template <int VPL>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t t, int lane, float (&x)[VPL]) {
  const int E = a.n_experts, first = lane * VPL;
  const int64_t at = t * E + first;
  if (VPL >= 2 && E % VPL == 0) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = -INFINITY;
    if (first >= E) return;
    if (a.dtype == EP_LOGITS_F32) {
      const float* p = reinterpret_cast<const float*>(a.logits) + at;
      if constexpr (VPL == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) x[j] = clean(__uint_as_float(v[j]));
      } else {
#pragma unroll
        for (int j = 0; j < VPL / 4; ++j) {
          const u32x4 v = load16(p + 4 * j);
#pragma unroll
          for (int q = 0; q < 4; ++q) x[4 * j + q] = clean(__uint_as_float(v[q]));
        }
      }
    } else {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(
          reinterpret_cast<const uint16_t*>(a.logits) + at);
      uint32_t v[VPL > 1 ? VPL / 2 : 1];
#pragma unroll
      for (int j = 0; j < VPL / 2; ++j) v[j] = p[j];
#pragma unroll
      for (int j = 0; j < VPL; ++j) x[j] = half_value(a, v[j / 2] >> (16 * (j & 1)));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) x[j] = first + j < E ? load_logit(a, at + j) : -INFINITY;
}

template <int VPL>
__device__ __forceinline__ void store_row(const RouteArgs& a, int64_t t, int lane,
                                          const float (&v)[VPL]) {
  const int E = a.n_experts, first = lane * VPL;
  const int64_t at = t * E + first;
  if (first >= E) return;
  if (VPL >= 2 && E % VPL == 0) {
    if (a.dtype == EP_LOGITS_F32) {
      float* p = reinterpret_cast<float*>(a.grad_logits) + at;
      if constexpr (VPL == 2) {
        *reinterpret_cast<u32x2*>(p) =
            u32x2{__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1])};
      } else {
#pragma unroll
        for (int j = 0; j < VPL / 4; ++j) {
          u32x4 o;
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] = __builtin_bit_cast(uint32_t, v[4 * j + q]);
          store16_nt(p + 4 * j, o);
        }
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

// Over the wave, the same in every lane: within rows of 16 lanes, then rows 0 and 2
// into 1 and 3, then the lower half into the upper, whose last lane has it all.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, lane_move<0x111>(v, v));        // row_shr 1, 2, 4, 8
  v = fmaxf(v, lane_move<0x112>(v, v));
  v = fmaxf(v, lane_move<0x114>(v, v));
  v = fmaxf(v, lane_move<0x118>(v, v));
  v = fmaxf(v, lane_move<0x142, 0xa>(v, v));   // row_bcast 15, 31
  v = fmaxf(v, lane_move<0x143, 0xc>(v, v));
  return read_lane(v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
  v += lane_move<0x111>(0.f, v);
  v += lane_move<0x112>(0.f, v);
  v += lane_move<0x114>(0.f, v);
  v += lane_move<0x118>(0.f, v);
  v += lane_move<0x142, 0xa>(0.f, v);
  v += lane_move<0x143, 0xc>(0.f, v);
  return read_lane(v, 63);
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const double o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}

// The largest value over the wave and its lowest index.
__device__ __forceinline__ void wave_best(double& v, int& i) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const double ov = __shfl_xor(v, d);
    const int oi = __shfl_xor(i, d);
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
}

constexpr int kNone = 0x7fffffff;

// Shares of the picks, lane k holding pick k's logit l (there: lane k has a pick):
// softmax over the picks, or their sigmoids over the sum.
__device__ __forceinline__ float pick_share(float l, bool there, int score) {
  const float low = score == EP_SCORE_SIGMOID ? fminf(l, 0.f) : l;
  const float top = wave_max(there ? low : -FLT_MAX);
  float e = there ? expf(low - top) : 0.f;
  if (score == EP_SCORE_SIGMOID) e /= 1.f + expf(-fabsf(l));
  const float sum = wave_sum(e);
  return there ? e / sum : 0.f;
}

// The picks of one token in binary64, lane k's id (or -1) in lane k: the definition,
// reduced over the wave group by group and pick by pick.
template <int VPL>
__device__ __forceinline__ int pick_binary64(const RouteArgs& a, int lane, const float (&x)[VPL],
                                             float top) {
  const int E = a.n_experts, per = E / a.n_groups;
  const bool top2 = a.n_groups > 1 && a.group_score == EP_GROUP_TOP2;
  double c[VPL], s[VPL];           // choice, score (with bias)
  double sum = 0.;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const double l = x[j];
    s[j] = a.score == EP_SCORE_SOFTMAX ? exp(l - top) : 1. / (1. + exp(-l));
    sum += s[j];
  }
  if (a.score == EP_SCORE_SOFTMAX) {
    sum = wave_sum(sum);
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = sum > 0. ? s[j] / sum : 0.;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int i = lane * VPL + j;
    bool there = x[j] > -INFINITY;
    if (a.bias) {
      const float b = i < E ? a.bias[i] : 0.f;
      there = there && b > -INFINITY;
      s[j] += b;
      c[j] = there ? s[j] : -INFINITY;
    } else {
      c[j] = x[j];
    }
    if (!there) s[j] = -INFINITY;
  }
  if (a.n_groups > 1) {
    double value = -INFINITY;      // lane g: the value of group g
    for (int g = 0; g < a.n_groups; ++g) {
      double v = -INFINITY;
      int best = kNone;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int i = lane * VPL + j;
        const double y = top2 ? s[j] : c[j];
        if (i / per == g && i < E && y > v) {
          v = y;
          best = i;
        }
      }
      wave_best(v, best);
      if (top2) {
        double w = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int i = lane * VPL + j;
          if (i / per == g && i < E && i != best && s[j] > w) w = s[j];
        }
        w = wave_max(w);
        if (w > -INFINITY) v += w;
      }
      if (lane == g) value = v;
    }
    uint64_t kept = 0;
    for (int n = 0; n < a.topk_groups; ++n) {
      double v = value;
      int g = v > -INFINITY ? lane : kNone;
      wave_best(v, g);
      if (g == kNone) break;
      kept |= 1ull << g;
      if (lane == g) value = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int g = (lane * VPL + j) / per;
      if (g >= a.n_groups || !(kept >> g & 1)) c[j] = -INFINITY;
    }
  }
  int id = -1;
  for (int k = 0; k < a.top_k; ++k) {
    double v = -INFINITY;
    int best = kNone;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (c[j] > v) {
        v = c[j];
        best = lane * VPL + j;
      }
    wave_best(v, best);
    if (best == kNone) break;
    if (lane == k) id = best;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (best == lane * VPL + j) c[j] = -INFINITY;
  }
  return id;
}

// Bound on the error of a binary32 score plus bias, over 1 + the largest such sum of the
// token: a softmax score is within s (|l - top| + 30) 2^-24 <= 31 * 2^-24 (the argument's
// rounding, expf, a sum of at most 16 + 6 additions, the division), a sigmoid within
// 4 * 2^-24, and the bias adds one rounding of the sum.
constexpr float kChoiceError = 0x1p-19f;

// The picks of one token in binary32.  Returns false where the keys are not exact
// (`exact`: they are the logits) and two that decide lie within their error.
// key: the choices, score: scores plus bias, -infinity for what cannot be picked; group:
// the groups of the lane's experts.  lanes: lanes of a group where that is a power of
// two of whole lanes, 0: no groups, -1: groups of any other size.
template <int VPL>
__device__ __forceinline__ bool pick_binary32(const RouteArgs& a, int lane, float (&key)[VPL],
                                              const float (&score)[VPL],
                                              const int (&group)[VPL], bool exact, int lanes,
                                              int& id) {
  float error = 0.f;
  if (!exact) {
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (score[j] > -INFINITY) most = fmaxf(most, fabsf(score[j]));
    error = kChoiceError * (1.f + wave_max(most));
  }
  bool sure = true;
  if (lanes != 0) {
    const bool top2 = a.group_score == EP_GROUP_TOP2;
    // the two largest of this lane's group (lanes > 0), or of group `lane`
    float v1 = -INFINITY, v2 = -INFINITY;
    if (lanes > 0) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const float y = top2 ? score[j] : key[j];
        v2 = fmaxf(v2, fminf(v1, y));
        v1 = fmaxf(v1, y);
      }
      for (int d = 1; d < lanes; d <<= 1) {
        const float o1 = __shfl_xor(v1, d), o2 = __shfl_xor(v2, d);
        v2 = fmaxf(fminf(v1, o1), fmaxf(v2, o2));
        v1 = fmaxf(v1, o1);
      }
    } else {
      for (int g = 0; g < a.n_groups; ++g) {
        float w1 = -INFINITY, w2 = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const float y = group[j] != g ? -INFINITY : top2 ? score[j] : key[j];
          w2 = fmaxf(w2, fminf(w1, y));
          w1 = fmaxf(w1, y);
        }
        const float m1 = wave_max(w1);
        float m2 = -INFINITY;
        if (top2) {
          // the second: one lane that has the first gives its second, the others their first
          const int win = (int)__builtin_ctzll(__ballot(w1 == m1));
          m2 = wave_max(lane == win ? w2 : w1);
        }
        if (lane == g) {
          v1 = m1;
          v2 = m2;
        }
      }
    }
    float value = v1;
    if (top2 && v2 > -INFINITY) value += v2;
    const int step = lanes > 0 ? lanes : 1, g = lane / step;
    int above = 0;                             // groups that come before this one
    for (int o = 0; o < a.n_groups; ++o) {
      const float v = read_lane(value, o * step);
      above += v > value || (v == value && o < g);
    }
    const bool mine = g < a.n_groups;
    const bool keep = mine && above < a.topk_groups;
    if (!exact && a.topk_groups < a.n_groups) {
      const float in = -wave_max(keep ? -value : -INFINITY);     // the last kept
      const float out = wave_max(mine && !keep ? value : -INFINITY);
      // (infinite values: a group without experts, a bias of +infinity)
      if (!(in - out > 4.f * error)) sure = out == -INFINITY;
    }
    const uint64_t kept = __ballot(keep);      // by lane, or by group
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (!(kept >> (lanes > 0 ? lane : group[j]) & 1)) key[j] = -INFINITY;
  }
  float before = INFINITY;
  id = -1;
  // one more pick than asked for, to see how near it comes
  const int picks = a.top_k + (exact ? 0 : 1);
  for (int k = 0; k < picks; ++k) {
    float best = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = fmaxf(best, key[j]);
    const float m = wave_max(best);
    if (m == -INFINITY) break;
    if (!exact && k > 0 && !(before - m > 2.f * error)) sure = false;
    before = m;
    if (k == a.top_k) break;
    const int win = (int)__builtin_ctzll(__ballot(best == m));
    int at = VPL;                              // the first of the lane's keys that is m
#pragma unroll
    for (int j = VPL - 1; j >= 0; --j)
      if (key[j] == m) at = j;
    const int i = win * VPL + __builtin_amdgcn_readlane(at, win);
    if (lane == k) id = i;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (lane * VPL + j == i) key[j] = -INFINITY;
  }
  return sure;
}

template <int VPL>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  const int64_t waves = (int64_t)gridDim.x * kRouteWaves;
  const int E = a.n_experts, per = E / a.n_groups;
  const bool exact = !a.bias && !(a.n_groups > 1 && a.group_score == EP_GROUP_TOP2);
  // lanes of a group, where that is a power of two of whole lanes
  const int span = per / VPL;
  const int lanes = a.n_groups == 1 ? 0 : per % VPL == 0 && (span & (span - 1)) == 0 ? span : -1;
  float bias[VPL];
  int group[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int i = lane * VPL + j;
    bias[j] = a.bias && i < E ? a.bias[i] : 0.f;
    group[j] = min(i / per, 63);     // past the last expert: whatever, its keys are -infinity
  }
  for (int64_t t = wave; t < a.tokens; t += waves) {
    float x[VPL];
    load_row<VPL>(a, t, lane, x);
    float top = x[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) top = fmaxf(top, x[j]);
    top = fmaxf(wave_max(top), -FLT_MAX);
    const bool dense = a.score == EP_SCORE_SOFTMAX && !a.renormalize;
    float sum = 0.f, key[VPL], score[VPL];
    if (!exact || dense) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        score[j] = a.score == EP_SCORE_SOFTMAX ? expf(x[j] - top) : 1.f / (1.f + expf(-x[j]));
        sum += score[j];
      }
      sum = a.score == EP_SCORE_SOFTMAX ? wave_sum(sum) : 1.f;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if (exact) {
        key[j] = x[j];
        continue;
      }
      if (a.score == EP_SCORE_SOFTMAX) score[j] *= inv;
      score[j] = x[j] > -INFINITY && bias[j] > -INFINITY ? score[j] + bias[j] : -INFINITY;
      key[j] = a.bias ? score[j] : x[j];
    }
    int id;
    if (!pick_binary32<VPL>(a, lane, key, score, group, exact, lanes, id))
      id = pick_binary64<VPL>(a, lane, x, top);
    const bool there = id >= 0;
    const float l = there ? load_logit(a, t * E + id) : -INFINITY;
    float w;
    if (a.renormalize)
      w = pick_share(l, there, a.score);
    else if (a.score == EP_SCORE_SIGMOID)
      w = 1.f / (1.f + expf(-l));
    else
      w = expf(l - top) / sum;
    if (lane < a.top_k) {
      a.topk_ids[t * a.top_k + lane] = id;
      a.topk_w[t * a.top_k + lane] = there ? a.scale * w : 0.f;
    }
  }
}

template <int VPL>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  const int64_t waves = (int64_t)gridDim.x * kRouteWaves;
  const int E = a.n_experts;
  for (int64_t t = wave; t < a.tokens; t += waves) {
    // lane k: pick k's id, gradient and logit
    int id = lane < a.top_k ? a.topk_ids[t * a.top_k + lane] : -1;
    float l = -INFINITY;
    if (id >= 0 && id < E) l = load_logit(a, t * E + id);
    const bool there = l > -INFINITY;
    if (!there) id = -1;
    const float g = there ? a.scale * a.grad_w[t * a.top_k + lane] : 0.f;
    float out[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) out[j] = 0.f;
    const bool dense = a.score == EP_SCORE_SOFTMAX && !a.renormalize;
    float d = g;                   // what pick k adds at its expert
    if (!dense) {
      if (a.renormalize) {
        const float p = pick_share(l, there, a.score);
        d = p * (g - wave_sum(g * p));
      } else {
        d = g / (1.f + expf(-l));
      }
      if (a.score == EP_SCORE_SIGMOID) d /= 1.f + expf(l);
      if (!there) d = 0.f;
    }
    for (int k = 0; k < a.top_k; ++k) {
      const int i = __builtin_amdgcn_readlane(id, k) - lane * VPL;
      const float v = read_lane(d, k);
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (i == j) out[j] += v;
    }
    if (dense) {
      float x[VPL], sum = 0.f, dot = 0.f;
      load_row<VPL>(a, t, lane, x);
      float top = x[0];
#pragma unroll
      for (int j = 1; j < VPL; ++j) top = fmaxf(top, x[j]);
      top = fmaxf(wave_max(top), -FLT_MAX);
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        x[j] = expf(x[j] - top);
        sum += x[j];
        dot += x[j] * out[j];
      }
      sum = wave_sum(sum);
      dot = wave_sum(dot);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      dot *= inv;
#pragma unroll
      for (int j = 0; j < VPL; ++j) out[j] = x[j] * inv * (out[j] - dot);
    }
    store_row<VPL>(a, t, lane, out);
  }
}

}  // namespace

#define EP_ROUTE_LAUNCH(KERNEL)                                                              \
  const int64_t blocks = (a.tokens + kRouteWaves - 1) / kRouteWaves;                          \
  const int64_t most = 16 * (int64_t)num_cus;                                                 \
  const dim3 grid((int)(blocks < most ? blocks : most)), block(kRouteThreads);                \
  const int vpl = (a.n_experts + 63) / 64;                                                    \
  if (vpl <= 1) hipLaunchKernelGGL(KERNEL<1>, grid, block, 0, st, a);                         \
  else if (vpl <= 2) hipLaunchKernelGGL(KERNEL<2>, grid, block, 0, st, a);                    \
  else if (vpl <= 4) hipLaunchKernelGGL(KERNEL<4>, grid, block, 0, st, a);                    \
  else if (vpl <= 8) hipLaunchKernelGGL(KERNEL<8>, grid, block, 0, st, a);                    \
  else hipLaunchKernelGGL(KERNEL<16>, grid, block, 0, st, a);                                 \
  return hipGetLastError();

hipError_t launch_route(const RouteArgs& a, int num_cus, hipStream_t st) {
  EP_ROUTE_LAUNCH(route_kernel)
}

hipError_t launch_route_backward(const RouteArgs& a, int num_cus, hipStream_t st) {
  EP_ROUTE_LAUNCH(route_backward_kernel)
}

}  // namespace ep
