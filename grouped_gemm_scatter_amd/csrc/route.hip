// Routing to experts: scores, the group limit, top-k picks and their weights for
// every token, and the gradient of the weights with respect to the logits.
// One wave per token; lane L holds experts L, L + 64, ... of the token's row.
//
// Which experts are picked is exact: without a bias the choice is the order of
// the logits themselves, and where a score is compared (a bias, a sum of two)
// it is computed in binary64.  Selection takes the largest (choice, lowest index)
// left, top_k times, by a reduction over the wave.
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

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t i) {
  float v;
  if (a.dtype == EP_LOGITS_F32)
    v = reinterpret_cast<const float*>(a.logits)[i];
  else if (a.dtype == EP_LOGITS_BF16)
    v = bf16_lo(reinterpret_cast<const uint16_t*>(a.logits)[i]);
  else
    v = (float)reinterpret_cast<const _Float16*>(a.logits)[i];
  // a missing expert (NaN, -infinity) is -infinity; +infinity the largest number
  return v != v ? -INFINITY : fminf(v, FLT_MAX);
}

__device__ __forceinline__ void store_grad(const RouteArgs& a, int64_t i, float v) {
  if (a.dtype == EP_LOGITS_F32)
    reinterpret_cast<float*>(a.grad_logits)[i] = v;
  else if (a.dtype == EP_LOGITS_BF16)
    reinterpret_cast<__bf16*>(a.grad_logits)[i] = (__bf16)v;
  else
    reinterpret_cast<_Float16*>(a.grad_logits)[i] = (_Float16)v;
}

template <class T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const T o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
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

template <int VPL>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  const int64_t waves = (int64_t)gridDim.x * kRouteWaves;
  const int E = a.n_experts, per = E / a.n_groups;
  const bool top2 = a.n_groups > 1 && a.group_score == EP_GROUP_TOP2;
  for (int64_t t = wave; t < a.tokens; t += waves) {
    float x[VPL];
    double c[VPL], s[VPL];         // choice, score (with bias)
    float top = -FLT_MAX;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int i = j * 64 + lane;
      x[j] = i < E ? load_logit(a, t * E + i) : -INFINITY;
      top = fmaxf(top, x[j]);
    }
    top = wave_max(top);
    if (a.bias || top2) {
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
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int i = j * 64 + lane;
      bool there = x[j] > -INFINITY;
      if (a.bias) {
        const float b = i < E ? a.bias[i] : 0.f;
        there = there && b > -INFINITY;
        s[j] += b;
        c[j] = there ? s[j] : -INFINITY;
      } else {
        c[j] = x[j];
      }
      if (top2) s[j] = there ? s[j] : -INFINITY;
    }
    if (a.n_groups > 1) {
      // lane g: the value of group g
      double value = -INFINITY;
      for (int g = 0; g < a.n_groups; ++g) {
        double v = -INFINITY;
        int best = kNone;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int i = j * 64 + lane;
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
            const int i = j * 64 + lane;
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
        const int g = (j * 64 + lane) / per;
        if (g >= a.n_groups || !(kept >> g & 1)) c[j] = -INFINITY;
      }
    }
    int id = -1;                   // lane k: pick k
    for (int k = 0; k < a.top_k; ++k) {
      double v = -INFINITY;
      int best = kNone;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (c[j] > v) {
          v = c[j];
          best = j * 64 + lane;
        }
      wave_best(v, best);
      if (best == kNone) break;
      if (lane == k) id = best;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (best == j * 64 + lane) c[j] = -INFINITY;
    }
    const bool there = id >= 0;
    const float l = there ? load_logit(a, t * E + id) : -INFINITY;
    float w;
    if (a.renormalize) {
      w = pick_share(l, there, a.score);
    } else if (a.score == EP_SCORE_SIGMOID) {
      w = 1.f / (1.f + expf(-l));
    } else {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) sum += expf(x[j] - top);
      w = expf(l - top) / wave_sum(sum);
    }
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
      const int i = __shfl(id, k);
      const float v = __shfl(d, k);
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (i == j * 64 + lane) out[j] += v;
    }
    if (dense) {
      float x[VPL], top = -FLT_MAX, sum = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int i = j * 64 + lane;
        x[j] = i < E ? load_logit(a, t * E + i) : -INFINITY;
        top = fmaxf(top, x[j]);
      }
      top = wave_max(top);
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
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int i = j * 64 + lane;
      if (i < E) store_grad(a, t * E + i, out[j]);
    }
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
