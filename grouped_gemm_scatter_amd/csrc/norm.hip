// RMS norm of rows with the residual's addition, outputs in the rows' type and in 8 bits,
// and its gradient.
//
//   s = x + residual (binary32, or x),   inv = 1 / sqrt(mean(s^2) + eps),   y = s inv w
//   with r the stored sums and g, h the gradients of y and of the stored sums:
//   dr = inv (g w - (r inv) (inv mean(g w r))) + h,   dw = sum over rows of g r inv
//
// Both are HBM streams.  A row is spread over TPR threads, a thread holding kHeld chunks of 8
// values in registers between the sum over the row and their use, so that every input is
// read once; what a row has beyond that (more than 16384 values, EXTRA) is read again.
// A 128-value block of 8-bit output is 16 neighbouring lanes' chunks.
//
// What they measured: 32768 rows of 7168 bf16 values, residual in and out, rows and codes out
// (2.12 GB): 370 to 383 us, 5.6 TB/s, 95% of the rate of a plain copy (four chunks a thread:
// 422), with 72 registers and six waves a SIMD, three workgroups of 512.  Their gradient
// (1.88 GB): 336 us, 5.6 TB/s, and 7 for the sum of the partial rows, with 114 registers and four
// waves.  One row: 4.6 us, a launch and two dependent trips to memory.  The gradient of 16-bit
// rows of over 16384 values beside 32-bit sums spills 12 registers.
#include <algorithm>

#include "ep_combine.h"
#include "ep_kernels.h"
#include "layer_kernels.h"

namespace ep {
namespace {

constexpr int kHeld = 2;

// 8 values of a type: their loads and stores, and the conversions.
template <int T>
struct Chunk {
  u32x4 v[T == EP_ROWS_F32 ? 2 : 1];
  static constexpr int BYTES = T == EP_ROWS_F32 ? 32 : 16;

  // STREAM: past the caches' replacement
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const uint8_t* row, int c) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint8_t* p = row + (size_t)c * BYTES + i * 16;
      v[i] = STREAM && T != EP_ROWS_F32 ? load16_nt(p) : load16(p);
    }
  }
  template <bool STREAM = false>
  __device__ __forceinline__ void store(uint8_t* row, int c) const {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      uint8_t* p = row + (size_t)c * BYTES + i * 16;
      if constexpr (STREAM && T != EP_ROWS_F32)
        store16_nt(p, v[i]);
      else
        *(global_u32x4*)p = v[i];
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == EP_ROWS_F32) {
        f[i] = __uint_as_float(v[0][i]);
        f[4 + i] = __uint_as_float(v[BYTES / 16 - 1][i]);
      } else if constexpr (T == EP_ROWS_BF16) {
        f[2 * i] = bf16_lo(v[0][i]);
        f[2 * i + 1] = bf16_hi(v[0][i]);
      } else {
        f[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)v[0][i]);
        f[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[0][i] >> 16));
      }
    }
  }
  // rounded to nearest even
  __device__ __forceinline__ void put(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == EP_ROWS_F32) {
        v[0][i] = __float_as_uint(f[i]);
        v[BYTES / 16 - 1][i] = __float_as_uint(f[4 + i]);
      } else if constexpr (T == EP_ROWS_BF16) {
        v[0][i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      } else {
        v[0][i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[2 * i]) |
                  (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[2 * i + 1]) << 16;
      }
    }
  }
};

// The weights of a chunk, in the rows' type or in 32 bits.
template <int XT>
__device__ __forceinline__ void load_weight(float (&w)[8], const NormArgs& a, int c) {
  if (a.weight_f32) {
    Chunk<EP_ROWS_F32> k;
    k.load(a.weight, c);
    k.get(w);
  } else {
    Chunk<XT> k;
    k.load(a.weight, c);
    k.get(w);
  }
}

template <int TPR> constexpr int kBlock = TPR < 256 ? 256 : TPR;

// Rows of a workgroup at a time.
template <int TPR> constexpr int kSlots = kBlock<TPR> / TPR;

// Sums of N values over the TPR threads of a row, in an order that does not depend on
// anything but TPR.  `s` is LDS of 2 N kBlock / 64 floats, of which one half is used by one
// set of rows and the other by the next.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* s, int parity) {
  constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
  for (int d = 1; d < W; d <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], d);
  if constexpr (TPR > 64) {
    constexpr int WAVES = TPR / 64, ALL = kBlock<TPR> / 64;
    float* at = s + parity * N * ALL;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) at[i * ALL + wave] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v[i] += at[i * ALL + wave / WAVES * WAVES + w];
    }
  }
}

__device__ __forceinline__ float inverse_rms(float sum_sq, int n, float eps) {
  return 1.f / __builtin_sqrtf(sum_sq / (float)n + eps);
}

// The 8-bit form of a chunk; all 16 lanes of its block take part.  The scale stays a
// normal number, so that no quotient is over 448.
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t row, int c,
                                            const float (&y)[8]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __builtin_fmaxf(top, __builtin_fabsf(y[i]));
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
  const float scale = top > 0.f ? __builtin_fmaxf(top / 448.f, 0x1p-126f) : 1.f;
  u32x2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i] / scale, y[4 * i + 1] / scale, 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2] / scale, y[4 * i + 3] / scale, p, true);
    o[i] = (uint32_t)p;
  }
  *reinterpret_cast<u32x2*>(a.codes + row * a.N + (int64_t)c * 8) = o;
  if ((c & 15) == 0) a.scales[row * (a.N / 128) + c / 16] = scale;
}

template <int TPR, int XT, int RT, bool STREAM, bool EXTRA>
__global__ __launch_bounds__(kBlock<TPR>) void rms_norm_kernel(NormArgs a) {
  constexpr int SLOTS = kSlots<TPR>;
  __shared__ float s_sum[2 * kBlock<TPR> / 64];
  const int place = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int chunks = a.N / 8;
  int parity = 0;
  for (int64_t first = (int64_t)blockIdx.x * SLOTS; first < a.rows;
       first += (int64_t)gridDim.x * SLOTS, parity ^= 1) {
    const bool there = first + slot < a.rows;
    const int64_t row = there ? first + slot : a.rows - 1;
    const uint8_t* x = a.x + row * a.N * (Chunk<XT>::BYTES / 8);
    const uint8_t* res = a.residual ? a.residual + row * a.N * (Chunk<RT>::BYTES / 8) : nullptr;

    // s of a chunk; 0 past the row's end, where the last chunk is loaded again
    auto sum = [&](const Chunk<XT>& xc, const Chunk<RT>& rc, bool in, float (&s)[8]) {
      xc.get(s);
      if (res) {
        float r[8];
        rc.get(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = in ? s[i] : 0.f;
    };
    auto load_sum = [&](int c, float (&s)[8]) {
      Chunk<XT> xc;
      Chunk<RT> rc{};
      xc.template load<STREAM>(x, c);
      if (res) rc.template load<STREAM>(res, c);
      sum(xc, rc, true, s);
    };
    float held[kHeld][8], ss[1] = {0.f};
    {
      Chunk<XT> xc[kHeld];
      Chunk<RT> rc[kHeld] = {};
#pragma unroll
      for (int h = 0; h < kHeld; ++h) xc[h].template load<STREAM>(x, min(place + h * TPR, chunks - 1));
      if (res)
#pragma unroll
        for (int h = 0; h < kHeld; ++h) rc[h].template load<STREAM>(res, min(place + h * TPR, chunks - 1));
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        sum(xc[h], rc[h], place + h * TPR < chunks, held[h]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = __builtin_fmaf(held[h][i], held[h][i], ss[0]);
      }
    }
    if constexpr (EXTRA)
      for (int c = place + kHeld * TPR; c < chunks; c += TPR) {
        float s[8];
        load_sum(c, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = __builtin_fmaf(s[i], s[i], ss[0]);
      }
    row_sums<TPR>(ss, s_sum, parity);
    const float inv = inverse_rms(ss[0], a.N, a.eps);

    auto finish = [&](int c, const float (&s)[8]) {
      float y[8];
      load_weight<XT>(y, a, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= s[i] * inv;
      if (a.residual_out) {
        Chunk<RT> k;
        k.put(s);
        k.template store<STREAM>(a.residual_out + row * a.N * (Chunk<RT>::BYTES / 8), c);
      }
      if (a.out) {
        Chunk<XT> k;
        k.put(y);
        k.template store<STREAM>(a.out + row * a.N * (Chunk<XT>::BYTES / 8), c);
      }
      if (a.codes) store_codes(a, row, c, y);
    };
    if (there) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (place + h * TPR < chunks) finish(place + h * TPR, held[h]);
      if constexpr (EXTRA)
        for (int c = place + kHeld * TPR; c < chunks; c += TPR) {
          float s[8];
          load_sum(c, s);
          finish(c, s);
        }
    }
  }
}

// A workgroup adds up g r inv of its rows, column by column, in registers (beyond kHeld
// chunks a thread in its part of the workspace, which nothing else touches), joins the
// sums of its row slots and leaves them as one row of the workspace.
template <int TPR, int XT, int RT, bool STREAM, bool EXTRA>
__global__ __launch_bounds__(kBlock<TPR>) void rms_norm_backward_kernel(NormArgs a) {
  constexpr int SLOTS = kSlots<TPR>;
  __shared__ float s_sum[4 * kBlock<TPR> / 64];
  __shared__ float s_dw[SLOTS > 1 ? kBlock<TPR> * kHeld * 8 : 1];
  const int place = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int chunks = a.N / 8;
  float* mine = a.partial + (size_t)blockIdx.x * a.N;
  float dw[kHeld][8] = {};
  int parity = 0;
  bool begun = false;
  for (int64_t first = (int64_t)blockIdx.x * SLOTS; first < a.rows;
       first += (int64_t)gridDim.x * SLOTS, parity ^= 1) {
    const bool there = first + slot < a.rows;
    const int64_t row = there ? first + slot : a.rows - 1;
    const int64_t at_x = row * a.N * (Chunk<XT>::BYTES / 8);
    const int64_t at_r = row * a.N * (Chunk<RT>::BYTES / 8);
    const uint8_t *g = a.grad_out + at_x, *r = a.x + at_r;
    const uint8_t* h0 = a.grad_residual ? a.grad_residual + at_r : nullptr;

    float sums[2] = {0.f, 0.f};        // r^2 and g w r
    auto add = [&](const Chunk<XT>& gk, const Chunk<RT>& rk, int c, bool in) {
      float gv[8], rv[8], w[8];
      gk.get(gv);
      rk.get(rv);
      load_weight<XT>(w, a, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = in ? rv[i] : 0.f;
        sums[0] = __builtin_fmaf(v, v, sums[0]);
        sums[1] = __builtin_fmaf(in ? gv[i] * w[i] : 0.f, v, sums[1]);
      }
    };
    Chunk<XT> gc[kHeld];
    Chunk<RT> rc[kHeld], hc[kHeld] = {};
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const int c = min(place + h * TPR, chunks - 1);
      gc[h].template load<STREAM>(g, c);
      rc[h].template load<STREAM>(r, c);
    }
    if (h0)
#pragma unroll
      for (int h = 0; h < kHeld; ++h) hc[h].template load<STREAM>(h0, min(place + h * TPR, chunks - 1));
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      add(gc[h], rc[h], min(place + h * TPR, chunks - 1), place + h * TPR < chunks);
    if constexpr (EXTRA)
      for (int c = place + kHeld * TPR; c < chunks; c += TPR) {
        Chunk<XT> gk;
        Chunk<RT> rk;
        gk.template load<STREAM>(g, c);
        rk.template load<STREAM>(r, c);
        add(gk, rk, c, true);
      }
    row_sums<TPR>(sums, s_sum, parity);
    const float inv = inverse_rms(sums[0], a.N, a.eps);
    // inv^2 itself may be past binary32 (rows of rms under 2^-64 with an eps as small): one
    // factor goes to the mean, the other to r
    const float shift = inv * (sums[1] / (float)a.N);

    auto finish = [&](int c, const Chunk<XT>& gk, const Chunk<RT>& rk, const Chunk<RT>& hk,
                      float (&dwc)[8]) {
      float gv[8], rv[8], hv[8], d[8];
      gk.get(gv);
      rk.get(rv);
      hk.get(hv);                     // zeros where there is none
      load_weight<XT>(d, a, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = rv[i] * inv;
        d[i] = inv * __builtin_fmaf(gv[i], d[i], -xh * shift) + hv[i];
        dwc[i] = __builtin_fmaf(gv[i], xh, dwc[i]);
      }
      if (a.grad_x) {
        Chunk<XT> k;
        k.put(d);
        k.template store<STREAM>(a.grad_x + at_x, c);
      }
      if (a.grad_sum) {
        Chunk<RT> k;
        k.put(d);
        k.template store<STREAM>(a.grad_sum + at_r, c);
      }
    };
    if (there) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (place + h * TPR < chunks) finish(place + h * TPR, gc[h], rc[h], hc[h], dw[h]);
      if constexpr (EXTRA)
        for (int c = place + kHeld * TPR; c < chunks; c += TPR) {
          Chunk<XT> gk;
          Chunk<RT> rk, hk{};
          gk.template load<STREAM>(g, c);
          rk.template load<STREAM>(r, c);
          if (h0) hk.template load<STREAM>(h0, c);
          Chunk<EP_ROWS_F32> k{};
          float dwc[8];
          if (begun) k.load(reinterpret_cast<const uint8_t*>(mine), c);
          k.get(dwc);
          finish(c, gk, rk, hk, dwc);
          k.put(dwc);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            reinterpret_cast<u32x4*>(mine)[2 * (size_t)c + i] = k.v[i];
        }
    }
    begun = true;
  }
  // one row of partial sums; the slots of a row's columns in the order of the slots
  if constexpr (SLOTS > 1) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) s_dw[((slot * kHeld + h) * TPR + place) * 8 + i] = dw[h][i];
    __syncthreads();
    for (int n = threadIdx.x; n < a.N; n += kBlock<TPR>) {
      float v = 0.f;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) v += s_dw[s * TPR * kHeld * 8 + n];
      mine[n] = v;
    }
  } else {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (place + h * TPR < chunks) {
        Chunk<EP_ROWS_F32> k;
        k.put(dw[h]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          reinterpret_cast<u32x4*>(mine)[2 * (size_t)(place + h * TPR) + i] = k.v[i];
      }
  }
}

// grad_weight[n] = sum of the partial rows: a workgroup takes 32 columns, 8 lanes of 4 by 32
// groups of rows, and joins the groups through LDS.
__global__ __launch_bounds__(256) void add_partials_kernel(const float* partial, int parts, int N,
                                                           float* out) {
  __shared__ f32x4 s[256];
  const int q = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int64_t n = (int64_t)blockIdx.x * 32 + q * 4;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int p = g; p < parts; p += 32)
    v += *reinterpret_cast<const f32x4*>(partial + (size_t)p * N + n);
  s[threadIdx.x] = v;
  __syncthreads();
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    if (g < d) s[threadIdx.x] += s[threadIdx.x + d * 8];
    __syncthreads();
  }
  if (g == 0) *reinterpret_cast<f32x4*>(out + n) = s[threadIdx.x];
}

// Threads a row: as few as hold it in kHeld chunks each.
int threads_per_row(int N) {
  int tpr = 16;
  while (tpr < 1024 && tpr * kHeld < N / 8) tpr *= 2;
  return tpr;
}

int rows_per_block(int tpr) { return tpr < 256 ? 256 / tpr : 1; }

template <int TPR, int XT, int RT, bool STREAM, bool EXTRA = false>
void launch_one(const NormArgs& a, bool backward, int grid, hipStream_t st) {
  if (backward)
    hipLaunchKernelGGL((rms_norm_backward_kernel<TPR, XT, RT, STREAM, EXTRA>), dim3(grid),
                       dim3(kBlock<TPR>), 0, st, a);
  else
    hipLaunchKernelGGL((rms_norm_kernel<TPR, XT, RT, STREAM, EXTRA>), dim3(grid), dim3(kBlock<TPR>),
                       0, st, a);
}

template <int XT, int RT, bool STREAM>
void launch_types(const NormArgs& a, bool backward, int tpr, int grid, hipStream_t st) {
  switch (tpr) {
    case 16: return launch_one<16, XT, RT, STREAM>(a, backward, grid, st);
    case 32: return launch_one<32, XT, RT, STREAM>(a, backward, grid, st);
    case 64: return launch_one<64, XT, RT, STREAM>(a, backward, grid, st);
    case 128: return launch_one<128, XT, RT, STREAM>(a, backward, grid, st);
    case 256: return launch_one<256, XT, RT, STREAM>(a, backward, grid, st);
    case 512: return launch_one<512, XT, RT, STREAM>(a, backward, grid, st);
  }
  if (a.N / 8 <= 1024 * kHeld) return launch_one<1024, XT, RT, STREAM>(a, backward, grid, st);
  launch_one<1024, XT, RT, STREAM, true>(a, backward, grid, st);
}

// Bytes of the rows that a call reads and writes.
int64_t moved_bytes(const NormArgs& a, bool backward) {
  const int64_t x = a.dtype == EP_ROWS_F32 ? 4 : 2, s = a.sum_dtype == EP_ROWS_F32 ? 4 : 2;
  const int64_t value =
      backward ? x + s + (a.grad_residual ? s : 0) + (a.grad_x ? x : 0) + (a.grad_sum ? s : 0)
               : x + (a.residual ? s : 0) + (a.residual_out ? s : 0) + (a.out ? x : 0) +
                     (a.codes ? 1 : 0);
  return a.rows * a.N * value;
}

// Calls that move more than this go past the caches' replacement: the loads and stores of
// 16-bit values, whole lines.  (Those of 32-bit values, half of every 32 bytes each, never
// do.)  Measured on rows of 7168 values, us streamed and not, by the bytes moved:
//                      79 MB          99 MB          119 MB         159 MB         479 MB
//   norm, bf16
//     alone            17.2 and 16.9  20.7 and 22.9  23.4 and 25.5  30.9 and 33.1   87.3 and  92.3
//     with a residual  16.5 and 15.7  19.8 and 22.5  23.0 and 27.2  29.4 and 34.0   83.4 and  88.9
//     and codes        19.2 and 18.1  23.3 and 25.4  26.4 and 29.8  32.9 and 36.4   84.1 and  92.4
//     beside fp32 sums 17.4 and 16.5  20.3 and 21.4  24.3 and 28.9  34.0 and 35.6   87.2 and  89.9
//   gradient, bf16
//     alone            33.8 and 30.2  37.7 and 36.9  40.8 and 39.5  48.7 and 47.8  110.7 and 113.0
//     with a residual  32.0 and 27.4  34.2 and 31.9  38.7 and 38.0  44.5 and 44.3   98.8 and 102.9
//     beside fp32 sums 24.7 and 21.5  27.8 and 24.1  31.7 and 32.6  37.8 and 39.7   83.3 and  84.5
constexpr int64_t kStreamNorm = 88 << 20, kStreamGradient = 128 << 20;

template <int XT, int RT>
void launch_types(const NormArgs& a, bool backward, int tpr, int grid, hipStream_t st) {
  if constexpr (XT != EP_ROWS_F32)
    if (moved_bytes(a, backward) >= (backward ? kStreamGradient : kStreamNorm))
      return launch_types<XT, RT, true>(a, backward, tpr, grid, st);
  launch_types<XT, RT, false>(a, backward, tpr, grid, st);
}

hipError_t launch(const NormArgs& a, bool backward, int tpr, int grid, hipStream_t st) {
  const bool wide = a.sum_dtype != a.dtype;      // the sums in 32 bits beside 16-bit rows
  switch (a.dtype) {
    case EP_ROWS_F32:
      launch_types<EP_ROWS_F32, EP_ROWS_F32>(a, backward, tpr, grid, st);
      break;
    case EP_ROWS_BF16:
      if (wide)
        launch_types<EP_ROWS_BF16, EP_ROWS_F32>(a, backward, tpr, grid, st);
      else
        launch_types<EP_ROWS_BF16, EP_ROWS_BF16>(a, backward, tpr, grid, st);
      break;
    default:
      if (wide)
        launch_types<EP_ROWS_F16, EP_ROWS_F32>(a, backward, tpr, grid, st);
      else
        launch_types<EP_ROWS_F16, EP_ROWS_F16>(a, backward, tpr, grid, st);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, int num_cus, hipStream_t st) {
  const int tpr = threads_per_row(a.N);
  const int per = rows_per_block(tpr);
  const int64_t grid = std::min<int64_t>((a.rows + per - 1) / per, 16 * (int64_t)num_cus);
  return launch(a, false, tpr, (int)grid, st);
}

// Partial rows of the weights' gradient: one for each workgroup.  Workgroups have at least
// two sets of rows each, since a partial row costs twice its bytes (512 rows of 7168: one
// 19.9 us a call, two 16.0, four 16.8, eight 23.2).
int norm_backward_parts(int64_t rows, int N, int num_cus) {
  const int tpr = threads_per_row(N), per = 2 * rows_per_block(tpr);
  return (int)std::min<int64_t>((rows + per - 1) / per, 1024 / std::max(tpr, 256) * (int64_t)num_cus);
}

hipError_t launch_rms_norm_backward(const NormArgs& a, int num_cus, hipStream_t st) {
  const int parts = norm_backward_parts(a.rows, a.N, num_cus);
  if (parts > 0) {
    const hipError_t err = launch(a, true, threads_per_row(a.N), parts, st);
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(add_partials_kernel, dim3(a.N / 32), dim3(256), 0, st, a.partial, parts, a.N,
                     a.grad_weight);
  return hipGetLastError();
}

}  // namespace ep
