// Grouped products with 4-bit weights and group scales: the up-projection with
// SwiGLU and the down-projection with the receive-buffer sink, for row groups so
// small that streaming the weights is the time.
//
//   y[m][n] = sum over groups g of scale[n][g] * (sum over k in g of x[m][k] v(code[n][k]))
//
// The code values (integers -8..7, or e2m1) are exact in bf16, so the inner sums are
// v_mfma_f32_16x16x32_bf16 on exact operands, one fp32 accumulator per group, and a
// group's scale enters once, in fp32.
//
// Packed weights: 16 rows x 128 k are one run of 1024 bytes in the order the MFMA
// reads its second operand: lane L's 16 bytes are row L % 16, dword i of them the
// codes of k = 32 i + 8 (L / 16) + 0..7, so a wave loads 1 KB contiguously and every
// dword is one MFMA's operand.  A row's scales of those 128 k are contiguous too.
//
// A workgroup of 4 waves takes 64 rows x 128 GEMM columns of one expert (its work
// table, sink and completion are those of the other grouped GEMMs); a wave takes 32
// columns, two 16-column blocks, in the up-projection a gate block and the up
// block of the same outputs, so SwiGLU needs no exchange.
#include "ep_combine.h"
#include "gemm_common.h"

namespace ep {
namespace {

using namespace gemm;

typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;

constexpr int kW4Threads = 256;
constexpr int kW4Rows = 64;        // rows of a tile
constexpr int kW4Cols = 128;       // GEMM columns of a tile

// The 8 codes of a packed dword as bf16 values.
template <int CODES>
__device__ __forceinline__ bf16x8 decode8(uint32_t v) {
  bf16x8 r;
  if constexpr (CODES == EP_W4_E2M1) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, 3);
    r = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = (__bf16)((float)((v >> (4 * j)) & 15) - 8.f);
  }
  return r;
}

__device__ __forceinline__ float scale_value(uint16_t s, int f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, s) : bf16_lo(s);
}

template <int CODES, int GROUP, bool SWIGLU>
__global__ __launch_bounds__(kW4Threads) void gemm_w4_kernel(W4Args wa) {
  constexpr int MT = kW4Rows / 16;                   // 16-row blocks
  constexpr int SPT = 128 / GROUP;                   // scales of a row per 128 k
  constexpr int OUT = SWIGLU ? kW4Cols / 2 : kW4Cols;  // output columns of a tile
  constexpr int PITCH = OUT * 2 + 16;                // bytes per staged output row
  __shared__ __attribute__((aligned(16))) uint8_t smem[kW4Rows * PITCH];
  __shared__ uint64_t s_rowdst[kW4Rows];
  __shared__ int s_base[kMaxLocalExperts + 1];
  __shared__ int s_gbeg[kMaxLocalExperts + 1];
  __shared__ uint8_t* s_recv[kMaxRanks];
  __shared__ int s_bad;
  __shared__ uint32_t s_done[kDoneWords];
  __shared__ int s_pend[kPendingMax];

  const GemmArgs& a = wa.g;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = a.K, N = a.N, KT = K / 128, NB = N / 16;
  const int El = a.s.n_experts;
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < kMaxRanks; ++i) s_recv[i] = a.s.recv[i];
  }
  init_done(s_done);
  if (!build_work_table<kW4Rows, kW4Threads>(a, N / kW4Cols, s_base, s_gbeg, &s_bad)) return;
  const int total = s_base[El];
  const int G = gridDim.x, per_xcd = G >> 3;         // G is a multiple of 8
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  PendingTiles pending;
  pending.done = s_done;
  pending.e = s_pend;
  pending.base = s_base;

  for (int round = 0;; ++round) {
    const int item = round * G + xcd * per_xcd + slot;
    if (item >= total) break;
    const TileWork t = tile_of<kW4Rows, kW4Cols>(a, s_base, s_gbeg, item);
    if (t.empty) {
      signal_empty_expert(a, t.e, pending);
      continue;
    }
    if (pending.n >= kPendingMax) {
      wait_vm<0>();
      prologue_barrier(a, pending);
    }
    const RowInfo ri =
        tid < kW4Rows ? load_row_info(a, t.e, t.g1, t.m_abs + tid) : RowInfo{-1, 0, 0};
    // the wave's two 16-column blocks of the weights
    int nb[2];
    const int tile = t.n_abs / kW4Cols;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      nb[i] = SWIGLU ? tile * (OUT / 16) + wave + i * (NB / 2) : tile * (OUT / 16) + wave * 2 + i;
    const int mt = (t.rows + 15) / 16;
    f32x4 acc[2][MT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int kt = 0; kt < KT; ++kt) {
      bf16x8 xf[MT][4];
#pragma unroll
      for (int j = 0; j < MT; ++j)
        if (j < mt) {
          // rows past m_end read the group's last row; they are not stored
          const int m = min(t.m_abs + j * 16 + (lane & 15), t.g1 - 1);
          const uint8_t* xr = a.x + ((size_t)m * K + kt * 128 + (lane >> 4) * 8) * 2;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            xf[j][i] = __builtin_bit_cast(bf16x8, load16(xr + i * 64));
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t blk = ((size_t)t.e * NB + nb[i]) * KT + kt;
        const u32x4 w = load16_nt(a.w + blk * 1024 + lane * 16);
        const uint16_t* sp = wa.scales + (blk * 16 + (lane & 15)) * SPT;
        f32x4 part[MT];
#pragma unroll
        for (int s = 0; s < SPT; ++s) {
          const float sc = scale_value(sp[s], wa.scale_f16);
#pragma unroll
          for (int j = 0; j < MT; ++j) part[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 4 / SPT; ++q) {
            const bf16x8 wf = decode8<CODES>(w[s * (4 / SPT) + q]);
#pragma unroll
            for (int j = 0; j < MT; ++j)
              if (j < mt)
                part[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[j][s * (4 / SPT) + q], wf,
                                                                  part[j], 0, 0, 0);
          }
#pragma unroll
          for (int j = 0; j < MT; ++j)
            if (j < mt)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[i][j][r] = __builtin_fmaf(sc, part[j][r], acc[i][j][r]);
        }
      }
    }

    // lane L holds rows 4 (L / 16) + 0..3 of column L % 16 of each block: staged in
    // LDS as bf16 rows, then stored 16 bytes a thread
#pragma unroll
    for (int i = 0; i < (SWIGLU ? 1 : 2); ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
        if (j < mt)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float y = acc[i][j][r];
            int col = (wave * 2 + i) * 16 + (lane & 15);
            if constexpr (SWIGLU) {
              y = y / (1.f + expf(-y)) * acc[1][j][r];
              col = wave * 16 + (lane & 15);
            }
            const int m = j * 16 + (lane >> 4) * 4 + r;
            *reinterpret_cast<__bf16*>(smem + m * PITCH + col * 2) = (__bf16)y;
          }
    if constexpr (!SWIGLU) {
      if (tid < kW4Rows) s_rowdst[tid] = row_destination(a, s_recv, ri, t.m_abs + tid);
    }
    __syncthreads();
    constexpr int TPR = OUT * 2 / 16, RPP = kW4Threads / TPR;
    const int cc = tid % TPR;
    for (int r = tid / TPR; r < t.rows; r += RPP) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(smem + r * PITCH + cc * 16);
      if constexpr (SWIGLU) {
        store16_nt(a.c_local + ((size_t)(t.m_abs + r) * (N / 2) + tile * OUT) * 2 + cc * 16, v);
      } else {
        const uint64_t dst = s_rowdst[r];
        if (dst)
          store16_nt(reinterpret_cast<uint8_t*>(dst) + (size_t)t.n_abs * 2 + cc * 16, v);
      }
    }
    if constexpr (!SWIGLU) {
      if (tid == 0) pending.e[pending.n] = t.e;
      ++pending.n;
    }
    __syncthreads();   // the staged tile is read; the next one may overwrite it
  }
  if constexpr (!SWIGLU) flush_pending(a, pending);
}

// Output dword d of a block of 16 rows x 128 k: lane (d / 4) % 64, dword d % 4.
__global__ __launch_bounds__(256) void pack_w4_codes_kernel(const uint8_t* codes, uint8_t* out,
                                                            int64_t dwords, int k) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  const int KT = k / 128;
  for (int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x; o < dwords; o += stride) {
    const int64_t blk = o >> 8;
    const int d = (int)(o & 255), lane = d >> 2, i = d & 3;
    const int64_t row = blk / KT * 16 + (lane & 15);     // row of the whole stack
    const int64_t k0 = blk % KT * 128 + 32 * i + 8 * (lane >> 4);
    reinterpret_cast<uint32_t*>(out)[o] =
        *reinterpret_cast<const uint32_t*>(codes + (row * k + k0) / 2);
  }
}

__global__ __launch_bounds__(256) void pack_w4_scales_kernel(const uint16_t* scales, uint16_t* out,
                                                             int64_t count, int k, int group) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  const int KT = k / 128, spt = 128 / group, gpr = k / group;
  for (int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x; o < count; o += stride) {
    const int64_t blk = o / (16 * spt);
    const int d = (int)(o % (16 * spt));
    const int64_t row = blk / KT * 16 + d / spt;
    out[o] = scales[row * gpr + blk % KT * spt + d % spt];
  }
}

template <int CODES, int GROUP>
hipError_t launch(const W4Args& a, bool swiglu, dim3 grid, hipStream_t st) {
  const dim3 block(kW4Threads);
  if (swiglu)
    hipLaunchKernelGGL((gemm_w4_kernel<CODES, GROUP, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((gemm_w4_kernel<CODES, GROUP, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_w4(const W4Args& a, bool swiglu, int num_cus, hipStream_t st) {
  const int64_t nt = a.g.N / kW4Cols, El = a.g.s.n_experts;
  const int64_t items = (int64_t(a.g.m_total) / kW4Rows + El) * nt + El;   // upper bound
  int64_t g = items < 4 * (int64_t)num_cus ? items : 4 * (int64_t)num_cus;
  const dim3 grid((int)((g + 7) / 8 * 8));
  switch (a.codes * 1000 + a.group) {
    case 32: return launch<EP_W4_INT4, 32>(a, swiglu, grid, st);
    case 64: return launch<EP_W4_INT4, 64>(a, swiglu, grid, st);
    case 128: return launch<EP_W4_INT4, 128>(a, swiglu, grid, st);
    case 1032: return launch<EP_W4_E2M1, 32>(a, swiglu, grid, st);
    case 1064: return launch<EP_W4_E2M1, 64>(a, swiglu, grid, st);
    case 1128: return launch<EP_W4_E2M1, 128>(a, swiglu, grid, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_pack_w4(const uint8_t* codes, const uint16_t* scales, uint8_t* codes_out,
                          uint16_t* scales_out, int64_t experts, int rows, int k, int group,
                          int num_cus, hipStream_t st) {
  const int64_t dwords = experts * rows * k / 8, count = experts * rows * (k / group);
  const int64_t most = 16 * (int64_t)num_cus;
  const int64_t gc = (dwords + 255) / 256, gs = (count + 255) / 256;
  hipLaunchKernelGGL(pack_w4_codes_kernel, dim3((int)(gc < most ? gc : most)), dim3(256), 0, st,
                     codes, codes_out, dwords, k);
  hipLaunchKernelGGL(pack_w4_scales_kernel, dim3((int)(gs < most ? gs : most)), dim3(256), 0, st,
                     scales, scales_out, count, k, group);
  return hipGetLastError();
}

}  // namespace ep
