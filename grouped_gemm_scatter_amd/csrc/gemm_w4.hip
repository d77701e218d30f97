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
// The decode tile: a workgroup of 4 waves takes 64 rows x 256 GEMM columns of one
// expert (work table, sink and completion are those of the other grouped GEMMs), each
// wave four 16-column blocks over the whole of K, in the up-projection two gate
// blocks and the up blocks of the same outputs, so SwiGLU needs no exchange.
// The narrow tile, for launches with too few of those: the same with 128 columns.
// The thin tile, for launches with too few tiles of either to fill the GPU: 16 rows x 64
// columns, every wave a quarter of K, the quarters' sums joined through LDS.
//
// What bounds it.  32 experts of about 31 rows, 7168 -> 2 x 2048, int4, groups of 128:
// 122 us for 503 MB, 4.1 TB/s, 69% of the rate of a plain copy.  The loads by themselves
// took 79 us and the arithmetic by itself 105: a SIMD's conversions (13 vector
// instructions for 8 codes of a lane) and MFMAs (one for every 16 rows of them) add up,
// whatever the number of waves.  The down-projection with groups of 32 (e2m1): 78 us for
// 283 MB, of which the sink's publication at the end of the launch is 8.  A single token:
// 32 us for 121 MB up, 23 for 61 MB down, bound by the memory's latency at either end of
// a tile.  Few large groups (1650 rows over 16 experts, 1536 -> 4096): 56 us, bound by
// the arithmetic and by tiles that do not fill their last round.
// Measured and left: four workgroups a CU of 48 x 128 tiles (129 us up), three a CU (the
// registers spill), four steps of weights ahead (no faster up, 3% slower down), a raised
// wave priority around the products (no change).
#include "ep_combine.h"
#include "gemm_common.h"

namespace ep {
namespace {

using namespace gemm;

typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;

constexpr int kW4Threads = 256;
constexpr int kW4Waves = kW4Threads / 64;

// Tile of a launch: ROWS x COLS GEMM columns, K split over SPLIT waves, BLOCKS
// 16-column blocks a wave, PER_CU workgroups resident on a CU.
struct DecodeTile {
  static constexpr int ROWS = 64, COLS = 256, SPLIT = 1, BLOCKS = 4, PER_CU = 2;
};
struct NarrowTile {
  static constexpr int ROWS = 64, COLS = 128, SPLIT = 1, BLOCKS = 2, PER_CU = 2;
};
struct ThinTile {
  static constexpr int ROWS = 16, COLS = 64, SPLIT = 4, BLOCKS = 4, PER_CU = 4;
};

// 1/16 of the signed integer in the low half of byte B.  (The mask makes the compiler select
// the byte in the conversion; that is left to it, since only then it keeps the conversion's
// result off registers that a matrix instruction still reads.)
template <int B>
__device__ __forceinline__ float off_i4(uint32_t v) {
  return __builtin_amdgcn_cvt_off_f32_i4((v >> (8 * B)) & 0xffu);
}

// The 8 codes of a packed dword as bf16 values: e2m1 values, or (code - 8) / 16.
// Both are exact: 4 conversions for e2m1, for int4 a shift, 8 conversions (the
// instruction takes a byte's low half) and 4 roundings of exact numbers.
// (int4 as unsigned codes through the fp8 conversion, 7 instructions, with -8 sum x
// from one more MFMA for each X fragment: the same time within 2%, and inexact zeros.)
template <int CODES>
__device__ __forceinline__ bf16x8 decode8(uint32_t v) {
  if constexpr (CODES == EP_W4_E2M1) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    // packed as two's complement, codes 0..3 in the low and 4..7 in the high halves of
    // the bytes
    const float l0 = off_i4<0>(v), l1 = off_i4<1>(v), l2 = off_i4<2>(v), l3 = off_i4<3>(v);
    v >>= 4;
    asm("" : "+v"(v));               // one shift for all, not one for each byte
    const float h0 = off_i4<0>(v), h1 = off_i4<1>(v), h2 = off_i4<2>(v), h3 = off_i4<3>(v);
    return bf16x8{(__bf16)l0, (__bf16)l1, (__bf16)l2, (__bf16)l3,
                  (__bf16)h0, (__bf16)h1, (__bf16)h2, (__bf16)h3};
  }
}

// A row's 2-byte scales of 128 k as one value.
template <int N> struct ScaleWord { typedef uint16_t type; };
template <> struct ScaleWord<2> { typedef uint32_t type; };
template <> struct ScaleWord<4> { typedef uint64_t type; };

// A weight format: code type, group and type of the scales.
template <int CODES_, int GROUP_, bool F16>
struct Format {
  static constexpr int CODES = CODES_, GROUP = GROUP_;
  typedef typename ScaleWord<128 / GROUP>::type word;
  static __device__ __forceinline__ float scale(uint16_t s) {
    constexpr float m = CODES == EP_W4_INT4 ? 16.f : 1.f;    // decode8's 1/16
    if constexpr (F16) return m * (float)__builtin_bit_cast(_Float16, s);
    return m * bf16_lo(s);
  }
};

// The codes and scales of one step of 128 k: NT 16-column blocks.
template <class F, int NT>
struct Weights {
  u32x4 w[NT];
  typename F::word s[NT];
};

// Loads through buffer descriptors: the address is a scalar base and offset plus one
// 32-bit offset a lane, which all blocks and steps share.  (64-bit addresses of every
// block kept so many registers that some spilled, and a reload in the K loop waits for
// the weights in flight.)
typedef __amdgpu_buffer_rsrc_t buffer;
__device__ __forceinline__ buffer make_buffer(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)0xffffffff, 0x00020000);
}
constexpr int kNontemporal = 2;
__device__ __forceinline__ u32x4 buffer_load16(buffer b, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, voff, soff, 0));
}
__device__ __forceinline__ u32x4 buffer_load16_nt(buffer b, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4,
                            __builtin_amdgcn_raw_buffer_load_b128(b, voff, soff, kNontemporal));
}
__device__ __forceinline__ void buffer_load_to(uint16_t& v, buffer b, uint32_t vo, uint32_t so) {
  v = __builtin_amdgcn_raw_buffer_load_b16(b, vo, so, 0);
}
__device__ __forceinline__ void buffer_load_to(uint32_t& v, buffer b, uint32_t vo, uint32_t so) {
  v = __builtin_amdgcn_raw_buffer_load_b32(b, vo, so, 0);
}
__device__ __forceinline__ void buffer_load_to(uint64_t& v, buffer b, uint32_t vo, uint32_t so) {
  v = __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(b, vo, so, 0));
}

// Where a wave's column blocks are: an expert's codes and scales, and the wave-uniform
// number of each block's first run of 1 KB.
template <int NT>
struct Blocks {
  buffer w, s;
  uint32_t run[NT];
};

template <class F, int NT>
__device__ __forceinline__ void load_weights(Weights<F, NT>& st, const Blocks<NT>& src, int kt,
                                             int lane) {
  constexpr uint32_t SB = 16 * (128 / F::GROUP) * 2;   // scale bytes of a run
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const uint32_t run = src.run[i] + kt;
    st.w[i] = buffer_load16_nt(src.w, lane * 16, run * 1024);
    buffer_load_to(st.s[i], src.s, (lane & 15) * (SB / 16), run * SB);
  }
}

// acc += scale * part, for one block.  The sums are made here: left free, the compiler
// sinks them past the next branch and keeps every `part` of a step in registers.
template <int MT>
__device__ __forceinline__ void add_group(f32x4 (&acc)[MT], const f32x4 (&part)[MT], float sc) {
#pragma unroll
  for (int j = 0; j < MT; ++j) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[j][r] = __builtin_fmaf(sc, part[j][r], acc[j][r]);
    asm volatile("" : "+v"(acc[j]));
  }
}

// One step: x(j, q) is the X fragment of row block j and quarter q of the 128 k.
template <class F, int MT, int NT, class X>
__device__ __forceinline__ void multiply_step(f32x4 (&acc)[NT][MT], const Weights<F, NT>& st,
                                              X x) {
  constexpr int SPT = 128 / F::GROUP, QPS = 4 / SPT;    // scales of a row per 128 k; quarters a scale
  // X fragments of a whole group for all blocks, or where those are many, of a quarter
  // at a time for two column blocks
  constexpr bool BY_QUARTER = QPS > 1 && (NT == 2 || QPS * MT > 8);
  constexpr int IB = BY_QUARTER ? 2 : NT;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i0 = 0; i0 < NT; i0 += IB)
#pragma unroll
    for (int s = 0; s < SPT; ++s) {
      if constexpr (BY_QUARTER) {
        f32x4 part[IB][MT];
#pragma unroll
        for (int q = 0; q < QPS; ++q) {
          bf16x8 xf[MT];
#pragma unroll
          for (int j = 0; j < MT; ++j) xf[j] = x(j, s * QPS + q);
#pragma unroll
          for (int i = 0; i < IB; ++i) {
            const bf16x8 wf = decode8<F::CODES>(st.w[i0 + i][s * QPS + q]);
#pragma unroll
            for (int j = 0; j < MT; ++j)
              part[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  xf[j], wf, q ? part[i][j] : zero, 0, 0, 0);
          }
        }
#pragma unroll
        for (int i = 0; i < IB; ++i)
          add_group(acc[i0 + i], part[i], F::scale((uint16_t)(st.s[i0 + i] >> (16 * s))));
      } else {
        bf16x8 xf[MT][QPS];
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int q = 0; q < QPS; ++q) xf[j][q] = x(j, s * QPS + q);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          f32x4 part[MT];
#pragma unroll
          for (int q = 0; q < QPS; ++q) {
            const bf16x8 wf = decode8<F::CODES>(st.w[i][s * QPS + q]);
#pragma unroll
            for (int j = 0; j < MT; ++j)
              part[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[j][q], wf, q ? part[j] : zero,
                                                                0, 0, 0);
          }
          add_group(acc[i], part, F::scale((uint16_t)(st.s[i] >> (16 * s))));
        }
      }
    }
}

// Waits for this wave's LDS accesses only, then for the workgroup: loads from global
// memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);                // lgkmcnt(0)
  raw_barrier();
}

// The decode tile's K loop.  All waves multiply the same X rows, which pass through
// LDS, two buffers of 128 k: the workgroup loads step k + 2 into registers while step k
// is multiplied, and writes it to LDS at the next step.  A row's sixteen 16-byte
// chunks are stored XORed with the row, so that neither the writes (a row by sixteen
// lanes) nor the reads (a chunk of sixteen rows) meet in a bank.  The weights of three
// steps are in registers or on their way.
template <class F, int MT, int NT>
__device__ __forceinline__ void multiply_shared(f32x4 (&acc)[NT][MT], const Blocks<NT>& src,
                                                buffer x, const uint32_t (&xoff)[MT],
                                                uint8_t* xs, int KT, int tid) {
  constexpr int BUF = MT * 4096;
  const int lane = tid & 63, row = tid >> 4;
  uint8_t* put = xs + row * 256 + ((tid & 15) ^ row) * 16;
  u32x4 xr[MT];
  Weights<F, NT> st[3];
  auto load_x = [&](int k) {
#pragma unroll
    for (int p = 0; p < MT; ++p) xr[p] = buffer_load16(x, xoff[p], k * 256);
  };
  auto put_x = [&](int k) {
#pragma unroll
    for (int p = 0; p < MT; ++p)
      *reinterpret_cast<u32x4*>(put + (k & 1) * BUF + p * 4096) = xr[p];
  };
  // The loads ahead are unconditional, past the end those of the last step again: with a
  // load under a condition the compiler does not know how many came after the one
  // that it waits for, and waits for all.
  auto step = [&](int k, Weights<F, NT>& w) {
    put_x(k + 1);
    load_x(min(k + 2, KT - 1));
    const uint8_t* xb = xs + (k & 1) * BUF + (lane & 15) * 256;
    multiply_step(acc, w, [&](int j, int q) {
      return *reinterpret_cast<const bf16x8*>(xb + j * 4096 +
                                              ((4 * q + (lane >> 4)) ^ (lane & 15)) * 16);
    });
    load_weights(w, src, min(k + 3, KT - 1), lane);
    lds_barrier();
  };
  load_x(0);
#pragma unroll
  for (int d = 0; d < 3; ++d) load_weights(st[d], src, min(d, KT - 1), lane);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  put_x(0);
  load_x(min(1, KT - 1));
  lds_barrier();
  for (int k = 0;;) {
    step(k, st[0]);
    if (++k >= KT) break;
    step(k, st[1]);
    if (++k >= KT) break;
    step(k, st[2]);
    if (++k >= KT) break;
  }
}

// The thin tile's: steps [k0, k1) of 16 rows, each wave its own k, X straight from L2.
template <class F, int NT>
struct ThinStep {
  Weights<F, NT> w;
  bf16x8 x[4];
};

template <class F, int NT>
__device__ __forceinline__ void multiply_thin(f32x4 (&acc)[NT][1], const Blocks<NT>& src,
                                              buffer x, uint32_t xoff, int k0, int k1,
                                              int lane) {
  ThinStep<F, NT> a, b;
  auto load = [&](ThinStep<F, NT>& st, int k) {
    load_weights(st.w, src, k, lane);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      st.x[q] = __builtin_bit_cast(bf16x8, buffer_load16(x, xoff + q * 64, k * 256));
  };
  auto multiply = [&](const ThinStep<F, NT>& st) {
    multiply_step(acc, st.w, [&](int, int q) { return st.x[q]; });
  };
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (k0 >= k1) return;
  load(a, k0);
  load(b, min(k0 + 1, k1 - 1));
  for (int k = k0;;) {
    multiply(a);
    load(a, min(k + 2, k1 - 1));
    if (++k >= k1) break;
    multiply(b);
    load(b, min(k + 2, k1 - 1));
    if (++k >= k1) break;
  }
}

// Staged output rows: lane L holds rows 4 (L / 16) + 0..3 of column L % 16 of a block.
template <int MT>
__device__ __forceinline__ void stage_block(uint8_t* smem, int pitch, const f32x4 (&y)[MT], int col,
                                            int lane) {
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<__bf16*>(smem + (j * 16 + (lane >> 4) * 4 + r) * pitch +
                                 (col + (lane & 15)) * 2) = (__bf16)y[j][r];
}

template <int MT>
__device__ __forceinline__ void swiglu(f32x4 (&g)[MT], const f32x4 (&u)[MT]) {
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) g[j][r] = g[j][r] / (1.f + expf(-g[j][r])) * u[j][r];
}

// build_work_table with the prefix over the experts made by a scan of one wave: the
// launch is short enough for a sequential prefix (1 us for 32 experts, 8 for 256) to count.
template <int BM>
__device__ __forceinline__ bool build_table(const GemmArgs& a, int nt, int* s_base, int* s_gbeg,
                                            int* s_bad) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int R = a.s.n_ranks, El = a.s.n_experts;
  if (tid == 0) *s_bad = 0;
  __syncthreads();
  for (int i = tid; i <= El * R; i += kW4Threads) {
    const int v = a.offsets[i], before = i > 0 ? a.offsets[i - 1] : 0;
    if (v < before || v > a.m_total || (i == 0 && v != 0) || (i == El * R && v != a.m_total))
      *s_bad = 1;
    if (i % R == 0) s_gbeg[i / R] = v;
  }
  __syncthreads();
  if (*s_bad) {
    if (tid == 0 && blockIdx.x == 0) latch_error(a.s.err, kErrBadGroup);
    return false;
  }
  if (tid < 64) {
    int base = 0;
    for (int e0 = 0; e0 < El; e0 += 64) {
      const int e = e0 + lane;
      int n = 0;                     // items of expert e: its tiles, or one to signal
      if (e < El) {
        const int me = s_gbeg[e + 1] - s_gbeg[e];
        n = me ? (me + BM - 1) / BM * nt : 1;
      }
      int sum = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(sum, d);
        if (lane >= d) sum += up;
      }
      if (e < El) s_base[e] = base + sum - n;
      base += __shfl(sum, 63);
    }
    if (lane == 0) s_base[El] = base;
  }
  __syncthreads();
  return true;
}

// The products of one tile with MT 16-row blocks, staged in LDS as bf16 rows.
template <class T, class F, bool SWIGLU, int MT>
__device__ __forceinline__ void tile_product(const W4Args& wa, const TileWork& t, uint8_t* smem,
                                             int pitch, int tid, int wave) {
  const GemmArgs& a = wa.g;
  // opaque, so that what derives from it is computed for each tile, not kept for every
  // tile shape across the others' K loops
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63;
  const int KT = a.K / 128, NB = a.N / 16;
  constexpr int PER = T::COLS / 16;                  // blocks of a tile
  constexpr int NT = T::BLOCKS;
  const int tile = t.n_abs / T::COLS;
  const int first = T::SPLIT > 1 ? 0 : wave * NT;
  // the wave's first output block of the tile, and its weight blocks
  const int ob = SWIGLU ? first / 2 : first;
  Blocks<NT> src;
  const size_t first_run = (size_t)t.e * NB * KT;
  src.w = make_buffer(a.w + first_run * 1024);
  src.s = make_buffer(wa.scales + first_run * (16 * (128 / F::GROUP)));
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    int nb = SWIGLU ? tile * (PER / 2) + ob + (i % (NT / 2)) + (i / (NT / 2)) * (NB / 2)
                    : tile * PER + ob + i;
    if constexpr (!SWIGLU) nb = min(nb, NB - 1);     // past the last column: not stored
    src.run[i] = (uint32_t)nb * KT;
  }
  // from the tile's first row, so that 32-bit offsets reach whatever m_total is
  const buffer x = make_buffer(a.x + (size_t)t.m_abs * a.K * 2);
  // rows past m_end read the group's last row; they are not stored
  auto row_offset = [&](int r) { return (uint32_t)min(r, t.g1 - 1 - t.m_abs) * (uint32_t)(a.K * 2); };
  f32x4 acc[NT][MT];
  if constexpr (T::SPLIT > 1) {
    static_assert(T::SPLIT == kW4Waves && NT == kW4Waves && MT == 1, "one block a wave at the end");
    // the wave's share of K
    multiply_thin<F>(acc, src, x, row_offset(lane & 15) + (lane >> 4) * 16,
                     wave * KT / T::SPLIT, (wave + 1) * KT / T::SPLIT, lane);
    // wave w adds up block w of all shares, in the order of k
    __shared__ f32x4 s_part[T::SPLIT][NT][64];
#pragma unroll
    for (int i = 0; i < NT; ++i) s_part[wave][i][lane] = acc[i][0];
    __syncthreads();
    f32x4 y[SWIGLU ? 2 : 1][1];
    const int mine = SWIGLU ? wave % (NT / 2) : wave;
#pragma unroll
    for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
      y[h][0] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < T::SPLIT; ++p) y[h][0] += s_part[p][mine + h * (NT / 2)][lane];
    }
    if constexpr (SWIGLU) swiglu(y[0], y[1]);
    if (!SWIGLU || wave < NT / 2) stage_block(smem, pitch, y[0], mine * 16, lane);
  } else {
    uint32_t xoff[MT];
#pragma unroll
    for (int p = 0; p < MT; ++p) xoff[p] = row_offset(p * 16 + (tid >> 4)) + (tid & 15) * 16;
    multiply_shared<F>(acc, src, x, xoff, smem, KT, tid);
    if constexpr (SWIGLU) {
#pragma unroll
      for (int i = 0; i < NT / 2; ++i) {
        swiglu(acc[i], acc[i + NT / 2]);
        stage_block(smem, pitch, acc[i], (ob + i) * 16, lane);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i) stage_block(smem, pitch, acc[i], (ob + i) * 16, lane);
    }
  }
}

template <class T, class F, bool SWIGLU>
__global__ __launch_bounds__(kW4Threads, T::PER_CU) void gemm_w4_kernel(W4Args wa) {
  constexpr int OUT = SWIGLU ? T::COLS / 2 : T::COLS;  // output columns of a tile
  constexpr int PITCH = OUT * 2 + 16;                // bytes per staged output row
  // the X rows on their way to the MFMAs, and after the K loop the finished tile
  constexpr int X_BYTES = T::SPLIT > 1 ? 0 : 2 * T::ROWS * 256, C_BYTES = T::ROWS * PITCH;
  __shared__ __attribute__((aligned(16))) uint8_t smem[X_BYTES > C_BYTES ? X_BYTES : C_BYTES];
  __shared__ uint64_t s_rowdst[T::ROWS];
  __shared__ int s_base[kMaxLocalExperts + 1];
  __shared__ int s_gbeg[kMaxLocalExperts + 1];
  __shared__ uint8_t* s_recv[kMaxRanks];
  __shared__ int s_bad;
  __shared__ uint32_t s_done[kDoneWords];
  __shared__ int s_pend[kPendingMax];

  const GemmArgs& a = wa.g;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int El = a.s.n_experts;
  const int width = SWIGLU ? a.N / 2 : a.N;          // output columns of a row
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < kMaxRanks; ++i) s_recv[i] = a.s.recv[i];
  }
  init_done(s_done);
  if (!build_table<T::ROWS>(a, (a.N + T::COLS - 1) / T::COLS, s_base, s_gbeg, &s_bad)) return;
  const int total = s_base[El];
  const int per_xcd = gridDim.x >> 3;                // the grid is a multiple of 8
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  PendingTiles pending;
  pending.done = s_done;
  pending.e = s_pend;
  pending.base = s_base;

  // each XCD (workgroups go round-robin over the eight) takes an equal run of the items,
  // its workgroups in turn
  const int end = (int)((int64_t)(xcd + 1) * total / 8);
  for (int item = (int)((int64_t)xcd * total / 8) + slot; item < end; item += per_xcd) {
    TileWork t = tile_of<T::ROWS, T::COLS>(a, s_base, s_gbeg, item);
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.g1 = __builtin_amdgcn_readfirstlane(t.g1);
    t.m_abs = __builtin_amdgcn_readfirstlane(t.m_abs);
    t.n_abs = __builtin_amdgcn_readfirstlane(t.n_abs);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if (t.empty) {
      signal_empty_expert(a, t.e, pending);
      continue;
    }
    if (pending.n >= kPendingMax) {
      wait_vm<0>();
      prologue_barrier<true>(a, pending);
    }
    // where the rows go: put into LDS at once, so that no register holds it across the K
    // loop, but in the thin tile, whose K loop is shorter than these loads
    RowInfo ri{-1, 0, 0};
    if constexpr (!SWIGLU) {
      if (tid < T::ROWS) {
        ri = load_row_info(a, t.e, t.g1, t.m_abs + tid);
        if (T::SPLIT == 1) s_rowdst[tid] = row_destination(a, s_recv, ri, t.m_abs + tid);
      }
    }
    const int mt = (t.rows + 15) / 16;
    if (T::ROWS == 16 || mt == 1)
      tile_product<T, F, SWIGLU, 1>(wa, t, smem, PITCH, tid, wave);
    else if (mt == 2)
      tile_product<T, F, SWIGLU, T::ROWS == 16 ? 1 : 2>(wa, t, smem, PITCH, tid, wave);
    else if (mt == 3)
      tile_product<T, F, SWIGLU, T::ROWS == 16 ? 1 : 3>(wa, t, smem, PITCH, tid, wave);
    else
      tile_product<T, F, SWIGLU, T::ROWS == 16 ? 1 : 4>(wa, t, smem, PITCH, tid, wave);
    if constexpr (!SWIGLU && T::SPLIT > 1) {
      if (tid < T::ROWS) s_rowdst[tid] = row_destination(a, s_recv, ri, t.m_abs + tid);
    }
    __syncthreads();
    const int col0 = t.n_abs / T::COLS * OUT;
    if (SWIGLU || !a.sink_on) {
      constexpr int TPR = OUT * 2 / 16, RPP = kW4Threads / TPR;
      const int cc = tid % TPR, col = col0 + cc * 8;
      if (col < width)
        for (int r = tid / TPR; r < t.rows; r += RPP)
          store16_nt(a.c_local + ((size_t)(t.m_abs + r) * width + col) * 2,
                     *reinterpret_cast<const u32x4*>(smem + r * PITCH + cc * 16));
    } else {
      // sent rows are written through: a fence per workgroup, each a write-back of its
      // XCD's L2, took 39 of the 62 us of a one-token launch and 20 of a decode step's 95
      constexpr int TPR = OUT * 2 / 16, RPP = kW4Threads / TPR;
      const int cc = tid % TPR, col = col0 + cc * 8;
      if (col < width)
        for (int r = tid / TPR; r < t.rows; r += RPP) {
          const uint64_t dst = s_rowdst[r];
          if (dst)
            store16_through(reinterpret_cast<uint8_t*>(dst) + (size_t)col * 2,
                            *reinterpret_cast<const u32x4*>(smem + r * PITCH + cc * 16));
        }
    }
    if constexpr (!SWIGLU) {
      if (tid == 0) pending.e[pending.n] = t.e;
      ++pending.n;
    }
    __syncthreads();   // the staged tile is read; the next one may overwrite it
  }
  if constexpr (!SWIGLU) flush_pending<true>(a, pending);
}

// Output dword d of a block of 16 rows x 128 k: lane (d / 4) % 64, dword d % 4.
__global__ __launch_bounds__(256) void pack_w4_codes_kernel(const uint8_t* codes, uint8_t* out,
                                                            int64_t dwords, int k, bool int4) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  const int KT = k / 128;
  for (int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x; o < dwords; o += stride) {
    const int64_t blk = o >> 8;
    const int d = (int)(o & 255), lane = d >> 2, i = d & 3;
    const int64_t row = blk / KT * 16 + (lane & 15);     // row of the whole stack
    const int64_t k0 = blk % KT * 128 + 32 * i + 8 * (lane >> 4);
    uint32_t v = *reinterpret_cast<const uint32_t*>(codes + (row * k + k0) / 2);
    if (int4) {
      // codes 0..3 to the low, 4..7 to the high halves of the bytes, as two's
      // complement of code - 8
      uint32_t r = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) r |= (v >> (4 * j) & 15u) << (8 * (j & 3) + (j & 4));
      v = r ^ 0x88888888u;
    }
    reinterpret_cast<uint32_t*>(out)[o] = v;
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

template <class T, class F>
hipError_t launch_tile(const W4Args& a, bool swiglu, int num_cus, hipStream_t st) {
  const int64_t nt = (a.g.N + T::COLS - 1) / T::COLS, El = a.g.s.n_experts;
  const int64_t items = (int64_t(a.g.m_total) / T::ROWS + El) * nt + El;   // upper bound
  const int64_t most = T::PER_CU * (int64_t)num_cus;
  const int64_t g = items < most ? items : most;
  const dim3 grid((int)((g + 7) / 8 * 8)), block(kW4Threads);
  if (swiglu)
    hipLaunchKernelGGL((gemm_w4_kernel<T, F, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((gemm_w4_kernel<T, F, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

// The tile by how many of each a launch is likely to have (only the device knows the
// groups): an expert's last tile is half full on average, and every expert has one.
// Measured at K 2048, group 64, equal groups, us (decode / narrow / thin tile):
//   E  4, N 2048, 16 rows each   21.3 / 14.4 /  9.8   128 thin tiles
//   E 16, N 2048, 16 rows        21.9 / 15.4 / 15.2   512
//   E  4, N 7168, 24 rows        23.4 / 16.7 / 21.8   896
//   E 32, N 2048,  1 row         23.7 / 20.6 / 21.1   1024, of one row
//   E 32, N 2048, 64 rows        32.1 / 29.6 / 72.7   512 narrow tiles
//   E 16, N 7168,  8 rows        32.4 / 35.2 / 35.9   896
//   E 32, N 2048, 128 rows       45.7 / 55.7 / 134    1024
// so: thin tiles up to two a CU, or up to four where they have few rows to repeat the
// weights for; narrow ones up to two a CU, which is one round of them; else the largest.
template <class F>
hipError_t launch(const W4Args& a, bool swiglu, int num_cus, hipStream_t st) {
  const int64_t El = a.g.s.n_experts, m = a.g.m_total, active = m < El ? m : El;
  auto tiles = [&](int rows, int cols) {
    const int64_t by_rows = m / rows + active / 2;
    return (by_rows > active ? by_rows : active) * ((a.g.N + cols - 1) / cols);
  };
  if (tiles(ThinTile::ROWS, ThinTile::COLS) <= (m <= 8 * active ? 4 : 2) * (int64_t)num_cus)
    return launch_tile<ThinTile, F>(a, swiglu, num_cus, st);
  if (tiles(NarrowTile::ROWS, NarrowTile::COLS) <= 2 * (int64_t)num_cus)
    return launch_tile<NarrowTile, F>(a, swiglu, num_cus, st);
  return launch_tile<DecodeTile, F>(a, swiglu, num_cus, st);
}

template <int CODES, int GROUP>
hipError_t launch(const W4Args& a, bool swiglu, int num_cus, hipStream_t st) {
  return a.scale_f16 ? launch<Format<CODES, GROUP, true>>(a, swiglu, num_cus, st)
                     : launch<Format<CODES, GROUP, false>>(a, swiglu, num_cus, st);
}

}  // namespace

hipError_t launch_gemm_w4(const W4Args& a, bool swiglu, int num_cus, hipStream_t st) {
  switch (a.codes * 1000 + a.group) {
    case 32: return launch<EP_W4_INT4, 32>(a, swiglu, num_cus, st);
    case 64: return launch<EP_W4_INT4, 64>(a, swiglu, num_cus, st);
    case 128: return launch<EP_W4_INT4, 128>(a, swiglu, num_cus, st);
    case 1032: return launch<EP_W4_E2M1, 32>(a, swiglu, num_cus, st);
    case 1064: return launch<EP_W4_E2M1, 64>(a, swiglu, num_cus, st);
    case 1128: return launch<EP_W4_E2M1, 128>(a, swiglu, num_cus, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_pack_w4(const uint8_t* codes, const uint16_t* scales, uint8_t* codes_out,
                          uint16_t* scales_out, int64_t experts, int rows, int k, int group,
                          bool int4, int num_cus, hipStream_t st) {
  const int64_t dwords = experts * rows * k / 8, count = experts * rows * (k / group);
  const int64_t most = 16 * (int64_t)num_cus;
  const int64_t gc = (dwords + 255) / 256, gs = (count + 255) / 256;
  hipLaunchKernelGGL(pack_w4_codes_kernel, dim3((int)(gc < most ? gc : most)), dim3(256), 0, st,
                     codes, codes_out, dwords, k, int4);
  hipLaunchKernelGGL(pack_w4_scales_kernel, dim3((int)(gs < most ? gs : most)), dim3(256), 0, st,
                     scales, scales_out, count, k, group);
  return hipGetLastError();
}

}  // namespace ep
