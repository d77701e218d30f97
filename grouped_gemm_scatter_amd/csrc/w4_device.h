// Device code shared by the kernels that read 4-bit weights and by those that read through
// buffer descriptors: code conversion, group scales, loads.
#pragma once

#include "ep_combine.h"
#include "ep_device.h"

namespace ep {

typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;

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

// Loads through buffer descriptors: the address is a scalar base and offset plus one
// 32-bit offset a lane, which all blocks and steps share.  (64-bit addresses of every
// block kept so many registers that some spilled, and a reload in the K loop waits for
// the weights in flight.)
typedef __amdgpu_buffer_rsrc_t buffer;
__device__ __forceinline__ buffer make_buffer(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)0xffffffff, 0x00020000);
}
// The same for step `at` of `end` (wave-uniform) where at < end, else a buffer that is empty:
// its loads give zeros and read nothing.  The length is the sign of a difference that the
// compiler does not see through: of a comparison it makes a vector register and a loop over
// the lanes around every load.
__device__ __forceinline__ int buffer_length(int at, int end) {
  int d = __builtin_amdgcn_readfirstlane(at - end);
  asm("" : "+s"(d));
  return d >> 31;
}
__device__ __forceinline__ buffer make_buffer(const void* p, int length) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, length, 0x00020000);
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

}  // namespace ep
