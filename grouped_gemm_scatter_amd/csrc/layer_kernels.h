// Kernel argument blocks and launchers of the calls around the EP-combine step: the norm in
// front of the layer and the layer for a few tokens.  (Apart from ep_kernels.h, which is
// part of the step's kernels: their stored HBM traffic holds while their sources do.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ep {

// RMS norm of rows and its gradient.
struct NormArgs {
  const uint8_t* x;          // [rows][N] dtype; backward: the stored sums, sum_dtype
  const uint8_t* residual;   // [rows][N] sum_dtype, or null
  const uint8_t* weight;     // [N] dtype, or fp32 with weight_f32
  uint8_t* residual_out;     // [rows][N] sum_dtype, or null
  uint8_t* out;              // [rows][N] dtype, or null
  uint8_t* codes;            // [rows][N] e4m3fn, or null
  float* scales;             // [rows][N/128]
  // backward
  const uint8_t* grad_out;        // [rows][N] dtype
  const uint8_t* grad_residual;   // [rows][N] sum_dtype, or null
  uint8_t* grad_x;                // [rows][N] dtype, or null
  uint8_t* grad_sum;              // [rows][N] sum_dtype, or null
  float* grad_weight;             // [N]
  float* partial;                 // [norm_backward_parts()][N]
  int64_t rows;
  int32_t N;                 // multiple of 128
  int32_t dtype;             // EP_ROWS_*
  int32_t sum_dtype;         // dtype or fp32
  int32_t weight_f32;
  float eps;
};
hipError_t launch_rms_norm(const NormArgs& a, int num_cus, hipStream_t st);
hipError_t launch_rms_norm_backward(const NormArgs& a, int num_cus, hipStream_t st);
int norm_backward_parts(int64_t rows, int N, int num_cus);

// Weights of one product of the layer for a few tokens.
struct MoeWeights {
  const uint8_t* w;          // bf16 rows, e4m3fn codes or packed 4-bit codes
  const void* scales;        // fp8: fp32 [E_l][rows/128][k/128]; 4-bit: packed
  int32_t codes;             // 4-bit: EP_W4_*
  int32_t group;             // 4-bit: 32, 64 or 128; 0: the handle's own dtype
  int32_t scale_f16;
  int32_t slice_major;       // bf16: [k/64][rows][64] within an expert
};

// The whole layer for a few tokens.
struct MoeArgs {
  const uint8_t* x;          // [tokens][hidden] bf16, or e4m3fn with x_scale
  const float* x_scale;      // [tokens][hidden/128] (fp8)
  const int32_t* topk_ids;   // [tokens][top_k]
  const float* topk_w;       // [tokens][top_k]
  uint8_t* h;                // workspace: [tokens*top_k][2][inter] bf16, two parts of a value
  uint8_t* out;              // [tokens][hidden] bf16
  MoeWeights w1, w2;
  int32_t fp8;
  int32_t tokens;            // of all ranks, 1..kMoeTokens
  int32_t top_k;             // tokens*top_k <= kMoePicks
  int32_t expert_lo;
  int32_t n_experts;         // E_l
  int32_t hidden;            // multiple of 128
  int32_t inter;             // multiple of 128
};
constexpr int kMoeTokens = 64;
constexpr int kMoePicks = 1024;
hipError_t launch_moe(const MoeArgs& a, int num_cus, hipStream_t st);

}  // namespace ep
