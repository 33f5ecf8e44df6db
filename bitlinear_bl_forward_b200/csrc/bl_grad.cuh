// Gradients through the ternary matmul (straight-through estimator).
//
// With the forward Y = (q / s) (gamma C)^T ("BitNet b1.58: The 1-Bit Ternary
// LLM Architecture Guide", section "The Mathematical Formulation of BitLinear",
// eq. (3)), round and clamp passed straight through, scales constant:
//   dX[m, k] = gamma sum_n dY[m, n] C[n, k]
//   dW[n, k] = sum_m dY[m, n] q[m, k] / s[m]
// Both are out[r, k] = sum_c B(r, c) A(c, k): A the stored low-bit matrix
// (rows c, k contiguous), B a view of dY.
#pragma once

#include <cuda_bf16.h>

#include "bl_common.cuh"

namespace bl {

enum GradKind : int { kGradInput = 0, kGradWeight = 1 };

struct GradArgs {
  const uint16_t* dY;    // bf16 [M, N]
  const uint8_t* A;      // packed ternary [N, K/4] (input) or int8 codes [M, K] (weight)
  const float* scale;    // [M] (weight)
  const float* gamma;    // device scalar (input)
  void* out;             // bf16 [M, K] (input); fp32 or bf16 [N, K] (weight)
  int M, K, N;
  int out_bf16, accumulate;
};

}  // namespace bl
