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

// 64 x 64 outputs a CTA, 4 x 4 a thread, fp32.
template <int KIND>
__global__ void __launch_bounds__(256) bl_grad_kernel(const GradArgs a) {
  __shared__ float sA[16][64], sB[16][65];
  const int R = KIND == kGradInput ? a.M : a.N, L = KIND == kGradInput ? a.N : a.M;
  const int k0 = blockIdx.x * 64, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int r0 = blockIdx.y * 64; r0 < R; r0 += gridDim.y * 64) {
    float acc[4][4] = {};
    for (int c0 = 0; c0 < L; c0 += 16) {
      for (int i = threadIdx.x; i < 16 * 64; i += 256) {
        const int c = c0 + (i >> 6), k = k0 + (i & 63);
        float v = 0.f;
        if (c < L) {
          if (KIND == kGradInput) {
            const uint8_t b = a.A[static_cast<size_t>(c) * (a.K / 4) + (k >> 4) * 4 + (k & 3)];
            v = static_cast<float>(static_cast<int>((b >> (2 * ((k >> 2) & 3))) & 3) - 1);
          } else {
            v = static_cast<float>(static_cast<int8_t>(a.A[static_cast<size_t>(c) * a.K + k])) / a.scale[c];
          }
        }
        sA[i >> 6][i & 63] = v;
      }
      for (int i = threadIdx.x; i < 16 * 64; i += 256) {
        int c, r;
        if (KIND == kGradInput) {
          c = i & 15;
          r = i >> 4;
        } else {
          r = i & 63;
          c = i >> 6;
        }
        float v = 0.f;
        if (c0 + c < L && r0 + r < R) {
          const size_t o = KIND == kGradInput ? static_cast<size_t>(r0 + r) * a.N + c0 + c
                                              : static_cast<size_t>(c0 + c) * a.N + r0 + r;
          v = __uint_as_float(static_cast<uint32_t>(a.dY[o]) << 16);
        }
        sB[c][r] = v;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 16; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] += sB[c][ty + 16 * i] * sA[c][tx + 16 * j];
      __syncthreads();
    }
    const float f = KIND == kGradInput ? *a.gamma : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + ty + 16 * i;
      if (r >= R) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const size_t o = static_cast<size_t>(r) * a.K + k0 + tx + 16 * j;
        float v = acc[i][j] * f;
        if (a.out_bf16) {
          __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.out);
          if (a.accumulate) v += __bfloat162float(y[o]);
          y[o] = __float2bfloat16_rn(v);
        } else {
          float* y = static_cast<float*>(a.out);
          y[o] = a.accumulate ? y[o] + v : v;
        }
      }
    }
  }
}

}  // namespace bl
