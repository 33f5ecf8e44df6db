// RMSNorm / LayerNorm of bf16 rows as an operator of its own, and its
// gradients (fp32 arithmetic, bf16 in and out).
//
// With K features, r = 1 / sqrt(stat + eps), xh = (x - mean) r, g = dY w:
//   forward   y  = xh w + b
//   backward  dx = r (g - xh mean_k(g xh) - mean_k(g))     (RMSNorm: no mean_k(g))
//             dw = sum_m dY xh,  db = sum_m dY
// "BitNet 2B4T Guide: Scaling Native 1.58-Bit LLMs", section "3. Sub-Layer
// Normalization (SubLN)" names the norm; the backward is its derivative.
//
// A CTA holds whole rows in registers (thread t owns the 16-byte chunks
// t, t + T, ...), so every row is read once and the sums over k are block
// reductions with one barrier each.  The backward's sums over m stay in the
// owning thread's registers over all rows of a CTA; the CTAs' partial sums
// meet in a second kernel that adds them in a fixed order (no atomics: the
// result does not depend on the run).
#pragma once

#include "bl_act.cuh"
#include "bl_common.cuh"

namespace bl {

constexpr int kNgMaxParts = 296;      // partial rows of the weight gradient (two CTAs an SM)
constexpr int kNgRowMaxK = 8192;      // widest row whose weight gradient stays in registers

__device__ __forceinline__ float2 warp_sum2(float2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

// Sum over the CTA, returned to every thread; one barrier.  `slot` alternates
// between two buffers: a buffer is written again only after the next
// reduction's barrier, which every reader of it has passed.
__device__ __forceinline__ float2 block_sum2(float2 v, float2* slot) {
  v = warp_sum2(v);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < nw ? slot[lane] : make_float2(0.f, 0.f);
  return warp_sum2(v);
}

__device__ __forceinline__ void unpack8_bf16(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 pack8_bf16(const float (&f)[8]) {
  return make_uint4(pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7]));
}

// 1 / sqrt(stat + eps): one rounding each.
__device__ __forceinline__ float norm_rstd(float stat, float eps) {
  return __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(stat, eps)));
}

// One row per CTA.  X and Y may be the same buffer (a thread writes only the
// chunks it has read), so neither is __restrict__.
template <int C, bool LAYER>
__global__ void __launch_bounds__(1024)
    bl_norm_fwd_kernel(const uint16_t* X, const uint16_t* __restrict__ weight, const uint16_t* __restrict__ bias,
                       float eps, int K, uint16_t* Y, float* __restrict__ mean, float* __restrict__ stat) {
  __shared__ float2 slots[2][32];
  const int nch = K >> 3;
  const size_t row = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(X + row * K);
  uint4* yr = reinterpret_cast<uint4*>(Y + row * K);
  uint4 v[C];
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    v[j] = i < nch ? xr[i] : make_uint4(0, 0, 0, 0);
    float f[8];
    unpack8_bf16(v[j], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s.x += LAYER ? f[e] : f[e] * f[e];
  }
  const float inv_k = 1.f / static_cast<float>(K);
  s = block_sum2(s, slots[0]);
  float mu = 0.f, st = s.x * inv_k;
  if (LAYER) {
    mu = st;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (threadIdx.x + j * blockDim.x < nch) {
        float f[8];
        unpack8_bf16(v[j], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s.x += (f[e] - mu) * (f[e] - mu);
      }
    }
    st = block_sum2(s, slots[1]).x * inv_k;
  }
  if (threadIdx.x == 0) {
    if (LAYER && mean) mean[row] = mu;
    if (stat) stat[row] = st;
  }
  const float r = norm_rstd(st, eps);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i < nch) {
      float f[8], w[8];
      unpack8_bf16(v[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (f[e] - mu) * r;
      if (weight) {
        unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(weight) + i), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= w[e];
      }
      if (bias) {
        unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(bias) + i), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += w[e];
      }
      yr[i] = pack8_bf16(f);
    }
  }
}

// xh of 8 elements: from bf16 X, or from the 8-bit checkpoint (q / s).
__device__ __forceinline__ void norm_xh_x(uint4 v, float mu, float r, float (&xh)[8]) {
  unpack8_bf16(v, xh);
#pragma unroll
  for (int e = 0; e < 8; ++e) xh[e] = (xh[e] - mu) * r;
}
__device__ __forceinline__ void norm_xh_q(uint2 q, float inv_s, float (&xh)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t w = e < 4 ? q.x : q.y;
    xh[e] = static_cast<float>(static_cast<int>(w << (24 - 8 * (e & 3))) >> 24) * inv_s;
  }
}

struct NormGradArgs {
  const uint16_t* dY;      // [M, K]
  const uint16_t* X;       // [M, K], or null: Xq and scale
  const int8_t* Xq;
  const float* scale;
  const uint16_t* weight;  // [K] or null
  const float* mean;       // [M] (LayerNorm on X)
  const float* stat;       // [M]
  uint16_t* dX;            // [M, K] or null; may be dY or X
  float* part;             // [gridDim.x][2][K] partial dw and db, when GRADS
  float eps;
  int M, K;
};

// Row gradients; with GRADS also this CTA's part of dw and db.
template <int C, bool LAYER, bool CKPT, bool GRADS>
__global__ void __launch_bounds__(C >= 8 ? 1024 : 512) bl_norm_bwd_kernel(const NormGradArgs a) {
  __shared__ float2 slots[2][32];
  const int nch = a.K >> 3;
  const float inv_k = 1.f / static_cast<float>(a.K);
  float dw[GRADS ? 8 * C : 1], db[GRADS ? 8 * C : 1];
#pragma unroll
  for (int e = 0; e < (GRADS ? 8 * C : 1); ++e) dw[e] = db[e] = 0.f;
  int buf = 0;
  for (int m = blockIdx.x; m < a.M; m += gridDim.x, buf ^= 1) {
    const size_t base = static_cast<size_t>(m) * a.K;
    const uint4* dyr = reinterpret_cast<const uint4*>(a.dY + base);
    const uint4* xr = reinterpret_cast<const uint4*>(a.X + base);
    const uint2* qr = reinterpret_cast<const uint2*>(a.Xq + base);
    const float r = norm_rstd(a.stat[m], a.eps);
    const float mu = (LAYER && !CKPT) ? a.mean[m] : 0.f;
    const float inv_s = CKPT ? __fdiv_rn(1.f, a.scale[m]) : 0.f;
    uint4 vy[C], vx[CKPT ? 1 : C];
    uint2 vq[CKPT ? C : 1];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      const bool in = i < nch;
      vy[j] = in ? dyr[i] : make_uint4(0, 0, 0, 0);
      if (CKPT)
        vq[j] = in ? qr[i] : make_uint2(0, 0);
      else
        vx[j] = in ? xr[i] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (i < nch) {
        float g[8], xh[8];
        unpack8_bf16(vy[j], g);
        if (CKPT)
          norm_xh_q(vq[j], inv_s, xh);
        else
          norm_xh_x(vx[j], mu, r, xh);
        if (GRADS) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dw[8 * j + e] += g[e] * xh[e];
            db[8 * j + e] += g[e];
          }
        }
        if (a.weight) {
          float w[8];
          unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(a.weight) + i), w);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s.x += g[e] * xh[e];
          if (LAYER) s.y += g[e];
        }
      }
    }
    if (a.dX == nullptr) continue;   // the same for every thread
    s = block_sum2(s, slots[buf]);
    const float c2 = s.x * inv_k, c1 = LAYER ? s.y * inv_k : 0.f;
    uint4* dxr = reinterpret_cast<uint4*>(a.dX + base);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (i < nch) {
        float g[8], xh[8];
        unpack8_bf16(vy[j], g);
        if (CKPT)
          norm_xh_q(vq[j], inv_s, xh);
        else
          norm_xh_x(vx[j], mu, r, xh);
        if (a.weight) {
          float w[8];
          unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(a.weight) + i), w);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = (g[e] - xh[e] * c2 - c1) * r;
        dxr[i] = pack8_bf16(g);
      }
    }
  }
  if (GRADS) {
    float4* pw = reinterpret_cast<float4*>(a.part + static_cast<size_t>(blockIdx.x) * 2 * a.K);
    float4* pb = pw + a.K / 4;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (i < nch) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = 8 * j + 4 * h;
          pw[2 * i + h] = make_float4(dw[e], dw[e + 1], dw[e + 2], dw[e + 3]);
          pb[2 * i + h] = make_float4(db[e], db[e + 1], db[e + 2], db[e + 3]);
        }
      }
    }
  }
}

// dw and db of wide rows: thread = 8 columns, blockIdx.y = part of the rows.
template <bool LAYER>
__global__ void __launch_bounds__(128) bl_norm_wgrad_cols_kernel(const NormGradArgs a, int rows_per_part) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (a.K >> 3)) return;
  float dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.f;
  const int m0 = blockIdx.y * rows_per_part, m1 = min(a.M, m0 + rows_per_part);
#pragma unroll 4
  for (int m = m0; m < m1; ++m) {
    const size_t base = static_cast<size_t>(m) * a.K;
    const float r = norm_rstd(a.stat[m], a.eps);
    const float mu = LAYER ? a.mean[m] : 0.f;
    float g[8], xh[8];
    unpack8_bf16(reinterpret_cast<const uint4*>(a.dY + base)[i], g);
    norm_xh_x(reinterpret_cast<const uint4*>(a.X + base)[i], mu, r, xh);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[e] += g[e] * xh[e];
      db[e] += g[e];
    }
  }
  float4* pw = reinterpret_cast<float4*>(a.part + static_cast<size_t>(blockIdx.y) * 2 * a.K);
  float4* pb = pw + a.K / 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    pw[2 * i + h] = make_float4(dw[4 * h], dw[4 * h + 1], dw[4 * h + 2], dw[4 * h + 3]);
    pb[2 * i + h] = make_float4(db[4 * h], db[4 * h + 1], db[4 * h + 2], db[4 * h + 3]);
  }
}

// Sums the parts in a fixed order: 32 columns a CTA, 32 threads a column.
// Columns 0..K-1 are dw, K..2K-1 db.
__global__ void __launch_bounds__(1024)
    bl_norm_wgrad_join_kernel(const float* __restrict__ part, int parts, int K, float* __restrict__ dweight,
                              float* __restrict__ dbias, int accumulate) {
  __shared__ float t[32][33];
  const int cx = threadIdx.x & 31, py = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;   // 2K is a multiple of 32
  float s = 0.f;
#pragma unroll 4
  for (int p = py; p < parts; p += 32) s += part[static_cast<size_t>(p) * 2 * K + c];
  t[py][cx] = s;
  __syncthreads();
  s = t[cx][py];   // column py of the block, part group cx
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (cx == 0) {
    const int col = blockIdx.x * 32 + py;
    float* out = col < K ? dweight : dbias;
    const int k = col < K ? col : col - K;
    if (out) out[k] = accumulate ? out[k] + s : s;
  }
}

}  // namespace bl
