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
//
// Bound by the bytes: one read of every input row and one write of every output
// row.  Measured (B200, 4096 x 2560, rows in HBM): forward 7.2 us, 5.8 TB/s (90%
// of a copy's rate); row gradients alone 10.1 us; with the weight's gradient 13
// (RMSNorm) to 16.7 us (LayerNorm) and 4 us for the join, against 9.6 us of bytes;
// from the checkpoint 11.8-12.1 us against 8.0 (one row a CTA: nothing is in flight
// between a row's sums and the next row's loads).
// There a group has seven steps, and what comes on top is the first fetch, the merge
// of the groups and the partial rows: neither fewer instructions a step (rows kept in
// registers between the passes) nor a hidden barrier (a step's dX behind the next
// step's sums) made it faster.
#pragma once

#include "bl_act.cuh"
#include "bl_common.cuh"
#include "bl_tc_common.cuh"

namespace bl {

constexpr unsigned int kSiteNormRows = 8;   // wait-site identifier (see bl_tc_common.cuh)
// CTAs of the weight gradient's partial rows: a multiple of a B200's SMs.  Fixed, so that
// the workspace query needs no device and the order of the sums does not depend on one.
constexpr int kNgSms = 148;
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

// Pairs of fp32 (one instruction for both halves; each half rounds as usual).
typedef uint64_t f2;
__device__ __forceinline__ f2 f2_make(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 f2_both(float v) { return f2_make(v, v); }
__device__ __forceinline__ float2 f2_get(f2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 f2_bf16(uint32_t w) { return f2_make(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ void f2_bf16x8(uint4 v, f2 (&f)[4]) {
  f[0] = f2_bf16(v.x);
  f[1] = f2_bf16(v.y);
  f[2] = f2_bf16(v.z);
  f[3] = f2_bf16(v.w);
}
__device__ __forceinline__ uint32_t f2_pack_bf16(f2 a) {
  uint32_t r;
  asm("{\n\t.reg .f32 x, y;\n\tmov.b64 {x, y}, %1;\n\tcvt.rn.bf16x2.f32 %0, y, x;\n\t}" : "=r"(r) : "l"(a));
  return r;
}

// 1 / sqrt(stat + eps), within two ulp (rsqrtf).  Every thread of a row forms it:
// a correctly rounded root and quotient would be a fifth of the backward's
// instructions.
__device__ __forceinline__ float norm_rstd(float stat, float eps) { return rsqrtf(__fadd_rn(stat, eps)); }

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

// xh of 8 elements: from bf16 X, (x - mu) r, or from the 8-bit checkpoint, q / s.
// (The difference first: folding -mu r into a product would lose what a large
// mean cancels.)
__device__ __forceinline__ void norm_xh_x(uint4 v, f2 neg_mu, f2 r, f2 (&xh)[4]) {
  f2_bf16x8(v, xh);
#pragma unroll
  for (int e = 0; e < 4; ++e) xh[e] = f2_mul(f2_add(xh[e], neg_mu), r);
}
__device__ __forceinline__ void norm_xh_q(uint2 q, f2 inv_s, f2 (&xh)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = e < 2 ? q.x : q.y;
    const int s = 16 * (e & 1);
    const float lo = static_cast<float>(static_cast<int>(w << (24 - s)) >> 24);
    const float hi = static_cast<float>(static_cast<int>(w << (16 - s)) >> 24);
    xh[e] = f2_mul(f2_make(lo, hi), inv_s);
  }
}

// dX of 8 elements from dY, the weight (all ones without one) and the row's
// means c2 = mean(g xh), c1 = mean(g): (dY w - c1 - xh c2) r.
__device__ __forceinline__ uint4 norm_dx8(const f2 (&dy)[4], const f2 (&w)[4], const f2 (&xh)[4], f2 neg_c1, f2 neg_c2,
                                          f2 r) {
  f2 d[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = f2_mul(f2_fma(xh[e], neg_c2, f2_fma(dy[e], w[e], neg_c1)), r);
  return make_uint4(f2_pack_bf16(d[0]), f2_pack_bf16(d[1]), f2_pack_bf16(d[2]), f2_pack_bf16(d[3]));
}

__device__ __forceinline__ void norm_weight8(const uint16_t* weight, int i, f2 (&w)[4]) {
  if (weight) {
    f2_bf16x8(__ldg(reinterpret_cast<const uint4*>(weight) + i), w);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = f2_both(1.f);
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
  float* part;             // [parts][part_cols]: partial dw (if wanted), then db (if wanted)
  float eps;
  int M, K;
  int want_w, want_b, part_cols;
};

// Sums of N values (a power of two, at most 32) over a group of nw warps,
// returned to every thread.  Within a warp each halving step adds one half of
// the values and hands the other half to the partner lane: N - 1 + 5 - log2 N
// shuffles instead of 5 N.  One barrier (id `bar`, 32 nw threads); `slot`
// ([32][N] floats) alternates between two buffers.  The barrier also takes a
// decision for the group: whether `ok` holds for all its threads.
template <int N>
__device__ __forceinline__ bool group_sum(float (&v)[N], float* slot, int w, int nw, int bar, bool ok) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int m = N / 2; m >= 1; m >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float keep = up ? v[i + m] : v[i], send = up ? v[i] : v[i + m];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  float t = v[0];
#pragma unroll
  for (int p = 16 / N; p >= 1; p >>= 1) t += __shfl_xor_sync(0xffffffffu, t, p);
  // lane l holds value l / (32 / N)
  if ((lane & (32 / N - 1)) == 0) slot[w * N + lane / (32 / N)] = t;
  ok = named_bar_and(bar, 32 * nw, ok);
  t = 0.f;
  for (int i = lane / N; i < nw; i += 32 / N) t += slot[i * N + (lane & (N - 1))];
#pragma unroll
  for (int p = N; p < 32; p <<= 1) t += __shfl_xor_sync(0xffffffffu, t, p);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, t, i);
  return ok;
}

// Row gradients, one row a CTA.
template <int C, bool LAYER, bool CKPT>
__global__ void __launch_bounds__(512) bl_norm_dx_kernel(const NormGradArgs a) {
  __shared__ float2 slot[32];
  const int nch = a.K >> 3;
  const float inv_k = 1.f / static_cast<float>(a.K);
  const int m = blockIdx.x;
  const size_t base = static_cast<size_t>(m) * a.K;
  uint4 vy[C], vx[CKPT ? 1 : C];
  uint2 vq[CKPT ? C : 1];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    const bool in = i < nch;
    vy[j] = in ? reinterpret_cast<const uint4*>(a.dY + base)[i] : make_uint4(0, 0, 0, 0);
    if (CKPT)
      vq[j] = in ? reinterpret_cast<const uint2*>(a.Xq + base)[i] : make_uint2(0, 0);
    else
      vx[j] = in ? reinterpret_cast<const uint4*>(a.X + base)[i] : make_uint4(0, 0, 0, 0);
  }
  const float r = norm_rstd(a.stat[m], a.eps);
  const float mu = CKPT ? __fdiv_rn(1.f, a.scale[m]) : LAYER ? a.mean[m] : 0.f;   // CKPT: 1 / scale
  const f2 f = f2_both(CKPT ? mu : r), nm = f2_both(-mu);
  f2 sx = 0, sy = 0;   // bit pattern of (0, 0)
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i < nch) {
      f2 dy[4], xh[4], w[4];
      f2_bf16x8(vy[j], dy);
      if (CKPT)
        norm_xh_q(vq[CKPT ? j : 0], f, xh);
      else
        norm_xh_x(vx[CKPT ? 0 : j], nm, f, xh);
      norm_weight8(a.weight, i, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 g = f2_mul(dy[e], w[e]);
        sx = f2_fma(g, xh[e], sx);
        if (LAYER) sy = f2_add(g, sy);
      }
    }
  }
  const float2 px = f2_get(sx), py = f2_get(sy);
  const float2 s = block_sum2(make_float2(px.x + px.y, py.x + py.y), slot);
  const f2 n2 = f2_both(-s.x * inv_k), n1 = f2_both(-s.y * inv_k), rr = f2_both(r);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i < nch) {
      f2 dy[4], xh[4], w[4];
      f2_bf16x8(vy[j], dy);
      if (CKPT)
        norm_xh_q(vq[CKPT ? j : 0], f, xh);
      else
        norm_xh_x(vx[CKPT ? 0 : j], nm, f, xh);
      norm_weight8(a.weight, i, w);
      reinterpret_cast<uint4*>(a.dX + base)[i] = norm_dx8(dy, w, xh, n1, n2, rr);
    }
  }
}

// Row gradients and this CTA's part of dw and db, rows of up to 8192.
//
// Bound by reading dY and X and writing dX once.  A group of threads takes R
// rows at a time; thread t owns the same columns of all of them, so that dw and
// db stay in its registers.  Bulk copies keep the group's ring of ST stages in
// shared memory filled, and both passes over a row (sums, then dX) read it there,
// which leaves the registers to the column sums.  A CTA has G groups, whose dw
// and db meet in shared memory: one partial row a CTA.
template <int C, int R, int G, int ST, bool LAYER>
__global__ void __launch_bounds__(G == 2 ? 640 : 512) bl_norm_bwd_kernel(const NormGradArgs a,
                                                                          unsigned long long limit_ns) {
  extern __shared__ __align__(128) uint8_t ring[];
  constexpr int NS = LAYER ? 2 * R : R;
  __shared__ float slots[G][2][32 * NS];
  __shared__ __align__(8) uint64_t full[G][ST];
  const int T = blockDim.x / G, grp = G == 2 && threadIdx.x >= T ? 1 : 0, tid = threadIdx.x - grp * T;
  const int nch = a.K >> 3, nw = T >> 5, w = tid >> 5;
  const int step = gridDim.x * G * R;
  const uint32_t row_bytes = 2 * a.K;
  const float inv_k = 1.f / static_cast<float>(a.K);
  uint8_t* my = ring + static_cast<size_t>(grp) * ST * R * 2 * row_bytes;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&full[grp][i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  auto fetch = [&](int m0, int st) {   // one thread: rows m0.. of dY, then of X
    const int n = min(R, a.M - m0);
    if (n <= 0) return;
    const uint32_t bytes = n * row_bytes;
    uint8_t* d = my + static_cast<size_t>(st) * R * 2 * row_bytes;
    mbar_arrive_expect_tx(&full[grp][st], 2 * bytes);
    bulk_load(d, a.dY + static_cast<size_t>(m0) * a.K, bytes, &full[grp][st]);
    bulk_load(d + R * row_bytes, a.X + static_cast<size_t>(m0) * a.K, bytes, &full[grp][st]);
  };
  f2 dw[4 * C], db[4 * C], wt[C][4];
#pragma unroll
  for (int e = 0; e < 4 * C; ++e) dw[e] = db[e] = 0;   // bit pattern of (0, 0)
#pragma unroll
  for (int j = 0; j < C; ++j) norm_weight8(a.weight, min(tid + j * T, nch - 1), wt[j]);
  int m0 = (blockIdx.x * G + grp) * R;
  if (tid == 0)
    for (int i = 0; i < ST && m0 + i * step < a.M; ++i) fetch(m0 + i * step, i);
  // the rows' statistics, one step ahead
  float stat[R], mean[R];
  auto stats = [&](int m) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const bool row = m + q < a.M;
      stat[q] = row ? a.stat[m + q] : 1.f;
      mean[q] = LAYER && row ? a.mean[m + q] : 0.f;
    }
  };
  stats(m0);
  bool ok = true;
  int it = 0;
  for (int st = 0, ph = 0; m0 < a.M; m0 += step, ++it) {
    f2 r[R], nm[R];
    float s[NS];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      r[q] = f2_both(norm_rstd(stat[q], a.eps));
      nm[q] = f2_both(-mean[q]);
    }
    if (m0 < a.M - step) stats(m0 + step);
    // a wait that gives up is recorded in the status word, and ends the group's
    // loop at the barrier below
    ok = mbar_wait(&full[grp][st], ph, nullptr, limit_ns, kSiteNormRows);
    const uint8_t* rows = my + static_cast<size_t>(st) * R * 2 * row_bytes;
    auto load = [&](int q, int i, f2 (&dy)[4], f2 (&xh)[4]) {
      f2_bf16x8(*reinterpret_cast<const uint4*>(rows + q * row_bytes + 16 * i), dy);
      norm_xh_x(*reinterpret_cast<const uint4*>(rows + (R + q) * row_bytes + 16 * i), nm[q], r[q], xh);
    };
#pragma unroll
    for (int q = 0; q < R; ++q) {
      f2 sx = 0, sy = 0;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int i = tid + j * T;
        if (i < nch && m0 + q < a.M) {
          f2 dy[4], xh[4];
          load(q, i, dy, xh);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f2 p = f2_mul(dy[e], xh[e]);
            dw[4 * j + e] = f2_add(dw[4 * j + e], p);
            db[4 * j + e] = f2_add(db[4 * j + e], dy[e]);
            sx = f2_fma(p, wt[j][e], sx);
            if (LAYER) sy = f2_fma(dy[e], wt[j][e], sy);
          }
        }
      }
      const float2 x = f2_get(sx), y = f2_get(sy);
      s[q] = x.x + x.y;
      if (LAYER) s[(LAYER ? R : 0) + q] = y.x + y.y;
    }
    // the barrier inside also says that the group has left the stage before
    if (a.dX)
      ok = group_sum<NS>(s, slots[grp][it & 1], w, nw, 1 + grp, ok);
    else
      ok = named_bar_and(1 + grp, T, ok);
    if (!ok) break;
    if (it > 0 && tid == 0 && m0 < a.M - (ST - 1) * step) fetch(m0 + (ST - 1) * step, st == 0 ? ST - 1 : st - 1);
    if (++st == ST) {
      st = 0;
      ph ^= 1;
    }
    if (!a.dX) continue;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (m0 + q >= a.M) continue;
      const f2 n2 = f2_both(-s[q] * inv_k), n1 = f2_both(LAYER ? -s[(LAYER ? R : 0) + q] * inv_k : 0.f);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int i = tid + j * T;
        if (i < nch) {
          f2 dy[4], xh[4];
          load(q, i, dy, xh);
          reinterpret_cast<uint4*>(a.dX + static_cast<size_t>(m0 + q) * a.K)[i] =
              norm_dx8(dy, wt[j], xh, n1, n2, r[q]);
        }
      }
    }
  }
  if (!ok) {
    // the column sums are not numbers then, and no copy of this group is in flight
    // when the CTA ends: rows were fetched for the steps up to it + ST - 2 (the first
    // ST before any step)
#pragma unroll
    for (int e = 0; e < 4 * C; ++e) dw[e] = db[e] = f2_both(__int_as_float(0x7FFFFFFF));
    if (tid == 0)
      for (int i = it, m = m0; i < (it ? it + ST - 1 : ST) && m < a.M; ++i, m += step)
        mbar_wait(&full[grp][i % ST], (i / ST) & 1, nullptr, limit_ns, kSiteDrain);
  }
  pdl_launch_dependents();
  if (G == 2) {
    ulonglong2* merge = reinterpret_cast<ulonglong2*>(ring);   // [2][K] floats
    __syncthreads();                                   // both groups have left the ring
    if (grp == 1) {
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = tid + j * T, e = 4 * j + 2 * h;
          if (i < nch) {
            merge[2 * i + h] = make_ulonglong2(dw[e], dw[e + 1]);
            merge[2 * (nch + i) + h] = make_ulonglong2(db[e], db[e + 1]);
          }
        }
    }
    __syncthreads();
    if (grp == 1) return;
  }
  const ulonglong2* merge = reinterpret_cast<const ulonglong2*>(ring);
  ulonglong2* pw = reinterpret_cast<ulonglong2*>(a.part + static_cast<size_t>(blockIdx.x) * a.part_cols);
  ulonglong2* pb = pw + (a.want_w ? a.K / 4 : 0);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int i = tid + j * T;
    if (i >= nch) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = 4 * j + 2 * h;
      ulonglong2 u = make_ulonglong2(dw[e], dw[e + 1]), v = make_ulonglong2(db[e], db[e + 1]);
      if (G == 2) {
        const ulonglong2 u2 = merge[2 * i + h], v2 = merge[2 * (nch + i) + h];
        u = make_ulonglong2(f2_add(u.x, u2.x), f2_add(u.y, u2.y));
        v = make_ulonglong2(f2_add(v.x, v2.x), f2_add(v.y, v2.y));
      }
      if (a.want_w) pw[2 * i + h] = u;
      if (a.want_b) pb[2 * i + h] = v;
    }
  }
}

// Row gradients of wide rows, which do not fit the registers: the sums in one
// pass over the row, dX in a second one (the row is in L2 by then).  A thread
// reads again only what it will overwrite itself, so dX may be dY or X.
// With weight gradients, bl_norm_wgrad_cols_kernel reads dY and X once more before.
// Measured (B200, LayerNorm): 2048 x 28672 73 us for dX, 47 for the columns, 15 for the
// join (135; 54 of bytes), 4096 x 16384 92 + 52 + 12 (156; 61), 257 x 28672 11 + 9 + 10
// (30; 6.8).
template <bool LAYER, bool CKPT>
__global__ void __launch_bounds__(1024) bl_norm_dx_wide_kernel(const NormGradArgs a) {
  __shared__ float2 slot[32];
  const int nch = a.K >> 3;
  const int m = blockIdx.x;
  const size_t base = static_cast<size_t>(m) * a.K;
  const float r = norm_rstd(a.stat[m], a.eps);
  const float mu = CKPT ? __fdiv_rn(1.f, a.scale[m]) : LAYER ? a.mean[m] : 0.f;
  const f2 f = f2_both(CKPT ? mu : r), nm = f2_both(-mu);
  auto load = [&](int i, f2 (&dy)[4], f2 (&xh)[4], f2 (&w)[4]) {
    f2_bf16x8(reinterpret_cast<const uint4*>(a.dY + base)[i], dy);
    if (CKPT)
      norm_xh_q(reinterpret_cast<const uint2*>(a.Xq + base)[i], f, xh);
    else
      norm_xh_x(reinterpret_cast<const uint4*>(a.X + base)[i], nm, f, xh);
    norm_weight8(a.weight, i, w);
  };
  f2 sx = 0, sy = 0;
#pragma unroll 2
  for (int i = threadIdx.x; i < nch; i += blockDim.x) {
    f2 dy[4], xh[4], w[4];
    load(i, dy, xh, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f2 g = f2_mul(dy[e], w[e]);
      sx = f2_fma(g, xh[e], sx);
      if (LAYER) sy = f2_add(g, sy);
    }
  }
  const float2 px = f2_get(sx), py = f2_get(sy);
  const float2 s = block_sum2(make_float2(px.x + px.y, py.x + py.y), slot);
  const float inv_k = 1.f / static_cast<float>(a.K);
  const f2 n2 = f2_both(-s.x * inv_k), n1 = f2_both(-s.y * inv_k), rr = f2_both(r);
#pragma unroll 2
  for (int i = threadIdx.x; i < nch; i += blockDim.x) {
    f2 dy[4], xh[4], w[4];
    load(i, dy, xh, w);
    reinterpret_cast<uint4*>(a.dX + base)[i] = norm_dx8(dy, w, xh, n1, n2, rr);
  }
}

// dw and db of wide rows: thread = 8 columns, blockIdx.y = part of the rows.
template <bool LAYER>
__global__ void __launch_bounds__(128) bl_norm_wgrad_cols_kernel(const NormGradArgs a, int rows_per_part) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (a.K >> 3)) return;
  f2 dw[4], db[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[e] = db[e] = 0;
  const int m0 = blockIdx.y * rows_per_part, m1 = min(a.M, m0 + rows_per_part);
#pragma unroll 4
  for (int m = m0; m < m1; ++m) {
    const size_t base = static_cast<size_t>(m) * a.K;
    const f2 r = f2_both(norm_rstd(a.stat[m], a.eps)), nm = f2_both(LAYER ? -a.mean[m] : 0.f);
    f2 dy[4], xh[4];
    f2_bf16x8(reinterpret_cast<const uint4*>(a.dY + base)[i], dy);
    norm_xh_x(reinterpret_cast<const uint4*>(a.X + base)[i], nm, r, xh);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dw[e] = f2_fma(dy[e], xh[e], dw[e]);
      db[e] = f2_add(dy[e], db[e]);
    }
  }
  ulonglong2* pw = reinterpret_cast<ulonglong2*>(a.part + static_cast<size_t>(blockIdx.y) * a.part_cols);
  ulonglong2* pb = pw + (a.want_w ? a.K / 4 : 0);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (a.want_w) pw[2 * i + h] = make_ulonglong2(dw[2 * h], dw[2 * h + 1]);
    if (a.want_b) pb[2 * i + h] = make_ulonglong2(db[2 * h], db[2 * h + 1]);
  }
}

// Sums the parts in a fixed order: 32 columns a CTA, 32 threads a column.
// Launched to start while the kernel before it still runs: it waits for that
// kernel's memory before it reads.
__global__ void __launch_bounds__(1024)
    bl_norm_wgrad_join_kernel(const float* __restrict__ part, int parts, int cols, int K, float* __restrict__ dweight,
                              float* __restrict__ dbias, int accumulate) {
  __shared__ float t[32][33];
  const int cx = threadIdx.x & 31, py = threadIdx.x >> 5;
  const float* p = part + blockIdx.x * 32 + cx;   // cols is a multiple of 32
  pdl_wait();
  float s = 0.f;
#pragma unroll 8
  for (int i = py; i < parts; i += 32) s += p[static_cast<size_t>(i) * cols];
  t[py][cx] = s;
  __syncthreads();
  s = t[cx][py];   // column py of the block, part group cx
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (cx == 0) {
    const int col = blockIdx.x * 32 + py;
    const bool w = dweight && col < K;
    float* out = w ? dweight + col : dbias + (dweight ? col - K : col);
    *out = accumulate ? *out + s : s;
  }
}

}  // namespace bl
