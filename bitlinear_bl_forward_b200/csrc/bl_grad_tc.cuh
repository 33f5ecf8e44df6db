// Gradients through the ternary matmul on the tensor cores (tcgen05 kind::f16,
// CTA pairs, bf16 operands, fp32 accumulators in tensor memory).
//
// Straight-through gradients of Y = (q / s) (gamma C)^T ("BitNet b1.58: The
// 1-Bit Ternary LLM Architecture Guide", section "The Mathematical Formulation
// of BitLinear", eq. (3)):
//   input   dX[m, k] = gamma sum_n dY[m, n] C[n, k]
//   weight  dW[n, k] = sum_m dY[m, n] q[m, k] / s[m]
// Both are D[k, r] = sum_c A[c, k] B[r, c]: A the stored low-bit matrix with
// k contiguous (packed ternary rows c = n, or int8 codes with rows c = m and a
// scale a row), B a view of dY (r = m, c contiguous; or r = n, r contiguous).
//
// A pair of CTAs computes 256 (k) x BN (r) per tile:
//   * every CTA brings its 128 k of the raw low-bit rows and half of the tile
//     of dY into shared memory with TMA, 64 or 128 rows of the sum a stage;
//   * converter warps expand the raw rows to bf16 into the swizzled operand
//     tile next to them (k contiguous: an MN-major operand, so nothing is
//     transposed).  C is exact in bf16.  q / s is not: an fp32 result takes it
//     as hi + lo, two bf16 with 2^-16 relative error together, and twice the
//     MMAs; a bf16 result takes hi alone, off by half a step of its own type;
//   * the leader issues tcgen05.mma.cta_group::2 (M = 256, N = BN, K = 16),
//     each tensor core reading only its half of dY from its own SM;
//   * eight epilogue warps drain one accumulator while the next one fills.
//     Lanes are k, so a warp's store of one r is 32 neighbouring k.
// The low-bit matrix is expanded once per tile and never exists in memory as
// bf16; A's conversion runs beside the MMAs.
// Tiles behind the last whole wave are cut along their sums (GtCut); the parts
// (fp32) meet in bl_grad_join_kernel in a fixed order.
// The tensor core truncates when it adds to an fp32 accumulator, so the error
// of a long sum grows with its length instead of its root: 1.0e-5 of the norm
// over 4096 tokens, hi + lo included (measured).  An fp32 result is therefore
// summed in segments of 2048 tokens, which the epilogue adds up with rounding
// (5.3e-6; a plain fp32 product: 1.1e-6): the pair that owns the tile stores the
// first segment and adds the others to its own output, which is still in L2.
// Segments of 1024 tokens cost 3% more.  bf16 results take their whole sum in one
// accumulator: short by up to 6.3e-9 of itself a term (8.2e-4 over 131072 terms of one
// sign, 1.4e-4 of mixed signs, where the output's rounding is 1.7e-3 of the norm).
//
// Order between the two CTAs.  Waits on barriers that the other CTA's threads or
// the leader's commits arrive on (ready, done, accfull, accempty) acquire at
// cluster scope; full is a CTA's own.  Arrivals on the leader's ready and accempty
// are relaxed at cluster scope, which is enough because no data crosses:
//   ready     an expanded tile is written, fenced and read in one SM's shared
//             memory: every writing lane passes fence.proxy.async, its warp meets,
//             and only then does one lane arrive, so the tile is visible to that
//             SM's tensor core before the leader can learn of it;
//   accempty  an accumulator is read (wait::ld) and handed back in one SM's tensor
//             memory; tcgen05.fence::before_thread_sync orders it before the arrival.
// A release at cluster scope on ready waits about 1300 clocks a stage for nothing:
// 2B down projection's dX 92 -> 134 us, 70B-class layer with 128 tokens 52 -> 75, 2B
// up projection's fp32 dW 182 -> 216, 4-bit-activation layer's bf16 dW 133 -> 178.
//
// What bounds it.  Per 64 rows of the sum and CTA, at BN = 256: 512 clocks of
// tensor work a term, against what passes through 128 bytes a clock of shared
// memory: A written and read (32 KB a term), dY in and read (32 KB, the read once
// a term), the raw rows in and out (4 or 16 KB).  That is 530 clocks for the
// input gradient, 640 for a bf16 and 1000 (of 1024) for an fp32 weight gradient.
// At BN <= 128 A's way through shared memory alone is 256 of them for 256 clocks of
// tensor work or less.  Measured (B200): 2B down projection, M = 4096, 91 us alone
// (1.59 PFLOP/s, the tensor pipe 84% active), 109 us in a seconds-long run under
// the power cap (1.33); 2B up projection's fp32 gradient 188 and 222 us (twice
// 0.77 PFLOP/s; pipe 92% active while a pair works); 4-bit-activation layer's bf16
// gradient 131 and 155 us (1.41; pipe 75%); 70B-class layer with 128 tokens 52 us and
// 5 for the join (1.06; pipe 58%).
#pragma once

#include <cuda_bf16.h>

#include "bl_common.cuh"
#include "bl_gemm_2sm.cuh"
#include "bl_grad.cuh"
#include "bl_tc_common.cuh"

namespace bl {

constexpr int kGtK = 128;                 // k a CTA (256 a pair)
constexpr int kGtEpiWarps = 8;
constexpr int kGtSegment = 2048;          // terms of the sum an fp32 result takes in one accumulator

// Rows of the sum a stage.  The issuing thread spends about 280 clocks a stage
// on waiting, committing and counting, while few MMAs are queued: at BN = 128 or
// less a stage of 64 rows is 256 clocks of tensor work and took 527, so those
// stages are 128 rows (77 -> 62 us for 128 tokens of a 70B-class layer).  At BN =
// 256 the deeper ring of 64-row stages wins (93 against 99 us for the 2B down
// projection), and the weight gradient's operands leave no room for more.
constexpr int gt_bc(int kind, int bn) { return kind == kGradInput && bn <= 128 ? 128 : 64; }

// TERMS: bf16 terms of A (2: hi + lo).
template <int KIND, int TERMS, int BN>
struct GtCfg {
  static constexpr int kBC = gt_bc(KIND, BN);
  static constexpr int kHalf = BN / 2;                         // r rows staged per CTA
  // K-major: boxes of 64 of the sum; MN-major: of 64 r (whole boxes)
  static constexpr int kBBytes = (KIND == kGradInput ? kHalf : (kHalf + 63) / 64 * 64) * kBC * 2;
  static constexpr int kRawBytes = KIND == kGradInput ? kBC * kGtK / 4 : kBC * kGtK;
  static constexpr int kBlockBytes = kBC * 128;                // 64 k of an expanded tile
  static constexpr int kTileBytes = 2 * kBlockBytes;           // one expanded operand tile
  static constexpr int kInBytes = kBBytes + kRawBytes;         // what TMA brings for a stage
  static constexpr int kASlotBytes = TERMS * kTileBytes;
  // Converter warps work in groups of four, each group on a stage of its own,
  // so that a stage's latency (waits, loads, conversion, proxy fence, arrival:
  // about 1000 clocks) overlaps the others'.  Measured on the 2B layers and the
  // 4-bit-activation layer with 2, 3 and 4 groups: input 97, 91, 91 us; weight
  // fp32 191, 191, 193; weight bf16 162, 150, 143 (half the tensor work beside the
  // same loads); two groups of eight warps are slower (fp32 193, bf16 157).
  static constexpr int kGroupWarps = 4;
  static constexpr int kGroups = KIND == kGradInput || TERMS == 2 ? 3 : 4;
  static constexpr int kFirstEpi = 2 + kGroupWarps * kGroups;
  static constexpr int kThreads = 32 * (kFirstEpi + kGtEpiWarps);
  static constexpr int kChunk = kHalf < 32 ? kHalf : 32;       // r of one epilogue step
  static constexpr int kOutBytes = TERMS == 2 ? 4096 : 2048;   // staging a warp: tiles of [32 r][32 k] bf16 or [16 r][32 k] fp32
  static constexpr int kOutTotal = kGtEpiWarps * kOutBytes;
  static constexpr int kASlots = kBC == 128 || TERMS == 2 ? 3 : 4;   // expanded operand tiles in flight
  static constexpr int kBudget = 227 * 1024 - 1024 - 512 - kOutTotal - kASlots * kASlotBytes;
  static constexpr int kMaxStages = kBudget / kInBytes;
  static constexpr int kStages = kMaxStages > 8 ? 8 : kMaxStages;
  static constexpr int kInOffset = kASlots * kASlotBytes;
  static constexpr int kSegment = TERMS == 2 ? kGtSegment / kBC : 1 << 30;
  static constexpr int kOutOffset = kInOffset + kStages * kInBytes;
  static constexpr int kBarOffset = kOutOffset + kOutTotal;
  static constexpr int kSmemBytes = kBarOffset + 512 + 1024;
  static constexpr int kTmemCols = 2 * BN <= 64 ? 64 : 2 * BN <= 128 ? 128 : 2 * BN <= 256 ? 256 : 512;
  static_assert(kStages >= 2 && kSmemBytes <= 227 * 1024, "shared memory");
  static_assert(kInBytes % 1024 == 0, "operand tiles are 1024-byte aligned");
  static_assert((3 * kStages + 5) * 8 + 8 <= 512, "barriers");
};

// How the tiles' sums are cut into the chunks that pairs take.  The first `whole`
// chunks are a tile each, written directly.  The stages of the other tiles (nkv a
// tile, in a row) are cut into chunks of `per`: a chunk is a part of a tile or runs
// from one tile into the next ones; what it has of a tile goes to an fp32 part of
// the tile's shape, and the tile's parts are added in the order of their chunks.
// nkv may be above the tile's own stages, so that chunks end with the tile.
struct GtCut {
  int whole, nkv, per, chunks;
  int over;   // 1: chunks may run over a tile's end (a tile and the next one have parts of the same chunk)
  // of tile whole + t: its first chunk behind the whole tiles, how many it has, and
  // where chunk c's part lies (every part has a place of its own)
  __host__ __device__ int first(int t) const { return t * nkv / per; }
  __host__ __device__ int parts(int t) const { return ((t + 1) * nkv - 1) / per - first(t) + 1; }
  __host__ __device__ int place(int t, int c) const { return c + over * t; }
};

struct GtArgs {
  const float* scale;   // [M] (weight)
  const float* gamma;   // device scalar (input), else null
  void* out;            // [R][K]
  int R, L, K;          // output rows, length of the sum, columns
  int kt, rt;           // tiles along k and r
  GtCut cut;
  int accumulate;       // out += (weight)
};

// Instruction descriptor: kind::f16, bf16 x bf16 -> f32; A MN-major, B
// MN-major or K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool b_mn) {
  return (1u << 4)                                   // D: f32
         | (1u << 7) | (1u << 10)                    // A, B: bf16
         | (1u << 15)                                // A: MN-major
         | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// High words of the operand descriptors (128-byte swizzle, 8-row atoms 1024
// bytes apart); the low word is the start address and, for MN-major operands,
// the bytes between blocks of 64 elements.
constexpr uint32_t kGtDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t gt_desc_mn_lo(uint32_t addr, uint32_t block_bytes) {
  return ((addr >> 4) & 0x3FFFu) | ((block_bytes >> 4) << 16);
}
__device__ __forceinline__ uint32_t gt_desc_k_lo(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | (1u << 16); }

// The four MMAs (K = 16 each) of one operand tile, A MN-major (2048 bytes a
// step) and B a step of BSTEP 16-byte units: one asm block, so that the issuing
// thread does little else.  The first accumulates when acc0 != 0.
template <int BSTEP>
__device__ __forceinline__ void mma_bf16_tile_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                                   uint32_t acc0) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t.reg .b32 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.eq.b32 q, %5, %5;\n\t"
      "mov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, p;\n\t"
      "add.u32 a, %1, 128;\n\t"
      "add.u32 b, %2, %6;\n\t"
      "mov.b64 da, {a, %3};\n\t"
      "mov.b64 db, {b, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, q;\n\t"
      "add.u32 a, %1, 256;\n\t"
      "add.u32 b, %2, %7;\n\t"
      "mov.b64 da, {a, %3};\n\t"
      "mov.b64 db, {b, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, q;\n\t"
      "add.u32 a, %1, 384;\n\t"
      "add.u32 b, %2, %8;\n\t"
      "mov.b64 da, {a, %3};\n\t"
      "mov.b64 db, {b, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, q;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(kGtDescHi), "r"(idesc), "r"(acc0), "n"(BSTEP), "n"(2 * BSTEP), "n"(3 * BSTEP)
      : "memory");
}

// Whether the phase has completed, without waiting for it.
__device__ __forceinline__ bool mbar_test_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// TMA store of a tile, and the reduction that adds it to fp32 in memory
// (rounding to nearest).  Every output element has one thread that adds to it, in
// order, so the result does not depend on the run.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* tmap, int x, int y, int z, const void* smem_src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(smem_src))
               : "memory");
}
__device__ __forceinline__ void tma_reduce_add_3d(const CUtensorMap* tmap, int x, int y, int z, const void* smem_src) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(smem_src))
               : "memory");
}
__device__ __forceinline__ void bulk_wait_group_read1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// Sixteen packed codes -> sixteen bf16 in {-1, 0, 1}.  Slice j of the word has
// the codes u = c + 1 of k = 4j..4j+3 in its bytes; u * 17 + 0x40 is the byte
// with nibbles (u + 4, u), which pick the high and the low byte of bf16(u - 1)
// from a table of six bytes.
__device__ __forceinline__ void expand16(uint32_t w, uint32_t (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t sel = ((w >> (2 * j)) & 0x03030303u) * 17u + 0x40404040u;
    v[2 * j] = __byte_perm(0x00800080u, 0x003F00BFu, sel);
    v[2 * j + 1] = __byte_perm(0x00800080u, 0x003F00BFu, sel >> 16);
  }
}

// Two codes (bytes B0, B0 + 1 of x, each q + 128) times r: the pair as fp32.
// 0x4B0000xx is 2^23 + xx; the subtraction leaves q exactly.
template <int B0>
__device__ __forceinline__ uint64_t codes2_f32(uint32_t x, uint64_t rr) {
  const uint32_t a = __byte_perm(x, 0x4B000000u, 0x7440 + B0), b = __byte_perm(x, 0x4B000000u, 0x7440 + B0 + 1);
  uint64_t v;
  asm("{\n\t.reg .b64 t, o;\n\t"
      "mov.b64 t, {%1, %2};\n\t"
      "mov.b64 o, {%3, %3};\n\t"
      "add.rn.f32x2 t, t, o;\n\t"
      "mul.rn.f32x2 %0, t, %4;\n\t}"
      : "=l"(v)
      : "r"(a), "r"(b), "r"(0xCB000080u), "l"(rr));   // -(2^23 + 128)
  return v;
}

// hi = bf16x2(v); lo = bf16x2(v - hi).
template <int TERMS>
__device__ __forceinline__ void split2(uint64_t v, uint32_t& hi, uint32_t& lo) {
  asm("{\n\t.reg .b32 a, b;\n\t"
      "mov.b64 {a, b}, %1;\n\t"
      "cvt.rn.bf16x2.f32 %0, b, a;\n\t}"
      : "=r"(hi)
      : "l"(v));
  if (TERMS == 2) {
    asm("{\n\t.reg .b32 a, b;\n\t.reg .b64 t;\n\t"
        "shl.b32 a, %1, 16;\n\t"
        "and.b32 b, %1, 0xffff0000;\n\t"
        "mov.b64 t, {a, b};\n\t"
        "sub.rn.f32x2 t, %2, t;\n\t"
        "mov.b64 {a, b}, t;\n\t"
        "cvt.rn.bf16x2.f32 %0, b, a;\n\t}"
        : "=r"(lo)
        : "r"(hi), "l"(v));
  }
}

template <int KIND, int TERMS, int BN>
__global__ void __launch_bounds__(GtCfg<KIND, TERMS, BN>::kThreads, 1)
    bl_grad_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmP,
                        const GtArgs P, unsigned long long limit_ns) {
  using C = GtCfg<KIND, TERMS, BN>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sOut = smem + C::kOutOffset;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);   // raw rows and dY have landed
  uint64_t* done = full + S;                                           // the MMAs have read the stage
  uint64_t* ready = done + S;       // leader's copy: both CTAs' converter warps have expanded the stage
  uint64_t* accfull = ready + S;
  uint64_t* accempty = accfull + 2;   // leader's copy: both CTAs' epilogue warps
  uint64_t* drain = accempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int nk = (P.L + C::kBC - 1) / C::kBC;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&done[s], 1);
      mbar_init(&ready[s], 2 * C::kGroupWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 2 * kGtEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();   // thread 0 comes last, and the barrier is a warp's instruction
  cluster_sync_all();   // barriers of both CTAs initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The pieces of this pair's chunks, in order: tile (k fastest, so that
  // neighbouring pairs share a slab of dY), stages [c0, c1) and its part's place (-1:
  // the whole tile).  Every role walks them by itself.
  struct Walk {
    int chunk, u, end;          // next stage of the chunk, its end (parts only)
    int kt, rt, c0, c1, place;
  };
  auto start = [&]() {
    Walk w;
    w.chunk = pair - npairs;
    w.u = w.end = 0;
    return w;
  };
  auto next = [&](Walk& w) {
    if (w.u >= w.end) {
      w.chunk += npairs;
      if (w.chunk >= P.cut.chunks) return false;
      if (w.chunk >= P.cut.whole) {
        w.u = (w.chunk - P.cut.whole) * P.cut.per;
        w.end = min((P.kt * P.rt - P.cut.whole) * P.cut.nkv, w.u + P.cut.per);
      }
    }
    int tile = w.chunk;
    w.c0 = 0;
    w.c1 = nk;
    w.place = -1;
    if (w.chunk >= P.cut.whole) {
      const int t = w.u / P.cut.nkv;
      tile = P.cut.whole + t;
      w.c0 = w.u - t * P.cut.nkv;
      w.c1 = min(nk, w.c0 + w.end - w.u);
      w.place = P.cut.place(t, w.chunk - P.cut.whole);
      w.u = min(w.end, (t + 1) * P.cut.nkv);
    }
    w.kt = tile % P.kt;
    w.rt = tile / P.kt;
    return true;
  };

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs; the whole warp, one lane issues) ----------------
    if (elect_one()) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
    }
    uint32_t g = 0;
    int s = 0;
    bool stop = false;
    for (Walk w = start(); !stop && next(w);) {
      const int k0 = w.kt * 2 * kGtK + static_cast<int>(rank) * kGtK;
      const int r0 = w.rt * BN + static_cast<int>(rank) * C::kHalf;
      for (int c = w.c0; c < w.c1; ++c, ++g) {
        if (g >= static_cast<uint32_t>(S) &&
            !__all_sync(0xffffffffu,
                        mbar_wait_cluster(&done[s], ((g / S) & 1) ^ 1u, abort_flag, limit_ns, kSiteProdEmpty))) {
          stop = true;
          break;
        }
        if (elect_one()) {
          uint8_t* sB = smem + C::kInOffset + s * C::kInBytes;
          mbar_arrive_expect_tx(&full[s], C::kInBytes);
          tma_load_2d(sB + C::kBBytes, &tmA, KIND == kGradInput ? k0 / 4 : k0, c * C::kBC, &full[s]);
          if (KIND == kGradInput) {
#pragma unroll
            for (int j = 0; j < C::kBC / 64; ++j)
              tma_load_2d(sB + j * C::kHalf * 128, &tmB, c * C::kBC + 64 * j, r0, &full[s]);
          } else {
#pragma unroll
            for (int j = 0; j < (C::kHalf + 63) / 64; ++j)
              tma_load_2d(sB + j * C::kBlockBytes, &tmB, r0 + 64 * j, c * C::kBC, &full[s]);
          }
        }
        if (++s == S) s = 0;
      }
    }
    const uint32_t issued = g;
    for (uint32_t t = 0; t < static_cast<uint32_t>(S) && t < issued; ++t) {
      const uint32_t last = t + S * ((issued - 1 - t) / S);
      mbar_wait(&full[t], (last / S) & 1, nullptr, limit_ns, kSiteDrain);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (leader only; the whole warp, one lane issues) ----------------
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16(2 * kGtK, BN, KIND == kGradWeight);
      constexpr uint32_t kBStep = KIND == kGradInput ? 2 : 128;   // 16 of the sum: 32 bytes K-major, 2048 MN-major
      const uint32_t base = smem_u32(smem);
      const uint32_t a0 = gt_desc_mn_lo(base, C::kBlockBytes);
      const uint32_t b0 = KIND == kGradInput ? gt_desc_k_lo(base + C::kInOffset)
                                             : gt_desc_mn_lo(base + C::kInOffset, C::kBlockBytes);
      int s = 0, as = 0, i = 0;
      uint32_t ph = 0;
      bool stop = false, seen = false;
      for (Walk w = start(); !stop && next(w);) {
        int c0 = w.c0;
        const int c1 = w.c1;
        while (c0 < c1) {   // a segment: the accumulator that was drained longest ago
          const int b = i & 1, ce = min(c1, c0 + min(C::kSegment, c1 - c0));
          // (every decision to give up is taken by the whole warp: elect.sync
          // below names all its lanes)
          if (i >= 2 &&
              !__all_sync(0xffffffffu,
                          mbar_wait_cluster(&accempty[b], ((i >> 1) & 1) ^ 1u, abort_flag, limit_ns, kSiteAcc))) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem + b * BN;
          uint32_t acc = 0;
          for (; c0 < ce; ++c0) {
            if (!__all_sync(0xffffffffu,
                            seen || mbar_wait_cluster(&ready[s], ph, abort_flag, limit_ns, kSiteMmaExfull))) {
              stop = true;
              break;
            }
            tc_fence_after();
            // look at the next stage's barrier now: the answer arrives while
            // this stage's MMAs are issued (a look that succeeds takes 165
            // clocks beside the converters' shared-memory traffic)
            const int sn = s + 1 == S ? 0 : s + 1;
            seen = mbar_test_wait_cluster(&ready[sn], sn ? ph : ph ^ 1u);
            if (elect_one()) {
              const uint32_t alo = a0 + as * (C::kASlotBytes / 16), blo = b0 + s * (C::kInBytes / 16);
#pragma unroll
              for (int j = 0; j < TERMS * (C::kBC / 64); ++j) {   // 64 of the sum each: hi, then lo
                constexpr int kB = C::kBC / 64;
                const uint32_t aj = (j / kB) * (C::kTileBytes / 16) + (j % kB) * 512;
                const uint32_t bj = (j % kB) * (KIND == kGradInput ? C::kHalf * 128 / 16 : 512);
                mma_bf16_tile_pair<kBStep>(d_tmem, alo + aj, blo + bj, idesc, j ? 1u : acc);
              }
              tc_commit_pair(&done[s], 3);
            }
            acc = 1;
            if (++as == C::kASlots) as = 0;
            if (++s == S) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (stop) break;
          if (elect_one()) tc_commit_pair(&accfull[b], 3);
          ++i;
        }
      }
      // no MMA of the pair may be in flight when either CTA frees its TMEM
      if (elect_one()) tc_commit_pair(drain, 1);
      mbar_wait(drain, 0, nullptr, limit_ns, kSiteDrain);
    }
  } else if (warp < C::kFirstEpi) {
    // ---------------- converters (both CTAs) ----------------
    const int grp = (warp - 2) / C::kGroupWarps;
    const int ct = threadIdx.x - 64 - grp * 32 * C::kGroupWarps;
    uint32_t g = 0;
    bool stop = false;
    for (Walk w = start(); !stop && next(w);) {
      for (int c = w.c0; c < w.c1; ++c, ++g) {
        if (g % C::kGroups != static_cast<uint32_t>(grp)) continue;
        const int s = g % S;
        const uint32_t sA = smem_u32(smem) + (g % C::kASlots) * C::kASlotBytes;
        const uint32_t raw = smem_u32(smem) + C::kInOffset + s * C::kInBytes + C::kBBytes;
        // The MMAs of the stage that last used the operand slot are done, and the
        // raw rows are here.  In this order: a parity tells a phase only from its
        // neighbours, and full[s]'s phase before this one belongs to another group's
        // stage, g - S, whose rows may land after those this group has just
        // expanded.  Once stage g - kASlots is through the MMAs, so is that one.
        auto wait_stage = [&]() {
          static_assert(C::kGroups <= C::kASlots && C::kASlots < S, "phases waited for are one ahead at most");
          bool ok = true;
          if (g >= static_cast<uint32_t>(C::kASlots)) {
            const uint32_t gp = g - C::kASlots;
            ok = mbar_wait_cluster(&done[gp % S], (gp / S) & 1, abort_flag, limit_ns, kSiteExpEmpty);
          }
          ok = ok && mbar_wait(&full[s], (g / S) & 1, abort_flag, limit_ns, kSiteExpFull);
          return __all_sync(0xffffffffu, ok) != 0;
        };
        if constexpr (KIND == kGradInput) {
          if (!wait_stage()) {
            stop = true;
            break;
          }
          // a quarter-warp takes four words of one 64-k block in two
          // neighbouring rows: the swizzle puts its eight 16-byte stores on
          // eight different bank groups
          const int row0 = 2 * (ct >> 4) + ((ct >> 2) & 1), gw = (ct & 3) + ((ct >> 3) & 1) * 4;
          constexpr int kRowStep = 32 * C::kGroupWarps / 8;
          uint32_t raw4[C::kBC / kRowStep];
#pragma unroll
          for (int i = 0; i < C::kBC / kRowStep; ++i)
            raw4[i] = ld_shared_u32(raw + (row0 + i * kRowStep) * 32 + gw * 4);
#pragma unroll
          for (int i = 0; i < C::kBC / kRowStep; ++i) {
            const int row = row0 + i * kRowStep;
            uint32_t v[8];
            expand16(raw4[i], v);
            const uint32_t rowa = sA + (gw >> 2) * C::kBlockBytes + row * 128, ch = 2 * (gw & 3), x = row & 7;
            st_shared_v4(rowa + ((ch ^ x) << 4), v[0], v[1], v[2], v[3]);
            st_shared_v4(rowa + (((ch + 1) ^ x) << 4), v[4], v[5], v[6], v[7]);
          }
        } else {
          constexpr int kRowStep = 32 * C::kGroupWarps / 16, kUnits = C::kBC / kRowStep;
          const int row0 = ct >> 4, u = ct & 15;   // 8 codes of a row
          float sc[kUnits];
#pragma unroll
          for (int i = 0; i < kUnits; ++i) {
            const int m = c * C::kBC + row0 + i * kRowStep;
            sc[i] = m < P.L ? __ldg(P.scale + m) : 1.f;
          }
          if (!wait_stage()) {
            stop = true;
            break;
          }
          uint2 q[kUnits];
#pragma unroll
          for (int i = 0; i < kUnits; ++i) q[i] = ld_shared_v2(raw + (row0 + i * kRowStep) * 128 + u * 8);
#pragma unroll
          for (int i = 0; i < kUnits; ++i) {
            const int row = row0 + i * kRowStep;
            // within 2^-23, far below the operand's step.  Scales above 2^126 would have a
            // subnormal reciprocal, flushed here; the entry point takes them up to 2^110,
            // where the lo of an fp32 result still is a normal bf16 or below 2^-16 of q / s.
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sc[i]));
            uint64_t rr;
            asm("mov.b64 %0, {%1, %1};" : "=l"(rr) : "f"(r));
            const uint32_t x0 = q[i].x ^ 0x80808080u, x1 = q[i].y ^ 0x80808080u;
            uint32_t hi[4], lo[4];
            split2<TERMS>(codes2_f32<0>(x0, rr), hi[0], lo[0]);
            split2<TERMS>(codes2_f32<2>(x0, rr), hi[1], lo[1]);
            split2<TERMS>(codes2_f32<0>(x1, rr), hi[2], lo[2]);
            split2<TERMS>(codes2_f32<2>(x1, rr), hi[3], lo[3]);
            const uint32_t at = sA + (u >> 3) * C::kBlockBytes + row * 128 + (((u & 7) ^ (row & 7)) << 4);
            st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
            if (TERMS == 2) st_shared_v4(at + C::kTileBytes, lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_smem();   // every writer, before the warp meets and one lane arrives
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(&ready[s], 0);
      }
    }
  } else {
    // ---------------- epilogue (both CTAs) ----------------
    // A warp has 32 k (its lanes) of half of the tile's r.  Results leave through
    // staging tiles and TMA: stores, or reductions that add to fp32 in memory (plain
    // stores of 128 bytes a warp took 7100 clocks a tile).  A bf16 result that is
    // added to is rounded once: what is there comes into the staging tile 16 bytes a
    // lane, and each lane adds its column.  Output of 8192 x 28672, 16 tokens: fp32 153
    // us stored, 403 added to (4.7 TB/s; 540 with plain loads instead of reductions);
    // bf16 128 and 271 us (930 with plain loads and stores of 2 bytes a lane; one
    // staging tile a warp, so that load, addition and store follow one another).
    const int q = warp & 3, half = (warp - C::kFirstEpi) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const float f = P.gamma ? *P.gamma : 1.f;
    uint8_t* so = sOut + (warp - C::kFirstEpi) * C::kOutBytes;
    int i = 0, buf = 0;
    Walk w = start();
    bool fresh = true;   // the piece's first segment
    for (w.c0 = w.c1 = 0;; ++i) {
      if (w.c0 >= w.c1) {
        if (!next(w)) break;
        fresh = true;
      }
      // (two terms: an fp32 result; one: a bf16 one; parts are fp32)
      const bool direct = w.place < 0, bf16 = TERMS == 1 && direct;
      const bool bf16_acc = KIND == kGradWeight && bf16 && P.accumulate;
      const CUtensorMap* tm = direct ? &tmD : &tmP;
      const int b = i & 1;
      const int kw = w.kt * 2 * kGtK + static_cast<int>(rank) * kGtK + q * 32;
      const int r0 = w.rt * BN + half * C::kHalf;
      const bool kin = kw < P.K;   // K is a multiple of 64: a warp's 32 k are all inside or all outside
      if (bf16_acc && kin) {
        // what will be added to, into L2 while the sum is formed
        for (int t = lane; t < C::kHalf && r0 + t < P.R; t += 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint16_t*>(P.out) +
                                                        static_cast<size_t>(r0 + t) * P.K + kw));
      }
      if (!__all_sync(0xffffffffu, mbar_wait_cluster(&accfull[b], (i >> 1) & 1, abort_flag, limit_ns, kSiteAcc) &&
                                       !*abort_flag))
        break;
      tc_fence_after();
      // the segments after the first add to what this warp stored itself: those
      // stores have to be complete
      const bool add = TERMS == 2 && ((direct && P.accumulate) || !fresh);
      if (add) {
        if (lane == 0) bulk_wait_group0();
        __syncwarp();
      }
#pragma unroll 1
      for (int c = 0; c < C::kHalf; c += C::kChunk) {
        uint32_t v[32];
        __syncwarp();   // tcgen05.ld is a warp's instruction, and lane 0 may still be issuing the last store
        if (C::kChunk == 32)
          tmem_ld_32x32b_x32(tmem + lane_base + b * BN + half * C::kHalf + c, v);
        else
          tmem_ld_32x32b_x16(tmem + lane_base + b * BN + half * C::kHalf + c, v);
        tmem_wait_ld();
        const int r = r0 + c;
        if (!kin || r >= P.R) continue;
        if (bf16) {
          if (lane == 0) bulk_wait_group_read0();   // the last store has read the tile
          __syncwarp();
          if (bf16_acc) {
            // rows (lane / 4) + 8 j of the chunk, 8 columns a lane
            const uint16_t* y = static_cast<const uint16_t*>(P.out) + static_cast<size_t>(r) * P.K + kw + (lane & 3) * 8;
            const uint32_t dst = smem_u32(so) + lane * 16;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int rr = (lane >> 2) + 8 * j;
              if (r + rr < P.R)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512 * j),
                             "l"(y + static_cast<size_t>(rr) * P.K)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int t = 0; t < C::kChunk; ++t)
              v[t] = __float_as_uint(
                  __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(so)[t * 32 + lane]) << 16) +
                  __uint_as_float(v[t]));
          }
#pragma unroll
          for (int t = 0; t < C::kChunk; ++t)
            reinterpret_cast<uint16_t*>(so)[t * 32 + lane] =
                __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[t]) * f));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(tm, kw, r, 0, so);
            bulk_commit_group();
          }
          continue;
        }
#pragma unroll
        for (int h = 0; h < C::kChunk; h += 16) {
          if (r + h >= P.R) break;
          uint8_t* tile = so + (TERMS == 2 ? buf * 2048 : 0);   // two tiles in turn, or one
          buf ^= 1;
          if (lane == 0) {
            if (TERMS == 2)
              bulk_wait_group_read1();
            else
              bulk_wait_group_read0();
          }
          __syncwarp();
#pragma unroll
          for (int t = 0; t < 16; ++t) reinterpret_cast<uint32_t*>(tile)[t * 32 + lane] = v[h + t];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            // in the result, or in a part of the tile's shape
            const int x = direct ? kw : kw - w.kt * 2 * kGtK, y = direct ? r + h : r + h - w.rt * BN;
            const int z = direct ? 0 : w.place;
            if (add)
              tma_reduce_add_3d(tm, x, y, z, tile);
            else
              tma_store_3d(tm, x, y, z, tile);
            bulk_commit_group();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(&accempty[b], 0);   // accumulator drained
      w.c0 += min(C::kSegment, w.c1 - w.c0);
      fresh = false;
    }
    if (lane == 0) bulk_wait_group0();   // outputs written before exit
  }
  if (P.cut.whole < P.kt * P.rt) pdl_launch_dependents();   // the join, which waits for this grid's end
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();   // the leader has drained its MMAs; both CTAs may free TMEM
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::kTmemCols);
  }
}

// out = f * (sum of a tile's parts, in order) (+ out), over the tiles that have
// parts.  A CTA takes kGtJoinRows rows of a tile, a thread four of them, so that
// four loads a part are in flight: the parts are in L2 and the loads' latency is
// what counts.  Launched as a dependent of the kernel that writes the parts.  With
// both, 8192 tokens of a 4096 x 4096 layer (bf16 weight gradient, 34 tiles in four
// parts) take 240 us, 249 with a float4 a thread and an ordinary launch.
constexpr int kGtJoinRows = 16;
__global__ void __launch_bounds__(256)
    bl_grad_join_kernel(const float* __restrict__ part, const GtCut cut, int bn, int kt, int R, int K, int part_rows,
                        int part_cols, const float* __restrict__ gamma, void* __restrict__ out, int out_bf16,
                        int accumulate) {
  pdl_wait();
  const int per_tile = bn / kGtJoinRows, t = blockIdx.x / per_tile;
  const int tile = cut.whole + t, kl = 4 * (threadIdx.x & 63), k = tile % kt * 2 * kGtK + kl;
  const int rl = (blockIdx.x - t * per_tile) * kGtJoinRows + (threadIdx.x >> 6), r0 = tile / kt * bn + rl;
  if (k >= K) return;
  const int parts = cut.parts(t);
  const size_t plane = static_cast<size_t>(part_rows) * part_cols;
  const float* src = part + cut.place(t, cut.first(t)) * plane + rl * part_cols + kl;
  float4 s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < parts; ++j) {
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * i;
      v[i] = r < R ? __ldcg(reinterpret_cast<const float4*>(src + j * plane + 4 * i * part_cols))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i].x += v[i].x;
      s[i].y += v[i].y;
      s[i].z += v[i].z;
      s[i].w += v[i].w;
    }
  }
  const float f = gamma ? *gamma : 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * i;
    if (r >= R) return;
    const size_t at = static_cast<size_t>(r) * K + k;
    float4 v = make_float4(s[i].x * f, s[i].y * f, s[i].z * f, s[i].w * f);
    if (out_bf16) {
      uint2* y = reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at);
      if (accumulate) {
        const uint2 o = *y;
        v.x += bf16_lo(o.x);
        v.y += bf16_hi(o.x);
        v.z += bf16_lo(o.y);
        v.w += bf16_hi(o.y);
      }
      *y = make_uint2(pack2_bf16(v.x, v.y), pack2_bf16(v.z, v.w));
    } else {
      float4* y = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
      if (accumulate) {
        const float4 o = *y;
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
      }
      *y = v;
    }
  }
}

// Rows of dY at a 16-byte stride (TMA needs one): [M, N] -> [M, ld].
__global__ void __launch_bounds__(256)
    bl_grad_pad_kernel(const uint16_t* __restrict__ src, uint16_t* __restrict__ dst, int M, int N, int ld) {
  for (int m = blockIdx.y; m < M; m += gridDim.y)
    for (int n = blockIdx.x * 256 + threadIdx.x; n < ld; n += gridDim.x * 256)
      dst[static_cast<size_t>(m) * ld + n] = n < N ? src[static_cast<size_t>(m) * N + n] : 0;
}

}  // namespace bl
