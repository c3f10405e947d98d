// Decode attention with query rows as the M side of the tensor-core tiles: for batches
// that share a prefix, and for capped, biased or windowed scores.
//
// For query row r = (sequence b, head) of kv head h, over the tokens t of b's context:
//   s_t = scale * q_r . k_t;  s_t = c tanh(s_t / c) with a cap c;  s_t += slope (t - (L_b - 1))
//   out_r = sum_t softmax_t(s) v_t,  tokens t < L_b - window masked.
// Sequences of one group hold the same blocks for their first tokens, so those tokens'
// K/V serve rows = sequences x G query rows of a kv head at once (G: query heads per kv
// head) and are read once for up to 256 of them. An item is
//   (group, kv head, tile of 256 rows) over the group's shared pages, or
//   (sequence, kv head) over the sequence's own pages,
// and consists of chunks of 128 tokens. All chunks of all items in a row are cut into one
// equal range per CTA (every CTA computes the same cuts from the lengths, so there is no
// work queue and the load is even whatever the lengths); the part of an item in one CTA is
// a segment, which leaves a normalised partial output and its log-sum-exp per row, and a
// second small launch merges a row's partials.
//
// Inside a CTA two pipes, each a softmax warpgroup with one TMEM score tile S (128 rows x
// 128 tokens, fp32), whose columns then hold the weights P (16 bits), and one output tile O:
//   S = Q . K^T  (Q 128 x D from shared memory, K 128 tokens x D)  tcgen05 kind::f16
//   O += P . V   (P from TMEM, V chunk as an MN-major operand)
// A wide segment (more than 128 rows) gives each pipe one of its two row tiles, and both
// read every chunk; in a narrow one the pipes take alternate chunks. S of a shared chunk is
// turned into weights in halves of 64 tokens, so that PV of the first half runs beside the
// softmax of the second; the tensor pipe works for one pipe while the other's warpgroup does
// its softmax. A sequence's own item has only G rows: they stand in Q four times, once for the
// TMEM lanes of each warp of a pipe, and each warp takes a quarter of the chunk's tokens (its
// P is zero elsewhere), with a maximum and a sum of its own; at the segment's end the four
// parts are joined through shared memory. One thread owns one row, so maxima and sums need
// no exchange. The running maximum is only followed when it grows by more than a threshold
// (2^8 in bf16, 2 in fp16), which spares nearly every rescaling of O; the final division
// makes up for it.
// P is the sum of two 16-bit terms, and PV takes twice the MMAs: a weight is off by at most
// 2^-16 of itself in bf16; in fp16, whose weights carry a factor 2^14, by 2^-22 of itself or
// 2^-39 of the running maximum (below 2^-17 of which the second term is subnormal), whichever
// is more. The denominator adds the weights before their rounding. bf16 weights carry a factor
// 2^-24, so that sums over 65536 tokens of V near the type's largest value stay finite (values
// of V below 2^-110 lose bits to it).
//
// Warps 0-3 and 4-7: the pipes. Warp 8: page loads (TMA) into a ring of K and V slots, the
// walk over segments. Warp 9: TMEM, both MMAs. Every wait is bounded.
//
// Measured (GB300, calls in a graph, merge included; bf16, head dim 128; the first case's K/V,
// 84 MB, stays in the L2, the others' does not). 128 sequences of 64/8 heads behind 16384
// shared tokens, 32 own ones: 98 us, 700 TFLOP/s (697 us without sharing), capped 148 us; the
// MMAs alone, two for each weight, take 54 us at the rate of a large library product. A wide
// chunk takes 2.2 us, some 4300 cycles, of which the tensor pipe works nearly three quarters:
// its softmax, on two warps a scheduler, bounds. 16 sequences (128 rows) behind 65536 tokens:
// 69 us, 3.9 TB/s (494 us); the ring's 160 KiB bound, which holds a V chunk until both halves
// of its PV are done. Own tokens only: 4 x 32768 at 32/8 heads 90 us, capped 94 us (6.0 and
// 5.7 TB/s of a copy's 6.7); 96 x 1024 at 64/8 heads 77 us, capped 80 us. The plan, launches
// and merge are 9 us of a call that has little to do.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pda_internal.h"
#include "ptx.cuh"
#include "row_attn.h"

namespace pda {
namespace row {

constexpr int kThreads = 320;
constexpr int kWarpLoad = 8;
constexpr int kWarpMma = 9;
constexpr int kHalf = kT * 128;   // 64 dims of 128 rows: 16 KiB
constexpr int kSegRing = 4;
constexpr int kSmallQ = 4;           // places for the queries of small segments, at most
constexpr int kQBars = 2 + kSmallQ;  // Q tiles, then those places
constexpr int kJoinBytes = 16 * 1024;
constexpr int kSegInts = 12;
constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kTmemCols = 512;

// What the merge needs to know of a sequence.
struct SeqPlan {
  int pre_start;   // where its tile's item of kv head 0 begins, in the row of all items
  int pre_stride;  // from one kv head's item to the next one's
  int pre_n;       // chunks of the shared part (0: none)
  int pre_row;     // row of its first query head in the item (tile 1 from kT on), + kWide if wide
  int own_start;   // where its own part's item of kv head 0 begins
  int own_n;       // chunks of its own part
  int pad0, pad1;
};
static_assert(sizeof(SeqPlan) == kPlanInts * 4, "plan entry");
constexpr int kWide = 1 << 16;

// What an item of n chunks costs, in the units that the cut counts: a chunk, and what comes on
// top once. (A unit is about 0.16 us: a wide chunk 2.2 us, an own one 1.5 us of the memory's
// time, a segment of one own chunk 2.2 us. A wide chunk at 11, 12, 13, 14, 15 and 16: 128
// sequences of 64/8 heads behind 16384 tokens 101.6, 101.6, 98.9, 97.4, 97.2, 100.3 us. Fixed
// parts of 4 / 14, 6 / 14, 8 / 16 and 6 / 20 for own and shared items: the same 102.6, 98.0,
// 100.8, 97.9 us, 96 sequences of 32 to 4096 tokens at 64/8 heads 69.3, 65.2, 65.5, 65.3 us.)
// Chunk 0 stands for the fixed part too, so that it belongs to the CTA in whose range the item
// begins.
enum ItemKind { kOwnItem, kTileItem, kWideItem };  // a sequence's own; shared, up to 128 rows; up to 256
__device__ __forceinline__ int item_chunk(int kind) { return kind == kWideItem ? 14 : kind == kTileItem ? 9 : 8; }
__device__ __forceinline__ int item_fixed(int kind) { return kind == kOwnItem ? 6 : 14; }
__device__ __forceinline__ int item_cost(int kind, int n) {
  return n > 0 ? item_fixed(kind) + n * item_chunk(kind) : 0;
}
// The chunks of an item that begin before position x of it.
__device__ __forceinline__ int chunk_at(int kind, int n, int x) {
  if (x <= 0) return 0;
  const int c = item_chunk(kind), y = x - item_fixed(kind);
  // ceil(y / c), the divisors written out so that none is a division
  const int up = kind == kWideItem ? (y + 13) / 14 : kind == kTileItem ? (y + 8) / 9 : (y + 7) / 8;
  return y <= c ? min(1, n) : min(n, up);
}

// Partial rows in the workspace: [B * Hq][2] of the segments that start a shared item (by
// pipe, or entry 0 for a wide one), [B * Hq][2] of those that start an own item, then per
// CTA 2 * cap rows of the one segment that continues another CTA's item.
__device__ __forceinline__ int64_t ws_first(const Params& p, bool own, int64_t row, int pipe) {
  return ((own ? (int64_t)p.B * p.Hq : 0) + row) * 2 + pipe;
}
__device__ __forceinline__ int64_t ws_next(const Params& p, int cta, int cap, int tile, int r) {
  return 4 * (int64_t)p.B * p.Hq + (int64_t)cta * 2 * cap + tile * cap + r;
}
__device__ __forceinline__ int ws_cap(const Params& p) { return min(kT, p.B * p.G); }

template <int D>
struct Layout {
  static constexpr int kTile = kT * D * 2;                // Q tile, K or V chunk
  static constexpr int kSlots = D == 128 ? 5 : 10;        // K and V slots, 160 KiB
  static constexpr int kOffQ = kSlots * kTile;
  // [pipe][16 KiB] for the join of a small segment's four parts: the second Q tile (an own
  // segment follows no wide one that still needs it), or at D 64 memory of its own
  static constexpr int kOffJoin = D == 128 ? kOffQ + kTile : kOffQ + 2 * kTile;
  static constexpr int kOffBar = kOffJoin + 2 * kJoinBytes;
  static constexpr int kBars = 2 * kSlots + 2 * kQBars + 2 * kSegRing + 15;
  static constexpr int kOffMl = kOffBar + kBars * 8;  // [pipe][4 warps][16 rows] maximum and sum
  static constexpr int kOffTmem = kOffMl + 2 * 4 * 16 * 8;
  static constexpr int kOffSeg = kOffTmem + 16;
  static constexpr int kOffScan = kOffSeg + kSegRing * kSegInts * 4;  // warp sums, start, total
  static constexpr int kOffCu = kOffScan + 16 * 4;
  static constexpr int kOffShared = kOffCu + (kMaxPrefixes + 4) * 2;
  static constexpr int kOffRow = kOffShared + kMaxPrefixes * 4;
  static constexpr int kBytes = kOffRow + kMaxPrefixes * 4;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
  static_assert((kMaxBatch + kMaxPrefixes) * 4 <= kSlots * kTile, "the plan's sums fit the ring");
};

template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (FP16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool FP16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if constexpr (FP16) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
}

// 32 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(
          r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Whether the phase with the given parity has completed; does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// One lane of the (converged) warp. The compiler knows of elect.sync that a single thread is
// active, and issues MMAs from uniform registers without a loop around each.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// D[tmem] (+)= A[tmem] * B[smem], issued by one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Eight consecutive floats (32-byte aligned) in one store.
__device__ __forceinline__ void store8(float* dst, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Pairs of floats in one 64-bit register: one instruction for two fused multiply-adds or sums.
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 scores x to weights 2^(x qs + neg): the TMEM columns at addr get 16 of first terms and 16
// of second ones; the sums add the weights as they were before.
template <bool FP16>
__device__ __forceinline__ void weights(uint32_t addr, const float* x, uint64_t qs2, uint64_t neg2,
                                        float& sum0, float& sum1) {
  uint32_t w[16], w2[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    float y0, y1;
    f32x2_split(f32x2_fma(f32x2(x[2 * q], x[2 * q + 1]), qs2, neg2), y0, y1);
    const float p0 = ex2_ftz(y0), p1 = ex2_ftz(y1);
    w[q] = pack16<FP16>(p0, p1);
    const float2 f = unpack16<FP16>(w[q]);
    w2[q] = pack16<FP16>(p0 - f.x, p1 - f.y);
    sum0 += p0;
    sum1 += p1;
  }
  tmem_st16(addr, w);
  tmem_st16(addr + 16, w2);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max32(const float* x) {
  float a[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int q = 4; q < 28; q += 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = max3(a[i], x[q + i], x[q + i + 4]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = fmaxf(a[i], x[28 + i]);
  return max3(fmaxf(a[0], a[1]), a[2], a[3]);
}

// tanh(y) / y for |y| <= 1/2 as a polynomial in y^2, off by at most 2^-25 (a score capped by way of
// it, with all roundings in fp32, by at most 2^-22.6 of itself): a weighted least-squares
// fit of the relative error on Chebyshev points, the weights drawn towards the largest errors
// (Lawson, "Contributions to the theory of linear least maximum approximations", 1961).
__device__ __forceinline__ constexpr float tanh_coeff(int i) {
  return i == 0 ? 1.f : i == 1 ? -0.33333069f : i == 2 ? 0.13324779f : i == 3 ? -0.05298607f : 0.017135005f;
}

// Products q . k of 32 tokens to capped and biased scores in base-2 units; far: the first
// token's distance from the context's last one (t - (L - 1)); live: the row counts.
__device__ __forceinline__ void score_mods(const Params& p, float* x, float slope, float far, bool live) {
  if (p.cap > 0.f) {
    const float c = p.cap * kLog2e;
    float most = 0.f;
#pragma unroll
    for (int q = 0; q < 32; ++q) most = fmaxf(most, fabsf(x[q]));
    if (__all_sync(0xffffffffu, !live || most * fabsf(p.cap_in) <= 0.5f)) {
      // what most caps see: two scores an instruction on the multiply-add pipe
      const uint64_t in2 = f32x2(p.cap_in, p.cap_in);
      uint64_t k2[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) k2[i] = f32x2(c * tanh_coeff(i), c * tanh_coeff(i));
#pragma unroll
      for (int q = 0; q < 32; q += 2) {
        const uint64_t y = f32x2_mul(f32x2(x[q], x[q + 1]), in2), z = f32x2_mul(y, y);
        uint64_t r = k2[4];
#pragma unroll
        for (int i = 3; i >= 0; --i) r = f32x2_fma(r, z, k2[i]);
        f32x2_split(f32x2_mul(r, y), x[q], x[q + 1]);
      }
    } else if (p.cap <= 128.f) {
      // c tanh(y) = c - 2 c / (1 + e^2y): off by at most a few 2^-24 c
      const float y2 = 2.f * kLog2e * p.cap_in;
#pragma unroll
      for (int q = 0; q < 32; ++q) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2_ftz(x[q] * y2) + 1.f));
        x[q] = fmaf(-2.f * c, r, c);
      }
    } else {  // a large cap: either, by the score
#pragma unroll
      for (int q = 0; q < 32; ++q) {
        const float y = x[q] * p.cap_in, z = y * y;
        const float poly = fmaf(fmaf(fmaf(fmaf(tanh_coeff(4), z, tanh_coeff(3)), z, tanh_coeff(2)), z, tanh_coeff(1)), z, tanh_coeff(0)) * y;
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2_ftz(y * (2.f * kLog2e)) + 1.f));
        x[q] = c * (fabsf(y) <= 0.5f ? poly : fmaf(-2.f, r, 1.f));
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 32; ++q) x[q] *= p.qscale;
  }
  if (p.slopes != nullptr) {
#pragma unroll
    for (int q = 0; q < 32; ++q) x[q] = fmaf(slope, far + (float)q, x[q]);
  }
}

__device__ __forceinline__ int context_len(const Params& p, int b) {
  const int L = __ldg(p.context_lens + b);
  const int64_t most = (int64_t)p.max_blocks * p.block_size;
  return L < 0 ? 0 : (L > most ? (int)most : L);
}

// The last prefix group g with cu[g] <= b, if b < cu[g + 1] (else -1).
__device__ __forceinline__ int group_of(const volatile uint16_t* cu, int P, int b) {
  int lo = 0, hi = P + 1;  // first g with cu[g] > b
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= b) lo = mid + 1; else hi = mid;
  }
  return lo >= 1 && lo <= P ? lo - 1 : -1;
}

// A sequence's own part: its first token and page, and its chunks.
struct Own {
  int L, first_tok, first_page, n;
};
__device__ __forceinline__ Own own_part(const Params& p, int len, int shared_pages) {
  Own o;
  o.L = len;
  o.first_tok = p.window > 0 && o.L > p.window ? o.L - p.window : 0;
  o.first_page = o.first_tok >> p.bs_log;
  if (shared_pages > 0) {
    o.first_page = shared_pages;
    o.first_tok = shared_pages << p.bs_log;
  }
  const int first = o.first_page << p.bs_log;
  o.n = o.L > first ? (o.L - first + kT - 1) / kT : 0;
  return o;
}

struct Seg {
  int n, wide, b0, n_seq, h, t0, t_end, t_lo, first, own, cc;
  int par;  // pipe of its first step: steps take the pipes in turns, across segments too
};
__device__ __forceinline__ void seg_put(volatile int* d, const Seg& s) {
  d[0] = s.n; d[1] = s.wide; d[2] = s.b0; d[3] = s.n_seq; d[4] = s.h; d[5] = s.t0;
  d[6] = s.t_end; d[7] = s.t_lo; d[8] = s.first; d[9] = s.own; d[10] = s.cc; d[11] = s.par;
}
__device__ __forceinline__ void seg_get(const volatile int* d, Seg& s) {
  s.n = d[0]; s.wide = d[1]; s.b0 = d[2]; s.n_seq = d[3]; s.h = d[4]; s.t0 = d[5];
  s.t_end = d[6]; s.t_lo = d[7]; s.first = d[8]; s.own = d[9]; s.cc = d[10]; s.par = d[11];
}

template <int D, bool FP16, bool MOD>
__global__ void __launch_bounds__(kThreads, 1)
    row_attn_kernel(const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v,
                    const __grid_constant__ CUtensorMap tmap_q,
                    const __grid_constant__ CUtensorMap tmap_q1, const Params p) {
  using L = Layout<D>;
  constexpr int NB = D / 64;
  constexpr int kSlots = L::kSlots;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t base_u32 = smem_u32(base);
  const uint32_t bar0 = base_u32 + L::kOffBar;
  auto kv_full = [&](int s) { return bar0 + 8u * s; };
  auto kv_empty = [&](int s) { return bar0 + 8u * (kSlots + s); };
  auto q_full = [&](int s) { return bar0 + 8u * (2 * kSlots + s); };
  auto q_empty = [&](int s) { return bar0 + 8u * (2 * kSlots + kQBars + s); };
  constexpr int kBar1 = 2 * kSlots + 2 * kQBars;
  auto seg_full = [&](int s) { return bar0 + 8u * (kBar1 + s); };
  auto seg_empty = [&](int s) { return bar0 + 8u * (kBar1 + kSegRing + s); };
  // of pipe t, and of half h of its score tile
  auto s_full = [&](int t) { return bar0 + 8u * (kBar1 + 2 * kSegRing + t); };
  auto p_full = [&](int t, int h) { return bar0 + 8u * (kBar1 + 2 * kSegRing + 2 + 2 * t + h); };
  auto pv_done = [&](int t, int h) { return bar0 + 8u * (kBar1 + 2 * kSegRing + 6 + 2 * t + h); };
  auto o_free = [&](int t) { return bar0 + 8u * (kBar1 + 2 * kSegRing + 10 + t); };
  auto joint = [&](int t) { return bar0 + 8u * (kBar1 + 2 * kSegRing + 12 + t); };
  const uint32_t drained = bar0 + 8u * (kBar1 + 2 * kSegRing + 14);
  // small segments' queries: rows 32 w .. 32 w + G - 1 of a tile for w < 4, so that tiles 8
  // (16) rows further in the same memory hold those of four (two) segments
  const int small_rows = p.G > 8 ? 16 : 8, n_small = 32 / small_rows;
  volatile int* seg_ring = reinterpret_cast<volatile int*>(base + L::kOffSeg);
  volatile int* scan = reinterpret_cast<volatile int*>(base + L::kOffScan);
  volatile uint16_t* cu = reinterpret_cast<volatile uint16_t*>(base + L::kOffCu);
  int* shared_pages = reinterpret_cast<int*>(base + L::kOffShared);  // of each group
  int* shared_row = reinterpret_cast<int*>(base + L::kOffRow);       // a sequence that holds them
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  const int G = p.G, spt = p.spt;  // sequences of a row tile
  // x / (2 spt) for x < 2^14 and the sequence of row r of a tile, without dividing
  auto tile_of = [&](int x) { return (int)__umulhi((unsigned)x, p.tile_mul); };
  auto seq_of = [&](int r) { return (int)((unsigned)r * p.group_mul >> 16); };
  bool failed = false;

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    for (int s = 0; s < kQBars; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(joint(s), 4);
      mbar_init(s_full(s), 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(p_full(s, h), 4);
        mbar_init(pv_done(s, h), 1);
      }
      mbar_init(o_free(s), 4);
    }
    mbar_init(drained, 1);
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(seg_full(s), 1);
      mbar_init(seg_empty(s), 9);
    }
    fence_mbar_init();
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    prefetch_tensormap(&tmap_q);
    prefetch_tensormap(&tmap_q1);
  }
  if (warp == kWarpMma) {
    tmem_alloc(base_u32 + L::kOffTmem, kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();

  // ------------------------------- the plan -------------------------------
  // What every element (the groups, then the sequences) costs, and the running sum; the
  // ring's memory holds them. What a thread needs of the inputs it loads at once.
  int P = p.P;
  int* sum = reinterpret_cast<int*>(base);
  const int my_len = tid < p.B ? context_len(p, tid) : 0;
  int my_prefix = 0;
  if (P > 0) {
    const int mine = tid <= P ? __ldg(p.cu_seqs + tid) : 0, next = tid < P ? __ldg(p.cu_seqs + tid + 1) : mine;
    my_prefix = tid < P ? max(0, __ldg(p.prefix_lens + tid)) : 0;
    if (tid <= P) cu[tid] = (uint16_t)mine;
    if (tid < P) shared_pages[tid] = shared_row[tid] = 0x7fffffff;
    if (__syncthreads_or(mine > next || mine < 0 || mine > p.B)) {
      P = 0;  // no grouping: every sequence reads its own table row
      if (tid == 0 && blockIdx.x == 0 && atomicCAS(p.err, 0, kErrCuSeqs) == 0) p.err[1] = 0;
    }
  }
  auto len_of = [&](int b) { return b == tid ? my_len : context_len(p, b); };
  const int my_group = P > 0 && tid < p.B ? group_of(cu, P, tid) : -1;
  auto group_at = [&](int b) { return P == 0 ? -1 : b == tid ? my_group : group_of(cu, P, b); };
  if (P > 0) {
    for (int b = tid; b < p.B; b += kThreads) {
      // an empty sequence (a padded batch) has no say, and its table row is not read
      const int g = group_at(b), n = len_of(b);
      const unsigned on = __activemask();
      const bool in = g >= 0 && n > 0;
      const int g0 = __shfl_sync(on, g, __ffs(on) - 1);
      if (__all_sync(on, g == g0)) {  // the warp's sequences are of one group
        const int least = __reduce_min_sync(on, in ? n : 0x7fffffff);
        const int row = __reduce_min_sync(on, in ? b : 0x7fffffff);
        if (g0 >= 0 && lane == __ffs(on) - 1) {
          atomicMin(shared_pages + g0, least);
          atomicMin(shared_row + g0, row);
        }
      } else if (in) {
        atomicMin(shared_pages + g, n);
        atomicMin(shared_row + g, b);
      }
    }
    __syncthreads();
    if (tid < P) {
      const int n = min(shared_pages[tid], my_prefix);
      shared_pages[tid] = cu[tid + 1] - cu[tid] > 1 && shared_row[tid] < p.B ? n >> p.bs_log : 0;
    }
    __syncthreads();
  }
  auto tiles_of = [&](int g) { return tile_of(cu[g + 1] - cu[g] + 2 * spt - 1); };
  auto group_chunks = [&](int g) { return ((shared_pages[g] << p.bs_log) + kT - 1) / kT; };
  // the last tile of a group may be narrow, the others are wide
  auto last_kind = [&](int g, int tiles) { return cu[g + 1] - cu[g] - (tiles - 1) * 2 * spt > spt ? kWideItem : kTileItem; };
  auto group_cost = [&](int g) {  // of one kv head
    const int n = group_chunks(g), tiles = tiles_of(g);
    return (tiles - 1) * item_cost(kWideItem, n) + item_cost(last_kind(g, tiles), n);
  };
  auto seq_shared = [&](int b) {
    const int g = P > 0 ? group_of(cu, P, b) : -1;
    return g >= 0 ? shared_pages[g] : 0;
  };
  const int n_elem = P + p.B;
  if (tid < P) sum[tid] = tiles_of(tid) > 0 ? p.Hkv * group_cost(tid) : 0;
  for (int b = tid; b < p.B; b += kThreads) {
    const int g = group_at(b);
    sum[P + b] = p.Hkv * item_cost(kOwnItem, own_part(p, len_of(b), g >= 0 ? shared_pages[g] : 0).n);
  }
  __syncthreads();
  const int per_thread = (n_elem + kThreads - 1) / kThreads;
  const int e0 = min(n_elem, tid * per_thread), e1 = min(n_elem, e0 + per_thread);
  {
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += sum[e];
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int v = scan[w];
      all += v;
      if (w < warp) before += v;
    }
    int at = before + incl - mine;
    for (int e = e0; e < e1; ++e) {
      const int n = sum[e];
      sum[e] = at;
      at += n;
    }
    if (tid == 0) scan[10] = all;
    __syncthreads();
  }
  const int total = scan[10];
  // no less than a chunk each: finer cuts would only leave empty ranges
  const int per = max(item_chunk(kOwnItem), (total + (int)gridDim.x - 1) / (int)gridDim.x);
  const int r0 = min((int64_t)total, (int64_t)blockIdx.x * per);
  const int r1 = min((int64_t)total, (int64_t)r0 + per);
  // the element that r0 falls into
  for (int e = e0; e < e1; ++e) {
    const int next = e + 1 < n_elem ? sum[e + 1] : total;
    if (r0 >= sum[e] && r0 < next) {
      scan[11] = e;
      scan[12] = r0 - sum[e];
    }
  }
  if (blockIdx.x == gridDim.x - 1) {  // for the merge, by the CTA with the least left to do
    if (tid == 0) p.plan[0] = per, p.plan[1] = (int)(0xffffffffu / (unsigned)per);
    SeqPlan* plan = reinterpret_cast<SeqPlan*>(p.plan + kPlanInts);
    for (int b = tid; b < p.B; b += kThreads) {
      SeqPlan s = {};
      const int g = group_at(b), len = len_of(b);
      if (g >= 0 && shared_pages[g] > 0 && len > 0) {
        const int i = b - cu[g], tile = tile_of(i), r = i - tile * 2 * spt;
        const int n_seq = min(2 * spt, cu[g + 1] - cu[g] - tile * 2 * spt);
        s.pre_n = group_chunks(g);
        s.pre_start = sum[g] + tile * item_cost(kWideItem, s.pre_n);
        s.pre_stride = group_cost(g);
        s.pre_row = (r >= spt ? kT + (r - spt) * G : r * G) + (n_seq > spt ? kWide : 0);
      }
      s.own_start = sum[P + b];
      s.own_n = own_part(p, len, g >= 0 ? shared_pages[g] : 0).n;
      plan[b] = s;
    }
  }
  fence_proxy_async_smem();  // the ring's memory goes to the TMA unit
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *reinterpret_cast<volatile uint32_t*>(base + L::kOffTmem), 0);
  auto tS = [&](int t) { return tmem + (uint32_t)(t * kT); };
  auto tO = [&](int t) { return tmem + (uint32_t)(2 * kT + t * D); };

  if (r0 < r1) {
    if (warp == kWarpLoad) {
      // ------------------------- segments and loads -------------------------
      const int PPS = kT >> p.bs_log;
      const int out_of_range = (int)(p.num_blocks * p.block_size);  // rows there read as zeros
      const int my_page = lane % PPS, my_half = lane / PPS;  // PPS * NB <= 32: a box per lane
      int fill = 0, qfill = 0, qsmall = 0, k = 0, cc = 0, par = 0;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        const bool ok = mbar_wait(bar, parity);
        if (!__all_sync(kFull, ok)) failed = true;
        return !failed;
      };
      auto publish = [&](const Seg& s) {
        const int slot = k % kSegRing;
        if (k >= kSegRing && !wait(seg_empty(slot), (k / kSegRing - 1) & 1)) return false;
        if (lane == 0) {
          seg_put(seg_ring + slot * kSegInts, s);
          mbar_arrive(seg_full(slot));
        }
        __syncwarp();
        ++k;
        return true;
      };
      // Sequences in order, with the own part and the first table entries of the next one and
      // the length of the one after it on their way, so that a change of sequence waits for
      // neither.
      auto len_at = [&](int b) { return b < p.B ? context_len(p, b) : 0; };
      auto own_at = [&](int b, int len) { return b < p.B ? own_part(p, len, seq_shared(b)) : Own{}; };
      auto page_end_of = [&](const Own& o) { return (o.L + p.block_size - 1) >> p.bs_log; };
      auto first_ids = [&](int b, const Own& o) {
        return o.n > 0 && o.first_page + my_page < page_end_of(o)
                   ? __ldg(p.block_table + (int64_t)b * p.max_blocks + o.first_page + my_page) : 0;
      };
      int e = scan[11], at = r0 - scan[12];  // the element, and where it begins
      Own own = {}, own1 = {};
      int ids = 0, ids1 = 0, len2 = 0;
      auto prime = [&](int b) {  // sequence b becomes the current one
        const int l0 = len_at(b), l1 = len_at(b + 1);
        len2 = len_at(b + 2);
        own = own_at(b, l0);
        ids = first_ids(b, own);
        own1 = own_at(b + 1, l1);
        ids1 = first_ids(b + 1, own1);
      };
      auto shift = [&]() {  // the next sequence becomes the current one
        ++e;
        own = own1;
        ids = ids1;
        own1 = own_at(e - P + 1, len2);
        ids1 = first_ids(e - P + 1, own1);
        len2 = len_at(e - P + 2);
      };
      if (e >= P) prime(e - P);
      // (h, tile) or h of the item that r0 falls into
      int h, tile = 0;
      {
        const int off = r0 - at;
        if (e >= P) {
          const int c = item_cost(kOwnItem, own.n);
          h = off / c;
          at += h * c;
        } else {
          const int c = group_cost(e), w = item_cost(kWideItem, group_chunks(e));
          h = off / c;
          tile = min((off - h * c) / w, tiles_of(e) - 1);
          at += h * c + tile * w;
        }
      }
      while (at < r1 && !failed) {
        const bool is_own = e >= P;
        Seg s;
        s.cc = cc;
        s.own = is_own;
        s.h = h;
        s.par = par;
        int page, page_end, n_item, kind, tiles = 1;
        if (is_own) {
          s.b0 = e - P;
          s.n_seq = 1;
          s.t_end = own.L;
          s.t_lo = own.first_tok;
          page = own.first_page;
          page_end = page_end_of(own);
          n_item = own.n;
          kind = kOwnItem;
        } else {
          tiles = tiles_of(e);
          s.b0 = cu[e] + tile * 2 * spt;
          s.n_seq = min(2 * spt, cu[e + 1] - s.b0);
          s.t_end = shared_pages[e] << p.bs_log;
          s.t_lo = 0;
          page = 0;
          page_end = shared_pages[e];
          n_item = group_chunks(e);
          kind = s.n_seq > spt ? kWideItem : kTileItem;
        }
        const int chunk = chunk_at(kind, n_item, r0 - at);
        const int n = chunk_at(kind, n_item, r1 - at) - chunk;
        const int32_t* table = p.block_table + (int64_t)(is_own ? e - P : shared_row[e]) * p.max_blocks;
        page += chunk * PPS;
        int id = ids;
        if (!is_own || chunk > 0) id = page + my_page < page_end ? __ldg(table + page + my_page) : 0;
        s.n = n;
        s.first = chunk == 0;
        s.wide = kind == kWideItem;
        s.t0 = page << p.bs_log;
        if (n > 0) {
          if (!s.wide) par ^= n & 1;
          if (!publish(s)) break;
        // the queries
        if (is_own) {
          if (qsmall == 0)  // the tile that the small places are in
            for (int i = max(0, qfill - 2); i < qfill; ++i)
              if (!wait(q_empty(i & 1), (i >> 1) & 1)) break;
          const int slot = qsmall % n_small;
          if (qsmall >= n_small && !failed) wait(q_empty(2 + slot), (qsmall / n_small - 1) & 1);
          if (failed) break;
          if (lane == 0) mbar_arrive_expect_tx(q_full(2 + slot), (uint32_t)(4 * G * 128 * NB));
          __syncwarp();
          if (lane < 4 * NB)
            tma_load_3d(base_u32 + L::kOffQ + (lane >> 2) * kHalf + ((lane & 3) * 32 + slot * small_rows) * 128,
                        &tmap_q1, (lane >> 2) * 64, s.h * G, s.b0, q_full(2 + slot));
          ++qsmall;
        } else {
          for (int t = 0; t <= s.wide; ++t, ++qfill) {
            const int slot = qfill & 1;
            if (qfill >= 2 && !wait(q_empty(slot), ((qfill >> 1) - 1) & 1)) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(q_full(slot), (uint32_t)(spt * G * 128 * NB));
#pragma unroll
              for (int i = 0; i < NB; ++i)
                tma_load_3d(base_u32 + L::kOffQ + slot * L::kTile + i * kHalf, &tmap_q, i * 64, s.h * G,
                            s.b0 + t * spt, q_full(slot));
            }
            __syncwarp();
          }
        }
        if (failed) break;
        for (int c = 0; c < n; ++c) {
          const int np = min(PPS, page_end - page);
          const int row = (unsigned)id < (unsigned long long)p.num_blocks ? id << p.bs_log : out_of_range;
          page += PPS;
          if (c + 1 < n) id = page + my_page < page_end ? __ldg(table + page + my_page) : 0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = fill % kSlots;
            if (fill >= kSlots && !wait(kv_empty(slot), (fill / kSlots - 1) & 1)) break;
            if (lane == 0)
              mbar_arrive_expect_tx(kv_full(slot), (uint32_t)(np * p.block_size * 128 * NB));
            __syncwarp();
            if (my_page < np && my_half < NB)
              tma_load_2d(base_u32 + slot * L::kTile + my_half * kHalf + my_page * p.block_size * 128,
                          kv ? &tmap_v : &tmap_k, s.h * D + my_half * 64, row, kv_full(slot));
            ++fill;
          }
          if (failed) break;
        }
        }
        cc += n;
        // on to the next item
        at += item_cost(kind, n_item);
        if (at < r1 && ++tile >= tiles) {
          tile = 0;
          if (++h == p.Hkv) {
            h = 0;
            if (is_own) {
              shift();
            } else {
              while (++e < P && group_chunks(e) * tiles_of(e) == 0) {}
              if (e == P) prime(0);
            }
            if (e >= P && own.n == 0) {  // the first sequence from here on that has chunks
              int b = e - P;
              unsigned some;
              do {
                ++b;
                some = __ballot_sync(kFull, own_at(b + lane, len_at(b + lane)).n > 0);
                b += some ? __ffs(some) - 1 : 31;
              } while (!some && b + 1 < p.B);
              e = P + b;
              prime(b);
            }
          }
        }
      }
      // all loads are issued: the merge may start launching (from the start on, its blocks
      // would sit beside this one and wait: 115 us where 98 us are possible)
      if (lane == 0) griddep_launch_dependents();
      Seg end = {};
      if (!failed) publish(end);
      // no copy may be in flight when the CTA exits: wait for the last releases, or after a
      // failed wait for the copies themselves
      if (failed) {
        for (int i = max(0, fill - kSlots); i < fill; ++i) mbar_wait(kv_full(i % kSlots), (i / kSlots) & 1);
        for (int i = max(0, qfill - 2); i < qfill; ++i) mbar_wait(q_full(i & 1), (i >> 1) & 1);
        for (int i = max(0, qsmall - n_small); i < qsmall; ++i)
          mbar_wait(q_full(2 + i % n_small), (i / n_small) & 1);
      }
      for (int i = max(0, fill - kSlots); i < fill && !failed; ++i) wait(kv_empty(i % kSlots), (i / kSlots) & 1);
      for (int i = max(0, qfill - 2); i < qfill && !failed; ++i) wait(q_empty(i & 1), (i >> 1) & 1);
      for (int i = max(0, qsmall - n_small); i < qsmall && !failed; ++i)
        wait(q_empty(2 + i % n_small), (i / n_small) & 1);
    } else if (warp == kWarpMma) {
      // -------------------------------- MMAs --------------------------------
      // What the warp does between two MMAs the tensor pipe, whose queue is short, waits for.
      // So each kind of segment has a loop of its own with little in it, and everything that
      // ends up in an MMA's operands is the same for the whole warp in the compiler's eyes too
      // (uniform registers, no branch on the outcome of a wait): a thread's own descriptors
      // cost 650 cycles a step on their way to the tensor pipe. After a wait that ran out,
      // the rest is walked through without waiting.
      constexpr uint32_t idesc_qk = idesc_f16(kT, kT, !FP16, false, false);
      constexpr uint32_t idesc_pv = idesc_f16(kT, D, !FP16, false, true);
      constexpr uint32_t kTileU = L::kTile >> 4, kHalfTileU = kHalf / 2 >> 4;  // in descriptor units
      // descriptors of the ring's first slot and of the first Q tile
      const uint64_t k_desc = sdesc_sw128(base_u32, 16, 1024);
      const uint64_t v_desc = sdesc_sw128(base_u32, kHalf, 1024);
      const uint64_t q_desc = sdesc_sw128(base_u32 + L::kOffQ, 16, 1024);
      int slot = 0;             // ring slot of the next chunk's K
      uint32_t phase = 0;       // and its phase
      int qfill = 0;            // Q tiles used
      uint32_t p_phase = 0;     // phases of p_full, bit 2 t + h
      uint32_t o_used = 0, o_phase = 0;  // bit t: the pipe had a segment; phase of o_free
      int k = 0;                // segments
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!failed && !mbar_wait(bar, parity)) failed = true;
      };
      auto next_slot = [](int& sl, uint32_t& ph) {
        const int up = sl + 2 >= kSlots;
        sl += 2 - up * kSlots;
        ph ^= (uint32_t)up;
      };
      auto commit = [&](uint32_t bar) {
        if (elect_one()) mma_commit(bar);
      };
      // scores of a chunk
      auto qk = [&](int t, uint32_t q_off, int sl) {
        const uint64_t qa = q_desc + q_off, kb = k_desc + (uint32_t)(sl * kTileU);
        const uint32_t d = tS(t);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t o = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
            mma_f16_ss(d, qa + o, kb + o, idesc_qk, i > 0 ? 1u : 0u);
          }
          mma_commit(s_full(t));
        }
      };
      auto v_slot = [&](int sl) { return sl + 1 == kSlots ? 0 : sl + 1; };
      auto v_wait = [&](int sl, uint32_t ph) {
        wait(kv_full(v_slot(sl)), sl + 1 == kSlots ? ph ^ 1 : ph);
      };
      // Pipe t's output tile is free for another segment.
      auto o_wait = [&](int t) {
        if ((o_used >> t) & 1) {
          wait(o_free(t), (o_phase >> t) & 1);
          o_phase ^= 1u << t;
        }
        o_used |= 1u << t;
      };
      auto p_wait = [&](int t, int h) {
        const int x = 2 * t + h;
        wait(p_full(t, h), (p_phase >> x) & 1);
        p_phase ^= 1u << x;
      };
      auto p_test = [&](int t, int h) {  // p_wait if it would not wait
        const int x = 2 * t + h;
        if (!__all_sync(kFull, mbar_test(p_full(t, h), (p_phase >> x) & 1))) return false;
        p_phase ^= 1u << x;
        return true;
      };
      // steps x 16 tokens from half h on, both terms of the weights
      auto pv = [&](auto steps, int t, int h, int vs, bool start) {
        const uint64_t vb = v_desc + (uint32_t)(vs * kTileU + h * kHalfTileU);
        const uint32_t pa = tS(t) + h * (kT / 2), o = tO(t);
        if (elect_one()) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int j = 0; j < decltype(steps)::value; ++j)
              mma_f16_ts(o, pa + (j >> 1) * 32 + u * 16 + (j & 1) * 8, vb + (uint32_t)(j * 2048 >> 4), idesc_pv,
                         u == 0 && j == 0 && start ? 0u : 1u);
          }
          mma_commit(pv_done(t, h));
        }
      };
      using Half = std::integral_constant<int, kT / 32>;
      using Whole = std::integral_constant<int, kT / 16>;
      int n = 0, own = 0, par = 0;
      auto seg_int = [&](int e, int i) { return __shfl_sync(kFull, seg_ring[e * kSegInts + i], 0); };
      // shared segments, one after the other
      while (true) {
        const int e = k % kSegRing;
        wait(seg_full(e), (k / kSegRing) & 1);
        if (__any_sync(kFull, failed)) break;
        n = seg_int(e, 0), own = seg_int(e, 9), par = seg_int(e, 11);
        const int wide = seg_int(e, 1);
        if (n == 0 || own) break;
        if (lane == 0) mbar_arrive(seg_empty(e));
        __syncwarp();
        ++k;
        int pslot = slot;
        uint32_t pphase = phase;
        if (wide) {
          // pipe 0's chunk (PV of its halves, the next chunk's scores), then pipe 1's
          const int f0 = qfill & 1, f1 = f0 ^ 1;
          const uint32_t q0 = f0 * kTileU, q1 = f1 * kTileU;
          wait(q_full(f0), (qfill >> 1) & 1);
          wait(q_full(f1), ((qfill + 1) >> 1) & 1);
          qfill += 2;
          wait(kv_full(slot), phase);
          tc_fence_after();
          qk(0, q0, slot);
          qk(1, q1, slot);
          commit(kv_empty(slot));
          next_slot(slot, phase);
          o_wait(0);
          o_wait(1);
          v_wait(pslot, pphase);
          p_wait(0, 0);
          for (int i = 0; i < n; ++i) {
            const int vs = v_slot(pslot);
            const bool more = i + 1 < n;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              tc_fence_after();
              pv(Half{}, t, 0, vs, i == 0);
              p_wait(t, 1);
              tc_fence_after();
              pv(Half{}, t, 1, vs, false);
              // while the tensor pipe is at it: what the next step waits for
              bool got = true;
              if (t == 0 || more) got = p_test(t ^ 1, 0);
              if (more) {
                if (t == 0) {
                  wait(kv_full(slot), phase);
                  tc_fence_after();
                }
                qk(t, t ? q1 : q0, slot);
              }
              if (!got) p_wait(t ^ 1, 0);
            }
            if (more) {  // the next chunk's V
              int ns = pslot;
              uint32_t np = pphase;
              next_slot(ns, np);
              v_wait(ns, np);
            }
            commit(kv_empty(vs));
            next_slot(pslot, pphase);
            if (more) {
              commit(kv_empty(slot));
              next_slot(slot, phase);
            }
          }
          commit(q_empty(f0));
          commit(q_empty(f1));
        } else {
          // chunks take the pipes in turns, each in two halves; the next chunk's scores before
          // this one's PV if its K is there
          const int f = qfill & 1;
          const uint32_t q0 = f * kTileU;
          wait(q_full(f), (qfill >> 1) & 1);
          ++qfill;
          auto scores = [&](int t) {
            wait(kv_full(slot), phase);
            tc_fence_after();
            qk(t, q0, slot);
            commit(kv_empty(slot));
            next_slot(slot, phase);
          };
          scores(par);
          for (int i = 0; i < n; ++i) {
            const int t = (par + i) & 1, vs = v_slot(pslot);
            bool more = i + 1 < n;
            if (more && __all_sync(kFull, mbar_test(kv_full(slot), phase))) {
              scores(t ^ 1);
              more = false;
            }
            v_wait(pslot, pphase);
            if (i < 2) o_wait(t);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              p_wait(t, h);
              tc_fence_after();
              pv(Half{}, t, h, vs, i < 2 && h == 0);
            }
            commit(kv_empty(vs));
            next_slot(pslot, pphase);
            if (more) scores(t ^ 1);
          }
          commit(q_empty(f));
        }
      }
      // Own segments: whole chunks, the pipes in turns, scores up to two chunks ahead,
      // beyond the segment's end too (it may have one chunk only). Where the next segment
      // or its K is not there yet, PV goes first.
      if (own && !__any_sync(kFull, failed)) {
        int kp = k, qleft = 0, vleft = 0, vi = 0, place = -1, pending = 0, tq = par, tp = par;
        uint32_t place_phase = 0;
        int pslot = slot;
        uint32_t pphase = phase;
        bool end = false;
        auto ready = [&](uint32_t bar, uint32_t parity) {  // waits if there is nothing else to do
          if (pending > 0) return (bool)__all_sync(kFull, mbar_test(bar, parity));
          wait(bar, parity);
          return true;
        };
        while (true) {
          while (!end && pending < 2) {
            if (qleft == 0) {
              const int e = k % kSegRing;
              if (!ready(seg_full(e), (k / kSegRing) & 1) || __any_sync(kFull, failed)) break;
              qleft = seg_int(e, 0);
              ++k;
              end = qleft == 0;
              if (end) break;
              if (++place == n_small) place = 0, place_phase ^= 1;
              wait(q_full(2 + place), place_phase);
            }
            if (!ready(kv_full(slot), phase)) break;
            tc_fence_after();
            const int sl = __shfl_sync(kFull, slot, 0), t = __shfl_sync(kFull, tq, 0);
            const int at = __shfl_sync(kFull, place * small_rows * 128 >> 4, 0);
            qk(t, (uint32_t)at, sl);
            commit(kv_empty(sl));
            if (--qleft == 0) commit(q_empty(2 + place));
            next_slot(slot, phase);
            tq ^= 1;
            ++pending;
          }
          if (pending == 0 || __any_sync(kFull, failed)) break;
          if (vleft == 0) {
            const int e = kp % kSegRing;
            vleft = seg_int(e, 0);
            if (lane == 0) mbar_arrive(seg_empty(e));
            __syncwarp();
            ++kp;
            vi = 0;
          }
          v_wait(pslot, pphase);
          if (vi < 2) o_wait(tp);
          p_wait(tp, 0);
          tc_fence_after();
          const int vs = __shfl_sync(kFull, v_slot(pslot), 0), t = __shfl_sync(kFull, tp, 0);
          pv(Whole{}, t, 0, vs, vi < 2);
          commit(kv_empty(vs));
          next_slot(pslot, pphase);
          tp ^= 1;
          ++vi;
          --vleft;
          --pending;
        }
      }
      // no MMA or arrival may be in flight when the CTA exits, not after a failed wait either
      commit(drained);
      failed |= !mbar_wait(drained, 0);
      failed = __any_sync(kFull, failed);
    } else {
      // ------------------------------- softmax -------------------------------
      const int t = warp >> 2, wq = warp & 3;
      const int r = wq * 32 + lane;  // row of the tile, and token row that this thread clears
      const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
      const uint32_t s_addr = tS(t) + lane_base, o_addr = tO(t) + lane_base;
      constexpr int kDims4Log = D == 128 ? 5 : 4;
      constexpr float kGrow = FP16 ? 1.f : 8.f;     // log2 of the growth that is let pass
      constexpr float kShift = FP16 ? 14.f : -24.f;  // log2 of the weights' factor
      const int cap_rows = ws_cap(p);
      uint32_t s_phase[2] = {0, 0};  // of PV of the halves, and of S (as of its first half)
      auto wait = [&](uint32_t bar, uint32_t parity) {
        const bool ok = mbar_wait(bar, parity);
        if (!__all_sync(kFull, ok)) failed = true;
        return !failed;
      };
      int meets = 0;
      [[maybe_unused]] float slope = 0.f, far0 = 0.f;
      // products q . k of 32 tokens to scores in base-2 units, those outside [lo, hi) -inf
      auto scores = [&](float* x, float far, bool row_on, bool part, int lo, int hi) {
        if constexpr (MOD) {
          if (part) {  // what masked columns hold must not choose the way of the others
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (q < lo || q >= hi) x[q] = 0.f;
          }
          score_mods(p, x, slope, far, row_on);
        } else
#pragma unroll
          for (int q = 0; q < 32; ++q) x[q] *= p.qscale;
        if (part) {
#pragma unroll
          for (int q = 0; q < 32; ++q)
            if (q < lo || q >= hi) x[q] = -INFINITY;
        }
      };
      auto shift = [&](float m) {
        const float neg = (m == -INFINITY ? 0.f : -m) + kShift;
        return f32x2(neg, neg);
      };
      auto meet = [&]() {  // the pipe's four warps, with what they wrote to shared memory
        __syncwarp();
        if (lane == 0) mbar_arrive(joint(t));
        return wait(joint(t), meets++ & 1);
      };
      for (int k = 0; !failed; ++k) {
        Seg s;
        if (!wait(seg_full(k % kSegRing), (k / kSegRing) & 1)) break;
        seg_get(seg_ring + (k % kSegRing) * kSegInts, s);
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty(k % kSegRing));
        if (s.n == 0) break;
        const int n_rows = (s.wide ? (t ? s.n_seq - spt : spt) : s.n_seq) * G;
        // own segments: every warp has the G rows, and a quarter of each chunk's tokens
        const int ri = s.own ? lane : r;
        const bool row_ok = ri < n_rows, warp_ok = s.own || wq * 32 < n_rows;
        const int rs = seq_of(ri), b = s.b0 + (s.wide && t ? spt : 0) + rs, hq = s.h * G + ri - rs * G;
        float m = -INFINITY, l = 0.f;  // running maximum (base 2), sum of the weights
        if constexpr (MOD) {
          slope = far0 = 0.f;
          if (p.slopes != nullptr && row_ok) {
            slope = __ldg(p.slopes + hq) * kLog2e;
            far0 = (float)(s.t0 - (context_len(p, b) - 1));
          }
        }
        int done = 0;  // steps of this pipe in the segment
        // Follows the running maximum once the largest score has outgrown it.
        auto follow = [&](float top) {
          if (__any_sync(kFull, row_ok && top > m + kGrow)) {
            const float mn = fmaxf(m, top);
            const float alpha = m == mn ? 1.f : ex2_ftz(m - mn);
            m = mn;
            l *= alpha;
            if (done > 0) {  // O has to be complete: PV of the step before
              const int h = s.own ? 0 : (done - 1) & 1;
              if (!wait(pv_done(t, h), s_phase[h] ^ 1)) return;
              tc_fence_after();
#pragma unroll 1
              for (int j = 0; j < D / 32; ++j) {
                float o[32];
                tmem_ld32(o_addr + j * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 32; ++q) o[q] *= alpha;
                tmem_st32(o_addr + j * 32, o);
              }
            }
          }
        };
        for (int i = s.wide ? 0 : s.par ^ t; i < s.n && !failed; i += s.wide ? 1 : 2) {
          const int t0 = s.t0 + i * kT;
          const int lo = max(0, s.t_lo - t0), hi = min(kT, s.t_end - t0);  // valid tokens of the chunk
          const bool part = lo > 0 || hi < kT;
          const float far = far0 + (float)(i * kT);
#pragma unroll 1
          for (int h = 0; h < (s.own ? 1 : 2); ++h) {
            if (h == 0) {
              if (!wait(s_full(t), s_phase[0])) break;
              tc_fence_after();
            }
            if (s.own) {
              // All 128 columns at once, 32 of them here.
              const int j = wq * 32;
              float x[32];
              tmem_ld32(s_addr + j, x);
              tmem_ld_wait();
              scores(x, far + (float)j, row_ok, part, lo - j, hi - j);
              follow(max32(x));
              float sum0 = 0.f, sum1 = 0.f;
              weights<FP16>(s_addr + j, x, f32x2(1.f, 1.f), shift(m), sum0, sum1);
#pragma unroll
              for (int q = 0; q < 32; ++q) x[q] = 0.f;
#pragma unroll 1
              for (int c = 0; c < kT; c += 32)
                if (c != j) tmem_st32(s_addr + c, x);
              l += sum0 + sum1;
              tmem_st_wait();
            } else if (warp_ok) {
              // Half the columns. (All 128 in registers, with the code that this unrolls to,
              // left eight warps waiting for instructions.)
              const int j = h * (kT / 2);
              float x[64];
              tmem_ld32(s_addr + j, x);
              tmem_ld32(s_addr + j + 32, x + 32);
              tmem_ld_wait();
              float qs = p.qscale, top;
              if (MOD || part) {
                scores(x, far + (float)j, row_ok, part, lo - j, hi - j);
                scores(x + 32, far + (float)(j + 32), row_ok, part, lo - j - 32, hi - j - 32);
                qs = 1.f;
              } else if (qs < 0.f) {  // the largest scaled score is the least product's
#pragma unroll
                for (int q = 0; q < 64; ++q) x[q] = -x[q];
                qs = -qs;
              }
              top = fmaxf(max32(x), max32(x + 32)) * qs;
              follow(top);
              const uint64_t qs2 = f32x2(qs, qs), neg2 = shift(m);
              float sum0 = 0.f, sum1 = 0.f;
              weights<FP16>(s_addr + j, x, qs2, neg2, sum0, sum1);
              weights<FP16>(s_addr + j + 32, x + 32, qs2, neg2, sum0, sum1);
              l += sum0 + sum1;
              tmem_st_wait();
            }
            if (part && h == 0 && (!s.wide || t == 0)) {
              // V rows of masked tokens are zeros: 0 times whatever they hold would be no zero
              const int f = 2 * (s.cc + i) + 1, slot = f % kSlots;
              if (!wait(kv_full(slot), (f / kSlots) & 1)) break;
#pragma unroll
              for (int j = 0; j < NB; ++j) {
                uint4* v = reinterpret_cast<uint4*>(base + slot * L::kTile + j * kHalf);
                for (int q = r; q < lo * 8; q += kT) v[q] = make_uint4(0, 0, 0, 0);
                for (int q = hi * 8 + r; q < kT * 8; q += kT) v[q] = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(t, h));
            s_phase[h] ^= 1;
            ++done;
          }
        }
        if (failed) break;
        // the segment's partial of this row
        const int64_t out_row = (int64_t)b * p.Hq + hq;
        const int64_t w = s.first ? ws_first(p, s.own, out_row, s.wide ? 0 : t)
                                  : ws_next(p, blockIdx.x, cap_rows, t, r);
        if (done == 0) {
          if (row_ok && (!s.own || wq == 0)) p.ws_lse[w] = -INFINITY;
          continue;
        }
        {
          const int h = s.own ? 0 : 1;  // of the last step
          if (!wait(pv_done(t, h), s_phase[h] ^ 1)) break;
        }
        tc_fence_after();
        if (s.own) {
          // the four warps' parts, all dims at once (G <= 8) or half of them at a time
          const int heads = small_rows, dims4_log = G > 8 ? kDims4Log - 1 : kDims4Log;  // rows and float4s of a round
          const int dims4 = 1 << dims4_log;
          float4* part4 = reinterpret_cast<float4*>(base + L::kOffJoin + t * kJoinBytes);  // [4][heads][dims4]
          float2* ml = reinterpret_cast<float2*>(base + L::kOffMl) + t * 64;               // [4][16]
          if (row_ok) ml[wq * 16 + lane] = make_float2(m, l);
          const int64_t w0 = s.first ? ws_first(p, true, (int64_t)s.b0 * p.Hq + s.h * G, t)
                                     : ws_next(p, blockIdx.x, cap_rows, t, 0);
          const int w_step = s.first ? 2 : 1;  // workspace rows from one head's to the next one's
#pragma unroll 1
          for (int d0 = 0; d0 < D / 4; d0 += dims4) {
            if (d0 > 0 && !meet()) break;  // the round before is read
#pragma unroll 1
            for (int j = 0; j < dims4; j += 8) {
              float o[32];
              tmem_ld32(o_addr + (d0 + j) * 4, o);
              tmem_ld_wait();
              if (row_ok) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  part4[(wq * heads + lane) * dims4 + j + (q ^ (lane & 7))] =
                      make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
              }
            }
            if (!meet()) break;
            for (int i = r; i < G * dims4; i += kT) {
              const int g = i >> dims4_log, c = i & (dims4 - 1);
              float2 v[4];
              float M = -INFINITY, sum = 0.f;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[q] = ml[q * 16 + g];
                M = fmaxf(M, v[q].x);
              }
              float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                // the warp saw tokens (or only scores that are NaN, whose sum is NaN)
                if (v[q].x != -INFINITY || v[q].y != 0.f) {
                  const float f = ex2_ftz(v[q].x - M);
                  const float4 o = part4[(q * heads + g) * dims4 + (c ^ (g & 7))];
                  sum = fmaf(f, v[q].y, sum);
                  a.x = fmaf(f, o.x, a.x), a.y = fmaf(f, o.y, a.y);
                  a.z = fmaf(f, o.z, a.z), a.w = fmaf(f, o.w, a.w);
                }
              }
              const float inv = 1.f / sum;
              const int64_t at = w0 + (int64_t)g * w_step;
              *reinterpret_cast<float4*>(p.ws_o + at * D + (d0 + c) * 4) =
                  make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
              if (d0 + c == 0) p.ws_lse[at] = M - kShift + log2f(sum);
            }
          }
          if (failed) break;
          // (The next segment's parts are written once its O is complete, which takes all
          // four warps' weights and so comes after their reads here.)
        } else if (warp_ok) {
          const float inv = 1.f / l;
          float* dst = p.ws_o + w * D;
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            float o[32];
            tmem_ld32(o_addr + j * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] *= inv;
            if (row_ok) {
#pragma unroll
              for (int q = 0; q < 32; q += 8) store8(dst + j * 32 + q, o + q);
            }
          }
          if (row_ok) p.ws_lse[w] = m - kShift + log2f(l);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free(t));
      }
    }
  }
  if (failed && lane == 0 && atomicCAS(p.err, 0, kErrWaitTimeout) == 0) p.err[1] = blockIdx.x;
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace row
}  // namespace pda
