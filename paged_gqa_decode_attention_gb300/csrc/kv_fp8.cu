// The block-scaled FP8 cache: quantising K/V rows as they are written, with or
// without rotary positions, and reading them back. The decode kernels read the
// same cache (paged_decode_attn_run_block_scaled).
//
// A cache is [num_blocks, block_size, Hkv, D] of E4M3 values with one fp32
// scale per block and kv head, [num_blocks, Hkv]; a stored value y stands for
// s * y. For the values x of a block and head,
//   s = 2^e with the smallest e >= kMinScaleExp for which max |x| <= 448 * 2^e,
//   y = rn_e4m3(x / s)   (to nearest, ties to even).
// A power of two costs an E4M3 value no precision (its steps are relative) and
// makes x / s and s * y exact, so a stored value depends on nothing but the
// block's exponent, and raising the exponent of a block rounds only values
// that become subnormal.
//
// A block that a call appends to behind tokens it holds keeps
// s' = max(s, needed by the new rows); where s' > s its earlier values become
// rn_e4m3(y * s / s'). One warp (two or four where it has over 256 vectors) owns the
// tile of one (block, K or V, head): nothing is exchanged between blocks of
// threads, no atomics, the result does not depend on any order.
//
// Bound by memory traffic: a row costs 2 bytes read and 1 written per value. A
// tile's rows are held in registers between the maximum and the rounding (NV
// 16-byte vectors a lane, at most 8: with 16 only two CTAs fit an SM and their
// chains of loads did not overlap, 51 us against 40), so each is read once.
// Measured on GB300 (back to back, copy rate 6784.5 GB/s): 41984 fp16 rows of 8
// heads, D 128, blocks of 32: 39.9 us, 6460 GB/s; 256 single bf16 tokens 4.1 us.
// With rotation 21631 bf16 rows at 32/8 heads take 99.4 us, 4940 GB/s (adjacent
// pairs 97.8, half the dimensions rotated 94.5): each q row is one chain of load,
// rotation and store, at 24 warps an SM, whose latency (first stall: long scoreboard)
// the exact rounding's instructions (57% of the issue slots) do not hide; no row is read
// twice. Read-back of 24058 tokens to bf16 or fp16: 24.5 us, 6030 GB/s, to fp32
// 40.4 us, 6100 GB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <string>

#include "paged_decode_attn.h"
#include "pda_internal.h"
#include "ptx.cuh"
#include "rope_math.cuh"
#include "row_sets.h"

namespace pda {
namespace {

constexpr int kAppendWarps = 8;
constexpr int kAppendThreads = 32 * kAppendWarps;
constexpr int kQPairs = 4;  // vector pairs of a q row in flight per lane
constexpr int kMinScaleExp = -60;
constexpr unsigned kAll = 0xffffffffu;

struct AppendParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride, qo_stride;  // elements between rows
  const int32_t* positions;  // [T] (rope)
  const float* cos_sin;      // [max_position, rot_dim] (rope)
  uint16_t* q_out;
  uint8_t* k_cache;  // [num_blocks, block_size, Hkv, D]
  uint8_t* v_cache;
  float* k_scale;    // [num_blocks, Hkv]
  float* v_scale;
  const int32_t* table;  // [B, max_blocks]
  const int32_t* lens;   // [B], the new rows included
  const int64_t* cu;     // [B + 1]
  int* err;              // optional {code, detail}
  int64_t num_blocks;
  int64_t T;
  int B, Hq, Hkv, block_size, max_blocks, max_position, rot_dim;
  int groups;      // CTAs per unit: ceil(2 Hkv / tiles per CTA)
  int64_t kv_ctas; // units * groups; later CTAs rotate q rows
};

__device__ __forceinline__ void record(int* err, int code, int detail) {
  if (err != nullptr && atomicCAS(err, 0, code) == 0) err[1] = detail;
}

// Work units: sequence b's new rows cu[b] .. cu[b + 1] get the unit slots
// base(b) .. base(b + 1) - 1, base(b) = floor(cu[b] / block_size) + b. That is
// at least floor(n / block_size) + 1 slots for n rows, which touch at most
// floor((n - 2) / block_size) + 2 blocks (n >= 2), so slot j takes the j-th
// touched block and the last slot also the one after it. The unit count
// floor(T / block_size) + B needs no device value.
//
// unit_sequence: the sequence of unit u (b = -1: none), its rows and its length: a
// 32-way search for the last b with base(b) <= u, one round of loads per factor
// of 32 of the batch; the last round's lanes have loaded what is known of their
// sequences along with it. Where cu does not ascend it gives some sequence or none,
// and the caller checks that u is one of that sequence's slots: then u still stands
// for one block of one sequence, and no other unit for the same one.
// (A division by a block size that the compiler does not know would cost more
// than the rows.)
template <int BS>
__device__ __forceinline__ int64_t block_index(int64_t x) {
  static_assert((BS & (BS - 1)) == 0, "a power of two");
  return x >> (BS == 16 ? 4 : BS == 32 ? 5 : 6);
}

struct UnitSeq {
  int b, len;
  int64_t r_lo, r_hi;
};
template <int BS>
__device__ __forceinline__ UnitSeq unit_sequence(const AppendParams& p, int64_t u, int lane) {
  int lo = 0, n = p.B;
  UnitSeq r;
  while (true) {
    const int step = (n + 31) >> 5;
    const int i = lane * step;
    int64_t c0 = 0, c1 = 0;
    int len = 0;
    bool le = false;
    if (i < n) {
      c0 = __ldg(p.cu + lo + i);
      if (step == 1) {
        c1 = __ldg(p.cu + lo + i + 1);
        len = __ldg(p.lens + lo + i);
      }
      le = block_index<BS>(c0) + (lo + i) <= u;
    }
    const int cnt = __popc(__ballot_sync(kAll, le));
    r.b = cnt == 0 ? -1 : lo + (cnt - 1) * step;
    if (cnt == 0 || step == 1) {
      const int src = cnt == 0 ? 0 : cnt - 1;
      r.r_lo = __shfl_sync(kAll, c0, src);
      r.r_hi = __shfl_sync(kAll, c1, src);
      r.len = __shfl_sync(kAll, len, src);
      return r;
    }
    n = min(step, n - (cnt - 1) * step);
    lo = r.b;
  }
}

// Rotates the pair of vectors (A, B) that hold both elements of 8 rotated pairs:
// c and s are their cosines and sines. Halves: pair i is (element i of A, element
// i of B); adjacent pairs: the two halves of word i of A, then of B.
template <typename F, bool kHalves>
__device__ __forceinline__ void rotate_pair(uint4& A, uint4& B, const float (&c)[8],
                                            const float (&s)[8]) {
  uint32_t* a = &A.x;
  uint32_t* b = &B.x;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (kHalves) {
      const float a0 = F::lo_f(a[w]), a1 = F::hi_f(a[w]), b0 = F::lo_f(b[w]), b1 = F::hi_f(b[w]);
      a[w] = rounded_dot2_x2<F, true>(a0, c[2 * w], -b0, s[2 * w], a1, c[2 * w + 1], -b1, s[2 * w + 1]);
      b[w] = rounded_dot2_x2<F, true>(b0, c[2 * w], a0, s[2 * w], b1, c[2 * w + 1], a1, s[2 * w + 1]);
    } else {
      float x = F::lo_f(a[w]), y = F::hi_f(a[w]);
      a[w] = rounded_dot2_x2<F, true>(x, c[w], -y, s[w], y, c[w], x, s[w]);
      x = F::lo_f(b[w]);
      y = F::hi_f(b[w]);
      b[w] = rounded_dot2_x2<F, true>(x, c[4 + w], -y, s[4 + w], y, c[4 + w], x, s[4 + w]);
    }
  }
}

// 8 cosines and sines from angle 8u on of a table row (rot / 2 cosines, then sines).
__device__ __forceinline__ void load_angles(const float* cs, int u, int half, float (&c)[8],
                                            float (&s)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(cs + 8 * u) + k);
    const float4 y = __ldg(reinterpret_cast<const float4*>(cs + half + 8 * u) + k);
    c[4 * k] = x.x;
    c[4 * k + 1] = x.y;
    c[4 * k + 2] = x.z;
    c[4 * k + 3] = x.w;
    s[4 * k] = y.x;
    s[4 * k + 1] = y.y;
    s[4 * k + 2] = y.z;
    s[4 * k + 3] = y.w;
  }
}

template <typename F>
struct Inf16;
template <>
struct Inf16<Bf16> {
  static constexpr uint32_t bits = 0x7f80u;
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b << 16); }
};
template <>
struct Inf16<Fp16> {
  static constexpr uint32_t bits = 0x7c00u;
  static __device__ __forceinline__ float value(uint32_t b) {
    return __half2float(__ushort_as_half((unsigned short)b));
  }
};

// Largest |x| of a 16-bit pair pattern, as a pattern; non-finite ones count 0.
__device__ __forceinline__ uint32_t finite_max(uint32_t w, uint32_t inf) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  return max(lo < inf ? lo : 0u, hi < inf ? hi : 0u);
}

// 2^e as above for a largest magnitude a (448 = 1.75 * 2^8).
__device__ __forceinline__ float block_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, kMinScaleExp);  // also zeros and subnormals
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ bool is_power_of_two(float s) {  // a normal one
  return (__float_as_uint(s) & 0x7fffffu) == 0;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Four E4M3 bytes times f (requantisation, read-back).
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float (&x)[4]) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 fa = __half22float2(__half2(a)), fb = __half22float2(__half2(b));
  x[0] = fa.x;
  x[1] = fa.y;
  x[2] = fb.x;
  x[3] = fb.y;
}

// One vector of 8 16-bit elements over the scale s, as 8 E4M3 bytes. E4M3 has
// no infinity: a non-finite element is stored as NaN.
template <typename F>
__device__ __forceinline__ uint2 quantise_any(uint4 x, float s) {
  auto q = [&](float a) { return isinf(a) ? __uint_as_float(0x7fc00000u) : __fdiv_rn(a, s); };
  uint2 y;
  y.x = e4m3x4(q(F::lo_f(x.x)), q(F::hi_f(x.x)), q(F::lo_f(x.y)), q(F::hi_f(x.y)));
  y.y = e4m3x4(q(F::lo_f(x.z)), q(F::hi_f(x.z)), q(F::lo_f(x.w)), q(F::hi_f(x.w)));
  return y;
}

// The same for finite elements and a power of two s whose reciprocal fits the
// 16-bit type (twice, for fp16: inv is its square root or near it), in 16-bit
// arithmetic. A product is exact except among the type's subnormals, and there it
// is nowhere near the E4M3 rounding borders (multiples of 2^-10; an fp16 product
// between 2^-11 and 2^-9 has its last bit at 2^-21 or above).
__device__ __forceinline__ uint2 quantise_pow2(uint4 x, uint32_t inv_a, uint32_t, Bf16) {
  const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162*>(&inv_a);
  auto q = [&](uint32_t w) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), f);
    return *reinterpret_cast<const uint32_t*>(&y);
  };
  const uint32_t a = q(x.x), b = q(x.y), c = q(x.z), d = q(x.w);
  return make_uint2(e4m3x4(Bf16::lo_f(a), Bf16::hi_f(a), Bf16::lo_f(b), Bf16::hi_f(b)),
                    e4m3x4(Bf16::lo_f(c), Bf16::hi_f(c), Bf16::lo_f(d), Bf16::hi_f(d)));
}
__device__ __forceinline__ uint2 quantise_pow2(uint4 x, uint32_t inv_a, uint32_t inv_b, Fp16) {
  const __half2 f = *reinterpret_cast<const __half2*>(&inv_a);
  const __half2 g = *reinterpret_cast<const __half2*>(&inv_b);
  auto q = [&](uint32_t w) {
    const __half2 y = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&w), f), g);
    return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(__half2_raw(y), __NV_SATFINITE, __NV_E4M3);
  };
  return make_uint2(q(x.x) | (q(x.y) << 16), q(x.z) | (q(x.w) << 16));
}

// Whether 1 / 2^e can be applied so, and the factors (pairs of the 16-bit type).
__device__ __forceinline__ bool pow2_factors(int e, uint32_t& a, uint32_t& b, Bf16) {
  a = (uint32_t)(127 - e) << 7;  // |e| <= 120
  a |= a << 16;
  b = 0;
  return e >= -120 && e <= 120;
}
__device__ __forceinline__ bool pow2_factors(int e, uint32_t& a, uint32_t& b, Fp16) {
  const int ea = -e / 2, eb = -e - ea;
  a = (uint32_t)(15 + ea) << 10;
  b = (uint32_t)(15 + eb) << 10;
  a |= a << 16;
  b |= b << 16;
  return e >= -28 && e <= 28;
}

enum Rope { kRopeNone = 0, kRopeHalves = 1, kRopePairs = 2 };

// CTAs below p.kv_ctas: a unit's tiles, W warps per tile; the others (rope):
// one q row per warp.
template <typename F, int D, int NV, int W, int kRope>
__global__ void __launch_bounds__(kAppendThreads, kRope == kRopeNone ? 4 : 3)
    append_kernel(const AppendParams p) {
  griddep_launch_dependents();  // the next grid may be set up; it waits for this one's end
  griddep_wait();
  // A lane's two vectors of a row are the A and B of one rotation item (8 pairs), or
  // any two where nothing rotates; kItems lanes cover a row.
  constexpr int kItems = D / 16;
  constexpr int BS = NV * W * 256 / D;  // block size
  constexpr int kRowsPerStep = 32 / kItems;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u16 = lane & (kItems - 1), sub = lane / kItems;
  const int half = p.rot_dim >> 1;
  const bool rotates = kRope != kRopeNone && 16 * u16 < p.rot_dim;
  int colA = 8 * u16, colB = 8 * u16 + D / 2;
  if constexpr (kRope == kRopeHalves) {
    colA = rotates ? 8 * u16 : 16 * u16;
    colB = rotates ? 8 * u16 + half : 16 * u16 + 8;
  } else if constexpr (kRope == kRopePairs) {
    colA = 16 * u16;
    colB = 16 * u16 + 8;
  }

  if (kRope != kRopeNone && blockIdx.x >= p.kv_ctas) {
    const int64_t r = ((int64_t)blockIdx.x - p.kv_ctas) * kAppendWarps + warp;
    const int64_t r_lo = __ldg(p.cu), r_hi = __ldg(p.cu + p.B);
    if (r < r_lo || r >= r_hi || r >= p.T) return;
    const int pos = __ldg(p.positions + r);
    if (pos < 0 || pos >= p.max_position) {
      if (lane == 0) record(p.err, kErrPosition, (int)r);
      return;
    }
    float c[8], s[8];
    if (rotates) load_angles(p.cos_sin + (int64_t)pos * p.rot_dim, u16, half, c, s);
    const uint16_t* src = p.q + r * p.q_stride;
    uint16_t* dst = p.q_out + r * p.qo_stride;
    for (int h0 = 0; h0 < p.Hq; h0 += kQPairs * kRowsPerStep) {
      uint4 A[kQPairs], B[kQPairs];
#pragma unroll
      for (int i = 0; i < kQPairs; ++i) {
        const int h = h0 + i * kRowsPerStep + sub;
        if (h < p.Hq) {
          A[i] = *reinterpret_cast<const uint4*>(src + h * D + colA);
          B[i] = *reinterpret_cast<const uint4*>(src + h * D + colB);
        }
      }
#pragma unroll
      for (int i = 0; i < kQPairs; ++i) {
        const int h = h0 + i * kRowsPerStep + sub;
        if (h < p.Hq) {
          if (rotates) rotate_pair<F, kRope == kRopeHalves>(A[i], B[i], c, s);
          *reinterpret_cast<uint4*>(dst + h * D + colA) = A[i];
          *reinterpret_cast<uint4*>(dst + h * D + colB) = B[i];
        }
      }
    }
    return;
  }

  __shared__ uint32_t s_max[kAppendWarps];
  const int u = (int)blockIdx.x / p.groups, grp = (int)blockIdx.x - u * p.groups;
  // Unit u also reports sequence u's rows where they descend or leave the input: the
  // search need not find such a sequence. (Requested before the search, so that
  // nothing waits for them; there are at least B units.)
  const bool reports = grp == 0 && threadIdx.x == 0 && u < p.B && p.err != nullptr;
  int64_t own_lo = 0, own_hi = 0;
  if (reports) {
    own_lo = __ldg(p.cu + u);
    own_hi = __ldg(p.cu + u + 1);
  }
  const UnitSeq seq = unit_sequence<BS>(p, u, lane);
  if (reports && (own_lo < 0 || own_hi < own_lo || own_hi > p.T)) record(p.err, kErrContextLen, u);
  const int b = seq.b, len = seq.len;
  if (b < 0) return;
  const int64_t r_lo = seq.r_lo, r_hi = seq.r_hi, n = r_hi - r_lo;
  constexpr int bs = BS;
  const int64_t base = block_index<BS>(r_lo) + b, slots = block_index<BS>(r_hi) + b + 1 - base;
  const int64_t j = u - base;
  if (n <= 0 || j < 0 || j >= slots || r_lo < 0 || r_hi > p.T) return;  // (reported above)
  if (n > len || len > INT_MAX - bs ||
      (int64_t)len > (int64_t)p.max_blocks * bs) {
    if (threadIdx.x == 0) record(p.err, kErrContextLen, b);
    return;
  }
  const int start = len - (int)n;
  const int last_page = (int)((unsigned)(len - 1) / bs);
  const int tile = grp * (kAppendWarps / W) + warp / W;
  const int wsub = warp % W;
  const bool has_tile = tile < 2 * p.Hkv;
  const bool is_v = tile >= p.Hkv;
  const int h = is_v ? tile - p.Hkv : tile;
  const uint16_t* x_rows = is_v ? p.v : p.k;
  const int64_t x_stride = is_v ? p.v_stride : p.k_stride;
  uint8_t* cache = is_v ? p.v_cache : p.k_cache;
  float* scales = is_v ? p.v_scale : p.k_scale;

  for (int page = (int)((unsigned)start / bs) + (int)j; page <= last_page; ++page) {
    const int t_lo = max(start, page * bs), t_hi = min(len, (page + 1) * bs);
    const int off = t_lo - page * bs, nr = t_hi - t_lo;
    const int64_t row0 = r_lo + (t_lo - start);
    // the rows and the block id are requested together
    const int blk = __ldg(p.table + (int64_t)b * p.max_blocks + page);
    uint4 x[NV];        // NV / 2 rows' A and B
    bool live[NV / 2];  // the row is written
    auto row_of = [&](int i) { return (i * W + wsub) * kRowsPerStep + sub; };
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) {
      live[i] = has_tile && row_of(i) < nr;
      x[2 * i] = x[2 * i + 1] = make_uint4(0, 0, 0, 0);
      if (live[i]) {
        const uint16_t* src = x_rows + (row0 + row_of(i)) * x_stride + h * D;
        x[2 * i] = __ldg(reinterpret_cast<const uint4*>(src + colA));
        x[2 * i + 1] = __ldg(reinterpret_cast<const uint4*>(src + colB));
      }
    }
    const bool blk_ok = blk >= 0 && blk < p.num_blocks;
    if (!blk_ok && threadIdx.x == 0) record(p.err, kErrBlockId, b);
    const bool active = has_tile && blk_ok;
    const int64_t sidx = (int64_t)(blk_ok ? blk : 0) * p.Hkv + (has_tile ? h : 0);
    float old = 0.f;
    if (active && off > 0) old = scales[sidx];
    if constexpr (kRope != kRopeNone) {
      int pos[NV / 2];
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) pos[i] = live[i] ? __ldg(p.positions + row0 + row_of(i)) : 0;
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        if (live[i]) {
          if (pos[i] < 0 || pos[i] >= p.max_position) {  // writes nothing (q's CTA reports it)
            live[i] = false;
            x[2 * i] = x[2 * i + 1] = make_uint4(0, 0, 0, 0);
          } else if (rotates && !is_v) {
            float c[8], s[8];
            load_angles(p.cos_sin + (int64_t)pos[i] * p.rot_dim, u16, half, c, s);
            rotate_pair<F, kRope == kRopeHalves>(x[2 * i], x[2 * i + 1], c, s);
          }
        }
      }
    }
    // largest magnitude of the tile
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                 __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
    }
    uint32_t m = __reduce_max_sync(kAll, max(m2 & 0xffffu, m2 >> 16));
    const bool nonfinite = m >= Inf16<F>::bits;  // warp-uniform, rare
    if (nonfinite) {
      m = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        m = max(m, max(max(finite_max(x[i].x, Inf16<F>::bits), finite_max(x[i].y, Inf16<F>::bits)),
                       max(finite_max(x[i].z, Inf16<F>::bits), finite_max(x[i].w, Inf16<F>::bits))));
      m = __reduce_max_sync(kAll, m);
    }
    if constexpr (W > 1) {
      if (lane == 0) s_max[warp] = m;
      __syncthreads();  // also: every warp of the tile has read the old scale
#pragma unroll
      for (int w = 0; w < W; ++w) m = max(m, s_max[warp - wsub + w]);
      __syncthreads();
    }
    if (active) {
      if (!(old > 0.f && old <= 3.402823466e38f)) old = 0.f;
      const float s = fmaxf(old, block_scale(Inf16<F>::value(m)));
      uint8_t* tile_base = cache + ((int64_t)blk * bs * p.Hkv + h) * D;
      const int64_t row_bytes = (int64_t)p.Hkv * D;
      if (off > 0 && s > old) {
        // the block's earlier values, 16 bytes a lane
        constexpr int kV16 = D / 16;
        const float f = __fdiv_rn(old, s);
        for (int i = wsub * 32 + lane; i < off * kV16; i += 32 * W) {
          uint4* a = reinterpret_cast<uint4*>(tile_base + (i / kV16) * row_bytes + (i % kV16) * 16);
          uint4 w = *a;
          uint32_t* ww = &w.x;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            float y[4];
            e4m3x4_to_float(ww[t], y);
            ww[t] = e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
          }
          *a = w;
        }
      }
      if (wsub == 0 && lane == 0) scales[sidx] = s;
      uint32_t fa, fb;
      const bool quick = pow2_factors((int)(__float_as_uint(s) >> 23) - 127, fa, fb, F()) &&
                         is_power_of_two(s) && !nonfinite;
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        if (live[i]) {
          uint8_t* dst = tile_base + (off + row_of(i)) * row_bytes;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint2 y;
            if (quick) y = quantise_pow2(x[2 * i + k], fa, fb, F());
            else y = quantise_any<F>(x[2 * i + k], s);
            *reinterpret_cast<uint2*>(dst + (k == 0 ? colA : colB)) = y;
          }
        }
      }
    }
    if (j != slots - 1) break;  // only a sequence's last slot goes on to the next block
  }
}

// --------------------------------- read-back ---------------------------------

template <typename T>
struct Pack;  // four fp32 values of a 16-byte store, or eight of a 16-bit one
template <>
struct Pack<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <typename F>
struct Pack16 {
  static constexpr int n = 8;
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(F::pack2(x[0], x[1]), F::pack2(x[2], x[3]), F::pack2(x[4], x[5]),
                      F::pack2(x[6], x[7]));
  }
};
template <>
struct Pack<Bf16> : Pack16<Bf16> {};
template <>
struct Pack<Fp16> : Pack16<Fp16> {};

struct GatherParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* lens;
  const int64_t* cu_rows;
  uint4* k_out;
  uint4* v_out;
  int* err;
  int64_t num_blocks, out_rows;
  int block_size, max_blocks, max_len, Hkv;
  uint32_t div_mul;  // ceil(2^32 / Hkv); 0 for Hkv = 1
};

constexpr int kGatherThreads = 256;
constexpr int kGatherVec = 4;  // vectors in flight per thread

// grid (pages, sequences, 2): one block's tokens of K (z = 0) or V. A block's
// rows are contiguous in the cache and in the output. x / Hkv is a multiplication
// (p.div_mul, exact for the x = token * Hkv + head of a block: ceil(2^32 / Hkv) * x
// is below the next multiple of 2^32 while x * Hkv < 2^32).
template <typename T, int D>
__global__ void __launch_bounds__(kGatherThreads) gather_fp8_kernel(const GatherParams p) {
  constexpr int E = Pack<T>::n;  // elements of an output vector
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.y, page = blockIdx.x;
  int L = __ldg(p.lens + b);
  if (L > p.max_len || L < 0) {
    if (page == 0 && blockIdx.z == 0 && threadIdx.x == 0) record(p.err, kErrContextLen, b);
    L = L < 0 ? 0 : p.max_len;
  }
  const int t0 = page * p.block_size;
  if (t0 >= L) return;
  const int nr = min(p.block_size, L - t0);
  const int blk = __ldg(p.table + (int64_t)b * p.max_blocks + page);
  const int64_t row0 = __ldg(p.cu_rows + b) + t0;
  if (blk < 0 || blk >= p.num_blocks || row0 < 0 || row0 + nr > p.out_rows) {
    if (threadIdx.x == 0) record(p.err, kErrBlockId, b);
    return;
  }
  const bool is_v = blockIdx.z != 0;
  const int64_t row_elems = (int64_t)p.Hkv * D;
  const uint8_t* src = (is_v ? p.v : p.k) + (int64_t)blk * p.block_size * row_elems;
  uint4* dst = (is_v ? p.v_out : p.k_out) + row0 * row_elems / E;
  const float* sc = (is_v ? p.v_scale : p.k_scale) + (int64_t)blk * p.Hkv;
  const int n = nr * (int)row_elems / E;
  constexpr int per_head = D / E;
  for (int i0 = threadIdx.x; i0 < n; i0 += kGatherThreads * kGatherVec) {
    uint2 w[kGatherVec];
    float s[kGatherVec];
#pragma unroll
    for (int t = 0; t < kGatherVec; ++t) {
      const int i = i0 + t * kGatherThreads;
      if (i < n) {
        if constexpr (E == 8) w[t] = __ldg(reinterpret_cast<const uint2*>(src) + i);
        else w[t].x = __ldg(reinterpret_cast<const uint32_t*>(src) + i);
        const uint32_t row_head = (uint32_t)i / per_head;
        const uint32_t row = p.Hkv == 1 ? row_head : __umulhi(row_head, p.div_mul);
        s[t] = __ldg(sc + (row_head - row * (uint32_t)p.Hkv));
      }
    }
#pragma unroll
    for (int t = 0; t < kGatherVec; ++t) {
      const int i = i0 + t * kGatherThreads;
      if (i < n) {
        float x[8];
        float y[4];
        e4m3x4_to_float(w[t].x, y);
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = y[q] * s[t];
        if constexpr (E == 8) {
          e4m3x4_to_float(w[t].y, y);
#pragma unroll
          for (int q = 0; q < 4; ++q) x[4 + q] = y[q] * s[t];
        }
        dst[i] = Pack<T>::pack(x);
      }
    }
  }
}

// ----------------------------------- host -----------------------------------

int fail(int code, const std::string& msg) { return set_last_error(code, msg.c_str()); }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Selects `device` for the scope and restores the caller's.
struct Dev {
  int prev = -1;
  cudaError_t err = cudaSuccess;
  explicit Dev(int d) {
    err = cudaGetDevice(&prev);
    if (err == cudaSuccess && prev != d) err = cudaSetDevice(d);
    else prev = -1;
  }
  ~Dev() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

int launched(const char* what, cudaError_t e) {
  if (e != cudaSuccess) return fail(PDA_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
  return PDA_OK;
}

Rows span(const void* p, int64_t bytes) {
  return Rows{(int64_t)reinterpret_cast<uintptr_t>(p), bytes, p ? bytes : 0, 1};
}

// Geometry that the FP8 decode kernels read.
int check_cache(int num_kv_heads, int head_dim, int block_size, int64_t num_blocks) {
  if (num_kv_heads < 1 || num_kv_heads > 65535)
    return fail(PDA_EINVAL, "num_kv_heads must be in [1, 65535]");
  if (head_dim < 1 || block_size < 1) return fail(PDA_EINVAL, "head_dim and block_size must be positive");
  if (head_dim != 64 && head_dim != 128) return fail(PDA_EUNSUPPORTED, "head_dim must be 64 or 128");
  if (block_size != 16 && block_size != 32 && block_size != 64)
    return fail(PDA_EUNSUPPORTED, "block_size must be 16, 32 or 64");
  if (num_blocks < 1 || num_blocks > INT_MAX / block_size)
    return fail(PDA_EINVAL, "num_blocks * block_size must be in [1, 2^31)");
  return PDA_OK;
}

// Launches with programmatic dependent launch, as the decode kernels: set-up overlaps
// the end of the previous grid in the stream (off with PDA_PDL=0).
template <typename P>
cudaError_t launch(void (*kernel)(const P), dim3 grid, int threads, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename F, int D, int NV, int W>
cudaError_t launch_append(const AppendParams& p, int rope, unsigned grid, cudaStream_t s) {
  return launch(rope == kRopeNone     ? append_kernel<F, D, NV, W, kRopeNone>
                : rope == kRopeHalves ? append_kernel<F, D, NV, W, kRopeHalves>
                                      : append_kernel<F, D, NV, W, kRopePairs>,
                dim3(grid), kAppendThreads, s, p);
}

template <typename F>
cudaError_t launch_append_geometry(const AppendParams& p, int D, int rope, unsigned grid,
                                   cudaStream_t s) {
  // NV * W * 32 = block_size * D / 8 vectors of a tile: at most 8 a lane, so that
  // four CTAs fit an SM and their chains of loads overlap
  const int tile = p.block_size * D;
  if (D == 64) {
    if (tile == 1024) return launch_append<F, 64, 4, 1>(p, rope, grid, s);
    if (tile == 2048) return launch_append<F, 64, 8, 1>(p, rope, grid, s);
    return launch_append<F, 64, 8, 2>(p, rope, grid, s);
  }
  if (tile == 2048) return launch_append<F, 128, 8, 1>(p, rope, grid, s);
  if (tile == 4096) return launch_append<F, 128, 8, 2>(p, rope, grid, s);
  return launch_append<F, 128, 8, 4>(p, rope, grid, s);
}

// Both append entry points; rope == kRopeNone: no q, no positions.
int append_impl(AppendParams p, int D, int dtype, int rope, int device, void* stream) {
  if (p.B < 0 || p.T < 0 || p.T > INT_MAX || p.max_blocks < 0 || device < 0)
    return fail(PDA_EINVAL, "negative size or device, or num_rows >= 2^31");
  if (dtype != PDA_BF16 && dtype != PDA_FP16) return fail(PDA_EINVAL, "dtype must be bf16 or fp16");
  const int st = check_cache(p.Hkv, D, p.block_size, p.num_blocks);
  if (st != PDA_OK) return st;
  const int64_t hkv_d = (int64_t)p.Hkv * D, hq_d = (int64_t)p.Hq * D;
  if (p.k_stride == 0) p.k_stride = hkv_d;
  if (p.v_stride == 0) p.v_stride = hkv_d;
  if (p.k_stride < hkv_d || p.v_stride < hkv_d)
    return fail(PDA_EINVAL, "a token stride is smaller than its row of heads");
  if ((p.k_stride | p.v_stride) % 8 != 0)
    return fail(PDA_EINVAL, "token strides must be multiples of 8 elements (16 bytes)");
  if (rope != kRopeNone) {
    if (p.Hq < 1 || p.Hq > 65535) return fail(PDA_EINVAL, "num_q_heads must be in [1, 65535]");
    if (p.rot_dim < 0 || p.rot_dim > D || p.rot_dim % 16 != 0)
      return fail(PDA_EINVAL, "rot_dim must be a multiple of 16 in [0, head_dim]");
    if (p.max_position < 0) return fail(PDA_EINVAL, "max_position < 0");
    if (p.q_stride == 0) p.q_stride = hq_d;
    if (p.qo_stride == 0) p.qo_stride = hq_d;
    if (p.q_stride < hq_d || p.qo_stride < hq_d)
      return fail(PDA_EINVAL, "a token stride is smaller than its row of heads");
    if ((p.q_stride | p.qo_stride) % 8 != 0)
      return fail(PDA_EINVAL, "token strides must be multiples of 8 elements (16 bytes)");
  }
  if (p.B == 0 || p.T == 0) return PDA_OK;
  if (p.max_blocks < 1) return fail(PDA_EINVAL, "max_blocks < 1");
  if (!p.k || !p.v || !p.k_cache || !p.v_cache || !p.k_scale || !p.v_scale || !p.table || !p.lens ||
      !p.cu || (rope != kRopeNone && (!p.q || !p.q_out || !p.positions || (p.rot_dim > 0 && !p.cos_sin))))
    return fail(PDA_EINVAL, "a required pointer is NULL");
  if (!aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.k_cache, 16) || !aligned(p.v_cache, 16) ||
      !aligned(p.q, 16) || !aligned(p.q_out, 16) || !aligned(p.cos_sin, 16))
    return fail(PDA_EINVAL, "rows, caches and the cos/sin table must be 16-byte aligned");
  if (!aligned(p.k_scale, 4) || !aligned(p.v_scale, 4) || !aligned(p.table, 4) ||
      !aligned(p.lens, 4) || !aligned(p.cu, 8) || !aligned(p.positions, 4) || !aligned(p.err, 4))
    return fail(PDA_EINVAL, "misaligned scales or index arrays");
  auto rows = [&](const void* x, int64_t stride, int64_t len) {
    return Rows{(int64_t)reinterpret_cast<uintptr_t>(x), stride * 2, x ? len * 2 : 0, p.T};
  };
  const int64_t cache_bytes = p.num_blocks * p.block_size * hkv_d;
  const int64_t scale_bytes = p.num_blocks * p.Hkv * 4;
  const Rows outs[6] = {span(p.k_cache, cache_bytes), span(p.v_cache, cache_bytes),
                        span(p.k_scale, scale_bytes), span(p.v_scale, scale_bytes),
                        span(p.err, 8), rows(p.q_out, p.qo_stride, hq_d)};
  const Rows ins[7] = {rows(p.k, p.k_stride, hkv_d), rows(p.v, p.v_stride, hkv_d),
                       span(p.table, (int64_t)p.B * p.max_blocks * 4), span(p.lens, p.B * 4ll),
                       span(p.cu, (p.B + 1) * 8ll), span(p.positions, p.T * 4),
                       span(p.cos_sin, (int64_t)p.max_position * p.rot_dim * 4)};
  const Rows rq = rows(p.q, p.q_stride, hq_d);
  for (int o = 0; o < 6; ++o) {
    for (const Rows& in : ins)
      if (overlaps(outs[o], in)) return fail(PDA_EALIAS, "an output overlaps an input");
    for (int j = o + 1; j < 6; ++j)
      if (overlaps(outs[o], outs[j])) return fail(PDA_EALIAS, "two outputs overlap");
    if (o < 5 && overlaps(outs[o], rq)) return fail(PDA_EALIAS, "an output overlaps q");
  }
  const bool q_in_place = p.q == p.q_out && p.q_stride == p.qo_stride;
  if (rope != kRopeNone && !q_in_place && overlaps(outs[5], rq))
    return fail(PDA_EALIAS, "q_out overlaps q (only the exact in-place form is allowed)");

  const int W = std::max(1, p.block_size * D / 2048);  // warps per tile
  const int tiles = kAppendWarps / W;
  p.groups = (2 * p.Hkv + tiles - 1) / tiles;
  p.kv_ctas = (p.T / p.block_size + p.B) * p.groups;
  const int64_t grid = p.kv_ctas + (rope != kRopeNone ? (p.T + kAppendWarps - 1) / kAppendWarps : 0);
  if (grid > INT_MAX) return fail(PDA_EINVAL, "too many rows for one launch");
  Dev guard(device);
  if (guard.err != cudaSuccess) return fail(PDA_ECUDA, "cudaSetDevice failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched("append launch",
                  dtype == PDA_BF16 ? launch_append_geometry<Bf16>(p, D, rope, (unsigned)grid, s)
                                    : launch_append_geometry<Fp16>(p, D, rope, (unsigned)grid, s));
}

}  // namespace
}  // namespace pda

using pda::fail;

extern "C" int paged_decode_attn_append_kv_fp8(
    const void* k, int64_t k_token_stride, const void* v, int64_t v_token_stride, int64_t num_rows,
    int num_kv_heads, int head_dim, int dtype, void* k_cache, void* v_cache, float* k_scale,
    float* v_scale, int64_t num_blocks, int block_size, const int32_t* block_table, int max_blocks,
    const int32_t* context_lens, const int64_t* cu_rows, int batch, int* err, int device,
    void* stream) {
  pda::AppendParams p = {};
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.k_stride = k_token_stride;
  p.v_stride = v_token_stride;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = block_table;
  p.lens = context_lens;
  p.cu = cu_rows;
  p.err = err;
  p.num_blocks = num_blocks;
  p.T = num_rows;
  p.B = batch;
  p.Hkv = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  return pda::append_impl(p, head_dim, dtype, pda::kRopeNone, device, stream);
}

extern "C" int paged_decode_attn_rope_append_kv_fp8(
    const void* q, int64_t q_token_stride, const void* k, int64_t k_token_stride, const void* v,
    int64_t v_token_stride, const int32_t* positions, const float* cos_sin_cache,
    int max_position, int rot_dim, int neox_style, int64_t num_rows, int num_q_heads,
    int num_kv_heads, int head_dim, int dtype, void* q_out, int64_t q_out_token_stride,
    void* k_cache, void* v_cache, float* k_scale, float* v_scale, int64_t num_blocks,
    int block_size, const int32_t* block_table, int max_blocks, const int32_t* context_lens,
    const int64_t* cu_rows, int batch, int* err, int device, void* stream) {
  pda::AppendParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_token_stride;
  p.k_stride = k_token_stride;
  p.v_stride = v_token_stride;
  p.qo_stride = q_out_token_stride;
  p.positions = positions;
  p.cos_sin = cos_sin_cache;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = block_table;
  p.lens = context_lens;
  p.cu = cu_rows;
  p.err = err;
  p.num_blocks = num_blocks;
  p.T = num_rows;
  p.B = batch;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.max_position = max_position;
  p.rot_dim = rot_dim;
  return pda::append_impl(p, head_dim, dtype, neox_style ? pda::kRopeHalves : pda::kRopePairs,
                          device, stream);
}

extern "C" int paged_decode_attn_gather_kv_fp8(
    const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
    int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
    const int32_t* block_table, int max_blocks, const int32_t* lens, const int64_t* cu_rows,
    int batch, int max_len, void* k_out, void* v_out, int64_t out_rows, int out_dtype, int* err,
    int device, void* stream) {
  if (max_blocks < 0 || batch < 0 || max_len < 0 || out_rows < 0 || device < 0)
    return fail(PDA_EINVAL, "negative size or device");
  if (batch > 65535) return fail(PDA_EINVAL, "batch > 65535");
  if (out_dtype != PDA_BF16 && out_dtype != PDA_FP16 && out_dtype != PDA_F32)
    return fail(PDA_EINVAL, "out_dtype must be PDA_BF16, PDA_FP16 or PDA_F32");
  const int st = pda::check_cache(num_kv_heads, head_dim, block_size, num_blocks);
  if (st != PDA_OK) return st;
  if (num_kv_heads > 8191) return fail(PDA_EUNSUPPORTED, "more than 8191 kv heads");
  if (batch == 0 || max_len == 0) return PDA_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !lens || !cu_rows ||
      (out_rows > 0 && (!k_out || !v_out)))
    return fail(PDA_EINVAL, "a required pointer is NULL");
  if (!pda::aligned(k_cache, 16) || !pda::aligned(v_cache, 16) || !pda::aligned(k_out, 16) ||
      !pda::aligned(v_out, 16) || !pda::aligned(k_scale, 4) || !pda::aligned(v_scale, 4) ||
      !pda::aligned(block_table, 4) || !pda::aligned(lens, 4) || !pda::aligned(cu_rows, 8) ||
      !pda::aligned(err, 4))
    return fail(PDA_EINVAL, "misaligned pointer");
  if ((int64_t)max_len > (int64_t)max_blocks * block_size)
    return fail(PDA_EINVAL, "max_len exceeds max_blocks * block_size");
  const int64_t elems = out_rows * num_kv_heads * head_dim;
  const int64_t out_bytes = elems * (out_dtype == PDA_F32 ? 4 : 2);
  const int64_t cache_bytes = num_blocks * block_size * num_kv_heads * head_dim;
  const pda::Rows outs[3] = {pda::span(k_out, out_bytes), pda::span(v_out, out_bytes),
                             pda::span(err, 8)};
  const pda::Rows ins[7] = {pda::span(k_cache, cache_bytes), pda::span(v_cache, cache_bytes),
                            pda::span(k_scale, num_blocks * num_kv_heads * 4),
                            pda::span(v_scale, num_blocks * num_kv_heads * 4),
                            pda::span(block_table, (int64_t)batch * max_blocks * 4),
                            pda::span(lens, batch * 4ll), pda::span(cu_rows, batch * 8ll)};
  for (int o = 0; o < 3; ++o) {
    for (const pda::Rows& in : ins)
      if (pda::overlaps(outs[o], in)) return fail(PDA_EALIAS, "an output overlaps an input");
    for (int j = o + 1; j < 3; ++j)
      if (pda::overlaps(outs[o], outs[j])) return fail(PDA_EALIAS, "two outputs overlap");
  }
  pda::GatherParams p;
  p.k = static_cast<const uint8_t*>(k_cache);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = block_table;
  p.lens = lens;
  p.cu_rows = cu_rows;
  p.k_out = static_cast<uint4*>(k_out);
  p.v_out = static_cast<uint4*>(v_out);
  p.err = err;
  p.num_blocks = num_blocks;
  p.out_rows = out_rows;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.max_len = max_len;
  p.Hkv = num_kv_heads;
  p.div_mul = num_kv_heads > 1 ? (uint32_t)(((1ull << 32) + num_kv_heads - 1) / num_kv_heads) : 0u;
  pda::Dev guard(device);
  if (guard.err != cudaSuccess) return fail(PDA_ECUDA, "cudaSetDevice failed");
  const dim3 grid((unsigned)((max_len + block_size - 1) / block_size), (unsigned)batch, 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto gather = [&](auto t) {
    using T = decltype(t);
    return pda::launch(head_dim == 64 ? pda::gather_fp8_kernel<T, 64> : pda::gather_fp8_kernel<T, 128>,
                       grid, pda::kGatherThreads, s, p);
  };
  return pda::launched("gather launch", out_dtype == PDA_BF16   ? gather(pda::Bf16())
                                        : out_dtype == PDA_FP16 ? gather(pda::Fp16())
                                                                : gather(float()));
}
