// Arithmetic shared by the kernels that rotate query and key heads: 16-bit
// unpacking and packing, and an exactly rounded two-term product sum.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace pda {

struct Bf16 {
  static __device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  // (RN(x) in the low half, RN(y) in the high half)
  static __device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

struct Fp16 {
  static __device__ __forceinline__ float lo_f(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
  }
  static __device__ __forceinline__ float hi_f(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
  static __device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// Round-to-odd conversion double -> float: truncate, then set the last bit
// if anything was cut off. Rounding that float to a format with at least two
// fewer significant bits (bf16: 8, fp16: 11, float: 24) gives the correctly
// rounded result of the double.
__device__ __forceinline__ float round_to_odd_float(double d) {
  const float f = __double2float_rz(d);
  return ((double)f != d) ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

// Two outputs, packed: RN_fmt(a0*b0 + c0*d0) in the low half and
// RN_fmt(a1*b1 + c1*d1) in the high half, for storage-format values a, c and
// fp32 b, d; equal to rounding the double-precision value (a*b and c*d are
// exact in double, the sum is rounded once) to the format.
// Fast path: r = fma(a, b, fl(c*d)) is within 2^-24 (|fl(c*d)| + |r|)(1 + 2^-23)
// + 2^-149 of the exact value; m is twice that bound. If rounding r - m down
// and r + m up gives the same storage values, the exact values, inside
// [r - m, r + m], round to them too. Otherwise (about one output in 10^4)
// both are recomputed in double and rounded through a round-to-odd float.
// The bound is kept tight (per output) because a warp takes the slow path
// whenever one of its lanes does.
// kCold: the double-precision path is a call, not inlined code, for kernels that
// unroll many of these and would not fit the instruction caches otherwise.
template <typename F>
__device__ __noinline__ uint32_t rounded_dot2_x2_exact(float a0, float b0, float c0, float d0,
                                                       float a1, float b1, float c1, float d1) {
  const double e0 = __dadd_rn(__dmul_rn((double)a0, (double)b0), __dmul_rn((double)c0, (double)d0));
  const double e1 = __dadd_rn(__dmul_rn((double)a1, (double)b1), __dmul_rn((double)c1, (double)d1));
  return F::pack2(round_to_odd_float(e0), round_to_odd_float(e1));
}

template <typename F, bool kCold = false>
__device__ __forceinline__ uint32_t rounded_dot2_x2(float a0, float b0, float c0, float d0,
                                                    float a1, float b1, float c1, float d1) {
  const float p0 = __fmul_rn(c0, d0), p1 = __fmul_rn(c1, d1);
  const float r0 = __fmaf_rn(a0, b0, p0), r1 = __fmaf_rn(a1, b1, p1);
  const float m0 = __fmaf_rn(fabsf(p0) + fabsf(r0), 0x1p-23f, 0x1p-147f);
  const float m1 = __fmaf_rn(fabsf(p1) + fabsf(r1), 0x1p-23f, 0x1p-147f);
  const uint32_t lo = F::pack2(__fsub_rd(r0, m0), __fsub_rd(r1, m1));
  const uint32_t hi = F::pack2(__fadd_ru(r0, m0), __fadd_ru(r1, m1));
  if (lo == hi) return lo;
  if constexpr (kCold) return rounded_dot2_x2_exact<F>(a0, b0, c0, d0, a1, b1, c1, d1);
  const double e0 = __dadd_rn(__dmul_rn((double)a0, (double)b0), __dmul_rn((double)c0, (double)d0));
  const double e1 = __dadd_rn(__dmul_rn((double)a1, (double)b1), __dmul_rn((double)c1, (double)d1));
  return F::pack2(round_to_odd_float(e0), round_to_odd_float(e1));
}

}  // namespace pda
