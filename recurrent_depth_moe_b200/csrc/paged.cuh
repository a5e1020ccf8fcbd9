// Device helpers of the paged key / value cache: e4m3 values with one power-of-two scale per
// (position, kv head), and the lookup of a position's page.
//
// A stored row is x ~ q * 2^E with q in e4m3 and E the smallest exponent that brings the row's
// largest finite magnitude to at most 448, the largest e4m3 value.  e4m3 is a floating format,
// so a power of two loses nothing against amax / 448: rounding stays relative (half a step of a
// 3-bit mantissa, 2^-4) except for values 2^-15 below the row's largest, and the read back
// value q * 2^E is exact in bf16.  The scale then costs one byte (E + 127) instead of four.
#pragma once
#include "common.cuh"
#include "kernels.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace rdt {

// 2^(b - 127) of a stored exponent byte (255, which the library never writes, gives inf)
__device__ __forceinline__ float exp_byte_scale(int b) { return __int_as_float(b ? b << 23 : 0x00400000); }

// exponent E of a row whose largest finite magnitude is amax: amax = m 2^x, 0.5 <= m < 1, and
// 448 = 0.875 * 2^9
__device__ __forceinline__ int row_exponent(float amax) {
  const int b = __float_as_int(amax);                            // x = (b >> 23) - 126; 0.875 is mantissa 0x600000
  return max((b >> 23) - 126 - 9 + ((b & 0x7fffff) > 0x600000), -127);   // (subnormal rows, and 0: -127; at most 120)
}
__device__ __forceinline__ float pow2_neg(int E) { return __int_as_float((127 - E) << 23); }   // 2^-E, -127 <= E <= 120

// magnitude for the row maximum: infinities and NaN take no part in the scale
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}
// e4m3 of x * inv, round to nearest even.  The scale leaves every finite value at or below 448, so
// the conversion's saturation never acts on one; e4m3 has no infinity, so +-inf is stored as NaN
// (as a NaN is), never as a large finite value: callers whose row holds one pass it through
// inf_to_nan.
__device__ __forceinline__ float inf_to_nan(float x) { return fabsf(x) <= 3.402823466e38f ? x : __int_as_float(0x7fffffff); }
__device__ __forceinline__ uint8_t to_e4m3(float x, float inv) {
  return (uint8_t)__nv_cvt_float_to_fp8(inf_to_nan(x) * inv, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float e4m3_f(uint8_t q) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(q, __NV_E4M3)));
}

// An index out of range: in the call's status word and in the cache's.
__device__ __forceinline__ void record_bad(const PagedView& c, DevStatus* st, int where, int detail) {
  record_status(st, ST_BOUNDS, where, detail);
  record_status(c.also, ST_BOUNDS, where, detail);
}
// Which page of its sequence a position is in.
__device__ __forceinline__ int page_index(const PagedView& c, int pos) {
  return c.ps_shift >= 0 ? pos >> c.ps_shift : pos / c.page_size;
}
// Page of position pos of sequence b, or -1 (recorded) if the position or
// the table's entry is out of range.
__device__ __forceinline__ int page_of(const PagedView& c, int b, int pos, DevStatus* st, int where) {
  const int pi = page_index(c, pos);
  if (pos < 0 || pi >= c.max_pages) {
    record_bad(c, st, where, pos);
    return -1;
  }
  const int page = __ldg(c.table + (long long)b * c.max_pages + pi);
  if (page < 0 || page >= c.n_pages) {
    record_bad(c, st, where + 1, page);
    return -1;
  }
  return page;
}

// Visible keys of sequence b: its length (0 without lens) plus len_add, inside what its table can hold.
__device__ __forceinline__ int visible_keys(const PagedView& c, const int* lens, int b, int len_add, DevStatus* st,
                                            int where) {
  const long long n = (long long)(lens ? __ldg(lens + b) : 0) + len_add, cap = (long long)c.max_pages * c.page_size;
  if (n > cap) {
    record_bad(c, st, where, (int)(n - len_add));
    return (int)cap;
  }
  return n > 0 ? (int)n : 0;
}

}  // namespace rdt
