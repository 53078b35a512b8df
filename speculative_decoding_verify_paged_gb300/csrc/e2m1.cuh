// The 4-bit pool's format: E2M1 codes, two a byte (the even value below), and an E4M3 scale for 16 values of a row.
//   value = code * s * scale,   s = E4M3(max |x| * (1 / (6 scale))),   code = E2M1(x * (1 / (s scale)))
// Every operation is fp32 and rounded to nearest, so the codes are determined to the bit. 6 is the largest code: s
// rounds to 3 bits of mantissa, up or down by 1/16 at most, and what then lies past 6 saturates.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sv_internal.cuh"

namespace sv {

__device__ __forceinline__ float max_nan(float x, float y) {  // a NaN if one is
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((uint8_t)code, __NV_E4M3)));
}
// The block scale of values up to `top` in size; inv6 = 1 / (6 scale).
__device__ __forceinline__ uint32_t block_scale(float top, float inv6) {
  return __nv_cvt_float_to_fp8(__fmul_rn(top, inv6), __NV_SATFINITE, __NV_E4M3);
}
// What values are multiplied with to become codes.
__device__ __forceinline__ float code_factor(uint32_t s, float scale) {
  const float step = __fmul_rn(e4m3_value(s), scale);
  return step > 0.f ? __frcp_rn(step) : 0.f;
}
__device__ __forceinline__ float top_of(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) m = max_nan(m, fabsf(x[j]));
  return m;
}
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float r) {
  uint32_t w;
  asm("{.reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};}"
      : "=r"(w)
      : "f"(__fmul_rn(x[0], r)), "f"(__fmul_rn(x[1], r)), "f"(__fmul_rn(x[2], r)), "f"(__fmul_rn(x[3], r)),
        "f"(__fmul_rn(x[4], r)), "f"(__fmul_rn(x[5], r)), "f"(__fmul_rn(x[6], r)), "f"(__fmul_rn(x[7], r)));
  return w;
}
// The codes of a word as fp16 pairs (exact), two codes of a byte each
__device__ __forceinline__ void widen8(uint32_t w, uint32_t &p0, uint32_t &p1, uint32_t &p2, uint32_t &p3) {
  asm("{.reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;}"
      : "=r"(p0), "=r"(p1), "=r"(p2), "=r"(p3)
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ float2 pair_of(uint32_t halves) { return __half22float2(*reinterpret_cast<const __half2 *>(&halves)); }


template <int LEFT> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ void copy_all(uint32_t dst, const uint8_t *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes into shared memory, zeros from byte n on
__device__ __forceinline__ void copy_some(uint32_t dst, const uint8_t *src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// N bytes of shared memory as words
template <int N> __device__ __forceinline__ void read_words(uint32_t at, uint32_t *w) {
  if constexpr (N == 4) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
  else if constexpr (N == 8) asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  else asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
}
__device__ __forceinline__ uint32_t read_byte(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(at));
  return x;
}
__device__ __forceinline__ uint32_t read_half(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(x) : "r"(at));
  return x;
}

}  // namespace sv
