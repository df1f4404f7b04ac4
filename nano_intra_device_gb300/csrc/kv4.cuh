// The 4-bit KV format on the device: e2m1 codes and e4m3 block scales.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv4.h"

namespace nf {

// Two codes (one byte of v) as an f16 pair, exact: channel 2i low, 2i + 1 high.
template <int BYTE>
__device__ __forceinline__ uint32_t e2m1_to_f16x2(uint32_t v) {
  uint32_t r;
  if (BYTE == 0)
    asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, a;}" : "=r"(r) : "r"(v));
  if (BYTE == 1)
    asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(r) : "r"(v));
  if (BYTE == 2)
    asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, c;}" : "=r"(r) : "r"(v));
  if (BYTE == 3)
    asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, d;}" : "=r"(r) : "r"(v));
  return r;
}
// The low two bytes of v, e4m3, as an f16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(r) : "r"(v));
  return r;
}
// Nearest codes of a pair, ties to even, saturating: lo in the low half of the byte.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float hi, float lo) {
  uint32_t r;
  asm("{.reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; mov.b32 %0, {t, 0, 0, 0};}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}
// Nearest e4m3, ties to even, saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  const uint32_t h = e4m3x2_to_f16x2(b);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t v) {
  __half2 h;
  *reinterpret_cast<uint32_t*>(&h) = v;
  return __half22float2(h);
}
// lo in the low half
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// max that keeps a NaN
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// 2^e for e in [-126, 127]
__host__ __device__ __forceinline__ float exp2_int(int e) {
#ifdef __CUDA_ARCH__
  return __int_as_float((e + 127) << 23);
#else
  union {
    uint32_t u;
    float f;
  } x;
  x.u = static_cast<uint32_t>(e + 127) << 23;
  return x.f;
#endif
}

}  // namespace nf
