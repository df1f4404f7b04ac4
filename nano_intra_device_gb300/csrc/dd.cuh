// Pairs of floats that stand for their sum (about 47 significant bits), for the
// few values that fp32 cannot place: fp64 arithmetic, at a sixty-fourth of the
// fp32 rate, takes a warp tens of microseconds for one such value.  The
// products and sums are Dekker's and Knuth's error-free transformations.
#pragma once
#include <math.h>
#include <stdint.h>

#include <cuda_runtime.h>

namespace nf {

struct dd {
  float h, l;
};

__host__ __device__ __forceinline__ dd dd_two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__host__ __device__ __forceinline__ dd dd_quick(float a, float b) {  // |a| >= |b|
  const float s = a + b;
  return {s, b - (s - a)};
}
__host__ __device__ __forceinline__ dd dd_prod(float a, float b) {
  const float p = a * b;
  return {p, fmaf(a, b, -p)};
}
__host__ __device__ __forceinline__ dd dd_add(dd a, dd b) {
  dd s = dd_two_sum(a.h, b.h);
  const dd t = dd_two_sum(a.l, b.l);
  s = dd_quick(s.h, s.l + t.h);
  return dd_quick(s.h, s.l + t.l);
}
__host__ __device__ __forceinline__ dd dd_mul(dd a, dd b) {
  const dd p = dd_prod(a.h, b.h);
  return dd_quick(p.h, p.l + fmaf(a.h, b.l, a.l * b.h));
}
__host__ __device__ __forceinline__ dd dd_mul(dd a, float b) {
  const dd p = dd_prod(a.h, b);
  return dd_quick(p.h, fmaf(a.l, b, p.l));
}
__host__ __device__ __forceinline__ dd dd_neg(dd a) { return {-a.h, -a.l}; }

// 1 / sqrt(m), one Newton step of second order from the fp32 value.
__host__ __device__ __forceinline__ dd dd_rsqrt(dd m) {
#ifdef __CUDA_ARCH__
  const float r = rsqrtf(m.h);
#else
  const float r = 1.f / sqrtf(m.h);
#endif
  const dd t = dd_mul(m, dd_prod(r, r));          // m r^2, near 1
  const float e = (1.f - t.h) - t.l;              // exact difference of neighbours of 1
  return dd_two_sum(r, r * (e * fmaf(0.375f, e, 0.5f)));
}

// cos and sin of 2 pi `turn` / 2^64: the nearest 64th of a turn from a table of
// the first quarter, the rest (at most 1/128) by Taylor series.
__host__ __device__ __forceinline__ void dd_cos_sin(uint64_t turn, dd* c, dd* s) {
  // cos(2 pi k / 64), k = 0 .. 16, as float pairs
  constexpr float T[17][2] = {
    {0x1p0f, 0.f}, {0x1.fd88dap-1f, 0x1.e89292p-28f},
    {0x1.f6297cp-1f, 0x1.feeb96p-26f}, {0x1.e9f416p-1f, -0x1.273a44p-26f},
    {0x1.d906bcp-1f, 0x1.e651a8p-26f}, {0x1.c38b30p-1f, -0x1.cfe84ap-26f},
    {0x1.a9b662p-1f, 0x1.21d434p-26f}, {0x1.8bc806p-1f, 0x1.62a2e8p-26f},
    {0x1.6a09e6p-1f, 0x1.9fcef4p-27f}, {0x1.44cf32p-1f, 0x1.424776p-27f},
    {0x1.1c73b4p-1f, -0x1.9465cep-27f}, {0x1.e2b5d4p-2f, -0x1.fe4272p-28f},
    {0x1.87de2ap-2f, 0x1.abaa58p-28f}, {0x1.294062p-2f, 0x1.dab3e0p-27f},
    {0x1.8f8b84p-3f, -0x1.cb2cfap-30f}, {0x1.917a6cp-4f, -0x1.eb25eap-31f},
    {0.f, 0.f},
  };
  const uint64_t near = turn + (1ull << 57);
  const uint32_t k = static_cast<uint32_t>(near >> 58);              // the 64th
  const int64_t rest = static_cast<int64_t>(turn - (static_cast<uint64_t>(k) << 58));
  // x = 2 pi rest / 2^64: 24 bits of rest, then the others
  const float r1 = static_cast<float>(static_cast<int32_t>(rest >> 34));  // 24 bits and a sign, exact
  const float r2 = static_cast<float>(static_cast<uint64_t>(rest) & ((1ull << 34) - 1)) * 0x1p-34f;
  const dd x = dd_mul(dd_two_sum(r1, r2), dd{0x1.921fb6p-28f, -0x1.777a5cp-53f});  // 2 pi 2^-30
  const dd q = dd_mul(x, x);
  // sin x = x (1 - q/6 + q^2/120 - q^3/5040), cos x = 1 - q/2 + q^2/24 - q^3/720 + q^4/40320
  const float q1 = q.h;
  dd ss = dd_mul(q, dd{-0x1.555556p-3f, 0x1.555556p-28f});           // -1/6
  ss = dd_add(ss, dd_two_sum(q1 * q1 * (1.f / 120.f), -q1 * q1 * q1 * (1.f / 5040.f)));
  ss = dd_add(dd{1.f, 0.f}, ss);
  const dd sx = dd_mul(ss, x);
  dd cx = dd_mul(q, -0.5f);
  const dd q2 = dd_mul(q, q);
  cx = dd_add(cx, dd_mul(q2, dd{0x1.555556p-5f, -0x1.555556p-30f}));  // 1/24
  cx = dd_add(cx, dd{q1 * q1 * q1 * fmaf(q1, 1.f / 40320.f, -1.f / 720.f), 0.f});
  cx = dd_add(dd{1.f, 0.f}, cx);
  // the table's angle: quadrant k / 16, step k % 16
  const int j = static_cast<int>(k & 15u);
  dd tc = {T[j][0], T[j][1]}, ts = {T[16 - j][0], T[16 - j][1]};
  const dd cc = dd_add(dd_mul(tc, cx), dd_neg(dd_mul(ts, sx)));
  const dd sn = dd_add(dd_mul(ts, cx), dd_mul(tc, sx));
  switch ((k >> 4) & 3u) {
    case 0: *c = cc; *s = sn; break;
    case 1: *c = dd_neg(sn); *s = cc; break;
    case 2: *c = dd_neg(cc); *s = dd_neg(sn); break;
    default: *c = sn; *s = dd_neg(cc); break;
  }
}

}  // namespace nf
