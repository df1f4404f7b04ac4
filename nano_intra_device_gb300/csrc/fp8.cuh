// Device-side helpers of the 8-bit operators: e4m3 products on tcgen05, copies and
// arrivals, the scale of a block and its codes, SwiGLU, launches.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp8.h"

namespace nf {

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs (K = 32 an instruction), fp32 accumulate.
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: e4m3 A and B (both K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 lanes x 16 columns, as the 32-column form.
__device__ __forceinline__ void tc_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// The cluster barrier in two halves, for threads that diverge in between.  Relaxed: it
// orders execution alone (barriers made before it are published by fence_mbar_init).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// The barrier before exit: no CTA leaves, and with it its shared memory, while a peer may
// still read there.  Released: the loads from peers that are before it in a thread's
// program are done when it arrives, whether or not their values were used (rows behind the
// last one are read and not stored, so the compiler may leave their loads in flight).
__device__ __forceinline__ void cluster_leave() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  cluster_wait();
}
// 16 bytes of a CTA of the cluster, by shared::cluster address.
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A tile into L2 alone.  Allowed ahead of pdl_wait(): L2 is where writes of the kernel
// ahead meet later reads, so a line taken early does not get stale.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
// One lane of a converged warp.  Products are issued under it rather than under
// `lane == 0`: their operands, computed by the whole warp, then stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// One arrival of the lanes for which `yes` holds, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint64_t* bar, bool yes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(yes ? 1u : 0u)
      : "memory");
}
// 4 bytes global -> shared (zeros where not `there`), and an arrival on an mbarrier once
// this thread's copies so far have landed.
__device__ __forceinline__ void copy4(float* dst, const float* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_copied(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// d += a b, a a value read from tensor memory.  Volatile: it must not be used ahead of
// the wait for its load.
__device__ __forceinline__ void fma_loaded(float& d, uint32_t a, float b) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(d) : "f"(__uint_as_float(a)), "f"(b));
}

// The larger magnitude; a NaN on either side stays.
__device__ __forceinline__ float absmax_nan(float m, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
  return r;
}
// The scale of a block whose largest magnitude is `top`: NaN where that is not finite.
__device__ __forceinline__ float f8_scale(float top) {
  return top <= 3.402823466e38f ? fmaxf(top / 448.f, 1.17549435e-38f) : __int_as_float(0x7fffffff);
}
// y / s in fp32, s > 0 with its rounded reciprocal inv: the product errs by an ulp or
// two, its remainder y - q s is exact in a fused multiply-add, and one correction by it
// gives the rounded quotient (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990); where s < 2^-100 the remainder may underflow
// and the quotient be an ulp off.  A block's values are often exact ties of codes (a
// ratio of two 8-bit significands times 448): the product alone settles one code in 2000
// of normal bf16 values otherwise.
__device__ __forceinline__ float f8_quotient(float y, float s, float inv) {
  const float q = y * inv;
  return fmaf(fmaf(-q, s, y), inv, q);
}
// Four values over their scale s (inv its reciprocal) as codes, value 0 in the low byte.
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d, float s, float inv) {
  const float2 x = make_float2(f8_quotient(a, s, inv), f8_quotient(b, s, inv));
  const float2 y = make_float2(f8_quotient(c, s, inv), f8_quotient(d, s, inv));
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The same for values that are themselves rounded, by the product with inv alone: off
// the nearest code where the quotient lies within 2^-22 of a border, as the values do.
__device__ __forceinline__ uint32_t f8_codes4_near(float a, float b, float c, float d, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// silu(g) u = g u / (1 + 2^(-g log2 e)): exponential and reciprocal by the hardware's
// approximations (2 and 1 units in the last place).  The rounded product g log2 e weighs more
// where the exponential does, at g < 0: ln 2 times its half step, and 2^-26 g of log2 e's own
// rounding, are some 2^-21 of the value at g = -8, 2^-19 at -32 and 2^-18 at -88, beside 2^-9
// of bf16's rounding and 2^-4 of e4m3's.  A g below -126 ln 2 gives zero, as the reciprocal of
// anything above 2^126 does; infinite g: NaN or g u.
__device__ __forceinline__ float silu_mul(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return g * r * u;
}

// A launch as a programmatic dependent of the stream's kernel ahead, in clusters of
// `cluster` CTAs: the kernel may start while that one ends, and calls pdl_wait() before
// it touches global memory.  What kernels ahead may have written is not read through the
// read-only path, whose lines may be as old as the kernel's start.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                             int cluster, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace nf
