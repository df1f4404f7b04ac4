// Values to e4m3 codes with a scale for each block of 128: rows (with RMSNorm and
// the residual's addition ahead of it, or through an index) and weight matrices.
//
//   s = max(max |y| / 448, 2^-126),  q = e4m3(y / s), to nearest, ties to even
//
// A block's largest value takes the largest code, 448.  The sum x + r, the norm's
// sum of squares and y are fp32; h is rounded to bf16 as it is stored, y only by
// its code; the quotient is rounded to fp32, then to the code.
//
// Bound by memory: one pass, 16-byte loads, a row in the registers of its CTA
// between the sum of squares and the codes.
#include "fp8.cuh"

namespace nf {
namespace {

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
  v[4] = bf16lo(u.z); v[5] = bf16hi(u.z); v[6] = bf16lo(u.w); v[7] = bf16hi(u.w);
}

// One CTA a row, VPT vectors of 8 columns a thread (vector j * blockDim + thread);
// 16 neighbouring threads hold a block of 128.
template <int VPT, bool NORM, bool RES>
__global__ void __launch_bounds__(512) f8_rows_kernel(const F8RowsArgs a) {
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, nvec = a.cols / 8;
  const int from = a.index ? a.index[row] : row;
  const bool there = from >= 0 && from < a.src_rows;
  const size_t at = static_cast<size_t>(there ? from : 0) * a.cols;
  const uint4* xr = reinterpret_cast<const uint4*>(a.x + at);
  float v[VPT][8];
  uint4 xv[VPT], rv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    xv[j] = rv[j] = make_uint4(0u, 0u, 0u, 0u);
    if (there && i < nvec) {
      xv[j] = xr[i];  // plain loads: h may be x or r
      if (RES) rv[j] = reinterpret_cast<const uint4*>(a.r + at)[i];
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    unpack8(xv[j], v[j]);
    if (RES) {
      float r[8];
      unpack8(rv[j], r);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] += r[k];
      const int i = j * blockDim.x + threadIdx.x;
      if (a.h && i < nvec)
        reinterpret_cast<uint4*>(a.h + at)[i] = make_uint4(pack_bf16(v[j][0], v[j][1]), pack_bf16(v[j][2], v[j][3]),
                                                           pack_bf16(v[j][4], v[j][5]), pack_bf16(v[j][6], v[j][7]));
    }
    if (NORM) {
#pragma unroll
      for (int k = 0; k < 8; ++k) ss += v[j][k] * v[j][k];
    }
  }
  if (NORM) {
    __shared__ float red[32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
    __syncthreads();
    float tot = 0.f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) tot += red[i];
    const float scale = 1.f / sqrtf(tot / a.cols + a.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = j * blockDim.x + threadIdx.x;
      if (i < nvec) {
        float g[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.g) + i), g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] = v[j][k] * scale * g[k];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * blockDim.x + threadIdx.x;
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = absmax_nan(top, v[j][k]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = absmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float s = f8_scale(top), inv = 1.f / s;
    if (i < nvec) {
      const uint2 c = make_uint2(f8_codes4(v[j][0], v[j][1], v[j][2], v[j][3], s, inv),
                                 f8_codes4(v[j][4], v[j][5], v[j][6], v[j][7], s, inv));
      reinterpret_cast<uint2*>(a.q + static_cast<size_t>(row) * a.cols)[i] = c;
      if ((i & 15) == 0) a.s[static_cast<size_t>(i >> 4) * a.rows + row] = s;
    }
  }
}

template <int VPT>
cudaError_t launch_rows(const F8RowsArgs& a, int threads, cudaStream_t stream) {
  if (!a.g) return launch_dependent(f8_rows_kernel<VPT, false, false>, a.rows, threads, 0, stream, a);
  if (a.r) return launch_dependent(f8_rows_kernel<VPT, true, true>, a.rows, threads, 0, stream, a);
  return launch_dependent(f8_rows_kernel<VPT, true, false>, a.rows, threads, 0, stream, a);
}

// One CTA a 128 x 128 block: thread t has vector t % 16 of the rows t / 16 + 16 i.
__global__ void __launch_bounds__(256)
    f8_weights_kernel(const __nv_bfloat16* __restrict__ w, uint8_t* __restrict__ q, float* __restrict__ s,
                      int rows, int cols, int row_blocks, int col_blocks) {
  pdl_trigger();
  pdl_wait();
  const int cb = blockIdx.x % col_blocks;
  const int rb = blockIdx.x / col_blocks % row_blocks;
  const size_t mat = blockIdx.x / col_blocks / row_blocks;
  const int c = cb * F8_BLOCK + (threadIdx.x & 15) * 8, r0 = rb * F8_BLOCK + (threadIdx.x >> 4);
  const size_t base = mat * rows * static_cast<size_t>(cols) + c;
  uint4 u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c < cols && r0 + 16 * i < rows)
      u[i] = __ldg(reinterpret_cast<const uint4*>(w + base + static_cast<size_t>(r0 + 16 * i) * cols));
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack8(u[i], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = absmax_nan(top, v[k]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = absmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  __shared__ float red[8];
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = absmax_nan(top, red[i]);
  const float sc = f8_scale(top), inv = 1.f / sc;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (c < cols && r0 + 16 * i < rows) {
      float v[8];
      unpack8(u[i], v);
      *reinterpret_cast<uint2*>(q + base + static_cast<size_t>(r0 + 16 * i) * cols) =
          make_uint2(f8_codes4(v[0], v[1], v[2], v[3], sc, inv), f8_codes4(v[4], v[5], v[6], v[7], sc, inv));
    }
  }
  if (threadIdx.x == 0) s[(mat * row_blocks + rb) * col_blocks + cb] = sc;
}

}  // namespace

cudaError_t launch_f8_rows(const F8RowsArgs& a, cudaStream_t stream) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.cols % 16 || a.cols > F8_MAX_COLS) return cudaErrorInvalidValue;
  const int nvec = a.cols / 8;
  auto threads = [&](int vpt) { return (nvec + 32 * vpt - 1) / (32 * vpt) * 32; };
  if (nvec <= 512) return launch_rows<1>(a, threads(1), stream);
  if (nvec <= 1024) return launch_rows<2>(a, threads(2), stream);
  if (nvec <= 2048) return launch_rows<4>(a, threads(4), stream);
  return launch_rows<8>(a, threads(8), stream);
}

cudaError_t launch_f8_weights(const __nv_bfloat16* w, uint8_t* q, float* s, int mats, int rows,
                              int cols, cudaStream_t stream) {
  const long long rb = (rows + F8_BLOCK - 1) / F8_BLOCK, cb = (cols + F8_BLOCK - 1) / F8_BLOCK;
  if (mats * rb * cb <= 0) return cudaSuccess;
  if (mats * rb * cb > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(f8_weights_kernel, static_cast<unsigned>(mats * rb * cb), 256, 0, stream, w, q, s, rows, cols,
                          static_cast<int>(rb), static_cast<int>(cb));
}

}  // namespace nf
