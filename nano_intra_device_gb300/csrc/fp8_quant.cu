// Values to e4m3 codes with a scale for each block of 128: rows (with RMSNorm and
// the residual's addition ahead of it, or through an index) and weight matrices.
//
//   s = max(max |y| / 448, 2^-126),  q = e4m3(y / s), to nearest, ties to even
//
// A block's largest value takes the largest code, 448.  The sum x + r, the norm's
// sum of squares and y are fp32; h is rounded to bf16 as it is stored, y only by
// its code; the quotient is rounded to fp32, then to the code.
//
// Bound by memory: one pass, 16-byte loads, a row of the norm in the registers of its
// CTA between the sum of squares and the codes.  Reached (of 6.68 TB/s copied): norm with
// residual, 4096 rows of 8192, 39 us = 6.0 TB/s; quantisation, 4096 rows of 14336, 28 us =
// 6.3 TB/s, by an index 4094 rows of 4096 8.7 us; two matrices of 14336 x 4096, 56 us =
// 6.3 TB/s.  Few rows: launch and latency, 1.4 to 2 us in a graph.
#include "fp8.cuh"

namespace nf {
namespace {

// Column blocks a thread quantises: as many loads are under way at once.  Where there are at
// most FEW_BLOCKS blocks an SM, or two blocks a row, one, which gives every SM work; one / four:
// 512 rows of 4096 (16384 blocks) 2.8 / 3.3 us, 1024 rows 4.5 / 4.1, 512 rows of 14336 6.7 /
// 5.6; 65536 rows of 256 13.0 / 13.3, of 384 18.9 / 15.2.
constexpr int FEW_BLOCKS = 128, QV = 4;
// Rows an SM up to which the norm takes one vector a thread: 1 / 2 vectors, rows of 4096,
// 1 row 1.96 / 2.26 us, 512 rows 5.2 / 6.2, 2048 rows 14.3 / 12.6.
constexpr int FEW_ROWS = 8;

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
  v[4] = bf16lo(u.z); v[5] = bf16hi(u.z); v[6] = bf16lo(u.w); v[7] = bf16hi(u.w);
}

// Vector i of a row (v; nothing from nvec on): `top` is its largest magnitude, the
// largest of 16 neighbouring threads the block's.  All lanes of a warp together.
__device__ __forceinline__ void store_block(const F8RowsArgs& a, int row, int i, int nvec, const float (&v)[8], float top) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = absmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float s = f8_scale(top), inv = 1.f / s;
  if (i < nvec) {
    reinterpret_cast<uint2*>(a.q + static_cast<size_t>(row) * a.cols)[i] =
        make_uint2(f8_codes4(v[0], v[1], v[2], v[3], s, inv), f8_codes4(v[4], v[5], v[6], v[7], s, inv));
    if ((i & 15) == 0) a.s[static_cast<size_t>(i >> 4) * a.rows + row] = s;
  }
}

// The norm: a row a warp (WARP) or a CTA, VPT vectors of 8 columns a thread, vector j *
// (threads of a row) + thread, so that 16 neighbouring threads hold a block of 128.
template <int VPT, bool RES, bool WARP>
__global__ void __launch_bounds__(512) f8_norm_kernel(const F8RowsArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int ti = WARP ? lane : threadIdx.x, tr = WARP ? 32 : blockDim.x, nvec = a.cols / 8;
  const int row = WARP ? blockIdx.x * warps + warp : blockIdx.x;
  if (row >= a.rows) return;  // (a whole warp)
  const size_t at = static_cast<size_t>(row) * a.cols;
  float v[VPT][8], ss = 0.f;
  uint4 xv[VPT], rv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * tr + ti;
    xv[j] = rv[j] = make_uint4(0u, 0u, 0u, 0u);
    if (i < nvec) {  // plain loads: h may be x or r
      xv[j] = reinterpret_cast<const uint4*>(a.x + at)[i];
      if (RES) rv[j] = reinterpret_cast<const uint4*>(a.r + at)[i];
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    unpack8(xv[j], v[j]);
    if (RES) {
      float r[8];
      unpack8(rv[j], r);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] += r[k];
      const int i = j * tr + ti;
      if (a.h && i < nvec)
        reinterpret_cast<uint4*>(a.h + at)[i] = make_uint4(pack_bf16(v[j][0], v[j][1]), pack_bf16(v[j][2], v[j][3]),
                                                           pack_bf16(v[j][4], v[j][5]), pack_bf16(v[j][6], v[j][7]));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += v[j][k] * v[j][k];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (!WARP) {
    __shared__ float red[16];
    if (lane == 0) red[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < warps; ++i) ss += red[i];
  }
  const float scale = 1.f / sqrtf(ss / a.cols + a.eps);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = j * tr + ti;
    float top = 0.f;
    if (i < nvec) {
      float g[8];
      unpack8(reinterpret_cast<const uint4*>(a.g)[i], g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[j][k] = v[j][k] * scale * g[k];
        top = absmax_nan(top, v[j][k]);
      }
    }
    store_block(a, row, i, nvec, v[j], top);
  }
}

template <int VPT, bool WARP>
cudaError_t launch_norm(const F8RowsArgs& a, int threads, cudaStream_t stream) {
  const int of_cta = WARP ? threads / 32 : 1;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.rows) + of_cta - 1) / of_cta);
  if (a.r) return launch_dependent(f8_norm_kernel<VPT, true, WARP>, grid, threads, 0, stream, 1, a);
  return launch_dependent(f8_norm_kernel<VPT, false, WARP>, grid, threads, 0, stream, 1, a);
}

// Given values: a CTA takes 16 rows (8 where a thread has several blocks: a shorter last
// wave, 4096 rows of 14336 28.0 us, by 16 rows 29.9, by 4 30.9) x V column blocks, 16 threads
// a block of 128, so that the scales of neighbouring rows, next to one another in memory, are
// written together.
constexpr int rows_of(int v) { return v == 1 ? 16 : 8; }
template <int V>
__global__ void __launch_bounds__(rows_of(V) * 16) f8_quant_kernel(const F8RowsArgs a, int col_groups) {
  pdl_trigger();
  pdl_wait();
  const int sub = threadIdx.x & 15, nvec = a.cols / 8;
  const int group = blockIdx.x / col_groups, row = group * rows_of(V) + (threadIdx.x >> 4);
  const int vec = (blockIdx.x - group * col_groups) * (V * 16) + sub;
  static_assert(V == 1 || V == 4, "column blocks");
  const int from = row < a.rows ? a.index ? a.index[row] : row : -1;
  const bool there = from >= 0 && from < a.src_rows;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(there ? from : 0) * a.cols);
  uint4 u[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    u[j] = make_uint4(0u, 0u, 0u, 0u);
    if (there && vec + 16 * j < nvec) u[j] = x[vec + 16 * j];
  }
  const int end = row < a.rows ? nvec : 0;
  if constexpr (V == 4) {
    // The four blocks' largest magnitudes at once: a lane hands on the two blocks, then the
    // one, that it does not keep, and ends with block sub % 4, whose scale and reciprocal it
    // takes for all (a division is a dozen instructions; made for each block by every lane,
    // 4096 rows of 14336 take 30.7 us, so 29.5).
    float t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
      unpack8(u[j], v);
      t[j] = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) t[j] = absmax_nan(t[j], v[k]);
    }
    auto over = [](float kept, float given, int lanes) { return absmax_nan(kept, __shfl_xor_sync(0xffffffffu, given, lanes)); };
    const bool odd = sub & 1, high = sub & 2;
    const float t0 = over(odd ? t[1] : t[0], odd ? t[0] : t[1], 1), t2 = over(odd ? t[3] : t[2], odd ? t[2] : t[3], 1);
    float top = over(high ? t2 : t0, high ? t0 : t2, 2);
    top = over(top, top, 4);
    top = over(top, top, 8);
    const float s = f8_scale(top), inv = 1.f / s;
    if (sub < 4 && vec + 15 * sub < end) a.s[static_cast<size_t>((vec - sub) / 16 + sub) * a.rows + row] = s;
    uint2* q = reinterpret_cast<uint2*>(a.q + static_cast<size_t>(row) * a.cols);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float sj = __shfl_sync(0xffffffffu, s, j, 16), ij = __shfl_sync(0xffffffffu, inv, j, 16);
      float v[8];
      unpack8(u[j], v);
      if (vec + 16 * j < end)
        q[vec + 16 * j] = make_uint2(f8_codes4(v[0], v[1], v[2], v[3], sj, ij), f8_codes4(v[4], v[5], v[6], v[7], sj, ij));
    }
  } else {
    float v[8], top = 0.f;
    unpack8(u[0], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = absmax_nan(top, v[k]);
    store_block(a, row, vec, end, v, top);
  }
}

template <int V>
cudaError_t launch_quant(const F8RowsArgs& a, cudaStream_t stream) {
  const int col_groups = (a.cols + V * F8_BLOCK - 1) / (V * F8_BLOCK);
  const long long grid = (static_cast<long long>(a.rows) + rows_of(V) - 1) / rows_of(V) * col_groups;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(f8_quant_kernel<V>, static_cast<unsigned>(grid), rows_of(V) * 16, 0, stream, 1, a, col_groups);
}

// One CTA a 128 x 128 block: thread t has vector t % 16 of the rows t / 16 + 16 i.
__global__ void __launch_bounds__(256)
    f8_weights_kernel(const __nv_bfloat16* w, uint8_t* q, float* s,
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
      u[i] = *reinterpret_cast<const uint4*>(w + base + static_cast<size_t>(r0 + 16 * i) * cols);
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

cudaError_t launch_f8_rows(const F8RowsArgs& a, int sms, cudaStream_t stream) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.cols % 16 || a.cols > F8_MAX_COLS) return cudaErrorInvalidValue;
  const int nvec = a.cols / 8;
  if (!a.g) {
    const long long blocks = static_cast<long long>(a.rows) * ((nvec + 15) / 16);
    return blocks <= FEW_BLOCKS * sms || nvec <= 32 ? launch_quant<1>(a, stream) : launch_quant<QV>(a, stream);
  }
  auto threads = [&](int vpt) { return (nvec + 32 * vpt - 1) / (32 * vpt) * 32; };
  // rows of at most 512 columns a warp each: 4096 rows of 256 3.6 us, by CTAs 4.5
  if (nvec <= 32) return launch_norm<1, true>(a, 128, stream);
  if (nvec <= 64) return launch_norm<2, true>(a, 128, stream);
  if (nvec <= 512 && (nvec <= 128 || a.rows <= FEW_ROWS * sms)) return launch_norm<1, false>(a, threads(1), stream);
  if (nvec <= 1024) return launch_norm<2, false>(a, threads(2), stream);
  if (nvec <= 2048) return launch_norm<4, false>(a, threads(4), stream);
  return launch_norm<8, false>(a, threads(8), stream);
}

cudaError_t launch_f8_weights(const __nv_bfloat16* w, uint8_t* q, float* s, int mats, int rows,
                              int cols, cudaStream_t stream) {
  const long long rb = (rows + F8_BLOCK - 1) / F8_BLOCK, cb = (cols + F8_BLOCK - 1) / F8_BLOCK;
  if (mats * rb * cb <= 0) return cudaSuccess;
  if (mats * rb * cb > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(f8_weights_kernel, static_cast<unsigned>(mats * rb * cb), 256, 0, stream, 1, w, q, s, rows, cols,
                          static_cast<int>(rb), static_cast<int>(cb));
}

}  // namespace nf
