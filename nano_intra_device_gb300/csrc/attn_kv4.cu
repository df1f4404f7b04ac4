// Attention over the 4-bit KV cache: a CTA takes one row and one KV head, its
// warps every fourth position, each with an online softmax of its own (base 2,
// fp32); the four states are joined at the end.
#include <math_constants.h>

#include "common.cuh"
#include "kv4.cuh"
#include "kv4.h"

namespace nf {
namespace {

template <int GRP, int D>
__global__ void __launch_bounds__(128) attn_kv4_rows_kernel(const Kv4AttnArgs a) {
  constexpr int CPL = D / 32;  // channels of a lane
  const int t = blockIdx.x / a.n_kv, g = blockIdx.x % a.n_kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = t, b0 = t, b1 = t + 1;
  if (a.tok_begin) {
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < a.n_seq; i += 128)
        if (a.tok_begin[i] < 0 || a.tok_begin[i + 1] < a.tok_begin[i] || a.tok_begin[i + 1] > a.n_tok)
          raise_status(a.status, ST_BAD_LEN);
    int lo = 0, hi = a.n_seq - 1;  // the last request that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.tok_begin[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
    b0 = a.tok_begin[s];
    b1 = a.tok_begin[s + 1];
    if (b0 < 0 || t < b0 || t >= b1 || b1 > a.n_tok) return;  // a row of no request
  }
  int len = a.seq_lens[s];
  if (len < 0 || len > static_cast<long long>(a.max_pages) * KV4_P) {
    raise_status(a.status, ST_BAD_LEN);
    len = 0;
  }
  const int n = max(len - (b1 - b0) + (t - b0) + 1, 0);
  float q[GRP][CPL], o[GRP][CPL], m[GRP], l[GRP];
#pragma unroll
  for (int h = 0; h < GRP; ++h) {
    m[h] = -CUDART_INF_F;
    l[h] = 0.f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      q[h][c] = __bfloat162float(a.q[(static_cast<size_t>(t) * a.n_q + g * GRP + h) * D + lane * CPL + c]);
      o[h][c] = 0.f;
    }
  }
  for (int p = warp; p < n; p += 4) {
    int page = a.block_table[static_cast<size_t>(s) * a.max_pages + p / KV4_P];
    if (page < 0 || page >= a.num_pages) {
      raise_status(a.status, ST_BAD_PAGE);
      page = 0;
    }
    const uint8_t* part = a.pool + (static_cast<size_t>(page) * a.n_kv + g) * 2 * kv4_part_bytes(D);
    float kv[2][CPL];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* code = part + i * kv4_part_bytes(D) + (p % KV4_P) * (D / 2) + lane * CPL / 2;
      const float sc = e4m3_to_f32(part[i * kv4_part_bytes(D) + 8 * D + (p % KV4_P) * (D / 16) + lane * CPL / 16]);
#pragma unroll
      for (int c = 0; c < CPL; c += 2) {
        const float2 x = f16x2_to_f32x2(e2m1_to_f16x2<0>(code[c / 2]));
        kv[i][c] = x.x * sc;
        kv[i][c + 1] = x.y * sc;
      }
    }
#pragma unroll
    for (int h = 0; h < GRP; ++h) {
      float x = 0.f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) x = fmaf(q[h][c], kv[0][c], x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x *= a.scale_log2;
      const float nm = fmaxf(m[h], x), w = exp2f(m[h] - nm), e = exp2f(x - nm);
      m[h] = nm;
      l[h] = l[h] * w + e;
#pragma unroll
      for (int c = 0; c < CPL; ++c) o[h][c] = fmaf(e, kv[1][c], o[h][c] * w);
    }
  }
  __shared__ float sm[4][GRP], sl[4][GRP], so[4][GRP][D];
#pragma unroll
  for (int h = 0; h < GRP; ++h) {
    if (lane == 0) {
      sm[warp][h] = m[h];
      sl[warp][h] = l[h];
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) so[warp][h][lane * CPL + c] = o[h][c];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < GRP * D; i += 128) {
    const int h = i / D, c = i % D;
    float M = -CUDART_INF_F, L = 0.f, O = 0.f;
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sm[w][h]);
    for (int w = 0; w < 4; ++w) {
      const float x = sm[w][h] == -CUDART_INF_F ? 0.f : exp2f(sm[w][h] - M);
      L += x * sl[w][h];
      O += x * so[w][h][c];
    }
    a.o[(static_cast<size_t>(t) * a.n_q + g * GRP + h) * D + c] =
        __float2bfloat16_rn(n > 0 ? O / L * a.v_scale : 0.f);
  }
}

template <int GRP, int D>
cudaError_t launch_t(const Kv4AttnArgs& a, cudaStream_t stream) {
  attn_kv4_rows_kernel<GRP, D><<<a.n_tok * a.n_kv, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_kv4(const Kv4AttnArgs& a, cudaStream_t stream) {
  const int grp = a.n_q / a.n_kv;
#define NF_KV4_CASE(G)                                          \
  if (grp == G) return a.head_dim == 128 ? launch_t<G, 128>(a, stream) : launch_t<G, 64>(a, stream);
  NF_KV4_CASE(1) NF_KV4_CASE(2) NF_KV4_CASE(4) NF_KV4_CASE(8)
#undef NF_KV4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace nf
