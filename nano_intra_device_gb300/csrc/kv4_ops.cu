// The small operators around the 4-bit KV cache: block tables and slot maps
// from request lengths, per-head norm + rotation + append, rows by slot.
#include <limits.h>

#include "common.cuh"
#include "kv4.cuh"
#include "kv4.h"

namespace nf {
namespace {

// ------------------------------------------------------------ block tables
//
// Three prefix sums over the requests (tokens, pages taken, pages given back)
// place everything.  A launch has to be one kernel, as a step's tables are a
// few microseconds of latency and no bandwidth: every CTA computes all the
// sums for itself (thread i the requests [i c, (i + 1) c), a block scan over the
// threads), then maps its own share of the tokens and of the requests.  No CTA
// reads what another one writes: the page of a token past the held ones comes
// from the ring, whose free part the call leaves alone, not from the table.
constexpr int BT_THREADS = 512;
constexpr int BT_WARPS = BT_THREADS / 32;

struct BtSeq {
  int held, len, ph, pl;  // positions and pages before and after
};
__device__ __forceinline__ BtSeq bt_seq(const BlockTableArgs& a, int s) {
  const long long most = static_cast<long long>(a.max_pages) * KV4_P;
  BtSeq r;
  r.held = static_cast<int>(min(static_cast<long long>(max(a.held[s], 0)), most));
  r.len = static_cast<int>(min(static_cast<long long>(max(a.seq_lens[s], 0)), most));
  r.ph = (r.held + KV4_P - 1) / KV4_P;
  r.pl = (r.len + KV4_P - 1) / KV4_P;
  return r;
}

struct BtSums {
  long long tok, take, back;
};

__global__ void __launch_bounds__(BT_THREADS) block_tables_kernel(const BlockTableArgs a) {
  __shared__ BtSums warp_sum[BT_WARPS + 1];
  __shared__ long long s_tok[BT_THREADS], s_take[BT_THREADS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = (a.n_seq + BT_THREADS - 1) / BT_THREADS;
  const long long first = static_cast<long long>(tid) * c;
  const int s0 = static_cast<int>(min(first, static_cast<long long>(a.n_seq)));
  const int s1 = static_cast<int>(min(first + c, static_cast<long long>(a.n_seq)));
  long long head = a.state_in[0] % a.num_pages;
  if (head < 0) head += a.num_pages;
  const long long count = min(max(a.state_in[1], 0), a.num_pages);

  BtSums own{0, 0, 0};
  for (int s = s0; s < s1; ++s) {
    const BtSeq q = bt_seq(a, s);
    own.tok += max(q.len - q.held, 0);
    own.take += max(q.pl - q.ph, 0);
    own.back += max(q.ph - q.pl, 0);
  }
  BtSums in = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, in.tok, o);
    const long long y = __shfl_up_sync(0xffffffffu, in.take, o);
    const long long z = __shfl_up_sync(0xffffffffu, in.back, o);
    if (lane >= o) {
      in.tok += x;
      in.take += y;
      in.back += z;
    }
  }
  if (lane == 31) warp_sum[warp + 1] = in;
  if (tid == 0) warp_sum[0] = BtSums{0, 0, 0};
  __syncthreads();
  if (tid < 3) {  // 16 warp totals: one thread a sum
    long long* p = &warp_sum[0].tok + tid;
    for (int w = 1; w <= BT_WARPS; ++w) p[3 * w] += p[3 * (w - 1)];
  }
  __syncthreads();
  BtSums at;  // before this thread's requests
  at.tok = warp_sum[warp].tok + in.tok - own.tok;
  at.take = warp_sum[warp].take + in.take - own.take;
  at.back = warp_sum[warp].back + in.back - own.back;
  s_tok[tid] = at.tok;
  s_take[tid] = at.take;
  const BtSums all = warp_sum[BT_WARPS];
  __syncthreads();
  const bool is_short = all.take > count;
  // page number i taken (i < count), and place i of the pages given back
  auto ring_at = [&](long long i) {
    const long long x = head + i;
    return static_cast<int>(x < a.num_pages ? x : x - a.num_pages);
  };

  if (blockIdx.x == 0 && tid == 0) {
    const long long back = is_short ? 0 : all.back;
    const long long left = count - (is_short ? 0 : all.take);
    a.state_out[0] = is_short ? static_cast<int>(head) : ring_at(all.take);
    a.state_out[1] = static_cast<int>(min(left + back, static_cast<long long>(a.num_pages)));
    a.state_out[2] = static_cast<int>(min(all.tok, static_cast<long long>(INT_MAX)));
    a.state_out[3] = static_cast<int>(
        min(max(all.take - count, 0LL), static_cast<long long>(INT_MAX)));
    a.tok_begin[a.n_seq] = a.state_out[2];
  }

  // requests: the warps take turns over the CTAs
  if (warp % gridDim.x == blockIdx.x) {
    for (int k = 0; k < c; ++k) {
      const bool live = s0 + k < s1;
      const int s = live ? s0 + k : 0;
      const BtSeq q = live ? bt_seq(a, s) : BtSeq{0, 0, 0, 0};
      const int grow = max(q.pl - q.ph, 0), back = max(q.ph - q.pl, 0);
      if (live) a.tok_begin[s] = static_cast<int>(min(at.tok, static_cast<long long>(INT_MAX)));
      // one entry, or `step`-strided entries from j0, of request r
      auto write = [&](int r, int ph, int pl, long long take, long long give, int j0, int step) {
        int* row = a.block_table + static_cast<size_t>(r) * a.max_pages;
        for (int j = ph + j0; j < pl; j += step)
          row[j] = is_short ? -1 : a.ring[ring_at(take + j - ph)];
        if (!is_short)
          for (int j = pl + j0; j < ph; j += step) {
            const long long to = count + give + j - pl;  // past the live part of the ring
            if (to < a.num_pages) a.ring[ring_at(to)] = row[j];
          }
      };
      const bool big = max(grow, back) > 4;
      if (live && !big) write(s, q.ph, q.pl, at.take, at.back, 0, 1);
      unsigned many = __ballot_sync(0xffffffffu, big);
      while (many) {  // a long request: the warp's lanes share its pages
        const int src = __ffs(many) - 1;
        many &= many - 1;
        const int r = __shfl_sync(0xffffffffu, s, src);
        const int ph = __shfl_sync(0xffffffffu, q.ph, src), pl = __shfl_sync(0xffffffffu, q.pl, src);
        const long long take = __shfl_sync(0xffffffffu, at.take, src);
        const long long give = __shfl_sync(0xffffffffu, at.back, src);
        write(r, ph, pl, take, give, lane, 32);
      }
      at.tok += max(q.len - q.held, 0);
      at.take += grow;
      at.back += back;
    }
  }

  // tokens
  const long long n = min(all.tok, static_cast<long long>(a.tok_cap));
  for (long long t = static_cast<long long>(blockIdx.x) * BT_THREADS + tid; t < n;
       t += static_cast<long long>(gridDim.x) * BT_THREADS) {
    int lo = 0, hi = BT_THREADS - 1;  // the last thread whose requests start at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_tok[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    long long tok = s_tok[lo], take = s_take[lo];
    int s = lo * c;
    BtSeq q = bt_seq(a, s);
    while (t - tok >= max(q.len - q.held, 0)) {  // ends: t lies in this thread's requests
      tok += max(q.len - q.held, 0);
      take += max(q.pl - q.ph, 0);
      q = bt_seq(a, ++s);
    }
    const int pos = q.held + static_cast<int>(t - tok), j = pos / KV4_P;
    int page;
    if (j < q.ph) page = a.block_table[static_cast<size_t>(s) * a.max_pages + j];
    else page = is_short ? -1 : a.ring[ring_at(take + j - q.ph)];
    a.tok_seq[t] = s;
    a.tok_pos[t] = pos;
    a.tok_slot[t] = page >= 0 && page < a.num_pages ? page * KV4_P + pos % KV4_P : -1;
  }
}

// --------------------------------------------- norm, rotation, append
//
// HBM-bound: every element of qkv is read once, q and the cache rows written
// once.  A head takes d / 16 lanes; each holds the 8 channels i and the 8
// channels i + d/2 that they rotate with, so a pair never leaves its lane and
// the loads and stores are 16 bytes.  The d/2 angles of a token are the same
// for all its heads: one thread each computes them once into shared memory.
//
// Rounding: q and k are normed and rotated in fp32 and rounded once.  A 4-bit
// code must not depend on how fp32 happened to round: where a K value or its
// block's largest lies within the fp32 error of a border between two codes
// (or two scales), the lane computes it again in fp64.  V comes in bf16, where
// the comparison is exact: 8 bits against borders of at most 7.
constexpr int QK_THREADS = 256;
constexpr int QK_MAX_TOK = 4;      // tokens a CTA handles at once
// Bound of the error of a rotated value relative to |a| + |b| of its pair: the
// tree sum of 16 squares a lane and 3 shuffles errs by 8 roundings of 2^-24,
// halved by the root; 1 / sqrt by two correctly rounded steps and the two
// products add 4, cos and sin 2^-22 with their angle, the rotation 2.
// 2^-24 (4 + 4 + 4 + 2) < 2^-20; doubled for safety.
constexpr float QK_ERR = 1.9073486e-6f;  // 2^-19

// Turns of 2^-64 that position pos makes, modulo one (negative ones backwards).
__device__ __forceinline__ uint64_t angle_turns(int pos, uint64_t freq) {
  return static_cast<uint64_t>(static_cast<int64_t>(pos)) * freq;
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  x[0] = bf16lo(u.x); x[1] = bf16hi(u.x); x[2] = bf16lo(u.y); x[3] = bf16hi(u.y);
  x[4] = bf16lo(u.z); x[5] = bf16hi(u.z); x[6] = bf16lo(u.w); x[7] = bf16hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// The scale byte for a block's largest magnitude t = a / 2^E, and its reciprocal.
__device__ __forceinline__ uint32_t scale_byte(float t) { return f32_to_e4m3(__fdiv_rn(t, 6.f)); }
__device__ __forceinline__ float scale_inv(uint32_t b) {
  const float s = e4m3_to_f32(b);
  return s > 0.f ? __fdiv_rn(1.f, s) : 0.f;  // a NaN or zero scale: zero codes
}

// Codes of 8 bf16-exact values x * 2^-E against the scale with reciprocal r.
// x has 8 significant bits and a border times the scale at most 7, so x / s is
// either exactly on a border or at least 2^-8 off it; x * r errs by 2^-23, and
// rounding the product to 16 bits restores exactly the ties.
__device__ __forceinline__ uint32_t codes_exact(const float (&x)[8], float mul, float r) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float u[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float p = x[i + k] * mul * r;
      u[k] = __uint_as_float((__float_as_uint(p) + 0x80u) & 0xFFFFFF00u);
    }
    // r = 0 marks a block of zero codes (0 * inf would be NaN)
    w |= (r > 0.f ? f32x2_to_e2m1x2(u[1], u[0]) : 0u) << (4 * i);
  }
  return w;
}

__device__ __forceinline__ float absmax8(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmax_nan(m, fabsf(x[i]));
  return m;
}

// To fp32 by rounding to odd: a later rounding to a few bits then gives what
// rounding x itself would, also where x lies next to a border.
__device__ __forceinline__ float to_f32_odd(double x) {
  const float f = __double2float_rz(x);
  return static_cast<double>(f) == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Everything a lane needs to form its pairs again in fp64.
struct QkLane {
  uint4 lo, hi;          // raw bf16 channels i .. i + 7 and i + d/2 .. (the head's row)
  const uint4* gain;     // the head's gain at this lane's channels (lo), NULL: none
  int gain_hi;           // uint4 offset of the hi channels' gain
  int pos, i0;           // position; first channel
  double r;              // 1 / sqrt(mean + eps)
};
__device__ __noinline__ void pair_f64(const QkLane& q, const RopeFreq& f, int i, double* lo,
                                      double* hi) {
  float a8[8], b8[8];
  unpack8(q.lo, a8);
  unpack8(q.hi, b8);
  double a = 0, b = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k == i) {
      a = a8[k];
      b = b8[k];
    }
  if (q.gain) {
    float g8[8], h8[8];
    unpack8(q.gain[0], g8);
    unpack8(q.gain[q.gain_hi], h8);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k == i) {
        a *= q.r * g8[k];
        b *= q.r * h8[k];
      }
  }
  const int64_t turn = static_cast<int64_t>(angle_turns(q.pos, f.freq[q.i0 + i]));
  double s, c;
  sincospi(static_cast<double>(turn) * 0x1p-63, &s, &c);
  *lo = a * c - b * s;
  *hi = b * c + a * s;
}

// Which of the 8 codes and scales an fp32 decision cannot settle.  x: values,
// e: their error bounds, t: the block's largest magnitude, te: its error.
__device__ __forceinline__ bool scale_open(float t, float te, float mul) {
  return scale_byte((t - te) * mul) != scale_byte((t + te) * mul);
}
__device__ __forceinline__ uint32_t codes_f32(const float (&x)[8], const float (&e)[8], float mul,
                                              float r, uint32_t* open) {
  uint32_t w = 0, o = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float u0 = x[i] * mul * r, u1 = x[i + 1] * mul * r;
    const float d0 = fmaf(fabsf(u0), 2.4e-7f, e[i] * mul * r), d1 = fmaf(fabsf(u1), 2.4e-7f, e[i + 1] * mul * r);
    const uint32_t a = f32x2_to_e2m1x2(u1 - d1, u0 - d0), b = f32x2_to_e2m1x2(u1 + d1, u0 + d0);
    w |= a << (4 * i);
    o |= (a ^ b) << (4 * i);
  }
  if (!(r > 0.f)) w = o = 0;
  *open = o;
  return w;
}

template <int D, bool FP4>
__global__ void __launch_bounds__(QK_THREADS)
    qk_norm_rope_kernel(const QkNormRopeArgs a, const __grid_constant__ RopeFreq f, int tok_cta) {
  constexpr int LPH = D / 16;         // lanes of a head
  constexpr int HPW = 32 / LPH;       // heads of a warp
  constexpr int HALF = D / 2;
  __shared__ __align__(16) float2 cs[QK_MAX_TOK][HALF];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hl = lane / LPH, l = lane % LPH;  // head of the warp, lane of the head
  const int t0 = blockIdx.x * tok_cta, nt = min(tok_cta, a.n_tok - t0);
  for (int k = threadIdx.x; k < nt * HALF; k += QK_THREADS) {
    const int t = k / HALF, i = k % HALF;
    const uint64_t turn = angle_turns(a.tok_pos[t0 + t], f.freq[i]);
    // the angle in units of 2^-31 pi: 24 bits through sincospif, and a
    // first-order step (below 10^-6) for the rest
    const int hi = static_cast<int>(turn >> 32);
    const float x = __int2float_rz(hi);
    const float rest = static_cast<float>(hi - static_cast<int>(x)) + static_cast<float>(static_cast<uint32_t>(turn)) * 0x1p-32f;
    float s, c;
    sincospif(x * (1.f / 2147483648.f), &s, &c);
    const float d = rest * (3.14159265f / 2147483648.f);
    cs[t][i] = make_float2(fmaf(-s, d, c), fmaf(c, d, s));
  }
  __syncthreads();
  const int heads = a.n_q + 2 * a.n_kv;
  const int groups = (heads + HPW - 1) / HPW;
  for (int it = warp; it < nt * groups; it += QK_THREADS / 32) {
    const int tl = it / groups, t = t0 + tl;
    const int h = (it % groups) * HPW + hl;
    const bool live = h < heads;
    const int hh = live ? h : heads - 1;  // idle lanes shadow the last head and store nothing
    const uint4* row = reinterpret_cast<const uint4*>(a.qkv + static_cast<size_t>(t) * a.ld + static_cast<size_t>(hh) * D);
    const uint4 ulo = row[l], uhi = row[LPH + l];
    const bool is_q = hh < a.n_q, is_v = hh >= a.n_q + a.n_kv;
    float lo[8], hi[8];
    unpack8(ulo, lo);
    unpack8(uhi, hi);
    const __nv_bfloat16* gain = is_q ? a.q_gain : is_v ? nullptr : a.k_gain;
    const uint4* g4 = gain ? reinterpret_cast<const uint4*>(gain) + l : nullptr;
    // sum of squares (every lane: the shuffles are the warp's)
    float sq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sq[i] = fmaf(lo[i], lo[i], hi[i] * hi[i]);
    float ss = ((sq[0] + sq[1]) + (sq[2] + sq[3])) + ((sq[4] + sq[5]) + (sq[6] + sq[7]));
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (g4) {
      const float r = __fdiv_rn(1.f, __fsqrt_rn(ss * (1.f / D) + a.eps));
      float g[8];
      unpack8(g4[0], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) lo[i] = lo[i] * r * g[i];
      unpack8(g4[LPH], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) hi[i] = hi[i] * r * g[i];
    }
    float err[8];
    if (!is_v) {
      const float4* c4 = reinterpret_cast<const float4*>(&cs[tl][8 * l]);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float4 c = c4[i / 2];
        const float x0 = lo[i], y0 = hi[i], x1 = lo[i + 1], y1 = hi[i + 1];
        err[i] = QK_ERR * (fabsf(x0) + fabsf(y0));
        err[i + 1] = QK_ERR * (fabsf(x1) + fabsf(y1));
        lo[i] = x0 * c.x - y0 * c.y;
        hi[i] = y0 * c.x + x0 * c.y;
        lo[i + 1] = x1 * c.z - y1 * c.w;
        hi[i + 1] = y1 * c.z + x1 * c.w;
      }
    }
    if (is_q && live) {
      uint4* out = reinterpret_cast<uint4*>(a.q + (static_cast<size_t>(t) * a.n_q + hh) * D);
      out[l] = pack8(lo);
      out[LPH + l] = pack8(hi);
    }
    const int slot = a.tok_slot[t];
    const bool store = live && !is_q && slot >= 0 && slot < a.num_pages * KV4_P;
    const int page = store ? slot / KV4_P : 0, prow = store ? slot % KV4_P : 0;
    const int kvh = is_q ? 0 : is_v ? hh - a.n_q - a.n_kv : hh - a.n_q;
    if (!FP4) {
      if (store) {
        __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(is_v ? a.v_pool : a.k_pool);
        uint4* out = reinterpret_cast<uint4*>(
            pool + ((static_cast<size_t>(page) * a.n_kv + kvh) * KV4_P + prow) * D);
        out[l] = is_v ? ulo : pack8(lo);
        out[LPH + l] = is_v ? uhi : pack8(hi);
      }
      continue;
    }
    if (__all_sync(0xffffffffu, is_q)) continue;  // no K or V among the warp's heads
    // 4 bits: a block is two neighbouring lanes, lo and hi halves separately
    const float mul = exp2_int(-(is_v ? a.v_exp : a.k_exp));
    float tlo = absmax8(lo), thi = absmax8(hi);
    tlo = fmax_nan(tlo, __shfl_xor_sync(0xffffffffu, tlo, 1));
    thi = fmax_nan(thi, __shfl_xor_sync(0xffffffffu, thi, 1));
    uint32_t blo = scale_byte(tlo * mul), bhi = scale_byte(thi * mul);
    uint32_t wlo, whi;
    if (is_v || is_q) {
      wlo = codes_exact(lo, mul, scale_inv(blo));
      whi = codes_exact(hi, mul, scale_inv(bhi));
    }
    uint32_t olo = 0, ohi = 0;
    bool slo = false, shi = false;
    if (!is_v && !is_q) {
      float e = err[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) e = fmaxf(e, err[i]);
      slo = scale_open(tlo, e, mul);
      shi = scale_open(thi, e, mul);
      wlo = codes_f32(lo, err, mul, scale_inv(blo), &olo);
      whi = codes_f32(hi, err, mul, scale_inv(bhi), &ohi);
    }
    slo |= __shfl_xor_sync(0xffffffffu, slo, 1);
    shi |= __shfl_xor_sync(0xffffffffu, shi, 1);
    if (__any_sync(0xffffffffu, olo || ohi || slo || shi)) {
      QkLane q;
      q.lo = ulo;
      q.hi = uhi;
      q.gain = g4;
      q.gain_hi = LPH;
      q.pos = a.tok_pos[t];
      q.i0 = 8 * l;
      float x[8], y[8];
      unpack8(ulo, x);
      unpack8(uhi, y);
      double sd = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        sd += static_cast<double>(x[i]) * x[i] + static_cast<double>(y[i]) * y[i];
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) sd += __shfl_xor_sync(0xffffffffu, sd, o);
      q.r = 1.0 / sqrt(sd / D + static_cast<double>(a.eps));
      double mlo = 0, mhi = 0;  // exact largest magnitudes of open blocks
      for (int i = 0; i < 8; ++i) {
        if (!(slo || shi)) continue;
        double u, v;
        pair_f64(q, f, i, &u, &v);
        mlo = fmax(mlo, fabs(u));
        mhi = fmax(mhi, fabs(v));
      }
      mlo = fmax(mlo, __shfl_xor_sync(0xffffffffu, mlo, 1));
      mhi = fmax(mhi, __shfl_xor_sync(0xffffffffu, mhi, 1));
      if (slo) blo = f32_to_e4m3(to_f32_odd(mlo * mul / 6.0));
      if (shi) bhi = f32_to_e4m3(to_f32_odd(mhi * mul / 6.0));
      const float rlo = scale_inv(blo), rhi = scale_inv(bhi);
      if (slo) wlo = codes_f32(lo, err, mul, rlo, &olo);
      if (shi) whi = codes_f32(hi, err, mul, rhi, &ohi);
      for (int i = 0; i < 8; ++i) {
        const uint32_t nib = 0xFu << (4 * i);
        if (!((olo | ohi) & nib)) continue;
        double u, v;
        pair_f64(q, f, i, &u, &v);
        if (olo & nib)
          wlo = (wlo & ~nib) | ((f32x2_to_e2m1x2(0.f, to_f32_odd(u * mul / e4m3_to_f32(blo))) & 0xFu) << (4 * i));
        if (ohi & nib)
          whi = (whi & ~nib) | ((f32x2_to_e2m1x2(0.f, to_f32_odd(v * mul / e4m3_to_f32(bhi))) & 0xFu) << (4 * i));
      }
    }
    if (store) {
      uint8_t* part = static_cast<uint8_t*>(a.k_pool) +
                      ((static_cast<size_t>(page) * a.n_kv + kvh) * 2 + (is_v ? 1 : 0)) * kv4_part_bytes(D);
      uint32_t* codes = reinterpret_cast<uint32_t*>(part + prow * (D / 2));
      codes[l] = wlo;
      codes[LPH + l] = whi;
      uint8_t* sc = part + 8 * D + prow * (D / 16);
      if ((l & 1) == 0) {
        sc[l / 2] = static_cast<uint8_t>(blo);
        sc[D / 32 + l / 2] = static_cast<uint8_t>(bhi);
      }
    }
  }
}

// ------------------------------------------------------------ rows by slot
//
// HBM-bound: a thread takes one block of 16 channels of K and the same of V
// (8 code bytes and a scale each), so neighbouring threads read and write
// neighbouring bytes and the stores are 16 bytes wide.
constexpr int RD_THREADS = 256;

// 16 codes under scale byte `b`, times 2^E: exact in fp32, rounded to bf16 only
// where 2^E leaves bf16's range.
__device__ __forceinline__ void block_to_bf16(uint2 w, uint32_t b, float mul, uint4* out) {
  const float s = e4m3_to_f32(b) * mul;
  const uint32_t word[2] = {w.x, w.y};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 x0 = f16x2_to_f32x2(e2m1_to_f16x2<0>(word[k])), x1 = f16x2_to_f32x2(e2m1_to_f16x2<1>(word[k]));
    const float2 x2 = f16x2_to_f32x2(e2m1_to_f16x2<2>(word[k])), x3 = f16x2_to_f32x2(e2m1_to_f16x2<3>(word[k]));
    out[k] = make_uint4(pack_bf16(x0.x * s, x0.y * s), pack_bf16(x1.x * s, x1.y * s),
                        pack_bf16(x2.x * s, x2.y * s), pack_bf16(x3.x * s, x3.y * s));
  }
}

template <int D>
__global__ void __launch_bounds__(RD_THREADS)
    kv4_read_kernel(const uint8_t* __restrict__ pool, int num_pages, int n_kv,
                    const int* __restrict__ slots, int n, float k_mul, float v_mul,
                    __nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ v) {
  const int bpt = n_kv * (D / 16);  // blocks of a token
  const long long total = static_cast<long long>(n) * bpt;
  for (long long i = static_cast<long long>(blockIdx.x) * RD_THREADS + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * RD_THREADS) {
    const int t = static_cast<int>(i / bpt), b = static_cast<int>(i % bpt);
    const int h = b / (D / 16), c = b % (D / 16);
    const int slot = slots[t];
    uint4 x[2] = {}, y[2] = {};
    if (slot >= 0 && slot < num_pages * KV4_P) {
      const uint8_t* part = pool + (static_cast<size_t>(slot / KV4_P) * n_kv + h) * 2 * kv4_part_bytes(D);
      const int row = slot % KV4_P;
      const uint8_t* code = part + row * (D / 2) + c * 8;
      const uint8_t* sc = part + 8 * D + row * (D / 16) + c;
      const uint2 kw = *reinterpret_cast<const uint2*>(code);
      const uint2 vw = *reinterpret_cast<const uint2*>(code + kv4_part_bytes(D));
      const uint32_t ks = sc[0], vs = sc[kv4_part_bytes(D)];
      block_to_bf16(kw, ks, k_mul, x);
      block_to_bf16(vw, vs, v_mul, y);
    }
    uint4* ko = reinterpret_cast<uint4*>(k) + i * 2;
    uint4* vo = reinterpret_cast<uint4*>(v) + i * 2;
    ko[0] = x[0];
    ko[1] = x[1];
    vo[0] = y[0];
    vo[1] = y[1];
  }
}

}  // namespace

cudaError_t launch_block_tables(const BlockTableArgs& a, int num_sms, cudaStream_t stream) {
  // a CTA for every 2048 tokens the caller has room for
  int grid = (a.tok_cap + 2047) / 2048;
  grid = grid < 1 ? 1 : grid > num_sms ? num_sms : grid;
  block_tables_kernel<<<grid, BT_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs& a, const RopeFreq& f, bool fp4, int num_sms,
                                cudaStream_t stream) {
  // one token a CTA until that fills the GPU, then up to 4, which share a
  // round of angles
  int tok = a.n_tok / (num_sms * 4);
  tok = tok < 1 ? 1 : tok > QK_MAX_TOK ? QK_MAX_TOK : tok;
  const int grid = (a.n_tok + tok - 1) / tok;
  if (a.head_dim == 128) {
    if (fp4) qk_norm_rope_kernel<128, true><<<grid, QK_THREADS, 0, stream>>>(a, f, tok);
    else qk_norm_rope_kernel<128, false><<<grid, QK_THREADS, 0, stream>>>(a, f, tok);
  } else {
    if (fp4) qk_norm_rope_kernel<64, true><<<grid, QK_THREADS, 0, stream>>>(a, f, tok);
    else qk_norm_rope_kernel<64, false><<<grid, QK_THREADS, 0, stream>>>(a, f, tok);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const uint8_t* pool, int num_pages, int n_kv, int head_dim,
                            const int* slots, int n, int k_exp, int v_exp, __nv_bfloat16* k,
                            __nv_bfloat16* v, int num_sms, cudaStream_t stream) {
  const long long total = static_cast<long long>(n) * n_kv * (head_dim / 16);
  const long long want = (total + RD_THREADS - 1) / RD_THREADS;
  const int grid = static_cast<int>(want < num_sms * 8LL ? want : num_sms * 8LL);
  const float km = exp2_int(k_exp), vm = exp2_int(v_exp);
  if (head_dim == 128)
    kv4_read_kernel<128><<<grid, RD_THREADS, 0, stream>>>(pool, num_pages, n_kv, slots, n, km, vm, k, v);
  else
    kv4_read_kernel<64><<<grid, RD_THREADS, 0, stream>>>(pool, num_pages, n_kv, slots, n, km, vm, k, v);
  return cudaGetLastError();
}

}  // namespace nf
