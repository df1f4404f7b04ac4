// The small operators around the 4-bit KV cache: block tables and slot maps
// from request lengths, per-head norm + rotation + append, rows by slot.
#include <limits.h>

#include "common.cuh"
#include "dd.cuh"
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
// Measured: 64 requests of one token 6.0 us, 1801 requests 8.2, 4096 with 1024
// prompts of 1000 tokens 16.4 (9.8 MB: 1.4 us of copy rate).  What bounds it is
// latency: the sums over the requests, then one round of table reads a block of
// tokens, while the same warps move the prompts' pages.
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

// Pages a lane moves by itself; more take a warp.  With three CTAs for 1801
// requests and four an SM for 4096, at 0 (a warp for every request), 4 and no limit:
// 12.3, 10.3, 20.5 us for 1801 with two prompts; 28.7, 27.8, 47.0 for 4096 with 1024.
constexpr int BT_FEW = 4;
constexpr int BT_PER = 4;                        // tokens of a thread and block
constexpr int BT_TOKENS = BT_THREADS * BT_PER;
constexpr int BT_REQS = 32;                      // requests for each of which a launch has a CTA at least

// What the tokens of a request in a block of tokens need: the request, the
// position of its first token there, the pages it held, those taken before it.
struct __align__(16) BtNote {
  int seq, pos, ph, take;
};

struct BtSums {
  long long tok, take, back;
};

__global__ void __launch_bounds__(BT_THREADS) block_tables_kernel(const BlockTableArgs a) {
  __shared__ BtSums warp_sum[BT_WARPS + 1];
  __shared__ long long s_tok[BT_THREADS], s_take[BT_THREADS], s_back[BT_THREADS];
  __shared__ BtNote s_note[BT_TOKENS];
  __shared__ int s_place[BT_TOKENS], s_top[BT_WARPS];
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
  s_back[tid] = at.back;
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

  // Entries of `step`-strided pages from j0 of request r.
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
  // Requests that move a few pages, a lane each; the CTAs take the k-th requests
  // of the warps' lanes in turn.
  for (int k = 0; k < c; ++k) {
    if (s0 + k >= s1) break;
    const int s = s0 + k;
    const BtSeq q = bt_seq(a, s);
    const int grow = max(q.pl - q.ph, 0), back = max(q.ph - q.pl, 0);
    if ((warp * c + k) % gridDim.x == blockIdx.x) {
      a.tok_begin[s] = static_cast<int>(min(at.tok, static_cast<long long>(INT_MAX)));
      if (max(grow, back) <= BT_FEW) write(s, q.ph, q.pl, at.take, at.back, 0, 1);
    }
    at.tok += max(q.len - q.held, 0);
    at.take += grow;
    at.back += back;
  }
  // Requests that move more, a warp each: a warp looks through its share, up to 32
  // at a time.
  const long long warps = static_cast<long long>(gridDim.x) * BT_WARPS;
  const int share = static_cast<int>(min((a.n_seq + warps - 1) / warps, 32ll));
  for (long long w0 = (static_cast<long long>(blockIdx.x) * BT_WARPS + warp) * share; w0 < a.n_seq; w0 += warps * share) {
    const int mine = static_cast<int>(min(w0 + lane, static_cast<long long>(a.n_seq - 1)));
    const BtSeq m = bt_seq(a, mine);
    unsigned many = __ballot_sync(0xffffffffu, lane < share && w0 + lane < a.n_seq && max(m.pl - m.ph, m.ph - m.pl) > BT_FEW);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const int s = static_cast<int>(w0) + src, own = s / c;
      const int ph = __shfl_sync(0xffffffffu, m.ph, src), pl = __shfl_sync(0xffffffffu, m.pl, src);
      long long take = 0, give = 0;
      for (int r = own * c + lane; r < s; r += 32) {
        const BtSeq p = bt_seq(a, r);
        take += max(p.pl - p.ph, 0);
        give += max(p.ph - p.pl, 0);
      }
      if (c > 1) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          take += __shfl_xor_sync(0xffffffffu, take, o);
          give += __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
      write(s, ph, pl, s_take[own] + take, s_back[own] + give, lane, 32);
    }
  }

  // Tokens, BT_TOKENS at a time.  The thread that owns a request notes at the
  // place of its first token in the block (or at place 0, if it began earlier)
  // what its tokens need; a running maximum over the places then tells every
  // token its request's place.
  const long long n = min(all.tok, static_cast<long long>(a.tok_cap));
  for (long long t0 = static_cast<long long>(blockIdx.x) * BT_TOKENS; t0 < n;
       t0 += static_cast<long long>(gridDim.x) * BT_TOKENS) {
    __syncthreads();  // the previous block's places are read
#pragma unroll
    for (int k = 0; k < BT_PER; ++k) s_place[tid * BT_PER + k] = 0;
    __syncthreads();
    long long tok = s_tok[tid], take = s_take[tid];
    const long long to = tid + 1 < BT_THREADS ? s_tok[tid + 1] : all.tok;
    if (tok < t0 + BT_TOKENS && to > t0)
      for (int s = s0; s < s1 && tok < t0 + BT_TOKENS; ++s) {
        const BtSeq q = bt_seq(a, s);
        const int m = max(q.len - q.held, 0);
        if (m > 0 && tok + m > t0) {
          const int at_place = static_cast<int>(max(tok - t0, 0ll));
          s_place[at_place] = at_place;
          s_note[at_place] = BtNote{s, static_cast<int>(q.held + max(t0 - tok, 0ll)), q.ph, static_cast<int>(take)};
        }
        tok += m;
        take += max(q.pl - q.ph, 0);
      }
    __syncthreads();
    // running maximum: this thread's BT_PER places, then over the threads
    int place[BT_PER], top = 0;
#pragma unroll
    for (int k = 0; k < BT_PER; ++k) place[k] = top = max(top, s_place[tid * BT_PER + k]);
    int in_top = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, in_top, o);
      if (lane >= o) in_top = max(in_top, y);
    }
    if (lane == 31) s_top[warp] = in_top;
    int before = __shfl_up_sync(0xffffffffu, in_top, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before = max(before, s_top[w]);
#pragma unroll
    for (int k = 0; k < BT_PER; ++k) s_place[tid * BT_PER + k] = max(before, place[k]);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < BT_PER; ++k) {
      const int i = k * BT_THREADS + tid;
      const long long t = t0 + i;
      if (t >= n) break;
      const int pl = s_place[i];
      const BtNote q = s_note[pl];
      const int pos = q.pos + i - pl, j = pos / KV4_P;
      int page;
      if (j < q.ph) page = a.block_table[static_cast<size_t>(q.seq) * a.max_pages + j];
      else page = is_short ? -1 : a.ring[ring_at(static_cast<long long>(q.take) + j - q.ph)];
      a.tok_seq[t] = q.seq;
      a.tok_pos[t] = pos;
      a.tok_slot[t] = page >= 0 && page < a.num_pages ? page * KV4_P + pos % KV4_P : -1;
    }
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
// block's largest lies within the fp32 error of a border between two codes (or
// two scales), about one head in two hundred, the lane computes it again in
// pairs of floats (dd.cuh).  V comes in bf16, where the comparison is exact: 8
// bits against borders of at most 7.
//
// Measured: 64 tokens of 32 + 8 + 8 heads of 128 into 4 bits 6 us, into bf16 2048
// tokens 16.4 us (50 MB: 7.4 at the copy rate): 512 CTAs of 4 tokens, 304 of which
// are resident at 106 registers, so 1.7 waves of 16 warps an SM, which memory latency
// bounds.  8191 tokens of 64 + 8 + 8 heads
// into 4 bits: 28 us for keys and values, which are bound by issue (the codes'
// and borders' arithmetic), then 46 us for the queries at 64 % of the DRAM rate.
constexpr int QK_THREADS = 256;
constexpr int QK_MAX_TOK = 8;      // tokens a CTA handles at once: 1, 2, 4 or 8, a power of two
// Bound of the error of a rotated value relative to |a| + |b| of its pair, in
// roundings of 2^-24: the tree sum of 16 squares a lane and 3 shuffles errs by 8,
// halved by the root; the mean and eps 1; rsqrtf, 2 units in the last place, 4;
// the two products 2; cos and sin with their angle 4; the rotation 2: 17 in
// all, a little over 2^-20.
constexpr float QK_ERR = 1.2e-6f;  // 20 x 2^-24

// Turns of 2^-64 that position pos makes, modulo one (negative ones backwards).
__device__ __forceinline__ uint64_t angle_turns(int pos, uint64_t freq) {
  return static_cast<uint64_t>(static_cast<int64_t>(pos)) * freq;
}
// An error bound, or none beside an infinity or a NaN, which rounding leaves alone.
__device__ __forceinline__ float finite_or_0(float d) { return d < 3e38f ? d : 0.f; }
// x rounded to 16 significant bits.
__device__ __forceinline__ float snap16(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x80u) & 0xFFFFFF00u);
}
// Scale byte of a block of bf16-exact values with largest magnitude t = a / 2^E.
// 8 significant bits against a border times 6 of at most 7: t / 6 is on a border
// between two scales or at least 2^-8 off it, and t times 1/6 errs by 2^-23, so
// 16 bits of the product restore exactly the ties.
__device__ __forceinline__ uint32_t scale_byte_exact(float t) {
  return t == t ? f32_to_e4m3(snap16(t * (1.f / 6.f))) : 0x7Fu;
}
// The same of a value known to +- e; *open where that leaves two bytes.
__device__ __forceinline__ uint32_t scale_byte_near(float t, float e, bool* open) {
  const float d = finite_or_0(fmaf(t, 2.4e-7f, e));  // and the product's rounding
  const uint32_t lo = f32_to_e4m3((t - d) * (1.f / 6.f)), hi = f32_to_e4m3((t + d) * (1.f / 6.f));
  *open = lo != hi;
  return hi;
}
// 1 / scale, to 2^-22; a NaN or zero scale: 0, which makes zero codes.
__device__ __forceinline__ float scale_inv(uint32_t b) {
  const float s = e4m3_to_f32(b);
  return s > 0.f ? __frcp_rn(s) : 0.f;
}

// Eight codes with the signs of zeros taken off: a zero is stored one way.
__device__ __forceinline__ uint32_t plain_zeros(uint32_t w) {
  const uint32_t m = w | (w >> 1) | (w >> 2);
  return w & (0x77777777u | ((m & 0x11111111u) << 3));
}

// Codes of 8 bf16-exact values times r = 2^-E / scale: as for the scale, 16 bits
// of the product restore exactly the ties.
__device__ __forceinline__ uint32_t codes_exact(const float2 (&x)[4], float r) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = __fmul2_rn(x[i], make_float2(r, r));
    w |= f32x2_to_e2m1x2(snap16(u.y), snap16(u.x)) << (8 * i);
  }
  return r > 0.f ? plain_zeros(w) : 0u;  // (0 times inf is NaN)
}

__device__ __forceinline__ float absmax8(const float2 (&x)[4]) {
  float m = fmax_nan(fabsf(x[0].x), fabsf(x[0].y));
#pragma unroll
  for (int i = 1; i < 4; ++i) m = fmax_nan(m, fmax_nan(fabsf(x[i].x), fabsf(x[i].y)));
  return m;
}

// Sign of v - b.
__device__ __forceinline__ int dd_side(dd v, float b) {
  const dd d = dd_add(v, dd{-b, 0.f});
  return d.h > 0.f ? 1 : d.h < 0.f ? -1 : 0;
}
// Nearest of the magnitudes grid(0) < grid(1) < ... < grid(last) to v * mul / s,
// ties to the even index, from the index k that fp32 gave (at most one off).
// Every product grid * s is exact: 2 to 5 bits by 4, or by 6.
template <typename Grid>
__device__ __forceinline__ uint32_t dd_nearest(dd v, float s, uint32_t k, uint32_t last, Grid grid) {
  if (k < last) {
    const int up = dd_side(v, 0.5f * (grid(k) + grid(k + 1)) * s);
    if (up > 0 || (up == 0 && (k & 1))) return k + 1;
  }
  if (k > 0) {
    const int down = dd_side(v, 0.5f * (grid(k - 1) + grid(k)) * s);
    if (down < 0 || (down == 0 && (k & 1))) return k - 1;
  }
  return k;
}
// Code of v (times 2^-E already) under the scale with byte b.
__device__ __forceinline__ uint32_t dd_code(dd v, uint32_t b) {
  const float s = e4m3_to_f32(b);
  if (!(s > 0.f)) return 0;
  const uint32_t sign = signbit(v.h) ? 8u : 0u;
  if (sign) v = dd_neg(v);
  const uint32_t k = f32x2_to_e2m1x2(0.f, __fdiv_rn(v.h, s)) & 7u;
  const uint32_t n = dd_nearest(v, s, k, 7, [](uint32_t i) { return i < 4 ? 0.5f * i : i < 6 ? i - 2.f : 2.f * i - 8.f; });
  return n ? sign | n : 0;
}
// Scale byte of a block with largest magnitude t (times 2^-E already).
__device__ __forceinline__ uint32_t dd_scale(dd t) {
  const uint32_t k = f32_to_e4m3(t.h * (1.f / 6.f));
  return k == 0x7Fu ? k : dd_nearest(t, 6.f, k, 126, [](uint32_t i) { return e4m3_to_f32(i); });
}

// What a lane needs to form its pairs again.
struct QkLane {
  uint4 lo, hi;          // raw bf16 channels i .. i + 7 and i + d/2 .. (the head's row)
  const uint4* gain;     // the head's gain at this lane's channels (lo), NULL: none
  int gain_hi;           // uint4 offset of the hi channels' gain
  int pos, i0;           // position; first channel
};
// Pair i of the lane, normed by r, rotated, times mul.
__device__ __forceinline__ void dd_pair(const QkLane& q, const RopeFreq& f, dd r, float mul, int i, dd* lo, dd* hi) {
  auto pick = [&](const uint4& u) {
    const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
    return (i & 1) ? bf16hi(w) : bf16lo(w);
  };
  dd a = {pick(q.lo), 0.f}, b = {pick(q.hi), 0.f};
  if (q.gain) {
    a = dd_mul(dd_mul(r, a.h), pick(q.gain[0]));
    b = dd_mul(dd_mul(r, b.h), pick(q.gain[q.gain_hi]));
  }
  dd c, s;
  dd_cos_sin(angle_turns(q.pos, f.freq[q.i0 + i]), &c, &s);
  *lo = dd_add(dd_mul(a, c), dd_neg(dd_mul(b, s)));
  *hi = dd_add(dd_mul(b, c), dd_mul(a, s));
  lo->h *= mul;
  lo->l *= mul;
  hi->h *= mul;
  hi->l *= mul;
}

// Codes of 8 values times r = 2^-E / scale, the values known to QK_ERR of sum;
// open: nibbles of those that lie within that of a border.
__device__ __forceinline__ uint32_t codes_near(const float2 (&x)[4], const float2 (&sum)[4], float r, uint32_t* open) {
  uint32_t below = 0, above = 0;
  const float2 r2 = make_float2(r, r), e2 = make_float2(r * QK_ERR, r * QK_ERR), one = make_float2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = __fmul2_rn(x[i], r2);
    float2 d = __ffma2_rn(make_float2(fabsf(u.x), fabsf(u.y)), make_float2(4.8e-7f, 4.8e-7f), __fmul2_rn(sum[i], e2));
    d.x = finite_or_0(d.x);
    d.y = finite_or_0(d.y);
    const float2 dn = __ffma2_rn(d, one, u), up = __fadd2_rn(u, d);
    below |= f32x2_to_e2m1x2(dn.y, dn.x) << (8 * i);
    above |= f32x2_to_e2m1x2(up.y, up.x) << (8 * i);
  }
  if (!(r > 0.f)) below = above = 0;
  below = plain_zeros(below);
  *open = below ^ plain_zeros(above);
  return below;
}

// 1 / sqrt(mean + eps) of the head, in pairs of floats: the squares of 8 bits are
// exact, the sums a tree.
template <int D>
__device__ __forceinline__ dd dd_norm(const QkLane& q, float eps) {
  const uint32_t raw[8] = {q.lo.x, q.lo.y, q.lo.z, q.lo.w, q.hi.x, q.hi.y, q.hi.z, q.hi.w};
  dd t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = dd_two_sum(bf16lo(raw[i]) * bf16lo(raw[i]), bf16hi(raw[i]) * bf16hi(raw[i]));
#pragma unroll
  for (int n = 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = dd_add(t[i], t[i + n]);
  dd ss = t[0];
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1)
    ss = dd_add(ss, dd{__shfl_xor_sync(0xffffffffu, ss.h, o), __shfl_xor_sync(0xffffffffu, ss.l, o)});
  return dd_rsqrt(dd_add(dd{ss.h * (1.f / D), ss.l * (1.f / D)}, dd{eps, 0.f}));
}

// What fp32 left open.  Every lane of the warp calls (shuffles); arguments by
// value, so that the callers' values stay in registers where nothing is open.
//
// Scale bytes (lo in the low byte, hi in the next) from the values of the bits in
// lo, hi, the only ones that may be their block's largest.
template <int D>
__device__ __noinline__ uint32_t settle_scales(QkLane q, const RopeFreq& f, float eps, float mul, uint32_t lo, uint32_t hi) {
  const dd r = dd_norm<D>(q, eps);
  auto larger = [](dd a, dd b) { return dd_add(b, dd_neg(a)).h > 0.f ? b : a; };
  auto mag = [](dd a) { return a.h < 0.f ? dd_neg(a) : a; };
  dd mlo = {0.f, 0.f}, mhi = {0.f, 0.f};
  for (uint32_t any = lo | hi; any; any &= any - 1) {
    const int i = __ffs(any) - 1;
    dd u, v;
    dd_pair(q, f, r, mul, i, &u, &v);
    if ((lo >> i) & 1) mlo = larger(mlo, mag(u));
    if ((hi >> i) & 1) mhi = larger(mhi, mag(v));
  }
  __syncwarp();
  mlo = larger(mlo, dd{__shfl_xor_sync(0xffffffffu, mlo.h, 1), __shfl_xor_sync(0xffffffffu, mlo.l, 1)});
  mhi = larger(mhi, dd{__shfl_xor_sync(0xffffffffu, mhi.h, 1), __shfl_xor_sync(0xffffffffu, mhi.l, 1)});
  return dd_scale(mlo) | (dd_scale(mhi) << 8);
}
// The codes of the nibbles that lo, hi mark, under the scale bytes blo, bhi, in
// the words wlo, whi.
template <int D>
__device__ __noinline__ uint2 settle_codes(QkLane q, const RopeFreq& f, float eps, float mul, uint32_t lo, uint32_t hi, uint32_t blo,
                                           uint32_t bhi, uint32_t wlo, uint32_t whi) {
  const dd r = dd_norm<D>(q, eps);
  for (uint32_t any = lo | hi; any;) {
    const int i = (__ffs(any) - 1) / 4;
    const uint32_t nib = 0xFu << (4 * i);
    any &= ~nib;
    dd u, v;
    dd_pair(q, f, r, mul, i, &u, &v);
    if (lo & nib) wlo = (wlo & ~nib) | (dd_code(u, blo) << (4 * i));
    if (hi & nib) whi = (whi & ~nib) | (dd_code(v, bhi) << (4 * i));
  }
  __syncwarp();
  return make_uint2(wlo, whi);
}
// Bits of the values that may be the largest of a block whose largest is near t.
__device__ __forceinline__ uint32_t near_largest(const float2 (&x)[4], float t) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m |= (fabsf(x[i].x) >= t ? 1u : 0u) << (2 * i) | (fabsf(x[i].y) >= t ? 2u : 0u) << (2 * i);
  return m;
}

// Two values at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 bf16x2_f32(uint32_t v) { return make_float2(bf16lo(v), bf16hi(v)); }

// A group of the warp's heads that are all queries: norm, rotation, one rounding.
// c, s: cos and sin of this lane's 8 angles.
template <int D>
__device__ __forceinline__ void q_group(const uint4& ulo, const uint4& uhi, const uint4& glo, const uint4& ghi, bool norm,
                                        float eps, const float2 (&c)[4], const float2 (&s)[4], uint4* out, bool live) {
  constexpr int LPH = D / 16;
  const uint32_t wl[4] = {ulo.x, ulo.y, ulo.z, ulo.w}, wh[4] = {uhi.x, uhi.y, uhi.z, uhi.w};
  float2 lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = bf16x2_f32(wl[i]);
    hi[i] = bf16x2_f32(wh[i]);
  }
  if (norm) {
    float2 a = mul2(lo[0], lo[0]), b = mul2(hi[0], hi[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      a = fma2(lo[i], lo[i], a);
      b = fma2(hi[i], hi[i], b);
    }
    a = __fadd2_rn(a, b);
    float ss = a.x + a.y;
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.f / D) + eps);
    const uint32_t gl[4] = {glo.x, glo.y, glo.z, glo.w}, gh[4] = {ghi.x, ghi.y, ghi.z, ghi.w};
    const float2 r2 = make_float2(r, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = mul2(mul2(lo[i], r2), bf16x2_f32(gl[i]));
      hi[i] = mul2(mul2(hi[i], r2), bf16x2_f32(gh[i]));
    }
  }
  uint32_t yl[4], yh[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 ns = make_float2(-s[i].x, -s[i].y);
    const float2 x = fma2(hi[i], ns, mul2(lo[i], c[i])), y = fma2(lo[i], s[i], mul2(hi[i], c[i]));
    yl[i] = pack_bf16(x.x, x.y);
    yh[i] = pack_bf16(y.x, y.y);
  }
  if (live) {
    out[0] = make_uint4(yl[0], yl[1], yl[2], yl[3]);
    out[LPH] = make_uint4(yh[0], yh[1], yh[2], yh[3]);
  }
}

// The heads of a group, as far as the kernel knows them when it is compiled.
enum GroupKind { GROUP_ANY, GROUP_K, GROUP_V };

// A group of the warp's heads of token t that holds keys or values: every lane's
// head hh (live or a stand-in), raw channels ulo, uhi; c, s as in q_group.
template <int D, bool FP4, GroupKind KIND>
__device__ __forceinline__ void kv_group(const QkNormRopeArgs& a, const RopeFreq& f, int t, int hh, bool live, int l,
                                         const uint4& ulo, const uint4& uhi, const float2 (&c)[4], const float2 (&s)[4]) {
  constexpr int LPH = D / 16;
  const bool is_q = KIND == GROUP_ANY && hh < a.n_q;
  const bool is_v = KIND == GROUP_V || (KIND == GROUP_ANY && hh >= a.n_q + a.n_kv);
  const uint32_t wl[4] = {ulo.x, ulo.y, ulo.z, ulo.w}, wh[4] = {uhi.x, uhi.y, uhi.z, uhi.w};
  float2 lo[4], hi[4], sum[4];  // sum: |a| + |b| of the pairs before the rotation
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = bf16x2_f32(wl[i]);
    hi[i] = bf16x2_f32(wh[i]);
    sum[i] = make_float2(0.f, 0.f);
  }
  const uint4* g4 = nullptr;
  if (KIND != GROUP_V) {
    const __nv_bfloat16* gain = is_q ? a.q_gain : is_v ? nullptr : a.k_gain;
    if (gain) g4 = reinterpret_cast<const uint4*>(gain) + l;
    // sum of squares, as a tree (every lane: the shuffles are the warp's)
    float2 sq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sq[i] = fma2(lo[i], lo[i], mul2(hi[i], hi[i]));
    const float2 s2 = __fadd2_rn(__fadd2_rn(sq[0], sq[1]), __fadd2_rn(sq[2], sq[3]));
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (g4) {
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const float2 r2 = make_float2(r, r);
      const uint4 x = g4[0], y = g4[LPH];
      const uint32_t gl[4] = {x.x, x.y, x.z, x.w}, gh[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = mul2(mul2(lo[i], r2), bf16x2_f32(gl[i]));
        hi[i] = mul2(mul2(hi[i], r2), bf16x2_f32(gh[i]));
      }
    }
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = lo[i], y = hi[i];
        sum[i] = make_float2(fabsf(x.x) + fabsf(y.x), fabsf(x.y) + fabsf(y.y));
        lo[i] = fma2(y, make_float2(-s[i].x, -s[i].y), mul2(x, c[i]));
        hi[i] = fma2(x, s[i], mul2(y, c[i]));
      }
    }
  }
  const uint4 ylo = make_uint4(pack_bf16(lo[0].x, lo[0].y), pack_bf16(lo[1].x, lo[1].y), pack_bf16(lo[2].x, lo[2].y), pack_bf16(lo[3].x, lo[3].y));
  const uint4 yhi = make_uint4(pack_bf16(hi[0].x, hi[0].y), pack_bf16(hi[1].x, hi[1].y), pack_bf16(hi[2].x, hi[2].y), pack_bf16(hi[3].x, hi[3].y));
  if (is_q && live) {
    uint4* out = reinterpret_cast<uint4*>(a.q + (static_cast<size_t>(t) * a.n_q + hh) * D);
    out[l] = ylo;
    out[LPH + l] = yhi;
  }
  const int slot = a.tok_slot[t];
  const bool store = live && !is_q && slot >= 0 && slot < a.num_pages * KV4_P;
  const int page = store ? slot / KV4_P : 0, prow = store ? slot % KV4_P : 0;
  const int kvh = is_q ? 0 : is_v ? hh - a.n_q - a.n_kv : hh - a.n_q;
  if (!FP4) {
    if (store) {
      __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(is_v ? a.v_pool : a.k_pool);
      uint4* out = reinterpret_cast<uint4*>(pool + ((static_cast<size_t>(page) * a.n_kv + kvh) * KV4_P + prow) * D);
      out[l] = is_v ? ulo : ylo;
      out[LPH + l] = is_v ? uhi : yhi;
    }
    return;
  }
  // 4 bits: a block is two neighbouring lanes, lo and hi halves separately
  const float mul = exp2_int(-(is_v ? a.v_exp : a.k_exp));
  float tlo = absmax8(lo) , thi = absmax8(hi);
  tlo = fmax_nan(tlo, __shfl_xor_sync(0xffffffffu, tlo, 1)) * mul;
  thi = fmax_nan(thi, __shfl_xor_sync(0xffffffffu, thi, 1)) * mul;
  uint32_t blo, bhi, wlo, whi, olo = 0, ohi = 0;  // scale bytes, codes, codes that fp32 cannot settle
  bool slo = false, shi = false;                  // the same of the scales
  float e = fmaxf(sum[0].x, sum[0].y);
#pragma unroll
  for (int i = 1; i < 4; ++i) e = fmaxf(e, fmaxf(sum[i].x, sum[i].y));
  const float e_other = KIND == GROUP_V ? 0.f : __shfl_xor_sync(0xffffffffu, e, 1);
  if (is_v || is_q) {
    blo = scale_byte_exact(tlo);
    bhi = scale_byte_exact(thi);
    wlo = codes_exact(lo, mul * scale_inv(blo));
    whi = codes_exact(hi, mul * scale_inv(bhi));
  } else {
    e = fmaxf(e, e_other) * (QK_ERR * mul);  // the block's largest value may be the other lane's
    blo = scale_byte_near(tlo, e, &slo);
    bhi = scale_byte_near(thi, e, &shi);
    wlo = codes_near(lo, sum, mul * scale_inv(blo), &olo);
    whi = codes_near(hi, sum, mul * scale_inv(bhi), &ohi);
  }
  if (KIND != GROUP_V && __any_sync(0xffffffffu, olo || ohi || slo || shi)) {
    QkLane q;
    q.lo = ulo;
    q.hi = uhi;
    q.gain = g4;
    q.gain_hi = LPH;
    q.pos = a.tok_pos[t];
    q.i0 = 8 * l;
    if (__any_sync(0xffffffffu, slo || shi)) {
      // both lanes of a block work out a scale that either left open
      slo |= __shfl_xor_sync(0xffffffffu, slo, 1);
      shi |= __shfl_xor_sync(0xffffffffu, shi, 1);
      // what is smaller than the largest by more than their errors is not it
      const uint32_t y = settle_scales<D>(q, f, a.eps, mul, slo ? near_largest(lo, (tlo - 4.f * e) / mul) : 0u,
                                          shi ? near_largest(hi, (thi - 4.f * e) / mul) : 0u);
      if (slo) {
        blo = y & 0xFFu;
        wlo = codes_near(lo, sum, mul * scale_inv(blo), &olo);
      }
      if (shi) {
        bhi = (y >> 8) & 0xFFu;
        whi = codes_near(hi, sum, mul * scale_inv(bhi), &ohi);
      }
    }
    if (__any_sync(0xffffffffu, olo || ohi)) {
      const uint2 y = settle_codes<D>(q, f, a.eps, mul, olo, ohi, blo, bhi, wlo, whi);
      wlo = y.x;
      whi = y.y;
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

// Which heads a launch takes.  The path of the queries needs half the registers of
// the keys' one, so many tokens take two launches, each with all the warps that
// its registers allow; few tokens take one.
enum QkPart { PART_ALL, PART_Q, PART_KV };

template <int D, bool FP4, QkPart PART>
__global__ void __launch_bounds__(QK_THREADS, PART == PART_Q ? 4 : 2)
    qk_norm_rope_kernel(const QkNormRopeArgs a, const __grid_constant__ RopeFreq f, int tok_cta) {
  constexpr int LPH = D / 16;         // lanes of a head
  constexpr int HPW = 32 / LPH;       // heads of a warp
  constexpr int HALF = D / 2, WARPS = QK_THREADS / 32;
  if (PART == PART_KV) pdl_trigger();  // the queries' launch may fill the SMs that this one leaves free
  __shared__ __align__(16) float co[QK_MAX_TOK][HALF], si[QK_MAX_TOK][HALF];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hl = lane / LPH, l = lane % LPH;  // head of the warp, lane of the head
  const int t0 = blockIdx.x * tok_cta, nt = min(tok_cta, a.n_tok - t0);
  // the warps of a token share its groups of heads
  const int wpt = WARPS / tok_cta, tl = warp / wpt, t = t0 + tl;
  const int heads = a.n_q + 2 * a.n_kv;
  const int groups = (heads + HPW - 1) / HPW;
  // (PART_Q and PART_KV: n_q is a multiple of a group)
  const int g_end = PART == PART_Q ? a.n_q / HPW : groups;
  int g = warp % wpt + (PART == PART_KV ? a.n_q / HPW : 0);
  const bool busy = tl < nt;
  // heads past the last shadow it and store nothing
  auto row_of = [&](int group) {
    return reinterpret_cast<const uint4*>(a.qkv + static_cast<size_t>(t) * a.ld + static_cast<size_t>(min(group * HPW + hl, heads - 1)) * D) + l;
  };
  uint4 ulo{}, uhi{};
  if (busy && g < g_end) {  // on their way while the angles are worked out
    const uint4* row = row_of(g);
    ulo = row[0];
    uhi = row[LPH];
  }
  for (int k = threadIdx.x; k < nt * HALF; k += QK_THREADS) {
    const int i = k % HALF;
    const uint64_t turn = angle_turns(a.tok_pos[t0 + k / HALF], f.freq[i]);
    // the angle in units of 2^-31 pi: 24 bits through sincospif, and a
    // first-order step (below 10^-6) for the rest
    const int hi = static_cast<int>(turn >> 32);
    const float x = __int2float_rz(hi);
    const float rest = static_cast<float>(hi - static_cast<int>(x)) + static_cast<float>(static_cast<uint32_t>(turn)) * 0x1p-32f;
    float s, c;
    sincospif(x * (1.f / 2147483648.f), &s, &c);
    const float d = rest * (3.14159265f / 2147483648.f);
    co[k / HALF][i] = fmaf(-s, d, c);
    si[k / HALF][i] = fmaf(c, d, s);
  }
  __syncthreads();
  if (!busy) {
    if (PART == PART_Q) pdl_wait();
    return;
  }
  float2 c2[4], s2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c2[i] = *reinterpret_cast<const float2*>(&co[tl][8 * l + 2 * i]);
    s2[i] = *reinterpret_cast<const float2*>(&si[tl][8 * l + 2 * i]);
  }
  uint4 glo{}, ghi{};
  if (PART != PART_KV && a.q_gain) {
    glo = reinterpret_cast<const uint4*>(a.q_gain)[l];
    ghi = reinterpret_cast<const uint4*>(a.q_gain)[LPH + l];
  }
  for (; g < g_end; g += wpt) {
    uint4 nlo = ulo, nhi = uhi;
    if (g + wpt < g_end) {
      const uint4* row = row_of(g + wpt);
      nlo = row[0];
      nhi = row[LPH];
    }
    const int h = g * HPW + hl;
    if (PART == PART_Q || (PART == PART_ALL && (g + 1) * HPW <= a.n_q))
      q_group<D>(ulo, uhi, glo, ghi, a.q_gain != nullptr, a.eps, c2, s2,
                 reinterpret_cast<uint4*>(a.q + (static_cast<size_t>(t) * a.n_q + h) * D) + l, true);
    else if (PART != PART_Q && g * HPW >= a.n_q + a.n_kv)
      kv_group<D, FP4, GROUP_V>(a, f, t, min(h, heads - 1), h < heads, l, ulo, uhi, c2, s2);
    else if (PART != PART_Q && g * HPW >= a.n_q && (g + 1) * HPW <= a.n_q + a.n_kv)
      kv_group<D, FP4, GROUP_K>(a, f, t, h, true, l, ulo, uhi, c2, s2);
    else if (PART == PART_ALL)
      kv_group<D, FP4, GROUP_ANY>(a, f, t, min(h, heads - 1), h < heads, l, ulo, uhi, c2, s2);
    ulo = nlo;
    uhi = nhi;
  }
  // what follows on the stream sees both launches complete
  if (PART == PART_Q) pdl_wait();
}

// ------------------------------------------------------------ rows by slot
//
// HBM-bound: a lane makes 8 channels of K and the same of V, so that a warp's
// stores are whole 512-byte runs; it has RD_ITEMS tokens' loads in flight.
// Measured: 30,000 tokens of 8 heads of 128 (158 MB) 29 us, 5.5 TB/s, 0.81 of the
// copy rate; 333 tokens of 2 heads of 64 3.3 us in a graph, a launch.
constexpr int RD_THREADS = 256;
constexpr int RD_ITEMS = 4;

// 8 codes under scale byte `b`, times 2^E: exact in fp32, rounded to bf16 only
// where 2^E leaves bf16's range.
__device__ __forceinline__ uint4 chunk_to_bf16(uint32_t w, uint32_t b, float mul) {
  const float s = e4m3_to_f32(b) * mul;
  const float2 x0 = f16x2_to_f32x2(e2m1_to_f16x2<0>(w)), x1 = f16x2_to_f32x2(e2m1_to_f16x2<1>(w));
  const float2 x2 = f16x2_to_f32x2(e2m1_to_f16x2<2>(w)), x3 = f16x2_to_f32x2(e2m1_to_f16x2<3>(w));
  return make_uint4(pack_bf16(x0.x * s, x0.y * s), pack_bf16(x1.x * s, x1.y * s),
                    pack_bf16(x2.x * s, x2.y * s), pack_bf16(x3.x * s, x3.y * s));
}

template <int D>
__global__ void __launch_bounds__(RD_THREADS)
    kv4_read_kernel(const uint8_t* __restrict__ pool, int num_pages, int n_kv,
                    const int* __restrict__ slots, int n, float k_mul, float v_mul,
                    uint4* __restrict__ k, uint4* __restrict__ v) {
  constexpr int CH = D / 8;  // chunks of a row
  const int tpc = RD_THREADS / CH;  // (token, head) rows that the CTA's threads cover at once
  const int c = threadIdx.x % CH, row0 = threadIdx.x / CH;
  const long long rows = static_cast<long long>(n) * n_kv;
  for (long long r0 = static_cast<long long>(blockIdx.x) * tpc * RD_ITEMS; r0 < rows;
       r0 += static_cast<long long>(gridDim.x) * tpc * RD_ITEMS) {
    uint32_t kw[RD_ITEMS], vw[RD_ITEMS], ks[RD_ITEMS], vs[RD_ITEMS];
    const long long tok0 = r0 / n_kv;  // the CTA's first token, and its head
    const unsigned head0 = static_cast<unsigned>(r0 - tok0 * n_kv);
#pragma unroll
    for (int i = 0; i < RD_ITEMS; ++i) {
      const long long r = r0 + i * tpc + row0;
      kw[i] = vw[i] = ks[i] = vs[i] = 0;
      if (r >= rows) continue;
      const unsigned local = head0 + i * tpc + row0, t = local / static_cast<unsigned>(n_kv);
      const unsigned h = local - t * n_kv;
      const int slot = slots[tok0 + t];
      if (slot >= 0 && slot < num_pages * KV4_P) {
        const uint8_t* part = pool + (static_cast<size_t>(slot / KV4_P) * n_kv + h) * 2 * kv4_part_bytes(D);
        const uint8_t* code = part + (slot % KV4_P) * (D / 2) + c * 4;
        const uint8_t* sc = part + 8 * D + (slot % KV4_P) * (D / 16) + c / 2;
        kw[i] = *reinterpret_cast<const uint32_t*>(code);
        vw[i] = *reinterpret_cast<const uint32_t*>(code + kv4_part_bytes(D));
        ks[i] = sc[0];
        vs[i] = sc[kv4_part_bytes(D)];
      }
    }
#pragma unroll
    for (int i = 0; i < RD_ITEMS; ++i) {
      const long long r = r0 + i * tpc + row0;
      if (r >= rows) break;
      k[r * CH + c] = chunk_to_bf16(kw[i], ks[i], k_mul);
      v[r * CH + c] = chunk_to_bf16(vw[i], vs[i], v_mul);
    }
  }
}

}  // namespace

cudaError_t launch_block_tables(const BlockTableArgs& a, int num_sms, cudaStream_t stream) {
  // a CTA for every block of tokens the caller has room for and for every BT_REQS
  // requests, up to two an SM.  1801 requests / 4096 with half a million tokens:
  // 8.2 / 16.4 us; without the second 12.3 / 16.4; blocks of half the tokens 9.0 /
  // 18.4; up to four CTAs an SM 20.4, one 20.5 (with the smaller blocks) for the latter
  const long long blocks = (static_cast<long long>(a.tok_cap) + BT_TOKENS - 1) / BT_TOKENS;
  const long long want = max(blocks, (static_cast<long long>(a.n_seq) + BT_REQS - 1) / BT_REQS);
  const int grid = static_cast<int>(min(want, 2ll * num_sms));
  block_tables_kernel<<<grid, BT_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, bool FP4>
static cudaError_t launch_qk(const QkNormRopeArgs& a, const RopeFreq& f, int tok, bool split, cudaStream_t stream) {
  const int grid = (a.n_tok + tok - 1) / tok;
  if (split) {
    qk_norm_rope_kernel<D, FP4, PART_KV><<<grid, QK_THREADS, 0, stream>>>(a, f, tok);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(QK_THREADS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<D, false, PART_Q>, a, f, tok);
  } else {
    qk_norm_rope_kernel<D, FP4, PART_ALL><<<grid, QK_THREADS, 0, stream>>>(a, f, tok);
  }
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs& a, const RopeFreq& f, bool fp4, int num_sms,
                                cudaStream_t stream) {
  // one token a CTA until that fills the GPU three times, then up to 8, a warp
  // each: fewer warps then load a token's angles and gains.  8191 tokens of 80
  // heads into 4 bits and back at 1, 2, 4, 8 tokens: 120, 96, 88 (in two launches),
  // 84 us, and 93 for 8 in one launch; 2048 tokens of 48 heads into bf16: 21 at 1,
  // 15 to 17 at 2 to 8.
  int tok = 1;
  while (tok < QK_MAX_TOK && a.n_tok >= 2 * tok * 3 * num_sms) tok *= 2;
  const int hpw = a.head_dim == 128 ? 4 : 8;  // heads of a group
  const bool split = tok == QK_MAX_TOK && a.n_q % hpw == 0 && a.n_kv % hpw == 0;
  if (a.head_dim == 128) return fp4 ? launch_qk<128, true>(a, f, tok, split, stream) : launch_qk<128, false>(a, f, tok, split, stream);
  return fp4 ? launch_qk<64, true>(a, f, tok, split, stream) : launch_qk<64, false>(a, f, tok, split, stream);
}

cudaError_t launch_kv4_read(const uint8_t* pool, int num_pages, int n_kv, int head_dim,
                            const int* slots, int n, int k_exp, int v_exp, __nv_bfloat16* k,
                            __nv_bfloat16* v, int num_sms, cudaStream_t stream) {
  const long long rows = static_cast<long long>(n) * n_kv;
  const int per = RD_THREADS / (head_dim / 8) * RD_ITEMS;
  const long long want = (rows + per - 1) / per;
  // CTAs an SM at most, 30,000 tokens: 8, 16, 32: 30.2, 29.1, 28.8 us
  const int grid = static_cast<int>(want < num_sms * 32LL ? want : num_sms * 32LL);
  const float km = exp2_int(k_exp), vm = exp2_int(v_exp);
  if (head_dim == 128)
    kv4_read_kernel<128><<<grid, RD_THREADS, 0, stream>>>(pool, num_pages, n_kv, slots, n, km, vm, reinterpret_cast<uint4*>(k), reinterpret_cast<uint4*>(v));
  else
    kv4_read_kernel<64><<<grid, RD_THREADS, 0, stream>>>(pool, num_pages, n_kv, slots, n, km, vm, reinterpret_cast<uint4*>(k), reinterpret_cast<uint4*>(v));
  return cudaGetLastError();
}

}  // namespace nf
