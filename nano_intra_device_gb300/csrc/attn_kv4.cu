// Attention of a few rows a request over the 4-bit KV cache.
//
// What bounds it: a page of one KV head is 18 d bytes (2304 at d = 128), which
// the GPU's copy rate delivers to one SM in about 100 clocks; the rest has to
// fit into those.  Per page and KV head a warp forms
//   S^T [16 positions x 8 columns] = K [16 x d] Q^T [d x 8],
//   O^T [d x 8] += V^T [d x 16] P^T [16 x 8]
// with m16n8k16 fp16 products.  The 8 columns are the GRP query heads of 8 / GRP
// neighbouring rows of one request (a decode row fills GRP of them), so a short
// chunk reads the cache once for 8 / GRP rows.
//  * Codes go straight from shared memory to operand registers: one conversion
//    instruction a byte (e2m1x2 -> f16x2) and one product with the block's
//    scale.  Both are exact: a code has 2 significant bits, a scale 4, and
//    their product lies in fp16's normal range or on its grid.
//  * Channels and positions are summed over, so their order in an operand is
//    free.  Thread c of a quad takes the channels [c d/4, (c + 1) d/4) of its K
//    rows, 16 contiguous bytes and two scales; for V, thread group g the
//    channels [g d/8, (g + 1) d/8) of its four positions, 8 bytes and a scale
//    each.  pos_of() orders the positions so that the K reads hit all
//    banks once and the V reads at most twice.
//  * Q enters in fp16 scaled by a power of two a column (its largest element to
//    2^14): bf16's 8 bits fit fp16's 11 down to 2^-28 of the largest element.
//  * P enters as fp16 of 2^7 times its share of the running maximum (2^-11
//    relative, exact zero only below 2^-32); the denominators sum the fp32
//    values.  The maximum is raised only when a score passes it by 2^8, so p
//    stays below 2^15.
//
// Work split: every warp gets the same number of pages.  The pages of all
// (request, column group, KV head) units are laid end to end, each unit behind
// a few slots that stand for its fixed cost, and warp w takes the slots
// [w quota, (w + 1) quota).  Every CTA derives its part from the lengths by a
// block-wide prefix sum; there is no work list, no counter to fetch from and no
// second launch.  A unit cut between warps is joined in shared memory by the
// CTA, one cut between CTAs through a record in the handle's workspace by the
// CTA that arrives last, in the order of the pieces either way: the result does
// not depend on timing.  The arrival counters are zero between launches.
#include <type_traits>

#include "common.cuh"
#include "kv4.cuh"
#include "kv4.h"
#include "mma_frag.cuh"

namespace nf {
namespace {

constexpr int KA_WARPS = 16;
constexpr int KA_THREADS = KA_WARPS * 32;
constexpr int KA_PG = 2;           // pages a warp works on at once (a ring stage)
constexpr int KA_RING = 9216;      // ring bytes of a warp: 2 stages at d = 128, 4 at d = 64
constexpr int KA_COLS = 8;
constexpr int KA_FIXED = 2;        // slots a unit costs beside its pages
constexpr int KA_MIN_QUOTA = 4;    // fewest slots of a warp
constexpr float KA_LAZY = 8.f;
constexpr float KA_SHIFT = 7.f;

template <int D>
struct KaLayout {
  static constexpr int SLOT = 18 * D;
  static constexpr int STAGES = KA_RING / (KA_PG * SLOT);
  static constexpr int REC = KA_COLS * D + 2 * KA_COLS;  // floats: O [column][d], m, l
  static constexpr int REC_OFF = KA_WARPS * KA_RING;
  static constexpr int BAR_OFF = REC_OFF + KA_WARPS * REC * 4;
  static constexpr int SMEM = BAR_OFF + KA_WARPS * STAGES * 8;
  static_assert(KA_RING % (KA_PG * SLOT) == 0 && REC * 4 <= KA_RING, "a record fits a drained ring");
};

// Page row of operand row r: neighbours (K: the two rows of eight lanes) differ
// in parity, and so do the rows 2t of t = 0 .. 3 in turn (V).
__device__ __forceinline__ int pos_of(int r) {
  return static_cast<int>((0x65742130u >> (4 * (r & 7))) & 7u) + (r & 8);
}

struct KaUnit {         // one (request, column group, KV head)
  long long key;        // its first slot
  int s, g;             // request, KV head
  int row0;             // first row in q and o
  int rows;             // live rows (1 .. 8 / GRP)
  int len;              // positions row row0 sees (may be <= 0)
  int pages;            // pages of the request
};

// Rows, visible length and pages of request s (0 rows: not ours).
struct KaSeq {
  int b0, rows, len, pages, groups;
};
template <int RG>
__device__ __forceinline__ KaSeq ka_seq(const Kv4AttnArgs& a, int s, bool report) {
  KaSeq q;
  q.b0 = s;
  q.rows = 1;
  if (a.tok_begin) {
    const int b0 = a.tok_begin[s], b1 = a.tok_begin[s + 1];
    q.b0 = b0;
    q.rows = b1 - b0;
    if (b0 < 0 || b1 < b0 || b1 > a.n_tok) {
      if (report) raise_status(a.status, ST_BAD_LEN);
      q.b0 = 0;
      q.rows = 0;
    }
  }
  q.len = a.seq_lens[s];
  if (q.len < 0 || q.len > static_cast<long long>(a.max_pages) * KV4_P) {
    if (report) raise_status(a.status, ST_BAD_LEN);
    q.len = 0;
  }
  q.pages = (q.len + KV4_P - 1) / KV4_P;
  q.groups = (q.rows + RG - 1) / RG;
  return q;
}
__device__ __forceinline__ long long ka_slots(const KaSeq& q, int n_kv) {
  return static_cast<long long>(q.pages + KA_FIXED) * q.groups * n_kv;
}

// a / b for a >= 0, b > 0; a 64-bit division costs several hundred clocks, and
// slot numbers past 32 bits are rare.
__device__ __forceinline__ long long udiv(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int B>
__device__ __forceinline__ uint32_t code_pair(const uint32_t (&w)[B], int i) {
  switch (i & 3) {
    case 0: return e2m1_to_f16x2<0>(w[i >> 2]);
    case 1: return e2m1_to_f16x2<1>(w[i >> 2]);
    case 2: return e2m1_to_f16x2<2>(w[i >> 2]);
    default: return e2m1_to_f16x2<3>(w[i >> 2]);
  }
}
// words of shared memory from a generic pointer
template <int W>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[W]) {
  if (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2 % W] = v.z; w[3 % W] = v.w;
  } else if (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1 % W] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ bool scale_nan(uint32_t b) { return (b & 0x7Fu) == 0x7Fu; }

// N floats to bf16, 16-byte stores.
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&x)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

template <int GRP, int D>
__global__ void __launch_bounds__(KA_THREADS, 1) attn_kv4_kernel(const Kv4AttnArgs a) {
  using Lay = KaLayout<D>;
  constexpr int RG = KA_COLS / GRP;      // rows of a unit
  constexpr int STAGES = Lay::STAGES, SLOT = Lay::SLOT;
  constexpr int KW = D / 32;             // words of a thread's K codes in a row
  constexpr int VW = D / 64;             // words of a thread's V codes in a row
  constexpr int KS = D / 16;             // k-steps of S, m-tiles of O
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_pre[KA_THREADS];
  __shared__ long long s_warp[KA_WARPS + 1];
  __shared__ KaUnit s_piece[KA_WARPS][2];  // what a warp leaves for the CTA to join; key -1: nothing
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lr = lane >> 2, lc = lane & 3;
  uint8_t* ring = smem + warp * KA_RING;
  float* head_rec = reinterpret_cast<float*>(smem + Lay::REC_OFF) + warp * Lay::REC;
  float* tail_rec = reinterpret_cast<float*>(ring);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF) + warp * STAGES;
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&bar[s], 1);
    fence_mbar_init();
    s_piece[warp][0].key = s_piece[warp][1].key = -1;
  }

  // ---- the slots before every run of requests: thread i sums [i c, (i + 1) c)
  const int c = (a.n_seq + KA_THREADS - 1) / KA_THREADS;
  {
    long long sum = 0;
    const int s0 = min(a.n_seq, tid * c), s1 = min(a.n_seq, s0 + c);
    for (int s = s0; s < s1; ++s) sum += ka_slots(ka_seq<RG>(a, s, blockIdx.x == 0), a.n_kv);
    long long in = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += x;
    }
    if (lane == 31) s_warp[warp] = in;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < KA_WARPS; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    s_pre[tid] = before + in - sum;
    if (tid == 0) s_warp[KA_WARPS] = all;
    __syncthreads();
  }
  const long long total = s_warp[KA_WARPS];
  const long long n_warps = static_cast<long long>(gridDim.x) * KA_WARPS;
  const long long quota = max(udiv(total + n_warps - 1, n_warps), static_cast<long long>(KA_MIN_QUOTA));
  const long long wid = static_cast<long long>(blockIdx.x) * KA_WARPS + warp;
  if (static_cast<long long>(blockIdx.x) * KA_WARPS * quota >= total) return;  // nothing for this CTA
  const long long end = min((wid + 1) * quota, total);
  long long x = wid * quota;  // next slot of this warp

  uint32_t gk = 0;  // pages this warp has consumed (ring position)
  bool failed = false;
  int s = 0;
  long long base = 0;  // first slot of request s
  KaSeq sq{0, 0, 0, 0, 0};
  if (x < end) {
    int lo = 0, hi = KA_THREADS - 1;  // last run that starts at or before x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pre[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    s = lo * c;
    base = s_pre[lo];
    for (;;) {  // 32 requests at a time
      const int r = s + lane;
      const long long n = r < a.n_seq ? ka_slots(ka_seq<RG>(a, r, false), a.n_kv) : 0;
      long long in = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, base + in > x);
      if (past) {
        const int j = __ffs(past) - 1;
        base += __shfl_sync(0xffffffffu, in - n, j);
        s += j;
        break;
      }
      base += __shfl_sync(0xffffffffu, in, 31);
      s += 32;
      if (s >= a.n_seq) break;  // not reached: x < total
    }
    if (s < a.n_seq) sq = ka_seq<RG>(a, s, false);
  }

  while (x < end && s < a.n_seq) {
    const long long per = sq.pages + KA_FIXED;
    if (x >= base + per * sq.groups * a.n_kv) {  // next request
      base += per * sq.groups * a.n_kv;
      if (++s < a.n_seq) sq = ka_seq<RG>(a, s, false);
      continue;
    }
    const int k = static_cast<int>(udiv(x - base, per));
    KaUnit u;
    u.key = base + k * per;
    u.s = s;
    u.g = k % a.n_kv;
    const int grp0 = (k / a.n_kv) * RG;  // first row of the group in the request
    u.row0 = sq.b0 + grp0;
    u.rows = min(RG, sq.rows - grp0);
    u.len = sq.len - sq.rows + grp0 + 1;
    u.pages = sq.pages;
    // pages [p0, p1) of the unit fall to this warp
    const int off = static_cast<int>(x - u.key);
    const int p0 = max(off - KA_FIXED, 0);
    const int p1 = static_cast<int>(min(end - u.key, per)) - KA_FIXED;
    x = min(end, u.key + per);
    const int h0 = 2 * lc, h1 = 2 * lc + 1;
    const int i0 = h0 / GRP, i1 = h1 / GRP;  // rows of this lane's accumulator columns
    const bool w0 = i0 < u.rows, w1 = i1 < u.rows;
    __nv_bfloat16* o0 = a.o + (static_cast<size_t>(u.row0 + (w0 ? i0 : 0)) * a.n_q + u.g * GRP + h0 % GRP) * D + lr * (D / 8);
    __nv_bfloat16* o1 = a.o + (static_cast<size_t>(u.row0 + (w1 ? i1 : 0)) * a.n_q + u.g * GRP + h1 % GRP) * D + lr * (D / 8);
    if (u.pages == 0) {  // nothing to see: zeros, by the warp of the unit's first slot
      if (off == 0) {
        const float z[D / 8] = {};
        if (w0) store_row(o0, z);
        if (w1) store_row(o1, z);
      }
      continue;
    }
    if (p1 <= p0) continue;  // only slots of the fixed cost
    const int npg = p1 - p0;

    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY;  // reference maxima of the columns h0, h1 (base 2)
    float n0 = KA_SHIFT, n1 = KA_SHIFT;    // what p's exponent adds: KA_SHIFT - m (m finite)
    float l0 = 0.f, l1 = 0.f;              // this lane's share of the denominators

    if (!failed) {
      // page ids, 32 at a time, the next 32 on their way
      const int* bt = a.block_table + static_cast<size_t>(u.s) * a.max_pages + p0;
      auto load_ids = [&](int b) {
        const int j = b + lane;
        int page = 0;
        if (j < npg) {
          page = bt[j];
          if (page < 0 || page >= a.num_pages) {  // never read outside the pool
            raise_status(a.status, ST_BAD_PAGE);
            page = 0;
          }
        }
        return page;
      };
      int ids = load_ids(0), ids_next = load_ids(32);
      int issued = 0;  // pages
      auto issue = [&](uint32_t st) {  // the piece's next pages into stage st (every lane calls)
        if (issued > 0 && (issued & 31) == 0) {
          ids = ids_next;
          ids_next = load_ids(issued + 32);
        }
        int page[KA_PG];
#pragma unroll
        for (int i = 0; i < KA_PG; ++i) page[i] = __shfl_sync(0xffffffffu, ids, (issued + i) & 31);
        const int n = min(KA_PG, npg - issued);
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar[st], n * SLOT);
#pragma unroll
          for (int i = 0; i < KA_PG; ++i)
            if (i < n)
              bulk_g2s(ring + (st * KA_PG + i) * SLOT, a.pool + (static_cast<size_t>(page[i]) * a.n_kv + u.g) * SLOT,
                       SLOT, &bar[st]);
        }
        issued += n;
      };
      if (lane == 0) fence_proxy_async_smem();  // the previous piece's reads come first
#pragma unroll
      for (int i = 0; i < STAGES; ++i)
        if (i * KA_PG < npg) issue((gk + i) % STAGES);

      // Q^T as the B operand: column lr, this thread's channels [lc d/4, ..) in
      // pairs 4 j + {0, 1} and 4 j + {2, 3}
      uint32_t qb[KS][2];
      float sc0, sc1;
      {
        const int ri = lr / GRP;
        const bool live = ri < u.rows;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + (static_cast<size_t>(u.row0 + (live ? ri : 0)) * a.n_q + u.g * GRP + lr % GRP) * D + lc * (D / 4));
        uint32_t raw[D / 8];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 v = src[i];
          raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          if (!live) raw[i] = 0;
          top = fmaxf(top, fmaxf(fabsf(bf16lo(raw[i])), fabsf(bf16hi(raw[i]))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        const int kq = top > 0.f ? max(-126, min(120, 14 - e)) : 0;
        const float mul = exp2_int(kq);
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qb[j][i] = pack_f16(bf16lo(raw[2 * j + i]) * mul, bf16hi(raw[2 * j + i]) * mul);
        const float back = a.scale_log2 * exp2_int(-kq);
        sc0 = __shfl_sync(0xffffffffu, back, h0 * 4);
        sc1 = __shfl_sync(0xffffffffu, back, h1 * 4);
      }
      const int lim0 = u.len + i0, lim1 = u.len + i1;  // positions the two columns see
      const int most = u.len + u.rows - 1;             // and the unit's last row
      const int kr = pos_of(lr);                       // page row of this thread's K rows kr, kr + 8
      const int va = pos_of(2 * lc), vb = pos_of(2 * lc + 1);

      const int plim = p1 * KV4_P;  // positions past the piece are another warp's

      // one ring stage: KA_PG pages from position pb on.  EDGE: some column does
      // not see all of their positions (a request's last pages, a piece's end).
      auto step = [&](const uint8_t* slot, const int pb, auto edge_) {
        constexpr bool EDGE = decltype(edge_)::value;
        float sc[KA_PG][4];
#pragma unroll
        for (int p = 0; p < KA_PG; ++p) {
          const uint8_t* sl = slot + p * SLOT;
          uint32_t ka[KW], kb[KW];
          lds_words(sl + kr * (D / 2) + lc * (D / 8), ka);
          lds_words(sl + (kr + 8) * (D / 2) + lc * (D / 8), kb);
          const uint8_t* ks = sl + 8 * D + kr * (D / 16) + lc * (D / 64);
          uint32_t sa[D / 64], sb[D / 64];  // scales as f16 pairs, one a 16-channel block
          if (D == 128) {
            const uint32_t ra = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks));
            const uint32_t rb = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks + 8 * (D / 16)));
            sa[0] = __byte_perm(ra, ra, 0x1010);
            sa[D / 64 - 1] = __byte_perm(ra, ra, 0x3232);
            sb[0] = __byte_perm(rb, rb, 0x1010);
            sb[D / 64 - 1] = __byte_perm(rb, rb, 0x3232);
          } else {
            const uint32_t both = e4m3x2_to_f16x2(__byte_perm(ks[0], ks[8 * (D / 16)], 0x0040));
            sa[0] = __byte_perm(both, both, 0x1010);
            sb[0] = __byte_perm(both, both, 0x3232);
          }
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            const uint32_t fa = sa[j / 4], fb = sb[j / 4];
            mma_f16(acc, hmul2_u(code_pair(ka, 2 * j), fa), hmul2_u(code_pair(kb, 2 * j), fb),
                    hmul2_u(code_pair(ka, 2 * j + 1), fa), hmul2_u(code_pair(kb, 2 * j + 1), fb), qb[j][0], qb[j][1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[p][i] = acc[i] * ((i & 1) ? sc1 : sc0);
        }
        // scaled scores, base 2: (position kr, h0), (kr, h1), (kr + 8, h0), (kr + 8, h1)
        unsigned bad = 0;  // NaN values of V at this thread's positions: bit 2 page + half
        if (EDGE) {
          // A NaN of V must reach the columns that see it and no other, so it
          // goes through P instead of V (0 * NaN is NaN).
#pragma unroll
          for (int p = 0; p < KA_PG; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int pos = pb + p * KV4_P + kr + 8 * i;
              if (pos >= min(lim0, plim)) sc[p][2 * i] = -INFINITY;
              if (pos >= min(lim1, plim)) sc[p][2 * i + 1] = -INFINITY;
              const uint8_t* vs = slot + p * SLOT + 17 * D + (kr + 8 * i) * (D / 16);
#pragma unroll
              for (int b = 0; b < D / 16; ++b)
                if (scale_nan(vs[b])) bad |= 1u << (2 * p + i);
            }
        }
        float x0 = fmaxf(sc[0][0], sc[0][2]), x1 = fmaxf(sc[0][1], sc[0][3]);
#pragma unroll
        for (int p = 1; p < KA_PG; ++p) {
          x0 = fmaxf(x0, fmaxf(sc[p][0], sc[p][2]));
          x1 = fmaxf(x1, fmaxf(sc[p][1], sc[p][3]));
        }
        if (__any_sync(0xffffffffu, x0 > m0 + KA_LAZY || x1 > m1 + KA_LAZY)) {
          float y0 = x0, y1 = x1;
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, d));
            y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, d));
          }
          const float r0 = fmaxf(m0, y0), r1 = fmaxf(m1, y1);
          // a column that has seen nothing yet holds zeros: any factor will do
          const float c0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - r0);
          const float c1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - r1);
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[i][0] *= c0;
            o[i][1] *= c1;
            o[i][2] *= c0;
            o[i][3] *= c1;
          }
          l0 *= c0;
          l1 *= c1;
          m0 = r0;
          m1 = r1;
          n0 = m0 == -INFINITY ? KA_SHIFT : KA_SHIFT - m0;
          n1 = m1 == -INFINITY ? KA_SHIFT : KA_SHIFT - m1;
        }
        uint32_t pt[KA_PG][2];
#pragma unroll
        for (int p = 0; p < KA_PG; ++p) {
          // the scaled scores are rounded before the maximum is taken off (no fused
          // step), so that the largest is at most 2^8 of it at any magnitude
          float e0 = ex2_approx(sc[p][0] + n0), e1 = ex2_approx(sc[p][1] + n1);
          float e2 = ex2_approx(sc[p][2] + n0), e3 = ex2_approx(sc[p][3] + n1);
          if (EDGE && bad) {
            const float nan = __int_as_float(0x7FC00000);
            const int pos = pb + p * KV4_P + kr;
            if ((bad >> (2 * p)) & 1) {
              if (pos < min(lim0, plim)) e0 = nan;
              if (pos < min(lim1, plim)) e1 = nan;
            }
            if ((bad >> (2 * p + 1)) & 1) {
              if (pos + 8 < min(lim0, plim)) e2 = nan;
              if (pos + 8 < min(lim1, plim)) e3 = nan;
            }
          }
          l0 += e0 + e2;
          l1 += e1 + e3;
          pt[p][0] = movmatrix_trans(pack_f16(e0, e1));  // positions 2 lc (+1), column lr
          pt[p][1] = movmatrix_trans(pack_f16(e2, e3));  // and 8 on
        }
#pragma unroll
        for (int p = 0; p < KA_PG; ++p) {
          const uint8_t* v = slot + p * SLOT + 9 * D + lr * (D / 16);
          uint32_t v0[VW], v1[VW], v2[VW], v3[VW];
          lds_words(v + va * (D / 2), v0);
          lds_words(v + vb * (D / 2), v1);
          lds_words(v + (va + 8) * (D / 2), v2);
          lds_words(v + (vb + 8) * (D / 2), v3);
          const uint8_t* vs = slot + p * SLOT + 17 * D + (lr * (D / 8)) / 16;
          uint32_t b0 = vs[va * (D / 16)], b1 = vs[vb * (D / 16)];
          uint32_t b2 = vs[(va + 8) * (D / 16)], b3 = vs[(vb + 8) * (D / 16)];
          if (EDGE) {  // positions no column sees, and NaNs (P has them): nothing
            const int pos = pb + p * KV4_P, lim = min(most, plim);
            if (pos + va >= lim || scale_nan(b0)) b0 = 0;
            if (pos + vb >= lim || scale_nan(b1)) b1 = 0;
            if (pos + va + 8 >= lim || scale_nan(b2)) b2 = 0;
            if (pos + vb + 8 >= lim || scale_nan(b3)) b3 = 0;
          }
          const uint32_t f01 = e4m3x2_to_f16x2(__byte_perm(b0, b1, 0x0040));
          const uint32_t f23 = e4m3x2_to_f16x2(__byte_perm(b2, b3, 0x0040));
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            const uint32_t c0 = code_pair(v0, i), c1 = code_pair(v1, i);
            const uint32_t c2 = code_pair(v2, i), c3 = code_pair(v3, i);
            mma_f16(o[i], hmul2_u(__byte_perm(c0, c1, 0x5410), f01), hmul2_u(__byte_perm(c0, c1, 0x7632), f01),
                    hmul2_u(__byte_perm(c2, c3, 0x5410), f23), hmul2_u(__byte_perm(c2, c3, 0x7632), f23), pt[p][0], pt[p][1]);
          }
        }
      };
      uint32_t st = gk % STAGES, ph = (gk / STAGES) & 1;
      for (int kp = 0; kp < npg; kp += KA_PG) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bar[st], ph, a.timeout_ns))) {
          if (lane == 0)  // what is still in flight lands before shared memory is used again
            for (int j = kp; j < issued; j += KA_PG) {
              mbar_wait(&bar[st], ph, a.timeout_ns);
              if (++st == STAGES) {
                st = 0;
                ph ^= 1;
              }
            }
          failed = true;
          break;
        }
        const int pb = (p0 + kp) * KV4_P;
        if (pb + KA_PG * KV4_P <= min(u.len, plim)) step(ring + st * (KA_PG * SLOT), pb, std::false_type{});
        else step(ring + st * (KA_PG * SLOT), pb, std::true_type{});
        ++gk;
        __syncwarp();
        if (issued < npg) {
          if (lane == 0) fence_proxy_async_smem();
          issue(st);
        }
        if (++st == STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (failed) {
      raise_status(a.status, ST_TIMEOUT);
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    // o[i]: channels lr d/8 + 2 i (+1) of columns h0 (entries 0, 2) and h1 (1, 3)
    float z0[D / 8], z1[D / 8];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      z0[2 * i] = o[i][0];
      z0[2 * i + 1] = o[i][2];
      z1[2 * i] = o[i][1];
      z1[2 * i + 1] = o[i][3];
    }
    if (p0 == 0 && p1 == u.pages) {  // the whole unit
      const float r0 = l0 == 0.f ? 0.f : a.v_scale / l0, r1 = l1 == 0.f ? 0.f : a.v_scale / l1;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        z0[i] *= r0;
        z1[i] *= r1;
      }
      if (w0) store_row(o0, z0);
      if (w1) store_row(o1, z1);
      continue;
    }
    // a piece: the warp's first when it began in another warp, else its last
    const int which = p0 > 0 ? 0 : 1;
    __syncwarp();
    float* rec = which == 0 ? head_rec : tail_rec;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      *reinterpret_cast<float4*>(rec + h0 * D + lr * (D / 8) + 4 * i) = make_float4(z0[4 * i], z0[4 * i + 1], z0[4 * i + 2], z0[4 * i + 3]);
      *reinterpret_cast<float4*>(rec + h1 * D + lr * (D / 8) + 4 * i) = make_float4(z1[4 * i], z1[4 * i + 1], z1[4 * i + 2], z1[4 * i + 3]);
    }
    if (lr == 0) {
      rec[KA_COLS * D + h0] = m0;
      rec[KA_COLS * D + h1] = m1;
      rec[KA_COLS * D + KA_COLS + h0] = l0;
      rec[KA_COLS * D + KA_COLS + h1] = l1;
    }
    if (lane == 0) s_piece[warp][which] = u;
  }
  __syncthreads();

  // ---- join the pieces of the CTA's warps.  Entry 2 w is the head piece of
  // warp w, 2 w + 1 its tail: a unit's pieces stand next to one another.  A warp
  // takes a column of a run of pieces at a time.
  const KaUnit* piece = &s_piece[0][0];
  auto rec_of = [&](int e) {
    return reinterpret_cast<const float*>((e & 1) ? smem + (e >> 1) * KA_RING
                                                  : smem + Lay::REC_OFF + (e >> 1) * Lay::REC * 4);
  };
  const long long my_key = lane < 2 * KA_WARPS ? piece[lane].key : -1;
  const unsigned valid = __ballot_sync(0xffffffffu, my_key >= 0);
  const unsigned before = valid & ((1u << lane) - 1);
  const long long prev = __shfl_sync(0xffffffffu, my_key, before ? 31 - __clz(before) : lane);
  const unsigned starts = __ballot_sync(0xffffffffu, my_key >= 0 && (!before || prev != my_key));
  const long long cta_begin = static_cast<long long>(blockIdx.x) * KA_WARPS * quota;
  const long long cta_end = cta_begin + KA_WARPS * quota;
  // the pages of a unit start, end in this CTA's slots
  auto starts_here = [&](const KaUnit& u) { return u.key + KA_FIXED >= cta_begin; };
  auto ends_here = [&](const KaUnit& u) { return u.key + KA_FIXED + u.pages <= cta_end; };
  constexpr int V = D / 32;  // floats of a lane
  int run = 0;
  for (unsigned left = starts; left; left &= left - 1, ++run) {
    const int e = __ffs(left) - 1;
    const unsigned more = left & (left - 1);
    const unsigned mine = valid & ~((1u << e) - 1) & (more ? (1u << (__ffs(more) - 1)) - 1 : ~0u);
    const KaUnit& u = piece[e];
    const bool from = starts_here(u), here = from && ends_here(u);
    const int cols = u.rows * GRP;
    for (int col = (warp + KA_WARPS - (run * KA_COLS) % KA_WARPS) % KA_WARPS; col < cols; col += KA_WARPS) {
      float M = -INFINITY, L = 0.f, O[V] = {};
      for (unsigned b = mine; b; b &= b - 1) M = fmaxf(M, rec_of(__ffs(b) - 1)[KA_COLS * D + col]);
      for (unsigned b = mine; b; b &= b - 1) {
        const float* r = rec_of(__ffs(b) - 1);
        const float mj = r[KA_COLS * D + col];
        const float w = mj == -INFINITY ? 1.f : exp2f(mj - M);  // a piece that saw nothing holds zeros (or NaN)
        L = fmaf(w, r[KA_COLS * D + KA_COLS + col], L);
#pragma unroll
        for (int i = 0; i < V; ++i) O[i] = fmaf(w, r[col * D + lane * V + i], O[i]);
      }
      if (here) {
        const float inv = L == 0.f ? 0.f : a.v_scale / L;
        uint32_t* dst = reinterpret_cast<uint32_t*>(
            a.o + (static_cast<size_t>(u.row0 + col / GRP) * a.n_q + u.g * GRP + col % GRP) * D + lane * V);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) dst[i] = pack_bf16(O[2 * i] * inv, O[2 * i + 1] * inv);
      } else {
        float* out = a.records + (static_cast<size_t>(blockIdx.x) * 2 + (from ? 1 : 0)) * Lay::REC;
#pragma unroll
        for (int i = 0; i < V; ++i) out[col * D + lane * V + i] = O[i];
        if (lane == 0) {
          out[KA_COLS * D + col] = M;
          out[KA_COLS * D + KA_COLS + col] = L;
        }
      }
    }
  }

  // ---- units cut between CTAs: at most the first and the last run
  __threadfence();
  __syncthreads();
  if (starts == 0) return;
  const int e_first = __ffs(starts) - 1, e_last = 31 - __clz(starts);
  for (int k = 0; k < 2; ++k) {
    if (k == 1 && e_last == e_first) break;
    const KaUnit& u = piece[k == 0 ? e_first : e_last];
    if (starts_here(u) && ends_here(u)) continue;
    const int first = static_cast<int>(udiv(u.key + KA_FIXED, quota * KA_WARPS));
    const int last = static_cast<int>(udiv(u.key + KA_FIXED + u.pages - 1, quota * KA_WARPS));
    if (tid == 0) {
      s_last = atomicAdd(&a.counters[first], 1) == last - first;
      if (s_last) a.counters[first] = 0;  // as the next launch expects it
    }
    __syncthreads();
    if (s_last) {
      __threadfence();
      const int cols = u.rows * GRP, n = last - first + 1;
      auto part = [&](int b) { return a.records + (static_cast<size_t>(first + b) * 2 + (b == 0 ? 1 : 0)) * Lay::REC; };
      // the ring is free: weights [column][n], then 1 / denominators
      float* w = reinterpret_cast<float*>(smem);
      float* inv = w + KA_COLS * gridDim.x;
      for (int col = warp; col < cols; col += KA_WARPS) {
        float M = -INFINITY;
        for (int b = lane; b < n; b += 32) M = fmaxf(M, w[col * n + b] = __ldcg(part(b) + KA_COLS * D + col));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        float L = 0.f;
        for (int b = lane; b < n; b += 32) {
          const float x = w[col * n + b] == -INFINITY ? 1.f : exp2f(w[col * n + b] - M);
          w[col * n + b] = x;
          L = fmaf(x, __ldcg(part(b) + KA_COLS * D + KA_COLS + col), L);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
        if (lane == 0) inv[col] = L == 0.f ? 0.f : a.v_scale / L;
      }
      __syncthreads();
      for (int i = tid; i < cols * D / 4; i += KA_THREADS) {
        const int col = i * 4 / D;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b0 = 0; b0 < n; b0 += 8) {  // 8 loads in flight
          float4 x[8];
#pragma unroll
          for (int b = 0; b < 8; ++b) x[b] = __ldcg(reinterpret_cast<const float4*>(part(min(b0 + b, n - 1))) + i);
#pragma unroll
          for (int b = 0; b < 8; ++b)
            if (b0 + b < n) {
              const float wb = w[col * n + b0 + b];
              O.x = fmaf(wb, x[b].x, O.x);
              O.y = fmaf(wb, x[b].y, O.y);
              O.z = fmaf(wb, x[b].z, O.z);
              O.w = fmaf(wb, x[b].w, O.w);
            }
        }
        const float s1 = inv[col];
        const int ch = i * 4 % D;
        *reinterpret_cast<uint2*>(a.o + (static_cast<size_t>(u.row0 + col / GRP) * a.n_q + u.g * GRP + col % GRP) * D + ch) =
            make_uint2(pack_bf16(O.x * s1, O.y * s1), pack_bf16(O.z * s1, O.w * s1));
      }
    }
    __syncthreads();
  }
}

template <int GRP, int D>
cudaError_t launch_t(const Kv4AttnArgs& a, cudaStream_t stream) {
  const int smem = KaLayout<D>::SMEM;
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(attn_kv4_kernel<GRP, D>), smem);
  if (e != cudaSuccess) return e;
  attn_kv4_kernel<GRP, D><<<a.grid, KA_THREADS, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv4_record_bytes(int head_dim) {
  return (head_dim == 128 ? KaLayout<128>::REC : KaLayout<64>::REC) * sizeof(float);
}

cudaError_t launch_attention_kv4(const Kv4AttnArgs& a, cudaStream_t stream) {
  const int grp = a.n_q / a.n_kv;
#define NF_KV4_CASE(G)                                          \
  if (grp == G) return a.head_dim == 128 ? launch_t<G, 128>(a, stream) : launch_t<G, 64>(a, stream);
  NF_KV4_CASE(1) NF_KV4_CASE(2) NF_KV4_CASE(4) NF_KV4_CASE(8)
#undef NF_KV4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace nf
