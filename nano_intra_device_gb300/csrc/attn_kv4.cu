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
//    relative, exact zero only below 2^-32).  Its lower bits would take a second
//    product with V, 8 matrix instructions beside the 16 of a page, in a kernel bound
//    by issue: 185 us against 168 for the 1000 rows below, 31.5 against 30.7 for the
//    64.  Without them the error of the bf16 output to the formula in 64 bits is 1 %
//    above that of fp32 weights.  The denominators sum the fp32
//    values.  The maximum m is raised only when p, as it is computed, would pass
//    2^15 (a score 2^8 times the maximum's share): beyond 2^24 a score's steps reach
//    what KA_SHIFT - m rounds off, so a bound on the score itself would not keep p
//    within fp16.
//
// The pages come by 16-byte asynchronous copies into a ring of two stages a warp,
// which runs on over the ends of units; nothing but the warp itself waits for
// them.  12 warps of 168 registers and two stages; 8 and 16 warps, rings of three
// and four stages and loads straight to registers were all slower.
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
//
// Measured, heads of 128:
//   1000 rows of 600 positions (median), 64 query and 8 KV heads, 917 MB: 168 us,
//     5.5 TB/s, 0.81 of the copy rate;
//   64 rows of 600, 32 and 8 heads, 70 MB: 31 us; one row of 65,543: 28 us.
// The first is bound by issue: about 105 clocks a page and KV head where the copy
// rate gives 98, with 60 % of the issue slots and 54 % of the arithmetic pipe
// (conversions, integer work) in use and the rest lost to fixed latencies.  The
// other two are bound by latency: 3 us of launch, 3 to find the slots, 5 to 7 for
// the last CTA's joins, whose code runs once and comes from memory.
#include <type_traits>

#include "common.cuh"
#include "kv4.cuh"
#include "kv4.h"
#include "mma_frag.cuh"

namespace nf {
namespace {

constexpr int KA_WARPS = 12;
constexpr int KA_THREADS = KA_WARPS * 32;
constexpr int KA_COLS = 8;
constexpr int KA_STAGES = 2;       // ring stages of a warp
constexpr int KA_GROUP = 4608;     // bytes of a stage: 2 pages at d = 128, 4 at d = 64
constexpr int KA_QUEUE = 8;        // pieces from what is worked on to what is fetched: at most one
                                   // a stage, the batch in use and the one after it
// Slots a unit costs beside its pages (query, epilogue, joins).  1000 rows of the
// table below at 1, 3, 5, 8, 12: 182, 171, 167, 170, 176 us; one long row 31, 30,
// 28, 30, 29; 64 rows 31, 30, 31, 31, 31.
constexpr uint32_t KA_FIXED = 5;
constexpr uint32_t KA_MIN_QUOTA = 8;  // fewest slots of a warp (1, 4, 8: the same)
constexpr float KA_LAZY = 8.f;
constexpr float KA_SHIFT = 7.f;
// What stands for -m where nothing was seen: any score passes the maximum, and a
// hidden one stays -infinity.
constexpr float KA_UNSEEN = 3.402823466e38f;

template <int D>
struct KaLayout {
  static constexpr int SLOT = 18 * D;                    // bytes of a (page, KV head)
  static constexpr int PG = KA_GROUP / SLOT;             // pages of a stage
  static constexpr int RING = KA_STAGES * KA_GROUP;
  static constexpr int REC = KA_COLS * D + 2 * KA_COLS;  // floats: O [column][d], m, l
  // a warp's ring, which also takes its last cut unit; its first cut unit
  static constexpr int REC_OFF = KA_WARPS * RING;
  static constexpr int SMEM = REC_OFF + KA_WARPS * REC * 4;
  static_assert(KA_GROUP % SLOT == 0 && REC * 4 <= RING, "a record fits a drained ring");
};

// Page row of operand row r (of 8): neighbours (K: the two rows of eight lanes)
// differ in parity, and so do the rows 2t of t = 0 .. 3 in turn (V), which keeps
// the shared-memory reads of K free of bank conflicts and those of V two-way.
__device__ __forceinline__ int pos_of(int r) {
  return static_cast<int>((0x65742130u >> (4 * (r & 7))) & 7u);
}

// A warp's part of one (request, column group, KV head) unit: pages [p0, p1).
struct __align__(16) KaPiece {
  uint32_t key;   // the unit's first slot; ~0u: none
  int g;          // KV head
  int row0;       // first row in q and o
  int rows;       // live rows (1 .. 8 / GRP)
  int len;        // positions row row0 sees (may be <= 0)
  int pages;      // pages of the request
  int p0, p1;
};
constexpr uint32_t KA_NONE = ~0u;

// Rows, visible length, pages and column groups of request s (0 groups: not ours).
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
  q.groups = q.rows > a.small_rows ? 0 : (q.rows + RG - 1) / RG;
  return q;
}
__device__ __forceinline__ long long ka_slots(const KaSeq& q, int n_kv) {
  return static_cast<long long>(q.pages + static_cast<int>(KA_FIXED)) * q.groups * n_kv;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with nothing to add to
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
template <int W>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[W]) {
  if constexpr (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// x times the low (0) or high (1) half of s
template <int H>
__device__ __forceinline__ uint32_t hmul2_half(uint32_t x, uint32_t s) {
  uint32_t r;
  if (H == 0)
    asm("{.reg .b16 l, h; .reg .b32 t; mov.b32 {l, h}, %2; mov.b32 t, {l, l}; mul.rn.f16x2 %0, %1, t;}" : "=r"(r) : "r"(x), "r"(s));
  else
    asm("{.reg .b16 l, h; .reg .b32 t; mov.b32 {l, h}, %2; mov.b32 t, {h, h}; mul.rn.f16x2 %0, %1, t;}" : "=r"(r) : "r"(x), "r"(s));
  return r;
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
  constexpr int SLOT = Lay::SLOT, PG = Lay::PG;
  constexpr int KW = D / 32;             // words of a thread's K codes in a row
  constexpr int VW = D / 64;             // words of a thread's V codes in a row
  constexpr int KS = D / 16;             // k-steps of S, m-tiles of O
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_warp[KA_WARPS];
  __shared__ uint32_t s_base[KA_WARPS];  // where each warp starts: a request's first slot and the request
  __shared__ int s_seq[KA_WARPS];
  __shared__ KaPiece s_queue[KA_WARPS][KA_QUEUE];
  __shared__ KaPiece s_piece[KA_WARPS][2];  // what a warp leaves for the CTA to join
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lr = lane >> 2, lc = lane & 3;
  if (lane == 0) s_piece[warp][0].key = s_piece[warp][1].key = KA_NONE;

  // ---- the slots of every request: thread i sums the requests [i c, (i + 1) c)
  const int c = (a.n_seq + KA_THREADS - 1) / KA_THREADS;
  uint32_t total, quota;
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
    long long before = in - sum, all = 0;
#pragma unroll
    for (int w = 0; w < KA_WARPS; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    if (all > 0xFFF00000ll) {  // 10 TB of pages: not a call that ends
      if (blockIdx.x == 0 && tid == 0) raise_status(a.status, ST_OVERFLOW);
      pdl_wait();
      return;
    }
    total = static_cast<uint32_t>(all);
    const uint32_t n_warps = gridDim.x * KA_WARPS;
    quota = max((total + n_warps - 1) / n_warps, KA_MIN_QUOTA);
    const uint32_t cta0 = blockIdx.x * KA_WARPS * quota;
    if (cta0 >= total) {  // nothing for this CTA
      pdl_wait();
      return;
    }
    // the thread whose requests hold a warp's first slot says where it starts
    uint32_t at = static_cast<uint32_t>(before);
    if (sum > 0 && at < cta0 + KA_WARPS * quota && at + static_cast<uint32_t>(sum) > cta0) {
      uint32_t w = at <= cta0 ? 0 : (at - cta0 + quota - 1) / quota;
      uint32_t x = cta0 + w * quota;
      for (int s = s0; s < s1 && w < KA_WARPS; ++s) {
        const uint32_t n = static_cast<uint32_t>(ka_slots(ka_seq<RG>(a, s, false), a.n_kv));
        while (w < KA_WARPS && x < at + n) {
          s_base[w] = at;
          s_seq[w] = s;
          ++w;
          x += quota;
        }
        at += n;
      }
    }
    __syncthreads();
  }
  const uint32_t wid = blockIdx.x * KA_WARPS + warp;
  const uint32_t end = min((wid + 1) * quota, total);
  uint32_t x = wid * quota;  // next slot of this warp
  int s = 0;
  uint32_t base = 0;         // first slot of request s
  KaSeq sq{0, 0, 0, 0, 0};
  if (x < end) {
    s = s_seq[warp];
    base = s_base[warp];
    sq = ka_seq<RG>(a, s, false);
  }
  const int h0 = 2 * lc, h1 = 2 * lc + 1;
  const int i0 = h0 / GRP, i1 = h1 / GRP;  // rows of this lane's accumulator columns
  auto out_row = [&](const KaPiece& u, int col) {
    return a.o + (static_cast<size_t>(u.row0 + col / GRP) * a.n_q + u.g * GRP + col % GRP) * D;
  };

  // ---- what is fetched.  A batch is up to 32 pages of one piece, an id a lane;
  // the next batch's ids are on their way while this one's pages are requested.
  // Batches run over the ends of pieces, so a unit's first pages arrive while the
  // one before it is worked on; the pieces wait in a queue meanwhile.
  KaPiece np;               // the piece the next batch belongs to
  np.p0 = np.p1 = 0;
  int np_s = 0;             // its request
  int np_at = 0;            // its next page to batch
  uint32_t pushed = 0, popped = 0;
  auto next_piece = [&]() -> bool {
    while (x < end) {
      const uint32_t per = sq.pages + KA_FIXED;
      const uint32_t past = base + per * static_cast<uint32_t>(sq.groups) * static_cast<uint32_t>(a.n_kv);
      if (x >= past) {  // next request
        base = past;
        if (++s >= a.n_seq) return false;
        sq = ka_seq<RG>(a, s, false);
        continue;
      }
      const uint32_t k = (x - base) / per;
      np.key = base + k * per;
      const int grp0 = static_cast<int>(k / a.n_kv) * RG;  // first row of the group in the request
      np.g = static_cast<int>(k % a.n_kv);
      np.row0 = sq.b0 + grp0;
      np.rows = min(RG, sq.rows - grp0);
      np.len = sq.len - sq.rows + grp0 + 1;
      np.pages = sq.pages;
      const uint32_t off = x - np.key;
      np.p0 = off > KA_FIXED ? static_cast<int>(off - KA_FIXED) : 0;
      np.p1 = static_cast<int>(min(end - np.key, per)) - static_cast<int>(KA_FIXED);
      x = min(end, np.key + per);
      if (np.pages == 0) {  // nothing to see: zeros, by the warp of the unit's first slot
        if (off == 0) {
          const float z[D / 8] = {};
          if (i0 < np.rows) store_row(out_row(np, h0) + lr * (D / 8), z);
          if (i1 < np.rows) store_row(out_row(np, h1) + lr * (D / 8), z);
        }
        continue;
      }
      if (np.p1 > np.p0) {  // else only slots of the fixed cost
        np_s = s;
        np_at = np.p0;
        return true;
      }
    }
    np.p0 = np.p1 = np_at = 0;
    return false;
  };
  int ids = 0, cnt = 0, at = 0, bg = 0;  // batch in use: ids, pages, next page, KV head
  int ids2 = 0, cnt2 = 0, bg2 = 0;       // batch after it
  auto load_batch = [&]() {              // -> ids2
    cnt2 = 0;
    if (np_at >= np.p1) {
      if (!next_piece()) return;
      if (lane == 0) s_queue[warp][pushed % KA_QUEUE] = np;
      ++pushed;
    }
    cnt2 = min(32, np.p1 - np_at);
    bg2 = np.g;
    ids2 = 0;
    if (lane < cnt2) {
      ids2 = a.block_table[static_cast<size_t>(np_s) * a.max_pages + np_at + lane];
      if (ids2 < 0 || ids2 >= a.num_pages) {  // never read outside the pool
        raise_status(a.status, ST_BAD_PAGE);
        ids2 = 0;
      }
    }
    np_at += cnt2;
  };
  const uint32_t ring = smem_u32(smem + warp * Lay::RING);
  constexpr int CHUNKS = SLOT / 16;  // 16-byte chunks of a page
  // Request the next group of pages (of one piece) into stage st.
  auto fetch = [&](int st) {
    if (at >= cnt) {
      ids = ids2;
      cnt = cnt2;
      bg = bg2;
      at = 0;
      load_batch();
    }
    const int n = min(PG, cnt - at);
    if (n > 0) {
      const uint8_t* src[PG];
#pragma unroll
      for (int i = 0; i < PG; ++i) {
        const int page = __shfl_sync(0xffffffffu, ids, (at + i) & 31);
        src[i] = a.pool + (static_cast<size_t>(page) * a.n_kv + bg) * SLOT;
      }
      const uint32_t dst = ring + st * KA_GROUP + lane * 16;
#pragma unroll
      for (int k = 0; k < KA_GROUP / 512; ++k) {  // chunk 32 k + lane of the group
        const int lo = 32 * k / CHUNKS, hi = (32 * k + 31) / CHUNKS;  // its page: one, or one of two
        const int pgi = lo == hi || lane < hi * CHUNKS - 32 * k ? lo : hi;
        const uint8_t* p = (pgi == lo ? src[lo] - lo * SLOT : src[hi] - hi * SLOT) + 512 * k + lane * 16;
        if (pgi < n) cp_async16(dst + 512 * k, p);
      }
      at += n;
    }
    cp_async_commit();  // also when empty: groups and commits stay in step
  };

  load_batch();
#pragma unroll
  for (int i = 0; i < KA_STAGES; ++i) fetch(i);

  // ---- what is worked on
  const int kr = pos_of(lr);                       // page rows kr, kr + 8 of this thread's K
  const int va = pos_of(2 * lc), vb = pos_of(2 * lc + 1);  // and va, vb, + 8 of its V
  const uint8_t* my_k = smem + warp * Lay::RING + kr * (D / 2) + lc * (D / 8);
  const uint8_t* my_ks = smem + warp * Lay::RING + 8 * D + kr * (D / 16) + lc * (D / 64);
  const uint8_t* my_va = smem + warp * Lay::RING + 9 * D + va * (D / 2) + lr * (D / 16);
  const uint8_t* my_vb = smem + warp * Lay::RING + 9 * D + vb * (D / 2) + lr * (D / 16);
  const uint8_t* my_sa = smem + warp * Lay::RING + 17 * D + va * (D / 16) + (lr * (D / 8)) / 16;
  const uint8_t* my_sb = smem + warp * Lay::RING + 17 * D + vb * (D / 16) + (lr * (D / 8)) / 16;
  int st = 0;
  __syncwarp();
  while (popped != pushed) {
    __syncwarp();  // lane 0 has queued it
    const KaPiece u = s_queue[warp][popped % KA_QUEUE];
    ++popped;
    const int npg = u.p1 - u.p0;

    // Q^T as the B operand: column lr, this thread's channels [lc d/4, ..) in
    // pairs 4 j + {0, 1} and 4 j + {2, 3}
    uint32_t qb[KS][2];
    float2 sc2;  // scales of the columns h0, h1
    {
      const bool live = lr / GRP < u.rows;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<size_t>(u.row0 + (live ? lr / GRP : 0)) * a.n_q + u.g * GRP + lr % GRP) * D + lc * (D / 4));
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
      // an infinity makes every score of the vector infinite or NaN, and their softmax
      // NaN, also where all are -inf, which would pass for hidden ones
      const float mul = top == INFINITY ? __int_as_float(0x7FC00000) : exp2_int(kq);
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qb[j][i] = pack_f16(bf16lo(raw[2 * j + i]) * mul, bf16hi(raw[2 * j + i]) * mul);
      const float back = a.scale_log2 * exp2_int(-kq);
      sc2.x = __shfl_sync(0xffffffffu, back, h0 * 4);
      sc2.y = __shfl_sync(0xffffffffu, back, h1 * 4);
    }
    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY;          // reference maxima of the columns h0, h1 (base 2)
    float2 n2 = make_float2(KA_UNSEEN, KA_UNSEEN); // what p's exponent adds: KA_SHIFT - m
    float2 l2 = make_float2(0.f, 0.f);             // this lane's share of the denominators
    const int plim = u.p1 * KV4_P;  // positions past the piece are another warp's
    const int lim0 = min(u.len + i0, plim), lim1 = min(u.len + i1, plim);  // the first hidden positions
    const int most = min(u.len + u.rows - 1, plim);                        // and of the unit's last row
    const int clear = min(u.len, plim);  // before it every column sees everything

    // A group of pages from position pb on, `off` bytes into the ring.  EDGE: some
    // column does not see all of it.
    auto step = [&](const int pb, const int off, auto edge_) {
      constexpr bool EDGE = decltype(edge_)::value;
      float sc[PG][4];
#pragma unroll
      for (int p = 0; p < PG; ++p) {
        const int at_p = off + p * SLOT;
        uint32_t ka[KW], kb[KW];
        lds_words(my_k + at_p, ka);
        lds_words(my_k + at_p + 8 * (D / 2), kb);
        uint32_t sa, sb;  // scales as f16 pairs; d = 64: one each
        if (D == 128) {
          sa = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(my_ks + at_p));
          sb = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(my_ks + at_p + 8 * (D / 16)));
        } else {
          sa = e4m3x2_to_f16x2(my_ks[at_p]);
          sb = e4m3x2_to_f16x2(my_ks[at_p + 8 * (D / 16)]);
        }
        float acc[4];
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          if (j == 0)
            mma_f16_zero(acc, hmul2_half<0>(code_pair(ka, 0), sa), hmul2_half<0>(code_pair(kb, 0), sb),
                         hmul2_half<0>(code_pair(ka, 1), sa), hmul2_half<0>(code_pair(kb, 1), sb), qb[0][0], qb[0][1]);
          else if (j < 4)
            mma_f16(acc, hmul2_half<0>(code_pair(ka, 2 * j), sa), hmul2_half<0>(code_pair(kb, 2 * j), sb),
                    hmul2_half<0>(code_pair(ka, 2 * j + 1), sa), hmul2_half<0>(code_pair(kb, 2 * j + 1), sb), qb[j][0], qb[j][1]);
          else
            mma_f16(acc, hmul2_half<1>(code_pair(ka, 2 * j), sa), hmul2_half<1>(code_pair(kb, 2 * j), sb),
                    hmul2_half<1>(code_pair(ka, 2 * j + 1), sa), hmul2_half<1>(code_pair(kb, 2 * j + 1), sb), qb[j][0], qb[j][1]);
        }
        // scaled scores, base 2: (position kr, h0), (kr, h1), (kr + 8, h0), (kr + 8, h1)
        const float2 lo = __fmul2_rn(make_float2(acc[0], acc[1]), sc2), hi = __fmul2_rn(make_float2(acc[2], acc[3]), sc2);
        sc[p][0] = lo.x;
        sc[p][1] = lo.y;
        sc[p][2] = hi.x;
        sc[p][3] = hi.y;
      }
      unsigned bad = 0;  // NaN values of V at this thread's positions: bit 2 page + half
      if (EDGE) {
        // A NaN of V must reach the columns that see it and no other, so it
        // goes through P instead of V (0 * NaN is NaN).
#pragma unroll
        for (int p = 0; p < PG; ++p)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int pos = pb + p * KV4_P + kr + 8 * i;
            if (pos >= lim0) sc[p][2 * i] = -INFINITY;
            if (pos >= lim1) sc[p][2 * i + 1] = -INFINITY;
            const uint8_t* vs = smem + warp * Lay::RING + off + p * SLOT + 17 * D + (kr + 8 * i) * (D / 16);
            for (int b = 0; b < D / 16; ++b)
              if (scale_nan(vs[b])) bad |= 1u << (2 * p + i);
          }
      }
      float x0 = fmaxf(sc[0][0], sc[0][2]), x1 = fmaxf(sc[0][1], sc[0][3]);
#pragma unroll
      for (int p = 1; p < PG; ++p) {
        x0 = fmaxf(x0, fmaxf(sc[p][0], sc[p][2]));
        x1 = fmaxf(x1, fmaxf(sc[p][1], sc[p][3]));
      }
      if (__any_sync(0xffffffffu, x0 + n2.x > KA_LAZY + KA_SHIFT || x1 + n2.y > KA_LAZY + KA_SHIFT)) {
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
        l2.x *= c0;
        l2.y *= c1;
        m0 = r0;
        m1 = r1;
        n2.x = m0 == -INFINITY ? KA_UNSEEN : KA_SHIFT - m0;
        n2.y = m1 == -INFINITY ? KA_UNSEEN : KA_SHIFT - m1;
      }
      uint32_t pt[PG][2];
#pragma unroll
      for (int p = 0; p < PG; ++p) {
        // the scaled scores are rounded before the maximum is taken off (no fused
        // step), as where the largest was compared
        float2 lo = __fadd2_rn(make_float2(sc[p][0], sc[p][1]), n2), hi = __fadd2_rn(make_float2(sc[p][2], sc[p][3]), n2);
        lo.x = ex2_approx(lo.x);
        lo.y = ex2_approx(lo.y);
        hi.x = ex2_approx(hi.x);
        hi.y = ex2_approx(hi.y);
        if (EDGE && bad) {
          const float nan = __int_as_float(0x7FC00000);
          const int pos = pb + p * KV4_P + kr;
          if ((bad >> (2 * p)) & 1) {
            if (pos < lim0) lo.x = nan;
            if (pos < lim1) lo.y = nan;
          }
          if ((bad >> (2 * p + 1)) & 1) {
            if (pos + 8 < lim0) hi.x = nan;
            if (pos + 8 < lim1) hi.y = nan;
          }
        }
        l2 = __fadd2_rn(l2, __fadd2_rn(lo, hi));
        pt[p][0] = movmatrix_trans(pack_f16(lo.x, lo.y));  // operand rows 2 lc (+1), column lr
        pt[p][1] = movmatrix_trans(pack_f16(hi.x, hi.y));  // and 8 on
      }
#pragma unroll
      for (int p = 0; p < PG; ++p) {
        const int at_p = off + p * SLOT;
        uint32_t v0[VW], v1[VW], v2[VW], v3[VW];
        lds_words(my_va + at_p, v0);
        lds_words(my_vb + at_p, v1);
        lds_words(my_va + at_p + 8 * (D / 2), v2);
        lds_words(my_vb + at_p + 8 * (D / 2), v3);
        uint32_t b0 = my_sa[at_p], b1 = my_sb[at_p], b2 = my_sa[at_p + 8 * (D / 16)], b3 = my_sb[at_p + 8 * (D / 16)];
        if (EDGE) {  // positions no column sees, and NaNs (P has them): nothing
          const int pos = pb + p * KV4_P;
          if (pos + va >= most || scale_nan(b0)) b0 = 0;
          if (pos + vb >= most || scale_nan(b1)) b1 = 0;
          if (pos + va + 8 >= most || scale_nan(b2)) b2 = 0;
          if (pos + vb + 8 >= most || scale_nan(b3)) b3 = 0;
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

    // batches of 32 pages end a group, so a piece's groups start at multiples of PG
    for (int i = 0; i < npg; i += PG) {
      cp_async_wait<KA_STAGES - 1>();
      __syncwarp();
      const int pb = (u.p0 + i) * KV4_P;
      if (pb + PG * KV4_P <= clear) step(pb, st * KA_GROUP, std::false_type{});
      else step(pb, st * KA_GROUP, std::true_type{});
      __syncwarp();
      fetch(st);
      st = st + 1 == KA_STAGES ? 0 : st + 1;
    }

#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l2.x += __shfl_xor_sync(0xffffffffu, l2.x, d);
      l2.y += __shfl_xor_sync(0xffffffffu, l2.y, d);
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
    if (npg == u.pages) {  // the whole unit
      const float r0 = l2.x == 0.f ? 0.f : a.v_scale / l2.x, r1 = l2.y == 0.f ? 0.f : a.v_scale / l2.y;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        z0[i] *= r0;
        z1[i] *= r1;
      }
      if (i0 < u.rows) store_row(out_row(u, h0) + lr * (D / 8), z0);
      if (i1 < u.rows) store_row(out_row(u, h1) + lr * (D / 8), z1);
    } else {
      // a piece: the warp's first when it began in another warp, else its last,
      // after which the ring is free
      const int which = u.p0 > 0 ? 0 : 1;
      if (which) {
        cp_async_wait<0>();
        __syncwarp();
      }
      float* rec = reinterpret_cast<float*>(which ? smem + warp * Lay::RING : smem + Lay::REC_OFF + warp * Lay::REC * 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        *reinterpret_cast<float4*>(rec + h0 * D + lr * (D / 8) + 4 * i) = make_float4(z0[4 * i], z0[4 * i + 1], z0[4 * i + 2], z0[4 * i + 3]);
        *reinterpret_cast<float4*>(rec + h1 * D + lr * (D / 8) + 4 * i) = make_float4(z1[4 * i], z1[4 * i + 1], z1[4 * i + 2], z1[4 * i + 3]);
      }
      if (lr == 0) {
        rec[KA_COLS * D + h0] = m0;
        rec[KA_COLS * D + h1] = m1;
        rec[KA_COLS * D + KA_COLS + h0] = l2.x;
        rec[KA_COLS * D + KA_COLS + h1] = l2.y;
      }
      if (lane == 0) s_piece[warp][which] = u;
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // ---- join the pieces of the CTA's warps.  Entry 2 w is the head piece of
  // warp w, 2 w + 1 its tail: a unit's pieces stand next to one another.  A warp
  // takes a column of a run of pieces at a time.
  const KaPiece* piece = &s_piece[0][0];
  auto rec_of = [&](int e) {
    return reinterpret_cast<const float*>((e & 1) ? smem + (e >> 1) * Lay::RING
                                                  : smem + Lay::REC_OFF + (e >> 1) * Lay::REC * 4);
  };
  const uint32_t my_key = lane < 2 * KA_WARPS ? piece[lane].key : KA_NONE;
  const unsigned valid = __ballot_sync(0xffffffffu, my_key != KA_NONE);
  const unsigned before = valid & ((1u << lane) - 1);
  const uint32_t prev = __shfl_sync(0xffffffffu, my_key, before ? 31 - __clz(before) : lane);
  const unsigned starts = __ballot_sync(0xffffffffu, my_key != KA_NONE && (!before || prev != my_key));
  const uint32_t cta_begin = blockIdx.x * KA_WARPS * quota, cta_end = cta_begin + KA_WARPS * quota;
  // the pages of a unit start, end in this CTA's slots
  auto starts_here = [&](const KaPiece& u) { return u.key + KA_FIXED >= cta_begin; };
  auto ends_here = [&](const KaPiece& u) { return u.key + KA_FIXED + u.pages <= cta_end; };
  constexpr int V = D / 32;  // floats of a lane
  int run = 0;
  for (unsigned left = starts; left; left &= left - 1, ++run) {
    const int e = __ffs(left) - 1;
    const unsigned more = left & (left - 1);
    const unsigned mine = valid & ~((1u << e) - 1) & (more ? (1u << (__ffs(more) - 1)) - 1 : ~0u);
    const KaPiece& u = piece[e];
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
  if (starts == 0) {
    pdl_wait();
    return;
  }
  const int e_first = __ffs(starts) - 1, e_last = 31 - __clz(starts);
  for (int k = 0; k < 2; ++k) {
    if (k == 1 && e_last == e_first) break;
    const KaPiece& u = piece[k == 0 ? e_first : e_last];
    if (starts_here(u) && ends_here(u)) continue;
    const int first = static_cast<int>((u.key + KA_FIXED) / (quota * KA_WARPS));
    const int last = static_cast<int>((u.key + KA_FIXED + u.pages - 1) / (quota * KA_WARPS));
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
  pdl_wait();
}

// Behind the tiles' launch the CTAs start on the SMs that it leaves: the two
// touch no common data, so only the end waits (pdl_wait at every exit; a no-op
// otherwise), which makes the stream's next launch wait for both.
template <int GRP, int D>
cudaError_t launch_t(const Kv4AttnArgs& a, bool behind, cudaStream_t stream) {
  const int smem = KaLayout<D>::SMEM;
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(attn_kv4_kernel<GRP, D>), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.grid), 1, 1);
  cfg.blockDim = dim3(KA_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_kv4_kernel<GRP, D>, a);
}

}  // namespace

size_t kv4_record_bytes(int head_dim) {
  return (head_dim == 128 ? KaLayout<128>::REC : KaLayout<64>::REC) * sizeof(float);
}

cudaError_t launch_attention_kv4(const Kv4AttnArgs& a, bool behind, cudaStream_t stream) {
  const int grp = a.n_q / a.n_kv;
#define NF_KV4_CASE(G)                                          \
  if (grp == G) return a.head_dim == 128 ? launch_t<G, 128>(a, behind, stream) : launch_t<G, 64>(a, behind, stream);
  NF_KV4_CASE(1) NF_KV4_CASE(2) NF_KV4_CASE(4) NF_KV4_CASE(8)
#undef NF_KV4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace nf
