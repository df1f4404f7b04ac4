// Causal attention of the rows of longer chunks over the 4-bit KV cache, on the
// 5th-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// A tile is 128 query vectors: 128 / GRP consecutive rows of one request and the
// GRP query heads of one KV head; a unit is two neighbouring tiles.  Per key
// block of 128 positions and tile
//   S = Q K^T   (M 128, N 128, K d),   O += P V   (M 128, N d, K 128),
// both with fp16 operands and fp32 accumulators.
//  * Four warps turn codes into fp16 operands: a lane loads half a row of a page
//    (a scale for every 16 channels), converts a byte an instruction, multiplies
//    by the scale (exact, see attn_kv4.cu) and stores 16-byte chunks in the
//    128-byte swizzle the products read; K has a ring of its own, V another.
//    The next block's codes are in registers while the ring is full.  Both tiles
//    use a block's operands: with one tile a CTA these four warps took issue
//    slots and shared memory from the softmax of every block (299 us against 290
//    in the case below).
//  * One thread issues the products, tile by tile: P V of one tile and its next S
//    run while the other tile's softmax does.  S of a tile stands in 128 columns
//    of tensor memory, P over their first half; the next S waits until P is read,
//    as products into different accumulators have no order of their own (12 us).
//  * Four softmax warps a tile, a thread a row: no exchange between threads.
//    Online softmax with a lazily raised maximum (base 2), P as fp16 of 2^7 times
//    its share of the running maximum, denominators summed in fp32.
// Q is scaled by a power of two a vector so that fp16 holds all of bf16's bits.
//
// Work split: the key blocks of all (unit, KV head) pairs are laid end to end
// (closed-form sums, as a unit's blocks grow with its position) and every CTA
// takes the same number.  A unit cut between CTAs is joined by the CTA that
// arrives last, from fp32 records in the handle's workspace, in the order of the
// pieces.  So a short chunk over a long prefix fills the GPU like a long prompt.
// The rings run on over the ends of units.
//
// Measured (1985 rows over 4099 positions, 32 query and 8 KV heads of 128, 166
// GFLOP, beside 63 decode rows): 221 us for this kernel, 244 for the
// call, 36 % of the cuBLAS bf16 rate.  What bounds it: the softmax warps, two on each of an
// SM's four schedulers, which issue in a third of the cycles; they wait for scores
// and for their own chains, and a sixth of the waits is for instructions (four
// roles' unrolled loops).  Tried and slower: two threads a row with the tiles one
// after the other (290; three quarters of the scores' reads and an exchange of
// maxima a block), four threads a row (354: 80 registers, spills), exponentials
// by the old maximum before the new one is known (327), P through shared memory
// with S issued ahead (274), S in two halves around the wait for P (355), one lane
// polling for its warp (387 against 309).
//
// Every wait is bounded; on expiry the kernel flags ST_TIMEOUT and every role
// leaves its loop.  Whichever role gave up, the products issued and the stores into
// tensor memory finish before it is freed; that wait has a limit of its own, as the
// caller's may be shorter than a product.
#include "common.cuh"
#include "kv4.cuh"
#include "kv4.h"
#include "mma_frag.cuh"

namespace nf {
namespace {

constexpr int KP_DQ_WARPS = 4;       // warps that make operands: two for K, two for V
constexpr int KP_SM_WARPS = 8;       // softmax warps: four a tile, one a tensor-memory lane quarter
constexpr int KP_MMA_WARP = KP_DQ_WARPS + KP_SM_WARPS;
constexpr int KP_WARPS = 16;         // registers are dealt by warpgroups of four: the last holds the
                                     // MMA warp and three that only take part in the prologue
constexpr int KP_THREADS = KP_WARPS * 32;
// 512 = 4 x 128 registers a thread at launch, dealt again by role (104 / 176 / 56:
// 245 us against 243, 96 / 184 / 48: 251)
constexpr int KP_DQ_REGS = 80, KP_SM_REGS = 184, KP_MMA_REGS = 64;
static_assert(KP_DQ_REGS + 2 * KP_SM_REGS + KP_MMA_REGS == 512, "the shares of the launch's registers");
constexpr int KP_M = 128;            // query vectors of a tile (tensor-memory lanes)
constexpr int KP_N = 128;            // positions of a key block
constexpr int KP_REGION = 128 * 128; // 128 rows x 128 bytes: 64 fp16 columns of 128 rows
constexpr int KP_FIXED = 1;          // blocks' worth of a unit's fixed cost (2, 4: 235, 232 us)
constexpr float KP_SLACK = 8.f;
constexpr float KP_SHIFT = 7.f;
constexpr float KP_UNSEEN = 3.402823466e38f;  // stands for -m where nothing was seen
constexpr uint32_t KP_TMEM_COLS = 512;
constexpr int KP_KST = 2, KP_VST = 2;  // ring stages of K and V
constexpr uint64_t KP_DRAIN_NS = 2000000000ull;

struct KpBars {
  uint64_t q_full[2];                        // by tile: its softmax warps have written Q
  uint64_t k_full[KP_KST], k_empty[KP_KST];  // full: two warps
  uint64_t v_full[KP_VST], v_empty[KP_VST];
  uint64_t s_full[2];                        // by tile: S of a block, and all products before it
  uint64_t p_full[2];                        // its softmax warps: P written (and O rescaled)
  uint64_t pv_done[2];                       // P is read: S of the next block may take its columns
  uint64_t o_full[2];                        // the last product of a piece
  uint64_t meet[2];                          // a bounded barrier of a tile's softmax warps
  uint64_t drain;
  uint32_t tmem_base;
  int abort, last[2];
  uint32_t v_nan[KP_VST][4];                 // positions whose V holds a NaN that not every row sees
  long long warp_sum[KP_WARPS];
  long long base;                            // where this CTA starts: a request's first slot
  int seq;                                   // and the request
};

template <int NCH>
struct KpLayout {
  static constexpr int D = NCH * 64;
  static constexpr int Q_BYTES = NCH * KP_REGION;   // [d/64][128 vectors][128 B]
  static constexpr int KV_BYTES = NCH * KP_REGION;  // 16 groups of 8 positions, each [d/64][8][128 B]
  static constexpr int KV_GROUP = NCH * 1024;
  static constexpr int K_OFF = 2 * Q_BYTES;
  static constexpr int V_OFF = K_OFF + KP_KST * KV_BYTES;
  static constexpr int BAR_OFF = V_OFF + KP_VST * KV_BYTES;
  static constexpr int SMEM = 1024 + BAR_OFF + static_cast<int>(sizeof(KpBars));
  static constexpr int TREC = KP_M * D + 2 * KP_M;  // floats of a tile's record: O, m, l
  static constexpr int REC = 2 * TREC;
};

template <int N>
__device__ __forceinline__ void kp_regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void kp_regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
// 32 lanes x 16 columns, as the 32-column forms.
__device__ __forceinline__ void tc_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tc_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// tcgen05.mma with A in tensor memory: a column holds two neighbours along K.
__device__ __forceinline__ void kp_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f16: fp16 A and B, fp32 D; B K-major or MN-major.
constexpr uint32_t kp_idesc(int M, int N, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24) | (b_mn ? 1u << 16 : 0u);
}

// A unit is R = 256 / GRP rows.  Its last row's limit lies k steps of R positions
// past a multiple of R: ceil(k / h) blocks, h = 128 / R, at least one; kp_sum is
// their sum over 1 .. m (m <= 0: minus one a step).  At GRP = 1 the step is a
// block, two a unit.
__device__ __forceinline__ long long kp_sum(long long m, int h) {
  if (m <= 0) return m;
  const long long q = m / h, r = m % h;
  return h * q * (q + 1) / 2 + r * (q + 1);
}

struct KpSeq {
  int b0, rows, len, units;
  long long c;  // steps up to the first row
};
template <int GRP>
__device__ __forceinline__ KpSeq kp_seq(const Kv4AttnArgs& a, int s) {
  constexpr int R = 2 * KP_M / GRP, U = R < KP_N ? R : KP_N;
  KpSeq q;
  const int b0 = a.tok_begin[s], b1 = a.tok_begin[s + 1];
  q.b0 = b0;
  q.rows = b0 < 0 || b1 < b0 || b1 > a.n_tok ? 0 : b1 - b0;
  q.len = a.seq_lens[s];
  if (q.len < 0 || q.len > static_cast<long long>(a.max_pages) * KV4_P) q.len = 0;
  q.units = q.rows > a.small_rows ? (q.rows + R - 1) / R : 0;
  const int first = q.len - q.rows;  // position of the first row
  q.c = first >= 0 ? (first + U - 1) / U : -(-first / U);
  return q;
}
template <int GRP>
__device__ __forceinline__ long long kp_blocks(const KpSeq& q, int i) {
  const long long k = GRP == 1 ? q.c + 2 * (i + 1LL) : q.c + i + 1;
  constexpr int h = GRP == 1 ? 1 : GRP / 2;
  return k <= 0 ? 1 : (k + h - 1) / h;
}
// Slots before unit i of a request.
template <int GRP>
__device__ __forceinline__ long long kp_before(const KpSeq& q, int i, int n_kv) {
  long long blocks;
  if (GRP == 1) {
    const long long one = min(static_cast<long long>(i), q.c < 0 ? -q.c / 2 : 0);  // units of one block
    blocks = one + (i - one) * q.c + i * (i + 1LL) - one * (one + 1);
  } else {
    blocks = kp_sum(q.c + i, GRP / 2) - kp_sum(q.c, GRP / 2);
  }
  return n_kv * (blocks + static_cast<long long>(i) * KP_FIXED);
}

struct KpPiece {
  long long key;      // the unit's first slot
  int s, g;
  int row0, rows;     // rows of q and o
  int pos0;           // position of row0 (may be negative)
  int len;            // positions of the request
  int nb, j0, j1;     // blocks of the unit, and those of this piece
  int nt;             // tiles of the unit: 1 or 2
};

// Walks the pieces of a CTA's slots; every warp keeps one.
template <int GRP>
struct KpWalk {
  long long x, end, base;
  int s;
  KpSeq q;
  __device__ __forceinline__ bool next(const Kv4AttnArgs& a, KpPiece& p) {
    constexpr int R = 2 * KP_M / GRP;
    while (x < end) {
      const long long all = kp_before<GRP>(q, q.units, a.n_kv);
      if (x >= base + all) {
        base += all;
        if (++s >= a.n_seq) return false;
        q = kp_seq<GRP>(a, s);
        continue;
      }
      int lo = 0, hi = q.units - 1;  // the last unit that starts at or before x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base + kp_before<GRP>(q, mid, a.n_kv) <= x) lo = mid;
        else hi = mid - 1;
      }
      const long long t0 = base + kp_before<GRP>(q, lo, a.n_kv);
      p.nb = static_cast<int>(kp_blocks<GRP>(q, lo));
      const int per = p.nb + KP_FIXED;
      p.g = static_cast<int>((x - t0) / per);
      p.key = t0 + static_cast<long long>(p.g) * per;
      p.s = s;
      p.row0 = q.b0 + lo * R;
      p.rows = min(R, q.rows - lo * R);
      p.nt = p.rows > R / 2 ? 2 : 1;
      p.pos0 = q.len - q.rows + lo * R;
      p.len = q.len;
      const int off = static_cast<int>(x - p.key);
      p.j0 = max(off - KP_FIXED, 0);
      p.j1 = static_cast<int>(min(end - p.key, static_cast<long long>(per))) - KP_FIXED;
      x = min(end, p.key + per);
      if (p.j1 > p.j0) return true;
    }
    return false;
  }
};

template <int GRP, int NCH>
__global__ void __launch_bounds__(KP_THREADS, 1) attn_kv4_prefill_kernel(const Kv4AttnArgs a) {
  using Lay = KpLayout<NCH>;
  constexpr int D = Lay::D;
  constexpr uint32_t IDESC_S = kp_idesc(KP_M, KP_N, false);
  constexpr uint32_t IDESC_PV = kp_idesc(KP_M, D, true);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sbase = smem_u32(smem);
  KpBars* bars = reinterpret_cast<KpBars*>(smem + Lay::BAR_OFF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t tmo = a.timeout_ns;

  pdl_trigger();  // the launch of few rows takes the SMs that this one leaves

  // ---- the slots of every request: thread i sums the requests [i c, (i + 1) c)
  KpWalk<GRP> walk;
  long long quota;
  {
    const int c = (a.n_seq + KP_THREADS - 1) / KP_THREADS;
    const int s0 = min(static_cast<long long>(a.n_seq), static_cast<long long>(tid) * c), s1 = min(a.n_seq, s0 + c);
    long long sum = 0;
    for (int s = s0; s < s1; ++s) {
      const KpSeq q = kp_seq<GRP>(a, s);
      sum += kp_before<GRP>(q, q.units, a.n_kv);
    }
    long long in = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += y;
    }
    if (lane == 31) bars->warp_sum[warp] = in;
    __syncthreads();
    long long at = in - sum, total = 0;
    for (int w = 0; w < KP_WARPS; ++w) {
      if (w < warp) at += bars->warp_sum[w];
      total += bars->warp_sum[w];
    }
    quota = (total + gridDim.x - 1) / gridDim.x;
    const long long x = blockIdx.x * quota;
    if (x >= total) return;  // nothing for this CTA
    if (at <= x && x < at + sum)
      for (int s = s0; s < s1; ++s) {
        const KpSeq q = kp_seq<GRP>(a, s);
        const long long n = kp_before<GRP>(q, q.units, a.n_kv);
        if (x < at + n) {
          bars->base = at;
          bars->seq = s;
          break;
        }
        at += n;
      }
    walk.x = x;
    walk.end = min(x + quota, total);
  }

  if (tid == 0) {
    for (int i = 0; i < KP_KST; ++i) {
      mbar_init(&bars->k_full[i], 2);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < KP_VST; ++i) {
      mbar_init(&bars->v_full[i], 2);
      mbar_init(&bars->v_empty[i], 1);
      for (int k = 0; k < 4; ++k) bars->v_nan[i][k] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], KP_SM_WARPS / 2);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], KP_SM_WARPS / 2);
      mbar_init(&bars->pv_done[i], 1);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->meet[i], KP_SM_WARPS / 2);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == KP_MMA_WARP) {
    tmem_alloc(&bars->tmem_base, KP_TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;  // columns [0, 256): S of the two tiles, P over it; [256, 256 + 2 d): O
  walk.base = bars->base;
  walk.s = bars->seq;
  walk.q = kp_seq<GRP>(a, walk.s);
  volatile int* abort_flag = &bars->abort;
  auto give_up = [&]() {
    raise_status(a.status, ST_TIMEOUT);
    *abort_flag = 1;
  };
  // One arrival a warp; what its lanes wrote before is ordered by the warp's
  // barrier.  All lanes poll: one lane's poll costs more than 32 at once.
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, tmo, abort_flag));
  };
  KpPiece p;

  if (warp < KP_DQ_WARPS) {
    kp_regs_less<KP_DQ_REGS>();
    // ------------------------------------------------------ operands from codes
    // Warps 0, 1: K; 2, 3: V; each four of a block's eight pages.  Lane: half
    // `hf` of page row `prow`; at d = 128 the second half's chunks go in the
    // order 4 .. 7, 0 .. 3, so that eight lanes' stores hit all banks.
    const bool is_k = warp < 2;
    uint64_t* full = is_k ? bars->k_full : bars->v_full;
    uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
    const int nst = is_k ? KP_KST : KP_VST;
    const uint32_t ring = sbase + (is_k ? Lay::K_OFF : Lay::V_OFF);
    const int prow = lane >> 1, hf = lane & 1, page0 = (warp & 1) * 4;
    constexpr int CW = D / 16;  // code words of a lane and page, one an 8-channel chunk
    const int part = is_k ? 0 : 9 * D;
    const int code_off = part + prow * (D / 2) + hf * (D / 4);
    const int scale_off = part + 8 * D + prow * (D / 16) + hf * (D / 32);
    // Three blocks are under way: one in registers (w, sc) to be made, one whose
    // page ids are here and whose codes are requested next, and one whose ids are
    // requested.  Nothing waits for a load before it is used.
    uint32_t w[4][CW], sc[4];  // codes and scale bytes of four pages
    struct Block {
      int s, g, j, pos0, last, npages;
      bool have;
    } made, ahead;
    made.have = ahead.have = false;
    int page = -1;  // id of page `lane` of `ahead`
    bool more = walk.next(a, p);
    int j = more ? p.j0 : 0;
    auto load_ids = [&]() {  // the walk's block becomes `ahead`
      ahead.have = more;
      page = -1;
      if (!more) return;
      ahead.s = p.s;
      ahead.g = p.g;
      ahead.j = j;
      ahead.pos0 = p.pos0;
      ahead.last = min(p.len, p.pos0 + p.rows) - 1;  // the tile's last visible position
      ahead.npages = (p.len + KV4_P - 1) / KV4_P;
      if (lane < 4 && j * 8 + page0 + lane < ahead.npages)
        page = a.block_table[static_cast<size_t>(p.s) * a.max_pages + j * 8 + page0 + lane];
      if (++j >= p.j1) {
        more = walk.next(a, p);
        j = more ? p.j0 : 0;
      }
    };
    auto load_codes = [&]() {  // `ahead` becomes `made`
      made = ahead;
      if (!made.have) return;
      if (lane < 4 && made.j * 8 + page0 + lane < made.npages && (page < 0 || page >= a.num_pages)) {
        raise_status(a.status, ST_BAD_PAGE);  // never read outside the pool
        page = 0;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int id = __shfl_sync(0xffffffffu, page, i);
#pragma unroll
        for (int k = 0; k < CW; ++k) w[i][k] = 0;
        sc[i] = 0;
        if (id >= 0 && made.j * KP_N + (page0 + i) * KV4_P + prow <= made.last) {
          // hidden positions hold zeros, whatever the cache has there
          const uint8_t* src = a.pool + (static_cast<size_t>(id) * a.n_kv + made.g) * (18 * D);
          const uint4 x = *reinterpret_cast<const uint4*>(src + code_off + (NCH == 2 ? hf * 16 : 0));
          w[i][0] = x.x; w[i][1] = x.y; w[i][2] = x.z; w[i][3] = x.w;
          if (NCH == 2) {
            const uint4 y = *reinterpret_cast<const uint4*>(src + code_off + (hf ^ 1) * 16);
            w[i][4 % CW] = y.x; w[i][5 % CW] = y.y; w[i][6 % CW] = y.z; w[i][7 % CW] = y.w;
            sc[i] = *reinterpret_cast<const uint32_t*>(src + scale_off);
          } else {
            sc[i] = *reinterpret_cast<const uint16_t*>(src + scale_off);
          }
        }
      }
    };
    load_ids();
    load_codes();
    load_ids();
    uint32_t n = 0;  // blocks made
    // the block whose arrival this warp leaves out (self-test of the waits)
    const uint32_t drop = static_cast<int>(blockIdx.x) == a.drop_cta && warp == 2 * a.drop_part ? a.drop_block : ~0u;
    while (made.have) {
      const uint32_t st = n % nst;
      if (!wait(&empty[st], ((n / nst) & 1) ^ 1)) {
        if (!*abort_flag) give_up();
        break;
      }
      uint32_t nan_bits = 0;  // V: pages whose row here holds a NaN that not every row of the tile sees
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!is_k && made.j * KP_N + (page0 + i) * KV4_P + prow > made.pos0) {
          // it must reach only the rows that do, through P (0 * NaN is NaN)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (((sc[i] >> (8 * k)) & 0x7Fu) == 0x7Fu) {
              nan_bits |= 1u << i;
              sc[i] &= ~(0xFFu << (8 * k));
            }
        }
        if (NCH == 2 && hf) sc[i] = __byte_perm(sc[i], 0, 0x1032);
      }
      const uint32_t dst = ring + st * Lay::KV_BYTES;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pos = (page0 + i) * KV4_P + prow;
        const uint32_t f01 = e4m3x2_to_f16x2(sc[i]), f23 = e4m3x2_to_f16x2(sc[i] >> 16);
        const uint32_t f[4] = {__byte_perm(f01, f01, 0x1010), __byte_perm(f01, f01, 0x3232),
                               __byte_perm(f23, f23, 0x1010), __byte_perm(f23, f23, 0x3232)};
        const uint32_t row = dst + (pos >> 3) * Lay::KV_GROUP + (NCH == 2 ? hf * 1024 : 0) + (pos & 7) * 128;
#pragma unroll
        for (int k = 0; k < CW; ++k) {  // chunk of 8 channels: one word, two chunks a scale
          const int ch = NCH == 2 ? k ^ (4 * hf) : 4 * hf + k;
          const uint32_t s2 = f[k / 2];
          st_shared_v4(row + ((ch ^ (pos & 7)) << 4),
                  make_uint4(hmul2_u(e2m1_to_f16x2<0>(w[i][k]), s2), hmul2_u(e2m1_to_f16x2<1>(w[i][k]), s2),
                             hmul2_u(e2m1_to_f16x2<2>(w[i][k]), s2), hmul2_u(e2m1_to_f16x2<3>(w[i][k]), s2)));
        }
      }
      if (!is_k) {
        // the block's NaN positions: this warp's two words (64 positions)
        uint32_t bits[2] = {0, 0};
        if (__any_sync(0xffffffffu, nan_bits != 0)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const unsigned rows = __ballot_sync(0xffffffffu, (nan_bits >> i) & 1);  // two lanes a row
            uint32_t r16 = 0;
            for (int r = 0; r < 16; ++r)
              if ((rows >> (2 * r)) & 3) r16 |= 1u << r;
            bits[i >> 1] |= r16 << (16 * (i & 1));
          }
        }
        if (lane == 0) {
          bars->v_nan[st][page0 >> 1] = bits[0];
          bars->v_nan[st][(page0 >> 1) + 1] = bits[1];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && n != drop) mbar_arrive(&full[st]);
      ++n;
      load_codes();
      load_ids();
    }
  } else if (warp >= KP_MMA_WARP) {
    kp_regs_less<KP_MMA_REGS>();
    // ------------------------------------------------------------ MMA issuer
    bool ok = true, any = false;
    uint32_t n = 0;                  // blocks
    uint32_t np0 = 0, np1 = 0;       // pieces and steps of either tile
    uint32_t st0 = 0, st1 = 0;
    uint32_t pv0 = 0, pv1 = 0;       // and the products that an S followed
    auto s_product = [&](int t, uint32_t block) {
      const uint32_t k_addr = sbase + Lay::K_OFF + (block % KP_KST) * Lay::KV_BYTES;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t adesc = desc_sw128_kmajor(sbase + t * Lay::Q_BYTES + (kk >> 2) * KP_REGION) + 2 * (kk & 3);
        const uint64_t bdesc = desc_sw128_kmajor_sbo(k_addr + (kk >> 2) * 1024, Lay::KV_GROUP) + 2 * (kk & 3);
        tc_mma_bf16(tmem + t * KP_N, adesc, bdesc, IDESC_S, kk > 0);
      }
      any = true;
      tc_commit(&bars->s_full[t]);
    };
    auto k_wait = [&](uint32_t block) -> bool {
      const bool good = mbar_wait(&bars->k_full[block % KP_KST], (block / KP_KST) & 1, tmo, abort_flag);
      tc_fence_after();
      return good;
    };
    while (warp == KP_MMA_WARP && ok && walk.next(a, p)) {
      if (lane == 0) {
        ok = mbar_wait(&bars->q_full[0], np0++ & 1, tmo, abort_flag) &&
             (p.nt == 1 || mbar_wait(&bars->q_full[1], np1++ & 1, tmo, abort_flag)) && k_wait(n);
        if (ok) {
          for (int t = 0; t < p.nt; ++t) s_product(t, n);
          tc_commit(&bars->k_empty[n % KP_KST]);
        }
        for (int j = p.j0; j < p.j1 && ok; ++j, ++n) {
          const uint32_t vs = n % KP_VST;
          const bool more = j + 1 < p.j1;
          ok = mbar_wait(&bars->v_full[vs], (n / KP_VST) & 1, tmo, abort_flag);
          for (int t = 0; t < p.nt && ok; ++t) {
            // P over S, then the next S over P
            ok = mbar_wait(&bars->p_full[t], (t ? st1++ : st0++) & 1, tmo, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t v_addr = sbase + Lay::V_OFF + vs * Lay::KV_BYTES;
#pragma unroll
            for (int kk = 0; kk < KP_N / 16; ++kk) {
              const uint64_t bdesc = desc_sw128_mnmajor(v_addr + kk * 2 * Lay::KV_GROUP, 1024, Lay::KV_GROUP);
              kp_mma_ts(tmem + 256 + t * D, tmem + t * KP_N + kk * 8, bdesc, IDESC_PV, j > p.j0 || kk > 0);
            }
            any = true;
            if (t == p.nt - 1) tc_commit(&bars->v_empty[vs]);
            if (more) {
              tc_commit(&bars->pv_done[t]);
              ok = (t > 0 || k_wait(n + 1)) && mbar_wait(&bars->pv_done[t], (t ? pv1++ : pv0++) & 1, tmo, abort_flag);
              if (!ok) break;
              tc_fence_after();
              s_product(t, n + 1);
              if (t == p.nt - 1) tc_commit(&bars->k_empty[(n + 1) % KP_KST]);
            } else {
              tc_commit(&bars->o_full[t]);
            }
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (!ok && lane == 0 && !*abort_flag) give_up();
    // Another role may give up after the last product was issued, so this wait does
    // not ask who did; otherwise the softmax warps wait for the same products.
    if (any) {
      tc_commit(&bars->drain);
      if (!mbar_wait(&bars->drain, 0, KP_DRAIN_NS)) raise_status(a.status, ST_TIMEOUT);
    }
    __syncwarp();
  } else {
    kp_regs_more<KP_SM_REGS>();
    // --------------------------------------------------- softmax and epilogue
    const int sw = warp - KP_DQ_WARPS;
    const int t = sw >> 2;             // the tile
    const int quarter = warp & 3;      // tensor-memory lanes this warp may access
    const int r = quarter * 32 + lane; // the vector (lane) this thread owns
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_tmem = tmem + lane_off + t * KP_N, o_tmem = tmem + lane_off + 256 + t * D;
    constexpr int RT = KP_M / GRP;     // rows of a tile
    uint32_t n = 0, np = 0, met = 0;   // blocks, pieces and meetings of this tile
    uint32_t blk = 0;                  // blocks of the CTA
    bool ok = true;
    auto meet = [&]() -> bool {
      arrive(&bars->meet[t]);
      const bool good = wait(&bars->meet[t], met & 1);
      ++met;
      return good;
    };
    while (ok && walk.next(a, p)) {
      if (t >= p.nt) {
        blk += p.j1 - p.j0;
        continue;
      }
      const int row = t * RT + r / GRP;
      const bool live = row < p.rows;
      const int qpos = live ? p.pos0 + row : -1;  // sees positions 0 .. qpos
      // of q and o; a row that is not there: the unit's first
      const size_t at = (static_cast<size_t>(p.row0 + (live ? row : 0)) * a.n_q + p.g * GRP + r % GRP) * D;
      // Q, scaled to fp16's range by the vector's largest element
      float scale;
      {
        const uint4* q4 = reinterpret_cast<const uint4*>(a.q + at);
        float top = 0.f;
        uint4 own[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint4 v = q4[c];
          if (!live) v = make_uint4(0, 0, 0, 0);
          top = fmaxf(top, fmax3(fmax3(fabsf(bf16lo(v.x)), fabsf(bf16hi(v.x)), fabsf(bf16lo(v.y))),
                                 fmax3(fabsf(bf16hi(v.y)), fabsf(bf16lo(v.z)), fabsf(bf16hi(v.z))),
                                 fmaxf(fabsf(bf16lo(v.w)), fabsf(bf16hi(v.w)))));
          own[c] = v;
        }
        const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        const int kq = top > 0.f ? max(-126, min(120, 14 - e)) : 0;
        // a vector with an infinity: NaN scores (attn_kv4.cu)
        const float mul = top == INFINITY ? __int_as_float(0x7FC00000) : exp2_int(kq);
        scale = fmaxf(a.scale_log2 * exp2_int(-kq), 1.17549435e-38f);  // 0 times a hidden score's -inf is NaN
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = own[c];
          st_shared_v4(sbase + t * Lay::Q_BYTES + (c >> 3) * KP_REGION + sw128(r, c & 7),
                  make_uint4(pack_f16(bf16lo(v.x) * mul, bf16hi(v.x) * mul), pack_f16(bf16lo(v.y) * mul, bf16hi(v.y) * mul),
                             pack_f16(bf16lo(v.z) * mul, bf16hi(v.z) * mul), pack_f16(bf16lo(v.w) * mul, bf16hi(v.w) * mul)));
        }
        fence_proxy_async_smem();
        arrive(&bars->q_full[t]);
      }
      float m_ref = -INFINITY, l = 0.f;
      float nm = KP_UNSEEN;  // what the exponents add: KP_SHIFT - m_ref
      for (int j = p.j0; j < p.j1; ++j, ++n, ++blk) {
        if (!wait(&bars->s_full[t], n & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float x[KP_N];
#pragma unroll
        for (int c = 0; c < KP_N / 32; ++c) tc_ld_32x32b_x32(s_tmem + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * c]));
        tc_wait_ld();
        const bool mixed = j * KP_N + KP_N - 1 > p.pos0;  // some row of the unit sees less than the block
        if (mixed) {
          const int see = qpos - j * KP_N;
#pragma unroll
          for (int i = 0; i < KP_N; ++i)
            if (i > see) x[i] = -INFINITY;
        }
        float mx;
        {
          float mx8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mx8[i] = fmax3(x[i], x[8 + i], x[16 + i]);
#pragma unroll
          for (int i = 24; i < KP_N - 8; i += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], x[i + k], x[i + 8 + k]);
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(mx8[k], x[KP_N - 8 + k]);
          mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])) * scale;
        }
        float corr = 1.f;
        if (mx + nm > KP_SLACK + KP_SHIFT) {  // also from -inf, where O and l are still zero
          corr = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - mx);
          m_ref = mx;
          nm = KP_SHIFT - mx;
          l *= corr;
        }
        // a raised maximum rescales the row of O; the product of the block before is
        // done, as it was issued before this S
        if (j > p.j0 && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t u[16];
            tc_ld_32x32b_x16(o_tmem + c * 16, u);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * corr);
            tc_st_32x32b_x16(o_tmem + c * 16, u);
          }
        }
        // p = 2^(s scale - m + shift); m = -inf: nothing seen yet, all p are 0
        if (__any_sync(0xffffffffu, fabsf(m_ref) > 8e6f && m_ref != -INFINITY)) {
          // Scores from 2^23 on have steps of 1 and more: the fused step could pass what
          // was compared, and with it fp16's range, by a power of two or more.  Below,
          // half a step is at most 2^-1: p stays under 2^15.5.
#pragma unroll
          for (int i = 0; i < KP_N; ++i) x[i] = ex2_approx(__fadd_rn(__fmul_rn(x[i], scale), nm));
        } else {
          const float2 sc2 = make_float2(scale, scale), nm2 = make_float2(nm, nm);
#pragma unroll
          for (int i = 0; i < KP_N / 2; ++i) {
            const float2 f = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), sc2, nm2);
            x[2 * i] = ex2_approx(f.x);
            x[2 * i + 1] = ex2_approx(f.y);
          }
        }
        if (mixed) {
          // NaN of V at positions that not every row sees: to the rows that do
          const uint32_t vs = blk % KP_VST;
          if (!wait(&bars->v_full[vs], (blk / KP_VST) & 1)) {
            ok = false;
            break;
          }
          const int see = qpos - j * KP_N;
#pragma unroll
          for (int k = 0; k < KP_N / 32; ++k) {
            const uint32_t nan = bars->v_nan[vs][k];
            if (nan) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (((nan >> i) & 1) && 32 * k + i <= see) x[32 * k + i] = __int_as_float(0x7FC00000);
            }
          }
        }
        // P as fp16 pairs over the first half of S, and the row's sum
        float2 ls4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ls4[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < KP_N / 64; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) ls4[i & 3] = __fadd2_rn(ls4[i & 3], make_float2(x[64 * c + 2 * i], x[64 * c + 2 * i + 1]));
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = pack_f16(x[64 * c + 2 * i], x[64 * c + 2 * i + 1]);
          tc_st_32x32b_x32(s_tmem + 32 * c, w);
        }
        tc_wait_st();
        tc_fence_before();
        arrive(&bars->p_full[t]);
        const float2 a2 = __fadd2_rn(__fadd2_rn(ls4[0], ls4[1]), __fadd2_rn(ls4[2], ls4[3]));
        l += a2.x + a2.y;
      }
      if (ok && !wait(&bars->o_full[t], np & 1)) ok = false;
      if (!ok) break;
      ++np;
      tc_fence_after();
      const bool whole = p.j0 == 0 && p.j1 == p.nb;
      const int first = static_cast<int>((p.key + KP_FIXED) / quota);
      const int last = static_cast<int>((p.key + KP_FIXED + p.nb - 1) / quota);
      auto rec_of = [&](int cta) {
        return a.tiles + (static_cast<size_t>(cta) * 2 + (cta == first ? 1 : 0)) * Lay::REC + t * Lay::TREC;
      };
      float* rec = rec_of(blockIdx.x);
      uint4* dst = reinterpret_cast<uint4*>(a.o + at);
      const float inv = l == 0.f ? 0.f : a.v_scale / l;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t u[32];
        tc_ld_32x32b_x32(o_tmem + c * 32, u);
        tc_wait_ld();
        if (whole) {
          if (live) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* f = reinterpret_cast<const float*>(u) + 8 * i;
              dst[c * 4 + i] = make_uint4(pack_bf16(f[0] * inv, f[1] * inv), pack_bf16(f[2] * inv, f[3] * inv),
                                          pack_bf16(f[4] * inv, f[5] * inv), pack_bf16(f[6] * inv, f[7] * inv));
            }
          }
        } else {  // four channels of all rows next to one another
          float4* out = reinterpret_cast<float4*>(rec) + c * 8 * KP_M + r;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float* f = reinterpret_cast<const float*>(u) + 4 * i;
            out[i * KP_M] = make_float4(f[0], f[1], f[2], f[3]);
          }
        }
      }
      tc_fence_before();
      if (whole) continue;
      rec[KP_M * D + r] = m_ref;
      rec[KP_M * D + KP_M + r] = l;
      __threadfence();
      if (!(ok = meet())) break;
      if (quarter == 0 && lane == 0) {
        int* counter = a.tile_counters + 2 * first + t;
        const int before = atomicAdd(counter, 1);
        bars->last[t] = before == last - first;
        if (before == last - first) *counter = 0;  // as the next launch expects it
      }
      if (!(ok = meet())) break;
      if (bars->last[t]) {
        __threadfence();
        float M = -INFINITY, Ls = 0.f;
        for (int b = first; b <= last; ++b) M = fmaxf(M, __ldcg(rec_of(b) + KP_M * D + r));
        for (int b = first; b <= last; ++b) {
          const float mb = __ldcg(rec_of(b) + KP_M * D + r);
          Ls = fmaf(mb == -INFINITY ? 1.f : exp2f(mb - M), __ldcg(rec_of(b) + KP_M * D + KP_M + r), Ls);
        }
        const float iv = Ls == 0.f ? 0.f : a.v_scale / Ls;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float4 acc[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int b = first; b <= last; ++b) {
            const float mb = __ldcg(rec_of(b) + KP_M * D + r);
            const float wb = mb == -INFINITY ? 1.f : exp2f(mb - M);
            const float4* in = reinterpret_cast<const float4*>(rec_of(b)) + c * 8 * KP_M + r;
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __ldcg(in + i * KP_M);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[i].x = fmaf(wb, v[i].x, acc[i].x);
              acc[i].y = fmaf(wb, v[i].y, acc[i].y);
              acc[i].z = fmaf(wb, v[i].z, acc[i].z);
              acc[i].w = fmaf(wb, v[i].w, acc[i].w);
            }
          }
          if (live) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = acc[2 * i], h = acc[2 * i + 1];
              dst[c * 4 + i] = make_uint4(pack_bf16(f.x * iv, f.y * iv), pack_bf16(f.z * iv, f.w * iv),
                                          pack_bf16(h.x * iv, h.y * iv), pack_bf16(h.z * iv, h.w * iv));
            }
          }
        }
      }
    }
    if (!ok && !*abort_flag) give_up();
    tc_wait_st();  // a rescaled row, if a wait behind it was given up
  }

  tc_fence_before();
  __syncthreads();
  if (warp == KP_MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, KP_TMEM_COLS);
  }
}

template <int GRP, int NCH>
cudaError_t launch_kp(const Kv4AttnArgs& a, cudaStream_t stream) {
  const int smem = KpLayout<NCH>::SMEM;
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(attn_kv4_prefill_kernel<GRP, NCH>), smem);
  if (e != cudaSuccess) return e;
  attn_kv4_prefill_kernel<GRP, NCH><<<a.grid, KP_THREADS, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv4_tile_record_bytes(int head_dim) {
  return (head_dim == 128 ? KpLayout<2>::REC : KpLayout<1>::REC) * sizeof(float);
}

cudaError_t launch_attention_kv4_prefill(const Kv4AttnArgs& a, cudaStream_t stream) {
  const int grp = a.n_q / a.n_kv;
#define NF_KP_CASE(G)                                          \
  if (grp == G) return a.head_dim == 128 ? launch_kp<G, 2>(a, stream) : launch_kp<G, 1>(a, stream);
  NF_KP_CASE(1) NF_KP_CASE(2) NF_KP_CASE(4) NF_KP_CASE(8)
#undef NF_KP_CASE
  return cudaErrorInvalidValue;
}

}  // namespace nf
