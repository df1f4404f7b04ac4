// Products of e4m3 operands with a scale for each block of 128, on tcgen05:
//
//   C[m, n] = sum_b a_s[b, m] b_s[n / 128, b] sum_{k in block b} a[m, k] b[n, k]
//
// for one matrix, or by groups of rows (experts) whose bounds are on the device.
//  * A tile is 128 rows of A x 256 rows of B (SwiGLU: 128 features' gate and up rows),
//    so a thread's row has one scale of A and a warp's columns one or two of B a
//    block of K.  A ring stage is one block of K: 128 bytes a row, one swizzled row.
//  * Scales are fp32 and change with every block of K, so a block's products go to
//    accumulators of their own in tensor memory (two, in turn, for each half of the
//    columns), and eight warps, four a half, add them, times their scale, to sums in
//    registers.  While they do, the tensor core fills the other accumulators.
//  * Warp 0 loads tiles by TMA, warps 1 and 2 issue the products of a half each, warp 3
//    copies the scales beside the tiles, warps 4 to 11 sum and run the epilogue.  Persistent CTAs, one an SM.
//  * What bounds it: the hand-over between products and sums.  A block of K is 528 cycles
//    of products (two halves of four instructions), but a half's accumulator goes issue,
//    completion, sums' loads, release, issue, some 1500 cycles for two blocks; about 800
//    cycles a block are reached, 57 % of the tensor pipe.  (What an SM takes in, 61 bytes a
//    cycle then, may bind beside it: not measured apart.)  In long runs the power limit
//    counts as well: 4096 x 8192 x 28672 takes 685 to 705 us (2.8 PFLOP/s) for the first dozens
//    of calls and 800 us (1590 MHz, 1360 W) after seconds.  Measured and not kept, on that
//    product at 711: one issuing warp for both halves 946, one for each accumulator 748,
//    sixteen summing warps of 64 columns 718, the next block's loads ahead of this one's
//    last sums 890, packed pairs of sums 893 (moves), one hand-over for all 256 columns
//    884, B multicast to two CTAs 703 (shorter products 4 to 7 % slower).
//  * A product with tiles for at most a half (a quarter) of the SMs is cut along K between
//    the two (four) CTAs of a cluster (SPLIT): each finishes its part of the tile's columns
//    (SwiGLU: of its rows), with the others' sums from their shared memory.
//  * Every wait is bounded; one that gives up flags the status word, and the kernel
//    drains what it has in flight (bounded) and frees tensor memory.
#include <type_traits>

#include "by_device.h"
#include "fp8.cuh"
#include "kernels.h"

namespace nf {
namespace {

constexpr int BM = 128, BN = 256, BK = F8_BLOCK;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int THREADS = 384;
// Registers: 384 threads start with 168 each (64,512); the first warpgroup keeps 40 (SPLIT:
// 72), the summing warps take 224 (208): 4 * 32 * 40 + 8 * 32 * 224 = 62,464, and as many
// with 72 and 208.  40 / 224 against 72 / 208: 2048 x 14336 x 4096 to 8 bits 180 / 189 us,
// 4096 x 8192 x 28672 704 / 706; 333 x 6144 x 4096 cut along K 16.9 / 15.6, 333 x 4096 x 14336
// 36.9 / 30.4.  With 56 / 216 or 64 / 208 the compiler moves sums about: 4096 x 8192 x 28672
// 836 and 760, 333 x 4096 x 14336 38.6 with 56 / 216.
constexpr int regs_few(bool split) { return split ? 72 : 40; }
constexpr int regs_sum(bool split) { return split ? 208 : 224; }
constexpr int TMEM_COLS = 512;
constexpr int STORE_BYTES = 2048;  // of a summing warp: 32 rows x 64 bytes of output
constexpr int TAIL_BYTES = 8192;

struct Tail {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t tfull[4];   // accumulators: half h of the columns, in turn 2 h and 2 h + 1
  uint64_t tempty[4];
  uint64_t pair[4];    // the two warps of 32 rows (SWIGLU8: the block's largest value)
  uint64_t drain[2];
  uint64_t ready;      // SPLIT: all CTAs' sums are in their shared memory
  uint32_t tmem_base;
  int abort;
  // for a drain after a wait gave up: the ring's stages and the phase of their last load,
  // the lanes that issue products (32: none issued)
  uint32_t issued, phases;
  int issuer[2];
  int tile0[F8_MAX_GROUPS + 1];  // first tile of each group
  int row0[F8_MAX_GROUPS + 1];   // first row of each group
  float a_s[8][BM];       // scales of the next blocks of K: of A's rows,
  float b_s[8][2];        // and of B's halves (SwiGLU: of gate and up)
  float top[2][8][32];    // SWIGLU8: by tile parity and warp, a row's largest value
};
constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + 8 * STORE_BYTES + TAIL_BYTES;
static_assert(sizeof(Tail) <= TAIL_BYTES && SMEM <= 232448, "shared memory");

__device__ uint32_t g_status;

struct Tile {
  int m0, m_lim, tn, e;
};

// SPLIT: CTAs of a cluster that take a part of K each of one tile (see the header).
template <int EPI, int SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_f8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const F8GemmArgs args) {
  constexpr bool SW = EPI == F8_SWIGLU || EPI == F8_SWIGLU8;
  constexpr int TN = SW ? BN / 2 : BN;  // output columns of a tile
  constexpr uint32_t IDESC = idesc_e4m3_f32(BM, BN / 2);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Tail* tail = reinterpret_cast<Tail*>(smem + STAGES * STAGE_BYTES + 8 * STORE_BYTES);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nk = (args.K + BK - 1) / BK, n_tiles = (args.N + TN - 1) / TN;
  const int nb = (args.N + F8_BLOCK - 1) / F8_BLOCK;
  const bool grouped = args.group_off != nullptr;
  const int rank = SPLIT > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = blockIdx.x / SPLIT, stride = gridDim.x / SPLIT;
  const int k0 = rank * nk / SPLIT, k1 = (rank + 1) * nk / SPLIT;
  const uint64_t tmo = args.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tail->full[s], 1 + 32);  // the tiles, the scales' 32 lanes
      mbar_init(&tail->empty[s], 2);
    }
    for (int a = 0; a < 4; ++a) {
      mbar_init(&tail->tfull[a], 2);  // the products, and the scales as their issuer saw them
      mbar_init(&tail->tempty[a], 4);
    }
    for (int a = 0; a < 2; ++a) mbar_init(&tail->drain[a], 1);
    mbar_init(&tail->ready, SPLIT);
    for (int a = 0; a < 4; ++a) mbar_init(&tail->pair[a], 2);
    tail->abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
  }
  pdl_wait();  // nothing before this reads or writes global memory
  // Tensor memory is taken once the kernel ahead is complete, and the kernel behind let
  // start once it is taken: neither can wait for columns that the other holds.
  if (warp == 1) {
    tmem_alloc(&tail->tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 2 && grouped) {
    // Rows and tiles of the groups.  Offsets are held within [0, M], and one below
    // the one before it counts as that one, so no offset leads out of a tensor.
    int top = 0, tiles = 0;
    for (int b = 0; b <= args.groups; b += 32) {
      const int i = b + lane;
      int o = i <= args.groups ? min(max(args.group_off[i], 0), args.M) : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, o, d);
        if (lane >= d) o = max(o, y);
      }
      o = max(o, top);
      const int up = __shfl_up_sync(0xffffffffu, o, 1);
      const int before = lane ? up : top;  // row0 of group i - 1
      int t = i > 0 && i <= args.groups ? (o - before + BM - 1) / BM * n_tiles : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t, d);
        if (lane >= d) t += y;
      }
      t += tiles;
      if (i <= args.groups) {
        tail->row0[i] = o;
        tail->tile0[i] = t;
      }
      top = __shfl_sync(0xffffffffu, o, 31);
      tiles = __shfl_sync(0xffffffffu, t, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  if (SPLIT > 1) {  // the peers' barriers exist before anything arrives on them
    cluster_arrive();
    cluster_wait();
  }
  const uint32_t tmem_base = tail->tmem_base;
  volatile int* abort_flag = &tail->abort;
  const int total = grouped ? tail->tile0[args.groups] : (args.M + BM - 1) / BM * n_tiles;
  auto decode = [&](int u) {
    Tile x;
    int r0 = 0, r1 = args.M;
    x.e = 0;
    if (grouped) {
      int lo = 0, hi = args.groups;  // tile0[lo] <= u < tile0[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (tail->tile0[mid] <= u) lo = mid;
        else hi = mid;
      }
      x.e = lo;
      u -= tail->tile0[lo];
      r0 = tail->row0[lo];
      r1 = tail->row0[lo + 1];
    }
    const int mt = (r1 - r0 + BM - 1) / BM;
    x.m0 = r0 + u % mt * BM;
    x.m_lim = r1;
    x.tn = u / mt;
    return x;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(regs_few(SPLIT > 1)));
    if (warp == 0 && lane == 0) {
      uint32_t st = 0, ph = 0, issued = 0, phases = 0;  // the stages, and the phase of their last load
      bool ok = true;
      for (int u = first; u < total && ok; u += stride) {
        const Tile x = decode(u);
        const int b0 = x.e * (SW ? 2 : 1) * args.N + x.tn * TN;
        const int b1 = SW ? b0 + args.N : b0 + 128;
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait(&tail->empty[st], ph ^ 1, tmo, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + st * STAGE_BYTES;
          uint64_t* bar = &tail->full[st];
          mbar_arrive_expect_tx(bar, STAGE_BYTES);
          tma_load_2d(sa, &tmA, bar, kb * BK, x.m0);
          if (SW) {  // a half of the columns: 64 features' gate rows, then their up rows
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tma_load_2d(sa + A_BYTES + i * (B_BYTES / 4), &tmB, bar, kb * BK, (i & 1 ? b1 : b0) + (i >> 1) * 64);
          } else {
            tma_load_2d(sa + A_BYTES, &tmB, bar, kb * BK, b0);
            tma_load_2d(sa + A_BYTES + B_BYTES / 2, &tmB, bar, kb * BK, b1);
          }
          issued |= 1u << st;
          phases = (phases & ~(1u << st)) | ph << st;
          if (++st == STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      tail->issued = issued;
      tail->phases = phases;
      if (!ok) {
        raise_status(&g_status, ST_TIMEOUT);
        *abort_flag = 1;
      }
    }
    if (warp == 1 || warp == 2) {
      const int h = warp - 1;
      const bool one = elect_one();
      uint32_t st = 0, ph = 0, acc = 0, aph = 0;
      bool ok = true, any = false;
      for (int u = first; u < total && ok; u += stride) {
#pragma unroll 1
        for (int kb = k0; kb < k1; ++kb) {
          // (the stage is there long before the accumulator is free)
          const uint32_t sa = smem_u32(smem + st * STAGE_BYTES), d = tmem_base + (2 * h + acc) * (BN / 2);
          const uint64_t ad = desc_sw128_kmajor(sa), bd = desc_sw128_kmajor(sa + A_BYTES + h * (B_BYTES / 2));
          ok = __all_sync(0xffffffffu, mbar_wait(&tail->full[st], ph, tmo, abort_flag) &&
                                           mbar_wait(&tail->tempty[2 * h + acc], aph ^ 1, tmo, abort_flag)) != 0;
          if (!ok) break;
          tc_fence_after();
          if (one) {
#pragma unroll
            for (int k = 0; k < BK / 32; ++k)  // 32 codes = 32 bytes along the swizzled row
              tc_mma_e4m3(d, ad + 2 * k, bd + 2 * k, IDESC, k != 0);
            tc_commit(&tail->tfull[2 * h + acc]);
            mbar_arrive(&tail->tfull[2 * h + acc]);
            tc_commit(&tail->empty[st]);
          }
          any = true;
          if (++st == STAGES) {
            st = 0;
            ph ^= 1;
          }
          if (++acc == 2) {
            acc = 0;
            aph ^= 1;
          }
        }
      }
      if (!ok && one) {
        raise_status(&g_status, ST_TIMEOUT);
        *abort_flag = 1;
      }
      if (one) tail->issuer[h] = any ? lane : 32;
    }
    if (warp == 3) {
      // Scales, copied beside the tiles: a slot is filled again 8 blocks of K later, when
      // the stage's products of 4 blocks before are done, so the sums of 2 further before.
      uint32_t st = 0, ph = 0, slot = 0;
      bool ok = true;
      for (int u = first; u < total && ok; u += stride) {
        const Tile x = decode(u);
        const int b0 = SW ? x.tn : min(2 * x.tn, nb - 1), b1 = SW ? nb + x.tn : min(2 * x.tn + 1, nb - 1);
        const float* as = args.a_s + static_cast<size_t>(k0) * args.M + x.m0 + lane;
        const float* bs = args.b_s + (static_cast<size_t>(x.e) * (SW ? 2 : 1) * nb + (lane ? b1 : b0)) * nk;
        const int rows = x.m_lim - x.m0 - lane;  // row 32 i of this lane's is there below it
#pragma unroll 1
        for (int kb = k0; kb < k1; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(&tail->empty[st], ph ^ 1, tmo, abort_flag)) != 0;
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) copy4(&tail->a_s[slot][lane + 32 * i], rows > 32 * i ? as + 32 * i : args.a_s, rows > 32 * i);
          if (lane < 2) copy4(&tail->b_s[slot][lane], bs + kb, true);
          mbar_arrive_copied(&tail->full[st]);
          as += args.M;
          slot = (slot + 1) % 8;
          if (++st == STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) {
        raise_status(&g_status, ST_TIMEOUT);
        *abort_flag = 1;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(regs_sum(SPLIT > 1)));
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row_in_tile = quarter * 32 + lane;
    uint8_t* mine = smem + STAGES * STAGE_BYTES + (warp - 4) * STORE_BYTES;
    // 16-byte chunk j of row r of the warp's 2 KB, so placed that rows are written and
    // read eight lanes at a time without bank conflicts
    auto slot = [&](int r, int j) { return reinterpret_cast<uint4*>(mine + r * 64 + ((j ^ (r >> 1 & 3)) << 4)); };
    uint32_t acc = 0, aph = 0, parity = 0, slot8 = 0;
    bool ok = true;
    for (int u = first; u < total && ok; u += stride) {
      // This thread's sums: 128 columns of its half (SwiGLU: 64 features' gate columns,
      // then their up columns).
      float sum[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) sum[i] = 0.f;
#pragma unroll 1
      for (int kb = k0; kb < k1; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&tail->tfull[2 * half + acc], aph, tmo, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + (2 * half + acc) * (BN / 2);
        uint32_t v[2][32];
        auto add = [&](int c, float s) {
#pragma unroll
          for (int i = 0; i < 32; ++i) fma_loaded(sum[c * 32 + i], v[c & 1][i], s);
        };
        tc_ld_32x32b_x32(tb, v[0]);
        tc_ld_32x32b_x32(tb + 32, v[1]);
        const float as = tail->a_s[slot8][row_in_tile];
        const float s0 = as * tail->b_s[slot8][SW ? 0 : half], s1 = SW ? as * tail->b_s[slot8][1] : s0;
        slot8 = (slot8 + 1) % 8;
        tc_wait_ld();
        add(0, s0);
        tc_ld_32x32b_x32(tb + 64, v[0]);
        add(1, s0);
        tc_ld_32x32b_x32(tb + 96, v[1]);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&tail->tempty[2 * half + acc], lane == 0);
        add(2, s1);
        add(3, s1);
        if (++acc == 2) {
          acc = 0;
          aph ^= 1;
        }
      }
      if (SPLIT > 1) {
        // Both halves' products have read the ring, which now takes the sums, four columns of
        // a row together, rows next to one another.  A CTA finishes its part of each half's
        // columns (SwiGLU: of the rows), with all CTAs' sums in their order (a load takes about
        // a microsecond: all 32 at once).
        asm volatile("bar.sync 1, 256;" ::: "memory");
        float4* ring = reinterpret_cast<float4*>(smem) + half * 32 * BM + row_in_tile;
        if (ok) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            ring[i * BM] = make_float4(sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]);
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        // (a release at cluster scope, behind the barrier that all of the CTA's writes precede)
        if (warp == 4 && lane < SPLIT) mbar_arrive_remote(cluster_map(smem_u32(&tail->ready), lane));
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tail->ready, 0, tmo)) && ok;
        if constexpr (SW) {
          // A feature's gate and up columns meet here, and an 8-bit block is a row's 128
          // features, so a CTA finishes rows: a warp 32 of them, FEAT features each (bf16
          // output by columns as below: 256 x 4096 x 14336 39 us, so 35).
          constexpr int ROW_WARPS = BM / SPLIT / 32, FEAT = 16 * ROW_WARPS, PART = FEAT / 4;
          const int w8 = warp - 4, chunk = w8 / ROW_WARPS;
          const int row = (rank * ROW_WARPS + w8 % ROW_WARPS) * 32 + lane;
          const int c4 = chunk / (64 / FEAT) * 32 + chunk % (64 / FEAT) * PART;  // first gate columns, in fours
          const Tile x = decode(u);
          const int n0 = x.tn * TN + chunk * FEAT;
          float o[FEAT], top = 0.f;
          if (ok) {
            const uint32_t mine8 = smem_u32(reinterpret_cast<float4*>(smem) + c4 * BM + row);
            float4 w[SPLIT][2 * PART];
#pragma unroll
            for (int r = 0; r < SPLIT; ++r) {
              const uint32_t at = cluster_map(mine8, r);
#pragma unroll
              for (int i = 0; i < 2 * PART; ++i) w[r][i] = ld_cluster_f4(at + (i / PART * 16 + i % PART) * (BM * 16));
            }
#pragma unroll
            for (int i = 0; i < 2 * PART; ++i)
#pragma unroll
              for (int r = 1; r < SPLIT; ++r) {
                w[0][i].x += w[r][i].x; w[0][i].y += w[r][i].y; w[0][i].z += w[r][i].z; w[0][i].w += w[r][i].w;
              }
#pragma unroll
            for (int i = 0; i < PART; ++i) {
              const float4 a = w[0][i], b = w[0][PART + i];
              o[4 * i] = silu_mul(a.x, b.x);
              o[4 * i + 1] = silu_mul(a.y, b.y);
              o[4 * i + 2] = silu_mul(a.z, b.z);
              o[4 * i + 3] = silu_mul(a.w, b.w);
            }
#pragma unroll
            for (int i = 0; i < FEAT; ++i) {
              if (n0 + i >= args.N) o[i] = 0.f;
              top = absmax_nan(top, o[i]);
            }
          }
          const int m = x.m0 + row;
          if constexpr (EPI == F8_SWIGLU) {
            if (ok && m < x.m_lim) {
#pragma unroll
              for (int j = 0; j < FEAT / 8; ++j) {
                const float* v = o + 8 * j;
                if (n0 + 8 * j < args.N)
                  *reinterpret_cast<uint4*>(args.C + static_cast<size_t>(m) * args.N + n0 + 8 * j) =
                      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
              }
            }
            break;  // one tile a cluster
          }
          tail->top[0][w8][lane] = top;
          asm volatile("bar.sync 1, 256;" ::: "memory");  // (also after a failure)
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < 8 / ROW_WARPS; ++j) top = absmax_nan(top, tail->top[0][w8 % ROW_WARPS + j * ROW_WARPS][lane]);
          const float s = f8_scale(top), inv = 1.f / s;
          if (m < x.m_lim) {
            if (chunk == 0) args.c_s[static_cast<size_t>(x.tn) * args.M + m] = s;
#pragma unroll
            for (int j = 0; j < FEAT / 16; ++j) {
              const float* v = o + 16 * j;
              if (n0 + 16 * j < args.N)
                *reinterpret_cast<uint4*>(args.q + static_cast<size_t>(m) * args.N + n0 + 16 * j) =
                    make_uint4(f8_codes4_near(v[0], v[1], v[2], v[3], inv), f8_codes4_near(v[4], v[5], v[6], v[7], inv),
                               f8_codes4_near(v[8], v[9], v[10], v[11], inv), f8_codes4_near(v[12], v[13], v[14], v[15], inv));
            }
          }
          break;
        }
        if (!ok) break;
        constexpr int PART = 32 / SPLIT;  // of a row's fours of columns
        float4 w[SPLIT][PART];
#pragma unroll
        for (int r = 0; r < SPLIT; ++r) {
          const uint32_t at = cluster_map(smem_u32(ring + rank * PART * BM), r);
#pragma unroll
          for (int i = 0; i < PART; ++i) w[r][i] = ld_cluster_f4(at + i * (BM * 16));
        }
#pragma unroll
        for (int i = 0; i < PART; ++i) {
          float4 t = w[0][i];
#pragma unroll
          for (int r = 1; r < SPLIT; ++r) {
            t.x += w[r][i].x; t.y += w[r][i].y; t.z += w[r][i].z; t.w += w[r][i].w;
          }
          sum[4 * i] = t.x; sum[4 * i + 1] = t.y; sum[4 * i + 2] = t.z; sum[4 * i + 3] = t.w;
        }
      }
      if (!ok) break;
      // Epilogue, 64 bytes of each of the warp's 32 rows at a time through its 2 KB.
      const Tile x = decode(u);
      const int mw = x.m0 + quarter * 32;  // first row of this warp
      if (EPI == F8_SWIGLU8) {
        const int n0 = x.tn * TN + half * 64;
        float o[64], top = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          o[i] = n0 + i < args.N ? silu_mul(sum[i], sum[64 + i]) : 0.f;
          top = absmax_nan(top, o[i]);
        }
        // the block's 128 features are this thread's and those of the other half's warp
        tail->top[parity][warp - 4][lane] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->pair[quarter]);
        if (!__all_sync(0xffffffffu, mbar_wait(&tail->pair[quarter], parity, tmo, abort_flag))) {
          ok = false;
          break;
        }
        top = absmax_nan(top, tail->top[parity][(warp - 4) ^ 4][lane]);
        parity ^= 1;
        const float s = f8_scale(top), inv = 1.f / s;
        if (half == 0 && mw + lane < x.m_lim) args.c_s[static_cast<size_t>(x.tn) * args.M + mw + lane] = s;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float* w = o + 16 * j;
          *slot(lane, j) = make_uint4(f8_codes4_near(w[0], w[1], w[2], w[3], inv), f8_codes4_near(w[4], w[5], w[6], w[7], inv),
                                      f8_codes4_near(w[8], w[9], w[10], w[11], inv), f8_codes4_near(w[12], w[13], w[14], w[15], inv));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + lane / 4, j = lane % 4, n = n0 + 16 * j;
          if (mw + r < x.m_lim && n < args.N)
            *reinterpret_cast<uint4*>(args.q + static_cast<size_t>(mw + r) * args.N + n) = *slot(r, j);
        }
        __syncwarp();
      } else {
        constexpr int CHUNKS = SW ? 2 : 4 / SPLIT;  // (a cut SwiGLU product is finished above)
#pragma unroll
        for (int h = 0; h < CHUNKS; ++h) {
          const int n0 = x.tn * TN + half * (TN / 2) + (rank * CHUNKS + h) * 32;
          if (EPI == F8_RESID) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = i * 8 + lane / 4, j = lane % 4, n = n0 + 8 * j;
              uint4 w = make_uint4(0u, 0u, 0u, 0u);
              if (mw + r < x.m_lim && n < args.N)
                w = *reinterpret_cast<const uint4*>(args.R + static_cast<size_t>(mw + r) * args.N + n);  // C may be R
              *slot(r, j) = w;
            }
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              w[i] = sum[h * 32 + j * 8 + i];
              if (SW) w[i] = silu_mul(w[i], sum[64 + h * 32 + j * 8 + i]);
            }
            if (EPI == F8_RESID) {
              const uint4 r = *slot(lane, j);
              w[0] += bf16lo(r.x); w[1] += bf16hi(r.x); w[2] += bf16lo(r.y); w[3] += bf16hi(r.y);
              w[4] += bf16lo(r.z); w[5] += bf16hi(r.z); w[6] += bf16lo(r.w); w[7] += bf16hi(r.w);
            }
            *slot(lane, j) = make_uint4(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7]));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + lane / 4, j = lane % 4, n = n0 + 8 * j;
            if (mw + r < x.m_lim && n < args.N)
              *reinterpret_cast<uint4*>(args.C + static_cast<size_t>(mw + r) * args.N + n) = *slot(r, j);
          }
          __syncwarp();
        }
      }
    }
    if (!ok) {
      raise_status(&g_status, ST_TIMEOUT);
      *abort_flag = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // Whoever gave up: products in flight end before tensor memory goes away, loads land
    // before shared memory does.
    if ((warp == 1 || warp == 2) && lane == tail->issuer[warp - 1]) {
      tc_commit(&tail->drain[warp - 1]);
      mbar_wait(&tail->drain[warp - 1], 0, F8_DRAIN_NS);
    }
    if (threadIdx.x == 0)
      for (int s = 0; s < STAGES; ++s)
        if (tail->issued & (1u << s)) mbar_wait(&tail->full[s], tail->phases >> s & 1, F8_DRAIN_NS);
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
  if (SPLIT > 1) cluster_leave();
}

// Counted where a poll finds it (counted by every thread that gives up, 4096 x 8192 x 28672
// takes 870 us, so 790: the compiler orders the sums otherwise).
__device__ uint32_t g_flags;
__global__ void count_flag_kernel() {
  if (atomicExch(&g_status, 0u)) ++g_flags;
}

// Clusters of SPLIT CTAs that the current device holds at once; asked once a device.
template <int EPI, int SPLIT>
cudaError_t most_clusters(int* most) {
  static ByDevice<1> kept;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return kept.get(dev, 0, most, [](int* n) {
    const auto kernel = gemm_f8_kernel<EPI, SPLIT>;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = SPLIT;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(SPLIT, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kernel), SMEM);
    return e == cudaSuccess ? cudaOccupancyMaxActiveClusters(n, kernel, &cfg) : e;
  });
}

template <int EPI, int SPLIT>
cudaError_t launch(const CUtensorMap& tmA, const CUtensorMap& tmB, const F8GemmArgs& args, int grid,
                   cudaStream_t stream) {
  const auto kernel = gemm_f8_kernel<EPI, SPLIT>;
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kernel), SMEM);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, grid, THREADS, SMEM, stream, SPLIT, tmA, tmB, args);
}

}  // namespace

cudaError_t launch_gemm_f8(int epi, const CUtensorMap& tmA, const CUtensorMap& tmB,
                           const F8GemmArgs& args, int sms, cudaStream_t stream) {
  const int tn = epi >= F8_SWIGLU ? BN / 2 : BN;
  const long long most = ((static_cast<long long>(args.M) + BM - 1) / BM + (args.group_off ? args.groups : 0)) *
                         ((args.N + tn - 1) / tn);
  if (most > 0x7fffffffLL || args.groups > F8_MAX_GROUPS) return cudaErrorInvalidValue;
  if (most <= 0) return cudaSuccess;
  // Tiles for at most half of the SMs, and eight blocks of K at least for each of two
  // CTAs.  Whole / cut: 333 x 6144 x 4096 18.4 / 15.8 us, 333 x 4096 x 14336 49 / 31,
  // 256 x 8192 x 28672 95 / 60; 512 x 2048 x 2048 11.5 either way, x 1024 8.4 / 9.5.  For at
  // most a quarter of the SMs four; two / four: 256 x 4096 x 14336 35 / 24, 256 x 4096 x 4096
  // 14.4 either way, x 2048 11.4 / 12.5, 256 x 2048 x 4096 SwiGLU 15.5 / 13.0.
  // A tile more than clusters fit is a second wave: 38 tiles of 256 x 4864 x 4096 in two parts
  // 14.8, in four (152 SMs, in groups that hold 36 clusters of four) 25.1.
  const int nk = (args.K + BK - 1) / BK;
  if (!args.group_off) {
    cudaError_t e = cudaSuccess;
    auto cut = [&](auto epilogue, auto split) {
      constexpr int EPI = decltype(epilogue)::value, SPLIT = decltype(split)::value;
      if (nk < 8 * SPLIT || SPLIT * most > sms) return false;
      int fit = 0;
      e = most_clusters<EPI, SPLIT>(&fit);
      if (e == cudaSuccess && most > fit) return false;
      if (e == cudaSuccess) e = launch<EPI, SPLIT>(tmA, tmB, args, static_cast<int>(SPLIT * most), stream);
      return true;
    };
    auto either = [&](auto epilogue) {
      return cut(epilogue, std::integral_constant<int, 4>{}) || cut(epilogue, std::integral_constant<int, 2>{});
    };
    if (epi == F8_STORE ? either(std::integral_constant<int, F8_STORE>{})
        : epi == F8_RESID  ? either(std::integral_constant<int, F8_RESID>{})
        : epi == F8_SWIGLU ? either(std::integral_constant<int, F8_SWIGLU>{})
                           : epi == F8_SWIGLU8 && either(std::integral_constant<int, F8_SWIGLU8>{}))
      return e;
  }
  const int grid = static_cast<int>(most < sms ? most : sms);
  switch (epi) {
    case F8_STORE: return launch<F8_STORE, 1>(tmA, tmB, args, grid, stream);
    case F8_RESID: return launch<F8_RESID, 1>(tmA, tmB, args, grid, stream);
    case F8_SWIGLU: return launch<F8_SWIGLU, 1>(tmA, tmB, args, grid, stream);
    case F8_SWIGLU8: return launch<F8_SWIGLU8, 1>(tmA, tmB, args, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t count_gemm_f8_flags(uint32_t* count, cudaStream_t stream) {
  count_flag_kernel<<<1, 1, 0, stream>>>();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? cudaMemcpyFromSymbolAsync(count, g_flags, 4, 0, cudaMemcpyDeviceToHost, stream) : e;
}

}  // namespace nf
