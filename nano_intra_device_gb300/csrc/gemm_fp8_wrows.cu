// The product of gemm_fp8.cu for few rows of A (a decode step, an expert's few
// tokens): B's rows are the 128-row operand and A's the N side.
//
// Such a product streams B once, 1 byte a value, and is bound by HBM.  So
//  * a tile is 128 features x TOK rows of A (16, 32, 64 or 128), its ring mostly B;
//  * the K range is split over the CTAs of a thread-block cluster (up to 8), each
//    with its own slice of B, and summed through distributed shared memory in rank
//    order, without workspace and the same at every run;
//  * a CTA of at most 64 accumulator columns takes no more than half of an SM (113 KB), so
//    that the next CTAs, of this launch or of the next product, start beside the ending
//    ones (64 rows of 8 experts of 2 x 14336 x 4096: 142 us; with rings of 220 KB 157);
//  * a block of K has its own accumulator, as in gemm_fp8.cu, but here a thread's row
//    is a feature and the scale changes from column to column: the products of A's
//    and B's scales go through a few floats of shared memory a warp;
//  * the exchange lays the sums out by row of A, 128 features a warp, so that SwiGLU,
//    the residual and the scale of an 8-bit output are a warp's own.
// By experts, a grid for the most tiles that the rows can make is launched and the
// CTAs find their group from the offsets; those past the last tile leave.
// Launched as a programmatic dependent of the kernel ahead.
// Every wait is bounded.  After one gave up the CTAs of a cluster still meet at the
// same exchange and the barrier before exit.
#include <algorithm>
#include <type_traits>

#include "by_device.h"
#include "fp8.cuh"
#include "kernels.h"

namespace nf {
namespace {

constexpr int WM = 128, BK = F8_BLOCK;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_STAGES = 8;
constexpr int TAIL_BYTES = 256;

template <int EPI, int TOK>
struct Cfg {
  static constexpr int NA = EPI >= F8_SWIGLU ? 2 : 1;   // operands of B (gate, up)
  static constexpr int COLS = NA * TOK;                 // columns of an accumulator
  static constexpr int HALVES = COLS > 64 ? 2 : 1;      // summing warps: 4 a half
  static constexpr int MINE = COLS / HALVES;            // columns of a thread
  static constexpr int THREADS = 64 + 128 * HALVES;
  static constexpr int ACCS = 4;                         // accumulators, in turn
  static constexpr int TMEM = ACCS * COLS < 32 ? 32 : ACCS * COLS;
  static constexpr int STAGE = NA * WM * BK + TOK * BK;
  static constexpr int SCALES = 4 * HALVES * 2 * MINE * 4;
  static constexpr int PER_SM = HALVES == 2 ? 1 : 2;     // CTAs that fit into an SM
  static constexpr int LIMIT = PER_SM == 2 ? 115712 : 232448;
  static constexpr int FIT = (LIMIT - 1024 - TAIL_BYTES - SCALES) / STAGE;
  static constexpr int STAGES = FIT < MAX_STAGES ? FIT : MAX_STAGES;
  static constexpr int SMEM = 1024 + STAGES * STAGE + SCALES + TAIL_BYTES;
  static_assert(STAGES >= 2 && SMEM <= LIMIT, "ring");
  static_assert(COLS * WM * 4 <= STAGES * STAGE, "the exchange reuses the ring");
  static_assert((TMEM & (TMEM - 1)) == 0 && TMEM <= 512 / PER_SM, "two CTAs' accumulators");
};

struct Tail {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t tfull[4];
  uint64_t tempty[4];
  uint64_t drain;
  uint64_t ready;  // every rank's sums are in its shared memory
  uint32_t tmem_base;
  int abort;
  int e, m0, m_lim, wt;  // this cluster's tile (m_lim 0: none)
};
static_assert(sizeof(Tail) <= TAIL_BYTES, "barrier block");

__device__ uint32_t g_status;

template <int EPI, int TOK>
__global__ void __launch_bounds__(Cfg<EPI, TOK>::THREADS, Cfg<EPI, TOK>::PER_SM)
    gemm_f8_wrows_kernel(const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmX, const F8GemmArgs args) {
  using C = Cfg<EPI, TOK>;
  constexpr int NA = C::NA, STAGES = C::STAGES, MINE = C::MINE, ACCS = C::ACCS;
  constexpr uint32_t IDESC = idesc_e4m3_f32(WM, TOK);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  float* xbuf = reinterpret_cast<float*>(smem);  // [column][feature], once the ring is done
  float* scales = reinterpret_cast<float*>(smem + STAGES * C::STAGE);
  Tail* tail = reinterpret_cast<Tail*>(smem + STAGES * C::STAGE + C::SCALES);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = args.splits, rank = static_cast<int>(cluster_rank());
  const int unit = static_cast<int>(cluster_id_x());
  const int nk = (args.K + BK - 1) / BK, nb = (args.N + F8_BLOCK - 1) / F8_BLOCK;
  const uint64_t tmo = args.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
    }
    for (int a = 0; a < ACCS; ++a) {
      mbar_init(&tail->tfull[a], 1);
      mbar_init(&tail->tempty[a], 4 * C::HALVES);
    }
    mbar_init(&tail->drain, 1);
    mbar_init(&tail->ready, S);
    tail->abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (threadIdx.x == 0 && !args.group_off) {
    // the first blocks of B are on their way from memory while the kernel ahead ends
    const int w = unit / ((args.M + TOK - 1) / TOK), a = rank * nk / S, n = (rank + 1) * nk / S - a;
    const int turn = static_cast<int>(static_cast<long long>(w) * n / nb) % n;
    for (int i = 0; i < min(STAGES, n); ++i) {
      const int kx = (a + (i + turn >= n ? i + turn - n : i + turn)) * BK;
      tma_prefetch_2d(&tmW, kx, w * WM);
      if (NA == 2) tma_prefetch_2d(&tmW, kx, w * WM + args.N);
    }
  }
  pdl_wait();  // nothing before this reads or writes global memory but into L2
  // Tensor memory is taken once the kernel ahead is complete, and the kernel behind let
  // start once it is taken: neither can wait for columns that the other holds.
  if (warp == 1) {
    tmem_alloc(&tail->tmem_base, C::TMEM);
    tmem_relinquish();
  }
  if (warp == 2) {
    if (!args.group_off) {
      if (lane == 0) {
        const int mt = (args.M + TOK - 1) / TOK;
        tail->e = 0;
        tail->m0 = unit % mt * TOK;
        tail->m_lim = args.M;
        tail->wt = unit / mt;
      }
    } else {
      // The group of this unit; offsets as in gemm_fp8.cu: within [0, M], never falling.
      int top = 0, tiles = 0;
      if (lane == 0) tail->m_lim = tail->m0 = tail->e = tail->wt = 0;
      __syncwarp();
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
        const int before = lane ? up : top;
        const int mt = i > 0 && i <= args.groups ? (o - before + TOK - 1) / TOK : 0;
        int t = mt * nb;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, t, d);
          if (lane >= d) t += y;
        }
        t += tiles;  // tiles up to and with group i - 1
        const int u = unit - (t - mt * nb);
        if (u >= 0 && u < mt * nb) {
          tail->e = i - 1;
          tail->m0 = before + u % mt * TOK;
          tail->m_lim = o;
          tail->wt = u / mt;
        }
        top = __shfl_sync(0xffffffffu, o, 31);
        tiles = __shfl_sync(0xffffffffu, t, 31);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  cluster_arrive();  // this CTA's barriers exist; each thread waits for the peers' further down
  const uint32_t tmem_base = tail->tmem_base;
  volatile int* abort_flag = &tail->abort;
  const int e = tail->e, m0 = tail->m0, m_lim = tail->m_lim, wt = tail->wt;
  const bool work = m0 < m_lim;  // the same in all CTAs of the cluster
  const int kb0 = rank * nk / S, klen = work ? (rank + 1) * nk / S - kb0 : 0;
  // The CTAs start together; each tile begins elsewhere in its K range, so that they do
  // not all ask for the same columns of B's rows at once.
  const int rot = klen > 0 ? static_cast<int>(static_cast<long long>(wt) * klen / nb) % klen : 0;
  auto kb_at = [&](int i) { return kb0 + (i + rot >= klen ? i + rot - klen : i + rot); };

  uint32_t issued = 0, phases = 0;  // thread 0: the ring's stages and the phase of their last load
  bool issuer = false;              // this thread has issued products
  if (warp == 0) {
    if (lane == 0) {
      const int w0 = e * NA * args.N + wt * WM;
      uint32_t st = 0, ph = 0;
      for (int i = 0; i < klen; ++i) {
        if (!mbar_wait(&tail->empty[st], ph ^ 1, tmo, abort_flag)) {
          raise_status(&g_status, ST_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        uint8_t* sa = smem + st * C::STAGE;
        uint64_t* bar = &tail->full[st];
        const int kx = kb_at(i) * BK;
        mbar_arrive_expect_tx(bar, C::STAGE);
        tma_load_2d(sa, &tmW, bar, kx, w0);
        if (NA == 2) tma_load_2d(sa + WM * BK, &tmW, bar, kx, w0 + args.N);
        tma_load_2d(sa + NA * WM * BK, &tmX, bar, kx, m0);
        issued |= 1u << st;
        phases = (phases & ~(1u << st)) | ph << st;
        if (++st == STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t st = 0, ph = 0, acc = 0, aph = 0;
      for (int i = 0; i < klen; ++i) {
        if (!mbar_wait(&tail->tempty[acc], aph ^ 1, tmo, abort_flag) ||
            !mbar_wait(&tail->full[st], ph, tmo, abort_flag)) {
          raise_status(&g_status, ST_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + st * C::STAGE), d = tmem_base + acc * C::COLS;
        const uint64_t w0 = desc_sw128_kmajor(sa), w1 = desc_sw128_kmajor(sa + WM * BK);
        const uint64_t xd = desc_sw128_kmajor(sa + NA * WM * BK);
#pragma unroll
        for (int k = 0; k < BK / 32; ++k) {
          tc_mma_e4m3(d, w0 + 2 * k, xd + 2 * k, IDESC, k != 0);
          if (NA == 2) tc_mma_e4m3(d + TOK, w1 + 2 * k, xd + 2 * k, IDESC, k != 0);
        }
        issuer = true;
        tc_commit(&tail->empty[st]);
        tc_commit(&tail->tfull[acc]);
        if (++st == STAGES) {
          st = 0;
          ph ^= 1;
        }
        if (++acc == ACCS) {
          acc = 0;
          aph ^= 1;
        }
      }
    }
  }
  if (warp < 2 || !work) {
    cluster_wait();
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int row = quarter * 32 + lane;  // feature of the tile
    float* sc = scales + (warp - 2) * 2 * MINE;
    float sum[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) sum[i] = 0.f;
    // Column half * MINE + lane + 32 i of the accumulator: its row of A, its operand of B.
    constexpr int CI = (MINE + 31) / 32, AHEAD = 4;
    const float* bs = args.b_s + (static_cast<size_t>(e) * NA * nb + wt) * nk;
    float px[AHEAD][CI], pw[AHEAD][CI];  // of the next blocks of K, each in its place of a ring
    auto fetch = [&](int i, int at) {
#pragma unroll
      for (int j = 0; j < CI; ++j) {
        const int c = half * MINE + lane + 32 * j, t = m0 + c % TOK;
        const bool on = i < klen && c < C::COLS && t < m_lim;
        const int kb = i < klen ? kb_at(i) : 0;
        px[at][j] = on ? args.a_s[static_cast<size_t>(kb) * args.M + t] : 0.f;
        pw[at][j] = on ? bs[(c / TOK) * static_cast<size_t>(nb) * nk + kb] : 0.f;
      }
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(i, i);
    uint32_t acc = 0, aph = 0;
    bool ok = true;
    auto block = [&](int i, int at) {
      float* p = sc + (at & 1) * MINE;
#pragma unroll
      for (int j = 0; j < CI; ++j)
        if (lane + 32 * j < MINE) p[lane + 32 * j] = px[at][j] * pw[at][j];
      fetch(i + AHEAD, at);
      // also makes p visible to the warp; it is overwritten two rounds later, behind the
      // next round's vote
      if (!__all_sync(0xffffffffu, mbar_wait(&tail->tfull[acc], aph, tmo, abort_flag))) return false;
      __syncwarp();
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * C::COLS + half * MINE;
      uint32_t v[MINE / 16 > 1 ? 2 : 1][16];
      tc_ld_32x32b_x16(tb, v[0]);
#pragma unroll
      for (int c = 0; c < MINE / 16; ++c) {
        tc_wait_ld();
        if (c + 1 < MINE / 16) {
          tc_ld_32x32b_x16(tb + 16 * (c + 1), v[(c + 1) & 1]);
        } else {
          tc_fence_before();
          __syncwarp();
          mbar_arrive_if(&tail->tempty[acc], lane == 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 s = *reinterpret_cast<const float4*>(p + 16 * c + 4 * j);
          float* d = sum + 16 * c + 4 * j;
          const uint32_t* a = v[c & 1] + 4 * j;
          fma_loaded(d[0], a[0], s.x);
          fma_loaded(d[1], a[1], s.y);
          fma_loaded(d[2], a[2], s.z);
          fma_loaded(d[3], a[3], s.w);
        }
      }
      if (++acc == ACCS) {
        acc = 0;
        aph ^= 1;
      }
      return true;
    };
#pragma unroll 1
    for (int i = 0; i < klen && ok; i += AHEAD)
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        if (ok && i + j < klen) ok = block(i + j, j);
    if (!ok) {
      raise_status(&g_status, ST_TIMEOUT);
      *abort_flag = 1;
    }
    // The exchange: this CTA's sums to its shared memory (every product that read the
    // ring has completed), then each rank adds all ranks' for its share of the rows.
    // After a failure the ring may still be written: nothing is stored.
    if (ok) {
#pragma unroll
      for (int j = 0; j < MINE; ++j) xbuf[(half * MINE + j) * WM + row] = sum[j];
    }
    cluster_wait();  // every peer's barriers exist
    asm volatile("bar.sync 1, %0;" ::"n"(128 * C::HALVES) : "memory");
    // (a release at cluster scope, behind the barrier that all of the CTA's writes precede)
    if (warp == 2 && lane < S) mbar_arrive_remote(cluster_map(smem_u32(&tail->ready), lane));
    if (!__all_sync(0xffffffffu, mbar_wait_cluster(&tail->ready, 0, tmo))) {
      raise_status(&g_status, ST_TIMEOUT);
      *abort_flag = 1;
    } else {
      const int nv = min(TOK, m_lim - m0);
      const int c0 = rank * nv / S, c1 = (rank + 1) * nv / S;
      const int n = wt * WM + lane * 4;  // a lane's 4 features
      const bool in = n < args.N;
      const uint32_t xa = smem_u32(xbuf) + lane * 16;
      // Columns together, so that 16 loads of peers' sums are under way a thread: one column at
      // a time 64 rows of 4096 x 14336 take 18.1 us, so 16.9; 64 x 6144 x 4096 12.0 and 11.3;
      // 128 x 4096 x 14336 18.9 and 18.4 (the sums' 64 KB a CTA).  RANKS: S or more.
      constexpr int NW = 4 * C::HALVES;
      auto finish = [&](auto ranks) {
        constexpr int RANKS = decltype(ranks)::value, G = TOK >= 32 ? 16 / (RANKS * NA) : 1;
        for (int c = c0 + (warp - 2); c < c1; c += NW * G) {
          float4 v[G][NA][RANKS];
          uint2 r[G];
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const int cg = c + NW * g;
            r[g] = make_uint2(0u, 0u);
            if (G == 1 || cg < c1) {
              if (EPI == F8_RESID && in)  // C may be R
                r[g] = *reinterpret_cast<const uint2*>(args.R + static_cast<size_t>(m0 + cg) * args.N + n);
#pragma unroll
              for (int j = 0; j < RANKS; ++j) {
                if (j < S) {
                  const uint32_t at = cluster_map(xa, j) + cg * (WM * 4);
#pragma unroll
                  for (int h = 0; h < NA; ++h) v[g][h][j] = ld_cluster_f4(at + h * (TOK * WM * 4));
                }
              }
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const int cg = c + NW * g;
            if (G > 1 && cg >= c1) break;
            const size_t t = static_cast<size_t>(m0 + cg);
            float s[NA][4] = {};
#pragma unroll
            for (int h = 0; h < NA; ++h)
#pragma unroll
              for (int j = 0; j < RANKS; ++j)
                if (j < S) {
                  s[h][0] += v[g][h][j].x; s[h][1] += v[g][h][j].y; s[h][2] += v[g][h][j].z; s[h][3] += v[g][h][j].w;
                }
            float(&o)[4] = s[0];
            if (NA == 2) {
#pragma unroll
              for (int k = 0; k < 4; ++k) o[k] = in ? silu_mul(o[k], s[NA - 1][k]) : 0.f;
            }
            if (EPI == F8_RESID) {
              o[0] += bf16lo(r[g].x); o[1] += bf16hi(r[g].x); o[2] += bf16lo(r[g].y); o[3] += bf16hi(r[g].y);
            }
            if (EPI == F8_SWIGLU8) {
              float top = 0.f;
#pragma unroll
              for (int k = 0; k < 4; ++k) top = absmax_nan(top, o[k]);
#pragma unroll
              for (int d = 16; d > 0; d >>= 1) top = absmax_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
              const float q = f8_scale(top), inv = 1.f / q;
              if (in) *reinterpret_cast<uint32_t*>(args.q + t * args.N + n) = f8_codes4_near(o[0], o[1], o[2], o[3], inv);
              if (lane == 0) args.c_s[static_cast<size_t>(wt) * args.M + t] = q;
            } else if (in) {
              *reinterpret_cast<uint2*>(args.C + t * args.N + n) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
            }
          }
        }
      };
      if (TOK < 32 || S > 4) finish(std::integral_constant<int, 8>{});
      else finish(std::integral_constant<int, 4>{});
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // Whoever gave up: products in flight end before tensor memory goes away, loads land
    // before shared memory does.
    if (issuer) {
      tc_commit(&tail->drain);
      mbar_wait(&tail->drain, 0, F8_DRAIN_NS);
    }
    if (threadIdx.x == 0)
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) mbar_wait(&tail->full[s], phases >> s & 1, F8_DRAIN_NS);
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM);
  }
  cluster_leave();
}

__device__ uint32_t g_flags;
__global__ void count_flag_kernel() {
  if (atomicExch(&g_status, 0u)) ++g_flags;
}

template <int EPI, int TOK>
void configure(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* at, int clusters, int splits, cudaStream_t stream) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(static_cast<unsigned>(clusters * splits), 1, 1);
  cfg->blockDim = dim3(Cfg<EPI, TOK>::THREADS, 1, 1);
  cfg->dynamicSmemBytes = Cfg<EPI, TOK>::SMEM;
  cfg->stream = stream;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(splits);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  // its barriers are made while the kernel ahead ends
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = at;
  cfg->numAttrs = 2;
}

template <int EPI, int TOK>
cudaError_t prepare() {
  return set_smem_limit(reinterpret_cast<const void*>(gemm_f8_wrows_kernel<EPI, TOK>), Cfg<EPI, TOK>::SMEM);
}

template <int EPI, int TOK>
cudaError_t launch(const CUtensorMap& tmW, const CUtensorMap& tmX, const F8GemmArgs& args, int clusters,
                   cudaStream_t stream) {
  const cudaError_t e = prepare<EPI, TOK>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute at[2];
  configure<EPI, TOK>(&cfg, at, clusters, args.splits, stream);
  return cudaLaunchKernelEx(&cfg, gemm_f8_wrows_kernel<EPI, TOK>, tmW, tmX, args);
}

// Clusters of `splits` CTAs that the current device holds at once, one CTA an SM (more is
// not reported for kernels with tensor memory); asked once a device.
template <int EPI, int TOK>
cudaError_t most_clusters(int splits, int* most) {
  static ByDevice<MAX_CLUSTER + 1> kept;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return kept.get(dev, splits, most, [splits](int* n) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at[2];
    configure<EPI, TOK>(&cfg, at, 1, splits, nullptr);
    cfg.numAttrs = 1;
    const cudaError_t e = prepare<EPI, TOK>();
    return e == cudaSuccess ? cudaOccupancyMaxActiveClusters(n, gemm_f8_wrows_kernel<EPI, TOK>, &cfg) : e;
  });
}

// f(epilogue, rows of A of a tile) with both as compile-time constants; -1 for others.
template <typename F>
int dispatch(int epi, int tok, F f) {
  using std::integral_constant;
  auto at = [&](auto e) {
    switch (tok) {
      case 16: return f(e, integral_constant<int, 16>{});
      case 32: return f(e, integral_constant<int, 32>{});
      case 64: return f(e, integral_constant<int, 64>{});
      case 128:
        if constexpr (F8_SWIGLU > decltype(e)::value) return f(e, integral_constant<int, 128>{});
      default: return -1;
    }
  };
  switch (epi) {
    case F8_STORE: return at(integral_constant<int, F8_STORE>{});
    case F8_RESID: return at(integral_constant<int, F8_RESID>{});
    case F8_SWIGLU: return at(integral_constant<int, F8_SWIGLU>{});
    case F8_SWIGLU8: return at(integral_constant<int, F8_SWIGLU8>{});
    default: return -1;
  }
}

}  // namespace

cudaError_t gemm_f8_wrows_choice(int epi, int M, int N, int K, int groups, F8RowsChoice* choice) {
  F8RowsChoice& c = *choice;
  const int rows = (M + groups - 1) / groups;  // of a group, were they even
  const int most = epi >= F8_SWIGLU ? 64 : 128;
  // by groups: room for twice the mean, as B is read again for each further tile
  const int want = groups > 1 ? 2 * rows : rows;
  c.tok = want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 || most == 64 ? 64 : 128;
  const long long wt = (N + WM - 1) / WM;
  c.units = groups > 1 ? wt * (M / c.tok + (M < groups ? M : groups)) : wt * ((M + c.tok - 1) / c.tok);
  // As many CTAs as the device holds at once, but four blocks of K each at least.  Where an
  // SM holds two, for one / both: 1 row of 4096 x 14336 15.3 / 13.2 us, of 10240 x 4096
  // 14.7 / 10.0, of 10240 x 14336 40.6 / 26.5, 64 rows of 14336 x 4096 18.3 / 15.1, 16 rows of
  // 14336 x 4096 SwiGLU 24.8 / 22.9.  A group of SMs that holds n clusters of s CTAs, one an
  // SM, holds 2 n of them two an SM, or n of 2 s.  One part more than fits is a second wave:
  // 1 row of 8192 x 4096 in 4 parts 8.5, in 5 13.9.
  const long long busy = wt * (groups > 1 ? (M < groups ? M : groups) : (M + c.tok - 1) / c.tok);
  const int nk = (K + BK - 1) / BK;
  c.splits = 1;
  for (int s = 2; s <= MAX_CLUSTER && 4 * s <= nk; ++s) {
    int fit = 0;
    const int e = dispatch(epi, c.tok, [&](auto epilogue, auto tok) {
      constexpr int EPI = decltype(epilogue)::value, TOK = decltype(tok)::value;
      int half = 0;
      cudaError_t e = most_clusters<EPI, TOK>(s, &fit);
      if (Cfg<EPI, TOK>::PER_SM == 1) return static_cast<int>(e);
      fit *= 2;
      if (e == cudaSuccess && s > 2) e = most_clusters<EPI, TOK>((s + 1) / 2, &half);
      fit = std::max(fit, half);
      return static_cast<int>(e);
    });
    if (e) return e < 0 ? cudaErrorInvalidValue : static_cast<cudaError_t>(e);
    if (busy <= fit) c.splits = s;
  }
  return cudaSuccess;
}

cudaError_t launch_gemm_f8_wrows(int epi, int tok, const CUtensorMap& tmW, const CUtensorMap& tmX,
                                 const F8GemmArgs& args, long long units, cudaStream_t stream) {
  if (units <= 0) return cudaSuccess;
  if (args.splits < 1 || args.splits > MAX_CLUSTER || units * args.splits > 0x7fffffffLL)
    return cudaErrorInvalidValue;
  const int e = dispatch(epi, tok, [&](auto e, auto k) {
    return static_cast<int>(launch<decltype(e)::value, decltype(k)::value>(tmW, tmX, args, static_cast<int>(units), stream));
  });
  return e < 0 ? cudaErrorInvalidValue : static_cast<cudaError_t>(e);
}

cudaError_t count_gemm_f8_wrows_flags(uint32_t* count, cudaStream_t stream) {
  count_flag_kernel<<<1, 1, 0, stream>>>();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? cudaMemcpyFromSymbolAsync(count, g_flags, 4, 0, cudaMemcpyDeviceToHost, stream) : e;
}

}  // namespace nf
