// Products of e4m3 operands with a scale for each block of 128, on tcgen05:
//
//   C[m, n] = sum_b a_s[b, m] b_s[n / 128, b] sum_{k in block b} a[m, k] b[n, k]
//
// for one matrix, or by groups of rows (experts) whose bounds are on the device.
//  * A tile is 128 rows of A x 256 rows of B (SwiGLU: 128 features' gate and up rows),
//    so a thread's row has one scale of A and a warp's columns one or two of B a
//    block of K.  A ring stage is one block of K: 128 bytes a row, one swizzled row.
//  * Scales are fp32 and change with every block of K, so a block's products go to an
//    accumulator of their own in tensor memory (two, in turn), and eight warps
//    add it, times its scale, to sums in registers (fp32, packed in pairs): while they
//    do, the tensor core fills the other accumulator.
//  * Warp 0 loads tiles by TMA, warp 1 issues the products, warps 4 to 11 sum and run
//    the epilogue.  Persistent CTAs, one an SM.
//  * Every wait is bounded; one that gives up flags the status word, and the kernel
//    drains what it has in flight (bounded) and frees tensor memory.
#include "fp8.cuh"
#include "kernels.h"

namespace nf {
namespace {

constexpr int BM = 128, BN = 256, BK = F8_BLOCK;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int THREADS = 384;
// Registers: 384 threads start with 168 each (64,512); the first warpgroup keeps 72,
// the summing warps take 208: 4 * 32 * 72 + 8 * 32 * 208 = 62,464.
constexpr int REGS_FEW = 72, REGS_SUM = 208;
constexpr int TMEM_COLS = 512;
constexpr int STORE_BYTES = 8 * 4096;  // 32 rows x 64 columns of bf16 a warp
constexpr int TAIL_BYTES = 1280;

struct Tail {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t pair[4];  // the two warps of 32 rows (SWIGLU8: the block's largest value)
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int tile0[F8_MAX_GROUPS + 1];  // first tile of each group
  int row0[F8_MAX_GROUPS + 1];   // first row of each group
};
constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + STORE_BYTES + TAIL_BYTES;
static_assert(sizeof(Tail) <= TAIL_BYTES && SMEM <= 232448, "shared memory");

__device__ uint32_t g_status;

struct Tile {
  int m0, m_lim, tn, e;
};

template <int EPI>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_f8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const F8GemmArgs args) {
  constexpr bool SW = EPI == F8_SWIGLU || EPI == F8_SWIGLU8;
  constexpr int TN = SW ? BN / 2 : BN;  // output columns of a tile
  constexpr uint32_t IDESC = idesc_e4m3_f32(BM, BN);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Tail* tail = reinterpret_cast<Tail*>(smem + STAGES * STAGE_BYTES + STORE_BYTES);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nk = (args.K + BK - 1) / BK, n_tiles = (args.N + TN - 1) / TN;
  const int nb = (args.N + F8_BLOCK - 1) / F8_BLOCK;
  const bool grouped = args.group_off != nullptr;
  const uint64_t tmo = args.timeout_ns;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tail->tfull[a], 1);
      mbar_init(&tail->tempty[a], 8);
    }
    for (int a = 0; a < 4; ++a) mbar_init(&tail->pair[a], 2);
    mbar_init(&tail->drain, 1);
    tail->abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(&tail->tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();  // nothing before this reads or writes global memory
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

  uint32_t issued = 0, phases = 0;  // thread 0: the ring's stages and the phase of their last load
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_FEW));
    if (warp == 0 && lane == 0) {
      uint32_t st = 0, ph = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        const Tile x = decode(u);
        const int b0 = x.e * (SW ? 2 : 1) * args.N + x.tn * TN;
        const int b1 = SW ? b0 + args.N : b0 + 128;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&tail->empty[st], ph ^ 1, tmo, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + st * STAGE_BYTES;
          uint64_t* bar = &tail->full[st];
          mbar_arrive_expect_tx(bar, STAGE_BYTES);
          tma_load_2d(sa, &tmA, bar, kb * BK, x.m0);
          tma_load_2d(sa + A_BYTES, &tmB, bar, kb * BK, b0);
          tma_load_2d(sa + A_BYTES + B_BYTES / 2, &tmB, bar, kb * BK, b1);
          issued |= 1u << st;
          phases = (phases & ~(1u << st)) | ph << st;
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
    }
    if (warp == 1 && lane == 0) {
      uint32_t st = 0, ph = 0, acc = 0, aph = 0;
      bool ok = true, any = false;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&tail->tempty[acc], aph ^ 1, tmo, abort_flag) ||
              !mbar_wait(&tail->full[st], ph, tmo, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + st * STAGE_BYTES);
          const uint64_t ad = desc_sw128_kmajor(sa), bd = desc_sw128_kmajor(sa + A_BYTES);
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)  // 32 codes = 32 bytes along the swizzled row
            tc_mma_e4m3(tmem_base + acc * BN, ad + 2 * k, bd + 2 * k, IDESC, k != 0);
          any = true;
          tc_commit(&tail->empty[st]);
          tc_commit(&tail->tfull[acc]);
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
      if (!ok) {
        raise_status(&g_status, ST_TIMEOUT);
        *abort_flag = 1;
        if (any) {  // the products already issued end before tensor memory goes away
          tc_commit(&tail->drain);
          mbar_wait(&tail->drain, 0, tmo);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SUM));
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row_in_tile = quarter * 32 + lane;
    // This thread's columns of the accumulator: chunks of 32 from col(c).  SwiGLU: 64
    // features' gate columns, then the same features' up columns.
    auto col = [&](int c) { return SW ? (c >> 1) * 128 + half * 64 + (c & 1) * 32 : half * 128 + c * 32; };
    uint8_t* mine = smem + STAGES * STAGE_BYTES + (warp - 4) * 4096;
    uint32_t acc = 0, aph = 0, parity = 0, pph = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
      const Tile x = decode(u);
      const int m = x.m0 + row_in_tile;
      const bool row_ok = m < x.m_lim;
      const int blk = SW ? x.tn : min(2 * x.tn + half, nb - 1);
      const float* bs0 = args.b_s + (static_cast<size_t>(x.e) * (SW ? 2 : 1) * nb + blk) * nk;
      const float* bs1 = SW ? bs0 + static_cast<size_t>(nb) * nk : bs0;
      const float* as = args.a_s + m;
      f32x2 sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      // scales, two blocks of K ahead of their use
      float sa[3], sb[3], sc[3];
      auto scales = [&](int kb, int i) {
        const bool on = kb < nk;
        sa[i] = on && row_ok ? __ldg(as + static_cast<size_t>(kb) * args.M) : 0.f;
        sb[i] = on ? __ldg(bs0 + kb) : 0.f;
        if (SW) sc[i] = on ? __ldg(bs1 + kb) : 0.f;
      };
      scales(0, 0);
      scales(1, 1);
      for (int kb = 0; kb < nk; ++kb) {
        scales(kb + 2, 2);
        if (!__all_sync(0xffffffffu, mbar_wait(&tail->tfull[acc], aph, tmo, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float s0 = sa[0] * sb[0], s1 = SW ? sa[0] * sc[0] : s0;
        const f32x2 p0 = pack_f32x2(s0, s0), p1 = pack_f32x2(s1, s1);
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN;
        uint32_t v[2][32];
        tc_ld_32x32b_x32(tb + col(0), v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tc_wait_ld();
          if (c < 3) {
            tc_ld_32x32b_x32(tb + col(c + 1), v[(c + 1) & 1]);
          } else {
            tc_fence_before();
            if (lane == 0) mbar_arrive(&tail->tempty[acc]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            fma_f32x2(sum[c * 16 + i], pack_b32x2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), c < 2 ? p0 : p1);
        }
        sa[0] = sa[1]; sa[1] = sa[2];
        sb[0] = sb[1]; sb[1] = sb[2];
        sc[0] = sc[1]; sc[1] = sc[2];
        if (++acc == 2) {
          acc = 0;
          aph ^= 1;
        }
      }
      if (!ok) break;
      // Epilogue, through the warp's own 4 KB: 32 rows x 128 bytes, 16-byte chunk j of
      // row r at chunk j ^ (r & 7), so that rows are written and 128-byte lines stored
      // without bank conflicts.
      auto slot = [&](int r, int j) { return reinterpret_cast<uint4*>(mine + r * 128 + ((j ^ (r & 7)) << 4)); };
      const int mw = x.m0 + quarter * 32;  // first row of this warp
      if (EPI == F8_SWIGLU8) {
        const int n0 = x.tn * TN + half * 64;
        float o[64], top = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float g0, g1, u0, u1;
          unpack_f32x2(sum[i], g0, g1);
          unpack_f32x2(sum[32 + i], u0, u1);
          const bool in = n0 + 2 * i < args.N;  // N is even
          o[2 * i] = in ? __fdividef(g0, 1.f + __expf(-g0)) * u0 : 0.f;
          o[2 * i + 1] = in ? __fdividef(g1, 1.f + __expf(-g1)) * u1 : 0.f;
          top = absmax_nan(absmax_nan(top, o[2 * i]), o[2 * i + 1]);
        }
        // The block's 128 features are this thread's and those of the other half's warp;
        // the codes take 2 KB of a warp's 4, so the largest values fit behind them.
        auto top_at = [&](int w) {
          return reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES + w * 4096 + 2048 + parity * 128);
        };
        top_at(warp - 4)[lane] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->pair[quarter]);
        if (!__all_sync(0xffffffffu, mbar_wait(&tail->pair[quarter], pph, tmo, abort_flag))) {
          ok = false;
          break;
        }
        top = absmax_nan(top, top_at((warp - 4) ^ 4)[lane]);
        parity ^= 1;
        pph ^= 1;
        const float s = f8_scale(top), inv = 1.f / s;
        auto slot8 = [&](int r, int j) { return reinterpret_cast<uint4*>(mine + r * 64 + ((j ^ (r >> 1 & 3)) << 4)); };
        if (half == 0 && row_ok) args.c_s[static_cast<size_t>(x.tn) * args.M + m] = s;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float* w = o + 16 * j;
          *slot8(lane, j) = make_uint4(f8_codes4(w[0], w[1], w[2], w[3], s, inv), f8_codes4(w[4], w[5], w[6], w[7], s, inv),
                                      f8_codes4(w[8], w[9], w[10], w[11], s, inv), f8_codes4(w[12], w[13], w[14], w[15], s, inv));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + lane / 4, j = lane % 4, n = n0 + 16 * j;
          if (mw + r < x.m_lim && n < args.N)
            *reinterpret_cast<uint4*>(args.q + static_cast<size_t>(mw + r) * args.N + n) = *slot8(r, j);
        }
        __syncwarp();
      } else {
#pragma unroll
        for (int h = 0; h < (SW ? 1 : 2); ++h) {
          const int n0 = SW ? x.tn * TN + half * 64 : x.tn * TN + half * 128 + h * 64;
          if (EPI == F8_RESID) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = i * 4 + lane / 8, j = lane % 8, n = n0 + 8 * j;
              uint4 w = make_uint4(0u, 0u, 0u, 0u);
              if (mw + r < x.m_lim && n < args.N)
                w = __ldg(reinterpret_cast<const uint4*>(args.R + static_cast<size_t>(mw + r) * args.N + n));
              *slot(r, j) = w;
            }
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              unpack_f32x2(sum[h * 32 + j * 4 + i], w[2 * i], w[2 * i + 1]);
              if (SW) {
                float u0, u1;
                unpack_f32x2(sum[32 + j * 4 + i], u0, u1);
                w[2 * i] = __fdividef(w[2 * i], 1.f + __expf(-w[2 * i])) * u0;
                w[2 * i + 1] = __fdividef(w[2 * i + 1], 1.f + __expf(-w[2 * i + 1])) * u1;
              }
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
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + lane / 8, j = lane % 8, n = n0 + 8 * j;
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
  if (threadIdx.x == 0 && *abort_flag)  // loads in flight land before shared memory goes away
    for (int s = 0; s < STAGES; ++s)
      if (issued & (1u << s)) mbar_wait(&tail->full[s], phases >> s & 1, tmo);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

__device__ uint32_t g_taken;
__global__ void take_status_kernel() { g_taken = atomicExch(&g_status, 0u); }

template <int EPI>
cudaError_t launch(const CUtensorMap& tmA, const CUtensorMap& tmB, const F8GemmArgs& args, int grid,
                   cudaStream_t stream) {
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(gemm_f8_kernel<EPI>), SMEM);
  if (e != cudaSuccess) return e;
  return launch_dependent(gemm_f8_kernel<EPI>, grid, THREADS, SMEM, stream, tmA, tmB, args);
}

}  // namespace

cudaError_t launch_gemm_f8(int epi, const CUtensorMap& tmA, const CUtensorMap& tmB,
                           const F8GemmArgs& args, int sms, cudaStream_t stream) {
  const int tn = epi >= F8_SWIGLU ? BN / 2 : BN;
  const long long most = ((args.M + BM - 1) / BM + (args.group_off ? args.groups : 0)) *
                         static_cast<long long>((args.N + tn - 1) / tn);
  if (most > 0x7fffffffLL || args.groups > F8_MAX_GROUPS) return cudaErrorInvalidValue;
  if (most <= 0) return cudaSuccess;
  const int grid = static_cast<int>(most < sms ? most : sms);
  switch (epi) {
    case F8_STORE: return launch<F8_STORE>(tmA, tmB, args, grid, stream);
    case F8_RESID: return launch<F8_RESID>(tmA, tmB, args, grid, stream);
    case F8_SWIGLU: return launch<F8_SWIGLU>(tmA, tmB, args, grid, stream);
    case F8_SWIGLU8: return launch<F8_SWIGLU8>(tmA, tmB, args, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t take_gemm_f8_status(uint32_t* bits, cudaStream_t stream) {
  void* at = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&at, g_taken);
  if (e != cudaSuccess) return e;
  take_status_kernel<<<1, 1, 0, stream>>>();
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyAsync(bits, at, 4, cudaMemcpyDeviceToHost, stream);
  return e == cudaSuccess ? cudaStreamSynchronize(stream) : e;
}

}  // namespace nf
