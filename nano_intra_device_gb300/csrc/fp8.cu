// C ABI of the 8-bit operators: argument checks, tensor maps, launches.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "../../include/nanoflow.h"
#include "by_device.h"
#include "fp8.h"
#include "fp8_choice.h"
#include "internal.h"
#include "kernels.h"

namespace {

std::atomic<int64_t> g_timeout_ns{2000000000};  // nf_fp8_set_timeout

nf_status fail8(nf_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return nf::set_last_error(s, buf);
}

#define NF_CUDA8(call)                                                                   \
  do {                                                                                   \
    cudaError_t e_ = (call);                                                             \
    if (e_ != cudaSuccess)                                                               \
      return fail8(NF_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_));         \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// What nf_fp8_poll goes by.  A wait that gives up raises a flag of its device, a poll that finds
// it counts it, and a host thread is told when the counts differ from what it saw last: no
// thread's poll takes a report away from another's.  A thread that begins with a product
// starts from the counts of the last poll by then: its own flags are counted later.
struct Flags {
  uint32_t tiles = 0, rows = 0;  // by the two product kernels
  bool begun = false;            // (of a thread) holds what the thread starts from
};
std::mutex g_mu;                         // of the counting as well
Flags g_counted[nf::MAX_DEVICES];        // under g_mu: as of the last poll
thread_local Flags t_seen[nf::MAX_DEVICES];  // what this thread was told of

void begin_products(int dev) {
  if (t_seen[dev].begun) return;
  std::lock_guard<std::mutex> lk(g_mu);
  t_seen[dev] = g_counted[dev];
  t_seen[dev].begun = true;
}

// The current device, for a section that keeps something by device.
nf_status device_number(int* dev) {
  NF_CUDA8(cudaGetDevice(dev));
  return *dev < nf::MAX_DEVICES ? NF_OK : fail8(NF_ERR_UNSUPPORTED, "device %d: %d are counted", *dev, nf::MAX_DEVICES);
}

// SM count of the current device (a cached attribute query).
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

nf_status check_rows(int32_t rows, int32_t cols, const char* what) {
  if (rows < 0) return fail8(NF_ERR_INVALID_ARG, "rows must not be negative (got %d)", rows);
  if (cols < 16 || cols % 16 || cols > nf::F8_MAX_COLS)
    return fail8(NF_ERR_INVALID_ARG, "%s must be a multiple of 16 in [16, %d] (got %d)", what,
                 nf::F8_MAX_COLS, cols);
  return NF_OK;
}

// The product's checks, for one matrix (group_off NULL, groups 1) or by groups.
nf_status gemm8(const void* A, const float* a_s, const void* B, const float* b_s,
                const int32_t* group_off, int32_t groups, void* C, float* c_s, const void* R,
                int32_t M, int32_t N, int32_t K, int32_t epilogue, int32_t max_sms, void* stream) {
  if (epilogue < NF_EPI_STORE || epilogue > NF_EPI_SWIGLU_FP8)
    return fail8(NF_ERR_INVALID_ARG, "unknown epilogue %d", epilogue);
  const bool eight = epilogue == NF_EPI_SWIGLU_FP8;
  const bool two = epilogue == NF_EPI_SWIGLU || eight;
  if (M < 0) return fail8(NF_ERR_INVALID_ARG, "M must not be negative (got %d)", M);
  if (K < 16 || K % 16) return fail8(NF_ERR_INVALID_ARG, "K must be a positive multiple of 16 (got %d)", K);
  if (N < 8 || N % (eight ? 16 : 8))
    return fail8(NF_ERR_INVALID_ARG, "N must be a positive multiple of %d (got %d)", eight ? 16 : 8, N);
  if (max_sms < 0) return fail8(NF_ERR_INVALID_ARG, "max_sms must not be negative (got %d)", max_sms);
  if (static_cast<int64_t>(groups) * N * (two ? 2 : 1) > 0x7fffffffLL - 256 || M > 0x7fffffff - 256 ||
      K > 0x7fffffff - 256)
    return fail8(NF_ERR_INVALID_ARG, "rows of A or B, or K, pass the 32-bit range");
  if (M == 0) return NF_OK;
  if (!A || !a_s || !B || !b_s || !C || (eight && !c_s) || (epilogue == NF_EPI_RESID && !R))
    return fail8(NF_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16) || (R && !aligned(R, 16)))
    return fail8(NF_ERR_INVALID_ARG, "matrices must be 16-byte aligned");
  if (!aligned(a_s, 4) || !aligned(b_s, 4) || (c_s && !aligned(c_s, 4)) || !aligned(group_off, 4))
    return fail8(NF_ERR_INVALID_ARG, "scales and offsets must be 4-byte aligned");
  const int sms = sm_count();
  if (sms <= 0) return fail8(NF_ERR_CUDA, "no CUDA device");
  int dev = 0;
  if (nf_status e = device_number(&dev)) return e;
  begin_products(dev);
  const bool capped = max_sms > 0 && max_sms < sms;
  const bool few = !capped && nf::few_rows(M, N, K, groups, two, sms);
  nf::F8RowsChoice c{};
  if (few) NF_CUDA8(nf::gemm_f8_wrows_choice(epilogue, M, N, K, groups, &c));
  CUtensorMap ta, tb;
  if (!nf::make_tmap_8bit(&ta, A, M, K, few ? c.tok : 128) ||
      !nf::make_tmap_8bit(&tb, B, static_cast<uint64_t>(groups) * N * (two ? 2 : 1), K,
                          two && !few ? 64 : 128))
    return fail8(NF_ERR_CUDA, "tensor map creation failed");
  nf::F8GemmArgs g{};
  g.M = M;
  g.N = N;
  g.K = K;
  g.a_s = a_s;
  g.b_s = b_s;
  g.group_off = group_off;
  g.groups = groups;
  g.C = eight ? nullptr : static_cast<__nv_bfloat16*>(C);
  g.R = static_cast<const __nv_bfloat16*>(R);
  g.q = eight ? static_cast<uint8_t*>(C) : nullptr;
  g.c_s = c_s;
  g.timeout_ns = static_cast<unsigned long long>(g_timeout_ns.load(std::memory_order_relaxed));
  if (few) {
    g.splits = c.splits;
    NF_CUDA8(nf::launch_gemm_f8_wrows(epilogue, c.tok, tb, ta, g, c.units, static_cast<cudaStream_t>(stream)));
  } else {
    NF_CUDA8(nf::launch_gemm_f8(epilogue, ta, tb, g, capped ? max_sms : sms, static_cast<cudaStream_t>(stream)));
  }
  return NF_OK;
}

}  // namespace

extern "C" {

nf_status nf_rmsnorm_fp8(const void* x, const void* r, const void* g, void* h, void* q, float* s,
                         int32_t rows, int32_t hidden, float eps, void* stream) {
  if (nf_status e = check_rows(rows, hidden, "hidden")) return e;
  if (!(eps >= 0.f)) return fail8(NF_ERR_INVALID_ARG, "eps must not be negative");
  if (rows == 0) return NF_OK;
  if (!x || !g || !q || !s) return fail8(NF_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(x, 16) || !aligned(r, 16) || !aligned(g, 16) || !aligned(h, 16) || !aligned(q, 16) || !aligned(s, 4))
    return fail8(NF_ERR_INVALID_ARG, "x, r, g, h and q must be 16-byte, s 4-byte aligned");
  if (h && !r) return fail8(NF_ERR_INVALID_ARG, "h without a residual r would be a copy of x");
  nf::F8RowsArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.r = static_cast<const __nv_bfloat16*>(r);
  a.g = static_cast<const __nv_bfloat16*>(g);
  a.h = static_cast<__nv_bfloat16*>(h);
  a.src_rows = a.rows = rows;
  a.cols = hidden;
  a.eps = eps;
  a.q = static_cast<uint8_t*>(q);
  a.s = s;
  NF_CUDA8(nf::launch_f8_rows(a, sm_count(), static_cast<cudaStream_t>(stream)));
  return NF_OK;
}

nf_status nf_quant_fp8(const void* x, int32_t src_rows, const int32_t* index, void* q, float* s,
                       int32_t rows, int32_t cols, void* stream) {
  if (nf_status e = check_rows(rows, cols, "cols")) return e;
  if (src_rows < 0) return fail8(NF_ERR_INVALID_ARG, "src_rows must not be negative (got %d)", src_rows);
  if (rows == 0) return NF_OK;
  if (!index && src_rows != rows)
    return fail8(NF_ERR_INVALID_ARG, "without an index, src_rows (%d) must be rows (%d)", src_rows, rows);
  if ((!x && src_rows) || !q || !s) return fail8(NF_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(x, 16) || !aligned(index, 4) || !aligned(q, 16) || !aligned(s, 4))
    return fail8(NF_ERR_INVALID_ARG, "x and q must be 16-byte, index and s 4-byte aligned");
  nf::F8RowsArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.index = index;
  a.src_rows = src_rows;
  a.rows = rows;
  a.cols = cols;
  a.q = static_cast<uint8_t*>(q);
  a.s = s;
  NF_CUDA8(nf::launch_f8_rows(a, sm_count(), static_cast<cudaStream_t>(stream)));
  return NF_OK;
}

nf_status nf_quant_fp8_weights(const void* w, void* q, float* s, int32_t mats, int32_t rows,
                               int32_t cols, void* stream) {
  if (mats < 0 || rows < 1) return fail8(NF_ERR_INVALID_ARG, "need mats >= 0 and rows >= 1");
  if (cols < 16 || cols % 16) return fail8(NF_ERR_INVALID_ARG, "cols must be a positive multiple of 16 (got %d)", cols);
  if (rows > 0x7fffffff - 256 || cols > 0x7fffffff - 256 ||
      static_cast<double>(mats) * ((rows + 127) / 128) * ((cols + 127) / 128) > 2147483647.0)
    return fail8(NF_ERR_INVALID_ARG, "more than 2^31 blocks");
  if (mats == 0) return NF_OK;
  if (!w || !q || !s) return fail8(NF_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(s, 4))
    return fail8(NF_ERR_INVALID_ARG, "w and q must be 16-byte, s 4-byte aligned");
  NF_CUDA8(nf::launch_f8_weights(static_cast<const __nv_bfloat16*>(w), static_cast<uint8_t*>(q), s, mats,
                                 rows, cols, static_cast<cudaStream_t>(stream)));
  return NF_OK;
}

nf_status nf_gemm_fp8(const void* A, const float* a_s, const void* B, const float* b_s, void* C,
                      float* c_s, const void* R, int32_t M, int32_t N, int32_t K, int32_t epilogue,
                      int32_t max_sms, void* stream) {
  return gemm8(A, a_s, B, b_s, nullptr, 1, C, c_s, R, M, N, K, epilogue, max_sms, stream);
}

nf_status nf_gemm_fp8_grouped(const void* A, const float* a_s, const void* B, const float* b_s,
                              const int32_t* group_off, int32_t groups, void* C, float* c_s,
                              int32_t M, int32_t N, int32_t K, int32_t epilogue, int32_t max_sms,
                              void* stream) {
  if (groups < 1 || groups > nf::F8_MAX_GROUPS)
    return fail8(NF_ERR_INVALID_ARG, "groups must lie in [1, %d] (got %d)", nf::F8_MAX_GROUPS, groups);
  if (epilogue == NF_EPI_RESID) return fail8(NF_ERR_INVALID_ARG, "the grouped product has no residual epilogue");
  if (M > 0 && !group_off) return fail8(NF_ERR_INVALID_ARG, "NULL argument");
  return gemm8(A, a_s, B, b_s, group_off, groups, C, c_s, nullptr, M, N, K, epilogue, max_sms, stream);
}

nf_status nf_fp8_set_timeout(int64_t timeout_ns) {
  if (timeout_ns < 1 || timeout_ns > 10000000000LL)
    return fail8(NF_ERR_INVALID_ARG, "timeout_ns must lie in [1, 1e10]");
  g_timeout_ns.store(timeout_ns, std::memory_order_relaxed);
  return NF_OK;
}

nf_status nf_fp8_poll(void* stream) {
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0;
  if (nf_status e = device_number(&dev)) return e;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  NF_CUDA8(cudaStreamIsCapturing(st, &capture));
  if (capture != cudaStreamCaptureStatusNone)
    return fail8(NF_ERR_INVALID_ARG, "the stream is being captured: a poll waits for it");
  NF_CUDA8(cudaStreamSynchronize(st));  // (polls do not wait for one another's streams)
  std::lock_guard<std::mutex> lk(g_mu);
  Flags now;
  NF_CUDA8(nf::count_gemm_f8_flags(&now.tiles, st));
  NF_CUDA8(nf::count_gemm_f8_wrows_flags(&now.rows, st));
  NF_CUDA8(cudaStreamSynchronize(st));
  now.begun = true;
  const bool more = now.tiles != t_seen[dev].tiles || now.rows != t_seen[dev].rows;
  t_seen[dev] = g_counted[dev] = now;
  if (!more) return NF_OK;
  return fail8(NF_ERR_TIMEOUT, "nf_gemm_fp8: a device-side wait timed out");
}

}  // extern "C"
