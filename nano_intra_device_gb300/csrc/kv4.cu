// C ABI of the 4-bit KV cache: argument checks, the attention handle, launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <new>

#include "../../include/nanoflow.h"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "kv4.h"

struct nf_kv4_s {
  nf_model_shape shape{};
  int num_pages = 0, max_pages = 0, device = 0, num_sms = 0;
  // one allocation: status word and the copy that a poll takes of it (256 bytes),
  // arrival counters, split records of the two kernels
  uint32_t* status = nullptr;
  int *counters = nullptr, *tile_counters = nullptr;
  float *records = nullptr, *tiles = nullptr;
  size_t counted = 0;  // bytes of the arrival counters, which a launch expects to be zero
  int64_t timeout_ns = 2000000000;
  int drop_cta = -1, drop_block = 0, drop_part = 0;
};

namespace {

nf_status fail4(nf_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return nf::set_last_error(s, buf);
}

#define NF_CUDA4(call)                                                                   \
  do {                                                                                   \
    cudaError_t e_ = (call);                                                             \
    if (e_ != cudaSuccess)                                                               \
      return fail4(NF_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_));         \
  } while (0)
#define NF_TRY4(expr)             \
  do {                            \
    nf_status s_ = (expr);        \
    if (s_ != NF_OK) return s_;   \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// SM count of the current device (a cached attribute query).
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// Zeros in device memory once this returns.  A memset on the default stream would
// neither be complete nor come before a call on a non-blocking stream, and would
// wait for whatever the default stream has to do.
cudaError_t zero_now(void* p, size_t bytes) {
  cudaStream_t s = nullptr;
  cudaError_t e = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(p, 0, bytes, s);
  const cudaError_t w = cudaStreamSynchronize(s);
  cudaStreamDestroy(s);
  return e != cudaSuccess ? e : w;
}

// status[1] = status[0], which becomes zero, in one step: a bit that a running call
// raises meanwhile is taken or stays.
__global__ void take_status_kernel(uint32_t* status) { status[1] = atomicExch(status, 0u); }

// The fields of a shape that the cache's operators use.
nf_status check_heads(const nf_model_shape* s) {
  if (!s) return fail4(NF_ERR_INVALID_ARG, "shape is NULL");
  if (s->head_dim != 64 && s->head_dim != 128)
    return fail4(NF_ERR_INVALID_ARG, "head_dim must be 64 or 128 (got %d)", s->head_dim);
  if (s->n_kv_heads <= 0 || s->n_kv_heads > 1024 || s->n_q_heads <= 0 || s->n_q_heads % s->n_kv_heads)
    return fail4(NF_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads (at most 1024)");
  const int grp = s->n_q_heads / s->n_kv_heads;
  if (grp != 1 && grp != 2 && grp != 4 && grp != 8)
    return fail4(NF_ERR_INVALID_ARG, "n_q_heads / n_kv_heads must be 1, 2, 4 or 8 (got %d)", grp);
  if (s->page_size != 16)
    return fail4(NF_ERR_INVALID_ARG, "page_size must be 16 (got %d)", s->page_size);
  return NF_OK;
}

// Slots and pool rows are 32-bit: num_pages * 16 below 2^31.
constexpr int kMaxPages = (1 << 27) - 1;
// Pages of a request in attention: the kernels count positions in 32 bits, past a
// request's last one by up to two key blocks, so the last 2^30 are left out.
constexpr int kMaxSeqPages = 1 << 26;

nf_status check_cache(const nf_kv_cache* c, bool fp4_only) {
  if (!c) return fail4(NF_ERR_INVALID_ARG, "cache is NULL");
  if (c->format != NF_KV_BF16 && c->format != NF_KV_FP4)
    return fail4(NF_ERR_INVALID_ARG, "unknown cache format %d", c->format);
  if (fp4_only && c->format != NF_KV_FP4)
    return fail4(NF_ERR_INVALID_ARG, "the cache must be NF_KV_FP4");
  if (c->num_pages < 1 || c->num_pages > kMaxPages)
    return fail4(NF_ERR_INVALID_ARG, "num_pages must lie in [1, %d] (got %d)", kMaxPages, c->num_pages);
  if (!c->k || (c->format == NF_KV_BF16 && !c->v))
    return fail4(NF_ERR_INVALID_ARG, "a cache pool is NULL");
  if (!aligned(c->k, 16) || (c->v && !aligned(c->v, 16)))
    return fail4(NF_ERR_INVALID_ARG, "pools must be 16-byte aligned");
  if (c->format == NF_KV_FP4) {
    if (c->v) return fail4(NF_ERR_INVALID_ARG, "an NF_KV_FP4 cache holds K and V in one pool: v must be NULL");
    if (c->k_exp < -64 || c->k_exp > 64 || c->v_exp < -64 || c->v_exp > 64)
      return fail4(NF_ERR_INVALID_ARG, "k_exp and v_exp must lie in [-64, 64]");
  }
  return NF_OK;
}

// A request of at most this many query vectors a KV head (rows * n_q / n_kv) goes
// to the kernel of few rows, which reads its cache once for 8 of them; a longer
// one to the tiles of 128, whose time hardly depends on how full they are.
// Measured, few rows against tiles, 32 query and 8 KV heads of 128, 16 requests
// of 2000 positions: 45 / 66 us at 32 vectors, 70 / 64 at 64, 92 / 64 at 96; 128
// requests of 500: 78 / 177, 129 / 182, 178 / 184.  With 8 query heads 70 / 66 at
// 64, with 64 heads 68 / 64 at 64 and 93 / 62 at 96.
constexpr int kSmallVecs = 64;
// The tiles' fixed cost is higher: a second launch, and a short unit is cut into
// pieces of one block, up to about 16, which one CTA joins one after the other.  One
// request of 32 rows and 4 heads a KV head, tiles / few rows, in a graph: over 100
// positions (one block, no join) 20.6 / 12.2 us, 500: 22.2 / 18.2, 2000: 32.7 / 19.9,
// 8000: 41.1 / 36.9; by single calls 32,000: 68 / 113.  So where the kernel of few
// rows can at most visit this many (page, KV head, 8 vectors) an SM, every request
// goes there.  The lengths are on the device, so the bound takes every request to be
// as long as the handle allows: a handle much wider than its requests sends chunks
// past kSmallVecs to the tiles however short they are (the 32 rows over 2000
// positions: 20 us in a handle of 512 pages a request, 33 in one of 40,000).
constexpr int kFewVisits = 500;

// Frequencies of (theta, head_dim), computed once for each pair in use: 64
// powl calls cost more than the launch.
const nf::RopeFreq* rope_freq(float theta, int d) {
  struct Entry {
    float theta = 0;
    int d = 0;
    nf::RopeFreq f;
  };
  thread_local Entry cache[4];
  thread_local int next = 0;
  for (Entry& e : cache)
    if (e.d == d && e.theta == theta) return &e.f;
  Entry& e = cache[next];
  next = (next + 1) % 4;
  e.theta = theta;
  e.d = d;
  const long double two64 = 18446744073709551616.0L, tau = 6.283185307179586476925286766559005768L;
  for (int i = 0; i < 64; ++i) {
    long double f = 0;
    if (i < d / 2) f = std::pow((long double)theta, -2.0L * i / d) / tau;
    f -= std::floor(f);  // whole turns do not matter (theta < 1)
    e.f.freq[i] = f * two64 >= two64 ? 0 : (uint64_t)(f * two64);
  }
  return &e.f;
}

}  // namespace

nf_status nf_kv4_pool_bytes(const nf_model_shape* shape, int32_t num_pages, size_t* bytes) {
  NF_TRY4(check_heads(shape));
  if (!bytes) return fail4(NF_ERR_INVALID_ARG, "bytes is NULL");
  if (num_pages < 1 || num_pages > kMaxPages)
    return fail4(NF_ERR_INVALID_ARG, "num_pages must lie in [1, %d] (got %d)", kMaxPages, num_pages);
  *bytes = (size_t)num_pages * shape->n_kv_heads * 2 * nf::kv4_part_bytes(shape->head_dim);
  return NF_OK;
}

nf_status nf_block_tables(const int32_t* held, const int32_t* seq_lens, int32_t n_seq,
                          int32_t* block_table, int32_t max_pages, int32_t* ring,
                          int32_t num_pages, const int32_t* state_in, int32_t* state_out,
                          int32_t* tok_begin, int32_t* tok_seq, int32_t* tok_pos,
                          int32_t* tok_slot, int32_t tok_cap, void* stream) {
  if (n_seq < 1) return fail4(NF_ERR_INVALID_ARG, "n_seq must be >= 1 (got %d)", n_seq);
  if (max_pages < 1 || max_pages > kMaxPages || num_pages < 1 || num_pages > kMaxPages)
    return fail4(NF_ERR_INVALID_ARG, "max_pages and num_pages must lie in [1, %d]", kMaxPages);
  if (tok_cap < 0) return fail4(NF_ERR_INVALID_ARG, "tok_cap must be >= 0 (got %d)", tok_cap);
  if (!held || !seq_lens || !block_table || !ring || !state_in || !state_out || !tok_begin ||
      (tok_cap > 0 && (!tok_seq || !tok_pos || !tok_slot)))
    return fail4(NF_ERR_INVALID_ARG, "NULL argument");
  if (state_in < state_out + 4 && state_out < state_in + 2)
    return fail4(NF_ERR_INVALID_ARG, "state_in and state_out overlap");
  const int sms = sm_count();
  if (sms <= 0) return fail4(NF_ERR_CUDA, "no CUDA device");
  nf::BlockTableArgs a{held,     seq_lens,  n_seq,   block_table, max_pages, ring,    num_pages,
                       state_in, state_out, tok_begin, tok_seq,   tok_pos,   tok_slot, tok_cap};
  NF_CUDA4(nf::launch_block_tables(a, sms, static_cast<cudaStream_t>(stream)));
  return NF_OK;
}

nf_status nf_qk_norm_rope(const nf_model_shape* shape, const void* qkv, int32_t ld,
                          const void* q_gain, const void* k_gain, const int32_t* tok_pos,
                          const int32_t* tok_slot, int32_t n_tok, void* q,
                          const nf_kv_cache* cache, void* stream) {
  NF_TRY4(check_heads(shape));
  NF_TRY4(check_cache(cache, false));
  if (!(shape->rms_eps >= 0.f) || !(shape->rope_theta > 0.f) || !std::isfinite(shape->rope_theta))
    return fail4(NF_ERR_INVALID_ARG, "rms_eps must be >= 0 and rope_theta positive");
  if (n_tok < 0) return fail4(NF_ERR_INVALID_ARG, "n_tok must be >= 0 (got %d)", n_tok);
  if (n_tok == 0) return NF_OK;
  if (!qkv || !tok_pos || !tok_slot || !q) return fail4(NF_ERR_INVALID_ARG, "NULL argument");
  const int width = (shape->n_q_heads + 2 * shape->n_kv_heads) * shape->head_dim;
  if (ld < width || ld % 8)
    return fail4(NF_ERR_INVALID_ARG, "ld must be a multiple of 8 and at least %d (got %d)", width, ld);
  if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(q_gain, 16) || !aligned(k_gain, 16))
    return fail4(NF_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  const int sms = sm_count();
  if (sms <= 0) return fail4(NF_ERR_CUDA, "no CUDA device");
  nf::QkNormRopeArgs a{};
  a.qkv = static_cast<const __nv_bfloat16*>(qkv);
  a.ld = ld;
  a.q_gain = static_cast<const __nv_bfloat16*>(q_gain);
  a.k_gain = static_cast<const __nv_bfloat16*>(k_gain);
  a.tok_pos = tok_pos;
  a.tok_slot = tok_slot;
  a.n_tok = n_tok;
  a.n_q = shape->n_q_heads;
  a.n_kv = shape->n_kv_heads;
  a.head_dim = shape->head_dim;
  a.eps = shape->rms_eps;
  a.q = static_cast<__nv_bfloat16*>(q);
  a.num_pages = cache->num_pages;
  a.k_pool = cache->k;
  a.v_pool = cache->v;
  a.k_exp = cache->k_exp;
  a.v_exp = cache->v_exp;
  NF_CUDA4(nf::launch_qk_norm_rope(a, *rope_freq(shape->rope_theta, shape->head_dim),
                                   cache->format == NF_KV_FP4, sms,
                                   static_cast<cudaStream_t>(stream)));
  return NF_OK;
}

nf_status nf_kv4_read(const nf_model_shape* shape, const nf_kv_cache* cache, const int32_t* slots,
                      int32_t n, void* k, void* v, void* stream) {
  NF_TRY4(check_heads(shape));
  NF_TRY4(check_cache(cache, true));
  if (n < 0) return fail4(NF_ERR_INVALID_ARG, "n must be >= 0 (got %d)", n);
  if (n == 0) return NF_OK;
  if (!slots || !k || !v) return fail4(NF_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(k, 16) || !aligned(v, 16))
    return fail4(NF_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  const int sms = sm_count();
  if (sms <= 0) return fail4(NF_ERR_CUDA, "no CUDA device");
  NF_CUDA4(nf::launch_kv4_read(static_cast<const uint8_t*>(cache->k), cache->num_pages,
                               shape->n_kv_heads, shape->head_dim, slots, n, cache->k_exp,
                               cache->v_exp, static_cast<__nv_bfloat16*>(k),
                               static_cast<__nv_bfloat16*>(v), sms,
                               static_cast<cudaStream_t>(stream)));
  return NF_OK;
}

nf_status nf_kv4_create(const nf_model_shape* shape, int32_t num_pages, int32_t max_pages_per_seq,
                        nf_kv4* out) {
  if (!out) return fail4(NF_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  NF_TRY4(check_heads(shape));
  if (num_pages < 1 || num_pages > kMaxPages)
    return fail4(NF_ERR_INVALID_ARG, "num_pages must lie in [1, %d] (got %d)", kMaxPages, num_pages);
  if (max_pages_per_seq < 1 || max_pages_per_seq > kMaxSeqPages)
    return fail4(NF_ERR_INVALID_ARG, "max_pages_per_seq must lie in [1, %d] (got %d)", kMaxSeqPages, max_pages_per_seq);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return fail4(NF_ERR_CUDA, "no CUDA device");
  }
  const int sms = sm_count();
  if (sms <= 0) return fail4(NF_ERR_CUDA, "no CUDA device");
  nf_kv4 h = new (std::nothrow) nf_kv4_s();
  if (!h) return fail4(NF_ERR_OOM, "out of host memory");
  h->shape = *shape;
  h->num_pages = num_pages;
  h->max_pages = max_pages_per_seq;
  h->device = dev;
  h->num_sms = sms;
  const size_t cnt = ((size_t)sms * 8 + 255) / 256 * 256;
  const size_t rec = ((size_t)sms * 2 * nf::kv4_record_bytes(shape->head_dim) + 255) / 256 * 256;
  const size_t tiles = (size_t)sms * 2 * nf::kv4_tile_record_bytes(shape->head_dim);
  h->counted = 2 * cnt;
  if (cudaMalloc(&h->status, 256 + h->counted + rec + tiles) != cudaSuccess ||
      zero_now(h->status, 256 + h->counted) != cudaSuccess) {
    cudaGetLastError();
    nf_kv4_destroy(h);
    return fail4(NF_ERR_OOM, "cudaMalloc of the workspace failed");
  }
  char* at = reinterpret_cast<char*>(h->status) + 256;
  h->counters = reinterpret_cast<int*>(at);
  h->tile_counters = reinterpret_cast<int*>(at + cnt);
  h->records = reinterpret_cast<float*>(at + 2 * cnt);
  h->tiles = reinterpret_cast<float*>(at + 2 * cnt + rec);
  *out = h;
  return NF_OK;
}

void nf_kv4_destroy(nf_kv4 h) {
  if (!h) return;
  if (h->status) cudaFree(h->status);
  delete h;
}

nf_status nf_kv4_poll(nf_kv4 h, int wait) {
  if (!h) return fail4(NF_ERR_INVALID_ARG, "handle is NULL");
  int dev = -1;
  NF_CUDA4(cudaGetDevice(&dev));
  if (dev != h->device)
    return fail4(NF_ERR_INVALID_ARG, "the handle belongs to device %d, the current one is %d", h->device, dev);
  if (wait) NF_CUDA4(cudaDeviceSynchronize());
  NF_CUDA4(cudaGetLastError());
  uint32_t st = 0;
  take_status_kernel<<<1, 1>>>(h->status);
  NF_CUDA4(cudaGetLastError());
  NF_CUDA4(cudaMemcpy(&st, h->status + 1, 4, cudaMemcpyDeviceToHost));
  if (st & nf::ST_TIMEOUT) {
    // pieces that were given up never arrived: the counters start over
    NF_CUDA4(cudaDeviceSynchronize());
    NF_CUDA4(zero_now(h->counters, h->counted));
    return fail4(NF_ERR_TIMEOUT, "a device wait timed out (status 0x%x)", st);
  }
  if (st)
    return fail4(NF_ERR_DEVICE, "device-side check failed (status 0x%x: %s%s%s)", st,
                 (st & nf::ST_BAD_PAGE) ? "page id out of range " : "",
                 (st & nf::ST_BAD_LEN) ? "bad sequence length or rows " : "",
                 (st & nf::ST_OVERFLOW) ? "too many pages for a call" : "");
  return NF_OK;
}

nf_status nf_kv4_set_timeout(nf_kv4 h, int64_t timeout_ns) {
  if (!h) return fail4(NF_ERR_INVALID_ARG, "handle is NULL");
  if (timeout_ns < 1 || timeout_ns > 10000000000LL)
    return fail4(NF_ERR_INVALID_ARG, "timeout_ns must lie in [1, 1e10]");
  h->timeout_ns = timeout_ns;
  return NF_OK;
}

nf_status nf_kv4_selftest_drop(nf_kv4 h, int32_t cta, int32_t part, int32_t block) {
  if (!h) return fail4(NF_ERR_INVALID_ARG, "handle is NULL");
  if (cta >= h->num_sms || (cta >= 0 && (part < 0 || part > 1 || block < 0)))
    return fail4(NF_ERR_INVALID_ARG, "cta must be below %d, part 0 or 1, block >= 0", h->num_sms);
  h->drop_cta = cta < 0 ? -1 : cta;
  h->drop_part = part;
  h->drop_block = block;
  return NF_OK;
}

nf_status nf_attention_kv4(nf_kv4 h, const void* q, const nf_kv_cache* cache,
                           const int32_t* block_table, const int32_t* seq_lens,
                           const int32_t* tok_begin, int32_t n_seq, int32_t n_tok, void* o,
                           void* stream) {
  if (!h) return fail4(NF_ERR_INVALID_ARG, "handle is NULL");
  NF_TRY4(check_cache(cache, true));
  if (n_seq < 0 || n_tok < 0) return fail4(NF_ERR_INVALID_ARG, "n_seq and n_tok must be >= 0");
  if (!tok_begin && n_tok != n_seq)
    return fail4(NF_ERR_INVALID_ARG, "without tok_begin n_tok must be n_seq (got %d and %d)", n_tok, n_seq);
  if (cache->num_pages != h->num_pages)
    return fail4(NF_ERR_INVALID_ARG, "the handle was made for %d pages, the cache has %d", h->num_pages,
                 cache->num_pages);
  if (n_seq == 0 || n_tok == 0) return NF_OK;
  if (!q || !block_table || !seq_lens || !o) return fail4(NF_ERR_INVALID_ARG, "NULL argument");
  if (!aligned(q, 16) || !aligned(o, 16))
    return fail4(NF_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  int dev = -1;
  NF_CUDA4(cudaGetDevice(&dev));
  if (dev != h->device)
    return fail4(NF_ERR_INVALID_ARG, "the handle belongs to device %d, the current one is %d", h->device, dev);
  nf::Kv4AttnArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.pool = static_cast<const uint8_t*>(cache->k);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.tok_begin = tok_begin;
  a.n_seq = n_seq;
  a.n_tok = n_tok;
  a.max_pages = h->max_pages;
  a.num_pages = h->num_pages;
  a.n_q = h->shape.n_q_heads;
  a.n_kv = h->shape.n_kv_heads;
  a.head_dim = h->shape.head_dim;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)a.head_dim) * std::ldexp(1.0, cache->k_exp));
  a.v_scale = nf::exp2_int(cache->v_exp);
  a.status = h->status;
  a.timeout_ns = static_cast<unsigned long long>(h->timeout_ns);
  a.drop_cta = h->drop_cta;
  a.drop_part = h->drop_part;
  a.drop_block = static_cast<uint32_t>(h->drop_block);
  a.grid = h->num_sms;
  a.records = h->records;
  a.counters = h->counters;
  a.tiles = h->tiles;
  a.tile_counters = h->tile_counters;
  const double visits = (double)n_tok * a.n_q / 8 * a.max_pages;
  a.small_rows = visits <= (double)kFewVisits * h->num_sms ? n_tok : kSmallVecs / (a.n_q / a.n_kv);
  const bool tiles = tok_begin && n_tok > a.small_rows;
  if (tiles) NF_CUDA4(nf::launch_attention_kv4_prefill(a, static_cast<cudaStream_t>(stream)));
  NF_CUDA4(nf::launch_attention_kv4(a, tiles, static_cast<cudaStream_t>(stream)));
  return NF_OK;
}
