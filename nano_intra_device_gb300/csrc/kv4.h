// Launch interface between the 4-bit KV cache's C ABI (kv4.cu) and its kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace nf {

constexpr int KV4_P = 16;  // positions of a page

// Bytes of K (or V) of one (page, KV head): 16 rows of codes, then 16 of scales.
__host__ __device__ constexpr int kv4_part_bytes(int head_dim) { return 9 * head_dim; }

struct BlockTableArgs {
  const int* held;
  const int* seq_lens;
  int n_seq;
  int* block_table;
  int max_pages;
  int* ring;
  int num_pages;
  const int* state_in;
  int* state_out;
  int *tok_begin, *tok_seq, *tok_pos, *tok_slot;
  int tok_cap;
};
cudaError_t launch_block_tables(const BlockTableArgs& a, int num_sms, cudaStream_t stream);

// freq[i] = theta^(-2i/d) / 2 pi in units of 2^-64 turns: position * freq[i]
// modulo 2^64 is the angle of any position, exact to the rounding of freq.
struct RopeFreq {
  uint64_t freq[64];
};

struct QkNormRopeArgs {
  const __nv_bfloat16* qkv;
  int64_t ld;
  const __nv_bfloat16 *q_gain, *k_gain;  // NULL: not normed
  const int *tok_pos, *tok_slot;
  int n_tok, n_q, n_kv, head_dim;
  float eps;
  __nv_bfloat16* q;
  int num_pages;
  // 16-bit pools, or the packed pool in k_pool
  void *k_pool, *v_pool;
  int k_exp, v_exp;
};
cudaError_t launch_qk_norm_rope(const QkNormRopeArgs& a, const RopeFreq& f, bool fp4, int num_sms,
                                cudaStream_t stream);

cudaError_t launch_kv4_read(const uint8_t* pool, int num_pages, int n_kv, int head_dim,
                            const int* slots, int n, int k_exp, int v_exp, __nv_bfloat16* k,
                            __nv_bfloat16* v, int num_sms, cudaStream_t stream);

struct Kv4AttnArgs {
  const __nv_bfloat16* q;  // [n_tok, n_q, d]
  __nv_bfloat16* o;
  const uint8_t* pool;
  const int* block_table;
  const int* seq_lens;
  const int* tok_begin;  // NULL: request s owns row s
  int n_seq, n_tok, max_pages, num_pages, n_q, n_kv, head_dim;
  float scale_log2;  // log2(e) / sqrt(d) * 2^k_exp
  float v_scale;     // 2^v_exp
  uint32_t* status;
  unsigned long long timeout_ns;
  // self-test: CTA drop_cta (-1: none) leaves out an arrival for its block drop_block
  // of K (drop_part 0) or V (1), so that what waits for it gives up
  int drop_cta, drop_part;
  uint32_t drop_block;
  int grid;              // CTAs, one an SM
  float* records;        // [grid][2] records of kv4_record_bytes
  int* counters;         // [grid], zero between launches
  // requests of more rows than small_rows are the prefill kernel's
  int small_rows;
  float* tiles;          // [grid][2] records of kv4_tile_record_bytes
  int* tile_counters;    // [grid][2], zero between launches
};
size_t kv4_record_bytes(int head_dim);
size_t kv4_tile_record_bytes(int head_dim);
cudaError_t launch_attention_kv4_prefill(const Kv4AttnArgs& a, cudaStream_t stream);
// behind: the stream's last launch is this call's tiles
cudaError_t launch_attention_kv4(const Kv4AttnArgs& a, bool behind, cudaStream_t stream);

}  // namespace nf
