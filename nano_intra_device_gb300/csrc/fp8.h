// Launch interface between the C ABI of the 8-bit operators (fp8.cu) and their kernels.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace nf {

constexpr int F8_BLOCK = 128;        // columns (and, for weights, rows) of a scale's block
constexpr int F8_MAX_GROUPS = 128;   // groups of rows of one product
// After a wait gave up: the limit of the waits for what is in flight already (loads,
// products), which takes microseconds, whatever the call's own limit is.
constexpr unsigned long long F8_DRAIN_NS = 20000000ULL;
// Columns of a row that one CTA norms, in registers.  Rows quantised without a norm are held
// to the same limit, though their kernel would take more.
constexpr int F8_MAX_COLS = 32768;

enum { F8_STORE = 0, F8_RESID = 1, F8_SWIGLU = 2, F8_SWIGLU8 = 3 };

// Rows to 8 bits: out row i is that of x row index[i] (NULL: i), an index outside
// [0, src_rows) a row of zeros.  g != NULL: RMSNorm first, of x + r (r NULL: x);
// h != NULL receives x + r.
struct F8RowsArgs {
  const __nv_bfloat16 *x, *r, *g;
  __nv_bfloat16* h;
  const int* index;
  int src_rows, rows, cols;
  float eps;
  uint8_t* q;
  float* s;  // [ceil(cols / 128)][rows]
};
cudaError_t launch_f8_rows(const F8RowsArgs& a, int sms, cudaStream_t stream);

// mats matrices [rows, cols] to 8 bits in 128 x 128 blocks, scales [mats][row block][column block].
cudaError_t launch_f8_weights(const __nv_bfloat16* w, uint8_t* q, float* s, int mats, int rows,
                              int cols, cudaStream_t stream);

struct F8GemmArgs {
  int M, N, K;           // N: output columns (the features for SwiGLU)
  const float* a_s;      // [ceil(K / 128)][M]
  const float* b_s;      // [groups][1, SwiGLU: 2][ceil(N / 128)][ceil(K / 128)]
  const int* group_off;  // NULL: one group of all rows; else device [groups + 1]
  int groups;
  __nv_bfloat16* C;      // STORE, RESID, SWIGLU
  const __nv_bfloat16* R;
  uint8_t* q;            // SWIGLU8
  float* c_s;            // SWIGLU8: [ceil(N / 128)][M]
  int splits;            // few rows: CTAs of a cluster, which split K
  unsigned long long timeout_ns;
};
// tmA: the rows of A in boxes of 128 rows, tmB: all groups' rows of B in boxes of 128
// (SwiGLU: 64) rows, x 128 columns.
cudaError_t launch_gemm_f8(int epi, const CUtensorMap& tmA, const CUtensorMap& tmB,
                           const F8GemmArgs& args, int sms, cudaStream_t stream);
// Takes the flag that a wait of the kernels of launch_gemm_f8 raised on the current device,
// and copies to *count, in the stream's order, how many flags were taken since the process
// began.  One call at a time on a device, until the stream has been waited for.
cudaError_t count_gemm_f8_flags(uint32_t* count, cudaStream_t stream);

// The same for few rows: tiles of 128 features x tok rows of A (tmX: the rows of A in
// boxes of tok rows; tok 16, 32, 64 and, but for SwiGLU, 128), `units` clusters of
// args.splits CTAs.
struct F8RowsChoice {
  int tok, splits;
  long long units;
};
cudaError_t gemm_f8_wrows_choice(int epi, int M, int N, int K, int groups, F8RowsChoice* choice);
cudaError_t launch_gemm_f8_wrows(int epi, int tok, const CUtensorMap& tmW, const CUtensorMap& tmX,
                                 const F8GemmArgs& args, long long units, cudaStream_t stream);
cudaError_t count_gemm_f8_wrows_flags(uint32_t* count, cudaStream_t stream);

}  // namespace nf
