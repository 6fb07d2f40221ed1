// Internal launch interface of the 8-bit operators and of the query/key norm with rotation (not part
// of the ABI).
#pragma once

#include "internal.h"

namespace moss {

// The current device's error word (allocated on first use, also while a stream is being captured);
// NULL if that fails.
unsigned* device_error_word();

// 8-bit [outer, inner] map (128-byte swizzle) of the 8-bit GEMM's operands.
bool make_tmap_i8_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint32_t box_inner,
                     uint32_t box_outer, std::string* err);

// 8-bit GEMM: c = (sum_k a b) a_scale[m] b_scale[n] + bias[n]; with gate and residual,
// c = residual + gate[n] * that (FP32).  a [M, K], b [N, K]; K a multiple of 16.
constexpr int kMaxI8K = 65536;
struct GemmI8Params {
  int M = 0, N = 0, K = 0;
  const float* a_scale = nullptr;   // [M]
  const float* b_scale = nullptr;   // [N]
  const bf16* bias = nullptr;       // [N] or NULL
  const float* gate = nullptr;      // [N], with residual
  const float* residual = nullptr;  // [M, N], may be c itself
  void* c = nullptr;                // [M, N] FP32 or BF16
  bool c_bf16 = false;
  int selftest = 0;                 // 0, or one of the failures below, in the grid's first CTA
};
enum : int { kI8SelftestFlatLoad = 1, kI8SelftestPairLoad = 2, kI8SelftestPairAccumulator = 3 };
cudaError_t launch_gemm_i8(const int8_t* a, const int8_t* b, const GemmI8Params& p, cudaStream_t s, unsigned* err,
                           std::string* emsg);
// Whether a call of these sizes runs the kernel that this failure is for, far enough to meet it.
bool gemm_i8_selftest_reaches(int kind, int M, int N, int K);

// Rows to 8-bit integers with one scale a row (dim a multiple of 16, at most kMaxRowDim).
constexpr int kMaxRowDim = 32768;
cudaError_t launch_quantize_i8(const void* x, bool is_bf16, int64_t x_stride, int8_t* q, float* scale, int rows,
                               int dim, cudaStream_t s);
cudaError_t launch_ln_mod_i8(const float* x, const float* shift, const float* mscale, int8_t* q, float* scale,
                             int rows, int dim, float eps, cudaStream_t s);
cudaError_t launch_swiglu_i8(const bf16* gu, int64_t gu_stride, int8_t* q, float* scale, int rows, int dim,
                             cudaStream_t s);

// Per-head RMSNorm and rotation of the queries and keys.  Strides in elements, between tokens; the
// launcher fills chunks, chunks_q and heads_per_chunk.
struct QkNormRopeParams {
  const void *q = nullptr, *k = nullptr;
  void *q_out = nullptr, *k_out = nullptr;
  int64_t q_stride = 0, k_stride = 0, q_out_stride = 0, k_out_stride = 0;
  const float *q_gain = nullptr, *k_gain = nullptr, *rope = nullptr;
  const int* positions = nullptr;
  int rows = 0, heads_q = 0, heads_k = 0, rot_dim = 0, n_pos = 0;
  float eps = 0.f;
  int heads_per_chunk = 0, chunks_q = 0, chunks = 0;
};
cudaError_t launch_qk_norm_rope(const QkNormRopeParams& p, int head_dim, bool halves, bool in_bf16, bool out_bf16,
                                cudaStream_t s, unsigned* err);

// The angles of launch_rope_table token by token: table[token * 64 + pair].
cudaError_t launch_rope_table_tokens(float2* table, int grid_h, int grid_w, int n_txt, cudaStream_t s);

}  // namespace moss
