// C ABI of the 8-bit linear path and of the query/key norm with rotation (declared in
// include/moss_dit.h): argument checks on the host, then one launch each.
#include <cstdio>
#include <cstring>

#include "../../include/moss_dit.h"
#include "ops_i8.h"

using namespace moss;

static_assert(int{kI8SelftestFlatLoad} == int{MOSS_I8_LOST_LOAD} && int{kI8SelftestPairLoad} == int{MOSS_I8_LOST_LOAD_PAIR} &&
              int{kI8SelftestPairAccumulator} == int{MOSS_I8_KEPT_ACCUMULATOR}, "as the header numbers them");

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int invalid(const char* msg) { return set_error(MOSS_ERR_INVALID_ARGUMENT, msg); }

int cuda_status(cudaError_t e, const char* what, const std::string& detail) {
  if (e == cudaSuccess) return set_error(MOSS_OK, "");
  return set_error(e == cudaErrorMemoryAllocation ? MOSS_ERR_OOM : MOSS_ERR_CUDA,
                   std::string(what) + ": " + (detail.empty() ? cudaGetErrorString(e) : detail));
}

bool known_dtype(int d) { return d == MOSS_DTYPE_F32 || d == MOSS_DTYPE_BF16; }
int64_t dtype_bytes(int d) { return d == MOSS_DTYPE_BF16 ? 2 : 4; }

// A set of `rows` byte ranges [base + r * stride, + width).
struct Span {
  uintptr_t base;
  int64_t width, stride, rows;
  Span(const void* p, int64_t w, int64_t s = 0, int64_t r = 1)
      : base(reinterpret_cast<uintptr_t>(p)), width(w), stride(s), rows(r) {}
  uintptr_t end() const { return base + static_cast<uintptr_t>(stride * (rows - 1) + width); }
};

// Whether two spans share a byte.  Rows of one stride that interleave (columns of one buffer) do not.
bool overlap(const Span& a, const Span& b) {
  if (a.end() <= b.base || b.end() <= a.base) return false;
  if (a.stride != b.stride || a.rows < 2) return true;
  const int64_t d = static_cast<int64_t>((b.base - a.base) % static_cast<uintptr_t>(a.stride));
  const int64_t off = b.base >= a.base ? d : static_cast<int64_t>((a.stride - static_cast<int64_t>((a.base - b.base) % static_cast<uintptr_t>(a.stride))) % a.stride);
  return off < a.width || off + b.width > a.stride;
}

int check_rows_out(const Span& in, int8_t* q, float* scale, int rows, int dim) {
  if (!q || !scale) return invalid("q and scale must not be NULL");
  if (!aligned(q, 16) || !aligned(scale, 4)) return invalid("q must be 16-byte aligned, scale 4-byte aligned");
  const Span sq(q, static_cast<int64_t>(rows) * dim), ss(scale, 4 * static_cast<int64_t>(rows));
  if (overlap(in, sq) || overlap(in, ss) || overlap(sq, ss)) return invalid("the outputs must not overlap the input or each other");
  return MOSS_OK;
}

// Whether `rows` rows `stride` bytes apart lie within an address space (and their offsets within 64 bits).
bool stride_fits(int64_t stride, int64_t rows) { return stride <= (int64_t{1} << 47) / (rows > 0 ? rows : 1); }

const char* kRowsDims = "rows must be >= 0 and dim a positive multiple of 16, at most 32768";
bool rows_dims_ok(int rows, int dim) { return rows >= 0 && dim >= 16 && dim % 16 == 0 && dim <= kMaxRowDim; }

}  // namespace

extern "C" {

int moss_op_quantize_i8(const void* x, int x_dtype, int64_t x_stride, int8_t* q, float* scale, int rows, int dim,
                        void* stream) {
  set_error(MOSS_OK, "");
  if (!known_dtype(x_dtype)) return invalid("x_dtype must be MOSS_DTYPE_F32 or MOSS_DTYPE_BF16");
  if (!rows_dims_ok(rows, dim)) return invalid(kRowsDims);
  const int64_t eb = dtype_bytes(x_dtype);
  if (x_stride < dim || x_stride % (16 / eb)) return invalid("x_stride must be >= dim and a multiple of 16 bytes");
  if (!stride_fits(x_stride, rows)) return invalid("x_stride is too long");
  if (rows == 0) return MOSS_OK;
  if (!x || !aligned(x, 16)) return invalid("x must not be NULL and must be 16-byte aligned");
  if (int rc = check_rows_out(Span(x, dim * eb, x_stride * eb, rows), q, scale, rows, dim)) return rc;
  count_launches(1);
  return cuda_status(launch_quantize_i8(x, x_dtype == MOSS_DTYPE_BF16, x_stride, q, scale, rows, dim,
                                        static_cast<cudaStream_t>(stream)), "quantize_i8", "");
}

int moss_op_ln_modulate_i8(const float* x, const float* shift, const float* scale, int8_t* q, float* q_scale, int rows,
                           int dim, void* stream) {
  set_error(MOSS_OK, "");
  if (!rows_dims_ok(rows, dim)) return invalid(kRowsDims);
  if (rows == 0) return MOSS_OK;
  if (!x || !shift || !scale) return invalid("pointers must not be NULL");
  if (!aligned(x, 16) || !aligned(shift, 16) || !aligned(scale, 16)) return invalid("16-byte alignment required");
  if (int rc = check_rows_out(Span(x, 4 * static_cast<int64_t>(rows) * dim), q, q_scale, rows, dim)) return rc;
  const Span sq(q, static_cast<int64_t>(rows) * dim), ss(q_scale, 4 * static_cast<int64_t>(rows));
  for (const float* v : {shift, scale})
    if (overlap(Span(v, 4 * static_cast<int64_t>(dim)), sq) || overlap(Span(v, 4 * static_cast<int64_t>(dim)), ss))
      return invalid("the outputs must not overlap shift or scale");
  count_launches(1);
  return cuda_status(launch_ln_mod_i8(x, shift, scale, q, q_scale, rows, dim, 1e-6f, static_cast<cudaStream_t>(stream)),
                     "ln_modulate_i8", "");
}

int moss_op_swiglu_i8(const void* gu, int64_t gu_stride, int8_t* q, float* scale, int rows, int dim, void* stream) {
  set_error(MOSS_OK, "");
  if (!rows_dims_ok(rows, dim)) return invalid(kRowsDims);
  if (gu_stride < 2 * static_cast<int64_t>(dim) || gu_stride % 8) return invalid("gu_stride must be >= 2 dim and a multiple of 8");
  if (!stride_fits(gu_stride, rows)) return invalid("gu_stride is too long");
  if (rows == 0) return MOSS_OK;
  if (!gu || !aligned(gu, 16)) return invalid("gu must not be NULL and must be 16-byte aligned");
  if (int rc = check_rows_out(Span(gu, 4 * static_cast<int64_t>(dim), 2 * gu_stride, rows), q, scale, rows, dim)) return rc;
  count_launches(1);
  return cuda_status(launch_swiglu_i8(static_cast<const bf16*>(gu), gu_stride, q, scale, rows, dim,
                                      static_cast<cudaStream_t>(stream)), "swiglu_i8", "");
}

static int gemm_i8_call(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale, const void* bias,
                        const float* gate, const float* residual, void* c, int c_dtype, int M, int N, int K,
                        void* stream, int selftest) {
  set_error(MOSS_OK, "");
  if (!known_dtype(c_dtype)) return invalid("c_dtype must be MOSS_DTYPE_F32 or MOSS_DTYPE_BF16");
  if (M < 0 || N < 1 || K < 16 || K % 16 || K > kMaxI8K)
    return invalid("need M >= 0, N >= 1 and K a multiple of 16, 16 <= K <= 65536");
  if ((gate == nullptr) != (residual == nullptr)) return invalid("gate and residual go together");
  if (residual && c_dtype != MOSS_DTYPE_F32) return invalid("the gated residual form writes FP32");
  if (((static_cast<int64_t>(M) + 15) / 16) * ((static_cast<int64_t>(N) + 127) / 128) * 8 > 0x7fffffff)
    return invalid("M * N is too large: ceil(M / 16) ceil(N / 128) must be below 2^28");
  const int64_t out = static_cast<int64_t>(M) * N * dtype_bytes(c_dtype);
  if (M == 0) return MOSS_OK;
  if (!a || !a_scale || !b || !b_scale || !c) return invalid("a, a_scale, b, b_scale and c must not be NULL");
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(c, 16) || !aligned(residual, 16))
    return invalid("a, b, c and residual must be 16-byte aligned");
  if (!aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(gate, 4) || !aligned(bias, 2))
    return invalid("a_scale, b_scale, gate and bias must be aligned to their elements");
  const Span sc(c, out);
  if (overlap(sc, Span(a, static_cast<int64_t>(M) * K)) || overlap(sc, Span(b, static_cast<int64_t>(N) * K)) ||
      overlap(sc, Span(a_scale, 4 * static_cast<int64_t>(M))) || overlap(sc, Span(b_scale, 4 * static_cast<int64_t>(N))) ||
      (bias && overlap(sc, Span(bias, 2 * static_cast<int64_t>(N)))) ||
      (gate && overlap(sc, Span(gate, 4 * static_cast<int64_t>(N)))) ||
      (residual && residual != c && overlap(sc, Span(residual, out))))
    return invalid("c must not overlap an input (it may be the residual itself)");
  unsigned* err = device_error_word();
  if (!err) return set_error(MOSS_ERR_CUDA, "device error word");
  GemmI8Params p;
  p.M = M; p.N = N; p.K = K;
  p.a_scale = a_scale; p.b_scale = b_scale; p.bias = static_cast<const bf16*>(bias);
  p.gate = gate; p.residual = residual; p.c = c; p.c_bf16 = c_dtype == MOSS_DTYPE_BF16;
  p.selftest = selftest;
  std::string detail;
  count_launches(1);
  const cudaError_t e = launch_gemm_i8(a, b, p, static_cast<cudaStream_t>(stream), err, &detail);
  return cuda_status(e, "gemm_i8", detail);
}

int moss_op_gemm_i8(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale, const void* bias,
                    const float* gate, const float* residual, void* c, int c_dtype, int M, int N, int K, void* stream) {
  return gemm_i8_call(a, a_scale, b, b_scale, bias, gate, residual, c, c_dtype, M, N, K, stream, 0);
}

int moss_selftest_gemm_i8_timeout(int failure, const int8_t* a, const float* a_scale, const int8_t* b,
                                  const float* b_scale, void* c, int M, int N, int K, void* stream) {
  set_error(MOSS_OK, "");
  if (failure != MOSS_I8_LOST_LOAD && failure != MOSS_I8_LOST_LOAD_PAIR && failure != MOSS_I8_KEPT_ACCUMULATOR)
    return invalid("unknown failure");
  if (M < 1 || N < 1 || !gemm_i8_selftest_reaches(failure, M, N, K)) return invalid("a call of these sizes does not reach the failure");
  return gemm_i8_call(a, a_scale, b, b_scale, nullptr, nullptr, nullptr, c, MOSS_DTYPE_BF16, M, N, K, stream, failure);
}

void moss_qk_norm_rope_args_init(moss_qk_norm_rope_args* a, uint32_t struct_size) {
  if (!a || struct_size < sizeof a->struct_size) return;
  moss_qk_norm_rope_args d;
  std::memset(&d, 0, sizeof d);
  d.struct_size = struct_size;
  d.in_dtype = d.out_dtype = MOSS_DTYPE_BF16;
  d.head_dim = d.rot_dim = 128;
  d.pairing = MOSS_ROPE_ADJACENT;
  d.eps = 1e-6f;
  std::memcpy(a, &d, struct_size < sizeof d ? struct_size : sizeof d);
}

int moss_op_qk_norm_rope(const moss_qk_norm_rope_args* a, void* stream) {
  set_error(MOSS_OK, "");
  if (!a) return invalid("args must not be NULL");
  if (a->struct_size != sizeof(moss_qk_norm_rope_args))
    return set_error(MOSS_ERR_ABI_MISMATCH, "moss_qk_norm_rope_args: struct_size differs from the library's");
  if (!known_dtype(a->in_dtype) || !known_dtype(a->out_dtype)) return invalid("in_dtype and out_dtype must be MOSS_DTYPE_F32 or MOSS_DTYPE_BF16");
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256)
    return set_error(MOSS_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  if (a->pairing != MOSS_ROPE_ADJACENT && a->pairing != MOSS_ROPE_HALVES) return invalid("unknown pairing");
  if (a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 8) return invalid("rot_dim must be a multiple of 8, at most head_dim");
  if (a->rows < 0 || a->heads_q < 1 || a->heads_k < 0) return invalid("need rows >= 0, heads_q >= 1, heads_k >= 0");
  if (a->heads_q > 65536 || a->heads_k > 65536) return invalid("at most 65536 heads");
  if (!(a->eps >= 0.f)) return invalid("eps must be >= 0");
  if (a->reserved != 0) return invalid("reserved must be 0");
  const int64_t ib = dtype_bytes(a->in_dtype), ob = dtype_bytes(a->out_dtype);
  const int64_t wq = static_cast<int64_t>(a->heads_q) * a->head_dim, wk = static_cast<int64_t>(a->heads_k) * a->head_dim;
  const bool has_k = a->heads_k > 0;
  if (a->q_stride < wq || a->q_out_stride < wq || (has_k && (a->k_stride < wk || a->k_out_stride < wk)))
    return invalid("a stride is shorter than its row of heads");
  if (!stride_fits(a->q_stride, a->rows) || !stride_fits(a->q_out_stride, a->rows) ||
      (has_k && (!stride_fits(a->k_stride, a->rows) || !stride_fits(a->k_out_stride, a->rows))))
    return invalid("a stride is too long");
  if (a->q_stride * ib % 16 || a->q_out_stride * ob % 16 || (has_k && (a->k_stride * ib % 16 || a->k_out_stride * ob % 16)))
    return invalid("strides must be multiples of 16 bytes");
  if (a->rows == 0) return MOSS_OK;
  if (!a->q || !a->q_out || (has_k && (!a->k || !a->k_out))) return invalid("q, q_out, k and k_out must not be NULL");
  if (a->rot_dim > 0 && (!a->rope || a->n_pos < 1)) return invalid("the rotation needs a rope table of n_pos >= 1 positions");
  if (a->positions && a->rot_dim == 0) return invalid("positions without a rotation");
  if (!aligned(a->q, 16) || !aligned(a->q_out, 16) || (has_k && (!aligned(a->k, 16) || !aligned(a->k_out, 16))) ||
      !aligned(a->q_gain, 16) || !aligned(a->k_gain, 16) || !aligned(a->rope, 16) || !aligned(a->positions, 4))
    return invalid("16-byte alignment required (positions: 4)");
  // Each output is its own input (same address, stride and type), or shares no byte with any input or
  // the other output.
  const Span iq(a->q, wq * ib, a->q_stride * ib, a->rows), oq(a->q_out, wq * ob, a->q_out_stride * ob, a->rows);
  const Span ik(has_k ? a->k : a->q, has_k ? wk * ib : 0, has_k ? a->k_stride * ib : 0, a->rows);
  const Span ok(has_k ? a->k_out : a->q_out, has_k ? wk * ob : 0, has_k ? a->k_out_stride * ob : 0, a->rows);
  const bool same_q = a->q == a->q_out && a->q_stride == a->q_out_stride && ib == ob;
  const bool same_k = has_k && a->k == a->k_out && a->k_stride == a->k_out_stride && ib == ob;
  if (!same_q && overlap(iq, oq)) return invalid("q_out overlaps q without being q");
  if (has_k && ((!same_k && overlap(ik, ok)) || overlap(ik, oq) || overlap(iq, ok) || overlap(oq, ok)))
    return invalid("the query and key buffers overlap");
  const Span aux[4] = {Span(a->q_gain, a->q_gain ? 4 * a->head_dim : 0), Span(a->k_gain, a->k_gain ? 4 * a->head_dim : 0),
                       Span(a->rope, a->rot_dim ? 4 * static_cast<int64_t>(a->n_pos) * a->rot_dim : 0),
                       Span(a->positions, a->positions ? 4 * static_cast<int64_t>(a->rows) : 0)};
  for (const Span& s : aux)
    if (s.width > 0 && (overlap(s, oq) || (has_k && overlap(s, ok)))) return invalid("an output overlaps the gains, the angles or the positions");
  unsigned* err = device_error_word();
  if (!err) return set_error(MOSS_ERR_CUDA, "device error word");
  QkNormRopeParams p;
  p.q = a->q; p.k = a->k; p.q_out = a->q_out; p.k_out = a->k_out;
  p.q_stride = a->q_stride; p.k_stride = a->k_stride; p.q_out_stride = a->q_out_stride; p.k_out_stride = a->k_out_stride;
  p.q_gain = a->q_gain; p.k_gain = a->k_gain; p.rope = a->rope; p.positions = a->positions;
  p.rows = a->rows; p.heads_q = a->heads_q; p.heads_k = a->heads_k; p.rot_dim = a->rot_dim;
  p.n_pos = a->rot_dim > 0 ? a->n_pos : 0;
  p.eps = a->eps;
  count_launches(1);
  return cuda_status(launch_qk_norm_rope(p, a->head_dim, a->pairing == MOSS_ROPE_HALVES, a->in_dtype == MOSS_DTYPE_BF16,
                                         a->out_dtype == MOSS_DTYPE_BF16, static_cast<cudaStream_t>(stream), err),
                     "qk_norm_rope", "");
}

int moss_op_rope_table(float* table, int grid_h, int grid_w, int n_txt, void* stream) {
  set_error(MOSS_OK, "");
  const int64_t n = static_cast<int64_t>(grid_h) * grid_w + n_txt;
  if (grid_h < 0 || grid_w < 0 || n_txt < 0 || n > (1 << 24)) return invalid("need grid_h, grid_w, n_txt >= 0 and at most 2^24 tokens");
  if (n == 0) return MOSS_OK;
  if (!table || !aligned(table, 16)) return invalid("table must not be NULL and must be 16-byte aligned");
  count_launches(1);
  return cuda_status(launch_rope_table_tokens(reinterpret_cast<float2*>(table), grid_h, grid_w, n_txt,
                                              static_cast<cudaStream_t>(stream)), "rope_table", "");
}

}  // extern "C"
