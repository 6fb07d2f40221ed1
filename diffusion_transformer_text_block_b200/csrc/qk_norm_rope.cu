// Per-head RMSNorm of the queries and keys and the rotation of their pairs, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * gain                      over the head_dim elements of a head
//   (y_a, y_b) <- (y_a cos - y_b sin, y_a sin + y_b cos)        pair i of the token's position
//
// Pairs: adjacent, (2i, 2i+1), the library's own rotation (SGLang cookbook, Qwen-Image 2.1:
// complex rotary multiplication); or halves, (i, i + rot_dim/2).  Elements from rot_dim on are
// normalised and not rotated.
//
// Bound by HBM: each element is read and written once.  head_dim / 8 lanes hold a head, 8 elements
// a lane, always the same 8 of a head: with halves a lane's elements are 4 of the first half and the
// 4 they pair with, so no pairing needs a shuffle.  A warp stays on one token and walks over some of
// its heads, so a lane reads its gains and angles once and folds them into 16 coefficients:
// (g_a cos, -g_b sin, g_a sin, g_b cos) per pair.  The first and the second elements of the pairs are
// kept apart, so that all the arithmetic goes two pairs an instruction.
#include "i8.cuh"
#include "ops_i8.h"

namespace moss {

namespace {

constexpr int kQkThreads = 256;
constexpr int kQkUnroll = 4;  // heads in flight per lane group

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A lane's 8 elements as they lie in memory (two pieces of 4), and apart: a, the pairs' first elements, and
// b, their second ones.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  float4 x, y;
  template <bool HALVES>
  __device__ __forceinline__ void load(const float* p, int o1, int o2) {
    x = *reinterpret_cast<const float4*>(p + o1);
    y = *reinterpret_cast<const float4*>(p + o2);
  }
  template <bool HALVES>
  __device__ __forceinline__ void split(float2 (&a)[2], float2 (&b)[2]) const {
    if (HALVES) {
      a[0] = make_float2(x.x, x.y); a[1] = make_float2(x.z, x.w);
      b[0] = make_float2(y.x, y.y); b[1] = make_float2(y.z, y.w);
    } else {
      a[0] = make_float2(x.x, x.z); a[1] = make_float2(y.x, y.z);
      b[0] = make_float2(x.y, x.w); b[1] = make_float2(y.y, y.w);
    }
  }
  template <bool HALVES>
  static __device__ __forceinline__ void store(float* p, int o1, int o2, const float2 (&a)[2], const float2 (&b)[2]) {
    float4* d1 = reinterpret_cast<float4*>(p + o1);
    float4* d2 = reinterpret_cast<float4*>(p + o2);
    if (HALVES) {
      *d1 = make_float4(a[0].x, a[0].y, a[1].x, a[1].y);
      *d2 = make_float4(b[0].x, b[0].y, b[1].x, b[1].y);
    } else {
      *d1 = make_float4(a[0].x, b[0].x, a[0].y, b[0].y);
      *d2 = make_float4(a[1].x, b[1].x, a[1].y, b[1].y);
    }
  }
};
template <>
struct Piece<bf16> {
  uint4 w;
  template <bool HALVES>
  __device__ __forceinline__ void load(const bf16* p, int o1, int o2) {
    if (HALVES) {
      const uint2 x = *reinterpret_cast<const uint2*>(p + o1), y = *reinterpret_cast<const uint2*>(p + o2);
      w = make_uint4(x.x, x.y, y.x, y.y);
    } else {
      w = *reinterpret_cast<const uint4*>(p + o1);
    }
  }
  template <bool HALVES>
  __device__ __forceinline__ void split(float2 (&a)[2], float2 (&b)[2]) const {
    if (HALVES) {
      a[0] = make_float2(lo_bf16(w.x), hi_bf16(w.x)); a[1] = make_float2(lo_bf16(w.y), hi_bf16(w.y));
      b[0] = make_float2(lo_bf16(w.z), hi_bf16(w.z)); b[1] = make_float2(lo_bf16(w.w), hi_bf16(w.w));
    } else {
      a[0] = make_float2(lo_bf16(w.x), lo_bf16(w.y)); a[1] = make_float2(lo_bf16(w.z), lo_bf16(w.w));
      b[0] = make_float2(hi_bf16(w.x), hi_bf16(w.y)); b[1] = make_float2(hi_bf16(w.z), hi_bf16(w.w));
    }
  }
  template <bool HALVES>
  static __device__ __forceinline__ void store(bf16* p, int o1, int o2, const float2 (&a)[2], const float2 (&b)[2]) {
    if (HALVES) {
      *reinterpret_cast<uint2*>(p + o1) = make_uint2(pack_bf16x2(a[0].x, a[0].y), pack_bf16x2(a[1].x, a[1].y));
      *reinterpret_cast<uint2*>(p + o2) = make_uint2(pack_bf16x2(b[0].x, b[0].y), pack_bf16x2(b[1].x, b[1].y));
    } else {
      *reinterpret_cast<uint4*>(p + o1) = make_uint4(pack_bf16x2(a[0].x, b[0].x), pack_bf16x2(a[0].y, b[0].y),
                                                     pack_bf16x2(a[1].x, b[1].x), pack_bf16x2(a[1].y, b[1].y));
    }
  }
};

// LPH lanes per head (head_dim = 8 LPH).
template <int LPH, bool HALVES, typename TI, typename TO>
__global__ void __launch_bounds__(kQkThreads, 4) qk_norm_rope_kernel(const QkNormRopeParams p, unsigned* err) {
  constexpr int kDim = 8 * LPH;
  constexpr int kPer = 32 / LPH;  // heads a warp works on at once
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kQkThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = unit / p.chunks;
  if (row >= p.rows) return;
  int chunk = static_cast<int>(unit - row * p.chunks);
  const bool is_q = chunk < p.chunks_q;
  if (!is_q) chunk -= p.chunks_q;
  const int heads = is_q ? p.heads_q : p.heads_k;
  const TI* src = static_cast<const TI*>(is_q ? p.q : p.k) + row * (is_q ? p.q_stride : p.k_stride);
  TO* dst = static_cast<TO*>(is_q ? p.q_out : p.k_out) + row * (is_q ? p.q_out_stride : p.k_out_stride);

  int pos = static_cast<int>(p.n_pos > 0 ? row % p.n_pos : 0);
  if (p.positions) {
    pos = __ldg(p.positions + row);
    if (pos < 0 || pos >= p.n_pos) {  // the row stays as it is
      if (lane == 0) atomicCAS(err, 0u, static_cast<unsigned>(kErrQkPosition));
      return;
    }
  }
  const int l = lane % LPH;
  // The lane's elements are [o1, o1 + 4) and [o2, o2 + 4) of its head.
  int o1 = 8 * l, o2 = 8 * l + 4;
  const bool turned = 8 * l < p.rot_dim;
  if (HALVES && turned) {
    o1 = 4 * l;
    o2 = p.rot_dim / 2 + 4 * l;
  }
  // Coefficients of the lane's 4 pairs, two a register pair: y_a = a ca + b sb, y_b = a sa + b cb.
  float2 ca[2], sb[2], sa[2], cb[2];
  {
    Piece<float> g = {make_float4(1.f, 1.f, 1.f, 1.f), make_float4(1.f, 1.f, 1.f, 1.f)};
    const float* gain = is_q ? p.q_gain : p.k_gain;
    if (gain) g.load<HALVES>(gain, o1, o2);
    float2 ga[2], gb[2];
    g.split<HALVES>(ga, gb);
    Piece<float> t = {make_float4(1.f, 0.f, 1.f, 0.f), make_float4(1.f, 0.f, 1.f, 0.f)};  // (cos, sin) of 4 pairs
    const float* angles = p.rope + (static_cast<int64_t>(pos) * (p.rot_dim / 2) + 4 * l) * 2;
    if (turned) t.load<false>(angles, 0, 4);
    float2 c[2], s[2];
    t.split<false>(c, s);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ca[i] = __fmul2_rn(ga[i], c[i]);
      sa[i] = __fmul2_rn(ga[i], s[i]);
      cb[i] = __fmul2_rn(gb[i], c[i]);
      sb[i] = __fmul2_rn(gb[i], make_float2(-s[i].x, -s[i].y));
    }
  }
  const int h_end = min(heads, (chunk + 1) * p.heads_per_chunk);
  const int group = lane / LPH;  // the lane's head among the kPer of a step
  // kQkUnroll steps at once; `left` heads from the first on, only the last round has too few.
  const auto round = [&](const TI* s, TO* d, int left) {
    Piece<TI> v[kQkUnroll];
#pragma unroll
    for (int i = 0; i < kQkUnroll; ++i)
      if (group + i * kPer < left) v[i].template load<HALVES>(s + i * kPer * kDim, o1, o2);
#pragma unroll
    for (int i = 0; i < kQkUnroll; ++i) {
      float2 a[2], b[2];
      v[i].template split<HALVES>(a, b);
      float2 q = __ffma2_rn(b[1], b[1], __ffma2_rn(b[0], b[0], __ffma2_rn(a[1], a[1], __fmul2_rn(a[0], a[0]))));
      float ss = q.x + q.y;
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(fmaf(ss, 1.0f / kDim, p.eps));
      const float2 rr = make_float2(r, r);
      float2 ya[2], yb[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        a[j] = __fmul2_rn(a[j], rr);
        b[j] = __fmul2_rn(b[j], rr);
        ya[j] = __ffma2_rn(a[j], ca[j], __fmul2_rn(b[j], sb[j]));
        yb[j] = __ffma2_rn(a[j], sa[j], __fmul2_rn(b[j], cb[j]));
      }
      if (group + i * kPer < left) Piece<TO>::template store<HALVES>(d + i * kPer * kDim, o1, o2, ya, yb);
    }
  };
  int h = chunk * p.heads_per_chunk;
  src += static_cast<int64_t>(h + group) * kDim;
  dst += static_cast<int64_t>(h + group) * kDim;
  constexpr int kRound = kPer * kQkUnroll;
  for (; h + kRound <= h_end; h += kRound, src += kRound * kDim, dst += kRound * kDim) round(src, dst, kRound);
  if (h < h_end) round(src, dst, h_end - h);
}

template <int LPH, bool HALVES, typename TI, typename TO>
cudaError_t launch_one(QkNormRopeParams p, cudaStream_t s, unsigned* err) {
  constexpr int kPer = 32 / LPH;
  // Heads per warp: all of a token's where there are enough tokens (gains and angles are then read
  // once), fewer until there are 16 warps a SM (333 tokens, 24 + 24 heads: 3.9 us, 5.9 with 32 a SM, whose
  // rounds are half empty, and 4.4 with 8).
  int hpc = ((p.heads_q > p.heads_k ? p.heads_q : p.heads_k) + kPer - 1) / kPer * kPer;
  const int64_t want = static_cast<int64_t>(num_sms()) * 16;
  while (hpc > kPer &&
         static_cast<int64_t>(p.rows) * ((p.heads_q + hpc - 1) / hpc + (p.heads_k + hpc - 1) / hpc) < want)
    hpc = (hpc / 2 + kPer - 1) / kPer * kPer;
  p.heads_per_chunk = hpc;
  p.chunks_q = (p.heads_q + hpc - 1) / hpc;
  p.chunks = p.chunks_q + (p.heads_k + hpc - 1) / hpc;
  const int64_t warps = static_cast<int64_t>(p.rows) * p.chunks;
  const unsigned grid = static_cast<unsigned>((warps + kQkThreads / 32 - 1) / (kQkThreads / 32));
  qk_norm_rope_kernel<LPH, HALVES, TI, TO><<<grid, kQkThreads, 0, s>>>(p, err);
  return cudaGetLastError();
}

template <int LPH, bool HALVES>
cudaError_t launch_types(const QkNormRopeParams& p, bool in_bf16, bool out_bf16, cudaStream_t s, unsigned* err) {
  if (in_bf16)
    return out_bf16 ? launch_one<LPH, HALVES, bf16, bf16>(p, s, err) : launch_one<LPH, HALVES, bf16, float>(p, s, err);
  return out_bf16 ? launch_one<LPH, HALVES, float, bf16>(p, s, err) : launch_one<LPH, HALVES, float, float>(p, s, err);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeParams& p, int head_dim, bool halves, bool in_bf16, bool out_bf16,
                                cudaStream_t s, unsigned* err) {
  switch (head_dim) {
    case 64: return halves ? launch_types<8, true>(p, in_bf16, out_bf16, s, err) : launch_types<8, false>(p, in_bf16, out_bf16, s, err);
    case 128: return halves ? launch_types<16, true>(p, in_bf16, out_bf16, s, err) : launch_types<16, false>(p, in_bf16, out_bf16, s, err);
    case 256: return halves ? launch_types<32, true>(p, in_bf16, out_bf16, s, err) : launch_types<32, false>(p, in_bf16, out_bf16, s, err);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moss
