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
// (g_a cos, g_b sin, g_a sin, g_b cos) per pair, 3 operations an element after the sum of squares.
#include "common.cuh"
#include "internal.h"

namespace moss {

namespace {

constexpr int kQkThreads = 256;
constexpr int kQkUnroll = 4;  // heads in flight per lane group

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const bf16* p, float* v) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
  v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
}
__device__ __forceinline__ void load8(const float* p, float* v) { load4(p, v); load4(p + 4, v + 4); }
__device__ __forceinline__ void load8(const bf16* p, float* v) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void store8(float* p, const float* v) { store4(p, v); store4(p + 4, v + 4); }
__device__ __forceinline__ void store8(bf16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// LPH lanes per head (head_dim = 8 LPH).
template <int LPH, bool HALVES, typename TI, typename TO>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkNormRopeParams p, unsigned* err) {
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
  float g[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  const float* gain = is_q ? p.q_gain : p.k_gain;
  if (gain) {
    load4(gain + o1, g);
    load4(gain + o2, g + 4);
  }
  // Pair i of the lane: elements (2i, 2i + 1), or with halves (i, i + 4).
  float ca[4], sb[4], sa[4], cb[4];
  {
    float t[8] = {1.f, 0.f, 1.f, 0.f, 1.f, 0.f, 1.f, 0.f};
    if (turned) load8(p.rope + (static_cast<int64_t>(pos) * (p.rot_dim / 2) + 4 * l) * 2, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = HALVES ? i : 2 * i, b = HALVES ? i + 4 : 2 * i + 1;
      ca[i] = g[a] * t[2 * i];
      sb[i] = g[b] * t[2 * i + 1];
      sa[i] = g[a] * t[2 * i + 1];
      cb[i] = g[b] * t[2 * i];
    }
  }
  const int h_end = min(heads, (chunk + 1) * p.heads_per_chunk);
  for (int h0 = chunk * p.heads_per_chunk + lane / LPH; h0 - lane / LPH < h_end; h0 += kPer * kQkUnroll) {
    float v[kQkUnroll][8];
#pragma unroll
    for (int i = 0; i < kQkUnroll; ++i) {
      const int h = h0 + i * kPer;
      if (h < h_end) {
        const TI* s = src + static_cast<int64_t>(h) * kDim;
        if (HALVES) {
          load4(s + o1, v[i]);
          load4(s + o2, v[i] + 4);
        } else {
          load8(s + o1, v[i]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kQkUnroll; ++i) {
      const int h = h0 + i * kPer;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(fmaf(ss, 1.0f / kDim, p.eps));
      float y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int a = HALVES ? j : 2 * j, b = HALVES ? j + 4 : 2 * j + 1;
        const float xa = v[i][a] * r, xb = v[i][b] * r;
        y[a] = fmaf(xa, ca[j], -(xb * sb[j]));
        y[b] = fmaf(xa, sa[j], xb * cb[j]);
      }
      if (h < h_end) {
        TO* d = dst + static_cast<int64_t>(h) * kDim;
        if (HALVES) {
          store4(d + o1, y);
          store4(d + o2, y + 4);
        } else {
          store8(d + o1, y);
        }
      }
    }
  }
}

template <int LPH, bool HALVES, typename TI, typename TO>
cudaError_t launch_one(QkNormRopeParams p, cudaStream_t s, unsigned* err) {
  constexpr int kPer = 32 / LPH;
  // Heads per warp: all of a token's where there are enough tokens (gains and angles are then read
  // once), fewer until the warps fill the GPU.
  int hpc = ((p.heads_q > p.heads_k ? p.heads_q : p.heads_k) + kPer - 1) / kPer * kPer;
  const int64_t want = static_cast<int64_t>(num_sms()) * 32;
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
