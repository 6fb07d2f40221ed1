// Rows to 8-bit integers, one scale a row: the operands of the 8-bit GEMM.
//
//   amax = max_j |h_j|,  scale = amax / 127,  q_j = round_half_even(127 h_j / amax)
//
// with h the row itself (BF16 or FP32), the modulated LayerNorm of an FP32 row, or the SwiGLU
// activation SiLU(g) * u of a BF16 row [g | u].  One pass: a row's h stays in registers (FP32)
// between the maximum and the rounding, so every input byte is read once and every output byte
// written once; the kernels are bound by HBM.  wpr warps share a row (8 / wpr rows per block of
// 256 threads), VPL units of 8 elements per lane.
//
// Rounding.  t = h * fl(127 / amax) is off 127 h / amax by at most 127 * 2^-24 = 7.6e-6, so the
// integer is certain unless t lies within that of a half-integer.  Adding 1.5 * 2^23 rounds the
// exact product to the nearest integer (half to even) and leaves its low byte in the sum's; the
// distance |t - q| of a unit's 8 elements is compared once with 1/2 - 1.6e-5, and a unit with an
// element closer to a border is redone in FP64, where 127 h is exact and a quotient that is no
// half-integer stays at least 2^-34 away from one.  So q equals the definition for every finite row.
#include "common.cuh"
#include "internal.h"

namespace moss {

namespace {

constexpr float kRoundMagic = 12582912.0f;          // 1.5 * 2^23
constexpr float kBorder = 0.5f - 1.6e-5f;
constexpr float kTinyAmax = 7.888609052210118e-31f;  // 2^-100: below it 127 / amax may overflow
constexpr int kRowThreads = 256;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Sum over the row's warps (part: one slot per warp of the block), and the same for the maximum of
// |h| as bits, in whose order NaN > infinity > every finite value.
__device__ __forceinline__ float row_sum(float s, float* part, int wib, int wpr, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (wpr == 1) return s;
  if (lane == 0) part[wib] = s;
  __syncthreads();
  const int w0 = wib & ~(wpr - 1);
  s = 0.f;
  for (int k = 0; k < wpr; ++k) s += part[w0 + k];
  return s;
}
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* part, int wib, int wpr, int lane) {
  m = __reduce_max_sync(0xffffffffu, m);
  if (wpr == 1) return m;
  if (lane == 0) part[wib] = m;
  __syncthreads();
  const int w0 = wib & ~(wpr - 1);
  m = part[w0];
  for (int k = 1; k < wpr; ++k) m = max(m, part[w0 + k]);
  return m;
}

enum RowSrc : int { kRowBf16 = 0, kRowF32 = 1, kRowLnMod = 2, kRowSwiglu = 3 };

template <int SRC, int VPL>
__global__ void __launch_bounds__(kRowThreads)
    rows_i8_kernel(const void* __restrict__ xin, int64_t x_stride, const float* __restrict__ shift,
                   const float* __restrict__ mscale, int8_t* __restrict__ q, float* __restrict__ scale, int rows,
                   int dim, int wpr, float eps) {
  __shared__ float part_s[2][8];
  __shared__ uint32_t part_m[8];
  const int wib = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int sub = wib & (wpr - 1);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (8 / wpr) + wib / wpr;
  const bool live = row < rows;  // block-wide barriers below: no early return
  const int units = dim >> 3;
  const int u0 = sub * 32 + lane, ustep = wpr * 32;

  float v[VPL][8];
  if constexpr (SRC == kRowBf16) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const bf16*>(xin) + row * x_stride);
    uint4 raw[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      raw[i] = live && u0 + i * ustep < units ? __ldg(p + u0 + i * ustep) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < VPL; ++i) unpack_bf16x8(raw[i], v[i]);
  } else if constexpr (SRC == kRowSwiglu) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const bf16*>(xin) + row * x_stride);
    uint4 rg[VPL], ru[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool in = live && u0 + i * ustep < units;
      rg[i] = in ? __ldg(p + u0 + i * ustep) : make_uint4(0, 0, 0, 0);
      ru[i] = in ? __ldg(p + units + u0 + i * ustep) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float g[8], u[8];
      unpack_bf16x8(rg[i], g);
      unpack_bf16x8(ru[i], u);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = __fdividef(g[e], 1.0f + __expf(-g[e])) * u[e];
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(xin) + row * x_stride);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int u = u0 + i * ustep;
      const bool in = live && u < units;
      const float4 a = in ? __ldg(p + 2 * u) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 b = in ? __ldg(p + 2 * u + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
      v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
    }
    if constexpr (SRC == kRowLnMod) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[i][e];
      const float mean = row_sum(s, part_s[0], wib, wpr, lane) / static_cast<float>(dim);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const bool in = u0 + i * ustep < units;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[i][e] = in ? v[i][e] - mean : 0.f;
          ss = fmaf(v[i][e], v[i][e], ss);
        }
      }
      const float rstd = rsqrtf(row_sum(ss, part_s[1], wib, wpr, lane) / static_cast<float>(dim) + eps);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int u = u0 + i * ustep;
        if (u < units) {
          const float4* sh = reinterpret_cast<const float4*>(shift) + 2 * u;
          const float4* sc = reinterpret_cast<const float4*>(mscale) + 2 * u;
          const float4 a = __ldg(sh), b = __ldg(sh + 1), c = __ldg(sc), d = __ldg(sc + 1);
          const float hs[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          const float hm[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = fmaf(v[i][e] * rstd, 1.0f + hm[e], hs[e]);
        }
      }
    }
  }

  float am = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) am = max_nan(am, fabsf(v[i][e]));
  const uint32_t abits = row_max(__float_as_uint(am), part_m, wib, wpr, lane);
  if (!live) return;
  const float amax = __uint_as_float(abits);
  const bool finite = abits < 0x7f800000u;
  if (sub == 0 && lane == 0) scale[row] = finite ? amax / 127.0f : __uint_as_float(0x7fffffffu);
  const bool tiny = amax < kTinyAmax;
  // A row of zeros, and one that is not finite, has q = 0 (inv = 0; its elements are skipped below).
  const bool zero = abits == 0 || !finite;
  const float inv = zero || tiny ? 0.f : 127.0f / amax;
  uint2* qr = reinterpret_cast<uint2*>(q + row * dim);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int u = u0 + i * ustep;
    if (u >= units) continue;
    uint32_t b[8];
    float far = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = fmaf(v[i][e], inv, kRoundMagic);
      const float d = fmaf(v[i][e], inv, kRoundMagic - r);
      b[e] = __float_as_uint(r);
      far = fmaxf(far, fabsf(d));
    }
    if (zero) {
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = 0;
    } else if (far > kBorder || tiny) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        b[e] = static_cast<uint32_t>(__double2int_rn(static_cast<double>(v[i][e]) * 127.0 / static_cast<double>(amax)));
    }
    uint2 o;
    o.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    qr[u] = o;
  }
}

template <int SRC>
cudaError_t launch_rows(const void* x, int64_t x_stride, const float* shift, const float* mscale, int8_t* q,
                        float* scale, int rows, int dim, float eps, cudaStream_t s) {
  const int units = dim / 8;
  // Warps per row: at most 4 units a lane where 8 warps reach that; all 8 warps on one row while
  // there are too few rows to fill the GPU otherwise.
  int wpr = 1;
  while (wpr < 8 && (units > 32 * wpr * 4 || static_cast<int64_t>(rows) * wpr * 2 <= num_sms() * 8)) wpr *= 2;
  const int vpl = (units + 32 * wpr - 1) / (32 * wpr);
  const unsigned grid = static_cast<unsigned>((rows + 8 / wpr - 1) / (8 / wpr));
#define MOSS_ROWS(V) \
  rows_i8_kernel<SRC, V><<<grid, kRowThreads, 0, s>>>(x, x_stride, shift, mscale, q, scale, rows, dim, wpr, eps)
  if (vpl <= 1) MOSS_ROWS(1);
  else if (vpl <= 2) MOSS_ROWS(2);
  else if (vpl <= 3) MOSS_ROWS(3);
  else if (vpl <= 4) MOSS_ROWS(4);
  else if (vpl <= 8) MOSS_ROWS(8);
  else MOSS_ROWS(16);
#undef MOSS_ROWS
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_i8(const void* x, bool is_bf16, int64_t x_stride, int8_t* q, float* scale, int rows,
                               int dim, cudaStream_t s) {
  return is_bf16 ? launch_rows<kRowBf16>(x, x_stride, nullptr, nullptr, q, scale, rows, dim, 0.f, s)
                 : launch_rows<kRowF32>(x, x_stride, nullptr, nullptr, q, scale, rows, dim, 0.f, s);
}

cudaError_t launch_ln_mod_i8(const float* x, const float* shift, const float* mscale, int8_t* q, float* scale,
                             int rows, int dim, float eps, cudaStream_t s) {
  return launch_rows<kRowLnMod>(x, dim, shift, mscale, q, scale, rows, dim, eps, s);
}

cudaError_t launch_swiglu_i8(const bf16* gu, int64_t gu_stride, int8_t* q, float* scale, int rows, int dim,
                             cudaStream_t s) {
  return launch_rows<kRowSwiglu>(gu, gu_stride, nullptr, nullptr, q, scale, rows, dim, 0.f, s);
}

}  // namespace moss
