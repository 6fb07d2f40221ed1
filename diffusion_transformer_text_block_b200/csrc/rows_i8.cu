// Rows to 8-bit integers, one scale a row: the operands of the 8-bit GEMM.
//
//   amax = max_j |h_j|,  scale = amax / 127,  q_j = round_half_even(127 h_j / amax)
//
// with h the row itself (BF16 or FP32), the modulated LayerNorm of an FP32 row, or the SwiGLU
// activation SiLU(g) * u of a BF16 row [g | u].  One pass: a row's h stays in registers (FP32)
// between the maximum and the rounding, so every input byte is read once and every output byte
// written once; the kernels are bound by HBM.  A team of 1, 2, 4 or 8 warps of a block of 256
// threads takes a row, VPL units of 8 elements a lane.
//
// Rounding.  Adding 1.5 * 2^23 to h * inv, inv = fl(127 / amax), in one FMA rounds the exact product
// to the nearest integer, half to even, and leaves it in the sum's low byte.  h * inv is off
// 127 h / amax by at most 127 * 2^-24 = 7.6e-6.
//   FP32 rows, and the LayerNorm's and SwiGLU's: the distance |t - q| of a unit's 8 elements is
//   compared once with 1/2 - 1.6e-5, and an element closer to a border is settled by an exact
//   comparison in FP64 (3 % of the SwiGLU kernel's time).
//   BF16 rows need no such check.  With 8-bit significands X of h and A of amax, 127 h / amax is
//   either a half-integer or, relatively, at least 1 / (254 * 255) away from one, far above FP32's
//   error.  It is a half-integer only for h = amax / 2 (63.5), which goes to 64 because inv is
//   rounded up, and for A = 254, where inv is a power of two and every product exact.
//   So q equals the definition for every finite row of h, h being in FP32.
#include "i8.cuh"
#include "ops_i8.h"

namespace moss {

namespace {

constexpr float kRoundMagic = 12582912.0f;          // 1.5 * 2^23
constexpr float kBorder = 0.5f - 1.6e-5f;
constexpr float kTinyAmax = 7.888609052210118e-31f;  // 2^-100: a row below it, where 127 / amax may
constexpr float kTinyUp = 1.2676506002282294e30f;     // overflow, is first made 2^100 larger (exactly)
constexpr int kRowThreads = 256;

// Three-input maximum of absolute values, a NaN kept (one instruction).
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The larger magnitudes of m's halves and of 8 BF16 values, as bits (NaN > infinity > finite).
__device__ __forceinline__ uint32_t max_bf16x8(uint32_t m, const uint4& p) {
  constexpr uint32_t k = 0x7fff7fffu;
  return __vimax3_u16x2(__vimax3_u16x2(m, p.x & k, p.y & k), p.z & k, p.w & k);
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& p, float2 (&v)[4]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// SiLU(g) u for 8 elements.  1 + e^-g passes 2^126, where the fast division gives 0, below g = -87.3, and FP32's
// range below -88.7, while SiLU(g) is a normal number down to -92 and one that a large u brings back further
// still.  Below -87, 1 + e^-g is e^-g in FP32 and SiLU(g) u = u e^(g/2) g e^(g/2), whose running product is never
// smaller than the result.  A unit takes that path for a gate whose BF16 pattern lies above that of -87 (0xc2ae):
// one comparison for 8 elements (9216 x 8192: 59.7 us with it, 60.8 without, in turn).
__device__ __forceinline__ void silu_mul8(const uint4& g8, const uint4& u8, float2 (&h)[4]) {
  float2 g[4], u[4];
  unpack_bf16x8(g8, g);
  unpack_bf16x8(u8, u);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    h[e] = __fmul2_rn(make_float2(__fdividef(g[e].x, 1.0f + __expf(-g[e].x)), __fdividef(g[e].y, 1.0f + __expf(-g[e].y))), u[e]);
  const uint32_t top = __vmaxu2(__vimax3_u16x2(g8.x, g8.y, g8.z), g8.w);
  if (max(top, top << 16) > 0xc2aeffffu) {
    const auto far = [](float h, float gate, float up) {
      const float a = __expf(0.5f * gate);
      return gate < -87.0f ? up * a * gate * a : h;
    };
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = make_float2(far(h[e].x, g[e].x, u[e].x), far(h[e].y, g[e].y, u[e].y));
  }
}

// The warps of one row: 2^SH of them (SH < 0: 2^shift, known at run time), `first` the block's warp they
// start at.
template <int SH>
struct Team {
  int warp, first, shift_, lane, id;
  __device__ __forceinline__ int shift() const { return SH < 0 ? shift_ : SH; }
  __device__ __forceinline__ void sync() const {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(32 << shift()) : "memory");
  }
};
__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
// Sum over the row's warps (part: one slot per warp of the block), and the maximum of |h| as bits, in
// whose order NaN > infinity > every finite value.
template <int SH>
__device__ __forceinline__ float row_sum(float s, float* part, const Team<SH>& t) {
  s = warp_sum(s);
  if (t.shift() == 0) return s;
  if (t.lane == 0) part[t.warp] = s;
  t.sync();
  s = part[t.first];
#pragma unroll
  for (int k = 1; k < 1 << t.shift(); ++k) s += part[t.first + k];
  return s;
}
template <int SH>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* part, const Team<SH>& t) {
  m = __reduce_max_sync(0xffffffffu, m);
  if (t.shift() == 0) return m;
  if (t.lane == 0) part[t.warp] = m;
  t.sync();
  m = part[t.first];
#pragma unroll
  for (int k = 1; k < 1 << t.shift(); ++k) m = max(m, part[t.first + k]);
  return m;
}

// r = magic + q, q the nearest integer to h inv.  Where that lies on the border to a neighbour, the side
// is decided exactly: 254 h against (2 q +- 1) amax, products of 33 bits at most, in FP64.
__device__ __forceinline__ float settle(float h, float amax, float inv, float r) {
  const float q = r - kRoundMagic;
  const float d = fmaf(h, inv, -q);
  if (fabsf(d) > kBorder) {
    const float up = copysignf(1.0f, d);
    const double over = fma(254.0, static_cast<double>(h), -(static_cast<double>(2.0f * q + up) * static_cast<double>(amax)));
    const double beyond = over * static_cast<double>(up);
    if (beyond > 0.0 || (beyond == 0.0 && (__float_as_uint(r) & 1u))) r += up;
  }
  return r;
}

enum RowSrc : int { kRowBf16 = 0, kRowF32 = 1, kRowLnMod = 2, kRowSwiglu = 3 };

// A lane's part of a row: VPL units of 8 elements.  16-bit rows: unit i is the 16 bytes u0 + i ustep.
// FP32 rows: unit i is the two quads (16 bytes) u0 + (2 i) ustep and u0 + (2 i + 1) ustep, so that a
// warp's load covers 512 neighbouring bytes there too.  With SH >= 0 the row is exactly 256 VPL 2^SH
// elements: the steps are constants and every lane's units lie inside it.
template <int SRC, int SH>
struct Lane {
  static constexpr bool kF32 = SRC == kRowF32 || SRC == kRowLnMod;
  int u0, ustep_, count;  // count: 16-byte pieces of a row of 16-bit h, quads of an FP32 one
  __device__ __forceinline__ int at(int i, int half) const {
    const int ustep = SH < 0 ? ustep_ : 32 << (SH < 0 ? 0 : SH);
    return kF32 ? u0 + (2 * i + half) * ustep : u0 + i * ustep;
  }
  __device__ __forceinline__ bool has(int i, int half) const { return SH >= 0 || at(i, half) < count; }
};

template <int SRC, int VPL, int SH>
struct RowPart {
  uint4 a[VPL], b[SRC == kRowBf16 ? 1 : VPL];
  __device__ __forceinline__ void load(const void* xin, int64_t x_stride, int64_t row, const Lane<SRC, SH>& l) {
    const uint4* p = static_cast<const uint4*>(xin) + row * (l.kF32 ? x_stride / 4 : x_stride / 8);
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      a[i] = l.has(i, 0) ? __ldg(p + l.at(i, 0)) : zero;
      if constexpr (SRC == kRowSwiglu) b[i] = l.has(i, 0) ? __ldg(p + l.count + l.at(i, 0)) : zero;
      if constexpr (Lane<SRC, SH>::kF32) b[i] = l.has(i, 1) ? __ldg(p + l.at(i, 1)) : zero;
    }
  }
  __device__ __forceinline__ void rows(float2 (&v)[VPL][4]) const {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if constexpr (SRC == kRowBf16) {
        unpack_bf16x8(a[i], v[i]);
      } else if constexpr (SRC == kRowSwiglu) {
        silu_mul8(a[i], b[i], v[i]);
      } else {
        v[i][0] = make_float2(__uint_as_float(a[i].x), __uint_as_float(a[i].y));
        v[i][1] = make_float2(__uint_as_float(a[i].z), __uint_as_float(a[i].w));
        v[i][2] = make_float2(__uint_as_float(b[i].x), __uint_as_float(b[i].y));
        v[i][3] = make_float2(__uint_as_float(b[i].z), __uint_as_float(b[i].w));
      }
    }
  }
};

// Blocks a SM that the registers allow: VPL units of 8 floats (BF16: 4 words until they are rounded) and
// some 40 others.
constexpr int row_blocks(int src, int vpl) {
  if (vpl <= 1) return 5;
  if (vpl <= 4) return vpl == 4 && (src == kRowF32 || src == kRowLnMod) ? 3 : 4;
  return vpl == 6 ? 3 : vpl <= 12 ? 2 : 1;
}

template <int SRC, int VPL, int SH>
__global__ void __launch_bounds__(kRowThreads, row_blocks(SRC, VPL))
    rows_i8_kernel(const void* __restrict__ xin, int64_t x_stride, const float* __restrict__ shift,
                   const float* __restrict__ mscale, int8_t* __restrict__ q, float* __restrict__ scale, int rows,
                   int dim, int shift_, float inv_dim, float eps) {
  __shared__ float part_s[2][8];
  __shared__ uint32_t part_m[2][8];
  const int warp = threadIdx.x >> 5;
  const int sh = SH < 0 ? shift_ : SH;
  const Team<SH> t = {warp, warp >> sh << sh, sh, static_cast<int>(threadIdx.x & 31), warp >> sh};
  const Lane<SRC, SH> l = {(warp - t.first) * 32 + t.lane, 32 << sh, Lane<SRC, SH>::kF32 ? dim >> 2 : dim >> 3};
  const int teams = 8 >> sh;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;

  RowPart<SRC, VPL, SH> part;
  int64_t row = static_cast<int64_t>(blockIdx.x) * teams + t.id;
  // The slots of the cross-warp sums alternate: a warp writes a slot again only after a barrier that
  // every warp of the team passed behind its reads.
  for (int flip = 0; row < rows; row += step, flip ^= 1) {
    float2 v[VPL][4];  // unit i of the lane: 8 elements; the arithmetic goes two elements an instruction
    part.load(xin, x_stride, row, l);
    if constexpr (SRC != kRowBf16) part.rows(v);
    if constexpr (SRC == kRowLnMod) {
      float2 s = both(0.f);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = __fadd2_rn(s, v[i][e]);
      const float mean = row_sum(s.x + s.y, part_s[0], t) * inv_dim;
      float2 ss = both(0.f);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!l.has(i, e >> 1)) continue;
          v[i][e] = __fadd2_rn(v[i][e], both(-mean));
          ss = __ffma2_rn(v[i][e], v[i][e], ss);
        }
      const float rstd = rsqrtf(row_sum(ss.x + ss.y, part_s[1], t) * inv_dim + eps);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!l.has(i, half)) continue;
          const float4 a = __ldg(reinterpret_cast<const float4*>(shift) + l.at(i, half));
          const float4 m = __ldg(reinterpret_cast<const float4*>(mscale) + l.at(i, half));
          float2* h = v[i] + 2 * half;
          h[0] = __ffma2_rn(__fmul2_rn(h[0], both(rstd)), __fadd2_rn(make_float2(m.x, m.y), both(1.0f)), make_float2(a.x, a.y));
          h[1] = __ffma2_rn(__fmul2_rn(h[1], both(rstd)), __fadd2_rn(make_float2(m.z, m.w), both(1.0f)), make_float2(a.z, a.w));
        }
    }

    uint32_t abits = 0;
    if constexpr (SRC == kRowBf16) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) abits = max_bf16x8(abits, part.a[i]);
      abits = max(abits & 0xffff0000u, abits << 16);
    } else {
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) am = max3_abs_nan(am, v[i][e].x, v[i][e].y);
      abits = __float_as_uint(am);
    }
    abits = row_max(abits, part_m[flip], t);
    float amax = __uint_as_float(abits);
    const bool finite = abits < 0x7f800000u;
    if (threadIdx.x == t.first * 32) scale[row] = finite ? amax / 127.0f : __uint_as_float(0x7fffffffu);
    const auto store = [&](int i, uint32_t lo, uint32_t hi) {  // a unit's 8 integers
      if constexpr (Lane<SRC, SH>::kF32) {
        uint32_t* qr = reinterpret_cast<uint32_t*>(q + row * dim);
        if (l.has(i, 0)) qr[l.at(i, 0)] = lo;
        if (l.has(i, 1)) qr[l.at(i, 1)] = hi;
      } else {
        if (l.has(i, 0)) reinterpret_cast<uint2*>(q + row * dim)[l.at(i, 0)] = make_uint2(lo, hi);
      }
    };
    if (!finite) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) store(i, 0, 0);
      continue;
    }
    if constexpr (SRC == kRowBf16) part.rows(v);
    if (amax < kTinyAmax) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = __fmul2_rn(v[i][e], both(kTinyUp));
      amax *= kTinyUp;
    }
    float inv = amax == 0.f ? 0.f : 127.0f / amax;  // a row of zeros: q = 0
    if (SRC == kRowBf16 && fmaf(inv, amax, -127.0f) < 0.f) inv = __uint_as_float(__float_as_uint(inv) + (amax > 0.f));
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float r[8];
      float far = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 s = __ffma2_rn(v[i][e], both(inv), both(kRoundMagic));
        r[2 * e] = s.x;
        r[2 * e + 1] = s.y;
        if constexpr (SRC != kRowBf16) {
          const float2 d = __ffma2_rn(v[i][e], both(inv), __ffma2_rn(s, both(-1.0f), both(kRoundMagic)));
          far = fmaxf(fmaxf(far, fabsf(d.x)), fabsf(d.y));
        }
      }
      if (SRC != kRowBf16 && far > kBorder) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          r[2 * e] = settle(v[i][e].x, amax, inv, r[2 * e]);
          r[2 * e + 1] = settle(v[i][e].y, amax, inv, r[2 * e + 1]);
        }
      }
      uint32_t b[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(r[e]);
      store(i, __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
            __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
    }
  }
}

struct RowArgs {
  const void* x;
  int64_t x_stride;
  const float *shift, *mscale;
  int8_t* q;
  float* scale;
  int rows, dim;
  float eps;
};

template <int SRC, int VPL, int SH>
cudaError_t launch_kernel(const RowArgs& a, int sh, cudaStream_t s) {
  const int teams = 8 >> sh;
  // A few waves of blocks that walk over the rows: 2 to 5 % better than one wave, and than a block for
  // every 8 / 2^sh rows.
  const int64_t blocks = (static_cast<int64_t>(a.rows) + teams - 1) / teams;
  const int64_t most = static_cast<int64_t>(num_sms()) * row_blocks(SRC, VPL) * (SRC == kRowBf16 ? 2 : 4);
  rows_i8_kernel<SRC, VPL, SH><<<static_cast<unsigned>(blocks < most ? blocks : most), kRowThreads, 0, s>>>(
      a.x, a.x_stride, a.shift, a.mscale, a.q, a.scale, a.rows, a.dim, sh, 1.0f / static_cast<float>(a.dim), a.eps);
  return cudaGetLastError();
}

// Rows that fill the lanes exactly have kernels without bounds checks and with constant steps: a third
// fewer instructions (LayerNorm of 9216 x 3072 33.1 -> 25.6 us, SwiGLU of 9216 x 8192 64.3 -> 58.8 us; now, with
// the border check, 27.2 to 28.7 = 0.75 to 0.79 and 59.7 to 61.2 us = 0.94 to 0.96 of the HBM rate).
template <int SRC, int VPL>
cudaError_t launch_shift(const RowArgs& a, int sh, cudaStream_t s) {
  if (a.dim == VPL << (8 + sh)) {
    switch (sh) {
      case 0: return launch_kernel<SRC, VPL, 0>(a, sh, s);
      case 1: return launch_kernel<SRC, VPL, 1>(a, sh, s);
      case 2: return launch_kernel<SRC, VPL, 2>(a, sh, s);
      default: return launch_kernel<SRC, VPL, 3>(a, sh, s);
    }
  }
  return launch_kernel<SRC, VPL, -1>(a, sh, s);
}

template <int SRC>
cudaError_t launch_rows(const RowArgs& a, cudaStream_t s) {
  const int units = a.dim / 8;
  // Units a lane where 8 warps or fewer reach that: 12 for BF16 rows (9216 x 3072 with part of the buffers left
  // in L2: 12.4 us with one warp a row, 14.6 with four; 14.5 with one where nothing is left), whose registers hold two elements a word; 4 for the others (LayerNorm without the
  // border check: 35 us with one warp, 25.6 with four).  More warps a row while there are too few rows to fill the GPU.
  const int most = SRC == kRowBf16 ? 12 : 4;
  int sh = 0;
  while (sh < 3 && (units > (most * 32 << sh) || (static_cast<int64_t>(a.rows) << (sh + 1)) <= num_sms() * 8)) ++sh;
  const int vpl = (units + (32 << sh) - 1) / (32 << sh);
  if (vpl <= 1) return launch_kernel<SRC, 1, -1>(a, sh, s);
  if (vpl <= 2) return launch_kernel<SRC, 2, -1>(a, sh, s);
  if (vpl <= 3) return launch_shift<SRC, 3>(a, sh, s);
  if (vpl <= 4) return launch_shift<SRC, 4>(a, sh, s);
  if constexpr (SRC == kRowBf16) {
    if (vpl <= 6) return launch_shift<SRC, 6>(a, sh, s);
    if (vpl <= 8) return launch_shift<SRC, 8>(a, sh, s);
    if (vpl <= 12) return launch_shift<SRC, 12>(a, sh, s);
  }
  if (vpl <= 8) return launch_kernel<SRC, 8, -1>(a, sh, s);
  return launch_kernel<SRC, 16, -1>(a, sh, s);
}

}  // namespace

cudaError_t launch_quantize_i8(const void* x, bool is_bf16, int64_t x_stride, int8_t* q, float* scale, int rows,
                               int dim, cudaStream_t s) {
  const RowArgs a = {x, x_stride, nullptr, nullptr, q, scale, rows, dim, 0.f};
  return is_bf16 ? launch_rows<kRowBf16>(a, s) : launch_rows<kRowF32>(a, s);
}

cudaError_t launch_ln_mod_i8(const float* x, const float* shift, const float* mscale, int8_t* q, float* scale,
                             int rows, int dim, float eps, cudaStream_t s) {
  return launch_rows<kRowLnMod>({x, dim, shift, mscale, q, scale, rows, dim, eps}, s);
}

cudaError_t launch_swiglu_i8(const bf16* gu, int64_t gu_stride, int8_t* q, float* scale, int rows, int dim,
                             cudaStream_t s) {
  return launch_rows<kRowSwiglu>({gu, gu_stride, nullptr, nullptr, q, scale, rows, dim, 0.f}, s);
}

}  // namespace moss
