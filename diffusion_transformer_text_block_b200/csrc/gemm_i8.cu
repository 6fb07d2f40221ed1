// 8-bit integer GEMM with a scale for each token and each output channel.
//
//   C[m, n] = (sum_k A[m, k] B[n, k]) a_scale[m] b_scale[n] + bias[n]
//   C[m, n] = residual[m, n] + gate[n] * (the same)                      with a gate and a residual
//
// A: activations [M, K], B: weights [N, K], signed 8 bits, K-contiguous.  The sums are exact: 32-bit
// integers in TMEM (|a|, |b| <= 128 and K <= kMaxI8K, so |sum| < 2^31).  The epilogue rounds a sum to
// FP32 (below 2^24 it is exact), and the rest is FP32 with one rounding to BF16 at the end where C
// is BF16.
//
// The weights are the wide operand in every kernel: few tokens then make a narrow tile and not an
// empty one, a thread of an epilogue holds one channel (its scale, bias and gate in registers), and a
// warp stores 32 neighbouring channels of a token (with a row a thread the epilogue of the CTA pairs
// was as long as their products: 196 us against 179 for 9216 x 9216 x 3072).
//
// `gemm_i8_one_kernel` (1 token) and `gemm_i8_few_kernel` (2..16): bound by the weights' bytes.  No
// tile, no barrier before the first load: warps read their channels with 16-byte loads straight into
// dp4a or mma.sync (the legacy tensor path, which at this rate of bytes is nowhere near its limit;
// tcgen05 would first have to bring the weights through shared memory).  One token through 9216 x 3072
// 7.5 us, 3.8 TB/s of weights; the launch and the first loads' latency are 2.5 us of that.
//
// `gemm_i8_flat_kernel` (a wave of tiles or less): one CTA per tile of 128 output channels and NT tokens
// (tcgen05.mma kind::i8, 128 x NT x 32), the K axis split over the CTAs of a cluster, whose partial
// sums meet in shared memory of the cluster (integers: the order does not matter).  Bound by latencies:
// of about 9.5 us for 77 tokens x 3072 x 4096 the first slot is full after 2.2, the weights have streamed
// after 4.6, the sums have met after 6.5 (clocks inside the kernel).
//   warp 0      TMA producer: 128 x 128 bytes of B and NT x 128 bytes of A per slot (128-byte swizzle)
//   warp 1      MMA issuer, four 32-deep steps a slot
//   warps 2..9  epilogue (two per TMEM lane quadrant, each half of the tokens)
//
// `gemm_i8_pair_kernel` (more tiles): persistent CTA pairs, 256 channels x 256 tokens a pair
// (tcgen05.mma.cta_group::2, 256 x 256 x 32) into one of two accumulators, seven 32 KB slots a CTA, the
// epilogue of a tile under the products of the next.  Bound by the tensor pipe and, in long runs, by the
// power cap: 9216 x 9216 x 3072 159 to 166 us = 3.1 to 3.3 PTOP/s, 8192^3 3.3 to 3.4 PTOP/s, 1.9 to 2.1 times
// the measured BF16 rate.  (256 x 128 tiles ran at half that rate; two pairs sharing a tile's K gained 6 to 19 % below
// 32 tiles and lost as much above.)
//   warp 0      TMA producer, in both CTAs, counted on the even CTA's barriers
//   warp 1      MMA issuer, even CTA only
//   warps 2..9  epilogue, in both CTAs
//   warp 10     even CTA: waits for the loads and meets warp 1 at a named barrier for each slot
#include "i8.cuh"
#include "ops_i8.h"

namespace moss {

namespace {

constexpr int kBK = 128;      // K bytes (= elements) per slot, one 128-byte swizzle row
constexpr int kTileN = 128;   // output channels per tile
constexpr int kFlatThreads = 320;
constexpr int kMaxSplit = 8;  // portable cluster size
static_assert(static_cast<int64_t>(kMaxI8K) * 128 * 128 <= (int64_t{1} << 30), "32-bit sums are exact");

// Pieces of `size` that n >= 1 elements fill, for every n of 31 bits.
__host__ __device__ constexpr int pieces(int n, int size) { return (n - 1) / size + 1; }
static_assert(pieces(0x7fffffff, 256) == 1 << 23 && pieces(256, 256) == 1 && pieces(257, 256) == 2 && pieces(1, 256) == 1, "");

template <int NT>
struct FlatShape {
  static constexpr int kWBytes = kTileN * kBK;
  static constexpr int kXBytes = NT * kBK;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kPartBytes = kTileN * NT * 4;  // partial sums a CTA receives from its cluster
  static constexpr int kMaxStages = (223 * 1024 - kPartBytes) / kStageBytes;
  static constexpr int kStages = kMaxStages < 10 ? kMaxStages : 10;
  static constexpr int kTmemCols = NT < 32 ? 32 : NT;
  static constexpr int kSmemBytes = kStages * kStageBytes + kPartBytes + NT * 4 + 1024 + 256;
  static_assert(kStageBytes % 1024 == 0 && kSmemBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Let the loads already issued land (bounded as well): after an abort too, no copy is in flight when
// the CTA reuses its slots or exits.
template <int STAGES>
__device__ __forceinline__ void drain_loads(uint64_t* full, const int (&armed)[STAGES]) {
  const uint64_t t0 = globaltimer_ns();
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    if (armed[s] < 0) continue;
    const uint32_t a = smem_u32(&full[s]);
    while (!mbar_try_wait(a, static_cast<uint32_t>(armed[s])) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
    }
  }
}

// The epilogue of one output value.
struct I8Channel {
  float scale, bias, gate;
};
__device__ __forceinline__ void store_value(const GemmI8Params& p, const I8Channel& ch, int acc, float a_scale, int m,
                                            int n) {
  float v = fmaf(__int2float_rn(acc) * a_scale, ch.scale, ch.bias);
  const int64_t at = static_cast<int64_t>(m) * p.N + n;
  if (p.residual) v = fmaf(ch.gate, v, p.residual[at]);
  if (p.c_bf16)
    static_cast<bf16*>(p.c)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p.c)[at] = v;
}

// The same for B tokens from m on, `count` of them inside C: every load before the first store.
template <int B>
__device__ __forceinline__ void store_values(const GemmI8Params& p, const I8Channel& ch, const uint32_t (&acc)[B],
                                             const float* scales, int m, int count, int n) {
  const int64_t at = static_cast<int64_t>(m) * p.N + n;
  float v[B];
#pragma unroll
  for (int i = 0; i < B; ++i) v[i] = fmaf(__int2float_rn(static_cast<int>(acc[i])) * scales[i], ch.scale, ch.bias);
  if (p.residual) {
    float r[B];
#pragma unroll
    for (int i = 0; i < B; ++i) r[i] = i < count ? p.residual[at + static_cast<int64_t>(i) * p.N] : 0.f;
#pragma unroll
    for (int i = 0; i < B; ++i) v[i] = fmaf(ch.gate, v[i], r[i]);
  }
  if (p.c_bf16) {
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (i < count) static_cast<bf16*>(p.c)[at + static_cast<int64_t>(i) * p.N] = __float2bfloat16_rn(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (i < count) static_cast<float*>(p.c)[at + static_cast<int64_t>(i) * p.N] = v[i];
  }
}

template <int NT>
__global__ void __launch_bounds__(kFlatThreads, 1)
    gemm_i8_flat_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const GemmI8Params p, int split, unsigned* err) {
  using S = FlatShape<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sX = smem + S::kStages * S::kWBytes;
  uint32_t* part = reinterpret_cast<uint32_t*>(smem + S::kStages * S::kStageBytes);
  float* scales = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes + S::kPartBytes);  // of the tile's tokens
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + NT);
  uint64_t* empty = full + S::kStages;
  uint64_t* tfull = empty + S::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int num_n = pieces(p.N, kTileN);
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int n0 = (tile % num_n) * kTileN;
  const int m0 = (tile / num_n) * NT;
  const int num_kb = pieces(p.K, kBK);
  const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * rank / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  // The producer warp needs neither TMEM nor the others: it announces its barriers and goes on, so the
  // first loads are under way while TMEM is allocated (about 0.7 us of a call of 7).
  tc_fence_before();
  if (warp == 0) {
    __syncwarp();
    asm volatile("bar.arrive 2, %0;" ::"n"(kFlatThreads) : "memory");
  } else {
    asm volatile("bar.sync 2, %0;" ::"n"(kFlatThreads) : "memory");
  }
  tc_fence_after();
  const uint32_t tmem_base = warp == 0 ? 0u : *tmem_slot;
  if (split > 1) cluster_arrive();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int armed[S::kStages];  // parity of the last phase armed on full[s], -1 = never
#pragma unroll
      for (int s2 = 0; s2 < S::kStages; ++s2) armed[s2] = -1;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1, err, kErrGemmI8Producer, abort_flag)) break;
        armed[stage] = static_cast<int>(phase);
        mbar_arrive_expect_tx(&full[stage], S::kStageBytes);
        if (p.selftest != kI8SelftestFlatLoad || blockIdx.x != 0 || kb != kb0)
          tma_load_2d(sW + stage * S::kWBytes, &tmW, &full[stage], kb * kBK, n0);
        tma_load_2d(sX + stage * S::kXBytes, &tmX, &full[stage], kb * kBK, m0);
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      drain_loads<S::kStages>(full, armed);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t kIdesc = idesc_i8(kTileN, NT);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full[stage], phase, err, kErrGemmI8Mma, abort_flag)) break;
        tc_fence_after();
        const uint32_t w0 = smem_u32(sW + stage * S::kWBytes);
        const uint32_t x0 = smem_u32(sX + stage * S::kXBytes);
#pragma unroll
        for (int k = 0; k < kBK / 32; ++k)
          mma_i8_ss(tmem_base, sdesc_sw128(w0 + k * 32, 16, 1024), sdesc_sw128(x0 + k * 32, 16, 1024), kIdesc,
                    (kb > kb0 || k > 0) ? 1u : 0u);
        tc_commit(&empty[stage]);
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // Also after an abort: TMEM is released below only once every MMA issued here has completed.
      tc_commit(tfull);
      const uint32_t a = smem_u32(tfull);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
  }

  const int quad = warp & 3;  // TMEM lane quadrant of an epilogue warp
  const int ln = quad * 32 + lane;
  const int n = n0 + ln;
  const int half = (warp - 2) >> 2;  // its half of the tokens
  const bool epi = warp >= 2;
  bool ok = false;
  I8Channel ch = {0.f, 0.f, 0.f};
  const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
  if (epi) {
    if (n < p.N) {
      ch.scale = __ldg(p.b_scale + n);
      if (p.bias) ch.bias = __bfloat162float(p.bias[n]);
      if (p.gate) ch.gate = __ldg(p.gate + n);
    }
    for (int i = half * 128 + ln; i < NT; i += 256) scales[i] = m0 + i < p.M ? __ldg(p.a_scale + m0 + i) : 0.f;
    asm volatile("bar.sync 1, 256;" ::: "memory");  // the eight epilogue warps
    ok = mbar_wait(tfull, 0, err, kErrGemmI8Epilogue, abort_flag) && !*abort_flag;
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
  }
  if (split == 1) {
    if (epi && ok) {
#pragma unroll 1
      for (int c = half * 16; c < NT && m0 + c < p.M; c += 32) {
        uint32_t v[16];
        tmem_ld16(tb + c, v);
        if (n < p.N) store_values<16>(p, ch, v, scales + c, m0 + c, min(16, p.M - m0 - c), n);
      }
    }
  } else {
    // split is a power of two: CTA r finishes the tile's tokens [r share, (r + 1) share), and every CTA
    // writes its partial sums of them to r's shared memory, [CTA][token][channel].
    static_assert(NT / kMaxSplit >= 4 && NT % 16 == 0, "four tokens have one owner");
    const int shift = __popc(NT / split - 1), share = 1 << shift;
    const int tokens = min(NT, p.M - m0);
    __syncwarp();
    cluster_wait();  // every CTA of the cluster has started
    if (epi && ok) {
      const uint32_t mine = smem_u32(part + rank * share * kTileN + ln);
#pragma unroll 1
      for (int c = half * 16; c < tokens; c += 32) {
        uint32_t v[16];
        tmem_ld16(tb + c, v);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {  // four tokens have one owner: share >= 4
          const uint32_t to = mapa_shared(mine + ((c + i) & (share - 1)) * kTileN * 4, (c + i) >> shift);
          if (c + i < tokens) {
#pragma unroll
            for (int j = 0; j < 4; ++j) st_cluster_u32(to + j * kTileN * 4, v[i + j]);
          }
        }
      }
    }
    __syncwarp();
    cluster_sync();
    if (epi && ok && n < p.N) {
      // Eight tokens a round: the code runs once or twice, and a longer body waits for its own instructions
      // (16 a round: 8.2 us instead of 7.4 for 24 x 3072 x 3072).
      constexpr int kB = 8;
      const int c0 = rank * share, count = min(share, tokens - c0);
#pragma unroll 1
      for (int i0 = half * kB; i0 < count; i0 += 2 * kB) {
        uint32_t sum[kB] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 2
        for (int r = 0; r < split; ++r)
#pragma unroll
          for (int i = 0; i < kB; ++i)
            if (i0 + i < count) sum[i] += part[(r * share + i0 + i) * kTileN + ln];
        store_values<kB>(p, ch, sum, scales + c0 + i0, m0 + c0 + i0, min(kB, count - i0), n);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::kTmemCols);
  }
}

template <int NT>
cudaError_t launch_flat(const int8_t* a, const int8_t* b, const GemmI8Params& p, int split, cudaStream_t s,
                        unsigned* err, std::string* emsg) {
  using S = FlatShape<NT>;
  static std::atomic<uint64_t> configured{0};
  if (!configured_on_device(configured)) {
    cudaError_t e = cudaFuncSetAttribute(gemm_i8_flat_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         S::kSmemBytes);
    if (e != cudaSuccess) return e;
    mark_configured_on_device(configured);
  }
  CUtensorMap tw, tx;
  if (!make_tmap_i8_2d(&tw, b, p.K, p.N, kBK, kTileN, emsg) || !make_tmap_i8_2d(&tx, a, p.K, p.M, kBK, NT, emsg))
    return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>(pieces(p.N, kTileN)) * pieces(p.M, NT);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * split));
  cfg.blockDim = dim3(kFlatThreads);
  cfg.dynamicSmemBytes = S::kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(split);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, gemm_i8_flat_kernel<NT>, tw, tx, p, split, err);
}

cudaError_t launch_flat_nt(int nt, const int8_t* a, const int8_t* b, const GemmI8Params& p, int split, cudaStream_t s,
                           unsigned* err, std::string* emsg) {
  switch (nt) {
    case 32: return launch_flat<32>(a, b, p, split, s, err, emsg);
    case 64: return launch_flat<64>(a, b, p, split, s, err, emsg);
    default: return launch_flat<128>(a, b, p, split, s, err, emsg);
  }
}

// ------------------------------------------------------------------------ a few tokens

// 16 bytes of weights, read once: past L1.
__device__ __forceinline__ int4 ld_weights(const int8_t* p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// D (16 x 8) += A (16 x 32, rows) B (32 x 8, columns), 8-bit integers: a.x, a.z of row lane / 4 and a.y,
// a.w of the row 8 below; b of column lane / 4; c[0..1] row lane / 4, columns 2 (lane % 4) + 0..1, c[2..3] 8 below.
__device__ __forceinline__ void mma_16832(int (&c)[4], int a0, int a1, int a2, int a3, int b0, int b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// wk warps of a block (a power of two) share 16 channels and take K in turns of U x 64 bytes.
template <int TG, int U, int W>
__global__ void __launch_bounds__(32 * W) gemm_i8_few_kernel(const int8_t* __restrict__ a,
                                                                   const int8_t* __restrict__ b, const GemmI8Params p,
                                                                   int wk) {
  __shared__ int part[W][TG * 8][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int sub = warp & (wk - 1);
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * (W / wk) + warp / wk) * 16;
  const int8_t* w0 = b + (n0 + g < p.N ? n0 + g : p.N - 1) * p.K;
  const int8_t* w1 = b + (n0 + g + 8 < p.N ? n0 + g + 8 : p.N - 1) * p.K;
  const int8_t* x = a + static_cast<int64_t>(g) * p.K;
  int acc[TG][4];
#pragma unroll
  for (int t = 0; t < TG; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0;
  const int4 zero = make_int4(0, 0, 0, 0);
  for (int k0 = sub * (U * 64); k0 < p.K; k0 += wk * (U * 64)) {
    int4 wa[U], wb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 64 + q * 16;
      wa[u] = k < p.K ? ld_weights(w0 + k) : zero;
      wb[u] = k < p.K ? ld_weights(w1 + k) : zero;
    }
#pragma unroll
    for (int t = 0; t < TG; ++t) {
      int4 xv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * 64 + q * 16;
        xv[u] = k < p.K && t * 8 + g < p.M ? __ldg(reinterpret_cast<const int4*>(x + static_cast<int64_t>(t) * 8 * p.K + k)) : zero;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        mma_16832(acc[t], wa[u].x, wb[u].x, wa[u].y, wb[u].y, xv[u].x, xv[u].y);
        mma_16832(acc[t], wa[u].z, wb[u].z, wa[u].w, wb[u].w, xv[u].z, xv[u].w);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TG; ++t) {
    part[warp][t * 8 + 2 * q][g] = acc[t][0];
    part[warp][t * 8 + 2 * q + 1][g] = acc[t][1];
    part[warp][t * 8 + 2 * q][g + 8] = acc[t][2];
    part[warp][t * 8 + 2 * q + 1][g + 8] = acc[t][3];
  }
  __syncthreads();
  // The group's wk warps finish its 16 x M outputs: lane % 16 the channel.
  const int64_t n = n0 + (lane & 15);
  if (n >= p.N) return;
  I8Channel ch = {__ldg(p.b_scale + n), 0.f, 0.f};
  if (p.bias) ch.bias = __bfloat162float(p.bias[n]);
  if (p.gate) ch.gate = __ldg(p.gate + n);
  const int w_first = warp - sub;
  for (int t = sub * 2 + (lane >> 4); t < p.M; t += 2 * wk) {
    int sum = 0;
    for (int k = 0; k < wk; ++k) sum += part[w_first + k][t][lane & 15];
    store_value(p, ch, sum, __ldg(p.a_scale + t), t, static_cast<int>(n));
  }
}

template <int TG, int U, int W>
cudaError_t launch_few_u(const int8_t* a, const int8_t* b, const GemmI8Params& p, cudaStream_t s) {
  int wk = 1;  // warps per group of 16 channels: K in one turn of each, if the block has so many
  while (wk < W && p.K > U * 64 * wk) wk *= 2;
  const int64_t groups = (static_cast<int64_t>(p.N) + 15) / 16;
  gemm_i8_few_kernel<TG, U, W><<<static_cast<unsigned>((groups * wk + W - 1) / W), 32 * W, 0, s>>>(a, b, p, wk);
  return cudaGetLastError();
}
template <int TG>
cudaError_t launch_few(const int8_t* a, const int8_t* b, const GemmI8Params& p, cudaStream_t s) {
  if (p.K <= 3072) return launch_few_u<TG, 6, 8>(a, b, p, s);
  if (p.K <= 4096) return launch_few_u<TG, 8, 8>(a, b, p, s);
  return launch_few_u<TG, 8, 16>(a, b, p, s);
}

// ------------------------------------------------------------------------ one token
// A warp holds R channels, 16 bytes of each a lane and turn: whole 512-byte pieces of the rows.
constexpr int kOneThreads = 256;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kOneRows = 8;

__device__ __forceinline__ int dot16(const int4& a, const int4& b, int c) {
  return __dp4a(a.w, b.w, __dp4a(a.z, b.z, __dp4a(a.y, b.y, __dp4a(a.x, b.x, c))));
}

__global__ void __launch_bounds__(kOneThreads) gemm_i8_one_kernel(const int8_t* __restrict__ a,
                                                                  const int8_t* __restrict__ b, const GemmI8Params p,
                                                                  int wk) {
  constexpr int R = kOneRows;
  __shared__ int part[kOneWarps][R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp & (wk - 1);
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * (kOneWarps / wk) + warp / wk) * R;
  const int8_t* w[R];
  int acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    w[r] = b + (n0 + r < p.N ? n0 + r : p.N - 1) * p.K;
    acc[r] = 0;
  }
  for (int k = (sub * 32 + lane) * 16; k < p.K; k += wk * 512) {
    int4 wv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) wv[r] = ld_weights(w[r] + k);
    const int4 x = __ldg(reinterpret_cast<const int4*>(a + k));
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = dot16(wv[r], x, acc[r]);
  }
  __syncwarp();
  int mine = 0;  // lane r: channel r
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int sum = __reduce_add_sync(0xffffffffu, acc[r]);
    if (lane == r) mine = sum;
  }
  if (wk > 1) {
    if (lane < R) part[warp][lane] = mine;
    __syncthreads();
    if (sub != 0) return;
    mine = 0;
    if (lane < R)
      for (int k = 0; k < wk; ++k) mine += part[warp + k][lane];
  }
  const int64_t n = n0 + lane;
  if (lane >= R || n >= p.N) return;
  I8Channel ch = {__ldg(p.b_scale + n), 0.f, 0.f};
  if (p.bias) ch.bias = __bfloat162float(p.bias[n]);
  if (p.gate) ch.gate = __ldg(p.gate + n);
  store_value(p, ch, mine, __ldg(p.a_scale), 0, static_cast<int>(n));
}

cudaError_t launch_one(const int8_t* a, const int8_t* b, const GemmI8Params& p, cudaStream_t s) {
  // Warps per group of channels: as many as leave the launch at 21 warps a SM, about one wave.
  const int64_t groups = (static_cast<int64_t>(p.N) + kOneRows - 1) / kOneRows;
  int wk = 1;
  while (wk < kOneWarps && groups * wk * 2 <= static_cast<int64_t>(num_sms()) * 21 && p.K > 512 * wk) wk *= 2;
  gemm_i8_one_kernel<<<static_cast<unsigned>((groups * wk + kOneWarps - 1) / kOneWarps), kOneThreads, 0, s>>>(a, b, p, wk);
  return cudaGetLastError();
}

// ------------------------------------------------------------------------ CTA pairs
constexpr int kPairThreads = 352;    // warp 0 TMA, warp 1 MMA, warps 2..9 epilogue, warp 10 hands the loads on

constexpr int kPairStages = 7;
constexpr int kPairOpBytes = 128 * kBK;                 // one operand's rows of one CTA in a slot
constexpr int kPairStageBytes = 2 * kPairOpBytes;       // 32 KB
constexpr int kPairSmemBytes = kPairStages * kPairStageBytes + 1024 + 256;
static_assert(kPairSmemBytes <= 227 * 1024, "shared memory");
constexpr int kPairGroupM = 16;      // M-tiles per band of the tile order

// The warp that waits for the loads and the one that issues the products meet slot by slot at named barrier 1,
// where both wait; the former says whether a slot failed to fill.
__device__ __forceinline__ void meet_announcing(bool failed) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %0, 0;\n\t"
      "bar.red.or.pred q, 1, 64, p;\n\t}" ::"r"(static_cast<uint32_t>(failed))
      : "memory");
}
// The other side: whether the slot is filled.  The calling thread with `issue` set multiplies it (w, x: the
// slot's descriptors, 32 bytes of K = 2 further each) before the answer is there, which takes longer than the barrier
// (9216 x 9216 x 3072: 162.4 us, 166.7 with the products behind the answer, in turn).  Products of a slot that failed
// to fill read what lies there; nothing takes their sums.
__device__ __forceinline__ bool meet_and_multiply(uint32_t d_tmem, uint64_t w, uint64_t x, uint32_t idesc,
                                                  uint32_t accumulate, bool issue) {
  uint32_t failed;
  asm volatile(
      "{\n\t.reg .pred none, failed, issue, acc;\n\t"
      "setp.ne.u32 none, 0, 0;\n\t"
      "setp.ne.u32 issue, %6, 0;\n\t"
      "setp.ne.u32 acc, %5, 0;\n\t"
      "bar.red.or.pred failed, 1, 64, none;\n\t"
      "tcgen05.fence::after_thread_sync;\n\t"
      "@issue tcgen05.mma.cta_group::2.kind::i8 [%1], %2, %3, %4, acc;\n\t"
      "setp.eq.u32 acc, 0, 0;\n\t"
      "@issue tcgen05.mma.cta_group::2.kind::i8 [%1], %7, %8, %4, acc;\n\t"
      "@issue tcgen05.mma.cta_group::2.kind::i8 [%1], %9, %10, %4, acc;\n\t"
      "@issue tcgen05.mma.cta_group::2.kind::i8 [%1], %11, %12, %4, acc;\n\t"
      "selp.u32 %0, 1, 0, failed;\n\t}"
      : "=r"(failed)
      : "r"(d_tmem), "l"(w), "l"(x), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(issue)), "l"(w + 2),
        "l"(x + 2), "l"(w + 4), "l"(x + 4), "l"(w + 6), "l"(x + 6)
      : "memory");
  return failed == 0;
}
static_assert(kBK / 32 == 4, "meet_and_multiply issues the products of one slot");

__device__ __forceinline__ void pair_tile(int tile, int num_m, int num_n, int& mb, int& nb) {
  const int band = tile / (kPairGroupM * num_n);
  const int m0 = band * kPairGroupM;
  const int bm = min(kPairGroupM, num_m - m0);
  const int idx = tile - band * kPairGroupM * num_n;
  mb = m0 + idx % bm;
  nb = idx / bm;
}

// The outputs of one channel for 32 tokens from m on, `tokens` of them inside C.
template <bool RESID, bool BF16OUT>
__device__ __forceinline__ void store_channel32(const GemmI8Params& p, const uint32_t (&acc)[32], const I8Channel& ch,
                                                int m, int tokens, int n) {
  const int64_t at = static_cast<int64_t>(m) * p.N + n;
  float res[32];
  if constexpr (RESID) {
#pragma unroll
    for (int i = 0; i < 32; ++i) res[i] = i < tokens ? p.residual[at + static_cast<int64_t>(i) * p.N] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (i >= tokens) continue;
    float v = fmaf(__int2float_rn(static_cast<int>(acc[i])) * __ldg(p.a_scale + m + i), ch.scale, ch.bias);
    if constexpr (RESID) v = fmaf(ch.gate, v, res[i]);
    if constexpr (BF16OUT)
      static_cast<bf16*>(p.c)[at + static_cast<int64_t>(i) * p.N] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(p.c)[at + static_cast<int64_t>(i) * p.N] = v;
  }
}

template <bool RESID, bool BF16OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    gemm_i8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const GemmI8Params p, unsigned* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sX = smem + kPairStages * kPairOpBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairStages * kPairStageBytes);
  uint64_t* empty = full + kPairStages;
  uint64_t* tfull = empty + kPairStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* peer_issued = abort_flag + 1;  // even CTA: slots that the odd one's producer has loaded in all

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: issues the MMAs, 1: its peer
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1;
  const int num_pairs = gridDim.x >> 1;
  const int num_m = pieces(p.M, 256);
  const int num_n = pieces(p.N, 256);
  const int num_tiles = num_m * num_n;
  const int num_kb = pieces(p.K, kBK);
  const int pair_slots = (num_tiles - pair + num_pairs - 1) / num_pairs * num_kb;  // of all the pair's tiles

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 16);  // eight epilogue warps of each CTA (used in the even CTA)
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised and their TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  int issued = 0;  // thread 0: slots loaded

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int armed[kPairStages];  // leader: parity of the last phase armed on full[s], -1 = never
#pragma unroll
      for (int s = 0; s < kPairStages; ++s) armed[s] = -1;
      for (int tile = pair; tile < num_tiles && ok; tile += num_pairs) {
        int mb, nb;
        pair_tile(tile, num_m, num_n, mb, nb);
        const int wrow = nb * 256 + static_cast<int>(rank) * 128, xrow = mb * 256 + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, err, kErrGemmI8Producer, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t full_leader = mapa_shared(smem_u32(&full[stage]), 0);
          if (leader) {
            armed[stage] = static_cast<int>(phase);
            mbar_arrive_expect_tx(&full[stage], 2 * kPairStageBytes);
          }
          if (p.selftest != kI8SelftestPairLoad || blockIdx.x != 0 || issued != 3)
            tma_load_2d_pair(sW + stage * kPairOpBytes, &tmW, full_leader, kb * kBK, wrow);
          tma_load_2d_pair(sX + stage * kPairOpBytes, &tmX, full_leader, kb * kBK, xrow);
          ++issued;
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (leader) drain_loads<kPairStages>(full, armed);
    }
  } else if (warp == 1) {
    if (leader) {
      // The warp learns of a filled slot by a named barrier, from warp 10: a poll of an mbarrier behind
      // queued MMAs holds up the next ones (171.8 us for 9216 x 9216 x 3072, 181.9 with polls here).  Both wait
      // at that barrier, and both go through every slot also after a failed wait, so neither can meet it twice
      // without the other.  From a slot that failed to fill on, no slot and no accumulator is handed on: the
      // producers of both CTAs come to rest, and no epilogue takes the sums.
      constexpr uint32_t kIdesc = idesc_i8(256, 256);
      int stage = 0;
      bool ok = true;
      int it = 0;
      for (int tile = pair; tile < num_tiles; tile += num_pairs, ++it) {
        const int acc = it & 1;
        if (lane == 0 && ok) ok = mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1, err, kErrGemmI8Mma, abort_flag);
        __syncwarp();
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 256;
        for (int kb = 0; kb < num_kb; ++kb) {
          const uint64_t w0 = sdesc_sw128(smem_u32(sW + stage * kPairOpBytes), 16, 1024);
          const uint64_t x0 = sdesc_sw128(smem_u32(sX + stage * kPairOpBytes), 16, 1024);
          if (!meet_and_multiply(d_tmem, w0, x0, kIdesc, kb, lane == 0 && ok)) ok = false;
          if (lane == 0 && ok) tc_commit_pair_both(&empty[stage], 0x3);  // the slot in both CTAs
          __syncwarp();
          if (++stage == kPairStages) stage = 0;
        }
        if (lane == 0 && ok) tc_commit_pair_both(&tfull[acc], 0x3);  // both CTAs' epilogues
      }
      // Every MMA issued by this thread has completed once `drain` flips: only then may
      // either CTA release its TMEM, on the normal path and after an abort alike.
      if (lane == 0) {
        tc_commit_pair(drain);
        const uint32_t a = smem_u32(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
        }
      }
      __syncwarp();
    }
  } else if (warp == 10) {
    if (leader) {
      // A wait that gives up is recorded and raises the abort flag; the warps meet for its slot all the same.
      int stage = 0;
      uint32_t phase = 0;
      bool failed = false;
      for (int i = 0; i < pair_slots; ++i) {
        if (lane == 0 && !mbar_wait(&full[stage], phase, err, kErrGemmI8Mma, abort_flag)) failed = true;
        __syncwarp();
        meet_announcing(failed);
        if (++stage == kPairStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else {
    const int quad = warp & 3;          // TMEM lane quadrant this warp may access
    const int half = (warp - 2) >> 2;   // which half of the tile's tokens it owns
    int it = 0;
    for (int tile = pair; tile < num_tiles; tile += num_pairs, ++it) {
      int mb, nb;
      pair_tile(tile, num_m, num_n, mb, nb);
      const int acc = it & 1;
      const int n = nb * 256 + static_cast<int>(rank) * 128 + quad * 32 + lane;  // the thread's channel
      const int m0 = mb * 256 + half * 128;
      // Operands of the epilogue that do not depend on the accumulator are fetched first.
      I8Channel ch = {0.f, 0.f, 0.f};
      if (n < p.N) {
        ch.scale = __ldg(p.b_scale + n);
        if (p.bias) ch.bias = __bfloat162float(p.bias[n]);
        if constexpr (RESID) ch.gate = __ldg(p.gate + n);
      }
      const bool ok = mbar_wait(&tfull[acc], (it >> 1) & 1, err, kErrGemmI8Epilogue, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;  // warp-uniform: TMEM loads are .sync.aligned
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256 + half * 128;
#pragma unroll 1
      for (int c = 0; c < 128 && m0 + c < p.M; c += 32) {
        uint32_t v[32];
        tmem_ld32(tb + c, v);
        const int tokens = p.M - m0 - c;
        if (n < p.N) {
          if (tokens >= 32)
            store_channel32<RESID, BF16OUT>(p, v, ch, m0 + c, 32, n);
          else
            store_channel32<RESID, BF16OUT>(p, v, ch, m0 + c, tokens, n);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && (p.selftest != kI8SelftestPairAccumulator || blockIdx.x != 0 || warp != 2)) {
        if (leader)
          mbar_arrive(&tempty[acc]);
        else
          mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) st_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1), 1);
  cluster_sync();  // the even CTA's MMAs into both TMEMs are complete (drained above)
  if (*abort_flag) {  // in either CTA, and now in both
    // The odd CTA may have loaded slots that the even one's producer, which stopped first, never armed (at
    // most one turn of them, since no slot was given back after that).  They are armed with the odd CTA's
    // bytes alone and waited for, so that no copy is in flight when a CTA exits.
    if (!leader && threadIdx.x == 0) st_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(peer_issued)), 0), issued);
    __syncwarp();
    cluster_sync();
    if (leader && threadIdx.x == 0) {
      const uint64_t t0 = globaltimer_ns();
      for (int i = issued; i < *peer_issued; ++i) {
        uint64_t* bar = &full[i % kPairStages];
        mbar_arrive_expect_tx(bar, kPairStageBytes);
        while (!mbar_try_wait(smem_u32(bar), (i / kPairStages) & 1) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
        }
      }
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <bool RESID, bool BF16OUT>
cudaError_t launch_pair(const int8_t* a, const int8_t* b, const GemmI8Params& p, cudaStream_t s, unsigned* err,
                        std::string* emsg) {
  static std::atomic<uint64_t> configured{0};
  if (!configured_on_device(configured)) {
    cudaError_t e = cudaFuncSetAttribute(gemm_i8_pair_kernel<RESID, BF16OUT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmemBytes);
    if (e != cudaSuccess) return e;
    mark_configured_on_device(configured);
  }
  CUtensorMap tw, tx;
  if (!make_tmap_i8_2d(&tw, b, p.K, p.N, kBK, 128, emsg) || !make_tmap_i8_2d(&tx, a, p.K, p.M, kBK, 128, emsg))
    return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>(pieces(p.M, 256)) * pieces(p.N, 256);
  const int pairs = static_cast<int>(tiles < num_sms() / 2 ? tiles : num_sms() / 2);
  gemm_i8_pair_kernel<RESID, BF16OUT><<<2 * pairs, kPairThreads, kPairSmemBytes, s>>>(tw, tx, p, err);
  return cudaGetLastError();
}

}  // namespace

// Which kernel, measured on a B200 (us; N x K of the weights):
//   1 token       one    3072 x 8192 6.3 (few 7.6), 16384 x 3072 10.2 (few 11.6)
//   2..16         few    8 x 9216 x 3072 7.3 (flat 10.2); from 9 tokens on only up to 8192 channels, since every
//                        warp reads the tokens again: 16 x 3072 x 3072 5.6 (flat 8.2), 16 x 16384 x 3072 17 (12.8)
//   one wave of   flat   256 x 3072 x 3072 11.4 (pairs 13.9), 64 x 9216 x 3072 10.8 (12.5); K split while the CTAs stay
//   tiles or less        one wave: 77 x 3072 x 4096 14.0 / 11.9 / 10.1 / 17.9 for 1 / 2 / 4 / 8 parts (24 to 192 CTAs), 9.6 to 10.1 now for 4
//   more tiles    pairs  512 x 9216 x 3072 16 (flat 25.6), 128 x 32768 x 3072 23.8 (29.9), 20 x 20480 x 3072 22.5 (21.6)
cudaError_t launch_gemm_i8(const int8_t* a, const int8_t* b, const GemmI8Params& p, cudaStream_t s, unsigned* err,
                           std::string* emsg) {
  if (p.M == 1) return launch_one(a, b, p, s);
  if (p.M <= 8) return launch_few<1>(a, b, p, s);
  if (p.M <= 16 && p.N <= 8192) return launch_few<2>(a, b, p, s);
  const int nt = p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
  const int64_t tiles = static_cast<int64_t>(pieces(p.N, kTileN)) * pieces(p.M, nt);
  if (tiles > num_sms()) {
    if (p.residual) return launch_pair<true, false>(a, b, p, s, err, emsg);
    return p.c_bf16 ? launch_pair<false, true>(a, b, p, s, err, emsg) : launch_pair<false, false>(a, b, p, s, err, emsg);
  }
  const int num_kb = pieces(p.K, kBK);
  int split = 1;
  while (split < kMaxSplit && tiles * split * 2 <= num_sms() && split * 2 <= num_kb) split *= 2;
  return launch_flat_nt(nt, a, b, p, split, s, err, emsg);
}

// Flat kernel: the rule above, a wave of tiles; pairs: three tiles or more for the first pair.
bool gemm_i8_selftest_reaches(int kind, int M, int N, int K) {
  if (M <= 16 || K < 256) return false;
  const int nt = M <= 32 ? 32 : M <= 64 ? 64 : 128;
  if (kind == kI8SelftestFlatLoad)
    return static_cast<int64_t>(pieces(N, kTileN)) * pieces(M, nt) <= num_sms();
  return static_cast<int64_t>(pieces(N, 256)) * pieces(M, 256) > num_sms() / 2 * 2;
}

}  // namespace moss
