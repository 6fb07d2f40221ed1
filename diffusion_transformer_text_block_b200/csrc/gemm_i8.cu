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
// `gemm_i8_flat_kernel`: one CTA per tile of 128 output channels and NT tokens.  The weights are the
// 128-row operand of tcgen05.mma (kind::i8, 128 x NT x 32), so few tokens make a narrow tile and not
// an empty one, and a thread of the epilogue holds one channel: a warp stores 32 neighbouring
// channels of a token.  The K axis of a tile is split over the CTAs of a cluster; their partial
// sums meet in shared memory of the cluster (integers: the order does not matter).
//   warp 0      TMA producer: 128 x 128 bytes of B and NT x 128 bytes of A per slot (128-byte swizzle)
//   warp 1      MMA issuer, four 32-deep steps a slot
//   warps 2..5  epilogue (one per TMEM lane quadrant)
#include "common.cuh"
#include "internal.h"

namespace moss {

namespace {

constexpr int kBK = 128;      // K bytes (= elements) per slot, one 128-byte swizzle row
constexpr int kTileN = 128;   // output channels per tile
constexpr int kFlatThreads = 192;
constexpr int kMaxSplit = 8;  // portable cluster size
static_assert(static_cast<int64_t>(kMaxI8K) * 128 * 128 <= (int64_t{1} << 30), "32-bit sums are exact");

template <int NT>
struct FlatShape {
  static constexpr int kWBytes = kTileN * kBK;
  static constexpr int kXBytes = NT * kBK;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kStages = (208 * 1024) / kStageBytes < 8 ? (208 * 1024) / kStageBytes : 8;
  static constexpr int kPartBytes = kTileN * NT * 4;  // partial sums of a tile, in the slots' place
  static constexpr int kTmemCols = NT < 32 ? 32 : NT;
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024 + 256;
  static_assert(kPartBytes <= kStages * kStageBytes, "partial sums fit the slots");
  static_assert(kStageBytes % 1024 == 0 && kSmemBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
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
__device__ __forceinline__ void store_value(const GemmI8Params& p, const I8Channel& ch, int acc, int m, int n) {
  float v = fmaf(__int2float_rn(acc) * __ldg(p.a_scale + m), ch.scale, ch.bias);
  const int64_t at = static_cast<int64_t>(m) * p.N + n;
  if (p.residual) v = fmaf(ch.gate, v, p.residual[at]);
  if (p.c_bf16)
    static_cast<bf16*>(p.c)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p.c)[at] = v;
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
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kStages * S::kStageBytes);
  uint64_t* empty = full + S::kStages;
  uint64_t* tfull = empty + S::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int num_n = (p.N + kTileN - 1) / kTileN;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int n0 = (tile % num_n) * kTileN;
  const int m0 = (tile / num_n) * NT;
  const int num_kb = (p.K + kBK - 1) / kBK;
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
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

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
    ok = mbar_wait(tfull, 0, err, kErrGemmI8Epilogue, abort_flag) && !*abort_flag;
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
  }
  if (split == 1) {
    if (epi && ok) {
#pragma unroll 1
      for (int c = 0; c < NT && m0 + c < p.M; c += 16) {
        uint32_t v[16];
        tmem_ld16(tb + c, v);
        if (n < p.N) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (m0 + c + i < p.M) store_value(p, ch, static_cast<int>(v[i]), m0 + c + i, n);
        }
      }
    }
  } else {
    // Every CTA of the cluster lays its partial sums out as [token][channel], then finishes its
    // share of the tokens.  The slots are free: all loads of this CTA fed MMAs that have completed.
    uint32_t* part = reinterpret_cast<uint32_t*>(smem);
    const int tokens = min(NT, p.M - m0);
    if (epi && ok) {
#pragma unroll 1
      for (int c = 0; c < tokens; c += 16) {
        uint32_t v[16];
        tmem_ld16(tb + c, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kTileN + ln] = v[i];
      }
    }
    __syncwarp();
    cluster_sync();
    if (epi && ok && n < p.N) {
      const int c0 = tokens * rank / split, c1 = tokens * (rank + 1) / split;
      for (int c = c0; c < c1; ++c) {
        const uint32_t at = smem_u32(part + c * kTileN + ln);
        uint32_t sum = 0;
        for (int r = 0; r < split; ++r) sum += ld_cluster_u32(mapa_shared(at, r));
        store_value(p, ch, static_cast<int>(sum), m0 + c, n);
      }
    }
    __syncwarp();
    cluster_sync();  // the peers have read this CTA's shared memory
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
  const int64_t tiles = static_cast<int64_t>((p.N + kTileN - 1) / kTileN) * ((p.M + NT - 1) / NT);
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

// ------------------------------------------------------------------------ CTA pairs
constexpr int kPairThreads = 320;    // warp 0 TMA, warp 1 MMA, warps 2..9 epilogue
constexpr int kPairStages = 6;
constexpr int kPairOpBytes = 128 * kBK;                 // one operand's rows of one CTA in a slot
constexpr int kPairStageBytes = 2 * kPairOpBytes;       // 32 KB
constexpr int kPairColBytes = 8 * 3 * 128 * 4;          // per epilogue warp: scale, bias, gate of its 128 columns
constexpr int kPairSmemBytes = kPairStages * kPairStageBytes + kPairColBytes + 1024 + 256;
static_assert(kPairSmemBytes <= 227 * 1024, "shared memory");
constexpr int kPairGroupM = 16;      // M-tiles per band of the tile order

__device__ __forceinline__ void pair_tile(int tile, int num_m, int num_n, int& mb, int& nb) {
  const int band = tile / (kPairGroupM * num_n);
  const int m0 = band * kPairGroupM;
  const int bm = min(kPairGroupM, num_m - m0);
  const int idx = tile - band * kPairGroupM * num_n;
  mb = m0 + idx % bm;
  nb = idx / bm;
}

// 32 neighbouring outputs of one row.  cs: the columns' scale, bias and gate (128 floats apart) in
// shared memory, read by all lanes at once.
template <bool RESID, bool BF16OUT>
__device__ __forceinline__ void store_row32(const GemmI8Params& p, const uint32_t (&acc)[32], float sa, int row, int col,
                                            const float* cs, bool vec) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 sc = *reinterpret_cast<const float4*>(cs + 4 * i);
    const float4 bi = *reinterpret_cast<const float4*>(cs + 128 + 4 * i);
    v[4 * i] = fmaf(__int2float_rn(static_cast<int>(acc[4 * i])) * sa, sc.x, bi.x);
    v[4 * i + 1] = fmaf(__int2float_rn(static_cast<int>(acc[4 * i + 1])) * sa, sc.y, bi.y);
    v[4 * i + 2] = fmaf(__int2float_rn(static_cast<int>(acc[4 * i + 2])) * sa, sc.z, bi.z);
    v[4 * i + 3] = fmaf(__int2float_rn(static_cast<int>(acc[4 * i + 3])) * sa, sc.w, bi.w);
  }
  const int64_t at = static_cast<int64_t>(row) * p.N + col;
  if (vec) {
    if constexpr (RESID) {
      const float4* r = reinterpret_cast<const float4*>(p.residual + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = r[i];
        const float4 g = *reinterpret_cast<const float4*>(cs + 256 + 4 * i);
        v[4 * i] = fmaf(g.x, v[4 * i], x.x);
        v[4 * i + 1] = fmaf(g.y, v[4 * i + 1], x.y);
        v[4 * i + 2] = fmaf(g.z, v[4 * i + 2], x.z);
        v[4 * i + 3] = fmaf(g.w, v[4 * i + 3], x.w);
      }
    }
    if constexpr (BF16OUT) {
      uint4* d = reinterpret_cast<uint4*>(static_cast<bf16*>(p.c) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                          pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
    } else {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.c) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (col + i >= p.N) continue;
      float y = v[i];
      if constexpr (RESID) y = fmaf(cs[256 + i], y, p.residual[at + i]);
      if constexpr (BF16OUT)
        static_cast<bf16*>(p.c)[at + i] = __float2bfloat16_rn(y);
      else
        static_cast<float*>(p.c)[at + i] = y;
    }
  }
}

template <bool RESID, bool BF16OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    gemm_i8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const GemmI8Params p, unsigned* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kPairStages * kPairOpBytes;
  float* sCol = reinterpret_cast<float*>(smem + kPairStages * kPairStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairStages * kPairStageBytes + kPairColBytes);
  uint64_t* empty = full + kPairStages;
  uint64_t* tfull = empty + kPairStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: issues the MMAs, 1: its peer
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1;
  const int num_pairs = gridDim.x >> 1;
  const int num_m = (p.M + 255) / 256;
  const int num_n = (p.N + 255) / 256;
  const int num_tiles = num_m * num_n;
  const int num_kb = (p.K + kBK - 1) / kBK;

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
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
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
        const int arow = mb * 256 + static_cast<int>(rank) * 128, brow = nb * 256 + static_cast<int>(rank) * 128;
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
          tma_load_2d_pair(sA + stage * kPairOpBytes, &tmA, full_leader, kb * kBK, arow);
          tma_load_2d_pair(sB + stage * kPairOpBytes, &tmB, full_leader, kb * kBK, brow);
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (leader) drain_loads<kPairStages>(full, armed);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      constexpr uint32_t kIdesc = idesc_i8(256, 256);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int it = 0;
      for (int tile = pair; tile < num_tiles && ok; tile += num_pairs, ++it) {
        const int acc = it & 1;
        if (!mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1, err, kErrGemmI8Mma, abort_flag)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 256;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait(&full[stage], phase, err, kErrGemmI8Mma, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + stage * kPairOpBytes);
          const uint32_t b0 = smem_u32(sB + stage * kPairOpBytes);
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            mma_i8_ss_pair(d_tmem, sdesc_sw128(a0 + k * 32, 16, 1024), sdesc_sw128(b0 + k * 32, 16, 1024), kIdesc,
                           (kb | k) != 0 ? 1u : 0u);
          tc_commit_pair_both(&empty[stage], 0x3);  // the slot in both CTAs
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok) tc_commit_pair_both(&tfull[acc], 0x3);  // both CTAs' epilogues
      }
      // Every MMA issued by this thread has completed once `drain` flips: only then may
      // either CTA release its TMEM, on the normal path and after an abort alike.
      tc_commit_pair(drain);
      const uint32_t a = smem_u32(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
  } else {
    const int quad = warp & 3;          // TMEM lane quadrant this warp may access
    const int half = (warp - 2) >> 2;   // which half of the tile's columns it owns
    float* cs = sCol + (warp - 2) * 384;
    const bool rows16 = p.N % (BF16OUT ? 8 : 4) == 0;  // rows of C start on 16 bytes
    int it = 0;
    for (int tile = pair; tile < num_tiles; tile += num_pairs, ++it) {
      int mb, nb;
      pair_tile(tile, num_m, num_n, mb, nb);
      const int acc = it & 1;
      const int row = mb * 256 + static_cast<int>(rank) * 128 + quad * 32 + lane;
      const int col0 = nb * 256 + half * 128;
      // Operands of the epilogue that do not depend on the accumulator are fetched first.
      const float sa = row < p.M ? __ldg(p.a_scale + row) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = lane + 32 * i, n = col0 + c;
        const bool in = n < p.N;
        cs[c] = in ? __ldg(p.b_scale + n) : 0.f;
        cs[128 + c] = in && p.bias ? __bfloat162float(p.bias[n]) : 0.f;
        if constexpr (RESID) cs[256 + c] = in ? __ldg(p.gate + n) : 0.f;
      }
      __syncwarp();
      const bool ok = mbar_wait(&tfull[acc], (it >> 1) & 1, err, kErrGemmI8Epilogue, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;  // warp-uniform: TMEM loads are .sync.aligned
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256 + half * 128;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        if (col0 + c >= p.N) break;  // warp-uniform
        uint32_t v[32];
        tmem_ld32(tb + c, v);
        if (row < p.M) store_row32<RESID, BF16OUT>(p, v, sa, row, col0 + c, cs + c, rows16 && col0 + c + 32 <= p.N);
      }
      tc_fence_before();
      __syncwarp();  // also: every lane is done with cs before the next tile's columns overwrite it
      if (lane == 0) {
        if (leader)
          mbar_arrive(&tempty[acc]);
        else
          mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the even CTA's MMAs into both TMEMs are complete (drained above)
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
  CUtensorMap ta, tb;
  if (!make_tmap_i8_2d(&ta, a, p.K, p.M, kBK, 128, emsg) || !make_tmap_i8_2d(&tb, b, p.K, p.N, kBK, 128, emsg))
    return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>((p.M + 255) / 256) * ((p.N + 255) / 256);
  const int pairs = static_cast<int>(tiles < num_sms() / 2 ? tiles : num_sms() / 2);
  gemm_i8_pair_kernel<RESID, BF16OUT><<<2 * pairs, kPairThreads, kPairSmemBytes, s>>>(ta, tb, p, err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_i8(const int8_t* a, const int8_t* b, const GemmI8Params& p, cudaStream_t s, unsigned* err,
                           std::string* emsg) {
  if (p.M > 256) {
    if (p.residual) return launch_pair<true, false>(a, b, p, s, err, emsg);
    return p.c_bf16 ? launch_pair<false, true>(a, b, p, s, err, emsg) : launch_pair<false, false>(a, b, p, s, err, emsg);
  }
  const int nt = p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : p.M <= 128 ? 128 : 256;
  const int64_t tiles = static_cast<int64_t>((p.N + kTileN - 1) / kTileN) * ((p.M + nt - 1) / nt);
  const int num_kb = (p.K + kBK - 1) / kBK;
  int split = 1;
  while (split < kMaxSplit && tiles * (split + 1) <= num_sms() && split + 1 <= num_kb) ++split;
  switch (nt) {
    case 16: return launch_flat<16>(a, b, p, split, s, err, emsg);
    case 32: return launch_flat<32>(a, b, p, split, s, err, emsg);
    case 64: return launch_flat<64>(a, b, p, split, s, err, emsg);
    case 128: return launch_flat<128>(a, b, p, split, s, err, emsg);
    default: return launch_flat<256>(a, b, p, split, s, err, emsg);
  }
}

}  // namespace moss
