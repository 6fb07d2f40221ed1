// Device-side additions of the 8-bit operators to the building blocks of common.cuh: error codes, the
// integer forms of tcgen05.mma, a narrow TMEM load and the two halves of a cluster barrier.
#pragma once

#include "common.cuh"

namespace moss {

// Error codes written to the device error word, beside those of common.cuh.
enum : unsigned {
  kErrGemmI8Producer = 0x111, kErrGemmI8Mma = 0x112, kErrGemmI8Epilogue = 0x113,
  kErrQkPosition = 0x401,  // a token's position lies outside the angle table (no wait gave up)
};

// D(tmem) (+)= A(smem desc) * B(smem desc), kind::i8: signed 8-bit integers, 32-bit integer sums.  K = 32 an
// instruction, so an operand's 32 bytes of K lie where kind::f16 has them.
__device__ __forceinline__ void mma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::i8: D format 2 = S32, A and B format 1 = signed 8 bits, both
// K-major; no saturation (the sums are exact).
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 lanes x 16 columns of 32-bit TMEM words (thread = lane), waiting for completion.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// The two halves of cluster_sync, for work between them.  Both want the whole warp converged.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace moss
