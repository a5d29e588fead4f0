// latent_mma.cuh -- pieces that the latent attention kernels share: the plan's prefix sum and the
// blocks' shares, and tensor-core helpers whose operands stay in uniform registers.
#pragma once

#include <cfloat>
#include <cmath>

#include "common.cuh"

namespace dsa {

constexpr int kPlanThreads = 1024;

// Inclusive prefix sum over the block's 1,024 threads (all of them call it).
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t s = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  return v + (warp ? warp_sums[warp - 1] : 0);
}

// The tiles [a, b) of a block's share, and the block whose share holds tile x.
__device__ __forceinline__ void share(int64_t tiles, int block, int blocks, int64_t* a, int64_t* b) {
  *a = tiles * block / blocks;
  *b = tiles * (block + 1) / blocks;
}
__device__ __forceinline__ int share_of(int64_t tiles, int64_t x, int blocks) {
  return static_cast<int>(((x + 1) * blocks - 1) / tiles);
}

// Shared-memory operand descriptors, 128-byte swizzle, 1,024 bytes from 8 rows to the next 8.  The
// low word holds the address and the leading offset: for a K-major operand (rows along M/N, 64
// values of K per 128-byte row) the latter is not used; for an MN-major one (rows along K, 64
// values along M/N) it is the distance to the next 64 values.  Addresses stay below 2^18, so the
// low word is advanced by plain additions of bytes / 16.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3FFFu) | ((lead >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x;\n\t"
      "elect.sync x|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// D (+)= A . B by the elected lane
__device__ __forceinline__ void umma_lo(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate,
                                        bool leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)leader)
      : "memory");
}

// fetch of `bytes` (a multiple of 16) from a 16-byte aligned address into L2
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// position in a ring of N stages and the parity of its full barriers
template <int N>
struct Ring {
  uint32_t s = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ float ex2_approx(float x) {   // relative error near 2^-22; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// 16 consecutive fp32 columns of the warp's TMEM lanes, and the wait for them
__device__ __forceinline__ void tmem_ld16(uint32_t a, float (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]),
        "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
      : "r"(a)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t a, const float (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(a),
      "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "f"(x[8]), "f"(x[9]),
      "f"(x[10]), "f"(x[11]), "f"(x[12]), "f"(x[13]), "f"(x[14]), "f"(x[15])
      : "memory");
}

// kind::f16 with fp16 A and B, fp32 accumulator, both K-major
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// 2^e, e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Exponent f of the scale 2^f that brings a largest magnitude of `top` to between 2^14 and 2^15,
// where fp16 holds it and what lies up to 2^28 below it in full; magnitudes below 2^lowest are
// lifted no further.
__device__ __forceinline__ int scale_exponent(float top, int lowest) {
  const int e = static_cast<int>((__float_as_uint(top) >> 23) & 0xFF) - 127;
  return (e < lowest ? lowest : e) - 14;
}
// Of queries and keys: lifted as far as pow2(-f) reaches.  Of values: the weights take the scale over,
// so those of one row's tiles must stay within fp32 of each other.
constexpr int kLowestFactor = -106, kLowestValue = -60;

// scale * log2(e) as m * 2^e, m in [1, 2): the factor of a score whose query and key were scaled by
// 2^f in all is m * 2^(e + f).  The exponents are summed first, since 2^-120 of a zero query times
// 2^-120 of a zero key is 0 in fp32, and a masked score of -inf times 0 is NaN.  Held at -126 below:
// scaled products stay under 2^38, so such scores are 0 to fp32 either way.
struct ScoreScale {
  float m;
  int e;
};
inline ScoreScale score_scale(float scale_log2) {
  ScoreScale s;
  s.m = 2.f * frexpf(scale_log2, &s.e);
  --s.e;
  return s;
}
// finite, so that a score of 0 stays 0
inline float scale_to_log2(float scale) { return fminf(scale * 1.4426950408889634f, FLT_MAX); }
__device__ __forceinline__ float score_factor(ScoreScale s, int f) {
  const int e = s.e + f;
  return s.m * pow2(e < -126 ? -126 : e > 127 ? 127 : e);
}

}  // namespace dsa
