// latent_fp4.cu -- rows of the 4-bit latent cache.
//
// A row keeps the 512-value latent as e2m1 codes (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) in
// blocks of 16 that share one e4m3 scale, and the 64-value rope key in bf16 (its values turn
// with the position and are shared by all heads, so their rounding would enter every score):
//   s = e4m3(min(amax / 6, 448)),  code = e2m1(x / s) to nearest, ties to the even code,
//   saturating at 6; s = 0 (amax at or below 6 * 2^-10) stores zero codes.
// A code times its scale has at most 2 + 4 significant bits, so the value a row stands for is
// exact in bf16 and the attention that reads it adds no rounding of its own.
//
// Bytes: 1,152 read and 416 written a row; 8,191 rows take 5.8 us either way with cold caches (2.0
// at the copy rate), less than the host takes for the call.  The quotient is rounded without a division per
// value: x * (1/s) carries a relative error of at most 2^-23, and x/s (an 8-bit significand by
// a 4-bit one) is either a midpoint between two codes or at least 2^-10 away from it, so
// snapping the product to multiples of 2^-13 (adding and subtracting 1,024) puts every midpoint
// exactly on itself before the conversion rounds it to even.

#include "latent.h"

namespace dsa {
namespace {

constexpr int kFp4Warps = 8;

// 8 e2m1 codes (first value in the lowest nibble) of 8 values already divided by their scale
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// e4m3 code of a value in [0, 448]
__device__ __forceinline__ uint32_t e4m3_code(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  // s eeee mmm: exponent bias 7, subnormals m * 2^-9
  const uint32_t e = (c >> 3) & 15u, m = c & 7u;
  return e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : static_cast<float>(m) * 0x1p-9f;
}

// One warp per row: lane l holds block l of the latent (16 values, 32 bytes read) and two values
// of the rope key.
__global__ void __launch_bounds__(kFp4Warps * 32) quantize_latent_fp4_kernel(int64_t n, const uint4* __restrict__ kv,
                                                                             const int64_t* __restrict__ rows,
                                                                             uint8_t* __restrict__ out,
                                                                             int64_t out_rows, int* err) {
  const int lane = threadIdx.x & 31;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kFp4Warps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kFp4Warps + (threadIdx.x >> 5); i < n; i += nw) {
    const int64_t r = rows ? rows[i] : i;
    if (r < 0 || r >= out_rows) {
      if (lane == 0) atomicOr(err, kErrBounds);
      continue;
    }
    const uint4* src = kv + i * (kLatDim / 8);
    const uint4 a = src[2 * lane], b = src[2 * lane + 1];
    const uint32_t rope = reinterpret_cast<const uint32_t*>(src)[kLatV / 2 + lane];
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float v[16], amax = 0.f;
    uint32_t top = 0u;                    // magnitudes of bf16 pairs compare as integers, NaN the largest
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      top = __vmaxu2(top, u[k] & 0x7FFF7FFFu);
      v[2 * k] = bf_lo(u[k]);
      v[2 * k + 1] = bf_hi(u[k]);
      amax = fmaxf(amax, fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
    }
    // codes cannot hold what is not finite: the row is written all the same, and reported
    if ((top & 0x7F80u) == 0x7F80u || (top >> 23) == 0xFFu) atomicOr(err, kErrBounds);
    const uint32_t sc = e4m3_code(fminf(__fdiv_rn(amax, 6.f), 448.f));
    const float s = e4m3_value(sc);
    const float inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
    uint32_t w[2];
#pragma unroll
    for (int hlf = 0; hlf < 2; ++hlf) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float y = v[8 * hlf + k];
        // beyond 6 every code is 6, so the cap at 8 (which keeps the snap exact) changes nothing
        const float t = __fsub_rn(__fadd_rn(fminf(__fmul_rn(fabsf(y), inv), 8.f), 1024.f), 1024.f);
        x[k] = copysignf(t, y);
      }
      w[hlf] = s > 0.f ? pack_e2m1x8(x) : 0u;
    }
    uint8_t* dst = out + r * kLatRow4;
    reinterpret_cast<uint2*>(dst)[lane] = make_uint2(w[0], w[1]);
    dst[kLatCodes + lane] = static_cast<uint8_t>(sc);
    reinterpret_cast<uint32_t*>(dst + kLatCodes + kLatScales)[lane] = rope;
  }
}

__global__ void __launch_bounds__(kFp4Warps * 32) dequantize_latent_fp4_kernel(int64_t n, const uint8_t* __restrict__ kv4,
                                                                               int64_t kv_rows,
                                                                               const int64_t* __restrict__ rows,
                                                                               uint4* __restrict__ out, int* err) {
  const int lane = threadIdx.x & 31;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kFp4Warps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kFp4Warps + (threadIdx.x >> 5); i < n; i += nw) {
    const int64_t r = rows ? rows[i] : i;
    const bool ok = r >= 0 && r < kv_rows;
    if (!ok && lane == 0) atomicOr(err, kErrBounds);
    const uint8_t* src = kv4 + (ok ? r : 0) * kLatRow4;
    uint2 c = reinterpret_cast<const uint2*>(src)[lane];
    float s = e4m3_value(src[kLatCodes + lane]);
    uint32_t rope = reinterpret_cast<const uint32_t*>(src + kLatCodes + kLatScales)[lane];
    if (!ok) c = make_uint2(0u, 0u), s = 0.f, rope = 0u;   // a row that is not there reads as zeros
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t byte = ((k < 4 ? c.x : c.y) >> (8 * (k & 3))) & 0xFFu;
      float x[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t nib = (byte >> (4 * j)) & 15u, e = (nib >> 1) & 3u, m = nib & 1u;
        const float mag = e ? __uint_as_float(((e + 126u) << 23) | (m << 22)) : 0.5f * static_cast<float>(m);
        x[j] = (nib & 8u ? -mag : mag) * s;
      }
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[0], x[1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&p);
    }
    uint4* dst = out + i * (kLatDim / 8);
    dst[2 * lane] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[2 * lane + 1] = make_uint4(w[4], w[5], w[6], w[7]);
    reinterpret_cast<uint32_t*>(dst)[kLatV / 2 + lane] = rope;
  }
}

int fp4_grid(int64_t n, int num_sms) {
  const int64_t want = (n + kFp4Warps - 1) / kFp4Warps, most = static_cast<int64_t>(num_sms) * 8;
  return static_cast<int>(want < most ? want : most);
}

}  // namespace

cudaError_t launch_quantize_latent_fp4(int64_t n, const void* kv, const int64_t* rows, uint8_t* out, int64_t out_rows,
                                       int* err, int num_sms, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  quantize_latent_fp4_kernel<<<fp4_grid(n, num_sms), kFp4Warps * 32, 0, s>>>(n, static_cast<const uint4*>(kv), rows, out,
                                                                             out_rows, err);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_latent_fp4(int64_t n, const uint8_t* kv4, int64_t kv_rows, const int64_t* rows, void* out,
                                         int* err, int num_sms, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  dequantize_latent_fp4_kernel<<<fp4_grid(n, num_sms), kFp4Warps * 32, 0, s>>>(n, kv4, kv_rows, rows,
                                                                               static_cast<uint4*>(out), err);
  return cudaGetLastError();
}

}  // namespace dsa
