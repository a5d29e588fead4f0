// latent_attention.cu -- dense (and, over a 4-bit cache, selected) attention in the absorbed
// form of multi-head latent attention.
//
//   x[t,h,s] = scale * (q[t,h] . c[s])  over the 576 cached values,
//   out[t,h] = sum_s softmax_s(x) * c[s][0..511],   lse[t,h] = ln sum_s exp(x[t,h,s]).
//
// First form: one warp per (token, head), an online softmax over the tokens it attends to.

#include "latent.h"

namespace dsa {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Are the offsets well formed?  (q_seq_offsets within [0, T] and non-decreasing, cache_offsets
// within [0, cache_rows] and non-decreasing)
__global__ void check_offsets_kernel(LatentArgs a, int* bad) {
  int b_bad = 0;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const int64_t q0 = a.q_seq_offsets[b], q1 = a.q_seq_offsets[b + 1];
    const int64_t c0 = a.cache_offsets[b], c1 = a.cache_offsets[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.T || c0 < 0 || c1 < c0 || c1 > a.cache_rows) b_bad = 1;
  }
  b_bad = __syncthreads_or(b_bad);
  if (threadIdx.x == 0) {
    *bad = b_bad;
    if (b_bad) atomicOr(a.err, kErrOffsets);
  }
}

__global__ void __launch_bounds__(kWarps * 32) latent_simple_kernel(LatentArgs a, const int* bad) {
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (r >= static_cast<int64_t>(a.T) * a.H) return;
  const int t = static_cast<int>(r / a.H);
  int64_t row0 = 0, len = 0;
  int n = 0;
  if (!*bad) {
    if (t < a.q_seq_offsets[0] || t >= a.q_seq_offsets[a.B]) return;   // a token of no sequence
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.q_seq_offsets[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    row0 = a.cache_offsets[lo];
    len = a.cache_offsets[lo + 1] - row0;
    if (a.k_sel >= 0) {
      n = a.k_sel;
    } else {
      const int p = a.positions[t];
      if (p >= -1 && p < len) n = p + 1;
      else if (lane == 0) atomicOr(a.err, kErrBounds);
    }
  }
  // lane l: latent values 16 l .. 16 l + 15 and rope values 2 l, 2 l + 1
  const uint4* qs = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + r * kLatDim);
  float q[18], o[16];
  {
    const uint4 u0 = qs[2 * lane], u1 = qs[2 * lane + 1];
    const uint32_t w[9] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w,
                           reinterpret_cast<const uint32_t*>(qs)[kLatV / 2 + lane]};
#pragma unroll
    for (int k = 0; k < 9; ++k) q[2 * k] = bf_lo(w[k]), q[2 * k + 1] = bf_hi(w[k]);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    int64_t pos = j;
    if (a.k_sel >= 0) {
      pos = a.idx[static_cast<int64_t>(t) * a.k_sel + j];
      if (pos >= len && lane == 0) atomicOr(a.err, kErrBounds);
      if (pos < 0 || pos >= len) continue;
    }
    float c[18];
    if (a.fp4) {
      const uint8_t* src = static_cast<const uint8_t*>(a.kv) + (row0 + pos) * kLatRow4;
      const uint2 w = reinterpret_cast<const uint2*>(src)[lane];
      const uint32_t sc = src[kLatCodes + lane];
      const uint32_t e8 = (sc >> 3) & 15u;
      const float s = e8 ? __uint_as_float(((e8 + 120u) << 23) | ((sc & 7u) << 20)) : static_cast<float>(sc & 7u) * 0x1p-9f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint32_t nib = ((k < 8 ? w.x : w.y) >> (4 * (k & 7))) & 15u, e = (nib >> 1) & 3u;
        const float mag = e ? __uint_as_float(((e + 126u) << 23) | ((nib & 1u) << 22)) : 0.5f * static_cast<float>(nib & 1u);
        c[k] = (nib & 8u ? -mag : mag) * s;
      }
      const uint32_t rp = reinterpret_cast<const uint32_t*>(src + kLatCodes + kLatScales)[lane];
      c[16] = bf_lo(rp), c[17] = bf_hi(rp);
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.kv) + (row0 + pos) * kLatDim);
      const uint4 u0 = src[2 * lane], u1 = src[2 * lane + 1];
      const uint32_t w[9] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w,
                             reinterpret_cast<const uint32_t*>(src)[kLatV / 2 + lane]};
#pragma unroll
      for (int k = 0; k < 9; ++k) c[2 * k] = bf_lo(w[k]), c[2 * k + 1] = bf_hi(w[k]);
    }
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < 18; ++k) x = fmaf(q[k], c[k], x);
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= a.scale;
    const float mn = fmaxf(m, x);
    const float f = m == -INFINITY ? 0.f : __expf(m - mn);
    const float p = x == -INFINITY ? 0.f : __expf(x - mn);
    l = l * f + p;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = fmaf(o[k], f, p * c[k]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
    w[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + r * kLatV);
  dst[2 * lane] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[2 * lane + 1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (lane == 0) a.lse[r] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

int64_t latent_workspace_bytes(int64_t, int64_t, int64_t, int) { return 16; }

cudaError_t launch_latent_attention(const LatentArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  int* bad = static_cast<int*>(a.workspace);
  check_offsets_kernel<<<1, 256, 0, s>>>(a, bad);
  const int64_t rows = static_cast<int64_t>(a.T) * a.H;
  latent_simple_kernel<<<static_cast<unsigned>((rows + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a, bad);
  return cudaGetLastError();
}

}  // namespace dsa
