// latent_expanded.cu -- attention in the expanded form of multi-head latent attention, for
// prompts: keys of 128 + 64 values (the first 128 up-projected from the latent for each head,
// the last 64 the shared rope key) and values of 128, up-projected too.
//
//   x[t,h,s] = scale * (q[t,h][0..127] . k[s,h] + q[t,h][128..191] . c[s][512..575]),
//   out[t,h] = sum_s softmax_s(x) * v[s,h].
//
// First form: one warp per (token, head), an online softmax over the prefix.

#include "latent.h"

namespace dsa {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

__global__ void check_offsets_kernel(ExpandedArgs a, int* bad) {
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

__global__ void __launch_bounds__(kWarps * 32) expanded_simple_kernel(ExpandedArgs a, const int* bad) {
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (r >= static_cast<int64_t>(a.T) * a.H) return;
  const int t = static_cast<int>(r / a.H), h = static_cast<int>(r % a.H);
  int64_t row0 = 0;
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
    const int64_t len = a.cache_offsets[lo + 1] - row0;
    const int p = a.positions[t];
    if (p >= -1 && p < len) n = p + 1;
    else if (lane == 0) atomicOr(a.err, kErrBounds);
  }
  const uint32_t* qs = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + r * 192);
  const uint2 q0 = reinterpret_cast<const uint2*>(qs)[lane];
  const uint32_t q1 = qs[64 + lane];
  const float q[6] = {bf_lo(q0.x), bf_hi(q0.x), bf_lo(q0.y), bf_hi(q0.y), bf_lo(q1), bf_hi(q1)};
  float o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    const uint2* kr = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.kv_exp) +
                                                     ((row0 + j) * a.H + h) * 256);
    const uint2 k0 = kr[lane], v = kr[32 + lane];
    const uint32_t k1 = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.kv) +
                                                          (row0 + j) * kLatDim + kLatV)[lane];
    float x = q[0] * bf_lo(k0.x) + q[1] * bf_hi(k0.x) + q[2] * bf_lo(k0.y) + q[3] * bf_hi(k0.y) + q[4] * bf_lo(k1) +
              q[5] * bf_hi(k1);
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= a.scale;
    const float mn = fmaxf(m, x);
    const float f = m == -INFINITY ? 0.f : __expf(m - mn);
    const float p = x == -INFINITY ? 0.f : __expf(x - mn);
    l = l * f + p;
    o[0] = fmaf(o[0], f, p * bf_lo(v.x));
    o[1] = fmaf(o[1], f, p * bf_hi(v.x));
    o[2] = fmaf(o[2], f, p * bf_lo(v.y));
    o[3] = fmaf(o[3], f, p * bf_hi(v.y));
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const __nv_bfloat162 b0 = __floats2bfloat162_rn(o[0] * inv, o[1] * inv), b1 = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
  reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + r * 128)[lane] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
}

}  // namespace

int64_t expanded_plan_bytes(int64_t, int64_t, int64_t, int) { return 16; }

cudaError_t launch_latent_expanded(const ExpandedArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  int* bad = static_cast<int*>(a.plan);
  check_offsets_kernel<<<1, 256, 0, s>>>(a, bad);
  const int64_t rows = static_cast<int64_t>(a.T) * a.H;
  expanded_simple_kernel<<<static_cast<unsigned>((rows + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a, bad);
  return cudaGetLastError();
}

}  // namespace dsa
