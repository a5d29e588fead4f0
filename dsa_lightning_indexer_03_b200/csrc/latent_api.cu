// latent_api.cu -- the C ABI of the latent-cache operators: argument checks, TMA descriptors and
// launches.

#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "handle.h"
#include "latent.h"

using namespace dsa;

namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_latent_encode = nullptr;
std::once_flag g_latent_encode_once;

// 2-D bf16 tensor [rows, inner], rows `stride` values apart, in 128-byte swizzled boxes of 64
// values x box_rows rows.
bool make_tmap(CUtensorMap* m, const void* base, uint64_t inner, uint64_t stride, uint64_t rows, uint32_t box_rows) {
  std::call_once(g_latent_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_latent_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_latent_encode) return false;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {stride * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return g_latent_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared checks of the latent attention entry points: sizes, then pointers.
dsa_status_t latent_checks(dsa_indexer_t h, int64_t T, const void* q, int32_t n_heads, const void* kv, int64_t cache_rows,
                           const int32_t* positions, const int32_t* q_seq_offsets, int32_t B,
                           const int64_t* cache_offsets, float scale, const void* out, const void* workspace) {
  if (!h || T < 0 || B < 1 || n_heads < 1 || n_heads > 1024) return DSA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return DSA_ERR_INVALID_ARG;
  if (T * n_heads > (int64_t(1) << 30) || T > (int64_t(1) << 30) || cache_rows < 1 || cache_rows > (int64_t(1) << 31) - (int64_t(1) << 20))
    return DSA_ERR_INVALID_ARG;
  if (T == 0) return DSA_OK;
  if (!q || !kv || !q_seq_offsets || !cache_offsets || !out || !workspace) return DSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv) || !aligned16(out) || !aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(positions) & 3) || (reinterpret_cast<uintptr_t>(q_seq_offsets) & 3) ||
      (reinterpret_cast<uintptr_t>(cache_offsets) & 7))
    return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

dsa_status_t latent_impl(dsa_indexer_t h, int64_t T, const void* q, int32_t n_heads, const void* kv, bool fp4,
                         int64_t cache_rows, const int32_t* positions, const int32_t* q_seq_offsets, int32_t B,
                         const int64_t* cache_offsets, const int32_t* idx, int32_t k_sel, float scale, void* out,
                         float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  const dsa_status_t st = latent_checks(h, T, q, n_heads, kv, cache_rows, positions, q_seq_offsets, B, cache_offsets,
                                        scale, out, workspace);
  if (st != DSA_OK || T == 0) return st;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3) || (reinterpret_cast<uintptr_t>(idx) & 3)) return DSA_ERR_INVALID_ARG;
  if (k_sel < 0 ? !positions : (!idx && k_sel > 0)) return DSA_ERR_INVALID_ARG;
  if (workspace_bytes < latent_workspace_bytes(T, B, n_heads, h->num_sms)) return DSA_ERR_WORKSPACE;
  LatentArgs a;
  a.T = static_cast<int>(T);
  a.B = B;
  a.H = n_heads;
  a.k_sel = k_sel;
  a.cache_rows = cache_rows;
  a.q = q;
  a.kv = kv;
  a.fp4 = fp4;
  a.positions = positions;
  a.q_seq_offsets = q_seq_offsets;
  a.cache_offsets = cache_offsets;
  a.idx = idx;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  a.num_sms = h->num_sms;
  a.err = h->ws.err;
  a.timeout_ns = timeout_ns();
  CUtensorMap tmQ, tmC;
  if (!make_tmap(&tmQ, q, kLatDim, kLatDim, uint64_t(T) * n_heads, 96)) return DSA_ERR_INVALID_ARG;
  if (fp4) tmC = tmQ;
  else if (!make_tmap(&tmC, kv, kLatDim, kLatDim, uint64_t(cache_rows), 64)) return DSA_ERR_INVALID_ARG;
  return launch_latent_attention(a, tmQ, tmC, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

extern "C" {

int64_t dsa_indexer_latent_attention_workspace(dsa_indexer_t h, int64_t T, int32_t B, int32_t n_heads) {
  if (!h || T < 0 || B < 1 || n_heads < 1 || n_heads > 1024 || T > (int64_t(1) << 30) || T * n_heads > (int64_t(1) << 30))
    return -1;
  return latent_workspace_bytes(T, B, n_heads, h->num_sms);
}

dsa_status_t dsa_indexer_latent_attention(dsa_indexer_t h, int64_t T, const void* q, int32_t n_heads,
                                          const void* kv_cache, int64_t cache_rows, const int32_t* positions,
                                          const int32_t* q_seq_offsets, int32_t B, const int64_t* cache_offsets,
                                          float scale, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                                          void* stream) {
  return latent_impl(h, T, q, n_heads, kv_cache, false, cache_rows, positions, q_seq_offsets, B, cache_offsets, nullptr,
                     -1, scale, out, lse, workspace, workspace_bytes, stream);
}

dsa_status_t dsa_indexer_latent_attention_fp4(dsa_indexer_t h, int64_t T, const void* q, int32_t n_heads,
                                              const void* kv_cache_fp4, int64_t cache_rows, const int32_t* positions,
                                              const int32_t* q_seq_offsets, int32_t B, const int64_t* cache_offsets,
                                              const int32_t* idx, int32_t k_sel, float scale, void* out, float* lse,
                                              void* workspace, int64_t workspace_bytes, void* stream) {
  return latent_impl(h, T, q, n_heads, kv_cache_fp4, true, cache_rows, positions, q_seq_offsets, B, cache_offsets, idx,
                     k_sel < 0 ? -1 : k_sel, scale, out, lse, workspace, workspace_bytes, stream);
}

dsa_status_t dsa_indexer_quantize_latent_fp4(dsa_indexer_t h, int64_t n, const void* kv, const int64_t* rows, void* out,
                                             int64_t out_rows, void* stream) {
  if (!h || n < 0 || out_rows < 0) return DSA_ERR_INVALID_ARG;
  if (n == 0) return DSA_OK;
  if (!kv || !out || n > (int64_t(1) << 34) || !aligned16(kv) || !aligned16(out) || (reinterpret_cast<uintptr_t>(rows) & 7))
    return DSA_ERR_INVALID_ARG;
  if (!rows && n > out_rows) return DSA_ERR_INVALID_ARG;
  return launch_quantize_latent_fp4(n, kv, rows, static_cast<uint8_t*>(out), out_rows, h->ws.err, h->num_sms,
                                    static_cast<cudaStream_t>(stream)) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t dsa_indexer_dequantize_latent_fp4(dsa_indexer_t h, int64_t n, const void* kv_fp4, int64_t kv_rows,
                                               const int64_t* rows, void* out, void* stream) {
  if (!h || n < 0 || kv_rows < 0) return DSA_ERR_INVALID_ARG;
  if (n == 0) return DSA_OK;
  if (!kv_fp4 || !out || n > (int64_t(1) << 34) || !aligned16(kv_fp4) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(rows) & 7) || kv_rows == 0)
    return DSA_ERR_INVALID_ARG;
  if (!rows && n > kv_rows) return DSA_ERR_INVALID_ARG;
  return launch_dequantize_latent_fp4(n, static_cast<const uint8_t*>(kv_fp4), kv_rows, rows, out, h->ws.err, h->num_sms,
                                      static_cast<cudaStream_t>(stream)) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

int64_t dsa_indexer_latent_expanded_workspace(dsa_indexer_t h, int64_t T, int32_t B, int32_t n_heads,
                                              int64_t cache_rows) {
  if (!h || T < 0 || B < 1 || n_heads < 1 || n_heads > 1024 || T > (int64_t(1) << 30) || T * n_heads > (int64_t(1) << 30) || cache_rows < 1 ||
      cache_rows > 65535 * int64_t(128))
    return -1;
  return expanded_workspace_bytes(T, B, n_heads, cache_rows, h->num_sms);
}

dsa_status_t dsa_indexer_latent_attention_expanded(dsa_indexer_t h, int64_t T, const void* q, int32_t n_heads,
                                                   const void* kv_cache, int64_t cache_rows, const void* W_ukv,
                                                   const int32_t* positions, const int32_t* q_seq_offsets, int32_t B,
                                                   const int64_t* cache_offsets, float scale, void* out,
                                                   void* workspace, int64_t workspace_bytes, void* stream) {
  const dsa_status_t st = latent_checks(h, T, q, n_heads, kv_cache, cache_rows, positions, q_seq_offsets, B,
                                        cache_offsets, scale, out, workspace);
  if (st != DSA_OK || T == 0) return st;
  if (!positions || !W_ukv || !aligned16(W_ukv)) return DSA_ERR_INVALID_ARG;
  if (cache_rows > 65535 * int64_t(128)) return DSA_ERR_UNSUPPORTED;
  if (workspace_bytes < expanded_workspace_bytes(T, B, n_heads, cache_rows, h->num_sms)) return DSA_ERR_WORKSPACE;
  CUtensorMap tmC, tmW;
  if (!make_tmap(&tmC, kv_cache, kLatV, kLatDim, uint64_t(cache_rows), 128) ||
      !make_tmap(&tmW, W_ukv, kLatV, kLatV, uint64_t(n_heads) * 256, 256))
    return DSA_ERR_INVALID_ARG;
  ExpandedArgs a;
  a.T = static_cast<int>(T);
  a.B = B;
  a.H = n_heads;
  a.cache_rows = cache_rows;
  a.q = q;
  a.kv = kv_cache;
  a.positions = positions;
  a.q_seq_offsets = q_seq_offsets;
  a.cache_offsets = cache_offsets;
  a.scale = scale;
  a.out = out;
  a.workspace = workspace;
  a.num_sms = h->num_sms;
  a.err = h->ws.err;
  a.timeout_ns = timeout_ns();
  return launch_latent_expanded(a, tmC, tmW, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
