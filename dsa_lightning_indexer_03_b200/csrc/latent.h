// latent.h -- launchers of the latent-cache operators (internal to the .so): dense attention
// in the absorbed form over a bf16 or 4-bit cache, the 4-bit rows, and the expanded form.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dsa {

constexpr int kLatDim = 576;      // cached values per token: latent, then the shared rope key
constexpr int kLatV = 512;        // the latent: the value part in the absorbed form
constexpr int kLatRope = 64;
constexpr int kLatBlock = 16;     // latent values that share one e4m3 scale in a 4-bit row
constexpr int kLatCodes = kLatV / 2;                  // bytes of codes of a 4-bit row
constexpr int kLatScales = kLatV / kLatBlock;         // bytes of scales, after the codes
constexpr int kLatRow4 = kLatCodes + kLatScales + 2 * kLatRope;   // 416: codes | scales | bf16 rope key

// Attention of T queries (H heads of 576 values) over a latent cache.  Dense: query t at
// position p of its sequence attends to rows 0..p (p = -1: to nothing).  With idx: to the
// positions its idx row holds (-1 = none).
struct LatentArgs {
  int T, B, H;
  int k_sel;                      // entries of an idx row; < 0: dense
  int64_t cache_rows;
  const void* q;                  // bf16 [T, H, 576]
  const void* kv;                 // bf16 [cache_rows, 576], or uint8 [cache_rows, 416] when fp4
  bool fp4;
  const int32_t* positions;       // [T] (dense)
  const int32_t* q_seq_offsets;   // [B+1]
  const int64_t* cache_offsets;   // [B+1]
  const int32_t* idx;             // [T, k_sel]
  float scale;
  void* out;                      // bf16 [T, H, 512]
  float* lse;                     // [T, H]
  void* workspace;
  int num_sms;
  int* err;
  uint64_t timeout_ns;
};

int64_t latent_workspace_bytes(int64_t T, int64_t B, int64_t H, int num_sms);
// tmQ: bf16 [T * H, 576], boxes of 64 values x 96 rows; tmC: the bf16 cache [cache_rows, 576],
// boxes of 64 values x 64 rows (not read when fp4)
cudaError_t launch_latent_attention(const LatentArgs& a, const CUtensorMap& tmQ, const CUtensorMap& tmC,
                                    cudaStream_t s);

// 4-bit rows of n bf16 rows kv [n, 576]: row i goes to row rows[i] of out (row i without rows)
cudaError_t launch_quantize_latent_fp4(int64_t n, const void* kv, const int64_t* rows, uint8_t* out, int64_t out_rows,
                                       int* err, int num_sms, cudaStream_t s);
// bf16 rows [n, 576] of rows rows[i] (row i without rows) of a 4-bit cache
cudaError_t launch_dequantize_latent_fp4(int64_t n, const uint8_t* kv4, int64_t kv_rows, const int64_t* rows, void* out,
                                         int* err, int num_sms, cudaStream_t s);

// Attention in the expanded form: q [T, H, 192] against the keys (128 + 64 values) and values
// (128) that W_ukv expands from the latent.
struct ExpandedArgs {
  int T, B, H;
  int64_t cache_rows;
  const void* q;                  // bf16 [T, H, 192]
  const void* kv;                 // bf16 [cache_rows, 576]
  const int32_t* positions;
  const int32_t* q_seq_offsets;
  const int64_t* cache_offsets;
  float scale;
  void* out;                      // bf16 [T, H, 128]
  void* workspace;
  int num_sms;
  int* err;
  uint64_t timeout_ns;
};

int64_t expanded_workspace_bytes(int64_t T, int64_t B, int64_t H, int64_t cache_rows, int num_sms);
// tmC: the latents of the cache [cache_rows, 512] (rows 576 values apart), boxes of 64 values x 128
// rows; tmW: W_ukv [H * 256, 512], boxes of 64 values x 256 rows
cudaError_t launch_latent_expanded(const ExpandedArgs& a, const CUtensorMap& tmC, const CUtensorMap& tmW, cudaStream_t s);

}  // namespace dsa
