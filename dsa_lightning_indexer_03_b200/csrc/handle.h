// handle.h -- what a dsa_indexer_t points to, and checks that the entry points share (internal to
// the .so).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "../../include/dsa_indexer.h"
#include "kernels.h"

struct dsa_indexer {
  dsa_indexer_config_t cfg;
  int device = 0;
  int num_sms = 0;
  __nv_bfloat16* WqT = nullptr;   // [n_heads*head_dim, q_latent_dim]
  __nv_bfloat16* WkwT = nullptr;  // [head_dim + n_heads, hidden_dim]
  float* gamma = nullptr;         // [head_dim]
  float* beta = nullptr;
  double* inv_freq = nullptr;     // [32] rotary frequencies (rope_dim > 0)
  CUtensorMap tm_WqT, tm_WkwT;
  dsa::TopkWorkspace ws{};
  std::vector<void*> allocs;
  // dsa_indexer_project runs the k|w GEMM (HBM-bound) on `side` next to the q GEMM
  // (tensor-bound) on the caller's stream, forked and joined with the two events
  cudaStream_t side = nullptr;
  cudaEvent_t ev_fork = nullptr, ev_join = nullptr;

  template <class T>
  bool alloc(T** p, size_t count) {
    void* q = nullptr;
    if (cudaMalloc(&q, count * sizeof(T) + 16) != cudaSuccess) return false;
    allocs.push_back(q);
    *p = static_cast<T*>(q);
    return true;
  }
  ~dsa_indexer() {
    if (ev_fork) cudaEventDestroy(ev_fork);
    if (ev_join) cudaEventDestroy(ev_join);
    if (side) cudaStreamDestroy(side);
    for (void* p : allocs) cudaFree(p);
  }
};

namespace dsa {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline uint64_t timeout_ns() { return wait_timeout_ns(); }

}  // namespace dsa
