// latent_expanded.cu -- attention in the expanded form of multi-head latent attention, for
// prompts: keys of 128 + 64 values (the first 128 up-projected from the latent for each head,
// the last 64 the shared rope key) and values of 128, up-projected too.
//
//   x[t,h,s] = scale * (q[t,h][0..127] . k[s,h] + q[t,h][128..191] . c[s][512..575]),
//   out[t,h] = sum_s softmax_s(x) * v[s,h].
//
// Keys, values and weights are held in fp16: as bf16 their three roundings of up to 2^-8 would
// triple the error that rounding out to bf16 leaves, in fp16 (2^-11 each) they add 2% to it.
// fp16's range is met by powers of two, which round nothing: a scale for each query row (taken
// out of q), and for each 128 tokens of a head one for its keys and one for its values, set by
// the largest magnitude; where the tokens' largest magnitudes lie further apart than 2^8, one for
// each token instead, so that none is rounded away beside another one, which a query need not even
// see.  The softmax then works on x + fv, fv the exponent of the value scale, so that the weights
// it hands to the product carry that scale; sums divide it out again.
//
// up_project_kernel: keys and values of every (128 tokens, head), [128, 512] x W_h^T [512, 256],
//   written as the 128-byte-swizzled images that the attention's MMAs read, so that it fetches
//   them with plain bulk copies.  One block per SM, the tokens' latents stay in shared memory
//   for all heads, W streams through a ring, and the epilogue of a head (8 warps) runs under
//   the MMAs of the next (two accumulators of 256 TMEM columns).
// expanded_kernel: one block of 12 warps per SM.  An item is (256 queries, head): two tiles of
//   128 rows, whose scores (128 columns each) and sums (128) fill TMEM.  One warp issues the MMAs
//   of a tile, so that the tensor core works on one tile while the softmax of the other runs;
//   four warps do that softmax, a thread per row, so that no warp waits for another one.  The
//   weights replace the scores in TMEM (the A operand of the second product).  K and V of 128 tokens
//   are 80 KB, read once for both tiles, through rings of four 16 KB and two 32 KB stages.
//   Items are taken in order from a counter, longest first among a sequence's; the heads go in
//   groups whose keys and values fit L2.  When there are too few long items for that to
//   balance, every block takes an equal share of all 128-token steps instead, and merge_expanded_kernel
//   joins the pieces of an item.
//
// Bound: the tensor core, 128 x 128 x (192 + 128) products in 1,280 cycles, and close behind
// it the 16,384 exponentials of those weights (1,024 cycles).  Measured: a step of both tiles takes
// 3,950 cycles, the chain of one of them (scores 1,400, maximum 550, weights 1,500, rest of the
// sums 500), and changing items 15,000; 8,192 tokens x 96 heads 2.21 ms in a row of calls, of
// which the up-projection is 0.21 (1.37 and 0.13 at the measured tensor rate).

#include <cuda_fp16.h>

#include "latent.h"
#include "latent_mma.cuh"

namespace dsa {
namespace {

constexpr int kTok = 128;                     // tokens of a step
constexpr int kRowsT = 128;                   // query rows of a tile
constexpr int kPair = 2 * kRowsT;
constexpr int kChunk = 16384;                 // 128 rows x 64 fp16
constexpr int kKvBytes = 5 * kChunk;          // keys (three chunks), then values (two), of 128 tokens
constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;
constexpr float kUnset = -1e38f;              // reference of a row without a token so far
constexpr float kLift = 7.f;                  // weights reach 2^(8 + 7): the upper end of fp16's range
// Largest distance, in powers of two, between the tokens of a tile that share a scale: a token that
// far below the largest is held to 2^-31 of its own largest value, and every weight to 2^-22 of the
// largest weight times value.  A tile beyond it costs its softmax two more passes over the
// scores and a third that reads them back: 8,192 tokens x 96 heads take 2.18 ms without one, 2.38 with one
// that all queries see and 7.6 with nothing else, where one scale a tile took 2.14 and rounded the
// smaller tokens away.  Looking for such tiles costs every call 1%.
constexpr int kSpread = 8;
constexpr float kOwnScale = 1000.f;           // in Ws::scale: the tokens' scales are in Ws::own
constexpr int64_t kL2Bytes = 48ll << 20;      // keys and values that a group of heads may take

struct Pair {           // up to 256 queries of a sequence
  int64_t kv_row0;      // cache row of the sequence's token 0
  int32_t tok0, ntok;   // first query, number of queries
  int32_t tile0;        // the sequence's first 128-token step among all
  int32_t seq_len;
  int32_t n[2];         // steps of either tile of rows
};

struct Steps {          // 128 tokens to expand
  int32_t row0, valid;  // first cache row, rows that some query attends to
};

struct Plan {
  int32_t pairs, tiles;     // entries of Ws::pair and Ws::step
  int64_t steps;            // over all pairs, of one head
  int32_t bad, merges;
  int32_t next, spoiled;    // items handed out; entries of Ws::spoiled
};

struct Merge {
  int32_t pair, head, first, last;   // an item in the shares of several blocks
};

struct Ws {
  Plan* plan;
  int32_t* seq_pair;    // [B+1] first pair of each sequence
  int32_t* seq_tile;    // [B+1] first step of each sequence
  int32_t* used;        // [B] tokens that some query attends to
  Pair* pair;           // [max pairs]
  int64_t* step0;       // [max pairs + 1] steps before each pair
  Steps* step;          // [max tiles]
  Merge* merge;         // [blocks]
  int2* spoiled;        // [T * H] a row of out to compute again, and the entry before it of the same warp
  float2* scale;        // [max tiles][H] exponents of the key and value scales, or kOwnScale
  float2* own;          // [max tiles][H][128] of the tokens, where they have scales of their own
  float2* ml;           // [2 * blocks][256] reference and sum of a piece's rows
  float* o;             // [2 * blocks][256][128]
  uint8_t* kv;          // [max tiles][H][kKvBytes]
  int64_t max_pairs, max_tiles, bytes;
};

Ws carve(void* base, int64_t T, int64_t B, int64_t H, int64_t cache_rows, int blocks) {
  Ws w;
  w.max_pairs = T / kPair + (B < T ? B : T) + 1;
  w.max_tiles = cache_rows / kTok + (B < T ? B : T) + 1;
  // parts 256 bytes apart from a 256-byte boundary, wherever the workspace itself starts
  uint8_t* const start = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(base) + 255) & ~uintptr_t(255));
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = start + off;
    off = (off + bytes + 255) & ~int64_t(255);
    return p;
  };
  w.plan = reinterpret_cast<Plan*>(take(sizeof(Plan)));
  w.seq_pair = reinterpret_cast<int32_t*>(take(4 * (B + 1)));
  w.seq_tile = reinterpret_cast<int32_t*>(take(4 * (B + 1)));
  w.used = reinterpret_cast<int32_t*>(take(4 * B));
  w.pair = reinterpret_cast<Pair*>(take(sizeof(Pair) * w.max_pairs));
  w.step0 = reinterpret_cast<int64_t*>(take(8 * (w.max_pairs + 1)));
  w.step = reinterpret_cast<Steps*>(take(sizeof(Steps) * w.max_tiles));
  w.merge = reinterpret_cast<Merge*>(take(sizeof(Merge) * blocks));
  w.spoiled = reinterpret_cast<int2*>(take(sizeof(int2) * T * H));
  w.scale = reinterpret_cast<float2*>(take(sizeof(float2) * w.max_tiles * H));
  w.own = reinterpret_cast<float2*>(take(sizeof(float2) * w.max_tiles * H * kTok));
  w.ml = reinterpret_cast<float2*>(take(sizeof(float2) * kPair * 2 * blocks));
  w.o = reinterpret_cast<float*>(take(int64_t(4) * kPair * 128 * 2 * blocks));
  w.kv = take(w.max_tiles * H * kKvBytes);
  w.bytes = off + 256;
  return w;
}

struct Params {
  int T, B, H;
  bool split;                   // equal shares of all steps instead of whole items
  int64_t cache_rows;
  const __nv_bfloat16* q;
  const __nv_bfloat16* kv;
  const int32_t* positions;
  const int32_t* q_seq_offsets;
  const int64_t* cache_offsets;
  ScoreScale scale;             // times log2(e)
  __nv_bfloat16* out;
  Ws ws;
  int* err;
  uint64_t timeout_ns;
};

// the last b with first[b] <= x, of n entries
__device__ __forceinline__ int last_at(const int32_t* first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ---------------------------------------------------------------- plan
__global__ void __launch_bounds__(kPlanThreads) expanded_plan_kernel(Params p, int blocks) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int64_t sums[32];
  const Ws& w = p.ws;
  const int tid = threadIdx.x, lane = tid & 31;
  int bad = 0;
  for (int b = tid; b < p.B; b += kPlanThreads) {
    const int64_t q0 = p.q_seq_offsets[b], q1 = p.q_seq_offsets[b + 1];
    const int64_t c0 = p.cache_offsets[b], c1 = p.cache_offsets[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.T || c0 < 0 || c1 < c0 || c1 > p.cache_rows) bad = 1;
    w.used[b] = 0;
  }
  bad = __syncthreads_or(bad);
  if (bad) {   // the attention kernel writes every row as attending to nothing
    if (tid == 0) {
      *w.plan = Plan{0, 0, 0, 1, 0, 0, 0};
      atomicOr(p.err, kErrOffsets);
    }
    return;
  }
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int n = b < p.B ? (p.q_seq_offsets[b + 1] - p.q_seq_offsets[b] + kPair - 1) / kPair : 0;
    const int inc = static_cast<int>(block_scan(n, sums));
    if (b < p.B) w.seq_pair[b + 1] = base + inc;
    base += static_cast<int>(sums[31]);
  }
  if (tid == 0) w.seq_pair[0] = 0;
  __syncthreads();
  const int pairs = base;
  // a warp per pair: its queries and the steps of its two tiles; a sequence's pairs in reverse
  // (with positions that rise, the longest first)
  int oob = 0;
  for (int k = tid >> 5; k < pairs; k += kPlanThreads / 32) {
    const int b = last_at(w.seq_pair, p.B, k);
    const int q0 = p.q_seq_offsets[b], q1 = p.q_seq_offsets[b + 1];
    const int i = w.seq_pair[b + 1] - 1 - k;     // counted from the sequence's first queries
    Pair pr;
    pr.kv_row0 = p.cache_offsets[b];
    pr.seq_len = static_cast<int32_t>(p.cache_offsets[b + 1] - pr.kv_row0);
    pr.tok0 = q0 + i * kPair;
    pr.ntok = q1 - pr.tok0 < kPair ? q1 - pr.tok0 : kPair;
    pr.tile0 = b;                                // replaced below
    int top = -1;
    for (int hf = 0; hf < 2; ++hf) {
      int m = -1;
      for (int j = hf * kRowsT + lane; j < (hf + 1) * kRowsT && j < pr.ntok; j += 32) {
        const int pos = p.positions[pr.tok0 + j];
        if (pos < -1 || pos >= pr.seq_len) oob = 1;
        else m = pos > m ? pos : m;
      }
      m = __reduce_max_sync(0xffffffffu, m);
      pr.n[hf] = (m + kTok) / kTok;
      top = m > top ? m : top;
    }
    if (lane == 0) {
      w.pair[k] = pr;
      atomicMax(&w.used[b], top + 1);
    }
  }
  if (oob) atomicOr(p.err, kErrBounds);
  __syncthreads();
  base = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int n = b < p.B ? (w.used[b] + kTok - 1) / kTok : 0;
    const int inc = static_cast<int>(block_scan(n, sums));
    if (b < p.B) w.seq_tile[b + 1] = base + inc;
    base += static_cast<int>(sums[31]);
  }
  if (tid == 0) w.seq_tile[0] = 0;
  __syncthreads();
  const int tiles = base;
  for (int k = tid; k < tiles; k += kPlanThreads) {
    const int b = last_at(w.seq_tile, p.B, k), j = (k - w.seq_tile[b]) * kTok;
    const int left = w.used[b] - j;
    w.step[k] = Steps{static_cast<int32_t>(p.cache_offsets[b] + j), left < kTok ? left : kTok};
  }
  int64_t steps = 0;
  for (int k0 = 0; k0 < pairs; k0 += kPlanThreads) {
    const int k = k0 + tid;
    int n = 0;
    if (k < pairs) {
      Pair& pr = w.pair[k];
      pr.tile0 = w.seq_tile[pr.tile0];
      n = pr.n[0] > pr.n[1] ? pr.n[0] : pr.n[1];
      if (n == 0) n = 1;                         // a pair without tokens still writes its rows
    }
    const int64_t inc = block_scan(n, sums);
    if (k < pairs) w.step0[k] = steps + inc - n;
    steps += sums[31];
  }
  if (tid == 0) w.step0[pairs] = steps;
  int* const count = reinterpret_cast<int*>(sums);
  __syncthreads();
  if (tid == 0) *count = 0;
  __syncthreads();
  if (p.split) {
    const int64_t all = steps * p.H;
    for (int64_t it = tid; it < static_cast<int64_t>(pairs) * p.H; it += kPlanThreads) {
      const int h = static_cast<int>(it / pairs), k = static_cast<int>(it % pairs);
      const int first = share_of(all, h * steps + w.step0[k], blocks), last = share_of(all, h * steps + w.step0[k + 1] - 1, blocks);
      if (first != last) w.merge[atomicAdd(count, 1)] = Merge{k, h, first, last};
    }
  }
  __syncthreads();
  if (tid == 0) *w.plan = Plan{pairs, tiles, steps, 0, *count, 0, 0};
}

// ---------------------------------------------------------------- helpers
// |v|, or 0 for NaN and infinities (they stay what they are under any scale)
__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.4028235e38f ? a : 0.f;
}

// D (+)= A[tmem] . B[smem] by the elected lane
__device__ __forceinline__ void umma_ta(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate,
                                        bool leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)leader)
      : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// 32 bytes, a whole sector, to a 32-byte aligned address
__device__ __forceinline__ void store32(void* p, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
// 16-byte units u, u + 1 (u even) of row r of a chunk: they lie at units u ^ (r & 7), (u + 1) ^ (r & 7),
// in the same 32 bytes
__device__ __forceinline__ void store_units(uint8_t* row, int r, int u, uint4 a, uint4 b) {
  store32(row + ((u ^ (r & 6)) * 16), r & 1 ? b : a, r & 1 ? a : b);
}

__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(smem_u32(bar), parity) && global_timer_ns() - t0 <= kDrainNs) {
  }
}

// ---------------------------------------------------------------- keys and values
constexpr int kUpStages = 3, kUpStage = 32768;      // 256 rows of W x 64 values
constexpr int kUpA = 8 * kChunk;                    // the latents of 128 tokens
constexpr int kUpThreads = 12 * 32;

struct UpMisc {
  uint64_t full[kUpStages], empty[kUpStages], a_full, a_empty, acc_full[2], acc_empty[2], mma_done;
  uint32_t tmem;
  int abort;
  float2 red[8];          // largest and smallest of the tokens' largest magnitudes, of a warp
};
constexpr int kUpSmem = kUpA + kUpStages * kUpStage + sizeof(UpMisc);
static_assert(kUpSmem <= 232448, "shared memory per block");

__global__ void __launch_bounds__(kUpThreads, 1)
    up_project_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmW, Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const sA = smem;
  uint8_t* const sB = smem + kUpA;
  UpMisc& mi = *reinterpret_cast<UpMisc*>(smem + kUpA + kUpStages * kUpStage);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Ws& w = p.ws;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kUpStages; ++s) {
      mbar_init(&mi.full[s], 1);
      mbar_init(&mi.empty[s], 1);
    }
    mbar_init(&mi.a_full, 1);
    mbar_init(&mi.a_empty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&mi.acc_full[b], 1);
      mbar_init(&mi.acc_empty[b], 8);
    }
    mbar_init(&mi.mma_done, 1);
    mi.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&mi.tmem, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  int64_t a0, a1;
  share(static_cast<int64_t>(w.plan->tiles) * p.H, blockIdx.x, gridDim.x, &a0, &a1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, mi.tmem, 0);
  const WaitCtl wc{p.err, &mi.abort, p.timeout_ns};
  const int H = p.H;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      uint32_t it = 0, loads = 0;
      for (int64_t i = a0; i < a1 && ok; ++i) {
        const int tile = static_cast<int>(i / H), h = static_cast<int>(i % H);
        const bool fresh = i == a0 || h == 0;
        if (fresh) {
          if (loads > 0 && !(ok = mbar_wait(&mi.a_empty, (loads - 1) & 1, wc))) break;
          mbar_arrive_expect_tx(&mi.a_full, kUpA);
          for (int c = 0; c < 8; ++c) tma_load_2d(sA + c * kChunk, &tmC, &mi.a_full, 64 * c, w.step[tile].row0);
          ++loads;
        }
        for (int c = 0; c < 8; ++c, ++it) {
          const uint32_t s = it % kUpStages;
          if (it >= kUpStages && !(ok = mbar_wait(&mi.empty[s], (it / kUpStages - 1) & 1, wc))) break;
          mbar_arrive_expect_tx(&mi.full[s], kUpStage);
          tma_load_2d(sB + s * kUpStage, &tmW, &mi.full[s], 64 * c, h * 256);
        }
      }
      if (!ok) {   // the loads in flight land before the block ends
        for (uint32_t k = it > kUpStages ? it - kUpStages : 0; k < it; ++k)
          drain(&mi.full[k % kUpStages], (k / kUpStages) & 1);
        if (loads > 0) drain(&mi.a_full, (loads - 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const bool leader = elect_one();
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc)); };
    auto commit = [&](uint64_t* bar) {
      if (leader) umma_commit(bar);
    };
    constexpr uint32_t idesc = umma_idesc_bf16(128, 256);
    const uint32_t a_lo = desc_lo(smem_u32(sA), 16), b_lo = desc_lo(smem_u32(sB), 16);
    Ring<kUpStages> rg;
    uint32_t nth = 0, loads = 0;
    bool ok = true;
    for (int64_t i = a0; i < a1 && ok; ++i, ++nth) {
      const int h = static_cast<int>(i % H);
      if (i == a0 || h == 0) {
        if (!(ok = wait(&mi.a_full, loads & 1))) break;
        ++loads;
      }
      const uint32_t buf = nth & 1;
      if (nth >= 2 && !(ok = wait(&mi.acc_empty[buf], (nth / 2 - 1) & 1))) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        if (!(ok = wait(&mi.full[rg.s], rg.phase))) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_lo(tmem + 256 * buf, a_lo + c * (kChunk >> 4) + 2 * k, b_lo + rg.s * (kUpStage >> 4) + 2 * k, idesc,
                  (c | k) != 0, leader);
        commit(&mi.empty[rg.s]);
        rg.next();
      }
      if (!ok) break;
      commit(&mi.acc_full[buf]);
      if (h == H - 1) commit(&mi.a_empty);
    }
    commit(&mi.mma_done);
    drain(&mi.mma_done, 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ---- epilogue: four warps for the keys, four for the values; a thread per token
    const int part = (warp - 4) >> 2, qd = warp & 3, r = qd * 32 + lane;
    bool ok = true;   // a wait that ran out is skipped from then on: the warps of a part meet at named barriers
    uint32_t nth = 0;
    uint4 rope[8];
    int valid = 0;
    for (int64_t i = a0; i < a1; ++i, ++nth) {
      const int64_t tile = i / H;
      const int h = static_cast<int>(i % H);
      if (i == a0 || h == 0) {
        const Steps st = w.step[tile];
        valid = st.valid;
        if (part == 0) {
          const uint4* src = reinterpret_cast<const uint4*>(p.kv + (st.row0 + static_cast<int64_t>(r < valid ? r : 0)) * kLatDim + kLatV);
#pragma unroll
          for (int u = 0; u < 8; ++u) rope[u] = src[u];
        }
      }
      const uint32_t buf = nth & 1, at = tmem + (static_cast<uint32_t>(qd * 32) << 16) + 256 * buf + 128 * part;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&mi.acc_full[buf], (nth / 2) & 1, wc));
      tc_fence_after();
      float top = 0.f;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        tmem_ld_32cols(at + 32 * c, x);
        tmem_ld_wait(x);
#pragma unroll
        for (int k = 0; k < 32; ++k) top = fmaxf(top, finite_abs(__uint_as_float(x[k])));
      }
      if (part == 0) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t v[4] = {rope[u].x, rope[u].y, rope[u].z, rope[u].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            top = fmaxf(top, fmaxf(finite_abs(__uint_as_float(v[k] << 16)), finite_abs(__uint_as_float(v[k] & 0xFFFF0000u))));
        }
      }
      if (r >= valid) top = 0.f;
      // tokens without a value but zeros (and what is not finite) fit any scale
      const uint32_t hi = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
      const uint32_t lo = __reduce_min_sync(0xffffffffu, top > 0.f ? __float_as_uint(top) : 0x7F800000u);
      if (lane == 0) mi.red[warp - 4] = make_float2(__uint_as_float(hi), __uint_as_float(lo));
      named_bar_sync(1 + part, 128);
      float most = 0.f, least = INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = mi.red[4 * part + k];
        most = fmaxf(most, v.x);
        least = fminf(least, v.y);
      }
      named_bar_sync(1 + part, 128);
      const bool own = static_cast<int>(__float_as_uint(most) >> 23) - static_cast<int>(__float_as_uint(least) >> 23) > kSpread;
      const int f = scale_exponent(own ? top : most, part == 0 ? kLowestFactor : kLowestValue);
      const float inv = pow2(-f);
      uint8_t* const dst = w.kv + (tile * H + h) * kKvBytes + part * 3 * kChunk + r * 128;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        tmem_ld_32cols(at + 32 * c, x);
        tmem_ld_wait(x);
        uint4 v[4];
        uint32_t* const o = reinterpret_cast<uint32_t*>(v);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          o[k] = r < valid ? pack_f16(__uint_as_float(x[2 * k]) * inv, __uint_as_float(x[2 * k + 1]) * inv) : 0u;
        store_units(dst + (c >> 1) * kChunk, r, 4 * (c & 1), v[0], v[1]);
        store_units(dst + (c >> 1) * kChunk, r, 4 * (c & 1) + 2, v[2], v[3]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&mi.acc_empty[buf]);
      if (part == 0) {
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
          const uint32_t v[8] = {rope[u].x, rope[u].y, rope[u].z, rope[u].w, rope[u + 1].x, rope[u + 1].y, rope[u + 1].z, rope[u + 1].w};
          uint4 t[2];
          uint32_t* const o = reinterpret_cast<uint32_t*>(t);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            o[k] = r < valid ? pack_f16(__uint_as_float(v[k] << 16) * inv, __uint_as_float(v[k] & 0xFFFF0000u) * inv) : 0u;
          store_units(dst + 2 * kChunk, r, u, t[0], t[1]);
        }
      }
      if (r == 0) (part == 0 ? w.scale[tile * H + h].x : w.scale[tile * H + h].y) = own ? kOwnScale : static_cast<float>(f);
      if (own) {
        float2* const t = w.own + (tile * H + h) * kTok + r;
        (part == 0 ? t->x : t->y) = static_cast<float>(f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- attention
constexpr int kKStages = 4, kVStages = 2, kVStage = 2 * kChunk;
constexpr int kQTile = 3 * kChunk;
constexpr int kThreads = 12 * 32;
// registers a thread: 168 at launch, then 88 (load, MMA) and 208 (softmax): 88 + 2 * 208 = 3 * 168
constexpr int kIssueRegs = 88, kSoftRegs = 208;
constexpr uint64_t kTurnNs = 20000;            // longest wait for the other tile's turn
constexpr uint32_t kTmemSum = 256;             // scores of tile i at 128 i, sums at 256 + 128 i

struct Misc {
  uint64_t full_k[kKStages], empty_k[kKStages], full_v[kVStages], empty_v[kVStages];
  uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], o_free[2], mma_done;
  uint32_t tmem;
  int abort;
  int item[2];                       // fetched items, in turn
  uint64_t item_full[2], item_empty[2];
  uint32_t turns[2];                 // softmax warps of a tile that are past their exponentials, in all
};
constexpr int kOffK = 2 * kQTile;
constexpr int kOffV = kOffK + kKStages * kChunk;
constexpr int kOffMisc = kOffV + kVStages * kVStage;
constexpr int kSmem = kOffMisc + sizeof(Misc);
static_assert(kSmem <= 232448, "shared memory per block");

struct Piece {
  Pair pr;
  int pair, head;
  int t0, n;            // first step, number of steps
  bool first, last;
};

// Items in order: a group of heads, the pairs, the heads of the group.
__device__ __forceinline__ void item_of(const Params& p, uint32_t pairs, uint32_t group, uint32_t it, int* pair, int* head) {
  const uint32_t per = group * pairs, g = it / per, rest = it - g * per;   // pairs * H stays below 2^31
  const uint32_t in = p.H - g * group < group ? p.H - g * group : group;
  *pair = rest / in;
  *head = g * group + rest % in;
}

// Exponents of token r's key and value scale in block blk = (tile, head) whose entry of Ws::scale is sc
__device__ __forceinline__ float2 token_scale(const Ws& w, float2 sc, int64_t blk, int r) {
  if (sc.x == kOwnScale || sc.y == kOwnScale) {
    const float2 t = w.own[blk * kTok + r];
    if (sc.x == kOwnScale) sc.x = t.x;
    if (sc.y == kOwnScale) sc.y = t.y;
  }
  return sc;
}

// Row (token, head) of out over its own prefix, by a warp: scores of 32 tokens at a time, a lane
// each, then four of the 128 dims a lane.  For rows that a NaN or an infinity beside their prefix
// spoiled (0 * NaN).  It may take long, so it runs where nobody waits for the warp.
__device__ __noinline__ void redo_row(const Params& p, int row) {
  const int lane = threadIdx.x & 31, t = row / p.H, head = row - t * p.H;
  const int tile0 = p.ws.seq_tile[last_at(p.q_seq_offsets, p.B, t)], lim = p.positions[t];
  const uint4* const q = reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(row) * 192);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 <= lim; s0 += 32) {
    const int64_t blk = static_cast<int64_t>(tile0 + s0 / kTok) * p.H + head;
    const uint8_t* const kv = p.ws.kv + blk * kKvBytes;
    const int r0 = s0 % kTok, r = r0 + lane;
    const float2 sc = token_scale(p.ws, p.ws.scale[blk], blk, r);
    const int n = lim - s0 < 31 ? lim - s0 + 1 : 32;
    float x = -INFINITY;
    if (lane < n) {
      x = 0.f;
#pragma unroll 4
      for (int u = 0; u < 24; ++u) {
        const uint4 a = q[u], k = *reinterpret_cast<const uint4*>(kv + (u >> 3) * kChunk + r * 128 + (((u & 7) ^ (r & 7)) * 16));
        const uint32_t av[4] = {a.x, a.y, a.z, a.w}, kvw[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&kvw[j]));
          x = fmaf(__uint_as_float(av[j] << 16), kf.x, fmaf(__uint_as_float(av[j] & 0xFFFF0000u), kf.y, x));
        }
      }
      x *= score_factor(p.scale, static_cast<int>(sc.x));
    }
    float top = x;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    top = fmaxf(m, top);
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - top), wt = top == -INFINITY ? 0.f : ex2_approx(x - top);
    m = top;
    float sum = wt;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = fmaf(l, f, sum);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] *= f;
    const float wv = wt * pow2(static_cast<int>(sc.y));
    for (int j = 0; j < n; ++j) {
      const float w = __shfl_sync(0xffffffffu, wv, j);
      const int rj = r0 + j;
      const uint2 v = *reinterpret_cast<const uint2*>(kv + (3 + (lane >> 4)) * kChunk + rj * 128 +
                                                      ((((lane & 15) >> 1) ^ (rj & 7)) * 16) + (lane & 1) * 8);
      const float2 v0 = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), v1 = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
      o[0] = fmaf(w, v0.x, o[0]);
      o[1] = fmaf(w, v0.y, o[1]);
      o[2] = fmaf(w, v1.x, o[2]);
      o[3] = fmaf(w, v1.y, o[3]);
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(row) * 128)[lane] = make_uint2(pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv));
}

// A tile whose tokens have scales of their own: the row's scores in TMEM become x + fv of each token
// (log2 units, -inf behind `rel`), and returned are the largest of them and the sum of
// 2^(x + fv - largest) / 2^fv.  The sum is taken from the rounded x + fv, as the weights are, so that what
// fp32 loses of a large score leaves their quotient as it is.  (-inf and 0 for a row that sees none
// of the tokens.)
__device__ __noinline__ float2 own_scores(const Params& p, float2 sc, int64_t blk, uint32_t ts, int fq, int rel) {
  const int lane = threadIdx.x & 31;
  float2 s[4];                                  // of tokens lane, lane + 32, ...
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] = token_scale(p.ws, sc, blk, lane + 32 * j);
  auto pick = [&](int c) { return c < 32 ? s[0] : c < 64 ? s[1] : c < 96 ? s[2] : s[3]; };
  float top = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < kTok; c += 16) {
    const float2 mine = pick(c);
    float x[16];
    tmem_ld16(ts + c, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int f = static_cast<int>(__shfl_sync(0xffffffffu, mine.x, (c & 16) + k));
      const float fv = __shfl_sync(0xffffffffu, mine.y, (c & 16) + k);
      x[k] = c + k <= rel ? fmaf(x[k], score_factor(p.scale, fq + f), fv) : -INFINITY;
      top = fmaxf(top, x[k]);
    }
    tmem_st16(ts + c, x);
  }
#pragma unroll 1
  for (int c = 0; c < kTok; c += 16) {
    const float2 mine = pick(c);
    float x[16];
    tmem_ld16(ts + c, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float fv = __shfl_sync(0xffffffffu, mine.y, (c & 16) + k);
      sum += x[k] == -INFINITY ? 0.f : ex2_approx(x[k] - top - fv);
    }
  }
  return make_float2(top, sum);
}

// The row's scores in TMEM become x * ak + fv less its reference, -inf behind `rel`: a difference of two
// rounded numbers, which is exact next to the reference.  (Not inlined: 128 more instructions
// in the loop cost every call 1%.)
__device__ __noinline__ void shift_scores(uint32_t ts, float ak, float fv, float m, int rel) {
#pragma unroll 1
  for (int c = 0; c < kTok; c += 16) {
    float x[16];
    tmem_ld16(ts + c, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = c + k <= rel ? fmaf(x[k], ak, fv) - m : -INFINITY;
    tmem_st16(ts + c, x);
  }
}

__global__ void __launch_bounds__(kThreads, 1) expanded_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const sQ = smem;
  uint8_t* const sK = smem + kOffK;
  uint8_t* const sV = smem + kOffV;
  Misc& mi = *reinterpret_cast<Misc*>(smem + kOffMisc);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Ws& w = p.ws;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&mi.full_k[s], 1);
      mbar_init(&mi.empty_k[s], 2);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&mi.full_v[s], 1);
      mbar_init(&mi.empty_v[s], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&mi.q_full[i], 4);
      mbar_init(&mi.s_full[i], 1);
      mbar_init(&mi.p_full[i][0], 4);
      mbar_init(&mi.p_full[i][1], 4);
      mbar_init(&mi.o_full[i], 1);
      mbar_init(&mi.o_free[i], 4);
      mbar_init(&mi.item_full[i], 1);
      mbar_init(&mi.item_empty[i], 10);   // 8 softmax and 2 MMA warps
      mi.turns[i] = 0;
    }
    mbar_init(&mi.mma_done, 2);
    mi.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&mi.tmem, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Plan plan = *w.plan;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (plan.bad) {
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; k < static_cast<int64_t>(p.T) * p.H * 16;
         k += static_cast<int64_t>(gridDim.x) * kThreads)
      reinterpret_cast<uint4*>(p.out)[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  const uint32_t tmem = __shfl_sync(0xffffffffu, mi.tmem, 0);
  const WaitCtl wc{p.err, &mi.abort, p.timeout_ns};
  // heads of a group: their keys and values fit L2
  int group = static_cast<int>(kL2Bytes / (static_cast<int64_t>(plan.tiles > 0 ? plan.tiles : 1) * kKvBytes));
  group = group < 1 ? 1 : group > p.H ? p.H : group;
  const int64_t items = static_cast<int64_t>(plan.pairs) * p.H, all = plan.steps * p.H;
  int64_t at, end;                    // shares: the block's steps
  share(all, blockIdx.x, gridDim.x, &at, &end);
  uint32_t fetched = 0;               // items so far
  // The next piece: of the block's share, or the next item of the counter, which warp 0 reads for
  // all (`mine`) and hands on through a ring of two.
  auto next = [&](Piece* pc, bool mine) {
    if (p.split) {
      if (at >= end) return false;
      const int h = static_cast<int>(at / plan.steps);
      const int64_t x = at - h * plan.steps;
      int lo = 0, hi = plan.pairs - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (w.step0[mid] <= x) lo = mid;
        else hi = mid - 1;
      }
      const int64_t s0 = w.step0[lo], s1 = w.step0[lo + 1];
      pc->pair = lo;
      pc->head = h;
      pc->t0 = static_cast<int>(x - s0);
      const int64_t stop = h * plan.steps + s1 < end ? h * plan.steps + s1 : end;
      pc->n = static_cast<int>(stop - at);
      pc->first = x == s0;
      pc->last = stop == h * plan.steps + s1;
      at = stop;
    } else {
      const uint32_t b = fetched & 1, ph = (fetched >> 1) & 1;
      int it;
      if (mine) {
        if (fetched >= 2 && !mbar_wait(&mi.item_empty[b], ph ^ 1, wc)) return false;
        it = atomicAdd(&w.plan->next, 1);
        if (it >= items) it = -1;
        *reinterpret_cast<volatile int*>(&mi.item[b]) = it;
        mbar_arrive(&mi.item_full[b]);
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait(&mi.item_full[b], ph, wc))) return false;
        it = *reinterpret_cast<volatile int*>(&mi.item[b]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.item_empty[b]);
      }
      ++fetched;
      if (it < 0) return false;
      item_of(p, plan.pairs, group, it, &pc->pair, &pc->head);
      pc->t0 = 0;
      pc->n = 0x7FFFFFFF;
      pc->first = pc->last = true;
    }
    pc->pr = w.pair[pc->pair];
    return true;
  };
  // steps of the piece that its tile i of rows takes part in
  auto steps_of = [](const Piece& pc, int i) {
    const int n = pc.pr.n[i] - pc.t0;
    return n < 0 ? 0 : n < pc.n ? n : pc.n;
  };
  Piece pc;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0) {
      // ============================================================ loads
      if (lane == 0) {
        bool ok = true;
        uint32_t ik = 0, iv = 0;
        while (ok && next(&pc, true)) {
          const int n0 = steps_of(pc, 0), n1 = steps_of(pc, 1), n = n0 > n1 ? n0 : n1;
          for (int t = 0; t < n && ok; ++t) {
            const uint8_t* const src =
                w.kv + (static_cast<int64_t>(pc.pr.tile0 + pc.t0 + t) * p.H + pc.head) * kKvBytes;
            for (int c = 0; c < 3; ++c, ++ik) {
              const uint32_t s = ik % kKStages;
              if (ik >= kKStages && !(ok = mbar_wait(&mi.empty_k[s], (ik / kKStages - 1) & 1, wc))) break;
              mbar_arrive_expect_tx(&mi.full_k[s], kChunk);
              bulk_load(sK + s * kChunk, src + c * kChunk, kChunk, &mi.full_k[s]);
            }
            if (!ok) break;
            const uint32_t s = iv % kVStages;
            if (iv >= kVStages && !(ok = mbar_wait(&mi.empty_v[s], (iv / kVStages - 1) & 1, wc))) break;
            mbar_arrive_expect_tx(&mi.full_v[s], kVStage);
            bulk_load(sV + s * kVStage, src + 3 * kChunk, kVStage, &mi.full_v[s]);
            ++iv;
          }
        }
        // the loads in flight land before the block ends, also when next() gave up waiting; after the
        // last item they have landed and this takes no time
        for (uint32_t k = ik > kKStages ? ik - kKStages : 0; k < ik; ++k) drain(&mi.full_k[k % kKStages], (k / kKStages) & 1);
        for (uint32_t k = iv > kVStages ? iv - kVStages : 0; k < iv; ++k) drain(&mi.full_v[k % kVStages], (k / kVStages) & 1);
      }
      __syncwarp();
    } else if (warp < 3) {
      // ============================================================ MMAs of tile i
      const int i = warp - 1;
      const bool leader = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc)); };
      auto commit = [&](uint64_t* bar) {
        if (leader) umma_commit(bar);
      };
      constexpr uint32_t idesc_s = idesc_f16(128, kTok), idesc_o = idesc_f16(128, 128) | (1u << 16);   // V MN-major
      const uint32_t q_lo = desc_lo(smem_u32(sQ + i * kQTile), 16), k_lo = desc_lo(smem_u32(sK), 16);
      const uint32_t v_lo = desc_lo(smem_u32(sV), kChunk);
      const uint32_t ts = tmem + 128 * i, to = tmem + kTmemSum + 128 * i;
      Ring<kKStages> rk;
      Ring<kVStages> rv;
      uint32_t segs = 0, done = 0;
      bool ok = true;
      while (ok && next(&pc, false)) {
        const int n = steps_of(pc, i), other = steps_of(pc, 1 - i);
        // S = Q . K^T of the next step
        auto scores = [&]() {
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            if (!wait(&mi.full_k[rk.s], rk.phase)) return false;
            tc_fence_after();
            const uint32_t a = q_lo + c * (kChunk >> 4), b = k_lo + rk.s * (kChunk >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_lo(ts, a + 2 * k, b + 2 * k, idesc_s, (c | k) != 0, leader);
            commit(&mi.empty_k[rk.s]);
            rk.next();
          }
          commit(&mi.s_full[i]);
          return true;
        };
        if (n > 0) {
          if (!(ok = wait(&mi.q_full[i], segs & 1))) break;
          tc_fence_after();
          if (!(ok = scores())) break;
          for (int t = 0; t < n && ok; ++t, ++done) {
            if (!(ok = wait(&mi.p_full[i][0], done & 1))) break;
            if (t == 0 && segs > 0 && !(ok = wait(&mi.o_free[i], (segs - 1) & 1))) break;
            // O += P . V, half of the tokens as soon as their weights are there
            if (!(ok = wait(&mi.full_v[rv.s], rv.phase))) break;
            tc_fence_after();
            const uint32_t b = v_lo + rv.s * (kVStage >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_ta(to, ts + 8 * k, b + k * 128, idesc_o, (t | k) != 0, leader);
            if (!(ok = wait(&mi.p_full[i][1], done & 1))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 4; k < 8; ++k) umma_ta(to, ts + 8 * k, b + k * 128, idesc_o, true, leader);
            commit(&mi.empty_v[rv.s]);
            rv.next();
            if (t == n - 1) commit(&mi.o_full[i]);
            else ok = scores();
          }
          ++segs;
        }
        // steps that only the other tile needs
        for (int t = n; t < other && ok; ++t) {
          for (int c = 0; c < 3; ++c) {
            if (!(ok = wait(&mi.full_k[rk.s], rk.phase))) break;
            if (leader) mbar_arrive(&mi.empty_k[rk.s]);
            rk.next();
          }
          if (!ok || !(ok = wait(&mi.full_v[rv.s], rv.phase))) break;
          if (leader) mbar_arrive(&mi.empty_v[rv.s]);
          rv.next();
        }
      }
      commit(&mi.mma_done);
      drain(&mi.mma_done, 0);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ============================================================ softmax of tile i, a thread per row
    const int i = (warp - 4) >> 2, qd = warp & 3;
    const int r = qd * 32 + lane;                         // row of the tile, TMEM lane
    const uint32_t tlane = tmem + (static_cast<uint32_t>(qd * 32) << 16);
    const uint32_t ts = tlane + 128 * i, to = tlane + kTmemSum + 128 * i;
    uint32_t done = 0, segs = 0, theirs = 0;              // steps of this tile, pieces, steps of the other
    int spoiled = -1;                                     // lane 0: the warp's last entry of Ws::spoiled
    bool ok = true;
    while (ok && next(&pc, false)) {
      const int n = steps_of(pc, i), other = steps_of(pc, 1 - i);
      const int tok = i * kRowsT + r;                     // query of the pair
      const bool real = tok < pc.pr.ntok;
      const int64_t row = static_cast<int64_t>(pc.pr.tok0 + tok) * p.H + pc.head;
      int lim = -1;
      if (real) {
        lim = p.positions[pc.pr.tok0 + tok];
        if (lim < -1 || lim >= pc.pr.seq_len) lim = -1;
      }
      int fq = 0;                                         // exponent of the row's scale
      if (n > 0) {
        // the warp's 32 rows of Q in fp16: lane l holds values 2l, 2l + 1 of each 64 of a row; all
        // of them are in flight at once
        const uint32_t* const src = reinterpret_cast<const uint32_t*>(p.q) +
                                    (static_cast<int64_t>(pc.pr.tok0 + i * kRowsT + qd * 32) * p.H + pc.head) * 96 + lane;
        const int have = pc.pr.ntok - i * kRowsT - qd * 32;
        uint32_t v[32][3];
#pragma unroll
        for (int k = 0; k < 32; ++k)
#pragma unroll
          for (int c = 0; c < 3; ++c) v[k][c] = k < have ? src[static_cast<int64_t>(k) * p.H * 96 + 32 * c] : 0u;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const int rr = qd * 32 + k;
          // magnitudes of bf16 pairs compare as integers (a row with an infinity is lost anyway)
          uint32_t top = __vmaxu2(__vmaxu2(v[k][0] & 0x7FFF7FFFu, v[k][1] & 0x7FFF7FFFu), v[k][2] & 0x7FFF7FFFu);
          top = __reduce_max_sync(0xffffffffu, top >> 16 > (top & 0xFFFFu) ? top >> 16 : top & 0xFFFFu);
          const int f = scale_exponent(__uint_as_float(top << 16), kLowestFactor);
          const float inv = pow2(-f);
#pragma unroll
          for (int c = 0; c < 3; ++c)
            *reinterpret_cast<uint32_t*>(sQ + i * kQTile + c * kChunk + rr * 128 + (((lane >> 2) ^ (rr & 7)) * 16) + (lane & 3) * 4) =
                pack_f16(__uint_as_float(v[k][c] << 16) * inv, __uint_as_float(v[k][c] & 0xFFFF0000u) * inv);
          if (lane == k) fq = f;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.q_full[i]);
      }
      const int low = __reduce_min_sync(0xffffffffu, real ? lim : 0x7FFFFFFF);   // of the warp's rows
      float m = kUnset, l = 0.f;
      const float2* const scales = w.scale + static_cast<int64_t>(pc.pr.tile0 + pc.t0) * p.H + pc.head;
      float2 sc = make_float2(0.f, 0.f);
      if (n > 0) sc = scales[0];
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++done) {
        const bool own = sc.x == kOwnScale || sc.y == kOwnScale;
        float ak = 1.f, fv = 0.f;              // own scales: in the scores already
        if (!own) ak = score_factor(p.scale, fq + static_cast<int>(sc.x)), fv = sc.y;
        const float2 here = sc;
        if (t + 1 < n) sc = scales[static_cast<int64_t>(t + 1) * p.H];
        const int pos0 = (pc.t0 + t) * kTok;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&mi.s_full[i], done & 1, wc));
        tc_fence_after();
        float2 sums = make_float2(0.f, 0.f);
        if (own) sums = own_scores(p, here, static_cast<int64_t>(pc.pr.tile0 + pc.t0 + t) * p.H + pc.head, ts, fq, lim - pos0);
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32cols(ts + 32 * c, x[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(x[c]);
        if (pos0 + kTok - 1 > low) {
          const int rel = lim - pos0;
#pragma unroll
          for (int c = 0; c < kTok; ++c)
            if (c > rel) x[c >> 5][c & 31] = 0xFF800000u;
        }
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 32; c += 2)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tops[k] = fmaxf(tops[k], fmaxf(__uint_as_float(x[k][c]), __uint_as_float(x[k][c + 1])));
        // the exponents of the weights stay below kLift + 8, in either form below: fp16 ends at 2^16
        const float most = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        float c2 = fv + kLift - m;
        const bool rise = fmaxf(fmaf(most, ak, fv) - m + kLift, fmaf(most, ak, c2)) > kLift + 8.f;
        bool exact = own;
        if (__any_sync(0xffffffffu, rise)) {
          // some row's reference rises
          const float now = rise ? fmaf(most, ak, fv) : m;
          // the sum of the weights in two halves: it carries no value scale, so it lasts where the
          // exponents of two tiles' values lie further apart than fp32 reaches
          const float f = ex2_approx(m - now), half = ex2_approx(0.5f * (m - now));
          m = now;
          l = l * half * half;
          if (t > 0) {
            // the sums so far (the scores' barrier covers the products before them)
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              float o[16];
              tmem_ld16(to + 16 * c, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= f;
              tmem_st16(to + 16 * c, o);
            }
          }
          c2 = fv + kLift - m;
          exact |= __any_sync(0xffffffffu, rise && fabsf(fmaf(most, ak, c2) - kLift) > 1.f);
        }
        if (exact) {
          // own scales, or scores so large that the rounding of m alone moves weights out of range
          shift_scores(ts, ak, fv, m, lim - pos0);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32cols(ts + 32 * c, x[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_wait(x[c]);
          ak = 1.f;
          c2 = kLift;
        }
        // The exponentials of the two tiles alternate, 0 before 1 in every step; left alone the tiles
        // fall into step, both softmaxes then wait for both products and a step takes twice as long.
        // Nothing depends on the order, so the wait is short and gives up without an error.
        {
          const uint32_t before = 4 * (theirs + (t + i < other ? t + i : other));
          const volatile uint32_t* const turns = &mi.turns[1 - i];
          if (static_cast<int32_t>(*turns - before) < 0) {
            const uint64_t t0 = global_timer_ns();
            while (static_cast<int32_t>(*turns - before) < 0 && global_timer_ns() - t0 < kTurnNs) {
            }
          }
          __syncwarp();
        }
        const float2 a2 = make_float2(ak, ak), b2 = make_float2(c2, c2);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int k = 2 * hf + (c >> 4), j = 2 * (c & 15);
            const float2 y = ffma2(make_float2(__uint_as_float(x[k][j]), __uint_as_float(x[k][j + 1])), a2, b2);
            const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            sum[c & 1] = __fadd2_rn(sum[c & 1], e);
            pk[c] = pack_f16(e.x, e.y);
          }
          if (hf == 1 && lane == 0) atomicAdd(&mi.turns[i], 1u);
          asm volatile(
              "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
              "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
              "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
              "tcgen05.wait::st.sync.aligned;" ::"r"(ts + 32 * hf),
              "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]), "r"(pk[7]),
              "r"(pk[8]), "r"(pk[9]), "r"(pk[10]), "r"(pk[11]), "r"(pk[12]), "r"(pk[13]), "r"(pk[14]), "r"(pk[15]),
              "r"(pk[16]), "r"(pk[17]), "r"(pk[18]), "r"(pk[19]), "r"(pk[20]), "r"(pk[21]), "r"(pk[22]), "r"(pk[23]),
              "r"(pk[24]), "r"(pk[25]), "r"(pk[26]), "r"(pk[27]), "r"(pk[28]), "r"(pk[29]), "r"(pk[30]), "r"(pk[31])
              : "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&mi.p_full[i][hf]);
        }
        sum[0] = __fadd2_rn(sum[0], sum[1]);
        l = own ? fmaf(sums.y, ex2_approx(sums.x - m + kLift), l) : fmaf(sum[0].x + sum[0].y, pow2(-static_cast<int>(fv)), l);
      }
      theirs += other;
      if (n > 0) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&mi.o_full[i], segs & 1, wc));
        tc_fence_after();
        ++segs;
      }
      const bool whole = pc.first && pc.last;
      const float inv = l != 0.f ? 1.f / l : 0.f;
      const int64_t slot = 2 * blockIdx.x + (pc.first ? 1 : 0);    // head pieces 0, tail pieces 1
      bool nan = false;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld_32cols(to + 32 * c, o);
          tmem_ld_wait(o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (real && whole) {
          uint4 v[4];
          uint32_t* const u = reinterpret_cast<uint32_t*>(v);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float v0 = __uint_as_float(o[2 * k]) * inv, v1 = __uint_as_float(o[2 * k + 1]) * inv;
            nan |= v0 != v0 || v1 != v1;
            u[k] = pack2(v0, v1);
          }
          __nv_bfloat16* const dst = p.out + row * 128 + 32 * c;
          if ((reinterpret_cast<uintptr_t>(p.out) & 16) == 0) {
            store32(dst, v[0], v[1]);
            store32(dst + 16, v[2], v[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(dst)[k] = v[k];
          }
        } else if (real && n > 0) {
          float* const dst = w.o + (slot * kPair + tok) * 128 + 32 * c;
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            store32(dst + k, make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]), make_uint4(o[k + 4], o[k + 5], o[k + 6], o[k + 7]));
        }
        __syncwarp();
      }
      if (!whole) w.ml[slot * kPair + tok] = make_float2(m, l);
      if (n > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.o_free[i]);
      }
      for (unsigned bad = __ballot_sync(0xffffffffu, nan && inv == inv); bad; bad &= bad - 1) {
        if (lane == 0) {
          const int e = atomicAdd(&w.plan->spoiled, 1);
          w.spoiled[e] = make_int2((pc.pr.tok0 + i * kRowsT + qd * 32 + __ffs(bad) - 1) * p.H + pc.head, spoiled);
          spoiled = e;
        }
      }
      __syncwarp();
    }
    // the warp's spoiled rows, when no other role waits for it any more
    for (int e = __shfl_sync(0xffffffffu, spoiled, 0); e >= 0;) {
      const int2 s = w.spoiled[e];
      redo_row(p, s.x);
      e = s.y;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- merge (shares)
// Rows of an item from its pieces, in the order of their steps; eight rows a warp, so that their
// loads are in flight together.
constexpr int kMergeThreads = 128, kMergeRows = 8;

__global__ void __launch_bounds__(kMergeThreads) merge_expanded_kernel(const __grid_constant__ Params p, int blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Ws& w = p.ws;
  const int merges = w.plan->merges, lane = threadIdx.x & 31;
  const int64_t all = w.plan->steps * p.H;
  for (int item = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5); item < merges * (kPair / kMergeRows);
       item += gridDim.x * (kMergeThreads / 32)) {
    const Merge mg = w.merge[item / (kPair / kMergeRows)];
    const Pair pr = w.pair[mg.pair];
    const int tok = item % (kPair / kMergeRows) * kMergeRows;
    if (tok >= pr.ntok) continue;
    float m[kMergeRows], l[kMergeRows];
    float4 o[kMergeRows];
#pragma unroll
    for (int r = 0; r < kMergeRows; ++r) m[r] = kUnset, l[r] = 0.f, o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = mg.first; k <= mg.last; ++k) {
      if (all < blocks) {      // with fewer steps than blocks some shares are empty
        int64_t x, y;
        share(all, k, blocks, &x, &y);
        if (x >= y) continue;
      }
      const int64_t at = static_cast<int64_t>(2 * k + (k == mg.first)) * kPair + tok;
      float2 v[kMergeRows];
      float4 c[kMergeRows];
#pragma unroll
      for (int r = 0; r < kMergeRows; ++r) {
        v[r] = w.ml[at + r];
        c[r] = reinterpret_cast<const float4*>(w.o + (at + r) * 128)[lane];
      }
#pragma unroll
      for (int r = 0; r < kMergeRows; ++r) {
        if (v[r].y == 0.f) continue;          // no token of the row in this piece: nothing was stored
        const float now = fmaxf(m[r], v[r].x), f0 = ex2_approx(m[r] - now), f1 = ex2_approx(v[r].x - now);
        const float m_was = m[r];
        m[r] = now;
        const float h0 = ex2_approx(0.5f * (m_was - now)), h1 = ex2_approx(0.5f * (v[r].x - now));
        l[r] = fmaf(l[r] * h0, h0, v[r].y * h1 * h1);
        o[r].x = fmaf(o[r].x, f0, c[r].x * f1);
        o[r].y = fmaf(o[r].y, f0, c[r].y * f1);
        o[r].z = fmaf(o[r].z, f0, c[r].z * f1);
        o[r].w = fmaf(o[r].w, f0, c[r].w * f1);
      }
    }
#pragma unroll
    for (int r = 0; r < kMergeRows; ++r) {
      if (tok + r >= pr.ntok) continue;
      const float inv = l[r] != 0.f ? 1.f / l[r] : 0.f;
      const int64_t row = static_cast<int64_t>(pr.tok0 + tok + r) * p.H + mg.head;
      reinterpret_cast<uint2*>(p.out + row * 128)[lane] =
          l[r] != 0.f ? make_uint2(pack2(o[r].x * inv, o[r].y * inv), pack2(o[r].z * inv, o[r].w * inv)) : make_uint2(0u, 0u);
      const bool nan = inv == inv && l[r] != 0.f && !(o[r].x == o[r].x && o[r].y == o[r].y && o[r].z == o[r].z && o[r].w == o[r].w);
      if (__any_sync(0xffffffffu, nan)) redo_row(p, static_cast<int>(row));   // each lane writes what it wrote above
    }
  }
}

}  // namespace

int64_t expanded_workspace_bytes(int64_t T, int64_t B, int64_t H, int64_t cache_rows, int num_sms) {
  return carve(nullptr, T, B, H, cache_rows, num_sms).bytes;
}

cudaError_t launch_latent_expanded(const ExpandedArgs& a, const CUtensorMap& tmC, const CUtensorMap& tmW, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int blocks = a.num_sms;
  Params p;
  p.T = a.T;
  p.B = a.B;
  p.H = a.H;
  p.cache_rows = a.cache_rows;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.kv = static_cast<const __nv_bfloat16*>(a.kv);
  p.positions = a.positions;
  p.q_seq_offsets = a.q_seq_offsets;
  p.cache_offsets = a.cache_offsets;
  p.scale = score_scale(scale_to_log2(a.scale));
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.ws = carve(a.workspace, a.T, a.B, a.H, a.cache_rows, blocks);
  p.err = a.err;
  p.timeout_ns = a.timeout_ns;
  // Whole items leave blocks idle in their last round; equal shares cost two more starts a block and
  // the merge, about as much as 12 steps.  Measured, items / shares: 2,000 tokens x 24 heads 83 / 116
  // us, ragged 3,802 x 32 130 / 177; 1,500 tokens after 6,500 x 32 heads 330 / 301, 1,000 after
  // 11,000 x 24 295 / 259.  From four items a block on the counter evens them out by itself.
  const int64_t items = (static_cast<int64_t>(a.T) + kPair - 1) / kPair * a.H;
  const int64_t idle = (blocks - items % blocks) % blocks, steps = a.cache_rows / (static_cast<int64_t>(a.B) * kTok) + 1;
  p.split = items < 4 * blocks && idle * steps > 12 * blocks;
  cudaError_t e = cudaFuncSetAttribute(up_project_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kUpSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(expanded_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  expanded_plan_kernel<<<1, kPlanThreads, 0, s>>>(p, blocks);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // the later kernels start while their predecessor runs out and wait for its results themselves
  cudaLaunchAttribute dep;
  dep.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  dep.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kUpThreads);
  cfg.dynamicSmemBytes = kUpSmem;
  cfg.stream = s;
  cfg.attrs = &dep;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, up_project_kernel, tmC, tmW, p)) != cudaSuccess) return e;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  if ((e = cudaLaunchKernelEx(&cfg, expanded_kernel, p)) != cudaSuccess) return e;
  if (!p.split) return cudaSuccess;
  cfg.gridDim = dim3(8 * blocks);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, merge_expanded_kernel, p, blocks);
}

}  // namespace dsa
