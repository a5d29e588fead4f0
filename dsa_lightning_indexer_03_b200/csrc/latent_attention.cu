// latent_attention.cu -- dense attention in the absorbed form of multi-head latent attention,
// over a bf16 or a 4-bit cache, and over the indexer's selection of a 4-bit cache.
//
//   x[r,s] = scale * (q[r] . c[s])  over the 576 cached values of a token,
//   out[r] = sum_s softmax_s(x[r]) c[s][0..511],   lse[r] = ln sum_s exp(x[r,s]),
//
// for the rows r = (token, head) of a sequence.  All rows of a sequence read the same cache
// rows, so they are taken in groups of up to 96 consecutive rows (one decode token of 96 heads,
// or several tokens of fewer), and a group's tokens in tiles of 128.
//
// The products run transposed: S^T = C . Q^T (M = 128 tokens, N = the group's rows, K = 576)
// and O^T += C_latent^T . P^T (M = 4 x 128 latent dims, N = rows, K = 128 tokens).  So M is
// always full (96 rows as M would waste a quarter of it), the whole 512-dim output of a group
// (4 x 96 fp32 columns) and its scores (96) fit in one SM's TMEM, and the scores of a tile are
// computed once.  Q (96 x 576, 108 KB) stays in shared memory; the cache streams through two
// rings: nine 64-value chunks of a tile for its scores, then the tile again (from L2) as pieces of
// 64 tokens x 128 dims for its values, since Q and a whole 144 KB tile do not fit together.
//
// latent_attention_kernel: persistent, one block of 20 (bf16) or 24 (4-bit) warps per SM.
//   fill      bf16: one thread a ring, with TMA, and a warp that zeroes the rows behind a
//             sequence's last token (0 * NaN is NaN).  4-bit: four warps a ring convert the rows,
//             to fp16, in which their values are exact; queries then are scaled by powers of two
//             into fp16 too (their rope part, and the rope keys, stay bf16: an MMA of their own).
//   softmax   12 warps, a thread per token and a third of the rows.  The reference m of a row is
//             its running maximum, raised only when a score exceeds it by more than 8 (log2 units,
//             so weights stay below 256, or 2^15 in fp16, whose weights start at 2^7 to keep light
//             ones): most tiles then need no maximum over the tokens, which lie across threads, only
//             a vote.  Sums are taken over the warp in every tile, over the warps at the end.
//             Weights go to shared memory in the values' type.
//   MMA       two warps, one for the scores and one for the values, so that the scores of the
//             next tile run beside the values of this one, and the softmax under both.
// Work: plan_kernel lists the groups and their tiles; the blocks take equal shares of all tiles
// in order, so a share may begin or end inside a group; such pieces leave unnormalised fp32
// sums and (m, l) in the workspace, which merge_kernel joins in a fixed order.
//
// A row of a bf16 cache that only some of a tile's queries may see can hold NaN or infinities; its
// weight for the others is 0, and 0 * NaN spoils their sums.  Such rows of out (NaN under a
// finite sum of weights) are listed and computed again by merge_kernel over their own prefix.
//
// Bound: 1,152 B (bf16) and 2 * 96 * 1,088 flop a cached token at 96 rows.  Measured: 7,400
// cycles a tile where the cache lies in L2 (a prompt chunk; the MMAs alone 3,260, the 765 KB of
// shared-memory traffic of both products' operands and the rings 6,000), 8,900 where it comes from
// memory (5,800 at the copy rate; a third of the rows is read twice all the same).  4-bit rows
// take 15,000: the conversion of a tile, once for each product, and the waits between its steps.

#include "latent.h"
#include "latent_mma.cuh"

namespace dsa {
namespace {

constexpr int kRows = 96;                    // rows (token, head) of a group
constexpr int kTile = 128;                   // tokens of a tile
constexpr int kQChunk = kRows * 128;         // 64 values of each row of Q
constexpr int kQBytes = 9 * kQChunk;
constexpr int kStage = 16384;                // 128 tokens x 64 values
constexpr int kRings = 5 * kStage;           // both rings: scores, values
constexpr int kPHalf = kTile * 128;          // weights of 64 rows: 128 tokens x 128 B
constexpr int kCols = 32;                    // rows of the group a softmax thread holds
constexpr int kSoftWarps = 12;

// Warps: fill, softmax (12), MMA (2 of 4).  A bf16 cache is filled by TMA from one thread a ring;
// 4-bit rows are converted by four warps a ring.  Registers a thread at launch, then of each kind
// of warp; the shares of the warpgroups add up to the launch's: 96 + 3 * 112 + 48 = 5 * 96 and
// 2 * 72 + 3 * 96 + 48 = 6 * 80 (with 64 to fill and 104 for the softmax the fill spilled, and the
// 4-bit decode batch of 32 took 734 us, not 593).
template <bool FP4>
struct Roles {
  static constexpr int kFill = FP4 ? 8 : 4, kMma = kFill + kSoftWarps, kThreads = (kMma + 4) * 32;
  static constexpr int kFillRegs = FP4 ? 72 : 96, kSoftRegs = FP4 ? 96 : 112, kMmaRegs = 48;
  // Stages of the rings; a stage of values holds 128 dims of kVTok tokens.  4-bit rows fill two
  // chunks of scores at a time, so that two such pairs make the ring, and values come by 32 tokens.
  static constexpr int kS = FP4 ? 4 : 3, kV = 2, kVTok = FP4 ? 32 : 64, kVStage = kVTok * 256;
  static_assert(kS * kStage + kV * kVStage <= kRings, "rings");
  // A row's reference lies this far (log2 units) below its maximum: fp16 weights use the range
  // up to 2^15, so that 131,072 tokens of 2^-26 of the heaviest still count; bf16 has fp32's range.
  static constexpr float kLift = FP4 ? 7.f : 0.f;
};
constexpr uint32_t kTmemS = 4 * kRows;       // O^T block j at 96 j, the scores behind them
constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;
constexpr float kUnset = -1e38f;             // reference of a row without a token so far
constexpr int64_t kSlotFloats = kRows * kLatV;

struct Group {
  int64_t kv_row0;     // cache row of the sequence's token 0
  int32_t row0;        // first row (token * H + head)
  int32_t nrows;
  int32_t seq_len;     // cache rows of the sequence
  int32_t ntok;        // tokens any of the rows attends to (dense), or entries of the idx row
  int32_t pad0, pad1;
};

struct Plan {          // header of the workspace
  int64_t tiles;       // over all groups
  int32_t groups;
  int32_t bad;         // malformed offsets
  int32_t spoiled;     // entries of Ws::spoiled
  int32_t merges;      // entries of Ws::merge
};

struct Merge {         // a group whose tiles lie in the shares of several blocks
  int32_t row0, nrows, first, last;   // its rows; the first and the last of the blocks
};

struct Ws {
  Plan* plan;
  int32_t* seq_group;   // [B+1] first group of each sequence
  Group* group;         // [max groups]
  int64_t* tile0;       // [max groups + 1] first tile of each group
  int32_t* spoiled;     // [T * H] rows of out to compute again
  Merge* merge;         // [blocks]
  float2* ml;           // [2 * blocks][96] reference and sum of the piece's rows
  float* o;             // [2 * blocks][96][512]
  int64_t max_groups;
  int64_t bytes;
};

// Groups: rows / 96 and one more ragged one per sequence (dense), or per token (selection).
int64_t max_groups(int64_t T, int64_t B, int64_t H) {
  const int64_t dense = T * H / kRows + (B < T ? B : T) + 1, sel = T * ((H + kRows - 1) / kRows);
  return dense > sel ? dense : sel;
}

Ws carve(void* base, int64_t T, int64_t B, int64_t H, int blocks) {
  Ws w;
  w.max_groups = max_groups(T, B, H);
  // parts 256 bytes apart from a 256-byte boundary, wherever the workspace itself starts
  uint8_t* const start = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(base) + 255) & ~uintptr_t(255));
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = start + off;
    off = (off + bytes + 255) & ~int64_t(255);
    return p;
  };
  w.plan = reinterpret_cast<Plan*>(take(sizeof(Plan)));
  w.seq_group = reinterpret_cast<int32_t*>(take(4 * (B + 1)));
  w.group = reinterpret_cast<Group*>(take(sizeof(Group) * w.max_groups));
  w.tile0 = reinterpret_cast<int64_t*>(take(8 * (w.max_groups + 1)));
  w.spoiled = reinterpret_cast<int32_t*>(take(4 * T * H));
  w.merge = reinterpret_cast<Merge*>(take(sizeof(Merge) * blocks));
  w.ml = reinterpret_cast<float2*>(take(sizeof(float2) * kRows * 2 * blocks));
  w.o = reinterpret_cast<float*>(take(4 * kSlotFloats * 2 * blocks));
  w.bytes = off + 256;
  return w;
}

struct Params {
  int T, B, H, k_sel;
  int64_t cache_rows;
  const __nv_bfloat16* q;
  const __nv_bfloat16* kv;     // bf16 cache, or
  const uint8_t* kv4;          // 4-bit cache
  const int32_t* positions;
  const int32_t* q_seq_offsets;
  const int64_t* cache_offsets;
  const int32_t* idx;
  float scale_log2;
  ScoreScale scale;            // the same, for scaled queries
  __nv_bfloat16* out;
  float* lse;
  Ws ws;
  int* err;
  uint64_t timeout_ns;
};

// ---------------------------------------------------------------- plan
__global__ void __launch_bounds__(kPlanThreads) latent_plan_kernel(Params p, int blocks) {
  asm volatile("griddepcontrol.launch_dependents;");

  __shared__ int64_t sums[32];
  const Ws& w = p.ws;
  const int tid = threadIdx.x;
  int bad = 0;
  for (int b = tid; b < p.B; b += kPlanThreads) {
    const int64_t q0 = p.q_seq_offsets[b], q1 = p.q_seq_offsets[b + 1];
    const int64_t c0 = p.cache_offsets[b], c1 = p.cache_offsets[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.T || c0 < 0 || c1 < c0 || c1 > p.cache_rows) bad = 1;
  }
  bad = __syncthreads_or(bad);
  if (bad) {   // merge_kernel writes every row as attending to nothing
    if (tid == 0) {
      w.plan->tiles = 0;
      w.plan->groups = 0;
      w.plan->bad = 1;
      w.plan->spoiled = 0;
      w.plan->merges = 0;
      atomicOr(p.err, kErrOffsets);
    }
    return;
  }
  const int per_tok = (p.H + kRows - 1) / kRows;   // groups of a token (selection)
  int64_t base = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int64_t n = 0;
    if (b < p.B) {
      const int64_t nq = p.q_seq_offsets[b + 1] - p.q_seq_offsets[b];
      n = p.k_sel >= 0 ? nq * per_tok : (nq * p.H + kRows - 1) / kRows;
    }
    const int64_t inc = block_scan(n, sums);
    if (b < p.B) w.seq_group[b + 1] = static_cast<int32_t>(base + inc);
    base += sums[31];
  }
  if (tid == 0) w.seq_group[0] = 0;
  __syncthreads();
  const int groups = static_cast<int>(base);
  int64_t tiles = 0;
  int oob = 0;
  for (int g0 = 0; g0 < groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    int64_t nt = 0;
    if (g < groups) {
      int lo = 0, hi = p.B - 1;   // the last sequence whose first group is at or below g
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (w.seq_group[mid] <= g) lo = mid;
        else hi = mid - 1;
      }
      const int k = g - w.seq_group[lo];
      const int q0 = p.q_seq_offsets[lo], q1 = p.q_seq_offsets[lo + 1];
      Group gr;
      gr.kv_row0 = p.cache_offsets[lo];
      gr.seq_len = static_cast<int32_t>(p.cache_offsets[lo + 1] - gr.kv_row0);
      gr.pad0 = gr.pad1 = 0;
      if (p.k_sel >= 0) {
        const int h0 = (k % per_tok) * kRows;
        gr.row0 = (q0 + k / per_tok) * p.H + h0;
        gr.nrows = p.H - h0 < kRows ? p.H - h0 : kRows;
        gr.ntok = p.k_sel;
      } else {
        gr.row0 = q0 * p.H + k * kRows;
        const int left = q1 * p.H - gr.row0;
        gr.nrows = left < kRows ? left : kRows;
        int top = -1;
        for (int t = gr.row0 / p.H; t <= (gr.row0 + gr.nrows - 1) / p.H; ++t) {
          const int pos = p.positions[t];
          if (pos < -1 || pos >= gr.seq_len) oob = 1;
          else top = pos > top ? pos : top;
        }
        gr.ntok = top + 1;
      }
      nt = gr.ntok > 0 ? (gr.ntok + kTile - 1) / kTile : 1;   // an empty group still writes its rows
      w.group[g] = gr;
    }
    const int64_t inc = block_scan(nt, sums);
    if (g < groups) w.tile0[g] = tiles + inc - nt;
    tiles += sums[31];
  }
  if (oob) atomicOr(p.err, kErrBounds);
  if (tid == 0) {
    w.tile0[groups] = tiles;
    w.plan->tiles = tiles;
    w.plan->groups = groups;
    w.plan->bad = 0;
    w.plan->spoiled = 0;
  }
  // groups that several blocks share
  int* const count = reinterpret_cast<int*>(sums);
  __syncthreads();
  if (tid == 0) *count = 0;
  __syncthreads();
  for (int g = tid; g < groups; g += kPlanThreads) {
    const int first = share_of(tiles, w.tile0[g], blocks), last = share_of(tiles, w.tile0[g + 1] - 1, blocks);
    if (first != last) w.merge[atomicAdd(count, 1)] = Merge{w.group[g].row0, w.group[g].nrows, first, last};
  }
  __syncthreads();
  if (tid == 0) w.plan->merges = *count;
}

// ---------------------------------------------------------------- pieces of PTX
// Lane c gets the maximum (or the sum) over the warp of v[c]: each step exchanges half of what is
// left, 31 shuffles in all (one reduction a column took 160, and the path runs cold).
template <bool MAX>
__device__ __forceinline__ float reduce_columns(float (&v)[kCols], int lane) {
#pragma unroll
  for (int w = 16; w; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + w], w);
      const float own = up ? v[i + w] : v[i];
      v[i] = MAX ? fmaxf(own, got) : own + got;
    }
  }
  return v[0];
}

// 32 consecutive fp32 columns of the warp's TMEM lanes, and the wait for them
__device__ __forceinline__ void tmem_ld32(uint32_t a, float (&x)[kCols]) {
  uint32_t r[32];
  tmem_ld_32cols(a, r);
  tmem_ld_wait(r);
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
}

// ---------------------------------------------------------------- 4-bit rows
// 32 values of a row: four words of codes (first value in the lowest nibble) and two scales.  Four
// neighbouring lanes take 128 values of a row, so that a load touches eight lines, not 32 (with a
// row a lane the loads alone kept the memory pipe busy for 9,000 cycles a tile).
struct Fp4Raw {
  uint4 w;
  uint32_t sc;
};

__device__ __forceinline__ Fp4Raw fp4_load(const uint8_t* base, int pos, int group) {
  Fp4Raw f = {};
  if (pos >= 0) {
    const uint8_t* const row = base + static_cast<int64_t>(pos) * kLatRow4;
    f.w = *reinterpret_cast<const uint4*>(row + 16 * group);
    f.sc = *reinterpret_cast<const uint16_t*>(row + kLatCodes + 2 * group);
  }
  return f;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Eight codes as eight fp16 values times their scale (exact: at most 2 + 4 significant bits, and
// magnitudes from 2^-10 to 2,880)
__device__ __forceinline__ uint4 fp4_word(uint32_t w, uint32_t s2) {
  uint4 r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "r"(w));
  return make_uint4(mul_f16x2(r.x, s2), mul_f16x2(r.y, s2), mul_f16x2(r.z, s2), mul_f16x2(r.w, s2));
}

// The 32 values as four 16-byte units of a 128-byte row r of a swizzled chunk (unit u at unit
// u ^ (r & 7)): the row's first four or last four (`upper`).  The lanes of a row's second chunk
// (`second`) store their units in another order, so that eight lanes never meet in a bank.
__device__ __forceinline__ void fp4_store(uint8_t* row, int r, bool upper, bool second, Fp4Raw f) {
  if (second) {
    f.w = make_uint4(f.w.z, f.w.w, f.w.x, f.w.y);
    f.sc = (f.sc >> 8) | (f.sc << 8);
  }
  const uint32_t w[4] = {f.w.x, f.w.y, f.w.z, f.w.w};
  const int u0 = (upper ? 4 : 0) ^ (second ? 2 : 0) ^ (r & 7);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    // e4m3 bits moved to fp16's fields read as 2^-8 of the scale, subnormals too
    const uint32_t s2 = mul_f16x2(((f.sc >> (8 * k)) & 0x7Fu) * 0x00800080u, 0x5C005C00u);
#pragma unroll
    for (int j = 0; j < 2; ++j) *reinterpret_cast<uint4*>(row + ((u0 ^ (2 * k + j)) * 16)) = fp4_word(w[2 * k + j], s2);
  }
}

// ---------------------------------------------------------------- attention
struct alignas(16) Misc {
  uint64_t full_s[4], empty_s[4];
  uint64_t full_v[2], empty_v[2], zero_req[2], zeroed[2];
  uint64_t q_full, q_empty, s_full, s_empty, p_full, pv_done, mma_done;
  uint32_t tmem;
  int abort;
  int first_group;
  int pad;
  alignas(16) float nm[kRows];       // minus the reference of each row (log2 units)
  alignas(16) float f[kRows];        // factor of a raised reference; at the end 1 / sum
  alignas(16) float qs[2][kRows];    // 4-bit cache: each row's factor to log2 units, pieces in turn
  alignas(16) int limit[kRows];      // last position the row attends to
  alignas(16) float red[kSoftWarps][kCols];
  int spoiled[kRows];                // the row's sums hold a NaN that its weights do not
};

constexpr int kOffRing = kQBytes;
constexpr int kOffP = kOffRing + kRings;
constexpr int kOffMisc = kOffP + 2 * kPHalf;
constexpr int kSmem = kOffMisc + static_cast<int>(sizeof(Misc)) + 1024;
static_assert(kSmem <= 232448, "shared memory per block");

// One block's walk over its pieces of groups, the same for every role.
struct Piece {
  Group g;
  int gi;         // group
  int t0, n;      // first tile inside the group, number of tiles
  bool first, last;   // holds the group's first / last tile
};

struct Walk {
  int64_t at, end;
  int gi;
  const Ws& w;
  __device__ Walk(const Ws& ws, int64_t a, int64_t b, int g) : at(a), end(b), gi(g), w(ws) {}
  __device__ bool next(Piece* p) {
    if (at >= end) return false;
    const int64_t s = w.tile0[gi], e = w.tile0[gi + 1];
    p->g = w.group[gi];
    p->gi = gi;
    p->t0 = static_cast<int>(at - s);
    const int64_t stop = e < end ? e : end;
    p->n = static_cast<int>(stop - at);
    p->first = at == s;
    p->last = stop == e;
    at = stop;
    ++gi;
    return true;
  }
};

// tokens of the group that tile t holds
__device__ __forceinline__ int tile_tokens(const Group& g, int t) {
  const int left = g.ntok - t * kTile;
  return left < kTile ? left : kTile;
}

// A thread's dims (tok, 128 + tok, ...) of 32 rows of a finished piece: out = sums * f, or the sums
// as they are to a slot of the workspace.  Not inlined: its addresses, live across the tiles'
// loop, would push the loop's own values out of the registers.
template <bool FP4>
__device__ __noinline__ void write_sums(const Params& p, const float* f, int* spoiled, uint32_t tlane, int tok, int c0,
                                        int row0, int nrows, bool any, float* slot) {
  const int lane = tok & 31;
#pragma unroll 1
  for (int u = 0; u < 8; ++u) {
    const int j = u & 3, cb = c0 + (u >> 2) * 16;         // block of dims, first of 16 rows
    if (cb >= nrows) break;
    float o[16];
    if (any) tmem_ld16(tlane + j * kRows + cb, o);
    const int dim = 128 * j + tok;
    if (!slot) {
      // even lanes keep row c, odd lanes row c + 1, each with its pair of dims
      __nv_bfloat16* const ob = p.out + static_cast<int64_t>(row0 + cb + (lane & 1)) * kLatV + (dim & ~1);
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const float i0 = f[cb + c], i1 = f[cb + c + 1];
        const float v0 = i0 != 0.f ? o[c] * i0 : 0.f, v1 = i1 != 0.f ? o[c + 1] * i1 : 0.f;
        if (!FP4) {
          if (v0 != v0 && i0 == i0) spoiled[cb + c] = 1;
          if (v1 != v1 && i1 == i1) spoiled[cb + c + 1] = 1;
        }
        const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? v0 : v1, 1);
        const uint32_t pr = lane & 1 ? pack2(got, v1) : pack2(v0, got);
        if (cb + c + (lane & 1) < nrows) *reinterpret_cast<uint32_t*>(ob + c * kLatV) = pr;
      }
    } else {
      float* const ob = slot + static_cast<int64_t>(cb) * kLatV + dim;
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (cb + c < nrows) ob[c * kLatV] = o[c];
    }
  }
}

template <bool FP4>
__global__ void __launch_bounds__(Roles<FP4>::kThreads, 1)
    latent_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmC,
                            const __grid_constant__ Params p) {
  using R = Roles<FP4>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sQ = smem;
  uint8_t* const sRing = smem + kOffRing;
  uint8_t* const sRingV = sRing + Roles<FP4>::kS * kStage;
  uint8_t* const sP = smem + kOffP;
  Misc& mi = *reinterpret_cast<Misc*>(smem + kOffMisc);

  constexpr int kMmaWarp = R::kMma;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Ws& w = p.ws;
  if (threadIdx.x == 0) {
    for (int s = 0; s < R::kS; ++s) {
      mbar_init(&mi.full_s[s], FP4 ? 128 : 1);
      mbar_init(&mi.empty_s[s], 1);
    }
    for (int s = 0; s < R::kV; ++s) {
      mbar_init(&mi.full_v[s], FP4 ? 128 : 1);
      mbar_init(&mi.empty_v[s], 1);
      mbar_init(&mi.zero_req[s], 1);
      mbar_init(&mi.zeroed[s], 1);
    }
    mbar_init(&mi.q_full, FP4 ? 128 : 1);
    mbar_init(&mi.q_empty, 1);
    mbar_init(&mi.s_full, 1);
    mbar_init(&mi.s_empty, kSoftWarps);
    mbar_init(&mi.p_full, kSoftWarps);
    mbar_init(&mi.pv_done, 1);
    mbar_init(&mi.mma_done, 2);
    mi.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&mi.tmem, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int64_t a0, a1;
  share(w.plan->tiles, blockIdx.x, gridDim.x, &a0, &a1);
  if (warp == 0 && a0 < a1) {
    // the group that holds tile a0: the last whose first tile is at or below it (32 probes a step)
    int lo = 0, n = w.plan->groups;
    while (n > 1) {
      const int step = (n + 31) / 32, i = lo + lane * step;
      const unsigned in = __ballot_sync(0xffffffffu, lane * step < n && w.tile0[i] <= a0);
      const int k = 31 - __clz(in);
      lo += k * step;
      n = n - k * step < step ? n - k * step : step;
    }
    if (lane == 0) mi.first_group = lo;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, mi.tmem, 0);
  const WaitCtl wc{p.err, &mi.abort, p.timeout_ns};
  Walk walk(w, a0, a1, mi.first_group);
  Piece pc;

  if (warp < R::kFill) {
    if (FP4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kFillRegs));
    // ============================================================ fill
    // stage `it` of a ring may be written once its previous contents have been read
    auto acquire = [&](uint64_t* empty, uint32_t it, uint32_t n) {
      return it < n || mbar_wait(&empty[it % n], (it / n - 1) & 1, wc);
    };
    // on an early exit the loads in flight land before the block ends
    auto drain = [&](uint64_t* bar, uint32_t parity) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(smem_u32(bar), parity) && global_timer_ns() - t0 <= kDrainNs) {
      }
    };
    // L2 keeps a tile between its two readings: without these hints 1.8 times the cache's bytes came
    // from memory (64 sequences of 8,192 tokens), and the decode batch of 64 takes 1.59 ms, not 1.49
    // (a prompt chunk, whose cache L2 holds anyway, 743 us, not 754).  Fetching the next tile into L2
    // as well made room for less of that and was a tenth slower.
    const uint64_t keep = l2_policy_evict_last(), drop = l2_policy_evict_first();
    uint32_t it = 0;        // stages of the warp's ring so far
    uint32_t segs = 0;      // pieces so far
    bool ok = true;
    if constexpr (FP4) {
      const bool scores = warp < 4;
      const int w4 = warp & 3, sub = lane >> 2, quad = lane & 3;   // row of eight, part of a row
      const bool upper = quad & 1, second = quad >> 1;
      while (ok && walk.next(&pc)) {
        if (pc.g.ntok == 0) continue;
        const uint8_t* const base = p.kv4 + pc.g.kv_row0 * kLatRow4;
        const int32_t* const sel = p.k_sel >= 0 ? p.idx + static_cast<int64_t>(pc.g.row0 / p.H) * p.k_sel : nullptr;
        // position of token j of tile t in the sequence, or -1
        auto pos_of = [&](int t, int j) {
          const int k = t * kTile + j;
          if (k >= pc.g.ntok) return -1;
          if (!sel) return k;
          const int pos = sel[k];
          if (pos >= pc.g.seq_len) atomicOr(p.err, kErrBounds);
          return pos < pc.g.seq_len ? pos : -1;
        };
        if (scores) {
          // Q with its latent part in fp16 (the type of the cache's values) and its rope part in
          // bf16, both times a power of two that fits the row into fp16
          if (segs > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait(&mi.q_empty, (segs - 1) & 1, wc)))) break;
          const uint32_t* const qsrc = reinterpret_cast<const uint32_t*>(p.q) + static_cast<int64_t>(pc.g.row0) * (kLatDim / 2) + lane;
#pragma unroll 2
          for (int rr = warp; rr < kRows; rr += 4) {
            uint32_t v[9], top = 0u;
#pragma unroll
            for (int c = 0; c < 9; ++c) v[c] = rr < pc.g.nrows ? qsrc[rr * (kLatDim / 2) + 32 * c] : 0u;
#pragma unroll
            for (int c = 0; c < 9; ++c) top = __vmaxu2(top, v[c] & 0x7FFF7FFFu);
            top = __reduce_max_sync(0xffffffffu, top >> 16 > (top & 0xFFFFu) ? top >> 16 : top & 0xFFFFu);
            const int f = scale_exponent(__uint_as_float(top << 16), kLowestFactor);
            const float inv = pow2(-f);
#pragma unroll
            for (int c = 0; c < 9; ++c) {
              const float lo = __uint_as_float(v[c] << 16) * inv, hi = __uint_as_float(v[c] & 0xFFFF0000u) * inv;
              *reinterpret_cast<uint32_t*>(sQ + c * kQChunk + rr * 128 + (((lane >> 2) ^ (rr & 7)) * 16) + (lane & 3) * 4) =
                  c < 8 ? pack_f16(lo, hi) : pack2(lo, hi);
            }
            if (lane == 0) mi.qs[segs & 1][rr] = score_factor(p.scale, f);
          }
          fence_proxy_async_smem();
          mbar_arrive(&mi.q_full);
          ++segs;
          auto prefetch = [&](int t) {
            if (t >= pc.t0 + pc.n) return;
            if (!sel) {            // rows follow one another: one instruction for all
              if (threadIdx.x == 0) prefetch_l2(base + static_cast<int64_t>(t) * kTile * kLatRow4, tile_tokens(pc.g, t) * kLatRow4);
              return;
            }
            const int pos = pos_of(t, threadIdx.x & 127);
            if (pos < 0) return;
            const uint8_t* const r = base + static_cast<int64_t>(pos) * kLatRow4;
#pragma unroll
            for (int k = 0; k < 4; ++k) asm volatile("prefetch.global.L2 [%0];" ::"l"(r + 128 * k));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(r + kLatRow4 - 16));
          };
          prefetch(pc.t0);
          for (int t = pc.t0; t < pc.t0 + pc.n && ok; ++t) {
            prefetch(t + 1);
            // the warp's 32 rows, eight at a time; two chunks (128 values) together
            int pos[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) pos[k] = pos_of(t, 32 * w4 + 8 * k + sub);
            Fp4Raw nx[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) nx[k] = fp4_load(base, pos[k], quad);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              Fp4Raw cur[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) cur[k] = nx[k];
              if (c < 3) {
#pragma unroll
                for (int k = 0; k < 4; ++k) nx[k] = fp4_load(base, pos[k], 4 * (c + 1) + quad);
              }
              const uint32_t s0 = it % R::kS, s1 = (it + 1) % R::kS;
              if (!(ok = __all_sync(0xffffffffu, acquire(mi.empty_s, it, R::kS) && acquire(mi.empty_s, it + 1, R::kS)))) break;
              uint8_t* const dst = sRing + (second ? s1 : s0) * kStage;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int r = 32 * w4 + 8 * k + sub;
                // a missing token's score is masked, whatever its row holds
                if (pos[k] >= 0) fp4_store(dst + r * 128, r, upper, second, cur[k]);
              }
              fence_proxy_async_smem();
              mbar_arrive(&mi.full_s[s0]);
              mbar_arrive(&mi.full_s[s1]);
              it += 2;
            }
            if (!ok) break;
            // the rope keys: eight lanes a row, a warp's four rows at a time
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int r = 4 * k + (lane >> 3);           // of the warp's 32; lane 4 (r & 7) holds its position
              const int a = __shfl_sync(0xffffffffu, pos[k >> 1], 4 * (r & 7));
              v[k] = a >= 0 ? *reinterpret_cast<const uint4*>(base + static_cast<int64_t>(a) * kLatRow4 + kLatCodes + kLatScales + 16 * (lane & 7))
                            : make_uint4(0u, 0u, 0u, 0u);
            }
            const uint32_t s = it % R::kS;
            if (!(ok = __all_sync(0xffffffffu, acquire(mi.empty_s, it, R::kS)))) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int r = 32 * w4 + 4 * k + (lane >> 3);
              *reinterpret_cast<uint4*>(sRing + s * kStage + r * 128 + (((lane & 7) ^ (r & 7)) * 16)) = v[k];
            }
            fence_proxy_async_smem();
            mbar_arrive(&mi.full_s[s]);
            ++it;
          }
        } else {
          for (int t = pc.t0; t < pc.t0 + pc.n && ok; ++t) {
            const int parts = (tile_tokens(pc.g, t) + R::kVTok - 1) / R::kVTok;
            // the warp's eight rows of each 32
            int pos[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) pos[k] = pos_of(t, 32 * k + 8 * w4 + sub);
#pragma unroll 1
            for (int j = 0; j < 4 && ok; ++j) {
              Fp4Raw raw[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) raw[k] = fp4_load(base, pos[k], 4 * j + quad);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k == parts) break;
                if (!(ok = acquire(mi.empty_v, it, R::kV))) break;
                const uint32_t s = it % R::kV;
                const int r = 8 * w4 + sub;                 // a missing token: codes and scales of zero
                fp4_store(sRingV + s * R::kVStage + (second ? R::kVStage / 2 : 0) + r * 128, r, upper, second, raw[k]);
                fence_proxy_async_smem();
                mbar_arrive(&mi.full_v[s]);
                ++it;
              }
            }
          }
        }
      }
    } else if (warp == 0 && lane == 0) {
      // scores: nine 64-value chunks of a tile
      while (ok && walk.next(&pc)) {
        if (pc.g.ntok == 0) continue;
        if (segs > 0 && !(ok = mbar_wait(&mi.q_empty, (segs - 1) & 1, wc))) break;
        mbar_arrive_expect_tx(&mi.q_full, kQBytes);
        for (int c = 0; c < 9; ++c) tma_load_2d(sQ + c * kQChunk, &tmQ, &mi.q_full, 64 * c, pc.g.row0);
        ++segs;
        for (int t = pc.t0; t < pc.t0 + pc.n && ok; ++t) {
          const bool two = tile_tokens(pc.g, t) > 64;
          const int y = static_cast<int>(pc.g.kv_row0) + t * kTile;
          for (int c = 0; c < 9; ++c) {
            if (!(ok = acquire(mi.empty_s, it, R::kS))) break;
            const uint32_t s = it % R::kS;
            mbar_arrive_expect_tx(&mi.full_s[s], two ? kStage : kStage / 2);
            const uint64_t pol = c < 8 ? keep : drop;
            tma_load_2d_hint(sRing + s * kStage, &tmC, &mi.full_s[s], 64 * c, y, pol);
            if (two) tma_load_2d_hint(sRing + s * kStage + kStage / 2, &tmC, &mi.full_s[s], 64 * c, y + 64, pol);
            ++it;
          }
        }
      }
      if (!ok) {
        for (uint32_t k = it > R::kS ? it - R::kS : 0; k < it; ++k)
          drain(&mi.full_s[k % R::kS], (k / R::kS) & 1);
        if (segs > 0) drain(&mi.q_full, (segs - 1) & 1);
      }
    } else if (warp == 1 && lane == 0) {
      // values: 64 tokens x 128 dims a stage
      while (ok && walk.next(&pc)) {
        if (pc.g.ntok == 0) continue;
        for (int t = pc.t0; t < pc.t0 + pc.n && ok; ++t) {
          const int v = tile_tokens(pc.g, t), halves = v > 64 ? 2 : 1;
          for (int k = 0; k < 4 * halves; ++k) {
            const int j = halves == 2 ? k >> 1 : k, hf = halves == 2 ? k & 1 : 0;
            const int y = static_cast<int>(pc.g.kv_row0) + t * kTile + 64 * hf;
            if (!(ok = acquire(mi.empty_v, it, R::kV))) break;
            const uint32_t s = it % R::kV;
            mbar_arrive_expect_tx(&mi.full_v[s], kStage);
            tma_load_2d_hint(sRingV + s * R::kVStage, &tmC, &mi.full_v[s], 128 * j, y, drop);
            tma_load_2d_hint(sRingV + s * R::kVStage + kStage / 2, &tmC, &mi.full_v[s], 128 * j + 64, y, drop);
            if (hf == halves - 1 && (v & 15)) mbar_arrive(&mi.zero_req[s]);
            ++it;
          }
        }
      }
      if (!ok)
        for (uint32_t k = it > R::kV ? it - R::kV : 0; k < it; ++k)
          drain(&mi.full_v[k % R::kV], (k / R::kV) & 1);
    } else if (warp == 2) {
      // zero the rows of a group's last tile that its MMAs read behind its last token
      uint32_t ph = 0;      // per-stage phase bits of zero_req
      while (ok && walk.next(&pc)) {
        if (pc.g.ntok == 0) continue;
        uint32_t stages = 0;
        for (int t = 0; t < pc.n; ++t) stages += tile_tokens(pc.g, pc.t0 + t) > 64 ? 8 : 4;
        const int v = tile_tokens(pc.g, pc.t0 + pc.n - 1);
        if (pc.last && (v & 15)) {
          const int halves = v > 64 ? 2 : 1;
          const int r0 = v - 64 * (halves - 1), r1 = (r0 + 15) & ~15;
          for (int j = 0; j < 4 && ok; ++j) {
            const uint32_t at = it + stages - 4 * halves + j * halves + (halves - 1), s = at % R::kV;
            ok = mbar_wait(&mi.zero_req[s], (ph >> s) & 1, wc) && mbar_wait(&mi.full_v[s], (at / R::kV) & 1, wc);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            ph ^= 1u << s;
            for (int u = lane; u < (r1 - r0) * 16; u += 32) {
              const int r = r0 + (u >> 4), un = u & 15;
              *reinterpret_cast<uint4*>(sRingV + s * R::kVStage + (un >> 3) * 8192 + r * 128 + (un & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&mi.zeroed[s]);
          }
        }
        it += stages;
      }
    }
    __syncwarp();
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kSoftRegs));
    // ============================================================ softmax
    const int wg = (warp - R::kFill) >> 2, qd = warp & 3;
    const int tok = qd * 32 + lane;                       // token of the tile, TMEM lane
    const uint32_t tlane = tmem + (static_cast<uint32_t>(qd * 32) << 16);
    const int wtid = (warp - R::kFill - 4 * wg) * 32 + lane;
    const int bar_id = 1 + wg;
    uint32_t done = 0, segs = 0;      // tiles and pieces with tokens so far
    // A wait that ran out is skipped from then on, but the walk goes on to its end: the warps of
    // a third meet at named barriers and none may leave the others there.  The results are then
    // worthless, and the error word says so.
    bool ok = true;
    while (walk.next(&pc)) {
      const Group& g = pc.g;
      // columns (rows of the group) of this third, of the N of the MMAs
      const int n16 = (g.nrows + 15) / 16 * 16, c0 = kCols * wg;
      const int nc = n16 - c0 < 0 ? 0 : n16 - c0 < kCols ? n16 - c0 : kCols;
      // rows' references and limits; columns without a row never raise theirs and weigh nothing
      int lim = -1;
      if (wtid < kCols) {
        const int r = c0 + wtid;
        const bool real = r < g.nrows;
        if (p.k_sel >= 0) {
          lim = 0;
        } else if (real) {
          lim = p.positions[(g.row0 + r) / p.H];
          if (lim >= g.seq_len || lim < -1) lim = -1;
        }
        mi.nm[r] = real ? -kUnset : -INFINITY;
        mi.limit[r] = lim;
        mi.spoiled[r] = 0;
        if (!real) lim = 0x7FFFFFFF;
      } else {
        lim = 0x7FFFFFFF;
      }
      int low = __reduce_min_sync(0xffffffffu, lim);   // of the third's rows (all in its first warp)
      if (wtid == 0) mi.red[warp - R::kFill][0] = __int_as_float(low);
      named_bar_sync(bar_id, 128);
      low = __float_as_int(mi.red[4 * wg][0]);
      named_bar_sync(bar_id, 128);
      float l = 0.f;          // lane c: sum of row c0 + c over the warp's tokens
      const int32_t* const sel = p.k_sel >= 0 ? p.idx + static_cast<int64_t>(g.row0 / p.H) * p.k_sel : nullptr;
      const float4* const nm4 = reinterpret_cast<const float4*>(mi.nm + c0);

      for (int t = 0; g.ntok > 0 && t < pc.n; ++t, ++done) {
        const int first_pos = (pc.t0 + t) * kTile;
        int pos = first_pos + tok;
        const bool masked = sel || first_pos + kTile - 1 > low;
        if (sel) {
          const int e = pos < g.ntok ? sel[pos] : -1;
          pos = e >= 0 && e < g.seq_len ? 0 : 0x7FFFFFFF;
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&mi.s_full, done & 1, wc));
        tc_fence_after();
        // y = x - m (log2 units) of the token against the rows, and their maximum
        float2 y[kCols / 2];
        float top = -INFINITY;
        auto scores = [&]() {
          float x[kCols];
          tmem_ld32(tlane + kTmemS + c0, x);
          if (masked) {
            const int4* const l4 = reinterpret_cast<const int4*>(mi.limit + c0);
#pragma unroll
            for (int c = 0; c < kCols / 4; ++c) {
              const int4 v = l4[c];
              x[4 * c] = pos <= v.x ? x[4 * c] : -INFINITY;
              x[4 * c + 1] = pos <= v.y ? x[4 * c + 1] : -INFINITY;
              x[4 * c + 2] = pos <= v.z ? x[4 * c + 2] : -INFINITY;
              x[4 * c + 3] = pos <= v.w ? x[4 * c + 3] : -INFINITY;
            }
          }
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) y[c] = make_float2(x[2 * c], x[2 * c + 1]);
        };
        const float4* const qs4 = reinterpret_cast<const float4*>(mi.qs[segs & 1] + c0);
        auto shift = [&]() {
#pragma unroll
          for (int c = 0; c < kCols / 4; ++c) {
            const float4 m = nm4[c];
            float4 k = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
            if (FP4) k = qs4[c];
            y[2 * c] = ffma2(y[2 * c], make_float2(k.x, k.y), make_float2(m.x, m.y));
            y[2 * c + 1] = ffma2(y[2 * c + 1], make_float2(k.z, k.w), make_float2(m.z, m.w));
          }
        };
        if (nc > 0) {
          scores();
          shift();
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) top = fmaxf(top, fmaxf(y[c].x, y[c].y));
        }
        if (named_bar_or(bar_id, 128, top > R::kLift + 8.f)) {
          // some row's reference rises: the tile's maximum of every row, over the tokens
          scores();
          {
            float v[kCols];
#pragma unroll
            for (int c = 0; c < kCols; ++c) v[c] = c & 1 ? y[c / 2].y : y[c / 2].x;
            mi.red[warp - R::kFill][lane] = reduce_columns<true>(v, lane);
          }
          named_bar_sync(bar_id, 128);
          if (wtid < nc) {
            float v = -INFINITY;
            for (int k = 0; k < 4; ++k) v = fmaxf(v, mi.red[4 * wg + k][wtid]);
            v = __fmul_rn(v, FP4 ? mi.qs[segs & 1][c0 + wtid] : p.scale_log2);
            const float old = -mi.nm[c0 + wtid];
            const float now = v > old + R::kLift + 8.f ? v - R::kLift : old;
            mi.nm[c0 + wtid] = -now;
            mi.f[c0 + wtid] = ex2_approx(old - now);
          }
          named_bar_sync(bar_id, 128);
          scores();      // again: kept across the reduction they would not fit the registers
          // The difference of the rounded product and the reference, which is one: next to it that is
          // exact, however large the scores.  A lift lost in rounding makes no weight past the type's
          // range (NaN stays).
          auto less = [](float x, float k, float nm) {
            const float v = __fadd_rn(__fmul_rn(x, k), nm);
            return v > R::kLift + 8.f ? R::kLift + 8.f : v;
          };
#pragma unroll
          for (int c = 0; c < kCols / 4; ++c) {
            const float4 m = nm4[c];
            float4 k = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
            if (FP4) k = qs4[c];
            y[2 * c] = make_float2(less(y[2 * c].x, k.x, m.x), less(y[2 * c].y, k.y, m.y));
            y[2 * c + 1] = make_float2(less(y[2 * c + 1].x, k.z, m.z), less(y[2 * c + 1].y, k.w, m.w));
          }
          l *= mi.f[c0 + lane];
          if (t > 0) {
            // the sums so far, once every earlier product has landed in them
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&mi.pv_done, (done - 1) & 1, wc));
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
#pragma unroll 1
              for (int cc = 0; cc < nc; cc += 16) {
                float o[16];
                const uint32_t a = tlane + j * kRows + c0 + cc;
                tmem_ld16(a, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= mi.f[c0 + cc + k];
                tmem_st16(a, o);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.s_empty);
        // weights: 2^y, summed before their rounding to the values' type, the operand type of the
        // product (lse keeps fp32's precision; out gets one rounding a weight, of up to 2^-8 in
        // bf16; in fp16 2^-11, and 2^-32 of the largest where a weight is below 2^-21 of it)
        uint32_t pk[kCols / 2];
        if (nc > 0) {
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {
            y[c] = make_float2(ex2_approx(y[c].x), ex2_approx(y[c].y));
            pk[c] = FP4 ? pack_f16(y[c].x, y[c].y) : pack2(y[c].x, y[c].y);
          }
        }
        // the weights' place in shared memory is free once the previous tile's product is done
        if (done > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&mi.pv_done, (done - 1) & 1, wc));
        if (nc > 0) {
#pragma unroll
          for (int u = 0; u < kCols / 8; ++u) {
            const int col = c0 + 8 * u;
            *reinterpret_cast<uint4*>(sP + (col >> 6) * kPHalf + tok * 128 + ((((col & 63) >> 3) ^ (tok & 7)) * 16)) =
                make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.p_full);
        // the rows' sums over the warp's tokens (32 sums a thread instead did not fit the registers)
        if (nc > 0) l += reduce_columns<false>(reinterpret_cast<float(&)[kCols]>(y), lane);
      }
      if (g.ntok > 0) ++segs;
      // the rows' sums over the warps
      named_bar_sync(bar_id, 128);
      mi.red[warp - R::kFill][lane] = l;
      named_bar_sync(bar_id, 128);
      const bool whole = pc.first && pc.last;
      const int slot = 2 * blockIdx.x + (pc.first ? 1 : 0);     // head pieces 0, tail pieces 1
      if (wtid < nc) {
        float sum = 0.f;
        for (int k = 0; k < 4; ++k) sum += mi.red[4 * wg + k][wtid];
        const int r = c0 + wtid;
        mi.f[r] = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        if (r < g.nrows) {
          const float m = -mi.nm[r];
          if (whole) p.lse[g.row0 + r] = sum == 0.f ? -INFINITY : fmaf(m, 0.69314718055994531f, logf(sum));
          else w.ml[static_cast<int64_t>(slot) * kRows + r] = make_float2(m, sum);
        }
      }
      named_bar_sync(bar_id, 128);
      if (g.ntok > 0) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&mi.pv_done, (done - 1) & 1, wc));
        tc_fence_after();
      }
      if (nc > 0)
        write_sums<FP4>(p, mi.f, mi.spoiled, tlane, tok, c0, g.row0, g.nrows, g.ntok > 0,
                        whole ? nullptr : w.o + slot * kSlotFloats);
      tc_fence_before();
      named_bar_sync(bar_id, 128);   // f, m and red are free for the next piece
      if (!FP4 && whole && wtid < nc && c0 + wtid < g.nrows && mi.spoiled[c0 + wtid])
        w.spoiled[atomicAdd(&w.plan->spoiled, 1)] = g.row0 + c0 + wtid;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kMmaRegs));
    // ============================================================ MMA issuers
    // One warp for the scores, one for the values: issuing takes 73 and 117 cycles an instruction
    // (its operands move to uniform registers), more than the 56 it runs for.  The whole warp walks
    // along and one elected lane issues (with a single lane in the loop 150 and 240 cycles).
    if (warp < kMmaWarp + 2) {
      const bool leader = elect_one();
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc)); };
      auto commit = [&](uint64_t* bar) {
        if (leader) umma_commit(bar);
      };
      uint32_t nth = 0;       // tiles so far
      if (warp == kMmaWarp) {
        Ring<R::kS> rg;
        uint32_t segs = 0;
        const uint32_t q_lo = desc_lo(smem_u32(sQ), 16), r_lo = desc_lo(smem_u32(sRing), 16);   // K-major
        while (ok && walk.next(&pc)) {
          if (pc.g.ntok == 0) continue;
          const int n16 = (pc.g.nrows + 15) / 16 * 16;
          if (!(ok = wait(&mi.q_full, segs & 1))) break;
          ++segs;
          for (int t = 0; t < pc.n && ok; ++t, ++nth) {
            if (nth > 0 && !(ok = wait(&mi.s_empty, (nth - 1) & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 9; ++c) {
              if (!(ok = wait(&mi.full_s[rg.s], rg.phase))) break;
              tc_fence_after();
              const uint32_t a = r_lo + rg.s * (kStage >> 4), b = q_lo + c * (kQChunk >> 4);
              const uint32_t idesc = FP4 && c < 8 ? idesc_f16(128, n16) : umma_idesc_bf16(128, n16);
#pragma unroll
              for (int k = 0; k < 4; ++k) umma_lo(tmem + kTmemS, a + 2 * k, b + 2 * k, idesc, (c | k) != 0, leader);
              commit(&mi.empty_s[rg.s]);
              rg.next();
            }
            if (!ok) break;
            commit(&mi.s_full);
            if (t == pc.n - 1) commit(&mi.q_empty);
          }
        }
      } else {
        Ring<R::kV> rg;
        uint32_t zph = 0;
        const uint32_t v_lo = desc_lo(smem_u32(sRingV), R::kVStage / 2), p_lo = desc_lo(smem_u32(sP), kPHalf);   // MN-major
        while (ok && walk.next(&pc)) {
          const Group& g = pc.g;
          if (g.ntok == 0) continue;
          const int n16 = (g.nrows + 15) / 16 * 16;
          const uint32_t idesc = (FP4 ? idesc_f16(128, n16) : umma_idesc_bf16(128, n16)) | (1u << 15) | (1u << 16);
          for (int t = 0; t < pc.n && ok; ++t, ++nth) {
            const int v = tile_tokens(g, pc.t0 + t), parts = (v + R::kVTok - 1) / R::kVTok;
            const bool zero = !FP4 && pc.last && t == pc.n - 1 && (v & 15);
            if (!(ok = wait(&mi.p_full, nth & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < 4 && ok; ++j) {
#pragma unroll 1
              for (int part = 0; part < parts; ++part) {
                if (zero && part == parts - 1) {
                  if (!(ok = wait(&mi.zeroed[rg.s], (zph >> rg.s) & 1))) break;
                  zph ^= 1u << rg.s;
                }
                if (!(ok = wait(&mi.full_v[rg.s], rg.phase))) break;
                tc_fence_after();
                const int left = v - R::kVTok * part;
                const uint32_t a = v_lo + rg.s * (R::kVStage >> 4), b = p_lo + part * (R::kVTok * 128 >> 4), d = tmem + j * kRows;
                if (left >= R::kVTok) {
#pragma unroll
                  for (int k = 0; k < R::kVTok / 16; ++k)
                    umma_lo(d, a + k * 128, b + k * 128, idesc, (t | part | k) != 0, leader);
                } else {
                  for (int k = 0; k < (left + 15) / 16; ++k)
                    umma_lo(d, a + k * 128, b + k * 128, idesc, (t | part | k) != 0, leader);
                }
                commit(&mi.empty_v[rg.s]);
                rg.next();
              }
            }
            if (ok) commit(&mi.pv_done);
          }
        }
      }
      // every MMA has finished before TMEM is freed, on an early exit too (bounded)
      commit(&mi.mma_done);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(smem_u32(&mi.mma_done), 0) && global_timer_ns() - t0 <= kDrainNs) {
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- merge
// Rows of the groups that several blocks share, from the pieces in a fixed order; with malformed offsets, rows of the call as attending to nothing.
constexpr int kMergeThreads = 128, kMergeRows = 2;

// Row `row` of out from its own prefix alone, by the block: scores of 128 tokens at a time, a
// thread each, then four of the 512 dims a thread.  For rows that a NaN or an infinity beside
// their prefix spoiled; lse is right already.
__device__ void redo_row(const Params& p, int64_t row) {
  __shared__ float sw[kMergeThreads];
  const int tid = threadIdx.x, t = static_cast<int>(row / p.H);
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.q_seq_offsets[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const __nv_bfloat16* const kv = p.kv + p.cache_offsets[lo] * kLatDim;
  const __nv_bfloat16* const q = p.q + row * kLatDim;
  const int n = p.positions[t] + 1;
  float m = -INFINITY, l = 0.f;
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < n; s0 += kMergeThreads) {
    float x = -INFINITY;
    if (s0 + tid < n) {
      x = 0.f;
      const __nv_bfloat16* const c = kv + static_cast<int64_t>(s0 + tid) * kLatDim;
      for (int d = 0; d < kLatDim; ++d) x = fmaf(__bfloat162float(q[d]), __bfloat162float(c[d]), x);
      x *= p.scale_log2;
    }
    __syncthreads();
    sw[tid] = x;
    __syncthreads();
    float top = m;
    for (int j = 0; j < kMergeThreads; ++j) top = fmaxf(top, sw[j]);
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - top);
    l *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] *= f;
    m = top;
    const int left = n - s0 < kMergeThreads ? n - s0 : kMergeThreads;
    for (int j = 0; j < left; ++j) {
      const float w = m == -INFINITY ? 0.f : ex2_approx(sw[j] - m);
      l += w;
      const __nv_bfloat16* const c = kv + static_cast<int64_t>(s0 + j) * kLatDim + 4 * tid;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = fmaf(w, __bfloat162float(c[k]), o[k]);
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  reinterpret_cast<uint2*>(p.out + row * kLatV)[tid] = make_uint2(pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv));
}

__global__ void __launch_bounds__(kMergeThreads) latent_merge_kernel(Params p, int blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Ws& w = p.ws;
  const int tid = threadIdx.x;
  const Plan plan = *w.plan;
  if (plan.bad) {
    const int64_t rows = static_cast<int64_t>(p.T) * p.H;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
      reinterpret_cast<uint2*>(p.out + r * kLatV)[tid] = make_uint2(0u, 0u);
      if (tid == 0) p.lse[r] = -INFINITY;
    }
    return;
  }
  for (int k = blockIdx.x; k < plan.spoiled; k += gridDim.x) redo_row(p, w.spoiled[k]);
  // two rows a block, a warp for every fourth piece (a long sequence alone has one from every block),
  // then the warps' sums
  __shared__ float4 so[kMergeThreads / 32][kMergeRows][kLatV / 4];
  __shared__ float2 sml[kMergeThreads / 32][kMergeRows];
  const int warp = tid >> 5, lane = tid & 31;
  for (int item = blockIdx.x; item < plan.merges * (kRows / kMergeRows); item += gridDim.x) {
    const Merge mg = w.merge[item / (kRows / kMergeRows)];
    const int r0 = item % (kRows / kMergeRows) * kMergeRows;
    if (r0 >= mg.nrows) continue;
    // pieces: the tail slot of the first block, then the head slots of the others; with fewer tiles
    // than blocks a share is one tile or empty, and the blocks are found from the tiles
    const bool few = plan.tiles < blocks;
    int64_t x0 = 0, x1 = 0, y;
    if (few) {
      share(plan.tiles, mg.first, blocks, &x0, &y);
      share(plan.tiles, mg.last, blocks, &x1, &y);
    }
    const int pieces = few ? static_cast<int>(x1 - x0) + 1 : mg.last - mg.first + 1;
    float m[kMergeRows], l[kMergeRows];
    float4 o[kMergeRows][4];
#pragma unroll
    for (int r = 0; r < kMergeRows; ++r) {
      m[r] = kUnset, l[r] = 0.f;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[r][d] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 2
    for (int n = warp; n < pieces; n += kMergeThreads / 32) {
      const int k = few ? share_of(plan.tiles, x0 + n, blocks) : mg.first + n;
      const int64_t at = static_cast<int64_t>(2 * k + (k == mg.first)) * kRows + r0;
      float2 v[kMergeRows];
      float4 c[kMergeRows][4];
#pragma unroll
      for (int r = 0; r < kMergeRows; ++r) {
        v[r] = w.ml[at + r];
#pragma unroll
        for (int d = 0; d < 4; ++d) c[r][d] = reinterpret_cast<const float4*>(w.o + (at + r) * kLatV)[lane + 32 * d];
      }
#pragma unroll
      for (int r = 0; r < kMergeRows; ++r) {
        if (v[r].y == 0.f) continue;          // no token of the row in this piece
        const float now = fmaxf(m[r], v[r].x), f0 = ex2_approx(m[r] - now), f1 = ex2_approx(v[r].x - now);
        m[r] = now;
        l[r] = fmaf(l[r], f0, v[r].y * f1);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          o[r][d].x = fmaf(o[r][d].x, f0, c[r][d].x * f1);
          o[r][d].y = fmaf(o[r][d].y, f0, c[r][d].y * f1);
          o[r][d].z = fmaf(o[r][d].z, f0, c[r][d].z * f1);
          o[r][d].w = fmaf(o[r][d].w, f0, c[r][d].w * f1);
        }
      }
    }
    __syncthreads();                          // so is free again
#pragma unroll
    for (int r = 0; r < kMergeRows; ++r) {
#pragma unroll
      for (int d = 0; d < 4; ++d) so[warp][r][lane + 32 * d] = o[r][d];
      if (lane == 0) sml[warp][r] = make_float2(m[r], l[r]);
    }
    __syncthreads();
    for (int r = 0; r < kMergeRows && r0 + r < mg.nrows; ++r) {
      float mm = kUnset, ll = 0.f;
      for (int k = 0; k < kMergeThreads / 32; ++k)
        if (sml[k][r].y != 0.f) mm = fmaxf(mm, sml[k][r].x);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < kMergeThreads / 32; ++k) {
        const float2 v = sml[k][r];
        if (v.y == 0.f) continue;
        const float f = ex2_approx(v.x - mm);
        const float4 c = so[k][r][tid];
        ll = fmaf(v.y, f, ll);
        a.x = fmaf(c.x, f, a.x);
        a.y = fmaf(c.y, f, a.y);
        a.z = fmaf(c.z, f, a.z);
        a.w = fmaf(c.w, f, a.w);
      }
      const float inv = ll != 0.f ? 1.f / ll : 0.f;
      const int64_t row = mg.row0 + r0 + r;
      reinterpret_cast<uint2*>(p.out + row * kLatV)[tid] =
          ll != 0.f ? make_uint2(pack2(a.x * inv, a.y * inv), pack2(a.z * inv, a.w * inv)) : make_uint2(0u, 0u);
      if (tid == 0) p.lse[row] = ll != 0.f ? fmaf(mm, 0.69314718055994531f, logf(ll)) : -INFINITY;
      const bool nan = ll == ll && ll != 0.f && !(a.x == a.x && a.y == a.y && a.z == a.z && a.w == a.w);
      if (p.kv && __syncthreads_or(nan)) redo_row(p, row);
    }
  }
}

}  // namespace

int64_t latent_workspace_bytes(int64_t T, int64_t B, int64_t H, int num_sms) {
  return carve(nullptr, T, B, H, num_sms).bytes;
}

cudaError_t launch_latent_attention(const LatentArgs& a, const CUtensorMap& tmQ, const CUtensorMap& tmC, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int blocks = a.num_sms;
  Params p;
  p.T = a.T;
  p.B = a.B;
  p.H = a.H;
  p.k_sel = a.k_sel;
  p.cache_rows = a.cache_rows;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.kv = a.fp4 ? nullptr : static_cast<const __nv_bfloat16*>(a.kv);
  p.kv4 = a.fp4 ? static_cast<const uint8_t*>(a.kv) : nullptr;
  p.positions = a.positions;
  p.q_seq_offsets = a.q_seq_offsets;
  p.cache_offsets = a.cache_offsets;
  p.idx = a.idx;
  p.scale_log2 = scale_to_log2(a.scale);
  p.scale = score_scale(p.scale_log2);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.ws = carve(a.workspace, a.T, a.B, a.H, blocks);
  p.err = a.err;
  p.timeout_ns = a.timeout_ns;
  auto kern = a.fp4 ? latent_attention_kernel<true> : latent_attention_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // the later two start while their predecessor runs out and wait for its results themselves
  latent_plan_kernel<<<1, kPlanThreads, 0, s>>>(p, blocks);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchAttribute dep;
  dep.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  dep.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(a.fp4 ? Roles<true>::kThreads : Roles<false>::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = &dep;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kern, tmQ, tmC, p)) != cudaSuccess) return e;
  cfg.gridDim = dim3(16 * blocks);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel, p, blocks);
}

}  // namespace dsa
