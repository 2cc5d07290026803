// Shared by the tree-attention sources: parameters, per-sequence bounds, the visibility bits
// of a query, the block-balanced schedule and the split plan.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

constexpr int kTreeMax = 1024;       // drafted tokens per sequence at most
// cached positions per sequence at most: positions and the blocks, pages and splits they are rounded up to
// stay inside 32 bits
constexpr int kTreeContext = 0x7FFFFF00;
constexpr int kTreeGroup = 4;        // CTAs that share a walk at most
constexpr int kTreeRows = 128;       // tensor-core kernel: query rows per tile
constexpr int kTreeBlk = 64;         // ... and cached tokens per block
constexpr int kTreeLead = 14;        // a unit's start and end take as long as this many blocks

struct TreePlan {
  int kernel;          // 0 CUDA cores, 1 tensor cores (tcgen05)
  int g;               // query heads per kv head
  int splits, chunk;   // kernel 0: token splits, tokens each
  int ctas;            // kernel 1: persistent CTAs
  int group;           // ... of which this many walk the same blocks for different row tiles
  int lead;            // ... and what a unit's start and end weigh, in blocks
  size_t ws_bytes, ws_ml_off;
};

struct TreeParams {
  const void* q;             // [Tq][Hq][D] act
  const int32_t* q_start;    // [B+1]
  const uint32_t* mask;      // [Tq][mask_words]
  const int32_t* tables;     // [B][max_blocks]
  const int32_t* lens;       // [B]
  int Tq, B, H, Hq, g, D;
  int max_tree, mask_words, max_blocks, max_context;
  const uint8_t* pages;
  const float* k_static;
  const float* v_static;
  int NB, bs, record, off_v, off_s, row_bytes, mode, cache_dtype, act_fp16;
  float scale_log2;
  void* out;
  int out_dtype;
  int splits, chunk, ctas, group, lead;
  int shares;                // ctas / group
  unsigned share_unit;       // 2^32 / shares, rounded down
  float* ws_o;
  float* ws_ml;
  int32_t* fault;
};

// Sequence b: its query rows start at q0, L drafted tokens, n cached positions (the drafted
// ones last).  L = 0 for a sequence without queries or one that is rejected: a context length
// outside [0, max_context] or the block table, more queries than positions or than max_tree,
// or query rows outside [0, Tq].
struct TreeSeq {
  int q0, L, n;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b, bool report = false) {
  TreeSeq s;
  s.q0 = p.q_start[b];
  const int q1 = p.q_start[b + 1];
  s.L = q1 - s.q0;
  s.n = p.lens[b];
  const bool ok = s.q0 >= 0 && s.L >= 0 && q1 <= p.Tq && s.L <= p.max_tree && s.n >= s.L && s.n <= p.max_context &&
                  s.n <= static_cast<long>(p.max_blocks) * p.bs;
  if (!ok) {
    if (report) record_fault(p.fault, KVQ_FAULT_CONTEXT);
    s.L = 0;
  }
  return s;
}

// Visibility of the 32 positions from `pos` on to the query whose mask row is `row`: bit i is
// position pos + i.  Positions below n - L are the prefix (all visible), position n - L + j is
// drafted token j (bit j of the row), positions from n on are not there.
__device__ __forceinline__ uint32_t visible32(const uint32_t* row, int pos, int n, int L) {
  const int j0 = pos - (n - L);                  // drafted index of the first position
  if (j0 + 32 <= 0) return 0xFFFFFFFFu;
  uint32_t w = 0;
  if (j0 < L) {
    const int words = (L + 31) >> 5;
    if (j0 >= 0) {
      const int k = j0 >> 5, sh = j0 & 31;
      w = row[k] >> sh;
      if (sh != 0 && k + 1 < words) w |= row[k + 1] << (32 - sh);
    } else {
      w = (row[0] << -j0) | ((1u << -j0) - 1u);  // the prefix part below the draft
    }
    const int have = L - j0;                     // positions of the word that exist
    if (have < 32) w &= (1u << have) - 1u;
  }
  return w;
}

// Block-balanced schedule of the tensor-core kernel.  A unit is one (sequence, kv head, row of
// `group` tiles of 128 query rows) and has ceil(n / 64) blocks; the blocks of all units (and `lead`
// before each unit's own, for what a unit costs besides), in the order (sequence, kv head, row of
// tiles), are cut into ctas / group contiguous ranges, one per group of CTAs.  The CTAs of a group walk the same blocks at the same time, each for its own tile
// of the row, so that the cache's bytes come from DRAM once for all of them (trees wider than one
// tile; with tiles as units of their own the tiles of a sequence were read at different times, and
// DRAM was the bound).  A CTA has at most two segments that do not hold a whole unit: one that
// does not begin its unit (partial slot 2 c) and one that begins but does not end it (slot
// 2 c + 1).
__device__ __forceinline__ int tree_tiles(const TreeParams& p, int L) {
  return (L * p.g + kTreeRows - 1) / kTreeRows;
}
__device__ __forceinline__ int tree_tile_rows(const TreeParams& p, int L) {
  return (tree_tiles(p, L) + p.group - 1) / p.group;
}
__device__ __forceinline__ int tree_blocks(int n) { return (n + kTreeBlk - 1) / kTreeBlk; }
// A unit weighs its blocks and `lead` more, for its start and end.
__device__ __forceinline__ unsigned tree_work(const TreeParams& p, const TreeSeq& s) {
  return s.L > 0 ? static_cast<unsigned>(tree_tile_rows(p, s.L) * p.H) * (tree_blocks(s.n) + p.lead) : 0;
}
// Start of share k when the work W is cut into p.shares about equal ones, or into shares of one block
// where there are not as many (none but the last ones is empty): W k / shares, by a product
// with 2^32 / shares (32 bits: the entry point refuses calls that could pass 2^31.  Divisions, and those
// of 64 bits above all, were microseconds of a small call.)
__device__ __forceinline__ unsigned tree_start(const TreeParams& p, unsigned W, int k) {
  const unsigned few = min(static_cast<unsigned>(k), W);
  return W <= static_cast<unsigned>(p.shares) ? few : k >= p.shares ? W : __umulhi(W, k * p.share_unit);
}
// The share that holds position u < W: an estimate, and the steps that it is off.
__device__ __forceinline__ int tree_share(const TreeParams& p, unsigned W, unsigned u) {
  if (W <= static_cast<unsigned>(p.shares)) return static_cast<int>(u);
  int k = min(p.shares - 1, static_cast<int>(__fdividef(static_cast<float>(u) * p.shares, static_cast<float>(W))));
  while (tree_start(p, W, k) > u) --k;
  while (tree_start(p, W, k + 1) <= u) ++k;
  return k;
}

bool tree_tc_supported(const Geometry& g, int group);
cudaError_t launch_tree_simt(const TreeParams& p, int act, cudaStream_t s);
cudaError_t launch_tree_tc(const TreeParams& p, const Geometry& g, cudaStream_t s);

}  // namespace kvq
