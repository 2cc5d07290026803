// Attention of drafted token trees on the 5th-generation tensor cores (tcgen05.mma,
// accumulators in tensor memory): head_dim 128, block size 16, INT8 / FP8 / BF16 / FP16 caches.
//
// A unit is one tile of 128 query rows (row r: drafted token r / g, head r % g) of one
// (sequence, kv head); it walks the sequence's positions in blocks of 64.  One persistent CTA
// per SM takes an equal share of all units' blocks (kvq_tree.cuh), so that a few long
// sequences and many short ones both fill the machine; a unit cut between CTAs leaves partial
// results (unnormalised O, exponent offset, sum) that tree_merge_kernel joins.
//
// Inside a CTA the blocks go to two streams in turn, each with its own running maximum, sum and
// output accumulator, joined once per unit: the chain of one block (S = Q K^T, softmax, O += P V)
// never waits for the softmax of the block before it.  Tensor memory holds three score buffers of 64
// columns (one per stream in use, one ahead; P replaces the scores it came from), Q (64) and the two
// accumulators (128 each): all 512 columns.
//
//   warps 0-3, 4-7  softmax of stream 0 / 1: one query row per thread;
//   warp 8          producer: block-table entries (32 pages at a time, the next 32 sent for into L2),
//                   one bulk copy per page record into a ring of six blocks (16-bit caches: four
//                   warps, each with one of a page's four TMA tensor copies straight into the tiles);
//   warp 9          issues S = Q K^T;  warp 18 issues O += P V;
//   warps 10-13     K converters, 14-17 V converters: codes -> fp16 tiles (exact), two warps per block.
//
// Measured (B200, bf16 results; one call behind an L2 flush / seconds of calls back to back, where the
// 1000 W cap holds the SMs at 1880, 1680 and 1590 MHz of 1965): ragged trees, 32 / 8 heads over 64 x 1024..8192
// FP8 237 / 240 us; trees of 16, 64 / 8 heads over 24 x 16384 INT8 302 / 342 us (2.8 / 2.5 TB/s of cache);
// trees of 64 over 8 x 16384 bf16 400 / 471 us (690 / 583 TFLOP/s; hi + lo P: three products for two).  No rate
// is the bound: DRAM is 31% busy (14% for bf16), the tensor pipe 32% (46%), the issue slots 52% (50%).  It is
// the latency of a block's chain, from its scores to its weights, that 19 warps of 96 registers do not
// cover.  About 6700 warp instructions go into 128 positions (a softmax warp 450 per 64, a converter
// warp 300 per 64).  What follows: scores, weights and sums are packed pairs, blocks that every row sees skip the maximum, two converter
// warps per block rather than four (331 -> 317 us), and the roles' loops are kept small, since together
// they have to fit the instruction cache (5% of the time when they did not).  Starting and ending a
// unit costs 8 us of a CTA, which the shares count.
//
// Query i sees the prefix and the drafted tokens of its mask row.  Blocks that hold prefix
// only, on pages that passed their table check, take a path without per-score tests; in the
// others a 32-bit word per row and 32 positions selects the visible scores (selected, never
// multiplied: a masked score may be NaN).  P is 0 at masked positions, which P V would still
// multiply with V: V rows outside the sequence are zeros in the tile, and a drafted row's
// infinities and NaN are left out of the tile and added in the end to the rows that see
// them.
//
// Rounding: K and V codes are exact in fp16, and q is (bf16 activations: scaled by a power of two per
// row; elements below 2^-26 of the row's largest lose bits).  P is one fp16 (11 bits) when the output is
// bf16 (8 bits) and the tiles are fp16, which leaves the output's own rounding eight times larger than P's
// (a pair there costs 306 -> 357 us in the INT8 case above and 239 -> 269 us in the FP8 one; the error against 64 bits,
// 0.0017 of the output, is that of binary32 probabilities as it is); otherwise P is a hi + lo pair of 16-bit
// halves (two MMAs; 22 bits in fp16, 17 in bf16).  fp16 has a smallest step besides, 2^-24: half of it is the absolute part of P's error (Range,
// below).  Scores, sums and O are binary32.
#include <algorithm>

#include "kvq_decode_common.cuh"
#include "kvq_ptx.cuh"
#include "kvq_tc.cuh"
#include "kvq_tree.cuh"

namespace kvq {
namespace {

constexpr int kD = 128, kBS = 16, kPPB = kTreeBlk / kBS;
constexpr int kThreads = 608;
constexpr int kSoftWarps = 8, kProdWarp = 8, kScoreWarp = 9, kConvWarp0 = 10, kOutWarp = 18;
constexpr int kTile = 16384;         // K or V of a block: 64 x 128 16-bit elements
constexpr int kNS = 3;               // score buffers: one in use per stream, one ahead
// slots of per-block scales and page flags: the K converters write block J's once S of block J - 2
// (16-bit caches: once P V of block J - 6) is complete, which came after P V of block J - 5 (J - 6),
// hence after the softmax of all blocks up to that: the slot of block J - 8 is free
constexpr int kNQ = 8;
// Where a row's P lies.  Re-basing puts its largest at 2^PLACE at most; log2 P above LIMIT, or 32 weights that sum
// (times the block's largest V scale) to more than SUM, ask for it.  fp16 tiles use the whole of
// fp16's range: what is placed high leaves the smallest weights, behind one position that takes nearly all, bits of
// their own (half a step, 2^-25, is 2^-31 of the largest; with the largest at 1 a sink of no value and 4000
// positions 2^18 below it came out further off than 2^-10 of them).  Higher still, what later positions
// exceed the largest by asks for re-basing more often (ragged FP8: 232 us at 2^5, 235 at 2^7, 242 at 2^9).  Per-token
// scales stay lower, since SUM holds for the block's largest V scale and may overstate P.  bf16 tiles have
// the range of binary32.
template <bool BF, bool PT>
struct Range {
  static constexpr float PLACE = BF ? 0.f : PT ? 5.f : 7.f;
  static constexpr float LIMIT = BF ? 8.f : 15.5f;
  static constexpr float SUM = BF ? 8192.f : PT ? 32500.f : 65000.f;    // (65504 is the largest fp16)
};
constexpr float kMostE = 90.f;       // log2 of the weights themselves stays below about this (V scales below 1)
// TMEM columns: scores / P of block J in [64 (J % 3), +64), Q in [192, 256), O of stream s in
// [256 + 128 s, +128)
constexpr uint32_t kTmemCols = 512, kTmQ = 192, kTmO = 256;

template <int CD, bool PT>
struct Layout {
  static constexpr bool DIRECT = CD == KVQ_DTYPE_BF16 || CD == KVQ_DTYPE_FP16;
  static constexpr bool BF = CD == KVQ_DTYPE_BF16;              // tile type
  static constexpr int ROWB = DIRECT ? 2 * kD : kD;
  static constexpr int OFF_V = kBS * ROWB, OFF_S = 2 * kBS * ROWB;
  static constexpr int REC = OFF_S + (PT ? 8 * kBS : 0);
  // K and V tile buffers (a K tile is free once S has read it, a V tile only after P V), and the
  // raw ring of blocks (8-bit caches)
  static constexpr int NBK = DIRECT ? 6 : 2, NBV = DIRECT ? 6 : 4;
  static constexpr int RS = DIRECT ? 0 : 6;
  static constexpr int RSD = RS > 0 ? RS : 1;                   // (a divisor)
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = NBK * kTile;
  static constexpr int RAW_OFF = V_OFF + NBV * kTile;
  static constexpr int KS_OFF = RAW_OFF + RS * kPPB * REC;      // float [kNQ][64] K scales (PT)
  static constexpr int VS_OFF = KS_OFF + (PT ? kNQ * kTreeBlk * 4 : 0);   // float [kNQ][64]: V scales
  static constexpr int VL_OFF = VS_OFF + (PT ? kNQ * kTreeBlk * 4 : 0);   // float [kNQ][64]: log2 of V scales
  static constexpr int KQ_OFF = VL_OFF + (PT ? kNQ * kTreeBlk * 4 : 0);   // float [8][64]: a softmax warp's score factors (PT)
  static constexpr int EX_OFF = KQ_OFF + (PT ? kSoftWarps * kTreeBlk * 4 : 0);   // float [2][2][128], int [4]: a unit's start and end
  static constexpr int WALK_OFF = EX_OFF + 4 * kTreeRows * 4 + 16;        // Walk [warps]
  static constexpr int MISC_OFF = WALK_OFF + (kThreads / 32 + 1) / 2 * 128;
  // vmax [kNQ][4]; nonfinite flags of scales [kNQ][4] and of V rows [NBV][4]; page masks of the raw
  // ring / tile buffers; pok [kNQ]; schedule [6]; tmem, abort;
  // blocks that each producer issued [4]
  static constexpr int NPOK = DIRECT ? NBK : RS;
  static constexpr int WORDS = 8 * kNQ + 4 * NBV + NPOK + kNQ + 6 + 2 + 4;
  static constexpr int BAR_OFF = (MISC_OFF + 4 * WORDS + 7) / 8 * 8;
  static_assert(MISC_OFF % 16 == 0, "vmax is read four at a time");
  static_assert(!DIRECT || NBK == NBV, "16-bit caches fill K and V of a buffer together");
  // raw_full, raw_empty [RS]; tile_full [NBK] (DIRECT); k_full, k_free [NBK]; v_full, v_free
  // [NBV]; s_full, s_free, p_full [kNS]; pv_done [2]; q_ready, o_full, sync, fin [2]
  static constexpr int NBARS = 2 * RS + 3 * NBK + 2 * NBV + 3 * kNS + 2 + 5;
  static constexpr int BYTES = 1024 + BAR_OFF + 8 * NBARS;
  static_assert(BYTES <= 227 * 1024, "fits the shared memory of one CTA");
  static_assert(BYTES > 114 * 1024, "one CTA per SM: its TMEM allocation never waits for a peer");
};

// One segment of the schedule: blocks [j0, j1) of a unit.
struct Seg {
  int b, kvh, tile, q0, L, n, nblk, j0, j1;
};

// A warp's place in the schedule, in shared memory; walk_next is a function of its own, since seven
// copies of it kept the loops of the roles from sharing the instruction cache.
struct Walk {
  Seg g;                                                      // the segment walk_next found
  int b, u, pos;                                              // where the next begins; pos: in the unit, its lead included
  int left;
};

// The next segment with a tile for this CTA (a short row of tiles has none for the last ones); the
// whole warp calls.
__device__ __noinline__ bool walk_next(const TreeParams& p, Walk* walk) {
  __syncwarp();
  Walk w = *walk;
  __syncwarp();
  bool found = false;
  while (w.left > 0 && !found) {
    const TreeSeq s = w.b < p.B ? tree_seq(p, w.b) : TreeSeq{0, 0, 0};
    const int tiles = tree_tiles(p, s.L), rows = tree_tile_rows(p, s.L);
    if (w.b >= p.B) break;
    if (w.u >= p.H * rows) {
      w.u = 0;
      ++w.b;
      continue;
    }
    w.g.kvh = w.u / rows;
    w.g.tile = (w.u - w.g.kvh * rows) * p.group + blockIdx.x % p.group;
    w.g.nblk = tree_blocks(s.n);
    const int take = min(p.lead + w.g.nblk - w.pos, w.left);
    w.g.j0 = max(w.pos - p.lead, 0);
    w.g.j1 = w.pos + take - p.lead;
    w.left -= take;
    w.pos = 0;
    ++w.u;
    found = w.g.j1 > w.g.j0 && w.g.tile < tiles;
    w.g.b = w.b;
    w.g.q0 = s.q0;
    w.g.L = s.L;
    w.g.n = s.n;
  }
  if ((threadIdx.x & 31) == 0) *walk = w;
  __syncwarp();
  return found;
}

struct Shared {
  uint64_t *raw_full, *raw_empty, *tile_full, *k_full, *k_free, *v_full, *v_free, *s_full, *s_free, *p_full, *pv_done,
      *q_ready, *o_full, *sync, *fin;
  int *pages, *pok, *snf, *vnf, *sched, *issued;
  float *vmax, *ks, *vs, *vl;
  uint32_t* tmem;
  volatile int* abort;
};

// Bounded wait that also gives up when another role has; the thread sleeps in the barrier.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = static_cast<uint32_t>(clock());
  while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
    if (*abort) return false;
    if (static_cast<uint32_t>(clock()) - t0 > static_cast<uint32_t>(kWaitCycles)) return false;
  }
  return true;
}

__device__ __forceinline__ void fail(const TreeParams& p, volatile int* abort) {
  record_fault(p.fault, KVQ_FAULT_TIMEOUT);
  *abort = 1;
}

// Swizzled byte offset of 16-byte chunk c (8 elements, c < 16) of row t in a tile of R rows.
template <int R>
__device__ __forceinline__ uint32_t tile_off(int t, int c) {
  return static_cast<uint32_t>((c >> 3) * (R * 128) + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}

// Descriptors of a tile's first k step.  K-major (rows M or N, contiguous along K): 8-row groups
// 1024 bytes apart; a step of 16 elements is 32 bytes on, the fifth in the second column half.
// MN-major (rows K, contiguous along N): column halves R * 128 bytes apart, a step of 16 rows 2048
// bytes on.  (Descriptors count 16 bytes.)
__device__ __forceinline__ uint64_t first_kmajor(uint32_t tile) { return tc::smem_desc(tile, 16u, 1024u); }
template <int R>
__device__ __forceinline__ uint64_t step_kmajor(int kk) { return (kk >> 2) * (R * 8) + (kk & 3) * 2; }
__device__ __forceinline__ uint64_t first_mnmajor(uint32_t tile) { return tc::smem_desc(tile, kTreeBlk * 128u, 1024u); }

// One thread of the warp issues (the operands stay in the warp's uniform registers, which a
// branch on the lane would take them out of).
__device__ __forceinline__ void mma_ts_one(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(0u) : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)) : "memory");
}

// Eight INT8 codes -> fp16, exactly: byte c + 128 under the exponent of 1024, less 1152.
__device__ __forceinline__ uint4 i8x8_to_f16(uint2 w) {
  const uint32_t a = w.x ^ 0x80808080u, b = w.y ^ 0x80808080u;
  uint4 u = make_uint4(__byte_perm(a, 0x64646464u, kLoPair), __byte_perm(a, 0x64646464u, kHiPair),
                       __byte_perm(b, 0x64646464u, kLoPair), __byte_perm(b, 0x64646464u, kHiPair));
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2& h = *reinterpret_cast<__half2*>(&(&u.x)[i]);
    h = __hsub2(h, bias);
  }
  return u;
}

__device__ __forceinline__ uint4 e4m3x8_to_f16(uint2 w) {
  return make_uint4(e4m3x2_to_f16x2(w.x & 0xFFFFu), e4m3x2_to_f16x2(w.x >> 16),
                    e4m3x2_to_f16x2(w.y & 0xFFFFu), e4m3x2_to_f16x2(w.y >> 16));
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float2 w) {
  return BF ? pack_bf16x2(w.x, w.y) : pack_f16x2(w.x, w.y);
}

// hi + lo split of two values into 16-bit pairs.
template <bool BF>
__device__ __forceinline__ void split2(float2 w, uint32_t& hi, uint32_t& lo) {
  hi = pack2<BF>(w);
  float2 h;
  if constexpr (BF) h = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi));
  else h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = pack2<BF>(__fadd2_rn(w, make_float2(-h.x, -h.y)));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// x 2^d for an integer d <= 0, in two steps (x may be as large as 2^d is small).
__device__ __forceinline__ float times_2(float x, float d) {
  const float h = truncf(0.5f * d);
  return x * ex2(h) * ex2(d - h);
}

__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
               : "memory");
}

// Bring a page record into L2 (a hint: it completes on its own and faults nothing).
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void prefetch_line(const void* src) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(src) : "memory");
}

// O or P columns [base, base + 16 n) of the warp's lanes times a power of two per lane: float32 values, or
// 16-bit pairs (f0 f1 may lie below fp16's smallest value where what it leaves of a large P does not).
__device__ __forceinline__ void scale_f32(uint32_t base, int n, float f) {
#pragma unroll 1
  for (int c = 0; c < n; ++c) {
    uint32_t r[16];
    tc::ld16(base + 16 * c, r);
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
    st8(base + 16 * c, r);
    st8(base + 16 * c + 8, r + 8);
  }
}
template <bool BF, bool HILO>
__device__ __forceinline__ void scale_p(uint32_t base, int n, float f0, float f1) {
#pragma unroll 1
  for (int c = 0; c < n; ++c) {
    uint32_t r[16];
    tc::ld16(base + 16 * c, r);
#pragma unroll
    for (int i = 0; i < (HILO ? 16 : 8); ++i) {
      if constexpr (BF) {
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&r[i]), __float2bfloat162_rn(f0 * f1));
        r[i] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __half2 v = __hmul2(__hmul2(*reinterpret_cast<__half2*>(&r[i]), __float2half2_rn(f0)), __float2half2_rn(f1));
        r[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    st8(base + 16 * c, r);
    if constexpr (HILO) st8(base + 16 * c + 8, r + 8);
  }
}

// 16-bit pairs of w whose exponent is all ones (infinity, NaN) set to zero; true if any was.
template <bool BF>
__device__ __forceinline__ bool drop_nonfinite(uint4& u) {
  constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t& w = (&u.x)[i];
    if ((w & e) == e) { w &= 0xFFFF0000u; any = true; }
    if (((w >> 16) & e) == e) { w &= 0xFFFFu; any = true; }
  }
  return any;
}

// Visibility of a row's columns [32 i, 32 i + 32) of block j: its mask bits, without the tokens
// of pages that failed their check (bit pp of pok: page pp of the block is there).
__device__ __forceinline__ uint32_t column_bits(const uint32_t* row, int pok, int j, int i, int n, int L) {
  const uint32_t pages = ((pok >> (2 * i)) & 1 ? 0xFFFFu : 0u) | ((pok >> (2 * i + 1)) & 1 ? 0xFFFF0000u : 0u);
  return visible32(row, j * kTreeBlk + 32 * i, n, L) & pages;
}

template <int CD, bool PT, bool HILO>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap rows) {
  using Y = Layout<CD, PT>;
  constexpr bool BF = Y::BF, DIRECT = Y::DIRECT;
  constexpr int NBK = Y::NBK, NBV = Y::NBV, kAll = (1 << kPPB) - 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Shared sh;
  {
    int* w = reinterpret_cast<int*>(smem + Y::MISC_OFF);
    sh.vmax = reinterpret_cast<float*>(w);                   // [kNQ][4]
    sh.snf = w + 4 * kNQ;                                    // [kNQ][4]
    sh.vnf = sh.snf + 4 * kNQ;                               // [NBV][4]
    sh.pages = sh.vnf + 4 * NBV;
    sh.pok = sh.pages + Y::NPOK;
    sh.sched = sh.pok + kNQ;                                 // [6]
    sh.tmem = reinterpret_cast<uint32_t*>(sh.sched + 6);
    sh.abort = reinterpret_cast<volatile int*>(sh.sched + 7);
    sh.issued = sh.sched + 8;                                // [4]
    sh.ks = reinterpret_cast<float*>(smem + Y::KS_OFF);
    sh.vs = reinterpret_cast<float*>(smem + Y::VS_OFF);
    sh.vl = reinterpret_cast<float*>(smem + Y::VL_OFF);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Y::BAR_OFF);
    auto take = [&](int n) { uint64_t* r = bar; bar += n; return r; };
    sh.raw_full = take(Y::RS);
    sh.raw_empty = take(Y::RS);
    sh.tile_full = take(NBK);
    sh.k_full = take(NBK);
    sh.k_free = take(NBK);
    sh.v_full = take(NBV);
    sh.v_free = take(NBV);
    sh.s_full = take(kNS);
    sh.s_free = take(kNS);
    sh.p_full = take(kNS);
    sh.pv_done = take(2);
    sh.q_ready = take(1);
    sh.o_full = take(1);
    sh.sync = take(1);
    sh.fin = take(2);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < Y::RS; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], 4);
    }
    for (int i = 0; i < NBK; ++i) {
      mbar_init(&sh.tile_full[i], 4);
      mbar_init(&sh.k_full[i], DIRECT ? 1 : 2);
      mbar_init(&sh.k_free[i], 1);
    }
    for (int i = 0; i < NBV; ++i) {
      mbar_init(&sh.v_full[i], DIRECT ? 4 : 2);
      mbar_init(&sh.v_free[i], 1);
    }
    for (int i = 0; i < kNS; ++i) {
      mbar_init(&sh.s_full[i], 2);
      mbar_init(&sh.s_free[i], 1);
      mbar_init(&sh.p_full[i], 4);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&sh.pv_done[i], 1);
    mbar_init(sh.q_ready, kSoftWarps);
    mbar_init(sh.o_full, 1);
    mbar_init(sh.sync, kSoftWarps);
    mbar_init(&sh.fin[0], 1);
    mbar_init(&sh.fin[1], 1);
    for (int i = 0; i < 4 * NBV; ++i) sh.vnf[i] = 0;
    *sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == kOutWarp) tc::tmem_alloc(sh.tmem, kTmemCols);
  griddep_wait();
  griddep_launch_dependents();                                // (after the wait: the merge reads this call's inputs early)
  if (warp == 0) {
    // this CTA's share of the blocks, and the unit it begins in
    unsigned W = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32)
      W += __reduce_add_sync(0xffffffffu, b0 + lane < p.B ? tree_work(p, tree_seq(p, b0 + lane, blockIdx.x == 0)) : 0);
    const unsigned w0 = tree_start(p, W, blockIdx.x / p.group), w1 = tree_start(p, W, blockIdx.x / p.group + 1);
    unsigned before = 0;
    int at_b = 0, at_u = 0, at_pos = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B && w1 > w0; b0 += 32) {
      const bool have = b0 + lane < p.B;
      const TreeSeq s = have ? tree_seq(p, b0 + lane) : TreeSeq{0, 0, 0};
      const unsigned w = have ? tree_work(p, s) : 0;
      unsigned sum = w;                                       // inclusive prefix
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned t = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += t;
      }
      const bool mine = before + sum - w <= w0 && w0 < before + sum;
      const unsigned m = __ballot_sync(0xffffffffu, mine);
      if (m) {
        const unsigned in = w0 - (before + sum - w), unit = tree_blocks(s.n) + p.lead;
        at_b = b0 + __ffs(m) - 1;
        at_u = __shfl_sync(0xffffffffu, in / max(unit, 1u), __ffs(m) - 1);
        at_pos = __shfl_sync(0xffffffffu, in % max(unit, 1u), __ffs(m) - 1);
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      sh.sched[0] = at_b;
      sh.sched[1] = at_u;
      sh.sched[2] = at_pos;
      sh.sched[3] = static_cast<int>(w1 - w0);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *sh.tmem;
  Walk* walk = reinterpret_cast<Walk*>(smem + Y::WALK_OFF) + warp;
  if (lane == 0) {
    walk->b = sh.sched[0];
    walk->u = sh.sched[1];
    walk->pos = sh.sched[2];
    walk->left = sh.sched[3];
  }
  Seg sg;
  auto next_segment = [&]() {
    const bool more = walk_next(p, walk);
    sg = walk->g;
    return more;
  };
  int J = 0;                                                  // blocks of the CTA so far

  if (warp == kProdWarp || (DIRECT && warp >= kConvWarp0 && warp < kConvWarp0 + 3)) {
    // ------------------------------------------------------------ producer
    // 16-bit caches: four warps, each with one of a page's four copies (K and V, two column halves:
    // a tensor copy takes about a hundred cycles to issue, and one warp issuing all sixteen of a
    // block was the bound), each announcing its own bytes; the first also sends for what comes next
    const int part = warp == kProdWarp ? 0 : warp - kConvWarp0 + 1;
    constexpr int kParts = DIRECT ? 4 : 1;
    bool run = true;
    int buf = 0, round = 0;                                   // of the raw ring / the tiles
    constexpr int RING = DIRECT ? NBK : Y::RSD;
    while (run && next_segment()) {
      const int npg = (sg.n + kBS - 1) / kBS;
      // table entries 32 pages (8 blocks) at a time, one per lane, the next 32 loaded while these
      // are used and their pages sent for into L2 (a block's own entries, read when it is due,
      // would put a load's latency between every two blocks)
      const int32_t* table = p.tables + static_cast<long>(sg.b) * p.max_blocks;
      const int base = sg.j0 * kPPB, stop = min(sg.j1 * kPPB, npg);
      int cur = -1, next = base + lane < stop ? table[base + lane] : -1;
      if (part == 0) {
        // the unit's q and mask rows, which softmax needs some blocks from now
        const int x0 = sg.tile * kTreeRows, x1 = min(x0 + kTreeRows, sg.L * p.g) - 1;
        for (int t = x0 / p.g + lane; t <= x1 / p.g; t += 32) {
          const long row = static_cast<long>(sg.q0) + t;
          prefetch_l2(static_cast<const uint16_t*>(p.q) + (row * p.Hq + static_cast<long>(sg.kvh) * p.g) * kD, p.g * kD * 2);
          prefetch_line(p.mask + row * p.mask_words);
        }
      }
      for (int j = sg.j0; j < sg.j1 && run; ++j, ++J) {
        const int at = (j - sg.j0) & 7;                       // block of the batch
        if (at == 0) {
          cur = next;
          const int k = j * kPPB + 32 + lane;
          next = k < stop ? table[k] : -1;
        } else if (at == 2 && part == 0 && next >= 0 && next < p.NB) {
          prefetch_l2(p.pages + (static_cast<long>(next) * p.H + sg.kvh) * Y::REC, Y::REC);
        }
        const int blk = __shfl_sync(0xffffffffu, cur, at * kPPB + (lane & (kPPB - 1)));
        const bool mine = lane < kPPB && j * kPPB + lane < stop;
        const bool valid = mine && blk >= 0 && blk < p.NB;
        if (mine && !valid && part == 0) record_fault(p.fault, KVQ_FAULT_BLOCK);
        const unsigned vm = __ballot_sync(0xffffffffu, valid);
        bool ok = true;
        if (lane == 0 && round > 0) {
          if constexpr (DIRECT)
            ok = wait(&sh.k_free[buf], (round - 1) & 1, sh.abort) && wait(&sh.v_free[buf], (round - 1) & 1, sh.abort);
          else
            ok = wait(&sh.raw_empty[buf], (round - 1) & 1, sh.abort);
        }
        run = __all_sync(0xffffffffu, ok);
        if (!run) break;
        uint64_t* full = DIRECT ? &sh.tile_full[buf] : &sh.raw_full[buf];
        if (lane == 0) {
          if (part == 0) sh.pages[buf] = static_cast<int>(vm);
          mbar_arrive_expect_tx(full, __popc(vm) * (Y::REC / kParts));
        }
        __syncwarp();
        if (valid) {
          if constexpr (DIRECT) {
            // 16 rows of K (parts 0, 1) or V (2, 3), one 128-byte half of their 256 bytes
            static_assert(Y::REC == 4 * kBS * 128, "a part's bytes");
            const int y = (blk * p.H + sg.kvh) * (2 * kBS) + (part >> 1) * kBS, hh = part & 1;
            tma_load_2d(smem + (part >> 1 ? Y::V_OFF : Y::K_OFF) + buf * kTile + hh * (kTile / 2) + lane * kBS * 128, &rows, full,
                        128 * hh, y);
          } else {
            bulk_load(smem + Y::RAW_OFF + (buf * kPPB + lane) * Y::REC,
                      p.pages + (static_cast<long>(blk) * p.H + sg.kvh) * Y::REC, Y::REC, full);
          }
        }
        if (++buf == RING) { buf = 0; ++round; }
      }
    }
    if (!run && lane == 0) fail(p, sh.abort);
    // every copy issued must land before the CTA may exit.  After a wait that ran out the parts may have
    // stopped at different blocks (by less than the ring, which turns only when all four have filled a
    // buffer): once all have stopped, the first arrives for those that did not come to a block, whose phase
    // then ends when the others' bytes are there.
    if constexpr (DIRECT) {
      if (lane == 0) sh.issued[part] = J;
      __syncwarp();
      asm volatile("bar.sync 1, 128;" ::: "memory");          // (the four parts: no wait above is without a bound)
    } else {
      if (lane == 0) sh.issued[0] = J;
    }
    if (lane == 0 && part == 0) {
      int most = 0;
      for (int k = 0; k < kParts; ++k) most = max(most, sh.issued[k]);
      for (int i = max(0, most - RING); i < most; ++i) {
        uint64_t* full = DIRECT ? &sh.tile_full[i % RING] : &sh.raw_full[i % RING];
        for (int k = 0; k < kParts; ++k)
          if (sh.issued[k] <= i) mbar_arrive(full);
        if (!mbar_drain(full, (i / RING) & 1)) record_fault(p.fault, KVQ_FAULT_TIMEOUT);
      }
    }
  } else if (warp >= kConvWarp0 && warp < kOutWarp) {
    // ------------------------------------------------------------ converters
    // 8-bit caches: two warps per block and tensor (four for every block spent more on what each block
    // costs a warp than on its codes): thread (c, rr) has 16-byte chunk c of rows rr + 4 k of every page;
    // K: thread ct also carries token ct's scales.  16-bit caches, V: token ct's zeros, and K's fourth
    // warp alone hands on the page flags
    const bool isv = warp >= kConvWarp0 + 4;
    const int cw = (warp - kConvWarp0) & 3, ct = (DIRECT ? cw : cw & 1) * 32 + lane;
    const int c = ct & 15, rr = ct >> 4;
    constexpr int kStep = DIRECT ? 1 : 2;
    bool run = true;
    int at = DIRECT ? 0 : cw >> 1;                            // this warp's next block of the CTA
    int raw = at, rpar = 0, kb = 0, kpar = 0;
    while (run && next_segment()) {
      const int first = sg.n - sg.L;                          // first drafted position
      const int end = J + sg.j1 - sg.j0;
      for (; at < end; at += kStep) {
        const int j = sg.j0 + at - J;
        if constexpr (!DIRECT) {
          kb = at & ((isv ? NBV : NBK) - 1);
          kpar = isv ? at / NBV : at / NBK;
        }
        const int slot = at & (kNQ - 1);
        bool ok = true;
        if constexpr (DIRECT) {
          ok = wait(&sh.tile_full[kb], kpar & 1, sh.abort);
        } else {
          ok = wait(&sh.raw_full[raw], rpar, sh.abort);
          if (ok && kpar > 0) ok = wait(isv ? &sh.v_free[kb] : &sh.k_free[kb], (kpar - 1) & 1, sh.abort);
        }
        run = __all_sync(0xffffffffu, ok);
        if (!run) break;
        const int pok = sh.pages[DIRECT ? kb : raw];
        const bool tail = j * kTreeBlk + kTreeBlk > first;    // holds drafted positions, or the end
        const bool whole = !tail && pok == kAll;
        bool nf = false;
        if constexpr (DIRECT) {
          if (isv && !whole && ct < kTreeBlk) {
            const int pos = j * kTreeBlk + ct;
            const bool keep = pos < sg.n && ((pok >> (ct / kBS)) & 1);
            uint8_t* tile = smem + Y::V_OFF + kb * kTile;
            if (!keep || pos >= first) {
#pragma unroll 1
              for (int cc = 0; cc < 16; ++cc) {
                uint4* a = reinterpret_cast<uint4*>(tile + tile_off<kTreeBlk>(ct, cc));
                uint4 u = keep ? *a : make_uint4(0, 0, 0, 0);
                const bool drop = drop_nonfinite<BF>(u);
                if (!keep || drop) *a = u;
                nf = nf || drop;
              }
            }
          }
        } else {
          uint8_t* tile = smem + (isv ? Y::V_OFF : Y::K_OFF) + kb * kTile;
          uint8_t* even = tile + tile_off<kTreeBlk>(rr, c);        // rows rr + 8 i, and
          uint8_t* odd = tile + tile_off<kTreeBlk>(rr + 4, c);     // rr + 4 + 8 i
          const uint8_t* src = smem + Y::RAW_OFF + raw * (kPPB * Y::REC);
          const uint8_t* row = src + (isv ? Y::OFF_V : 0) + rr * Y::ROWB + 8 * c;
          uint2 w[kPPB][4];
#pragma unroll
          for (int pp = 0; pp < kPPB; ++pp)
#pragma unroll
            for (int k = 0; k < 4; ++k) w[pp][k] = *reinterpret_cast<const uint2*>(row + pp * Y::REC + 4 * k * Y::ROWB);
          float kscale = 0.f, vscale = 0.f;
          if constexpr (PT) {
            if (!isv) {
              const float* sc = reinterpret_cast<const float*>(src + (ct >> 4) * Y::REC + Y::OFF_S) + (ct & 15);
              kscale = sc[0];
              vscale = sc[kBS];
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.raw_empty[raw]);
          raw += 2;
          if (raw >= Y::RS) { raw -= Y::RS; rpar ^= 1; }
          auto code16 = [&](const uint2& x) { return CD == KVQ_DTYPE_INT8 ? i8x8_to_f16(x) : e4m3x8_to_f16(x); };
#pragma unroll
          for (int pp = 0; pp < kPPB; ++pp)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>((k & 1 ? odd : even) + (pp * kBS + 8 * (k >> 1)) * 128) = code16(w[pp][k]);
          if (!whole) {
            // rows that are not there to zeros, and drafted V without its infinities and NaN
#pragma unroll 1
            for (int i = 0; i < 4 * kPPB; ++i) {
              const int t = 4 * i + rr, pos = j * kTreeBlk + t;
              uint4* a = reinterpret_cast<uint4*>(tile + tile_off<kTreeBlk>(t, c));
              if (!(((pok >> (i >> 2)) & 1) && pos < sg.n)) {
                *a = make_uint4(0, 0, 0, 0);
              } else if (CD == KVQ_DTYPE_FP8_E4M3 && isv && pos >= first) {
                uint4 u = *a;
                if (drop_nonfinite<false>(u)) {
                  *a = u;
                  nf = true;
                }
              }
            }
          }
          if constexpr (PT) {
            if (!isv) {
              bool sf = false;
              if (!whole) {
                const int pos = j * kTreeBlk + ct;
                if (!(pos < sg.n && ((pok >> (ct / kBS)) & 1))) kscale = vscale = 0.f;
                if (pos >= first && !(fabsf(vscale) <= 3.4e38f)) {   // an unusable drafted row
                  vscale = 0.f;
                  sf = true;
                }
              }
              const float va = fabsf(vscale);
              sh.ks[slot * kTreeBlk + ct] = kscale;
              sh.vs[slot * kTreeBlk + ct] = vscale;
              sh.vl[slot * kTreeBlk + ct] = __log2f(va);
              // bit patterns order as magnitudes do (a NaN of the prefix lies above all of them)
              const unsigned m = __reduce_max_sync(0xffffffffu, va <= 3.4e38f ? __float_as_uint(va) : 0u);
              sf = __any_sync(0xffffffffu, sf);
              if (lane == 0) {
                sh.vmax[slot * 4 + (cw & 1)] = __uint_as_float(m);
                sh.snf[slot * 4 + (cw & 1)] = sf;
              }
            }
          }
        }
        if (isv && tail) {
          nf = __any_sync(0xffffffffu, nf);
          if (lane == 0) sh.vnf[kb * 4 + (ct >> 5)] = nf;
        }
        if (!isv && (DIRECT ? lane == 0 : ct == 0)) sh.pok[slot] = pok;
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(isv ? &sh.v_full[kb] : &sh.k_full[kb]);
        }
        if constexpr (DIRECT) {
          if (++kb == NBK) { kb = 0; ++kpar; }
        }
      }
      J = end;
    }
    if (!run && lane == 0) fail(p, sh.abort);
  } else if (warp == kScoreWarp) {
    // ------------------------------------------------------------ S = Q K^T
    // (the whole warp runs the loop, so that descriptors stay in uniform registers)
    const uint32_t tiles = smem_u32(smem);
    constexpr uint32_t idS = tc::idesc_f16(BF, false, kTreeRows, kTreeBlk);
    const uint64_t dk = first_kmajor(tiles + Y::K_OFF);
    bool ok = true;
    int unit = 0, kb = 0, kround = 0, sb = 0, sround = 0;
    while (ok && next_segment()) {
      ok = __all_sync(0xffffffffu, wait(sh.q_ready, unit & 1, sh.abort));
      for (int j = sg.j0; j < sg.j1 && ok; ++j, ++J) {
        // the score buffer: P V of block J - 3 has read it
        bool fine = sround == 0 || wait(&sh.s_free[sb], (sround - 1) & 1, sh.abort);
        if (fine) fine = wait(&sh.k_full[kb], kround & 1, sh.abort);
        if (DIRECT && fine) fine = wait(&sh.tile_full[kb], kround & 1, sh.abort);
        ok = __all_sync(0xffffffffu, fine);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_one(tbase + kTreeBlk * sb, tbase + kTmQ + 8 * kk, dk + kb * (kTile / 16) + step_kmajor<kTreeBlk>(kk), idS, kk > 0);
        commit_one(&sh.k_free[kb]);
        commit_one(&sh.s_full[sb]);
        // (and this warp's own arrival: it hands on what it acquired from the K converters, the
        // block's scales and page flags)
        if (lane == 0) mbar_arrive(&sh.s_full[sb]);
        if (++kb == NBK) { kb = 0; ++kround; }
        if (++sb == kNS) { sb = 0; ++sround; }
      }
      ++unit;
    }
    if (!ok && lane == 0) fail(p, sh.abort);
    // one more commit covers every MMA issued above: TMEM is freed only after it arrives
    commit_one(&sh.fin[0]);
    if (!mbar_drain(&sh.fin[0], 0) && lane == 0) record_fault(p.fault, KVQ_FAULT_TIMEOUT);
    __syncwarp();
  } else if (warp == kOutWarp) {
    // ------------------------------------------------------------ O += P V
    constexpr uint32_t idPV = tc::idesc_f16(BF, true, kTreeRows, kD);
    const uint64_t dv = first_mnmajor(smem_u32(smem) + Y::V_OFF);
    bool ok = true;
    int vb = 0, vround = 0, sb = 0, sround = 0;
    while (ok && next_segment()) {
      for (int j = sg.j0; j < sg.j1 && ok; ++j, ++J) {
        const int st = J & 1;
        bool fine = wait(&sh.v_full[vb], vround & 1, sh.abort);
        if (fine) fine = wait(&sh.p_full[sb], sround & 1, sh.abort);
        ok = __all_sync(0xffffffffu, fine);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int pa = 0; pa < (HILO ? 2 : 1); ++pa)
#pragma unroll
          for (int kk = 0; kk < kTreeBlk / 16; ++kk)
            mma_ts_one(tbase + kTmO + 128 * st, tbase + kTreeBlk * sb + 16 * kk + 8 * pa, dv + vb * (kTile / 16) + kk * 128,
                       idPV, j > sg.j0 + 1 || pa > 0 || kk > 0);
        commit_one(&sh.v_free[vb]);
        commit_one(&sh.s_free[sb]);
        commit_one(&sh.pv_done[st]);
        if (j == sg.j1 - 1) commit_one(sh.o_full);
        if (++vb == NBV) { vb = 0; ++vround; }
        if (++sb == kNS) { sb = 0; ++sround; }
      }
    }
    if (!ok && lane == 0) fail(p, sh.abort);
    commit_one(&sh.fin[1]);
    if (!mbar_drain(&sh.fin[1], 0) && lane == 0) record_fault(p.fault, KVQ_FAULT_TIMEOUT);
    __syncwarp();
  } else if (warp < kSoftWarps) {
    // ------------------------------------------------------------ softmax
    const int st = warp >> 2, quarter = warp & 3;
    const int r = 32 * quarter + lane;                        // row of the tile (TMEM lane)
    const uint32_t lanes = tbase + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t obase = lanes + kTmO + 128 * st;
    float* ex = reinterpret_cast<float*>(smem + Y::EX_OFF);   // [2][2][128] at a unit's end, [2][128] at its start
    int* exf = reinterpret_cast<int*>(ex + 512);              // [2] nonfinite drafted rows seen
    int unit = 0, syncs = 0, seen = 0;                        // seen: blocks of this stream
    bool ok = true;
    auto sync8 = [&]() -> bool {                              // the eight softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.sync);
      const bool fine = wait(sh.sync, syncs & 1, sh.abort);
      ++syncs;
      return __all_sync(0xffffffffu, fine);
    };
    while (ok && next_segment()) {
      // this thread's row, worked out where it is needed from the segment in shared memory (what stays in
      // registers across the blocks is spilled there)
      struct Row {
        bool ok;                                              // it exists
        long q;                                               // row of q and out
        const uint32_t* mask;
      };
      auto row = [&]() {
        const Seg& g = walk->g;
        const int x = g.tile * kTreeRows + r;
        Row w;
        w.ok = x < g.L * p.g;
        const int tok = w.ok ? x / p.g : 0;
        const long at = static_cast<long>(g.q0) + tok;
        w.q = at * p.Hq + static_cast<long>(g.kvh) * p.g + (x - tok * p.g);
        w.mask = p.mask + at * p.mask_words;
        return w;
      };
      const bool warp_ok = 32 * quarter < sg.L * p.g - sg.tile * kTreeRows;
      // --- this row's q, channels [64 st, 64 st + 64), to tensor memory
      float qsc = p.scale_log2;
      int notes = 0;                                        // (uniform) bit 0: drafted rows with infinities or NaN; 1: rows of unlike qsc
      {
        if (p.mode == KVQ_SCALE_PER_HEAD) qsc *= p.k_static[sg.kvh];
        if (p.mode == KVQ_SCALE_PER_TENSOR) qsc *= p.k_static[0];
        uint4 u[8];
        const Row mine = row();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          u[i] = mine.ok ? reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + mine.q * kD + 64 * st)[i]
                        : make_uint4(0, 0, 0, 0);
        if constexpr (!BF) {
          if (!p.act_fp16) {
            // bf16 activations in fp16 tiles: a power of two brings each row's largest |q| to 2^13 .. 2^14, so
            // that elements down to 2^-27 of it keep all their bits (bf16 has fewer than fp16).  A row takes
            // the one of the warp's largest row where that loses nothing (its own largest is then 2 or
            // more: 2^-15 of it whole, the rest within 2^-26 of it), its own where the rows differ by more.
            __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(reinterpret_cast<const __nv_bfloat162*>(&u[i])[e]));
            ex[st * kTreeRows + r] = fmaxf(__low2float(top), __high2float(top));   // (64 of 128 channels)
            ok = sync8();
            if (!ok) break;
            const float amax = fmaxf(ex[r], ex[kTreeRows + r]);
            const bool usable = amax > 0.f && amax <= 3.4e38f;
            int eq = usable ? max(exponent_of(amax) - 13, -100) : -100;
            const int most = __reduce_max_sync(0xffffffffu, eq);
            if (!usable || eq >= most - 12) eq = most;        // (a row with an infinity sets no other row's)
            const float down = pow2i(-eq);
            qsc *= pow2i(eq);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float v[8];
              unpack8<__nv_bfloat16>(u[i], v);
              u[i] = make_uint4(pack_f16x2(v[0] * down, v[1] * down), pack_f16x2(v[2] * down, v[3] * down),
                                pack_f16x2(v[4] * down, v[5] * down), pack_f16x2(v[6] * down, v[7] * down));
            }
          }
        }
        const uint32_t flip = qsc < 0.f ? 0x80008000u : 0u;   // a negative static scale: in q's sign
        qsc = fabsf(qsc);
        if (PT && !__all_sync(0xffffffffu, qsc == __shfl_sync(0xffffffffu, qsc, 0))) notes = 2;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint32_t w[8] = {u[i].x ^ flip, u[i].y ^ flip, u[i].z ^ flip, u[i].w ^ flip,
                                 u[i + 1].x ^ flip, u[i + 1].y ^ flip, u[i + 1].z ^ flip, u[i + 1].w ^ flip};
          st8(lanes + kTmQ + 32 * st + 4 * i, w);
        }
        tc::st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.q_ready);
      }
      const int first = sg.n - sg.L;
      // P holds e = 2^(x - m) times the token's V scale, l sums e, O accumulates P V.  m is an integer near
      // the running maximum of x + log2 V scale over what this row sees, less PLACE, raised when P outgrows
      // its range, so that every factor between two of its values is a power of two and re-basing is exact.  The
      // V scale belongs to the maximum, and only the row's own tokens do: a large scale would otherwise
      // leave the other tokens' P no bits in fp16, for rows that do not see it or give it no weight.
      float m = -INFINITY, moff = 0.f, l = 0.f;               // moff: m, or 0 before the first score
      bool begun = false;
      for (int jj = J + ((J ^ st) & 1); jj < J + sg.j1 - sg.j0; jj += 2) {
        const int j = sg.j0 + jj - J;
        const int sb = jj % kNS, slot = jj % kNQ;
        const uint32_t sbase = lanes + kTreeBlk * sb;
        ok = __all_sync(0xffffffffu, wait(&sh.s_full[sb], (jj / kNS) & 1, sh.abort));
        if (!ok) break;
        tc::fence_after_sync();
        const int pok = sh.pok[slot];
        // (uniform) every row sees the whole block, and the rows share score factors
        const bool fast = j * kTreeBlk + kTreeBlk <= first && pok == kAll && notes < 2;
        if (!fast && j * kTreeBlk + kTreeBlk > first) {
          // drafted rows that hold infinities or NaN (the V converters' flags come with the tile)
          const int kb = jj % NBV;
          ok = __all_sync(0xffffffffu, wait(&sh.v_full[kb], (jj / NBV) & 1, sh.abort));
          notes |= sh.vnf[kb * 4] | sh.vnf[kb * 4 + 1] | sh.vnf[kb * 4 + 2] | sh.vnf[kb * 4 + 3];
          if (PT) notes |= sh.snf[slot * 4] | sh.snf[slot * 4 + 1];
        }
        // this stream's block before: its P V must be complete before O is touched (rare)
        auto settle = [&]() {
          if (seen > 0 && !wait(&sh.pv_done[st], (seen - 1) & 1, sh.abort)) ok = false;
          tc::fence_after_sync();
        };
        if (warp_ok) {
          float* kq = reinterpret_cast<float*>(smem + Y::KQ_OFF) + warp * kTreeBlk;
          if (PT && fast) {
            // each token's score factor, once for the warp's 32 rows: K scale times theirs
            const float2 f = reinterpret_cast<const float2*>(sh.ks + slot * kTreeBlk)[lane];
            __syncwarp();                                     // (the block before has been read)
            reinterpret_cast<float2*>(kq)[lane] = make_float2(f.x * qsc, f.y * qsc);
            __syncwarp();
          }
          auto factor = [&](int c) {
            return PT ? *reinterpret_cast<const float4*>(kq + c) : make_float4(qsc, qsc, qsc, qsc);
          };
          const float* vsp = sh.vs + slot * kTreeBlk;
          const float* vlp = sh.vl + slot * kTreeBlk;
          using Rg = Range<BF, PT>;
          float most = Rg::SUM;
          if constexpr (PT) {
            const float2 v2 = *reinterpret_cast<const float2*>(sh.vmax + slot * 4);
            most = Rg::SUM * pow2i(min(-exponent_of(fmaxf(v2.x, v2.y)), static_cast<int>(kMostE) - 15));
          }
          float2 lsum = make_float2(0.f, 0.f);
          // the m that the row's largest P so far (log2 top) and largest weight (log2 mx) ask for
          auto wanted = [&](float top, float mx) {
            return PT ? fmaxf(ceilf(top) - Rg::PLACE, ceilf(mx) - kMostE) : ceilf(top) - Rg::PLACE;
          };
          // m raised to mn for the lanes that ask: l and O (and P of the block's columns before column c0)
          // into the new domain (in two steps: l may be large where V scales are small)
          auto rebase = [&](bool ask, float mn, int c0) {
            float f0 = 1.f, f1 = 1.f;
            if (ask) {
              const int d = m == -INFINITY ? -1000 : static_cast<int>(fmaxf(m - mn, -1000.f));
              f0 = pow2i(d / 2);
              f1 = pow2i(d - d / 2);
              m = moff = mn;
            }
            l = l * f0 * f1;
            lsum = make_float2(lsum.x * f0 * f1, lsum.y * f0 * f1);
            tc::st_wait();
            if (begun) {
              settle();
              scale_f32(obase, 8, f0 * f1);
            }
            scale_p<BF, HILO>(sbase, c0 / 16, f0, f1);
          };
          // --- 32 columns at a time: scores times the K scale, e, its sum, and P over the scores
          // they came from
          auto block = [&](auto masked) {
            constexpr bool MASKED = decltype(masked)::value;
            const uint32_t* mrow = MASKED ? row().mask : nullptr;
#pragma unroll 1
            for (int cc = 0; cc < kTreeBlk / 32; ++cc) {
              uint32_t s[32];
              float2 t[16];
              // the scores of the 32 columns in the exponent's units (by the row's own factor)
              auto load = [&]() {
                tc::ld32(sbase + 32 * cc, s);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  float4 f = make_float4(qsc, qsc, qsc, qsc);
                  if constexpr (PT) {
                    f = *reinterpret_cast<const float4*>(sh.ks + slot * kTreeBlk + 32 * cc + 2 * i);
                    f = make_float4(f.x * qsc, f.y * qsc, f.z * qsc, f.w * qsc);
                  }
                  t[i] = __fmul2_rn(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), make_float2(f.x, f.y));
                  t[i + 1] = __fmul2_rn(make_float2(__uint_as_float(s[2 * i + 2]), __uint_as_float(s[2 * i + 3])), make_float2(f.z, f.w));
                }
              };
              auto largest = [&]() {
                float m0 = fmaxf(t[0].x, t[0].y), m1 = fmaxf(t[1].x, t[1].y);
#pragma unroll
                for (int i = 2; i < 16; i += 2) {
                  m0 = max3(m0, t[i].x, t[i].y);
                  m1 = max3(m1, t[i + 1].x, t[i + 1].y);
                }
                return fmaxf(m0, m1);
              };
              auto largest_p = [&]() {                        // log2 of the largest P (before 2^-m)
                float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  const float4 v = *reinterpret_cast<const float4*>(vlp + 32 * cc + 2 * i);
                  m0 = max3(m0, t[i].x + v.x, t[i].y + v.y);
                  m1 = max3(m1, t[i + 1].x + v.z, t[i + 1].y + v.w);
                }
                return fmaxf(m0, m1);
              };
              if constexpr (!MASKED) {
                tc::ld32(sbase + 32 * cc, s);
              } else {
                load();
                const uint32_t vis = column_bits(mrow, pok, j, cc, sg.n, sg.L);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  if (!((vis >> (2 * i)) & 1u)) t[i].x = -INFINITY;
                  if (!((vis >> (2 * i + 1)) & 1u)) t[i].y = -INFINITY;
                }
                const float mx = largest(), top = PT ? largest_p() : mx;
                const bool ask = top > m + Rg::LIMIT || (PT && mx > m + (kMostE + 8.f));
                if (__any_sync(0xffffffffu, ask)) rebase(ask, wanted(top, mx), 32 * cc);
              }
              uint32_t ph[16], pl[HILO ? 16 : 1];
              // from the scores in t, or (blocks that every row sees) straight from S
              auto weights = [&](auto scaled) {
                const float2 noff = make_float2(-moff, -moff);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  float2 a, b;
                  if constexpr (decltype(scaled)::value) {
                    a = __fadd2_rn(t[i], noff);
                    b = __fadd2_rn(t[i + 1], noff);
                  } else {
                    const float4 f = factor(32 * cc + 2 * i);
                    a = __ffma2_rn(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), make_float2(f.x, f.y), noff);
                    b = __ffma2_rn(make_float2(__uint_as_float(s[2 * i + 2]), __uint_as_float(s[2 * i + 3])), make_float2(f.z, f.w), noff);
                  }
                  a = make_float2(ex2(a.x), ex2(a.y));
                  b = make_float2(ex2(b.x), ex2(b.y));
                  sum = __fadd2_rn(sum, __fadd2_rn(a, b));
                  if constexpr (PT) {
                    const float4 f = *reinterpret_cast<const float4*>(vsp + 32 * cc + 2 * i);
                    a = __fmul2_rn(a, make_float2(f.x, f.y));
                    b = __fmul2_rn(b, make_float2(f.z, f.w));
                  }
                  if constexpr (HILO) {
                    split2<BF>(a, ph[i], pl[i]);
                    split2<BF>(b, ph[i + 1], pl[i + 1]);
                  } else {
                    ph[i] = pack2<BF>(a);
                    ph[i + 1] = pack2<BF>(b);
                  }
                }
                return sum;
              };
              float2 sum = weights(masked);
              if constexpr (!MASKED) {
                // every column is visible: the maximum need not be known as long as the 32 weights, times
                // the block's largest V scale, sum to no more than SUM: P then stays inside fp16.  It is
                // found, from the scores again, for a row's first columns and when that fails.
                const bool ask = sum.x + sum.y > most || m == -INFINITY;
                if (__any_sync(0xffffffffu, ask)) {
                  load();
                  const float mx = largest(), mn = wanted(PT ? largest_p() : mx, mx);
                  // (every row that has grown, not only those that ask: fewer times in all, 242 against 255 us
                  // in the ragged FP8 case above)
                  const bool raise = mn > m;
                  if (__any_sync(0xffffffffu, raise)) rebase(raise, mn, 32 * cc);
                  // (from t, whose largest m was made of: S times the factor less m, rounded once, leaves
                  // ulp(x) / 2 there, which is more than fits an exponent once scores reach 2^31)
                  sum = weights(std::true_type{});
                }
              }
              lsum = __fadd2_rn(lsum, sum);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                st8(sbase + 32 * cc + 16 * h, ph + 8 * h);
                if constexpr (HILO) st8(sbase + 32 * cc + 16 * h + 8, pl + 8 * h);
              }
              (void)pl;
            }
          };
          if (fast) block(std::false_type{});
          else block(std::true_type{});
          l += lsum.x + lsum.y;
          tc::st_wait();
        }
        begun = true;
        ++seen;
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[sb]);
        if (!ok) break;
      }
      J += sg.j1 - sg.j0;
      if (!ok) break;
      // --- the unit's end: both streams' (offset, sum) through shared memory, then stream st joins
      // the two accumulators for output channels [64 st, 64 st + 64)
      ok = __all_sync(0xffffffffu, wait(sh.o_full, unit & 1, sh.abort));
      ++unit;
      if (!ok) break;
      tc::fence_after_sync();
      ex[(2 * st) * 128 + r] = moff;
      ex[(2 * st + 1) * 128 + r] = l;
      if (threadIdx.x < 2) exf[threadIdx.x] = 0;
      ok = sync8();
      if (!ok) break;
      if ((notes & 1) && lane == 0) atomicOr(&exf[0], 1);
      const float o0 = ex[r], l0 = ex[128 + r], o1 = ex[256 + r], l1 = ex[384 + r];
      ok = sync8();
      if (!ok) break;
      const bool nonfinite = exf[0] != 0;
      // a stream whose sum is 0 saw nothing (or had no block: its accumulator is unwritten)
      const bool has0 = l0 != 0.f, has1 = l1 != 0.f;
      const float off = has0 && has1 ? fmaxf(o0, o1) : has0 ? o0 : has1 ? o1 : -INFINITY;
      const float w0 = has0 ? ex2(o0 - off) : 0.f, w1 = has1 ? ex2(o1 - off) : 0.f;
      const float lt = (has0 ? times_2(l0, o0 - off) : 0.f) + (has1 ? times_2(l1, o1 - off) : 0.f);
      const Seg& g = walk->g;
      const Row mine = row();
      const bool whole = sg.j0 == 0 && sg.j1 == g.nblk;
      float vmul = 1.f;
      if (p.mode == KVQ_SCALE_PER_HEAD) vmul = p.v_static[g.kvh];
      if (p.mode == KVQ_SCALE_PER_TENSOR) vmul = p.v_static[0];
      const float mul = whole ? (lt != 0.f ? vmul / lt : 0.f) : vmul;
      const long prow = (2L * blockIdx.x + (sg.j0 == 0 ? 1 : 0)) * kTreeRows + r;    // partial row
      if (!whole && st == 0 && mine.ok) *reinterpret_cast<float2*>(p.ws_ml + 2 * prow) = make_float2(off, lt);
      if (warp_ok) {
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          const int d0 = 64 * st + 16 * cc;
          uint32_t a[16], b[16];
          tc::ld16_issue(lanes + kTmO + d0, a);
          tc::ld16_issue(lanes + kTmO + 128 + d0, b);
          tc::ld_wait16(a);
          tc::ld_wait16(b);
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = ((has0 ? __uint_as_float(a[i]) * w0 : 0.f) + (has1 ? __uint_as_float(b[i]) * w1 : 0.f)) * mul;
          if (nonfinite && mine.ok) {
            // drafted rows with infinities or NaN in V: their other elements were in the tile; these
            // are added to the rows that see them
            for (int pos = max(first, sg.j0 * kTreeBlk); pos < min(sg.n, sg.j1 * kTreeBlk); ++pos) {
              const int t = pos - first;
              if (!((mine.mask[t >> 5] >> (t & 31)) & 1u)) continue;
              const int blk = p.tables[static_cast<long>(g.b) * p.max_blocks + pos / kBS];
              if (blk < 0 || blk >= p.NB) continue;
              const uint8_t* rec = p.pages + (static_cast<long>(blk) * p.H + g.kvh) * Y::REC;
              const uint8_t* row = rec + Y::OFF_V + (pos % kBS) * Y::ROWB;
              float s = 1.f;
              if constexpr (PT) s = reinterpret_cast<const float*>(rec + Y::OFF_S)[kBS + pos % kBS];
              for (int i = 0; i < 16; ++i) {
                float e;
                if constexpr (CD == KVQ_DTYPE_INT8) e = static_cast<float>(static_cast<int8_t>(row[d0 + i]));
                else if constexpr (CD == KVQ_DTYPE_FP8_E4M3) e = e4m3_to_float(row[d0 + i]);
                else if constexpr (CD == KVQ_DTYPE_BF16) e = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[d0 + i]);
                else e = __half2float(reinterpret_cast<const __half*>(row)[d0 + i]);
                e *= s;
                if (!(fabsf(e) <= 3.4028235e38f)) v[i] += e;
              }
            }
          }
          if (!mine.ok) continue;
          if (!whole) {
            float4* dst = reinterpret_cast<float4*>(p.ws_o + prow * kD + d0);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else if (p.out_dtype == KVQ_DTYPE_FP32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + mine.q * kD + d0);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            const bool bf = p.out_dtype == KVQ_DTYPE_BF16;
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + mine.q * kD + d0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float x0 = v[8 * i + 2 * e], x1 = v[8 * i + 2 * e + 1];
                w[e] = bf ? pack_bf16x2(x0, x1) : pack_f16x2(x0, x1);
              }
              dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      tc::fence_before_sync();
      // every warp has read the accumulators and the exchange area before the next unit begins
      ok = sync8();
    }
    if (!ok && lane == 0) fail(p, sh.abort);
  }
  // ---------------------------------------------------------------- teardown
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kOutWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, kTmemCols);
  }
}

// Joins the partial results of units cut between CTAs: a warp per query row, 4 channels per lane, and
// `per_warp` rows one after another, so that large calls read the schedule once for many rows.  A
// unit that lies in one CTA's range was written by that CTA.  What bounds it is the chain of loads: the
// schedule is worked out before the wait for the attention kernel (which let this one start only after
// its own wait: what ran before it is complete), and N partial rows are on their way at a time: 16 where
// one row is all a warp has (1032 tokens, 17 parts a row: the call takes 20.5 us, 25 with 8 behind a look
// at their sums), 8 where more warps per SM hide the loads.
template <int N>
__global__ void __launch_bounds__(256, N == 16 ? 2 : 4) tree_merge_kernel(TreeParams p, int per_warp) {
  const int b = blockIdx.z, kvh = blockIdx.y, lane = threadIdx.x & 31;
  const TreeSeq s = tree_seq(p, b);
  unsigned W = 0, before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int bb = b0 + lane;
    const unsigned w = bb < p.B ? tree_work(p, tree_seq(p, bb)) : 0;
    W += __reduce_add_sync(0xffffffffu, w);
    before += __reduce_add_sync(0xffffffffu, bb < b ? w : 0);
  }
  const int nblk = tree_blocks(s.n);
  const unsigned unit0 = before + p.lead;                     // the sequence's first unit's first block
  int last = -1, member = 0, c0 = 0, c1 = 0;                  // the tile before; the shares of its first and last block
  bool waited = false;
#pragma unroll 1
  for (int k = 0; k < per_warp; ++k) {
    const int x = (blockIdx.x * per_warp + k) * 8 + (threadIdx.x >> 5);   // row of the sequence and kv head
    const int tile = x / kTreeRows, r = x % kTreeRows;
    if (x < s.L * p.g && tile != last) {
      last = tile;
      const int group = tile / p.group;
      member = tile - group * p.group;
      const unsigned U0 = unit0 + (kvh * tree_tile_rows(p, s.L) + group) * (nblk + p.lead);
      c0 = tree_share(p, W, U0);
      c1 = tree_share(p, W, U0 + nblk - 1);
    }
    if (!waited) griddep_wait();
    waited = true;
    if (x >= s.L * p.g) return;
    if (c0 == c1) continue;
    auto row_of = [&](int c) { return (2 * (c * p.group + member) + (c == c0 ? 1 : 0)) * kTreeRows + r; };
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* o = p.ws_o + 4 * lane;
#pragma unroll 1
    for (int k0 = c0; k0 <= c1; k0 += N) {
      // lane t < N has the (offset, sum) of group k0 + t
      const int n = min(N, c1 - k0 + 1);
      float2 ml = make_float2(0.f, 0.f);
      if (lane < n) ml = *reinterpret_cast<const float2*>(p.ws_ml + 2 * row_of(k0 + lane));
      float4 v[N];
#pragma unroll
      for (int t = 0; t < N; ++t)
        v[t] = t < n ? *reinterpret_cast<const float4*>(o + static_cast<long>(row_of(k0 + t)) * kD) : make_float4(0.f, 0.f, 0.f, 0.f);
      float mx = ml.y != 0.f ? ml.x : -INFINITY;              // (a sum of 0: nothing seen, and v is zeros)
      const float mk = mx;
#pragma unroll
      for (int d = N / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      mx = __shfl_sync(0xffffffffu, mx, 0);
      if (mx > M) {
        const float f = M == -INFINITY ? 0.f : ex2(M - mx);
        L = M == -INFINITY ? 0.f : times_2(L, M - mx);
        M = mx;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
      }
      const float w = ml.y != 0.f ? ex2(mk - M) : 0.f;
      if (ml.y != 0.f) L += times_2(ml.y, mk - M);
#pragma unroll
      for (int t = 0; t < N; ++t) {
        const float wt = __shfl_sync(0xffffffffu, w, t);
        acc.x = fmaf(v[t].x, wt, acc.x);
        acc.y = fmaf(v[t].y, wt, acc.y);
        acc.z = fmaf(v[t].z, wt, acc.z);
        acc.w = fmaf(v[t].w, wt, acc.w);
      }
    }
#pragma unroll
    for (int d = N / 2; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    L = __shfl_sync(0xffffffffu, L, 0);
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const int tok = x / p.g;
    const long e0 = ((static_cast<long>(s.q0) + tok) * p.Hq + static_cast<long>(kvh) * p.g + (x - tok * p.g)) * kD + 4 * lane;
    if (p.out_dtype == KVQ_DTYPE_FP32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + e0) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
      const bool bf = p.out_dtype == KVQ_DTYPE_BF16;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + e0) =
          bf ? make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv))
             : make_uint2(pack_f16x2(acc.x * inv, acc.y * inv), pack_f16x2(acc.z * inv, acc.w * inv));
    }
  }
}

template <int CD, bool PT, bool HILO>
cudaError_t launch(const TreeParams& p, const Geometry& g, cudaStream_t s) {
  using Y = Layout<CD, PT>;
  if (g.record != Y::REC) return cudaErrorInvalidValue;
  // (every call: the attribute belongs to the current device's copy of the kernel)
  cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<CD, PT, HILO>, cudaFuncAttributeMaxDynamicSharedMemorySize, Y::BYTES);
  if (e != cudaSuccess) return e;
  CUtensorMap rows = {};
  if constexpr (Y::DIRECT) {
    const long nrows = static_cast<long>(g.NB) * g.H * 2 * kBS;
    if (!make_rows_map(&rows, p.pages, nrows, Y::ROWB, kBS)) return cudaErrorInvalidValue;
  }
  tree_tc_kernel<CD, PT, HILO><<<p.ctas, kThreads, Y::BYTES, s>>>(p, rows);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // rows per warp: about four times the CTAs that the SMs hold (most find units that were not cut)
  const long most = static_cast<long>(p.max_tree) * p.g, warps = most * p.H * p.B;
  const bool one = warps <= 2L * 8 * p.ctas;
  const int per_warp = one ? 1 : static_cast<int>(std::min((warps + 16L * 8 * p.ctas - 1) / (16L * 8 * p.ctas), (most + 7) / 8));
  const dim3 grid(static_cast<unsigned>((most + 8L * per_warp - 1) / (8L * per_warp)), p.H, p.B);
  return one ? launch_dependent(tree_merge_kernel<16>, grid, dim3(256), 0, s, p, per_warp)
             : launch_dependent(tree_merge_kernel<8>, grid, dim3(256), 0, s, p, per_warp);
}

}  // namespace

bool tree_tc_supported(const Geometry& g, int group) {
  return group >= 1 && g.D == kD && g.bs == kBS && !low_bit(g.cache_dtype) && g.scale_mode != KVQ_SCALE_PER_CHANNEL;
}

cudaError_t launch_tree_tc(const TreeParams& p, const Geometry& g, cudaStream_t s) {
  const bool pt = g.scale_mode == KVQ_SCALE_PER_TOKEN_HEAD, hilo = p.out_dtype != KVQ_DTYPE_BF16;
  switch (g.cache_dtype) {
    case KVQ_DTYPE_INT8:
      if (pt) return hilo ? launch<KVQ_DTYPE_INT8, true, true>(p, g, s) : launch<KVQ_DTYPE_INT8, true, false>(p, g, s);
      return hilo ? launch<KVQ_DTYPE_INT8, false, true>(p, g, s) : launch<KVQ_DTYPE_INT8, false, false>(p, g, s);
    case KVQ_DTYPE_FP8_E4M3:
      if (pt) return hilo ? launch<KVQ_DTYPE_FP8_E4M3, true, true>(p, g, s) : launch<KVQ_DTYPE_FP8_E4M3, true, false>(p, g, s);
      return hilo ? launch<KVQ_DTYPE_FP8_E4M3, false, true>(p, g, s) : launch<KVQ_DTYPE_FP8_E4M3, false, false>(p, g, s);
    case KVQ_DTYPE_FP16: return hilo ? launch<KVQ_DTYPE_FP16, false, true>(p, g, s) : launch<KVQ_DTYPE_FP16, false, false>(p, g, s);
    case KVQ_DTYPE_BF16: return launch<KVQ_DTYPE_BF16, false, true>(p, g, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
