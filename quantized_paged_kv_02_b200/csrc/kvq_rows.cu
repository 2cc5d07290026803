// Cache rows by slot: read back as K and V of the activation type (kvq_gather), and the
// accepted path of a drafted tree moved to its final positions (kvq_tree_commit).
//
// Both are bound by bytes.  kvq_gather: D / 16 lanes per (K or V, kv head) row, 16 elements
// each, so a lane's codes are one load and its output two 16-byte stores; a thread reads the
// same column of several rows, four rows' loads in flight.  Values are the dequantized values
// of include/kvq.h, formed in binary32 and rounded once to the activation type.
//
// kvq_tree_commit: the j-th accepted row moves from position first + path[j] to first + j.
// The path is strictly increasing, so path[j] >= j: a destination never lies beyond its
// source, and moving the rows in order, each batch read whole before it is written, never
// overwrites a row still to be read.  Codes and per-token scales move as bytes.
//
// Measured (B200, behind an L2 flush / back to back): gather of 32-head INT8 rows 18 / 12 us for 2048 tokens,
// 45 / 41 for 8192, 141 / 138 for 32640, so some 13 us of start and end and then 1.04 times the bytes' time
// at copy speed; 32640 x 8 INT4 rows 49 / 47 us, 1.5 times the bytes' time a further row: their unpacking has the
// issue slots 79% busy, DRAM 28%.  Commit of 256 trees of 64 over 32 bf16 heads 24 / 20 us (10.9 at copy
// speed): two dependent loads (path, table) before a row's bytes can be asked for, in 2.6 waves of
// CTAs; DRAM 20% busy.
#include <algorithm>

#include "kvq_checks.cuh"
#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"

namespace kvq {
namespace {

struct GatherParams {
  const int32_t* slots;
  const uint8_t* pages;
  const float* k_static;
  const float* v_static;
  int NB, bs, H;
  int record, off_v, off_s, row_bytes, mode;
  void* k_out;
  void* v_out;
  int32_t* fault;
};

constexpr int kRowThreads = 256;

__device__ __forceinline__ float2 half2_at(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// An integer below 2^23 as a float, without a conversion (those run at a quarter of the rate).
__device__ __forceinline__ float small_float(uint32_t i) { return __uint_as_float(i | 0x4B000000u) - 8388608.f; }

// Codes of one lane: 16 elements.
template <int CD> struct Codes { uint4 w; };                       // 8-bit codes
template <> struct Codes<KVQ_DTYPE_BF16> { uint4 w[2]; };
template <> struct Codes<KVQ_DTYPE_INT4> { uint2 w; };
template <> struct Codes<KVQ_DTYPE_INT2> { uint32_t w; };

template <int CD>
__device__ __forceinline__ void load_codes(Codes<CD>& c, const uint8_t* row, int l) {
  if constexpr (CD == KVQ_DTYPE_BF16) {
    c.w[0] = reinterpret_cast<const uint4*>(row)[2 * l];
    c.w[1] = reinterpret_cast<const uint4*>(row)[2 * l + 1];
  } else {
    c.w = reinterpret_cast<const decltype(c.w)*>(row)[l];
  }
}

// 16 elements of one row as packed 16-bit outputs.  `prm`: the low-bit parameters of a K row per
// channel (scale [16], zero point [16], as loaded), else unused; `s`, `z`: the row's scale and zero
// point (per token and group, per token, or static).
template <typename TA, int CD>
__device__ __forceinline__ void row_values(const Codes<CD>& c, const uint4* prm, bool channel, float s, float z, bool fz,
                                           const float4* chan, uint32_t* out) {
  if constexpr (CD == KVQ_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i] = (&c.w[0].x)[i];
      out[4 + i] = (&c.w[1].x)[i];
    }
    return;
  } else {
    float x[16];
    if constexpr (CD == KVQ_DTYPE_INT4 || CD == KVQ_DTYPE_INT2) {
      auto code = [&](int i) {
        if constexpr (CD == KVQ_DTYPE_INT4) return small_float(((i < 8 ? c.w.x : c.w.y) >> (4 * (i & 7))) & 15u);
        else return small_float((c.w >> (2 * i)) & 3u);
      };
      // code * s + minimum, or (code - z) * s
      auto value = [&](float q, float sv, float zv) { return fz ? fmaf(q, sv, zv) : (q - zv) * sv; };
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 sv = make_float2(s, s), zv = make_float2(z, z);
        if (channel) {
          sv = half2_at((&prm[i >> 2].x)[i & 3]);
          zv = half2_at((&prm[2 + (i >> 2)].x)[i & 3]);
        }
        x[2 * i] = value(code(2 * i), sv.x, zv.x);
        x[2 * i + 1] = value(code(2 * i + 1), sv.y, zv.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = (&c.w.x)[i];
        float4 f = make_float4(s, s, s, s);
        if (chan != nullptr) f = chan[i];
        __half2 h8[2];                         // (E4M3 is exact in fp16)
        if constexpr (CD == KVQ_DTYPE_FP8_E4M3) {
          const uint32_t lo = e4m3x2_to_f16x2(w & 0xFFFFu), hi = e4m3x2_to_f16x2(w >> 16);
          h8[0] = *reinterpret_cast<const __half2*>(&lo);
          h8[1] = *reinterpret_cast<const __half2*>(&hi);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v;
          if constexpr (CD == KVQ_DTYPE_INT8)   // byte + 128 under the exponent of 2^23
            v = __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4B000000u, 0x7650u + e)) - 8388736.f;
          else
            v = e & 1 ? __high2float(h8[e >> 1]) : __low2float(h8[e >> 1]);
          x[4 * i + e] = v * (&f.x)[e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out[i] = std::is_same<TA, __nv_bfloat16>::value ? pack_bf16x2(x[2 * i], x[2 * i + 1])
                                                      : pack_f16x2(x[2 * i], x[2 * i + 1]);
  }
}

// grid (ceil(T / tokens), columns): CTA x reads back the rows of `tokens` slots.  A thread keeps one
// (K or V, head, lane) column for all its tokens, `par` tokens side by side in a CTA where a token
// has few columns, four rows' loads in flight; INT4 / INT2 keys whose parameters are per channel
// load those again only when the block changes.
template <typename TA, int CD, int D>
__global__ void __launch_bounds__(kRowThreads, 4) gather_kernel(GatherParams p, int T, int tokens, int par, int bs_shift) {
  constexpr int LPR = D / 16;
  constexpr bool LB = CD == KVQ_DTYPE_INT4 || CD == KVQ_DTYPE_INT2;
  constexpr int U = 4;
  const int t0 = blockIdx.x * tokens, nt = min(tokens, T - t0);
  const int cols = 2 * p.H * LPR;
  int sub = 0, col = blockIdx.y * kRowThreads + threadIdx.x;
  if (par > 1) {
    sub = threadIdx.x / cols;
    col = threadIdx.x - sub * cols;
    if (sub >= par) return;
  }
  if (col >= cols) return;
  const int r = col / LPR, l = col - r * LPR, kv = r >= p.H ? 1 : 0, h = r - kv * p.H;
  const bool channel = LB && kv == 0 && p.mode != KVQ_SCALE_INT4_PER_TOKEN;
  const bool fz = p.mode == KVQ_SCALE_KIVI_FLOAT_ZERO;
  const float* st = kv ? p.v_static : p.k_static;
  float fixed = 1.f;
  float4 chan[4];
  if constexpr (!LB && CD != KVQ_DTYPE_BF16) {
    if (p.mode == KVQ_SCALE_PER_HEAD) fixed = st[h];
    if (p.mode == KVQ_SCALE_PER_TENSOR) fixed = st[0];
    if (p.mode == KVQ_SCALE_PER_CHANNEL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) chan[i] = reinterpret_cast<const float4*>(st + static_cast<long>(h) * D + 16 * l)[i];
    }
  }
  uint16_t* out = static_cast<uint16_t*>(kv ? p.v_out : p.k_out) + static_cast<long>(h) * D + 16 * l;
  uint4 prm[4];
  int prm_blk = -1;
  // (slots are int32, so at most 2^31 of them can be named)
  const long pool = static_cast<long>(p.NB) * p.bs, nslots = pool < (1L << 31) ? pool : (1L << 31);
  auto parameters = [&](int blk) {              // per channel: scale [D], then zero point [D]
    const uint8_t* base = p.pages + (static_cast<long>(blk) * p.H + h) * p.record + p.off_s + 32 * l;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      prm[i] = reinterpret_cast<const uint4*>(base)[i];
      prm[2 + i] = reinterpret_cast<const uint4*>(base + 2 * D)[i];
    }
    prm_blk = blk;
  };
  for (int k0 = sub; k0 < nt; k0 += U * par) {
    Codes<CD> c[U];
    float s[U];
    uint32_t sz[U];
    int slot[U], blk[U];
#pragma unroll
    for (int a = 0; a < U; ++a) {
      const int k = k0 + a * par;
      slot[a] = k < nt ? p.slots[t0 + k] : -1;
      if (slot[a] < 0 || slot[a] >= nslots) {
        if (slot[a] != -1 && col == 0) record_fault(p.fault, KVQ_FAULT_SLOT);
        slot[a] = -1;
      }
    }
#pragma unroll
    for (int a = 0; a < U; ++a) {
      if (slot[a] < 0) continue;
      blk[a] = bs_shift >= 0 ? slot[a] >> bs_shift : slot[a] / p.bs;
      const int off = slot[a] - blk[a] * p.bs;
      const uint8_t* rec = p.pages + (static_cast<long>(blk[a]) * p.H + h) * p.record;
      load_codes<CD>(c[a], rec + (kv ? p.off_v : 0) + off * p.row_bytes, l);
      if constexpr (LB) {
        if (a == 0 && channel && blk[0] != prm_blk) parameters(blk[0]);   // beside the codes
      }
      s[a] = fixed;
      sz[a] = 0;
      if constexpr (LB) {
        // per token and 64-channel group: (scale, zero point) [bs][D/64], K's before V's
        if (!channel) sz[a] = reinterpret_cast<const uint32_t*>(rec + p.off_s + (kv ? 4 * D : 0))[off * (D / 64) + l / 4];
      } else if constexpr (CD != KVQ_DTYPE_BF16) {
        if (p.mode == KVQ_SCALE_PER_TOKEN_HEAD) s[a] = reinterpret_cast<const float*>(rec + p.off_s)[(kv ? p.bs : 0) + off];
      }
    }
#pragma unroll
    for (int a = 0; a < U; ++a) {
      if (slot[a] < 0) continue;
      float z = 0.f;
      if constexpr (LB) {
        if (channel) {
          if (blk[a] != prm_blk) parameters(blk[a]);
        } else {
          const float2 f = half2_at(sz[a]);
          s[a] = f.x;
          z = f.y;
        }
      }
      uint32_t w[8];
      row_values<TA, CD>(c[a], prm, channel, s[a], z, fz, p.mode == KVQ_SCALE_PER_CHANNEL ? chan : nullptr, w);
      uint4* dst = reinterpret_cast<uint4*>(out + static_cast<long>(t0 + k0 + a * par) * p.H * D);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <typename TA, int CD>
cudaError_t launch_gather_dim(const GatherParams& p, int D, int shift, int T, cudaStream_t s) {
  const int cols = 2 * p.H * (D / 16), par = std::max(1, kRowThreads / cols);
  const int slices = (cols + kRowThreads - 1) / kRowThreads;
  // four rows per thread (one round of loads), fewer below four CTAs per SM; eight, for the parameters
  // they share, once there are more
  const int one = std::max(1, device_sm_count() * par / slices);   // rows that give each SM one CTA
  const int each = T >= 4 * 8 * one ? 8 : std::max(1, std::min(4, T / (4 * one)));
  const int tokens = each * par;
  const dim3 grid((T + tokens - 1) / tokens, slices);
  if (D == 64) gather_kernel<TA, CD, 64><<<grid, kRowThreads, 0, s>>>(p, T, tokens, par, shift);
  else gather_kernel<TA, CD, 128><<<grid, kRowThreads, 0, s>>>(p, T, tokens, par, shift);
  return cudaGetLastError();
}

template <typename TA>
cudaError_t launch_gather(const GatherParams& p, int cd, int D, int shift, int T, cudaStream_t s) {
  switch (cd) {
    case KVQ_DTYPE_INT8: return launch_gather_dim<TA, KVQ_DTYPE_INT8>(p, D, shift, T, s);
    case KVQ_DTYPE_FP8_E4M3: return launch_gather_dim<TA, KVQ_DTYPE_FP8_E4M3>(p, D, shift, T, s);
    case KVQ_DTYPE_INT4: return launch_gather_dim<TA, KVQ_DTYPE_INT4>(p, D, shift, T, s);
    case KVQ_DTYPE_INT2: return launch_gather_dim<TA, KVQ_DTYPE_INT2>(p, D, shift, T, s);
    default: return launch_gather_dim<TA, KVQ_DTYPE_BF16>(p, D, shift, T, s);   // 16-bit rows as they are
  }
}

// ------------------------------------------------------------------ commit
struct CommitParams {
  const int32_t* path;         // [B][max_accept]
  const int32_t* accepted;     // [B]
  const int32_t* q_start;      // [B+1]
  const int32_t* tables;
  const int32_t* lens;
  int32_t* new_lens;           // or null
  uint8_t* pages;
  int max_accept, max_blocks, B;
  int NB, bs, H, record, off_v, off_s, row_bytes;
  bool scales;                 // per-token scales move too
  int32_t* fault;
};

constexpr int kCommitRows = 64;      // rows whose records are looked up together
constexpr int kCommitUnits = 4;      // 16-byte pieces a thread carries per batch

// grid (B, head tiles): CTA (b, y) moves the accepted rows of heads y, y + gridDim.y, ...
// The threads check the path and look its rows' records up, then read their pieces of as many
// rows as fit their registers, and after a barrier write them.
__global__ void __launch_bounds__(kRowThreads, 6) commit_kernel(CommitParams p) {
  __shared__ long src_at[kCommitRows], dst_at[kCommitRows];   // record of (block, head 0); source -1: stays
  __shared__ int src_off[kCommitRows], dst_off[kCommitRows];
  __shared__ int bad;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int32_t* path = p.path + static_cast<long>(b) * p.max_accept;
  const int32_t* table = p.tables + static_cast<long>(b) * p.max_blocks;
  // (the first rows' path is read beside the lengths, not behind them)
  const int pv = tid < p.max_accept ? path[tid] : 0, before = tid > 0 && tid < p.max_accept ? path[tid - 1] : -1;
  const int n = p.lens[b], a = p.accepted[b], L = p.q_start[b + 1] - p.q_start[b];
  const long first = static_cast<long>(n) - L;
  const bool report = blockIdx.y == 0 && tid == 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  if (!(L >= 0 && first >= 0 && n <= static_cast<long>(p.max_blocks) * p.bs && a >= 0 && a <= L && a <= p.max_accept)) {
    if (report) {
      record_fault(p.fault, KVQ_FAULT_CONTEXT);
      if (p.new_lens != nullptr) p.new_lens[b] = n;
    }
    return;
  }
  // record of (block, head 0) and offset of row j's source and destination, kept at i
  auto look = [&](int j, int s, int prev, int i) -> bool {
    if (!(s > prev && s >= 0 && s < L)) return false;
    const int sp = static_cast<int>(first) + s, dp = static_cast<int>(first) + j;
    const int sq = sp / p.bs, dq = dp / p.bs;
    const int sb = table[sq], db = table[dq];
    if (sb < 0 || sb >= p.NB || db < 0 || db >= p.NB) return false;
    if (i >= 0) {
      src_at[i] = sp == dp ? -1 : static_cast<long>(sb) * p.H * p.record;
      dst_at[i] = static_cast<long>(db) * p.H * p.record;
      src_off[i] = sp - sq * p.bs;
      dst_off[i] = dp - dq * p.bs;
    }
    return true;
  };
  // the whole path is checked first: nothing of a bad one moves
  if (tid < a && !look(tid, pv, before, tid < kCommitRows ? tid : -1)) bad = 1;
  for (int j = tid + kRowThreads; j < a; j += kRowThreads)
    if (!look(j, path[j], path[j - 1], -1)) bad = 1;
  __syncthreads();
  if (bad) {
    if (report) {
      record_fault(p.fault, KVQ_FAULT_TREE);
      if (p.new_lens != nullptr) p.new_lens[b] = n;
    }
    return;
  }
  if (report && p.new_lens != nullptr) p.new_lens[b] = static_cast<int>(first) + a;
  const int chunks = p.row_bytes / 16;                  // 16-byte pieces of a K (or V) row: 4, 8 or 16
  const int shift = chunks == 16 ? 4 : chunks == 8 ? 3 : 2;
  const int heads = (p.H - blockIdx.y + gridDim.y - 1) / gridDim.y;
  const int per_row = heads * 2 * chunks;
  for (int j0 = 0; j0 < a; j0 += kCommitRows) {
    const int m = min(kCommitRows, a - j0);
    if (j0 > 0) {
      __syncthreads();
      if (tid < m) look(j0 + tid, path[j0 + tid], path[j0 + tid - 1], tid);
      __syncthreads();
    }
    // rows in order: a batch of whole rows is read before any of it is written (several rounds
    // only when one row alone exceeds a batch: its pieces are disjoint)
    const int fit = max(1, kCommitUnits * kRowThreads / per_row);
    for (int r0 = 0; r0 < m; r0 += fit) {
      const int mr = min(fit, m - r0), items = mr * per_row;
      for (int i0 = 0; i0 < items; i0 += kCommitUnits * kRowThreads) {
        uint4 w[kCommitUnits];
        uint8_t* to[kCommitUnits];
#pragma unroll
        for (int u = 0; u < kCommitUnits; ++u) {
          const int i = i0 + u * kRowThreads + tid;
          to[u] = nullptr;
          if (i < items) {
            const int rr = i / per_row, rest = i - rr * per_row, r = r0 + rr;
            const int hk = rest >> shift, c = rest & (chunks - 1);
            const long head = static_cast<long>(blockIdx.y + (hk >> 1) * gridDim.y) * p.record + ((hk & 1) ? p.off_v : 0) + 16 * c;
            if (src_at[r] >= 0) {
              w[u] = *reinterpret_cast<const uint4*>(p.pages + src_at[r] + head + src_off[r] * p.row_bytes);
              to[u] = p.pages + dst_at[r] + head + dst_off[r] * p.row_bytes;
            }
          }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kCommitUnits; ++u)
          if (to[u] != nullptr) *reinterpret_cast<uint4*>(to[u]) = w[u];
        __syncthreads();
      }
      // the same rows' scales: one per row, head and K or V
      for (int i0 = 0; p.scales && i0 < mr * heads * 2; i0 += kRowThreads) {
        const int i = i0 + tid;
        float s = 0.f;
        float* to = nullptr;
        if (i < mr * heads * 2) {
          const int rr = i / (heads * 2), hk = i - rr * heads * 2, r = r0 + rr;
          const long head = static_cast<long>(blockIdx.y + (hk >> 1) * gridDim.y) * p.record + p.off_s + ((hk & 1) ? 4 * p.bs : 0);
          if (src_at[r] >= 0) {
            s = reinterpret_cast<const float*>(p.pages + src_at[r] + head)[src_off[r]];
            to = reinterpret_cast<float*>(p.pages + dst_at[r] + head) + dst_off[r];
          }
        }
        __syncthreads();
        if (to != nullptr) *to = s;
        __syncthreads();
      }
    }
  }
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_gather(const kvq_cache_desc* c, const int32_t* slots, int num_rows, void* k_out,
                      void* v_out, cudaStream_t stream) {
  Geometry g;
  const kvq_status st = validate_desc(c, &g);
  if (st != KVQ_OK) return st;
  if (num_rows < 0) return KVQ_ERR_INVALID_ARG;
  if (num_rows == 0) return KVQ_OK;
  if (slots == nullptr || k_out == nullptr || v_out == nullptr || !aligned(k_out) || !aligned(v_out))
    return KVQ_ERR_INVALID_ARG;
  const size_t bytes = static_cast<size_t>(num_rows) * g.H * g.D * 2;
  if (bytes_overlap(k_out, bytes, v_out, bytes)) return KVQ_ERR_INVALID_ARG;
  const GatherParams p{slots, static_cast<const uint8_t*>(c->pages), c->k_scales, c->v_scales, g.NB, g.bs, g.H,
                       g.record, g.off_v, g.off_s, g.row_bytes, g.scale_mode, k_out, v_out, c->fault};
  int shift = -1;
  if ((g.bs & (g.bs - 1)) == 0) for (shift = 0; (1 << shift) < g.bs; ++shift) {}
  const cudaError_t e = g.act_dtype == KVQ_DTYPE_BF16
                            ? launch_gather<__nv_bfloat16>(p, g.cache_dtype, g.D, shift, num_rows, stream)
                            : launch_gather<__half>(p, g.cache_dtype, g.D, shift, num_rows, stream);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_tree_commit(const kvq_cache_desc* c, const int32_t* path, int max_accept,
                           const int32_t* accepted, int batch, const int32_t* q_start,
                           const int32_t* block_tables, int max_blocks_per_seq,
                           const int32_t* context_lens, int32_t* new_lens, cudaStream_t stream) {
  Geometry g;
  const kvq_status st = validate_desc(c, &g);
  if (st != KVQ_OK) return st;
  if (batch < 0 || max_accept < 0 || max_blocks_per_seq < 1) return KVQ_ERR_INVALID_ARG;
  if (low_bit(g.cache_dtype)) return KVQ_ERR_UNSUPPORTED;
  if (batch == 0) return KVQ_OK;
  if ((max_accept > 0 && path == nullptr) || accepted == nullptr || q_start == nullptr ||
      block_tables == nullptr || context_lens == nullptr)
    return KVQ_ERR_INVALID_ARG;
  // (a sequence's CTAs, one per tile of heads, all read these, while the first writes its new length)
  const size_t n = static_cast<size_t>(batch) * sizeof(int32_t);
  if (new_lens != nullptr &&
      (bytes_overlap(new_lens, n, context_lens, n) || bytes_overlap(new_lens, n, accepted, n) ||
       bytes_overlap(new_lens, n, q_start, n + sizeof(int32_t)) || bytes_overlap(new_lens, n, path, n * max_accept) ||
       bytes_overlap(new_lens, n, block_tables, n * max_blocks_per_seq)))
    return KVQ_ERR_INVALID_ARG;
  const CommitParams p{path, accepted, q_start, block_tables, context_lens, new_lens,
                       static_cast<uint8_t*>(c->pages), max_accept, max_blocks_per_seq, batch,
                       g.NB, g.bs, g.H, g.record, g.off_v, g.off_s, g.row_bytes,
                       g.scale_mode == KVQ_SCALE_PER_TOKEN_HEAD, c->fault};
  // heads are spread over CTAs until every SM has a few
  const int tiles = std::max(1, std::min(g.H, 16 * device_sm_count() / batch));
  commit_kernel<<<dim3(batch, tiles), kRowThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
