// Cache rows by slot: read back as K and V of the activation type (kvq_gather), and the
// accepted path of a drafted tree moved to its final positions (kvq_tree_commit).
//
// Both are bound by bytes.  kvq_gather: one CTA per listed row (token); D / 16 lanes per
// (K or V, kv head) row, 16 elements each, so a lane's codes are one load and its output two
// 16-byte stores; two rows' loads are in flight per lane.  Values are the dequantized values
// of include/kvq.h, formed in binary32 and rounded once to the activation type.
//
// kvq_tree_commit: the j-th accepted row moves from position first + path[j] to first + j.
// The path is strictly increasing, so path[j] >= j: a destination never lies beyond its
// source, and moving the rows in order, each batch read whole before it is written, never
// overwrites a row still to be read.  Codes and per-token scales move as bytes.
#include <algorithm>

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

// grid T: row t of the output is the cache row of slots[t] (left as it was for -1).  Lane
// group i of the CTA takes (K or V, head) rows i, i + groups, ...
template <typename TA, int CD, int D>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(GatherParams p, int bs_shift) {
  constexpr int LPR = D / 16;
  constexpr int GROUPS = kRowThreads / LPR;
  constexpr bool LB = CD == KVQ_DTYPE_INT4 || CD == KVQ_DTYPE_INT2;
  const int t = blockIdx.x, l = threadIdx.x % LPR;
  const int slot = p.slots[t];
  const long nslots = static_cast<long>(p.NB) * p.bs;
  if (slot < 0 || slot >= nslots) {
    if (slot != -1 && threadIdx.x == 0) record_fault(p.fault, KVQ_FAULT_SLOT);
    return;
  }
  const int blk = bs_shift >= 0 ? slot >> bs_shift : slot / p.bs;
  const int off = slot - blk * p.bs;
  const uint8_t* rec0 = p.pages + static_cast<long>(blk) * p.H * p.record;
  for (int r = threadIdx.x / LPR; r < 2 * p.H; r += GROUPS) {
    const int kv = r >= p.H ? 1 : 0, h = r - kv * p.H;
    const uint8_t* rec = rec0 + static_cast<long>(h) * p.record;
    Codes<CD> c;
    load_codes<CD>(c, rec + (kv ? p.off_v : 0) + off * p.row_bytes, l);
    uint32_t out[8];
    if constexpr (CD == KVQ_DTYPE_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        out[i] = (&c.w[0].x)[i];
        out[4 + i] = (&c.w[1].x)[i];
      }
    } else {
      float x[16];
      if constexpr (LB) {
        constexpr int BITS = CD == KVQ_DTYPE_INT4 ? 4 : 2;
        const uint8_t* prm = rec + p.off_s;
        const bool fz = p.mode == KVQ_SCALE_KIVI_FLOAT_ZERO;
        auto code = [&](int i) {
          if constexpr (BITS == 4) return static_cast<float>(((i < 8 ? c.w.x : c.w.y) >> (4 * (i & 7))) & 15u);
          else return static_cast<float>((c.w >> (2 * i)) & 3u);
        };
        // code * s + minimum, or (code - z) * s
        auto value = [&](float q, float s, float z) { return fz ? fmaf(q, s, z) : (q - z) * s; };
        if (kv == 0 && p.mode != KVQ_SCALE_INT4_PER_TOKEN) {
          // per channel: scale [D], then zero point [D]
          uint4 s[2], z[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            s[i] = reinterpret_cast<const uint4*>(prm)[2 * l + i];
            z[i] = reinterpret_cast<const uint4*>(prm + 2 * D)[2 * l + i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 sv = half2_at((&s[i >> 2].x)[i & 3]), zv = half2_at((&z[i >> 2].x)[i & 3]);
            x[2 * i] = value(code(2 * i), sv.x, zv.x);
            x[2 * i + 1] = value(code(2 * i + 1), sv.y, zv.y);
          }
        } else {
          // per token and 64-channel group: (scale, zero point) [bs][D/64]
          const float2 sz = half2_at(
              reinterpret_cast<const uint32_t*>(prm + (kv ? 4 * D : 0))[off * (D / 64) + l / 4]);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = value(code(i), sz.x, sz.y);
        }
      } else {
        const float* st = kv ? p.v_static : p.k_static;
        float s = 1.f;
        if (p.mode == KVQ_SCALE_PER_TOKEN_HEAD)
          s = reinterpret_cast<const float*>(rec + p.off_s)[(kv ? p.bs : 0) + off];
        else if (p.mode == KVQ_SCALE_PER_HEAD) s = st[h];
        else if (p.mode == KVQ_SCALE_PER_TENSOR) s = st[0];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = (&c.w.x)[i];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint8_t b = static_cast<uint8_t>(w >> (8 * e));
            x[4 * i + e] = CD == KVQ_DTYPE_INT8 ? static_cast<float>(static_cast<int8_t>(b)) : e4m3_to_float(b);
          }
        }
        if (p.mode == KVQ_SCALE_PER_CHANNEL) {
          const float4* cs = reinterpret_cast<const float4*>(st + static_cast<long>(h) * D + 16 * l);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f = cs[i];
            x[4 * i] *= f.x;
            x[4 * i + 1] *= f.y;
            x[4 * i + 2] *= f.z;
            x[4 * i + 3] *= f.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= s;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        out[i] = std::is_same<TA, __nv_bfloat16>::value ? pack_bf16x2(x[2 * i], x[2 * i + 1])
                                                        : pack_f16x2(x[2 * i], x[2 * i + 1]);
    }
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv ? p.v_out : p.k_out) +
                                          (static_cast<long>(t) * p.H + h) * D) + 2 * l;
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

template <typename TA, int CD>
cudaError_t launch_gather_dim(const GatherParams& p, int D, int shift, int T, cudaStream_t s) {
  if (D == 64) gather_kernel<TA, CD, 64><<<T, kRowThreads, 0, s>>>(p, shift);
  else gather_kernel<TA, CD, 128><<<T, kRowThreads, 0, s>>>(p, shift);
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

constexpr int kCommitRows = 32;      // rows looked up and moved per batch
constexpr int kCommitUnits = 4;      // 16-byte pieces a thread carries per batch

// grid (B, head tiles): CTA (b, y) moves the accepted rows of heads y, y + gridDim.y, ...
// Thread 0..31 look up a batch of rows; all threads then read their pieces of it, and after
// a barrier write them.
__global__ void __launch_bounds__(kRowThreads) commit_kernel(CommitParams p) {
  __shared__ long src_at[kCommitRows], dst_at[kCommitRows];   // record of (block, head 0), or -1
  __shared__ int src_off[kCommitRows], dst_off[kCommitRows];
  __shared__ int bad;
  const int b = blockIdx.x;
  const int n = p.lens[b], a = p.accepted[b], L = p.q_start[b + 1] - p.q_start[b];
  const long first = static_cast<long>(n) - L;
  const bool report = blockIdx.y == 0;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  bool ok = L >= 0 && first >= 0 && n <= static_cast<long>(p.max_blocks) * p.bs && a >= 0 && a <= L && a <= p.max_accept;
  if (!ok) {
    if (report && threadIdx.x == 0) {
      record_fault(p.fault, KVQ_FAULT_CONTEXT);
      if (p.new_lens != nullptr) p.new_lens[b] = n;
    }
    return;
  }
  const int32_t* path = p.path + static_cast<long>(b) * p.max_accept;
  const int32_t* table = p.tables + static_cast<long>(b) * p.max_blocks;
  // the whole path is checked first: nothing of a bad one moves
  for (int j = threadIdx.x; j < a; j += kRowThreads) {
    const int s = path[j];
    bool fine = s >= 0 && s < L && (j == 0 || s > path[j - 1]);
    if (fine) {
      const int sb = table[(first + s) / p.bs], db = table[(first + j) / p.bs];
      fine = sb >= 0 && sb < p.NB && db >= 0 && db < p.NB;
    }
    if (!fine) bad = 1;
  }
  __syncthreads();
  if (bad) {
    if (report && threadIdx.x == 0) {
      record_fault(p.fault, KVQ_FAULT_TREE);
      if (p.new_lens != nullptr) p.new_lens[b] = n;
    }
    return;
  }
  if (report && threadIdx.x == 0 && p.new_lens != nullptr) p.new_lens[b] = static_cast<int>(first) + a;
  const int chunks = p.row_bytes / 16;                  // 16-byte pieces of a K (or V) row
  const int heads = (p.H - blockIdx.y + gridDim.y - 1) / gridDim.y;
  const int per_row = heads * 2 * chunks;
  for (int j0 = 0; j0 < a; j0 += kCommitRows) {
    const int m = min(kCommitRows, a - j0);
    __syncthreads();
    if (threadIdx.x < m) {
      const long s = first + path[j0 + threadIdx.x], d = first + j0 + threadIdx.x;
      src_at[threadIdx.x] = s == d ? -1 : static_cast<long>(table[s / p.bs]) * p.H * p.record;
      dst_at[threadIdx.x] = static_cast<long>(table[d / p.bs]) * p.H * p.record;
      src_off[threadIdx.x] = static_cast<int>(s % p.bs);
      dst_off[threadIdx.x] = static_cast<int>(d % p.bs);
    }
    __syncthreads();
    // rows in order: a batch of whole rows is read before any of it is written
    const int fit = max(1, kCommitUnits * kRowThreads / per_row);
    for (int r0 = 0; r0 < m; r0 += fit) {
      const int items = min(fit, m - r0) * per_row;
      for (int i0 = 0; i0 < items; i0 += kCommitUnits * kRowThreads) {
        // (several rounds only when one row alone exceeds a batch: its pieces are disjoint)
        uint4 w[kCommitUnits];
        float sc[kCommitUnits];
        long to[kCommitUnits];
        int sc_to[kCommitUnits];
#pragma unroll
        for (int u = 0; u < kCommitUnits; ++u) {
          const int i = i0 + u * kRowThreads + threadIdx.x;
          to[u] = -1;
          sc_to[u] = -1;
          if (i < items) {
            const int r = r0 + i / per_row, rest = i % per_row;
            const int hk = rest / chunks, c = rest - hk * chunks;
            const int h = blockIdx.y + (hk >> 1) * gridDim.y, kv = hk & 1;
            if (src_at[r] >= 0) {
              const long rec_s = src_at[r] + static_cast<long>(h) * p.record, rec_d = dst_at[r] + static_cast<long>(h) * p.record;
              const int row = kv ? p.off_v : 0;
              w[u] = *reinterpret_cast<const uint4*>(p.pages + rec_s + row + src_off[r] * p.row_bytes + 16 * c);
              to[u] = rec_d + row + dst_off[r] * p.row_bytes + 16 * c;
              if (p.scales && c == 0) {
                sc[u] = reinterpret_cast<const float*>(p.pages + rec_s + p.off_s)[kv * p.bs + src_off[r]];
                sc_to[u] = kv * p.bs + dst_off[r];
              }
            }
          }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kCommitUnits; ++u) {
          if (to[u] >= 0) *reinterpret_cast<uint4*>(p.pages + to[u]) = w[u];
          if (sc_to[u] >= 0) {
            // the record: back from the row piece's address (c == 0)
            const int kv = sc_to[u] >= p.bs ? 1 : 0;
            const long rec = to[u] - (kv ? p.off_v : 0) - static_cast<long>(sc_to[u] - kv * p.bs) * p.row_bytes;
            reinterpret_cast<float*>(p.pages + rec + p.off_s)[sc_to[u]] = sc[u];
          }
        }
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
      block_tables == nullptr || context_lens == nullptr || new_lens == context_lens)
    return KVQ_ERR_INVALID_ARG;
  const CommitParams p{path, accepted, q_start, block_tables, context_lens, new_lens,
                       static_cast<uint8_t*>(c->pages), max_accept, max_blocks_per_seq, batch,
                       g.NB, g.bs, g.H, g.record, g.off_v, g.off_s, g.row_bytes,
                       g.scale_mode == KVQ_SCALE_PER_TOKEN_HEAD, c->fault};
  // heads are spread over CTAs until every SM has a few
  const int tiles = std::max(1, std::min(g.H, 8 * device_sm_count() / batch));
  commit_kernel<<<dim3(batch, tiles), kRowThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
