// Attention of drafted token trees over the paged cache: entry points, plan, the CUDA-core
// kernel for geometries without a tensor-core kernel, and its split reduce.
//
// Query i of sequence b (i < L) sees the prefix p < n - L and the drafted positions n - L + j
// whose bit j is set in its mask row:  o = sum_p softmax_p(scale q . k_p) v_p over those.
//
// CUDA-core kernel.  A CTA takes 16 query rows (row r: token r / g, head r % g) of one
// (sequence, kv head) and one split of the positions, 32 at a time: K and V rows are
// dequantized once into shared memory for the 16 rows, two scores per thread, one warp per
// two rows for the running maximum and sum, then D / 16 output channels per thread.  Masked
// positions are left out by selection, never by multiplication, so that a masked row's
// infinities and NaN reach nobody.  It is the fallback (head_dim 64, block sizes other than 16,
// per-channel scales), bound by shared-memory reads: trees of 16, 8 / 4 heads of 64 over 8 x 4096 INT8
// take 238 us.
#include <algorithm>
#include <cmath>

#include "kvq_ptx.cuh"
#include "kvq_tree.cuh"

namespace kvq {
namespace {

constexpr int kSimtRows = 16, kSimtTok = 32, kSimtThreads = 256;

__device__ __forceinline__ void tree_store(const TreeParams& p, long idx, float v) {
  if (p.out_dtype == KVQ_DTYPE_FP32) static_cast<float*>(p.out)[idx] = v;
  else if (p.out_dtype == KVQ_DTYPE_BF16) static_cast<__nv_bfloat16*>(p.out)[idx] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p.out)[idx] = __float2half_rn(v);
}

// Dequantized element d of row `off` of a record.
__device__ __forceinline__ float cache_value(const TreeParams& p, const uint8_t* rec, int kv, int h, int off, int d) {
  const uint8_t* row = rec + (kv ? p.off_v : 0) + off * p.row_bytes;
  if (p.cache_dtype == KVQ_DTYPE_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[d]);
  if (p.cache_dtype == KVQ_DTYPE_FP16) return __half2float(reinterpret_cast<const __half*>(row)[d]);
  const float* st = kv ? p.v_static : p.k_static;
  const float s = p.mode == KVQ_SCALE_PER_TOKEN_HEAD ? reinterpret_cast<const float*>(rec + p.off_s)[(kv ? p.bs : 0) + off]
                  : p.mode == KVQ_SCALE_PER_HEAD     ? st[h]
                  : p.mode == KVQ_SCALE_PER_CHANNEL  ? st[static_cast<long>(h) * p.D + d]
                                                     : st[0];
  return (p.cache_dtype == KVQ_DTYPE_INT8 ? static_cast<float>(static_cast<int8_t>(row[d])) : e4m3_to_float(row[d])) * s;
}

// grid (row tiles x splits, H, B)
template <typename TA, int D>
__global__ void __launch_bounds__(kSimtThreads) tree_simt_kernel(TreeParams p) {
  __shared__ float ks[kSimtTok][D + 1], vs[kSimtTok][D];
  __shared__ float qs[kSimtRows][D], sc[kSimtRows][kSimtTok];
  __shared__ float row_m[kSimtRows], row_f[kSimtRows], row_l[kSimtRows];
  const int b = blockIdx.z, kvh = blockIdx.y;
  const int tile = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  griddep_wait();
  const TreeSeq s = tree_seq(p, b, blockIdx.x == 0 && kvh == 0 && tid == 0);
  const int R = s.L * p.g, r0 = tile * kSimtRows;
  if (r0 >= R) return;
  const int lo = split * p.chunk, hi = s.n - lo > p.chunk ? lo + p.chunk : s.n;
  for (int e = tid; e < kSimtRows * D; e += kSimtThreads) {
    const int r = r0 + e / D, d = e % D;
    float x = 0.f;
    if (r < R) {
      const long row = (static_cast<long>(s.q0) + r / p.g) * p.Hq + static_cast<long>(kvh) * p.g + r % p.g;
      x = Act<TA>::to_f(static_cast<const TA*>(p.q)[row * D + d]);
    }
    qs[e / D][d] = x * p.scale_log2;
  }
  if (tid < kSimtRows) {
    row_m[tid] = -INFINITY;
    row_l[tid] = 0.f;
  }
  constexpr int DPT = kSimtRows * D / kSimtThreads;        // output channels per thread
  const int orow = tid / (kSimtThreads / kSimtRows), od = tid % (kSimtThreads / kSimtRows) * DPT;
  float o[DPT];
#pragma unroll
  for (int i = 0; i < DPT; ++i) o[i] = 0.f;
  for (int t0 = lo; t0 < hi; t0 += kSimtTok) {
    __syncthreads();
    for (int e = tid; e < kSimtTok * D; e += kSimtThreads) {
      const int t = e / D, d = e % D, pos = t0 + t;
      float kx = 0.f, vx = 0.f;
      if (pos < hi) {
        const int blk = p.tables[static_cast<long>(b) * p.max_blocks + pos / p.bs];
        if (blk >= 0 && blk < p.NB) {
          const uint8_t* rec = p.pages + (static_cast<long>(blk) * p.H + kvh) * p.record;
          kx = cache_value(p, rec, 0, kvh, pos % p.bs, d);
          vx = cache_value(p, rec, 1, kvh, pos % p.bs, d);
        } else if (d == 0 && tile == 0 && pos % p.bs == 0) {
          record_fault(p.fault, KVQ_FAULT_BLOCK);
        }
      }
      ks[t][d] = kx;
      vs[t][d] = vx;
    }
    __syncthreads();
    for (int e = tid; e < kSimtRows * kSimtTok; e += kSimtThreads) {
      const int r = e / kSimtTok, t = e % kSimtTok;
      float a = 0.f;
#pragma unroll 8
      for (int d = 0; d < D; ++d) a = fmaf(qs[r][d], ks[t][d], a);
      sc[r][t] = a;
    }
    __syncthreads();
    for (int r = warp; r < kSimtRows; r += kSimtThreads / 32) {
      const int row = r0 + r;
      uint32_t vis = 0;
      if (row < R) vis = visible32(p.mask + (static_cast<long>(s.q0) + row / p.g) * p.mask_words, t0, s.n, s.L);
      const int pos = t0 + lane;
      bool see = ((vis >> lane) & 1u) && pos < hi;
      if (see) {
        const int blk = p.tables[static_cast<long>(b) * p.max_blocks + pos / p.bs];
        see = blk >= 0 && blk < p.NB;
      }
      float x = see ? sc[r][lane] : -INFINITY, mx = x;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float m0 = row_m[r], m = fmaxf(m0, mx);
      const float e = see ? exp2f(x - (m == -INFINITY ? 0.f : m)) : 0.f;
      float sum = e;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      // -1 marks a masked position: it is left out of P V
      sc[r][lane] = see ? e : -1.f;
      __syncwarp();
      if (lane == 0) {
        const float f = m0 == -INFINITY ? 0.f : exp2f(m0 - m);
        row_m[r] = m;
        row_f[r] = f;
        row_l[r] = row_l[r] * f + sum;
      }
    }
    __syncthreads();
    const float f = row_f[orow];
#pragma unroll
    for (int i = 0; i < DPT; ++i) o[i] *= f;
    for (int t = 0; t < kSimtTok; ++t) {
      const float e = sc[orow][t];
      if (e == -1.f) continue;
#pragma unroll
      for (int i = 0; i < DPT; ++i) o[i] = fmaf(e, vs[t][od + i], o[i]);
    }
  }
  __syncthreads();
  const int r = r0 + orow;
  if (r >= R) return;
  const long row = (static_cast<long>(s.q0) + r / p.g) * p.Hq + static_cast<long>(kvh) * p.g + r % p.g;
  const float m = row_m[orow], l = row_l[orow];
  if (p.splits == 1) {
#pragma unroll
    for (int i = 0; i < DPT; ++i) tree_store(p, row * D + od + i, l != 0.f ? o[i] / l : 0.f);
    return;
  }
  const long part = row * p.splits + split;
#pragma unroll
  for (int i = 0; i < DPT; ++i) p.ws_o[part * D + od + i] = o[i];
  if (od == 0) {
    p.ws_ml[2 * part] = m;
    p.ws_ml[2 * part + 1] = l;
  }
}

// One warp per query row: the log-sum-exp merge of its splits.
__global__ void __launch_bounds__(256) tree_simt_reduce_kernel(TreeParams p) {
  griddep_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);       // (token, head) of the sequence
  const TreeSeq s = tree_seq(p, b);
  if (i >= s.L * p.Hq) return;
  const long row = static_cast<long>(s.q0) * p.Hq + i;
  const int S = (s.n - 1) / p.chunk + 1;
  const float* ml = p.ws_ml + 2 * row * p.splits;
  const float* o = p.ws_o + row * p.splits * p.D;
  float M = -INFINITY;
  for (int k = 0; k < S; ++k) M = fmaxf(M, ml[2 * k]);
  float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < S; ++k) {
    if (ml[2 * k + 1] == 0.f) continue;                    // nothing visible in this split
    const float w = ml[2 * k] == -INFINITY ? 1.f : exp2f(ml[2 * k] - M);
    L = fmaf(ml[2 * k + 1], w, L);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 32 * e < p.D) acc[e] = fmaf(o[static_cast<long>(k) * p.D + lane + 32 * e], w, acc[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < p.D) tree_store(p, row * p.D + lane + 32 * e, L != 0.f ? acc[e] / L : 0.f);
}

template <typename TA>
void launch_simt_dim(const TreeParams& p, dim3 grid, cudaStream_t s) {
  if (p.D == 64) tree_simt_kernel<TA, 64><<<grid, kSimtThreads, 0, s>>>(p);
  else tree_simt_kernel<TA, 128><<<grid, kSimtThreads, 0, s>>>(p);
}

kvq_status plan_tree(const Geometry& g, int batch, int num_q_heads, int max_tree, int max_context, TreePlan* p) {
  if (low_bit(g.cache_dtype)) return KVQ_ERR_UNSUPPORTED;
  if (max_tree > kTreeMax) return KVQ_ERR_UNSUPPORTED;
  max_context = std::min(max_context, kTreeContext);
  const int sms = device_sm_count();
  p->g = num_q_heads / g.H;
  p->kernel = tree_tc_supported(g, p->g) ? 1 : 0;
  p->ws_bytes = p->ws_ml_off = 0;
  p->splits = p->chunk = p->ctas = 0;
  p->group = 1;
  p->lead = 0;
  if (p->kernel == 1) {
    // CTAs in groups of as many as a tree has row tiles, at most kTreeGroup; two partial slots per
    // CTA, each one tile of rows
    const long tiles = (static_cast<long>(max_tree) * p->g + kTreeRows - 1) / kTreeRows;
    p->group = static_cast<int>(std::max(1L, std::min(tiles, static_cast<long>(std::min(kTreeGroup, sms)))));
    p->ctas = sms / p->group * p->group;
    // Starting and ending a unit costs a CTA as much as kTreeLead blocks (q's way to tensor memory, a
    // pipeline that fills and drains, masked blocks, the output).  Shares that count it keep a CTA with
    // many short sequences from ending last: contexts of 1024 to 8192 (64 sequences, 8 kv heads) 260 us
    // with 3, 243 with 6, 238 with 10, 233 with 14.  Not where CTAs have few blocks anyway: the parts
    // would get longer.
    const long blocks = static_cast<long>(batch) * g.H * ((tiles + p->group - 1) / p->group) * ((static_cast<long>(max_context) + kTreeBlk - 1) / kTreeBlk);
    static_assert((kTreeLead + 1L) << 27 < 1L << 31, "the schedule counts in 32 bits");
    if (blocks >= 1L << 27) return KVQ_ERR_UNSUPPORTED;
    if (blocks >= 16L * (p->ctas / p->group)) p->lead = kTreeLead;
    const size_t rows = static_cast<size_t>(2) * sms * kTreeRows;
    p->ws_ml_off = rows * g.D * sizeof(float);
    p->ws_bytes = p->ws_ml_off + rows * 2 * sizeof(float);
    return KVQ_OK;
  }
  // enough splits for about four CTAs per SM, none shorter than 256 positions
  const long tiles = (static_cast<long>(std::max(max_tree, 1)) * p->g + kSimtRows - 1) / kSimtRows;
  const long units = std::max(1L, static_cast<long>(batch) * g.H * tiles);
  long S = (4L * sms + units - 1) / units;
  S = std::max(1L, std::min(S, (static_cast<long>(max_context) + 255) / 256));
  const long chunk = std::max(1L, ((static_cast<long>(max_context) + S - 1) / S + kSimtTok - 1) / kSimtTok) * kSimtTok;
  S = std::max(1L, (static_cast<long>(max_context) + chunk - 1) / chunk);
  p->splits = static_cast<int>(S);
  p->chunk = static_cast<int>(chunk);
  return KVQ_OK;
}

// Partials of the CUDA-core kernel are held per query row; the caller knows num_q_tokens only
// through max_tree, so they are sized for batch * max_tree rows.
size_t simt_rows(int batch, int num_q_heads, int max_tree) {
  return static_cast<size_t>(batch) * max_tree * num_q_heads;
}

void finish_plan(const Geometry& g, int batch, int num_q_heads, int max_tree, TreePlan* p) {
  if (p->kernel == 0 && p->splits > 1) {
    const size_t rows = simt_rows(batch, num_q_heads, max_tree) * p->splits;
    p->ws_ml_off = (rows * g.D * sizeof(float) + 255) / 256 * 256;
    p->ws_bytes = p->ws_ml_off + rows * 2 * sizeof(float);
  }
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

cudaError_t launch_tree_simt(const TreeParams& p, int act, cudaStream_t s) {
  const int tiles = (p.max_tree * p.g + kSimtRows - 1) / kSimtRows;
  const dim3 grid(tiles * p.splits, p.H, p.B);
  if (act == KVQ_DTYPE_BF16) launch_simt_dim<__nv_bfloat16>(p, grid, s);
  else launch_simt_dim<__half>(p, grid, s);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_dependent(tree_simt_reduce_kernel, dim3((p.max_tree * p.Hq + 7) / 8, p.B), dim3(256), 0, s, p);
}

}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_tree_workspace_size(const kvq_cache_desc* c, int batch, int num_q_heads, int max_tree,
                                   int max_context, size_t* bytes) {
  if (c == nullptr || bytes == nullptr) return KVQ_ERR_INVALID_ARG;
  // the pool's pointers are not looked at: any aligned stand-in passes the check
  kvq_cache_desc d = *c;
  d.pages = d.residual = reinterpret_cast<void*>(16);
  d.k_scales = d.v_scales = reinterpret_cast<float*>(16);
  Geometry g;
  kvq_status st = validate_desc(&d, &g);
  if (st != KVQ_OK) return st;
  if (batch < 0 || num_q_heads < 1 || num_q_heads % g.H != 0 || max_tree < 0 || max_context < 0)
    return KVQ_ERR_INVALID_ARG;
  TreePlan p;
  st = plan_tree(g, batch, num_q_heads, max_tree, max_context, &p);
  if (st != KVQ_OK) return st;
  finish_plan(g, batch, num_q_heads, max_tree, &p);
  *bytes = p.ws_bytes;
  return KVQ_OK;
}

kvq_status kvq_tree_attention(const kvq_cache_desc* c, const void* q, int num_q_tokens, int batch,
                              int num_q_heads, const int32_t* q_start, int max_tree,
                              const uint32_t* tree_mask, int mask_words, const int32_t* block_tables,
                              int max_blocks_per_seq, const int32_t* context_lens, int max_context,
                              float softmax_scale, void* out, int32_t out_dtype, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  Geometry g;
  kvq_status st = validate_desc(c, &g);
  if (st != KVQ_OK) return st;
  if (batch < 0 || num_q_tokens < 0 || num_q_heads < 1 || num_q_heads % g.H != 0 || max_tree < 0 ||
      max_context < 0 || max_blocks_per_seq < 1 || mask_words < (max_tree + 31) / 32)
    return KVQ_ERR_INVALID_ARG;
  if (out_dtype != KVQ_DTYPE_BF16 && out_dtype != KVQ_DTYPE_FP16 && out_dtype != KVQ_DTYPE_FP32)
    return KVQ_ERR_INVALID_ARG;
  if (!(softmax_scale >= 0.f) || !std::isfinite(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  TreePlan plan;
  st = plan_tree(g, batch, num_q_heads, max_tree, max_context, &plan);
  if (st != KVQ_OK) return st;
  if (batch > 65535 || g.H > 65535) return KVQ_ERR_UNSUPPORTED;
  if (batch == 0 || num_q_tokens == 0 || max_tree == 0) return KVQ_OK;
  if (q == nullptr || q_start == nullptr || tree_mask == nullptr || block_tables == nullptr ||
      context_lens == nullptr || out == nullptr)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned(q) || !aligned(out)) return KVQ_ERR_INVALID_ARG;
  finish_plan(g, batch, num_q_heads, max_tree, &plan);
  TreeParams p{};
  if (plan.ws_bytes > 0) {
    if (workspace == nullptr || workspace_bytes < plan.ws_bytes || !aligned(workspace)) return KVQ_ERR_INVALID_ARG;
    // the CUDA-core kernel's partials are indexed by query row
    if (plan.kernel == 0 && static_cast<long>(num_q_tokens) > static_cast<long>(batch) * max_tree) return KVQ_ERR_INVALID_ARG;
    p.ws_o = static_cast<float*>(workspace);
    p.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.ws_ml_off);
  }
  p.q = q;
  p.q_start = q_start;
  p.mask = tree_mask;
  p.tables = block_tables;
  p.lens = context_lens;
  p.Tq = num_q_tokens;
  p.B = batch;
  p.H = g.H;
  p.Hq = num_q_heads;
  p.g = plan.g;
  p.D = g.D;
  p.max_tree = max_tree;
  p.mask_words = mask_words;
  p.max_blocks = max_blocks_per_seq;
  p.max_context = std::min(max_context, kTreeContext);
  p.pages = static_cast<const uint8_t*>(c->pages);
  p.k_static = c->k_scales;
  p.v_static = c->v_scales;
  p.NB = g.NB;
  p.bs = g.bs;
  p.record = g.record;
  p.off_v = g.off_v;
  p.off_s = g.off_s;
  p.row_bytes = g.row_bytes;
  p.mode = g.scale_mode;
  p.cache_dtype = g.cache_dtype;
  p.act_fp16 = g.act_dtype == KVQ_DTYPE_FP16;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(g.D));
  p.scale_log2 = scale * kLog2e;
  p.out = out;
  p.out_dtype = out_dtype;
  p.splits = plan.splits;
  p.chunk = plan.chunk;
  p.ctas = plan.ctas;
  p.group = plan.group;
  p.lead = plan.lead;
  p.shares = plan.kernel == 1 ? plan.ctas / plan.group : 1;
  p.share_unit = static_cast<unsigned>(std::min((1LL << 32) / p.shares, 0xFFFFFFFFLL));
  p.fault = c->fault;
  const cudaError_t e = plan.kernel == 1 ? launch_tree_tc(p, g, stream) : launch_tree_simt(p, g.act_dtype, stream);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
