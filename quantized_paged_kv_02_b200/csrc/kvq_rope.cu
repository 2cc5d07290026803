// Rotary position embedding, alone (kvq_rope) and fused with quantize-on-write of K and V
// (kvq_rope_write).
//
// Pair p of a head at position t turns by the angle t * f_p:
//   (a, b) -> (a cos - b sin, b cos + a sin) * m,   m the attention factor of the scaling,
// with (a, b) = (x[p], x[p + rot/2]) in the half layout and (x[2p], x[2p+1]) in the
// interleaved one; dimensions from rot on pass through.  The angle is formed in turns, in
// binary64 (t * f_p / 2 pi, less its nearest integer), because in binary32 a position of 2^16
// already leaves no more than 8 bits below one radian, with the products' low parts, since at 2^31
// binary64 alone leaves no more than 24 (3e-7 rad).  Cosine and sine are rounded to binary32 once.
//
// What bounds it: bytes (16-bit rows in, 16-bit rows and codes out; 3 flops per element), so
// the work per element is kept below the copy's.  A CTA takes up to four tokens, whose cosines
// and sines (at most 64 pairs each) are computed once, one per thread, into shared memory, while
// the first rows are on their way; every head then shares them.  D / 16 lanes hold one row, lane
// i the 16-byte chunks i and i + D/16 (in the half layout with a partly rotated head, i and
// i + rot/16), so both elements of a pair are always in one lane, each load of a lane group is
// contiguous, and the rotation may run in place.  The rows of a CTA's tokens form one list, 32 (64
// for head_dim 64) at a time, the loads of the next two turns in flight.  The quantizers are kvq_write's, fed
// with the rotated binary32 values (no rounding to 16 bits in between).
//
// Measured (B200): 16411 tokens of 32 / 8 bf16 heads, 64 of 128 dimensions interleaved, 61 us, 5.5 TB/s
// (one token per CTA 76 us: every CTA waited for its own sines); 24 tokens 6 us, a launch and one chain of
// loads; 32768 tokens of 64 / 8 heads with quantize-on-write to INT8 231 us, 5.5 TB/s of the bytes it
// cannot do without.
#include <algorithm>
#include <climits>
#include <cmath>

#include "kvq_checks.cuh"
#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"

namespace kvq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;       // tokens per CTA at most
constexpr int kNoCache = -1;         // CD of kvq_rope: K rows go to k_out

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_out;
  long q_stride, k_stride, v_stride, qo_stride, ko_stride;   // elements between tokens
  int Hq, H;
  const int32_t* pos;
  const double* freqs;       // [rot/2] radians per position
  double mscale;
  int rot;
  const int32_t* slots;
  uint8_t* pages;
  const float* k_static;
  const float* v_static;
  int NB, bs, record, off_v, off_s, mode;
  int32_t* fault;
};

template <typename TA>
__device__ __forceinline__ uint4 pack8(const float* x) {
  if constexpr (std::is_same<TA, __nv_bfloat16>::value)
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  else
    return make_uint4(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]), pack_f16x2(x[4], x[5]),
                      pack_f16x2(x[6], x[7]));
}

// Codes of one 8-element chunk of a row (chunk c of kv head h), stored into its record.
template <int CD, int D>
__device__ __forceinline__ void store_codes(uint8_t* row, int c, const float* x, float s, bool per_token,
                                            const float* chan) {
  uint2 w;
  if (chan == nullptr && s != 0.f) {
    w = quant8_same_scale<CD>(x, s, __frcp_rn(s), per_token);
  } else {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float cs = chan != nullptr ? chan[8 * c + i] : s;
      e[i] = CD == KVQ_DTYPE_INT8 ? quant_int8(x[i], cs) : quant_fp8(x[i], cs);
    }
    w = make_uint2(pack4_low_bytes(e[0], e[1], e[2], e[3]), pack4_low_bytes(e[4], e[5], e[6], e[7]));
  }
  *reinterpret_cast<uint2*>(row + 8 * c) = w;
}

// grid (ceil(T / tokens), slices): tokens blockIdx.x * tokens ..; slice y takes every gridDim.y-th
// group of kRopeThreads / LPR entries of their row list.  Rows of a token: Hq of q, H of k, and
// with a cache H of v.
template <typename TA, int CD, int D, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(RopeParams p, int T, int tokens) {
  constexpr int LPR = D / 16;                 // lanes per row, two 16-byte chunks each
  constexpr int RPB = kRopeThreads / LPR;     // rows per turn of the CTA
  constexpr bool CACHE = CD != kNoCache;
  constexpr bool CODES = CD == KVQ_DTYPE_INT8 || CD == KVQ_DTYPE_FP8_E4M3;
  constexpr int AHEAD = 2;                    // turns whose loads are in flight
  __shared__ __align__(16) float cosv[kRopeTokens][D / 2];
  __shared__ __align__(16) float sinv[kRopeTokens][D / 2];
  __shared__ int blk_of[kRopeTokens], off_of[kRopeTokens];   // (a cache) block, or -1: nothing stored
  const int t0 = blockIdx.x * tokens, nt = min(tokens, T - t0), l = threadIdx.x % LPR;
  const int rows = p.Hq + (CACHE ? 2 : 1) * p.H, total = nt * rows;
  const int pairs = p.rot / 2;

  int c0, c1, p0, p1;                         // the lane's chunks, and their first pairs
  bool turns0, turns1;                        // whether each chunk is rotated
  if constexpr (HALF) {
    const int r8 = p.rot / 16;
    turns0 = turns1 = l < r8;
    c0 = turns0 ? l : 2 * l;
    c1 = turns0 ? l + r8 : 2 * l + 1;
    p0 = 8 * l;
    p1 = p0 + 4;
  } else {
    c0 = l;
    c1 = l + LPR;
    turns0 = 8 * c0 < p.rot;
    turns1 = 8 * c1 < p.rot;
    p0 = 4 * c0;
    p1 = 4 * c1;
  }

  // entry `at` of the list: token t0 + tk, row r of it
  const int step = gridDim.y * RPB, start = blockIdx.y * RPB;
  auto advance = [&](int& tk, int& r) {
    r += step;
    while (r >= rows && tk < nt) { r -= rows; ++tk; }
  };
  auto source = [&](int tk, int r) -> const uint4* {
    const long t = t0 + tk;
    const void* base;
    long at;
    if (r < p.Hq) { base = p.q; at = t * p.q_stride + static_cast<long>(r) * D; }
    else if (r < p.Hq + p.H) { base = p.k; at = t * p.k_stride + static_cast<long>(r - p.Hq) * D; }
    else { base = p.v; at = t * p.v_stride + static_cast<long>(r - p.Hq - p.H) * D; }
    return reinterpret_cast<const uint4*>(static_cast<const TA*>(base) + at);
  };
  int tk = 0, r = start + threadIdx.x / LPR;
  while (r >= rows && tk < nt) { r -= rows; ++tk; }
  int ltk = tk, lr = r;                       // what is loaded next
  uint4 u[AHEAD][2];
#pragma unroll
  for (int a = 0; a < AHEAD; ++a) {
    u[a][0] = u[a][1] = make_uint4(0, 0, 0, 0);
    if (ltk < nt) {
      const uint4* src = source(ltk, lr);
      u[a][0] = src[c0];
      u[a][1] = src[c1];
    }
    advance(ltk, lr);
  }
  if constexpr (CACHE) {
    if (threadIdx.x < nt) {
      const int slot = p.slots[t0 + threadIdx.x];
      const bool in = slot >= 0 && slot < static_cast<long>(p.NB) * p.bs;
      if (!in && slot != -1 && blockIdx.y == 0) record_fault(p.fault, KVQ_FAULT_SLOT);
      blk_of[threadIdx.x] = in ? slot / p.bs : -1;
      off_of[threadIdx.x] = in ? slot % p.bs : 0;
    }
  }
  for (int i = threadIdx.x; i < nt * pairs; i += kRopeThreads) {
    // 1 / 2 pi as the sum of two binary64: what turns are left above whole ones is the remainder of
    // product with the first (one FMA, exact to its last bit) plus the small parts
    constexpr double kInvTwoPi = 0x1.45f306dc9c883p-3, kInvTwoPiLow = -0x1.6b01ec5417056p-57;
    const int k = i / pairs, f = i - k * pairs;
    const double t = p.pos[t0 + k], w = p.freqs[f], angle = t * w, low = fma(t, w, -angle);
    const double whole = rint(angle * kInvTwoPi);
    const double turn = fma(angle, kInvTwoPi, -whole) + fma(angle, kInvTwoPiLow, low * kInvTwoPi);
    double sn, cs;
    sincospi(2.0 * turn, &sn, &cs);
    cosv[k][f] = static_cast<float>(cs * p.mscale);
    sinv[k][f] = static_cast<float>(sn * p.mscale);
  }
  __syncthreads();

  // one entry; then the load of the entry two turns on into the registers it leaves
  auto entry = [&](uint4 (&u)[2]) {
    const uint4 w0 = u[0], w1 = u[1];
    if (ltk < nt) {
      const uint4* src = source(ltk, lr);
      u[0] = src[c0];
      u[1] = src[c1];
    }
    advance(ltk, lr);
    const bool have = tk < nt, is_q = r < p.Hq, is_v = r >= p.Hq + p.H;
    const int k = have ? tk : 0;
    float x[16];
    unpack8<TA>(w0, x);
    unpack8<TA>(w1, x + 8);
    if (!is_v) {
      if constexpr (HALF) {
        if (turns0) {
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 c4 = *reinterpret_cast<const float4*>(&cosv[k][p0 + i]), s4 = *reinterpret_cast<const float4*>(&sinv[k][p0 + i]);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float2 a = make_float2(x[i + e], x[i + e + 1]), b = make_float2(x[i + e + 8], x[i + e + 9]);
              const float2 c = e ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
              const float2 s = e ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y);
              const float2 y = __ffma2_rn(a, c, __fmul2_rn(b, make_float2(-s.x, -s.y))), z = __ffma2_rn(b, c, __fmul2_rn(a, s));
              x[i + e] = y.x;
              x[i + e + 1] = y.y;
              x[i + e + 8] = z.x;
              x[i + e + 9] = z.y;
            }
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 0 ? turns0 : turns1) {
            const int at = h == 0 ? p0 : p1;
            const float4 c4 = *reinterpret_cast<const float4*>(&cosv[k][at]), s4 = *reinterpret_cast<const float4*>(&sinv[k][at]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[8 * h + 2 * i], b = x[8 * h + 2 * i + 1], c = (&c4.x)[i], s = (&s4.x)[i];
              x[8 * h + 2 * i] = fmaf(a, c, -b * s);
              x[8 * h + 2 * i + 1] = fmaf(b, c, a * s);
            }
          }
        }
      }
    }
    if ((is_q || !CACHE) && have) {
      const long t = t0 + tk;
      uint4* dst = is_q ? reinterpret_cast<uint4*>(static_cast<TA*>(p.q_out) + t * p.qo_stride + static_cast<long>(r) * D)
                        : reinterpret_cast<uint4*>(static_cast<TA*>(p.k_out) + t * p.ko_stride + static_cast<long>(r - p.Hq) * D);
      dst[c0] = turns0 ? pack8<TA>(x) : w0;
      dst[c1] = turns1 ? pack8<TA>(x + 8) : w1;
    }
    if constexpr (CACHE) if (__any_sync(0xffffffffu, have && !is_q)) {   // (most warps hold q rows only)
      const int blk = blk_of[k], off = off_of[k];
      const int h = r - p.Hq - (is_v ? p.H : 0);
      const bool keep = have && !is_q && blk >= 0;
      uint8_t* rec = p.pages + (static_cast<long>(blk) * p.H + h) * p.record;
      if constexpr (CODES) {
        // (a warp may hold q rows too: they take part in the maximum only)
        const bool per_token = p.mode == KVQ_SCALE_PER_TOKEN_HEAD;
        float s = 0.f;
        if (per_token) {
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          s = div_rn(m, QMax<CD>::v);
        }
        if (keep) {
          const float* st = is_v ? p.v_static : p.k_static;
          const float* chan = nullptr;
          if (p.mode == KVQ_SCALE_PER_HEAD) s = st[h];
          if (p.mode == KVQ_SCALE_PER_TENSOR) s = st[0];
          if (p.mode == KVQ_SCALE_PER_CHANNEL) chan = st + static_cast<long>(h) * D;
          if (per_token && l == 0) reinterpret_cast<float*>(rec + p.off_s)[(is_v ? p.bs : 0) + off] = s;
          uint8_t* row = rec + (is_v ? p.off_v : 0) + off * D;
          store_codes<CD, D>(row, c0, x, s, per_token, chan);
          store_codes<CD, D>(row, c1, x + 8, s, per_token, chan);
        }
      } else if (keep) {
        uint4* row = reinterpret_cast<uint4*>(rec + (is_v ? p.off_v : 0) + off * 2 * D);
        row[c0] = !is_v && turns0 ? pack8<TA>(x) : w0;
        row[c1] = !is_v && turns1 ? pack8<TA>(x + 8) : w1;
      }
    }
    advance(tk, r);
  };
  // the trip count is the same for every thread of the CTA (the shuffles need whole warps): entries
  // past the end of the list stand in with zeros and store nothing
  for (int base = start; base < total; base += 2 * step) {
    entry(u[0]);
    if (base + step < total) entry(u[1]);
  }
}

template <typename TA, int CD, int D>
cudaError_t launch_layout(const RopeParams& p, bool half, int T, cudaStream_t s) {
  const int rpb = kRopeThreads / (D / 16);
  const int rows = p.Hq + (CD == kNoCache ? 1 : 2) * p.H;
  // one token per CTA until every SM has three CTAs, then up to four; with fewer tokens than that
  // a token's rows go to CTAs of their own
  const int sms = device_sm_count(), passes = (rows + rpb - 1) / rpb;
  const int tokens = std::max(1, std::min(kRopeTokens, T / (3 * sms)));
  const int ctas = (T + tokens - 1) / tokens;
  const int slices = std::max(1, std::min(passes, 2 * sms / std::max(ctas, 1)));
  const dim3 grid(ctas, slices);
  if (half) rope_kernel<TA, CD, D, true><<<grid, kRopeThreads, 0, s>>>(p, T, tokens);
  else rope_kernel<TA, CD, D, false><<<grid, kRopeThreads, 0, s>>>(p, T, tokens);
  return cudaGetLastError();
}

template <typename TA, int CD>
cudaError_t launch_dim(const RopeParams& p, int D, bool half, int T, cudaStream_t s) {
  return D == 64 ? launch_layout<TA, CD, 64>(p, half, T, s) : launch_layout<TA, CD, 128>(p, half, T, s);
}

template <typename TA>
cudaError_t launch_rope(const RopeParams& p, int cd, int D, bool half, int T, cudaStream_t s) {
  switch (cd) {
    case KVQ_DTYPE_INT8: return launch_dim<TA, KVQ_DTYPE_INT8>(p, D, half, T, s);
    case KVQ_DTYPE_FP8_E4M3: return launch_dim<TA, KVQ_DTYPE_FP8_E4M3>(p, D, half, T, s);
    case kNoCache: return launch_dim<TA, kNoCache>(p, D, half, T, s);
    default: return launch_dim<TA, KVQ_DTYPE_BF16>(p, D, half, T, s);   // rows stored as they are
  }
}

bool finite_positive(double x) { return std::isfinite(x) && x > 0.0; }

// Checks a rope descriptor; *mscale the factor of cosine and sine.
kvq_status check_rope(const kvq_rope_desc* r, int head_dim, double* mscale) {
  if (r == nullptr) return KVQ_ERR_INVALID_ARG;
  if (r->layout != KVQ_ROPE_HALF && r->layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim % 2 != 0 || r->rot_dim > head_dim) return KVQ_ERR_INVALID_ARG;
  if (!finite_positive(r->theta) || !std::isfinite(r->attention_factor) || r->attention_factor < 0.0)
    return KVQ_ERR_INVALID_ARG;
  double m = 1.0;
  switch (r->scaling) {
    case KVQ_ROPE_SCALE_NONE: break;
    case KVQ_ROPE_SCALE_LINEAR:
    case KVQ_ROPE_SCALE_NTK:
      if (!finite_positive(r->factor)) return KVQ_ERR_INVALID_ARG;
      if (r->scaling == KVQ_ROPE_SCALE_NTK && r->rot_dim < 4) return KVQ_ERR_INVALID_ARG;
      break;
    case KVQ_ROPE_SCALE_WAVELENGTH:
    case KVQ_ROPE_SCALE_YARN:
      if (!finite_positive(r->factor) || r->original_context < 1 || !finite_positive(r->low) ||
          !finite_positive(r->high) || r->low >= r->high)
        return KVQ_ERR_INVALID_ARG;
      if (r->scaling == KVQ_ROPE_SCALE_YARN) {
        if (r->theta == 1.0) return KVQ_ERR_INVALID_ARG;
        if (r->factor > 1.0) m = 0.1 * std::log(r->factor) + 1.0;
      }
      break;
    default: return KVQ_ERR_INVALID_ARG;
  }
  if (r->attention_factor > 0.0) m = r->attention_factor;
  if (mscale) *mscale = m;
  return KVQ_OK;
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// One [T][heads][D] tensor with a token stride: present, aligned, rows not overlapping.
bool rows_ok(const void* p, int64_t stride, int heads, int D) {
  return p != nullptr && aligned(p) && stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * D;
}

// T rows of `wide` elements each, `stride` elements apart.
struct Rows {
  const void* at;
  int64_t stride, wide;
};

// Do two tensors of T such rows (16-bit elements) overlap?  Columns of one buffer, which have one stride, lie
// between one another; tensors of different strides within one range count as overlapping.
bool rows_overlap(const Rows& a, const Rows& b, int T) {
  if (!bytes_overlap(a.at, 2 * ((T - 1) * a.stride + a.wide), b.at, 2 * ((T - 1) * b.stride + b.wide))) return false;
  if (a.stride != b.stride || T == 1) return true;
  const int64_t s = 2 * a.stride;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at)) % s;
  const int64_t from = d < 0 ? d + s : d;                    // b's rows begin here in a's period
  return from < 2 * a.wide || from + 2 * b.wide > s;
}

// May `out` be written while `in` is read?  As its own input (same rows) or apart from it.
bool in_place(const Rows& out, const Rows& in, int T) {
  return (out.at == in.at && out.stride == in.stride) || !rows_overlap(out, in, T);
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_rope_frequencies(const kvq_rope_desc* r, double* freqs, double* attention_factor) {
  constexpr double kPi = 3.14159265358979323846;
  double m = 1.0;
  const kvq_status st = check_rope(r, INT_MAX, &m);
  if (st != KVQ_OK) return st;
  if (freqs != nullptr) {
    const double rot = r->rot_dim;
    double theta = r->theta;
    if (r->scaling == KVQ_ROPE_SCALE_NTK) theta *= std::pow(r->factor, rot / (rot - 2.0));
    // YaRN: the pair that makes `turns` turns within the original context
    auto pair_of = [&](double turns) {
      return rot * std::log(r->original_context / (turns * 2.0 * kPi)) / (2.0 * std::log(r->theta));
    };
    double lo = 0.0, hi = 0.0;
    if (r->scaling == KVQ_ROPE_SCALE_YARN) {
      lo = std::max(std::floor(pair_of(r->high)), 0.0);
      hi = std::min(std::ceil(pair_of(r->low)), rot - 1.0);
    }
    for (int i = 0; i < r->rot_dim / 2; ++i) {
      const double f = std::pow(theta, -2.0 * i / rot);
      double keep = 1.0;                         // share of the unscaled frequency
      if (r->scaling == KVQ_ROPE_SCALE_LINEAR) keep = 0.0;
      if (r->scaling == KVQ_ROPE_SCALE_WAVELENGTH) {
        const double turns = r->original_context * f / (2.0 * kPi);
        keep = std::min(std::max((turns - r->low) / (r->high - r->low), 0.0), 1.0);
      }
      if (r->scaling == KVQ_ROPE_SCALE_YARN)
        keep = 1.0 - std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      freqs[i] = keep == 1.0 ? f : (1.0 - keep) * f / r->factor + keep * f;
    }
  }
  if (attention_factor != nullptr) *attention_factor = m;
  return KVQ_OK;
}

kvq_status kvq_rope(const kvq_rope_desc* r, const double* freqs, int32_t act_dtype, int head_dim,
                    const int32_t* positions, int num_tokens, const void* q, int64_t q_stride,
                    int num_q_heads, void* q_out, int64_t q_out_stride, const void* k,
                    int64_t k_stride, int num_kv_heads, void* k_out, int64_t k_out_stride,
                    cudaStream_t stream) {
  if (act_dtype != KVQ_DTYPE_BF16 && act_dtype != KVQ_DTYPE_FP16) return KVQ_ERR_INVALID_ARG;
  if (head_dim < 1 || num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0) return KVQ_ERR_INVALID_ARG;
  RopeParams p{};
  const kvq_status st = check_rope(r, head_dim, &p.mscale);
  if (st != KVQ_OK) return st;
  if ((head_dim != 64 && head_dim != 128) || r->rot_dim % 16 != 0) return KVQ_ERR_UNSUPPORTED;
  if (num_tokens == 0 || num_q_heads + num_kv_heads == 0) return KVQ_OK;
  if (freqs == nullptr || positions == nullptr) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (!rows_ok(q, q_stride, num_q_heads, head_dim) || !rows_ok(q_out, q_out_stride, num_q_heads, head_dim)))
    return KVQ_ERR_INVALID_ARG;
  if (num_kv_heads > 0 && (!rows_ok(k, k_stride, num_kv_heads, head_dim) || !rows_ok(k_out, k_out_stride, num_kv_heads, head_dim)))
    return KVQ_ERR_INVALID_ARG;
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim, kw = static_cast<int64_t>(num_kv_heads) * head_dim;
  const Rows rq{q, q_stride, qw}, rqo{q_out, q_out_stride, qw}, rk{k, k_stride, kw}, rko{k_out, k_out_stride, kw};
  if (num_q_heads > 0 && !in_place(rqo, rq, num_tokens)) return KVQ_ERR_INVALID_ARG;
  if (num_kv_heads > 0 && !in_place(rko, rk, num_tokens)) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads > 0 && num_kv_heads > 0 &&
      (rows_overlap(rqo, rk, num_tokens) || rows_overlap(rko, rq, num_tokens) || rows_overlap(rqo, rko, num_tokens)))
    return KVQ_ERR_INVALID_ARG;
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.qo_stride = q_out_stride;
  p.ko_stride = k_out_stride;
  p.Hq = num_q_heads;
  p.H = num_kv_heads;
  p.pos = positions;
  p.freqs = freqs;
  p.rot = r->rot_dim;
  const bool half = r->layout == KVQ_ROPE_HALF;
  const cudaError_t e = act_dtype == KVQ_DTYPE_BF16
                            ? launch_rope<__nv_bfloat16>(p, kNoCache, head_dim, half, num_tokens, stream)
                            : launch_rope<__half>(p, kNoCache, head_dim, half, num_tokens, stream);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_rope_write(const kvq_cache_desc* c, const kvq_rope_desc* r, const double* freqs,
                          const int32_t* positions, int num_tokens, const void* q, int64_t q_stride,
                          int num_q_heads, void* q_out, int64_t q_out_stride, const void* k_new,
                          int64_t k_stride, const void* v_new, int64_t v_stride,
                          const int32_t* slot_mapping, cudaStream_t stream) {
  Geometry g;
  kvq_status st = validate_desc(c, &g);
  if (st != KVQ_OK) return st;
  if (num_tokens < 0 || num_q_heads < 0) return KVQ_ERR_INVALID_ARG;
  RopeParams p{};
  st = check_rope(r, g.D, &p.mscale);
  if (st != KVQ_OK) return st;
  if (low_bit(g.cache_dtype) || r->rot_dim % 16 != 0) return KVQ_ERR_UNSUPPORTED;
  if (num_tokens == 0) return KVQ_OK;
  if (freqs == nullptr || positions == nullptr || slot_mapping == nullptr) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (!rows_ok(q, q_stride, num_q_heads, g.D) || !rows_ok(q_out, q_out_stride, num_q_heads, g.D)))
    return KVQ_ERR_INVALID_ARG;
  if (!rows_ok(k_new, k_stride, g.H, g.D) || !rows_ok(v_new, v_stride, g.H, g.D)) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads > 0) {
    const int64_t qw = static_cast<int64_t>(num_q_heads) * g.D, kw = static_cast<int64_t>(g.H) * g.D;
    const Rows out{q_out, q_out_stride, qw};
    if (!in_place(out, {q, q_stride, qw}, num_tokens) || rows_overlap(out, {k_new, k_stride, kw}, num_tokens) ||
        rows_overlap(out, {v_new, v_stride, kw}, num_tokens))
      return KVQ_ERR_INVALID_ARG;
  }
  p.q = q;
  p.k = k_new;
  p.v = v_new;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.qo_stride = q_out_stride;
  p.Hq = num_q_heads;
  p.H = g.H;
  p.pos = positions;
  p.freqs = freqs;
  p.rot = r->rot_dim;
  p.slots = slot_mapping;
  p.pages = static_cast<uint8_t*>(c->pages);
  p.k_static = c->k_scales;
  p.v_static = c->v_scales;
  p.NB = g.NB;
  p.bs = g.bs;
  p.record = g.record;
  p.off_v = g.off_v;
  p.off_s = g.off_s;
  p.mode = g.scale_mode;
  p.fault = c->fault;
  const bool half = r->layout == KVQ_ROPE_HALF;
  const cudaError_t e = g.act_dtype == KVQ_DTYPE_BF16
                            ? launch_rope<__nv_bfloat16>(p, g.cache_dtype, g.D, half, num_tokens, stream)
                            : launch_rope<__half>(p, g.cache_dtype, g.D, half, num_tokens, stream);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
