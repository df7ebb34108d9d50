// kvpool_rope.cu -- per-head norms of queries and keys with the position
// rotation in the same pass: what a model does to the rows that it hands to
// append and decode_attend.
//
// For one head x of a token at position p:
//   y = x / sqrt(mean(x^2) + eps) * w
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
// over the pairs (a, b) of the first rot_dim dims, t = p * freq_i.
//
// The table holds freq_i / (2 pi) as a 64-bit fraction of a turn, so p *
// table[i] modulo 2^64 is the angle's place in its turn: the integer product
// loses nothing at any position (p * freq_i in fp32 is off by 0.06 rad at p =
// 2^20), and three integer multiplies replace a 64-bit float product and its
// range reduction.  Its top 32 bits as a signed number, times 2^-31, are the
// angle in units of pi in [-1, 1): off by 2^-25 turns at most.
//
// Bound: HBM (one read and one write of every value).  A warp takes one token
// and a run of its heads: the lanes work out the token's rot_dim / 2 sines and
// cosines once (two per lane at 128 dims), pass them through shared memory,
// and then stream heads, 8 values (16 bytes of bf16) per lane and four loads
// ahead.  Norms are held in fp32; one rounding at the store.
#include <cmath>

#include <cuda_runtime.h>

#include "device_util.cuh"
#include "kvpool_internal.h"

namespace kvp {
namespace {

constexpr int kRopeWarps = 4;    // warps per CTA
constexpr int kRopeAhead = 4;    // heads per lane group in flight
constexpr int kRopeMaxDim = 256;

struct RopeTensor {
  const uint8_t* in;
  uint8_t* out;
  const float* w;
  int64_t in_tok, in_head, out_tok, out_head;  // strides in bytes
  int32_t heads, steps;                        // steps: warp steps over the heads of one token
};

struct RopeParams {
  RopeTensor t[2];  // queries, keys
  const int64_t* pos;
  const uint64_t* table;
  int64_t n_tokens;
  int32_t head_dim, rot_dim, lanes, group;  // lanes with values per head, lanes per head (a power of two)
  int32_t interleaved, runs, run_steps;     // runs: warps per token, steps of each
  float eps, inv_dim;
};

// 8 values from memory in fp32
template <int T>
struct Vec8;
template <>
struct Vec8<KVPOOL_BF16> {
  uint4 r;
  __device__ __forceinline__ void load(const uint8_t* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void put(uint8_t* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<KVPOOL_F32> {
  float4 a, b;
  __device__ __forceinline__ void load(const uint8_t* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void put(uint8_t* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

template <int T, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const __grid_constant__ RopeParams P) {
  pdl_start();
  __shared__ float2 turn[kRopeWarps][kRopeMaxDim / 2];  // (cos, sin) of the warp's token
  constexpr int kValBytes = T == KVPOOL_BF16 ? 2 : 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t task = (int64_t)blockIdx.x * kRopeWarps + warp;
  const int64_t tok = task / P.runs;
  if (tok >= P.n_tokens) return;
  const int s0 = (int)(task - tok * P.runs) * P.run_steps;
  const int s1 = min(s0 + P.run_steps, P.t[0].steps + P.t[1].steps);
  const int sub = lane / P.group, l = lane % P.group;  // head within a step, lane within the head
  const int per_step = 32 / P.group;
  const bool on = l < P.lanes;

  const int half = P.rot_dim / 2;
  if (half > 0) {
    const uint64_t p = (uint64_t)P.pos[tok];
    for (int i = lane; i < half; i += 32) {
      const int32_t t = (int32_t)((p * P.table[i]) >> 32);
      float s, c;
      sincospif((float)t * 0x1p-31f, &s, &c);
      turn[warp][i] = make_float2(c, s);
    }
    __syncwarp();
  }
  // this lane's angles: of its 8 values (pairs half a rotation apart) or of its 4 pairs
  const bool rot = on && 8 * l < P.rot_dim;
  constexpr int kAng = INTER ? 4 : 8;
  float2 cs[kAng];
  const bool low = 8 * l < half;  // pairs half a rotation apart: the first of its pairs?
#pragma unroll
  for (int j = 0; j < kAng; ++j)
    cs[j] = rot ? turn[warp][INTER ? 4 * l + j : (low ? 8 * l : 8 * l - half) + j] : make_float2(1.0f, 0.0f);
  const int partner = (lane - l) + (rot ? (low ? l + half / 8 : l - half / 8) : l);

  float w[8];
  int have = -1;  // tensor whose weights w holds
  for (int s = s0; s < s1; s += kRopeAhead) {
    Vec8<T> v[kRopeAhead];
#pragma unroll
    for (int u = 0; u < kRopeAhead; ++u) {
      const int st = s + u;
      if (st < s1) {
        const int which = st >= P.t[0].steps;
        const RopeTensor& X = P.t[which];
        const int h = (st - (which ? P.t[0].steps : 0)) * per_step + sub;
        if (on && h < X.heads) v[u].load(X.in + tok * X.in_tok + h * X.in_head + l * 8 * kValBytes);
      }
    }
#pragma unroll
    for (int u = 0; u < kRopeAhead; ++u) {
      const int st = s + u;
      if (st >= s1) break;
      const int which = st >= P.t[0].steps;
      const RopeTensor& X = P.t[which];
      if (have != which) {
        have = which;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = X.w && on ? X.w[8 * l + j] : 1.0f;
      }
      const int h = (st - (which ? P.t[0].steps : 0)) * per_step + sub;
      const bool mine = on && h < X.heads;
      float x[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
      if (mine) v[u].get(x);
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
      for (int o = P.group / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(fmaf(ss, P.inv_dim, P.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
      if constexpr (INTER) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[2 * j] = fmaf(x[2 * j], cs[j].x, -x[2 * j + 1] * cs[j].y);
          y[2 * j + 1] = fmaf(x[2 * j + 1], cs[j].x, x[2 * j] * cs[j].y);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float z = __shfl_sync(0xffffffffu, x[j], partner);
          y[j] = fmaf(x[j], cs[j].x, low ? -z * cs[j].y : z * cs[j].y);
        }
      }
      if (mine) Vec8<T>::put(X.out + tok * X.out_tok + h * X.out_head + l * 8 * kValBytes, y);
    }
  }
}

bool heads_ok(const kvpool_heads* h, int32_t dtype) {
  const int64_t unit = dtype == KVPOOL_BF16 ? 8 : 4;  // values in 16 bytes
  return reinterpret_cast<uintptr_t>(h->data) % 16 == 0 && h->token_stride % unit == 0 && h->head_stride % unit == 0;
}

}  // namespace
}  // namespace kvp

extern "C" int kvpool_rope_table(int32_t rot_dim, const double* h_inv_freq, uint64_t* h_table) {
  using namespace kvp;
  if (rot_dim < 0 || rot_dim > kRopeMaxDim || rot_dim % 16 != 0) return KVPOOL_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!h_inv_freq || !h_table)) return KVPOOL_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!std::isfinite(h_inv_freq[i])) return KVPOOL_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double turns = h_inv_freq[i] / 6.283185307179586476925286766559;
    const double f = turns - std::floor(turns);  // [0, 1]: 1 where a tiny negative one rounds up
    h_table[i] = f >= 1.0 ? 0u : (uint64_t)std::ldexp(f, 64);
  }
  return KVPOOL_OK;
}

extern "C" int kvpool_qk_norm_rope(int32_t dtype, int32_t head_dim, int64_t n_tokens, const kvpool_heads* q,
                                   const kvpool_heads* k, const kvpool_heads* q_out, const kvpool_heads* k_out,
                                   const float* d_q_weight, const float* d_k_weight, float eps, int32_t rot_dim,
                                   int32_t interleaved, const uint64_t* d_table, const int64_t* d_positions,
                                   void* stream) {
  using namespace kvp;
  if (dtype != KVPOOL_F32 && dtype != KVPOOL_BF16) return KVPOOL_ERR_INVALID_ARG;
  if (head_dim < 8 || head_dim > kRopeMaxDim || head_dim % 8 != 0) return KVPOOL_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0 || (interleaved != 0 && interleaved != 1))
    return KVPOOL_ERR_INVALID_ARG;
  if (n_tokens < 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return KVPOOL_ERR_INVALID_ARG;
  const kvpool_heads* in[2] = {q, k};
  const kvpool_heads* out[2] = {q_out, k_out};
  const float* wt[2] = {d_q_weight, d_k_weight};
  RopeParams P{};
  int group = 1;
  while (group * 8 < head_dim) group *= 2;
  const int per_step = 32 / group;
  const int64_t vb = dtype == KVPOOL_BF16 ? 2 : 4;
  for (int i = 0; i < 2; ++i) {
    if (!in[i] || in[i]->heads == 0) continue;  // no such heads
    if (in[i]->heads < 0 || in[i]->heads > 65536 || !out[i] || out[i]->heads != in[i]->heads)
      return KVPOOL_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!in[i]->data || !out[i]->data)) return KVPOOL_ERR_INVALID_ARG;
    if (!heads_ok(in[i], dtype) || !heads_ok(out[i], dtype)) return KVPOOL_ERR_INVALID_ARG;
    RopeTensor& X = P.t[i];
    X.in = static_cast<const uint8_t*>(in[i]->data);
    X.out = static_cast<uint8_t*>(const_cast<void*>(out[i]->data));
    X.w = wt[i];
    X.in_tok = in[i]->token_stride * vb;
    X.in_head = in[i]->head_stride * vb;
    X.out_tok = out[i]->token_stride * vb;
    X.out_head = out[i]->head_stride * vb;
    X.heads = in[i]->heads;
    X.steps = (X.heads + per_step - 1) / per_step;
  }
  const int steps = P.t[0].steps + P.t[1].steps;
  if (n_tokens == 0 || steps == 0) return KVPOOL_OK;
  if (rot_dim > 0 && (!d_table || !d_positions)) return KVPOOL_ERR_INVALID_ARG;
  P.pos = d_positions;
  P.table = d_table;
  P.n_tokens = n_tokens;
  P.head_dim = head_dim;
  P.rot_dim = rot_dim;
  P.lanes = head_dim / 8;
  P.group = group;
  P.interleaved = interleaved;
  P.eps = eps;
  P.inv_dim = 1.0f / (float)head_dim;
  // warps per token: one takes all its heads (its angles are worked out once)
  // unless there are too few tokens to fill the GPU
  constexpr int64_t kFill = 152 * 32;  // warps that keep every SM's loads in flight
  P.run_steps = kRopeAhead;
  while (P.run_steps < steps && n_tokens * ((steps + 2 * P.run_steps - 1) / (2 * P.run_steps)) >= kFill) P.run_steps *= 2;
  while (P.run_steps > 1 && n_tokens * ((steps + P.run_steps - 1) / P.run_steps) < kFill) P.run_steps /= 2;
  P.runs = (steps + P.run_steps - 1) / P.run_steps;
  const int64_t ctas = (n_tokens * P.runs + kRopeWarps - 1) / kRopeWarps;
  if (ctas > 0x7FFFFFFF) return KVPOOL_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)ctas), block(kRopeWarps * 32);
  cudaError_t e;
  if (dtype == KVPOOL_BF16)
    e = interleaved ? launch_kernel(true, rope_kernel<KVPOOL_BF16, true>, grid, block, 0, s, P)
                    : launch_kernel(true, rope_kernel<KVPOOL_BF16, false>, grid, block, 0, s, P);
  else
    e = interleaved ? launch_kernel(true, rope_kernel<KVPOOL_F32, true>, grid, block, 0, s, P)
                    : launch_kernel(true, rope_kernel<KVPOOL_F32, false>, grid, block, 0, s, P);
  return e == cudaSuccess ? KVPOOL_OK : KVPOOL_ERR_CUDA;
}
