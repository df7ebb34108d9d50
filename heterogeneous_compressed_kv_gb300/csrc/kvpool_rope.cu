// kvpool_rope.cu -- per-head norms of queries and keys with the position
// rotation in the same pass: what a model does to the rows that it hands to
// append and decode_attend.
//
// For one head x of a token at position p:
//   y = x / sqrt(mean(x^2) + eps) * w
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
// over the pairs (a, b) of the first rot_dim dims, t = p * freq_i.
//
// The table holds freq_i / (2 pi) modulo 1 as a 64-bit fraction of a turn, so p
// * table[i] modulo 2^64 is the angle's place in its turn: the integer product
// loses nothing of the table (p * freq_i in fp32 is off by 0.06 rad at p = 2^20),
// and three integer multiplies replace a 64-bit float product and its range
// reduction.  Its top 32 bits as a signed number, times 2^-31, are the angle in
// units of pi in [-1, 1): off by 2^-25 turns at most.  The table itself is a
// quotient in doubles (two roundings) cut off at 2^-64: an angle of N turns at
// position p is off by N 2^-52 + p 2^-64 more, 2^-25 turns at 2^27 of them.
//
// Bound: HBM (one read and one write of every value).  A warp takes one token
// and a run of its heads: the lanes work out the token's rot_dim / 2 sines and
// cosines once (two per lane at 128 dims), pass them through shared memory,
// and then stream heads, 8 values (16 bytes of bf16) per lane and four loads
// ahead.  Norms are held in fp32; one rounding at the store.
//
// What the first form lost was instructions (214 a step of two 128-dim heads,
// 66% of the issue slots at 3.7 TB/s): the weights are now multiplied into the
// sines and cosines once per token and tensor, so that with r = 1 / sqrt(...)
//   y = r * (x * (w cos) + z * (w_z sin)),  z the pair's other value,
// z travels between lanes as it was loaded (two bf16 to a word), and fp32 pairs
// share instructions.
//
// Measured (bf16, heads of 128): 65,537 tokens x 20 heads 116 us, 5.8 TB/s (0.86
// of the copy rate; DRAM 68% busy and the issue slots 60%, 64 registers);
// 8,192 tokens x 32 heads 23.5 us (0.85); 32 tokens x 32 heads 2.7 us, a
// launch's latency.  Few heads: 4,099 tokens x 8 heads of 64 in fp32 6.3 us for 2.5
// us of traffic -- a token is two steps, a warp takes one token at most and here
// one step of it, so that 1 KB is in flight for a position, a table row and a
// sine read and worked out before it.
#include <cmath>
#include <type_traits>

#include <cuda_runtime.h>

#include "device_util.cuh"
#include "kvpool_internal.h"
#include "kvpool_pair.cuh"
#include "kvpool_rows.h"

namespace kvp {
namespace {

constexpr int kRopeWarps = 4;    // warps per CTA
constexpr int kRopeAhead = 4;    // steps (heads per lane group) in flight
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
  int32_t rot_dim, lanes;   // lanes with values per head
  int32_t runs, run_steps;  // runs: warps per token, steps of each
  float eps, inv_dim;
};

// 8 values as loaded: W words, V = 8 / W of them to a word
template <int T>
struct Vec8;
template <>
struct Vec8<KVPOOL_BF16> {
  static constexpr int W = 4;
  uint32_t w[4];
  __device__ __forceinline__ void load(const uint8_t* p) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
  }
  // values 2i and 2i + 1 in fp32
  __device__ __forceinline__ uint64_t pair(int i) const {
    return pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void put(uint8_t* p, const uint64_t* y) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(y[i]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
      o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
  }
};
template <>
struct Vec8<KVPOOL_F32> {
  static constexpr int W = 8;
  uint32_t w[8];
  __device__ __forceinline__ void load(const uint8_t* p) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ uint64_t pair(int i) const {
    return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  static __device__ __forceinline__ void put(uint8_t* p, const uint64_t* y) {
    const float2 a = unpack2(y[0]), b = unpack2(y[1]), c = unpack2(y[2]), d = unpack2(y[3]);
    reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
    reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
  }
};

// G: lanes of a head (of which head_dim / 8 have values)
template <int T, bool INTER, int G>
__global__ void __launch_bounds__(kRopeWarps * 32, T == KVPOOL_BF16 ? 8 : 5) rope_kernel(const __grid_constant__ RopeParams P) {
  pdl_start();
  // cosines and sines of the warps' tokens, in two rows: a lane takes 4 or 8
  // neighbours of each in 16-byte loads (as pairs, 8 bytes each, their bank
  // conflicts cost more than the heads' shuffles)
  __shared__ __align__(16) float turn[kRopeWarps][2][G * 4];
  constexpr int kVecBytes = T == KVPOOL_BF16 ? 16 : 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t task = (int64_t)blockIdx.x * kRopeWarps + warp;
  const int64_t tok = P.runs == 1 ? task : task / P.runs;
  if (tok >= P.n_tokens) return;
  const int s0 = (int)(task - tok * P.runs) * P.run_steps;
  const int s1 = min(s0 + P.run_steps, P.t[0].steps + P.t[1].steps);
  const int sub = lane / G, l = lane % G;  // head within a step, lane within the head
  constexpr int per_step = 32 / G;
  const bool on = l < P.lanes;

  // The batch of steps st .. st + 3 of tensor X, of which those below b and of
  // a head that there is: pointers are of step st.
  Vec8<T> v[kRopeAhead];
  auto load = [&](const RopeTensor& X, const uint8_t* in, int st, int b, int left) {
    const int64_t in_step = per_step * X.in_head;
#pragma unroll
    for (int u = 0; u < kRopeAhead; ++u) {
#pragma unroll
      for (int i = 0; i < Vec8<T>::W; ++i) v[u].w[i] = 0u;
      if (st + u < b && u * per_step < left) v[u].load(in + u * in_step);
    }
  };
  auto in_ptr = [&](const RopeTensor& X, int st) {
    return X.in + tok * X.in_tok + (int64_t)(st * per_step + sub) * X.in_head + l * kVecBytes;
  };
  // the first batch is on its way while the angles are worked out
  {
    const int which = s0 >= P.t[0].steps, a = s0 - (which ? P.t[0].steps : 0);
    const RopeTensor& X = P.t[which];
    load(X, in_ptr(X, a), a, min(s1 - s0 + a, X.steps), on ? X.heads - (a * per_step + sub) : 0);
  }
  bool loaded = true;

  const int half = P.rot_dim / 2;
  if (half > 0) {
    const uint64_t p = (uint64_t)P.pos[tok];
    for (int i = lane; i < half; i += 32) {
      const int32_t t = (int32_t)((p * P.table[i]) >> 32);
      float s, c;
      sincospif((float)t * 0x1p-31f, &s, &c);
      turn[warp][0][i] = c;
      turn[warp][1][i] = s;
    }
    __syncwarp();
  }
  const bool rot = on && 8 * l < P.rot_dim;
  const bool low = 8 * l < half;  // pairs half a rotation apart: the first of its pairs?
  const int partner = (lane - l) + (rot ? (low ? l + half / 8 : l - half / 8) : l);
  const int other = partner - (lane - l);  // the partner's lane within the head

#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const RopeTensor& X = P.t[which];
    const int from = which ? P.t[0].steps : 0;
    const int a = max(s0 - from, 0), b = min(s1 - from, X.steps);  // steps of this tensor
    if (a >= b) continue;
    const uint8_t* in = in_ptr(X, a);
    uint8_t* out = X.out + tok * X.out_tok + (int64_t)(a * per_step + sub) * X.out_head + l * kVecBytes;
    const int64_t in_step = per_step * X.in_head, out_step = per_step * X.out_head;
    int left = on ? X.heads - (a * per_step + sub) : 0;  // heads from this lane's first one on
    // weight times cosine of the value's own, weight times signed sine of the pair's other value
    uint64_t wc[4], ws[4];
    float c[8], sn[8], w[8], wz[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = w[j] = wz[j] = 1.0f, sn[j] = 0.0f;
    if (rot) {
      constexpr int kAng = INTER ? 4 : 8;
      const int at = INTER ? 4 * l : low ? 8 * l : 8 * l - half;
      float x[kAng], y[kAng];
#pragma unroll
      for (int j = 0; j < kAng; j += 4) {
        *reinterpret_cast<float4*>(x + j) = *reinterpret_cast<const float4*>(&turn[warp][0][at + j]);
        *reinterpret_cast<float4*>(y + j) = *reinterpret_cast<const float4*>(&turn[warp][1][at + j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = x[INTER ? j / 2 : j];
        sn[j] = (INTER ? j % 2 == 0 : low) ? -y[INTER ? j / 2 : j] : y[INTER ? j / 2 : j];
      }
    }
    if (X.w && on) {
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        *reinterpret_cast<float4*>(w + j) = *reinterpret_cast<const float4*>(X.w + 8 * l + j);
        if (!INTER) *reinterpret_cast<float4*>(wz + j) = *reinterpret_cast<const float4*>(X.w + 8 * other + j);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wc[i] = pack2(c[2 * i] * w[2 * i], c[2 * i + 1] * w[2 * i + 1]);
      ws[i] = INTER ? pack2(sn[2 * i] * w[2 * i + 1], sn[2 * i + 1] * w[2 * i])
                    : pack2(sn[2 * i] * wz[2 * i], sn[2 * i + 1] * wz[2 * i + 1]);
    }
#pragma unroll 1
    for (int st = a; st < b; st += kRopeAhead) {
      if (!loaded) load(X, in, st, b, left);
      loaded = false;
#pragma unroll
      for (int u = 0; u < kRopeAhead; ++u) {
        if (st + u >= b) break;
        uint64_t sq = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) sq = fma2(v[u].pair(i), v[u].pair(i), sq);
        const float2 f = unpack2(sq);
        float ss = f.x + f.y;
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(fmaf(ss, P.inv_dim, P.eps));
        Vec8<T> z;
        if constexpr (!INTER) {
#pragma unroll
          for (int i = 0; i < Vec8<T>::W; ++i) z.w[i] = __shfl_sync(0xffffffffu, v[u].w[i], partner);
        }
        const uint64_t r2 = pack2(r, r);
        uint64_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t x = v[u].pair(i);
          uint64_t zz;
          if constexpr (INTER) {
            const float2 q = unpack2(x);
            zz = pack2(q.y, q.x);
          } else {
            zz = z.pair(i);
          }
          y[i] = mul2(fma2(zz, ws[i], mul2(x, wc[i])), r2);
        }
        if (u * per_step < left) Vec8<T>::put(out + u * out_step, y);
      }
      in += kRopeAhead * in_step;
      out += kRopeAhead * out_step;
      left -= kRopeAhead * per_step;
    }
  }
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
  const int group = head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32;  // lanes of a head
  const int per_step = 32 / group;
  const int64_t vb = dtype == KVPOOL_BF16 ? 2 : 4;
  for (int i = 0; i < 2; ++i) {
    if (!in[i] || in[i]->heads == 0) continue;  // no such heads
    if (in[i]->heads < 0 || in[i]->heads > 65536 || !out[i] || out[i]->heads != in[i]->heads)
      return KVPOOL_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!in[i]->data || !out[i]->data)) return KVPOOL_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(wt[i]) % 16 != 0) return KVPOOL_ERR_INVALID_ARG;
    if (!rows_aligned(*in[i], dtype) || !rows_aligned(*out[i], dtype)) return KVPOOL_ERR_INVALID_ARG;
    if (!rows_apart(*out[i], n_tokens, head_dim)) return KVPOOL_ERR_INVALID_ARG;
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
  for (int i = 0; i < 2; ++i) {  // an output is its own input or lies apart from everything
    if (P.t[i].steps == 0) continue;
    for (int j = 0; j < 2; ++j) {
      if (P.t[j].steps == 0) continue;
      if (!(i == j && rows_same(*out[i], *in[i], n_tokens)) && rows_meet(*out[i], n_tokens, *in[j], n_tokens, head_dim, vb))
        return KVPOOL_ERR_INVALID_ARG;
      if (i < j && rows_meet(*out[i], n_tokens, *out[j], n_tokens, head_dim, vb)) return KVPOOL_ERR_INVALID_ARG;
    }
  }
  const int steps = P.t[0].steps + P.t[1].steps;
  if (n_tokens == 0 || steps == 0) return KVPOOL_OK;
  if (rot_dim > 0 && (!d_table || !d_positions)) return KVPOOL_ERR_INVALID_ARG;
  P.pos = d_positions;
  P.table = d_table;
  P.n_tokens = n_tokens;
  P.rot_dim = rot_dim;
  P.lanes = head_dim / 8;
  P.eps = eps;
  P.inv_dim = 1.0f / (float)head_dim;
  // warps per token: one takes all its heads (its angles are worked out once)
  // unless there are too few tokens to fill the GPU
  const int sms = device_sms();
  if (sms < 1) return KVPOOL_ERR_CUDA;
  const int64_t fill = 32LL * sms;  // warps that keep every SM's loads in flight
  P.run_steps = kRopeAhead;
  while (P.run_steps < steps && n_tokens * ((steps + 2 * P.run_steps - 1) / (2 * P.run_steps)) >= fill) P.run_steps *= 2;
  while (P.run_steps > 1 && n_tokens * ((steps + P.run_steps - 1) / P.run_steps) < fill) P.run_steps /= 2;
  P.runs = (steps + P.run_steps - 1) / P.run_steps;
  const int64_t ctas = (n_tokens * P.runs + kRopeWarps - 1) / kRopeWarps;
  if (ctas > 0x7FFFFFFF) return KVPOOL_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)ctas), block(kRopeWarps * 32);
  auto go = [&](auto t, auto inter) {
    constexpr int T = decltype(t)::value;
    constexpr bool I = decltype(inter)::value;
    return group == 8    ? launch_kernel(true, rope_kernel<T, I, 8>, grid, block, 0, s, P)
           : group == 16 ? launch_kernel(true, rope_kernel<T, I, 16>, grid, block, 0, s, P)
                         : launch_kernel(true, rope_kernel<T, I, 32>, grid, block, 0, s, P);
  };
  auto types = [&](auto inter) {
    return dtype == KVPOOL_BF16 ? go(std::integral_constant<int, KVPOOL_BF16>(), inter)
                                : go(std::integral_constant<int, KVPOOL_F32>(), inter);
  };
  const cudaError_t e = interleaved ? types(std::true_type()) : types(std::false_type());
  return e == cudaSuccess ? KVPOOL_OK : KVPOOL_ERR_CUDA;
}
