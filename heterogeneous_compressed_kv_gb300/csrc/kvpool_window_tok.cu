// kvpool_window_tok.cu -- window attention of single tokens (at most 16 query
// rows per key head): bound by the K and V rows it reads once.
//
// A CTA of four warps takes the rows of one segment and key head and a part of
// the keys that they see (the first tokens and the window as one list).  No
// staging: a lane's loads are whole 16-byte pieces of K and V rows that serve
// as matrix fragments as they arrive, so every warp keeps 8 KB in flight and a
// dozen warps per SM cover the memory's latency.
//
// bf16: S^T = K Q^T with mma m16n8k16, 16 keys x 8 rows.  The index along the
// head's dims is permuted so that lane (g, t) = (lane / 4, lane % 4) of a
// 32-dim piece holds dims 8t .. 8t + 7 of keys g and g + 8 -- one 16-byte load
// each -- and the same dims of query row g.  O^T = V^T P^T: lane (g, t) loads
// dims 8g .. 8g + 7 of keys 2t, 2t + 1, 2t + 8, 2t + 9; two byte permutes make
// the pairs along the keys that the fragment wants; P^T comes from S^T by an
// 8 x 8 transposition of bf16 pairs (movmatrix).  The 5th-generation products
// (128 rows) would do the same with 8 to 128 times the padding.
// A weight goes into the product as two bf16 numbers whose sum holds 16 of its
// bits (off by 2^-18 of it at most): one alone would be off by 2^-9, as much as
// the output's own rounding.  The second product takes 0 to 4% of the time
// (most with 16 rows to a key head).
// fp32: FMAs; four lanes per key, each lane its own running softmax per row.
//
// Measured: 64 requests under a window of 4,096 (16 query heads on 4 key heads
// of 128) 81 - 82 us, 6.6 TB/s (0.97 of the copy rate); 32 requests under 128 (16
// heads) 8.5 - 10.4 us against 5.1 us of reading: launch and one round of
// loads' latency.  Four CTAs to an SM: three took 98 and 14.5 us.
// fp32: the same 64 requests 229 us for 142 us of reading, with 4 heads of 64 100
// for 71; 32 under 128 14.7 for 10.2 (16 heads of 128) and 5.2 for 1.3 (4 of 64).
// Four rows of 128 take 255 registers, which leaves two CTAs to an SM.
#include <cuda_runtime.h>

#include "kvpool_fma.cuh"
#include "kvpool_mma.cuh"
#include "kvpool_window.h"

namespace kvp {
namespace {

constexpr int kTokWarps = 4;

// token of the u-th key of an item's list
__device__ __forceinline__ int tok_of(const WinItem& w, int u) { return u < w.n_s ? u : w.lo + (u - w.n_s); }

// this split's part [a, b) of the list, in whole groups of 64 keys
__device__ __forceinline__ void tok_range(const WinItem& w, int& a, int& b) {
  const int n = w.n_s + w.n_w, g = (n + 63) / 64;
  a = min(n, (int)((int64_t)g * w.split / w.n_split) * 64);
  b = min(n, (int)((int64_t)g * (w.split + 1) / w.n_split) * 64);
}

// Merge the warps' states (m, l, o in shared memory) and write the rows' final
// outputs, or the split's partial.  o: [kTokWarps][rows][D].
template <int T, int D>
__device__ void tok_finish(const WinParams& P, const WinItem& w, const float* so, const float2* sml, int row0, int rows,
                           int stride) {
  const WinSeg& S = P.segs[w.seg];
  for (int i = threadIdx.x; i < rows * (D / 4); i += kTokWarps * 32) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kTokWarps; ++k) m = fmaxf(m, sml[k * stride + r].x);
    const float base = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kTokWarps; ++k) {
      const float2 ml = sml[k * stride + r];
      const float f = ex2f(ml.x - base);
      const float4 x = *reinterpret_cast<const float4*>(so + ((int64_t)k * stride + r) * D + c);
      l = fmaf(ml.y, f, l);
      o.x = fmaf(x.x, f, o.x);
      o.y = fmaf(x.y, f, o.y);
      o.z = fmaf(x.z, f, o.z);
      o.w = fmaf(x.w, f, o.w);
    }
    const int row = row0 + r;
    if (w.n_split > 1) {
      const int64_t pr = (int64_t)w.slot * P.tile_rows + row;
      *reinterpret_cast<float4*>(P.part_o + pr * D + c) = o;
      if (c == 0) P.part_ml[pr] = make_float2(m, l);
      continue;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int64_t tok = S.q_row0 + w.tok0 + row / P.group;
    const int h = w.hk * P.group + row % P.group;
    const int64_t at = tok * P.o_tok + h * P.o_head + c;
    if constexpr (T == KVPOOL_F32)
      *reinterpret_cast<float4*>(P.out + 4 * at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    else
      *reinterpret_cast<uint2*>(P.out + 2 * at) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (P.lse && c == 0) P.lse[tok * P.q_heads + h] = win_lse(m, l);
  }
}

// ---- bf16: NT tiles of 8 rows ------------------------------------------------------
template <int D, int NT>
__global__ void __launch_bounds__(kTokWarps * 32, NT == 1 ? 4 : 2) window_tok_kernel(const __grid_constant__ WinParams P) {
  pdl_start();
  __shared__ float so[kTokWarps][NT * 8][D];
  __shared__ float2 sml[kTokWarps][NT * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const WinItem w = win_item(P, blockIdx.x);
  const WinSeg& S = P.segs[w.seg];
  const int rows = w.n_tok * P.group;
  constexpr int C = D / 32;  // 32-dim pieces of a row

  // query fragments: row 8n + g, dims 32c + 8t .. + 7
  uint4 q[NT][C];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int r = 8 * n + g;
      q[n][c] = make_uint4(0, 0, 0, 0);
      if (r < rows)
        q[n][c] = *reinterpret_cast<const uint4*>(
            P.q + 2 * ((S.q_row0 + w.tok0 + r / P.group) * P.q_tok +
                       (int64_t)(w.hk * P.group + r % P.group) * P.q_head + 32 * c + 8 * t));
    }
  // the positions of this lane's score columns (rows 8n + 2t, + 1)
  int pos[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) pos[n][e] = w.pos0 + (8 * n + 2 * t + e) / P.group;
  const uint8_t* kb = P.k + 2 * (S.k_start * P.k_tok + w.hk * P.k_head + 8 * t);
  const uint8_t* vb = P.v + 2 * (S.k_start * P.v_tok + w.hk * P.v_head + 8 * g);

  float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
  }
  int a, b;
  tok_range(w, a, b);
  for (int u0 = a + 16 * warp; u0 < b; u0 += 16 * kTokWarps) {
    // keys behind the end repeat the last one (masked below)
    uint4 kf[2][C], vf[4][D / 64];
    int tk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      tk[i] = tok_of(w, min(u0 + g + 8 * i, b - 1));
      const uint8_t* p = kb + 2 * (int64_t)tk[i] * P.k_tok;
#pragma unroll
      for (int c = 0; c < C; ++c) kf[i][c] = ld_stream16(p + 64 * c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = u0 + 2 * t + (i & 1) + 8 * (i >> 1);
      const uint8_t* p = vb + 2 * (int64_t)tok_of(w, min(u, b - 1)) * P.v_tok;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) vf[i][h] = ld_stream16(p + 128 * h);
    }
    uint32_t pt[NT][2][2];  // [piece of the weights][keys 0 - 7, 8 - 15]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        mma_bf16(s, kf[0][c].x, kf[1][c].x, kf[0][c].y, kf[1][c].y, q[n][c].x, q[n][c].y);
        mma_bf16(s, kf[0][c].z, kf[1][c].z, kf[0][c].w, kf[1][c].w, q[n][c].z, q[n][c].w);
      }
      // s[2i + e]: key g + 8i, row 2t + e
      float mx[2], corr[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool see = u0 + g + 8 * i < b && win_sees(P, pos[n][e], tk[i]);
          s[2 * i + e] = see ? s[2 * i + e] * P.scale_log2 : -INFINITY;
        }
        mx[e] = fmaxf(s[e], s[2 + e]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], off));
        mx[e] = fmaxf(mx[e], m[n][e]);
        const float base = mx[e] == -INFINITY ? 0.0f : mx[e];
        corr[e] = ex2f(m[n][e] - base);
        m[n][e] = mx[e];
        s[e] = ex2f(s[e] - base);
        s[2 + e] = ex2f(s[2 + e] - base);
        l[n][e] = fmaf(l[n][e], corr[e], s[e] + s[2 + e]);  // this lane's keys only
      }
      if (__any_sync(0xffffffffu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[n][i][j] *= corr[j & 1];
      }
      // the weights' first 8 bits, then the next 8
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t pk = pack_bf16(s[2 * i], s[2 * i + 1]);
          s[2 * i] -= __uint_as_float(pk << 16);
          s[2 * i + 1] -= __uint_as_float(pk & 0xFFFF0000u);
          pt[n][x][i] = transpose8x8(pk);  // row g, keys 2t, 2t + 1 (+ 8)
        }
    }
    // O^T tiles: lane's dims 64h + 8g + 2j (rows g) and + 1 (rows g + 8)
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      const uint32_t v0[4] = {vf[0][h].x, vf[0][h].y, vf[0][h].z, vf[0][h].w};
      const uint32_t v1[4] = {vf[1][h].x, vf[1][h].y, vf[1][h].z, vf[1][h].w};
      const uint32_t v2[4] = {vf[2][h].x, vf[2][h].y, vf[2][h].z, vf[2][h].w};
      const uint32_t v3[4] = {vf[3][h].x, vf[3][h].y, vf[3][h].z, vf[3][h].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = __byte_perm(v0[j], v1[j], 0x5410), a1 = __byte_perm(v0[j], v1[j], 0x7632);
        const uint32_t a2 = __byte_perm(v2[j], v3[j], 0x5410), a3 = __byte_perm(v2[j], v3[j], 0x7632);
#pragma unroll
        for (int x = 1; x >= 0; --x)
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_bf16(o[n][4 * h + j], a0, a1, a2, a3, pt[n][x][0], pt[n][x][1]);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
      const int r = 8 * n + 2 * t + e;
      if (g == 0) sml[warp][r] = make_float2(m[n][e], l[n][e]);
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float2*>(&so[warp][r][64 * h + 8 * g + 2 * j]) =
              make_float2(o[n][4 * h + j][e], o[n][4 * h + j][2 + e]);
    }
  __syncthreads();
  tok_finish<KVPOOL_BF16, D>(P, w, &so[0][0][0], &sml[0][0], 0, rows, NT * 8);
}

// ---- fp32: R rows at a time -----------------------------------------------------------
template <int D, int R>
__global__ void __launch_bounds__(kTokWarps * 32) window_tok_f32_kernel(const __grid_constant__ WinParams P) {
  pdl_start();
  __shared__ float so[kTokWarps][R][D];
  __shared__ float2 sml[kTokWarps][R];
  __shared__ __align__(16) float sq[R][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const WinItem w = win_item(P, blockIdx.x);
  const WinSeg& S = P.segs[w.seg];
  const int row0 = blockIdx.y * R;
  const int rows = min(R, w.n_tok * P.group - row0);
  if (rows <= 0) return;  // (the whole CTA)
  for (int i = threadIdx.x; i < R * (D / 4); i += kTokWarps * 32) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4)), row = row0 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
      x = *reinterpret_cast<const float4*>(P.q + 4 * ((S.q_row0 + w.tok0 + row / P.group) * P.q_tok +
                                                      (int64_t)(w.hk * P.group + row % P.group) * P.q_head + c));
    *reinterpret_cast<float4*>(&sq[r][c]) = x;
  }
  __syncthreads();
  int pos[R];
#pragma unroll
  for (int r = 0; r < R; ++r) pos[r] = w.pos0 + (row0 + r) / P.group;
  const uint8_t* kb = P.k + 4 * (S.k_start * P.k_tok + w.hk * P.k_head + 4 * t);
  const uint8_t* vb = P.v + 4 * (S.k_start * P.v_tok + w.hk * P.v_head + 4 * t);
  // lane (g, t): key g of a group of 8, dims 16i + 4t .. + 3
  constexpr int I = D / 16;
  float m[R], l[R], o[R][4 * I];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int j = 0; j < 4 * I; ++j) o[r][j] = 0.0f;
  }
  int a, b;
  tok_range(w, a, b);
  for (int u0 = a + 8 * warp; u0 < b; u0 += 8 * kTokWarps) {
    const bool in = u0 + g < b;
    const int tk = tok_of(w, min(u0 + g, b - 1));
    float4 k[I], v[I];
#pragma unroll
    for (int i = 0; i < I; ++i) k[i] = *reinterpret_cast<const float4*>(kb + 4 * ((int64_t)tk * P.k_tok + 16 * i));
#pragma unroll
    for (int i = 0; i < I; ++i) v[i] = *reinterpret_cast<const float4*>(vb + 4 * ((int64_t)tk * P.v_tok + 16 * i));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(&sq[r][16 * i + 4 * t]);
        s0 = fmaf(x.x, k[i].x, fmaf(x.y, k[i].y, s0));
        s1 = fmaf(x.z, k[i].z, fmaf(x.w, k[i].w, s1));
      }
      float s = s0 + s1;
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s = in && win_sees(P, pos[r], tk) ? s * P.scale_log2 : -INFINITY;
      const float mx = fmaxf(m[r], s);
      const float base = mx == -INFINITY ? 0.0f : mx;
      const float corr = ex2f(m[r] - base), p = ex2f(s - base);
      m[r] = mx;
      l[r] = fmaf(l[r], corr, p);
#pragma unroll
      for (int i = 0; i < I; ++i) {
        o[r][4 * i] = fmaf(p, v[i].x, o[r][4 * i] * corr);
        o[r][4 * i + 1] = fmaf(p, v[i].y, o[r][4 * i + 1] * corr);
        o[r][4 * i + 2] = fmaf(p, v[i].z, o[r][4 * i + 2] * corr);
        o[r][4 * i + 3] = fmaf(p, v[i].w, o[r][4 * i + 3] * corr);
      }
    }
  }
  // the eight keys' states of a warp into one
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float mx = m[r];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float f = ex2f(m[r] - (mx == -INFINITY ? 0.0f : mx));
    l[r] *= f;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
#pragma unroll
    for (int j = 0; j < 4 * I; ++j) {
      o[r][j] *= f;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) o[r][j] += __shfl_xor_sync(0xffffffffu, o[r][j], off);
    }
    if (g == 0) {
      if (t == 0) sml[warp][r] = make_float2(mx, l[r]);
#pragma unroll
      for (int i = 0; i < I; ++i)
        *reinterpret_cast<float4*>(&so[warp][r][16 * i + 4 * t]) =
            make_float4(o[r][4 * i], o[r][4 * i + 1], o[r][4 * i + 2], o[r][4 * i + 3]);
    }
  }
  __syncthreads();
  tok_finish<KVPOOL_F32, D>(P, w, &so[0][0][0], &sml[0][0], row0, rows, R);
}

template <int D>
cudaError_t launch_tok(const WinParams& P, int dtype, cudaStream_t s) {
  const dim3 block(kTokWarps * 32);
  if (dtype == KVPOOL_BF16)
    return P.tile_rows <= 8 ? launch_kernel(true, window_tok_kernel<D, 1>, dim3(P.n_items), block, 0, s, P)
                            : launch_kernel(true, window_tok_kernel<D, 2>, dim3(P.n_items), block, 0, s, P);
  if (P.tile_rows == 1) return launch_kernel(true, window_tok_f32_kernel<D, 1>, dim3(P.n_items), block, 0, s, P);
  if (P.tile_rows == 2) return launch_kernel(true, window_tok_f32_kernel<D, 2>, dim3(P.n_items), block, 0, s, P);
  return launch_kernel(true, window_tok_f32_kernel<D, 4>, dim3(P.n_items, (P.tile_rows + 3) / 4), block, 0, s, P);
}

}  // namespace

int launch_window_tok(const WinParams& P, int dtype, int head_dim, void* stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return (int)(head_dim == 128 ? launch_tok<128>(P, dtype, s) : launch_tok<64>(P, dtype, s));
}

}  // namespace kvp
