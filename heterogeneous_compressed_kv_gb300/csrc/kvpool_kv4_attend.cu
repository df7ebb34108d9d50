// kvpool_kv4_attend.cu -- attention of a ragged batch over the 4-bit paged
// cache, with the weight that every token got.
//
//   out = sum_t softmax_t(scale <q, k_t>) v_t over t <= p, p the query's place;
//   lse = log sum_t exp(scale <q, k_t>);
//   weights[t] = decay * weights[t] + sum over the key head's query rows of
//   exp(scale <q, k_t> - lse).
//
// A segment with at most 64 query rows to a key head (single tokens, drafts)
// goes through the kernel below; a longer one's tokens are read back to bf16
// (exact) or fp32 rows and go through window attention.
//
// Bound: reading the cache, 1.125 bytes for a key's and a value's number.  The
// keys of a segment and head are cut into parts of equal length, so that all
// parts of the launch are one wave of CTAs.  A CTA of four warps takes a part;
// each warp has a ring of pairs of tiles (32 tokens, one bulk copy), so that up to
// 220 KB are in flight on a multiprocessor without a register held for them.
//
// A tile's products are mma m16n8k16 in fp16: S^T = K Q^T over 16 keys x 8 rows,
// O^T = V^T P^T.  Codes times their scale are exact in fp16.  Queries are
// multiplied by a power of two that brings their row's largest value to 2^14 ..
// 2^15: a bf16 one is exact then, or off by 2^-39 of the largest (half of fp16's
// smallest step); an fp32 one goes in as two halves that hold 22 bits.  Softmax
// weights go in as one half for bf16 outputs (off by 2^-11 of it, the outputs'
// own rounding is 2^-8) and as two for fp32 ones (2^-22), between 2^6 and 2^14 for
// the largest so far, so that small ones are off by 2^-31 of that at most.  The
// unit changes only when a weight passes 2^14 (a running maximum kept exactly
// takes three shuffles and a rescaling test of every tile).
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include <cuda_runtime.h>

#include "kvpool_fma.cuh"
#include "kvpool_kv4.h"
#include "kvpool_mma.cuh"
#include "kvpool_rows.h"

namespace kvp {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxGroup = 16;   // query heads per key head
constexpr int kMaxRows = 64;    // query rows per key head of this file's kernel
constexpr int kMergeWarps = 4;
constexpr float kUp = 6.0f, kMost = 14.0f;  // see the kernel's c

struct Kv4Seg {
  int64_t q_row0;      // first query row
  int64_t score_base;  // first score (weights wanted)
  int32_t q_len, k_len;
  int32_t n_parts;     // parts that each head's keys are cut into
  int32_t item_base;   // first work item: (part * row tiles + row tile) * kv_heads + head
  int32_t part_base;   // first partial (partials wanted)
  int32_t row_base;    // first of the rows (head, row) that have partials
  int32_t key_base;    // first block of keys whose weights are summed
  int32_t table_row;
};

struct Kv4Params {
  Kv4Cache c;
  const uint8_t* q;
  uint8_t* out;
  float* lse;      // [q_rows][q_heads] or null
  float* weights;  // or null
  int64_t q_tok, q_head, o_tok, o_head;  // strides in values
  int64_t w_seg, w_head;
  int32_t group;
  int32_t tile_rows;       // rows of a row tile
  int32_t part_pairs;      // pairs of tiles of a part
  float scale_log2;        // softmax scale times log2(e) and the keys' scale
  float decay;
  int32_t n_segs, n_items, n_rows, n_blocks;
  float* part_o;    // [partials][tile_rows][head_dim]
  float2* part_ml;  // [partials][tile_rows]: (exponent of the weights' unit, sum)
  float* lse2;      // [n_rows], log2 domain (weights wanted)
  float* scores;    // log2 domain (weights wanted)
  Kv4Seg segs[kKv4MaxSegs];
};

template <typename F>
__device__ __forceinline__ int find_seg(const Kv4Params& P, int x, F base) {
  int lo = 0, hi = P.n_segs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base(P.segs[mid]) <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int score_pitch(int k_len) { return (k_len + 3) & ~3; }

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t a) { return __half22float2(*reinterpret_cast<const __half2*>(&a)); }
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

constexpr int kStages = 3;
constexpr int kPair = 2;  // tiles of a stage

template <int D, int NT>
struct Kv4Smem {
  union {
    uint8_t ring[kWarps][kStages][kPair * Kv4Tile<D>::kBytes];
    float o[kWarps][NT * 8][D];  // once the ring is done with
  };
  float2 ml[kWarps][NT * 8];
  uint64_t bar[kWarps][kStages];
};

// The keys of a tile as the lane's share of fragments: keys g and g + 8, dims
// D / 4 * t and on, eight dims to a word; sc: [key][half of the lane's dims]
template <int D>
struct Kv4Keys {
  uint32_t k0[D / 32], k1[D / 32], sc[2][2];
  __device__ __forceinline__ void load(const uint8_t* tile, int lane) {
    const int g = lane >> 2, t = lane & 3;
    if constexpr (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(tile + lane * 16), y = *reinterpret_cast<const uint4*>(tile + 512 + lane * 16);
      k0[0] = x.x, k0[1] = x.y, k0[2] = x.z, k0[3] = x.w;
      k1[0] = y.x, k1[1] = y.y, k1[2] = y.z, k1[3] = y.w;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t h =
            e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(tile + Kv4Tile<D>::kKs + (g + 8 * i) * 8 + 2 * t));
        sc[i][0] = __byte_perm(h, h, 0x1010);
        sc[i][1] = __byte_perm(h, h, 0x3232);
      }
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(tile + lane * 8), y = *reinterpret_cast<const uint2*>(tile + 256 + lane * 8);
      k0[0] = x.x, k0[1] = x.y;
      k1[0] = y.x, k1[1] = y.y;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t h = tile[Kv4Tile<D>::kKs + (g + 8 * i) * 4 + t];
        sc[i][0] = sc[i][1] = e4m3x2_to_f16x2((uint16_t)(h | h << 8));
      }
    }
  }
};

// NT: tiles of 8 query rows; F32: fp32 queries and outputs
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 && !F32 ? 4 : 2) kv4_attend_kernel(const __grid_constant__ Kv4Params P) {
  pdl_start();
  using L = Kv4Tile<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Kv4Smem<D, NT>& sm = *reinterpret_cast<Kv4Smem<D, NT>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int kPieces = F32 ? 2 : 1;
  constexpr int KS = D / 16;  // steps of 16 dims

  // ---- the work item ----
  const int seg = find_seg(P, blockIdx.x, [](const Kv4Seg& s) { return s.item_base; });
  const Kv4Seg& S = P.segs[seg];
  const int n_rows = S.q_len * P.group, row_tiles = (n_rows + P.tile_rows - 1) / P.tile_rows;
  int r = blockIdx.x - S.item_base;
  const int slot = S.part_base + r;
  const int head = r % P.c.kv_heads;
  r /= P.c.kv_heads;
  const int row0 = r % row_tiles * P.tile_rows, part = r / row_tiles;
  const int rows = min(P.tile_rows, n_rows - row0);
  const int pos0 = S.k_len - S.q_len + row0 / P.group;  // the first row's place
  // keys that some row sees (may be < 1); where scores are kept, every key has one
  const int seen = P.scores ? S.k_len : S.k_len - S.q_len + (row0 + rows - 1) / P.group + 1;
  // pairs of tiles a + warp, + kWarps, ... below b
  const int a = part * P.part_pairs;
  const int b = min((max(seen, 0) + kPair * kKv4Tile - 1) / (kPair * kKv4Tile), a + P.part_pairs);
  const int n_my = b > a + warp ? (b - a - warp + kWarps - 1) / kWarps : 0;

  // ---- the ring ----
  uint64_t* bar = sm.bar[warp];
  if (lane < kStages) mbar_init(&bar[lane], 1);
  mbar_fence_init();
  __syncwarp();
  // Page ids of 16 of the warp's pairs, and of the next 16: lane 2i + j has the
  // one of tile j of pair i (a pair in one page has two equal ones).  A tile
  // behind the segment's last one is never looked up: its pair is in one page,
  // or it is not copied.
  const int last = (S.k_len - 1) / kKv4Tile;
  auto ids_from = [&](int i) {
    const int tile = kPair * (a + warp + kWarps * (i + (lane >> 1))) + (lane & 1);
    return i + (lane >> 1) < n_my ? kv4_page(P.c, S.table_row, min(tile, last)) : 0;
  };
  int ids = ids_from(0), ids_next = ids_from(16);
  auto issue = [&](int i, int stage) {
    if (i > 0 && (i & 15) == 0) {
      ids = ids_next;
      ids_next = ids_from(i + 16);
    }
    // (a bad page: page 0, flagged)
    const int id0 = max(__shfl_sync(0xffffffffu, ids, 2 * (i & 15)), 0);
    const int id1 = max(__shfl_sync(0xffffffffu, ids, 2 * (i & 15) + 1), 0);
    const int tile = kPair * (a + warp + kWarps * i);
    if (lane == 0) {
      uint64_t* mb = &bar[stage];
      uint8_t* dst = sm.ring[warp][stage];
      const uint8_t* src = P.c.pages + kv4_tile_offset<D>(P.c, id0, head, tile);
      if (P.c.page_shift > 0) {  // both tiles in one page
        mbar_arrive_expect_tx(mb, kPair * L::kBytes);
        bulk_g2s(dst, src, kPair * L::kBytes, mb);
      } else {
        mbar_arrive_expect_tx(mb, (tile < last ? kPair : 1) * L::kBytes);
        bulk_g2s(dst, src, L::kBytes, mb);
        if (tile < last) bulk_g2s(dst + L::kBytes, P.c.pages + kv4_tile_offset<D>(P.c, id1, head, tile + 1), L::kBytes, mb);
      }
    }
  };
  int issued = 0;
  for (; issued < min(kStages, n_my); ++issued) issue(issued, issued);

  // ---- queries: row 8n + g, dims D / 4 * t .. as fp16 pieces ----
  constexpr int vb = F32 ? 4 : 2;
  uint32_t q[kPieces][NT][2 * KS];
  float mul[NT][2];  // score scale of rows 8n + 2t, + 1
  int pos[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float x[4 * KS];
    const int row = row0 + 8 * n + g;
    const uint8_t* p = P.q + vb * ((S.q_row0 + row / P.group) * P.q_tok +
                                   (int64_t)(head * P.group + row % P.group) * P.q_head + 4 * KS * t);
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4 * KS; i += 16 / vb) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (8 * n + g < rows) w = *reinterpret_cast<const uint4*>(p + vb * i);
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
          x[i + j] = __uint_as_float(v[j]);
        } else {
          x[i + 2 * j] = __uint_as_float(v[j] << 16);
          x[i + 2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4 * KS; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^(14 - e), e the exponent of the largest value (at least -110)
    const int e = max((int)(amax >> 23) - 127, -110);
    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23), down = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
      const float x0 = x[2 * i] * up, x1 = x[2 * i + 1] * up;
      q[0][n][i] = pack_f16(x0, x1);
      if constexpr (F32) {
        const float2 h = unpack_f16(q[0][n][i]);
        q[1][n][i] = pack_f16(x0 - h.x, x1 - h.y);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      mul[n][c] = P.scale_log2 * __shfl_sync(0xffffffffu, down, 4 * (2 * t + c));
      pos[n][c] = min(S.k_len - 1, S.k_len - S.q_len + (row0 + 8 * n + 2 * t + c) / P.group);
    }
  }

  // A row's weights are 2^(score + c): c is such that the largest score seen when
  // it was last set gave 2^kUp, and is set anew when one passes 2^kMost (`most`;
  // -inf before the row's first score).
  float c[NT][2], most[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    c[n][0] = c[n][1] = 0.0f;
    most[n][0] = most[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
  }
  float* scores = nullptr;
  const int pitch = score_pitch(S.k_len);
  if (P.scores) scores = P.scores + S.score_base + ((int64_t)head * n_rows + row0) * pitch;

  // ---- pairs of tiles ----
  int stage = 0, phase = 0;
#pragma unroll 1
  for (int i = 0; i < n_my; ++i) {
    if (!warp_wait(&bar[stage], phase, P.c.err)) {  // (flagged) the copies on their way, then the end
      for (int j = i + 1; j < issued; ++j) warp_wait(&bar[j % kStages], j / kStages & 1, P.c.err);
      break;
    }
    const uint8_t* ring = sm.ring[warp][stage];
    const int u0 = (a + warp + kWarps * i) * kPair * kKv4Tile;
    float s[kPair][NT][4];  // [2i + c]: key g + 8i of the tile, row 8n + 2t + c
#pragma unroll
    for (int y = 0; y < kPair; ++y) {
      Kv4Keys<D> K;
      K.load(ring + y * L::kBytes, lane);
      float s2[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[y][n][j] = s2[n][j] = 0.0f;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t k0[4], k1[4];
        e2m1x8_to_f16x2x4(K.k0[w], k0);
        e2m1x8_to_f16x2x4(K.k1[w], k1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          k0[j] = mul_f16x2(k0[j], K.sc[0][w / 2]);
          k1[j] = mul_f16x2(k1[j], K.sc[1][w / 2]);
        }
#pragma unroll
        for (int x = kPieces - 1; x >= 0; --x)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(s[y][n], k0[0], k1[0], k0[1], k1[1], q[x][n][4 * w], q[x][n][4 * w + 1]);
            mma_f16(s2[n], k0[2], k1[2], k0[3], k1[3], q[x][n][4 * w + 2], q[x][n][4 * w + 3]);
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[y][n][j] += s2[n][j];
    }
    if (scores) {
#pragma unroll
      for (int y = 0; y < kPair; ++y)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = 8 * n + 2 * t + (j & 1), u = u0 + kKv4Tile * y + g + 8 * (j >> 1);
            if (row < rows && u < S.k_len)
              scores[(int64_t)row * pitch + u] = u <= pos[n][j & 1] ? s[y][n][j] * mul[n][j & 1] : -INFINITY;
          }
    }
    bool high = false;
#pragma unroll
    for (int y = 0; y < kPair; ++y)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[y][n][j] = fmaf(s[y][n][j], mul[n][j & 1], c[n][j & 1]);
    if (u0 + kPair * kKv4Tile - 1 > pos0) {  // some row does not see some key
#pragma unroll
      for (int y = 0; y < kPair; ++y)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (u0 + kKv4Tile * y + g + 8 * (j >> 1) > pos[n][j & 1]) s[y][n][j] = -INFINITY;
    }
    float mx[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[n][e] = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e]));
        high |= mx[n][e] > most[n][e];
      }
    if (__any_sync(0xffffffffu, high)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], off));
          if (!(mx[n][e] > most[n][e])) continue;
          const float d = kUp - mx[n][e], f = ex2f(d);  // (the first time, l and o are zeros or NaN)
          c[n][e] += d;
          most[n][e] = kMost;
          l[n][e] = l[n][e] == 0.0f ? 0.0f : l[n][e] * f;
#pragma unroll
          for (int y = 0; y < kPair; ++y) s[y][n][e] += d, s[y][n][2 + e] += d;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            o[n][x][e] = o[n][x][e] == 0.0f ? 0.0f : o[n][x][e] * f;
            o[n][x][2 + e] = o[n][x][2 + e] == 0.0f ? 0.0f : o[n][x][2 + e] * f;
          }
        }
    }
#pragma unroll
    for (int y = 0; y < kPair; ++y) {
      uint32_t pt[kPieces][NT][2];  // [keys 0 - 7, 8 - 15]
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[y][n][j] = ex2f(s[y][n][j]);
        l[n][0] += s[y][n][0] + s[y][n][2];  // this lane's keys only
        l[n][1] += s[y][n][1] + s[y][n][3];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t pk = pack_f16(s[y][n][2 * j], s[y][n][2 * j + 1]);
          if constexpr (F32) {
            const float2 h = unpack_f16(pk);
            pt[1][n][j] = transpose8x8(pack_f16(s[y][n][2 * j] - h.x, s[y][n][2 * j + 1] - h.y));
          }
          pt[0][n][j] = transpose8x8(pk);  // row g, keys 2t, 2t + 1 (+ 8)
        }
      }
      // values: lane's dims D / 8 * g and on of the token pairs t and t + 4
      constexpr int W = D / 32;  // words of 4 dims
      uint32_t v0[W], v1[W];
      const uint8_t* tile = ring + y * L::kBytes;
      const uint8_t* p = tile + L::kV + t * D + (g ^ kv4_swizzle<D>(t)) * L::kChunk;  // (t and t + 4 swizzle alike)
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(p), z = *reinterpret_cast<const uint4*>(p + 4 * D);
        v0[0] = x.x, v0[1] = x.y, v0[2] = x.z, v0[3] = x.w;
        v1[0] = z.x, v1[1] = z.y, v1[2] = z.z, v1[3] = z.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p), z = *reinterpret_cast<const uint2*>(p + 4 * D);
        v0[0] = x.x, v0[1] = x.y;
        v1[0] = z.x, v1[1] = z.y;
      }
      const int grp = g * L::kChunk / kKv4Group;
      uint32_t e0 = *reinterpret_cast<const uint16_t*>(tile + L::kVs + t * (D / 8) + 2 * grp);
      uint32_t e1 = *reinterpret_cast<const uint16_t*>(tile + L::kVs + (t + 4) * (D / 8) + 2 * grp);
      if (u0 + kKv4Tile * (y + 1) > S.k_len) {  // places behind the last token may hold anything
        const int left = S.k_len - u0 - kKv4Tile * y - 2 * t;
        e0 &= left >= 2 ? 0xFFFFu : left == 1 ? 0xFFu : 0u;
        e1 &= left >= 10 ? 0xFFFFu : left == 9 ? 0xFFu : 0u;
      }
      const uint32_t f0 = e4m3x2_to_f16x2((uint16_t)e0), f1 = e4m3x2_to_f16x2((uint16_t)e1);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t x[4], z[4];
        e2m1x8_to_f16x2x4(v0[w], x);
        e2m1x8_to_f16x2x4(v1[w], z);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = mul_f16x2(x[j], f0);
          z[j] = mul_f16x2(z[j], f1);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (F32) {  // a tile's own sum, added with rounding (the tensor core cuts a running sum off)
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(d, x[2 * j], x[2 * j + 1], z[2 * j], z[2 * j + 1], pt[1][n][0], pt[1][n][1]);
              mma_f16(d, x[2 * j], x[2 * j + 1], z[2 * j], z[2 * j + 1], pt[0][n][0], pt[0][n][1]);
#pragma unroll
              for (int k = 0; k < 4; ++k) o[n][2 * w + j][k] += d[k];
            } else {
              mma_f16(o[n][2 * w + j], x[2 * j], x[2 * j + 1], z[2 * j], z[2 * j + 1], pt[0][n][0], pt[0][n][1]);
            }
          }
      }
    }
    __syncwarp();  // the pair is read
    if (issued < n_my) issue(issued++, stage);
    if (++stage == kStages) stage = 0, phase ^= 1;
  }

  // ---- the warps' states into one ----
  __syncthreads();  // every warp's ring is done with (and no copy on its way)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
      const int row = 8 * n + 2 * t + e;
      // the exponent of the weights' unit (-inf: the row saw nothing)
      if (g == 0) sm.ml[warp][row] = make_float2(l[n][e] == 0.0f ? -INFINITY : -c[n][e], l[n][e]);
#pragma unroll
      for (int x = 0; x < D / 16; ++x)  // dims D / 8 * g + 2x, + 1
        *reinterpret_cast<float2*>(&sm.o[warp][row][L::kChunk * g + 2 * x]) = make_float2(o[n][x][e], o[n][x][2 + e]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += kWarps * 32) {
    const int row = i / (D / 4), c = 4 * (i % (D / 4));
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, sm.ml[k][row].x);
    const float base = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float2 ml = sm.ml[k][row];
      const float f = ex2f(ml.x - base);
      const float4 y = *reinterpret_cast<const float4*>(&sm.o[k][row][c]);
      sum = fmaf(ml.y, f, sum);
      x.x = fmaf(y.x, f, x.x);
      x.y = fmaf(y.y, f, x.y);
      x.z = fmaf(y.z, f, x.z);
      x.w = fmaf(y.w, f, x.w);
    }
    if (S.n_parts > 1) {
      const int64_t pr = (int64_t)slot * P.tile_rows + row;
      *reinterpret_cast<float4*>(P.part_o + pr * D + c) = x;
      if (c == 0) P.part_ml[pr] = make_float2(mx, sum);
      continue;
    }
    const float inv = sum > 0.0f ? P.c.v_scale / sum : sum == 0.0f ? 0.0f : sum;  // (a NaN stays one)
    const int gr = row0 + row;
    const int64_t tok = S.q_row0 + gr / P.group;
    const int h = head * P.group + gr % P.group;
    const int64_t at = tok * P.o_tok + h * P.o_head + c;
    if constexpr (F32)
      *reinterpret_cast<float4*>(P.out + 4 * at) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    else
      *reinterpret_cast<uint2*>(P.out + 2 * at) = make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    if (c == 0) {
      const float z = sum == 0.0f ? -INFINITY : mx + log2f(sum);
      if (P.lse) P.lse[tok * (P.c.kv_heads * P.group) + h] = z * 0.69314718055994531f;
      if (P.lse2) P.lse2[S.row_base + head * n_rows + gr] = z;
    }
  }
}

// One warp per row (head, row) of a segment whose keys were cut: out = sum_s
// 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s, parts in order.
template <int D, bool F32>
__global__ void __launch_bounds__(kMergeWarps * 32) kv4_merge_kernel(const __grid_constant__ Kv4Params P) {
  pdl_start();
  const int lane = threadIdx.x & 31, id = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  if (id >= P.n_rows) return;
  const int seg = find_seg(P, id, [](const Kv4Seg& s) { return s.row_base; });
  const Kv4Seg& S = P.segs[seg];
  if (S.n_parts <= 1) return;
  const int n_rows = S.q_len * P.group, row_tiles = (n_rows + P.tile_rows - 1) / P.tile_rows;
  const int head = (id - S.row_base) / n_rows, gr = (id - S.row_base) % n_rows;
  const int64_t step = (int64_t)row_tiles * P.c.kv_heads;  // partials of a part
  const int64_t slot0 = S.part_base + (int64_t)(gr / P.tile_rows) * P.c.kv_heads + head;
  constexpr int V = D / 32;
  float m = -INFINITY, l = 0.0f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < S.n_parts; ++s) {
    const int64_t pr = (slot0 + s * step) * P.tile_rows + gr % P.tile_rows;
    const float2 ml = P.part_ml[pr];
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = P.part_o[pr * D + lane * V + i];
    const float mx = fmaxf(m, ml.x);
    const float base = mx == -INFINITY ? 0.0f : mx;
    const float fa = ex2f(m - base), fb = ex2f(ml.x - base);
    l = l * fa + ml.y * fb;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = acc[i] * fa + x[i] * fb;
    m = mx;
  }
  const float inv = l > 0.0f ? P.c.v_scale / l : l == 0.0f ? 0.0f : l;
  const int64_t tok = S.q_row0 + gr / P.group;
  const int h = head * P.group + gr % P.group;
  const int64_t at = tok * P.o_tok + h * P.o_head + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if constexpr (F32)
      *reinterpret_cast<float2*>(P.out + 4 * (at + i)) = make_float2(acc[i] * inv, acc[i + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(P.out + 2 * (at + i)) = pack_bf16(acc[i] * inv, acc[i + 1] * inv);
  }
  if (lane == 0) {
    const float z = l == 0.0f ? -INFINITY : m + log2f(l);
    if (P.lse) P.lse[tok * (P.c.kv_heads * P.group) + h] = z * 0.69314718055994531f;
    if (P.lse2) P.lse2[id] = z;
  }
}

// A CTA sums the weights of kWeightKeys keys of a segment and head, rows in
// order (the same sum on every run); a row that saw nothing gives none.
constexpr int kWeightThreads = 128, kWeightKeys = 4 * kWeightThreads;
__global__ void __launch_bounds__(kWeightThreads) kv4_weights_kernel(const __grid_constant__ Kv4Params P) {
  pdl_start();
  const int seg = find_seg(P, blockIdx.x, [](const Kv4Seg& s) { return s.key_base; });
  const Kv4Seg& S = P.segs[seg];
  const int r = blockIdx.x - S.key_base, head = r % P.c.kv_heads;
  const int t0 = r / P.c.kv_heads * kWeightKeys + 4 * threadIdx.x;
  const int n_rows = S.q_len * P.group, pitch = score_pitch(S.k_len);
  if (t0 >= S.k_len) return;
  const float* s = P.scores + S.score_base + (int64_t)head * n_rows * pitch + t0;
  const float* z = P.lse2 + S.row_base + head * n_rows;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int i = 0; i < n_rows; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(s + (int64_t)i * pitch);
    const float y = z[i];
    if (y == -INFINITY) continue;
    w[0] += ex2f(x.x - y);
    w[1] += ex2f(x.y - y);
    w[2] += ex2f(x.z - y);
    w[3] += ex2f(x.w - y);
  }
  float* out = P.weights + S.table_row * P.w_seg + head * P.w_head + t0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t0 + i < S.k_len) out[i] = P.decay == 0.0f ? w[i] : fmaf(P.decay, out[i], w[i]);
}

// ---- host -------------------------------------------------------------------
bool is_prompt(const kvpool_kv4_args* a, int64_t q_len) { return q_len * (a->q.heads / a->cache.kv_heads) > kMaxRows; }

int check_args(const kvpool_kv4_args* a, int32_t n, const int64_t* q_len, const int64_t* k_len, int64_t* total_q) {
  if (!a || n < 0) return KVPOOL_ERR_INVALID_ARG;
  const int rc = kv4_check(&a->cache, n);
  if (rc != KVPOOL_OK) return rc;
  const int32_t hk = a->cache.kv_heads;
  if (a->dtype != KVPOOL_F32 && a->dtype != KVPOOL_BF16) return KVPOOL_ERR_INVALID_ARG;
  if (a->out.heads != a->q.heads || a->q.heads < hk || a->q.heads > kKv4MaxHeads || a->q.heads % hk != 0 ||
      a->q.heads / hk > kMaxGroup)
    return KVPOOL_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale) || !std::isfinite(a->decay) || a->q_rows < 0 || a->q_rows > 0x7FFFFFFF)
    return KVPOOL_ERR_INVALID_ARG;
  if (!rows_aligned(a->q, a->dtype) || !rows_aligned(a->out, a->dtype) || !rows_apart(a->out, a->q_rows, a->cache.head_dim))
    return KVPOOL_ERR_INVALID_ARG;
  if (n > 0 && (!q_len || !k_len)) return KVPOOL_ERR_INVALID_ARG;
  int64_t q = 0, most = 0;
  bool keys = false;
  for (int i = 0; i < n; ++i) {
    if (q_len[i] < 0 || q_len[i] > (1 << 30) || k_len[i] < 0 || k_len[i] > kv4_tokens(&a->cache)) return KVPOOL_ERR_INVALID_ARG;
    if (q_len[i] == 0) continue;
    if (a->d_weights && is_prompt(a, q_len[i])) return KVPOOL_ERR_INVALID_ARG;
    q += q_len[i];
    most = std::max(most, k_len[i]);
    keys |= k_len[i] > 0;
  }
  if (q > a->q_rows) return KVPOOL_ERR_INVALID_ARG;
  if (q > 0 && (!a->q.data || !a->out.data)) return KVPOOL_ERR_INVALID_ARG;
  if (keys && (!a->cache.d_pages || !a->cache.d_table || a->cache.n_pages < 1)) return KVPOOL_ERR_INVALID_ARG;
  if (a->d_weights && (reinterpret_cast<uintptr_t>(a->d_weights) % 4 != 0 ||
                       (hk > 1 && a->weight_head_stride < most) ||
                       (n > 1 && a->weight_stride < (int64_t)(hk - 1) * a->weight_head_stride + most)))
    return KVPOOL_ERR_INVALID_ARG;
  *total_q = q;
  return KVPOOL_OK;
}

constexpr int64_t kMinPairs = 8;  // pairs of tiles of a part, at least

// Where a launch's workspace lies, in bytes from its start.
struct Space {
  int64_t part_ml, lse2, scores, total;
};

// Segments [i0, n) of one launch (at most kKv4MaxSegs that are no prompts);
// returns the next segment, or -1 (too large for one launch).
int32_t plan(const kvpool_kv4_args* a, int32_t i0, int32_t n, const int64_t* q_len, const int64_t* k_len, int64_t* q_row,
             int n_sms, Kv4Params* P, Space* w) {
  const int hk = a->cache.kv_heads, group = a->q.heads / hk;
  int32_t i = i0;
  int64_t row = *q_row, most_rows = 0;
  P->n_segs = 0;
  for (; i < n && P->n_segs < kKv4MaxSegs; ++i) {
    if (q_len[i] > 0 && !is_prompt(a, q_len[i])) {
      Kv4Seg& S = P->segs[P->n_segs++];
      S = Kv4Seg{};
      S.q_row0 = row;
      S.q_len = (int32_t)q_len[i];
      S.k_len = (int32_t)k_len[i];
      S.table_row = i - i0;
      most_rows = std::max(most_rows, q_len[i] * group);
    }
    row += q_len[i];
  }
  *q_row = row;
  P->tile_rows = most_rows <= 8 ? 8 : 16;
  auto row_tiles = [&](const Kv4Seg& S) { return ((int64_t)S.q_len * group + P->tile_rows - 1) / P->tile_rows; };
  auto pairs = [&](const Kv4Seg& S) {
    return std::max<int64_t>(1, ((int64_t)S.k_len + kPair * kKv4Tile - 1) / (kPair * kKv4Tile));
  };
  auto items = [&](int64_t part) {
    int64_t x = 0;
    for (int s = 0; s < P->n_segs; ++s) {
      const Kv4Seg& S = P->segs[s];
      x += (pairs(S) + part - 1) / part * row_tiles(S) * hk;
    }
    return x;
  };
  // the shortest parts that are one wave of CTAs together
  const int64_t want = (int64_t)n_sms * (P->tile_rows == 8 && a->dtype == KVPOOL_BF16 ? 4 : 2);
  int64_t lo = kMinPairs, hi = kMinPairs;
  while (hi < (1 << 26) && items(hi) > want) hi *= 2;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (items(mid) <= want) hi = mid;
    else lo = mid + 1;
  }
  P->part_pairs = (int32_t)lo;
  int64_t item = 0, partials = 0, rows = 0, blocks = 0, scores = 0;
  bool cut = false;
  for (int s = 0; s < P->n_segs; ++s) {
    Kv4Seg& S = P->segs[s];
    const int64_t parts = (pairs(S) + lo - 1) / lo, its = parts * row_tiles(S) * hk;
    S.n_parts = (int32_t)parts;
    S.item_base = (int32_t)item;
    S.part_base = (int32_t)partials;
    S.row_base = (int32_t)rows;
    S.key_base = (int32_t)blocks;
    S.score_base = scores;
    item += its;
    if (parts > 1) partials += its, cut = true;
    rows += (int64_t)S.q_len * group * hk;
    if (a->d_weights) {
      blocks += ((int64_t)S.k_len + kWeightKeys - 1) / kWeightKeys * hk;
      scores += (int64_t)S.q_len * group * hk * ((S.k_len + 3) & ~3);
    }
  }
  if (item > (1 << 30) || partials > (1 << 30) || rows > (1 << 30) || blocks > (1 << 30)) return -1;
  P->n_items = (int32_t)item;
  P->n_rows = (int32_t)rows;
  P->n_blocks = (int32_t)blocks;
  w->part_ml = partials * P->tile_rows * a->cache.head_dim * 4;
  w->lse2 = w->part_ml + partials * P->tile_rows * 8;
  w->scores = w->lse2 + (a->d_weights ? (rows * 4 + 15) / 16 * 16 : 0);
  w->total = w->scores + 4 * scores;
  if (!cut) w->part_ml = -1;
  return i;
}

// The prompts: runs of segments that are prompts (or have no queries), whose
// tokens are read back to rows of the queries' type.
struct Run {
  int32_t first, end;
  int64_t q_row, q_rows, kv_rows, bytes;  // bytes: keys' and values' rows
};
bool next_run(const kvpool_kv4_args* a, int32_t* i, int64_t* q_row, int32_t n, const int64_t* q_len, const int64_t* k_len,
              Run* run) {
  while (*i < n && (q_len[*i] == 0 || !is_prompt(a, q_len[*i]))) *q_row += q_len[(*i)++];
  if (*i >= n) return false;
  *run = Run{*i, *i, *q_row, 0, 0, 0};
  for (; *i < n && (q_len[*i] == 0 || is_prompt(a, q_len[*i])); ++*i) {
    run->q_rows += q_len[*i];
    if (q_len[*i] > 0) run->kv_rows += k_len[*i];
  }
  *q_row += run->q_rows;
  run->end = *i;
  run->bytes = run->kv_rows * a->cache.kv_heads * a->cache.head_dim * (a->dtype == KVPOOL_BF16 ? 2 : 4);
  return true;
}

// The window call of a run: everything up to the query is visible.
struct WindowCall {
  kvpool_window_args args;
  std::unique_ptr<int64_t[]> start, len;  // [segments of the run], keys read back
};
bool window_call(const kvpool_kv4_args* a, const Run& run, const int64_t* q_len, const int64_t* k_len, void* space,
                 WindowCall* w) {
  const int32_t n = run.end - run.first;
  w->start.reset(new (std::nothrow) int64_t[n]);
  w->len.reset(new (std::nothrow) int64_t[n]);
  if (!w->start || !w->len) return false;
  int64_t at = 0;
  for (int32_t i = 0; i < n; ++i) {
    w->len[i] = q_len[run.first + i] > 0 ? k_len[run.first + i] : 0;
    w->start[i] = at;
    at += w->len[i];
  }
  const int64_t vb = a->dtype == KVPOOL_BF16 ? 2 : 4;
  kvpool_window_args& x = w->args;
  x = kvpool_window_args{};
  x.dtype = a->dtype;
  x.head_dim = a->cache.head_dim;
  x.q = a->q;
  x.out = a->out;
  x.q.data = static_cast<const uint8_t*>(a->q.data) + vb * run.q_row * a->q.token_stride;
  x.out.data = static_cast<const uint8_t*>(a->out.data) + vb * run.q_row * a->out.token_stride;
  const int64_t row = (int64_t)a->cache.kv_heads * a->cache.head_dim;
  x.k = kvpool_heads{space, row, a->cache.head_dim, a->cache.kv_heads, 0};
  x.v = x.k;
  x.v.data = static_cast<uint8_t*>(space) + run.bytes;
  x.q_rows = run.q_rows;
  x.kv_rows = run.kv_rows;
  x.d_lse = a->d_lse ? a->d_lse + run.q_row * a->q.heads : nullptr;
  x.window = 1 << 30;
  x.scale = a->scale;
  return true;
}

template <int D, int NT, bool F32>
cudaError_t launch_attend(const Kv4Params& P, cudaStream_t s) {
  constexpr int smem = (int)sizeof(Kv4Smem<D, NT>);
  auto* kern = kv4_attend_kernel<D, NT, F32>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e == cudaSuccess ? launch_kernel(true, kern, dim3(P.n_items), dim3(kWarps * 32), smem, s, P) : e;
}

template <int D, bool F32>
cudaError_t launch_all(const Kv4Params& P, bool cut, cudaStream_t s) {
  cudaError_t e = P.tile_rows == 8 ? launch_attend<D, 1, F32>(P, s) : launch_attend<D, 2, F32>(P, s);
  if (e == cudaSuccess && cut)
    e = launch_kernel(true, kv4_merge_kernel<D, F32>, dim3((P.n_rows + kMergeWarps - 1) / kMergeWarps), dim3(kMergeWarps * 32),
                      0, s, P);
  if (e == cudaSuccess && P.n_blocks > 0)
    e = launch_kernel(true, kv4_weights_kernel, dim3(P.n_blocks), dim3(kWeightThreads), 0, s, P);
  return e;
}

}  // namespace
}  // namespace kvp

extern "C" int64_t kvpool_kv4_workspace(const kvpool_kv4_args* a, int32_t n, const int64_t* h_q_len, const int64_t* h_k_len) {
  using namespace kvp;
  int64_t total = 0, most = 0;
  const int rc = check_args(a, n, h_q_len, h_k_len, &total);
  if (rc != KVPOOL_OK) return rc;
  if (total == 0) return 0;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  std::unique_ptr<Kv4Params> P(new (std::nothrow) Kv4Params);
  if (!P) return KVPOOL_ERR_INVALID_ARG;
  Space w;
  int64_t row = 0;
  for (int32_t i = 0; i < n;) {
    i = plan(a, i, n, h_q_len, h_k_len, &row, dev->sms, P.get(), &w);
    if (i < 0) return KVPOOL_ERR_INVALID_ARG;
    most = std::max(most, w.total);
  }
  Run run;
  row = 0;
  for (int32_t i = 0; next_run(a, &i, &row, n, h_q_len, h_k_len, &run);) {
    WindowCall call;
    if (!window_call(a, run, h_q_len, h_k_len, nullptr, &call)) return KVPOOL_ERR_INVALID_ARG;
    call.args.k.data = call.args.v.data = reinterpret_cast<const void*>((uintptr_t)16);  // (sizes only)
    const int64_t x = kvpool_window_workspace(&call.args, run.end - run.first, h_q_len + run.first, call.start.get(),
                                              call.len.get());
    if (x < 0) return x;
    most = std::max(most, 2 * run.bytes + x);
  }
  return most;
}

extern "C" int kvpool_kv4_attend(const kvpool_kv4_args* a, int32_t n, const int64_t* h_q_len, const int64_t* h_k_len,
                                 void* d_workspace, int64_t workspace_bytes, void* stream) {
  using namespace kvp;
  int64_t total = 0;
  const int bad = check_args(a, n, h_q_len, h_k_len, &total);
  if (bad != KVPOOL_OK || total == 0) return bad;
  if (!rows_same(a->out, a->q, total) &&
      rows_meet(a->out, total, a->q, total, a->cache.head_dim, a->dtype == KVPOOL_BF16 ? 2 : 4))
    return KVPOOL_ERR_INVALID_ARG;
  const int64_t need = kvpool_kv4_workspace(a, n, h_q_len, h_k_len);
  if (need < 0) return (int)need;
  if (need > 0 && (!d_workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(d_workspace) % 16 != 0))
    return KVPOOL_ERR_INVALID_ARG;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  std::unique_ptr<Kv4Params> P(new (std::nothrow) Kv4Params);
  if (!P) return KVPOOL_ERR_INVALID_ARG;
  uint8_t* space = static_cast<uint8_t*>(d_workspace);
  P->q = static_cast<const uint8_t*>(a->q.data);
  P->out = static_cast<uint8_t*>(const_cast<void*>(a->out.data));
  P->lse = a->d_lse;
  P->q_tok = a->q.token_stride;
  P->q_head = a->q.head_stride;
  P->o_tok = a->out.token_stride;
  P->o_head = a->out.head_stride;
  P->w_seg = a->weight_stride;
  P->w_head = a->weight_head_stride;
  P->group = a->q.heads / a->cache.kv_heads;
  P->scale_log2 = a->scale * 1.4426950408889634f * a->cache.k_scale;
  P->decay = a->decay;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Space w;
  int64_t row = 0;
  for (int32_t i = 0; i < n;) {
    const int32_t first = i;
    i = plan(a, i, n, h_q_len, h_k_len, &row, dev->sms, P.get(), &w);
    if (P->n_segs == 0) continue;
    P->c = kv4_cache(&a->cache, first, dev->err);
    P->weights = a->d_weights ? a->d_weights + first * a->weight_stride : nullptr;
    P->part_o = reinterpret_cast<float*>(space);
    P->part_ml = reinterpret_cast<float2*>(space + std::max<int64_t>(w.part_ml, 0));
    P->lse2 = a->d_weights ? reinterpret_cast<float*>(space + w.lse2) : nullptr;
    P->scores = a->d_weights ? reinterpret_cast<float*>(space + w.scores) : nullptr;
    const bool cut = w.part_ml >= 0, f32 = a->dtype == KVPOOL_F32;
    const cudaError_t e = a->cache.head_dim == 128 ? (f32 ? launch_all<128, true>(*P, cut, s) : launch_all<128, false>(*P, cut, s))
                                                   : (f32 ? launch_all<64, true>(*P, cut, s) : launch_all<64, false>(*P, cut, s));
    if (e != cudaSuccess) return KVPOOL_ERR_CUDA;
  }
  Run run;
  row = 0;
  for (int32_t i = 0; next_run(a, &i, &row, n, h_q_len, h_k_len, &run);) {
    WindowCall call;
    if (!window_call(a, run, h_q_len, h_k_len, space, &call)) return KVPOOL_ERR_INVALID_ARG;
    const int32_t m = run.end - run.first;
    std::unique_ptr<int64_t[]> zero(new (std::nothrow) int64_t[m]());
    if (!zero) return KVPOOL_ERR_INVALID_ARG;
    int rc = kv4_load_rows(&a->cache, a->dtype, call.args.k, call.args.v, m, run.first, zero.get(), call.len.get(), dev->err,
                           stream);
    if (rc != KVPOOL_OK) return rc;
    rc = kvpool_window_attend(&call.args, m, h_q_len + run.first, call.start.get(), call.len.get(), space + 2 * run.bytes,
                              workspace_bytes - 2 * run.bytes, stream);
    if (rc != KVPOOL_OK) return rc;
  }
  return KVPOOL_OK;
}
