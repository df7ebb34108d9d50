// kvpool_kv4_attend.cu -- attention of a ragged batch over the 4-bit paged
// cache, with the weight that every token got.
//
//   out = sum_t softmax_t(scale <q, k_t>) v_t over t <= p, p the query's place;
//   lse = log sum_t exp(scale <q, k_t>);
//   weights[t] = decay * weights[t] + sum over the key head's query rows of
//   exp(scale <q, k_t> - lse).
//
// Single tokens, drafts and all fp32 queries go through the kernel below; the
// tokens of longer bf16 segments are read back to rows (keys in bf16, values in
// fp16, exact) and go through window attention where that pays.
//
// Bound: reading the cache, 1.125 bytes for a key's and a value's number.  The
// whole list of keys, across segments and heads, is cut into equal shares, one to
// each warp that the GPU holds (16 to a multiprocessor).  A warp has a ring of pairs of tiles (32 tokens, one bulk copy), so that up to
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
//
// Measured (heads of 128): one request behind 1,048,576 tokens of 16 heads 352 us
// for 2.42 GB, 6.9 TB/s (1.01 of the measured copy); an eighth of it 57 us a call,
// 49 inside the kernel.  64 requests of 1 to 16,384 tokens, 16 heads on 4, 69 us
// (311 MB), with the tokens' weights 85 (their scores are 34 MB, written and read
// again); 32 of 1 to 8,192 24 us for 76 MB, of which the kernel takes 16.6, 3.4
// before its first data, and the merging launch after it 5.  A tile takes a warp
// 260 instructions (64 conversions of codes, 64 products with scales, 16 matrix
// instructions); issue slots 54% busy, the integer pipe 49%, the tensor pipe 30%.
// Measured and not kept: a running maximum kept exactly (333 instructions to a
// tile, 465 us for the million tokens); a CTA of four warps to a part of equal
// length (ragged lengths leave 20% of a wave idle: 69 us where shares took 62) or
// several waves of them (68); a CTA's share over several units (the ring drains at
// each: 79 to 101 us); barriers that keep a CTA's warps together; skipping pairs
// that no row of a tile sees (fp32 prompts among their own tokens 81 -> 72 us, but
// the registers it takes cost single tokens 3 to 8%).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <memory>
#include <new>

#include <cuda_runtime.h>

#include "kvpool_fma.cuh"
#include "kvpool_kv4.h"
#include "kvpool_mma.cuh"
#include "kvpool_rows.h"
#include "kvpool_window.h"

namespace kvp {
namespace {

constexpr int kMaxGroup = 16;  // query heads per key head
constexpr int kMaxRows = 64;   // query rows per key head whose weights are summed; bf16 rows that are no prompt
constexpr int kPair = 2;       // tiles of a stage
constexpr float kUp = 6.0f, kMost = 14.0f;  // see the kernel's c

// A launch is one list of pairs of tiles: segments in order, of each its units
// (row tile, key head; heads fastest) in order, of each its keys.  The list is cut
// into equal shares, one to a warp: the end of a unit, whole units, the start of one.
struct Kv4Seg {
  int64_t q_row0;     // first query row
  int64_t score_base; // first score (weights wanted)
  int64_t pair_base;  // first pair of the list
  int32_t q_len, k_len;
  int32_t row_base;   // first of its rows (head, row)
  int32_t key_base;   // first block of keys whose weights are summed
  int32_t table_row;
  int32_t unit_base;  // first unit
};

struct Kv4Params {
  Kv4Cache c;
  const uint8_t* q;
  uint8_t* out;
  float* lse;      // [q_rows][q_heads] or null
  float* weights;  // or null
  int64_t q_tok, q_head, o_tok, o_head;  // strides in values
  int64_t w_seg, w_head;
  int64_t n_pairs, share;  // pairs of the list, of a share (of the first `longer` shares one more)
  int32_t longer, n_shares;
  int32_t n_units, unit_warps;  // unit_warps > 0: a CTA of so many warps takes a whole unit
  int32_t group;
  int32_t tile_rows;  // rows of a row tile
  float scale_log2;   // softmax scale times log2(e) and the keys' scale
  float decay;
  int32_t n_segs, n_rows, n_blocks;  // rows (head, row), blocks of keys whose weights are summed
  int32_t turns;
  float* part_o;    // [share][its first unit, its last][tile_rows][head_dim]
  float2* part_ml;  // [share][2][tile_rows]: (exponent of the weights' unit, sum)
  float* lse2;      // [rows] of whole units, log2 domain (weights wanted)
  float* scores;    // log2 domain (weights wanted)
  Kv4Seg segs[kKv4MaxSegs];
};

// a share's first pair, and the share that has pair x of the list
__device__ __forceinline__ int64_t share_start(const Kv4Params& P, int share) { return share * P.share + min(share, P.longer); }
__device__ __forceinline__ int share_of(const Kv4Params& P, int64_t x) {
  const int64_t y = P.longer * (P.share + 1);
  if (P.n_pairs >> 32) return (int)(x < y ? x / (P.share + 1) : P.longer + (x - y) / P.share);
  const uint32_t d = (uint32_t)P.share + (x < y ? 1 : 0);
  return x < y ? (uint32_t)x / d : P.longer + (uint32_t)(x - y) / d;
}

__device__ __forceinline__ int seg_pairs(const Kv4Seg& S) {
  return max(1, (S.k_len + kPair * kKv4Tile - 1) / (kPair * kKv4Tile));
}

// The shares first .. last that have a part of a unit whose pairs start at x0, and
// where the rows of a share's part lie.
struct Kv4Parts {
  int64_t x0;
  int first, last;
};
__device__ __forceinline__ Kv4Parts parts_of(const Kv4Params& P, const Kv4Seg& S, int unit) {
  if (P.unit_warps > 0) return Kv4Parts{0, 0, 0};  // whole units
  const int pairs = seg_pairs(S);
  const int64_t x0 = S.pair_base + (int64_t)unit * pairs;
  return Kv4Parts{x0, share_of(P, x0), share_of(P, x0 + pairs - 1)};
}
__device__ __forceinline__ int64_t part_row(const Kv4Params& P, const Kv4Parts& u, int share) {
  return (2 * (int64_t)share + (share_start(P, share) < u.x0 ? 1 : 0)) * P.tile_rows;
}

template <typename F>
__device__ __forceinline__ int find_seg(const Kv4Params& P, int64_t x, F base) {
  int lo = 0, hi = P.n_segs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base(P.segs[mid]) <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// a row's log-sum-exp in the log2 domain: -inf where it saw nothing
__device__ __forceinline__ float lse2_of(float unit, float sum) { return sum == 0.0f ? -INFINITY : unit + log2f(sum); }

__device__ __forceinline__ int score_pitch(int k_len) { return (k_len + 3) & ~3; }

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

// four neighbouring values of an output, times inv
template <bool F32>
__device__ __forceinline__ void put4(uint8_t* out, int64_t at, float4 y, float inv) {
  if constexpr (F32)
    *reinterpret_cast<float4*>(out + 4 * at) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
  else
    *reinterpret_cast<uint2*>(out + 2 * at) = make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
}

constexpr int kStages = 3;

// One CTA fills a multiprocessor's registers: 16 warps, or 8 where a warp holds
// more rows or pieces.
__host__ __device__ constexpr int kv4_warps(int NT, bool F32) { return NT == 1 && !F32 ? 16 : 8; }

template <int D>
struct alignas(128) Kv4Smem {  // a warp's
  union {
    uint8_t ring[kStages][kPair * Kv4Tile<D>::kBytes];
    float o[16][D];  // its rows, for the CTA's other warps (once the ring is done with)
  };
  uint64_t bar[kStages];
  float2 ml[16];
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

// NT: tiles of 8 query rows; F32: fp32 queries and outputs; UNIT: a CTA's warps
// share one unit and join their states in shared memory
template <int D, int NT, bool F32, bool UNIT>
__global__ void __launch_bounds__(kv4_warps(NT, F32) * 32, 1) kv4_attend_kernel(const __grid_constant__ Kv4Params P) {
  pdl_launch();
  using L = Kv4Tile<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  Kv4Smem<D>& sm = reinterpret_cast<Kv4Smem<D>*>(smem_raw)[warp];
  constexpr int kPieces = F32 ? 2 : 1;
  constexpr int KS = D / 16;  // steps of 16 dims
  const int share = warp * gridDim.x + blockIdx.x;
  if (!UNIT && share >= P.n_shares) return pdl_wait();
  if (lane < kStages) mbar_init(&sm.bar[lane], 1);
  mbar_fence_init();
  __syncwarp();

  // ---- the ring ----
  int seg, n_my;  // the first pair's segment, pairs
  int64_t x_first;
  if constexpr (UNIT) {
    seg = find_seg(P, blockIdx.x, [](const Kv4Seg& s) { return s.unit_base; });
    const int pairs = seg_pairs(P.segs[seg]), warps = blockDim.x >> 5;
    const int first = (int)((int64_t)pairs * warp / warps);
    n_my = (int)((int64_t)pairs * (warp + 1) / warps) - first;
    x_first = P.segs[seg].pair_base + (int64_t)(blockIdx.x - P.segs[seg].unit_base) * pairs + first;
  } else {
    x_first = share_start(P, share);
    n_my = (int)(share_start(P, share + 1) - x_first);
    seg = find_seg(P, x_first, [](const Kv4Seg& s) { return s.pair_base; });
  }
  auto unit_of = [&](const Kv4Seg& S, int pairs, int64_t x) {
    const int64_t off = x - S.pair_base;
    return off >> 32 ? (int)(off / pairs) : (int)((uint32_t)off / (uint32_t)pairs);
  };
  // Places of 16 of the share's pairs, and of the next 16: lane 2i + j has the one
  // of tile j of pair i.  (-1: no such tile; a bad page, which is flagged: page 0)
  int ahead = seg;
  auto places_from = [&](int i) -> int64_t {
    i += lane >> 1;
    if (i >= n_my) return -1;
    const int64_t x = x_first + i;
    while (ahead + 1 < P.n_segs && P.segs[ahead + 1].pair_base <= x) ++ahead;
    const Kv4Seg& S = P.segs[ahead];
    const int pairs = seg_pairs(S), unit = unit_of(S, pairs, x);
    const int tile = kPair * (int)(x - S.pair_base - (int64_t)unit * pairs) + (lane & 1);
    if (tile * kKv4Tile >= S.k_len) return -1;
    return kv4_tile_offset<D>(P.c, max(kv4_page(P.c, S.table_row, tile), 0), unit % P.c.kv_heads, tile);
  };
  pdl_wait();
  int64_t places = places_from(0), places_next = places_from(16);
  int issued = 0;
  auto issue = [&](int to) {
    if (issued > 0 && (issued & 15) == 0) {
      places = places_next;
      places_next = places_from(issued + 16);
    }
    const int64_t p0 = __shfl_sync(0xffffffffu, places, 2 * (issued & 15));
    const int64_t p1 = __shfl_sync(0xffffffffu, places, 2 * (issued & 15) + 1);
    ++issued;
    if (lane != 0) return;
    uint64_t* mb = &sm.bar[to];
    uint8_t* dst = sm.ring[to];
    if (p0 < 0) {  // a segment without tokens: its scores are all masked
      mbar_arrive(mb);
    } else if (P.c.page_shift > 0) {  // both tiles in one page
      mbar_arrive_expect_tx(mb, kPair * L::kBytes);
      bulk_g2s(dst, P.c.pages + p0, kPair * L::kBytes, mb);
    } else {
      mbar_arrive_expect_tx(mb, (p1 < 0 ? 1 : kPair) * L::kBytes);
      bulk_g2s(dst, P.c.pages + p0, L::kBytes, mb);
      if (p1 >= 0) bulk_g2s(dst + L::kBytes, P.c.pages + p1, L::kBytes, mb);
    }
  };
  while (issued < min(kStages, n_my)) issue(issued);

  int stage = 0, phase = 0;  // of the pair that is read next
  int done = 0;
#pragma unroll 1
  do {  // (a share has a pair at least; a CTA's warp may have none of its unit)
    // ---- a part: the share's keys of a unit ----
    if (!UNIT)
      while (seg + 1 < P.n_segs && P.segs[seg + 1].pair_base <= x_first + done) ++seg;
    const Kv4Seg& S = P.segs[seg];
    const int pairs = seg_pairs(S), unit = UNIT ? blockIdx.x - S.unit_base : unit_of(S, pairs, x_first + done);
    const int a = (int)(x_first + done - S.pair_base - (int64_t)unit * pairs);  // the part's pairs of the unit: a .. b - 1
    const int b = min(pairs, a + (n_my - done));
    const bool first_unit = done == 0, whole_unit = b - a == pairs;
    done += b - a;
    const int n_rows = S.q_len * P.group;
    const int head = unit % P.c.kv_heads, row0 = unit / P.c.kv_heads * P.tile_rows;
    const int rows = min(P.tile_rows, n_rows - row0);
    const int pos0 = S.k_len - S.q_len + row0 / P.group;  // the first row's place

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
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      // an infinity makes NaNs of all the row's scores (an infinite product with keys of one sign might be -inf alone)
      const float down = amax >= 0x7F800000u ? NAN : __uint_as_float((uint32_t)(127 - 14 + e) << 23);
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
#pragma unroll 1
    for (int i = a; i < b; ++i) {
      if (!warp_wait(&sm.bar[stage], phase, P.c.err)) {  // (flagged) the copies on their way, then the end
        for (int j = done - b + i + 1; j < issued; ++j) {
          if (++stage == kStages) stage = 0, phase ^= 1;
          warp_wait(&sm.bar[stage], phase, P.c.err);
        }
        if (!UNIT) return;
        break;
      }
      const uint8_t* ring = sm.ring[stage];
      const int u0 = i * kPair * kKv4Tile;
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
      if (issued < n_my) issue(stage);
      if (++stage == kStages) stage = 0, phase ^= 1;
    }

    // ---- the part's rows: dims D / 8 * g and on of rows 8n + 2t, + 1 ----
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const float m = sum == 0.0f ? -INFINITY : -c[n][e];  // the exponent of the weights' unit
        const int row = 8 * n + 2 * t + e, gr = row0 + row;
        float y[D / 8];
#pragma unroll
        for (int x = 0; x < D / 16; ++x) y[2 * x] = o[n][x][e], y[2 * x + 1] = o[n][x][2 + e];
        if constexpr (UNIT) {
#pragma unroll
          for (int x = 0; x < D / 8; x += 4)
            *reinterpret_cast<float4*>(&sm.o[row][L::kChunk * g + x]) = make_float4(y[x], y[x + 1], y[x + 2], y[x + 3]);
          if (g == 0) sm.ml[row] = make_float2(m, sum);
          continue;
        }
        if (row >= rows) continue;
        if (!whole_unit) {
          const int64_t pr = (2 * (int64_t)share + (first_unit ? 0 : 1)) * P.tile_rows + row;
#pragma unroll
          for (int x = 0; x < D / 8; x += 4)
            *reinterpret_cast<float4*>(P.part_o + pr * D + L::kChunk * g + x) = make_float4(y[x], y[x + 1], y[x + 2], y[x + 3]);
          if (g == 0) P.part_ml[pr] = make_float2(m, sum);
          continue;
        }
        const float inv = sum > 0.0f ? P.c.v_scale / sum : sum == 0.0f ? 0.0f : sum;  // (a NaN stays one)
        const int64_t tok = S.q_row0 + gr / P.group;
        const int h = head * P.group + gr % P.group;
        const int64_t at = tok * P.o_tok + h * P.o_head + L::kChunk * g;
#pragma unroll
        for (int x = 0; x < D / 8; x += 8) {
          if constexpr (F32) {
            *reinterpret_cast<float4*>(P.out + 4 * (at + x)) =
                make_float4(y[x] * inv, y[x + 1] * inv, y[x + 2] * inv, y[x + 3] * inv);
            *reinterpret_cast<float4*>(P.out + 4 * (at + x + 4)) =
                make_float4(y[x + 4] * inv, y[x + 5] * inv, y[x + 6] * inv, y[x + 7] * inv);
          } else {
            *reinterpret_cast<uint4*>(P.out + 2 * (at + x)) =
                make_uint4(pack_bf16(y[x] * inv, y[x + 1] * inv), pack_bf16(y[x + 2] * inv, y[x + 3] * inv),
                           pack_bf16(y[x + 4] * inv, y[x + 5] * inv), pack_bf16(y[x + 6] * inv, y[x + 7] * inv));
          }
        }
        if (g == 0) {
          const float z = lse2_of(m, sum);
          if (P.lse) P.lse[tok * (P.c.kv_heads * P.group) + h] = z * 0.69314718055994531f;
          if (P.lse2) P.lse2[S.row_base + head * n_rows + gr] = z;
        }
      }
    if constexpr (UNIT) {
      __syncthreads();
      const Kv4Smem<D>* all = reinterpret_cast<const Kv4Smem<D>*>(smem_raw);
      const int warps = blockDim.x >> 5;
      for (int i = threadIdx.x; i < rows * (D / 4); i += blockDim.x) {
        const int row = i / (D / 4), x = 4 * (i % (D / 4)), gr = row0 + row;
        float mx = -INFINITY;
        for (int k = 0; k < warps; ++k) mx = fmaxf(mx, all[k].ml[row].x);
        const float base = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < warps; ++k) {
          const float2 ml = all[k].ml[row];
          const float f = ex2f(ml.x - base);
          const float4 z = *reinterpret_cast<const float4*>(&all[k].o[row][x]);
          sum = fmaf(ml.y, f, sum);
          y.x = fmaf(z.x, f, y.x), y.y = fmaf(z.y, f, y.y), y.z = fmaf(z.z, f, y.z), y.w = fmaf(z.w, f, y.w);
        }
        const float inv = sum > 0.0f ? P.c.v_scale / sum : sum == 0.0f ? 0.0f : sum;  // (a NaN stays one)
        const int64_t tok = S.q_row0 + gr / P.group;
        const int h = head * P.group + gr % P.group;
        const int64_t at = tok * P.o_tok + h * P.o_head + x;
        put4<F32>(P.out, at, y, inv);
        if (x == 0) {
          const float z = lse2_of(mx, sum);
          if (P.lse) P.lse[tok * (P.c.kv_heads * P.group) + h] = z * 0.69314718055994531f;
          if (P.lse2) P.lse2[S.row_base + head * n_rows + gr] = z;
        }
      }
    }
  } while (!UNIT && done < n_my);
}

// What is left once every part is done, in one launch.  The first CTAs merge the
// rows (head, row) of segments whose keys were cut: out = sum_s
// 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.  The others sum the
// weights of kWeightKeys keys of a segment and head, rows in order (the same sums
// on every run), from the rows' log-sum-exps, which each works out of the parts'
// (unit, sum)s; a row that saw nothing gives none.
constexpr int kFinishThreads = 512;  // at most (of a merging CTA)
constexpr int kWeightThreads = 128, kWeightKeys = 4 * kWeightThreads;

// the state (unit, sum, outputs) of `from` joins the one of `to`
__device__ __forceinline__ void join_state(float& m, float& l, float4& o, float fm, float fl, float4 fo) {
  const float mx = fmaxf(m, fm), base = mx == -INFINITY ? 0.0f : mx;
  const float a = ex2f(m - base), b = ex2f(fm - base);
  m = mx;
  l = l * a + fl * b;
  o = make_float4(o.x * a + fo.x * b, o.y * a + fo.y * b, o.z * a + fo.z * b, o.w * a + fo.w * b);
}

// `slices` groups of D / 4 threads merge row `id`, each every slices-th part: one
// group of a CTA's several, or the whole CTA.
template <int D, bool F32>
__device__ void kv4_merge_row(const Kv4Params& P, int id, int slices) {
  constexpr int kLanes = D / 4, kMost = kFinishThreads / kLanes, kAtOnce = 8;
  __shared__ float4 so[kMost][kLanes];
  __shared__ float2 sml[kMost];
  const int slice = slices > 1 ? threadIdx.x / kLanes : 0, lane = threadIdx.x % kLanes;
  const int seg = find_seg(P, id, [](const Kv4Seg& s) { return s.row_base; });
  const Kv4Seg& S = P.segs[seg];
  const int n_rows = S.q_len * P.group;
  const int head = (id - S.row_base) / n_rows, gr = (id - S.row_base) % n_rows;
  const Kv4Parts u = parts_of(P, S, gr / P.tile_rows * P.c.kv_heads + head);
  pdl_wait();
  if (u.first == u.last) return;  // the unit's warp wrote the outputs
  float m = -INFINITY, l = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = u.first + slice; c0 <= u.last; c0 += kAtOnce * slices) {
    float2 ml[kAtOnce];
    float4 o[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int c = c0 + i * slices;
      ml[i] = make_float2(-INFINITY, 0.0f);
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c > u.last) continue;
      const int64_t r = part_row(P, u, c) + gr % P.tile_rows;
      ml[i] = P.part_ml[r];
      o[i] = *reinterpret_cast<const float4*>(P.part_o + r * D + 4 * lane);
    }
    float mx = m;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) mx = fmaxf(mx, ml[i].x);
    const float base = mx == -INFINITY ? 0.0f : mx, f = ex2f(m - base);
    m = mx;
    l *= f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float g = ex2f(ml[i].x - base);
      l = fmaf(ml[i].y, g, l);
      acc = make_float4(fmaf(o[i].x, g, acc.x), fmaf(o[i].y, g, acc.y), fmaf(o[i].z, g, acc.z), fmaf(o[i].w, g, acc.w));
    }
  }
  if (slices > 1) {
    so[slice][lane] = acc;
    if (lane == 0) sml[slice] = make_float2(m, l);
    __syncthreads();
    if (slice != 0) return;
    for (int i = 1; i < slices; ++i) join_state(m, l, acc, sml[i].x, sml[i].y, so[i][lane]);
  }
  const float inv = l > 0.0f ? P.c.v_scale / l : l == 0.0f ? 0.0f : l;
  const int64_t tok = S.q_row0 + gr / P.group;
  const int h = head * P.group + gr % P.group;
  const int64_t at = tok * P.o_tok + h * P.o_head + 4 * lane;
  put4<F32>(P.out, at, acc, inv);
  if (lane == 0 && P.lse) P.lse[tok * (P.c.kv_heads * P.group) + h] = lse2_of(m, l) * 0.69314718055994531f;
}

// The weights of P.turns * kWeightKeys keys, by kWeightThreads threads.
__device__ void kv4_weights_block(const Kv4Params& P, int block) {
  __shared__ float z[kMaxRows];  // the rows' log-sum-exps, log2 domain
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = find_seg(P, block, [](const Kv4Seg& s) { return s.key_base; });
  const Kv4Seg& S = P.segs[seg];
  const int r = block - S.key_base, head = r % P.c.kv_heads;
  const int t0 = r / P.c.kv_heads * (P.turns * kWeightKeys) + 4 * threadIdx.x;  // and kWeightKeys on, `turns` times
  const int n_rows = S.q_len * P.group, pitch = score_pitch(S.k_len);
  const float* s = P.scores + S.score_base + (int64_t)head * n_rows * pitch + t0;
  pdl_wait();
  // the first rows' scores of two turns are on their way while the sums are worked out
  float4 x[2][4];
  auto load = [&](int turn, int i0) {
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = kWeightKeys * (turn + y);
        if (turn + y < P.turns && t0 + at < S.k_len && i0 + i < n_rows) x[y][i] = *reinterpret_cast<const float4*>(s + at + (int64_t)(i0 + i) * pitch);
      }
  };
  load(0, 0);
  for (int row = warp; row < n_rows; row += kWeightThreads / 32) {
    const Kv4Parts u = parts_of(P, S, row / P.tile_rows * P.c.kv_heads + head);
    if (u.first == u.last) {
      if (lane == 0) z[row] = P.lse2[S.row_base + head * n_rows + row];
      continue;
    }
    float m = -INFINITY, l = 0.0f;
    for (int c = u.first + lane; c <= u.last; c += 32) {
      const float2 y = P.part_ml[part_row(P, u, c) + row % P.tile_rows];
      const float mx = fmaxf(m, y.x), base = mx == -INFINITY ? 0.0f : mx;
      l = l * ex2f(m - base) + y.y * ex2f(y.x - base);
      m = mx;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float fm = __shfl_xor_sync(0xffffffffu, m, off), fl = __shfl_xor_sync(0xffffffffu, l, off);
      const float mx = fmaxf(m, fm), base = mx == -INFINITY ? 0.0f : mx;
      // (both lanes of a pair add the same two terms: in the same order)
      const float a = l * ex2f(m - base), b = fl * ex2f(fm - base);
      l = a + b;
      m = mx;
    }
    if (lane == 0) z[row] = lse2_of(m, l);
  }
  __syncthreads();
  float* out = P.weights + S.table_row * P.w_seg + head * P.w_head + t0;
#pragma unroll 1
  for (int turn = 0; turn < P.turns && t0 + kWeightKeys * turn < S.k_len; turn += 2) {
    float w[2][4] = {};
#pragma unroll 1
    for (int i0 = 0; i0 < n_rows; i0 += 4) {
      if (turn > 0 || i0 > 0) load(turn, i0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i0 + i >= n_rows || z[i0 + i] == -INFINITY) continue;
        const float lse = z[i0 + i];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          w[y][0] += ex2f(x[y][i].x - lse);
          w[y][1] += ex2f(x[y][i].y - lse);
          w[y][2] += ex2f(x[y][i].z - lse);
          w[y][3] += ex2f(x[y][i].w - lse);
        }
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = kWeightKeys * (turn + y) + i;
        if (turn + y < P.turns && t0 + at < S.k_len) out[at] = P.decay == 0.0f ? w[y][i] : fmaf(P.decay, out[at], w[y][i]);
      }
  }
}

template <int D, bool F32>
__global__ void __launch_bounds__(kFinishThreads) kv4_finish_kernel(const __grid_constant__ Kv4Params P, int n_merge, int slices) {
  pdl_launch();  // (the wait follows in both parts)
  if ((int)blockIdx.x >= n_merge) return kv4_weights_block(P, blockIdx.x - n_merge);
  if (slices > 1) return kv4_merge_row<D, F32>(P, blockIdx.x, slices);  // (the whole CTA)
  const int id = blockIdx.x * (kWeightThreads / (D / 4)) + threadIdx.x / (D / 4);
  if (id < P.n_rows) kv4_merge_row<D, F32>(P, id, 1);
  else pdl_wait();
}

// ---- host -------------------------------------------------------------------
int64_t group_rows(const kvpool_kv4_args* a, int64_t q_len) { return q_len * (a->q.heads / a->cache.kv_heads); }

// Rows that tokens are read back to: a token's heads one after the other.
kvpool_heads read_back_rows(const kvpool_kv4_args* a, void* space) {
  const int32_t d = a->cache.head_dim, hk = a->cache.kv_heads;
  return kvpool_heads{space, (int64_t)hk * d, d, hk, 0};
}

// Do segments of more than kMaxRows bf16 rows to a key head go through window
// attention (5th-generation products, after reading their tokens back)?  Its
// launches take 10 to 20 us before the first product; the kernel above takes 1.8
// us for every 1,216 pairs of tiles and 16 rows beside 8.  (200 queries of 16 heads
// on 4 among their own 200 tokens 9.3 us here and 17.0 there, 1,024 among theirs
// 61 and 27, 2 x 128 behind 8,000 tokens 83 and 36.)  fp32 rows never do: window
// attention's FMAs take 2.3 to 5.6 times as long (1,024 queries among their own
// tokens 189 us and 81, 256 behind 16,384 1,421 and 253).
//
// Nor do calls whose scale or strides its tensor-core form does not take (a scale
// that is not positive, queries alike over an axis: 300 queries of 8 heads on 2
// behind 6,000 tokens 191 us by its multiply-adds, 25 here), and
// segments without tokens have nothing to read back.
bool prompts_pay(const kvpool_kv4_args* a, int32_t n, const int64_t* q_len, const int64_t* k_len) {
  if (a->dtype == KVPOOL_F32) return false;
  double pairs = 0;
  for (int32_t i = 0; i < n; ++i)
    if (group_rows(a, q_len[i]) > kMaxRows && k_len[i] > 0)
      pairs += (double)((group_rows(a, q_len[i]) + 15) / 16) * a->cache.kv_heads * (double)(k_len[i] / (kPair * kKv4Tile) + 1);
  if (!(pairs > 8192)) return false;
  kvpool_window_args w{};
  w.dtype = a->dtype;
  w.scale = a->scale;
  w.q = a->q;
  w.q_rows = a->q_rows;
  w.k = w.v = read_back_rows(a, nullptr);
  return window_tc_able(&w);
}
bool is_prompt(const kvpool_kv4_args* a, bool prompts, int64_t q_len, int64_t k_len) {
  return prompts && group_rows(a, q_len) > kMaxRows && k_len > 0;
}

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
    if (a->d_weights && group_rows(a, q_len[i]) > kMaxRows) return KVPOOL_ERR_INVALID_ARG;
    q += q_len[i];
    most = std::max(most, k_len[i]);
    keys |= k_len[i] > 0;
  }
  if (q > a->q_rows) return KVPOOL_ERR_INVALID_ARG;
  if (q > 0 && (!a->q.data || !a->out.data)) return KVPOOL_ERR_INVALID_ARG;
  if (keys && (!a->cache.d_pages || !a->cache.d_table || a->cache.n_pages < 1)) return KVPOOL_ERR_INVALID_ARG;
  if (a->d_weights && (reinterpret_cast<uintptr_t>(a->d_weights) % 4 != 0 || a->weight_stride < 0 || a->weight_head_stride < 0 ||
                       !runs_apart(n, a->weight_stride, hk, a->weight_head_stride, most)))
    return KVPOOL_ERR_INVALID_ARG;
  *total_q = q;
  return KVPOOL_OK;
}

constexpr int64_t kMinPairs = 2;  // of a share
// The most pairs of a bf16 share or of a warp's part of a unit, and the rounds of
// shares that this may take: the tensor core cuts its running sums of outputs off,
// up to 2^-23 of the sum at every tile.  (One share to a warp left outputs 0.11% too
// small for 1,500 requests behind the same 1,048,576 tokens, 8 heads on 2, and 0.033%
// for 160 requests, 16 heads on 4; these 0.013% there.  15.8 -> 13.6 ms for those, 5.42
// -> 5.48 for 64 of them.  fp32 outputs are summed with rounding.)
constexpr int64_t kMaxPairs = 1024, kMaxRounds = 16;

// Where a launch's workspace lies, in bytes from its start.
struct Space {
  int64_t part_ml, lse2, scores, total;
};

// Which form is the quicker one: a CTA of 4, 8 or 16 warps for every unit (no
// merging launch; the answer), or equal shares (0).  Times in us, fitted to 34
// batches of equal and of ragged lengths, of 16 to 524,288 tokens: a round (one
// pair to each warp of a multiprocessor) takes 0.55 us and 1/16 more for each
// warp, a wave of unit CTAs 3.5 beside its rounds, shares 8.5 and up to 0.004 for
// every row to merge.  (152 requests of 256 tokens, 4 key heads: 8.9 us as units,
// 13.9 as shares; 32 of 4,096 18.7 and 22.2; 256 of 1 to 2,048 43.6 and 51; 32 of
// 1 to 8,192 30.4 and 23.2; one of 16,384 55 and 12.4.)  The batches were of 16 bf16
// heads on 4 of 128; with heads of 64, fp32, 16 heads on one and 4 on 4, ten batches
// each, the rule's form is the quickest or within 5% of it, but for three (11 to 15%).
int unit_warps(int64_t units, int64_t most_pairs, int64_t pairs, int64_t rows, int64_t shares, int n_sms, int64_t warps_per_sm, bool f32) {
  auto round_us = [](double warps) { return 0.55 + 0.0625 * warps; };
  const double rounds = (double)pairs / (double)shares;
  double best = 8.5 + rounds * round_us(std::min((double)warps_per_sm, (double)shares / n_sms) + 3.0) +
                0.004 * (double)rows * std::min(1.0, rounds / 8);
  int answer = 0;
  for (int w = 4; w <= warps_per_sm; w *= 2) {
    if (!f32 && most_pairs > w * kMaxPairs) continue;
    const double waves = (double)units * w / (double)(n_sms * warps_per_sm);
    const double round = round_us((double)std::min<int64_t>(warps_per_sm, (units + n_sms - 1) / n_sms * w));
    const double longest = (double)((most_pairs + w - 1) / w) * round + 3.5, mean = (double)pairs / (double)units / w * round + 3.5;
    const double t = 0.5 + (waves > 1.0 ? waves * mean + 0.5 * longest : longest);
    if (t < best) best = t, answer = w;
  }
  return answer;
}

// Segments [i0, n) of one launch (at most kKv4MaxSegs that are no prompts);
// returns the next segment, or -1 (too large for one launch).
int32_t plan(const kvpool_kv4_args* a, bool prompts, int32_t i0, int32_t n, const int64_t* q_len, const int64_t* k_len, int64_t* q_row,
             int n_sms, Kv4Params* P, Space* w) {
  const int hk = a->cache.kv_heads, group = a->q.heads / hk;
  int32_t i = i0;
  int64_t row = *q_row, most_rows = 0, rows = 0, blocks = 0, scores = 0;
  P->n_segs = 0;
  for (; i < n && P->n_segs < kKv4MaxSegs; ++i) {
    if (q_len[i] > 0 && !is_prompt(a, prompts, q_len[i], k_len[i])) {
      Kv4Seg& S = P->segs[P->n_segs++];
      S.q_row0 = row;
      S.q_len = (int32_t)q_len[i];
      S.k_len = (int32_t)k_len[i];
      S.table_row = i - i0;
      S.row_base = (int32_t)rows;
      S.score_base = scores;
      most_rows = std::max(most_rows, q_len[i] * group);
      rows += q_len[i] * group * hk;
      if (a->d_weights) {
        blocks += (k_len[i] + kWeightKeys - 1) / kWeightKeys * hk;  // of one turn
        scores += q_len[i] * group * hk * ((k_len[i] + 3) & ~3);
      }
    }
    row += q_len[i];
  }
  if (rows + blocks > (1 << 30)) return -1;
  *q_row = row;
  // a block's row sums are worth several turns where there are many keys (64 requests 19.5 us -> 16 with four)
  P->turns = blocks >= 16LL * n_sms ? 4 : blocks >= 8LL * n_sms ? 2 : 1;
  blocks = 0;
  for (int s = 0; a->d_weights && s < P->n_segs; ++s) {
    P->segs[s].key_base = (int32_t)blocks;
    blocks += (P->segs[s].k_len + (int64_t)P->turns * kWeightKeys - 1) / (P->turns * kWeightKeys) * hk;
  }
  P->tile_rows = most_rows <= 8 ? 8 : 16;
  P->n_pairs = 0;
  int64_t n_units = 0;
  int most = 1;
  for (int s = 0; s < P->n_segs; ++s) {
    Kv4Seg& S = P->segs[s];
    S.pair_base = P->n_pairs;
    S.unit_base = (int32_t)n_units;
    const int units = (S.q_len * group + P->tile_rows - 1) / P->tile_rows * hk;
    const int pairs = std::max(1, (S.k_len + kPair * kKv4Tile - 1) / (kPair * kKv4Tile));
    n_units += units;
    most = std::max(most, pairs);
    P->n_pairs += (int64_t)units * pairs;
  }
  P->n_units = (int32_t)n_units;
  // a share to each warp that the GPU holds, of kMinPairs pairs at least, or several
  const bool f32 = a->dtype == KVPOOL_F32;
  const int64_t warps = (int64_t)n_sms * kv4_warps(P->tile_rows / 8, f32);
  const int64_t shares = std::max<int64_t>(1, std::min(warps, P->n_pairs / kMinPairs));
  const int64_t rounds = f32 ? 1 : std::min(kMaxRounds, std::max<int64_t>(1, (P->n_pairs / shares + kMaxPairs - 1) / kMaxPairs));
  P->n_shares = (int32_t)(shares * rounds);
  P->share = P->n_pairs / P->n_shares;
  if (P->share > (1 << 30)) return -1;
  P->longer = (int32_t)(P->n_pairs % P->n_shares);
  P->unit_warps = unit_warps(P->n_units, most, P->n_pairs, rows, shares, n_sms, warps / n_sms, f32);
  P->n_rows = (int32_t)rows;
  P->n_blocks = (int32_t)blocks;
  const int64_t parts = P->unit_warps == 0 && P->n_shares > 1 ? 2 * (int64_t)P->n_shares * P->tile_rows : 0;
  w->part_ml = parts * a->cache.head_dim * 4;
  w->lse2 = w->part_ml + parts * 8;
  w->scores = w->lse2 + (a->d_weights ? (rows * 4 + 15) / 16 * 16 : 0);
  w->total = w->scores + 4 * scores;
  return i;
}

// The prompts: runs of segments that are prompts (or have no queries), whose
// tokens are read back to rows of 16-bit numbers.  A run's rows take up to kRunBytes of the
// workspace; a segment of more tokens is a run by itself, taken in pieces: of so
// many keys, and of queries whose running states take up to kStateBytes.  Measured
// with 2^26, 2^28, 2^29, 2^30 and 2^31 bytes of rows, and all at once: 1,024 queries
// of 16 heads behind 1,048,576 tokens 10.7, 8.7, 8.0, 7.6, 7.5 and 7.4 ms (8.6 GB of
// rows); 64 drafts of 5 tokens, 64 heads on 4, behind 65,536 6.2, 3.8, 3.5, 3.3, 3.1
// and 3.1 ms (8.6 GB); 8 x 512 queries, 16 heads on 8, behind 131,072 5.2, 4.7, 4.2,
// 3.7, 3.8 and 4.0 ms (4.3 GB).
constexpr int64_t kRunBytes = 1ll << 31, kStateBytes = 1ll << 26;
int64_t token_bytes(const kvpool_kv4_args* a) { return 4LL * a->cache.kv_heads * a->cache.head_dim; }  // of a key's and a value's rows

struct Run {
  int32_t first, end;
  int64_t q_row, q_rows, kv_rows;
};
bool next_run(const kvpool_kv4_args* a, bool prompts, int32_t* i, int64_t* q_row, int32_t n, const int64_t* q_len, const int64_t* k_len,
              Run* run) {
  while (*i < n && (q_len[*i] == 0 || !is_prompt(a, prompts, q_len[*i], k_len[*i]))) *q_row += q_len[(*i)++];
  if (*i >= n) return false;
  *run = Run{*i, *i, *q_row, 0, 0};
  for (; *i < n && (q_len[*i] == 0 || is_prompt(a, prompts, q_len[*i], k_len[*i])); ++*i) {
    const int64_t keys = q_len[*i] > 0 ? k_len[*i] : 0;
    if (run->kv_rows > 0 && (run->kv_rows + keys) * token_bytes(a) > kRunBytes) break;
    run->q_rows += q_len[*i];
    run->kv_rows += keys;
  }
  *q_row += run->q_rows;
  run->end = *i;
  return true;
}

// A run's workspace: keys' rows, values' rows, states of a segment in pieces, and
// what window attention asks for.
struct RunSpace {
  int64_t rows;           // bytes of the keys' rows
  int64_t state_o, state_ml;
  int64_t queries, keys;  // the most of a piece (0: no pieces)
  int64_t window() const { return 2 * rows + state_o + state_ml; }  // where that starts
};
RunSpace run_space(const kvpool_kv4_args* a, const Run& run, const int64_t* q_len, const int64_t* k_len) {
  RunSpace s{};
  s.rows = run.kv_rows * token_bytes(a) / 2;
  if (2 * s.rows <= kRunBytes) return s;
  const int64_t tile = 2 * (kTcTileRows / (a->q.heads / a->cache.kv_heads));
  const int64_t state = (int64_t)a->q.heads * (a->cache.head_dim + 2) * 4;
  const int64_t most = kStateBytes / state;
  s.queries = std::min(q_len[run.first], most < tile ? most : most / tile * tile);
  s.keys = kRunBytes / token_bytes(a) / 128 * 128;
  s.rows = s.keys * token_bytes(a) / 2;
  s.state_o = s.queries * a->q.heads * a->cache.head_dim * 4;
  s.state_ml = (s.queries * a->q.heads * 8 + 15) / 16 * 16;
  return s;
}

// The window call of query rows `row` .. row + queries - 1 over `keys` rows read
// back: everything up to the query is visible.
kvpool_window_args window_call(const kvpool_kv4_args* a, const RunSpace& s, uint8_t* space, int64_t row, int64_t queries, int64_t keys) {
  kvpool_window_args x{};
  x.dtype = a->dtype;
  x.head_dim = a->cache.head_dim;
  x.q = a->q;
  x.out = a->out;
  x.q.data = static_cast<const uint8_t*>(a->q.data) + 2 * row * a->q.token_stride;
  x.out.data = static_cast<const uint8_t*>(a->out.data) + 2 * row * a->out.token_stride;
  x.k = read_back_rows(a, space);
  x.v = read_back_rows(a, space + s.rows);
  x.q_rows = queries;
  x.kv_rows = keys;
  x.d_lse = a->d_lse ? a->d_lse + row * a->q.heads : nullptr;
  x.window = 1 << 30;
  x.scale = a->scale;
  return x;
}

// Call f(first query, queries, first key, keys, dense) for every piece of a
// segment, in order; it returns a KVPOOL_ code, of which the first that is none ends this.
template <typename F>
int each_piece(const RunSpace& s, int64_t q_len, int64_t k_len, F f) {
  for (int64_t q0 = 0; q0 < q_len; q0 += s.queries) {
    const int64_t nq = std::min(s.queries, q_len - q0), last = k_len - q_len + q0 + nq;  // keys up to the last query
    const int64_t keys = std::max<int64_t>(1, last);  // (queries at places below 0 see none of one key)
    for (int64_t k0 = 0; k0 < keys; k0 += s.keys) {
      const int64_t nk = std::min(s.keys, keys - k0);
      WinDense d;
      d.pieces = true;
      d.begin = k0 == 0;
      d.end = k0 + nk == keys;
      d.behind = last - (k0 + nk);
      const int rc = f(q0, nq, k0, nk, d);
      if (rc != KVPOOL_OK) return rc;
    }
  }
  return KVPOOL_OK;
}

// The segments of a run as window attention takes them: keys read back, one after the other.
struct RunKeys {
  std::unique_ptr<int64_t[]> start, len, zero;
  bool fill(const Run& run, const int64_t* q_len, const int64_t* k_len) {
    const int32_t n = run.end - run.first;
    start.reset(new (std::nothrow) int64_t[n]);
    len.reset(new (std::nothrow) int64_t[n]);
    zero.reset(new (std::nothrow) int64_t[n]());
    if (!start || !len || !zero) return false;
    int64_t at = 0;
    for (int32_t i = 0; i < n; ++i) {
      len[i] = q_len[run.first + i] > 0 ? k_len[run.first + i] : 0;
      start[i] = at;
      at += len[i];
    }
    return true;
  }
};

template <int D, int NT, bool F32, bool UNIT>
cudaError_t launch_attend(const Kv4Params& P, int n_sms, cudaStream_t s) {
  constexpr int smem = (int)sizeof(Kv4Smem<D>);  // of a warp
  auto* kern = kv4_attend_kernel<D, NT, F32, UNIT>;
  static std::atomic<uint64_t> told;  // the devices (of 64) that know of the kernel's shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !(told.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem * kv4_warps(NT, F32));
    if (e == cudaSuccess) told.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  // neighbouring shares go to different multiprocessors: few of them still use all
  const int held = n_sms * kv4_warps(NT, F32), rounds = (P.n_shares + held - 1) / held;
  const int ctas = UNIT ? P.n_units : std::min(n_sms * rounds, P.n_shares);
  const int warps = UNIT ? P.unit_warps : (P.n_shares + ctas - 1) / ctas;
  return launch_kernel(true, kern, dim3(ctas), dim3(warps * 32), smem * warps, s, P);
}
template <int D, int NT, bool F32>
cudaError_t launch_form(const Kv4Params& P, int n_sms, cudaStream_t s) {
  return P.unit_warps > 0 ? launch_attend<D, NT, F32, true>(P, n_sms, s) : launch_attend<D, NT, F32, false>(P, n_sms, s);
}

template <int D, bool F32>
cudaError_t launch_all(const Kv4Params& P, int n_sms, cudaStream_t s) {
  cudaError_t e = P.tile_rows == 8 ? launch_form<D, 1, F32>(P, n_sms, s) : launch_form<D, 2, F32>(P, n_sms, s);
  const bool parts = P.unit_warps == 0 && P.n_shares > 1;
  auto* kern = kv4_finish_kernel<D, F32>;
  int n_merge = 0;
  // A row of a unit in n parts takes n / slices / 8 loads' latencies: rows of few parts, or too many rows for one
  // wave of CTAs, go four or eight to a CTA, others take a CTA of 128 or 512 threads each (512 rows of 19 parts: 28.5
  // us a call with 512 threads, 23.5 with 128)
  constexpr int kRows = kWeightThreads / (D / 4);  // or slices of 128 threads
  int slices = 1;
  // Where weights are summed as well, one launch for both is worth more until 64 parts (4 requests of 4,000 tokens, 4 key
  // heads: 10.9 us against 15.6); behind them the sides change with the case (16,000 tokens, 150 parts: 25.8 against
  // 22.0 at a head of 128, 16.4 against 17.8 at 64; one request of 60,000: 62 against 34).
  if (parts && P.n_shares / (P.n_blocks > 0 ? 64 : 16) >= P.n_units && P.n_rows <= n_sms) {
    if (e == cudaSuccess)
      e = launch_kernel(true, kern, dim3(P.n_rows), dim3(kFinishThreads), 0, s, P, P.n_rows, kFinishThreads / (D / 4));
  } else if (parts) {
    slices = P.n_shares / 6 >= P.n_units && P.n_rows <= 8 * n_sms ? kRows : 1;
    n_merge = slices > 1 ? P.n_rows : (P.n_rows + kRows - 1) / kRows;
  }
  if (e == cudaSuccess && n_merge + P.n_blocks > 0)
    e = launch_kernel(true, kern, dim3(n_merge + P.n_blocks), dim3(kWeightThreads), 0, s, P, n_merge, slices);
  return e;
}

}  // namespace
}  // namespace kvp

namespace kvp {
namespace {

// Bytes that the call's launches take, one after the other (a negative error code).
int64_t space_of(const kvpool_kv4_args* a, int32_t n, const int64_t* q_len, const int64_t* k_len, int n_sms, Kv4Params* P) {
  const bool prompts = prompts_pay(a, n, q_len, k_len);
  Space w;
  int64_t row = 0, most = 0;
  for (int32_t i = 0; i < n;) {
    i = plan(a, prompts, i, n, q_len, k_len, &row, n_sms, P, &w);
    if (i < 0) return KVPOOL_ERR_INVALID_ARG;
    most = std::max(most, w.total);
  }
  Run run;
  row = 0;
  uint8_t* const none = reinterpret_cast<uint8_t*>((uintptr_t)16);  // (sizes only)
  for (int32_t i = 0; next_run(a, prompts, &i, &row, n, q_len, k_len, &run);) {
    const RunSpace s = run_space(a, run, q_len, k_len);
    int64_t window = 0;
    if (s.queries > 0) {
      const int64_t zero = 0;
      int64_t known[2] = {0, 0};  // (a piece like the one before asks for as much)
      const int rc = each_piece(s, q_len[run.first], k_len[run.first], [&](int64_t q0, int64_t nq, int64_t, int64_t nk, const WinDense& d) {
        if (nq == known[0] && nk == known[1]) return (int)KVPOOL_OK;
        known[0] = nq, known[1] = nk;
        const kvpool_window_args x = window_call(a, s, none, run.q_row + q0, nq, nk);
        const int64_t y = window_space(&x, 1, &nq, &zero, &nk, &d);
        window = std::max(window, y);
        return y < 0 ? (int)y : (int)KVPOOL_OK;
      });
      if (rc != KVPOOL_OK) return rc;
    } else {
      RunKeys keys;
      if (!keys.fill(run, q_len, k_len)) return KVPOOL_ERR_INVALID_ARG;
      const kvpool_window_args x = window_call(a, s, none, run.q_row, run.q_rows, run.kv_rows);
      const WinDense d;
      window = window_space(&x, run.end - run.first, q_len + run.first, keys.start.get(), keys.len.get(), &d);
      if (window < 0) return window;
    }
    most = std::max(most, s.window() + window);
  }
  return most;
}

}  // namespace
}  // namespace kvp

extern "C" int64_t kvpool_kv4_workspace(const kvpool_kv4_args* a, int32_t n, const int64_t* h_q_len, const int64_t* h_k_len) {
  using namespace kvp;
  int64_t total = 0;
  const int rc = check_args(a, n, h_q_len, h_k_len, &total);
  if (rc != KVPOOL_OK) return rc;
  if (total == 0) return 0;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  std::unique_ptr<Kv4Params> P(new (std::nothrow) Kv4Params);
  return P ? space_of(a, n, h_q_len, h_k_len, dev->sms, P.get()) : KVPOOL_ERR_INVALID_ARG;
}

extern "C" int kvpool_kv4_attend(const kvpool_kv4_args* a, int32_t n, const int64_t* h_q_len, const int64_t* h_k_len,
                                 void* d_workspace, int64_t workspace_bytes, void* stream) {
  using namespace kvp;
  int64_t total = 0;
  const int bad = check_args(a, n, h_q_len, h_k_len, &total);
  if (bad != KVPOOL_OK || total == 0) return bad;
  const int64_t vb = a->dtype == KVPOOL_BF16 ? 2 : 4;
  if (!rows_same(a->out, a->q, total) && rows_meet(a->out, total, a->q, total, a->cache.head_dim, vb)) return KVPOOL_ERR_INVALID_ARG;
  if (kv4_meets(&a->cache, a->out, total, vb) || kv4_meets(&a->cache, d_workspace, workspace_bytes)) return KVPOOL_ERR_INVALID_ARG;
  // the log-sum-exps, the weights and (below) the workspace lie apart from all else
  int64_t most = 0;  // places of a segment's weights
  for (int32_t i = 0; a->d_weights && i < n; ++i)
    if (h_q_len[i] > 0) most = std::max(most, h_k_len[i]);
  auto on_rows = [&](const void* p, __int128 bytes) {
    return rows_touch(a->q, total, a->cache.head_dim, vb, p, bytes) || rows_touch(a->out, total, a->cache.head_dim, vb, p, bytes);
  };
  auto on_weights = [&](const void* p, __int128 bytes) {
    return runs_touch(a->d_weights, n, a->weight_stride, a->cache.kv_heads, a->weight_head_stride, most, p, bytes);
  };
  const __int128 lse_bytes = a->d_lse ? (__int128)4 * total * a->q.heads : 0;
  if (kv4_meets(&a->cache, a->d_lse, lse_bytes) || on_rows(a->d_lse, lse_bytes) || on_weights(a->d_lse, lse_bytes) ||
      kv4_meets(&a->cache, a->d_weights, n, a->weight_stride, a->weight_head_stride, most))
    return KVPOOL_ERR_INVALID_ARG;
  for (const kvpool_heads& h : {a->q, a->out})
    if (on_weights(h.data, (__int128)vb * ((__int128)(total - 1) * h.token_stride + (__int128)(h.heads - 1) * h.head_stride + a->cache.head_dim)))
      return KVPOOL_ERR_INVALID_ARG;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  std::unique_ptr<Kv4Params> P(new (std::nothrow) Kv4Params);
  if (!P) return KVPOOL_ERR_INVALID_ARG;
  const bool prompts = prompts_pay(a, n, h_q_len, h_k_len);
  Space w;
  int64_t row = 0;
  const int32_t next = plan(a, prompts, 0, n, h_q_len, h_k_len, &row, dev->sms, P.get(), &w);
  bool whole = next == n;  // one launch is the whole call
  for (int32_t i = 0; whole && i < n; ++i) whole = !is_prompt(a, prompts, h_q_len[i], h_k_len[i]);
  const int64_t need = whole ? w.total : space_of(a, n, h_q_len, h_k_len, dev->sms, P.get());
  if (need < 0) return (int)need;
  if (need > 0 && (!d_workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(d_workspace) % 16 != 0))
    return KVPOOL_ERR_INVALID_ARG;
  const uintptr_t at = reinterpret_cast<uintptr_t>(d_workspace), lse = reinterpret_cast<uintptr_t>(a->d_lse);
  if (need > 0 && (on_rows(d_workspace, need) || on_weights(d_workspace, need) || (lse_bytes > 0 && lse < at + need && at < lse + lse_bytes)))
    return KVPOOL_ERR_INVALID_ARG;
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
  row = 0;
  for (int32_t i = 0; i < n;) {
    const int32_t first = i;
    i = whole ? n : plan(a, prompts, i, n, h_q_len, h_k_len, &row, dev->sms, P.get(), &w);
    if (P->n_segs == 0) continue;
    P->c = kv4_cache(&a->cache, first, dev->err);
    P->weights = a->d_weights ? a->d_weights + first * a->weight_stride : nullptr;
    P->part_o = reinterpret_cast<float*>(space);
    P->part_ml = reinterpret_cast<float2*>(space + w.part_ml);
    P->lse2 = a->d_weights ? reinterpret_cast<float*>(space + w.lse2) : nullptr;
    P->scores = a->d_weights ? reinterpret_cast<float*>(space + w.scores) : nullptr;
    const bool f32 = a->dtype == KVPOOL_F32;
    const cudaError_t e = a->cache.head_dim == 128 ? (f32 ? launch_all<128, true>(*P, dev->sms, s) : launch_all<128, false>(*P, dev->sms, s))
                                                   : (f32 ? launch_all<64, true>(*P, dev->sms, s) : launch_all<64, false>(*P, dev->sms, s));
    if (e != cudaSuccess) return KVPOOL_ERR_CUDA;
  }
  Run run;
  row = 0;
  for (int32_t i = 0; !whole && next_run(a, prompts, &i, &row, n, h_q_len, h_k_len, &run);) {
    const RunSpace r = run_space(a, run, h_q_len, h_k_len);
    // keys and values of m segments from table row `first` on are read back and attended to
    auto part = [&](int32_t first, int32_t m, const int64_t* start, const int64_t* q_len, const int64_t* at, const int64_t* len,
                    const kvpool_window_args& x, WinDense d) {
      d.v_scale = a->cache.v_scale;
      const int rc = kv4_load_rows(&a->cache, x.k, x.v, m, first, start, len, dev->err, stream);
      return rc != KVPOOL_OK ? rc : window_run(&x, m, q_len, at, len, &d, space + r.window(), workspace_bytes - r.window(), stream);
    };
    int rc;
    if (r.queries > 0) {
      const int64_t zero = 0;
      rc = each_piece(r, h_q_len[run.first], h_k_len[run.first], [&](int64_t q0, int64_t nq, int64_t k0, int64_t nk, WinDense d) {
        d.acc_o = reinterpret_cast<float*>(space + 2 * r.rows);
        d.acc_ml = reinterpret_cast<float2*>(space + 2 * r.rows + r.state_o);
        return part(run.first, 1, &k0, &nq, &zero, &nk, window_call(a, r, space, run.q_row + q0, nq, nk), d);
      });
    } else {
      RunKeys keys;
      if (!keys.fill(run, h_q_len, h_k_len)) return KVPOOL_ERR_INVALID_ARG;
      rc = part(run.first, run.end - run.first, keys.zero.get(), h_q_len + run.first, keys.start.get(), keys.len.get(),
                window_call(a, r, space, run.q_row, run.q_rows, run.kv_rows), WinDense{});
    }
    if (rc != KVPOOL_OK) return rc;
  }
  return KVPOOL_OK;
}
