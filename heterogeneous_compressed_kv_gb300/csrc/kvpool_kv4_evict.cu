// kvpool_kv4_evict.cu -- the heaviest tokens of a 4-bit paged cache into other
// pages: of a segment's tokens every key head keeps the first n_sink, the last
// n_recent and of the others the ones of largest weight (ties to the lowest
// place), in their order.
//
// Two kernels.  The first finds what stays: a cluster of CTAs takes the weights of
// one segment and key head, a slice each, which stays in shared memory; four
// passes over 8 bits of an order-keeping integer of the weight narrow the last
// weight that stays (histograms in shared memory, added up over the cluster), a
// count by warp slices gives every slice its first place, and the places go out in
// order.  The second moves the tokens, a warp to two tiles of 16 of them.
//
// Measured: 4 segments of 65,536 to 131,072 tokens x 8 heads of 128 cut to 16,384
// 74 us: 29 the selection (of it 6 the weights' way in, 3.5 and three times 2.9 the
// passes -- cluster barriers and remote sums --, 5 the places' way out), 43 the
// moving (75 MB each way, of which reads fetch whole 64-byte pieces for a token's
// 8 and 16 bytes of scales and every other nibble of its values: about 240 MB in
// all).  16 of 2,048 to 4,096 tokens x 4 heads cut to 1,024 15 us (11 and 4), one
// round of latencies after the other.  One segment of 1,048,576 tokens cut to 16,384,
// whose slices do not fit shared memory (every pass reads the weights again, 8 CTAs to
// a head): 192 us with 1 head, 223 with 8.
// Measured and not kept: eight histograms of the first pass, one to every eighth
// lane (33.8 us where one took 32.2).
#include <algorithm>
#include <atomic>
#include <memory>
#include <new>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "kvpool_kv4.h"
#include "kvpool_rows.h"

namespace kvp {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxShared = 49152;  // keys of a CTA's slice in shared memory
constexpr int kMoveWarps = 4;

struct EvictSeg {
  int32_t k_len;
  int32_t task_base;  // first task of the moving kernel: tiles * kv_heads + head
  int32_t table_row;  // of the first launch's tables, weights and outputs
};

struct EvictParams {
  Kv4Cache c;  // table: the tokens' places
  const int32_t* out_table;
  int64_t out_stride;
  const float* w;
  float* out_w;   // or null
  int32_t* index; // [segments][kv_heads][keep]
  int64_t w_seg, w_head, ow_seg, ow_head;
  int32_t keep, sink, recent, ow_width;
  int32_t cluster;
  int32_t n_segs, n_tasks;
  EvictSeg segs[kKv4MaxSegs];
};

// A larger weight has a larger key; -0 and +0 are alike and a NaN is the largest.
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0xFFFFFFFFu : score_key(w); }
// the weight again (a NaN for any NaN, +0 for -0)
__device__ __forceinline__ float key_weight(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// SHARED: a CTA's slice of the weights stays in shared memory as keys (up to
// kMaxShared of them), otherwise every pass reads it again.
template <bool SHARED>
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const __grid_constant__ EvictParams P) {
  pdl_start();
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ uint32_t hist[4][256];
  __shared__ uint2 counts[kSelWarps];  // (above the last weight that stays, equal to it) of a warp's slice
  __shared__ uint32_t sh_digit, sh_left;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = P.cluster, rank = blockIdx.x % C, id = blockIdx.x / C;
  const int head = id % P.c.kv_heads;
  const EvictSeg& S = P.segs[id / P.c.kv_heads];
  const int n = S.k_len, keep = P.keep;
  const float* w = P.w + S.table_row * P.w_seg + head * P.w_head;
  float* ow = P.out_w ? P.out_w + S.table_row * P.ow_seg + head * P.ow_head : nullptr;
  int32_t* index = P.index + ((int64_t)S.table_row * P.c.kv_heads + head) * keep;
  const int all = C * kSelThreads, at = rank * kSelThreads + tid;
  // behind what stays: no token, no weight
  const int kept = min(n, keep);
  for (int i = kept + at; i < keep; i += all) index[i] = -1;
  if (ow)
    for (int i = kept + at; i < P.ow_width; i += all) ow[i] = 0.0f;
  if (n <= keep) {
    for (int i = at; i < n; i += all) {
      index[i] = i;
      if (ow) ow[i] = w[i];
    }
    return;  // (the whole cluster)
  }
  // the first and the last tokens stay
  for (int i = at; i < P.sink + P.recent; i += all) {
    const int t = i < P.sink ? i : n - P.recent + (i - P.sink), to = i < P.sink ? i : keep - P.recent + (i - P.sink);
    index[to] = t;
    if (ow) ow[to] = w[t];
  }
  const int lo = P.sink, hi = n - P.recent, want = keep - P.sink - P.recent;  // want < hi - lo
  if (want == 0) return;
  const int warps = C * kSelWarps, per = ((hi - lo + warps - 1) / warps + 127) & ~127;  // a warp's slice
  const int a = min(hi, lo + (rank * kSelWarps + warp) * per), b = min(hi, a + per);
  for (int i = tid; i < 4 * 256; i += kSelThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  // The keys of weights i .. i + 3; 0, which is no weight's, behind the slice.
  uint32_t* slice = keys + warp * per;
  auto keys_at = [&](int i) {
    if constexpr (SHARED) return *reinterpret_cast<const uint4*>(slice + (i - a));
    return make_uint4(i < b ? weight_key(w[i]) : 0u, i + 1 < b ? weight_key(w[i + 1]) : 0u, i + 2 < b ? weight_key(w[i + 2]) : 0u,
                      i + 3 < b ? weight_key(w[i + 3]) : 0u);
  };
  if (SHARED) {
#pragma unroll 1
    for (int i0 = a; i0 < b; i0 += 512) {
      float x[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) x[u] = i0 + 32 * u + lane < b ? w[i0 + 32 * u + lane] : 0.0f;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int i = i0 + 32 * u + lane;
        if (i < a + per) slice[i - a] = i < b ? weight_key(x[u]) : 0u;
      }
    }
    __syncwarp();
  }
  uint32_t prefix = 0, left = want;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
#pragma unroll 2
    for (int i = a + 4 * lane; i < b; i += 128) {
      const uint4 k = keys_at(i);
      const uint32_t key[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (key[u] != 0 && (pass == 0 || key[u] >> (shift + 8) == prefix)) atomicAdd(&hist[pass][key[u] >> shift & 255], 1u);
    }
    cluster.sync();
    // counts from the largest digit down: thread i holds digit 255 - i
    if (tid < 256) {
      uint32_t x = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < C) x += cluster.map_shared_rank(&hist[pass][0], r)[255 - tid];
      uint32_t up = x;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, up, off);
        if (lane >= off) up += y;
      }
      if (lane == 31) counts[warp].x = up;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      for (int k = 0; k < warp; ++k) up += counts[k].x;
      if (up >= left && up - x < left) {  // one thread
        sh_digit = 255 - tid;
        sh_left = left - (up - x);
      }
    }
    __syncthreads();
    prefix = prefix << 8 | sh_digit;
    left = sh_left;
    __syncthreads();
  }
  // `prefix` is the key of the last weight that stays, `left` how many of those equal to it do
  uint2 mine = make_uint2(0, 0);
#pragma unroll 2
  for (int i = a + 4 * lane; i < b; i += 128) {
    const uint4 k = keys_at(i);
    mine.x += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
    mine.y += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
  }
  mine.x = __reduce_add_sync(0xffffffffu, mine.x);
  mine.y = __reduce_add_sync(0xffffffffu, mine.y);
  if (lane == 0) counts[warp] = mine;
  cluster.sync();
  uint32_t above = 0, equal = 0;  // before this warp's slice
  for (int i = lane; i < rank * kSelWarps + warp; i += 32) {
    const uint2 x = cluster.map_shared_rank(&counts[0], i / kSelWarps)[i % kSelWarps];
    above += x.x;
    equal += x.y;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
#pragma unroll 1
  for (int i0 = a; i0 < b; i0 += 128) {
    const int i = i0 + 4 * lane;
    const uint4 k = i < b ? keys_at(i) : make_uint4(0, 0, 0, 0);
    const uint32_t key[4] = {k.x, k.y, k.z, k.w};
    uint32_t here = 0;  // above (low half) and equal (high half)
#pragma unroll
    for (int u = 0; u < 4; ++u) here += (key[u] > prefix ? 1u : 0u) + (key[u] == prefix ? 1u << 16 : 0u);
    uint32_t up = here;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, up, off);
      if (lane >= off) up += y;
    }
    uint32_t n_above = above + ((up - here) & 0xFFFF), n_equal = equal + ((up - here) >> 16);
    const uint32_t total = __shfl_sync(0xffffffffu, up, 31);
    above += total & 0xFFFF;
    equal += total >> 16;
    if (here == 0) continue;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool gt = key[u] > prefix, eq = key[u] == prefix;
      if (gt || (eq && n_equal < left)) {
        const int to = P.sink + n_above + min(n_equal, left);
        index[to] = i + u;
        if (ow) ow[to] = key_weight(key[u]);
      }
      n_above += gt;
      n_equal += eq;
    }
  }
  cluster.sync();  // no CTA ends while another one reads its counts
}

// A warp moves two tiles of 16 tokens of one head, one after the other: their
// places are looked up at once.
constexpr int kMoveTiles = 2;
template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32) kv4_move_kernel(const __grid_constant__ EvictParams P) {
  using L = Kv4Tile<D>;
  const int task = blockIdx.x * kMoveWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (task >= P.n_tasks) return;
  int lo = 0, hi = P.n_segs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.segs[mid].task_base <= task) lo = mid;
    else hi = mid - 1;
  }
  const EvictSeg& S = P.segs[lo];
  const int head = (task - S.task_base) % P.c.kv_heads, tile0 = (task - S.task_base) / P.c.kv_heads * kMoveTiles;
  const int left = min(S.k_len, P.keep) - tile0 * kKv4Tile;  // tokens from there on (at least one)
  Kv4Cache to = P.c;
  to.table = P.out_table;
  to.table_stride = P.out_stride;
  const int to_tile = tile0 + lane / kKv4Tile;
  const int to_id = lane / kKv4Tile * kKv4Tile < left ? kv4_page(to, S.table_row, to_tile) : -1;
  const int64_t to_off = to_id < 0 ? -1 : kv4_tile_offset<D>(P.c, to_id, head, to_tile);
  // lane r: the place of token r of the tiles; a bad page id reads as zeros
  int64_t off = -1;
  int slot = 0;
  if (lane < left) {
    const int t = P.index[((int64_t)S.table_row * P.c.kv_heads + head) * P.keep + tile0 * kKv4Tile + lane];
    slot = t % kKv4Tile;
    const int id = kv4_page(P.c, S.table_row, t / kKv4Tile);
    if (id >= 0) off = kv4_tile_offset<D>(P.c, id, head, t / kKv4Tile);
  }
  const uint8_t* pages = P.c.pages;
#pragma unroll 1
  for (int y0 = 0; y0 < kMoveTiles; ++y0) {
    const int n = min(kKv4Tile, left - y0 * kKv4Tile);
    const int64_t dst_off = __shfl_sync(0xffffffffu, to_off, y0 * kKv4Tile);
    if (dst_off < 0) continue;  // (no such tile, or a bad page: the whole warp)
    uint8_t* dst = P.c.pages + dst_off;
    auto off_of = [&](int r) { return __shfl_sync(0xffffffffu, off, y0 * kKv4Tile + r); };
    auto slot_of = [&](int r) { return __shfl_sync(0xffffffffu, slot, y0 * kKv4Tile + r); };
    // all loads first (nothing that is written is read)
    constexpr int KI = D / 64;  // 16-byte pieces of keys to a lane
    uint4 k[KI];
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int x = i * 32 + lane, r = x / (D / 32), c = x % (D / 32);
      const int64_t o = off_of(r);
      const int sl = slot_of(r);
      k[i] = o >= 0 ? *reinterpret_cast<const uint4*>(pages + o + sl * (D / 2) + 16 * c) : make_uint4(0, 0, 0, 0);
    }
    // scales: of token `lane`'s keys (8 or 4 bytes), of pair `lane`'s values (16 or 8: two tokens' bytes alternate)
    constexpr int G = D / kKv4Group, SW = G / 4;
    uint32_t ks[SW], vs[2 * SW];
    {
      const int64_t o = off_of(lane % kKv4Tile);
      const int sl = slot_of(lane % kKv4Tile);
#pragma unroll
      for (int i = 0; i < SW; ++i) ks[i] = o >= 0 ? reinterpret_cast<const uint32_t*>(pages + o + L::kKs + sl * G)[i] : 0;
    }
    {
      const int j = lane % 8;
      const int64_t o0 = off_of(2 * j), o1 = off_of(2 * j + 1);
      const int s0 = slot_of(2 * j), s1 = slot_of(2 * j + 1);
#pragma unroll
      for (int i = 0; i < 2 * SW; ++i) {
        const uint32_t x = o0 >= 0 ? reinterpret_cast<const uint32_t*>(pages + o0 + L::kVs + (s0 >> 1) * 2 * G)[i] : 0;
        const uint32_t y = o1 >= 0 ? reinterpret_cast<const uint32_t*>(pages + o1 + L::kVs + (s1 >> 1) * 2 * G)[i] : 0;
        vs[i] = (x >> 8 * (s0 & 1) & 0x00FF00FFu) | (y >> 8 * (s1 & 1) & 0x00FF00FFu) << 8;
      }
    }
    constexpr int VW = D / 64;  // 8-byte words of a V chunk
    uint2 v[2][VW];             // pairs lane / 8 and + 4, chunk lane % 8
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = lane / 8 + 4 * i, c = lane % 8;
#pragma unroll
      for (int y = 0; y < VW; ++y) v[i][y] = make_uint2(0, 0);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int64_t o = off_of(2 * j + y);
        const int sl = slot_of(2 * j + y), p = sl >> 1;
        if (o < 0) continue;
        const uint8_t* src = pages + o + L::kV + p * D + (c ^ kv4_swizzle<D>(p)) * L::kChunk;
#pragma unroll
        for (int z = 0; z < VW; ++z) {
          const uint2 x = *reinterpret_cast<const uint2*>(src + 8 * z);
          v[i][z].x |= (x.x >> 4 * (sl & 1) & 0x0F0F0F0Fu) << 4 * y;
          v[i][z].y |= (x.y >> 4 * (sl & 1) & 0x0F0F0F0Fu) << 4 * y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int x = i * 32 + lane, r = x / (D / 32), c = x % (D / 32);
      if (r < n) *reinterpret_cast<uint4*>(dst + r * (D / 2) + 16 * c) = k[i];
    }
    if (lane < n) {
#pragma unroll
      for (int i = 0; i < SW; ++i) reinterpret_cast<uint32_t*>(dst + L::kKs + lane * G)[i] = ks[i];
    }
    if (lane < 8 && 2 * lane < n) {
      uint32_t* p = reinterpret_cast<uint32_t*>(dst + L::kVs + lane * 2 * G);
#pragma unroll
      for (int i = 0; i < 2 * SW; ++i) p[i] = 2 * lane + 1 < n ? vs[i] : (vs[i] & 0x00FF00FFu) | (p[i] & 0xFF00FF00u);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = lane / 8 + 4 * i, c = lane % 8;
      if (2 * j >= n) continue;
      uint2* p = reinterpret_cast<uint2*>(dst + L::kV + j * D + (c ^ kv4_swizzle<D>(j)) * L::kChunk);
#pragma unroll
      for (int z = 0; z < VW; ++z) {
        uint2 x = v[i][z];
        if (2 * j + 1 >= n) {  // the place of the pair's second token stays
          const uint2 old = p[z];
          x = make_uint2((x.x & 0x0F0F0F0Fu) | (old.x & 0xF0F0F0F0u), (x.y & 0x0F0F0F0Fu) | (old.y & 0xF0F0F0F0u));
        }
        p[z] = x;
      }
    }
  }
}

int check_args(const kvpool_kv4_evict_args* a, int32_t n, const int64_t* k_len, int64_t* most) {
  if (!a || n < 0) return KVPOOL_ERR_INVALID_ARG;
  const int rc = kv4_check(&a->cache, n);
  if (rc != KVPOOL_OK) return rc;
  const kvpool_kv4& c = a->cache;
  if (a->keep < 1 || a->keep > (1 << 30) || a->n_sink < 0 || a->n_recent < 0 || a->n_sink > a->keep ||
      a->n_recent > a->keep - a->n_sink)
    return KVPOOL_ERR_INVALID_ARG;
  if (n > 0 && !k_len) return KVPOOL_ERR_INVALID_ARG;
  int64_t len = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (k_len[i] < 0 || k_len[i] > kv4_tokens(&c)) return KVPOOL_ERR_INVALID_ARG;
    len = std::max(len, k_len[i]);
  }
  *most = len;
  if (n == 0) return KVPOOL_OK;
  if (!a->d_index || reinterpret_cast<uintptr_t>(a->d_index) % 4 != 0) return KVPOOL_ERR_INVALID_ARG;
  if (a->out_table_rows < n || a->out_table_stride < 0 || reinterpret_cast<uintptr_t>(a->d_out_table) % 4 != 0 ||
      a->out_table_width < 0 || (int64_t)a->out_table_width * c.page_tokens < std::min<int64_t>(len, a->keep))
    return KVPOOL_ERR_INVALID_ARG;
  if (len > 0 && (!c.d_pages || !c.d_table || c.n_pages < 1 || !a->d_out_table || !a->d_weights)) return KVPOOL_ERR_INVALID_ARG;
  auto strides = [&](const float* p, int64_t seg, int64_t head, int64_t width, bool out) {
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0 || seg < 0 || head < 0 || seg > (1ll << 40) || head > (1ll << 40)) return false;
    if (!out) return true;
    return runs_apart(n, seg, c.kv_heads, head, width);
  };
  if (!strides(a->d_weights, a->weight_stride, a->weight_head_stride, len, false)) return KVPOOL_ERR_INVALID_ARG;
  const __int128 index_bytes = (__int128)4 * n * c.kv_heads * a->keep,
                 out_table_bytes = a->out_table_width > 0 ? 4 * ((__int128)(n - 1) * a->out_table_stride + a->out_table_width) : 0;
  auto touch = [](const void* p, __int128 np, const void* q, __int128 nq) {
    const __int128 x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return p && q && np > 0 && nq > 0 && x < y + nq && y < x + np;
  };
  if (kv4_meets(&c, a->d_index, index_bytes) || touch(a->d_index, index_bytes, a->d_out_table, out_table_bytes) ||
      runs_touch(a->d_weights, n, a->weight_stride, c.kv_heads, a->weight_head_stride, len, a->d_index, index_bytes))
    return KVPOOL_ERR_INVALID_ARG;
  if (a->d_out_weights) {
    if (a->out_weight_width < a->keep ||
        !strides(a->d_out_weights, a->out_weight_stride, a->out_weight_head_stride, a->out_weight_width, true))
      return KVPOOL_ERR_INVALID_ARG;
    auto end = [&](const float* p, int64_t seg, int64_t head, int64_t width) {
      return reinterpret_cast<uintptr_t>(p + (n - 1) * seg + (c.kv_heads - 1) * head + width);
    };
    if (len > 0 && reinterpret_cast<uintptr_t>(a->d_weights) < end(a->d_out_weights, a->out_weight_stride, a->out_weight_head_stride, a->out_weight_width) &&
        reinterpret_cast<uintptr_t>(a->d_out_weights) < end(a->d_weights, a->weight_stride, a->weight_head_stride, len))
      return KVPOOL_ERR_INVALID_ARG;
    auto on = [&](const void* p, __int128 bytes) {
      return runs_touch(a->d_out_weights, n, a->out_weight_stride, c.kv_heads, a->out_weight_head_stride, a->out_weight_width, p, bytes);
    };
    if (kv4_meets(&c, a->d_out_weights, n, a->out_weight_stride, a->out_weight_head_stride, a->out_weight_width) ||
        on(a->d_out_table, out_table_bytes) || on(a->d_index, index_bytes))
      return KVPOOL_ERR_INVALID_ARG;
  }
  return KVPOOL_OK;
}

template <bool SHARED>
cudaError_t launch_select(const EvictParams& P, int64_t slice, cudaStream_t s) {
  auto* kern = kv4_select_kernel<SHARED>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.n_segs * P.c.kv_heads * P.cluster);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  if (SHARED) {
    cfg.dynamicSmemBytes = 4 * slice;
    static std::atomic<uint64_t> told;  // the devices (of 64) that know of the kernel's shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(told.load(std::memory_order_relaxed) >> dev & 1)) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * (int)kMaxShared);
      if (e == cudaSuccess) told.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) return e;
  }
  // not before the kernel ahead has ended: CTAs that wait hold the threads and the
  // shared memory that it needs (a loop of evictions of 4 x 131,072 tokens 87 us a call instead of 79.5; the kernel that moves likewise)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = P.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P);
}

}  // namespace
}  // namespace kvp

extern "C" int kvpool_kv4_evict(const kvpool_kv4_evict_args* a, int32_t n, const int64_t* h_k_len, void* stream) {
  using namespace kvp;
  int64_t most = 0;
  const int rc = check_args(a, n, h_k_len, &most);
  if (rc != KVPOOL_OK || n == 0) return rc;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  std::unique_ptr<EvictParams> P(new (std::nothrow) EvictParams);
  if (!P) return KVPOOL_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int hk = a->cache.kv_heads;
  P->w_seg = a->weight_stride;
  P->w_head = a->weight_head_stride;
  P->ow_seg = a->out_weight_stride;
  P->ow_head = a->out_weight_head_stride;
  P->out_stride = a->out_table_stride;
  P->keep = a->keep;
  P->sink = a->n_sink;
  P->recent = a->n_recent;
  P->ow_width = a->out_weight_width;
  // CTAs to a segment and head: as many as fill the GPU together, of 2,048 weights at least
  P->cluster = 1;
  while (P->cluster < kMaxCluster && (int64_t)std::min(n, kKv4MaxSegs) * hk * P->cluster * 2 <= 2 * dev->sms &&
         most >= 4096 * P->cluster)
    P->cluster *= 2;
  // keys of the longest segment's slice, as the kernel cuts it
  const int64_t warps = (int64_t)P->cluster * kSelWarps, between = std::max<int64_t>(0, most - a->n_sink - a->n_recent);
  const int64_t slice = (((between + warps - 1) / warps + 127) & ~(int64_t)127) * kSelWarps;
  for (int32_t i = 0; i < n;) {
    const int32_t first = i;
    P->n_segs = 0;
    int64_t tasks = 0;
    for (; i < n && P->n_segs < kKv4MaxSegs; ++i) {
      const int64_t tiles = (std::min<int64_t>(h_k_len[i], a->keep) + kMoveTiles * kKv4Tile - 1) / (kMoveTiles * kKv4Tile);
      if (tiles * hk > (1 << 30)) return KVPOOL_ERR_INVALID_ARG;
      if (tasks > 0 && tasks + tiles * hk > (1 << 30)) break;
      EvictSeg& S = P->segs[P->n_segs++];
      S.k_len = (int32_t)h_k_len[i];
      S.task_base = (int32_t)tasks;
      S.table_row = i - first;
      tasks += tiles * hk;
    }
    P->n_tasks = (int32_t)tasks;
    P->c = kv4_cache(&a->cache, first, dev->err);
    P->out_table = a->d_out_table + first * a->out_table_stride;
    P->w = a->d_weights + first * a->weight_stride;
    P->out_w = a->d_out_weights ? a->d_out_weights + first * a->out_weight_stride : nullptr;
    P->index = a->d_index + (int64_t)first * hk * a->keep;
    cudaError_t e = slice <= kMaxShared ? launch_select<true>(*P, slice, s) : launch_select<false>(*P, slice, s);
    if (e == cudaSuccess && P->n_tasks > 0) {
      const dim3 grid((unsigned)((P->n_tasks + kMoveWarps - 1) / kMoveWarps)), block(kMoveWarps * 32);
      e = a->cache.head_dim == 128 ? launch_kernel(false, kv4_move_kernel<128>, grid, block, 0, s, *P)
                                   : launch_kernel(false, kv4_move_kernel<64>, grid, block, 0, s, *P);
    }
    if (e != cudaSuccess) return KVPOOL_ERR_CUDA;
  }
  return KVPOOL_OK;
}
