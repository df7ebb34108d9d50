// kvpool_window.h -- work plan of window attention, shared by its kernels.
#pragma once

#include "device_util.cuh"
#include "kvpool_internal.h"

namespace kvp {

constexpr int kMaxWinSegs = 256;  // segments per launch
constexpr int kWinMaxGroup = 16;  // query heads per key head

// One segment (a request's queries and its cached tokens) of a launch.  Its
// queries are cut into tiles of tile_tokens tokens; a tile holds the rows
// (token, query head of the group) of one key head, the group's heads fastest.
struct WinSeg {
  int64_t q_row0;     // first query row
  int64_t k_start;    // cache row of the token at position 0
  int32_t q_len, k_len;
  int32_t item_base;  // first work item: ((tile * n_split + split) * kv_heads + head)
  int32_t n_split;    // parts that each tile's keys are cut into
  int32_t part_base;  // first partial slot (n_split > 1)
  int32_t merge_base; // (tile, key head)s of the split segments before this one
};

struct WinParams {
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* out;
  float* lse;  // [q_rows][q_heads] or null
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head;  // strides in values
  int32_t q_heads, kv_heads, group;
  int32_t window, n_sink;
  float scale_log2;  // softmax scale times log2(e)
  int32_t tile_tokens, tile_rows;
  int32_t n_segs, n_items;
  int32_t n_merge, merge_rows;  // (tile, key head)s to merge, the most rows that one has
  float* part_o;    // [slots][tile_rows][head_dim]
  float2* part_ml;  // [slots][tile_rows]: (max in the log2 domain, sum)
  uint32_t* err;
  WinSeg segs[kMaxWinSegs];
};

// A work item: queries tok0 .. tok0 + n_tok - 1 of a segment (positions pos0
// ...) under key head hk.  The keys that some query of the tile sees are the
// first n_s tokens (sinks before the window) and tokens lo .. lo + n_w - 1;
// every query of the tile at a position >= 0 sees all of the first n_s.
struct WinItem {
  int seg, hk, tok0, n_tok, split, n_split, slot;
  int pos0, n_s, lo, n_w;
};

__device__ __forceinline__ int win_find_seg(const WinParams& P, int item) {
  int lo = 0, hi = P.n_segs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.segs[mid].item_base <= item) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ WinItem win_item(const WinParams& P, int item) {
  WinItem w;
  w.seg = win_find_seg(P, item);
  const WinSeg& S = P.segs[w.seg];
  int r = item - S.item_base;
  w.slot = S.part_base + r;
  w.hk = r % P.kv_heads;
  r /= P.kv_heads;
  w.n_split = S.n_split;
  w.split = r % S.n_split;
  w.tok0 = (r / S.n_split) * P.tile_tokens;
  w.n_tok = min(P.tile_tokens, S.q_len - w.tok0);
  w.pos0 = S.k_len - S.q_len + w.tok0;
  const int hi = w.pos0 + w.n_tok - 1;  // the last query's own position
  w.lo = max(0, w.pos0 - P.window + 1);
  // a window of 0: of these, only the first tokens are anybody's
  w.n_w = max(0, (P.window > 0 ? hi : min(hi, P.n_sink - 1)) - w.lo + 1);
  w.n_s = max(0, min(P.n_sink, min(w.lo, hi + 1)));
  return w;
}

// does the query at position p see the token at position t?
__device__ __forceinline__ bool win_sees(const WinParams& P, int p, int t) {
  return t <= p && (t > p - P.window || t < P.n_sink);
}

// A row's log-sum-exp from its maximum (log2 domain) and sum: -inf where it saw
// nothing, NaN where its sum is one (a NaN or an infinity among its scores)
__device__ __forceinline__ float win_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Single-token form: at most 16 query rows per key head, the whole segment in
// one tile.  Returns a cudaError_t.
constexpr int kTokRows = 16;
int launch_window_tok(const WinParams& P, int dtype, int head_dim, void* stream);

// Tensor-core form of a launch of prompts (bf16); tiles of two times
// tile_tokens / 2 tokens.  Returns a cudaError_t.
constexpr int kTcTileRows = 128;
int launch_window_tc(const WinParams& P, int head_dim, int64_t q_rows, int64_t kv_rows, int n_sms, void* stream);

}  // namespace kvp
