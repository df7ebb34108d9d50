// kvpool_kv4.h -- the paged cache held in 4 bits: its layout and what the
// kernels that write, read and shrink it share.
//
// A page holds page_tokens tokens of every key head; the record of a page and
// head is page_tokens / 16 tiles of 16 tokens, each in one piece:
//   K codes   [16 tokens][D / 2]   dims 2i (low nibble) and 2i + 1 in byte i
//   V codes   [8 pairs][D]         tokens 2j (low nibble) and 2j + 1 in byte d
//                                  of pair j, D / 8 dims to a chunk (below)
//   K scales  [16 tokens][D / 16]  e4m3
//   V scales  [8 pairs][D / 16][2] e4m3, token 2j first
// Keys are multiplied along the dims and values along the tokens, so that is
// how two codes share a byte: one conversion makes the pair of halves that a
// matrix fragment wants.  Chunk c of V pair j lies in place c ^ kv4_swizzle(j):
// the 32 lanes of a fragment (8 chunks of 4 pairs) then read shared memory
// without bank conflicts, while a pair's codes stay together for the kernels
// that move single tokens.
#pragma once

#include "device_util.cuh"
#include "kvpool_internal.h"

namespace kvp {

constexpr int kKv4Tile = 16;      // tokens
constexpr int kKv4Group = 16;     // values that share a scale
constexpr int kKv4MaxSegs = 256;  // segments per launch
constexpr int kKv4MaxHeads = 1024;

template <int D>
struct Kv4Tile {
  static constexpr int kV = kKv4Tile * D / 2;
  static constexpr int kKs = kKv4Tile * D;
  static constexpr int kVs = kKs + D;
  static constexpr int kBytes = kKv4Tile * D + 2 * D;
  static constexpr int kChunk = D / 8;  // bytes of a V chunk (one lane's dims)
};

struct Kv4Cache {
  uint8_t* pages;
  const int32_t* table;  // [rows][table_stride] page ids, already at the launch's first segment
  int64_t table_stride;
  int32_t n_pages, kv_heads;
  int32_t page_shift;  // log2 of a page's tiles
  float k_scale, v_scale;
  uint32_t* err;
};

template <int D>
__device__ __forceinline__ int kv4_swizzle(int pair) {
  return D == 128 ? 2 * (pair & 3) : 4 * ((pair >> 1) & 1);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t a) { return __half22float2(*reinterpret_cast<const __half2*>(&a)); }

// The page id of a tile of table row `row`, or -1 (and a flag) if it is none.
__device__ __forceinline__ int kv4_page(const Kv4Cache& C, int64_t row, int tile) {
  const int id = C.table[row * C.table_stride + (tile >> C.page_shift)];
  if ((unsigned)id < (unsigned)C.n_pages) return id;
  atomicOr(C.err, (uint32_t)kErrBadBlock);
  return -1;
}
template <int D>
__device__ __forceinline__ int64_t kv4_tile_offset(const Kv4Cache& C, int id, int head, int tile) {
  return ((((int64_t)id * C.kv_heads + head) << C.page_shift) + (tile & ((1 << C.page_shift) - 1))) * Kv4Tile<D>::kBytes;
}

// Host: the checks of a cache that every call makes, and what the kernels take
// of it for table rows row0 and on.  Returns KVPOOL_OK or an error.
int kv4_check(const kvpool_kv4* c, int64_t rows);
Kv4Cache kv4_cache(const kvpool_kv4* c, int64_t row0, uint32_t* err);
// Do n tokens' rows of h lie on the cache's pages or its table?
bool kv4_meets(const kvpool_kv4* c, const kvpool_heads& h, int64_t n, int64_t vb);
bool kv4_meets(const kvpool_kv4* c, const void* p, __int128 bytes);
// The same for n segments' weights (fp32 runs of len places, per segment and head).
bool kv4_meets(const kvpool_kv4* c, const float* w, int64_t n, int64_t seg_stride, int64_t head_stride, int64_t len);
inline int64_t kv4_tokens(const kvpool_kv4* c) { return (int64_t)c->table_width * c->page_tokens; }

// Read len[i] tokens from place start[i] on of table rows row0 + i into rows of k
// (bf16) and v (fp16, not multiplied by v_scale), one segment after the other.
// Returns a KVPOOL_ code.
int kv4_load_rows(const kvpool_kv4* c, const kvpool_heads& k, const kvpool_heads& v, int32_t n, int64_t row0,
                  const int64_t* start, const int64_t* len, uint32_t* err, void* stream);

}  // namespace kvp
