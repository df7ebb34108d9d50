// kvpool_window_tc.cu -- window attention of prompts on the 5th-generation
// tensor cores (bf16).
//
// A work item is 256 query rows (token, query head of the group) of one key
// head: two tiles of 128 rows that share every K and V tile of 128 keys.
// Persistent CTAs, one per SM, of ten warps: one issues the tensor copies
// (Q tiles, and a ring of K and V tiles), one the matrix products, and a group
// of four per query tile does its softmax, a thread per row.  Scores S = Q K^T
// go to tensor memory; the softmax reads a row, keeps the running maximum and
// sum in fp32, and writes the weights back as bf16 over the scores; O += P V
// accumulates in tensor memory.  While one tile's rows go through the softmax
// the products of the other tile run, so the tensor core and the exponentials
// (both about 1,024 cycles per 128 x 128 x 128 tile pair and side) overlap.
//
// The bf16 weights are the one rounding besides the output's own (2^-8 of a
// weight, against sums of the unrounded ones).  A second piece of each, and a
// second product with V, was measured: 32,768 tokens under a window of 4,096
// 1,075 us against 770, 4 x 2,048 under 128 44.3 against 38.6.  Against 64 bits the
// outputs are off by 2.0e-3 to 2.3e-3 of their norm, where their own rounding
// alone leaves 1.5e-3 to 1.7e-3.
//
// The 4-bit cache's values are exact in fp16 (F16): their tiles and the weights are
// fp16 then (2^-11 of a weight), in units of 2^-6 of the row's maximum or older
// maximum, so that the largest is 2^6 to 2^14 and what fp16's smallest step takes
// from small ones is 2^-31 of it.
//
// The outputs are rescaled only when a row's maximum grows by more than 2^8:
// until then its weights are taken against the older maximum (bf16 keeps its
// relative precision up to 2^8, the sums are fp32), so the read-modify-write
// of O leaves the critical path.
//
// The tensor core cuts its sums off instead of rounding them: 65,536 additions of 16
// keys' products in a row left outputs 0.7% too small (4,096 queries behind 1,048,576
// tokens, values of one sign; error 7.2e-3 of their norm, their rounding alone is
// 1.7e-3).  So a sum in tensor memory is 16,384 keys long at most; a thread then adds
// its row's to fp32 sums in the workspace (20 MB, L2), with rounding (1.68e-3
// there).  Calls without such items run a kernel without this.  With it, prompts over
// the 4-bit cache take 1% longer with heads of 128 (65,536 queries of 16 heads on 4
// behind their own 11.4 -> 11.5 ms) and 3% with 64, others no longer (16,384 queries,
// 16 heads on 8 of 64, window 100,000 7.08 -> 7.03 ms).  Measured and not kept: vector
// atomics instead of reading the sums, the same in a function of its own (12% there).
//
// Rows of K and V behind a segment, or between the first tokens and the window,
// never count: scores are masked, and such V rows are not copied (boxes of 16
// and of 1 row up to the last one that holds values, zeros behind it).
//
// Bound: the chain scores -> softmax -> outputs -> next scores of a query tile,
// which one other tile covers.  32,768 tokens x 16 heads of 128 under a window of
// 4,096 take 770 us, 1,335 TFLOP/s of visible products (0.69 of the library
// product's rate; partial tiles compute up to 6% more than is visible).  At 8,192
// tokens the tensor pipe is busy 52% of the time and 56% of an active SM's, the
// exponentials' 27%, issue slots 33%; warps wait on loads and barriers (3.5 of 7.5
// cycles per instruction).  The power limit takes 6% (1,940 of 2,070 MHz in a loop
// of calls, where the library product falls to 1,450).
// Short windows: 4 x 2,048 queries x 16 heads under a window of 128 38.6 us, of which
// the tiles' 128-key steps compute 3 keys for 1 that is seen; tensor pipe 16% busy,
// issue slots 22%, loads and barriers 6.2 of 11.7 cycles per instruction,
// instruction fetch 1.0.
// Measured and not kept: K and V tiles of its own for each query tile (38.8 us
// against 36.6 there), two threads per row (174 against 164 us for 8,192 tokens
// under 4,096), outputs staged for whole-line stores (slower).
#include <cuda.h>
#include <cuda_runtime.h>

#include "kvpool_fma.cuh"
#include "kvpool_tcgen05.cuh"
#include "kvpool_window.h"

namespace kvp {
namespace {

constexpr int kTcKeys = 128;
constexpr int kTcThreads = 320;
constexpr int kTcTable = 96;  // items of a CTA that are worked out at its start
constexpr float kRescale = 8.0f;  // log2 growth of the maximum that rescales O
constexpr float kF16Up = 6.0f;    // log2 of the maximum's weight, F16

template <int D>
struct TcShape {
  static constexpr int kTileBytes = 128 * D * 2;  // a Q, K or V tile: D / 64 runs of 128 rows x 128 bytes
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kBarOff = (2 + kStages) * kTileBytes;
  static constexpr int kTableOff = kBarOff + 512;
  static constexpr int kSmem = kTableOff + kTcTable * 64 + 1024;  // + slack to align the tiles to 1,024 bytes
};

struct TcMaps {
  CUtensorMap q, k, v, v16, v1;  // v16, v1: boxes of 16 rows and of one
};

// A work item as the roles take it: its keys are the first n_s tokens and n_w
// from lo on, in steps [a, b) of 128.
struct TcItem {
  int hk, q_row, k_row, n_tok, pos0, part, slot, k_len;  // part: its rows are partials
  int n_s, lo, n_w, a, b;
  int pad[3];
};
static_assert(sizeof(TcItem) == 64, "the item table's stride");

// Step st of a key list: 128 keys from token t0 on, of which those before `end` count.
struct TcStep {
  int t0, end;
  bool sink;
};
__device__ __forceinline__ TcStep tc_step(const TcItem& w, int st) {
  const int st_s = (w.n_s + kTcKeys - 1) / kTcKeys;
  TcStep c;
  c.sink = st < st_s;
  c.t0 = c.sink ? st * kTcKeys : w.lo + (st - st_s) * kTcKeys;
  c.end = c.sink ? w.n_s : w.lo + w.n_w;
  return c;
}
// Rows of the step's tile that hold values; the others, behind the first tokens
// or behind the segment, may hold anything
__device__ __forceinline__ int tc_valid(const WinParams& P, const TcItem& w, int st) {
  const TcStep c = tc_step(w, st);
  return min(kTcKeys, (c.sink || P.window == 0 ? c.end : w.k_len) - c.t0);
}
// A query tile of an item: n tokens at positions p0 .. p1
struct TcTile {
  int n, p0, p1;
};
__device__ __forceinline__ TcTile tc_tile(const WinParams& P, const TcItem& w, int t) {
  const int tt = P.tile_tokens / 2;
  TcTile q;
  q.n = max(0, min(tt, w.n_tok - t * tt));
  q.p0 = w.pos0 + t * tt;
  q.p1 = q.p0 + q.n - 1;
  return q;
}

// The steps of [a, b) that some row of a query tile needs: those before `sink`
// (first tokens) and those in [lo, hi).
struct TcNeed {
  int sink, lo, hi;
  __device__ __forceinline__ bool operator()(int st) const { return st < sink || (st >= lo && st < hi); }
  __device__ __forceinline__ bool more(int st) const { return st + 1 < sink || max(st + 1, lo) < hi; }
  __device__ __forceinline__ int last(int a) const { return hi > lo ? hi - 1 : sink > a ? sink - 1 : -1; }
};
__device__ __forceinline__ TcNeed tc_need(const WinParams& P, const TcItem& w, const TcTile& q) {
  TcNeed n{w.a, w.a, w.a};
  if (q.n <= 0) return n;
  const int st_s = (w.n_s + kTcKeys - 1) / kTcKeys;
  // window steps: step st holds tokens lo + (st - st_s) * 128 ..
  const int first = max(0, q.p0 - P.window + 1 - w.lo) / kTcKeys;  // of the first token in the window
  const int past = q.p1 < w.lo ? 0 : (q.p1 - w.lo) / kTcKeys + 1;
  const int sinks = P.n_sink > w.lo ? (P.n_sink - w.lo + kTcKeys - 1) / kTcKeys : 0;  // first tokens behind lo
  n.sink = min(w.b, max(w.a, st_s + min(sinks, past)));
  n.lo = max(n.sink, st_s + first);
  n.hi = max(n.lo, min(w.b, st_s + past));
  return n;
}

// k-th item of a CTA: back and forth over the CTAs, the last (longest) tiles first
__device__ __forceinline__ int tc_nth(const WinParams& P, int k) {
  const int g = gridDim.x, c = blockIdx.x;
  const int i = k * g + ((k & 1) ? g - 1 - c : c);
  return i < P.n_items ? P.n_items - 1 - i : -1;
}

__device__ __forceinline__ TcItem tc_make(const WinParams& P, int item) {
  const WinItem w = win_item(P, item);
  const WinSeg& S = P.segs[w.seg];
  const int n = (w.n_s + kTcKeys - 1) / kTcKeys + (w.n_w + kTcKeys - 1) / kTcKeys;
  TcItem x;
  x.hk = w.hk;
  x.q_row = (int)S.q_row0 + w.tok0;
  x.k_row = (int)S.k_start;
  x.n_tok = w.n_tok;
  x.pos0 = w.pos0;
  x.part = w.n_split > 1 || P.pieces;
  x.slot = w.slot;
  x.k_len = S.k_len;
  x.n_s = w.n_s;
  x.lo = w.lo;
  x.n_w = w.n_w;
  x.a = (int)((int64_t)n * w.split / w.n_split);
  x.b = (int)((int64_t)n * (w.split + 1) / w.n_split);
  x.pad[0] = x.pad[1] = x.pad[2] = 0;
  return x;
}

// ---- softmax of one row -----------------------------------------------------------
__device__ __forceinline__ float tc_max32(const uint32_t* x, float mx) {
  float a[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < 32; j += 2)
    a[(j >> 1) & 3] = max3(a[(j >> 1) & 3], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
  return fmaxf(max3(a[0], a[1], a[2]), a[3]);
}
__device__ __forceinline__ float tc_max64(const uint32_t* x, float mx) { return tc_max32(x + 32, tc_max32(x, mx)); }

// weights 2^(x scale - base) of 32 scores as bf16 or fp16 to 16 words of tensor
// memory, and their fp32 sums (packed pairs)
template <bool F16>
__device__ __forceinline__ void tc_weights32(const uint32_t* x, float scale, float base, uint64_t* sum, uint32_t addr) {
  const uint64_t scale2 = pack2(scale, scale), base2 = pack2(-base, -base);
  uint32_t pk[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 y = unpack2(fma2(pack2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), scale2, base2));
    const float p0 = ex2f(y.x), p1 = ex2f(y.y);
    sum[j & 1] = add2(sum[j & 1], pack2(p0, p1));
    if constexpr (F16) {
      const __half2 z = __floats2half2_rn(p0, p1);
      pk[j] = *reinterpret_cast<const uint32_t*>(&z);
    } else {
      const __nv_bfloat162 z = __floats2bfloat162_rn(p0, p1);
      pk[j] = *reinterpret_cast<const uint32_t*>(&z);
    }
  }
  tmem_st16(addr, pk);
}
// Take a step's maximum into the row's; the whole warp rescales its sums and
// outputs (in tensor memory from `to` on) when some row's grew by too much.
template <int D>
__device__ __forceinline__ void tc_maximum(float mn, bool& first, float& m, float& l, uint32_t to) {
  if (first) {
    m = fmaxf(m, mn);
    first = false;
  } else if (__any_sync(0xffffffffu, mn > m + kRescale)) {
    const float m2 = fmaxf(m, mn);
    const float f = m2 == -INFINITY ? 1.0f : ex2f(m - m2);
    m = m2;
    l *= f;
#pragma unroll 1
    for (int i = 0; i < D / 16; ++i) {
      uint32_t o[16];
      tmem_ld16(to + 16 * i, o);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
      tmem_st16(to + 16 * i, o);
    }
  }
}

// A row's sums outside tensor memory, and the maximum that they were taken against.
struct TcSums {
  uint4* o;  // four numbers, the next four 128 further
  float* m;
  // the sums, times f, to x
  __device__ __forceinline__ void add(int i, float f, uint32_t* x) const {
    const uint4 z = __ldcg(o + i * 128);
    x[0] = __float_as_uint(fmaf(__uint_as_float(z.x), f, __uint_as_float(x[0])));
    x[1] = __float_as_uint(fmaf(__uint_as_float(z.y), f, __uint_as_float(x[1])));
    x[2] = __float_as_uint(fmaf(__uint_as_float(z.z), f, __uint_as_float(x[2])));
    x[3] = __float_as_uint(fmaf(__uint_as_float(z.w), f, __uint_as_float(x[3])));
  }
};
// what a number taken against the maximum `then` is worth against the one now
__device__ __forceinline__ float tc_factor(float then, float now) { return then == -INFINITY ? 0.0f : ex2f(then - now); }
template <int D>
__device__ __forceinline__ TcSums tc_sums(const WinParams& P, int t, int row) {
  float* base = P.sums + (int64_t)(2 * blockIdx.x + t) * 128 * (D + 1);
  return TcSums{reinterpret_cast<uint4*>(base) + row, base + 128 * D + row};
}

// F16: weights and V in fp16; SUMS: some items have more than kTcSumSteps steps
template <int D, bool F16, bool SUMS>
__global__ void __launch_bounds__(kTcThreads, 1) window_tc_kernel(const __grid_constant__ WinParams P,
                                                                  const __grid_constant__ TcMaps M) {
  using Sh = TcShape<D>;
  constexpr int NS = Sh::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t* q_tile = smem;
  uint8_t* ring = smem + 2 * Sh::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kBarOff);
  uint64_t *kv_full = bars, *kv_free = kv_full + NS, *q_full = kv_free + NS, *q_free = q_full + 2, *s_full = q_free + 2,
           *p_ready = s_full + 2, *o_full = p_ready + 2, *o_free = o_full + 2, *drain = o_free + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  TcItem* table = reinterpret_cast<TcItem*>(smem + Sh::kTableOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_free[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_free[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[t], 4);
      mbar_init(&o_full[t], 1);
      mbar_init(&o_free[t], 4);
    }
    mbar_init(drain, 1);
    mbar_fence_init();
  }
  // The CTA's first items, a thread each (the divisions and the search for the
  // segment cost ~2,000 cycles, once instead of per item and role)
  if (threadIdx.x >= 32 && threadIdx.x < 32 + kTcTable) {
    const int item = tc_nth(P, threadIdx.x - 32);
    if (item >= 0) table[threadIdx.x - 32] = tc_make(P, item);
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // columns: S0, S1 (128 each), O0, O1 (128 each)
  pdl_start();  // nothing before touches what an earlier kernel writes
  auto item_of = [&](int k, int item) -> TcItem {
    if (k < kTcTable) return table[k];
    return tc_make(P, item);
  };

  if (warp == 8) {
    // ---- tensor copies (one lane issues them) ----
    const bool leader = elect_one();
    int stage = 0, n_q[2] = {0, 0}, issued = 0;
    uint32_t round = 0;  // of the ring
    bool ok = true;
    // the tile's first `valid` rows
    auto load = [&](const CUtensorMap* map, int hk, int row, int valid) {
      if (round > 0) ok = ok && warp_wait(&kv_free[stage], (round - 1) & 1, P.err);
      if (!ok) return;
      uint8_t* tile = ring + stage * Sh::kTileBytes;
      if (valid == kTcKeys) {
        if (leader) {
          mbar_arrive_expect_tx(&kv_full[stage], Sh::kTileBytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tma_load_3d(tile + c * 16384, map, 64 * c, hk, row, &kv_full[stage]);
        }
      } else {
        // A V tile that ends early: its rows in boxes of 16 and of 1, and zeros
        // in the rest of the last 16 (the product takes whole groups of 16; 0
        // times a NaN there would reach every row)
        const int n16 = (valid + 15) / 16;
        for (int h = 0; h < D / 64; ++h) {
          uint4* base = reinterpret_cast<uint4*>(tile + h * 16384);
          for (int j = valid * 8 + lane; j < n16 * 128; j += 32) base[j] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
        if (leader) {
          mbar_arrive_expect_tx(&kv_full[stage], valid * D * 2);
          for (int r = 0; r < valid;) {
            const bool many = valid - r >= 16;
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(tile + c * 16384 + r * 128, many ? &M.v16 : &M.v1, 64 * c, hk, row + r, &kv_full[stage]);
            r += many ? 16 : 1;
          }
        }
      }
      __syncwarp();
      ++issued;
      if (++stage == NS) {
        stage = 0;
        ++round;
      }
    };
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int item = tc_nth(P, k);
      if (item < 0) break;
      const TcItem w = item_of(k, item);
      const int tt = P.tile_tokens / 2;
      auto load_q = [&](int t) {
        if (w.n_tok <= t * tt) return;
        if (n_q[t] > 0) ok = ok && warp_wait(&q_free[t], (n_q[t] - 1) & 1, P.err);
        if (!ok) return;
        if (leader) {
          mbar_arrive_expect_tx(&q_full[t], tt * P.group * D * 2);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(q_tile + t * Sh::kTileBytes + c * 16384, &M.q, 64 * c, 0, w.hk, w.q_row + t * tt, &q_full[t]);
        }
        __syncwarp();
        ++n_q[t];
      };
#pragma unroll 1
      for (int st = w.a; st < w.b && ok; ++st) {
        const int t0 = tc_step(w, st).t0;
        if (st == w.a) load_q(0);
        if (ok) load(&M.k, w.hk, w.k_row + t0, kTcKeys);
        if (st == w.a && ok) load_q(1);
        if (ok) load(&M.v, w.hk, w.k_row + t0, tc_valid(P, w, st));
      }
    }
    // the CTA does not end while copies land in its shared memory
    for (int i = issued > NS ? issued - NS : 0; i < issued; ++i) warp_wait(&kv_full[i % NS], (i / NS) & 1, P.err);
    for (int t = 0; t < 2; ++t)
      if (n_q[t] > 0) warp_wait(&q_full[t], (n_q[t] - 1) & 1, P.err);
  } else if (warp == 9) {
    // ---- matrix products (one thread) ----
    if (elect_one()) {
      constexpr uint32_t kIdQK = bf16_idesc(128, kTcKeys, false), kIdPV = bf16_idesc(128, D, true, F16);
      const uint64_t q_desc = smem_desc(smem_addr(q_tile), 16), k_desc = smem_desc(smem_addr(ring), 16),
                     v_desc = smem_desc(smem_addr(ring), 16384);
      int stage = 0;
      uint32_t round = 0;
      int n_q[2] = {0, 0}, n_p[2] = {0, 0}, n_o[2] = {0, 0};
      bool ok = true;
      auto next = [&]() {
        if (++stage == NS) {
          stage = 0;
          ++round;
        }
      };
      // the ring's next tile is there; returns its stage
      auto take = [&]() {
        const int s = stage;
        if (!mbar_wait_word(&kv_full[s], round & 1, P.err)) ok = false;
        next();
        return s;
      };
      // O_t += P_t V, V in ring stage vs, over n16 groups of 16 keys
      auto outputs = [&](int t, int vs, int n16, bool begun, bool last) {
        ok = ok && mbar_wait_word(&p_ready[t], n_p[t] & 1, P.err);
        ++n_p[t];
        if (ok && !begun && n_o[t] > 0) ok = mbar_wait_word(&o_free[t], (n_o[t] - 1) & 1, P.err);
        if (!ok) return;
        tc_fence_after();
        const uint64_t vd = v_desc + vs * (Sh::kTileBytes >> 4);
        if (n16 == kTcKeys / 16) {
#pragma unroll
          for (int c = 0; c < kTcKeys / 16; ++c)
            mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * c, vd + c * (2048 >> 4), kIdPV, begun || c > 0);
        } else {
#pragma unroll 1
          for (int c = 0; c < n16; ++c)
            mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * c, vd + c * (2048 >> 4), kIdPV, begun || c > 0);
        }
        if (last) {
          mma_commit(&o_full[t]);
          ++n_o[t];
        }
      };
      // S_t = Q_t K^T, K in ring stage ks
      auto scores = [&](int t, int ks, bool begun, bool last) {
        if (!begun) {
          ok = ok && mbar_wait_word(&q_full[t], n_q[t] & 1, P.err);
          ++n_q[t];
        }
        if (!ok) return;
        tc_fence_after();
        const uint64_t qd = q_desc + t * (Sh::kTileBytes >> 4), kd = k_desc + ks * (Sh::kTileBytes >> 4);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t off = ((c / 4) * 16384 + (c % 4) * 32) >> 4;
          mma_ss(tmem + 128 * t, qd + off, kd + off, kIdQK, c > 0);
        }
        mma_commit(&s_full[t]);
        if (last) mma_commit(&q_free[t]);
      };
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        const int item = tc_nth(P, k);
        if (item < 0) break;
        const TcItem w = item_of(k, item);
        const int a = w.a, b = w.b;
        if (a >= b) continue;
        const TcTile q[2] = {tc_tile(P, w, 0), tc_tile(P, w, 1)};
        const TcNeed need[2] = {tc_need(P, w, q[0]), tc_need(P, w, q[1])};
        const int last[2] = {need[0].last(a), need[1].last(a)};
        bool seen_q[2] = {false, false};
        bool seen_pv[2] = {false, false};
        if (SUMS) n_p[0] &= 1, n_p[1] &= 1;
        int vs = 0, v16 = 0;  // of the step before: V's stage and its groups of 16 keys
        // round st: outputs of step st - 1, then scores of step st
#pragma unroll 1
        for (int st = a; st <= b && ok; ++st) {
          int ks = 0;
          if (st < b) ks = take();
          if (!ok) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && st > a && need[t](st - 1)) {
              const bool end = st - 1 == last[t] || (SUMS && (n_p[t] + 1) % kTcSumSteps == 0);
              outputs(t, vs, v16, seen_pv[t], end);
              seen_pv[t] = !SUMS || !end;
            }
            if (ok && st < b && need[t](st)) {
              scores(t, ks, seen_q[t], st == last[t]);
              seen_q[t] = true;
            }
          }
          if (!ok) break;
          if (st > a) mma_commit(&kv_free[vs]);
          if (st == b) break;
          mma_commit(&kv_free[ks]);
          vs = take();
          v16 = (tc_valid(P, w, st) + 15) / 16;
        }
        // a tile whose rows need no step was loaded all the same: take its Q
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && q[t].n > 0 && !seen_q[t]) {
            ok = mbar_wait_word(&q_full[t], n_q[t] & 1, P.err);
            ++n_q[t];
            mma_commit(&q_free[t]);
          }
      }
      // every product and its arrivals are done before the CTA ends
      mma_commit(drain);
      mbar_wait_word(drain, 0, P.err);
    }
    __syncwarp();
  } else {
    // ---- softmax of query tile t: a thread per row ----
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // 32 lanes per warp, lane in bits 16..
    const uint32_t ts = tmem + lane_base + 128 * t, to = tmem + lane_base + 256 + 128 * t;
    const int r_tok = row / P.group, r_head = row % P.group;
    const int tt = P.tile_tokens / 2;
    const float scale = P.scale_log2;
    constexpr float kUp = F16 ? kF16Up : 0.0f;  // (m - 0 is m: the bf16 form's bits are without it)
    int n_s = 0, n_o = 0;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int item = tc_nth(P, k);
      if (item < 0) break;
      const TcItem w = item_of(k, item);
      const TcTile q = tc_tile(P, w, t);
      const TcNeed need = tc_need(P, w, q);
      const int pos = q.p0 + r_tok;
      bool mine = r_tok < q.n && row < tt * P.group;
      // m: of the scaled scores (log2).  A row that is not the tile's has no say in when its warp rescales, since its scores
      // are of other segments' queries (or of outputs that are written over them meanwhile), or of what shared memory held:
      // it starts where nothing is larger.
      float m = mine ? -INFINITY : INFINITY, l = 0.0f;
      bool first = true;
      // SUMS: the item's steps are counted from the barrier's parity on (0 or 1), here and where the products are issued
      if (SUMS) n_s &= 1;
      // (two loops: what is done once in kTcSumSteps steps stays out of the inner one's registers)
      int st = w.a;
#pragma unroll 1
      while (true) {
#pragma unroll 1
        for (; st < w.b; ++st) {
          if (!need(st)) continue;
          const TcStep c = tc_step(w, st);
          if (!warp_wait(&s_full[t], n_s & 1, P.err)) {
            ok = false;
            break;
          }
          ++n_s;
          tc_fence_after();
          // a tile in the middle: every row of the query tile sees all of it
          const bool whole = c.t0 + kTcKeys <= c.end &&
                             (c.sink || (c.t0 + kTcKeys - 1 <= q.p0 &&
                                         (c.t0 > q.p1 - P.window || c.t0 + kTcKeys <= P.n_sink)));
          const int hi = min(c.sink ? c.end - 1 : pos, c.end - 1) - c.t0;  // last column that the row sees
          const int lo = c.sink ? 0 : pos - P.window + 1 - c.t0;            // first of the window
          const int sk = c.sink ? 0 : P.n_sink - c.t0;                     // columns before it: first tokens
          uint64_t sum[2] = {0, 0};
          if (whole) {
            // the row's 128 scores in registers: maximum, weights
            uint32_t x[128];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, x + 32 * i);
            tmem_wait_ld();
            tc_maximum<D>(tc_max64(x + 64, tc_max64(x, -INFINITY)) * scale, first, m, l, to);
            const float base = m == -INFINITY ? 0.0f : m - kUp;
#pragma unroll
            for (int i = 0; i < 4; ++i) tc_weights32<F16>(x + 32 * i, scale, base, sum, ts + 16 * i);
          } else {
            // 32 scores at a time, twice (little code: it is run through cold);
            // a quarter that none of the warp's rows sees is skipped
            uint32_t x[32];
            auto quarter = [&](int i) {  // false: nobody sees it
              const int h = hi - 32 * i, g = lo - 32 * i, f = sk - 32 * i;
              const uint32_t le = h < 0 ? 0u : h >= 31 ? ~0u : (2u << h) - 1u;
              const uint32_t ge = g <= 0 ? ~0u : g >= 32 ? 0u : ~((1u << g) - 1u);
              const uint32_t lt = f <= 0 ? 0u : f >= 32 ? ~0u : (1u << f) - 1u;
              const uint32_t see = le & (ge | lt);
              if (!__any_sync(0xffffffffu, see != 0u)) return false;
              tmem_ld32(ts + 32 * i, x);
              tmem_wait_ld();
              if (!__all_sync(0xffffffffu, see == ~0u)) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!((see >> j) & 1u)) x[j] = 0xFF800000u;  // -inf
              }
              return true;
            };
            float mx = -INFINITY;
#pragma unroll 1
            for (int i = 0; i < 4; ++i)
              if (quarter(i)) mx = tc_max32(x, mx);
            tc_maximum<D>(mx * scale, first, m, l, to);
            const float base = m == -INFINITY ? 0.0f : m - kUp;
            // weights of columns 32 i .. 32 i + 31 go to words 16 i .. 16 i + 15: over scores that have been read by then
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              if (quarter(i)) {
                tc_weights32<F16>(x, scale, base, sum, ts + 16 * i);
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = 0u;
                tmem_st16(ts + 16 * i, x);
              }
            }
          }
          const float2 sa = unpack2(sum[0]), sb = unpack2(sum[1]);
          l += (sa.x + sa.y) + (sb.x + sb.y);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[t]);
          if (SUMS && n_s % kTcSumSteps == 0 && need.more(st)) break;
        }
        if (!SUMS || !ok || st >= w.b) break;
        // a sum is full, and more steps follow: it joins the row's outside tensor memory
        if (!warp_wait(&o_full[t], n_o & 1, P.err)) {
          ok = false;
          break;
        }
        ++n_o;
        tc_fence_after();
        uint32_t o[D];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) tmem_ld32(to + 32 * i, o + 32 * i);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[t]);  // (the next sum may begin)
        const TcSums sums = tc_sums<D>(P, t, row);
        if (n_s > kTcSumSteps) {
          const float f = tc_factor(*sums.m, m);
#pragma unroll
          for (int i = 0; i < D / 4; ++i) sums.add(i, f, o + 4 * i);
        }
        *sums.m = m;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) __stcg(sums.o + i * 128, make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
        ++st;
      }
      if (!ok) break;
      // ---- outputs of the tile ----
      if constexpr (SUMS || !F16) {  // worked out again, not kept over the loops (SUMS with heads of 64 took 3% longer, 4 x 2,048
                                     // queries under a window of 128 2%; the other form is the quicker one with it kept)
        int own = row;
        asm volatile("" : "+r"(own));
        mine = r_tok < q.n && own < tt * P.group;
      }
      const int64_t tok = w.q_row + t * tt + r_tok;
      const int head = w.hk * P.group + r_head;
      if (F16 && !w.part) l = win_sum(P, pos, l);
      const float inv = l > 0.0f ? P.v_scale / l : l;  // (a NaN stays one)
      if (!first) {
        if (!warp_wait(&o_full[t], n_o & 1, P.err)) break;
        ++n_o;
        tc_fence_after();
      }
      const int64_t pr = (int64_t)w.slot * P.tile_rows + t * tt * P.group + row;
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        __syncwarp();
        if (!first) {
          tmem_ld32(to + 32 * i, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        if (i == D / 32 - 1 && !first) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free[t]);
        }
        if (SUMS && n_s > kTcSumSteps) {
          const TcSums sums = tc_sums<D>(P, t, row);
          const float f = tc_factor(*sums.m, m);
#pragma unroll
          for (int j = 0; j < 8; ++j) sums.add(8 * i + j, f, o + 4 * j);
        }
        if (mine && w.part) {
          float4* dst = reinterpret_cast<float4*>(P.part_o + pr * D + 32 * i);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[j] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]), __uint_as_float(o[4 * j + 2]),
                                 __uint_as_float(o[4 * j + 3]));
        } else if (mine) {
          uint4* dst = reinterpret_cast<uint4*>(P.out + 2 * (tok * P.o_tok + head * P.o_head + 32 * i));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[8 * j + 2 * e]) * inv,
                                                             __uint_as_float(o[8 * j + 2 * e + 1]) * inv);
              x[e] = *reinterpret_cast<const uint32_t*>(&y);
            }
            dst[j] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      if (mine) {
        if (w.part) P.part_ml[pr] = make_float2(l > 0.0f ? m - kUp : -INFINITY, l);
        else if (P.lse) P.lse[tok * P.q_heads + head] = win_lse(m - kUp, l);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free(tmem, 512);
}

// ---- host ---------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// a stride in bytes; an axis of length 1 takes any legal one
cuuint64_t stride_bytes(int64_t values, int64_t extent) { return extent > 1 ? (cuuint64_t)values * 2 : 16; }

template <int D, bool F16, bool SUMS>
cudaError_t launch_tc(const WinParams& P, const TcMaps& M, int ctas, cudaStream_t s) {
  auto* kern = window_tc_kernel<D, F16, SUMS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TcShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(true, kern, dim3(ctas), dim3(kTcThreads), TcShape<D>::kSmem, s, P, M);
}

template <int D>
cudaError_t launch_dim(const WinParams& P, const TcMaps& M, int ctas, cudaStream_t s) {
  if (P.long_sums) return P.dense ? launch_tc<D, true, true>(P, M, ctas, s) : launch_tc<D, false, true>(P, M, ctas, s);
  return P.dense ? launch_tc<D, true, false>(P, M, ctas, s) : launch_tc<D, false, false>(P, M, ctas, s);
}

}  // namespace

int launch_window_tc(const WinParams& P, int head_dim, int64_t q_rows, int64_t kv_rows, int n_sms, void* stream) {
  if (!encode_fn()) return (int)cudaErrorNotSupported;
  TcMaps M;
  const cuuint64_t d = head_dim, g = P.group, hk = P.kv_heads;
  const cuuint64_t qd[4] = {d, g, hk, (cuuint64_t)q_rows};
  const cuuint64_t qs[3] = {stride_bytes(P.q_head, g), stride_bytes(P.q_head * P.group, hk), stride_bytes(P.q_tok, q_rows)};
  const cuuint32_t qb[4] = {64, (cuuint32_t)g, 1, (cuuint32_t)(P.tile_tokens / 2)};
  const cuuint64_t kd[3] = {d, hk, (cuuint64_t)kv_rows};
  const cuuint64_t ks[2] = {stride_bytes(P.k_head, hk), stride_bytes(P.k_tok, kv_rows)};
  const cuuint64_t vs[2] = {stride_bytes(P.v_head, hk), stride_bytes(P.v_tok, kv_rows)};
  const cuuint32_t kb[3] = {64, 1, kTcKeys}, b16[3] = {64, 1, 16}, b1[3] = {64, 1, 1};
  if (!encode(&M.q, P.q, 4, qd, qs, qb) || !encode(&M.k, P.k, 3, kd, ks, kb) || !encode(&M.v, P.v, 3, kd, vs, kb) ||
      !encode(&M.v16, P.v, 3, kd, vs, b16) || !encode(&M.v1, P.v, 3, kd, vs, b1))
    return (int)cudaErrorInvalidValue;
  const int ctas = P.n_items < n_sms ? P.n_items : n_sms;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return (int)(head_dim == 128 ? launch_dim<128>(P, M, ctas, s) : launch_dim<64>(P, M, ctas, s));
}

}  // namespace kvp
