// kvpool_window.cu -- attention of a ragged batch of queries over raw K/V
// tokens with a sliding window and a few first tokens that stay visible: what
// computes a prompt's own outputs in a window layer while append takes its
// tokens into the cache ("Why does V4 split pools? ..." s3.3: the window is
// the exact local part of attention).
//
//   out = sum_t softmax_t(scale <q, k_t>) v_t over t <= p with t > p - window
//   or t < n_sink;  lse = log sum_t exp(scale <q, k_t>);  a query that sees
//   nothing gives zeros and -inf.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <memory>
#include <mutex>
#include <new>

#include <cuda_runtime.h>

#include "kvpool_fma.cuh"
#include "kvpool_rows.h"
#include "kvpool_window.h"

namespace kvp {
namespace {

constexpr int kMaxDevices = 64;
__device__ uint32_t g_ops_error;  // device error word of the calls that have no pool

template <int T>
__device__ __forceinline__ float4 load4(const uint8_t* base, int64_t i) {
  if constexpr (T == KVPOOL_F32) {
    return *reinterpret_cast<const float4*>(base + 4 * i);
  } else {
    const uint2 r = *reinterpret_cast<const uint2*>(base + 2 * i);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
  }
}
template <int T>
__device__ __forceinline__ void store4(uint8_t* base, int64_t i, float4 x) {
  if constexpr (T == KVPOOL_F32) {
    *reinterpret_cast<float4*>(base + 4 * i) = x;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(base + 2 * i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// ---- fp32 FMA tiles: 32 rows, 64 keys per step ----------------------------------
template <int T, int D>
__global__ void __launch_bounds__(kFmaThreads) window_fma_kernel(const __grid_constant__ WinParams P) {
  pdl_start();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  FmaSmem<D>& sm = *reinterpret_cast<FmaSmem<D>*>(smem_raw);
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const WinItem w = win_item(P, blockIdx.x);
  const WinSeg& S = P.segs[w.seg];
  const int rows = w.n_tok * P.group;
  for (int i = tid; i < kFmaRows * (D / 4); i += kFmaThreads) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
      x = load4<T>(P.q, (S.q_row0 + w.tok0 + r / P.group) * P.q_tok +
                            (int64_t)(w.hk * P.group + r % P.group) * P.q_head + c);
    *reinterpret_cast<float4*>(&sm.q[r][c]) = x;
  }
  int pos[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) pos[r] = 4 * ty + r < rows ? w.pos0 + (4 * ty + r) / P.group : -1;
  FmaTile<D> f;
  f.init();
  // steps over the first n_s tokens, then over the window's; this split's share
  const int st_s = (w.n_s + kFmaKeys - 1) / kFmaKeys, st_w = (w.n_w + kFmaKeys - 1) / kFmaKeys;
  const int n_st = st_s + st_w;
  const int a = (int)((int64_t)n_st * w.split / w.n_split), b = (int)((int64_t)n_st * (w.split + 1) / w.n_split);
  struct Step {
    int t0, end;  // tokens from `end` on are nobody's: read as zeros
    bool sink;
  };
  auto step_of = [&](int st) {
    const bool sink = st < st_s;
    return Step{sink ? st * kFmaKeys : w.lo + (st - st_s) * kFmaKeys, sink ? w.n_s : w.lo + w.n_w, sink};
  };
  auto load = [&](int st) {  // fp32 rows by asynchronous copies
    const Step c = step_of(st);
    for (int i = tid; i < kFmaKeys * (D / 4); i += kFmaThreads) {
      const int r = i / (D / 4), x = 4 * (i % (D / 4));
      const bool in = c.t0 + r < c.end;
      const int64_t ka = in ? (S.k_start + c.t0 + r) * P.k_tok + w.hk * P.k_head + x : 0;
      const int64_t va = in ? (S.k_start + c.t0 + r) * P.v_tok + w.hk * P.v_head + x : 0;
      if constexpr (T == KVPOOL_F32) {
        cp_async16(smem_addr(&sm.k[r][x]), P.k + 4 * ka, in ? 16 : 0);
        cp_async16(smem_addr(&sm.v[r][x]), P.v + 4 * va, in ? 16 : 0);
      } else {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(&sm.k[r][x]) = in ? load4<T>(P.k, ka) : zero;
        *reinterpret_cast<float4*>(&sm.v[r][x]) = in ? load4<T>(P.v, va) : zero;
      }
    }
    cp_async_commit();
  };
  for (int st = a; st < b; ++st) {
    load(st);
    cp_async_wait<0>();
    __syncthreads();
    const Step c = step_of(st);
    f.step(
        sm, ty, tx,
        [&](int r, int j) {
          return c.t0 + j < c.end && (c.sink ? pos[r] >= 0 : win_sees(P, pos[r], c.t0 + j));
        },
        [&](int) { return P.scale_log2; }, [](int) { return 1.0f; });
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 4 * ty + r;
    if (row >= rows) continue;
    if (w.n_split > 1) {
      const int64_t pr = (int64_t)w.slot * P.tile_rows + row;
      if (tx == 0) P.part_ml[pr] = make_float2(f.m[r], f.l[r]);
      f.put(P.part_o + pr * D, r, tx);
      continue;
    }
    const float inv = f.l[r] > 0.0f ? 1.0f / f.l[r] : 0.0f;
    const int64_t tok = S.q_row0 + w.tok0 + row / P.group;
    const int h = w.hk * P.group + row % P.group;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4<T>(P.out, tok * P.o_tok + h * P.o_head + 64 * c + 4 * tx,
                make_float4(f.o[r][4 * c] * inv, f.o[r][4 * c + 1] * inv, f.o[r][4 * c + 2] * inv,
                            f.o[r][4 * c + 3] * inv));
    if (P.lse && tx == 0)
      P.lse[tok * P.q_heads + h] = win_lse(f.m[r], f.l[r]);
  }
}

// ---- merge of the splits ------------------------------------------------------
// One warp per row of a tile whose keys were split: out = sum_s 2^(m_s - M)
// o_s / sum_s 2^(m_s - M) l_s, splits in order (the same sum on every run).  With a
// segment in pieces the sums go on where those of the piece before ended.
constexpr int kMergeWarps = 8;
template <int T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) window_merge_kernel(const __grid_constant__ WinParams P) {
  pdl_start();
  const int lane = threadIdx.x & 31;
  // blockIdx.x counts the (tile, key head)s of split segments
  int seg = 0;
  for (int lo = 0, hi = P.n_segs - 1; lo <= hi;) {  // the last segment whose first one is not behind it
    const int mid = (lo + hi) >> 1;
    if (P.segs[mid].merge_base <= (int)blockIdx.x) {
      seg = mid;
      lo = mid + 1;
    } else {
      hi = mid - 1;
    }
  }
  const int tile_head = blockIdx.x - P.segs[seg].merge_base;
  const int item = P.segs[seg].item_base + (tile_head / P.kv_heads) * P.segs[seg].n_split * P.kv_heads +
                   tile_head % P.kv_heads;  // its first split
  const WinItem w = win_item(P, item);
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  if (row >= w.n_tok * P.group) return;
  const WinSeg& S = P.segs[w.seg];
  constexpr int V = D / 32;
  const int64_t tok = S.q_row0 + w.tok0 + row / P.group;
  const int h = w.hk * P.group + row % P.group;
  const int64_t state = tok * P.q_heads + h;  // (pieces)
  float m = -INFINITY, l = 0.0f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  if (P.pieces && !P.acc_begin) {
    const float2 ml = P.acc_ml[state];
    m = ml.x, l = ml.y;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = P.acc_o[state * D + lane * V + i];
  }
#pragma unroll 4
  for (int s = 0; s < w.n_split; ++s) {
    const int64_t pr = ((int64_t)w.slot + (int64_t)s * P.kv_heads) * P.tile_rows + row;
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
  if (P.pieces && !P.acc_end) {
    if (lane == 0) P.acc_ml[state] = make_float2(m, l);
#pragma unroll
    for (int i = 0; i < V; ++i) P.acc_o[state * D + lane * V + i] = acc[i];
    return;
  }
  l = win_sum(P, w.pos0 + row / P.group, l);
  const float inv = l > 0.0f ? P.v_scale / l : l;  // (a NaN stays one)
  const int64_t at = tok * P.o_tok + h * P.o_head + lane * V;
  if constexpr (T == KVPOOL_F32) {
#pragma unroll
    for (int i = 0; i < V; ++i) reinterpret_cast<float*>(P.out)[at + i] = acc[i] * inv;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2)
      *reinterpret_cast<__nv_bfloat162*>(P.out + 2 * (at + i)) = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
  }
  if (P.lse && lane == 0) P.lse[tok * P.q_heads + h] = win_lse(m, l);
}

// ---- host plan ------------------------------------------------------------------
constexpr int32_t kMaxLen = 1 << 30;

int check_args(const kvpool_window_args* a, int32_t n, const int64_t* q_len, const int64_t* k_start,
               const int64_t* k_len, int64_t* total_q) {
  if (!a || n < 0) return KVPOOL_ERR_INVALID_ARG;
  if (a->dtype != KVPOOL_F32 && a->dtype != KVPOOL_BF16) return KVPOOL_ERR_INVALID_ARG;
  if (a->head_dim != 64 && a->head_dim != 128) return KVPOOL_ERR_INVALID_ARG;
  if (a->k.heads < 1 || a->v.heads != a->k.heads || a->out.heads != a->q.heads || a->q.heads < a->k.heads ||
      a->q.heads > 1024 || a->q.heads % a->k.heads != 0 || a->q.heads / a->k.heads > kWinMaxGroup)
    return KVPOOL_ERR_INVALID_ARG;
  if (a->window < 0 || a->n_sink < 0 || !std::isfinite(a->scale) || a->q_rows < 0 || a->kv_rows < 0)
    return KVPOOL_ERR_INVALID_ARG;
  if (a->q_rows > 0x7FFFFFFF || a->kv_rows > 0x7FFFFFFF) return KVPOOL_ERR_INVALID_ARG;
  if (!rows_aligned(a->q, a->dtype) || !rows_aligned(a->k, a->dtype) || !rows_aligned(a->v, a->dtype) ||
      !rows_aligned(a->out, a->dtype) || !rows_apart(a->out, a->q_rows, a->head_dim))
    return KVPOOL_ERR_INVALID_ARG;
  if (n > 0 && (!q_len || !k_start || !k_len)) return KVPOOL_ERR_INVALID_ARG;
  int64_t q = 0;
  bool keys = false;
  for (int i = 0; i < n; ++i) {
    if (q_len[i] < 0 || q_len[i] > kMaxLen || k_len[i] < 0 || k_len[i] > kMaxLen) return KVPOOL_ERR_INVALID_ARG;
    if (k_len[i] > 0 && (k_start[i] < 0 || k_start[i] > a->kv_rows - k_len[i])) return KVPOOL_ERR_INVALID_ARG;
    q += q_len[i];
    keys |= q_len[i] > 0 && k_len[i] > 0;
  }
  if (q > a->q_rows) return KVPOOL_ERR_INVALID_ARG;
  if (q > 0 && (!a->q.data || !a->out.data)) return KVPOOL_ERR_INVALID_ARG;
  if (keys && (!a->k.data || !a->v.data)) return KVPOOL_ERR_INVALID_ARG;
  *total_q = q;
  return KVPOOL_OK;
}

// Does the output lie on rows that the call reads, other than as its queries
// themselves?  (A tile's queries are read by the CTAs that write its outputs,
// or by a kernel before the one that does.)
bool out_meets_inputs(const kvpool_window_args* a, int32_t n, const int64_t* q_len, const int64_t* k_start,
                      const int64_t* k_len, int64_t total_q) {
  const int64_t vb = a->dtype == KVPOOL_BF16 ? 2 : 4;
  if (!rows_same(a->out, a->q, total_q) && rows_meet(a->out, total_q, a->q, total_q, a->head_dim, vb)) return true;
  int64_t first = INT64_MAX, end = 0;  // K and V rows of the segments
  for (int i = 0; i < n; ++i)
    if (q_len[i] > 0 && k_len[i] > 0) {
      first = std::min(first, k_start[i]);
      end = std::max(end, k_start[i] + k_len[i]);
    }
  if (first >= end) return false;
  for (kvpool_heads h : {a->k, a->v}) {
    h.data = static_cast<const uint8_t*>(h.data) + vb * first * h.token_stride;
    if (rows_meet(a->out, total_q, h, end - first, a->head_dim, vb)) return true;
  }
  return false;
}

// ---- which kernel takes a segment ------------------------------------------------
enum Form { kFormTok, kFormTc, kFormFma, kForms };

// The tensor copies' limits: strides of used axes positive and below 2^40
// bytes; the softmax takes the maximum before the scale, so that is positive.
bool tc_able(const kvpool_window_args* a) {
  if (a->dtype != KVPOOL_BF16 || !(a->scale > 0.0f)) return false;
  auto ok = [](int64_t stride, int64_t extent) { return extent <= 1 || (stride > 0 && stride < (1ll << 38)); };
  return ok(a->q.token_stride, a->q_rows) && ok(a->q.head_stride, a->q.heads) && ok(a->q.head_stride * 16, a->k.heads) &&
         ok(a->k.token_stride, a->kv_rows) && ok(a->k.head_stride, a->k.heads) && ok(a->v.token_stride, a->kv_rows) &&
         ok(a->v.head_stride, a->v.heads);
}

Form form_of(const kvpool_window_args* a, bool tc, const WinDense* dense, int64_t q_len, int64_t k_len) {
  const int64_t rows = q_len * (a->q.heads / a->k.heads);
  return rows <= kTokRows && !dense ? kFormTok : tc && k_len > 0 ? kFormTc : kFormFma;
}

// the most keys that a tile of the segment sees
int64_t tile_keys(const kvpool_window_args* a, int64_t q_len, int64_t k_len, int tile_tokens) {
  const int64_t w = (int64_t)a->window + std::min<int64_t>(tile_tokens, q_len) + a->n_sink;
  return std::min<int64_t>(k_len, w);
}

// Long key lists under few query tiles (no window): the length of parts, each a
// work item, that makes k rounds of one item to every multiprocessor shortest, an
// item taking as long as 256 keys beside its own (two prompts of 1,024 and 768
// queries, 16 heads on 4, behind up to 32,768 tokens read back from a 4-bit cache:
// 360 us a call whole, 263 in parts).
int64_t even_part(const kvpool_window_args* a, const WinParams& P, int n_sms) {
  auto items = [&](int64_t part) {
    int64_t x = 0;
    for (int s = 0; s < P.n_segs; ++s) {
      const WinSeg& S = P.segs[s];
      const int64_t keys = std::max<int64_t>(1, tile_keys(a, S.q_len, S.k_len, P.tile_tokens));
      x += (int64_t)((S.q_len + P.tile_tokens - 1) / P.tile_tokens) * a->k.heads * ((keys + part - 1) / part);
    }
    return x;
  };
  const int64_t whole = items(kMaxLen);
  int64_t best = kMaxLen, cost = INT64_MAX;
  for (int64_t k = 1; k <= 6; ++k) {
    if (k * n_sms < whole) continue;
    int64_t lo = 1, hi = kMaxLen / 128;  // in steps of 128 keys
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (items(128 * mid) <= k * n_sms) hi = mid;
      else lo = mid + 1;
    }
    if (k * (128 * lo + 256) < cost) cost = k * (128 * lo + 256), best = 128 * lo;
  }
  return best;
}

// Keys of a bf16 single-token item at most: the tensor core cuts its sums off instead
// of rounding them (about 2^-23 of the sum each time), and a warp's outputs are one
// sum of two products for every 64 keys of the item.  160 requests behind 1,048,576
// tokens, uncut: outputs 0.18% too small (values of one sign; error 2.4e-3 of their
// norm, their rounding alone 1.69e-3), in parts of it 1.69e-3 (50.1 -> 39.6 ms: more
// items, evener waves).
constexpr int64_t kTokSumKeys = 65536;

// Fill segments [i0, n) of one launch (at most kMaxWinSegs with queries);
// returns the next segment.  A launch with few tiles cuts each tile's keys
// into parts (merged by a second kernel) so that the GPU is filled.
int plan_launch(const kvpool_window_args* a, Form form, bool tc, const WinDense* dense, int32_t i0, int32_t n,
                const int64_t* q_len, const int64_t* k_start, const int64_t* k_len, int64_t q_row0, int n_sms, WinParams* P, int64_t* next_row,
                int64_t* slots) {
  const int Hk = a->k.heads;
  int64_t most = 1;  // queries of a single-token segment
  if (form == kFormTok)
    for (int j = i0, m = 0; j < n && m < kMaxWinSegs; ++j)
      if (q_len[j] > 0 && form_of(a, tc, dense, q_len[j], k_len[j]) == form) most = std::max(most, q_len[j]), ++m;
  P->tile_tokens = form == kFormTok  ? (int32_t)most
                   : form == kFormTc ? 2 * (kTcTileRows / P->group)
                                     : kFmaRows / P->group;
  P->tile_rows = P->tile_tokens * P->group;
  int i = i0;
  P->n_segs = 0;
  int64_t tiles = 0;
  for (; i < n && P->n_segs < kMaxWinSegs; ++i) {
    if (q_len[i] > 0 && form_of(a, tc, dense, q_len[i], k_len[i]) == form) {
      WinSeg& S = P->segs[P->n_segs++];
      S = WinSeg{};
      S.q_row0 = q_row0;
      S.k_start = k_len[i] > 0 ? k_start[i] : 0;
      S.q_len = (int32_t)q_len[i];
      S.k_len = (int32_t)k_len[i];
      tiles += (int64_t)((q_len[i] + P->tile_tokens - 1) / P->tile_tokens) * Hk;
    }
    q_row0 += q_len[i];
  }
  *next_row = q_row0;
  // Work items that fill the GPU, and the fewest keys of one.  Tensor-core and
  // single-token items are counted down to one wave (one and four CTAs to a
  // multiprocessor; a few past it would double the time); fp32 ones up (prompts
  // of 1,021 tokens: 53, 41, 44, 46 us at 2, 4, 6, 8 to a multiprocessor).
  const int64_t min_keys = form == kFormTok ? 256 : form == kFormTc ? 128 : kFmaKeys;
  const int64_t want = n_sms * (form == kFormTc ? 1LL : 4LL);
  const int64_t fill = tiles == 0 ? 1 : form == kFormFma ? (want + tiles - 1) / tiles : std::max<int64_t>(1, want / tiles);
  const int64_t part = dense && form == kFormTc && tiles > 0 ? even_part(a, *P, n_sms) : 0;
  int64_t items = 0, slot = 0, merge = 0, rows = 0;
  for (int s = 0; s < P->n_segs; ++s) {
    WinSeg& S = P->segs[s];
    const int64_t st = (int64_t)((S.q_len + P->tile_tokens - 1) / P->tile_tokens) * Hk;
    const int64_t keys = tile_keys(a, S.q_len, S.k_len, P->tile_tokens);
    int64_t split = std::max<int64_t>(1, part > 0 ? (keys + part - 1) / part : std::min(fill, (keys + min_keys - 1) / min_keys));
    if (form == kFormTok && a->dtype == KVPOOL_BF16) split = std::max(split, (keys + kTokSumKeys - 1) / kTokSumKeys);
    S.n_split = (int32_t)split;
    S.item_base = (int32_t)items;
    S.part_base = (int32_t)slot;
    S.merge_base = (int32_t)merge;
    items += st * split;
    if (split > 1 || P->pieces) {
      slot += st * split;
      merge += st;
      rows = std::max<int64_t>(rows, std::min<int64_t>(S.q_len, P->tile_tokens) * P->group);
    }
  }
  // the longest sum, in steps (first tokens and window apart)
  int64_t steps = 0;
  for (int s = 0; form == kFormTc && s < P->n_segs; ++s) {
    const int64_t all = tile_keys(a, P->segs[s].q_len, P->segs[s].k_len, P->tile_tokens) / 128 + 2;
    steps = std::max(steps, (all + P->segs[s].n_split - 1) / P->segs[s].n_split);
  }
  P->long_sums = steps > kTcSumSteps;
  P->n_items = items <= (1 << 30) ? (int32_t)items : -1;
  P->n_merge = (int32_t)merge;
  P->merge_rows = (int32_t)rows;
  *slots = slot;
  return i;
}

void fill_params(const kvpool_window_args* a, const WinDense* dense, WinParams* P) {
  const WinDense d = dense ? *dense : WinDense{};
  P->pieces = d.pieces;
  P->acc_begin = d.begin;
  P->acc_end = d.end;
  P->behind = (int32_t)d.behind;
  P->acc_o = d.acc_o;
  P->acc_ml = d.acc_ml;
  P->dense = dense != nullptr;
  P->v_scale = d.v_scale;
  P->q = static_cast<const uint8_t*>(a->q.data);
  P->k = static_cast<const uint8_t*>(a->k.data);
  P->v = static_cast<const uint8_t*>(a->v.data);
  P->out = static_cast<uint8_t*>(const_cast<void*>(a->out.data));
  P->lse = a->d_lse;
  P->q_tok = a->q.token_stride;
  P->q_head = a->q.head_stride;
  P->k_tok = a->k.token_stride;
  P->k_head = a->k.head_stride;
  P->v_tok = a->v.token_stride;
  P->v_head = a->v.head_stride;
  P->o_tok = a->out.token_stride;
  P->o_head = a->out.head_stride;
  P->q_heads = a->q.heads;
  P->kv_heads = a->k.heads;
  P->group = a->q.heads / a->k.heads;
  P->window = std::min(a->window, kMaxLen);
  P->n_sink = std::min(a->n_sink, kMaxLen);
  P->scale_log2 = a->scale * 1.4426950408889634f;
}

// A launch's workspace: partial outputs, their maxima and sums, and the tensor-core form's sums.
struct WinSpace {
  int64_t part_ml, sums, total;
};
WinSpace win_space(const WinParams& P, int head_dim, int64_t slots, int n_sms) {
  WinSpace w;
  w.part_ml = slots * P.tile_rows * head_dim * 4;
  w.sums = (w.part_ml + slots * P.tile_rows * 8 + 15) / 16 * 16;
  const int64_t ctas = P.long_sums ? std::min<int64_t>(P.n_items, n_sms) : 0;
  w.total = w.sums + ctas * 2 * kTcTileRows * (head_dim + 1) * 4;
  return w;
}

template <int T, int D>
cudaError_t launch_fma(const WinParams& P, cudaStream_t s) {
  constexpr int smem = (int)sizeof(FmaSmem<D>);
  auto* kern = window_fma_kernel<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e == cudaSuccess ? launch_kernel(true, kern, dim3(P.n_items), dim3(kFmaThreads), smem, s, P) : e;
}

template <int T, int D>
cudaError_t launch_merge(const WinParams& P, cudaStream_t s) {
  return launch_kernel(true, window_merge_kernel<T, D>, dim3(P.n_merge, (P.merge_rows + kMergeWarps - 1) / kMergeWarps),
                       dim3(kMergeWarps * 32), 0, s, P);
}

}  // namespace

int device_sms() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if ((sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return 0;
  known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

const OpsDevice* ops_device() {
  static std::mutex mu;
  static OpsDevice info[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  OpsDevice& d = info[dev];
  if (!d.err) {
    void* p = nullptr;
    const int sms = device_sms();
    if (sms < 1 || cudaGetSymbolAddress(&p, g_ops_error) != cudaSuccess || !p) return nullptr;
    d.sms = sms;
    d.err = static_cast<uint32_t*>(p);
  }
  return &d;
}

bool window_tc_able(const kvpool_window_args* a) { return tc_able(a); }

int64_t window_space(const kvpool_window_args* a, int32_t n, const int64_t* h_q_len, const int64_t* h_k_start,
                     const int64_t* h_k_len, const WinDense* dense) {
  int64_t total = 0;
  const int rc = check_args(a, n, h_q_len, h_k_start, h_k_len, &total);
  if (rc != KVPOOL_OK) return rc;
  if (total == 0) return 0;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  const int sms = dev->sms;
  std::unique_ptr<WinParams> P(new (std::nothrow) WinParams);
  if (!P) return KVPOOL_ERR_INVALID_ARG;
  fill_params(a, dense, P.get());
  const bool tc = tc_able(a);
  int64_t most = 0;
  for (int f = 0; f < kForms; ++f)
    for (int64_t i = 0, row = 0, slots = 0; i < n;) {
      i = plan_launch(a, (Form)f, tc, dense, (int32_t)i, n, h_q_len, h_k_start, h_k_len, row, sms, P.get(), &row, &slots);
      if (P->n_items < 0) return KVPOOL_ERR_INVALID_ARG;
      if (P->n_segs > 0) most = std::max(most, win_space(*P, a->head_dim, slots, sms).total);
    }
  return most;
}

int window_run(const kvpool_window_args* a, int32_t n, const int64_t* h_q_len, const int64_t* h_k_start,
               const int64_t* h_k_len, const WinDense* dense, void* d_workspace, int64_t workspace_bytes, void* stream) {
  int64_t total = 0;
  const int rc = check_args(a, n, h_q_len, h_k_start, h_k_len, &total);
  if (rc != KVPOOL_OK) return rc;
  if (total == 0) return KVPOOL_OK;
  if (out_meets_inputs(a, n, h_q_len, h_k_start, h_k_len, total)) return KVPOOL_ERR_INVALID_ARG;
  const int64_t need = window_space(a, n, h_q_len, h_k_start, h_k_len, dense);
  if (need < 0) return (int)need;
  if (need > 0 && (!d_workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(d_workspace) % 16 != 0))
    return KVPOOL_ERR_INVALID_ARG;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  const int sms = dev->sms;
  std::unique_ptr<WinParams> P(new (std::nothrow) WinParams);
  if (!P) return KVPOOL_ERR_INVALID_ARG;
  fill_params(a, dense, P.get());
  P->err = dev->err;
  const bool tc = tc_able(a);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for (int f = 0; f < kForms; ++f)
    for (int64_t i = 0, row = 0, slots = 0; i < n;) {
      i = plan_launch(a, (Form)f, tc, dense, (int32_t)i, n, h_q_len, h_k_start, h_k_len, row, sms, P.get(), &row, &slots);
      if (P->n_segs == 0) continue;
      const WinSpace w = win_space(*P, a->head_dim, slots, sms);
      uint8_t* space = static_cast<uint8_t*>(d_workspace);
      P->part_o = reinterpret_cast<float*>(space);
      P->part_ml = reinterpret_cast<float2*>(space + w.part_ml);
      P->sums = reinterpret_cast<float*>(space + w.sums);
      cudaError_t e = cudaSuccess;
      if (f == kFormTok) e = (cudaError_t)launch_window_tok(*P, a->dtype, a->head_dim, stream);
      else if (f == kFormTc) e = (cudaError_t)launch_window_tc(*P, a->head_dim, a->q_rows, a->kv_rows, sms, stream);
      else if (a->dtype == KVPOOL_F32)
        e = a->head_dim == 128 ? launch_fma<KVPOOL_F32, 128>(*P, s) : launch_fma<KVPOOL_F32, 64>(*P, s);
      else
        e = a->head_dim == 128 ? launch_fma<KVPOOL_BF16, 128>(*P, s) : launch_fma<KVPOOL_BF16, 64>(*P, s);
      if (e == cudaSuccess && slots > 0) {
        if (a->dtype == KVPOOL_F32)
          e = a->head_dim == 128 ? launch_merge<KVPOOL_F32, 128>(*P, s) : launch_merge<KVPOOL_F32, 64>(*P, s);
        else
          e = a->head_dim == 128 ? launch_merge<KVPOOL_BF16, 128>(*P, s) : launch_merge<KVPOOL_BF16, 64>(*P, s);
      }
      if (e != cudaSuccess) return KVPOOL_ERR_CUDA;
    }
  return KVPOOL_OK;
}

}  // namespace kvp

extern "C" int64_t kvpool_window_workspace(const kvpool_window_args* a, int32_t n, const int64_t* h_q_len,
                                           const int64_t* h_k_start, const int64_t* h_k_len) {
  return kvp::window_space(a, n, h_q_len, h_k_start, h_k_len, nullptr);
}

extern "C" int kvpool_window_attend(const kvpool_window_args* a, int32_t n, const int64_t* h_q_len,
                                    const int64_t* h_k_start, const int64_t* h_k_len, void* d_workspace,
                                    int64_t workspace_bytes, void* stream) {
  return kvp::window_run(a, n, h_q_len, h_k_start, h_k_len, nullptr, d_workspace, workspace_bytes, stream);
}

extern "C" int kvpool_window_check(void* stream, uint32_t* h_flags) {
  using namespace kvp;
  uint32_t word = 0;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  uint32_t* err = dev->err;
  const uint32_t zero = 0;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess ||
      cudaMemcpy(&word, err, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess ||
      (word && cudaMemcpy(err, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess))
    return KVPOOL_ERR_CUDA;
  if (h_flags) *h_flags = word;
  return word == 0 ? KVPOOL_OK : KVPOOL_ERR_DEVICE_CHECK;
}
