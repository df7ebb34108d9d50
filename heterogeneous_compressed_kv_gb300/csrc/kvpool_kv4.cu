// kvpool_kv4.cu -- tokens into the 4-bit paged cache and back out.
//
// Of 16 neighbouring values x of a head the cache holds s = e4m3(amax / 6), amax
// their largest magnitude, and the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to x / s
// (ties to the even code); s times such a number has at most 6 bits, so what is
// read back is exact in bf16.
//
// Bound: memory, at sizes that fill the GPU; the smallest call is one launch.  A
// warp takes a tile of 16 tokens of one head, so that no two warps share a byte
// (two tokens' values do), and asks for all of it before it needs the first row.
// Measured (bf16, 16 heads of 128): 6,656 tokens stored 13.4 us (69.9 MB, 0.77 of
// the copy rate; a value takes 8 instructions, the integer pipe is the next bound),
// read back 9.3 us (the cache and much of the output stay in L2); 65,536 tokens of
// 8 heads read back 53.9 us, 6.4 TB/s (0.94); 32 tokens 3.9 and 2.4 us.  fp32, the
// same 6,656 tokens: stored 48.5 us (124 MB, 0.38; a division for every value bounds
// it), read back 32.0 (0.57).
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include <cuda_runtime.h>

#include "kvpool_kv4.h"
#include "kvpool_pair.cuh"
#include "kvpool_rows.h"

namespace kvp {
namespace {

constexpr int kWarps = 4;

struct MoveSeg {
  int64_t row0;   // first row of k and v
  int32_t start;  // position of the first token
  int32_t n;
  int32_t task_base;  // first task: tile * kv_heads + head
  int32_t table_row;
};

struct MoveParams {
  Kv4Cache c;
  const uint8_t* k;
  const uint8_t* v;
  int64_t k_tok, k_head, v_tok, v_head;  // strides in bytes
  int32_t n_segs, n_tasks;
  MoveSeg segs[kKv4MaxSegs];
};

struct MoveTask {
  int head, tile, lo, hi;  // the segment's tokens of the tile: slots lo .. hi - 1
  int64_t row;             // k and v row of slot 0
  int64_t off;             // the tile's place in the pages, < 0: a bad page id
};

template <int D>
__device__ __forceinline__ MoveTask move_task(const MoveParams& P, int task) {
  int lo = 0, hi = P.n_segs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.segs[mid].task_base <= task) lo = mid;
    else hi = mid - 1;
  }
  const MoveSeg& S = P.segs[lo];
  const int r = task - S.task_base;
  MoveTask t;
  t.head = r % P.c.kv_heads;
  t.tile = S.start / kKv4Tile + r / P.c.kv_heads;
  const int first = t.tile * kKv4Tile;  // (at most 2^30)
  t.lo = max(0, S.start - first);
  t.hi = min(kKv4Tile, S.start + S.n - first);
  t.row = S.row0 + (first - S.start);
  const int id = kv4_page(P.c, S.table_row, t.tile);
  t.off = id < 0 ? -1 : kv4_tile_offset<D>(P.c, id, t.head, t.tile);
  return t;
}

// 8 values of a row as loaded
template <int T>
struct Raw8;
template <>
struct Raw8<KVPOOL_BF16> {
  uint4 r;
  __device__ __forceinline__ void load(const uint8_t* p, bool in) {
    r = in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<KVPOOL_F32> {
  float4 a, b;
  __device__ __forceinline__ void load(const uint8_t* p, bool in) {
    a = b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <int T>
__device__ __forceinline__ void store8(uint8_t* p, const float* x) {
  if constexpr (T == KVPOOL_F32) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The scale of a group, of which a lane has one half and its neighbour the other,
// and what quotients by it are made with: a code, and its value or a multiple of
// its reciprocal.  A NaN or an infinity makes the scale NaN: the whole group reads
// back as NaN.
template <int T>
struct Scale {
  uint32_t code;
  float by;
};

__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ Scale<KVPOOL_F32> scale_of(const Raw8<KVPOOL_F32>& raw, float inv_scale) {
  float x[8];
  raw.get(x);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  if (amax >= 0x7F800000u) return {0x7F, 0.0f};
  const float top = __uint_as_float(amax) * inv_scale;  // (a power of two; past fp32's range: the largest scale)
  const uint32_t s = f32x2_to_e4m3x2(__fdiv_rn(top, 6.0f), 0.0f) & 0xFFu;
  return {s, e4m3x2_to_f32x2((uint16_t)s).x};
}

// For bf16 a product with a reciprocal stands for the quotient.  With a rounding
// that brings a quotient that is a border between two codes back to it: a bf16
// number (8 bits) is 6 times a border between two scales (5 bits), or a border
// between two codes times a scale (7 bits), or at least 2^-8 of it away, where the
// product is off by 2^-22 of it and the rounding (to fp16's 11 bits; to multiples of
// 2^-11 beside borders from 0.25 to 5) by less than 2^-10.  (With quotients 6,656
// tokens of 16 heads x 128 took 30.9 us.)
__device__ __forceinline__ Scale<KVPOOL_BF16> scale_of(const Raw8<KVPOOL_BF16>& raw, float inv_scale) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t m = max_abs_bf16x2(max_abs_bf16x2(raw.r.x & kAbs, raw.r.y & kAbs), max_abs_bf16x2(raw.r.z & kAbs, raw.r.w & kAbs));
  m = max_abs_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t amax = max(m << 16, m & 0xFFFF0000u);  // (NaN is the largest)
  if (amax >= 0x7F800000u) return {0x7F, 0.0f};
  const float top = __uint_as_float(amax) * inv_scale;  // (a power of two; past fp32's range: the largest scale)
  uint16_t s;
  asm("{.reg .b32 h;\n\tcvt.rn.f16x2.f32 h, %1, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 %0, h;}" : "=h"(s) : "f"(top * (1.0f / 6.0f)));
  const float f = e4m3x2_to_f32x2(s).x;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(f));
  return {s & 0xFFu, f > 0.0f ? r * inv_scale : 0.0f};
}

// eight values' quotients, as the codes' rounding takes them
__device__ __forceinline__ void quotients(const Raw8<KVPOOL_F32>& raw, float inv_scale, const Scale<KVPOOL_F32>& s, float* q) {
  raw.get(q);
  // The fp32 quotient stands for x / s: it lies on a border between two codes only
  // where x / s does (x and border * s are fp32 numbers, so unequal ones differ by
  // more than the quotient's rounding).
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = s.by > 0.0f ? __fdiv_rn(q[i] * inv_scale, s.by) : 0.0f;
}
__device__ __forceinline__ void quotients(const Raw8<KVPOOL_BF16>& raw, float, const Scale<KVPOOL_BF16>& s, float* q) {
  raw.get(q);
  constexpr float kGrid = 6144.0f;  // 1.5 * 2^12: a sum with it is a multiple of 2^-11 (what is beyond 6 stays there)
  const uint64_t by = pack2(s.by, s.by), up = pack2(kGrid, kGrid), down = pack2(-kGrid, -kGrid);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = unpack2(add2(fma2(pack2(q[2 * i], q[2 * i + 1]), by, up), down));
    q[2 * i] = y.x, q[2 * i + 1] = y.y;
  }
}

// byte i: the codes of a[i] (low nibble) and b[i]
__device__ __forceinline__ uint32_t codes4(float a0, float b0, float a1, float b1, float a2, float b2, float a3, float b3) {
  uint32_t r;
  asm("{.reg .b8 t0, t1, t2, t3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
      "mov.b32 %0, {t0, t1, t2, t3};}"
      : "=r"(r)
      : "f"(a0), "f"(b0), "f"(a1), "f"(b1), "f"(a2), "f"(b2), "f"(a3), "f"(b3));
  return r;
}

// A warp takes a tile of one head: the lanes of a row hold 8 dims each.  All of
// its loads are on their way before the first is needed.
template <int T, int D>
__global__ void __launch_bounds__(kWarps * 32) kv4_store_kernel(const __grid_constant__ MoveParams P) {
  pdl_start();
  using L = Kv4Tile<D>;
  const int task = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (task >= P.n_tasks) return;
  const MoveTask t = move_task<D>(P, task);
  if (t.off < 0) return;
  uint8_t* tile = P.c.pages + t.off;
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a row, rows at a time
  constexpr int kK = kKv4Tile / kPer, kV = kKv4Tile / 2 / kPer;  // steps over the keys, the pairs of values
  constexpr int vb = T == KVPOOL_F32 ? 4 : 2;
  const int sub = lane / kLanes, l = lane % kLanes;
  const uint8_t* k = P.k + t.row * P.k_tok + t.head * P.k_head + 8 * vb * l;
  const uint8_t* v = P.v + t.row * P.v_tok + t.head * P.v_head + 8 * vb * l;
  const float k_inv = 1.0f / P.c.k_scale, v_inv = 1.0f / P.c.v_scale;
  Raw8<T> rk[kK], rv[kV][2];
#pragma unroll
  for (int it = 0; it < kK; ++it) {
    const int r = it * kPer + sub;
    rk[it].load(k + r * P.k_tok, r >= t.lo && r < t.hi);
  }
#pragma unroll
  for (int it = 0; it < kV; ++it)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int r = 2 * (it * kPer + sub) + y;
      rv[it][y].load(v + r * P.v_tok, r >= t.lo && r < t.hi);
    }
#pragma unroll
  for (int it = 0; it < kK; ++it) {
    const int r = it * kPer + sub;
    const bool in = r >= t.lo && r < t.hi;
    if (!__any_sync(0xffffffffu, in)) continue;
    const auto s = scale_of(rk[it], k_inv);
    float q[8];
    quotients(rk[it], k_inv, s, q);
    if (in) {
      *reinterpret_cast<uint32_t*>(tile + r * (D / 2) + 4 * l) = codes4(q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]);
      if (l % 2 == 0) tile[L::kKs + r * (D / kKv4Group) + l / 2] = (uint8_t)s.code;
    }
  }
#pragma unroll
  for (int it = 0; it < kV; ++it) {
    const int j = it * kPer + sub, r = 2 * j;
    const bool in0 = r >= t.lo && r < t.hi, in1 = r + 1 >= t.lo && r + 1 < t.hi;
    if (!__any_sync(0xffffffffu, in0 || in1)) continue;
    const auto s0 = scale_of(rv[it][0], v_inv), s1 = scale_of(rv[it][1], v_inv);
    float q0[8], q1[8];
    quotients(rv[it][0], v_inv, s0, q0);
    quotients(rv[it][1], v_inv, s1, q1);
    if (!in0 && !in1) continue;
    const int chunk = 8 * l / L::kChunk, at = 8 * l % L::kChunk;
    uint2* p = reinterpret_cast<uint2*>(tile + L::kV + j * D + (chunk ^ kv4_swizzle<D>(j)) * L::kChunk + at);
    const uint2 w = make_uint2(codes4(q0[0], q1[0], q0[1], q1[1], q0[2], q1[2], q0[3], q1[3]),
                               codes4(q0[4], q1[4], q0[5], q1[5], q0[6], q1[6], q0[7], q1[7]));
    uint8_t* sc = tile + L::kVs + j * (D / 8) + l / 2 * 2;
    if (in0 && in1) {
      *p = w;
      if (l % 2 == 0) *reinterpret_cast<uint16_t*>(sc) = (uint16_t)(s0.code | s1.code << 8);
    } else {  // the pair's other token stays
      const uint32_t mine = in0 ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
      const uint2 old = *p;
      *p = make_uint2((w.x & mine) | (old.x & ~mine), (w.y & mine) | (old.y & ~mine));
      if (l % 2 == 0) sc[in0 ? 0 : 1] = (uint8_t)(in0 ? s0.code : s1.code);
    }
  }
}

// HALVES: values as fp16 numbers and without v_scale (codes times their scale are
// exact in fp16, and then in a product of fp16 numbers)
template <int T, int D, bool HALVES>
__global__ void __launch_bounds__(kWarps * 32) kv4_load_kernel(const __grid_constant__ MoveParams P) {
  pdl_start();
  using L = Kv4Tile<D>;
  const int task = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (task >= P.n_tasks) return;
  const MoveTask t = move_task<D>(P, task);
  const bool bad = t.off < 0;  // reads as zeros
  const uint8_t* tile = P.c.pages + (bad ? 0 : t.off);
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;
  constexpr int kK = kKv4Tile / kPer, kV = kKv4Tile / 2 / kPer;
  constexpr int vb = T == KVPOOL_F32 ? 4 : 2;
  const int sub = lane / kLanes, l = lane % kLanes;
  uint8_t* k = const_cast<uint8_t*>(P.k) + t.row * P.k_tok + t.head * P.k_head + 8 * vb * l;
  uint8_t* v = const_cast<uint8_t*>(P.v) + t.row * P.v_tok + t.head * P.v_head + 8 * vb * l;
  uint32_t kc[kK], ks[kK], vs[kV];
  uint2 vc[kV];
#pragma unroll
  for (int it = 0; it < kK; ++it) {
    const int r = it * kPer + sub;
    kc[it] = bad ? 0 : *reinterpret_cast<const uint32_t*>(tile + r * (D / 2) + 4 * l);
    ks[it] = bad ? 0 : tile[L::kKs + r * (D / kKv4Group) + l / 2];
  }
#pragma unroll
  for (int it = 0; it < kV; ++it) {
    const int j = it * kPer + sub, chunk = 8 * l / L::kChunk, at = 8 * l % L::kChunk;
    vc[it] = make_uint2(0, 0);
    vs[it] = 0;
    if (bad) continue;
    vc[it] = *reinterpret_cast<const uint2*>(tile + L::kV + j * D + (chunk ^ kv4_swizzle<D>(j)) * L::kChunk + at);
    vs[it] = *reinterpret_cast<const uint16_t*>(tile + L::kVs + j * (D / 8) + l / 2 * 2);
  }
#pragma unroll
  for (int it = 0; it < kK; ++it) {
    const int r = it * kPer + sub;
    if (r < t.lo || r >= t.hi) continue;
    uint32_t h[4];
    const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)(ks[it] | ks[it] << 8));
    e2m1x8_to_f16x2x4(kc[it], h);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_f16(mul_f16x2(h[i], s2));
      x[2 * i] = f.x * P.c.k_scale;
      x[2 * i + 1] = f.y * P.c.k_scale;
    }
    store8<T>(k + r * P.k_tok, x);
  }
#pragma unroll
  for (int it = 0; it < kV; ++it) {
    const int r = 2 * (it * kPer + sub);
    const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)vs[it]);
    uint32_t h[8];
    e2m1x8_to_f16x2x4(vc[it].x, h);
    e2m1x8_to_f16x2x4(vc[it].y, h + 4);
    const bool in0 = r >= t.lo && r < t.hi, in1 = r + 1 >= t.lo && r + 1 < t.hi;
    if constexpr (HALVES) {
      uint32_t x[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = mul_f16x2(h[2 * i], s2), b = mul_f16x2(h[2 * i + 1], s2);
        x[0][i] = __byte_perm(a, b, 0x5410);
        x[1][i] = __byte_perm(a, b, 0x7632);
      }
      if (in0) *reinterpret_cast<uint4*>(v + r * P.v_tok) = make_uint4(x[0][0], x[0][1], x[0][2], x[0][3]);
      if (in1) *reinterpret_cast<uint4*>(v + (r + 1) * P.v_tok) = make_uint4(x[1][0], x[1][1], x[1][2], x[1][3]);
    } else {
      float x0[8], x1[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = unpack_f16(mul_f16x2(h[i], s2));
        x0[i] = f.x * P.c.v_scale;
        x1[i] = f.y * P.c.v_scale;
      }
      if (in0) store8<T>(v + r * P.v_tok, x0);
      if (in1) store8<T>(v + (r + 1) * P.v_tok, x1);
    }
  }
}

bool power_of_two(float x) {
  int e;
  return x > 0.0f && std::isfinite(x) && std::frexp(x, &e) == 0.5f && e - 1 >= -16 && e - 1 <= 16;
}

enum Move { kStore, kLoad, kLoadHalves };
template <int T, int D>
cudaError_t launch_move(Move what, const MoveParams& P, cudaStream_t s) {
  const dim3 grid((unsigned)((P.n_tasks + kWarps - 1) / kWarps)), block(kWarps * 32);
  if constexpr (T == KVPOOL_BF16)
    if (what == kLoadHalves) return launch_kernel(true, kv4_load_kernel<T, D, true>, grid, block, 0, s, P);
  return what == kStore ? launch_kernel(true, kv4_store_kernel<T, D>, grid, block, 0, s, P)
                        : launch_kernel(true, kv4_load_kernel<T, D, false>, grid, block, 0, s, P);
}

int move_rows(Move what, const kvpool_kv4* c, int32_t dtype, const kvpool_heads& k, const kvpool_heads& v, int32_t n,
              int64_t row0, const int64_t* start, const int64_t* len, uint32_t* err, void* stream) {
  std::unique_ptr<MoveParams> P(new (std::nothrow) MoveParams);
  if (!P) return KVPOOL_ERR_INVALID_ARG;
  const int64_t vb = dtype == KVPOOL_BF16 ? 2 : 4;
  P->k = static_cast<const uint8_t*>(k.data);
  P->v = static_cast<const uint8_t*>(v.data);
  P->k_tok = k.token_stride * vb;
  P->k_head = k.head_stride * vb;
  P->v_tok = v.token_stride * vb;
  P->v_head = v.head_stride * vb;
  int64_t row = 0;
  for (int32_t i = 0; i < n;) {
    const int32_t first = i;
    P->c = kv4_cache(c, row0 + first, err);
    P->n_segs = 0;
    int64_t tasks = 0;
    for (; i < n && P->n_segs < kKv4MaxSegs; ++i) {
      if (len[i] == 0) continue;
      const int64_t tiles = (start[i] + len[i] - 1) / kKv4Tile - start[i] / kKv4Tile + 1;
      if (tasks > 0 && tasks + tiles * c->kv_heads > (1 << 30)) break;  // the next launch takes it
      MoveSeg& S = P->segs[P->n_segs++];
      S.row0 = row;
      S.start = (int32_t)start[i];
      S.n = (int32_t)len[i];
      S.task_base = (int32_t)tasks;
      S.table_row = i - first;
      tasks += tiles * c->kv_heads;
      row += len[i];
    }
    if (P->n_segs == 0) continue;
    if (tasks > 0x7FFFFFFF) return KVPOOL_ERR_INVALID_ARG;
    P->n_tasks = (int32_t)tasks;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == KVPOOL_F32)
      e = c->head_dim == 128 ? launch_move<KVPOOL_F32, 128>(what, *P, s) : launch_move<KVPOOL_F32, 64>(what, *P, s);
    else
      e = c->head_dim == 128 ? launch_move<KVPOOL_BF16, 128>(what, *P, s) : launch_move<KVPOOL_BF16, 64>(what, *P, s);
    if (e != cudaSuccess) return KVPOOL_ERR_CUDA;
  }
  return KVPOOL_OK;
}

// the checks that store and load share
int check_rows(const kvpool_kv4* c, int32_t dtype, const kvpool_heads* k, const kvpool_heads* v, int64_t rows, int32_t n,
               const int64_t* start, const int64_t* len, int64_t* total) {
  if (n < 0 || rows < 0 || rows > 0x7FFFFFFF || !k || !v) return KVPOOL_ERR_INVALID_ARG;
  const int rc = kv4_check(c, n);
  if (rc != KVPOOL_OK) return rc;
  if (dtype != KVPOOL_F32 && dtype != KVPOOL_BF16) return KVPOOL_ERR_INVALID_ARG;
  if (k->heads != c->kv_heads || v->heads != c->kv_heads || !rows_aligned(*k, dtype) || !rows_aligned(*v, dtype))
    return KVPOOL_ERR_INVALID_ARG;
  if (n > 0 && (!start || !len)) return KVPOOL_ERR_INVALID_ARG;
  const int64_t most = kv4_tokens(c);
  int64_t sum = 0, tiles = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (len[i] < 0 || len[i] > most || start[i] < 0 || start[i] > most - len[i]) return KVPOOL_ERR_INVALID_ARG;
    sum += len[i];
    tiles = std::max(tiles, len[i] / kKv4Tile + 2);
  }
  if (sum > rows || tiles * c->kv_heads > (1 << 30)) return KVPOOL_ERR_INVALID_ARG;
  if (sum > 0 && (!k->data || !v->data || !c->d_pages || !c->d_table)) return KVPOOL_ERR_INVALID_ARG;
  const int64_t vb = dtype == KVPOOL_BF16 ? 2 : 4;
  if (kv4_meets(c, *k, sum, vb) || kv4_meets(c, *v, sum, vb)) return KVPOOL_ERR_INVALID_ARG;
  *total = sum;
  return KVPOOL_OK;
}

}  // namespace

int kv4_check(const kvpool_kv4* c, int64_t rows) {
  if (!c || kvpool_kv4_page_bytes(c->kv_heads, c->head_dim, c->page_tokens) < 0) return KVPOOL_ERR_INVALID_ARG;
  if (c->n_pages < 0 || c->n_pages > 0x7FFFFFFF || reinterpret_cast<uintptr_t>(c->d_pages) % 16 != 0)
    return KVPOOL_ERR_INVALID_ARG;
  if (c->table_rows < 0 || rows > c->table_rows || c->table_width < 0 || c->table_stride < 0 ||
      reinterpret_cast<uintptr_t>(c->d_table) % 4 != 0)
    return KVPOOL_ERR_INVALID_ARG;
  if (kv4_tokens(c) > (1 << 30)) return KVPOOL_ERR_INVALID_ARG;
  if (!power_of_two(c->k_scale) || !power_of_two(c->v_scale)) return KVPOOL_ERR_INVALID_ARG;
  return KVPOOL_OK;
}

namespace {
__int128 page_bytes(const kvpool_kv4* c) {
  return (__int128)c->n_pages * kvpool_kv4_page_bytes(c->kv_heads, c->head_dim, c->page_tokens);
}
__int128 table_bytes(const kvpool_kv4* c) {
  return c->table_rows > 0 && c->table_width > 0 ? 4 * ((__int128)(c->table_rows - 1) * c->table_stride + c->table_width) : 0;
}
}  // namespace

bool kv4_meets(const kvpool_kv4* c, const kvpool_heads& h, int64_t n, int64_t vb) {
  return rows_touch(h, n, c->head_dim, vb, c->d_pages, page_bytes(c)) || rows_touch(h, n, c->head_dim, vb, c->d_table, table_bytes(c));
}

bool kv4_meets(const kvpool_kv4* c, const void* p, __int128 bytes) {
  auto touch = [&](const void* q, __int128 n) {
    const __int128 a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && bytes > 0 && n > 0 && a < b + n && b < a + bytes;
  };
  return touch(c->d_pages, page_bytes(c)) || touch(c->d_table, table_bytes(c));
}

bool kv4_meets(const kvpool_kv4* c, const float* w, int64_t n, int64_t seg_stride, int64_t head_stride, int64_t len) {
  return runs_touch(w, n, seg_stride, c->kv_heads, head_stride, len, c->d_pages, page_bytes(c)) ||
         runs_touch(w, n, seg_stride, c->kv_heads, head_stride, len, c->d_table, table_bytes(c));
}

Kv4Cache kv4_cache(const kvpool_kv4* c, int64_t row0, uint32_t* err) {
  Kv4Cache C{};
  C.pages = static_cast<uint8_t*>(c->d_pages);
  C.table = c->d_table + row0 * c->table_stride;
  C.table_stride = c->table_stride;
  C.n_pages = (int32_t)c->n_pages;
  C.kv_heads = c->kv_heads;
  for (int t = c->page_tokens / kKv4Tile; t > 1; t >>= 1) ++C.page_shift;
  C.k_scale = c->k_scale;
  C.v_scale = c->v_scale;
  C.err = err;
  return C;
}

int kv4_load_rows(const kvpool_kv4* c, const kvpool_heads& k, const kvpool_heads& v, int32_t n, int64_t row0,
                  const int64_t* start, const int64_t* len, uint32_t* err, void* stream) {
  return move_rows(kLoadHalves, c, KVPOOL_BF16, k, v, n, row0, start, len, err, stream);
}

}  // namespace kvp

extern "C" int64_t kvpool_kv4_page_bytes(int32_t kv_heads, int32_t head_dim, int32_t page_tokens) {
  if (kv_heads < 1 || kv_heads > kvp::kKv4MaxHeads || (head_dim != 64 && head_dim != 128)) return KVPOOL_ERR_INVALID_ARG;
  if (page_tokens < kvp::kKv4Tile || page_tokens > 1024 || (page_tokens & (page_tokens - 1)) != 0)
    return KVPOOL_ERR_INVALID_ARG;
  return (int64_t)kv_heads * page_tokens * head_dim * 9 / 8;
}

extern "C" int kvpool_kv4_store(const kvpool_kv4* c, int32_t dtype, const kvpool_heads* k, const kvpool_heads* v,
                                int64_t rows, int32_t n, const int64_t* h_start, const int64_t* h_n_new, void* stream) {
  using namespace kvp;
  int64_t total = 0;
  const int rc = check_rows(c, dtype, k, v, rows, n, h_start, h_n_new, &total);
  if (rc != KVPOOL_OK || total == 0) return rc;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  return move_rows(kStore, c, dtype, *k, *v, n, 0, h_start, h_n_new, dev->err, stream);
}

extern "C" int kvpool_kv4_load(const kvpool_kv4* c, int32_t dtype, const kvpool_heads* k, const kvpool_heads* v,
                               int64_t rows, int32_t n, const int64_t* h_start, const int64_t* h_len, void* stream) {
  using namespace kvp;
  int64_t total = 0;
  const int rc = check_rows(c, dtype, k, v, rows, n, h_start, h_len, &total);
  if (rc != KVPOOL_OK) return rc;
  const int64_t vb = dtype == KVPOOL_BF16 ? 2 : 4;
  if (!rows_apart(*k, total, c->head_dim) || !rows_apart(*v, total, c->head_dim) ||
      rows_meet(*k, total, *v, total, c->head_dim, vb))
    return KVPOOL_ERR_INVALID_ARG;
  if (total == 0) return KVPOOL_OK;
  const OpsDevice* dev = ops_device();
  if (!dev) return KVPOOL_ERR_CUDA;
  return move_rows(kLoad, c, dtype, *k, *v, n, 0, h_start, h_len, dev->err, stream);
}
