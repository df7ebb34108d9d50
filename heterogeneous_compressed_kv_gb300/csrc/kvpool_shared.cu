// kvpool_shared.cu -- the HCA entries that a whole decode batch shares, read
// once for all its requests ("Ch 12 Inference framework: heterogeneous KV
// scheduling" s2.2: many requests reference the same blocks).
//
// decode_attend at one query per head streams every request's entries past one
// vector each.  Behind a shared prefix the same entries meet the queries of n
// requests: per head a dense product, scores [n x entries] and outputs [n x
// dim].  A CTA takes one head, a run of the shared entries and a block of
// requests (32 in the FMA form, 64 in the bf16 one), and leaves a partial (max,
// sum, output) per request and head in the slots behind the request's other
// splits; the ordinary merge joins them.
//
// Measured as whole steps of 16 heads x 128 in bf16, no tokens of the requests'
// own (decode_attend in brackets): 32 requests behind 1,024 entries 17.9 us (28.4;
// the shared entries' kernel by itself 6.9), 64 behind 8,192 (kvpool_shared_tc.cu)
// 43.7 us (440).  Where it does not pay (shared_pays) the caller does not come here.
#include <algorithm>

#include <cuda_runtime.h>

#include "device_util.cuh"
#include "kvpool_fma.cuh"
#include "kvpool_internal.h"
#include "kvpool_mma.cuh"
#include "kvpool_shared.h"

namespace kvp {
namespace {

constexpr int kSharedRows = 64;  // requests of a CTA of the small products

// 4 values of a row of codes in fp32 (fp8: without the scale)
template <int T>
__device__ __forceinline__ float4 codes4(const uint8_t* row, int i) {
  if constexpr (T == KVPOOL_F32) {
    return *reinterpret_cast<const float4*>(row + 4 * i);
  } else if constexpr (T == KVPOOL_BF16) {
    const uint2 r = *reinterpret_cast<const uint2*>(row + 2 * i);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
  } else {
    const uint32_t r = *reinterpret_cast<const uint32_t*>(row + i);
    const float2 a = e4m3x2_to_f32x2((uint16_t)(r & 0xFFFFu)), b = e4m3x2_to_f32x2((uint16_t)(r >> 16));
    return make_float4(a.x, a.y, b.x, b.y);
  }
}

// ---- fp32 FMA form: every type ---------------------------------------------------
template <int IN, int CACHE, int D>
__global__ void __launch_bounds__(kFmaThreads) shared_fma_kernel(const __grid_constant__ AttendParams P,
                                                                 const __grid_constant__ SharedShape H) {
  pdl_start();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  FmaSmem<D>& sm = *reinterpret_cast<FmaSmem<D>*>(smem_raw);
  __shared__ float scales[2][kFmaKeys];
  const PoolDesc& pd = P.pool;
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int h = blockIdx.x, split = blockIdx.y, i0 = blockIdx.z * kFmaRows;
  const int rows = min(kFmaRows, P.n - i0);
  const int a = (int)((int64_t)H.n_entries * split / H.n_split);
  const int b = (int)((int64_t)H.n_entries * (split + 1) / H.n_split);
  const float qscale = 1.4426950408889634f * rsqrtf((float)D);
  for (int i = tid; i < kFmaRows * (D / 4); i += kFmaThreads) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
      x = codes4<IN>(static_cast<const uint8_t*>(P.q) + ((int64_t)(P.row0 + i0 + r) * pd.HD + h * D) * pd.isz, c);
    *reinterpret_cast<float4*>(&sm.q[r][c]) = x;
  }
  FmaTile<D> t;
  t.init();
  auto load = [&](int e0) {  // fp32 rows by asynchronous copies
    for (int i = tid; i < kFmaKeys * (D / 4); i += kFmaThreads) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4));
      const bool in = e0 + r < b;
      const uint8_t* ent = in ? shared_entry(P, shared_id(P, H, e0 + r)) : pd.arena;
      const uint8_t* kr = ent + h * D * pd.vs;
      if constexpr (CACHE == KVPOOL_F32) {
        cp_async16(smem_addr(&sm.k[r][c]), in ? kr + 4 * c : ent, in ? 16 : 0);
        cp_async16(smem_addr(&sm.v[r][c]), in ? kr + 4 * (pd.HD + c) : ent, in ? 16 : 0);
      } else {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (in) {
          x = codes4<CACHE>(kr, c);
          y = codes4<CACHE>(kr + pd.HD * pd.vs, c);
          if (CACHE == KVPOOL_FP8_E4M3 && c == 0) {
            const uint32_t s2 = *reinterpret_cast<const uint32_t*>(ent + 2 * pd.HD);
            scales[0][r] = qscale * __uint_as_float(s2 << 16);
            scales[1][r] = __uint_as_float(s2 & 0xFFFF0000u);
          }
        }
        *reinterpret_cast<float4*>(&sm.k[r][c]) = x;
        *reinterpret_cast<float4*>(&sm.v[r][c]) = y;
      }
    }
    cp_async_commit();
  };
  for (int e0 = a; e0 < b; e0 += kFmaKeys) {
    load(e0);
    cp_async_wait<0>();
    __syncthreads();
    const int n = b - e0;
    t.step(
        sm, ty, tx, [&](int, int j) { return j < n; },
        [&](int j) { return CACHE != KVPOOL_FP8_E4M3 ? qscale : j < n ? scales[0][j] : 0.0f; },
        [&](int j) { return CACHE != KVPOOL_FP8_E4M3 ? 1.0f : j < n ? scales[1][j] : 0.0f; });
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 4 * ty + r;
    if (row >= rows) continue;
    const int64_t slot = shared_slot(P, i0 + row, split);
    t.put(P.part_o + slot * pd.HD + h * D, r, tx);
    if (tx == 0) *reinterpret_cast<float2*>(P.part_ml + (slot * pd.heads + h) * 2) = make_float2(t.m[r], t.l[r]);
  }
}

// ---- bf16 queries and cache: tensor cores -----------------------------------------
// Eight warps share stages of 128 entries (K and V of the head, asynchronous
// copies through a ring of three): RG groups of 16 requests times 8 / RG groups
// of keys.  Fragments as in the single-token window attention: S^T = K Q^T, 16
// keys x 8 requests per product, lane (g, t) holding dims 8t .. 8t + 7 of a
// 32-dim piece; O^T = V^T P^T with V's pairs along the keys from byte permutes.
//
// The outputs are fp32 and the cache is bf16, so a bf16 weight would be the one
// rounding that shows (2^-9): each weight is taken apart into three bf16 numbers
// whose sum holds its 24 bits, and O^T takes three products.  Scores are exact
// products summed in fp32.  Each group of keys has products of its own that are
// then added to the outputs with rounding: 30 requests of 64 heads x 64 behind
// 16,384 entries are off by 2.9e-7 of the outputs' norm (in one running sum 6.9e-6,
// and the longer the run the more) for 2% of the time.
constexpr int kMmaWarps = 8, kMmaKeys = 128, kMmaStages = 3;

template <int D>
struct MmaShared {
  static constexpr int kTile = kMmaKeys * D * 2;  // K or V of a stage
  static constexpr int kSmem = kMmaStages * 2 * kTile;
  static_assert(kSmem >= kMmaWarps * 16 * D * 4, "the warps' outputs reuse the stages");
};

// 16-byte piece u of row r: swizzled so that both fragments' loads (two rows x
// four pieces, four rows two apart x two pieces) meet eight different banks
__device__ __forceinline__ int shared_piece(int r, int u) { return u ^ (r & 6) ^ ((r & 1) << 2); }

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

template <int D, int RG>
__global__ void __launch_bounds__(kMmaWarps * 32, 1) shared_mma_kernel(const __grid_constant__ AttendParams P,
                                                                       const __grid_constant__ SharedShape H) {
  pdl_start();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ float2 sml[kMmaWarps][16];
  constexpr int kTile = MmaShared<D>::kTile, C = D / 32, U = D / 8, KG = kMmaWarps / RG;
  constexpr int KB = KG <= 2 ? 2 : 1;  // blocks of 16 keys that a warp takes at once
  const PoolDesc& pd = P.pool;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rg = warp % RG, kg = warp / RG;
  const int h = blockIdx.x, split = blockIdx.y, i0 = blockIdx.z * kSharedRows;
  const int rows = min(kSharedRows, P.n - i0);
  const int a = (int)((int64_t)H.n_entries * split / H.n_split);
  const int b = (int)((int64_t)H.n_entries * (split + 1) / H.n_split);
  const float qscale = 1.4426950408889634f * rsqrtf((float)D);
  const uint32_t base = smem_addr(smem_raw);

  // query fragments: request 16 rg + 8n + g, dims 32c + 8t .. + 7
  uint4 q[2][C];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int r = 16 * rg + 8 * n + g;
      q[n][c] = make_uint4(0, 0, 0, 0);
      if (r < rows)
        q[n][c] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(P.q) +
                                                  2 * ((int64_t)(P.row0 + i0 + r) * pd.HD + h * D + 32 * c + 8 * t));
    }
  // four threads copy an entry: pieces tid % 4, + 4, ... of its K and V
  const int n_st = (b - a + kMmaKeys - 1) / kMmaKeys;
  const int ce = tid >> 2, cu = tid & 3;
  // their block ids are asked for a stage ahead; entries behind the end repeat
  // the last one (masked below)
  int32_t next[2];
  auto look_up = [&](int st) {
#pragma unroll
    for (int x = 0; x < 2; ++x) next[x] = shared_id(P, H, min(a + st * kMmaKeys + 64 * x + ce, b - 1));
  };
  look_up(0);
  auto copy = [&](int st) {
    if (st < n_st) {
      const int32_t id[2] = {next[0], next[1]};
      if (st + 1 < n_st) look_up(st + 1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint8_t* src = shared_entry(P, id[x]) + h * D * 2;
        const uint32_t dst = base + (st % kMmaStages) * 2 * kTile + (64 * x + ce) * D * 2;
#pragma unroll
        for (int u = 0; u < U; u += 4) {
          const uint32_t at = shared_piece(ce, u + cu) * 16;
          cp_async16(dst + at, src + (u + cu) * 16);
          cp_async16(dst + kTile + at, src + pd.HD * 2 + (u + cu) * 16);
        }
      }
    }
    cp_async_commit();
  };
  for (int st = 0; st < kMmaStages - 1; ++st) copy(st);

  float m[2][2], l[2][2], o[2][D / 16][4];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
  }
  for (int st = 0; st < n_st; ++st) {
    cp_async_wait<kMmaStages - 2>();
    __syncthreads();  // the stage has landed for all; the one copied next has been read by all
    copy(st + kMmaStages - 1);
    const uint32_t sk = base + (st % kMmaStages) * 2 * kTile, sv = sk + kTile;
    const int n_key = min(kMmaKeys, b - a - st * kMmaKeys);
    for (int k0 = 16 * KB * kg; k0 < n_key; k0 += 16 * KB * KG) {
      float s[KB][2][4] = {};
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          const uint4 ka = lds16(sk + (k0 + 16 * k + g) * D * 2 + shared_piece(g, 4 * c + t) * 16);
          const uint4 kb = lds16(sk + (k0 + 16 * k + 8 + g) * D * 2 + shared_piece(g, 4 * c + t) * 16);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            mma_bf16(s[k][n], ka.x, kb.x, ka.y, kb.y, q[n][c].x, q[n][c].y);
            mma_bf16(s[k][n], ka.z, kb.z, ka.w, kb.w, q[n][c].z, q[n][c].w);
          }
        }
      uint32_t pt[KB][2][3][2];  // [16 keys][requests][piece of the weights][keys 0 - 7, 8 - 15]
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float corr[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = -INFINITY;
#pragma unroll
          for (int k = 0; k < KB; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& x = s[k][n][2 * i + e];
              x = k0 + 16 * k + 8 * i + g < n_key ? x * qscale : -INFINITY;
              mx = fmaxf(mx, x);
            }
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          mx = fmaxf(mx, m[n][e]);  // finite: some key of the group counts
          corr[e] = ex2f(m[n][e] - mx);
          m[n][e] = mx;
          l[n][e] *= corr[e];
#pragma unroll
          for (int k = 0; k < KB; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& x = s[k][n][2 * i + e];
              x = ex2f(x - mx);
              l[n][e] += x;  // this lane's keys only
            }
        }
        if (__any_sync(0xffffffffu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][i][j] *= corr[j & 1];
        }
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
          for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t pk = pack_bf16(s[k][n][2 * i], s[k][n][2 * i + 1]);
              s[k][n][2 * i] -= __uint_as_float(pk << 16);
              s[k][n][2 * i + 1] -= __uint_as_float(pk & 0xFFFF0000u);
              pt[k][n][x][i] = transpose8x8(pk);
            }
      }
      // Products of these keys alone, then a rounded sum: the tensor core cuts
      // off what it adds to, every time, so one running sum would lose more the
      // longer the run (see kvpool_shared_tc.cu)
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh) {
        float add[4][2][4] = {};
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = k0 + 16 * k + 2 * t + (i & 1) + 8 * (i >> 1);
            v[i] = lds16(sv + r * D * 2 + shared_piece(r & 7, 8 * hh + g) * 16);
          }
          const uint32_t v0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, v1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
          const uint32_t v2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, v3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
          uint32_t f[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[j][0] = __byte_perm(v0[j], v1[j], 0x5410);
            f[j][1] = __byte_perm(v0[j], v1[j], 0x7632);
            f[j][2] = __byte_perm(v2[j], v3[j], 0x5410);
            f[j][3] = __byte_perm(v2[j], v3[j], 0x7632);
          }
          // eight independent sums in a row
#pragma unroll
          for (int x = 2; x >= 0; --x)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int n = 0; n < 2; ++n)
                mma_bf16(add[j][n], f[j][0], f[j][1], f[j][2], f[j][3], pt[k][n][x][0], pt[k][n][x][1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][4 * hh + j][i] += add[j][n][i];
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  // the key groups' states of a request into one
  float* so = reinterpret_cast<float*>(smem_raw);  // [warp][16][D]
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
      const int r = 8 * n + 2 * t + e;
      if (g == 0) sml[warp][r] = make_float2(m[n][e], l[n][e]);
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float2*>(so + (warp * 16 + r) * D + 64 * hh + 8 * g + 2 * j) =
              make_float2(o[n][4 * hh + j][e], o[n][4 * hh + j][2 + e]);
    }
  __syncthreads();
  for (int i = tid; i < min(rows, 16 * RG) * (D / 4); i += kMmaWarps * 32) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < KG; ++k) mx = fmaxf(mx, sml[k * RG + r / 16][r % 16].x);
    float ls = 0.0f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < KG; ++k) {
      const int wp = k * RG + r / 16;
      const float2 ml = sml[wp][r % 16];
      const float f = ex2f(ml.x - mx);
      const float4 y = *reinterpret_cast<const float4*>(so + (wp * 16 + r % 16) * D + c);
      ls = fmaf(ml.y, f, ls);
      x.x = fmaf(y.x, f, x.x);
      x.y = fmaf(y.y, f, x.y);
      x.z = fmaf(y.z, f, x.z);
      x.w = fmaf(y.w, f, x.w);
    }
    const int64_t slot = shared_slot(P, i0 + r, split);
    *reinterpret_cast<float4*>(P.part_o + slot * pd.HD + h * D + c) = x;
    if (c == 0) *reinterpret_cast<float2*>(P.part_ml + (slot * pd.heads + h) * 2) = make_float2(mx, ls);
  }
}

template <int D, int RG>
cudaError_t launch_mma_t(const AttendParams& p, const SharedShape& h, cudaStream_t s) {
  auto* kern = shared_mma_kernel<D, RG>;
  constexpr int smem = MmaShared<D>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(h.pdl != 0, kern, dim3(p.pool.heads, h.n_split, (p.n + kSharedRows - 1) / kSharedRows),
                       dim3(kMmaWarps * 32), smem, s, p, h);
}
// the fewest groups of 16 requests that hold a CTA's
template <int D>
cudaError_t launch_mma(const AttendParams& p, const SharedShape& h, cudaStream_t s) {
  return p.n <= 16 ? launch_mma_t<D, 1>(p, h, s) : p.n <= 32 ? launch_mma_t<D, 2>(p, h, s) : launch_mma_t<D, 4>(p, h, s);
}

template <int IN, int CACHE, int D>
cudaError_t launch_shared_t(const AttendParams& p, const SharedShape& h, cudaStream_t s) {
  auto* kern = shared_fma_kernel<IN, CACHE, D>;
  constexpr int smem = (int)sizeof(FmaSmem<D>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(h.pdl != 0, kern, dim3(p.pool.heads, h.n_split, (p.n + kFmaRows - 1) / kFmaRows),
                       dim3(kFmaThreads), smem, s, p, h);
}

template <int IN, int CACHE>
cudaError_t launch_shared_d(const AttendParams& p, const SharedShape& h, cudaStream_t s) {
  return p.pool.head_dim == 128 ? launch_shared_t<IN, CACHE, 128>(p, h, s) : launch_shared_t<IN, CACHE, 64>(p, h, s);
}

}  // namespace

// bf16 on the 5th-generation tensor cores or on the small products?  The
// former read an entry once for up to 128 requests and need a tile of 128
// entries to get going; measured as whole steps of 16 heads x 128 (small
// products / 5th generation, us):
//   entries     32 requests    64 requests    128 requests
//   1,024       17.9 / 23.3    26.2 / 30.3    39.9 / 48.5
//   2,048       22.1 / 25.5    31.7 / 31.5    50.0 / 48.1
//   4,096       26.7 / 28.1    39.4 / 35.1    67.6 / 51.0
//   8,192       36.7 / 35.9    55.7 / 43.7     102 / 59.9
bool shared_tc(int n, int n_entries) { return n > 32 && n_entries >= 2048; }

// Splits of the shared entries for n requests: CTAs (head, split, block of
// requests) that fill the GPU (the FMA form: with three to an SM; the
// 5th-generation form: each takes two), of at least 64 entries each.
int shared_splits(const PoolDesc& pd, int n, int n_entries, int n_sms) {
  const bool mma = pd.in_dtype == KVPOOL_BF16 && pd.cache_dtype == KVPOOL_BF16;
  const bool tc = mma && shared_tc(n, n_entries);
  const int rows = !mma ? kFmaRows : tc ? kSharedTcRows : kSharedRows;
  const int per = pd.heads * ((n + rows - 1) / rows);
  const int most = !mma ? 3 * n_sms / per : tc ? 2 * std::max(1, n_sms / per) : n_sms / per;
  return std::max(1, std::min(most, (n_entries + 63) / 64));
}

// Does it pay?  What the call saves is n requests' reading of the entries: a time
// per entry and request that depends on the entry's values (heads x head_dim) and
// type, half as much again where there is more to read than one wave of
// decode_attend's longest splits takes.  What it costs is another launch and
// partial results (start, and kShareRequest for each request), and the tiles that
// a multiprocessor works through one after another: 128 entries by up to 64
// requests (small products) or 128 (5th generation, in two runs), 64 entries by 32
// requests in the FMA form, which takes as long for 2 requests as for 32.
//
// Times in ns, fitted to steps of 4 and 16 heads x 64 and 8, 16 and 32 x 128, 2 to
// 128 requests, 128 to 8,192 entries, every type.  Some of them, shared / each its
// own in us, at 16 x 128:
//                   8 requests,  32 requests,  64 requests,  64 requests,
//                   2,048 entries  1,024         512          8,192
//   bf16            16.6 / 18.8  20.1 / 29.2   26.0 / 30.6   44.0 / 442
//   bf16 on fp8     59.6 / 17.4  28.4 / 26.3   31.7 / 26.7    276 / 328
//   fp32 on bf16    57.0 / 19.8  29.3 / 31.4   35.0 / 33.5    284 / 474
//   fp32            54.8 / 42.7  33.4 / 79.4   42.9 / 86.3    259 / 1,717
// Of all 2,520 steps the slower side is taken in 89, by more than 3% in 59; of 336
// of layers with CSA (fp8 and bf16), in 61 and 23.  With 64 MB of reading saved as
// the rule for every type, steps that shared an fp8 cache's entries took up to 8
// times as long as those that did not.
constexpr double kShareRequest = 25.0;
bool shared_pays(const PoolDesc& pd, int n, int n_entries, int n_sms) {
  if (n < 2 || n_entries < 1) return false;
  // an entry read by one request, at these values per entry
  constexpr double kValues[4] = {256, 1024, 2048, 4096};
  constexpr double kRead[3][4] = {{0.34, 1.04, 1.87, 4.05}, {0.25, 0.34, 0.56, 1.75}, {0.25, 0.29, 0.45, 1.2}};
  const double* t = kRead[pd.cache_dtype];
  int k = 0;
  while (k < 2 && pd.HD > kValues[k + 1]) ++k;
  const double per_entry = t[k] + (t[k + 1] - t[k]) * (pd.HD - kValues[k]) / (kValues[k + 1] - kValues[k]);
  const double entries = (double)n * n_entries;
  const double read = entries * per_entry * (entries > 3.0 * n_sms * attend_max_split_len() ? 1.5 : 1.0);

  struct Cost {
    double tile64, tile128, start;  // a tile of heads of 64 and of 128
  };
  const bool mma = pd.in_dtype == KVPOOL_BF16 && pd.cache_dtype == KVPOOL_BF16;
  const bool tc = mma && shared_tc(n, n_entries);
  const Cost c = tc                                  ? Cost{400, 650, 7000}
                 : mma                               ? Cost{400, 2500, 2800}
                 : pd.cache_dtype == KVPOOL_FP8_E4M3 ? Cost{3200, 8200, 5000}
                 : pd.cache_dtype == KVPOOL_BF16     ? Cost{2600, 7500, 4000}
                                                     : Cost{1950, 4800, 6500};
  const int rows = !mma ? kFmaRows : tc ? kSharedTcRows : kSharedRows, keys = mma ? kMmaKeys : kFmaKeys;
  const int runs = shared_splits(pd, n, n_entries, n_sms), per_cta = tc ? 2 : 1;
  const int64_t ctas = (int64_t)pd.heads * ((n + rows - 1) / rows) * ((runs + per_cta - 1) / per_cta);
  const int64_t run = (n_entries + runs - 1) / runs;
  const double tiles = (double)((run + keys - 1) / keys * per_cta) * (double)((ctas + n_sms - 1) / n_sms);
  return read > tiles * (pd.head_dim == 64 ? c.tile64 : c.tile128) + c.start + kShareRequest * n;
}

int launch_shared(const AttendParams& p, int n_entries, int n_split, bool pdl, void* stream, int* n_kernels) {
  const SharedShape h{n_entries, n_split, p.reqs[0].slot, pdl};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  *n_kernels += 1;
  switch (p.pool.in_dtype * 3 + p.pool.cache_dtype) {
    case KVPOOL_F32 * 3 + KVPOOL_F32: return (int)launch_shared_d<KVPOOL_F32, KVPOOL_F32>(p, h, s);
    case KVPOOL_F32 * 3 + KVPOOL_BF16: return (int)launch_shared_d<KVPOOL_F32, KVPOOL_BF16>(p, h, s);
    case KVPOOL_F32 * 3 + KVPOOL_FP8_E4M3: return (int)launch_shared_d<KVPOOL_F32, KVPOOL_FP8_E4M3>(p, h, s);
    case KVPOOL_BF16 * 3 + KVPOOL_F32: return (int)launch_shared_d<KVPOOL_BF16, KVPOOL_F32>(p, h, s);
    case KVPOOL_BF16 * 3 + KVPOOL_BF16:
      return (int)(shared_tc(p.n, n_entries) ? launch_shared_tc(p, h, s)
                   : p.pool.head_dim == 128 ? launch_mma<128>(p, h, s)
                                            : launch_mma<64>(p, h, s));
    case KVPOOL_BF16 * 3 + KVPOOL_FP8_E4M3: return (int)launch_shared_d<KVPOOL_BF16, KVPOOL_FP8_E4M3>(p, h, s);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace kvp
