// kvpool_shared.cu -- the HCA entries that a whole decode batch shares, read
// once for all its requests ("Ch 12 Inference framework: heterogeneous KV
// scheduling" s2.2: many requests reference the same blocks).
//
// decode_attend at one query per head streams every request's entries past one
// vector each.  Behind a shared prefix the same entries meet the queries of n
// requests: per head a dense product, scores [n x entries] and outputs [n x
// dim].  A CTA takes one head, a run of the shared entries and up to 64
// requests, and leaves a partial (max, sum, output) per request and head in
// the slots behind the request's other splits; the ordinary merge joins them.
#include <algorithm>

#include <cuda_runtime.h>

#include "device_util.cuh"
#include "kvpool_fma.cuh"
#include "kvpool_internal.h"

namespace kvp {
namespace {

constexpr int kSharedRows = 64;  // requests of a CTA

struct SharedShape {
  int32_t n_entries, n_split, slot;  // slot: the request whose table holds the shared ids
};

__device__ __forceinline__ const uint8_t* shared_entry(const AttendParams& P, const SharedShape& H, int e) {
  const PoolDesc& pd = P.pool;
  int32_t b = reinterpret_cast<const int32_t*>(pd.arena + pd.table)[(int64_t)H.slot * pd.max_bpr + e];
  if (b < 0 || b >= pd.max_blocks) {
    flag_error(pd, kErrBadBlock);
    b = 0;
  }
  return pd.arena + P.layer.hca_pool + (int64_t)b * P.layer.hca_stride;
}

__device__ __forceinline__ int64_t shared_slot(const AttendParams& P, int i, int split) {
  const AttendReq& R = P.reqs[i];
  return R.part_base + R.n_split0 + R.n_split1 + split;
}

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
  extern __shared__ __align__(16) uint8_t smem_raw[];
  FmaSmem<D>& sm = *reinterpret_cast<FmaSmem<D>*>(smem_raw);
  __shared__ float scales[2][kFmaKeys];
  const PoolDesc& pd = P.pool;
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int h = blockIdx.x, split = blockIdx.y, i0 = blockIdx.z * kSharedRows;
  const int rows = min(kSharedRows, P.n - i0);
  const int a = (int)((int64_t)H.n_entries * split / H.n_split);
  const int b = (int)((int64_t)H.n_entries * (split + 1) / H.n_split);
  const float qscale = 1.4426950408889634f * rsqrtf((float)D);
  for (int i = tid; i < kSharedRows * (D / 4); i += kFmaThreads) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
      x = codes4<IN>(static_cast<const uint8_t*>(P.q) + ((int64_t)(P.row0 + i0 + r) * pd.HD + h * D) * pd.isz, c);
    *reinterpret_cast<float4*>(&sm.q[r][c]) = x;
  }
  FmaTile<D> t;
  t.init();
  for (int e0 = a; e0 < b; e0 += kFmaKeys) {
    __syncthreads();
    for (int i = tid; i < kFmaKeys * (D / 4); i += kFmaThreads) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4));
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (e0 + r < b) {
        const uint8_t* ent = shared_entry(P, H, e0 + r);
        x = codes4<CACHE>(ent + h * D * pd.vs, c);
        y = codes4<CACHE>(ent + (pd.HD + h * D) * pd.vs, c);
        if (CACHE == KVPOOL_FP8_E4M3 && c == 0) {
          const uint32_t s2 = *reinterpret_cast<const uint32_t*>(ent + 2 * pd.HD);
          scales[0][r] = qscale * __uint_as_float(s2 << 16);
          scales[1][r] = __uint_as_float(s2 & 0xFFFF0000u);
        }
      }
      *reinterpret_cast<float4*>(&sm.k[r][c]) = x;
      *reinterpret_cast<float4*>(&sm.v[r][c]) = y;
    }
    __syncthreads();
    const int n = b - e0;
    t.step(
        sm, ty, tx, [&](int, int j) { return j < n; },
        [&](int j) { return CACHE != KVPOOL_FP8_E4M3 ? qscale : j < n ? scales[0][j] : 0.0f; },
        [&](int j) { return CACHE != KVPOOL_FP8_E4M3 ? 1.0f : j < n ? scales[1][j] : 0.0f; });
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

template <int IN, int CACHE, int D>
cudaError_t launch_shared_t(const AttendParams& p, const SharedShape& h, cudaStream_t s) {
  auto* kern = shared_fma_kernel<IN, CACHE, D>;
  constexpr int smem = (int)sizeof(FmaSmem<D>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(true, kern, dim3(p.pool.heads, h.n_split, (p.n + kSharedRows - 1) / kSharedRows),
                       dim3(kFmaThreads), smem, s, p, h);
}

template <int IN, int CACHE>
cudaError_t launch_shared_d(const AttendParams& p, const SharedShape& h, cudaStream_t s) {
  return p.pool.head_dim == 128 ? launch_shared_t<IN, CACHE, 128>(p, h, s) : launch_shared_t<IN, CACHE, 64>(p, h, s);
}

}  // namespace

// Splits of the shared entries for n requests: CTAs (head, split, 64
// requests) that fill the GPU twice over, of at least 64 entries each.
int shared_splits(const PoolDesc& pd, int n, int n_entries, int n_sms) {
  const int per = pd.heads * ((n + kSharedRows - 1) / kSharedRows);
  return std::max(1, std::min((2 * n_sms + per - 1) / per, (n_entries + 63) / 64));
}

int launch_shared(const AttendParams& p, int n_entries, int n_split, void* stream, int* n_kernels) {
  const SharedShape h{n_entries, n_split, p.reqs[0].slot};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  *n_kernels += 1;
  switch (p.pool.in_dtype * 3 + p.pool.cache_dtype) {
    case KVPOOL_F32 * 3 + KVPOOL_F32: return (int)launch_shared_d<KVPOOL_F32, KVPOOL_F32>(p, h, s);
    case KVPOOL_F32 * 3 + KVPOOL_BF16: return (int)launch_shared_d<KVPOOL_F32, KVPOOL_BF16>(p, h, s);
    case KVPOOL_F32 * 3 + KVPOOL_FP8_E4M3: return (int)launch_shared_d<KVPOOL_F32, KVPOOL_FP8_E4M3>(p, h, s);
    case KVPOOL_BF16 * 3 + KVPOOL_F32: return (int)launch_shared_d<KVPOOL_BF16, KVPOOL_F32>(p, h, s);
    case KVPOOL_BF16 * 3 + KVPOOL_BF16: return (int)launch_shared_d<KVPOOL_BF16, KVPOOL_BF16>(p, h, s);
    case KVPOOL_BF16 * 3 + KVPOOL_FP8_E4M3: return (int)launch_shared_d<KVPOOL_BF16, KVPOOL_FP8_E4M3>(p, h, s);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace kvp
