// kvpool_fma.cuh -- attention of a tile of 32 query rows over steps of 64 keys
// in fp32 FMAs: the step that the fp32 forms of the attention kernels share.
//
// Bound by shared-memory loads beside the FMAs: a thread's 4 rows x 4 keys take
// 8 16-byte loads per 64 FMAs.  Tiles are small (128 threads) so that several
// CTAs share an SM: while one waits for its keys the others compute, which
// takes less shared memory than a second buffer, and few rows still make many
// tiles.
//
// Measured: 3 prompts of 1,021 fp32 tokens x 4 heads of 64 under a window of 256
// 41 us (issue slots 47% busy at 14 warps to an SM).  Not kept, no faster there:
// fp32 pairs in one instruction (40.8), the next step's keys and values on
// their way during a step (42.4), five CTAs to an SM with the weights in the
// keys' place (42.9).
#pragma once

#include "device_util.cuh"

namespace kvp {

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr int kFmaRows = 32, kFmaKeys = 64, kFmaThreads = 128;

template <int D>
struct FmaSmem {
  float q[kFmaRows][D + 4];
  float k[kFmaKeys][D + 4];
  float v[kFmaKeys][D];
  float p[kFmaRows][kFmaKeys + 4];
};

// The state of thread (ty, tx) = (tid / 16, tid % 16): rows 4 ty .. 4 ty + 3,
// keys tx, tx + 16, tx + 32 and tx + 48 of a step's scores, dims 4 tx .. 4 tx + 3 (and 64 more)
// of the outputs.  The running maximum (log2 domain) and sum are the same in
// the 16 threads of a row.
template <int D>
struct FmaTile {
  float m[4], l[4], o[4][D / 16];

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[r][c] = 0.0f;
    }
  }

  // scores of the staged keys times ks(key), masked by see(row of the thread,
  // key of the step); weights times vs(key) for the values
  template <class See, class KScale, class VScale>
  __device__ __forceinline__ void step(FmaSmem<D>& sm, int ty, int tx, See see, KScale ks, VScale vs) {
    float s[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[r][j] = 0.0f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = *reinterpret_cast<const float4*>(&sm.q[4 * ty + r][c]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 k = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][c]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s[r][j] = fmaf(x[r].x, k.x, fmaf(x[r].y, k.y, fmaf(x[r].z, k.z, fmaf(x[r].w, k.w, s[r][j]))));
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[r][j] = see(r, tx + 16 * j) ? s[r][j] * ks(tx + 16 * j) : -INFINITY;
        mx = fmaxf(mx, s[r][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      mx = fmaxf(mx, m[r]);
      const float base = mx == -INFINITY ? 0.0f : mx;
      const float corr = ex2f(m[r] - base);
      float ps = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = ex2f(s[r][j] - base);
        ps += p;
        sm.p[4 * ty + r][tx + 16 * j] = p * vs(tx + 16 * j);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
      l[r] = l[r] * corr + ps;
      m[r] = mx;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[r][c] *= corr;
    }
    __syncwarp();  // a row's weights are written and read by the same half-warp
#pragma unroll 2
    for (int j = 0; j < kFmaKeys; j += 4) {
      float p[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.p[4 * ty + r][j]);
        p[r][0] = x.x, p[r][1] = x.y, p[r][2] = x.z, p[r][3] = x.w;
      }
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const float4 y = *reinterpret_cast<const float4*>(&sm.v[j + jj][64 * c + 4 * tx]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            o[r][4 * c] = fmaf(p[r][jj], y.x, o[r][4 * c]);
            o[r][4 * c + 1] = fmaf(p[r][jj], y.y, o[r][4 * c + 1]);
            o[r][4 * c + 2] = fmaf(p[r][jj], y.z, o[r][4 * c + 2]);
            o[r][4 * c + 3] = fmaf(p[r][jj], y.w, o[r][4 * c + 3]);
          }
        }
    }
  }

  __device__ __forceinline__ void put(float* row_o, int r, int tx) const {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      *reinterpret_cast<float4*>(row_o + 64 * c + 4 * tx) =
          make_float4(o[r][4 * c], o[r][4 * c + 1], o[r][4 * c + 2], o[r][4 * c + 3]);
  }
};

}  // namespace kvp
