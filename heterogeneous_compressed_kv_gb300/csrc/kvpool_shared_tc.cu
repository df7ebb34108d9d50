// kvpool_shared_tc.cu -- the shared HCA entries of a decode batch on the
// 5th-generation tensor cores (bf16 queries and cache).
//
// A CTA takes one head, a run of the shared entries and up to 128 requests:
// the requests' queries are the 128 rows of S = Q K^T and O += P V over tiles
// of 128 entries, in two runs with a partial result each.  Thirteen warps: four gather the entries (through the block
// table: a tensor copy would want them adjacent) into a ring of K and V tiles
// with asynchronous copies, one thread issues the products, and eight do the
// softmax, two threads per row.  The scores of the next tile are computed while
// the weights of this one are (two score tiles in tensor memory).
//
// The outputs are fp32 and the cache is bf16, so a bf16 weight would be the one
// rounding that shows (2^-9): each weight is taken apart into three bf16 numbers
// whose sum holds its 24 bits, and O += P V takes three products.  Two of the
// weights' pieces lie over the scores, the third beside them.
// Measured: 64 requests behind 8,192 entries of 16 heads x 128 24 us.  The first
// tile is there after 5.4 us (parameters, block ids, entries: three reads in a
// row), a tile's K and V take 1.9 us (4.9 TB/s over the CTAs; four tiles of 32 KB
// in flight), a run's outputs 1.7 us.  Without its softmax the step would take
// 4.5 us less, with one product of three 2.4 us, with its entries in the L2 cache
// 3 us.  Four rows to a gathering tensor copy in place of the threads' 16-byte
// ones: 68 us a step instead of 46.
// The tensor core cuts each sum's last bit off instead of rounding it, 24 times
// per tile, so that a running sum loses the more the longer it is: of the outputs'
// norm 1.4e-6 over 4 tiles of random entries and 2.9e-6 over 8 (each other fp32
// step together 0.3e-6; decode_attend 0.6e-6).  Hence two runs to a CTA, and a sum
// of 8 tiles at most, after which it is added to its run's partial in global
// memory (by the threads that wrote it).  Behind 16,384 entries (64 requests of 16
// heads x 128, runs of 8 tiles) sums of 4 took 69.5 us a step and sums of 8 58.6.
// Outputs are rescaled when a row's maximum grows by more than 2^8 (see
// kvpool_window_tc.cu).
#include <cuda_runtime.h>

#include "kvpool_fma.cuh"
#include "kvpool_shared.h"
#include "kvpool_tcgen05.cuh"

namespace kvp {
namespace {

constexpr int kKeys = 128;
constexpr int kSoftmaxWarps = 8, kCopyWarps = 4;
constexpr int kThreads = 32 * (kSoftmaxWarps + 1 + kCopyWarps);
constexpr int kLag = 3;  // tiles on their way behind the one being started
constexpr float kGrow = 8.0f;
constexpr int kRunTiles = 8;  // tiles that are summed in tensor memory

template <int D>
struct Shape {
  static constexpr int kTileBytes = 128 * D * 2;  // D / 64 runs of 128 rows x 128 bytes
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kBarOff = (1 + kStages) * kTileBytes;
  static constexpr int kSwapOff = kBarOff + 256;
  static constexpr int kSmem = kSwapOff + 3 * 256 * 4 + 1024;
  static_assert(kLag < kStages, "a tile is announced before the ring needs its stage");
};

// tiles go out as K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1): the order of their use
__device__ __forceinline__ bool tile_is_k(int i, int n, int& j) {
  if (i == 0 || n == 1) {
    j = 0;
    return i == 0;
  }
  if (i == 2 * n - 1) {
    j = n - 1;
    return false;
  }
  j = (i + 1) / 2 - (i % 2 == 0 ? 1 : 0);
  return i % 2 == 1;
}

// LONG: runs of more than kRunTiles tiles
template <int D, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) shared_tc_kernel(const __grid_constant__ AttendParams P,
                                                                const __grid_constant__ SharedShape H) {
  pdl_start();
  using Sh = Shape<D>;
  constexpr int NS = Sh::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t* ring = smem + Sh::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kBarOff);
  // scores, weights, outputs: two barriers in turn (with one, a phase could pass
  // while a slow waiter still looks for the one before, or a wait be taken for
  // the phase before the one before it)
  uint64_t *kv_full = bars, *kv_free = kv_full + NS, *s_full = kv_free + NS, *p_ready = s_full + 2, *pv_done = p_ready + 2,
           *swap = pv_done + 2, *drain = swap + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const PoolDesc& pd = P.pool;
  uint32_t* err = reinterpret_cast<uint32_t*>(pd.arena + pd.err);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x, split = 2 * blockIdx.y, i0 = blockIdx.z * kSharedTcRows;
  const int rows = min(kSharedTcRows, P.n - i0);
  // the two runs: entries [a, mid) in n0 tiles, [mid, b) in the others
  const int a = (int)((int64_t)H.n_entries * split / H.n_split);
  const int mid = (int)((int64_t)H.n_entries * (split + 1) / H.n_split);
  const int b = split + 2 > H.n_split ? mid : (int)((int64_t)H.n_entries * (split + 2) / H.n_split);
  const int n0 = (mid - a + kKeys - 1) / kKeys, n_tile = n0 + (b - mid + kKeys - 1) / kKeys;
  // first entry of tile j, and the end of its run
  auto tile_at = [&](int j) { return j < n0 ? a + j * kKeys : mid + (j - n0) * kKeys; };
  auto run_end = [&](int j) { return j < n0 ? mid : b; };
  // is tile j the first of its sum in tensor memory?
  auto fresh = [&](int j) { return LONG ? (j < n0 ? j : j - n0) % kRunTiles == 0 : j == 0 || j == n0; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], kCopyWarps);
      mbar_init(&kv_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], kSoftmaxWarps);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&swap[i], 2);
    mbar_fence_init();
  }
  __syncthreads();
  // columns: scores 0 - 127 and 128 - 255, outputs 256 - 383, third pieces 384 - 447 and 448 - 511
  uint32_t tmem = 0;
  // The copy warps start at once; the others stage the queries first (in one
  // go, the loads in flight together: started one by one, and with the copies
  // behind them, the first product waited 3 us longer)
  if (warp <= kSoftmaxWarps) {
    if (warp == kSoftmaxWarps) {
      tmem_alloc(tmem_slot, 512);
    } else {
      // row r, 16-byte piece u of each run of 64 dims at u ^ (r % 8)
      constexpr int kEach = 128 * (D / 8) / (32 * kSoftmaxWarps);
      uint4 x[kEach];
#pragma unroll
      for (int y = 0; y < kEach; ++y) {
        const int i = threadIdx.x + y * 32 * kSoftmaxWarps, r = i / (D / 8), u = i % (D / 8);
        x[y] = make_uint4(0, 0, 0, 0);
        if (r < rows)
          x[y] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(P.q) +
                                                 2 * ((int64_t)(P.row0 + i0 + r) * pd.HD + h * D + 8 * u));
      }
#pragma unroll
      for (int y = 0; y < kEach; ++y) {
        const int i = threadIdx.x + y * 32 * kSoftmaxWarps, r = i / (D / 8), u = i % (D / 8);
        *reinterpret_cast<uint4*>(smem + (u / 8) * 16384 + r * 128 + (((u % 8) ^ (r & 7)) << 4)) = x[y];
      }
      fence_proxy_async();
    }
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(32 * (kSoftmaxWarps + 1)) : "memory");
    tc_fence_after();
    tmem = *tmem_slot;
  }

  if (warp > kSoftmaxWarps) {
    // ---- copies: four threads per entry ----
    const int ct = threadIdx.x - 32 * (kSoftmaxWarps + 1), r0 = ct >> 2, u0 = ct & 3;
    // block ids of rows r0 + 32 i of a tile (entries behind the end: none)
    auto look_up = [&](int j, int32_t* id) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = tile_at(j) + r0 + 32 * i;
        id[i] = e < run_end(j) ? shared_id(P, H, e) : INT32_MIN;
      }
    };
    int32_t next[4];                  // ids of the K tile to come, asked for a tile ahead
    const uint8_t *now[4], *last[4];  // addresses of the newest K tile's rows, and of the one's before
    look_up(0, next);
#pragma unroll
    for (int i = 0; i < 4; ++i) now[i] = last[i] = nullptr;
    bool ok = true;
    const int n = 2 * n_tile;
    int told = 0;
    for (int i = 0; i < n && ok; ++i) {
      const int stage = i % NS;
      if (i >= NS) ok = warp_wait(&kv_free[stage], (i / NS - 1) & 1, err);
      if (!ok) break;
      int j;
      const bool is_k = tile_is_k(i, n_tile, j);
      if (is_k) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          last[x] = now[x];
          now[x] = next[x] == INT32_MIN ? nullptr : shared_entry(P, next[x]) + h * D * 2 + u0 * 16;
        }
        if (j + 1 < n_tile) look_up(j + 1, next);
      }
      // V of tile j: that of the K before the newest one, or of the last K
      const bool newest = is_k || j == n_tile - 1;
      const uint32_t dst = smem_addr(ring) + stage * Sh::kTileBytes;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = r0 + 32 * x;
        const uint8_t* src = newest ? now[x] : last[x];
        const uint32_t bytes = src ? 16u : 0u;  // none: zeros
        const uint8_t* from = src ? src + (is_k ? 0 : pd.HD * 2) : pd.arena;
#pragma unroll
        for (int u = 0; u < D / 8; u += 4)
          cp_async16(dst + ((u + u0) / 8) * 16384 + r * 128 + ((((u + u0) % 8) ^ (r & 7)) << 4), src ? from + u * 16 : from,
                     bytes);
      }
      cp_async_commit();
      if (i >= kLag) {
        cp_async_wait<kLag>();
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[told % NS]);
        ++told;
      }
    }
    cp_async_wait<0>();
    fence_proxy_async();
    __syncwarp();
    for (; ok && told < n; ++told)
      if (lane == 0) mbar_arrive(&kv_full[told % NS]);
    __syncwarp();
  } else if (warp == kSoftmaxWarps) {
    // ---- products (one thread) ----
    if (elect_one()) {
      constexpr uint32_t kIdQK = bf16_idesc(128, kKeys, false), kIdPV = bf16_idesc(128, D, true);
      const uint64_t qd = smem_desc(smem_addr(smem), 16), k_desc = smem_desc(smem_addr(ring), 16),
                     v_desc = smem_desc(smem_addr(ring), 16384);
      bool ok = true;
      int i = 0;  // tiles used
#pragma unroll 1
      for (int j = 0; j <= n_tile && ok; ++j) {  // scores of tile j, then outputs of tile j - 1
        if (j < n_tile) {
          const int stage = i % NS;
          ok = mbar_wait_word(&kv_full[stage], (i / NS) & 1, err);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = k_desc + stage * (Sh::kTileBytes >> 4);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t off = ((c / 4) * 16384 + (c % 4) * 32) >> 4;
            mma_ss(tmem + 128 * (j & 1), qd + off, kd + off, kIdQK, c > 0);
          }
          mma_commit(&s_full[j & 1]);
          mma_commit(&kv_free[stage]);
          ++i;
        }
        if (j > 0) {
          const int stage = i % NS, e = (j - 1) & 1;
          ok = mbar_wait_word(&kv_full[stage], (i / NS) & 1, err) && mbar_wait_word(&p_ready[e], ((j - 1) >> 1) & 1, err);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_desc + stage * (Sh::kTileBytes >> 4);
          // pieces: the smallest first
          const uint32_t piece[3] = {tmem + 384 + 64 * e, tmem + 128 * e + 64, tmem + 128 * e};
#pragma unroll
          for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int c = 0; c < kKeys / 16; ++c)
              mma_ts(tmem + 256, piece[x] + 8 * c, vd + c * (2048 >> 4), kIdPV, !fresh(j - 1) || x > 0 || c > 0);
          mma_commit(&pv_done[e]);
          mma_commit(&kv_free[stage]);
          ++i;
        }
      }
      // every product and its arrivals are done before the CTA ends
      mma_commit(drain);
      mbar_wait_word(drain, 0, err);
    }
    __syncwarp();
  } else {
    // ---- softmax: two threads per row, 64 columns each ----
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t base_lane = tmem + ((uint32_t)(warp & 3) << 21);
    const bool live = 32 * (warp & 3) < rows;  // some row of the warp is a request's
    const float scale = 1.4426950408889634f * rsqrtf((float)D);
    uint64_t* pair = &swap[warp & 3];
    float* told = reinterpret_cast<float*>(smem + Sh::kSwapOff) + 128 * half + row;
    const int other = half ? -128 : 128;
    int n_swap = 0;
    // the other thread's value of the row (buffers in turn)
    auto exchange = [&](float x, float& y) {
      float* p = told + (n_swap % 3) * 256;
      *p = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair);
      const bool done = warp_wait(pair, n_swap & 1, err);
      y = p[other];
      ++n_swap;
      return done;
    };
    float m = -INFINITY, l = 0.0f;    // of the sum in tensor memory
    float run_m = -INFINITY, run_l = 0.0f;  // of the run's sums before it
    bool ok = true;
    // (looked up before the first scores are there: an index of its own for each
    // lane makes 32 reads of the parameters, 2 us when they are cold)
    const int64_t slot0 = shared_slot(P, min(i0 + row, P.n - 1), split);
    // The sum in tensor memory, whose last tile is j, goes to its run's partial:
    // as it is where it is the run's first one, else added to what is there
    auto put = [&](int j, float m, float l) {
      const int run = j >= n0;
      const bool first = !LONG || j - (run ? n0 : 0) < kRunTiles;
      const int64_t slot = slot0 + run;
      float4* dst = reinterpret_cast<float4*>(P.part_o + slot * pd.HD + h * D + (D / 2) * half);
      float theirs;
      if (!warp_wait(&pv_done[j & 1], (j >> 1) & 1, err) || !exchange(l, theirs)) return false;
      tc_fence_after();
      l += theirs;
      float fo = 0.0f, fn = 1.0f;
      if (!first) {
        const float m2 = fmaxf(run_m, m);
        fo = ex2f(run_m - m2);
        fn = ex2f(m - m2);
        m = m2;
        l = fmaf(run_l, fo, l * fn);
      }
      run_m = m;
      run_l = l;
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 16) {
        uint32_t o[16];
        float4 old[4];
        if (!first && row < rows) {
#pragma unroll
          for (int y = 0; y < 4; ++y) old[y] = dst[c / 4 + y];
        }
        __syncwarp();
        tmem_ld16(base_lane + 256 + (D / 2) * half + c, o);
        tmem_wait_ld();
        if (row < rows) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float4 x = make_float4(__uint_as_float(o[4 * y]), __uint_as_float(o[4 * y + 1]),
                                   __uint_as_float(o[4 * y + 2]), __uint_as_float(o[4 * y + 3]));
            if (!first) {
              const float4 w = old[y];
              x.x = fmaf(w.x, fo, x.x * fn);
              x.y = fmaf(w.y, fo, x.y * fn);
              x.z = fmaf(w.z, fo, x.z * fn);
              x.w = fmaf(w.w, fo, x.w * fn);
            }
            dst[c / 4 + y] = x;
          }
        }
      }
      if (row < rows && half == 0)
        *reinterpret_cast<float2*>(P.part_ml + (slot * pd.heads + h) * 2) = make_float2(m, l);
      return true;
    };
#pragma unroll 1
    for (int j = 0; j < n_tile; ++j) {
      if (!warp_wait(&s_full[j & 1], (j >> 1) & 1, err)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (live) {
        const uint32_t ts = base_lane + 128 * (j & 1);
        uint32_t x[64];
        tmem_ld32(ts + 64 * half, x);
        tmem_ld32(ts + 64 * half + 32, x + 32);
        tmem_wait_ld();
        const int n_key = run_end(j) - tile_at(j) - 64 * half;  // columns of this half that count
        if (n_key < 64) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= n_key) x[c] = 0xFF800000u;  // -inf
        }
        float mx = -INFINITY, theirs;
#pragma unroll
        for (int c = 0; c < 64; c += 2) mx = max3(mx, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        // (also: both halves' scores are in registers before weights are written over them)
        if (!exchange(mx, theirs)) {
          ok = false;
          break;
        }
        const float mn = fmaxf(mx, theirs) * scale;  // finite: some key of the tile counts
        const float m0 = m, l0 = l;
        if (fresh(j)) {
          m = mn;
          l = 0.0f;
        } else if (__any_sync(0xffffffffu, mn > m + kGrow)) {
          if (!warp_wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float m2 = fmaxf(m, mn), f = ex2f(m - m2);
          m = m2;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 16) {
            uint32_t o[16];
            const uint32_t at = base_lane + 256 + (D / 2) * half + c;
            tmem_ld16(at, o);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            tmem_st16(at, o);
          }
        }
        float sum[2] = {0.0f, 0.0f};
        const uint32_t to[3] = {ts + 32 * half, ts + 64 + 32 * half, base_lane + 384 + 64 * (j & 1) + 32 * half};
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t pk[3][16];
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            float p0 = ex2f(fmaf(__uint_as_float(x[c + 2 * y]), scale, -m));
            float p1 = ex2f(fmaf(__uint_as_float(x[c + 2 * y + 1]), scale, -m));
            sum[0] += p0;
            sum[1] += p1;
#pragma unroll
            for (int z = 0; z < 3; ++z) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(p0, p1);
              pk[z][y] = *reinterpret_cast<const uint32_t*>(&v);
              p0 -= __uint_as_float(pk[z][y] << 16);
              p1 -= __uint_as_float(pk[z][y] & 0xFFFF0000u);
            }
          }
#pragma unroll
          for (int z = 0; z < 3; ++z) tmem_st16(to[z] + c / 2, pk[z]);
        }
        l += sum[0] + sum[1];
        tmem_wait_st();
        // a sum leaves before the next one's first product replaces it
        if (j > 0 && fresh(j) && !put(j - 1, m0, l0)) {
          ok = false;
          break;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[j & 1]);
    }
    if (ok && live) put(n_tile - 1, m, l);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftmaxWarps) tmem_free(tmem, 512);
}

template <int D, bool LONG>
cudaError_t launch_l(const AttendParams& p, const SharedShape& h, cudaStream_t s) {
  auto* kern = shared_tc_kernel<D, LONG>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(h.pdl != 0, kern, dim3(p.pool.heads, (h.n_split + 1) / 2, (p.n + kSharedTcRows - 1) / kSharedTcRows),
                       dim3(kThreads), Shape<D>::kSmem, s, p, h);
}

template <int D>
cudaError_t launch_t(const AttendParams& p, const SharedShape& h, cudaStream_t s) {
  return h.n_entries > (int64_t)h.n_split * kRunTiles * kKeys ? launch_l<D, true>(p, h, s) : launch_l<D, false>(p, h, s);
}

}  // namespace

cudaError_t launch_shared_tc(const AttendParams& p, const SharedShape& h, cudaStream_t s) {
  return p.pool.head_dim == 128 ? launch_t<128>(p, h, s) : launch_t<64>(p, h, s);
}

}  // namespace kvp
