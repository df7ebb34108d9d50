// kvpool_shared.h -- shared HCA entries of a decode batch: what the kernels of
// kvpool_shared.cu and kvpool_shared_tc.cu have in common.
#pragma once

#include "device_util.cuh"
#include "kvpool_internal.h"

namespace kvp {

struct SharedShape {
  int32_t n_entries, n_split, slot;  // slot: the request whose table holds the shared ids
  int32_t pdl;                       // programmatic dependent launch
};

// the block id of shared entry e as it stands in the table, and the entry's
// address (the id is looked at there: a load that is early enough costs nothing)
__device__ __forceinline__ int32_t shared_id(const AttendParams& P, const SharedShape& H, int e) {
  return reinterpret_cast<const int32_t*>(P.pool.arena + P.pool.table)[(int64_t)H.slot * P.pool.max_bpr + e];
}
__device__ __forceinline__ const uint8_t* shared_entry(const AttendParams& P, int32_t b) {
  if (b < 0 || b >= P.pool.max_blocks) {
    flag_error(P.pool, kErrBadBlock);
    b = 0;
  }
  return P.pool.arena + P.layer.hca_pool + (int64_t)b * P.layer.hca_stride;
}

// partial slot of a request of the launch
__device__ __forceinline__ int64_t shared_slot(const AttendParams& P, int i, int split) {
  const AttendReq& R = P.reqs[i];
  return R.part_base + R.n_split0 + R.n_split1 + split;
}

// bf16 queries and cache on the 5th-generation tensor cores; a cudaError_t
constexpr int kSharedTcRows = 128;  // requests of a CTA
cudaError_t launch_shared_tc(const AttendParams& p, const SharedShape& h, cudaStream_t s);

}  // namespace kvp
