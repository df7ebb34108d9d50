// kvpool_rows.h -- host checks of the callers' rows (kvpool_heads).
#pragma once

#include <stdint.h>

#include "kvpool.h"

namespace kvp {

// data and strides in whole pieces of 16 bytes, strides not negative
inline bool rows_aligned(const kvpool_heads& h, int32_t dtype) {
  const int64_t unit = dtype == KVPOOL_BF16 ? 8 : 4;  // values in 16 bytes
  return reinterpret_cast<uintptr_t>(h.data) % 16 == 0 && h.token_stride % unit == 0 && h.head_stride % unit == 0 &&
         h.token_stride >= 0 && h.head_stride >= 0;
}

// No value of an output has two places in it: the axis of the larger stride
// steps over the whole of the other one (axes of length 1 take any stride).
inline bool rows_apart(const kvpool_heads& h, int64_t tokens, int32_t dim) {
  const int64_t ts = h.token_stride, hs = h.head_stride;
  if (tokens <= 1 || h.heads <= 1) return (tokens <= 1 || ts >= dim) && (h.heads <= 1 || hs >= dim);
  const int64_t lo = ts < hs ? ts : hs, hi = ts < hs ? hs : ts, n = ts < hs ? tokens : h.heads;  // n: the inner axis
  return lo >= dim && (hi - dim) / (n - 1) >= lo;  // hi >= lo * (n - 1) + dim
}

}  // namespace kvp
