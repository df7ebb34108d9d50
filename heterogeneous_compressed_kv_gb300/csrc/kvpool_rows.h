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

// The same places in the same order?
inline bool rows_same(const kvpool_heads& a, const kvpool_heads& b, int64_t tokens) {
  return a.data == b.data && a.heads == b.heads && (tokens <= 1 || a.token_stride == b.token_stride) &&
         (a.heads <= 1 || a.head_stride == b.head_stride);
}

// Do na tokens of a and nb of b share a value (of vb bytes)?  Tensors in one
// piece of memory share their strides, as the parts of a fused projection do:
// head h of token t of a and head g of token u of b then meet where (t - u)
// token strides and (h - g) head strides are less than dim from the distance of
// the two tensors.  With strides that differ they are taken to meet.
inline bool rows_meet(const kvpool_heads& a, int64_t na, const kvpool_heads& b, int64_t nb, int32_t dim, int64_t vb) {
  if (na <= 0 || nb <= 0 || a.heads <= 0 || b.heads <= 0) return false;
  using Wide = __int128;
  constexpr int64_t kMost = (int64_t)1 << 60;  // more bytes than any memory: strides that no tensor has
  auto bytes = [&](const kvpool_heads& h, int64_t n) {
    const Wide x = (Wide)vb * ((Wide)(n - 1) * h.token_stride + (Wide)(h.heads - 1) * h.head_stride + dim);
    return x < kMost ? (int64_t)x : kMost;
  };
  const int64_t an = bytes(a, na), bn = bytes(b, nb);
  if (an == kMost || bn == kMost) return true;
  const int64_t d0 = (int64_t)(reinterpret_cast<uintptr_t>(b.data) - reinterpret_cast<uintptr_t>(a.data));
  if (d0 >= an || -d0 >= bn) return false;
  if ((na > 1 && nb > 1 && a.token_stride != b.token_stride) || (a.heads > 1 && b.heads > 1 && a.head_stride != b.head_stride))
    return true;
  const int64_t ts = vb * (na > 1 ? a.token_stride : nb > 1 ? b.token_stride : 0);
  const int64_t hs = vb * (a.heads > 1 ? a.head_stride : b.heads > 1 ? b.head_stride : 0);
  const int64_t row = vb * dim;
  for (int64_t j = 1 - (int64_t)b.heads; j < a.heads; ++j) {  // heads between the two
    const int64_t r = d0 - j * hs;                            // i token strides are nearest to r
    const int64_t at = ts > 0 ? r / ts : 0;
    for (int up = 0; up < 2; ++up) {
      int64_t i = at + (r < 0 ? -up : up);
      i = i > na - 1 ? na - 1 : i < 1 - nb ? 1 - nb : i;
      const int64_t d = r - i * ts;
      if (d < row && -d < row) return true;
    }
  }
  return false;
}

// Does the memory from the first value of n tokens' rows to the last one share a
// byte with [p, p + bytes)?
inline bool rows_touch(const kvpool_heads& h, int64_t n, int32_t dim, int64_t vb, const void* p, __int128 bytes) {
  if (n <= 0 || h.heads <= 0 || bytes <= 0 || !p) return false;
  const __int128 a = reinterpret_cast<uintptr_t>(h.data), b = reinterpret_cast<uintptr_t>(p);
  const __int128 an = (__int128)vb * ((__int128)(n - 1) * h.token_stride + (__int128)(h.heads - 1) * h.head_stride + dim);
  return a < b + bytes && b < a + an;
}

// Are n1 x n2 runs of `len` values, s1 and s2 values apart, in places of their own?
inline bool runs_apart(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t len) {
  if (len <= 0 || n1 <= 0 || n2 <= 0) return true;
  if (n1 == 1 || n2 == 1) return (n1 == 1 || s1 >= len) && (n2 == 1 || s2 >= len);
  const int64_t lo = s1 < s2 ? s1 : s2, hi = s1 < s2 ? s2 : s1, n = s1 < s2 ? n1 : n2;
  return lo >= len && (hi - len) / (n - 1) >= lo;
}

// Does one of n1 x n2 runs of `len` 4-byte values, s1 and s2 values apart, share a
// byte with [p, p + bytes)?
inline bool runs_touch(const void* runs, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t len, const void* p, __int128 bytes) {
  if (!runs || !p || n1 <= 0 || n2 <= 0 || len <= 0 || bytes <= 0) return false;
  const __int128 a = reinterpret_cast<uintptr_t>(runs), b = reinterpret_cast<uintptr_t>(p);
  if (a >= b + bytes || b >= a + 4 * ((__int128)(n1 - 1) * s1 + (__int128)(n2 - 1) * s2 + len)) return false;
  for (int64_t i = 0; i < n1; ++i)  // (hardly ever: it lies among them)
    for (int64_t j = 0; j < n2; ++j) {
      const __int128 x = a + 4 * ((__int128)i * s1 + (__int128)j * s2);
      if (x < b + bytes && b < x + 4 * (__int128)len) return true;
    }
  return false;
}

}  // namespace kvp
