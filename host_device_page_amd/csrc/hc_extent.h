// How far the arguments of a forward-pass call reach in memory, from its sizes and strides alone.
// A count times a stride can pass 64 bits, so the products are taken in 128; what does not fit is
// kTooFar, which no allocation holds.
#pragma once

#include <stdint.h>

namespace hc {

constexpr int64_t kTooFar = -1;

inline int64_t extent(__int128 bytes) { return bytes > INT64_MAX ? kTooFar : (int64_t)bytes; }

// Bytes of an [n][heads][dim] tensor of 2-byte elements from its first one, strides (of the token
// and of the head, >= 0) in elements: 0 when it is empty.
inline int64_t tensor_bytes(const int64_t* stride, int64_t n, int64_t heads, int64_t dim) {
  if (n <= 0 || heads <= 0) return 0;
  return extent(2 * ((__int128)(n - 1) * stride[0] + (__int128)(heads - 1) * stride[1] + dim));
}

// No two heads of such a tensor share an element: tokens lie outside heads or heads outside tokens.
inline bool rows_apart(const int64_t* stride, int64_t n, int64_t heads, int64_t dim) {
  const int inner = heads > 1 && (n <= 1 || stride[1] <= stride[0]) ? 1 : 0;
  const int64_t count[2] = {n, heads};
  __int128 need = dim;
  for (int k : {inner, 1 - inner}) {
    if (count[k] <= 1) continue;
    if (stride[k] < need) return false;
    need += (__int128)stride[k] * (count[k] - 1);
  }
  return true;
}

// Bytes of a table of int64 entries from its first one: 0 when it has none.
inline int64_t table_bytes(int64_t rows, int64_t width, int64_t stride) {
  if (rows <= 0 || width <= 0) return 0;
  return extent(8 * ((__int128)(rows - 1) * stride + width));
}

}  // namespace hc
