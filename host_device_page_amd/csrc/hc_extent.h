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

// [a, a + an) and [b, b + bn) share a byte.
inline bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Bytes of a table of int64 entries from its first one: 0 when it has none.
inline int64_t table_bytes(int64_t rows, int64_t width, int64_t stride) {
  if (rows <= 0 || width <= 0) return 0;
  return extent(8 * ((__int128)(rows - 1) * stride + width));
}

// A tensor of `elem`-byte elements, strides (of the token and of the head) in elements.
struct Tensor {
  const void* at;
  int64_t stride[2];
  int64_t n, heads, dim;
  int32_t elem = 2;
  int64_t bytes() const { return elem == 2 ? tensor_bytes(stride, n, heads, dim) : table_bytes(n, dim, stride[0]); }
};
// A table as one: a row of entries per "token".
inline Tensor table_tensor(const void* at, int64_t rows, int64_t width, int64_t stride) {
  return {at, {stride, 0}, rows, 1, width, 8};
}

// Two tensors of the same element size, whose extents fit, share an element.  Views of one buffer lie
// between each other's tokens and heads, so where both step alike the heads are compared one by one; tensors
// of unlike head strides are compared token by token, of unlike token strides as a whole, and may be
// taken to share what they only enclose.
inline bool share(const Tensor& a, const Tensor& b) {
  if (!overlap(a.at, a.bytes(), b.at, b.bytes())) return false;
  if (a.n > 1 && b.n > 1 && a.stride[0] != b.stride[0]) return true;
  const int64_t token = a.elem * (a.n > 1 ? a.stride[0] : b.n > 1 ? b.stride[0] : 0);
  const bool alike = a.heads <= 1 || b.heads <= 1 || a.stride[1] == b.stride[1];
  const int64_t head = alike ? a.elem * (a.heads > 1 ? a.stride[1] : b.heads > 1 ? b.stride[1] : 0) : 0;
  // bytes compared: a head's, or all from a token's first head to its last
  const int64_t an = a.elem * (alike ? a.dim : (a.heads - 1) * a.stride[1] + a.dim);
  const int64_t bn = b.elem * (alike ? b.dim : (b.heads - 1) * b.stride[1] + b.dim);
  const int64_t off = (int64_t)((uintptr_t)b.at - (uintptr_t)a.at);
  for (int64_t h = alike ? -(a.heads - 1) : 0; h <= (alike ? b.heads - 1 : 0); h++) {
    // token i of a meets token j of b where (i - j) * token is in (low, high)
    const int64_t low = off + h * head - an, high = off + h * head + bn;
    int64_t k = 0;
    if (token > 0) {
      k = low >= 0 ? low / token + 1 : -((-low - 1) / token);  // the least with k * token > low
      if (k < 1 - b.n) k = 1 - b.n;
      if (k > a.n - 1) continue;
    }
    if (k * token > low && k * token < high) return true;
  }
  return false;
}

}  // namespace hc
