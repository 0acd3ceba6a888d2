// Pages for the new tokens of a batch, and where each of them goes.
//
//   fresh(s) = ceil((len + added) / P) - ceil(len / P)         pages that row s needs
//   token j of row s: position p = len + j, page p / P: the row's own entry below ceil(len / P), else
//   free page first + sum of fresh before s + p / P - ceil(len / P)
//
// Two prefix sums over the rows and then every token by itself.  One launch: each workgroup takes a range
// of tokens and goes over all rows for the sums, 8 bytes each of two lists, instead of waiting for
// another to publish them; a token that begins a page enters it in the table, so no entry that a workgroup reads is
// written by another.  Latency bounds it, a batch's lists are a few hundred kilobytes at most: 64 sequences with a
// token each 3.5 us, 512 with 67000 tokens 7 us.  Thousands of rows cost what a workgroup takes to go over them, 3.5
// us a thousand, once for every half million tokens: calls of 3000 rows 14 us, 8192 32, 32768 118 and with two million
// tokens 914.  (Quotients in 32 bits where they fit gave nothing.)
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hc_forward.h"

namespace hc {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kTokens = 1024;  // of a workgroup

struct Grow {
  int64_t len, added, fresh;
  bool ok;
};
__device__ __forceinline__ Grow grow_of(const ExtendArgs& a, int64_t s) {
  Grow g = {0, 0, 0, true};
  if (s >= a.table.rows) return g;
  const int64_t most = a.table.width * a.P;
  g.len = a.table.lens[s];
  g.added = a.added[s];
  g.ok = g.len >= 0 && g.len <= most && g.added >= 0 && g.added <= a.room && g.added <= most - g.len;
  if (!g.ok) g.added = 0;
  if (g.ok) g.fresh = (g.len + g.added + a.P - 1) / a.P - (g.len + a.P - 1) / a.P;
  return g;
}

// Exclusive prefixes of x and y over the workgroup, and their sums.
__device__ __forceinline__ void prefix_both(int64_t* x, int64_t* y, int64_t* s, int64_t* x_sum, int64_t* y_sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int64_t xi = *x, yi = *y;
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t u = __shfl_up(xi, d), v = __shfl_up(yi, d);
    if (lane >= d) xi += u, yi += v;
  }
  if (lane == 63) s[2 * wave] = xi, s[2 * wave + 1] = yi;
  __syncthreads();
  int64_t xb = 0, yb = 0, xt = 0, yt = 0;
  for (int w = 0; w < waves; w++) {
    if (w < wave) xb += s[2 * w], yb += s[2 * w + 1];
    xt += s[2 * w], yt += s[2 * w + 1];
  }
  *x = xb + xi - *x;
  *y = yb + yi - *y;
  *x_sum = xt;
  *y_sum = yt;
}

__global__ __launch_bounds__(kMaxThreads) void k_extend_pages(ExtendArgs a) {
  __shared__ int64_t s_start[kMaxThreads], s_page[kMaxThreads], s_len[kMaxThreads], s_sum[2 * kMaxThreads / 64];
  const int64_t t0 = (int64_t)blockIdx.x * kTokens, t1 = t0 + kTokens < a.room ? t0 + kTokens : a.room;
  const int64_t free0 = a.first_free ? *a.first_free : 0;
  int64_t start = 0, page = 0;  // of the rows gone over
  for (int64_t s0 = 0; s0 < a.table.rows; s0 += blockDim.x) {
    const int64_t s = s0 + threadIdx.x;
    const Grow g = grow_of(a, s);
    int64_t x = g.added, y = g.fresh, x_sum, y_sum;
    prefix_both(&x, &y, s_sum, &x_sum, &y_sum);
    s_start[threadIdx.x] = start + x;
    s_page[threadIdx.x] = page + y;
    s_len[threadIdx.x] = g.len;
    __syncthreads();
    const int rows = a.table.rows - s0 < blockDim.x ? (int)(a.table.rows - s0) : (int)blockDim.x;
    if (blockIdx.x == 0 && s < a.table.rows) {
      a.q_start[s] = start + x;
      a.kv_len[s] = g.len + g.added;
      if (!g.ok || (g.added > 0 && start + x + g.added > a.room)) report_wrong<DeviceAtomic>(a.wrong, kWrongLengths, s);
    }
    // Pages that begin past the room: kv_len counts their tokens, so what stood in their entries would be taken for the
    // row's own page by the next call.  A workgroup takes every gridDim.x-th entry of a row.
    if (s < a.table.rows && g.added > 0 && start + x + g.added > a.room) {
      int64_t* row = const_cast<int64_t*>(a.table.entries) + s * a.table.stride;
      const int64_t held = (g.len + a.P - 1) / a.P, fits = a.room - (start + x);  // tokens that have room, or below 0
      const int64_t kept = fits > 0 ? (g.len + fits + a.P - 1) / a.P : held;
      for (int64_t e = kept + blockIdx.x; e < held + g.fresh; e += gridDim.x)
        if (row[e] >= 0 && row[e] < a.pages) row[e] = -1;
    }
    const int64_t lo = start > t0 ? start : t0, hi = start + x_sum < t1 ? start + x_sum : t1;
    for (int64_t t = lo + threadIdx.x; t < hi; t += blockDim.x) {
      int r = 0, n = rows;  // the last row that starts at or before t: those behind it that add nothing start later
      while (n > 1) {
        const int half = n >> 1;
        if (s_start[r + half] <= t) r += half;
        n -= half;
      }
      const int64_t len = s_len[r], p = len + t - s_start[r], e = p / a.P, held = (len + a.P - 1) / a.P;
      int64_t* at = const_cast<int64_t*>(a.table.entries) + (s0 + r) * a.table.stride + e;
      int64_t id;
      if (e < held) {
        id = *at;
      } else {
        const int64_t k = s_page[r] + e - held;
        id = free0 >= 0 && free0 <= a.n_free && k < a.n_free - free0 ? a.free_pages[free0 + k] : -1;
      }
      const bool ok = id >= 0 && id < a.pages;
      if (!ok) report_wrong<DeviceAtomic>(a.wrong, kWrongIndex, s0 + r);
      if (e >= held && (p % a.P == 0)) *at = ok ? id : -1;
      a.slots[t] = ok ? id * a.P + p % a.P : -1;
      a.positions[t] = p;
    }
    start += x_sum;
    page += y_sum;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.q_start[a.table.rows] = start;
    *a.used = page;
  }
  for (int64_t t = (start > t0 ? start : t0) + threadIdx.x; t < t1; t += blockDim.x) {
    a.slots[t] = -1;
    a.positions[t] = 0;
  }
}

}  // namespace

hipError_t launch_extend_pages(const ExtendArgs& a, hipStream_t stream) {
  const int64_t groups = a.room > 0 ? (a.room + kTokens - 1) / kTokens : 1;
  (void)hipGetLastError();
  k_extend_pages<<<dim3((unsigned)groups), a.table.rows <= 256 ? 256 : kMaxThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace hc
