// Page tables over the device pool: copying pages, branching sequences, finding free pages
// and packing the live ones.
//
// A page is live when a table row names it within its length, so nothing but the tables has
// to be kept: marks over the pool's pages come from one pass over the entries, and a scan of
// the marks gives the free list, or for packing the pairs (k-th live page at or above the
// live count L, k-th dead page below L).  Sources lie at or above L and targets below it, so
// the pairs can be copied in any order and at once.
//
// The data of a page is contiguous in every layer and sub-buffer (P rows, or one block), so a
// pair is copied in pieces of 32 KiB, each one batch of eight 16-byte loads per lane before
// its stores; memory bounds it (64 children of 8 prompts over 32 layers, 621 MB, 116 us = 5.3 TB/s; 176 of 227
// live pages of 8 layers moved in 149 us).  Tables of a few thousand entries cost launches, not bandwidth,
// so marks are cleared, set and scanned by one small launch (three for large tables) and the
// entries rewritten by the launch that copies.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hc_forward.h"

namespace hc {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;
constexpr int64_t kPiece = (int64_t)kThreads * 16 * kUnroll;
constexpr int kScanThreads = 1024;

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) const v4u* gload_t;
typedef __attribute__((address_space(1))) v4u* gstore_t;

__device__ __forceinline__ void flag(WrongWord* wrong, Wrong kind, int64_t pos) {
  report_wrong<DeviceAtomic>(wrong, kind, pos);
}

// Entries of row s that count: ceil(len / P), 0 for a length out of bounds.
__device__ __forceinline__ int64_t row_entries(const PageTable& t, int64_t s, int32_t P, bool* bad) {
  const int64_t len = t.lens[s];
  *bad = len < 0 || len > t.width * P;
  return *bad ? 0 : (len + P - 1) / P;
}

// Bytes of one page of sub-buffer b in one layer, and of its first `rows` rows.
__device__ __forceinline__ int64_t page_bytes(const Geom& g, int b, int64_t rows) {
  return g.sub[b].gran == HC_PAGE_BLOCKS ? g.sub[b].elem : rows * g.sub[b].elem;
}

// One piece of a page pair: bytes [off, min(off + kPiece, bytes)) of (sub b, layer l).
__device__ __forceinline__ void copy_piece(const Geom& g, int b, int64_t l, int64_t from, int64_t to, int64_t off,
                                           int64_t bytes) {
  const int64_t page = page_bytes(g, b, g.P);
  const uint64_t base = g.sub[b].layers[l];
  const gload_t src = reinterpret_cast<gload_t>(base + (uint64_t)(from * page + off));
  const gstore_t dst = reinterpret_cast<gstore_t>(base + (uint64_t)(to * page + off));
  const int vecs = (int)((bytes - off < kPiece ? bytes - off : kPiece) / 16);
  // every lane loads, past the end the last vector: loads under a condition do not leave together
  v4u v[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; k++) {
    const int i = k * kThreads + threadIdx.x;
    v[k] = src[i < vecs ? i : vecs - 1];
  }
#pragma unroll
  for (int k = 0; k < kUnroll; k++) {
    const int i = k * kThreads + threadIdx.x;
    if (i < vecs) dst[i] = v[k];
  }
}

// Pieces of a page in one layer, over the sub-buffers, and the sub-buffer of piece i of them.
struct Pieces {
  int32_t end[HC_MAX_SUBBUFS];
};
__host__ __device__ inline int64_t pieces_of(int64_t bytes) { return (bytes + kPiece - 1) / kPiece; }

Pieces layer_pieces(const Geom& g) {
  Pieces p;
  int64_t n = 0;
  for (int b = 0; b < HC_MAX_SUBBUFS; b++) {
    if (b < g.nsub) n += pieces_of(g.sub[b].gran == HC_PAGE_BLOCKS ? g.sub[b].elem : g.P * g.sub[b].elem);
    p.end[b] = (int32_t)n;
  }
  return p;
}

// Copies unit u of a list of n pairs: layer-major, then pair, then piece, so that what is in flight is
// many pages of one layer and not one page of many layers, whose addresses differ by a layer's
// power of two.  `pair` gives pair i's pages and the rows of it that move (0: nothing).
template <class Pair>
__device__ __forceinline__ void copy_unit(const Geom& g, const Pieces& pc, int64_t n, int64_t u, const Pair& pair) {
  const int32_t per_layer = pc.end[g.nsub - 1];
  const int64_t row = u / per_layer;
  const int32_t piece = (int32_t)(u - row * per_layer);
  const int64_t l = row / n, i = row - l * n;
  int b = 0;
  while (piece >= pc.end[b]) b++;
  int64_t from, to, rows;
  pair(i, &from, &to, &rows, piece == 0 && l == 0);
  if (rows <= 0) return;
  const int64_t off = (int64_t)(piece - (b ? pc.end[b - 1] : 0)) * kPiece;
  const int64_t bytes = page_bytes(g, b, rows);
  if (off < bytes) copy_piece(g, b, l, from, to, off, bytes);
}

__global__ __launch_bounds__(kThreads) void k_copy_pages(Geom g, Pieces pc, const int64_t* __restrict__ src,
                                                         const int64_t* __restrict__ dst, int64_t n,
                                                         WrongWord* __restrict__ wrong) {
  const int64_t pages = g.S / g.P;
  const int64_t units = n * g.L * pc.end[g.nsub - 1];
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x)
    copy_unit(g, pc, n, u, [&](int64_t i, int64_t* from, int64_t* to, int64_t* rows, bool first) {
      *from = src[i];
      *to = dst[i];
      const bool ok = *from >= 0 && *from < pages && *to >= 0 && *to < pages;
      if (!ok && first && threadIdx.x == 0) flag(wrong, kWrongIndex, i);
      *rows = ok && *from != *to ? g.P : 0;
    });
}

// Exclusive prefix of `x` over the workgroup and its sum; s: one entry per wave.
__device__ __forceinline__ int64_t block_prefix(int64_t x, int64_t* s, int64_t* sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int64_t incl = x;
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 63) s[wave] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < waves; w++) {
    if (w < wave) before += s[w];
    total += s[w];
  }
  __syncthreads();
  *sum = total;
  return before + incl - x;
}

// Numbers the children that need a page of their own and writes that entry of their rows.
__global__ __launch_bounds__(kScanThreads) void k_fork_plan(int32_t P, int64_t pages, ForkArgs a,
                                                            WrongWord* __restrict__ wrong) {
  __shared__ int64_t s_wave[kScanThreads / 64];
  int64_t taken = 0;
  for (int64_t i0 = 0; i0 < a.n; i0 += blockDim.x) {
    const int64_t i = i0 + threadIdx.x;
    int64_t len = 0;
    if (i < a.n) {
      const int64_t r = a.parents[i];
      if (r >= 0 && r < a.table.rows) {
        bool bad;
        row_entries(a.table, r, P, &bad);
        len = bad ? 0 : a.table.lens[r];
        if (bad) flag(wrong, kWrongLengths, i);
      } else {
        flag(wrong, kWrongIndex, i);
      }
    }
    int64_t sum;
    const int64_t rank = taken + block_prefix(len % P != 0 ? 1 : 0, s_wave, &sum);
    taken += sum;
    if (len % P != 0) {
      int64_t page = rank < a.n_free ? a.free_pages[rank] : -1;
      if (page < 0 || page >= pages) {
        flag(wrong, kWrongIndex, i);
        page = -1;
      }
      a.out[i * a.out_stride + len / P] = page;
    }
  }
  if (threadIdx.x == 0) *a.used = taken;
}

// The other entries of the children's rows, and the filled rows of the shared last pages.
__global__ __launch_bounds__(kThreads) void k_fork(Geom g, Pieces pc, ForkArgs a, int64_t units,
                                                   WrongWord* __restrict__ wrong) {
  const int64_t pages = g.S / g.P;
  auto length = [&](int64_t r) -> int64_t {
    bool bad;
    if (r < 0 || r >= a.table.rows) return 0;
    row_entries(a.table, r, g.P, &bad);
    return bad ? 0 : a.table.lens[r];
  };
  const int64_t entries = a.n * a.table.width;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < entries; e += (int64_t)gridDim.x * kThreads) {
    const int64_t i = e / a.table.width, j = e - i * a.table.width;
    const int64_t r = a.parents[i];
    const int64_t len = length(r);
    if (j == len / g.P && len % g.P != 0) continue;  // its own page, numbered already
    int64_t page = -1;
    if (j < len / g.P) {
      page = a.table.entries[r * a.table.stride + j];
      if (page < 0 || page >= pages) {
        flag(wrong, kWrongIndex, i);
        page = -1;
      }
    }
    a.out[i * a.out_stride + j] = page;
  }
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x)
    copy_unit(g, pc, a.n, u, [&](int64_t i, int64_t* from, int64_t* to, int64_t* rows, bool first) {
      const int64_t r = a.parents[i];
      const int64_t len = length(r);
      *rows = len % g.P;
      if (!*rows) return;
      *from = a.table.entries[r * a.table.stride + len / g.P];
      *to = a.out[i * a.out_stride + len / g.P];
      if (*from < 0 || *from >= pages) {
        if (first && threadIdx.x == 0) flag(wrong, kWrongIndex, i);
        *rows = 0;
      } else if (*to < 0 || *to == *from) {
        *rows = 0;
      }
    });
}

// Workspace of the liveness calls: [0] the live count, [1] the number of pairs, then an int32
// per page three times: mark (then the page's new number), pair sources, pair targets.
struct Work {
  int64_t* head;
  int32_t *mark, *from, *to;
};
__host__ __device__ inline Work work_of(void* w, int64_t pages) {
  Work k;
  k.head = reinterpret_cast<int64_t*>(w);
  k.mark = reinterpret_cast<int32_t*>(k.head + 2);
  k.from = k.mark + pages;
  k.to = k.from + pages;
  return k;
}

// The lengths of a table without entries, none of which a pass over the entries sees.
__device__ __forceinline__ void check_lengths(const PageTable& t, int32_t P, WrongWord* wrong, int64_t first,
                                              int64_t step) {
  if (t.width > 0) return;
  for (int64_t s = first; s < t.rows; s += step) {
    bool bad;
    row_entries(t, s, P, &bad);
    if (bad) flag(wrong, kWrongLengths, s);
  }
}

__global__ __launch_bounds__(kThreads) void k_clear(int32_t* __restrict__ mark, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) mark[i] = 0;
}

__global__ __launch_bounds__(kThreads) void k_mark(PageTable t, int32_t P, int64_t pages, int32_t* __restrict__ mark,
                                                   WrongWord* __restrict__ wrong) {
  check_lengths(t, P, wrong, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
  const int64_t entries = t.rows * t.width;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < entries; e += (int64_t)gridDim.x * kThreads) {
    const int64_t s = e / t.width, j = e - s * t.width;
    bool bad;
    const int64_t n = row_entries(t, s, P, &bad);
    if (bad && j == 0) flag(wrong, kWrongLengths, s);
    if (j >= n) continue;
    const int64_t p = t.entries[s * t.stride + j];
    if (p >= 0 && p < pages)
      mark[p] = 1;
    else
      flag(wrong, kWrongIndex, e);
  }
}

// The free list, or (compact) the pairs and every page's new number, from the marks.
__global__ __launch_bounds__(kScanThreads) void k_scan(Work w, int64_t pages, int64_t* __restrict__ free_pages,
                                                       int64_t* __restrict__ count, int32_t compact) {
  __shared__ int64_t s_wave[kScanThreads / 64];
  int64_t mine = 0, live, sum;
  for (int64_t p = threadIdx.x; p < pages; p += blockDim.x) mine += w.mark[p];
  block_prefix(mine, s_wave, &live);
  if (threadIdx.x == 0) *count = compact ? live : pages - live;
  int64_t movers = 0, holes = 0;
  for (int64_t p0 = 0; p0 < pages; p0 += blockDim.x) {
    const int64_t p = p0 + threadIdx.x;
    const bool in = p < pages;
    const bool on = in && w.mark[p] != 0;
    if (!compact) {
      const int64_t rank = holes + block_prefix(in && !on ? 1 : 0, s_wave, &sum);
      holes += sum;
      if (in && !on) free_pages[rank] = p;
      continue;
    }
    const bool mover = on && p >= live, hole = in && !on && p < live;
    const int64_t m = movers + block_prefix(mover ? 1 : 0, s_wave, &sum);
    movers += sum;
    const int64_t h = holes + block_prefix(hole ? 1 : 0, s_wave, &sum);
    holes += sum;
    if (mover) w.from[m] = (int32_t)p;
    if (hole) w.to[h] = (int32_t)p;
    if (in) w.mark[p] = (int32_t)p;
  }
  if (!compact) return;
  __syncthreads();  // the lists are whole (one workgroup wrote them): as many movers as holes
  if (threadIdx.x == 0) w.head[1] = movers;
  for (int64_t k = threadIdx.x; k < movers; k += blockDim.x) w.mark[w.from[k]] = w.to[k];
}

// Clear, mark and scan in one workgroup, the marks a bit a page in LDS.
constexpr int64_t kLiveEntries = 16384;
constexpr int64_t kLivePages = 131072;

__global__ __launch_bounds__(kScanThreads) void k_live(PageTable t, int32_t P, int64_t pages, Work w,
                                                       int64_t* __restrict__ free_pages, int64_t* __restrict__ count,
                                                       int32_t compact, WrongWord* __restrict__ wrong) {
  __shared__ uint32_t s_live[kLivePages / 32];
  __shared__ int64_t s_wave[kScanThreads / 64];
  const int words = (int)((pages + 31) / 32);
  for (int i = threadIdx.x; i < words; i += kScanThreads) s_live[i] = 0;
  __syncthreads();
  check_lengths(t, P, wrong, threadIdx.x, kScanThreads);
  const int entries = (int)(t.rows * t.width), width = (int)t.width;
  for (int e = threadIdx.x; e < entries; e += kScanThreads) {
    const int s = e / width, j = e - s * width;
    bool bad;
    const int64_t n = row_entries(t, s, P, &bad);
    if (bad && j == 0) flag(wrong, kWrongLengths, s);
    if (j >= n) continue;
    const int64_t p = t.entries[s * t.stride + j];
    if (p >= 0 && p < pages)
      atomicOr(&s_live[p >> 5], 1u << (p & 31));
    else
      flag(wrong, kWrongIndex, e);
  }
  __syncthreads();
  int64_t mine = 0, live, sum;
  for (int i = threadIdx.x; i < words; i += kScanThreads) mine += __popc(s_live[i]);
  block_prefix(mine, s_wave, &live);
  if (threadIdx.x == 0) *count = compact ? live : pages - live;
  // movers (live, at or above the live count) in the low half, holes (dead, below it) in the high half;
  // for the free list every dead page is a hole
  int64_t before = 0;
  for (int i0 = 0; i0 < words; i0 += kScanThreads) {
    const int i = i0 + threadIdx.x;
    uint32_t on = 0, off = 0;
    if (i < words) {
      const int64_t left = pages - (int64_t)i * 32;
      const uint32_t all = left >= 32 ? ~0u : (1u << left) - 1;
      on = s_live[i];
      off = ~on & all;
      if (compact) {
        const int64_t below = live - (int64_t)i * 32;  // pages of the word below the live count
        const uint32_t low = below <= 0 ? 0 : below >= 32 ? ~0u : (1u << below) - 1;
        on &= ~low;
        off &= low;
        for (int k = 0; k < 32 && k < left; k++) w.mark[i * 32 + k] = i * 32 + k;
      }
    }
    const int64_t rank = before + block_prefix((int64_t)__popc(on) | (int64_t)__popc(off) << 32, s_wave, &sum);
    before += sum;
    int64_t m = rank & 0xffffffff, h = rank >> 32;
    for (; off; off &= off - 1) {
      const int p = i * 32 + __ffs(off) - 1;
      if (compact) w.to[h++] = p;
      else free_pages[h++] = p;
    }
    if (compact)
      for (; on; on &= on - 1) w.from[m++] = i * 32 + __ffs(on) - 1;
  }
  if (!compact) return;
  const int64_t movers = before & 0xffffffff;
  __syncthreads();  // the lists are whole: as many movers as holes
  if (threadIdx.x == 0) w.head[1] = movers;
  for (int64_t k = threadIdx.x; k < movers; k += kScanThreads) w.mark[w.from[k]] = w.to[k];
}

__global__ __launch_bounds__(kThreads) void k_compact(Geom g, Pieces pc, PageTable t, Work w,
                                                      int64_t* out, int64_t out_stride) {
  const int64_t pages = g.S / g.P;
  const int64_t entries = t.rows * t.width;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < entries; e += (int64_t)gridDim.x * kThreads) {
    const int64_t s = e / t.width, j = e - s * t.width;
    bool bad;
    const int64_t n = row_entries(t, s, g.P, &bad);
    const int64_t p = t.entries[s * t.stride + j];
    out[s * out_stride + j] = j < n && p >= 0 && p < pages ? (int64_t)w.mark[p] : p;
  }
  const int64_t moves = w.head[1];
  const int64_t units = moves * g.L * pc.end[g.nsub - 1];
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x)
    copy_unit(g, pc, moves, u, [&](int64_t i, int64_t* from, int64_t* to, int64_t* rows, bool) {
      *from = w.from[i];
      *to = w.to[i];
      *rows = g.P;
    });
}

unsigned grid_of(int64_t items, int32_t num_cus) {
  const int64_t cap = (int64_t)num_cus * 8;
  return (unsigned)(items < 1 ? 1 : (items < cap ? items : cap));
}

// The free list or the pairs, by one launch for tables that one workgroup gets through sooner than three
// launches start.  A free list by one launch and by three, in us a call: 1024 pages and 432 entries
// 11.4 and 16.1, 16384 entries 12.6 and 17.2, 32768 entries 21.1 and 17.4; 16384 pages and 16384 entries 15.7
// and 37.8; 131072 pages and 16384 entries 75 and 256.
hipError_t launch_live(const Geom& g, const PageTable& t, const Work& w, int64_t* free_pages, int64_t* count,
                       int32_t compact, WrongWord* wrong, int32_t num_cus, hipStream_t stream) {
  const int64_t pages = g.S / g.P, entries = t.rows * t.width;
  if (entries <= kLiveEntries && pages <= kLivePages) {
    k_live<<<dim3(1), kScanThreads, 0, stream>>>(t, g.P, pages, w, free_pages, count, compact, wrong);
    return hipGetLastError();
  }
  k_clear<<<dim3((unsigned)((pages + kThreads - 1) / kThreads)), kThreads, 0, stream>>>(w.mark, pages);
  if (t.rows > 0)
    k_mark<<<dim3(grid_of(((t.width > 0 ? entries : t.rows) + kThreads - 1) / kThreads, num_cus)), kThreads, 0, stream>>>(
        t, g.P, pages, w.mark, wrong);
  k_scan<<<dim3(1), kScanThreads, 0, stream>>>(w, pages, free_pages, count, compact);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_copy_pages(const Geom& g, const int64_t* src, const int64_t* dst, int64_t n, WrongWord* wrong,
                             int32_t num_cus, hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  const Pieces pc = layer_pieces(g);
  const int64_t units = n * g.L * pc.end[g.nsub - 1];
  (void)hipGetLastError();
  k_copy_pages<<<dim3(grid_of(units, num_cus)), kThreads, 0, stream>>>(g, pc, src, dst, n, wrong);
  return hipGetLastError();
}

hipError_t launch_fork_pages(const Geom& g, const ForkArgs& a, WrongWord* wrong, int32_t num_cus, hipStream_t stream) {
  const Pieces pc = layer_pieces(g);
  const int64_t units = a.n * g.L * pc.end[g.nsub - 1];
  (void)hipGetLastError();
  k_fork_plan<<<dim3(1), kScanThreads, 0, stream>>>(g.P, g.S / g.P, a, wrong);
  if (a.n > 0) k_fork<<<dim3(grid_of(units, num_cus)), kThreads, 0, stream>>>(g, pc, a, units, wrong);
  return hipGetLastError();
}

int64_t pages_workspace(const Geom& g) { return 16 + (g.S / g.P) * 12; }

hipError_t launch_free_pages(const Geom& g, const PageTable& t, int64_t* pages, int64_t* count, void* work,
                             WrongWord* wrong, int32_t num_cus, hipStream_t stream) {
  const Work w = work_of(work, g.S / g.P);
  (void)hipGetLastError();
  return launch_live(g, t, w, pages, count, 0, wrong, num_cus, stream);
}

hipError_t launch_compact_pages(const Geom& g, const PageTable& t, int64_t* out, int64_t out_stride, int64_t* count,
                                void* work, WrongWord* wrong, int32_t num_cus, hipStream_t stream) {
  const Work w = work_of(work, g.S / g.P);
  (void)hipGetLastError();
  hipError_t e = launch_live(g, t, w, nullptr, count, 1, wrong, num_cus, stream);
  if (e != hipSuccess) return e;
  if (t.rows * t.width == 0) return hipSuccess;  // nothing is named, nothing moves
  k_compact<<<dim3((unsigned)num_cus * 8), kThreads, 0, stream>>>(g, layer_pieces(g), t, w, out, out_stride);
  return hipGetLastError();
}

}  // namespace hc
