// Attention of a chunk of new tokens over the cached tokens of their sequences.
//
//   s_j = scale * q . k_j,  m = max s_j,  l = sum exp(s_j - m),  o = sum exp(s_j - m) v_j / l
//
// over the keys j that the row sees, in one pass: a step over some keys with maximum m' scales
// what was summed so far by exp(m - max(m, m')).  Exponentials are base 2, with log2(e) folded
// into the scale.
//
// The keys that a block of rows can see are [0, sinks) and [lo, hi); they are walked as one list of
// n = min(sinks, lo) + hi - lo positions, so a window costs what it shows, however long the cache.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <utility>

#include "hc_forward.h"

namespace hc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  typedef __bf16 elem;
  typedef bf16x8 v8;
  static __device__ __forceinline__ f32x4 mfma16(v8 a, v8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(v8 a, v8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
struct F16 {
  typedef _Float16 elem;
  typedef f16x8 v8;
  static __device__ __forceinline__ f32x4 mfma16(v8 a, v8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(v8 a, v8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

__device__ __forceinline__ void flag(WrongWord* wrong, Wrong kind, int64_t pos) {
  report_wrong<DeviceAtomic>(wrong, kind, pos);
}

// A sequence's rows and cached tokens; ok only when they are inside the call's bounds.
struct Seq {
  int64_t q0;
  int kv, m;
  bool ok;
};
__device__ __forceinline__ Seq sequence(const AttendArgs& a, int64_t s) {
  Seq r;
  r.q0 = a.q_start ? a.q_start[s] : s;
  const int64_t q1 = a.q_start ? a.q_start[s + 1] : s + 1;
  const int64_t kv = a.kv_len[s];
  r.ok = r.q0 >= 0 && q1 >= r.q0 && q1 <= a.q_rows && q1 - r.q0 <= a.max_q && kv >= 0 && kv <= a.max_kv;
  r.kv = r.ok ? (int)kv : 0;
  r.m = r.ok ? (int)(q1 - r.q0) : 0;
  return r;
}

// The keys that rows at positions [p0, p1] can see, as a list: i < sk is key i, others key
// lo + i - sk.  Rows, keys and positions are below 2^30 in size, so 32 bits hold them.
struct Span {
  int lo, sk, n;
  __device__ __forceinline__ int key(int i) const { return i < sk ? i : lo + (i - sk); }
};
__device__ __forceinline__ Span span_of(const AttendArgs& a, int kv, int p0, int p1) {
  Span s;
  int hi = kv;
  s.lo = 0;
  if (a.causal) {
    hi = p1 + 1 < kv ? p1 + 1 : kv;
    hi = hi < 0 ? 0 : hi;
    if (a.window > 0 && p0 - a.window + 1 > 0) s.lo = p0 - a.window + 1;
    if (s.lo > hi) s.lo = hi;
  }
  s.sk = a.sinks < s.lo ? a.sinks : s.lo;
  s.n = s.sk + hi - s.lo;
  return s;
}
__device__ __forceinline__ bool visible(const AttendArgs& a, int p, int j) {
  return !a.causal | ((j <= p) & ((a.window == 0) | (p - j < a.window) | (j < a.sinks)));
}

// Of the 64 keys at positions base, base + 1, ... of a span those that a row at position p sees, a bit
// each; `there`: those that are there at all.  In positions of the list: not past p, and past p - window or
// below sinks (a window starts at or before p, so the sinks in front of it are never past p).
__device__ __forceinline__ uint64_t first_bits(int n) {  // n of them: none below 0, all from 64 on
  return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ uint64_t sees(const AttendArgs& a, const Span& s, uint64_t there, int p, int base) {
  if (!a.causal) return there;
  const int at = p - s.lo + s.sk - base;  // the row's own key
  uint64_t m = there & first_bits(at + 1);
  if (a.window > 0) m &= first_bits(a.sinks - base) | ~first_bits(at - a.window + 1);
  return m;
}

// |scale| in base 2, above 0: hidden scores are -infinity and have to stay that.  For a scale of 0 it is fp32's
// least number, which brings the largest scores down to 2^-21, so that all weights are alike.
__device__ __forceinline__ float weight_scale(const AttendArgs& a) {
  return a.scale == 0.f ? 0x1p-149f : fabsf(a.scale) * kLog2e;
}

constexpr uint32_t kNoSlot = 0xffffffffu;  // layers hold fewer rows: 2^32 of the smallest are 512 GiB

// Slot of key j (below 2^31) of sequence s in two steps, so that a kernel can load a table entry long
// before it needs the slot: a wait for a load waits for all that were issued before it.
struct Entry {
  int64_t page;      // what the table says
  int64_t at;        // its place in the table, -1: no key
  uint32_t rest;     // token inside the entry
};
__device__ __forceinline__ Entry entry_of(const AttendArgs& a, int64_t s, uint32_t j) {
  const uint32_t e = (uint32_t)(((uint64_t)j * a.entry_magic) >> a.entry_shift);  // j / entry
  Entry r;
  r.at = s * a.table_stride + e;
  r.rest = j - e * (uint32_t)a.entry;
  r.page = a.table[r.at];
  return r;
}
// kNoSlot for no key, and for a bad table entry, which is reported.
__device__ __forceinline__ uint32_t slot_from(const AttendArgs& a, const Entry& e) {
  if (e.at < 0) return kNoSlot;
  if (e.page < 0 || e.page >= a.entries) {
    flag(a.wrong, kWrongIndex, e.at);
    return kNoSlot;
  }
  return (uint32_t)e.page * (uint32_t)a.entry + e.rest;
}
__device__ __forceinline__ uint32_t slot_of(const AttendArgs& a, int64_t s, uint32_t j) {
  return slot_from(a, entry_of(a, s, j));
}

// 16 bytes a lane from memory into LDS, lane i to lds + 16 i (lds the same in all lanes), past the
// registers.  Nothing waits for it but lds_arrived, of the wave that loaded.
// (m0 is reserved, which the compiler remarks on: it keeps no values of its own there, but what it puts there for an
// instruction has to be put there again behind this.)
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_load(const uint8_t* from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
}
__device__ __forceinline__ void lds_arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}

// ---------------------------------------------------------------- one row, key by key
// Softmax sums of one query row over positions [i0, i1) of its span, by one wave: lanes take keys
// for the scores and dims for the sum, and nothing of a key that the row does not see is touched.
// The tiled kernels multiply hidden keys' values by a weight of 0, which is NaN where the value is
// not finite; they do the rows that came out NaN again with this, unless the sum of weights is NaN too: then a score
// that the row sees is, and so is the row.  (One row costs as much as a hundred in tiles: 2048 rows behind 14336, all of
// NaN queries, took 160 ms, now 0.6.)  s_q: DK floats of this wave's.
template <class T, int DK, int DV>
__device__ __forceinline__ void exact_row(const AttendArgs& a, int64_t s, int64_t row, int h, int p, Span span,
                                       int i0, int i1, float* s_q, float* o, float* m_out, float* l_out) {
  typedef typename T::elem elem;
  const int lane = threadIdx.x & 63;
  const int hk = h / a.group;
  const elem* qp = reinterpret_cast<const elem*>(a.q) + row * a.q_stride[0] + h * a.q_stride[1];
  __builtin_amdgcn_wave_barrier();
  for (int i = lane; i < DK; i += 64) s_q[i] = (float)qp[i];
  __builtin_amdgcn_wave_barrier();
  constexpr int ND = DV / 64;
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < ND; c++) o[c] = 0.f;
  const float scale = a.scale * kLog2e;
#pragma unroll 1
  for (int base = i0; base < i1; base += 64) {
    const int i = base + lane;
    float x = -INFINITY;
    uint32_t slot = kNoSlot;
    if (i < i1) {
      const int j = span.key(i);
      if (visible(a, p, j)) slot = slot_of(a, s, (uint32_t)j);
    }
    if (slot != kNoSlot) {
      const v4u* kp = reinterpret_cast<const v4u*>(a.k_rows + 2 * ((int64_t)slot * a.k_row + (int64_t)hk * DK));
      x = 0.f;
#pragma unroll 1
      for (int v = 0; v < DK / 8; v++) {
        const f32x8 kv = __builtin_convertvector(__builtin_bit_cast(typename T::v8, kp[v]), f32x8);
#pragma unroll
        for (int c = 0; c < 8; c++) x += kv[c] * s_q[v * 8 + c];
      }
      x *= scale;
    }
    float top = x;
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    // a score that is NaN is not a maximum, and makes the sums NaN
    const float next = fmaxf(m, top);
    const float zero = next == -INFINITY ? 0.f : next;
    const float keep = exp2f(m - zero), e = slot != kNoSlot ? exp2f(x - zero) : 0.f;
    m = next;
    float sum = e;
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    l = l * keep + sum;
#pragma unroll
    for (int c = 0; c < ND; c++) o[c] *= keep;
    uint64_t todo = __ballot(slot != kNoSlot);
    while (todo) {
      const int j = __builtin_ctzll(todo);
      todo &= todo - 1;
      const float pj = __shfl(e, j);
      const uint32_t sj = __shfl(slot, j);
      const elem* vp = reinterpret_cast<const elem*>(a.v_rows) + (int64_t)sj * a.v_row + (int64_t)hk * (DK == DV ? DV : 0);
#pragma unroll
      for (int c = 0; c < ND; c++) o[c] += pj * (float)vp[c * 64 + lane];
    }
  }
  *m_out = m;
  *l_out = l;
}

// ---------------------------------------------------------------- the list of work items
// A sequence's query rows times the heads of a KV head's group make row lists of m * group rows,
// row r being token r / group and head r % group of the group; R rows make a row tile.  An item is
// (sequence, KV head, row tile, split): `splits` items share a tile's keys.  Every workgroup works
// out the list for itself from the lengths, so that its number of items follows the lengths as
// they are on the device: a sequence gets a split per C keys, C being the whole call's keys over
// the wanted number of items.
struct Item {
  int64_t s;
  Seq q;
  int32_t hk, tile, split, splits;
  int64_t index;  // place in the list: where its partial result lies, if its tile is split
};

struct PlanCount {
  int64_t tiles, n;  // row tiles of the sequence, positions of the span of all its rows
};
__device__ __forceinline__ PlanCount plan_count(const AttendArgs& a, int64_t s, int R, Seq* q) {
  *q = sequence(a, s);
  PlanCount c = {0, 0};
  if (!q->ok || q->m == 0) return c;
  c.tiles = ((int64_t)q->m * a.group + R - 1) / R;
  c.n = span_of(a, q->kv, q->kv - q->m, q->kv - 1).n;
  return c;
}

__device__ __forceinline__ int64_t wave_prefix(int64_t x) {  // inclusive
  const int lane = threadIdx.x & 63;
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// What the joining launch has to know of an item that has a place for a partial result, behind all of those.
struct Part {
  int64_t splits;  // of the tile whose first split the item is, else 0
  int64_t q0, m, tile_hk;
};

// Keys of a split, for a call of `work` pairs of row tiles and keys.
__device__ __forceinline__ int64_t split_keys(const AttendArgs& a, int64_t work) {
  const int64_t C = (work * a.kv_heads + a.target - 1) / a.target;
  return C < a.min_split ? a.min_split : C;
}

// Item `rest` of a sequence's: its row tiles from the last, whose rows see the most keys, to the first.
__device__ __forceinline__ void set_item(const AttendArgs& a, Item* it, int64_t s, const Seq& q, int64_t tiles,
                                         int64_t splits, int64_t rest) {
  it->s = s;
  it->splits = (int32_t)splits;
  const int64_t unit = rest / it->splits, back = unit / a.kv_heads;
  it->split = (int32_t)(rest - unit * it->splits);
  it->hk = (int32_t)(unit - back * a.kv_heads);
  it->tile = (int32_t)(tiles - 1 - back);
  it->q = q;
  it->index = blockIdx.x;
}

// Finds item blockIdx.x of the list (256 threads; s_plan: 8 int64); false when the list is shorter.
// `parts`: where the items' Parts are kept, when there is a joining launch.
// SPLIT_FIRST: calls with fewer places of partial results than items, in which the items of split tiles come first in
// the list, so that a partial result's place stays its item's.  (Kernels of their own: the other calls' loops get
// registers as if there were none, which otherwise cost 1.5 % of a chunk of 2048.)
// FEW: calls of a few sequences have a way of their own, in the kernels of few rows (in those of many it
// cost 3 % of a chunk of 2048, 575 us for 560, by the registers that the compiler then gave the loop).
template <bool FEW, bool SPLIT_FIRST>
__device__ __forceinline__ bool find_item(const AttendArgs& a, int R, int64_t* s_plan, Part* parts, Item* it) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t want = blockIdx.x;
  int64_t work = 0;
  Seq q = {0, 0, 0, true};
  PlanCount c = {0, 0};
  bool found = false;
  if (FEW && !SPLIT_FIRST && a.num_seqs <= 4) {
    // a few sequences: every thread goes over them by itself, without the steps of a reduction and a
    // prefix over threads (1.5 us of a single sequence's decoding)
    for (int64_t s = 0; s < a.num_seqs; s++) {
      c = plan_count(a, s, R, &q);
      if (blockIdx.x == 0 && threadIdx.x == 0 && !q.ok) flag(a.wrong, kWrongLengths, s);
      work += c.tiles * c.n;
    }
    const int64_t C = split_keys(a, work);
    int64_t at = 0;
    for (int64_t s = 0; s < a.num_seqs && !found; s++) {
      if (a.num_seqs > 1) c = plan_count(a, s, R, &q);
      const int64_t splits = c.n <= C ? 1 : (c.n + C - 1) / C, mine = c.tiles * splits * a.kv_heads;
      found = want < at + mine;
      if (found) set_item(a, it, s, q, c.tiles, splits, want - at);
      at += mine;
    }
  } else {
    for (int64_t s = threadIdx.x; s < a.num_seqs; s += 256) {
      c = plan_count(a, s, R, &q);
      if (blockIdx.x == 0 && !q.ok) flag(a.wrong, kWrongLengths, s);
      work += c.tiles * c.n;
    }
    for (int d = 1; d < 64; d <<= 1) work += __shfl_xor(work, d);
    if (lane == 0) s_plan[wave] = work;
    __syncthreads();
    work = 0;
    for (int w = 0; w < 4; w++) work += s_plan[w];
    const int64_t C = split_keys(a, work);
    int64_t before = 0;
    bool split_ones = false;
    if (SPLIT_FIRST) {
      int64_t first = 0;
      for (int64_t s = threadIdx.x; s < a.num_seqs; s += 256) {
        if (a.num_seqs > 256) c = plan_count(a, s, R, &q);
        if (c.n > C) first += c.tiles * ((c.n + C - 1) / C) * a.kv_heads;
      }
      for (int d = 1; d < 64; d <<= 1) first += __shfl_xor(first, d);
      __syncthreads();
      if (lane == 0) s_plan[wave] = first;
      __syncthreads();
      first = 0;
      for (int w = 0; w < 4; w++) first += s_plan[w];
      split_ones = want < first;
      before = split_ones ? 0 : first;
    }
    for (int64_t s0 = 0; s0 < a.num_seqs; s0 += 256) {
      const int64_t s = s0 + threadIdx.x;
      if (a.num_seqs > 256) {  // else they are at hand
        c = {0, 0};
        if (s < a.num_seqs) c = plan_count(a, s, R, &q);
      }
      const int64_t splits = c.n <= C ? 1 : (c.n + C - 1) / C;
      const int64_t mine = SPLIT_FIRST && (splits > 1) != split_ones ? 0 : c.tiles * splits * a.kv_heads;
      const int64_t incl = wave_prefix(mine);
      __syncthreads();
      if (lane == 63) s_plan[wave] = incl;
      __syncthreads();
      int64_t at = before + incl - mine;
      for (int w = 0; w < 4; w++) {
        if (w < wave) at += s_plan[w];
        before += s_plan[w];
      }
      found = want < before;
      __syncthreads();
      if (want >= at && want < at + mine) {
        s_plan[0] = s;
        s_plan[1] = splits;
        s_plan[2] = want - at;
        s_plan[3] = c.tiles;
        s_plan[4] = q.q0;
        s_plan[5] = q.kv;
        s_plan[6] = q.m;
      }
      if (found) break;
    }
    __syncthreads();
    if (found)
      set_item(a, it, s_plan[0], {s_plan[4], (int)s_plan[5], (int)s_plan[6], true}, s_plan[3], s_plan[1], s_plan[2]);
    __syncthreads();
  }
  if ((SPLIT_FIRST ? want < a.slots : a.join_parts > 0) && threadIdx.x == 0) {
    Part p = {0, 0, 0, 0};
    if (found && it->split == 0) p = {it->splits, it->q.q0, it->q.m, (int64_t)it->tile * a.kv_heads + it->hk};
    parts[want] = p;
  }
  return found;
}

// Floats of a partial result: per row the sum over values, then maximum and sum of weights.
template <int DV>
__host__ __device__ constexpr int64_t partial_floats(int R) {
  return (int64_t)R * (DV + 2);
}
template <int DV, int R>
__device__ __forceinline__ Part* parts_of(const AttendArgs& a) {
  return reinterpret_cast<Part*>(a.work + a.slots * partial_floats<DV>(R));
}

// ---------------------------------------------------------------- few rows: decoding
// Rows: up to 16 (token, head) pairs of one KV head, so K and V are read once for all of them.
// What bounds it is memory: 2 * 16 * D operations on 4 * D bytes of a key.  So a wave works alone
// on tiles of 32 keys, rows of K straight from memory into the operand registers of the
// product, the next tile's K and V on their way while one is computed, and waves and splits are
// joined only at the end.
//
//   S^T = K Q^T   (A: 16 keys, B: 16 rows): a lane ends with one row's scores of 8 of the 32 keys,
//                 keys 16 t + 4 (lane / 16) + r, so a row's maximum and sum need two lane swaps
//   O^T += V^T P^T (B: the same lane's 8 weights as they stand): the order of the keys inside the
//                 product is free, so V^T is read in that order: V goes through LDS and comes
//                 back transposed, four keys of a dim a lane
//
// Measured: 64 sequences up to 8192 tokens, 8 KV heads of 128, 208 us = 5.3 TB/s; 32 sequences in a window
// of 4096 with 4 sinks, scattered slots, heads of 64, 62 us = 4.2 TB/s; one sequence of 1500 8 us and 4 us to
// join. Eight workgroups a compute unit in the list of items: 4 213 us, 16 217 us, 32 254 us on the
// first; three waves a SIMD instead of two (which spills) 232 us.
constexpr int kRowTile = 16;
constexpr int kKeys = 32;

template <int D>
__device__ __forceinline__ int v_swizzle(int row) {  // 16-byte chunks of a V row change places by its row:
  return D == 128 ? 2 * (row & 7) : 2 * ((row >> 1) & 3);  // the transposing reads then spread over all banks
}

template <class T, int D, bool SPLIT_FIRST>
__global__ __launch_bounds__(256, 2) void k_attend_decode(AttendArgs a) {
  typedef typename T::v8 v8;
  typedef typename T::elem elem;
  constexpr int KS = D / 32;            // product steps over the head
  constexpr int DT = D / 16;            // 16-dim tiles of the output
  constexpr int CH = D / 8;             // 16-byte chunks of a row
  constexpr int VL = kKeys * CH / 64;   // V loads of a lane
  __shared__ __align__(16) uint8_t s_v[4][kKeys * D * 2];
  __shared__ float s_m[4][kRowTile], s_l[4][kRowTile], s_q[4][D];
  __shared__ int64_t s_plan[8];
  Item it;
  if (!find_item<true, SPLIT_FIRST>(a, kRowTile, s_plan, parts_of<D, kRowTile>(a), &it)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int rows_all = it.q.m * a.group;
  const int r0 = it.tile * kRowTile;
  const int rows = rows_all - r0 < kRowTile ? rows_all - r0 : kRowTile;
  // this lane's row
  const int r = r0 + (col < rows ? col : 0);
  const int tok = r / a.group, h = it.hk * a.group + (r - tok * a.group);
  const int64_t row = it.q.q0 + tok;
  const int p = it.q.kv - it.q.m + tok;
  const int p_first = it.q.kv - it.q.m + r0 / a.group, p_last = it.q.kv - it.q.m + (r0 + rows - 1) / a.group;
  const Span span = span_of(a, it.q.kv, p_first, p_last);
  // this split's part of the span
  const int part = ((span.n + it.splits - 1) / it.splits + 127) / 128 * 128;
  const int i0 = (int64_t)it.split * part < span.n ? it.split * part : span.n;
  const int i1 = i0 + part < span.n ? i0 + part : span.n;
  v8 q[KS];
  {
    const v4u* qp = reinterpret_cast<const v4u*>(a.q + 2 * (row * a.q_stride[0] + h * a.q_stride[1]));
#pragma unroll
    for (int i = 0; i < KS; i++) {
      const v4u x = qp[i * 4 + quad];
      q[i] = __builtin_bit_cast(v8, col < rows ? x : v4u{0, 0, 0, 0});
    }
  }
  f32x4 o[DT] = {};
  float m = -INFINITY, l = 0.f;
  const float scale = a.scale * kLog2e;
  const uint8_t* kb = a.k_rows + 2 * (int64_t)it.hk * D;
  const uint8_t* vb = a.v_rows + 2 * (int64_t)it.hk * D;
  const uint64_t k_row = 2 * a.k_row, v_row = 2 * a.v_row;
  uint8_t* sv = s_v[wave];
  // Slot of the tile's key lane % 32, kNoSlot past the end and for a key that no row sees: with one
  // token a tile (decoding) that is every hidden key, whose values then are zeros in the product.
  auto entry = [&](int base) {
    const int i = base + (lane & 31);
    const int j = span.key(i < i1 ? i : i0);
    Entry e = {0, -1, 0};
    if (i < i1 && (p_first != p_last || visible(a, p_first, j))) e = entry_of(a, it.s, (uint32_t)j);
    return e;
  };
  v4u kreg[2][KS], vreg[VL];
  auto load_k = [&](uint32_t slot) {
#pragma unroll
    for (int t = 0; t < 2; t++) {
      const uint32_t sl = __shfl(slot, t * 16 + col);
      const v4u* kp = reinterpret_cast<const v4u*>(kb + (sl == kNoSlot ? 0 : sl * k_row));
#pragma unroll
      for (int i = 0; i < KS; i++) kreg[t][i] = kp[i * 4 + quad];
    }
  };
  auto load_v = [&](uint32_t slot) {
#pragma unroll
    for (int c = 0; c < VL; c++) {
      const int x = c * 64 + lane;
      const uint32_t sl = __shfl(slot, x / CH);
      const v4u y = *reinterpret_cast<const v4u*>(vb + (sl == kNoSlot ? 0 : sl * v_row) + (x % CH) * 16);
      vreg[c] = sl == kNoSlot ? v4u{0, 0, 0, 0} : y;
    }
  };
  int base = i0 + wave * kKeys;
  Entry next_entry = entry(base + 128);
  uint32_t slot = slot_from(a, entry(base)), slot_next = kNoSlot;
  if (base < i1) {
    load_k(slot);
    load_v(slot);
  }
  for (; base < i1; base += 128) {
    f32x4 st[2] = {};
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int i = 0; i < KS; i++) st[t] = T::mfma16(__builtin_bit_cast(v8, kreg[t][i]), q[i], st[t]);
    const uint32_t there = (uint32_t)__ballot(slot != kNoSlot);
    const bool more = base + 128 < i1;
    slot_next = slot_from(a, next_entry);
    next_entry = entry(base + 256);
    if (more) load_k(slot_next);
    // V into LDS, and the next tile's on its way
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int c = 0; c < VL; c++) {
      const int x = c * 64 + lane, key = x / CH;
      *reinterpret_cast<v4u*>(sv + key * D * 2 + ((x % CH) ^ v_swizzle<D>(key)) * 16) = vreg[c];
    }
    if (more) load_v(slot_next);
    // hidden keys: past the end, bad entries, and those that this row does not see
    const bool whole = there == 0xffffffffu &&
                       (!a.causal || (span.key(base + kKeys - 1) <= p_first &&
                                      (a.window == 0 || p_last - span.key(base) < a.window)));
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; e++) x[e] = st[e / 4][e % 4] * scale;
    if (!whole) {
      const uint32_t see = (uint32_t)sees(a, span, there, p, base) >> (quad * 4);
#pragma unroll
      for (int e = 0; e < 8; e++) x[e] = (see >> (e / 4 * 16 + e % 4)) & 1 ? x[e] : -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 8; e++) top = fmaxf(top, x[e]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float next = fmaxf(m, top);
    const float zero = next == -INFINITY ? 0.f : next;
    const float keep = __builtin_amdgcn_exp2f(m - zero);
    m = next;
    float sum = 0.f;
    f32x8 w;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      w[e] = __builtin_amdgcn_exp2f(x[e] - zero);
      sum += w[e];
    }
    l = l * keep + sum;  // this lane's keys; the quads are summed at the end
    const v8 wt = __builtin_convertvector(w, v8);  // the weight's one rounding, as the product's operand
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int d = 0; d < DT; d++) {
      s16x4 v[2];
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const int key = t * 16 + quad * 4 + col / 4;
        const int chunk = (d * 2 + (col & 3) / 2) ^ v_swizzle<D>(key);
        v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(sv + key * D * 2 + chunk * 16 + (col & 1) * 8));
      }
      const v8 vt = __builtin_bit_cast(v8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
      o[d] *= keep;
      o[d] = T::mfma16(vt, wt, o[d]);
    }
    slot = slot_next;
  }
  // Join the four waves through LDS (over V, which is done with): 16 threads to a row, 8 or 4 dims each.
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (lane < kRowTile) {
    s_m[wave][lane] = m;
    s_l[wave][lane] = l;
  }
  __syncthreads();  // every wave is done with V: a wave's sums take more LDS than its values did
  float* so = reinterpret_cast<float*>(&s_v[0][0]);  // [wave][row][D]
  if (col < rows) {
#pragma unroll
    for (int d = 0; d < DT; d++) *reinterpret_cast<f32x4*>(so + (wave * kRowTile + col) * D + d * 16 + quad * 4) = o[d];
  }
  __syncthreads();
  constexpr int E = D / 16;
  const int rr = threadIdx.x / 16, d0 = threadIdx.x % 16 * E;
  const bool valid = rr < rows;  // all lanes stay: a row that came out NaN takes the whole wave
  float m_all = s_m[0][rr];
  for (int w = 1; w < 4; w++) m_all = fmaxf(m_all, s_m[w][rr]);
  const float zero = m_all == -INFINITY ? 0.f : m_all;
  float l_all = 0.f, acc[E] = {};
#pragma unroll
  for (int w = 0; w < 4; w++) {
    const float f = __builtin_amdgcn_exp2f(s_m[w][rr] - zero);
    l_all += s_l[w][rr] * f;
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] += so[(w * kRowTile + rr) * D + d0 + e] * f;
  }
  bool nan = false;
#pragma unroll
  for (int e = 0; e < E; e++) nan |= acc[e] != acc[e];
  const uint64_t bits = __ballot(nan && valid && l_all == l_all);  // a row's 16 threads are in one wave
  const bool bad = (bits >> (lane & 48)) & 0xffff;
  float* part_o = a.work + it.index * partial_floats<D>(kRowTile);
  float* part_ml = part_o + kRowTile * D;
  auto finish = [&](int y, float mm, float ll) {
    if (it.splits > 1) {
      part_ml[y * 2] = mm;
      part_ml[y * 2 + 1] = ll;
    } else if (a.lse) {
      const int rt = (r0 + y) / a.group, rh = it.hk * a.group + (r0 + y - rt * a.group);
      a.lse[(it.q.q0 + rt) * a.q_heads + rh] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
  };
  if (valid && !bad) {
    if (it.splits > 1) {
#pragma unroll
      for (int e = 0; e < E; e++) part_o[rr * D + d0 + e] = acc[e];
    } else {
      typedef elem ev __attribute__((ext_vector_type(E)));
      typedef float fv __attribute__((ext_vector_type(E)));
      const int rt = (r0 + rr) / a.group, rh = it.hk * a.group + (r0 + rr - rt * a.group);
      fv y;
#pragma unroll
      for (int e = 0; e < E; e++) y[e] = l_all == 0.f ? 0.f : acc[e] / l_all;
      *reinterpret_cast<ev*>(reinterpret_cast<elem*>(a.out) + (it.q.q0 + rt) * a.out_stride[0] + rh * a.out_stride[1] + d0) =
          __builtin_convertvector(y, ev);
    }
    if (d0 == 0) finish(rr, m_all, l_all);
  }
  // rows that came out NaN, by the wave that holds them
  if (bits) {
    for (int k = 0; k < 4; k++) {
      const int y = wave * 4 + k;
      if (!((bits >> (k * 16)) & 0xffff)) continue;
      const int rt = (r0 + y) / a.group, rh = it.hk * a.group + (r0 + y - rt * a.group);
      float oo[D / 64], mm, ll;
      exact_row<T, D, D>(a, it.s, it.q.q0 + rt, rh, it.q.kv - it.q.m + rt, span, i0, i1, s_q[wave], oo, &mm, &ll);
      for (int c = 0; c < D / 64; c++) {
        if (it.splits > 1)
          part_o[y * D + c * 64 + lane] = oo[c];
        else
          reinterpret_cast<elem*>(a.out)[(it.q.q0 + rt) * a.out_stride[0] + rh * a.out_stride[1] + c * 64 + lane] =
              (elem)(ll == 0.f ? 0.f : oo[c] / ll);
      }
      if (lane == 0) finish(y, mm, ll);
    }
  }
}

// ---------------------------------------------------------------- many rows: chunks and prompts
// A workgroup takes 128 (token, head) rows of one KV head, 32 a wave, and walks its keys in tiles of
// 64 whose K and V all four waves read from LDS.  4 * D operations on a pair make it bound by the
// matrix cores, and next to them by the exponentials and by LDS, 2 * 64 * D * 2 bytes a wave and tile.
//
// The products are the decoding kernel's in their 32 x 32 form: S^T = K Q^T leaves a lane with one
// row's scores of 32 of the 64 keys, 8 q + 4 (lane / 32) + r of each 32, which are the operand of
// O^T += V^T P^T as they stand; V comes from LDS transposed, in that order of the keys.  The next tile
// is loaded into the other half of LDS while one is computed: one barrier a tile.
//
// Measured: a chunk of 2048 behind 14336 cached, 32/8 heads of 128, 548 to 578 us over machines = 890 to 940 TFLOP/s;
// four prompts of unequal lengths up to 4096 of fp16 16/4 heads of 64, 114 to 121 us = 530 to 560 TFLOP/s, of
// equal lengths 646, one of 16384 757: short prompts behind long ones leave places empty at the end. Waves in a product go before others (s_setprio): two waves of a
// SIMD that multiply at the same time would also compute weights at the same time, 574 us for 557.
//
// The maximum that a row's weights are relative to is replaced only when it grows by more than
// 2^8: until then weights of up to 2^8 are summed, which loses nothing in fp32 or as operands, and the
// sums need not be scaled.
constexpr int kTileRows = 128;
constexpr int kTileKeys = 64;
constexpr float kGrow = 8.f;

// Which chunk of a K row lies at a place of it, and back: 16 rows' same chunk in 16 places.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int chunk) {
  return chunk ^ (D == 128 ? row & 15 : (row >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int k_place(int row, int chunk) {
  return row * D * 2 + k_chunk<D>(row, chunk) * 16;
}
// Of a V row: four rows' 32 dims side by side.
template <int D>
__device__ __forceinline__ int v_chunk(int row, int chunk) {
  return chunk ^ (D == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2);
}
template <int D>
__device__ __forceinline__ int v_place(int row, int chunk) {
  return row * D * 2 + v_chunk<D>(row, chunk) * 16;
}

template <class T, int D, bool SPLIT_FIRST>
__global__ __launch_bounds__(256, 2) void k_attend_tiles(AttendArgs a) {
  constexpr int R = kTileRows;
  typedef typename T::v8 v8;
  typedef typename T::elem elem;
  constexpr int KS = D / 16;                    // product steps over the head
  constexpr int DT = D / 32;                    // 32-dim tiles of the output
  constexpr int CH = D / 8;                     // 16-byte chunks of a row
  constexpr int W = 4;                          // waves
  constexpr int LD = kTileKeys * CH / (64 * W);      // loads of a wave, K and V each
  constexpr int BUF = kTileKeys * D * 2;        // bytes of a K or V tile
  __shared__ __align__(256) uint8_t s_k[2][BUF], s_v[2][BUF];
  __shared__ int64_t s_plan[8];
  Item it;
  if (!find_item<false, SPLIT_FIRST>(a, R, s_plan, parts_of<D, R>(a), &it)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int64_t rows_all = (int64_t)it.q.m * a.group;
  const int64_t t0 = (int64_t)it.tile * R;
  const int rows_tile = rows_all - t0 < R ? (int)(rows_all - t0) : R;
  // this lane's row, and the positions of the tile's and the wave's first and last rows
  const int rr = wave * 32 + col;
  const bool live = rr < rows_tile;
  const int64_t r = t0 + (live ? rr : 0);
  const int tok = (int)(r / a.group), h = it.hk * a.group + (int)(r - (int64_t)tok * a.group);
  const int64_t row = it.q.q0 + tok;
  const int before = it.q.kv - it.q.m;
  const int p = before + tok;
  const int p_first = before + (int)(t0 / a.group), p_last = before + (int)((t0 + rows_tile - 1) / a.group);
  const Span span = span_of(a, it.q.kv, p_first, p_last);
  const int part = ((span.n + it.splits - 1) / it.splits + kTileKeys - 1) / kTileKeys * kTileKeys;
  const int i0 = (int64_t)it.split * part < span.n ? it.split * part : span.n;
  const int i1 = i0 + part < span.n ? i0 + part : span.n;
  // weights are exp2(c * score - c * maximum); a negative scale turns the queries' sign
  const float c = weight_scale(a);
  v8 q[KS];
  {
    const v4u* qp = reinterpret_cast<const v4u*>(a.q + 2 * (row * a.q_stride[0] + h * a.q_stride[1]));
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < KS; i++) {
      const v4u x = qp[i * 2 + half] ^ flip;
      q[i] = __builtin_bit_cast(v8, live ? x : v4u{0, 0, 0, 0});
    }
  }
  auto entry = [&](int base) {  // of key `lane` of the tile
    const int i = base + lane;
    Entry e = {0, -1, 0};
    if (i < i1) e = entry_of(a, it.s, (uint32_t)span.key(i));
    return e;
  };
  // One instruction carries 64 chunks; the swizzle is in which chunk of its row a lane fetches, the same
  // one in every instruction.  Rows of K and V are equally far apart, so a key's lane works out where its
  // rows are once and the lanes that fetch them only add their own part.
  constexpr int RL = 64 / CH;  // rows of an instruction
  const int from = wave * RL + lane / CH;  // a lane's first row, the next W RL on
  const uint8_t* kl = a.k_rows + 2 * (int64_t)it.hk * D + k_chunk<D>(from, lane % CH) * 16;
  const uint8_t* vl = a.v_rows + 2 * (int64_t)it.hk * D + v_chunk<D>(from, lane % CH) * 16;
  auto load = [&](uint32_t slot, int buf) {
    const uint64_t row = slot == kNoSlot ? 0 : (uint64_t)slot * (2 * a.k_row);
    const uint32_t lo = (uint32_t)row, hi = (uint32_t)(row >> 32);
#pragma unroll
    for (int x = 0; x < LD; x++) {
      const int key = x * W * RL + from;
      const uint64_t at = (uint64_t)__shfl(hi, key) << 32 | __shfl(lo, key);
      lds_load(kl + at, lds_offset(s_k[buf] + (x * W + wave) * 1024));
      lds_load(vl + at, lds_offset(s_v[buf] + (x * W + wave) * 1024));
    }
  };
  f32x16 o[DT] = {};
  float m = -INFINITY, l = 0.f;
  Entry next_entry = entry(i0 + kTileKeys);
  uint32_t slot = slot_from(a, entry(i0));
  if (i0 < i1) load(slot, 0);
  lds_arrived();
  __syncthreads();
  int buf = 0;
  for (int base = i0; base < i1; base += kTileKeys) {
    const uint64_t there = __ballot(slot != kNoSlot);
    slot = slot_from(a, next_entry);
    next_entry = entry(base + 2 * kTileKeys);
    if (base + kTileKeys < i1) load(slot, buf ^ 1);
    if (there != ~0ull) {  // what was fetched in place of no key must not reach the product: its value is zero
      for (int x = threadIdx.x; x < kTileKeys * CH; x += 64 * W)
        if (!((there >> (x / CH)) & 1)) *reinterpret_cast<v4u*>(s_v[buf] + x * 16) = v4u{0, 0, 0, 0};
      __syncthreads();
    }
    __builtin_amdgcn_s_setprio(1);  // waves in a product before others: two of a SIMD then fall out of step
    f32x16 st[2] = {};
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int i = 0; i < KS; i++) {
        const v8 k = *reinterpret_cast<const v8*>(s_k[buf] + k_place<D>(u * 32 + col, i * 2 + half));
        st[u] = T::mfma32(k, q[i], st[u]);
      }
    __builtin_amdgcn_s_setprio(0);
    float x[32];
#pragma unroll
    for (int e = 0; e < 32; e++) x[e] = st[e / 16][e % 16];
    const bool whole = there == ~0ull && (!a.causal || (span.key(base + kTileKeys - 1) <= p_first &&
                                                        (a.window == 0 || p_last - span.key(base) < a.window)));
    if (!whole) {
      const uint64_t see = sees(a, span, there, p, base) >> (half * 4);
      const uint32_t part[2] = {(uint32_t)see, (uint32_t)(see >> 32)};
#pragma unroll
      for (int e = 0; e < 32; e++) x[e] = (part[e / 16] >> (e % 16 / 4 * 8 + e % 4)) & 1 ? x[e] : -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 32; e++) top = fmaxf(top, x[e]);
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any((top - m) * c > kGrow || (m == -INFINITY && top != -INFINITY))) {
      const float next = fmaxf(m, top);
      const float keep = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - next) * c);
      m = next;
      l *= keep;
#pragma unroll
      for (int d = 0; d < DT; d++) o[d] *= keep;
    }
    const float zero = m == -INFINITY ? 0.f : m * c;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 32; e++) {
      x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c, -zero));
      sum += x[e];
    }
    l += sum;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 4; s++) {
      f32x8 w;
#pragma unroll
      for (int e = 0; e < 8; e++) w[e] = x[s * 8 + e];
      const v8 wt = __builtin_convertvector(w, v8);
#pragma unroll
      for (int d = 0; d < DT; d++) {
        s16x4 v[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
          const int key = s * 16 + t * 8 + half * 4 + (lane & 15) / 4;
          const int at = d * 32 + (lane & 16) + (lane & 3) * 4;  // dim
          v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4)(s_v[buf] + v_place<D>(key, at / 8) + (at & 4) * 2));
        }
        const v8 vt = __builtin_bit_cast(v8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        o[d] = T::mfma32(vt, wt, o[d]);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    buf ^= 1;
    lds_arrived();
    __syncthreads();
  }
  l += __shfl_xor(l, 32);
  bool nan = false;
#pragma unroll
  for (int d = 0; d < DT; d++)
#pragma unroll
    for (int e = 0; e < 16; e++) nan |= o[d][e] != o[d][e];
  uint64_t again = __ballot(nan && live && l == l);
  again = (again | again >> 32) & 0xffffffffu;
  const bool mine = live && !((again >> col) & 1);
  const float log2_max = m == -INFINITY ? -INFINITY : m * c;  // of the weights, in the joining kernel's unit
  float* part_o = a.work + it.index * partial_floats<D>(R);
  float* part_ml = part_o + R * D;
  elem* op = reinterpret_cast<elem*>(a.out) + row * a.out_stride[0] + h * a.out_stride[1];
  if (mine) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int dim = d * 32 + e * 8 + half * 4;
        f32x4 y = {o[d][e * 4], o[d][e * 4 + 1], o[d][e * 4 + 2], o[d][e * 4 + 3]};
        if (it.splits > 1) {
          *reinterpret_cast<f32x4*>(part_o + rr * D + dim) = y;
        } else {
          typedef elem e4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<e4*>(op + dim) = __builtin_convertvector(y * inv, e4);
        }
      }
    if (half == 0) {
      if (it.splits > 1) {
        part_ml[rr * 2] = log2_max;
        part_ml[rr * 2 + 1] = l;
      } else if (a.lse) {
        a.lse[row * a.q_heads + h] = l == 0.f ? -INFINITY : (log2_max + log2f(l)) * kLn2;
      }
    }
  }
  // rows that came out NaN, one after the other (a wave's own LDS: the tiles are done with)
  float* s_q = reinterpret_cast<float*>(s_k[0]) + wave * D;
  while (again) {
    const int w = __builtin_ctzll(again);
    again &= again - 1;
    const int64_t ra = t0 + wave * 32 + w;
    const int ta = (int)(ra / a.group), ha = it.hk * a.group + (int)(ra - (int64_t)ta * a.group);
    float oo[D / 64], mm, ll;
    exact_row<T, D, D>(a, it.s, it.q.q0 + ta, ha, before + ta, span, i0, i1, s_q, oo, &mm, &ll);
    elem* oa = reinterpret_cast<elem*>(a.out) + (it.q.q0 + ta) * a.out_stride[0] + ha * a.out_stride[1];
    for (int x = 0; x < D / 64; x++) {
      if (it.splits > 1) part_o[(wave * 32 + w) * D + x * 64 + lane] = oo[x];
      else oa[x * 64 + lane] = (elem)(ll == 0.f ? 0.f : oo[x] / ll);
    }
    if (lane == 0) {
      if (it.splits > 1) {
        part_ml[(wave * 32 + w) * 2] = mm;
        part_ml[(wave * 32 + w) * 2 + 1] = ll;
      } else if (a.lse) {
        a.lse[(it.q.q0 + ta) * a.q_heads + ha] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      }
    }
  }
}

// ---------------------------------------------------------------- a latent cache: one row is key and value
// 576 dims of a key against every head of a token, 512 of them its value, so a tile of 64 keys (72 KiB,
// two of them in LDS) is read into LDS once for both products, and its four waves cut the work
// without doing any twice: scores by keys, values by dims, 128 a wave.  The maxima of the waves' keys
// and then the weights go through LDS: three barriers a tile.  Measured: 32 sequences up to 6000 tokens and 16 heads
// 32 us and 5 us to join; a chunk of 512 behind 3988 with 32 heads 190 to 193 us = 784 to 796 TFLOP/s.
constexpr int kLatKeys = 64;
constexpr int kLatDim = 576;
constexpr int kLatValue = 512;
constexpr int kLatBytes = kLatDim * 2;
constexpr int kLatTile = kLatKeys * kLatBytes;

// A tile lies in LDS in nine blocks of 64 dims: [dims / 64][key][128 bytes], so that one instruction
// brings 8 keys' 128 bytes and a lane's nine of a key differ by constants.  Inside the 128 bytes 16-byte
// chunk x lies at place x ^ lat_swizzle(key), which spreads both 16 keys' same chunk and the four
// keys by 64 bytes of a transposing read over all banks.
constexpr int kLatBlock = kLatKeys * 128;
__device__ __forceinline__ int lat_swizzle(int key) { return ((key >> 1) & 1) << 2 | ((key >> 2) & 3); }

// What both latent kernels share: their item's place in the sequence, and the tiles on their way.
struct Latent {
  Item it;
  int64_t t0;     // the row tile's first row
  int rows;       // rows of it
  int before, p_first, p_last;
  Span span;
  int i0, i1;     // this split's part of the span
  // row x of the tile (past the end: its first): token and head
  __device__ __forceinline__ int token(const AttendArgs& a, int x) const {
    return (int)((t0 + (x < rows ? x : 0)) / a.group);
  }
  __device__ __forceinline__ int head(const AttendArgs& a, int x, int tok) const {
    return (int)(t0 + (x < rows ? x : 0) - (int64_t)tok * a.group);
  }
  __device__ __forceinline__ Entry entry(const AttendArgs& a, int base) const {  // of key `lane` of a tile
    const int i = base + (threadIdx.x & 63);
    Entry e = {0, -1, 0};
    if (i < i1) e = entry_of(a, it.s, (uint32_t)span.key(i));
    return e;
  }
  __device__ __forceinline__ bool whole(const AttendArgs& a, int base, uint64_t there) const {
    return there == ~0ull && (!a.causal || (span.key(base + kLatKeys - 1) <= p_first &&
                                            (a.window == 0 || p_last - span.key(base) < a.window)));
  }
};

template <int R, bool SPLIT_FIRST>
__device__ __forceinline__ bool latent_item(const AttendArgs& a, int64_t* s_plan, Latent* t) {
  if (!find_item<(R <= 32), SPLIT_FIRST>(a, R, s_plan, parts_of<kLatValue, R>(a), &t->it)) return false;
  const Seq& q = t->it.q;
  const int64_t rows_all = (int64_t)q.m * a.group;
  t->t0 = (int64_t)t->it.tile * R;
  t->rows = rows_all - t->t0 < R ? (int)(rows_all - t->t0) : R;
  t->before = q.kv - q.m;
  t->p_first = t->before + (int)(t->t0 / a.group);
  t->p_last = t->before + (int)((t->t0 + t->rows - 1) / a.group);
  t->span = span_of(a, q.kv, t->p_first, t->p_last);
  const int n = t->span.n, splits = t->it.splits;
  const int part = ((n + splits - 1) / splits + kLatKeys - 1) / kLatKeys * kLatKeys;
  t->i0 = (int64_t)t->it.split * part < n ? t->it.split * part : n;
  t->i1 = t->i0 + part < n ? t->i0 + part : n;
  return true;
}

// 16 bytes a lane from memory into LDS, lane i to lds + 16 i (lds the same in all lanes), past the
// registers, from OFFSET bytes on in memory (the instruction adds its offset to both addresses).
template <int OFFSET>
__device__ __forceinline__ void lds_load_at(const uint8_t* from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2" ::"s"(lds), "v"(from),
               "n"(OFFSET)
               : "memory", "m0");
}
template <int... B>
__device__ __forceinline__ void latent_load_key(const uint8_t* from, uint32_t lds, std::integer_sequence<int, B...>) {
  (lds_load_at<B * 128>(from, lds + B * (kLatBlock - 128)), ...);
}
// A tile of keys into LDS, 16 of them a wave; slot: of key `lane`.
__device__ __forceinline__ void latent_load(const AttendArgs& a, uint32_t slot, const uint8_t* to) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int x = 0; x < 2; x++) {
    const int key = wave * 16 + x * 8 + lane / 8;
    const uint32_t sl = __shfl(slot, key);
    latent_load_key(a.k_rows + (uint64_t)(sl == kNoSlot ? 0 : sl) * kLatBytes + ((lane & 7) ^ lat_swizzle(key)) * 16,
                    lds_offset(to) + (wave * 16 + x * 8) * 128, std::make_integer_sequence<int, kLatBytes / 128>());
  }
}

// What was fetched in place of no key must not reach the product.
__device__ __forceinline__ void latent_clear(uint64_t there, uint8_t* tile) {
  for (int x = threadIdx.x; x < kLatTile / 16; x += 256)
    if (!((there >> (x % (kLatBlock / 16) / 8)) & 1)) *reinterpret_cast<v4u*>(tile + x * 16) = v4u{0, 0, 0, 0};
  __syncthreads();
}

// Rows that came out NaN, but for those whose sum of weights is NaN, shared out over the waves; s_sum: four parts of
// R rows' sums, s_q: kLatDim floats of this wave's.
template <class T>
__device__ __forceinline__ void latent_again(const AttendArgs& a, const Latent& t, const uint32_t* s_nan,
                                             const float* s_sum, int R, float* s_q, float* part_o, float* part_ml) {
  typedef typename T::elem elem;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int x = wave; x < t.rows; x += 4) {
    if (!((s_nan[x >> 5] >> (x & 31)) & 1)) continue;
    const float sum = s_sum[x] + s_sum[R + x] + s_sum[2 * R + x] + s_sum[3 * R + x];
    if (sum != sum) continue;
    const int tok = t.token(a, x), h = t.head(a, x, tok);
    const int64_t row = t.it.q.q0 + tok;
    float o[kLatValue / 64], m, l;
    exact_row<T, kLatDim, kLatValue>(a, t.it.s, row, h, t.before + tok, t.span, t.i0, t.i1, s_q, o, &m, &l);
    elem* op = reinterpret_cast<elem*>(a.out) + row * a.out_stride[0] + h * a.out_stride[1];
    for (int d = 0; d < kLatValue / 64; d++) {
      if (t.it.splits > 1) part_o[x * kLatValue + d * 64 + lane] = o[d];
      else op[d * 64 + lane] = (elem)(l == 0.f ? 0.f : o[d] / l);
    }
    if (lane == 0) {
      if (t.it.splits > 1) {
        part_ml[x * 2] = m;
        part_ml[x * 2 + 1] = l;
      } else if (a.lse) {
        a.lse[row * a.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
  }
}

// Writes four dims of a row, of the result or of a split's part of it.
template <class T>
__device__ __forceinline__ void latent_store(const AttendArgs& a, const Latent& t, float* part_o, int x, int64_t row,
                                             int h, int dim, f32x4 y, float inv) {
  typedef typename T::elem elem;
  typedef elem e4 __attribute__((ext_vector_type(4)));
  if (t.it.splits > 1)
    *reinterpret_cast<f32x4*>(part_o + x * kLatValue + dim) = y;
  else
    *reinterpret_cast<e4*>(reinterpret_cast<elem*>(a.out) + row * a.out_stride[0] + h * a.out_stride[1] + dim) =
        __builtin_convertvector(y * inv, e4);
}

// Up to 16 or 32 rows (RB of 16): decoding.  Bound by memory: 2 * 1088 operations a row on the 1152 bytes of a
// key.  Scores in 16 x 16 products, wave w taking keys 16 w of the tile against all rows.
template <class T, int RB, bool SPLIT_FIRST>
__global__ __launch_bounds__(256, 1) void k_attend_latent_few(AttendArgs a) {
  typedef typename T::v8 v8;
  constexpr int R = 16 * RB;
  constexpr int KS = kLatDim / 32;
  constexpr int DT = 8;  // 16-dim tiles of a wave
  __shared__ __align__(16) uint8_t s_k[2 * kLatTile];
  __shared__ __align__(16) uint8_t s_p[R * kLatKeys * 2];
  __shared__ float s_max[4][R], s_sum[4][R];
  __shared__ uint32_t s_nan[1];
  __shared__ int64_t s_plan[8];
  Latent t;
  if (!latent_item<R, SPLIT_FIRST>(a, s_plan, &t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const float c = weight_scale(a);
  v8 q[RB][KS];
  int p[RB];
#pragma unroll
  for (int b = 0; b < RB; b++) {
    const int x = b * 16 + col, tok = t.token(a, x), h = t.head(a, x, tok);
    p[b] = t.before + tok;
    const v4u* qp = reinterpret_cast<const v4u*>(a.q + 2 * ((t.it.q.q0 + tok) * a.q_stride[0] + h * a.q_stride[1]));
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < KS; i++) {
      const v4u y = qp[i * 4 + quad] ^ flip;
      q[b][i] = __builtin_bit_cast(v8, x < t.rows ? y : v4u{0, 0, 0, 0});
    }
  }
  // chunk 4 i + quad of key 16 wave + col: the swizzle changes its lowest three bits, two cases of i
  const int key = wave * 16 + col;
  int k_at[2];
  for (int i = 0; i < 2; i++) k_at[i] = key * 128 + ((i * 4 + quad) ^ lat_swizzle(key)) * 16;
  // dims 128 wave + 16 d of keys 32 s + 16 t + 4 quad + (lane & 15) / 4: four cases of d
  const int vkey = quad * 4 + (lane & 15) / 4;
  int v_at[4];
  for (int d = 0; d < 4; d++)
    v_at[d] = wave * 2 * kLatBlock + vkey * 128 + ((d * 2 + ((lane & 3) >> 1)) ^ lat_swizzle(vkey)) * 16 + (lane & 1) * 8;
  f32x4 o[RB][DT] = {};
  float m[RB], l[RB];
  for (int b = 0; b < RB; b++) m[b] = -INFINITY, l[b] = 0.f;
  Entry next_entry = t.entry(a, t.i0 + kLatKeys);
  uint32_t slot = slot_from(a, t.entry(a, t.i0));
  if (t.i0 < t.i1) latent_load(a, slot, s_k);
  lds_arrived();
  if (threadIdx.x == 0) s_nan[0] = 0;
  __syncthreads();
  int off = 0;
  f32x4 st[RB];   // scores of a tile, hidden ones -infinity
  float top[RB];  // its maxima
  // The scores of the tile at LDS `off`, while the next tile is loaded.
  auto score = [&](int base) {
    const uint64_t there = __ballot(slot != kNoSlot);
    slot = slot_from(a, next_entry);
    next_entry = t.entry(a, base + 2 * kLatKeys);
    if (base + kLatKeys < t.i1) latent_load(a, slot, s_k + (kLatTile - off));
    if (there != ~0ull) latent_clear(there, s_k + off);
#pragma unroll
    for (int b = 0; b < RB; b++) st[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KS; i++) {
      const v8 k = *reinterpret_cast<const v8*>(s_k + off + k_at[i & 1] + (i >> 1) * kLatBlock);
#pragma unroll
      for (int b = 0; b < RB; b++) st[b] = T::mfma16(k, q[b][i], st[b]);
    }
    const bool whole = t.whole(a, base, there);
#pragma unroll
    for (int b = 0; b < RB; b++) {
      float x[4] = {st[b][0], st[b][1], st[b][2], st[b][3]};
      if (!whole) {
        const uint32_t see = (uint32_t)(sees(a, t.span, there, p[b], base) >> (wave * 16)) >> (quad * 4);
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = (see >> e) & 1 ? x[e] : -INFINITY;
      }
      float y = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      y = fmaxf(y, __shfl_xor(y, 16));
      y = fmaxf(y, __shfl_xor(y, 32));
      if (quad == 0) s_max[wave][b * 16 + col] = y;
      st[b] = f32x4{x[0], x[1], x[2], x[3]};
    }
    __syncthreads();
    bool grows = false;
#pragma unroll
    for (int b = 0; b < RB; b++) {
      const int x = b * 16 + col;
      top[b] = fmaxf(fmaxf(s_max[0][x], s_max[1][x]), fmaxf(s_max[2][x], s_max[3][x]));
      grows |= (top[b] - m[b]) * c > kGrow || (m[b] == -INFINITY && top[b] != -INFINITY);
    }
    return __any(grows) != 0;  // the same rows and numbers in every wave, so all decide alike
  };
  // The sums are scaled outside the loop over tiles: a product's sums that other instructions touch
  // inside a loop are moved between the two register files in every round of it.
  int base = t.i0;
  if (base < t.i1) score(base);
  while (base < t.i1) {
#pragma unroll
    for (int b = 0; b < RB; b++) {
      const float next = fmaxf(m[b], top[b]);
      const float keep = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m[b] - next) * c);
      m[b] = next;
      l[b] *= keep;
#pragma unroll
      for (int d = 0; d < DT; d++) o[b][d] *= keep;
    }
    bool grows = false;
    do {
#pragma unroll
      for (int b = 0; b < RB; b++) {
        const int x = b * 16 + col;
        const float zero = m[b] == -INFINITY ? 0.f : m[b] * c;
        f32x4 w;
#pragma unroll
        for (int e = 0; e < 4; e++) w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(st[b][e], c, -zero));
        l[b] += w[0] + w[1] + w[2] + w[3];
        typedef typename T::elem e4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<e4*>(s_p + x * kLatKeys * 2 + (((wave >> 1) * 4 + quad) ^ (x & 7)) * 16 + (wave & 1) * 8) =
            __builtin_convertvector(w, e4);
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; s++) {
        v8 w[RB];
#pragma unroll
        for (int b = 0; b < RB; b++) {
          const int x = b * 16 + col;
          w[b] = *reinterpret_cast<const v8*>(s_p + x * kLatKeys * 2 + ((s * 4 + quad) ^ (x & 7)) * 16);
        }
#pragma unroll
        for (int d = 0; d < DT; d++) {
          s16x4 v[2];
#pragma unroll
          for (int u = 0; u < 2; u++)
            v[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4)(s_k + off + v_at[d & 3] + (d >> 2) * kLatBlock + (s * 32 + u * 16) * 128));
          const v8 vt = __builtin_bit_cast(v8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
          for (int b = 0; b < RB; b++) o[b][d] = T::mfma16(vt, w[b], o[b][d]);
        }
      }
      off = kLatTile - off;
      lds_arrived();
      __syncthreads();
      base += kLatKeys;
      if (base >= t.i1) break;
      grows = score(base);
    } while (!grows);
  }
#pragma unroll
  for (int b = 0; b < RB; b++) {
    l[b] += __shfl_xor(l[b], 16);
    l[b] += __shfl_xor(l[b], 32);
    if (quad == 0) s_sum[wave][b * 16 + col] = l[b];
    bool nan = false;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int e = 0; e < 4; e++) nan |= o[b][d][e] != o[b][d][e];
    uint64_t bits = __ballot(nan);
    bits |= bits >> 32;
    bits |= bits >> 16;
    if (lane == 0 && (bits & 0xffff)) atomicOr(s_nan, (uint32_t)(bits & 0xffff) << (b * 16));
  }
  __syncthreads();
  float* part_o = a.work + t.it.index * partial_floats<kLatValue>(R);
  float* part_ml = part_o + R * kLatValue;
#pragma unroll
  for (int b = 0; b < RB; b++) {
    const int x = b * 16 + col;
    const float sum = s_sum[0][x] + s_sum[1][x] + s_sum[2][x] + s_sum[3][x];
    if (x >= t.rows || (((s_nan[0] >> x) & 1) && sum == sum)) continue;
    const int tok = t.token(a, x), h = t.head(a, x, tok);
    const int64_t row = t.it.q.q0 + tok;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int d = 0; d < DT; d++) latent_store<T>(a, t, part_o, x, row, h, wave * 128 + d * 16 + quad * 4, o[b][d], inv);
    if (wave == 0 && quad == 0) {
      const float log2_max = m[b] == -INFINITY ? -INFINITY : m[b] * c;
      if (t.it.splits > 1) {
        part_ml[x * 2] = log2_max;
        part_ml[x * 2 + 1] = sum;
      } else if (a.lse) {
        a.lse[row * a.q_heads + h] = sum == 0.f ? -INFINITY : (log2_max + log2f(sum)) * kLn2;
      }
    }
  }
  latent_again<T>(a, t, s_nan, &s_sum[0][0], R, reinterpret_cast<float*>(s_k) + wave * kLatDim, part_o, part_ml);
}

// 64 rows: chunks, and many heads.  Bound by the matrix cores and LDS: 240 KiB are read from it for 2176
// cycles of products.  Scores in 32 x 32 products, wave (i, j) taking rows 32 i, whose queries stay in
// registers, and keys 32 j.
constexpr int kLatRows = 64;

template <class T, bool SPLIT_FIRST>
__global__ __launch_bounds__(256, 1) void k_attend_latent(AttendArgs a) {
  typedef typename T::v8 v8;
  constexpr int KS = kLatDim / 16;
  constexpr int DT = 4;  // 32-dim tiles of a wave
  __shared__ __align__(16) uint8_t s_k[2 * kLatTile];
  __shared__ __align__(16) uint8_t s_p[kLatRows * kLatKeys * 2];
  __shared__ float s_max[2][kLatRows], s_sum[4][kLatRows];
  __shared__ uint32_t s_nan[2];
  __shared__ int64_t s_plan[8];
  Latent t;
  if (!latent_item<kLatRows, SPLIT_FIRST>(a, s_plan, &t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int wi = wave >> 1, wj = wave & 1;
  const int rr = wi * 32 + col;  // this lane's row of the scores
  const int tok = t.token(a, rr), p = t.before + tok;
  const float c = weight_scale(a);
  v8 q[KS];
  {
    const v4u* qp = reinterpret_cast<const v4u*>(
        a.q + 2 * ((t.it.q.q0 + tok) * a.q_stride[0] + t.head(a, rr, tok) * a.q_stride[1]));
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < KS; i++) {
      const v4u x = qp[i * 2 + half] ^ flip;
      q[i] = __builtin_bit_cast(v8, rr < t.rows ? x : v4u{0, 0, 0, 0});
    }
  }
  // chunk 2 i + half of key 32 j + col: the swizzle changes its lowest three bits, four cases of i
  const int key = wj * 32 + col;
  int k_at[4];
  for (int i = 0; i < 4; i++) k_at[i] = key * 128 + ((i * 2 + half) ^ lat_swizzle(key)) * 16;
  // dims 128 wave + 32 d of keys 16 s + 8 u + 4 half + (lane & 15) / 4: two cases of d, two of u
  int v_at[2][2];
  for (int d = 0; d < 2; d++)
    for (int u = 0; u < 2; u++) {
      const int k = u * 8 + half * 4 + (lane & 15) / 4;
      v_at[d][u] = wave * 2 * kLatBlock + k * 128 + ((d * 4 + (lane & 16) / 8 + (lane & 3) / 2) ^ lat_swizzle(k)) * 16 +
                   (lane & 1) * 8;
    }
  auto p_place = [&](int row, int chunk) { return row * kLatKeys * 2 + (chunk ^ (row & 7)) * 16; };
  f32x16 o[2][DT] = {};
  float m[2] = {-INFINITY, -INFINITY}, l = 0.f;  // maxima of rows col and 32 + col; this lane's part of row rr's sum
  Entry next_entry = t.entry(a, t.i0 + kLatKeys);
  uint32_t slot = slot_from(a, t.entry(a, t.i0));
  if (t.i0 < t.i1) latent_load(a, slot, s_k);
  lds_arrived();
  if (threadIdx.x < 2) s_nan[threadIdx.x] = 0;
  __syncthreads();
  int off = 0;
  float x[16], top[2];  // scores of a tile, hidden ones -infinity, and its maxima
  auto score = [&](int base) {
    const uint64_t there = __ballot(slot != kNoSlot);
    slot = slot_from(a, next_entry);
    next_entry = t.entry(a, base + 2 * kLatKeys);
    if (base + kLatKeys < t.i1) latent_load(a, slot, s_k + (kLatTile - off));
    if (there != ~0ull) latent_clear(there, s_k + off);
    // groups of operands, the next on its way while one is multiplied; left to itself the compiler
    // fetches all 36 first and runs out of registers
    constexpr int G = 4;
    f32x16 st = {};
    v8 k[2][G];
#pragma unroll
    for (int i = 0; i < G; i++) k[0][i] = *reinterpret_cast<const v8*>(s_k + off + k_at[i & 3]);
#pragma unroll
    for (int g = 0; g < KS / G; g++) {
      if (g + 1 < KS / G) {
#pragma unroll
        for (int i = 0; i < G; i++)
          k[(g + 1) & 1][i] = *reinterpret_cast<const v8*>(s_k + off + k_at[i & 3] + (g + 1) * kLatBlock);
      }
#pragma unroll
      for (int i = 0; i < G; i++) st = T::mfma32(k[g & 1][i], q[g * G + i], st);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int e = 0; e < 16; e++) x[e] = st[e];
    if (!t.whole(a, base, there)) {
      const uint32_t see = (uint32_t)(sees(a, t.span, there, p, base) >> (wj * 32)) >> (half * 4);
#pragma unroll
      for (int e = 0; e < 16; e++) x[e] = (see >> (e / 4 * 8 + e % 4)) & 1 ? x[e] : -INFINITY;
    }
    float y = x[0];
#pragma unroll
    for (int e = 1; e < 16; e++) y = fmaxf(y, x[e]);
    y = fmaxf(y, __shfl_xor(y, 32));
    if (half == 0) s_max[wj][rr] = y;
    __syncthreads();
    bool grows = false;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      top[i] = fmaxf(s_max[0][i * 32 + col], s_max[1][i * 32 + col]);
      grows |= (top[i] - m[i]) * c > kGrow || (m[i] == -INFINITY && top[i] != -INFINITY);
    }
    return __any(grows) != 0;  // the same rows and numbers in every wave, so all decide alike
  };
  int base = t.i0;
  if (base < t.i1) score(base);
  while (base < t.i1) {  // the sums are scaled outside the loop over tiles, as above
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const float next = fmaxf(m[i], top[i]);
      const float keep = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m[i] - next) * c);
      m[i] = next;
      l *= wi == i ? keep : 1.f;
#pragma unroll
      for (int d = 0; d < DT; d++) o[i][d] *= keep;
    }
    bool grows = false;
    do {
      const float mine = wi ? m[1] : m[0];
      const float zero = mine == -INFINITY ? 0.f : mine * c;
      float sum = 0.f;
#pragma unroll
      for (int s = 0; s < 2; s++) {
        f32x8 w;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[s * 8 + e], c, -zero));
          sum += w[e];
        }
        *reinterpret_cast<v8*>(s_p + p_place(rr, (wj * 2 + s) * 2 + half)) = __builtin_convertvector(w, v8);
      }
      l += sum;
      __syncthreads();
      // values and weights a step ahead as well (201 us for a chunk of 512 behind 3988, else 210)
      v8 vf[2][DT], w[2][2];
      auto fetch = [&](int s, int h) {
        w[h][0] = *reinterpret_cast<const v8*>(s_p + p_place(col, s * 2 + half));
        w[h][1] = *reinterpret_cast<const v8*>(s_p + p_place(32 + col, s * 2 + half));
#pragma unroll
        for (int d = 0; d < DT; d++) {
          s16x4 v[2];
#pragma unroll
          for (int u = 0; u < 2; u++)
            v[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4)(s_k + off + v_at[d & 1][u] + (d >> 1) * kLatBlock + s * 16 * 128));
          vf[h][d] = __builtin_bit_cast(v8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        }
      };
      fetch(0, 0);
#pragma unroll
      for (int s = 0; s < 4; s++) {
        if (s < 3) fetch(s + 1, (s + 1) & 1);
#pragma unroll
        for (int d = 0; d < DT; d++) {
          o[0][d] = T::mfma32(vf[s & 1][d], w[s & 1][0], o[0][d]);
          o[1][d] = T::mfma32(vf[s & 1][d], w[s & 1][1], o[1][d]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      off = kLatTile - off;
      lds_arrived();
      __syncthreads();
      base += kLatKeys;
      if (base >= t.i1) break;
      grows = score(base);
    } while (!grows);
  }
  // sums of a row: two key halves times two lane halves
  s_sum[wj * 2 + half][rr] = l;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    bool nan = false;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int e = 0; e < 16; e++) nan |= o[i][d][e] != o[i][d][e];
    const uint64_t b = __ballot(nan);
    if (lane == 0 && b) atomicOr(&s_nan[i], (uint32_t)(b | b >> 32));
  }
  __syncthreads();
  float* part_o = a.work + t.it.index * partial_floats<kLatValue>(kLatRows);
  float* part_ml = part_o + kLatRows * kLatValue;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int x = i * 32 + col;
    const float sum = s_sum[0][x] + s_sum[1][x] + s_sum[2][x] + s_sum[3][x];
    if (x >= t.rows || (((s_nan[i] >> col) & 1) && sum == sum)) continue;
    const int tx = t.token(a, x), hx = t.head(a, x, tx);
    const int64_t row = t.it.q.q0 + tx;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int e = 0; e < 4; e++)
        latent_store<T>(a, t, part_o, x, row, hx, wave * 128 + d * 32 + e * 8 + half * 4,
                        f32x4{o[i][d][e * 4], o[i][d][e * 4 + 1], o[i][d][e * 4 + 2], o[i][d][e * 4 + 3]}, inv);
    if (wave == 0 && half == 0) {
      const float log2_max = m[i] == -INFINITY ? -INFINITY : m[i] * c;
      if (t.it.splits > 1) {
        part_ml[x * 2] = log2_max;
        part_ml[x * 2 + 1] = sum;
      } else if (a.lse) {
        a.lse[row * a.q_heads + hx] = sum == 0.f ? -INFINITY : (log2_max + log2f(sum)) * kLn2;
      }
    }
  }
  latent_again<T>(a, t, s_nan, &s_sum[0][0], kLatRows, reinterpret_cast<float*>(s_k) + wave * kLatDim, part_o, part_ml);
}

// Joins the splits of a row tile, a wave a row.  A workgroup looks at the item of one place; all but the first
// split of a tile that was split have nothing to do.
template <class T, int DV, int R>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a) {
  typedef typename T::elem elem;
  const int64_t first = blockIdx.x / a.join_parts;
  const Part p = parts_of<DV, R>(a)[first];
  // a q_start that goes back (reported) can make more items than the call has room for
  if (p.splits <= 1 || first + p.splits > a.slots) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tile = p.tile_hk / a.kv_heads;
  const int hk = (int)(p.tile_hk - tile * a.kv_heads);
  const int rr = (int)(blockIdx.x % a.join_parts) * 4 + wave;
  const int64_t r = tile * R + rr;
  if (rr >= R || r >= p.m * a.group) return;
  constexpr int ND = DV / 64;
  float m = -INFINITY, l = 0.f, o[ND] = {};
#pragma unroll 4
  for (int k = 0; k < (int)p.splits; k++) {
    const float* po = a.work + (first + k) * partial_floats<DV>(R);
    const float pm = po[R * DV + rr * 2], pl = po[R * DV + rr * 2 + 1];
    float v[ND];
#pragma unroll
    for (int c = 0; c < ND; c++) v[c] = po[rr * DV + c * 64 + lane];
    const float next = fmaxf(m, pm);
    const float zero = next == -INFINITY ? 0.f : next;
    const float keep = __builtin_amdgcn_exp2f(m - zero), add = __builtin_amdgcn_exp2f(pm - zero);
    m = next;
    l = l * keep + pl * add;
#pragma unroll
    for (int c = 0; c < ND; c++) o[c] = o[c] * keep + v[c] * add;
  }
  const int64_t rt = r / a.group;
  const int h = hk * a.group + (int)(r - rt * a.group);
  elem* op = reinterpret_cast<elem*>(a.out) + (p.q0 + rt) * a.out_stride[0] + h * a.out_stride[1];
#pragma unroll
  for (int c = 0; c < ND; c++) op[c * 64 + lane] = (elem)(l == 0.f ? 0.f : o[c] / l);
  if (a.lse && lane == 0) a.lse[(p.q0 + rt) * a.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Row tiles of R rows that a call can have at most: each sequence rounds up once.
int64_t most_tiles(const AttendArgs& a, int R) {
  return a.q_rows * a.group / R + (a.num_seqs < a.q_rows ? a.num_seqs : a.q_rows);
}

// The kernel for a call: the rows of its row tiles.  64 sequences up to 8192 tokens, 32/8 heads of 128, with several
// new tokens each, in tiles of 16 and of 128 rows: 17 to 32 rows of a KV head 298 and 273 us, 48 rows 370 and
// 278, 64 rows 482 and 285 (16 rows fit one tile, 230); 16/4 heads of 64: 32 rows 88 and 70, 48 rows 102 and 71.
// So from 17 rows on tiles of 128 are ahead, and the border of 32 is a tenth to a fifth too slow for what is
// between.  32 sequences up to 6000 tokens of a latent cache, in tiles of 32 and of 64 rows: 20 rows 43.0 and 45.1 us, 32
// rows 46.0 and 45.3, 40 rows 62.9 and 48.0, 64 rows 70.0 and 52.1.
int tile_rows(const AttendArgs& a, int32_t head_dim) {
  const int64_t rows = a.max_q * a.group;
  if (head_dim == kLatDim) return rows <= 16 ? 16 : rows <= 32 ? 32 : kLatRows;
  return rows <= 2 * kRowTile ? kRowTile : kTileRows;
}

// How the list of items is made for a call of tiles of R rows, and the number of items at most: a split of
// C keys has at least `min_split` of them, and the whole call's keys over C is at most `target`.
//
// min_split: few rows, with 64, 128 and 256 keys at least: one sequence of 4000 21.4, 15.8 and 15.2 us, 16 of 600 27.9,
// 21.3 and 18.7, one of 1500 of a latent cache 18.8, 18.3 and 21.1.  Many rows, with 128, 256 and 512: a chunk of 64 behind
// 1436 22.8, 22.3 and 26.6, of 256 behind 1744 35.1, 34.9 and 33.5, of 32 of a latent cache behind 1468 35.5, 36.1 and 43.6.
//
// Calls of many rows are split when their row tiles, which the host knows, are fewer than the target, or when some of
// several sequences may be so long that their one tile each (a decoding row beside a chunk) would run on alone; else one
// launch does all.  The second rule, applied and not: a chunk of 4096 beside one row of 32768 keys 250 and 876 us, beside
// four of 65536 387 and 1668, a latent chunk of 512 beside one of 32768 71 and 1258; beside one of 16384 it would gain
// too (255 and 517).  Calls whose sequences keep the GPU busy anyway pay for it: a chunk of 4096 beside 63
// rows of 8192 686 and 670, of 32768 1772 and 1756, four fp16 prompts up to 4096 139 and 127; hence not for
// shorter ones.
//
// A latent cache's target leaves places to the tiles themselves.  With the whole GPU as its target: 32 sequences
// up to 6000 of 16 heads 52.4 us for 38.4, 16 sequences up to 16384 of 128 heads 129 for 90; but half the GPU, which
// it comes down to, is too little where tiles are many: a chunk of 255 tokens of 32 heads 118 for 194, and from 128 tiles
// on, where a call counts as filling that half and is not split, 64 sequences up to 16384 of 128 heads 358 for 705.
//
// Only split tiles have partial results.  A split tile of n > C keys has at most (n + C - 1) / C < 2 n / C
// splits, so that they are less than twice the target, however many row tiles the call has.  A call of more
// items than that has just those places, and takes the split tiles first; of another the list is left in the order
// of the sequences, which is found sooner (a sequence of 1500 12.0 us for 12.8, 64 up to 8192 207.3 for 208.1).
constexpr int64_t kLongKeys = 16384;
struct Plan {
  int64_t items, joins;  // joins: workgroups of the second launch, 0: no split can be
  bool few_places;       // fewer places of partial results than items
};
Plan plan(AttendArgs* a, int R, int32_t head_dim, int32_t num_cus) {
  const bool latent = head_dim == kLatDim, few = R <= 32;
  a->min_split = few ? 128 : 256;
  Plan p = {most_tiles(*a, R) * a->kv_heads, 0, false};
  // items that run at once: 8 or 2 workgroups a compute unit, and one of a latent cache, where the
  // whole list, `tiles` longer than the target at most, should be one round
  a->target = (int64_t)num_cus * (few ? 8 : 2);
  if (latent) a->target = num_cus - p.items > num_cus / 2 ? num_cus - p.items : num_cus / 2;
  a->join_parts = 0;
  a->slots = 0;
  const int64_t most_splits = (a->max_kv + a->min_split - 1) / a->min_split;
  const bool fills = a->q_rows * a->group / R * a->kv_heads >= a->target;
  if (most_splits > 1 && (few || !fills || (a->num_seqs > 1 && a->max_kv > kLongKeys))) {
    const int64_t rows = a->max_q * a->group < R ? a->max_q * a->group : R;  // of a tile at most
    a->join_parts = (int32_t)((rows + 3) / 4);
    p.items += most_splits - 1 <= a->target / p.items ? p.items * (most_splits - 1) : a->target;
    p.few_places = p.items > 2 * a->target;
    a->slots = p.few_places ? 2 * a->target : p.items;
    p.joins = a->slots * a->join_parts;
  } else {
    a->min_split = a->max_kv + 1;
  }
  return p;
}

// kernels: of calls whose items all have a place for a partial result, or that are not split, and of others.
template <class T, int DV, int R>
hipError_t launch_split(void (*const (&kernels)[2])(AttendArgs), AttendArgs a, int32_t num_cus, hipStream_t stream) {
  const Plan p = plan(&a, R, DV == kLatValue ? kLatDim : DV, num_cus);
  if (p.items > 0x7fffffff || p.joins > 0x7fffffff) return hipErrorInvalidValue;
  kernels[p.few_places]<<<dim3((unsigned)p.items), 256, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.joins == 0) return e;
  k_attend_join<T, DV, R><<<dim3((unsigned)p.joins), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <class T, int RB>
hipError_t launch_latent_few(const AttendArgs& a, int32_t num_cus, hipStream_t stream) {
  return launch_split<T, kLatValue, 16 * RB>({k_attend_latent_few<T, RB, false>, k_attend_latent_few<T, RB, true>}, a,
                                             num_cus, stream);
}
template <class T, int D>
hipError_t launch_decode(const AttendArgs& a, int32_t num_cus, hipStream_t stream) {
  return launch_split<T, D, kRowTile>({k_attend_decode<T, D, false>, k_attend_decode<T, D, true>}, a, num_cus, stream);
}
template <class T, int D>
hipError_t launch_tiles(const AttendArgs& a, int32_t num_cus, hipStream_t stream) {
  return launch_split<T, D, kTileRows>({k_attend_tiles<T, D, false>, k_attend_tiles<T, D, true>}, a, num_cus, stream);
}

template <class T>
hipError_t launch_for(const AttendArgs& a, int32_t head_dim, int32_t num_cus, hipStream_t stream) {
  (void)hipGetLastError();
  const int R = tile_rows(a, head_dim);
  if (head_dim == kLatDim)
    return R == 16   ? launch_latent_few<T, 1>(a, num_cus, stream)
           : R == 32 ? launch_latent_few<T, 2>(a, num_cus, stream)
                     : launch_split<T, kLatValue, kLatRows>({k_attend_latent<T, false>, k_attend_latent<T, true>}, a,
                                                            num_cus, stream);
  if (R == kRowTile)
    return head_dim == 64 ? launch_decode<T, 64>(a, num_cus, stream) : launch_decode<T, 128>(a, num_cus, stream);
  return head_dim == 64 ? launch_tiles<T, 64>(a, num_cus, stream) : launch_tiles<T, 128>(a, num_cus, stream);
}

}  // namespace

int64_t attend_workspace(const AttendArgs& args, int32_t head_dim, int32_t num_cus) {
  const int R = tile_rows(args, head_dim);
  if (args.q_rows <= 0 || args.num_seqs <= 0) return 0;
  AttendArgs a = args;
  const Plan p = plan(&a, R, head_dim, num_cus);
  if (p.joins == 0) return 0;
  const int64_t floats = head_dim == 64 ? partial_floats<64>(R) : head_dim == 128 ? partial_floats<128>(R)
                                                                                 : partial_floats<kLatValue>(R);
  return a.slots * (4 * floats + (int64_t)sizeof(Part));
}

hipError_t launch_attend(const AttendArgs& a, int32_t dtype, int32_t head_dim, int32_t num_cus, hipStream_t stream) {
  if (a.q_rows <= 0 || a.num_seqs <= 0) return hipSuccess;
  return dtype == HC_BF16 ? launch_for<Bf16>(a, head_dim, num_cus, stream) : launch_for<F16>(a, head_dim, num_cus, stream);
}

}  // namespace hc
