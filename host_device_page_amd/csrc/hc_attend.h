// What the attention kernels over caches of elements (hc_attend.hip) and of 4 bits (hc_attend_mxfp4.hip) share: a
// sequence's rows and keys, where tokens are, what a row sees, one row computed key by key, and the list of
// work items.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

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

constexpr uint32_t kNoSlot = (uint32_t)kMaxAttendSlots;  // pools of an attention call have fewer

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
// OFFSET: bytes on from there, in memory and in LDS (the instruction adds its offset to both addresses).
#pragma clang diagnostic ignored "-Winline-asm"
template <int OFFSET>
__device__ __forceinline__ void lds_load_at(const uint8_t* from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2" ::"s"(lds), "v"(from),
               "n"(OFFSET)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_load(const uint8_t* from, uint32_t lds) { lds_load_at<0>(from, lds); }
__device__ __forceinline__ void lds_arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}

// Keys and values of a token's KV head, of a cache of elements.  (A latent cache's values are in its key rows, one head.)
template <class T, int DK, int DV>
struct ElementRows {
  typedef typename T::elem elem;
  struct Key {
    const v4u* at;
    __device__ __forceinline__ Key(const AttendArgs& a, uint32_t slot, int hk)
        : at(reinterpret_cast<const v4u*>(a.k_rows + 2 * ((int64_t)slot * a.k_row + (int64_t)hk * DK))) {}
    __device__ __forceinline__ typename T::v8 eight(int v) const { return __builtin_bit_cast(typename T::v8, at[v]); }
  };
  struct Value {
    const elem* at;
    __device__ __forceinline__ Value(const AttendArgs& a, uint32_t slot, int hk)
        : at(reinterpret_cast<const elem*>(a.v_rows) + (int64_t)slot * a.v_row + (int64_t)hk * (DK == DV ? DV : 0)) {}
    __device__ __forceinline__ elem one(int d) const { return at[d]; }
  };
};

// ---------------------------------------------------------------- one row, key by key
// Softmax sums of one query row over positions [i0, i1) of its span, by one wave: lanes take keys
// for the scores and dims for the sum, and nothing of a key that the row does not see is touched.
// The tiled kernels multiply hidden keys' values by a weight of 0, which is NaN where the value is
// not finite; they do the rows that came out NaN again with this, unless the sum of weights is NaN too: then a score
// that the row sees is, and so is the row.  (One row costs as much as a hundred in tiles: 2048 rows behind 14336, all of
// NaN queries, took 160 ms, now 0.6.)  s_q: DK floats of this wave's.
template <class T, int DK, int DV, class Rows>
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
      const typename Rows::Key kp(a, slot, hk);
      x = 0.f;
#pragma unroll 1
      for (int v = 0; v < DK / 8; v++) {
        const f32x8 kv = __builtin_convertvector(kp.eight(v), f32x8);
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
      const typename Rows::Value vp(a, sj, hk);
#pragma unroll
      for (int c = 0; c < ND; c++) o[c] += pj * (float)vp.one(c * 64 + lane);
    }
  }
  *m_out = m;
  *l_out = l;
}

// In the kernels of many rows, of a latent cache and of 4-bit rows the maximum that a row's weights are relative to
// is replaced only when it grows by more than 2^8: until then weights of up to 2^8 are summed, which loses nothing
// in fp32 or as operands, and the sums need not be scaled.
constexpr float kGrow = 8.f;

// Rows of a row tile: of the kernels of few rows (decoding), of many, and of a latent cache's.
constexpr int kRowTile = 16;
constexpr int kTileRows = 128;
constexpr int kLatRows = 64;
constexpr int kLatDim = 576;
constexpr int kLatValue = 512;

// ---------------------------------------------------------------- the list of work items
// A sequence's query rows times the heads of a KV head's group make row lists of m * group rows,
// row r being token r / group and head r % group of the group; R rows make a row tile.  An item is
// (sequence, KV head, row tile, split): `splits` items share a tile's keys.  Every workgroup works
// out the list for itself from the lengths, so that its number of items follows the lengths as
// they are on the device: a sequence gets a split per C keys, C being the whole call's keys over
// the wanted number of items, but min_split at least, which the host knows: some keys, and over 4-bit rows a share of
// the call's max_kv, so that there a bound far above the lengths makes fewer items.
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


// ---------------------------------------------------------------- splits: how many, and their join
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
// Kernels with a rule of their own say the workgroups of a compute unit (per_cu) and the least keys of a split, and
// of how many KV heads an item is (heads; a->kv_heads then counts items of a tile).  Few tiles' list should be one round
// of workgroups, tiles included; of many, two rounds, since their tiles are of unlike lengths, but of a latent cache one,
// whose partial results are long.  (4-bit rows.  64 sequences up to 8192, few tiles: a target of the whole round
// 100 us, less the tiles 82; up to half a round of tiles for a quarter: 128 up to 2048 54 for 56.  Many, in one round and in
// two: 256 up to 8192 317 and 285, 512 up to 2000 198 and 168, all of 1000 148 and 157; of a latent cache 512 of 500
// 46 and 76, 128 up to 6000 68 and 76, 256 117 and 117.)
Plan plan(AttendArgs* a, int R, int32_t head_dim, int32_t num_cus, int heads = 0, int per_cu = 0, int least = 0) {
  const bool latent = head_dim == kLatDim, few = R <= 32;
  a->min_split = least ? least : few ? 128 : 256;
  Plan p = {most_tiles(*a, R) * a->kv_heads, 0, false};
  // items that run at once: 8 or 2 workgroups a compute unit, and one of a latent cache, where the
  // whole list, `tiles` longer than the target at most, should be one round
  a->target = (int64_t)num_cus * (per_cu ? per_cu : few ? 8 : 2);
  if (per_cu) a->target = 2 * p.items <= a->target ? a->target - p.items : latent ? a->target : 2 * a->target;
  if (latent && !per_cu) a->target = num_cus - p.items > num_cus / 2 ? num_cus - p.items : num_cus / 2;
  a->join_parts = 0;
  a->slots = 0;
  const int64_t most_splits = (a->max_kv + a->min_split - 1) / a->min_split;
  const bool fills = a->q_rows * a->group / R * a->kv_heads >= a->target;
  // (a call whose sequences have no rows has no tile to split, however many rows the tensor has)
  if (most_splits > 1 && a->max_q > 0 && (few || !fills || (a->num_seqs > 1 && a->max_kv > kLongKeys))) {
    const int64_t rows = a->max_q * a->group < R ? a->max_q * a->group : R;  // of a tile at most
    a->join_parts = (int32_t)(heads ? rows * heads : (rows + 3) / 4);
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
typedef void (*AttendKernel)(AttendArgs);
hipError_t launch_planned(const AttendKernel (&kernels)[2], AttendKernel join, const AttendArgs& a, const Plan& p,
                          hipStream_t stream) {
  if (p.items > 0x7fffffff || p.joins > 0x7fffffff) return hipErrorInvalidValue;
  kernels[p.few_places]<<<dim3((unsigned)p.items), 256, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.joins == 0) return e;
  join<<<dim3((unsigned)p.joins), 256, 0, stream>>>(a);
  return hipGetLastError();
}
template <class T, int DV, int R>
hipError_t launch_split(const AttendKernel (&kernels)[2], AttendArgs a, int32_t num_cus, hipStream_t stream) {
  const Plan p = plan(&a, R, DV == kLatValue ? kLatDim : DV, num_cus);
  return launch_planned(kernels, k_attend_join<T, DV, R>, a, p, stream);
}

}  // namespace
}  // namespace hc
