// Attention over a cache held in 4 bits: the formulas and the list of work items are hc_attend.hip's, the
// rows hc_mxfp4.h's.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "hc_attend_latent.h"
#include "hc_attend_tiles.h"
#include "hc_mxfp4.h"

namespace hc {
namespace {

template <class T>
constexpr bool kIsBf16 = false;
template <>
constexpr bool kIsBf16<Bf16> = true;

// Keys and values of a token's KV head in 4 bits, rounded to T's elements.  HEADS: KV heads of an item.
template <class T, int DK, int DV, int HEADS = 1>
struct MxRows {
  struct Head {
    const uint8_t *codes, *scales;
    __device__ __forceinline__ Head(const uint8_t* row, int heads, int hk)
        : codes(row + hk * (DK / 2)), scales(row + mxfp4_codes((int64_t)heads * DK) + hk * (DK / kMxBlock)) {}
    __device__ __forceinline__ typename T::v8 eight(int v) const {
      return __builtin_bit_cast(typename T::v8, mx_decode<kIsBf16<T>>(reinterpret_cast<const uint32_t*>(codes)[v],
                                                                      mx_scale(scales[v / 4])));
    }
    __device__ __forceinline__ typename T::elem one(int d) const {
      return __builtin_bit_cast(typename T::v8, mx_decode<kIsBf16<T>>((uint32_t)codes[d / 2] >> (d & 1) * 4,
                                                                      mx_scale(scales[d / kMxBlock])))[0];
    }
  };
  struct Key : Head {
    __device__ __forceinline__ Key(const AttendArgs& a, uint32_t slot, int hk)
        : Head(a.k_rows + (int64_t)slot * a.k_row, a.kv_heads * HEADS, hk) {}
  };
  struct Value : Head {  // DK == DV, or a latent cache's only head
    __device__ __forceinline__ Value(const AttendArgs& a, uint32_t slot, int hk)
        : Head(a.v_rows + (int64_t)slot * a.v_row, a.kv_heads * HEADS, hk) {}
  };
};

// ---------------------------------------------------------------- few rows: decoding
// Rows and products are the decoding kernel's of the cache of elements, 16 (token, head) pairs of a KV head; what differs is
// how little is read, 68 bytes of a key's 128 dims, and that a row's heads lie next to each other in it.
//
// A workgroup takes up to four KV heads, and reads their part of a row in one piece, straight into LDS; from there
// every wave takes its own head's codes and scales into registers, and the next tile is on its way while they
// are computed.  Waves that share a head take 32 keys of a tile each and are joined at the end.  (Waves that load their
// head's 64 bytes themselves ask for each line of memory several times: 64 sequences up to 8192 tokens took 93 us so,
// and 130 with one head to a workgroup.)
//
// Measured: 64 sequences up to 8192 tokens, 32/8 heads of 128, 73 us and 7 us to join = 4.0 TB/s of rows; 256 of them
// 4.1; 32 sequences in a window of 4096 with 4 sinks, scattered slots, fp16 heads of 64, 26 and 6 us; one
// sequence of 1500 13 us.  Four workgroups a compute unit (128 registers a lane) for three: 82 us for 85 on the first.
//
//   K  the order of the dims inside a product is free, so a lane takes D / 4 dims of a key next to each other,
//      one read and one scale, and the queries the same.
//   V  a block of 32 dims of a key and its scale a lane, 64 dims at a time through LDS as elements and back
//      transposed.
constexpr int kFewKeys = 32;  // of a wave and tile

// Where the 16-byte chunk of a key's 64 dims of V lies; written and read without conflicts.
__device__ __forceinline__ int few_place(int key, int chunk) {
  const int x = ((key >> 1) & 1) << 2 | ((key >> 2) & 1) << 1 | ((key >> 3) & 1);
  return key * 128 + (chunk ^ x) * 16;
}

// A tile of rows in LDS: CPR chunks of codes a key, in places that 16 keys' same chunk does not share, and
// S4 dwords of scales.
template <int D, int HEADS>
struct FewStage {
  static constexpr int W = 4;  // waves
  static constexpr int KW = W / HEADS;
  static constexpr int KEYS = kFewKeys * KW;
  static constexpr int CPR = HEADS * D / 32;
  static constexpr int CODES = KEYS * CPR * 16;
  static constexpr int S4 = HEADS * D / 128 > 0 ? HEADS * D / 128 : 1;
  static constexpr int SCALES = KEYS * S4 * 4;
  static constexpr int LOADS = KEYS * CPR / (64 * W);  // of a wave, K and V each
  static __device__ __forceinline__ int turn(int key) { return CPR >= 16 ? key & 15 : (key / (16 / CPR)) & (CPR - 1); }
  static __device__ __forceinline__ int place(int key, int chunk) { return (key * CPR + (chunk ^ turn(key))) * 16; }
};

// The keys of a split, where they are.
struct FewKeys {
  const AttendArgs& a;
  const int64_t* table;  // the sequence's row
  int64_t row;
  Span span;
  int i1, p;
  bool one;              // a tile of one token (decoding), at position p: a key that it does not see is none
  uint32_t bad = ~0u;    // the first entry that is not in the pool, kept for the end
  struct Key {
    int64_t page;
    uint32_t e, rest;  // place in the table's row, token inside the entry
    bool seen;
  };
  __device__ __forceinline__ FewKeys(const AttendArgs& args, int64_t s, const Span& sp, int end, int p_first, int p_last)
      : a(args), table(args.table + s * args.table_stride), row(s * args.table_stride), span(sp), i1(end), p(p_first),
        one(p_first == p_last) {}
  // The table entry of the i-th on its way, without a branch: past the end it is the last one's.
  __device__ __forceinline__ Key at(int i) const {
    const uint32_t j = span.key(i < i1 ? i : i1 - 1);
    Key k;
    k.e = (uint32_t)(((uint64_t)j * a.entry_magic) >> a.entry_shift);  // j / entry
    k.rest = j - k.e * (uint32_t)a.entry;
    k.page = table[k.e];
    k.seen = i < i1 && (!one || visible(a, p, (int)j));
    return k;
  }
  // Its slot; 0 for no key, of which `there` then has no bit.
  __device__ __forceinline__ uint32_t slot(const Key& k, uint64_t* there) {
    const bool ok = k.page >= 0 && k.page < a.entries;
    bad = k.seen && !ok && k.e < bad ? k.e : bad;
    *there = __ballot(k.seen && ok);
    return k.seen && ok ? (uint32_t)k.page * (uint32_t)a.entry + k.rest : 0u;
  }
  __device__ __forceinline__ void report() const {
    if (bad != ~0u) flag(a.wrong, kWrongIndex, row + bad);
  }
};

// The maximum over the four lanes that are 16 apart, without LDS.
__device__ __forceinline__ float max_of_quads(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t y = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
  const auto b = __builtin_amdgcn_permlane32_swap(y, y, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// 4 bytes a lane from memory into LDS, lane i to lds + 4 i (lds the same in all lanes), as lds_load.
__device__ __forceinline__ void lds_load_dword(const uint8_t* from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
}

// The items of a tile in another order: eight splits of one group of KV heads, then the same eight of the next, so that
// items which read the same rows are eight workgroups apart, on the same XCD at the same time, and its L2 reads
// the lines that both of them need once.  (`index`, where an item's partial result lies, stays in the list's order.)
__device__ __forceinline__ void pair_groups(const AttendArgs& a, Item* it) {
  const int at = it->hk * it->splits + it->split, whole = it->splits / 8 * 8;
  // a q_start that goes back (reported) can make more items than there are places: the last tile stays as it is
  if (it->index - at + it->splits * a.kv_heads > a.slots) return;
  if (at < whole * a.kv_heads) {
    const int chunk = at / (8 * a.kv_heads), rest = at - chunk * 8 * a.kv_heads;
    it->hk = rest / 8;
    it->split = chunk * 8 + rest % 8;
  } else {
    const int rest = at - whole * a.kv_heads, left = it->splits - whole;
    it->hk = rest / left;
    it->split = whole + rest - it->hk * left;
  }
  it->index += it->hk * it->splits + it->split - at;
}

template <class T, int D, int HEADS, bool SPLIT_FIRST>
__global__ __launch_bounds__(256, 4) void k_attend_mxfp4_few(AttendArgs a) {
  typedef typename T::v8 v8;
  typedef typename T::elem elem;
  typedef MxRows<T, D, D, HEADS> Rows;
  typedef FewStage<D, HEADS> Stage;
  constexpr int W = Stage::W;
  constexpr int KW = Stage::KW;         // waves that share a head's keys
  constexpr int G = Stage::KEYS;
  constexpr int KS = D / 32;            // product steps over the head: dwords of a lane and key
  constexpr int DT = D / 16;            // 16-dim tiles of the output
  constexpr int VL = D / 64;            // 64 dims of V at a time
  constexpr int R = kRowTile;
  constexpr int SL = G <= 64 ? 1 : G / 64;  // keys of a lane
  typedef uint32_t kw_t __attribute__((ext_vector_type(KS)));
  // codes of K and V, their scales, and 64 dims of 32 keys a wave; behind the loop the waves' sums
  constexpr int kStage = 2 * (Stage::CODES + Stage::SCALES), kAll = kStage + W * kFewKeys * 128;
  constexpr int kJoin = KW > 1 ? W * 64 * DT * 16 : 0;
  __shared__ __align__(16) uint8_t s_all[kAll > kJoin ? kAll : kJoin];
  __shared__ float s_ml[W][64][2];
  __shared__ int64_t s_plan[8];
  Item it;
  if (!find_item<true, SPLIT_FIRST>(a, R, s_plan, parts_of<D, R * HEADS>(a), &it)) return;
  if (a.kv_heads > 1) pair_groups(a, &it);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4, kw = wave / HEADS, hw = wave - kw * HEADS;
  const int hk = it.hk * HEADS + hw;
  const int rows_all = it.q.m * a.group;
  const int r0 = it.tile * R;
  const int rows = rows_all - r0 < R ? rows_all - r0 : R;
  // this lane's row
  const bool live = col < rows;
  const int r = r0 + (live ? col : 0);
  const int tok = r / a.group, h = hk * a.group + (r - tok * a.group);
  const int64_t row = it.q.q0 + tok;
  const int p = it.q.kv - it.q.m + tok;
  const int p_first = it.q.kv - it.q.m + r0 / a.group, p_last = it.q.kv - it.q.m + (r0 + rows - 1) / a.group;
  const Span span = span_of(a, it.q.kv, p_first, p_last);
  // this split's part of the span
  const int part = ((span.n + it.splits - 1) / it.splits + G - 1) / G * G;
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
      const v4u x = qp[quad * KS + i] ^ flip;
      q[i] = __builtin_bit_cast(v8, live ? x : v4u{0, 0, 0, 0});
    }
  }
  f32x4 o[DT] = {};
  float m = -INFINITY, l = 0.f;
  uint8_t* sk = s_all;
  uint8_t* sv = s_all + Stage::CODES;
  uint8_t* ssk = s_all + 2 * Stage::CODES;
  uint8_t* ssv = ssk + Stage::SCALES;
  uint8_t* st_v = s_all + kStage + wave * kFewKeys * 128;
  FewKeys keys(a, it.s, span, i1, p_first, p_last);
  // A tile's rows on their way into LDS.  (Rows of K and V are equally long.)
  const uint32_t row_bytes = (uint32_t)a.k_row;
  const int codes = (int)mxfp4_codes((int64_t)a.kv_heads * HEADS * D);
  const uint8_t* k_at = a.k_rows + it.hk * HEADS * (D / 2);
  const uint8_t* v_at = a.v_rows + it.hk * HEADS * (D / 2);
  const int scale0 = codes + (it.hk * HEADS * (D / 32) & ~3);  // a single head of 64 has two bytes of a dword
  auto load = [&](const uint32_t (&slot)[SL]) {
    auto slot_at = [&](int key) {
      uint32_t x = __shfl(slot[0], key & 63);
      for (int n = 1; n < SL; n++) {
        const uint32_t y = __shfl(slot[n], key & 63);
        x = key >> 6 == n ? y : x;
      }
      return x;
    };
#pragma unroll
    for (int n = 0; n < Stage::LOADS; n++) {
      const int at = (n * W + wave) * 64 + lane, key = at / Stage::CPR, chunk = at % Stage::CPR ^ Stage::turn(key);
      const uint64_t off = (uint64_t)slot_at(key) * row_bytes + chunk * 16;
      lds_load(k_at + off, lds_offset(sk + (n * W + wave) * 1024));
      lds_load(v_at + off, lds_offset(sv + (n * W + wave) * 1024));
    }
    // dwords of scales, K's and then V's: 64 a wave
    constexpr int N = G * Stage::S4;
    if (wave * 64 < 2 * N) {
      const int at = wave * 64 + lane, is_v = at >= N, d = at - (is_v ? N : 0), key = d / Stage::S4;
      const uint8_t* rows_at = is_v ? a.v_rows : a.k_rows;
      lds_load_dword(rows_at + (uint64_t)slot_at(key) * row_bytes + scale0 + d % Stage::S4 * 4, lds_offset(ssk + wave * 256));
    }
  };
  // V: a lane's block of 64 dims, and its key: 16 lanes next to each other write 16 places
  const int block = lane & 1;
  const int vkey = ((lane >> 1) & 1) | ((lane >> 2) & 3) << 2 | ((lane >> 4) & 1) << 1 | (lane >> 5) << 4;
  const int key0 = kw * kFewKeys;  // the wave's first of the tile
  const int byte0 = hw * (D / 32) + (HEADS * D < 128 ? (hk & 1) * 2 : 0);
  uint64_t there[SL] = {}, there_next[SL] = {};
  uint32_t slot[SL];
  FewKeys::Key next[SL];
  if (i0 < i1) {
#pragma unroll
    for (int n = 0; n < SL; n++) slot[n] = keys.slot(keys.at(i0 + n * 64 + lane), &there[n]);
    load(slot);
#pragma unroll
    for (int n = 0; n < SL; n++) next[n] = keys.at(i0 + G + n * 64 + lane);
  }
  for (int tile0 = i0; tile0 < i1; tile0 += G) {
    const int base = tile0 + key0;  // the wave's keys
    const bool more = tile0 + G < i1;
#pragma unroll
    for (int n = 0; n < SL; n++) slot[n] = more ? keys.slot(next[n], &there_next[n]) : 0;
    lds_arrived();
    __syncthreads();
    kw_t kc[2];
    v4u vc[VL];
    uint32_t ks[2], vs[VL];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      const int key = key0 + t * 16 + col;
      if (D == 128)
        kc[t] = *reinterpret_cast<const kw_t*>(sk + Stage::place(key, hw * 4 + quad));
      else
        kc[t] = *reinterpret_cast<const kw_t*>(sk + Stage::place(key, hw * 2 + quad / 2) + (quad & 1) * 8);
      ks[t] = ssk[key * Stage::S4 * 4 + byte0 + quad * KS / 4];
    }
#pragma unroll
    for (int g = 0; g < VL; g++) {
      const int key = key0 + vkey;
      vc[g] = *reinterpret_cast<const v4u*>(sv + Stage::place(key, hw * (D / 32) + g * 2 + block));
      vs[g] = ssv[key * Stage::S4 * 4 + byte0 + g * 2 + block];
    }
    __syncthreads();  // every wave has its codes: the next tile's may come
    if (more) {
      load(slot);
#pragma unroll
      for (int n = 0; n < SL; n++) next[n] = keys.at(tile0 + 2 * G + n * 64 + lane);
    }
    const uint32_t here = (uint32_t)(there[SL > 1 ? key0 / 64 : 0] >> (key0 & 63));  // the wave's keys
    f32x4 st[2] = {};
#pragma unroll
    for (int i = 0; i < KS; i++)
#pragma unroll
      for (int t = 0; t < 2; t++)
        st[t] = T::mfma16(__builtin_bit_cast(v8, mx_decode<kIsBf16<T>>(kc[t][i], mx_scale(ks[t]))), q[i], st[t]);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; e++) x[e] = st[e / 4][e % 4];
    // hidden keys: past the end, bad entries, and those that this row does not see
    const bool whole = here == ~0u && (!a.causal || (span.key(base + kFewKeys - 1) <= p_first &&
                                                     (a.window == 0 || p_last - span.key(base) < a.window)));
    if (!whole) {
      const uint32_t see = (uint32_t)sees(a, span, here, p, base) >> (quad * 4);
#pragma unroll
      for (int e = 0; e < 8; e++) x[e] = (see >> (e / 4 * 16 + e % 4)) & 1 ? x[e] : -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 8; e++) top = fmaxf(top, x[e]);
    top = max_of_quads(top);
    if (__any((top - m) * c > kGrow || (m == -INFINITY && top != -INFINITY))) {
      const float grown = fmaxf(m, top);
      const float keep = grown == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - grown) * c);
      m = grown;
      l *= keep;
#pragma unroll
      for (int d = 0; d < DT; d++) o[d] *= keep;
    }
    const float zero = m == -INFINITY ? 0.f : m * c;
    f32x8 w;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c, -zero));
      sum += w[e];
    }
    l += sum;  // this lane's keys; the quads are summed at the end
    const v8 wt = __builtin_convertvector(w, v8);  // the weight's one rounding, as the product's operand
    if (here != ~0u && !((here >> vkey) & 1)) {  // what was fetched in place of no key must not reach the product
#pragma unroll
      for (int g = 0; g < VL; g++) vc[g] = v4u{0, 0, 0, 0}, vs[g] = 127;
    }
#pragma unroll
    for (int g = 0; g < VL; g++) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 4; i++)
        *reinterpret_cast<v4u*>(st_v + few_place(vkey, block * 4 + i)) = mx_decode<kIsBf16<T>>(vc[g][i], mx_scale(vs[g]));
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int d = 0; d < 4; d++) {
        s16x4 v[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
          const int key = t * 16 + quad * 4 + col / 4;
          v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4)(st_v + few_place(key, d * 2 + (col & 3) / 2) + (col & 1) * 8));
        }
        const v8 vt = __builtin_bit_cast(v8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        o[g * 4 + d] = T::mfma16(vt, wt, o[g * 4 + d]);
      }
    }
#pragma unroll
    for (int n = 0; n < SL; n++) there[n] = there_next[n];
  }
  keys.report();
  __syncthreads();  // the tiles are done with
  float* s_q = reinterpret_cast<float*>(s_all) + wave * (KW > 1 ? 64 * DT * 4 : D);  // this wave's
  if (KW > 1) {  // the first wave of a head takes in the others', a lane its own places
    if (kw > 0) {
#pragma unroll
      for (int d = 0; d < DT; d++) reinterpret_cast<f32x4*>(s_q)[d * 64 + lane] = o[d];
      s_ml[wave][lane][0] = m;
      s_ml[wave][lane][1] = l;
    }
    __syncthreads();
    if (kw > 0) return;
#pragma unroll
    for (int w = 1; w < KW; w++) {
      const int from = w * HEADS + hw;
      const float mw = s_ml[from][lane][0], next = fmaxf(m, mw);
      const float zero = next == -INFINITY ? 0.f : next;
      const float keep = __builtin_amdgcn_exp2f((m - zero) * c), add = __builtin_amdgcn_exp2f((mw - zero) * c);
      m = next;
      l = l * keep + s_ml[from][lane][1] * add;
#pragma unroll
      for (int d = 0; d < DT; d++) o[d] = o[d] * keep + reinterpret_cast<const f32x4*>(s_all)[(from * DT + d) * 64 + lane] * add;
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  bool nan = false;
#pragma unroll
  for (int d = 0; d < DT; d++)
#pragma unroll
    for (int e = 0; e < 4; e++) nan |= o[d][e] != o[d][e];
  uint64_t again = __ballot(nan && live && l == l);
  again |= again >> 32;
  again = (again | again >> 16) & 0xffff;
  const float log2_max = m == -INFINITY ? -INFINITY : m * c;  // of the weights, in the joining kernel's unit
  float* part_o = a.work + it.index * partial_floats<D>(R * HEADS);
  float* part_ml = part_o + R * HEADS * D;
  if (live && !((again >> col) & 1)) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    elem* op = reinterpret_cast<elem*>(a.out) + row * a.out_stride[0] + h * a.out_stride[1];
#pragma unroll
    for (int d = 0; d < DT; d++) {
      typedef elem e4 __attribute__((ext_vector_type(4)));
      if (it.splits > 1)
        *reinterpret_cast<f32x4*>(part_o + (hw * R + col) * D + d * 16 + quad * 4) = o[d];
      else
        *reinterpret_cast<e4*>(op + d * 16 + quad * 4) = __builtin_convertvector(o[d] * inv, e4);
    }
    if (quad == 0) {
      if (it.splits > 1) {
        part_ml[(hw * R + col) * 2] = log2_max;
        part_ml[(hw * R + col) * 2 + 1] = l;
      } else if (a.lse) {
        a.lse[row * a.q_heads + h] = l == 0.f ? -INFINITY : (log2_max + log2f(l)) * kLn2;
      }
    }
  }
  // rows that came out NaN, one after the other
  while (again) {
    const int y = __builtin_ctzll(again);
    again &= again - 1;
    const int ta = (r0 + y) / a.group, ha = hk * a.group + (r0 + y - ta * a.group);
    float oo[D / 64], mm, ll;
    exact_row<T, D, D, Rows>(a, it.s, it.q.q0 + ta, ha, it.q.kv - it.q.m + ta, span, i0, i1, s_q, oo, &mm, &ll);
    elem* oa = reinterpret_cast<elem*>(a.out) + (it.q.q0 + ta) * a.out_stride[0] + ha * a.out_stride[1];
    for (int x = 0; x < D / 64; x++) {
      if (it.splits > 1) part_o[(hw * R + y) * D + x * 64 + lane] = oo[x];
      else oa[x * 64 + lane] = (elem)(ll == 0.f ? 0.f : oo[x] / ll);
    }
    if (lane == 0) {
      if (it.splits > 1) {
        part_ml[(hw * R + y) * 2] = mm;
        part_ml[(hw * R + y) * 2 + 1] = ll;
      } else if (a.lse) {
        a.lse[(it.q.q0 + ta) * a.q_heads + ha] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      }
    }
  }
}

// A latent cache, up to 16 rows a tile: one row of 320 bytes is key and value.  A wave takes 32 keys, by itself: their
// rows come straight into its own part of LDS, their scores leave the weights in the registers that the sums
// take them from, for all 512 dims, and the waves meet at the split's end only.  What bounds it is the
// conversion of every code twice, as key and as value, on two waves a SIMD.
//
// V needs no transposition: which dims a product's 16 rows are is free, so they are every eighth, of which a lane has
// the eight in one dword of a key's codes; two keys' pairs of dims become two dims' pairs of keys by two byte
// permutations.  (Through LDS as elements, as above: 64 KiB a wave and tile, 7.3 us a tile of 128 keys on two
// workgroups a compute unit.)
constexpr int kMxLatKeys = 4 * kFewKeys;  // of a tile of all waves
// A wave's rows in LDS: chunks 0 to 7 and 8 to 15 of 8 keys by 128 bytes, then chunks 16 to 19 (the last codes and the
// scales) of 16 keys by 64, each what one load brings.  Places are turned by the key, so that 16 keys' same chunk is
// in 16 places.
constexpr int kMxLatTail = 8192;
constexpr int kMxLatStage = 10240;
__device__ __forceinline__ int mx_lat_turn(int key) { return (key >> 1) & 7; }
__device__ __forceinline__ int mx_lat_tail_turn(int key) { return (key >> 2) & 3; }

// Waits for this wave's reads of LDS, which a load into it does not.
__device__ __forceinline__ void lds_read() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <class T, bool SPLIT_FIRST>
__global__ __launch_bounds__(256, 2) void k_attend_mxfp4_latent_few(AttendArgs a) {
  typedef typename T::v8 v8;
  typedef typename T::elem elem;
  typedef MxRows<T, kLatDim, kLatValue> Rows;
  constexpr int R = kRowTile;
  constexpr int DT = kLatValue / 16, KS = kLatDim / 32;
  constexpr int G = kMxLatKeys;
  constexpr int kQ = KS * 64 * 16, kStages = 4 * kMxLatStage, kJoin = 2 * 4 * 64 * (DT / 4) * 16;
  __shared__ __align__(16) uint8_t s_all[kStages + kQ > kJoin ? kStages + kQ : kJoin];  // behind the loop two quarters of the four waves' sums
  __shared__ float s_ml[4][64][2];
  __shared__ uint32_t s_nan;
  __shared__ int64_t s_plan[8];
  Item it;
  if (!find_item<true, SPLIT_FIRST>(a, R, s_plan, parts_of<kLatValue, R>(a), &it)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int rows_all = it.q.m * a.group;
  const int r0 = it.tile * R;
  const int rows = rows_all - r0 < R ? rows_all - r0 : R;
  // this lane's row
  const bool live = col < rows;
  const int r = r0 + (live ? col : 0);
  const int tok = r / a.group, h = r - tok * a.group;
  const int64_t row = it.q.q0 + tok;
  const int p = it.q.kv - it.q.m + tok;
  const int p_first = it.q.kv - it.q.m + r0 / a.group, p_last = it.q.kv - it.q.m + (r0 + rows - 1) / a.group;
  const Span span = span_of(a, it.q.kv, p_first, p_last);
  // this split's part of the span
  const int part = ((span.n + it.splits - 1) / it.splits + G - 1) / G * G;
  const int i0 = (int64_t)it.split * part < span.n ? it.split * part : span.n;
  const int i1 = i0 + part < span.n ? i0 + part : span.n;
  // weights are exp2(c * score - c * maximum); a negative scale turns the queries' sign
  const float c = weight_scale(a);
  uint8_t* sk = s_all + wave * kMxLatStage;
  v4u* s_q = reinterpret_cast<v4u*>(s_all + kStages);
  f32x4 o[DT] = {};
  float m = -INFINITY, l = 0.f;
  FewKeys keys(a, it.s, span, i1, p_first, p_last);
  const uint32_t row_bytes = (uint32_t)a.k_row;
  auto load = [&](uint32_t slot) {
#pragma unroll
    for (int n = 0; n < 4; n++) {
      const int key = n * 8 + lane / 8;
      const uint8_t* at = a.k_rows + (uint64_t)__shfl(slot, key) * row_bytes + ((lane & 7) ^ mx_lat_turn(key)) * 16;
      lds_load(at, lds_offset(sk + n * 1024));
      lds_load(at + 128, lds_offset(sk + 4096 + n * 1024));
    }
#pragma unroll
    for (int n = 0; n < 2; n++) {
      const int key = n * 16 + lane / 4;
      lds_load(a.k_rows + (uint64_t)__shfl(slot, key) * row_bytes + 256 + ((lane & 3) ^ mx_lat_tail_turn(key)) * 16,
               lds_offset(sk + kMxLatTail + n * 1024));
    }
  };
  // K: key col (and 16 on), chunk 4 g + quad: two cases of g.  Scales 4 g + quad, and the last two blocks.
  const uint8_t *k_at[2], *v_at[2][2];
  for (int g = 0; g < 2; g++)
    k_at[g] = sk + col / 8 * 1024 + col % 8 * 128 + ((g * 4 + quad) ^ mx_lat_turn(col)) * 16;
  const uint8_t* tail = sk + kMxLatTail + col * 64;
  const uint8_t* k_tail = tail + ((quad / 2) ^ mx_lat_tail_turn(col)) * 16 + (quad & 1) * 8;
  const uint8_t* k_scale = tail + (2 ^ mx_lat_tail_turn(col)) * 16 + quad;
  const uint8_t* k_last = tail + (3 ^ mx_lat_tail_turn(col)) * 16 + quad / 2;
  // V: keys 4 quad + r (and 16 on), chunk 4 g + col / 4, dword col % 4: two cases of g, two of r.
  for (int g = 0; g < 2; g++)
    for (int u = 0; u < 2; u++)
      v_at[g][u] = sk + quad / 2 * 1024 + (quad & 1) * 512 + u * 256 +
                   ((g * 4 + col / 4) ^ mx_lat_turn(quad * 4 + u * 2)) * 16 + (col & 3) * 4;
  const uint8_t* v_scale = sk + kMxLatTail + quad * 256 + (2 ^ quad) * 16 + col / 4;
  int base = i0 + wave * kFewKeys;  // keys of lanes 0 to 31, and of 32 to 63 again
  uint64_t there = 0;
  FewKeys::Key next = {};
  FewKeys::Key first = {};
  if (base < i1) first = keys.at(base + (lane & 31));
  // Queries as the products take them, a wave every fourth: of the first 16 blocks a lane has 32 dims of one in four
  // products, of the last two 16 dims in two.  On their way before the rows, and waited for behind.
  v4u q_in[(KS + 3) / 4];
  {
    const v4u* qp = reinterpret_cast<const v4u*>(a.q + 2 * (row * a.q_stride[0] + h * a.q_stride[1]));
#pragma unroll
    for (int n = 0; n < (KS + 3) / 4; n++) {
      const int i = n * 4 + wave < KS ? n * 4 + wave : KS - 1;
      q_in[n] = qp[i < 16 ? (i / 4 * 4 + quad) * 4 + i % 4 : 64 + quad * 2 + i - 16];
    }
  }
  if (base < i1) {
    load(keys.slot(first, &there));
    if (base + G < i1) next = keys.at(base + G + (lane & 31));
  }
  {
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int n = 0; n < (KS + 3) / 4; n++)
      if (n * 4 + wave < KS) s_q[(n * 4 + wave) * 64 + lane] = live ? q_in[n] ^ flip : v4u{0, 0, 0, 0};
  }
  __syncthreads();  // the queries are in LDS
  for (; base < i1; base += G) {
    const bool more = base + G < i1;
    lds_arrived();
    __builtin_amdgcn_wave_barrier();
    f32x4 st[2] = {};
#pragma unroll
    for (int g = 0; g < 5; g++) {
      v4u kc[2];
      float ks[2];
#pragma unroll
      for (int t = 0; t < 2; t++) {
        if (g < 4) {
          kc[t] = *reinterpret_cast<const v4u*>(k_at[g & 1] + g / 2 * 4096 + t * 2048);
          ks[t] = mx_scale(k_scale[t * 1024 + g * 4]);
        } else {
          typedef uint32_t u2 __attribute__((ext_vector_type(2)));
          const u2 y = *reinterpret_cast<const u2*>(k_tail + t * 1024);
          kc[t] = v4u{y[0], y[1], 0, 0};
          ks[t] = mx_scale(k_last[t * 1024]);
        }
      }
#pragma unroll
      for (int i = 0; i < (g < 4 ? 4 : 2); i++) {
        const v8 q = __builtin_bit_cast(v8, s_q[(g * 4 + i) * 64 + lane]);
#pragma unroll
        for (int t = 0; t < 2; t++)
          st[t] = T::mfma16(__builtin_bit_cast(v8, mx_decode<kIsBf16<T>>(kc[t][i], ks[t])), q, st[t]);
      }
    }
    const uint32_t here = (uint32_t)there;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; e++) x[e] = st[e / 4][e % 4];
    // hidden keys: past the end, bad entries, and those that this row does not see
    const bool whole = here == ~0u && (!a.causal || (span.key(base + kFewKeys - 1) <= p_first &&
                                                     (a.window == 0 || p_last - span.key(base) < a.window)));
    if (!whole) {
      const uint32_t see = (uint32_t)sees(a, span, here, p, base) >> (quad * 4);
#pragma unroll
      for (int e = 0; e < 8; e++) x[e] = (see >> (e / 4 * 16 + e % 4)) & 1 ? x[e] : -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 8; e++) top = fmaxf(top, x[e]);
    top = max_of_quads(top);
    if (__any((top - m) * c > kGrow || (m == -INFINITY && top != -INFINITY))) {
      const float grown = fmaxf(m, top);
      const float keep = grown == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - grown) * c);
      m = grown;
      l *= keep;
#pragma unroll
      for (int d = 0; d < DT; d++) o[d] *= keep;
    }
    const float zero = m == -INFINITY ? 0.f : m * c;
    f32x8 w;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c, -zero));
      sum += w[e];
    }
    l += sum;  // this lane's keys; the quads are summed at the end
    const v8 wt = __builtin_convertvector(w, v8);  // the weight's one rounding, as the product's operand
    // four of a lane's keys at a time: 4 quad + r, and 16 on
#pragma unroll
    for (int g = 0; g < 4; g++) {
      uint32_t vc[8];
      float vs[8];
#pragma unroll
      for (int e = 0; e < 8; e++) {
        vc[e] = *reinterpret_cast<const uint32_t*>(v_at[g & 1][e % 4 / 2] + g / 2 * 4096 + e / 4 * 2048 + e % 2 * 128);
        vs[e] = mx_scale(v_scale[e / 4 * 1024 + e % 4 * 64 + g * 4]);
      }
      if (here != ~0u) {  // what was fetched in place of no key must not reach the product: its value is zero
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const bool some = (here >> (e / 4 * 16 + quad * 4 + e % 4)) & 1;
          vc[e] = some ? vc[e] : 0u;
          vs[e] = some ? vs[e] : 1.f;
        }
      }
      v4u d[8];  // a key's eight dims
#pragma unroll
      for (int e = 0; e < 8; e++) d[e] = mx_decode<kIsBf16<T>>(vc[e], vs[e]);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v4u even, odd;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          even[e] = __builtin_amdgcn_perm(d[2 * e + 1][i], d[2 * e][i], 0x05040100u);
          odd[e] = __builtin_amdgcn_perm(d[2 * e + 1][i], d[2 * e][i], 0x07060302u);
        }
        o[g * 8 + 2 * i] = T::mfma16(__builtin_bit_cast(v8, even), wt, o[g * 8 + 2 * i]);
        o[g * 8 + 2 * i + 1] = T::mfma16(__builtin_bit_cast(v8, odd), wt, o[g * 8 + 2 * i + 1]);
      }
    }
    if (more) {
      const uint32_t slot = keys.slot(next, &there);
      lds_read();  // the tile's codes are in registers: the next one's may come
      load(slot);
      if (base + 2 * G < i1) next = keys.at(base + 2 * G + (lane & 31));
    }
  }
  keys.report();
  // The waves' sums are joined by quarters of the dims, one a wave, two at a time in LDS.
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  s_ml[wave][lane][0] = m;
  s_ml[wave][lane][1] = l;
  if (threadIdx.x == 0) s_nan = 0;
  __syncthreads();  // the tiles are done with
  float f[4], m_all = -INFINITY, l_all = 0.f;
#pragma unroll
  for (int w = 0; w < 4; w++) m_all = fmaxf(m_all, s_ml[w][lane][0]);
#pragma unroll
  for (int w = 0; w < 4; w++) {
    f[w] = __builtin_amdgcn_exp2f((s_ml[w][lane][0] - (m_all == -INFINITY ? 0.f : m_all)) * c);
    l_all += s_ml[w][lane][1] * f[w];
  }
  f32x4* so = reinterpret_cast<f32x4*>(s_all);
  f32x4 acc[DT / 4];
#pragma unroll
  for (int half = 0; half < 2; half++) {
    if (half) __syncthreads();
#pragma unroll
    for (int d = 0; d < DT / 2; d++) so[(wave * (DT / 2) + d) * 64 + lane] = o[half * (DT / 2) + d];
    __syncthreads();
    if (wave / 2 == half) {
#pragma unroll
      for (int d = 0; d < DT / 4; d++) {
        acc[d] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; w++) acc[d] += so[(w * (DT / 2) + (wave & 1) * (DT / 4) + d) * 64 + lane] * f[w];
      }
    }
  }
  bool nan = false;
#pragma unroll
  for (int d = 0; d < DT / 4; d++)
#pragma unroll
    for (int e = 0; e < 4; e++) nan |= acc[d][e] != acc[d][e];
  uint64_t bits = __ballot(nan && live && l_all == l_all);
  bits |= bits >> 32;
  bits = (bits | bits >> 16) & 0xffff;
  if (lane == 0 && bits) atomicOr(&s_nan, (uint32_t)bits);
  __syncthreads();
  uint32_t again = s_nan;
  const float log2_max = m_all == -INFINITY ? -INFINITY : m_all * c;  // of the weights, in the joining kernel's unit
  float* part_o = a.work + it.index * partial_floats<kLatValue>(R);
  float* part_ml = part_o + R * kLatValue;
  auto finish = [&](int y, int64_t row_y, int head, float mm, float ll) {
    if (it.splits > 1) {
      part_ml[y * 2] = mm;
      part_ml[y * 2 + 1] = ll;
    } else if (a.lse) {
      a.lse[row_y * a.q_heads + head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
  };
  if (live && !((again >> col) & 1)) {
    const float inv = l_all == 0.f ? 0.f : 1.f / l_all;
    elem* op = reinterpret_cast<elem*>(a.out) + row * a.out_stride[0] + h * a.out_stride[1];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const int dim = wave * 128 + quad * 32 + e * 8;
      f32x8 y;
#pragma unroll
      for (int d = 0; d < 8; d++) y[d] = acc[d][e];
      if (it.splits > 1)
        *reinterpret_cast<f32x8*>(part_o + col * kLatValue + dim) = y;
      else
        *reinterpret_cast<v8*>(op + dim) = __builtin_convertvector(y * inv, v8);
    }
    if (wave == 0 && quad == 0) finish(col, row, h, log2_max, l_all);
  }
  // rows that came out NaN, shared out over the waves
  float* s_row = reinterpret_cast<float*>(s_all) + wave * kLatDim;
  while (again) {
    const int y = __builtin_ctz(again);
    again &= again - 1;
    if ((y & 3) != wave) continue;
    const int ta = (r0 + y) / a.group, ha = r0 + y - ta * a.group;
    float oo[kLatValue / 64], mm, ll;
    exact_row<T, kLatDim, kLatValue, Rows>(a, it.s, it.q.q0 + ta, ha, it.q.kv - it.q.m + ta, span, i0, i1, s_row, oo, &mm,
                                           &ll);
    elem* oa = reinterpret_cast<elem*>(a.out) + (it.q.q0 + ta) * a.out_stride[0] + ha * a.out_stride[1];
    for (int x = 0; x < kLatValue / 64; x++) {
      if (it.splits > 1) part_o[y * kLatValue + x * 64 + lane] = oo[x];
      else oa[x * 64 + lane] = (elem)(ll == 0.f ? 0.f : oo[x] / ll);
    }
    if (lane == 0) finish(y, it.q.q0 + ta, ha, mm, ll);
  }
}

// Joins the splits of rows, PER waves of a workgroup a row: with the greatest maximum known first, from one load a split
// over the lanes, the sums are loaded together instead of one after the other.  A workgroup looks at the
// item of one place; all but the first split of a tile that was split have nothing to do.
template <class T, int D, int HEADS, int PER>
__global__ __launch_bounds__(256) void k_attend_mxfp4_join(AttendArgs a) {
  typedef typename T::elem elem;
  typedef float f2 __attribute__((ext_vector_type(2)));
  constexpr int R = kRowTile, ND = D / 64;
  __shared__ float s_w[4][64], s_o[4][D], s_l[4];
  const int64_t first = blockIdx.x / a.join_parts;
  const Part p = parts_of<D, R * HEADS>(a)[first];
  // a q_start that goes back (reported) can make more items than the call has room for
  if (p.splits <= 1 || first + p.splits > a.slots) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), turn = wave % PER;
  const int64_t tile = p.tile_hk / a.kv_heads;
  const int part = (int)(blockIdx.x % a.join_parts), per = a.join_parts / HEADS, hw = part / per;
  const int y = (part - hw * per) * (4 / PER) + wave / PER;
  const int64_t r = tile * R + y;
  const bool some = y < R && r < p.m * a.group;
  const int hk = (int)(p.tile_hk - tile * a.kv_heads) * HEADS + hw, rr = hw * R + (some ? y : 0), splits = (int)p.splits;
  const float* part_o = a.work + first * partial_floats<D>(R * HEADS) + rr * D;
  const float* part_ml = a.work + first * partial_floats<D>(R * HEADS) + R * HEADS * D + rr * 2;
  auto ml = [&](int k) { return *reinterpret_cast<const f2*>(part_ml + k * partial_floats<D>(R * HEADS)); };
  float m = -INFINITY;
  for (int k = lane; k < splits; k += 64) m = fmaxf(m, ml(k)[0]);
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float zero = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[ND] = {};
  for (int k0 = turn; k0 < splits; k0 += 64 * PER) {  // splits k0, k0 + PER, ...
    const int mine = k0 + PER * lane, left = (splits - k0 + PER - 1) / PER, n = left < 64 ? left : 64;
    f2 v = {-INFINITY, 0.f};
    if (mine < splits) v = ml(mine);
    const float w = __builtin_amdgcn_exp2f(v[0] - zero);
    l += v[1] * w;
    s_w[wave][lane] = w;
    __builtin_amdgcn_wave_barrier();
    const float* po = part_o + k0 * partial_floats<D>(R * HEADS) + lane;
#pragma unroll 8
    for (int j = 0; j < n; j++) {
      const float f = s_w[wave][j];
#pragma unroll
      for (int c = 0; c < ND; c++) o[c] += po[c * 64] * f;
      po += PER * partial_floats<D>(R * HEADS);
    }
    __builtin_amdgcn_wave_barrier();
  }
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
  if (PER > 1) {
#pragma unroll
    for (int c = 0; c < ND; c++) s_o[wave][c * 64 + lane] = o[c];
    if (lane == 0) s_l[wave] = l;
    __syncthreads();
    if (turn > 0) return;
    for (int w = 1; w < PER; w++) {
      l += s_l[wave + w];
#pragma unroll
      for (int c = 0; c < ND; c++) o[c] += s_o[wave + w][c * 64 + lane];
    }
  }
  if (!some) return;
  const int64_t rt = r / a.group;
  const int h = hk * a.group + (int)(r - rt * a.group);
  elem* op = reinterpret_cast<elem*>(a.out) + (p.q0 + rt) * a.out_stride[0] + h * a.out_stride[1];
#pragma unroll
  for (int c = 0; c < ND; c++) op[c * 64 + lane] = (elem)(l == 0.f ? 0.f : o[c] / l);
  if (a.lse && lane == 0) a.lse[(p.q0 + rt) * a.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- tiles of 4-bit rows, as elements into LDS
// A tile's codes wait in registers while the tile before is computed, 16 bytes and a scale for a
// block of 32 elements, and are written to LDS as elements beside its second product, by one wave for all four.
// 16 lanes next to each other write all banks.
template <class T, int D>
struct MxTiles {
  typedef MxRows<T, D, D> Rows;
  static constexpr bool kZeros = true;
  static constexpr int N = D == 128 ? 2 : 1;  // blocks of a lane: of K and V, or of one of them
  const uint8_t *codes_at[N], *scales_at[N];
  int key, block;
  bool is_v;  // N == 1
  v4u codes[N] = {};
  uint32_t scales[N] = {};
  __device__ __forceinline__ MxTiles(const AttendArgs& a, int hk, int lane, int wave) {
    const int64_t scales0 = mxfp4_codes((int64_t)a.kv_heads * D);
    if (D == 128) {
      key = wave * 16 + ((lane >> 2) & 3) * 4 + (lane >> 4);
      block = lane & 3;
      is_v = false;
    } else {
      key = (wave & 1) * 32 + lane / 2;
      block = lane & 1;
      is_v = wave >= 2;
    }
#pragma unroll
    for (int n = 0; n < N; n++) {
      const uint8_t* rows = N == 2 ? (n ? a.v_rows : a.k_rows) : (is_v ? a.v_rows : a.k_rows);
      codes_at[n] = rows + hk * (D / 2) + block * 16;
      scales_at[n] = rows + scales0 + hk * (D / 32) + block;
    }
  }
  __device__ __forceinline__ void load(const AttendArgs& a, uint32_t slot, uint8_t*, uint8_t*) {
    const uint32_t sl = __shfl(slot, key);
    const uint64_t at = sl == kNoSlot ? 0 : (uint64_t)sl * a.k_row;
#pragma unroll
    for (int n = 0; n < N; n++) {
      const v4u y = *reinterpret_cast<const v4u*>(codes_at[n] + at);
      const uint32_t z = scales_at[n][at];
      codes[n] = sl == kNoSlot ? v4u{0, 0, 0, 0} : y;
      scales[n] = sl == kNoSlot ? 127 : z;
    }
  }
  // Behind the last tile the codes of the one before are written again, to LDS that is done with.
  __device__ __forceinline__ void step(int i, uint8_t* k, uint8_t* v) {
    const int chunk = block * 4 + i;
#pragma unroll
    for (int n = 0; n < N; n++) {
      const v4u y = mx_decode<kIsBf16<T>>(codes[n][i], mx_scale(scales[n]));
      if (N == 2) *reinterpret_cast<v4u*>(n ? v + v_place(key, chunk) : k + k_place(key, chunk)) = y;
      else *reinterpret_cast<v4u*>(is_v ? v + v_place(key, chunk) : k + k_place(key, chunk)) = y;
    }
  }
  __device__ __forceinline__ void arrive(bool first, uint8_t* k, uint8_t* v) {
    if (!first) return;
#pragma unroll
    for (int i = 0; i < 4; i++) step(i, k, v);
  }
  // Where a row's chunk lies: read, 16 rows' same chunk of K and four rows' 32 dims of V lie in different banks.
  static __device__ __forceinline__ int k_place(int row, int chunk) {
    return row * D * 2 + (chunk ^ (D == 128 ? (row & 3) << 2 | ((row >> 2) & 3) : (row >> 1) & 7)) * 16;
  }
  static __device__ __forceinline__ int v_place(int row, int chunk) {
    return row * D * 2 +
           (chunk ^ (D == 128 ? (row & 3) << 2 | ((row >> 2) & 3) : ((row >> 1) & 1) << 2 | ((row >> 1) & 3))) * 16;
  }
};

// 64 keys of a latent cache: 18 blocks a key, 1152 in all, 16 lanes taking two blocks next to each other of
// eight keys, whose places are in all banks.
template <class T>
struct MxLatent {
  typedef MxRows<T, kLatDim, kLatValue> Rows;
  static constexpr bool kZeros = true;
  static constexpr int N = 5;  // rounds over the workgroup's 16 sixteens of lanes, the last of them half empty
  v4u codes[N] = {};
  uint32_t scales[N] = {};
  __device__ __forceinline__ explicit MxLatent(const AttendArgs&) {}
  // Pair of blocks, key and the lane's block of the pair, in round n; false: none.
  static __device__ __forceinline__ bool place(int n, int* pair, int* key, int* b) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int u = n * 16 + wave * 4 + (lane >> 4), octet = u / 9;
    *pair = u - octet * 9;
    *b = lane & 1;
    *key = ((lane >> 1) & 1) | (octet & 1) << 1 | ((lane >> 2) & 1) << 2 | ((lane >> 3) & 1) << 3 | (octet >> 1) << 4;
    return u < 72;
  }
  __device__ __forceinline__ void load(const AttendArgs& a, uint32_t slot, uint8_t*) {
#pragma unroll
    for (int n = 0; n < N; n++) {
      int pair, key, b;
      const bool some = place(n, &pair, &key, &b);
      const uint32_t sl = __shfl(slot, some ? key : 0);
      const uint8_t* at = a.k_rows + (sl == kNoSlot ? 0 : (uint64_t)sl * a.k_row);
      const int block = some ? pair * 2 + b : 0;
      const v4u y = *reinterpret_cast<const v4u*>(at + block * 16);
      const uint32_t z = at[mxfp4_codes(kLatDim) + block];
      codes[n] = sl == kNoSlot ? v4u{0, 0, 0, 0} : y;
      scales[n] = sl == kNoSlot ? 127 : z;
    }
  }
  // (Behind the last tile as in MxTiles.)
  __device__ __forceinline__ void round(int n, uint8_t* to) {
    int pair, key, b;
    if (!place(n, &pair, &key, &b)) return;
#pragma unroll
    for (int i = 0; i < 4; i++)
      *reinterpret_cast<v4u*>(to + pair * kLatBlock + key * 128 + ((b * 4 + i) ^ lat_swizzle(key)) * 16) =
          mx_decode<kIsBf16<T>>(codes[n][i], mx_scale(scales[n]));
  }
  __device__ __forceinline__ void step(int s, uint8_t* to) {
    round(s, to);
    if (s == 3) round(4, to);
  }
  __device__ __forceinline__ void arrive(bool first, uint8_t* to) {
    if (!first) return;
#pragma unroll
    for (int s = 0; s < 4; s++) step(s, to);
  }
};

// ---------------------------------------------------------------- many rows of a latent cache: its tokens as elements first
// Every row tile of a sequence converts all keys that it sees, beside products that one wave a SIMD leaves waiting.
// Where a sequence has many tiles and the call's tokens as elements are not many bytes, they are converted once, by a launch of
// their own, into the workspace, with a table that says where, and the kernels over elements do the rest.  (A
// bad entry, or bad lengths, are reported here; what those kernels report of this table goes to words that
// nobody reads.)
//
// Measured, converted in the kernel and first: four sequences of 8000 tokens and 16 heads with 8 new tokens each 50 and
// 57 us, 16 64 and 67, 32 97 and 89, 64 179 and 144, 128 467 and 341; a chunk of 512 behind 3988 with 32 heads 281 and
// 226.  One rule for the whole call: the decoding rows beside a chunk are converted too.  Converted in the kernel and first,
// 16 heads, 63 decoding rows of 1800 to 3600 beside a chunk of 32 behind 1500 83 and 125 us (the chunk alone 38, the rows
// alone 39), beside one of 512 behind 3000 216 and 209; 32 heads, 31 rows up to 6000 beside a chunk of 512 behind 3988 596
// and 458, of 2048 behind 2000 1090 and 835; 128 heads, 512 behind 3988 1359 and 1013.  And a max_kv so far above the
// lengths that the rows would not fit turns it off (the chunk of 512 alone 269 for 200).  (K and V of heads of 128: 512 new
// tokens each 322 and 330, a chunk of 2048 behind 14336 612 and 590 for 67 MB of workspace; not done.)
constexpr int kExpandTokens = 8;                       // of a workgroup
constexpr int64_t kExpandRows = 8 * kLatRows;           // of a sequence, at least
constexpr int64_t kExpandBytes = (int64_t)256 << 20;    // of the workspace, at most

// The workspace: words for reports, the rows, the table, then what the attention needs.
struct Expand {
  int64_t tokens, table_at, work_at;
};
Expand expand_of(const AttendArgs& a) {
  Expand e;
  e.tokens = a.num_seqs * a.max_kv;
  e.table_at = 256 + e.tokens * kLatDim * 2;
  e.work_at = (e.table_at + e.tokens * 8 + 255) / 256 * 256;
  return e;
}
bool expands(const AttendArgs& a, int32_t head_dim) {
  return head_dim == kLatDim && a.max_kv > 0 && a.max_q * a.group >= kExpandRows &&
         a.num_seqs <= kExpandBytes / (kLatDim * 2 + 8) / a.max_kv;
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_expand_latent(AttendArgs a, Expand e) {
  __shared__ uint32_t s_slot[kExpandTokens];
  const int64_t per = (a.max_kv + kExpandTokens - 1) / kExpandTokens, s = blockIdx.x / per;
  const int j0 = (int)(blockIdx.x - s * per) * kExpandTokens;
  const Seq q = sequence(a, s);
  if (!q.ok && j0 == 0 && threadIdx.x == 0) flag(a.wrong, kWrongLengths, s);
  if (q.m == 0 || j0 >= q.kv) return;
  const Span span = span_of(a, q.kv, q.kv - q.m, q.kv - 1);  // of all the sequence's rows: nothing else is read
  const int64_t row0 = s * a.max_kv + j0;
  uint8_t* work = reinterpret_cast<uint8_t*>(a.work);
  if (threadIdx.x < kExpandTokens) {
    const int j = j0 + threadIdx.x;
    uint32_t slot = kNoSlot;
    if (j < span.sk || (j >= span.lo && j < span.lo + span.n - span.sk)) slot = slot_of(a, s, (uint32_t)j);
    s_slot[threadIdx.x] = slot;
    if (j < q.kv) reinterpret_cast<int64_t*>(work + e.table_at)[row0 + threadIdx.x] = slot == kNoSlot ? -1 : row0 + threadIdx.x;
  }
  __syncthreads();
  constexpr int kVecs = kLatDim / 8;
  for (int i = threadIdx.x; i < kExpandTokens * kVecs; i += 256) {
    const int t = i / kVecs, w = i - t * kVecs;
    if (s_slot[t] == kNoSlot) continue;
    const uint8_t* row = a.k_rows + (uint64_t)s_slot[t] * a.k_row;
    const uint32_t codes = reinterpret_cast<const uint32_t*>(row)[w];
    const float scale = mx_scale(row[mxfp4_codes(kLatDim) + w / 4]);
    reinterpret_cast<v4u*>(work + 256 + (row0 + t) * kLatDim * 2)[w] = mx_decode<BF16>(codes, scale);
  }
}

// The call over the elements.
AttendArgs expanded(const AttendArgs& args, const Expand& e) {
  AttendArgs a = args;
  uint8_t* w = reinterpret_cast<uint8_t*>(a.work);
  a.wrong = reinterpret_cast<WrongWord*>(w);
  a.k_rows = a.v_rows = w + 256;
  a.k_row = a.v_row = kLatDim;
  a.table = reinterpret_cast<const int64_t*>(w + e.table_at);
  a.table_width = a.table_stride = a.max_kv;
  a.entry = 1;  // slots
  a.entry_shift = 31;
  a.entry_magic = 1u << 31;
  a.entries = e.tokens;
  a.work = reinterpret_cast<float*>(w + e.work_at);
  return a;
}

hipError_t launch_expanded(const AttendArgs& a, int32_t dtype, int32_t num_cus, hipStream_t stream) {
  const Expand e = expand_of(a);
  const int64_t groups = a.num_seqs * ((a.max_kv + kExpandTokens - 1) / kExpandTokens);
  (void)hipGetLastError();
  (dtype == HC_BF16 ? k_expand_latent<true> : k_expand_latent<false>)<<<dim3((unsigned)groups), 256, 0, stream>>>(a, e);
  const hipError_t err = hipGetLastError();
  return err != hipSuccess ? err : launch_attend(expanded(a, e), dtype, kLatDim, num_cus, stream);
}

// The kernel for a call: the rows of its row tiles.  64 sequences up to 8192 tokens, 32/8 heads of 128, with several
// new tokens each, in tiles of 16 and of 128 rows: 20 rows of a KV head 96 and 312 us, 32 rows 127 and 315, 48 rows 165
// and 317, 64 rows 195 and 325; 32 sequences up to 6000 tokens of a latent cache, in tiles of 16 and of 64 rows: 20 rows
// 32.0 and 49.2 us, 32 rows 36.3 and 51.4, 64 rows 48.8 and 58.4, 128 rows 110.6 and 102.1.
int tile_rows(const AttendArgs& a, int32_t head_dim) {
  const int64_t rows = a.max_q * a.group;
  return rows <= 4 * kRowTile ? kRowTile : head_dim == kLatDim ? kLatRows : kTileRows;
}

// KV heads of an item of few rows: as many as divide the heads, up to the waves.  (Eight, with eight waves: 64
// sequences up to 8192 of eight heads 83 us for 82, one sequence of 1500 15.6 for 14.0, 32 in a window of 4096 of fp16
// heads of 64 31.5 for 34.)
int heads_of(const AttendArgs& a) { return a.kv_heads % 4 == 0 ? 4 : a.kv_heads % 2 == 0 ? 2 : 1; }

// How calls of few rows are split: four workgroups a compute unit, splits of 32 keys and more (of 64: a sequence of 1500
// 14.0 us for 13.0) and no more than 128 of them (of 32768 keys: 64 splits 33 us, 128 24, 512 57; all of eight KV heads, four
// an item, whose tiles are 32 keys; two an item walk 64 and one 128, to which a split's part is rounded up, so
// that some of their splits have no key: a sequence of 1500 with 1, 2, 3 and 4 KV heads 13.0, 12.8, 13.3 and 13.3 us).  The
// least split is a 128th of max_kv, not of the length, which only the device knows: under a bound of 8192, 32768, 131072 and 2^20 a
// sequence of 1500 15.1, 21.5, 43 and 74 us for 14.4 under its own length, a window of 4096 in 32768 under 131072 and 2^20 46
// and 184 for 22; 64 sequences up to 8192 under 131072 122 for 118.  And joined: where
// there are few rows a workgroup a row (a sequence of 32768 24 us, by waves 35), else a wave, since empty workgroups
// cost more then (32 sequences of 16 heads in a window 34.3 us by workgroups, 32.4 by waves).
// A latent cache: two workgroups a compute unit and tiles of 128 keys (32 sequences up to 6000 of 16 heads 35 us; one
// workgroup 38, four 50).
constexpr int kFewPerCu = 4, kFewLeast = 32, kFewSplits = 128, kFewAlone = 128, kMxLatPerCu = 2;
Plan few_plan(AttendArgs* a, int32_t head_dim, int heads, int32_t num_cus, bool* alone = nullptr) {
  const bool latent = head_dim == kLatDim;
  const int most = (int)(a->max_kv / kFewSplits), tile = latent ? kMxLatKeys : kFewLeast;
  Plan p = plan(a, kRowTile, head_dim, num_cus, heads, latent ? kMxLatPerCu : kFewPerCu, most > tile ? most : tile);
  const bool row = a->q_rows * a->q_heads <= kFewAlone;
  if (alone) *alone = row;
  if (p.joins > 0 && !row) {
    a->join_parts = (a->join_parts / heads + 3) / 4 * heads;
    p.joins = a->slots * a->join_parts;
  }
  return p;
}

template <class T, int D, int HEADS>
hipError_t launch_few(AttendArgs a, int32_t num_cus, hipStream_t stream) {
  a.kv_heads /= HEADS;
  bool alone;
  const Plan p = few_plan(&a, D, HEADS, num_cus, &alone);
  return launch_planned({k_attend_mxfp4_few<T, D, HEADS, false>, k_attend_mxfp4_few<T, D, HEADS, true>},
                        alone ? k_attend_mxfp4_join<T, D, HEADS, 4> : k_attend_mxfp4_join<T, D, HEADS, 1>, a, p, stream);
}
template <class T, int D>
hipError_t launch_heads(const AttendArgs& a, int32_t num_cus, hipStream_t stream) {
  if (tile_rows(a, D) == kTileRows)
    return launch_split<T, D, kTileRows>(
        {k_attend_tiles<T, D, MxTiles<T, D>, false>, k_attend_tiles<T, D, MxTiles<T, D>, true>}, a, num_cus, stream);
  const int heads = heads_of(a);
  return heads == 4   ? launch_few<T, D, 4>(a, num_cus, stream)
         : heads == 2 ? launch_few<T, D, 2>(a, num_cus, stream)
                      : launch_few<T, D, 1>(a, num_cus, stream);
}
template <class T>
hipError_t launch_latent_few(AttendArgs a, int32_t num_cus, hipStream_t stream) {
  bool alone;
  const Plan p = few_plan(&a, kLatDim, 1, num_cus, &alone);
  return launch_planned({k_attend_mxfp4_latent_few<T, false>, k_attend_mxfp4_latent_few<T, true>},
                        alone ? k_attend_mxfp4_join<T, kLatValue, 1, 4> : k_attend_mxfp4_join<T, kLatValue, 1, 1>, a, p, stream);
}

template <class T>
hipError_t launch_for(const AttendArgs& a, int32_t head_dim, int32_t num_cus, hipStream_t stream) {
  (void)hipGetLastError();
  if (head_dim == 64) return launch_heads<T, 64>(a, num_cus, stream);
  if (head_dim == 128) return launch_heads<T, 128>(a, num_cus, stream);
  const int R = tile_rows(a, head_dim);
  return R == kRowTile ? launch_latent_few<T>(a, num_cus, stream)
         : launch_split<T, kLatValue, kLatRows>(
                         {k_attend_latent<T, MxLatent<T>, false>, k_attend_latent<T, MxLatent<T>, true>}, a, num_cus,
                         stream);
}

}  // namespace

int64_t attend_mxfp4_workspace(const AttendArgs& args, int32_t head_dim, int32_t num_cus) {
  if (args.q_rows <= 0 || args.num_seqs <= 0) return 0;
  const int R = tile_rows(args, head_dim);
  if (expands(args, head_dim)) {
    const Expand e = expand_of(args);
    return e.work_at + attend_workspace(expanded(args, e), head_dim, num_cus);
  }
  const bool few = R == kRowTile;
  const int heads = few && head_dim != kLatDim ? heads_of(args) : 1;
  AttendArgs a = args;
  a.kv_heads /= heads;
  const Plan p = few ? few_plan(&a, head_dim, heads, num_cus) : plan(&a, R, head_dim, num_cus);
  if (p.joins == 0) return 0;
  const int64_t floats = head_dim == 64    ? partial_floats<64>(R * heads)
                         : head_dim == 128 ? partial_floats<128>(R * heads)
                                           : partial_floats<kLatValue>(R);
  return a.slots * (4 * floats + (int64_t)sizeof(Part));
}

hipError_t launch_attend_mxfp4(const AttendArgs& a, int32_t dtype, int32_t head_dim, int32_t num_cus, hipStream_t stream) {
  if (a.q_rows <= 0 || a.num_seqs <= 0) return hipSuccess;
  if (expands(a, head_dim)) return launch_expanded(a, dtype, num_cus, stream);
  return dtype == HC_BF16 ? launch_for<Bf16>(a, head_dim, num_cus, stream) : launch_for<F16>(a, head_dim, num_cus, stream);
}

}  // namespace hc
