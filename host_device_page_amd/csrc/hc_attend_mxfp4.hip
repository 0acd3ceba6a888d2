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
// how little is read: 68 bytes of a key's 128 dims.
//
// HEADS waves take a KV head each and the same keys, so that a workgroup reads HEADS * 64 bytes of a row in one
// piece and its waves share the lines that a head's 64 bytes do not fill; the other waves share a head's
// keys in turns of 64, and are joined at the end.
//
//   K  straight into the operand registers: the order of the dims inside a product is free, so a lane
//      takes D / 4 dims of a key next to each other, one load and one scale, and the queries the same.
//   V  16 bytes a lane, a block of a key and its scale, through LDS as elements and back transposed.
template <int D>
__device__ __forceinline__ int few_place(int key, int chunk) {  // of 32 keys; written and read without conflicts
  const int x = D == 128 ? 2 * (key & 7) | ((key >> 3) & 1) : 2 * ((key >> 1) & 3) | ((key >> 3) & 1);
  return key * D * 2 + (chunk ^ x) * 16;
}

template <class T, int D, int HEADS, bool SPLIT_FIRST>
__global__ __launch_bounds__(256, 2) void k_attend_mxfp4_few(AttendArgs a) {
  typedef typename T::v8 v8;
  typedef typename T::elem elem;
  typedef MxRows<T, D, D, HEADS> Rows;
  constexpr int KW = 4 / HEADS;         // waves that share a head's keys
  constexpr int KS = D / 32;            // product steps over the head: dwords of a lane and key
  constexpr int DT = D / 16;            // 16-dim tiles of the output
  constexpr int VL = 64 * (D / 32) / 64;  // V loads of a lane
  constexpr int VK = 64 / VL;           // keys of one
  constexpr int R = kRowTile;
  typedef uint32_t kw_t __attribute__((ext_vector_type(KS)));
  __shared__ __align__(16) uint8_t s_v[4][32 * D * 2];
  __shared__ float s_ml[4][64][2];
  __shared__ int64_t s_plan[8];
  Item it;
  if (!find_item<true, SPLIT_FIRST>(a, R, s_plan, parts_of<D, R * HEADS>(a), &it)) return;
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
  constexpr int G = 64 * KW;
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
  // V: a lane's block, and its key among the VK of a load: 16 lanes next to each other write 16 places
  const int block = lane % (D / 32);
  const int vkey = D == 128 ? (lane >> 4) * 2 + ((lane >> 2) & 1) + ((lane >> 3) & 1) * 8
                            : ((lane >> 1) & 1) + ((lane >> 2) & 1) * 2 + ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 8 +
                                  (lane >> 5) * 16;
  const int64_t codes = mxfp4_codes((int64_t)a.kv_heads * HEADS * D);
  const uint8_t* kc_at = a.k_rows + hk * (D / 2) + quad * (D / 8);
  const uint8_t* ks_at = a.k_rows + codes + hk * (D / 32) + quad * KS / 4;
  const uint8_t* vc_at = a.v_rows + hk * (D / 2) + block * 16;
  const uint8_t* vs_at = a.v_rows + codes + hk * (D / 32) + block;
  uint8_t* sv = s_v[wave];
  // Slot of the tile's key `lane`, kNoSlot past the end and for a key that no row sees: with one
  // token a tile (decoding) that is every hidden key, whose values then are zeros in the product.
  auto entry = [&](int base) {
    const int i = base + lane;
    const int j = span.key(i < i1 ? i : i0);
    Entry e = {0, -1, 0};
    if (i < i1 && (p_first != p_last || visible(a, p_first, j))) e = entry_of(a, it.s, (uint32_t)j);
    return e;
  };
  kw_t kc[4];
  v4u vc[VL];
  uint32_t ks[4], vs[VL];
  auto load_k = [&](uint32_t slot) {
#pragma unroll
    for (int t = 0; t < 4; t++) {
      const uint32_t sl = __shfl(slot, t * 16 + col);
      const uint64_t at = sl == kNoSlot ? 0 : (uint64_t)sl * a.k_row;
      kc[t] = *reinterpret_cast<const kw_t*>(kc_at + at);
      ks[t] = ks_at[at];
    }
  };
  auto load_v = [&](uint32_t slot) {
#pragma unroll
    for (int x = 0; x < VL; x++) {
      const uint32_t sl = __shfl(slot, x * VK + vkey);
      const uint64_t at = sl == kNoSlot ? 0 : (uint64_t)sl * a.v_row;
      const v4u y = *reinterpret_cast<const v4u*>(vc_at + at);
      const uint32_t z = vs_at[at];
      vc[x] = sl == kNoSlot ? v4u{0, 0, 0, 0} : y;
      vs[x] = sl == kNoSlot ? 127 : z;
    }
  };
  int base = i0 + kw * 64;
  Entry next_entry = entry(base + G);
  uint32_t slot = slot_from(a, entry(base)), slot_next = kNoSlot;
  if (base < i1) {
    load_k(slot);
    load_v(slot);
  }
  for (; base < i1; base += G) {
    f32x4 st[4] = {};
#pragma unroll
    for (int t = 0; t < 4; t++)
#pragma unroll
      for (int i = 0; i < KS; i++)
        st[t] = T::mfma16(__builtin_bit_cast(v8, mx_decode<kIsBf16<T>>(kc[t][i], mx_scale(ks[t]))), q[i], st[t]);
    const uint64_t there = __ballot(slot != kNoSlot);
    const bool more = base + G < i1;
    slot_next = slot_from(a, next_entry);
    next_entry = entry(base + 2 * G);
    if (more) load_k(slot_next);
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; e++) x[e] = st[e / 4][e % 4];
    // hidden keys: past the end, bad entries, and those that this row does not see
    const bool whole = there == ~0ull && (!a.causal || (span.key(base + 63) <= p_first &&
                                                        (a.window == 0 || p_last - span.key(base) < a.window)));
    if (!whole) {
      const uint64_t see = sees(a, span, there, p, base) >> (quad * 4);
      const uint32_t part2[2] = {(uint32_t)see, (uint32_t)(see >> 32)};
#pragma unroll
      for (int e = 0; e < 16; e++) x[e] = (part2[e / 8] >> (e % 8 / 4 * 16 + e % 4)) & 1 ? x[e] : -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 16; e++) top = fmaxf(top, x[e]);
    top = fmaxf(top, __shfl_xor(top, 16));
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
    for (int e = 0; e < 16; e++) {
      x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c, -zero));
      sum += x[e];
    }
    l += sum;  // this lane's keys; the quads are summed at the end
#pragma unroll
    for (int u = 0; u < 2; u++) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int y = u * VL / 2; y < (u + 1) * VL / 2; y++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          *reinterpret_cast<v4u*>(sv + few_place<D>((y - u * VL / 2) * VK + vkey, block * 4 + i)) =
              mx_decode<kIsBf16<T>>(vc[y][i], mx_scale(vs[y]));
      if (u == 1 && more) load_v(slot_next);
      f32x8 w;
#pragma unroll
      for (int e = 0; e < 8; e++) w[e] = x[u * 8 + e];
      const v8 wt = __builtin_convertvector(w, v8);  // the weight's one rounding, as the product's operand
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int d = 0; d < DT; d++) {
        s16x4 v[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
          const int key = t * 16 + quad * 4 + col / 4;
          v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4)(sv + few_place<D>(key, d * 2 + (col & 3) / 2) + (col & 1) * 8));
        }
        const v8 vt = __builtin_bit_cast(v8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        o[d] = T::mfma16(vt, wt, o[d]);
      }
    }
    slot = slot_next;
  }
  if (KW > 1) {  // the first wave of a head takes in the others', a lane its own places
    __builtin_amdgcn_wave_barrier();
    f32x4* so = reinterpret_cast<f32x4*>(sv);
    if (kw > 0) {
#pragma unroll
      for (int d = 0; d < DT; d++) so[d * 64 + lane] = o[d];
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
      for (int d = 0; d < DT; d++) o[d] = o[d] * keep + reinterpret_cast<const f32x4*>(s_v[from])[d * 64 + lane] * add;
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
    exact_row<T, D, D, Rows>(a, it.s, it.q.q0 + ta, ha, it.q.kv - it.q.m + ta, span, i0, i1, reinterpret_cast<float*>(sv),
                             oo, &mm, &ll);
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

// ---------------------------------------------------------------- tiles of 4-bit rows, as elements into LDS
// A tile's codes wait in registers while the tile before is computed, 16 bytes and a scale for a
// block of 32 elements, and are written to LDS as elements behind its products, by one wave for all four.
// 16 lanes next to each other write all banks.
template <class T, int D>
struct MxTiles {
  typedef MxRows<T, D, D> Rows;
  static constexpr bool kZeros = true;
  static constexpr int N = D == 128 ? 2 : 1;  // blocks of a lane: of K and V, or of one of them
  const uint8_t *codes_at[N], *scales_at[N];
  int key, block;
  bool is_v;  // N == 1
  v4u codes[N];
  uint32_t scales[N];
  __device__ __forceinline__ MxTiles(const AttendArgs& a, int hk) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  __device__ __forceinline__ void arrive(bool more, uint8_t* k, uint8_t* v) {
    if (!more) return;
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const v4u y = mx_decode<kIsBf16<T>>(codes[n][i], mx_scale(scales[n]));
        const int chunk = block * 4 + i;
        if (N == 2) *reinterpret_cast<v4u*>(n ? v + v_place(key, chunk) : k + k_place(key, chunk)) = y;
        else *reinterpret_cast<v4u*>(is_v ? v + v_place(key, chunk) : k + k_place(key, chunk)) = y;
      }
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
  v4u codes[N];
  uint32_t scales[N];
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
  __device__ __forceinline__ void arrive(bool more, uint8_t* to) {
    if (!more) return;
#pragma unroll
    for (int n = 0; n < N; n++) {
      int pair, key, b;
      if (!place(n, &pair, &key, &b)) continue;
#pragma unroll
      for (int i = 0; i < 4; i++)
        *reinterpret_cast<v4u*>(to + pair * kLatBlock + key * 128 + ((b * 4 + i) ^ lat_swizzle(key)) * 16) =
            mx_decode<kIsBf16<T>>(codes[n][i], mx_scale(scales[n]));
    }
  }
};

int tile_rows(const AttendArgs& a, int32_t head_dim) {
  const int64_t rows = a.max_q * a.group;
  if (head_dim == kLatDim) return rows <= 16 ? 16 : rows <= 32 ? 32 : kLatRows;
  return rows <= 2 * kRowTile ? kRowTile : kTileRows;
}

// KV heads of an item of few rows: as many as divide the heads.
int heads_of(const AttendArgs& a) { return a.kv_heads % 4 == 0 ? 4 : a.kv_heads % 2 == 0 ? 2 : 1; }

template <class T, int D, int HEADS>
hipError_t launch_few(AttendArgs a, int32_t num_cus, hipStream_t stream) {
  a.kv_heads /= HEADS;
  return launch_split<T, D, kRowTile, HEADS>({k_attend_mxfp4_few<T, D, HEADS, false>, k_attend_mxfp4_few<T, D, HEADS, true>}, a,
                                             num_cus, stream);
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
template <class T, int RB>
hipError_t launch_latent_few(const AttendArgs& a, int32_t num_cus, hipStream_t stream) {
  return launch_split<T, kLatValue, 16 * RB>({k_attend_latent_few<T, RB, MxLatent<T>, false>,
                                              k_attend_latent_few<T, RB, MxLatent<T>, true>}, a, num_cus, stream);
}

template <class T>
hipError_t launch_for(const AttendArgs& a, int32_t head_dim, int32_t num_cus, hipStream_t stream) {
  (void)hipGetLastError();
  if (head_dim == 64) return launch_heads<T, 64>(a, num_cus, stream);
  if (head_dim == 128) return launch_heads<T, 128>(a, num_cus, stream);
  const int R = tile_rows(a, head_dim);
  return R == 16   ? launch_latent_few<T, 1>(a, num_cus, stream)
         : R == 32 ? launch_latent_few<T, 2>(a, num_cus, stream)
                   : launch_split<T, kLatValue, kLatRows>(
                         {k_attend_latent<T, MxLatent<T>, false>, k_attend_latent<T, MxLatent<T>, true>}, a, num_cus,
                         stream);
}

}  // namespace

int64_t attend_mxfp4_workspace(const AttendArgs& args, int32_t head_dim, int32_t num_cus) {
  if (args.q_rows <= 0 || args.num_seqs <= 0) return 0;
  const int R = tile_rows(args, head_dim), heads = head_dim != kLatDim && R == kRowTile ? heads_of(args) : 1;
  AttendArgs a = args;
  a.kv_heads /= heads;
  const Plan p = plan(&a, R, head_dim, num_cus, heads);
  if (p.joins == 0) return 0;
  const int64_t floats = head_dim == 64    ? partial_floats<64>(R * heads)
                         : head_dim == 128 ? partial_floats<128>(R * heads)
                                           : partial_floats<kLatValue>(R);
  return a.slots * (4 * floats + (int64_t)sizeof(Part));
}

hipError_t launch_attend_mxfp4(const AttendArgs& a, int32_t dtype, int32_t head_dim, int32_t num_cus, hipStream_t stream) {
  if (a.q_rows <= 0 || a.num_seqs <= 0) return hipSuccess;
  return dtype == HC_BF16 ? launch_for<Bf16>(a, head_dim, num_cus, stream) : launch_for<F16>(a, head_dim, num_cus, stream);
}

}  // namespace hc
