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

#include "hc_attend_latent.h"
#include "hc_attend_tiles.h"

namespace hc {
namespace {

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
      exact_row<T, D, D, ElementRows<T, D, D>>(a, it.s, it.q.q0 + rt, rh, it.q.kv - it.q.m + rt, span, i0, i1, s_q[wave], oo, &mm, &ll);
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

// ---------------------------------------------------------------- tiles of elements, straight from memory into LDS
// 64 keys of heads of D.
// Which chunk of a K row lies at a place of it, and back: 16 rows' same chunk in 16 places.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int chunk) {
  return chunk ^ (D == 128 ? row & 15 : (row >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int tile_k_place(int row, int chunk) {
  return row * D * 2 + k_chunk<D>(row, chunk) * 16;
}
// Of a V row: four rows' 32 dims side by side.
template <int D>
__device__ __forceinline__ int v_chunk(int row, int chunk) {
  return chunk ^ (D == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2);
}
template <int D>
__device__ __forceinline__ int tile_v_place(int row, int chunk) {
  return row * D * 2 + v_chunk<D>(row, chunk) * 16;
}

template <class T, int D>
struct ElementTiles {
  typedef ElementRows<T, D, D> Rows;
  static constexpr bool kZeros = false;
  static constexpr int CH = D / 8;   // 16-byte chunks of a row
  static constexpr int W = 4;        // waves
  static constexpr int LD = kTileKeys * CH / (64 * W);  // loads of a wave, K and V each
  // One instruction carries 64 chunks; the swizzle is in which chunk of its row a lane fetches, the same
  // one in every instruction.  Rows of K and V are equally far apart, so a key's lane works out where its
  // rows are once and the lanes that fetch them only add their own part.
  static constexpr int RL = 64 / CH;  // rows of an instruction
  const int wave, from;               // a lane's first row, the next W RL on
  const uint8_t *const kl, *const vl;
  __device__ __forceinline__ ElementTiles(const AttendArgs& a, int hk, int lane, int w)
      : wave(w), from(w * RL + lane / CH), kl(a.k_rows + 2 * (int64_t)hk * D + k_chunk<D>(from, lane % CH) * 16),
        vl(a.v_rows + 2 * (int64_t)hk * D + v_chunk<D>(from, lane % CH) * 16) {}
  __device__ __forceinline__ void load(const AttendArgs& a, uint32_t slot, const uint8_t* k, const uint8_t* v) const {
    const uint64_t row = slot == kNoSlot ? 0 : (uint64_t)slot * (2 * a.k_row);
    const uint32_t lo = (uint32_t)row, hi = (uint32_t)(row >> 32);
#pragma unroll
    for (int x = 0; x < LD; x++) {
      const int key = x * W * RL + from;
      const uint64_t at = (uint64_t)__shfl(hi, key) << 32 | __shfl(lo, key);
      lds_load(kl + at, lds_offset(k + (x * W + wave) * 1024));
      lds_load(vl + at, lds_offset(v + (x * W + wave) * 1024));
    }
  }
  __device__ __forceinline__ void step(int, const uint8_t*, const uint8_t*) {}
  __device__ __forceinline__ void arrive(bool, const uint8_t*, const uint8_t*) { lds_arrived(); }
  static __device__ __forceinline__ int k_place(int row, int chunk) { return tile_k_place<D>(row, chunk); }
  static __device__ __forceinline__ int v_place(int row, int chunk) { return tile_v_place<D>(row, chunk); }
};

// 64 keys of a latent cache.
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

template <class T>
struct ElementLatent {
  typedef ElementRows<T, kLatDim, kLatValue> Rows;
  static constexpr bool kZeros = false;
  __device__ __forceinline__ explicit ElementLatent(const AttendArgs&) {}
  __device__ __forceinline__ void load(const AttendArgs& a, uint32_t slot, const uint8_t* to) { latent_load(a, slot, to); }
  __device__ __forceinline__ void step(int, const uint8_t*) {}
  __device__ __forceinline__ void arrive(bool, const uint8_t*) { lds_arrived(); }
};

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

template <class T, int RB>
hipError_t launch_latent_few(const AttendArgs& a, int32_t num_cus, hipStream_t stream) {
  return launch_split<T, kLatValue, 16 * RB>({k_attend_latent_few<T, RB, ElementLatent<T>, false>,
                                               k_attend_latent_few<T, RB, ElementLatent<T>, true>}, a,
                                             num_cus, stream);
}
template <class T, int D>
hipError_t launch_decode(const AttendArgs& a, int32_t num_cus, hipStream_t stream) {
  return launch_split<T, D, kRowTile>({k_attend_decode<T, D, false>, k_attend_decode<T, D, true>}, a, num_cus, stream);
}
template <class T, int D>
hipError_t launch_tiles(const AttendArgs& a, int32_t num_cus, hipStream_t stream) {
  return launch_split<T, D, kTileRows>({k_attend_tiles<T, D, ElementTiles<T, D>, false>,
                                        k_attend_tiles<T, D, ElementTiles<T, D>, true>}, a, num_cus, stream);
}

template <class T>
hipError_t launch_for(const AttendArgs& a, int32_t head_dim, int32_t num_cus, hipStream_t stream) {
  (void)hipGetLastError();
  const int R = tile_rows(a, head_dim);
  if (head_dim == kLatDim)
    return R == 16   ? launch_latent_few<T, 1>(a, num_cus, stream)
           : R == 32 ? launch_latent_few<T, 2>(a, num_cus, stream)
                     : launch_split<T, kLatValue, kLatRows>({k_attend_latent<T, ElementLatent<T>, false>,
                                                             k_attend_latent<T, ElementLatent<T>, true>}, a,
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
