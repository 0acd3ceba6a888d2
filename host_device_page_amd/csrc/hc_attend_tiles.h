// Attention of many rows over K and V of heads of 64 and 128, whatever the cache holds.
#pragma once

#include "hc_attend.h"

namespace hc {
namespace {

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
constexpr int kTileKeys = 64;

// Source: how a tile of keys and values gets into LDS, and where their 16-byte chunks lie there.
//   load(a, slot, k, v)    starts on the tile whose key `lane` is in `slot`, into LDS k and v
//   step(s, k, v)          beside the s-th of the four products of weights and values: may put a part of it there
//   arrive(first, k, v)    what load started is in LDS, behind the four steps but for the first tile
//   kZeros                 values of keys that are not there arrive as zeros
//   Rows                   one row of the cache, for exact_row
template <class T, int D, class Source, bool SPLIT_FIRST>
__global__ __launch_bounds__(256, 2) void k_attend_tiles(AttendArgs a) {
  constexpr int R = kTileRows;
  typedef typename T::v8 v8;
  typedef typename T::elem elem;
  constexpr int KS = D / 16;                    // product steps over the head
  constexpr int DT = D / 32;                    // 32-dim tiles of the output
  constexpr int CH = D / 8;                     // 16-byte chunks of a row
  constexpr int W = 4;                          // waves
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
  Source source(a, it.hk, lane, wave);
  f32x16 o[DT] = {};
  float m = -INFINITY, l = 0.f;
  Entry next_entry = entry(i0 + kTileKeys);
  uint32_t slot = slot_from(a, entry(i0));
  if (i0 < i1) source.load(a, slot, s_k[0], s_v[0]);
  source.arrive(true, s_k[0], s_v[0]);
  __syncthreads();
  int buf = 0;
  for (int base = i0; base < i1; base += kTileKeys) {
    const uint64_t there = __ballot(slot != kNoSlot);
    slot = slot_from(a, next_entry);
    next_entry = entry(base + 2 * kTileKeys);
    if (base + kTileKeys < i1) source.load(a, slot, s_k[buf ^ 1], s_v[buf ^ 1]);
    if (!Source::kZeros && there != ~0ull) {  // what was fetched in place of no key must not reach the product: its value is zero
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
        const v8 k = *reinterpret_cast<const v8*>(s_k[buf] + Source::k_place(u * 32 + col, i * 2 + half));
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
      source.step(s, s_k[buf ^ 1], s_v[buf ^ 1]);
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
              (lds_s16x4)(s_v[buf] + Source::v_place(key, at / 8) + (at & 4) * 2));
        }
        const v8 vt = __builtin_bit_cast(v8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        o[d] = T::mfma32(vt, wt, o[d]);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    buf ^= 1;
    source.arrive(false, s_k[buf], s_v[buf]);
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
    exact_row<T, D, D, typename Source::Rows>(a, it.s, it.q.q0 + ta, ha, before + ta, span, i0, i1, s_q, oo, &mm, &ll);
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

}  // namespace
}  // namespace hc
