// Attention over a latent cache, one row of 576 dims key and value at once, whatever the cache holds.
#pragma once

#include "hc_attend.h"

namespace hc {
namespace {

// ---------------------------------------------------------------- a latent cache: one row is key and value
// 576 dims of a key against every head of a token, 512 of them its value, so a tile of 64 keys (72 KiB,
// two of them in LDS) is read into LDS once for both products, and its four waves cut the work
// without doing any twice: scores by keys, values by dims, 128 a wave.  The maxima of the waves' keys
// and then the weights go through LDS: three barriers a tile.  Measured: 32 sequences up to 6000 tokens and 16 heads
// 32 us and 5 us to join; a chunk of 512 behind 3988 with 32 heads 190 to 193 us = 784 to 796 TFLOP/s.
constexpr int kLatKeys = 64;
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

// Source, in the kernels below: how a tile of keys gets into LDS.
//   load(a, slot, to)    starts on the tile whose key `lane` is in `slot`, into LDS `to`
//   step(s, to)          beside the s-th of the four products of weights and values of many rows: may put a part there
//   arrive(first, to)    what load started is in LDS, behind the four steps but for the first tile
//   kZeros               keys that are not there arrive as zeros
//   Rows                 one row of the cache, for exact_row

// What was fetched in place of no key must not reach the product.
__device__ __forceinline__ void latent_clear(uint64_t there, uint8_t* tile) {
  for (int x = threadIdx.x; x < kLatTile / 16; x += 256)
    if (!((there >> (x % (kLatBlock / 16) / 8)) & 1)) *reinterpret_cast<v4u*>(tile + x * 16) = v4u{0, 0, 0, 0};
  __syncthreads();
}

// Rows that came out NaN, but for those whose sum of weights is NaN, shared out over the waves; s_sum: four parts of
// R rows' sums, s_q: kLatDim floats of this wave's.
template <class T, class Rows>
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
    exact_row<T, kLatDim, kLatValue, Rows>(a, t.it.s, row, h, t.before + tok, t.span, t.i0, t.i1, s_q, o, &m, &l);
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
template <class T, int RB, class Source, bool SPLIT_FIRST>
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
  Source source(a);
  if (t.i0 < t.i1) source.load(a, slot, s_k);
  source.arrive(true, s_k);
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
    if (base + kLatKeys < t.i1) source.load(a, slot, s_k + (kLatTile - off));
    if (!Source::kZeros && there != ~0ull) latent_clear(there, s_k + off);
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
      source.arrive(false, s_k + off);
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
  latent_again<T, typename Source::Rows>(a, t, s_nan, &s_sum[0][0], R, reinterpret_cast<float*>(s_k) + wave * kLatDim, part_o, part_ml);
}

// 64 rows: chunks, and many heads.  Bound by the matrix cores and LDS: 240 KiB are read from it for 2176
// cycles of products.  Scores in 32 x 32 products, wave (i, j) taking rows 32 i, whose queries stay in
// registers, and keys 32 j.

template <class T, class Source, bool SPLIT_FIRST>
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
  Source source(a);
  if (t.i0 < t.i1) source.load(a, slot, s_k);
  source.arrive(true, s_k);
  if (threadIdx.x < 2) s_nan[threadIdx.x] = 0;
  __syncthreads();
  int off = 0;
  float x[16], top[2];  // scores of a tile, hidden ones -infinity, and its maxima
  auto score = [&](int base) {
    const uint64_t there = __ballot(slot != kNoSlot);
    slot = slot_from(a, next_entry);
    next_entry = t.entry(a, base + 2 * kLatKeys);
    if (base + kLatKeys < t.i1) source.load(a, slot, s_k + (kLatTile - off));
    if (!Source::kZeros && there != ~0ull) latent_clear(there, s_k + off);
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
        source.step(s, s_k + (kLatTile - off));
#pragma unroll
        for (int d = 0; d < DT; d++) {
          o[0][d] = T::mfma32(vf[s & 1][d], w[s & 1][0], o[0][d]);
          o[1][d] = T::mfma32(vf[s & 1][d], w[s & 1][1], o[1][d]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      off = kLatTile - off;
      source.arrive(false, s_k + off);
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
  latent_again<T, typename Source::Rows>(a, t, s_nan, &s_sum[0][0], kLatRows, reinterpret_cast<float*>(s_k) + wave * kLatDim, part_o, part_ml);
}

}  // namespace
}  // namespace hc
