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

#include "hc_forward.h"

namespace hc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  typedef __bf16 elem;
  typedef bf16x8 v8;
};
struct F16 {
  typedef _Float16 elem;
  typedef f16x8 v8;
};

__device__ __forceinline__ void flag(int32_t* err, int bit, int64_t pos) {
  atomicOr(err, bit);
  atomicMin(reinterpret_cast<unsigned long long*>(err + 2), (unsigned long long)pos);
}

// A sequence's rows and cached tokens; ok only when they are inside the call's bounds.
struct Seq {
  int64_t q0, kv;
  int64_t m;
  bool ok;
};
__device__ __forceinline__ Seq sequence(const AttendArgs& a, int64_t s) {
  Seq r;
  r.q0 = a.q_start ? a.q_start[s] : s;
  const int64_t q1 = a.q_start ? a.q_start[s + 1] : s + 1;
  r.kv = a.kv_len[s];
  r.m = q1 - r.q0;
  r.ok = r.q0 >= 0 && r.m >= 0 && q1 <= a.q_rows && r.m <= a.max_q && r.kv >= 0 && r.kv <= a.max_kv;
  return r;
}

// The keys that rows at positions [p0, p1] can see, as a list: i < sk is key i, others key
// lo + i - sk.
struct Span {
  int64_t lo, sk, n;
  __device__ __forceinline__ int64_t key(int64_t i) const { return i < sk ? i : lo + (i - sk); }
};
__device__ __forceinline__ Span span_of(const AttendArgs& a, int64_t kv, int64_t p0, int64_t p1) {
  Span s;
  int64_t hi = kv;
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
__device__ __forceinline__ bool visible(const AttendArgs& a, int64_t p, int64_t j) {
  if (!a.causal) return true;
  return j <= p && (a.window == 0 || p - j < a.window || j < a.sinks);
}

// Slot of key j, -1 for a bad table entry.
__device__ __forceinline__ int64_t slot_of(const AttendArgs& a, int64_t s, int64_t j) {
  const int64_t e = j / a.entry;
  const int64_t t = a.table[s * a.table_stride + e];
  if (t < 0 || t >= a.S / a.entry) {
    flag(a.err, kErrIndex, s * a.table_stride + e);
    return -1;
  }
  return t * a.entry + (j - e * a.entry);
}

// One wave per (row, head): lanes take keys for the scores and dims for the sum.
template <class T, int DK, int DV>
__global__ __launch_bounds__(256) void k_attend_rows(AttendArgs a) {
  __shared__ float s_q[4][DK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x == 0)
    for (int64_t s = threadIdx.x; s < a.num_seqs; s += blockDim.x)
      if (!sequence(a, s).ok) flag(a.err, kErrLengths, s);
  const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
  const int64_t row = unit / a.q_heads;
  const int h = (int)(unit - row * a.q_heads);
  if (row >= a.q_rows) return;
  int64_t s = row;
  if (a.q_start) {  // the last sequence that starts at or before the row
    int64_t l = 0, r = a.num_seqs;
    while (r - l > 1) {
      const int64_t mid = (l + r) / 2;
      if (a.q_start[mid] <= row) l = mid; else r = mid;
    }
    s = l;
  }
  if (s >= a.num_seqs) return;
  const Seq q = sequence(a, s);
  if (!q.ok || row < q.q0 || row >= q.q0 + q.m) return;
  const int64_t p = q.kv - q.m + (row - q.q0);
  const Span span = span_of(a, q.kv, p, p);
  const int hk = h / a.group;
  typedef typename T::elem elem;
  const elem* qp = reinterpret_cast<const elem*>(a.q) + row * a.q_stride[0] + h * a.q_stride[1];
  for (int i = lane; i < DK; i += 64) s_q[wave][i] = (float)qp[i];
  __builtin_amdgcn_wave_barrier();
  constexpr int ND = DV / 64;
  float o[ND] = {}, m = -INFINITY, l = 0.f;
  const float scale = a.scale * kLog2e;
  for (int64_t i0 = 0; i0 < span.n; i0 += 64) {
    const int64_t i = i0 + lane;
    float x = -INFINITY;
    int64_t slot = -1;
    if (i < span.n) {
      const int64_t j = span.key(i);
      if (visible(a, p, j)) slot = slot_of(a, s, j);
    }
    if (slot >= 0) {
      const v4u* kp = reinterpret_cast<const v4u*>(a.k_rows + 2 * (slot * a.k_row + (int64_t)hk * DK));
      x = 0.f;
      for (int v = 0; v < DK / 8; v++) {
        const f32x8 kv = __builtin_convertvector(__builtin_bit_cast(typename T::v8, kp[v]), f32x8);
#pragma unroll
        for (int c = 0; c < 8; c++) x += kv[c] * s_q[wave][v * 8 + c];
      }
      x *= scale;
    }
    float top = x;
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    // a score that is NaN is not a maximum, and makes the sums below NaN
    const float next = fmaxf(m, top);
    const float base = next == -INFINITY ? 0.f : next;
    const float keep = exp2f(m - base), e = slot >= 0 ? exp2f(x - base) : 0.f;
    m = next;
    float sum = e;
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    l = l * keep + sum;
#pragma unroll
    for (int c = 0; c < ND; c++) o[c] *= keep;
    uint64_t todo = __ballot(slot >= 0);
    while (todo) {
      const int j = __builtin_ctzll(todo);
      todo &= todo - 1;
      const float pj = __shfl(e, j);
      const int64_t sj = __shfl(slot, j);
      const elem* vp = reinterpret_cast<const elem*>(a.v_rows) + sj * a.v_row + (int64_t)hk * (DK == DV ? DV : 0);
#pragma unroll
      for (int c = 0; c < ND; c++) o[c] += pj * (float)vp[c * 64 + lane];
    }
  }
  elem* op = reinterpret_cast<elem*>(a.out) + row * a.out_stride[0] + h * a.out_stride[1];
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < ND; c++) op[c * 64 + lane] = (elem)(l == 0.f ? 0.f : o[c] * inv);
  if (a.lse && lane == 0) a.lse[row * a.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <class T>
hipError_t launch_for(const AttendArgs& a, int32_t head_dim, hipStream_t stream) {
  const int64_t units = a.q_rows * a.q_heads;
  const dim3 grid((unsigned)((units + 3) / 4));
  (void)hipGetLastError();
  if (head_dim == 64) k_attend_rows<T, 64, 64><<<grid, 256, 0, stream>>>(a);
  else if (head_dim == 128) k_attend_rows<T, 128, 128><<<grid, 256, 0, stream>>>(a);
  else k_attend_rows<T, 576, 512><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t attend_workspace(const AttendArgs&, int32_t, int32_t) { return 0; }

hipError_t launch_attend(const AttendArgs& a, int32_t dtype, int32_t head_dim, int32_t, hipStream_t stream) {
  if (a.q_rows <= 0 || a.num_seqs <= 0) return hipSuccess;
  return dtype == HC_BF16 ? launch_for<Bf16>(a, head_dim, stream) : launch_for<F16>(a, head_dim, stream);
}

}  // namespace hc
