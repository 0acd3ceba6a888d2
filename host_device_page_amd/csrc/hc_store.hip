// Rotary positions and the store of new tokens into a layer of the pool.
//
// Pair (x1, x2) of a token at position p turns by a = p * f: y1 = m (x1 cos a - x2 sin a),
// y2 = m (x2 cos a + x1 sin a).  The angle is needed as a fraction of a turn only, so f is
// kept as f / 2 pi in units of 2^-64 and p * f is one wrapping 64-bit product, whose top 32
// bits are the signed fraction in [-1/2, 1/2): exact for every position, where p * f in fp32
// is off by 0.06 radians at p = 10^6.
//
// The call reads each input element and writes each output element once, so memory bounds
// it (and the launch, for a decoding step's few tokens).  A workgroup takes a few tokens and
// a range of heads: first its sines and cosines into LDS, one per (token, pair) and shared by
// all its heads, then 16-byte vectors: a lane that rotates loads both vectors of its eight
// pairs (half layout) or the one that holds four (interleaved) and writes the same places,
// which is why queries may be rotated in place.
//
// Pairs of a rope of several axes take the position of their axis; everything else is the same, so that
// the axis is looked up in kernels of their own (AXES) only.
//
// A cache held in 4 bits (MX): a lane takes 16 bytes of keys or values, four lanes a block of 32
// elements and its scale, whose bits come from the largest magnitude's without a logarithm.  Rotated
// keys are computed in 64 bits and reach the 4-bit rounding unrounded: in fp32 one of a million would be
// on the wrong side of a border, half of its value off.
//
// Measured: 8192 tokens of 32 + 8 + 8 heads of 128, 201 MB, 45 us = 4.4 TB/s; 2048 tokens of a latent cache 19 us =
// 4.3 TB/s; 32 tokens 3.9 us, their heads over several workgroups each.
// In 4 bits: 8192 tokens 43 us, 177 MB at 4.1 TB/s, and 12 us to fetch them; 32 tokens 4.8 and 2.5 us.  Several axes: 8192
// tokens 46 us, 32 tokens 3.7.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hc_forward.h"
#include "hc_mxfp4.h"

namespace hc {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // tokens of a workgroup at most

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));

template <class V8>
__device__ __forceinline__ f32x8 widen(v4u x) {
  return __builtin_convertvector(__builtin_bit_cast(V8, x), f32x8);
}
template <class V8>
__device__ __forceinline__ v4u narrow(f32x8 x) {  // rounds to nearest, the one rounding of the rotation
  return __builtin_bit_cast(v4u, __builtin_convertvector(x, V8));
}

// A lane's eight elements of a head of keys (rotated: r is the vector's place in the rotated ones) or
// values into a row of 4 bits; `pair` sines and cosines of the token.
template <class V8>
__device__ __forceinline__ void store_mxfp4(const StoreArgs& a, const v4u* src, uint8_t* row, int heads_before, int dim,
                                            int x, int r, int rv, const double* s_cos, const double* s_sin) {
  const f32x8 u = widen<V8>(src[x]);
  float f[8];
  if (r < 0 || r >= rv) {
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] = u[j];
  } else if (a.rope.interleaved) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const double c = s_cos[r * 4 + j], s = s_sin[r * 4 + j];
      f[2 * j] = mx_beside((double)u[2 * j] * c - (double)u[2 * j + 1] * s);
      f[2 * j + 1] = mx_beside((double)u[2 * j + 1] * c + (double)u[2 * j] * s);
    }
  } else {  // the pair's other element is half a rotation away
    const bool first = r < rv / 2;
    const int p = first ? r : r - rv / 2;
    const f32x8 w = widen<V8>(src[first ? x + rv / 2 : x - rv / 2]);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const double c = s_cos[p * 8 + j], s = s_sin[p * 8 + j];
      f[j] = mx_beside((double)u[j] * c + (double)w[j] * (first ? -s : s));
    }
  }
  uint32_t top = 0;  // largest magnitude, as bits: NaN above infinity above all others
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const uint32_t y = __float_as_uint(f[j]) & 0x7fffffffu;
    top = y > top ? y : top;
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    const uint32_t y = __shfl_xor(top, d);
    top = y > top ? y : top;
  }
  const uint32_t byte = mx_scale_byte(top);
  mx_hold<__is_same(V8, bf16x8)>(f, byte);
  const int64_t at = (int64_t)heads_before * dim + x * 8;
  *reinterpret_cast<uint32_t*>(row + at / 2) = byte == 255 ? 0 : mx_encode(f, mx_scale(byte));
  if ((x & 3) == 0) row[mxfp4_codes((int64_t)a.kv_heads * dim) + at / kMxBlock] = (uint8_t)byte;
}

template <class V8, bool AXES, bool MX>
__global__ __launch_bounds__(kThreads) void k_store_tokens(StoreArgs a, int32_t tokens, int32_t splits) {
  __shared__ float s_cos[kTokens][HC_MAX_ROT_DIM / 2], s_sin[kTokens][HC_MAX_ROT_DIM / 2];
  __shared__ double s_cos64[MX ? kTokens : 1][HC_MAX_ROT_DIM / 2], s_sin64[MX ? kTokens : 1][HC_MAX_ROT_DIM / 2];
  __shared__ int64_t s_slot[kTokens];
  const int64_t t0 = (int64_t)(blockIdx.x / splits) * tokens;
  const int split = blockIdx.x % splits;
  const int count = a.n - t0 < tokens ? (int)(a.n - t0) : tokens;
  const int pairs = a.rope.rot_dim / 2;
  if ((int)threadIdx.x < count) {
    const int64_t slot = a.slots[t0 + threadIdx.x];
    const bool ok = slot >= 0 && slot < a.S;
    if (!ok && slot != -1 && split == 0) report_wrong<DeviceAtomic>(a.wrong, kWrongIndex, t0 + threadIdx.x);
    s_slot[threadIdx.x] = ok ? slot : -1;
  }
  for (int i = threadIdx.x; i < count * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    const int64_t position = a.positions[AXES ? a.rope.axis[p] * a.n + t0 + t : t0 + t];
    const uint64_t turn = (uint64_t)position * a.rope.turns[p];
    if constexpr (MX) {
      double s, c;
      sincospi((double)(int64_t)turn * 0x1p-63, &s, &c);
      s_cos64[t][p] = c * a.rope.magnitude64;
      s_sin64[t][p] = s * a.rope.magnitude64;
      s_cos[t][p] = (float)s_cos64[t][p];
      s_sin[t][p] = (float)s_sin64[t][p];
    } else {
      const float half = (float)(int32_t)(turn >> 32) * 0x1p-31f;  // angle / pi, in [-1, 1)
      float s, c;
      sincospif(half, &s, &c);
      s_cos[t][p] = c * a.rope.magnitude;
      s_sin[t][p] = s * a.rope.magnitude;
    }
  }
  __syncthreads();
  // The heads of queries, keys and values in one row of work, cut evenly over the splits.
  const int d_vecs = a.head_dim / 8, v_vecs = a.value_dim / 8;
  const int q_work = a.q_heads * d_vecs, k_work = a.kv_heads * d_vecs, v_work = a.kv_heads * v_vecs;
  const int all = q_work + k_work + v_work;
  // (MX: in whole blocks of four vectors, whose lanes work together)
  constexpr int U = MX ? 4 : 1;
  const int w0 = (int)((int64_t)(all / U) * split / splits) * U, w1 = (int)((int64_t)(all / U) * (split + 1) / splits) * U;
  const int r0 = a.rope.rot_offset / 8, rv = a.rope.rot_dim / 8;
  for (int i = threadIdx.x; i < count * (w1 - w0); i += kThreads) {
    const int t = i / (w1 - w0);
    int w = w0 + i - t * (w1 - w0);
    const int64_t slot = s_slot[t];
    if (slot < 0) continue;
    const bool is_q = w < q_work, is_v = w >= q_work + k_work;
    w -= is_q ? 0 : (is_v ? q_work + k_work : q_work);
    const int vecs = is_v ? v_vecs : d_vecs;
    const int h = w / vecs, x = w - h * vecs;
    const int64_t* in = is_q ? a.q_stride : (is_v ? a.v_stride : a.k_stride);
    const uint8_t* from = (is_q ? a.q : (is_v ? a.v : a.k)) + 2 * ((t0 + t) * in[0] + h * in[1]);
    if constexpr (MX) {
      if (!is_q) {
        const int dim = is_v ? a.value_dim : a.head_dim;
        uint8_t* row = (is_v ? a.v_rows : a.k_rows) + slot * mxfp4_row((int64_t)a.kv_heads * dim);
        store_mxfp4<V8>(a, reinterpret_cast<const v4u*>(from), row, h, dim, x, is_v ? -1 : x - r0, rv, s_cos64[t],
                        s_sin64[t]);
        continue;
      }
    }
    uint8_t* to = is_q ? a.q_out + 2 * ((t0 + t) * a.q_out_stride[0] + h * a.q_out_stride[1])
                       : (is_v ? a.v_rows + 2 * ((slot * a.kv_heads + h) * (int64_t)a.value_dim)
                               : a.k_rows + 2 * ((slot * a.kv_heads + h) * (int64_t)a.head_dim));
    const v4u* src = reinterpret_cast<const v4u*>(from);
    v4u* dst = reinterpret_cast<v4u*>(to);
    const int r = x - r0;
    if (is_v || r < 0 || r >= rv) {
      dst[x] = src[x];
    } else if (a.rope.interleaved) {
      const f32x8 u = widen<V8>(src[x]);
      f32x8 y;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float c = s_cos[t][r * 4 + j], s = s_sin[t][r * 4 + j];
        y[2 * j] = u[2 * j] * c - u[2 * j + 1] * s;
        y[2 * j + 1] = u[2 * j + 1] * c + u[2 * j] * s;
      }
      dst[x] = narrow<V8>(y);
    } else if (r < rv / 2) {  // the lane of the first half writes both
      const f32x8 u1 = widen<V8>(src[x]), u2 = widen<V8>(src[x + rv / 2]);
      f32x8 y1, y2;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float c = s_cos[t][r * 8 + j], s = s_sin[t][r * 8 + j];
        y1[j] = u1[j] * c - u2[j] * s;
        y2[j] = u2[j] * c + u1[j] * s;
      }
      dst[x] = narrow<V8>(y1);
      dst[x + rv / 2] = narrow<V8>(y2);
    }
  }
}

// Eight elements a lane: 4 bytes of codes in, 16 bytes out, neighbours next to each other on both sides.  Written bytes
// bound it, four times those that are read.  A workgroup takes a few tokens, and a lane up to four of their
// vectors at once.
constexpr int kFetch = 4;
template <bool BF16>
__global__ __launch_bounds__(kThreads) void k_fetch_mxfp4(FetchArgs a, int32_t tokens) {
  const int d_vecs = a.kv_heads * (a.head_dim / 8), all = d_vecs + a.kv_heads * (a.value_dim / 8);
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int count = a.n - t0 < tokens ? (int)(a.n - t0) : tokens;
  const int64_t k_row = mxfp4_row((int64_t)a.kv_heads * a.head_dim), v_row = mxfp4_row((int64_t)a.kv_heads * a.value_dim);
  for (int i0 = threadIdx.x; i0 < count * all; i0 += kThreads * kFetch) {
    uint32_t codes[kFetch], scale[kFetch];
    uint8_t* to[kFetch];
#pragma unroll
    for (int n = 0; n < kFetch; n++) {
      to[n] = nullptr;
      const int i = i0 + n * kThreads;
      if (i >= count * all) continue;
      const int t = i / all;
      int w = i - t * all;
      const int64_t slot = a.slots[t0 + t];
      if (slot < 0 || slot >= a.S) {
        if (w == 0 && slot != -1) report_wrong<DeviceAtomic>(a.wrong, kWrongIndex, t0 + t);
        continue;
      }
      const bool is_v = w >= d_vecs;
      w -= is_v ? d_vecs : 0;
      const int dim = is_v ? a.value_dim : a.head_dim, h = w / (dim / 8), x = w - h * (dim / 8);
      const uint8_t* row = is_v ? a.v_rows + slot * v_row : a.k_rows + slot * k_row;
      codes[n] = reinterpret_cast<const uint32_t*>(row)[w];
      scale[n] = row[mxfp4_codes((int64_t)a.kv_heads * dim) + w / 4];
      to[n] = (is_v ? a.v + 2 * ((t0 + t) * a.v_stride[0] + h * a.v_stride[1])
                    : a.k + 2 * ((t0 + t) * a.k_stride[0] + h * a.k_stride[1])) + 16 * x;
    }
#pragma unroll
    for (int n = 0; n < kFetch; n++)
      if (to[n]) *reinterpret_cast<v4u*>(to[n]) = mx_decode<BF16>(codes[n], mx_scale(scale[n]));
  }
}

template <class V8>
void (*store_kernel(bool axes, bool mxfp4))(StoreArgs, int32_t, int32_t) {
  if (mxfp4) return axes ? k_store_tokens<V8, true, true> : k_store_tokens<V8, false, true>;
  return axes ? k_store_tokens<V8, true, false> : k_store_tokens<V8, false, false>;
}

}  // namespace

hipError_t launch_store(const StoreArgs& a, int32_t dtype, bool mxfp4, int32_t num_cus, hipStream_t stream) {
  if (a.n <= 0) return hipSuccess;
  // Few tokens: one a workgroup, and its heads over up to 8 workgroups.  Of 32 + 8 + 8 heads of 128, in a graph: one
  // token with its heads over 1, 8 and 16 workgroups 4.25, 3.23 and 3.18 us, 32 tokens 4.50, 3.32 and 3.52; four
  // tokens a workgroup for one 4.00 for 3.32 us at 32 tokens, 12.9 for 12.5 at 2048, 35.2 for 35.8 at 8192.
  const int64_t fill = (int64_t)num_cus * 4;
  const int32_t tokens = a.n >= fill * kTokens ? kTokens : 1;
  const int64_t groups = (a.n + tokens - 1) / tokens;
  int32_t splits = 1;
  while (splits < 8 && groups * splits * 2 <= fill) splits *= 2;
  if (groups * splits > 0x7fffffff) return hipErrorInvalidValue;
  (void)hipGetLastError();
  const bool axes = a.rope.rot_dim > 0 && a.rope.axes > 1;
  auto kernel = dtype == HC_BF16 ? store_kernel<bf16x8>(axes, mxfp4) : store_kernel<f16x8>(axes, mxfp4);
  kernel<<<dim3((unsigned)(groups * splits)), kThreads, 0, stream>>>(a, tokens, splits);
  return hipGetLastError();
}

hipError_t launch_fetch_mxfp4(const FetchArgs& a, int32_t dtype, int32_t num_cus, hipStream_t stream) {
  if (a.n <= 0) return hipSuccess;
  const int32_t tokens = a.n >= (int64_t)num_cus * 4 * kTokens ? kTokens : 1;
  const int64_t groups = (a.n + tokens - 1) / tokens;
  if (groups > 0x7fffffff) return hipErrorInvalidValue;
  (void)hipGetLastError();
  (dtype == HC_BF16 ? k_fetch_mxfp4<true> : k_fetch_mxfp4<false>)<<<dim3((unsigned)groups), kThreads, 0, stream>>>(a, tokens);
  return hipGetLastError();
}

}  // namespace hc
