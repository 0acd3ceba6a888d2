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
// Measured: 8192 tokens of 32 + 8 + 8 heads of 128, 201 MB, 45 us = 4.4 TB/s; 2048 tokens of a latent cache 19 us =
// 4.3 TB/s; 32 tokens 3.9 us, their heads over several workgroups each.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hc_forward.h"

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

template <class V8>
__global__ __launch_bounds__(kThreads) void k_store_tokens(StoreArgs a, int32_t tokens, int32_t splits) {
  __shared__ float s_cos[kTokens][HC_MAX_ROT_DIM / 2], s_sin[kTokens][HC_MAX_ROT_DIM / 2];
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
    const uint64_t turn = (uint64_t)a.positions[t0 + t] * a.rope.turns[p];
    const float half = (float)(int32_t)(turn >> 32) * 0x1p-31f;  // angle / pi, in [-1, 1)
    float s, c;
    sincospif(half, &s, &c);
    s_cos[t][p] = c * a.rope.magnitude;
    s_sin[t][p] = s * a.rope.magnitude;
  }
  __syncthreads();
  // The heads of queries, keys and values in one row of work, cut evenly over the splits.
  const int d_vecs = a.head_dim / 8, v_vecs = a.value_dim / 8;
  const int q_work = a.q_heads * d_vecs, k_work = a.kv_heads * d_vecs, v_work = a.kv_heads * v_vecs;
  const int all = q_work + k_work + v_work;
  const int w0 = (int)((int64_t)all * split / splits), w1 = (int)((int64_t)all * (split + 1) / splits);
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

}  // namespace

hipError_t launch_store(const StoreArgs& a, int32_t dtype, int32_t num_cus, hipStream_t stream) {
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
  auto kernel = dtype == HC_BF16 ? k_store_tokens<bf16x8> : k_store_tokens<f16x8>;
  kernel<<<dim3((unsigned)(groups * splits)), kThreads, 0, stream>>>(a, tokens, splits);
  return hipGetLastError();
}

}  // namespace hc
