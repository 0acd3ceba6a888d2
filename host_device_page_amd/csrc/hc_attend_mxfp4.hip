// Attention over a cache held in 4 bits: the formulas and the list of work items are hc_attend.hip's, the
// rows hc_mxfp4.h's.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "hc_attend.h"
#include "hc_mxfp4.h"

namespace hc {
namespace {

template <class T>
constexpr bool kIsBf16 = false;
template <>
constexpr bool kIsBf16<Bf16> = true;

// Keys and values of a token's KV head in 4 bits, rounded to T's elements.
template <class T, int DK, int DV>
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
        : Head(a.k_rows + (int64_t)slot * a.k_row, a.kv_heads, hk) {}
  };
  struct Value : Head {  // DK == DV, or a latent cache's only head
    __device__ __forceinline__ Value(const AttendArgs& a, uint32_t slot, int hk)
        : Head(a.v_rows + (int64_t)slot * a.v_row, a.kv_heads, hk) {}
  };
};

// Row tiles of 16, a wave a row, key by key.
constexpr int kRows = 16;

template <class T, int DK, int DV>
__global__ __launch_bounds__(256) void k_attend_mxfp4(AttendArgs a) {
  typedef typename T::elem elem;
  __shared__ float s_q[4][DK];
  __shared__ int64_t s_plan[8];
  Item it;
  if (!find_item<false, false>(a, kRows, s_plan, nullptr, &it)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int x = wave; x < kRows; x += 4) {
    const int64_t r = (int64_t)it.tile * kRows + x;
    if (r >= (int64_t)it.q.m * a.group) return;
    const int tok = (int)(r / a.group), h = it.hk * a.group + (int)(r - (int64_t)tok * a.group);
    const int p = it.q.kv - it.q.m + tok;
    const Span span = span_of(a, it.q.kv, p, p);
    float o[DV / 64], m, l;
    exact_row<T, DK, DV, MxRows<T, DK, DV>>(a, it.s, it.q.q0 + tok, h, p, span, 0, span.n, s_q[wave], o, &m, &l);
    elem* op = reinterpret_cast<elem*>(a.out) + (it.q.q0 + tok) * a.out_stride[0] + h * a.out_stride[1];
    for (int c = 0; c < DV / 64; c++) op[c * 64 + lane] = (elem)(l == 0.f ? 0.f : o[c] / l);
    if (a.lse && lane == 0) a.lse[(it.q.q0 + tok) * a.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <class T>
void (*kernel_for(int32_t head_dim))(AttendArgs) {
  return head_dim == 64 ? k_attend_mxfp4<T, 64, 64> : head_dim == 128 ? k_attend_mxfp4<T, 128, 128> : k_attend_mxfp4<T, 576, 512>;
}

}  // namespace

int64_t attend_mxfp4_workspace(const AttendArgs&, int32_t, int32_t) { return 0; }

hipError_t launch_attend_mxfp4(const AttendArgs& args, int32_t dtype, int32_t head_dim, int32_t, hipStream_t stream) {
  AttendArgs a = args;
  if (a.q_rows <= 0 || a.num_seqs <= 0) return hipSuccess;
  a.target = 1;
  a.min_split = a.max_kv + 1;
  const int64_t items = (a.q_rows * a.group / kRows + (a.num_seqs < a.q_rows ? a.num_seqs : a.q_rows)) * a.kv_heads;
  if (items > 0x7fffffff) return hipErrorInvalidValue;
  (void)hipGetLastError();
  (dtype == HC_BF16 ? kernel_for<Bf16>(head_dim) : kernel_for<F16>(head_dim))<<<dim3((unsigned)items), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace hc
