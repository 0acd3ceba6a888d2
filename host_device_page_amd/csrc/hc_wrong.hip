// Takes what kernels reported, of the transfers (error bits, then the smallest position) and of the
// forward pass, for hc_pool_sync.
#include <hip/hip_runtime.h>

#include "hc_internal.h"
#include "hc_wrong.h"

namespace hc {
namespace {

__global__ void k_take_reports(int32_t* err, WrongWord* words, TakenReports* out) {
  out->bits = (unsigned)atomicExch(err, 0);
  out->position = DeviceAtomic::exchange(reinterpret_cast<WrongWord*>(err + 2), kNothing);
  take_wrong<DeviceAtomic>(words, out->words);
}

}  // namespace

hipError_t launch_take_reports(int32_t* err, WrongWord* words, TakenReports* out, hipStream_t stream) {
  (void)hipGetLastError();
  k_take_reports<<<dim3(1), 1, 0, stream>>>(err, words, out);
  return hipGetLastError();
}

}  // namespace hc
