// Refusals of the attention calls for pools that no test can allocate: the entry points themselves, over a made-up pool, under
// AddressSanitizer + UBSan.  No device is asked and nothing is launched: what the library's other files do is stood in for below.
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "hc_forward.h"

#define CHECK(cond)                                                      \
  do {                                                                   \
    if (!(cond)) {                                                       \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
      exit(1);                                                           \
    }                                                                    \
  } while (0)

static hc::Geom geom;
static uint64_t bases[2 * HC_MAX_SUBBUFS];

extern "C" int roctxRangePushA(const char*) { return 0; }
extern "C" int roctxRangePop() { return 0; }
extern "C" const char* hipGetErrorString(hipError_t) { return ""; }

namespace hc {
int set_error(int code, const char*, ...) { return code; }
void pool_view(const hc_pool*, PoolView* out) { *out = {&geom, bases, nullptr, 0, 256, true}; }
int pool_forward(hc_pool* pool, void*, PoolView* out) {
  pool_view(pool, out);
  return HC_OK;
}
int BufferCheck::buffer(const void*, int64_t, int32_t, bool, const char*) { return HC_OK; }
hipError_t launch_store(const StoreArgs&, int32_t, bool, int32_t, hipStream_t) { return hipSuccess; }
hipError_t launch_fetch_mxfp4(const FetchArgs&, int32_t, int32_t, hipStream_t) { return hipSuccess; }
hipError_t launch_extend_pages(const ExtendArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_copy_pages(const Geom&, const int64_t*, const int64_t*, int64_t, WrongWord*, int32_t, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_fork_pages(const Geom&, const ForkArgs&, WrongWord*, int32_t, hipStream_t) { return hipSuccess; }
int64_t pages_workspace(const Geom&) { return 0; }
hipError_t launch_free_pages(const Geom&, const PageTable&, int64_t*, int64_t*, void*, WrongWord*, int32_t, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_compact_pages(const Geom&, const PageTable&, int64_t*, int64_t, int64_t*, void*, WrongWord*, int32_t,
                                hipStream_t) {
  return hipSuccess;
}
static int launches = 0;
int64_t attend_workspace(const AttendArgs&, int32_t, int32_t) { return 0; }
int64_t attend_mxfp4_workspace(const AttendArgs&, int32_t, int32_t) { return 0; }
static hipError_t launched(const AttendArgs& a) {
  // what the kernels rely on: a slot fits 32 bits and is not the one that stands for none
  CHECK(a.entries * a.entry <= 0xffffffffll);
  launches++;
  return hipSuccess;
}
hipError_t launch_attend(const AttendArgs& a, int32_t, int32_t, int32_t, hipStream_t) { return launched(a); }
hipError_t launch_attend_mxfp4(const AttendArgs& a, int32_t, int32_t, int32_t, hipStream_t) { return launched(a); }
}  // namespace hc

static void slots_beyond_32_bits() {
  const int64_t limit = (int64_t)1 << 32;
  static int64_t lists[16];
  int taken = 0;
  for (int64_t S : {limit / 2, limit - 64, limit - 1, limit, limit + 64, 2 * limit, (int64_t)1 << 40})
    for (int mxfp4 = 0; mxfp4 < 2; mxfp4++)
      for (int entry : {1, 64}) {
        memset(&geom, 0, sizeof(geom));
        geom.nsub = 2, geom.L = 1, geom.P = 64, geom.S = S;
        for (int b = 0; b < 2; b++) geom.sub[b].gran = HC_TOKEN_ROWS, geom.sub[b].elem = mxfp4 ? 48 : 128;
        hc_attend_desc d;
        memset(&d, 0, sizeof(d));
        d.dtype = HC_BF16, d.q_heads = d.kv_heads = 1, d.head_dim = d.value_dim = 64;
        d.entry_tokens = entry, d.causal = 1, d.scale = 1.f;
        d.num_seqs = d.q_rows = d.max_q = d.table_width = 1, d.max_kv = entry;
        d.q = lists, d.out = lists + 2, d.kv_len = lists + 4, d.table = lists + 6;
        d.q_stride[0] = d.q_stride[1] = d.out_stride[0] = d.out_stride[1] = 64;
        static uint16_t heads[2][64];
        d.q = heads[0], d.out = heads[1];
        int64_t bytes = -1;
        hc_pool* pool = reinterpret_cast<hc_pool*>(lists);
        const int want = S < limit ? HC_OK : HC_ERR_UNSUPPORTED;
        CHECK((mxfp4 ? hc_attend_mxfp4_workspace_bytes : hc_attend_workspace_bytes)(pool, &d, &bytes) == want);
        CHECK((mxfp4 ? hc_attend_mxfp4 : hc_attend)(pool, &d, nullptr) == want);
        taken += want == HC_OK;
      }
  CHECK(taken == 12 && hc::launches == taken);
}

int main() {
  slots_beyond_32_bits();
  printf("attend_host ok\n");
  return 0;
}
