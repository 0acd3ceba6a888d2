// Arguments of the forward-pass kernels (hc_store.hip, hc_attend.hip, hc_attend_mxfp4.hip, hc_pages.hip,
// hc_extend.hip) as hc_forward.cpp hands them over, checked.  Plain values only, so a launch recorded into
// a graph carries everything it needs.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "hc.h"
#include "hc_internal.h"
#include "hc_wrong.h"

namespace hc {

// The turn per position of each rotated pair, as a fraction of 2^64: position * turns,
// modulo 2^64, is the angle's fraction of a full turn, exact but for the rounding of
// `turns` itself (position * 2^-65 of a turn).
struct RopeTable {
  uint64_t turns[HC_MAX_ROT_DIM / 2];
  float magnitude;
  int32_t rot_dim, rot_offset, interleaved;  // rot_dim 0: nothing is rotated
  double magnitude64;
  int32_t axes;                              // of positions: `axis` is read where there are several
  uint8_t axis[HC_MAX_ROT_DIM / 2];          // whose position a pair takes
};

struct StoreArgs {
  RopeTable rope;
  const int64_t* slots;
  const int64_t* positions;
  const uint8_t *q, *k, *v;
  uint8_t* q_out;
  uint8_t *k_rows, *v_rows;  // the layer's sub-buffers
  WrongWord* wrong;  // the pool's words of what is found wrong
  int64_t n, S;
  int64_t q_stride[2], q_out_stride[2], k_stride[2], v_stride[2];  // elements
  int32_t q_heads, kv_heads, head_dim, value_dim;
};
hipError_t launch_store(const StoreArgs& a, int32_t dtype, bool mxfp4, int32_t num_cus, hipStream_t stream);

struct FetchArgs {
  const int64_t* slots;
  const uint8_t *k_rows, *v_rows;  // the layer's sub-buffers
  uint8_t *k, *v;
  WrongWord* wrong;
  int64_t n, S;
  int64_t k_stride[2], v_stride[2];  // elements
  int32_t kv_heads, head_dim, value_dim;
};
hipError_t launch_fetch_mxfp4(const FetchArgs& a, int32_t dtype, int32_t num_cus, hipStream_t stream);

// Attention keeps slots in 32 bits, the last of them for "no slot".  (2^32 rows of one head of 64 in 4 bits, the smallest, are
// 192 GiB, which a layer can have.)
constexpr int64_t kMaxAttendSlots = 0xffffffff;
struct AttendArgs {
  const uint8_t* q;
  uint8_t* out;
  float* lse;
  const int64_t *q_start, *kv_len, *table;
  const uint8_t *k_rows, *v_rows;
  WrongWord* wrong;  // the pool's words of what is found wrong
  float* work;  // partial results of split sequences
  int64_t q_stride[2], out_stride[2], table_width, table_stride;
  int64_t k_row, v_row;  // elements from token to token in the layer's rows
  int64_t num_seqs, q_rows, max_q, max_kv;
  int32_t window, sinks;
  int64_t entries;                     // table entries of the pool: S / entry
  int64_t target, min_split, slots;    // how the work is split (set by launch_attend); places of partial results
  uint32_t entry_magic, entry_shift;   // j / entry == (j * magic) >> shift for j < 2^31
  int32_t q_heads, kv_heads, group, entry, causal;
  int32_t join_parts;                  // workgroups of the joining launch to a row tile
  float scale;
};
// The same over rows in 4 bits: k_row and v_row are bytes.
hipError_t launch_attend_mxfp4(const AttendArgs& a, int32_t dtype, int32_t head_dim, int32_t num_cus,
                               hipStream_t stream);
int64_t attend_mxfp4_workspace(const AttendArgs& a, int32_t head_dim, int32_t num_cus);
// Bytes of workspace that launch_attend needs for these sizes.
int64_t attend_workspace(const AttendArgs& a, int32_t head_dim, int32_t num_cus);
hipError_t launch_attend(const AttendArgs& a, int32_t dtype, int32_t head_dim, int32_t num_cus, hipStream_t stream);

struct PageTable {
  const int64_t* entries;
  const int64_t* lens;
  int64_t rows, width, stride;
};
struct ForkArgs {
  PageTable table;
  const int64_t* parents;
  const int64_t* free_pages;
  int64_t n, n_free;
  int64_t* out;
  int64_t out_stride;
  int64_t* used;
};
struct ExtendArgs {
  PageTable table;   // entries are written too
  const int64_t *added, *free_pages, *first_free;
  int64_t n_free, pages;
  int64_t *kv_len, *q_start, *slots, *positions, *used;
  int64_t room;
  WrongWord* wrong;
  int32_t P;
};
hipError_t launch_extend_pages(const ExtendArgs& a, hipStream_t stream);
hipError_t launch_copy_pages(const Geom& g, const int64_t* src, const int64_t* dst, int64_t n, WrongWord* wrong,
                             int32_t num_cus, hipStream_t stream);
hipError_t launch_fork_pages(const Geom& g, const ForkArgs& a, WrongWord* wrong, int32_t num_cus, hipStream_t stream);
int64_t pages_workspace(const Geom& g);
hipError_t launch_free_pages(const Geom& g, const PageTable& t, int64_t* pages, int64_t* count, void* work,
                             WrongWord* wrong, int32_t num_cus, hipStream_t stream);
hipError_t launch_compact_pages(const Geom& g, const PageTable& t, int64_t* out, int64_t out_stride, int64_t* count,
                                void* work, WrongWord* wrong, int32_t num_cus, hipStream_t stream);

}  // namespace hc
