// Entry points of the forward-pass operators on a pool's device side: argument checks on the
// host, then one or a few launches on the caller's stream.  Nothing here allocates device
// memory or waits, so every call can be recorded into a graph.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <new>

#include <rocprofiler-sdk-roctx/roctx.h>

#include "hc_extent.h"
#include "hc_forward.h"

using hc::PoolView;
using hc::set_error;

struct hc_rope {
  hc::RopeTable table;
  double frequency[HC_MAX_ROT_DIM / 2];
  double magnitude;
};

namespace {

struct TraceRange {
  explicit TraceRange(const char* name) { roctxRangePushA(name); }
  ~TraceRange() { roctxRangePop(); }
  TraceRange(const TraceRange&) = delete;
  TraceRange& operator=(const TraceRange&) = delete;
};

#define HC_TRY(call)              \
  do {                            \
    const int rc_ = (call);       \
    if (rc_ != HC_OK) return rc_; \
  } while (0)

int launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return HC_OK;
  return set_error(HC_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
}

constexpr int64_t kMaxRows = (int64_t)1 << 31;      // rows, sequences and tokens of one call
constexpr int64_t kMaxTokens = (int64_t)1 << 30;    // of an attention call: 32-bit positions
constexpr int64_t kMaxStride = (int64_t)1 << 40;    // elements; the extents themselves are checked too

int check_extent(const void* q, int64_t bytes, int32_t align, bool host_ok, hc::BufferCheck& check, const char* what) {
  if (bytes == hc::kTooFar) return set_error(HC_ERR_INVALID, "%s: its strides reach past every allocation", what);
  return check.buffer(q, bytes, align, host_ok, what);
}

int check_tensor(const void* q, const int64_t* stride, int64_t n, int64_t heads, int64_t dim, bool writes,
                 hc::BufferCheck& check, const char* what) {
  const int64_t count[2] = {n, heads};
  for (int k = 0; k < 2; k++) {
    if (count[k] <= 1) continue;  // no step is taken
    if (stride[k] < 0 || stride[k] > kMaxStride)
      return set_error(HC_ERR_INVALID, "%s: stride %lld out of range", what, (long long)stride[k]);
    if (stride[k] % 8 != 0)
      return set_error(HC_ERR_UNSUPPORTED, "%s: strides must be multiples of 8 elements", what);
  }
  if (writes && !hc::rows_apart(stride, n, heads, dim)) return set_error(HC_ERR_INVALID, "%s: its rows overlap", what);
  return check_extent(q, hc::tensor_bytes(stride, n, heads, dim), 16, false, check, what);
}

int check_list(const int64_t* q, int64_t n, hc::BufferCheck& check, const char* what) {
  return check.buffer(q, n * (int64_t)sizeof(int64_t), 8, true, what);
}

// Written lists and counters stay in device memory.
int check_out_list(const int64_t* q, int64_t n, hc::BufferCheck& check, const char* what) {
  return check.buffer(q, n * (int64_t)sizeof(int64_t), 8, false, what);
}

struct Span {
  const void* at;
  int64_t bytes;
};
bool overlap(const Span& a, const Span& b) { return hc::overlap(a.at, a.bytes, b.at, b.bytes); }
Span span_of(const hc::Tensor& t) { return {t.at, t.bytes()}; }

// Sub-buffer b holds token rows of exactly `elems` 2-byte elements.
int check_rows(const PoolView& v, int b, int64_t elems, const char* what) {
  if (b >= v.geom->nsub || v.geom->sub[b].gran != HC_TOKEN_ROWS)
    return set_error(HC_ERR_INVALID, "the pool's sub-buffer %d does not hold %s token rows", b, what);
  if (v.geom->sub[b].elem != 2 * elems)
    return set_error(HC_ERR_INVALID, "%s rows of %lld elements, the pool's are %lld bytes", what, (long long)elems,
                     (long long)v.geom->sub[b].elem);
  return HC_OK;
}

int check_layer(const PoolView& v, int32_t layer, int32_t dtype) {
  if (layer < 0 || layer >= v.geom->L) return set_error(HC_ERR_INVALID, "layer %d out of range [0, %d)", layer, v.geom->L);
  if (dtype != HC_BF16 && dtype != HC_F16) return set_error(HC_ERR_INVALID, "unknown dtype %d", dtype);
  return HC_OK;
}

uint8_t* layer_rows(const PoolView& v, int b, int32_t layer) {
  return (uint8_t*)(uintptr_t)v.bases[(size_t)b * v.geom->L + layer];
}

Span layer_span(const PoolView& v, int b, int32_t layer) {
  return {layer_rows(v, b, layer), v.geom->S * v.geom->sub[b].elem};
}

}  // namespace

extern "C" {

int hc_rope_create(const hc_rope_desc* d, hc_rope** out) {
  if (!out) return set_error(HC_ERR_INVALID, "out is null");
  *out = nullptr;
  if (!d) return set_error(HC_ERR_INVALID, "desc is null");
  if (d->rot_dim <= 0 || d->rot_dim > HC_MAX_ROT_DIM)
    return set_error(HC_ERR_INVALID, "rot_dim must be in [16, %d]", HC_MAX_ROT_DIM);
  if (d->rot_dim % 16 != 0) return set_error(HC_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16");
  if (d->rot_offset < 0) return set_error(HC_ERR_INVALID, "rot_offset must be >= 0");
  if (d->rot_offset % 8 != 0) return set_error(HC_ERR_UNSUPPORTED, "rot_offset must be a multiple of 8");
  if (d->scaling < HC_ROPE_NONE || d->scaling > HC_ROPE_YARN) return set_error(HC_ERR_INVALID, "unknown scaling");
  if (!(d->base > 1.0) || !isfinite(d->base)) return set_error(HC_ERR_INVALID, "base must be above 1 and finite");
  if (d->scaling != HC_ROPE_NONE && (!(d->factor > 0.0) || !isfinite(d->factor)))
    return set_error(HC_ERR_INVALID, "factor must be above 0 and finite");
  if (!(d->magnitude >= 0.0) || !isfinite(d->magnitude))
    return set_error(HC_ERR_INVALID, "magnitude must be >= 0 and finite");
  if (d->scaling == HC_ROPE_LLAMA3 &&
      (!(d->low_freq_factor > 0.0) || !(d->high_freq_factor > d->low_freq_factor) || !isfinite(d->high_freq_factor)))
    return set_error(HC_ERR_INVALID, "0 < low_freq_factor < high_freq_factor is needed");
  if (d->scaling == HC_ROPE_YARN &&
      (!(d->beta_slow > 0.0) || !(d->beta_fast >= d->beta_slow) || !isfinite(d->beta_fast)))
    return set_error(HC_ERR_INVALID, "0 < beta_slow <= beta_fast is needed");
  if ((d->scaling == HC_ROPE_LLAMA3 || d->scaling == HC_ROPE_YARN) && d->original_context <= 0)
    return set_error(HC_ERR_INVALID, "original_context must be above 0");
  hc_rope* r = new (std::nothrow) hc_rope();
  if (!r) return set_error(HC_ERR_NOMEM, "rope allocation failed");
  const double pi2 = 6.283185307179586476925286766559;
  const int pairs = d->rot_dim / 2;
  double lo = 0.0, hi = 0.0;
  r->magnitude = d->magnitude > 0.0 ? d->magnitude : 1.0;
  if (d->scaling == HC_ROPE_YARN) {
    auto pair_of = [&](double turns) {
      return pairs * log((double)d->original_context / (turns * pi2)) / log(d->base);
    };
    lo = fmax(floor(pair_of(d->beta_fast)), 0.0);
    hi = fmin(ceil(pair_of(d->beta_slow)), (double)(d->rot_dim - 1));
    if (d->magnitude == 0.0) r->magnitude = 0.1 * log(d->factor) + 1.0;
  }
  for (int i = 0; i < pairs; i++) {
    const double f0 = exp(-log(d->base) * (2.0 * i / d->rot_dim));
    double keep = 1.0;  // share of the unscaled frequency
    if (d->scaling == HC_ROPE_LINEAR) {
      keep = 0.0;
    } else if (d->scaling == HC_ROPE_LLAMA3) {
      const double turns = (double)d->original_context * f0 / pi2;
      keep = (turns - d->low_freq_factor) / (d->high_freq_factor - d->low_freq_factor);
    } else if (d->scaling == HC_ROPE_YARN) {
      keep = 1.0 - (i - lo) / fmax(hi - lo, 0.001);
    }
    keep = fmin(fmax(keep, 0.0), 1.0);
    const double f = d->scaling == HC_ROPE_NONE ? f0 : f0 * keep + f0 / d->factor * (1.0 - keep);
    r->frequency[i] = f;
    // f / 2 pi in units of 2^-64, modulo a turn; long double has the 64 bits
    long double turn = (long double)f / 6.283185307179586476925286766559L;
    turn -= floorl(turn);
    const long double scaled = turn * 18446744073709551616.0L;
    r->table.turns[i] = scaled >= 18446744073709551615.0L ? 0 : (uint64_t)(scaled + 0.5L);
  }
  r->table.magnitude = (float)r->magnitude;
  r->table.rot_dim = d->rot_dim;
  r->table.rot_offset = d->rot_offset;
  r->table.interleaved = d->interleaved != 0;
  *out = r;
  return HC_OK;
}

int hc_rope_destroy(hc_rope* r) {
  delete r;
  return HC_OK;
}

int hc_rope_frequencies(const hc_rope* r, double* f, double* magnitude) {
  if (!r || !f || !magnitude) return set_error(HC_ERR_INVALID, "null argument");
  memcpy(f, r->frequency, sizeof(double) * (size_t)(r->table.rot_dim / 2));
  *magnitude = r->magnitude;
  return HC_OK;
}

int hc_store_tokens(hc_pool* pool, const hc_store_desc* d, void* stream) {
  if (!pool || !d) return set_error(HC_ERR_INVALID, "null argument");
  TraceRange range("hc_store_tokens");
  PoolView v;
  hc::pool_view(pool, &v);
  HC_TRY(check_layer(v, d->layer, d->dtype));
  if (d->n < 0 || d->n >= kMaxRows) return set_error(HC_ERR_INVALID, "n must be in [0, 2^31)");
  if (d->q_heads < 0 || d->kv_heads <= 0 || d->head_dim <= 0 || d->value_dim < 0)
    return set_error(HC_ERR_INVALID, "bad head counts or sizes");
  if (d->head_dim % 8 != 0 || d->value_dim % 8 != 0)
    return set_error(HC_ERR_UNSUPPORTED, "head_dim and value_dim must be multiples of 8");
  if ((int64_t)d->q_heads * d->head_dim > (1 << 20))
    return set_error(HC_ERR_UNSUPPORTED, "q_heads * head_dim above 2^20");
  if (d->q_heads == 0 && (d->q || d->q_out)) return set_error(HC_ERR_INVALID, "queries given with q_heads 0");
  HC_TRY(check_rows(v, 0, (int64_t)d->kv_heads * d->head_dim, "key"));
  if (d->value_dim > 0) HC_TRY(check_rows(v, 1, (int64_t)d->kv_heads * d->value_dim, "value"));
  if (d->value_dim == 0 && d->v) return set_error(HC_ERR_INVALID, "values given with value_dim 0");
  if (d->rope && d->rope->table.rot_offset + d->rope->table.rot_dim > d->head_dim)
    return set_error(HC_ERR_INVALID, "the rotated elements [%d, %d) are not inside a head of %d",
                     d->rope->table.rot_offset, d->rope->table.rot_offset + d->rope->table.rot_dim, d->head_dim);
  HC_TRY(hc::pool_forward(pool, stream, &v));
  hc::BufferCheck check(v.device);
  if (d->n == 0) return HC_OK;
  HC_TRY(check_list(d->slots, d->n, check, "slots"));
  if (d->rope) HC_TRY(check_list(d->positions, d->n, check, "positions"));
  HC_TRY(check_tensor(d->k, d->k_stride, d->n, d->kv_heads, d->head_dim, false, check, "k"));
  if (d->value_dim > 0)
    HC_TRY(check_tensor(d->v, d->v_stride, d->n, d->kv_heads, d->value_dim, false, check, "v"));
  if (d->q_heads > 0) {
    HC_TRY(check_tensor(d->q, d->q_stride, d->n, d->q_heads, d->head_dim, false, check, "q"));
    HC_TRY(check_tensor(d->q_out, d->q_out_stride, d->n, d->q_heads, d->head_dim, true, check, "q_out"));
    if (d->q_out == d->q && ((d->n > 1 && d->q_out_stride[0] != d->q_stride[0]) ||
                             (d->q_heads > 1 && d->q_out_stride[1] != d->q_stride[1])))
      return set_error(HC_ERR_INVALID, "q_out in place of q needs q's strides");
  }
  const hc::Tensor q = {d->q, {d->q_stride[0], d->q_stride[1]}, d->n, d->q_heads, d->head_dim};
  const hc::Tensor q_out = {d->q_out, {d->q_out_stride[0], d->q_out_stride[1]}, d->n, d->q_heads, d->head_dim};
  const hc::Tensor k = {d->k, {d->k_stride[0], d->k_stride[1]}, d->n, d->kv_heads, d->head_dim};
  const hc::Tensor v_in = {d->v, {d->v_stride[0], d->v_stride[1]}, d->n, d->value_dim > 0 ? d->kv_heads : 0,
                           d->value_dim};
  const Span slots = {d->slots, 8 * d->n}, positions = {d->positions, d->rope ? 8 * d->n : 0};
  if ((q_out.at != q.at && share(q_out, q)) || share(q_out, k) || share(q_out, v_in) ||
      overlap(span_of(q_out), slots) || overlap(span_of(q_out), positions))
    return set_error(HC_ERR_INVALID, "q_out overlaps what is read");
  for (int b = 0; b < (d->value_dim > 0 ? 2 : 1); b++)
    for (const Span& x : {span_of(q), span_of(q_out), span_of(k), span_of(v_in), slots, positions})
      if (overlap(x, layer_span(v, b, d->layer)))
        return set_error(HC_ERR_INVALID, "the call's buffers must not overlap the layer's rows");
  hc::StoreArgs a;
  memset(&a, 0, sizeof(a));
  if (d->rope) a.rope = d->rope->table;
  a.slots = d->slots;
  a.positions = d->positions;
  a.q = (const uint8_t*)d->q;
  a.k = (const uint8_t*)d->k;
  a.v = (const uint8_t*)d->v;
  a.q_out = (uint8_t*)d->q_out;
  a.k_rows = layer_rows(v, 0, d->layer);
  a.v_rows = d->value_dim > 0 ? layer_rows(v, 1, d->layer) : nullptr;
  a.wrong = v.wrong;
  a.n = d->n;
  a.S = v.geom->S;
  for (int k = 0; k < 2; k++) {
    a.q_stride[k] = d->q_stride[k];
    a.q_out_stride[k] = d->q_out_stride[k];
    a.k_stride[k] = d->k_stride[k];
    a.v_stride[k] = d->v_stride[k];
  }
  a.q_heads = d->q_heads;
  a.kv_heads = d->kv_heads;
  a.head_dim = d->head_dim;
  a.value_dim = d->value_dim;
  return launched(hc::launch_store(a, d->dtype, v.num_cus, (hipStream_t)stream), "store");
}

}  // extern "C"

namespace {

// The checks of sizes, and the kernel arguments that follow from them.
int attend_sizes(const PoolView& v, const hc_attend_desc* d, hc::AttendArgs* a) {
  HC_TRY(check_layer(v, d->layer, d->dtype));
  if (d->kv_heads <= 0 || d->q_heads <= 0 || d->q_heads % d->kv_heads != 0)
    return set_error(HC_ERR_INVALID, "q_heads %d is not a multiple of kv_heads %d", d->q_heads, d->kv_heads);
  if (d->q_heads / d->kv_heads > 128) return set_error(HC_ERR_UNSUPPORTED, "more than 128 query heads per KV head");
  if (d->q_heads > 65536) return set_error(HC_ERR_UNSUPPORTED, "more than 65536 query heads");
  const bool latent = d->value_in_key != 0;
  if (latent ? !(d->head_dim == 576 && d->value_dim == 512 && d->kv_heads == 1)
             : !(d->head_dim == d->value_dim && (d->head_dim == 64 || d->head_dim == 128)))
    return set_error(HC_ERR_UNSUPPORTED,
                     "head_dim / value_dim %d / %d with %d KV heads: 64 / 64, 128 / 128, or 576 / 512 with "
                     "value_in_key and one KV head",
                     d->head_dim, d->value_dim, d->kv_heads);
  HC_TRY(check_rows(v, 0, (int64_t)d->kv_heads * d->head_dim, "key"));
  if (!latent) HC_TRY(check_rows(v, 1, (int64_t)d->kv_heads * d->value_dim, "value"));
  if (d->entry_tokens != 1 && d->entry_tokens != v.geom->P)
    return set_error(HC_ERR_INVALID, "entry_tokens must be 1 or the pool's page_size %d", v.geom->P);
  if (!isfinite(d->scale)) return set_error(HC_ERR_INVALID, "scale must be finite");
  if (d->window < 0 || d->sinks < 0) return set_error(HC_ERR_INVALID, "window and sinks must be >= 0");
  if (d->window > 0 && !d->causal) return set_error(HC_ERR_INVALID, "a window needs causal");
  if (d->num_seqs < 0 || d->num_seqs > kMaxTokens || d->q_rows < 0 || d->q_rows > kMaxTokens || d->max_q < 0 ||
      d->max_q > kMaxTokens || d->max_kv < 0 || d->max_kv > kMaxTokens)
    return set_error(HC_ERR_INVALID, "num_seqs, q_rows, max_q and max_kv must be in [0, 2^30]");
  if (d->table_width < 0 || d->table_width >= kMaxRows || d->table_stride < 0 || d->table_stride > kMaxStride ||
      (d->num_seqs > 1 && d->table_stride < d->table_width))
    return set_error(HC_ERR_INVALID, "bad table_width or table_stride");
  if (d->max_kv > d->table_width * d->entry_tokens)
    return set_error(HC_ERR_INVALID, "max_kv %lld is more than a table row holds", (long long)d->max_kv);
  memset(a, 0, sizeof(*a));
  a->q_stride[0] = d->q_stride[0];
  a->q_stride[1] = d->q_stride[1];
  a->out_stride[0] = d->out_stride[0];
  a->out_stride[1] = d->out_stride[1];
  a->table_width = d->table_width;
  a->table_stride = d->table_stride;
  a->k_row = (int64_t)d->kv_heads * d->head_dim;
  a->v_row = latent ? a->k_row : (int64_t)d->kv_heads * d->value_dim;
  a->num_seqs = d->num_seqs;
  a->q_rows = d->q_rows;
  a->max_q = d->max_q < d->q_rows ? d->max_q : d->q_rows;
  a->max_kv = d->max_kv;
  // a window that covers every sequence hides nothing
  a->window = d->window < d->max_kv ? (int32_t)d->window : 0;
  a->sinks = a->window > 0 ? (int32_t)(d->sinks < d->max_kv ? d->sinks : d->max_kv) : 0;
  a->q_heads = d->q_heads;
  a->kv_heads = d->kv_heads;
  a->group = d->q_heads / d->kv_heads;
  a->entry = d->entry_tokens;
  a->entries = v.geom->S / d->entry_tokens;
  // with 2^shift >= 2^31 * entry, ceil(2^shift / entry) is below 2^32 and off by less than 1 / entry
  // over all j < 2^31
  a->entry_shift = 31;
  while (((int64_t)1 << (a->entry_shift - 31)) < a->entry) a->entry_shift++;
  a->entry_magic = (uint32_t)((((uint64_t)1 << a->entry_shift) + (uint64_t)a->entry - 1) / (uint64_t)a->entry);
  a->causal = d->causal != 0;
  a->scale = d->scale;
  return HC_OK;
}

}  // namespace

extern "C" {

int hc_attend_workspace_bytes(const hc_pool* pool, const hc_attend_desc* d, int64_t* out_bytes) {
  if (!pool || !d || !out_bytes) return set_error(HC_ERR_INVALID, "null argument");
  PoolView v;
  hc::pool_view(pool, &v);
  hc::AttendArgs a;
  HC_TRY(attend_sizes(v, d, &a));
  *out_bytes = hc::attend_workspace(a, d->head_dim, v.num_cus);
  return HC_OK;
}

int hc_attend(hc_pool* pool, const hc_attend_desc* d, void* stream) {
  if (!pool || !d) return set_error(HC_ERR_INVALID, "null argument");
  TraceRange range("hc_attend");
  PoolView v;
  hc::pool_view(pool, &v);
  hc::AttendArgs a;
  HC_TRY(attend_sizes(v, d, &a));
  HC_TRY(hc::pool_forward(pool, stream, &v));
  hc::BufferCheck check(v.device);
  if (d->q_rows == 0 || d->num_seqs == 0) return HC_OK;
  if (!d->q_start && d->q_rows < d->num_seqs)
    return set_error(HC_ERR_INVALID, "without q_start every sequence has a row: q_rows is below num_seqs");
  HC_TRY(check_tensor(d->q, d->q_stride, d->q_rows, d->q_heads, d->head_dim, false, check, "q"));
  HC_TRY(check_tensor(d->out, d->out_stride, d->q_rows, d->q_heads, d->value_dim, true, check, "out"));
  HC_TRY(check.buffer(d->lse, d->lse ? 4 * d->q_rows * d->q_heads : 0, 4, false, "lse"));
  if (d->q_start) HC_TRY(check_list(d->q_start, d->num_seqs + 1, check, "q_start"));
  HC_TRY(check_list(d->kv_len, d->num_seqs, check, "kv_len"));
  HC_TRY(check_extent(d->table, hc::table_bytes(d->num_seqs, d->table_width, d->table_stride), 8, true, check, "table"));
  const int64_t work = hc::attend_workspace(a, d->head_dim, v.num_cus);
  if (work > 0) {
    if (d->workspace_bytes < work)
      return set_error(HC_ERR_INVALID, "workspace_bytes %lld below the %lld that are needed",
                       (long long)d->workspace_bytes, (long long)work);
    HC_TRY(check.buffer(d->workspace, work, 16, false, "workspace"));
  }
  const hc::Tensor q = {d->q, {d->q_stride[0], d->q_stride[1]}, d->q_rows, d->q_heads, d->head_dim};
  const hc::Tensor out = {d->out, {d->out_stride[0], d->out_stride[1]}, d->q_rows, d->q_heads, d->value_dim};
  if (share(q, out)) return set_error(HC_ERR_INVALID, "out must not overlap q");
  const Span writes[] = {span_of(out), {d->lse, d->lse ? 4 * d->q_rows * d->q_heads : 0}, {d->workspace, work}};
  const Span reads[] = {span_of(q),
                        {d->q_start, d->q_start ? 8 * (d->num_seqs + 1) : 0},
                        {d->kv_len, 8 * d->num_seqs},
                        {d->table, hc::table_bytes(d->num_seqs, d->table_width, d->table_stride)},
                        layer_span(v, 0, d->layer),
                        layer_span(v, d->value_in_key ? 0 : 1, d->layer)};
  for (int w = 0; w < 3; w++) {
    for (int r = w == 0 ? 1 : 0; r < 6; r++)  // out and q are compared above
      if (overlap(writes[w], reads[r]))
        return set_error(HC_ERR_INVALID, "out, lse and the workspace must not overlap what is read");
    for (int o = 0; o < w; o++)
      if (overlap(writes[w], writes[o]))
        return set_error(HC_ERR_INVALID, "out, lse and the workspace must not overlap each other");
  }
  a.q = (const uint8_t*)d->q;
  a.out = (uint8_t*)d->out;
  a.lse = d->lse;
  a.q_start = d->q_start;
  a.kv_len = d->kv_len;
  a.table = d->table;
  a.k_rows = layer_rows(v, 0, d->layer);
  a.v_rows = layer_rows(v, d->value_in_key ? 0 : 1, d->layer);
  a.wrong = v.wrong;
  a.work = (float*)d->workspace;
  return launched(hc::launch_attend(a, d->dtype, d->head_dim, v.num_cus, (hipStream_t)stream), "attention");
}

}  // extern "C"

namespace {

int page_pool(const PoolView& v) {
  if (!v.pages) return set_error(HC_ERR_INVALID, "the pool's device_slots are not whole pages");
  if (v.geom->S / v.geom->P >= kMaxRows) return set_error(HC_ERR_UNSUPPORTED, "more than 2^31 pages");
  return HC_OK;
}

int table_sizes(int64_t rows, int64_t width, int64_t stride) {
  if (rows < 0 || rows >= kMaxRows || width < 0 || width >= kMaxRows)
    return set_error(HC_ERR_INVALID, "table_rows and table_width must be in [0, 2^31)");
  if (stride < 0 || stride > kMaxStride || (rows > 1 && stride < width))
    return set_error(HC_ERR_INVALID, "table_stride is below table_width");
  return HC_OK;
}

int check_table(const int64_t* table, const int64_t* lens, int64_t rows, int64_t width, int64_t stride,
                hc::BufferCheck& check) {
  HC_TRY(check_extent(table, hc::table_bytes(rows, width, stride), 8, true, check, "table"));
  return check_list(lens, rows, check, "lens");
}

// The workspace, apart from the call's other buffers.
int check_work(const PoolView& v, const void* work, int64_t bytes, hc::BufferCheck& check,
               std::initializer_list<Span> others) {
  const int64_t need = hc::pages_workspace(*v.geom);
  if (bytes < need)
    return set_error(HC_ERR_INVALID, "workspace_bytes %lld below the %lld that are needed", (long long)bytes,
                     (long long)need);
  HC_TRY(check.buffer(work, need, 16, false, "workspace"));
  for (const Span& o : others)
    if (overlap({work, need}, o)) return set_error(HC_ERR_INVALID, "the workspace overlaps another buffer");
  return HC_OK;
}

}  // namespace

extern "C" {

int hc_copy_pages(hc_pool* pool, const int64_t* src, const int64_t* dst, int64_t n, void* stream) {
  if (!pool) return set_error(HC_ERR_INVALID, "pool is null");
  TraceRange range("hc_copy_pages");
  PoolView v;
  hc::pool_view(pool, &v);
  HC_TRY(page_pool(v));
  if (n < 0 || n >= kMaxRows) return set_error(HC_ERR_INVALID, "n must be in [0, 2^31)");
  HC_TRY(hc::pool_forward(pool, stream, &v));
  hc::BufferCheck check(v.device);
  HC_TRY(check_list(src, n, check, "src"));
  HC_TRY(check_list(dst, n, check, "dst"));
  return launched(hc::launch_copy_pages(*v.geom, src, dst, n, v.wrong, v.num_cus, (hipStream_t)stream), "page copy");
}

int hc_fork_pages(hc_pool* pool, const int64_t* table, int64_t table_rows, int64_t table_width, int64_t table_stride,
                  const int64_t* lens, const int64_t* parents, int64_t n, const int64_t* free_pages, int64_t n_free,
                  int64_t* out_table, int64_t out_stride, int64_t* used, void* stream) {
  if (!pool) return set_error(HC_ERR_INVALID, "pool is null");
  TraceRange range("hc_fork_pages");
  PoolView v;
  hc::pool_view(pool, &v);
  HC_TRY(page_pool(v));
  HC_TRY(table_sizes(table_rows, table_width, table_stride));
  HC_TRY(table_sizes(n, table_width, out_stride));
  if (n_free < 0 || n_free >= kMaxRows) return set_error(HC_ERR_INVALID, "n_free must be in [0, 2^31)");
  HC_TRY(hc::pool_forward(pool, stream, &v));
  hc::BufferCheck check(v.device);
  HC_TRY(check_table(table, lens, table_rows, table_width, table_stride, check));
  HC_TRY(check_list(parents, n, check, "parents"));
  HC_TRY(check_list(free_pages, n_free, check, "free_pages"));
  const hc::Tensor in = hc::table_tensor(table, table_rows, table_width, table_stride);
  const hc::Tensor out = hc::table_tensor(out_table, n, table_width, out_stride);
  HC_TRY(check_extent(out_table, out.bytes(), 8, false, check, "out_table"));
  HC_TRY(check_out_list(used, 1, check, "used"));
  bool shared = share(in, out) || overlap(span_of(in), {used, 8});
  for (const Span& r : {Span{lens, 8 * table_rows}, Span{parents, 8 * n}, Span{free_pages, 8 * n_free}, Span{used, 8}})
    shared |= overlap(r, span_of(out)) || (r.at != used && overlap(r, {used, 8}));
  if (shared) return set_error(HC_ERR_INVALID, "out_table and used must not overlap each other or what is read");
  hc::ForkArgs a = {{table, lens, table_rows, table_width, table_stride}, parents, free_pages, n, n_free, out_table,
                    out_stride, used};
  return launched(hc::launch_fork_pages(*v.geom, a, v.wrong, v.num_cus, (hipStream_t)stream), "fork");
}

int hc_pages_workspace_bytes(const hc_pool* pool, int64_t* out_bytes) {
  if (!pool || !out_bytes) return set_error(HC_ERR_INVALID, "null argument");
  PoolView v;
  hc::pool_view(pool, &v);
  HC_TRY(page_pool(v));
  *out_bytes = hc::pages_workspace(*v.geom);
  return HC_OK;
}

int hc_free_pages(hc_pool* pool, const int64_t* table, int64_t table_rows, int64_t table_width, int64_t table_stride,
                  const int64_t* lens, int64_t* free_pages, int64_t* count, void* workspace, int64_t workspace_bytes,
                  void* stream) {
  if (!pool) return set_error(HC_ERR_INVALID, "pool is null");
  TraceRange range("hc_free_pages");
  PoolView v;
  hc::pool_view(pool, &v);
  HC_TRY(page_pool(v));
  HC_TRY(table_sizes(table_rows, table_width, table_stride));
  HC_TRY(hc::pool_forward(pool, stream, &v));
  hc::BufferCheck check(v.device);
  HC_TRY(check_table(table, lens, table_rows, table_width, table_stride, check));
  const Span in = {table, hc::table_bytes(table_rows, table_width, table_stride)}, lengths = {lens, 8 * table_rows};
  const Span list = {free_pages, 8 * (v.geom->S / v.geom->P)}, number = {count, 8};
  HC_TRY(check.buffer(free_pages, list.bytes, 8, false, "free_pages"));
  HC_TRY(check_out_list(count, 1, check, "count"));
  if (overlap(in, list) || overlap(lengths, list) || overlap(number, in) || overlap(number, lengths) ||
      overlap(number, list))
    return set_error(HC_ERR_INVALID, "free_pages and count must not overlap each other or what is read");
  HC_TRY(check_work(v, workspace, workspace_bytes, check, {in, lengths, list, number}));
  const hc::PageTable t = {table, lens, table_rows, table_width, table_stride};
  return launched(hc::launch_free_pages(*v.geom, t, free_pages, count, workspace, v.wrong, v.num_cus,
                                        (hipStream_t)stream),
                  "free list");
}

int hc_compact_pages(hc_pool* pool, const int64_t* table, int64_t table_rows, int64_t table_width,
                     int64_t table_stride, const int64_t* lens, int64_t* out_table, int64_t out_stride,
                     int64_t* count, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!pool) return set_error(HC_ERR_INVALID, "pool is null");
  TraceRange range("hc_compact_pages");
  PoolView v;
  hc::pool_view(pool, &v);
  HC_TRY(page_pool(v));
  HC_TRY(table_sizes(table_rows, table_width, table_stride));
  HC_TRY(table_sizes(table_rows, table_width, out_stride));
  HC_TRY(hc::pool_forward(pool, stream, &v));
  hc::BufferCheck check(v.device);
  HC_TRY(check_table(table, lens, table_rows, table_width, table_stride, check));
  const hc::Tensor in = hc::table_tensor(table, table_rows, table_width, table_stride);
  const hc::Tensor out = hc::table_tensor(out_table, table_rows, table_width, out_stride);
  const Span lengths = {lens, 8 * table_rows}, number = {count, 8};
  HC_TRY(check_extent(out_table, out.bytes(), 8, false, check, "out_table"));
  HC_TRY(check_out_list(count, 1, check, "count"));
  if (share(in, out) && !(table == out_table && (table_stride == out_stride || table_rows == 1)))
    return set_error(HC_ERR_INVALID, "out_table overlaps the table without being it");
  if (overlap(lengths, span_of(out)) || overlap(number, span_of(out)) || overlap(number, span_of(in)) ||
      overlap(number, lengths))
    return set_error(HC_ERR_INVALID, "out_table and count must not overlap each other or what is read");
  HC_TRY(check_work(v, workspace, workspace_bytes, check, {span_of(in), lengths, span_of(out), number}));
  const hc::PageTable t = {table, lens, table_rows, table_width, table_stride};
  return launched(hc::launch_compact_pages(*v.geom, t, out_table, out_stride, count, workspace, v.wrong, v.num_cus,
                                           (hipStream_t)stream),
                  "compaction");
}

}  // extern "C"
