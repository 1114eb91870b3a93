// C ABI of the ragged-batch calls: argument validation and launches.
#include <algorithm>

#include "batch.cuh"
#include "decode.cuh"

namespace {

size_t dtype_bytes(int dtype) {
  return dtype == KVATTN_F32 ? 4 : dtype == KVATTN_F16 || dtype == KVATTN_BF16 ? 2 : 0;
}

int validate_batch(const kvattn_kv_desc* desc, const kvattn_batch* b) {
  const int st = validate_desc(desc);
  if (st) return st;
  if (!b || b->reserved != 0) return KVATTN_ERR_INVALID_ARG;
  if (b->n_seqs < 0 || b->n_rows < 0 || b->n_rows > INT32_MAX || b->max_rows < 0 || b->max_blocks < 0 ||
      b->max_blocks > (INT32_MAX / kPageTokens) + 1)
    return KVATTN_ERR_INVALID_ARG;
  // units are searched and counted in 32 bits
  if (static_cast<int64_t>(b->n_seqs) * desc->n_kv_heads > (1 << 27)) return KVATTN_ERR_UNSUPPORTED_SHAPE;
  if (b->n_seqs > 0 && (!b->row_start || !b->pos_start || (b->max_blocks > 0 && !b->page_table)))
    return KVATTN_ERR_INVALID_ARG;
  return KVATTN_OK;
}

// A token array of `heads` heads.  Inputs may repeat or overlap rows, outputs may not.
int validate_rows(const kvattn_rows* r, int64_t n_rows, int heads, bool output) {
  if (!r || r->reserved != 0 || !r->data || !aligned16(r->data)) return KVATTN_ERR_INVALID_ARG;
  const size_t size = dtype_bytes(r->dtype);
  if (!size) return KVATTN_ERR_UNSUPPORTED_FORMAT;
  const int64_t unit = static_cast<int64_t>(16 / size);
  const int64_t rs = n_rows > 1 ? r->row_stride : 0, hs = heads > 1 ? r->head_stride : 0;
  constexpr int64_t kMost = int64_t{1} << 40;  // elements: n_rows * stride stays below 2^63 bytes
  if (rs < 0 || hs < 0 || rs > kMost / (n_rows > 1 ? n_rows : 1) * 64 || hs > kMost || rs % unit || hs % unit)
    return KVATTN_ERR_INVALID_ARG;
  if (output) {
    const bool heads_inside = (heads == 1 || hs >= kHeadDim) && (n_rows <= 1 || rs >= hs * (heads - 1) + kHeadDim);
    const bool rows_inside = (n_rows <= 1 || rs >= kHeadDim) && (heads == 1 || hs >= rs * (n_rows - 1) + kHeadDim);
    if (!heads_inside && !rows_inside) return KVATTN_ERR_INVALID_ARG;
  }
  return KVATTN_OK;
}

RowsView view_of(const kvattn_rows* r, int64_t n_rows, int heads) {
  return RowsView{r->data, n_rows > 1 ? r->row_stride : 0, heads > 1 ? r->head_stride : 0};
}

BatchParams params_of(const kvattn_kv_desc* d, const kvattn_batch* b) {
  BatchParams p{};
  p.k_pool = static_cast<uint8_t*>(d->k_pool);
  p.v_pool = static_cast<uint8_t*>(d->v_pool);
  p.k_stride = d->k_page_stride;
  p.v_stride = d->v_page_stride;
  p.n_pages = d->n_pages;
  p.row_start = b->row_start;
  p.pos_start = b->pos_start;
  p.page_table = b->page_table;
  p.n_rows = b->n_rows;
  p.n_seqs = b->n_seqs;
  p.max_rows = b->max_rows;
  p.max_blocks = b->max_blocks;
  p.n_kv = d->n_kv_heads;
  return p;
}

long long most_tiles_of(const kvattn_kv_desc* d, const kvattn_batch* b) {
  return static_cast<long long>(b->n_seqs) * d->n_kv_heads * 8 * std::max(b->max_blocks, 1);
}

// What a decode supports beyond validate_batch: query rows of a unit that the kernels hold ...
bool decode_rows_ok(const kvattn_kv_desc* d, const kvattn_batch* b) {
  return static_cast<int64_t>(d->n_q_heads / d->n_kv_heads) * b->max_rows <= 24;
}

// ... and a line of all units' tiles (and a few per unit beside them) that is counted in 32 bits.
bool decode_tiles_ok(const kvattn_kv_desc* d, const kvattn_batch* b) { return most_tiles_of(d, b) <= (1ll << 30); }

// The workspace of a decode: where every unit's partials are, and two partials per group.
struct BatchPlan {
  int sms;
  long long most_tiles;  // of all units together
  size_t lse_off, o_off, bytes;
};

BatchPlan plan_batch(const kvattn_kv_desc* d, const kvattn_batch* b) {
  BatchPlan p{};
  p.sms = sm_budget_of(d);
  const long long units = static_cast<long long>(b->n_seqs) * d->n_kv_heads;
  p.most_tiles = most_tiles_of(d, b);
  const int row_tiles = batch_row_tiles(d->n_q_heads / d->n_kv_heads * std::max(b->max_rows, 1));
  const size_t slots = static_cast<size_t>(batch_group_bound(p.sms, row_tiles)) * 2 * row_tiles * 8;
  p.lse_off = round_up(sizeof(int2) * std::max(units, 1ll), 256);
  p.o_off = round_up(p.lse_off + sizeof(float) * slots, 256);
  p.bytes = p.o_off + sizeof(float) * slots * kHeadDim;
  return p;
}

// The grid of append and read: four warps per (tile slot, head), two such per CTA.
bool too_many_tiles(const kvattn_kv_desc* d, const kvattn_batch* b) {
  return (b->n_rows / 16 + 2ll * b->n_seqs) * d->n_kv_heads / 2 >= INT32_MAX;
}

bool nothing_to_do(const kvattn_batch* b) { return b->n_seqs == 0 || b->n_rows == 0 || b->max_rows == 0; }

}  // namespace

extern "C" {

KVATTN_API int kvattn_append_batch(const kvattn_kv_desc* desc, const kvattn_batch* batch, const kvattn_rows* k,
                                   const kvattn_rows* v, kvattn_stream_t stream) {
  const CallRange range_("kvattn_append_batch");
  int st = validate_batch(desc, batch);
  if (st) return st;
  if (nothing_to_do(batch)) return KVATTN_OK;
  if ((st = validate_rows(k, batch->n_rows, desc->n_kv_heads, false))) return st;
  if ((st = validate_rows(v, batch->n_rows, desc->n_kv_heads, false))) return st;
  if (k->dtype != v->dtype) return KVATTN_ERR_UNSUPPORTED_FORMAT;
  if (too_many_tiles(desc, batch)) return KVATTN_ERR_UNSUPPORTED_SHAPE;
  int dev;
  if ((st = current_device_checked(&dev))) return st;
  const cudaError_t e = launch_append_batch(params_of(desc, batch), view_of(k, batch->n_rows, desc->n_kv_heads),
                                            view_of(v, batch->n_rows, desc->n_kv_heads), k->dtype,
                                            key_format_id(desc->k_fmt), value_format_id(desc->v_fmt),
                                            static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVATTN_OK : cuda_fail(e);
}

KVATTN_API int kvattn_read_batch(const kvattn_kv_desc* desc, const kvattn_batch* batch, const kvattn_rows* k,
                                 const kvattn_rows* v, kvattn_stream_t stream) {
  const CallRange range_("kvattn_read_batch");
  int st = validate_batch(desc, batch);
  if (st) return st;
  if (nothing_to_do(batch) || (!k && !v)) return KVATTN_OK;
  if (k && (st = validate_rows(k, batch->n_rows, desc->n_kv_heads, true))) return st;
  if (v && (st = validate_rows(v, batch->n_rows, desc->n_kv_heads, true))) return st;
  if (k && v && k->dtype != v->dtype) return KVATTN_ERR_UNSUPPORTED_FORMAT;
  if (too_many_tiles(desc, batch)) return KVATTN_ERR_UNSUPPORTED_SHAPE;
  int dev;
  if ((st = current_device_checked(&dev))) return st;
  const RowsView none{nullptr, 0, 0};
  const cudaError_t e = launch_read_batch(params_of(desc, batch), k ? view_of(k, batch->n_rows, desc->n_kv_heads) : none,
                                          v ? view_of(v, batch->n_rows, desc->n_kv_heads) : none,
                                          k ? k->dtype : v->dtype, key_format_id(desc->k_fmt),
                                          value_format_id(desc->v_fmt), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVATTN_OK : cuda_fail(e);
}

KVATTN_API size_t kvattn_decode_batch_workspace_size(const kvattn_kv_desc* desc, const kvattn_batch* batch) {
  if (validate_batch(desc, batch) || !decode_rows_ok(desc, batch) || !decode_tiles_ok(desc, batch)) return 0;
  return plan_batch(desc, batch).bytes;
}

KVATTN_API int kvattn_decode_batch(const kvattn_kv_desc* desc, const kvattn_batch* batch, const kvattn_rows* q,
                                   const int32_t* page_logical, const int32_t* n_pages, int32_t window,
                                   const kvattn_rows* out, float* lse, void* ws, size_t ws_bytes,
                                   kvattn_stream_t stream) {
  const CallRange range_("kvattn_decode_batch");
  int st = validate_batch(desc, batch);
  if (st) return st;
  if (window < 0) return KVATTN_ERR_INVALID_ARG;
  if (!decode_rows_ok(desc, batch)) return KVATTN_ERR_UNSUPPORTED_SHAPE;
  if (nothing_to_do(batch)) return KVATTN_OK;
  if ((st = validate_rows(q, batch->n_rows, desc->n_q_heads, false))) return st;
  if ((st = validate_rows(out, batch->n_rows, desc->n_q_heads, true))) return st;
  if (q->dtype != out->dtype) return KVATTN_ERR_UNSUPPORTED_FORMAT;
  if (!lse) return KVATTN_ERR_INVALID_ARG;
  if (!decode_tiles_ok(desc, batch)) return KVATTN_ERR_UNSUPPORTED_SHAPE;
  const BatchPlan plan = plan_batch(desc, batch);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) return KVATTN_ERR_INVALID_ARG;
  if (ws_bytes < plan.bytes) return KVATTN_ERR_WORKSPACE_TOO_SMALL;
  int dev;
  if ((st = current_device_checked(&dev))) return st;
  BatchDecodeParams p{};
  p.b = params_of(desc, batch);
  p.q = view_of(q, batch->n_rows, desc->n_q_heads);
  p.out = view_of(out, batch->n_rows, desc->n_q_heads);
  p.lse = lse;
  p.page_logical = page_logical;
  p.n_list = n_pages;
  p.group = desc->n_q_heads / desc->n_kv_heads;
  p.window = window;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.unit_parts = reinterpret_cast<int2*>(w);
  p.part_lse = reinterpret_cast<float*>(w + plan.lse_off);
  p.part_o = reinterpret_cast<float*>(w + plan.o_off);
  const cudaError_t e = launch_decode_batch(p, q->dtype, key_format_id(desc->k_fmt), value_format_id(desc->v_fmt),
                                            plan.sms, plan.most_tiles, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVATTN_OK : cuda_fail(e);
}

}  // extern "C"
