// cross_api.cu -- host side of the entry points over packed rows without a
// rotation (include/kvq.h): argument validation and dispatch.
#include <cuda_runtime.h>

#include "kvq_check.h"

using kvq::aligned;
using kvq::check_layer;
using kvq::check_rows;
using kvq::kHeadDim;
using kvq::overlap;
using kvq::span_bytes;

namespace {

// The parts of a shared-prefix step's workspace.
struct PrefixPlan {
  kvq::DecodePlan own;
  kvq::CrossPlan shared;
  int64_t xo_off, xml_off, cross_off, ws_bytes;
};

PrefixPlan plan_prefix(const kvq_layer &layer, const kvq_layer &prefix, int max_len,
                       int max_prefix, int sms) {
  PrefixPlan p;
  const int64_t rows = static_cast<int64_t>(layer.n_seqs) * layer.n_q_heads;
  p.own = kvq::plan_decode(layer, max_len, sms);
  p.shared = kvq::plan_cross(prefix, layer.n_seqs, max_prefix, sms);
  p.xo_off = (p.own.ws_bytes + 15) / 16 * 16;
  p.xml_off = p.xo_off + rows * kHeadDim * 4;
  p.cross_off = (p.xml_off + rows * 8 + 15) / 16 * 16;
  p.ws_bytes = p.cross_off + p.shared.ws_bytes;
  return p;
}

int check_prefix(const kvq_layer *layer, const kvq_layer *prefix, int32_t max_len,
                 int32_t max_prefix) {
  int st = check_layer(layer);
  if (st != KVQ_OK) return st;
  if ((st = check_layer(prefix)) != KVQ_OK) return st;
  if (prefix->n_kv_heads != layer->n_kv_heads || prefix->n_q_heads != layer->n_q_heads)
    return KVQ_EINVAL;
  if (!kvq::decode_shape_ok(layer) || prefix->n_seqs > kvq::kCrossMaxSeqs) return KVQ_EINVAL;
  if (max_len <= 0 || max_prefix <= 0) return KVQ_EINVAL;
  return max_len > layer->capacity || max_prefix > prefix->capacity ? KVQ_ECAPACITY : KVQ_OK;
}

}  // namespace

extern "C" {

int kv_append_rows(const kvq_layer *layer, const kvq_rows *k, const kvq_rows *v, int64_t n_rows,
                   const int32_t *n_new, const int32_t *row_start, int32_t update_lens,
                   void *stream) {
  int st = check_layer(layer);
  if (st != KVQ_OK) return st;
  if (!k || !v) return KVQ_EINVAL;
  if ((st = kvq::check_packed(layer, n_rows, n_new, row_start, false)) != KVQ_OK) return st;
  if (n_rows == 0) return KVQ_OK;  // (an empty batch's tensors have no address)
  if ((st = check_rows(*k, false, n_rows, layer->n_kv_heads)) != KVQ_OK) return st;
  if ((st = check_rows(*v, false, n_rows, layer->n_kv_heads)) != KVQ_OK) return st;
  if (k->type != v->type) return KVQ_EUNSUPPORTED;
  const int sms = kvq::device_sms();
  if (sms <= 0) return KVQ_ECUDA;
  const cudaError_t e =
      kvq::launch_append_rope(*layer, nullptr, nullptr, *k, *v, n_rows, n_new, row_start, nullptr,
                              nullptr, update_lens, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

int kv_read_rows(const kvq_layer *layer, const kvq_rows *k, const kvq_rows *v, int64_t n_rows,
                 const int32_t *n_read, const int32_t *row_start, const int32_t *first,
                 void *stream) {
  int st = check_layer(layer);
  if (st != KVQ_OK) return st;
  if (!k && !v) return KVQ_EINVAL;
  if ((st = kvq::check_packed(layer, n_rows, n_read, row_start, false)) != KVQ_OK) return st;
  if (!aligned(first, 4)) return KVQ_EALIGN;
  if (n_rows == 0) return KVQ_OK;
  const int heads = layer->n_kv_heads;
  if (k && (st = check_rows(*k, true, n_rows, heads)) != KVQ_OK) return st;
  if (v && (st = check_rows(*v, true, n_rows, heads)) != KVQ_OK) return st;
  if (k && v &&
      overlap(k->data, span_bytes(*k, n_rows, heads), v->data, span_bytes(*v, n_rows, heads)) &&
      !kvq::interleaved(*k, *v, n_rows, heads))
    return KVQ_EINVAL;
  const int sms = kvq::device_sms();
  if (sms <= 0) return KVQ_ECUDA;
  const cudaError_t e = kvq::launch_read_rows(*layer, k, v, n_rows, n_read, row_start, first, sms,
                                              static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

int attn_cross_workspace(const kvq_layer *layer, int64_t n_rows, int32_t max_len, size_t *bytes) {
  const int st = check_layer(layer);
  if (st != KVQ_OK) return st;
  if (!bytes || !kvq::rows_fit(layer, n_rows) || max_len <= 0 ||
      layer->n_seqs > kvq::kCrossMaxSeqs)
    return KVQ_EINVAL;
  if (max_len > layer->capacity) return KVQ_ECAPACITY;
  const int sms = kvq::device_sms();
  if (sms <= 0) return KVQ_ECUDA;
  *bytes = static_cast<size_t>(kvq::plan_cross(*layer, n_rows, max_len, sms).ws_bytes);
  return KVQ_OK;
}

int attn_cross(const kvq_layer *layer, const kvq_rows *q, int64_t n_rows, const int32_t *n_new,
               const int32_t *row_start, float scale, const kvq_rows *out, float *lse,
               int32_t max_len, void *workspace, size_t ws_bytes, void *stream) {
  int st = check_layer(layer);
  if (st != KVQ_OK) return st;
  if (!q || !out || max_len <= 0 || !(scale > 0.0f) || !isfinite(scale) ||
      layer->n_seqs > kvq::kCrossMaxSeqs)
    return KVQ_EINVAL;
  if (max_len > layer->capacity) return KVQ_ECAPACITY;
  if ((st = kvq::check_packed(layer, n_rows, n_new, row_start, true)) != KVQ_OK) return st;
  if (n_rows == 0) return KVQ_OK;
  const int heads = layer->n_q_heads;
  if ((st = check_rows(*q, false, n_rows, heads)) != KVQ_OK) return st;
  if ((st = check_rows(*out, true, n_rows, heads)) != KVQ_OK) return st;
  if (q->type == KVQ_T_F32 || out->type != q->type) return KVQ_EUNSUPPORTED;
  if (!aligned(lse, 4)) return KVQ_EALIGN;
  // (a row's query is read by every block that takes a part of its keys)
  if (overlap(q->data, span_bytes(*q, n_rows, heads), out->data, span_bytes(*out, n_rows, heads)) &&
      !kvq::interleaved(*q, *out, n_rows, heads))
    return KVQ_EINVAL;
  if (!workspace) return KVQ_EWORKSPACE;
  if (!aligned(workspace, 16)) return KVQ_EALIGN;
  const int sms = kvq::device_sms();
  if (sms <= 0) return KVQ_ECUDA;
  const kvq::CrossPlan pl = kvq::plan_cross(*layer, n_rows, max_len, sms);
  if (ws_bytes < static_cast<size_t>(pl.ws_bytes)) return KVQ_EWORKSPACE;
  const kvq::CrossOut to = {out->data, lse, nullptr, nullptr};
  const cudaError_t e = kvq::launch_cross(*layer, pl, *q, n_rows, n_new, row_start, scale, to,
                                          out->row_stride, out->head_stride, max_len, workspace,
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

int attn_decode_prefix_workspace(const kvq_layer *layer, const kvq_layer *prefix, int32_t max_len,
                                 int32_t max_prefix, size_t *bytes) {
  const int st = check_prefix(layer, prefix, max_len, max_prefix);
  if (st != KVQ_OK) return st;
  if (!bytes) return KVQ_EINVAL;
  const int sms = kvq::device_sms();
  if (sms <= 0) return KVQ_ECUDA;
  *bytes = static_cast<size_t>(plan_prefix(*layer, *prefix, max_len, max_prefix, sms).ws_bytes);
  return KVQ_OK;
}

int attn_decode_prefix(const kvq_layer *layer, const kvq_layer *prefix,
                       const int32_t *group_start, const void *q, float scale, void *out,
                       float *lse, int32_t max_len, int32_t max_prefix, void *workspace,
                       size_t ws_bytes, void *stream) {
  int st = check_prefix(layer, prefix, max_len, max_prefix);
  if (st != KVQ_OK) return st;
  if (!q || !out || !(scale > 0.0f) || !isfinite(scale)) return KVQ_EINVAL;
  if (!group_start && prefix->n_seqs != 1) return KVQ_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 8) || (lse && !aligned(lse, 4)) || !aligned(group_start, 4))
    return KVQ_EALIGN;
  const int64_t d = kHeadDim, nb = layer->n_seqs * (layer->n_q_heads * d * 2);
  if (overlap(q, nb, out, nb)) return KVQ_EINVAL;
  if (!workspace) return KVQ_EWORKSPACE;
  if (!aligned(workspace, 16)) return KVQ_EALIGN;
  const int sms = kvq::device_sms();
  if (sms <= 0) return KVQ_ECUDA;
  const PrefixPlan pl = plan_prefix(*layer, *prefix, max_len, max_prefix, sms);
  if (ws_bytes < static_cast<size_t>(pl.ws_bytes)) return KVQ_EWORKSPACE;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const kvq_rows qr = {const_cast<void *>(q), layer->n_q_heads * d, d, KVQ_T_F16, 0};
  float *xo = reinterpret_cast<float *>(ws + pl.xo_off);
  float2 *xml = reinterpret_cast<float2 *>(ws + pl.xml_off);
  cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  // one prefix without group_start: its rows are the batch (padded form, all of it)
  cudaError_t e = kvq::launch_cross(*prefix, pl.shared, qr, layer->n_seqs, nullptr, group_start,
                                    scale, {nullptr, nullptr, xo, xml}, 0, 0, max_prefix,
                                    ws + pl.cross_off, st_);
  if (e == cudaSuccess) {
    const kvq::PrefixPart part = {xo, xml, group_start, prefix->n_seqs};
    e = kvq::launch_decode(*layer, pl.own, q, scale, out, lse, max_len, workspace, st_, nullptr,
                           nullptr, nullptr, nullptr, &part);
  }
  return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

}  // extern "C"
