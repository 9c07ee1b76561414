// rope_api.cu -- host side of the rotary-position entry points (include/kvq.h):
// frequencies, argument validation, dispatch.
#include <cuda_runtime.h>

#include <math.h>

#include "kvq_check.h"

namespace kvq {

uint64_t turns_of(double f) {
  // 1 / (2 pi) = hi + lo to 106 bits
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double t = f * hi, e = fma(f, hi, -t) + f * lo;  // t + e: the turns
  const double r = ldexp(t, 64), n = floor(r);
  // n < 2^64 (f < 2 pi); the rest is below 2^12 in size
  return static_cast<uint64_t>(n) + static_cast<uint64_t>(llround((r - n) + ldexp(e, 64)));
}

namespace {

constexpr double kTwoPi = 6.283185307179586;

// Strides and pointer of a set of rows [n][heads][128].
int check_rows(const kvq_rows &r, bool is_written, int64_t n, int32_t heads) {
  if (!r.data || r.reserved != 0) return KVQ_EINVAL;
  if (r.type != KVQ_T_F16 && r.type != KVQ_T_BF16 && r.type != KVQ_T_F32) return KVQ_EUNSUPPORTED;
  if (r.row_stride < 0 || r.head_stride < 0) return KVQ_EINVAL;
  const int64_t sz = type_bytes(r.type);
  if (!aligned(r.data, 16) || r.row_stride * sz % 16 || r.head_stride * sz % 16) return KVQ_EALIGN;
  if (is_written) {  // no two rows may share a place
    const int64_t d = kHeadDim;
    const bool heads_inside = (heads == 1 || r.head_stride >= d) &&
                              (n == 1 || r.row_stride >= (heads - 1) * r.head_stride + d);
    const bool rows_inside = (n == 1 || r.row_stride >= d) &&
                             (heads == 1 || r.head_stride >= (n - 1) * r.row_stride + d);
    if (!heads_inside && !rows_inside) return KVQ_EINVAL;
  }
  return KVQ_OK;
}

int64_t span_bytes(const kvq_rows &r, int64_t n, int32_t heads) {
  return ((n - 1) * r.row_stride + (heads - 1) * r.head_stride + kHeadDim) * type_bytes(r.type);
}

}  // namespace
}  // namespace kvq

using kvq::aligned;
using kvq::check_layer;
using kvq::check_rope;

extern "C" {

int kvq_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, double orig_len,
                   double low, double high, double *freqs) {
  if (!freqs || rot_dim < 2 || rot_dim > kvq::kHeadDim || rot_dim % 2 != 0) return KVQ_EINVAL;
  if (!(base > 1.0) || !isfinite(base)) return KVQ_EINVAL;
  if (scaling < KVQ_ROPE_PLAIN || scaling > KVQ_ROPE_YARN) return KVQ_EUNSUPPORTED;
  if (scaling != KVQ_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return KVQ_EINVAL;
  const bool blend = scaling == KVQ_ROPE_PARTS || scaling == KVQ_ROPE_YARN;
  if (blend && (!(orig_len > 0.0) || !isfinite(orig_len) || !(low > 0.0) || !(high > low) ||
                !isfinite(high)))
    return KVQ_EINVAL;
  const int n = rot_dim / 2;
  if (scaling == KVQ_ROPE_NTK && n > 1)
    base *= pow(factor, rot_dim / static_cast<double>(rot_dim - 2));
  if (!isfinite(base)) return KVQ_EINVAL;
  double l = 0.0, h = 0.0;
  if (scaling == KVQ_ROPE_YARN) {
    const double turn = rot_dim / (2.0 * log(base));
    l = fmax(floor(turn * log(orig_len / (high * kvq::kTwoPi))), 0.0);
    h = fmin(ceil(turn * log(orig_len / (low * kvq::kTwoPi))), rot_dim - 1.0);
  }
  for (int i = 0; i < n; ++i) {
    const double f = pow(base, -2.0 * i / rot_dim);
    double keep = 1.0;
    if (scaling == KVQ_ROPE_LINEAR) keep = 0.0;
    if (scaling == KVQ_ROPE_PARTS)
      keep = fmin(fmax((orig_len * f / kvq::kTwoPi - low) / (high - low), 0.0), 1.0);
    if (scaling == KVQ_ROPE_YARN) keep = 1.0 - fmin(fmax((i - l) / fmax(h - l, 0.001), 0.0), 1.0);
    freqs[i] = keep == 1.0 ? f : f * keep + f / factor * (1.0 - keep);
  }
  return KVQ_OK;
}

int kvq_rope_table(const double *freqs, int32_t rot_dim, int32_t n_pos, float *table,
                   void *stream) {
  if (!freqs || !table || rot_dim < 2 || rot_dim > kvq::kHeadDim || rot_dim % 2 != 0 || n_pos <= 0)
    return KVQ_EINVAL;
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!(freqs[i] >= 0.0) || !(freqs[i] < kvq::kTwoPi)) return KVQ_EINVAL;
  if (!aligned(table, 16)) return KVQ_EALIGN;
  const cudaError_t e =
      kvq::launch_rope_table(freqs, rot_dim, n_pos, table, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

int kvq_rope_apply(const kvq_rope *rope, const kvq_rows *x, const kvq_rows *y, int64_t n_rows,
                   int32_t n_heads, const int32_t *positions, int32_t pos0, int32_t transpose,
                   int32_t *err, void *stream) {
  int st = check_rope(rope);
  if (st != KVQ_OK) return st;
  if (!x || !y || n_rows < 0 || n_rows > INT32_MAX || n_heads <= 0 || n_heads > 65536)
    return KVQ_EINVAL;
  if (n_rows == 0) return KVQ_OK;
  if ((st = kvq::check_rows(*x, false, n_rows, n_heads)) != KVQ_OK) return st;
  if ((st = kvq::check_rows(*y, true, n_rows, n_heads)) != KVQ_OK) return st;
  if (y->type != x->type && y->type != KVQ_T_F16) return KVQ_EUNSUPPORTED;
  if (!aligned(positions, 4) || !aligned(err, 4)) return KVQ_EALIGN;
  const bool same = x->data == y->data && x->type == y->type &&
                    (n_rows == 1 || x->row_stride == y->row_stride) &&
                    (n_heads == 1 || x->head_stride == y->head_stride);
  if (!same && kvq::overlap(x->data, kvq::span_bytes(*x, n_rows, n_heads), y->data,
                            kvq::span_bytes(*y, n_rows, n_heads)))
    return KVQ_EINVAL;
  const cudaError_t e =
      kvq::launch_rope_apply(*rope, *x, *y, n_rows, n_heads, positions, pos0, transpose, err,
                             static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

int kv_append_rope(const kvq_layer *layer, const kvq_rope *rope, const kvq_rows *q,
                   const kvq_rows *k, const kvq_rows *v, int64_t n_rows, const int32_t *n_new,
                   const int32_t *row_start, const int32_t *positions, void *q_out,
                   int32_t update_lens, void *stream) {
  int st = check_layer(layer);
  if (st != KVQ_OK) return st;
  if ((st = check_rope(rope)) != KVQ_OK) return st;
  if (!k || !v || n_rows < 0 || n_rows > INT32_MAX) return KVQ_EINVAL;
  if ((n_new == nullptr) == (row_start == nullptr)) return KVQ_EINVAL;
  if (n_new && n_rows % layer->n_seqs != 0) return KVQ_EINVAL;
  if (!aligned(n_new, 4) || !aligned(row_start, 4) || !aligned(positions, 4)) return KVQ_EALIGN;
  if (n_rows == 0) return KVQ_OK;  // (an empty batch's tensors have no address)
  if ((q == nullptr) != (q_out == nullptr)) return KVQ_EINVAL;
  if ((st = kvq::check_rows(*k, false, n_rows, layer->n_kv_heads)) != KVQ_OK) return st;
  if ((st = kvq::check_rows(*v, false, n_rows, layer->n_kv_heads)) != KVQ_OK) return st;
  if (k->type != v->type) return KVQ_EUNSUPPORTED;
  if (q) {
    if ((st = kvq::check_rows(*q, false, n_rows, layer->n_q_heads)) != KVQ_OK) return st;
    if (q->type != k->type) return KVQ_EUNSUPPORTED;
    if (!aligned(q_out, 16)) return KVQ_EALIGN;
    const int64_t d = kvq::kHeadDim, nb = n_rows * layer->n_q_heads * d * 2;
    const bool same = q->data == q_out && q->type == KVQ_T_F16 &&
                      (n_rows == 1 || q->row_stride == layer->n_q_heads * d) &&
                      (layer->n_q_heads == 1 || q->head_stride == d);
    if (!same && kvq::overlap(q->data, kvq::span_bytes(*q, n_rows, layer->n_q_heads), q_out, nb))
      return KVQ_EINVAL;
    if (kvq::overlap(k->data, kvq::span_bytes(*k, n_rows, layer->n_kv_heads), q_out, nb) ||
        kvq::overlap(v->data, kvq::span_bytes(*v, n_rows, layer->n_kv_heads), q_out, nb))
      return KVQ_EINVAL;
  }
  const int sms = kvq::device_sms();
  if (sms <= 0) return KVQ_ECUDA;
  const cudaError_t e = kvq::launch_append_rope(*layer, *rope, q, *k, *v, n_rows, n_new, row_start,
                                                positions, q_out, update_lens, sms,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

int kv_evict_delta(const kvq_layer *layer, const int32_t *evict, const int32_t *n_evicted,
                   int32_t max_evict, int32_t *delta, void *stream) {
  const int st = check_layer(layer);
  if (st != KVQ_OK) return st;
  if (!evict || !n_evicted || max_evict < 0 || !delta) return KVQ_EINVAL;
  if (layer->n_seqs > kvq::kShiftMaxSeqs) return KVQ_EINVAL;
  if (!aligned(evict, 4) || !aligned(n_evicted, 4) || !aligned(delta, 4)) return KVQ_EALIGN;
  const cudaError_t e = kvq::launch_evict_delta(*layer, evict, n_evicted, max_evict, delta,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

int kv_rope_shift(const kvq_layer *layer, const kvq_rope *rope, const int32_t *delta,
                  void *stream) {
  int st = check_layer(layer);
  if (st != KVQ_OK) return st;
  if ((st = check_rope(rope)) != KVQ_OK) return st;
  if (!delta || layer->n_seqs > kvq::kShiftMaxSeqs) return KVQ_EINVAL;
  if (!aligned(delta, 4)) return KVQ_EALIGN;
  const cudaError_t e =
      kvq::launch_rope_shift(*layer, *rope, delta, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

}  // extern "C"
