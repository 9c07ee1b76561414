// kvq_check.h -- host-side argument validation shared by every entry point of
// libkvq, so that all of them apply the same rules (include/kvq.h: "Errors").
#pragma once

#include <math.h>
#include <stdint.h>

#include "../../include/kvq.h"
#include "kvq_launch.h"

namespace kvq {

constexpr int kHeadDim = 128;

inline bool valid_codec(int c) {
  return c == KVQ_F16 || c == KVQ_Q8_0 || c == KVQ_Q4_0 || c == KVQ_TURBO4;
}

inline bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
  const uint8_t *x = static_cast<const uint8_t *>(a), *y = static_cast<const uint8_t *>(b);
  return x < y + nb && y < x + na;
}

// The layer descriptor: geometry, codecs, cache pointers and their
// alignment, and (paged layers) the block table.
inline int check_layer(const kvq_layer *L) {
  if (!L) return KVQ_EINVAL;
  if (L->head_dim != kHeadDim) return KVQ_EUNSUPPORTED;
  if (!valid_codec(L->codec_k) || !valid_codec(L->codec_v)) return KVQ_EUNSUPPORTED;
  if (L->n_seqs <= 0 || L->n_kv_heads <= 0 || L->n_q_heads <= 0 || L->capacity <= 0 ||
      L->reserved != 0)
    return KVQ_EINVAL;
  if (L->n_q_heads % L->n_kv_heads != 0) return KVQ_EINVAL;
  if (!L->k_cache || !L->v_cache || !L->seq_lens) return KVQ_EINVAL;
  if (L->capacity % 256 != 0) return KVQ_EALIGN;
  if (L->pages_per_seq < 0) return KVQ_EINVAL;
  if (L->pages_per_seq > 0) {  // paged: a block table over pools of n_pages pages
    if (!L->block_table || L->n_pages <= 0) return KVQ_EINVAL;
    if (static_cast<int64_t>(L->pages_per_seq) * 256 != L->capacity) return KVQ_EINVAL;
    if (!aligned(L->block_table, 4)) return KVQ_EALIGN;
  }
  if (!aligned(L->k_cache, 16) || !aligned(L->v_cache, 16) || !aligned(L->seq_lens, 4) ||
      (L->err && !aligned(L->err, 4)))
    return KVQ_EALIGN;
  return KVQ_OK;
}

// The rotary descriptor.
inline int check_rope(const kvq_rope *r) {
  if (!r || !r->table || r->n_pos <= 0 || r->rot_dim < 2 || r->rot_dim > kHeadDim ||
      r->rot_dim % 2 != 0 || !isfinite(r->magnitude))
    return KVQ_EINVAL;
  if (r->layout != KVQ_ROPE_INTERLEAVED && r->layout != KVQ_ROPE_HALF) return KVQ_EUNSUPPORTED;
  return aligned(r->table, 16) ? KVQ_OK : KVQ_EALIGN;
}

// Strides and pointer of a set of rows [n][heads][128].
inline int check_rows(const kvq_rows &r, bool is_written, int64_t n, int32_t heads) {
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

inline int64_t span_bytes(const kvq_rows &r, int64_t n, int32_t heads) {
  return ((n - 1) * r.row_stride + (heads - 1) * r.head_stride + kHeadDim) * type_bytes(r.type);
}

// Whether a and b, whose ranges meet, are views of one tensor that share no place: with the
// same strides, each lies in its own part of every period, the larger stride (rows or heads
// of one beside those of the other) or the smaller one (beside each other in every head or row).
inline bool interleaved(const kvq_rows &a, const kvq_rows &b, int64_t n, int32_t heads) {
  const int64_t sa = type_bytes(a.type), sb = type_bytes(b.type);
  const int64_t row = a.row_stride * sa, head = a.head_stride * sa;
  if ((n > 1 && row != b.row_stride * sb) || (heads > 1 && head != b.head_stride * sb)) return false;
  const int64_t at = static_cast<uint8_t *>(b.data) - static_cast<uint8_t *>(a.data);
  auto apart = [&](int64_t period, int64_t inner) {  // inner: from the first to the last value's row
    if (period <= 0) return false;
    const int64_t d = (at % period + period) % period;
    return d >= inner + kHeadDim * sa && d + inner + kHeadDim * sb <= period;
  };
  if (n == 1 || heads == 1) return apart(n > 1 ? row : heads > 1 ? head : 0, 0);
  const bool rows_outside = row >= head;
  const int64_t large = rows_outside ? row : head, small = rows_outside ? head : row;
  return apart(large, ((rows_outside ? heads : n) - 1) * small) ||
         (small > 0 && large % small == 0 && apart(small, 0));
}

// At most 2^31 - 1 rows times query heads (any n_rows: no product that could wrap).
inline bool rows_fit(const kvq_layer *L, int64_t n_rows) {
  return n_rows >= 0 && n_rows <= INT32_MAX / L->n_q_heads;
}

// Which rows belong to which sequence: row_start (packed), n_new (padded) or
// neither (one row per sequence).
inline int check_packed(const kvq_layer *L, int64_t n_rows, const int32_t *n_new,
                        const int32_t *row_start, bool one_each) {
  if (!rows_fit(L, n_rows)) return KVQ_EINVAL;
  if (n_new && row_start) return KVQ_EINVAL;
  if (!n_new && !row_start && (!one_each || n_rows != L->n_seqs)) return KVQ_EINVAL;
  if (n_new && n_rows % L->n_seqs != 0) return KVQ_EINVAL;
  return aligned(n_new, 4) && aligned(row_start, 4) ? KVQ_OK : KVQ_EALIGN;
}

// Decode streams: (sequence, kv head, group of up to 8 query heads).
inline bool decode_shape_ok(const kvq_layer *L) {
  const int64_t G = L->n_q_heads / L->n_kv_heads;
  const int64_t streams = static_cast<int64_t>(L->n_seqs) * L->n_kv_heads * ((G + 7) / 8);
  return L->n_seqs <= kDecodeMaxSeqs && streams <= kDecodeMaxStreams;
}

// Everything a decode call checks before its scratch memory: the layer, the
// query and output pointers and max_len.
inline int check_decode_call(const kvq_layer *L, const void *q, const void *out,
                             const float *lse, int32_t max_len) {
  const int st = check_layer(L);
  if (st != KVQ_OK) return st;
  if (!q || !out || max_len <= 0) return KVQ_EINVAL;
  if (!decode_shape_ok(L)) return KVQ_EINVAL;
  if (max_len > L->capacity) return KVQ_ECAPACITY;
  if (!aligned(q, 8) || !aligned(out, 8) || (lse && !aligned(lse, 4))) return KVQ_EALIGN;
  return KVQ_OK;
}

}  // namespace kvq
