// kvq_packed.cuh -- rows of a batch's sequences, packed or padded: which rows
// of [n_rows] belong to which sequence (include/kvq.h: kv_append_rope).
#pragma once

#include "kvq_device.cuh"

namespace kvq {

struct PackedRows {
  const int32_t *row_start;  // packed: sequence s has rows row_start[s] .. row_start[s + 1] - 1
  const int32_t *n_new;      // padded: rows s * per_seq .. + n_new[s] - 1; both null: all per_seq
  int64_t n_rows, per_seq;
  int n_seqs;
};

// Rows of sequence s from `first` on; 0 and `bad` where the caller's entries
// are out of range.
__device__ __forceinline__ int64_t packed_rows(const PackedRows &p, int s, int64_t &first,
                                               bool &bad) {
  if (p.row_start) {
    const int a = p.row_start[s], b = p.row_start[s + 1];
    bad = a < 0 || b < a || b > p.n_rows;
    first = a;
    return bad ? 0 : b - a;
  }
  first = s * p.per_seq;
  const int64_t n = p.n_new ? p.n_new[s] : p.per_seq;
  bad = n < 0 || n > p.per_seq;
  return bad ? 0 : n;
}

// The sequence of a row, and the row's index in it; false for padding.
__device__ __forceinline__ bool packed_find(const PackedRows &p, int64_t row, int &s, int64_t &i) {
  int lo = 0;
  if (!p.row_start) {
    lo = static_cast<int>(row / p.per_seq);
  } else {
    int hi = p.n_seqs;  // the last s with row_start[s] <= row
    while (lo + 1 < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.row_start[mid] <= row) lo = mid;
      else hi = mid;
    }
  }
  s = lo;
  bool bad;
  int64_t first;
  const int64_t n = packed_rows(p, s, first, bad);
  i = row - first;
  return i >= 0 && i < n;
}

// KVQ_DEVERR_ROWS for entries out of range (one block).
__device__ __forceinline__ void packed_check(const PackedRows &p, int32_t *err) {
  for (int s = threadIdx.x; s < p.n_seqs; s += blockDim.x) {
    bool bad;
    int64_t first;
    packed_rows(p, s, first, bad);
    if (bad) set_err(err, KVQ_DEVERR_ROWS);
  }
}

}  // namespace kvq
