// append_rope.cu -- quantize-on-append with the rotary rotation applied on
// the way: new keys are rotated in fp32 and encoded from there, values are
// encoded as they come, and the queries of the same rows are rotated to fp16
// beside them.
#include <cuda_runtime.h>

#include "kvq_encode.cuh"
#include "kvq_launch.h"
#include "kvq_rope.cuh"

namespace kvq {
namespace {

constexpr int kArWarps = 8;
constexpr int kArThreads = kArWarps * 32;
constexpr int kHeadsPerWarp = 8;  // heads of one row that share a warp's angles

struct AppendRopeParams {
  RopeArgs rope;
  const uint8_t *x[3];     // q, k, v rows
  int64_t row[3], head[3];  // strides in bytes
  __half *q_out;
  uint8_t *cache[2];
  int codec[2];
  const int32_t *seq_lens, *n_new, *row_start, *positions;
  const int32_t *table;  // paged layers: block table; nullptr: contiguous
  int32_t *err;
  int64_t n_rows, max_new;  // max_new: padded rows per sequence
  int n_seqs, n_q, n_kv, capacity, pages_per_seq, n_pages;
  int q_chunks, kv_chunks;  // chunks of kHeadsPerWarp heads
};

// New rows of sequence s, 0 and KVQ_DEVERR_ROWS where the caller's entries
// are out of range.
__device__ __forceinline__ int64_t new_rows(const AppendRopeParams &p, int s, bool &bad) {
  bad = false;
  if (p.row_start) {
    const int a = p.row_start[s], b = p.row_start[s + 1];
    bad = a < 0 || b < a || b > p.n_rows;
    return bad ? 0 : b - a;
  }
  const int n = p.n_new[s];
  bad = n < 0 || n > p.max_new;
  return bad ? 0 : n;
}

// The sequence of a row and its index there; false for padding.
__device__ __forceinline__ bool find_row(const AppendRopeParams &p, int64_t row, int &s,
                                         int64_t &i) {
  if (!p.row_start) {
    s = static_cast<int>(row / p.max_new);
    i = row - s * p.max_new;
    return i < p.n_new[s];
  }
  int lo = 0, hi = p.n_seqs;  // the last s with row_start[s] <= row
  while (lo + 1 < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.row_start[mid] <= row) lo = mid;
    else hi = mid;
  }
  s = lo;
  i = row - p.row_start[s];
  return i >= 0 && row < p.row_start[s + 1];
}

// One warp per (row, up to eight heads of q, k or v).
template <int T>
__global__ void __launch_bounds__(kArThreads) append_rope_kernel(AppendRopeParams p) {
  constexpr int S = sizeof(typename RowType<T>::type);
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s < p.n_seqs; s += kArThreads) {
      bool bad;
      new_rows(p, s, bad);
      if (bad) set_err(p.err, KVQ_DEVERR_ROWS);
    }
  const int per_row = p.q_chunks + 2 * p.kv_chunks;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kArWarps + (threadIdx.x >> 5);
  const int64_t row = item / per_row;
  if (row >= p.n_rows) return;
  int chunk = static_cast<int>(item % per_row), which = 0;
  if (chunk >= p.q_chunks) {
    chunk -= p.q_chunks;
    which = 1 + chunk / p.kv_chunks;
    chunk %= p.kv_chunks;
  }
  int s;
  int64_t i;
  if (!find_row(p, row, s, i)) return;
  const int64_t slot = static_cast<int64_t>(p.seq_lens[s]) + i;
  const int h0 = chunk * kHeadsPerWarp, h1 = min(h0 + kHeadsPerWarp, which == 0 ? p.n_q : p.n_kv);
  const uint8_t *x = p.x[which] + row * p.row[which] + 4 * lane * S;
  LaneAngles a;
  if (which < 2)
    a = lane_angles(p.rope, rope_row(p.rope, p.positions ? p.positions[row] : slot, p.err), lane);
  if (which == 0) {
    for (int h = h0; h < h1; ++h) {
      float v[4];
      load4<T>(x + h * p.head[0], v);
      rotate_lane(p.rope, a, lane, v);
      store4<KVQ_T_F16>(p.q_out + (row * p.n_q + h) * kD + 4 * lane, v);
    }
    return;
  }
  if (slot < 0 || slot >= p.capacity) {
    if (lane == 0) set_err(p.err, KVQ_DEVERR_CAPACITY);
    return;
  }
  const int side = which - 1, codec = p.codec[side];
  int64_t unit = static_cast<int64_t>(s) * p.n_kv * (p.capacity / kUnitTokens) + slot / kUnitTokens;
  int64_t step = p.capacity / kUnitTokens;  // units from one kv head to the next
  if (p.table) {
    const int pg =
        page_of(p.table, p.pages_per_seq, p.n_pages, s, slot / (kUnitTokens * kPageUnits));
    if (pg < 0) {
      if (lane == 0) set_err(p.err, KVQ_DEVERR_PAGE);
      return;
    }
    unit = static_cast<int64_t>(pg) * p.n_kv * kPageUnits + (slot / kUnitTokens) % kPageUnits;
    step = kPageUnits;
  }
  const int r = static_cast<int>(slot % kUnitTokens);
  for (int h = h0; h < h1; ++h) {
    float v[4];
    load4<T>(x + h * p.head[which], v);
    uint8_t *u = p.cache[side] + (unit + h * step) * unit_bytes(codec);
    if (side == 0) {
      rotate_lane(p.rope, a, lane, v);
      encode_f32_row_into<0>(codec, v, u, r, lane);
    } else {
      encode_f32_row_into<1>(codec, v, u, r, lane);
    }
  }
}

// Advance the lengths once every row has been placed.
__global__ void advance_lens_kernel(AppendRopeParams p, int32_t *seq_lens) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s >= p.n_seqs) return;
  bool bad;
  const int64_t v = seq_lens[s] + new_rows(p, s, bad);
  if (!bad) seq_lens[s] = static_cast<int32_t>(v > p.capacity ? p.capacity : v);
}

}  // namespace

cudaError_t launch_append_rope(const kvq_layer &L, const kvq_rope &rope, const kvq_rows *q,
                               const kvq_rows &k, const kvq_rows &v, int64_t n_rows,
                               const int32_t *n_new, const int32_t *row_start,
                               const int32_t *positions, void *q_out, int update_lens,
                               cudaStream_t stream) {
  AppendRopeParams p;
  p.rope = rope_args(rope);
  const kvq_rows *rows[3] = {q ? q : &k, &k, &v};
  for (int i = 0; i < 3; ++i) {
    p.x[i] = static_cast<const uint8_t *>(rows[i]->data);
    p.row[i] = rows[i]->row_stride * type_bytes(rows[i]->type);
    p.head[i] = rows[i]->head_stride * type_bytes(rows[i]->type);
  }
  p.q_out = static_cast<__half *>(q_out);
  p.cache[0] = static_cast<uint8_t *>(L.k_cache);
  p.cache[1] = static_cast<uint8_t *>(L.v_cache);
  p.codec[0] = L.codec_k;
  p.codec[1] = L.codec_v;
  p.seq_lens = L.seq_lens;
  p.n_new = n_new;
  p.row_start = row_start;
  p.positions = positions;
  p.table = L.pages_per_seq > 0 ? L.block_table : nullptr;
  p.err = L.err;
  p.n_rows = n_rows;
  p.max_new = n_rows / L.n_seqs;
  p.n_seqs = L.n_seqs;
  p.n_q = L.n_q_heads;
  p.n_kv = L.n_kv_heads;
  p.capacity = L.capacity;
  p.pages_per_seq = L.pages_per_seq;
  p.n_pages = L.n_pages;
  p.q_chunks = q ? (p.n_q + kHeadsPerWarp - 1) / kHeadsPerWarp : 0;
  p.kv_chunks = (p.n_kv + kHeadsPerWarp - 1) / kHeadsPerWarp;
  if (n_rows > 0) {
    const int64_t items = n_rows * (p.q_chunks + 2 * p.kv_chunks);
    const dim3 grid(static_cast<unsigned>((items + kArWarps - 1) / kArWarps)), block(kArThreads);
    const cudaError_t e =
        k.type == KVQ_T_F16    ? launch_pdl(append_rope_kernel<KVQ_T_F16>, grid, block, 0, stream, p)
        : k.type == KVQ_T_BF16 ? launch_pdl(append_rope_kernel<KVQ_T_BF16>, grid, block, 0, stream, p)
                               : launch_pdl(append_rope_kernel<KVQ_T_F32>, grid, block, 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  if (!update_lens || n_rows == 0) return cudaSuccess;
  return launch_pdl(advance_lens_kernel, dim3((L.n_seqs + 127) / 128), dim3(128), 0, stream, p,
                    L.seq_lens);
}

}  // namespace kvq
