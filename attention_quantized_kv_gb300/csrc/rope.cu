// rope.cu -- rotary positions: the angle table, the rotation of rows, and the
// re-rotation of cached keys after an eviction moved them.
#include <cuda_runtime.h>

#include <math.h>

#include "kvq_encode.cuh"
#include "kvq_launch.h"
#include "kvq_rope.cuh"

namespace kvq {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = kRopeWarps * 32;

// ------------------------------------------------------------------ table

struct TableParams {
  float2 *table;
  int64_t n;             // n_pos * pairs
  int pairs;
  uint64_t turns[kD / 2];  // frequency in units of 2^-64 turns per position
};

// One (position, plane) per thread.  pos * turns mod 2^64 is the angle as an
// exact fraction of a turn; the nearest quarter turn is taken off as an
// integer, so the remainder in [-1/8, 1/8] turns is exact too and rounds once
// to fp32 whatever the position.
__global__ void __launch_bounds__(kRopeThreads) table_kernel(TableParams p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x;
  if (i >= p.n) return;
  const uint64_t pos = static_cast<uint64_t>(i / p.pairs);
  const uint64_t u = pos * p.turns[i % p.pairs];
  const uint32_t quarter = static_cast<uint32_t>((u + (1ull << 61)) >> 62);
  const int64_t r = static_cast<int64_t>(u - (static_cast<uint64_t>(quarter) << 62));
  float s, c;
  sincospif(static_cast<float>(r) * 0x1p-63f, &s, &c);
  const float co = (quarter & 1) ? s : c, si = (quarter & 1) ? c : s;
  p.table[i] = make_float2((quarter + 1) & 2 ? -co : co, quarter & 2 ? -si : si);
}

// ------------------------------------------------------------------ apply

struct ApplyParams {
  RopeArgs rope;
  const uint8_t *x;
  uint8_t *y;
  int64_t x_row, x_head, y_row, y_head;  // strides in bytes
  int64_t n_rows;
  const int32_t *positions;
  int32_t *err;
  int n_heads, pos0, chunks;
  float sign;
};

constexpr int kHeadsPerWarp = 8;  // heads of one row that share a warp's angles

template <int TI, int TO>
__global__ void __launch_bounds__(kRopeThreads) apply_kernel(ApplyParams p) {
  constexpr int SI = sizeof(typename RowType<TI>::type), SO = sizeof(typename RowType<TO>::type);
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int64_t row = item / p.chunks;
  if (row >= p.n_rows) return;
  const int h0 = static_cast<int>(item % p.chunks) * kHeadsPerWarp;
  const int64_t pos = p.positions ? p.positions[row] : p.pos0 + row;
  const LaneAngles a = lane_angles(p.rope, rope_row(p.rope, pos, p.err), lane, p.sign);
  const uint8_t *x = p.x + row * p.x_row + 4 * lane * SI;
  uint8_t *y = p.y + row * p.y_row + 4 * lane * SO;
  for (int h = h0; h < p.n_heads && h < h0 + kHeadsPerWarp; ++h) {
    float v[4];
    load4<TI>(x + h * p.x_head, v);
    rotate_lane(p.rope, a, lane, v);
    store4<TO>(y + h * p.y_head, v);
  }
}

// ------------------------------------------------------------------ shift

struct DeltaParams {
  const int32_t *seq_lens, *evict, *n_evicted;
  int32_t *delta;
  int capacity, max_evict;
};

// delta[s][w] = -(evicted tokens before the one that moves to w).  evict[j] - j
// kept tokens lie before evicted token j, a non-decreasing count, so that
// number is the count of j with evict[j] - j <= w: a binary search.
__global__ void __launch_bounds__(kRopeThreads) delta_kernel(DeltaParams p) {
  grid_dependency_wait();
  const int s = blockIdx.y;
  const int w = blockIdx.x * kRopeThreads + threadIdx.x;
  const int len = min(p.seq_lens[s], p.capacity);
  const int n = max(0, min(p.n_evicted[s], p.max_evict));
  if (w >= len - n) return;
  const int32_t *e = p.evict + static_cast<int64_t>(s) * p.max_evict;
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (e[mid] - mid <= w) lo = mid + 1;
    else hi = mid;
  }
  p.delta[static_cast<int64_t>(s) * p.capacity + w] = -lo;
}

struct ShiftParams {
  RopeArgs rope;
  uint8_t *k;
  const int32_t *seq_lens, *delta, *table;
  int32_t *err;
  int codec, n_kv, capacity, pages_per_seq, n_pages;
};

// One warp per (sequence, token): its K rows of every kv head.
__global__ void __launch_bounds__(kRopeThreads) shift_kernel(ShiftParams p) {
  grid_dependency_wait();
  const int s = blockIdx.y, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  if (t >= min(p.seq_lens[s], p.capacity)) return;
  const int d = p.delta[static_cast<int64_t>(s) * p.capacity + t];
  if (d == 0) return;
  int64_t unit = static_cast<int64_t>(s) * p.n_kv * (p.capacity / kUnitTokens) + t / kUnitTokens;
  int64_t step = p.capacity / kUnitTokens;
  if (p.table) {
    const int pg = page_of(p.table, p.pages_per_seq, p.n_pages, s, t / (kUnitTokens * kPageUnits));
    if (pg < 0) {
      if (lane == 0) set_err(p.err, KVQ_DEVERR_PAGE);
      return;
    }
    unit = static_cast<int64_t>(pg) * p.n_kv * kPageUnits + (t / kUnitTokens) % kPageUnits;
    step = kPageUnits;
  }
  const int64_t by = d;
  const LaneAngles a =
      lane_angles(p.rope, rope_row(p.rope, by < 0 ? -by : by, p.err), lane, d < 0 ? -1.0f : 1.0f);
  for (int h = 0; h < p.n_kv; ++h) {
    uint8_t *u = p.k + (unit + h * step) * unit_bytes(p.codec);
    float x[4];
    load_row<0>(p.codec, u, t % kUnitTokens, lane, x);
    rotate_lane(p.rope, a, lane, x);
    __syncwarp();  // every lane has read its part before any is written
    encode_f32_row_into<0>(p.codec, x, u, t % kUnitTokens, lane);
  }
}

template <int TI, int TO>
cudaError_t launch_apply_t(const ApplyParams &p, cudaStream_t stream) {
  const int64_t blocks = (p.n_rows * p.chunks + kRopeWarps - 1) / kRopeWarps;
  apply_kernel<TI, TO><<<static_cast<unsigned>(blocks), kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(const double *freqs, int rot_dim, int n_pos, float *table,
                              cudaStream_t stream) {
  TableParams p;
  p.table = reinterpret_cast<float2 *>(table);
  p.pairs = rot_dim / 2;
  p.n = static_cast<int64_t>(n_pos) * p.pairs;
  for (int i = 0; i < p.pairs; ++i) p.turns[i] = turns_of(freqs[i]);
  const int64_t blocks = (p.n + kRopeThreads - 1) / kRopeThreads;
  table_kernel<<<static_cast<unsigned>(blocks), kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rope_apply(const kvq_rope &rope, const kvq_rows &x, const kvq_rows &y,
                              int64_t n_rows, int n_heads, const int32_t *positions, int pos0,
                              int transpose, int32_t *err, cudaStream_t stream) {
  ApplyParams p;
  p.rope = rope_args(rope);
  p.x = static_cast<const uint8_t *>(x.data);
  p.y = static_cast<uint8_t *>(y.data);
  p.x_row = x.row_stride * type_bytes(x.type);
  p.x_head = x.head_stride * type_bytes(x.type);
  p.y_row = y.row_stride * type_bytes(y.type);
  p.y_head = y.head_stride * type_bytes(y.type);
  p.n_rows = n_rows;
  p.positions = positions;
  p.err = err;
  p.n_heads = n_heads;
  p.pos0 = pos0;
  p.chunks = (n_heads + kHeadsPerWarp - 1) / kHeadsPerWarp;
  p.sign = transpose ? -1.0f : 1.0f;
  if (x.type == KVQ_T_F16) return launch_apply_t<KVQ_T_F16, KVQ_T_F16>(p, stream);
  if (x.type == KVQ_T_BF16)
    return y.type == KVQ_T_BF16 ? launch_apply_t<KVQ_T_BF16, KVQ_T_BF16>(p, stream)
                                : launch_apply_t<KVQ_T_BF16, KVQ_T_F16>(p, stream);
  return y.type == KVQ_T_F32 ? launch_apply_t<KVQ_T_F32, KVQ_T_F32>(p, stream)
                             : launch_apply_t<KVQ_T_F32, KVQ_T_F16>(p, stream);
}

cudaError_t launch_evict_delta(const kvq_layer &L, const int32_t *evict, const int32_t *n_evicted,
                               int max_evict, int32_t *delta, cudaStream_t stream) {
  DeltaParams p{L.seq_lens, evict, n_evicted, delta, L.capacity, max_evict};
  const dim3 grid((L.capacity + kRopeThreads - 1) / kRopeThreads, L.n_seqs);
  return launch_pdl(delta_kernel, grid, dim3(kRopeThreads), 0, stream, p);
}

cudaError_t launch_rope_shift(const kvq_layer &L, const kvq_rope &rope, const int32_t *delta,
                              cudaStream_t stream) {
  ShiftParams p;
  p.rope = rope_args(rope);
  p.rope.magnitude = 1.0f;  // the rows carry it already
  p.k = static_cast<uint8_t *>(L.k_cache);
  p.seq_lens = L.seq_lens;
  p.delta = delta;
  p.table = L.pages_per_seq > 0 ? L.block_table : nullptr;
  p.err = L.err;
  p.codec = L.codec_k;
  p.n_kv = L.n_kv_heads;
  p.capacity = L.capacity;
  p.pages_per_seq = L.pages_per_seq;
  p.n_pages = L.n_pages;
  const dim3 grid((L.capacity + kRopeWarps - 1) / kRopeWarps, L.n_seqs);
  return launch_pdl(shift_kernel, grid, dim3(kRopeThreads), 0, stream, p);
}

}  // namespace kvq
