// cross.cu -- attention of packed query rows to every cached key of their
// sequence, without a causal mask: cross attention to an encoder's states, and
// the shared part of a decode step behind a common prefix.
//
// o = softmax(scale q K^T) V over the keys below the sequence's length, query
// head h reading kv head h / (n_q / n_kv).
#include <cuda_runtime.h>

#include <math.h>

#include "kvq_launch.h"
#include "kvq_packed.cuh"
#include "kvq_rope.cuh"
#include "kvq_row_decode.cuh"

namespace kvq {
namespace {

constexpr int kCrossWarps = 8;

struct CrossParams {
  const uint8_t *cache[2];
  int codec[2];
  const uint8_t *q;
  int64_t q_row, q_head, out_row, out_head;  // strides in bytes
  int q_type, out_type;
  CrossOut out;
  PackedRows rows;
  const int32_t *seq_lens, *table;
  int32_t *err;
  int n_q, n_kv, G, capacity, max_len, pages_per_seq, n_pages;
  float scale_log2;
};

// A warp per (row, query head), one key after the other.
__global__ void __launch_bounds__(kCrossWarps * 32)
    cross_kernel(const __grid_constant__ CrossParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0) packed_check(p.rows, p.err);
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kCrossWarps + (threadIdx.x >> 5);
  const int64_t row = item / p.n_q;
  const int head = static_cast<int>(item % p.n_q), kvh = head / p.G;
  if (row >= p.rows.n_rows) return;
  int s;
  int64_t i;
  if (!packed_find(p.rows, row, s, i)) return;
  int len = p.seq_lens[s];
  if (len > p.max_len) {
    set_err(p.err, KVQ_DEVERR_MAXLEN);
    len = p.max_len;
  }
  float q[4];
  const uint8_t *qr = p.q + row * p.q_row + head * p.q_head + 8 * lane;
  if (p.q_type == KVQ_T_BF16) load4<KVQ_T_BF16>(qr, q);
  else load4<KVQ_T_F16>(qr, q);
  float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int t = 0; t < len; ++t) {
    const int j = t / kUnitTokens, r = t % kUnitTokens;
    int64_t unit = (static_cast<int64_t>(s) * p.n_kv + kvh) * (p.capacity / kUnitTokens) + j;
    if (p.table) {
      int pg = page_of(p.table, p.pages_per_seq, p.n_pages, s, j / kPageUnits);
      if (pg < 0) {
        set_err(p.err, KVQ_DEVERR_PAGE);
        pg = 0;  // read pool page 0 in its place
      }
      unit = (static_cast<int64_t>(pg) * p.n_kv + kvh) * kPageUnits + j % kPageUnits;
    }
    float x[4];
    decode_row_lane<0>(p.codec[0], p.cache[0] + unit * unit_bytes(p.codec[0]), r, lane, x);
    float a = q[0] * x[0] + q[1] * x[1] + q[2] * x[2] + q[3] * x[3];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) a += __shfl_xor_sync(0xffffffffu, a, k);
    a *= p.scale_log2;
    const float mn = fmaxf(m, a), f = m == -INFINITY ? 0.0f : exp2f(m - mn);
    const float e = mn == -INFINITY ? 0.0f : exp2f(a - mn);
    decode_row_lane<1>(p.codec[1], p.cache[1] + unit * unit_bytes(p.codec[1]), r, lane, x);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = fmaf(o[k], f, e * x[k]);
    l = fmaf(l, f, e);
    m = mn;
  }
  const int64_t at = row * p.n_q + head;
  if (p.out.xo) {  // unnormalised, for a merge
    *reinterpret_cast<float4 *>(p.out.xo + at * kD + 4 * lane) = make_float4(o[0], o[1], o[2], o[3]);
    if (lane == 0) p.out.xml[at] = make_float2(m, l);
    return;
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] *= inv;
  uint8_t *y = static_cast<uint8_t *>(p.out.out) + row * p.out_row + head * p.out_head + 8 * lane;
  if (p.out_type == KVQ_T_BF16) store4<KVQ_T_BF16>(y, o);
  else store4<KVQ_T_F16>(y, o);
  if (p.out.lse && lane == 0)
    p.out.lse[at] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

CrossPlan plan_cross(const kvq_layer &L, int64_t n_rows, int num_sms) {
  CrossPlan pl;
  pl.ws_bytes = 16;
  return pl;
}

cudaError_t launch_cross(const kvq_layer &L, const CrossPlan &pl, const kvq_rows &q,
                         int64_t n_rows, const int32_t *n_new, const int32_t *row_start,
                         float scale, const CrossOut &out, int64_t out_row, int64_t out_head,
                         int out_type, int max_len, void *workspace, cudaStream_t stream) {
  CrossParams p;
  p.cache[0] = static_cast<const uint8_t *>(L.k_cache);
  p.cache[1] = static_cast<const uint8_t *>(L.v_cache);
  p.codec[0] = L.codec_k;
  p.codec[1] = L.codec_v;
  p.q = static_cast<const uint8_t *>(q.data);
  p.q_row = q.row_stride * type_bytes(q.type);
  p.q_head = q.head_stride * type_bytes(q.type);
  p.q_type = q.type;
  p.out = out;
  p.out_row = out_row * 2;
  p.out_head = out_head * 2;
  p.out_type = out_type;
  p.rows = {row_start, n_new, n_rows, n_rows / L.n_seqs, L.n_seqs};
  p.seq_lens = L.seq_lens;
  p.table = L.pages_per_seq > 0 ? L.block_table : nullptr;
  p.err = L.err;
  p.n_q = L.n_q_heads;
  p.n_kv = L.n_kv_heads;
  p.G = L.n_q_heads / L.n_kv_heads;
  p.capacity = L.capacity;
  p.max_len = max_len;
  p.pages_per_seq = L.pages_per_seq;
  p.n_pages = L.n_pages;
  p.scale_log2 = scale * 1.4426950408889634f;
  const int64_t blocks = (n_rows * L.n_q_heads + kCrossWarps - 1) / kCrossWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(cross_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kCrossWarps * 32), 0,
                    stream, p);
}

}  // namespace kvq
