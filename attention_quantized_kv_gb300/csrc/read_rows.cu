// read_rows.cu -- cached rows read back as values (fp16, bf16 or fp32): every
// row decoded exactly in fp32 and rounded once to the output's type.
#include <cuda_runtime.h>

#include "kvq_launch.h"
#include "kvq_packed.cuh"
#include "kvq_rope.cuh"
#include "kvq_row_decode.cuh"

namespace kvq {
namespace {

constexpr int kReadWarps = 8;

struct ReadParams {
  const uint8_t *cache[2];
  uint8_t *out[2];          // nullptr: side not read
  int64_t row[2], head[2];  // strides in bytes
  int type[2], codec[2];
  PackedRows rows;
  const int32_t *first, *seq_lens, *table;
  int32_t *err;
  int n_kv, capacity, pages_per_seq, n_pages;
};

// A warp per (row, kv head, side).
__global__ void __launch_bounds__(kReadWarps * 32)
    read_rows_kernel(const __grid_constant__ ReadParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0) packed_check(p.rows, p.err);
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5);
  const int64_t row = item / (2 * p.n_kv);
  const int h = static_cast<int>(item % (2 * p.n_kv)) >> 1, side = item & 1;
  if (row >= p.rows.n_rows || !p.out[side]) return;
  int s;
  int64_t i;
  if (!packed_find(p.rows, row, s, i)) return;
  const int64_t t = (p.first ? p.first[s] : 0) + i;
  if (t < 0 || t >= p.seq_lens[s] || t >= p.capacity) {
    set_err(p.err, KVQ_DEVERR_SEQLEN);
    return;
  }
  const int64_t j = t / kUnitTokens;
  int64_t unit = (static_cast<int64_t>(s) * p.n_kv + h) * (p.capacity / kUnitTokens) + j;
  if (p.table) {
    const int pg = page_of(p.table, p.pages_per_seq, p.n_pages, s, j / kPageUnits);
    if (pg < 0) {
      set_err(p.err, KVQ_DEVERR_PAGE);
      return;
    }
    unit = (static_cast<int64_t>(pg) * p.n_kv + h) * kPageUnits + j % kPageUnits;
  }
  const int codec = p.codec[side], r = static_cast<int>(t % kUnitTokens);
  const uint8_t *u = p.cache[side] + unit * unit_bytes(codec);
  float x[4];
  if (side == 0) decode_row_lane<0>(codec, u, r, lane, x);
  else decode_row_lane<1>(codec, u, r, lane, x);
  uint8_t *y = p.out[side] + row * p.row[side] + h * p.head[side];
  if (p.type[side] == KVQ_T_F32) store4<KVQ_T_F32>(y + 16 * lane, x);
  else if (p.type[side] == KVQ_T_BF16) store4<KVQ_T_BF16>(y + 8 * lane, x);
  else store4<KVQ_T_F16>(y + 8 * lane, x);
}

}  // namespace

cudaError_t launch_read_rows(const kvq_layer &L, const kvq_rows *k, const kvq_rows *v,
                             int64_t n_rows, const int32_t *n_read, const int32_t *row_start,
                             const int32_t *first, cudaStream_t stream) {
  ReadParams p;
  p.cache[0] = static_cast<const uint8_t *>(L.k_cache);
  p.cache[1] = static_cast<const uint8_t *>(L.v_cache);
  p.codec[0] = L.codec_k;
  p.codec[1] = L.codec_v;
  const kvq_rows *rows[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    p.out[i] = rows[i] ? static_cast<uint8_t *>(rows[i]->data) : nullptr;
    p.type[i] = rows[i] ? rows[i]->type : KVQ_T_F16;
    p.row[i] = rows[i] ? rows[i]->row_stride * type_bytes(p.type[i]) : 0;
    p.head[i] = rows[i] ? rows[i]->head_stride * type_bytes(p.type[i]) : 0;
  }
  p.rows = {row_start, n_read, n_rows, n_rows / L.n_seqs, L.n_seqs};
  p.first = first;
  p.seq_lens = L.seq_lens;
  p.table = L.pages_per_seq > 0 ? L.block_table : nullptr;
  p.err = L.err;
  p.n_kv = L.n_kv_heads;
  p.capacity = L.capacity;
  p.pages_per_seq = L.pages_per_seq;
  p.n_pages = L.n_pages;
  const int64_t blocks = (n_rows * 2 * L.n_kv_heads + kReadWarps - 1) / kReadWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(read_rows_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kReadWarps * 32),
                    0, stream, p);
}

}  // namespace kvq
