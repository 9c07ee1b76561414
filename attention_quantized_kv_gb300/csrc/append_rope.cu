// append_rope.cu -- quantize-on-append with the rotary rotation applied on
// the way: new keys are rotated in fp32 and encoded from there, values are
// encoded as they come, and the queries of the same rows are rotated to fp16
// beside them.
//
// One launch reads each value once and writes each code once.  Device times on
// one GB300 against the bytes at the measured 6.78 TB/s: 32768 prompt tokens of
// 32 q / 4 kv heads into f16 caches 103 us (0.98), K f16 / V q8_0 106 us (0.93),
// q8_0 109 us (0.88), q4_0 113 us (0.83), turbo4 138 us (0.68): HBM bounds the
// first; the last issues 106 M warp instructions, 84 us of them at full issue,
// and 0.61 per scheduler and cycle behind loads and dependent instructions.
// 2048 tokens into q8_0 caches 12.8 us (0.55) and a mixed batch of 1821 rows
// 14.4 us (0.54): two waves of blocks, each a chain of dependent loads (row ->
// length -> page, and only then the rows).  16 single tokens of 40 q / 8 kv
// heads 3.4 us, one such chain.
#include <cuda_runtime.h>

#include "kvq_encode.cuh"
#include "kvq_launch.h"
#include "kvq_quad.cuh"

namespace kvq {
namespace {

constexpr int kArWarps = 8;
constexpr int kArThreads = kArWarps * 32;
constexpr int kMaxHeads = 8;  // heads of one row that share a warp's angles
constexpr int kRowSlotsPerSm = 128;  // rows x heads per SM up to which an append goes by rows

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
  int q_hpw, hpw;           // heads per warp item, of q and of k or v
  int q_chunks, kv_chunks;  // items of a row's q, of its k (or v) heads
  int64_t kv_blocks;             // prompts: blocks that place keys and values
  int kind;                      // quad_kind
  bool eight;                    // eight_lanes
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
  if (!p.n_new) return 1;  // one row per sequence
  const int n = p.n_new[s];
  bad = n < 0 || n > p.max_new;
  return bad ? 0 : n;
}

// The sequence of a row and its index there; false for padding.
__device__ __forceinline__ bool find_row(const AppendRopeParams &p, int64_t row, int &s, int &i,
                                         int &n) {
  if (!p.row_start) {
    s = static_cast<int>(row / p.max_new);
    i = static_cast<int>(row - s * p.max_new);
    n = p.n_new ? p.n_new[s] : 1;
    return i < n && n <= p.max_new;
  }
  int lo = 0, hi = p.n_seqs;  // the last s with row_start[s] <= row
  while (lo + 1 < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.row_start[mid] <= row) lo = mid;
    else hi = mid;
  }
  s = lo;
  const int a = p.row_start[s], b = p.row_start[s + 1];
  i = static_cast<int>(row - a);
  n = b - a;
  return a >= 0 && row >= a && row < b && b <= p.n_rows;
}

// find_row of one row by a whole warp: each round narrows the range 32 times,
// so up to 32 sequences cost one dependent load.
__device__ __forceinline__ bool find_row_warp(const AppendRopeParams &p, int64_t row, int lane,
                                              int &s, int &i) {
  if (!p.row_start) {
    int n;
    return find_row(p, row, s, i, n);
  }
  int lo = 0, n = p.n_seqs;
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < n && p.row_start[lo + at] <= row);
    const int k = max(__popc(le) - 1, 0) * step;
    lo += k;
    n = min(step, n - k);
  }
  s = lo;
  const int a = p.row_start[s], b = p.row_start[s + 1];
  i = static_cast<int>(row - a);
  return a >= 0 && row >= a && row < b && b <= p.n_rows;
}

// Unit of kv head 0 that holds slot `slot` of sequence s; -1 and the error
// bit where there is no place.
__device__ __forceinline__ int64_t unit_of(const AppendRopeParams &p, int s, int64_t slot) {
  if (slot < 0 || slot >= p.capacity) {
    set_err(p.err, KVQ_DEVERR_CAPACITY);
    return -1;
  }
  const int64_t j = slot / kUnitTokens;
  if (!p.table) return static_cast<int64_t>(s) * p.n_kv * (p.capacity / kUnitTokens) + j;
  const int pg = page_of(p.table, p.pages_per_seq, p.n_pages, s, j / kPageUnits);
  if (pg < 0) {
    set_err(p.err, KVQ_DEVERR_PAGE);
    return -1;
  }
  return static_cast<int64_t>(pg) * p.n_kv * kPageUnits + j % kPageUnits;
}
// Units from one kv head to the next.
__device__ __forceinline__ int64_t unit_step(const AppendRopeParams &p) {
  return p.table ? kPageUnits : p.capacity / kUnitTokens;
}

__device__ __forceinline__ void check_counts(const AppendRopeParams &p) {
  if (blockIdx.x != 0) return;
  for (int s = threadIdx.x; s < p.n_seqs; s += kArThreads) {
    bool bad;
    new_rows(p, s, bad);
    if (bad) set_err(p.err, KVQ_DEVERR_ROWS);
  }
}

// Where dim d of token row r lies in an f16 unit of V.  A token's values lie
// four to a 128-byte line there, so a row is stored one value per lane, dims
// 32 j + lane: 8 lines per store.  (Four consecutive dims per lane, as the
// encoders hold them, touch 32 each time; a window of 16 single tokens took
// 8 us longer that way.)
__device__ __forceinline__ uint8_t *v_f16_place(uint8_t *unit, int r, int d) {
  return unit + (d >> 4) * 512 + (4 * ((d & 15) >> 1) + ((r & 7) >> 1)) * 16 +
         ((r >> 3) * 4 + (d & 1) * 2 + (r & 1)) * 2;
}

// One warp: up to 16 heads of q of one row (planes that eight lanes hold).
template <int T>
__device__ __forceinline__ void q_item(const AppendRopeParams &p, int64_t row, int chunk,
                                       int lane) {
  constexpr int N = T == KVQ_T_F32 ? 2 : 4;
  const int h0 = chunk * p.q_hpw;
  rotate_heads_eight<T, KVQ_T_F16, N>(
      p.rope, p.x[0] + row * p.row[0] + h0 * p.head[0], p.head[0],
      reinterpret_cast<uint8_t *>(p.q_out + (row * p.n_q + h0) * kD), 2 * kD,
      min(p.q_hpw, p.n_q - h0), 1.0f, lane, [&]() -> const float * {
        int s, i;
        if (!find_row_warp(p, row, lane, s, i)) return nullptr;
        return rope_row(
            p.rope, p.positions ? p.positions[row] : static_cast<int64_t>(p.seq_lens[s]) + i,
            p.err);
      });
}

// One warp: up to hpw heads of q (which 0), k (1) or v (2) of one row, every
// value requested before the row's place and angles are looked up.
template <int T>
__device__ __forceinline__ void row_item(const AppendRopeParams &p, int64_t row, int which,
                                         int chunk, int lane) {
  using Raw = typename RowType<T>::raw4;
  constexpr int S = sizeof(typename RowType<T>::type);
  const int per = which == 0 ? p.q_hpw : p.hpw;
  const int h0 = chunk * per, nh = min(per, (which == 0 ? p.n_q : p.n_kv) - h0);
  const uint8_t *x = p.x[which] + row * p.row[which] + h0 * p.head[which] + 4 * lane * S;
  Raw raw[kMaxHeads];
#pragma unroll
  for (int h = 0; h < kMaxHeads; ++h)
    if (h < nh) raw[h] = *reinterpret_cast<const Raw *>(x + h * p.head[which]);
  int s, i;
  if (!find_row_warp(p, row, lane, s, i)) return;
  const int64_t slot = static_cast<int64_t>(p.seq_lens[s]) + i;
  LaneAngles a;
  if (which < 2)
    a = lane_angles(p.rope, rope_row(p.rope, p.positions ? p.positions[row] : slot, p.err), lane);
  if (which == 0) {
    with_lanes(p.rope, [&](auto lanes) {
#pragma unroll
      for (int h = 0; h < kMaxHeads; ++h)
        if (h < nh) {
          float v[4];
          load4<T>(&raw[h], v);
          rotate_lane<decltype(lanes)::value>(p.rope, a, lane, v);
          store4<KVQ_T_F16>(p.q_out + (row * p.n_q + h0 + h) * kD + 4 * lane, v);
        }
    });
    return;
  }
  const int64_t unit = unit_of(p, s, slot), step = unit_step(p);
  if (unit < 0) return;
  const int r = static_cast<int>(slot % kUnitTokens), codec = p.codec[which - 1];
#pragma unroll 1
  for (int h = 0; h < nh; ++h) {
    float v[4];
    Raw w = raw[0];  // (a rotating window instead of an indexed array: registers)
    load4<T>(&w, v);
#pragma unroll
    for (int k = 0; k + 1 < kMaxHeads; ++k) raw[k] = raw[k + 1];
    uint8_t *u = p.cache[which - 1] + (unit + (h0 + h) * step) * unit_bytes(codec);
    if (which == 1) {
      rotate_lane(p.rope, a, lane, v);
      encode_f32_row_into<0>(codec, v, u, r, lane);
    } else if (codec == KVQ_F16) {
      const uint32_t lo = pack_half2(v[0], v[1]), hi = pack_half2(v[2], v[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // dim 32 j + lane: of lane 8 j + lane / 4
        const uint32_t a = __shfl_sync(0xffffffffu, lo, 8 * j + (lane >> 2));
        const uint32_t b = __shfl_sync(0xffffffffu, hi, 8 * j + (lane >> 2));
        st_u16(v_f16_place(u, r, 32 * j + lane), ((lane & 2) ? b : a) >> (16 * (lane & 1)));
      }
    } else {
      encode_f32_row_into<1>(codec, v, u, r, lane);
    }
  }
}

// Decode steps and other short appends: one warp per row item.
template <int T>
__global__ void __launch_bounds__(kArThreads)
    append_rows_kernel(const __grid_constant__ AppendRopeParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  check_counts(p);
  const int lane = threadIdx.x & 31, per_row = p.q_chunks + 2 * p.kv_chunks;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kArWarps + (threadIdx.x >> 5);
  const int64_t row = item / per_row;
  if (row >= p.n_rows) return;
  int chunk = static_cast<int>(item % per_row), which = 0;
  if (chunk >= p.q_chunks) {
    chunk -= p.q_chunks;
    which = 1 + chunk / p.kv_chunks;
    chunk %= p.kv_chunks;
  }
  if (which == 0 && p.eight) q_item<T>(p, row, chunk, lane);
  else row_item<T>(p, row, which, chunk, lane);
}

// ------------------------------------------------------------------ prompts
//
// A prompt fills whole 16-token units, whose bytes interleave their tokens
// (include/kvq.h): written row by row the V side would go out as 2-byte
// stores, one 32-byte sector each.  So one warp takes a whole unit of one kv
// head, and stores it as contiguous 512-byte pieces.
// The window's rows are copied into shared memory, 16 of them in flight (K rows
// read into registers instead, 32768 rows: f16 106 instead of 103 us, q8_0 112
// instead of 110 us).
//   K: every quad of lanes takes two rows in the unit's own order, rotates,
//      encodes and stores them (kvq_quad.cuh), whatever units they belong to.
//   V: two lanes per row encode its four blocks; the unit is put together 16
//      bytes per lane from the 16 rows' codes.
//
// Packed rows are cut into windows of 16, whatever the lengths.  For V a
// window's warp places the rows of every unit whose first new row lies in the
// window: no other warp writes that unit, so an incomplete one with enough new
// rows is put together over its old bytes; rows of others are stored one by
// one.

// A staged row: the input's 128 values, replaced (but for f16) by 128 one-byte
// codes and the block scales (4, or 1 for turbo4) behind them.
template <int T>
struct Stage {
  static constexpr int S = sizeof(typename RowType<T>::type);
  static constexpr int kPitch = kD * S + 16;  // rows 4 banks apart
  static constexpr int kWarpBytes = kUnitTokens * kPitch;
  static constexpr int kBytes = kArWarps * kWarpBytes;
};
// New rows of a unit that are worth putting it together over its old bytes; 3,
// 8, 12 or 16: a prompt of 2047 rows 11.4, 11.4, 11.4, 13.3 us, 16 prompts of
// 16 rows 10.9, 9.3, 9.4, 9.4 us, 64 of 16 rows 19.7, 14.9, 14.0, 13.4 us.
constexpr int kGroupRows = 12;
constexpr int kScaleAt = kD;  // byte offset of a staged row's scales

// Copy the rows of `mask` (bit j: row j of the 16 at x) into their stage slots.
template <int T>
__device__ __forceinline__ void stage_rows(uint8_t *stage, const uint8_t *x, int64_t row_bytes,
                                           unsigned mask, int lane) {
  constexpr int kLanes = kD * Stage<T>::S / 16;  // lanes that carry one row
  constexpr int kPerPass = 32 / kLanes;
#pragma unroll
  for (int j0 = 0; j0 < kUnitTokens; j0 += kPerPass) {
    const int j = j0 + lane / kLanes, off = (lane % kLanes) * 16;
    if ((mask >> j) & 1u)
      copy_async16(stage + j * Stage<T>::kPitch + off, x + j * row_bytes + off);
  }
  copy_async_wait_all();
  __syncwarp();
}

// Encode the staged row at `row`, of which the lane holds x, in place (turbo4).
__device__ __forceinline__ void encode_staged_turbo4(const float (&x)[4], uint8_t *row, int lane) {
  int q[4];
  __half d16;
  encode_turbo4(x, lane, q, d16);
  reinterpret_cast<uint32_t *>(row)[lane] = (q[0] & 0xff) | ((q[1] & 0xff) << 8) |
                                            ((q[2] & 0xff) << 16) |
                                            (static_cast<uint32_t>(q[3] & 0xff) << 24);
  if (lane == 0) *reinterpret_cast<__half *>(row + kScaleAt) = d16;
}

// Store a staged row as token row r of a unit of V (f16: the input's values, of
// type T, still).
template <int T>
__device__ __forceinline__ void store_staged(int codec, const uint8_t *row, uint8_t *unit, int r,
                                             int lane) {
  if (codec == KVQ_F16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const auto v = reinterpret_cast<const typename RowType<T>::type *>(row)[32 * j + lane];
      st_u16(v_f16_place(unit, r, 32 * j + lane),
             __half_as_ushort(__float2half_rn(static_cast<float>(v))));
    }
    return;
  }
  const uint32_t w = reinterpret_cast<const uint32_t *>(row)[lane];
  int q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = (w >> (8 * i)) & 0xff;
  const __half d16 =
      reinterpret_cast<const __half *>(row + kScaleAt)[codec == KVQ_TURBO4 ? 0 : lane >> 3];
  store_row<1>(codec, unit, r, lane, make_uint2(0u, 0u), q, d16);
}

// The bytes of a V unit's chunk c that belong to the token rows of the mask.
__device__ __forceinline__ uint4 chunk_mask(int codec, int c, unsigned rows) {
  const int data = codec == KVQ_F16 ? 256 : codec == KVQ_Q8_0 ? 128 : 64, k = c - data;
  const int tig = c & 3;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (c < data && nibble_codec(codec)) {  // byte par * 2 + rh: row 2 tig + par + 8 rh
      o[i] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if ((rows >> (2 * tig + (b >> 1) + 8 * (b & 1))) & 1u) o[i] |= 0xffu << (8 * b);
    } else {  // halves par of rows 2 tig + par + 8 rh
      const int r = c < data              ? 2 * tig + 8 * (codec == KVQ_F16 ? i >> 1 : i & 1)
                    : codec == KVQ_TURBO4 ? 2 * (2 * k + (i >> 1)) + 8 * (i & 1)
                                          : 2 * (k >> 1) + 8 * (i & 1);
      o[i] = ((rows >> r) & 1u ? 0x0000ffffu : 0u) | ((rows >> (r + 1)) & 1u ? 0xffff0000u : 0u);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// 16 bytes of a V unit, chunk c, from the staged rows: the inverse of the
// placement formulas of include/kvq.h.
template <int T>
__device__ __forceinline__ uint4 unit_chunk(int codec, const uint8_t *s, int c) {
  constexpr int kPitch = Stage<T>::kPitch;
  auto w16 = [&](int r, int byte) -> uint32_t {
    return *reinterpret_cast<const uint16_t *>(s + r * kPitch + byte);
  };
  uint32_t o[4];
  const int tig = c & 3, gq = (c >> 2) & 7, hi = c >> 5;
  if (codec == KVQ_F16) {  // hi = mt: dims 16 mt + 2 gq, + 1 of rows 2 tig + par + 8 rh
#pragma unroll
    for (int rh = 0; rh < 2; ++rh) {
      uint32_t h[2];  // par: the row's two values as fp16
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const uint8_t *at = s + (2 * tig + par + 8 * rh) * kPitch + (16 * hi + 2 * gq) * Stage<T>::S;
        if (T == KVQ_T_F32) {
          const float2 x = *reinterpret_cast<const float2 *>(at);
          h[par] = pack_half2(x.x, x.y);
        } else {
          h[par] = *reinterpret_cast<const uint32_t *>(at);
          if (T == KVQ_T_BF16)
            h[par] = pack_half2(__uint_as_float(h[par] << 16), __uint_as_float(h[par] & 0xffff0000u));
        }
      }
      o[2 * rh] = __byte_perm(h[0], h[1], 0x5410);
      o[2 * rh + 1] = __byte_perm(h[0], h[1], 0x7632);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
  const int data = codec == KVQ_Q8_0 ? 128 : 64;  // chunks of codes, then of scales
  const int k = c - data;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (c >= data) {
      // turbo4: one scale per row, tig 2k and 2k + 1; else tig = k / 2, blocks
      // 2 (k % 2) and + 1; rh; par
      const int r = (codec == KVQ_TURBO4 ? 2 * (2 * k + (i >> 1)) : 2 * (k >> 1)) + 8 * (i & 1);
      const int at = kScaleAt + (codec == KVQ_TURBO4 ? 0 : 2 * (2 * (k & 1) + (i >> 1)));
      o[i] = w16(r, at) | (w16(r + 1, at) << 16);
    } else if (codec == KVQ_Q8_0) {  // (mt & 1, rh): dims 32 hi + 16 (mt & 1) + 2 gq, + 1
      const int d = 32 * hi + 16 * (i >> 1) + 2 * gq, r = 2 * tig + 8 * (i & 1);
      o[i] = w16(r, d) | (w16(r + 1, d) << 16);
    } else {  // mt = 4 hi + i: byte par * 2 + rh, levels of dims d low, d + 16 high
      const int mt = 4 * hi + i, d = 32 * (mt >> 1) + 8 * (mt & 1) + gq;
      o[i] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint8_t *row = s + (2 * tig + (b >> 1) + 8 * (b & 1)) * kPitch;
        // (a slot without a row holds anything: it must not reach other bytes)
        o[i] |= ((row[d] | (static_cast<uint32_t>(row[d + 16]) << 4)) & 0xffu) << (8 * b);
      }
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Encode the staged rows' four 32-value blocks in place, lane l blocks
// 2 (l / 16) and + 1 of row l % 16, each in registers: one division per block
// and no exchange between lanes (q8_0 and q4_0).  slots: those that hold a row.
template <int T, int DC>
__device__ __forceinline__ void encode_staged_blocks(uint8_t *stage, unsigned slots, int lane) {
  const bool live = (slots >> (lane & 15)) & 1u;
  uint8_t *row = stage + (lane & 15) * Stage<T>::kPitch;
  const int b0 = 2 * (lane >> 4);
  uint32_t code[2][8];
  __half d16[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float x[32];
#pragma unroll
    for (int i = 0; i < 32 * Stage<T>::S / 16; ++i) {
      const uint4 raw =
          *reinterpret_cast<const uint4 *>(row + (b0 + k) * 32 * Stage<T>::S + 16 * i);
      if (T == KVQ_T_F32) {
        load4<T>(&raw, reinterpret_cast<float(&)[4]>(x[4 * i]));
      } else {
        load4<T>(&raw, reinterpret_cast<float(&)[4]>(x[8 * i]));
        load4<T>(&raw.z, reinterpret_cast<float(&)[4]>(x[8 * i + 4]));
      }
    }
    float d;
    if (DC == KVQ_Q8_0) {
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) a = fmaxf(a, fabsf(x[i]));
      d = __fdiv_rn(a, 127.0f);
    } else {
      float hi = -INFINITY, lo = INFINITY;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        hi = fmaxf(hi, x[i]);
        lo = fminf(lo, x[i]);
      }
      float m = hi > -lo ? hi : lo;
      if (hi == -lo) {  // the first of them (none: all NaN)
        m = 0.0f;
#pragma unroll
        for (int i = 31; i >= 0; --i)
          if (fabsf(x[i]) == hi) m = x[i];
      }
      d = __fdiv_rn(m, -8.0f);
    }
    d16[k] = __float2half_rn(d);
    const float rcp = d != 0.0f ? __frcp_rn(d) : 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      const uint2 c = quad_codes8<DC>(reinterpret_cast<const float(&)[8]>(x[i]), d, rcp, live);
      code[k][i / 4] = DC == KVQ_Q8_0 ? c.x : clamp15x4(c.x);
      code[k][i / 4 + 1] = DC == KVQ_Q8_0 ? c.y : clamp15x4(c.y);
    }
  }
  __syncwarp();  // both lanes of a row have read it before its codes replace it
  uint4 *out = reinterpret_cast<uint4 *>(row + 32 * b0);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    out[2 * k] = make_uint4(code[k][0], code[k][1], code[k][2], code[k][3]);
    out[2 * k + 1] = make_uint4(code[k][4], code[k][5], code[k][6], code[k][7]);
  }
  *reinterpret_cast<__half2 *>(row + kScaleAt + 2 * b0) = __halves2half2(d16[0], d16[1]);
}

// A window's 16 rows of K, at x, which may lie in any units: lane j knows row
// j's position, unit (-1: none) and row there.  All of them are requested at
// once; then every quad turns, encodes and stores rows g and g + 8, one after
// the other where the encoder's registers are many.
template <int T, int CODEC>
__device__ __forceinline__ void quad_window(const AppendRopeParams &p, const uint8_t *x,
                                            int64_t pos, int64_t unit, int r, uint8_t *stage,
                                            int lane) {
  constexpr int S = Stage<T>::S;
  const int g = lane >> 2, w = lane & 3;
  stage_rows<T>(stage, x, p.row[1], __ballot_sync(0xffffffffu, unit >= 0), lane);
#pragma unroll (CODEC == KVQ_F16 ? 2 : 1)
  for (int rh = 0; rh < 2; ++rh) {
    const int64_t at = __shfl_sync(0xffffffffu, unit, g + 8 * rh);
    const int64_t ps = __shfl_sync(0xffffffffu, pos, g + 8 * rh);
    const int rr = __shfl_sync(0xffffffffu, r, g + 8 * rh);
    const uint8_t *mine = stage + (g + 8 * rh) * Stage<T>::kPitch;
    float v[8][4];
#pragma unroll
    for (int c = 0; c < 8; ++c) load4<T>(mine + (16 * c + 4 * w) * S, v[c]);
    const float *row = at >= 0 ? rope_row(p.rope, ps, p.err) : p.rope.table;
    if (p.kind == kQuadAny)
      quad_rotate_any<false>(
          p.rope, row, w, 1.0f, [&](int d, float(&o)[4]) { load4<T>(mine + d * S, o); },
          [&](int d) { return load1<T>(mine + d * S); }, v);
    else
      quad_rotate<false>(p.rope, p.kind, row, w, 1.0f, v);
    QuadCodes<CODEC> q;
    quad_encode<CODEC>(v, w, at >= 0, q);
    if (at >= 0) quad_store_row<CODEC>(p.cache[0] + at * unit_bytes(CODEC), rr, w, q);
  }
}

// Lane j's row r0 + j of a window (lanes below 16; the others hold none): its
// sequence's new rows n, its index i among them, its position, its unit of kv
// head 0 (-1: no place) and its row there.
struct WindowRow {
  int64_t pos = 0, unit = -1;
  int i = 0, n = 0, r = 0;
};
__device__ __forceinline__ WindowRow window_row(const AppendRopeParams &p, int64_t r0, int lane) {
  WindowRow w;
  const int64_t row = r0 + lane;
  int s = 0;
  if (lane < kUnitTokens && row < p.n_rows && find_row(p, row, s, w.i, w.n)) {
    const int64_t slot = static_cast<int64_t>(p.seq_lens[s]) + w.i;
    w.pos = p.positions ? p.positions[row] : slot;
    w.r = static_cast<int>(slot & (kUnitTokens - 1));
    w.unit = unit_of(p, s, slot);
  }
  return w;
}

template <int T>
__device__ __forceinline__ void k_window(const AppendRopeParams &p, int64_t r0, int h,
                                         uint8_t *stage, int lane) {
  const WindowRow w = window_row(p, r0, lane);
  const uint8_t *x = p.x[1] + r0 * p.row[1] + h * p.head[1];
  const int64_t unit = w.unit < 0 ? -1 : w.unit + h * unit_step(p);
  switch (p.codec[0]) {
    case KVQ_F16: quad_window<T, KVQ_F16>(p, x, w.pos, unit, w.r, stage, lane); break;
    case KVQ_Q8_0: quad_window<T, KVQ_Q8_0>(p, x, w.pos, unit, w.r, stage, lane); break;
    case KVQ_Q4_0: quad_window<T, KVQ_Q4_0>(p, x, w.pos, unit, w.r, stage, lane); break;
    default: quad_window<T, KVQ_TURBO4>(p, x, w.pos, unit, w.r, stage, lane); break;
  }
}

template <int T>
__device__ __forceinline__ void v_window(const AppendRopeParams &p, int64_t r0, int h,
                                         uint8_t *stage, int lane) {
  constexpr int kPitch = Stage<T>::kPitch, S = Stage<T>::S;
  const int codec = p.codec[1];
  const WindowRow w = window_row(p, r0, lane);
  const uint8_t *x = p.x[2] + r0 * p.row[2] + h * p.head[2];
  const int64_t unit = w.unit < 0 ? -1 : w.unit + h * unit_step(p);
  const int r = w.r;
  // The new rows of this row's unit: how many, and whether this is the first.
  const int before = min(r, w.i), count = before + min(kUnitTokens - r, w.n - w.i);
  const unsigned few = __ballot_sync(0xffffffffu, unit >= 0 && count < kGroupRows);
  unsigned first = __ballot_sync(0xffffffffu, unit >= 0 && before == 0 && count >= kGroupRows);
  // Stage slots: token rows of a unit, or (few) rows of the window.
#pragma unroll 1
  for (bool group = few == 0; !group || first; group = true) {
    const int j0 = group ? __ffs(first) - 1 : 0;  // row r0 + j0 goes to slot k0
    const int k0 = group ? __shfl_sync(0xffffffffu, r, j0) : 0;
    const unsigned slots =
        group ? ((1u << __shfl_sync(0xffffffffu, count, j0)) - 1) << k0 : few;
    uint4 *dst = nullptr;
    if (group) {
      first &= first - 1;
      dst = reinterpret_cast<uint4 *>(p.cache[1] +
                                      __shfl_sync(0xffffffffu, unit, j0) * unit_bytes(codec));
      // an incomplete unit's old bytes, asked for beside the rows
      if (slots != (1u << kUnitTokens) - 1 && lane * 128 < unit_bytes(codec))
        asm volatile("prefetch.global.L1 [%0];\n" ::"l"(reinterpret_cast<uint8_t *>(dst) + lane * 128));
    }
    stage_rows<T>(stage, x + (j0 - k0) * p.row[2], p.row[2], slots, lane);
    if (codec == KVQ_Q8_0) {
      encode_staged_blocks<T, KVQ_Q8_0>(stage, slots, lane);
    } else if (codec == KVQ_Q4_0) {
      encode_staged_blocks<T, KVQ_Q4_0>(stage, slots, lane);
    } else if (codec == KVQ_TURBO4) {  // (f16: converted on the way out)
#pragma unroll 1
      for (unsigned m = slots; m; m &= m - 1) {
        uint8_t *row = stage + (__ffs(m) - 1) * kPitch;
        float v[4];
        load4<T>(row + 4 * lane * S, v);
        __syncwarp();  // every lane has read its part before the codes replace it
        encode_staged_turbo4(v, row, lane);
      }
    }
    __syncwarp();
    if (group) {
      const int chunks = unit_bytes(codec) / 16;
      if (slots == (1u << kUnitTokens) - 1) {
        for (int c = lane; c < chunks; c += 32) dst[c] = unit_chunk<T>(codec, stage, c);
      } else {
        constexpr int kAhead = 4;  // old pieces requested at once
        for (int c0 = lane; c0 < chunks; c0 += 32 * kAhead) {
          uint4 old[kAhead];
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
            if (c0 + 32 * i < chunks) old[i] = dst[c0 + 32 * i];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int c = c0 + 32 * i;
            if (c >= chunks) break;
            const uint4 m = chunk_mask(codec, c, slots), b = old[i];
            const uint4 a = unit_chunk<T>(codec, stage, c);
            dst[c] = make_uint4((a.x & m.x) | (b.x & ~m.x), (a.y & m.y) | (b.y & ~m.y),
                                (a.z & m.z) | (b.z & ~m.z), (a.w & m.w) | (b.w & ~m.w));
          }
        }
      }
    } else {
#pragma unroll 1
      for (unsigned m = slots; m; m &= m - 1) {
        const int k = __ffs(m) - 1;
        store_staged<T>(codec, stage + k * kPitch,
                        p.cache[1] + __shfl_sync(0xffffffffu, unit, k) * unit_bytes(codec),
                        __shfl_sync(0xffffffffu, r, k), lane);
      }
    }
    __syncwarp();  // the slots are free again
  }
}

template <int T>
__global__ void __launch_bounds__(kArThreads, T == KVQ_T_F32 ? 2 : 3)
    append_prompt_kernel(const __grid_constant__ AppendRopeParams p) {
  extern __shared__ __align__(16) uint8_t stage[];
  grid_dependency_wait();
  grid_launch_dependents();
  check_counts(p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Blocks of keys and values (first every (window, kv head) of K, then of V)
  // alternate with blocks of q rows while there are both: the encoders'
  // instructions and the q rows' bytes share an SM (32768 rows, q8_0: 111 us;
  // all of K and V first 118, spread over the whole grid 116; 2048 rows 13.0,
  // 12.8, 14.7 us).
  const int64_t b = blockIdx.x, pairs = min(p.kv_blocks, static_cast<int64_t>(gridDim.x) - p.kv_blocks);
  const bool kv = b < 2 * pairs ? b % 2 == 0 : b - pairs < p.kv_blocks;
  const int64_t at = b < 2 * pairs ? b / 2 : kv ? b - pairs : b - p.kv_blocks;
  if (kv) {
    const int64_t item = at * kArWarps + warp;
    const int64_t per_side = (p.n_rows + kUnitTokens - 1) / kUnitTokens * p.n_kv;
    if (item >= 2 * per_side) return;
    uint8_t *mine = stage + warp * Stage<T>::kWarpBytes;
    if (item < per_side)
      k_window<T>(p, item / p.n_kv * kUnitTokens, static_cast<int>(item % p.n_kv), mine, lane);
    else
      v_window<T>(p, (item - per_side) / p.n_kv * kUnitTokens,
                  static_cast<int>((item - per_side) % p.n_kv), mine, lane);
  } else {
    const int64_t item = at * kArWarps + warp;
    const int64_t row = item / p.q_chunks;
    if (row >= p.n_rows) return;
    if (p.eight) q_item<T>(p, row, static_cast<int>(item % p.q_chunks), lane);
    else row_item<T>(p, row, 0, static_cast<int>(item % p.q_chunks), lane);
  }
}

template <int T>
void set_q_items(AppendRopeParams &p, int hpw) {
  p.q_hpw = hpw;
  if (p.q_chunks) p.q_chunks = (p.n_q + hpw - 1) / hpw;
}

template <int T>
cudaError_t launch_rows(AppendRopeParams &p, int num_sms, cudaStream_t stream) {
  // A row's k and v heads go to one warp each while the grid is small (the
  // encoder's latency is paid once), to up to eight, sharing the angles, when
  // it is not; q heads four at a time where eight lanes hold a row.
  const int64_t slots = p.n_rows * (p.n_q * (p.q_chunks > 0) + 2 * p.n_kv);
  while (p.hpw < kMaxHeads && slots / p.hpw > static_cast<int64_t>(num_sms) * 16) p.hpw *= 2;
  set_q_items<T>(p, p.eight ? (p.hpw > 4 ? p.hpw : 4) : p.hpw);
  p.kv_chunks = (p.n_kv + p.hpw - 1) / p.hpw;
  const int64_t items = p.n_rows * (p.q_chunks + 2 * p.kv_chunks);
  const int64_t blocks = (items + kArWarps - 1) / kArWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(append_rows_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kArThreads), 0,
                    stream, p);
}

template <int T>
cudaError_t launch_prompt(AppendRopeParams &p, cudaStream_t stream) {
  static std::atomic<uint64_t> optin{0};
  const cudaError_t e = smem_optin(append_prompt_kernel<T>, Stage<T>::kBytes, optin);
  if (e != cudaSuccess) return e;
  set_q_items<T>(p, !p.eight ? kMaxHeads : T == KVQ_T_F32 ? 8 : 16);
  const int64_t windows = (p.n_rows + kUnitTokens - 1) / kUnitTokens;
  p.kv_blocks = (windows * 2 * p.n_kv + kArWarps - 1) / kArWarps;
  const int64_t blocks = p.kv_blocks + (p.n_rows * p.q_chunks + kArWarps - 1) / kArWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(append_prompt_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kArThreads),
                    Stage<T>::kBytes, stream, p);
}

template <int T>
cudaError_t launch_append_t(AppendRopeParams &p, int num_sms, cudaStream_t stream) {
  // Short appends go row by row, whatever their sequences: the chain of one
  // row is 3 us, of a window 6 to 10.  With 40 q / 8 kv heads and f16 caches
  // 256 rows take 5.7 us by rows and 6.6 (one sequence) to 9.7 us (64) by
  // windows, 512 rows 9.7 and 7.7 to 10.7 us, 2048 rows 31 and 11.4 to 18 us;
  // q8_0 caches cross at the same sizes.
  const int64_t slots = p.n_rows * (p.n_q * (p.q_chunks > 0) + 2 * p.n_kv);
  return slots > static_cast<int64_t>(num_sms) * kRowSlotsPerSm
             ? launch_prompt<T>(p, stream)
             : launch_rows<T>(p, num_sms, stream);
}

// Advance the lengths once every row has been placed.
__global__ void advance_lens_kernel(AppendRopeParams p, int32_t *seq_lens) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s >= p.n_seqs) return;
  bool bad;
  const int64_t old = seq_lens[s], v = old + new_rows(p, s, bad);
  if (!bad && old >= 0) seq_lens[s] = static_cast<int32_t>(v > p.capacity ? p.capacity : v);
}

}  // namespace

cudaError_t launch_append_rope(const kvq_layer &L, const kvq_rope &rope, const kvq_rows *q,
                               const kvq_rows &k, const kvq_rows &v, int64_t n_rows,
                               const int32_t *n_new, const int32_t *row_start,
                               const int32_t *positions, void *q_out, int update_lens,
                               int num_sms, cudaStream_t stream) {
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
  p.kind = quad_kind(p.rope);
  p.eight = eight_lanes(p.rope);
  p.q_hpw = p.hpw = 1;
  p.q_chunks = q ? 1 : 0;
  if (n_rows > 0) {
    const cudaError_t e = k.type == KVQ_T_F16    ? launch_append_t<KVQ_T_F16>(p, num_sms, stream)
                          : k.type == KVQ_T_BF16 ? launch_append_t<KVQ_T_BF16>(p, num_sms, stream)
                                                 : launch_append_t<KVQ_T_F32>(p, num_sms, stream);
    if (e != cudaSuccess) return e;
  }
  if (!update_lens || n_rows == 0) return cudaSuccess;
  return launch_pdl(advance_lens_kernel, dim3((L.n_seqs + 127) / 128), dim3(128), 0, stream, p,
                    L.seq_lens);
}

}  // namespace kvq
