// rope.cu -- rotary positions: the angle table, the rotation of rows, and the
// re-rotation of cached keys after an eviction moved them.
//
// All three move bytes: what they cannot do without, at the measured copy rate
// of 6.78 TB/s, is the floor of the figures below (device times on one GB300).
#include <cuda_runtime.h>

#include <math.h>

#include "kvq_launch.h"
#include "kvq_quad.cuh"

namespace kvq {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = kRopeWarps * 32;
constexpr int kTableBlocks = 8;  // of the table kernel's grid per SM, of which six are resident
constexpr int kSmallGrid = 8;    // warps per SM below which a row's heads are spread

// ------------------------------------------------------------------ table

struct TableParams {
  float *table;
  int64_t n_pos;
  int pairs, cols;         // planes; columns of one thread's planes
  uint64_t turns[kD / 2];  // frequency in units of 2^-64 turns per position
};

// Terms of the Taylor series of sin and cos in turns: (2 pi)^n / n!.
constexpr double kTurn = 6.283185307179586477;  // 2 pi
__host__ __device__ constexpr double turn_term(int n) {
  return n == 0 ? 1.0 : turn_term(n - 1) * kTurn / n;
}

// (cos, sin) of u * 2^-64 turns for two angles at once (one polynomial
// instruction serves both).  The nearest quarter turn is taken off as an
// integer, so the remainder t in [-1/8, 1/8] turns is exact (its 56 upper
// bits are used) and rounds once to fp32 whatever the position (2^-24 of at
// most pi / 4 rad).  The Taylor series end at t^9 and t^10, what is left out
// being below 2e-9; 2 pi t is taken with 2 pi as the sum of two floats, so that
// the last addition's rounding is the only other one of its size.  In all
// within 1.3 * 2^-24 (measured on the host over 4M values), inside the
// documented 2^-23.
__device__ __forceinline__ float2 both(float k) { return make_float2(k, k); }
__device__ __forceinline__ void cos_sin_turns(uint64_t u0, uint64_t u1, float2 &first,
                                              float2 &second) {
  constexpr float k1 = static_cast<float>(kTurn), k1lo = static_cast<float>(kTurn - k1);
  constexpr float k2 = turn_term(2), k3 = turn_term(3), k4 = turn_term(4), k5 = turn_term(5),
                  k6 = turn_term(6), k7 = turn_term(7), k8 = turn_term(8), k9 = turn_term(9),
                  k10 = turn_term(10);
  // the quarter and the remainder's upper word: the lower word stays
  const uint32_t h0 = static_cast<uint32_t>(u0 >> 32), h1 = static_cast<uint32_t>(u1 >> 32);
  const uint32_t q0 = (h0 + (1u << 29)) >> 30, q1 = (h1 + (1u << 29)) >> 30;
  // turns of a remainder: its top 24 bits exactly, the 32 below them added
  // with one rounding
  auto turns = [](uint32_t h, uint32_t lo) {
    const float top = static_cast<float>(static_cast<int32_t>(h & ~0xffu));
    const float rest = static_cast<float>(__funnelshift_l(lo, h, 24));
    return fmaf(rest, 0x1p-56f, top * 0x1p-32f);
  };
  const float2 t = make_float2(turns(h0 - (q0 << 30), static_cast<uint32_t>(u0)),
                               turns(h1 - (q1 << 30), static_cast<uint32_t>(u1)));
  const float2 t2 = __fmul2_rn(t, t);
  float2 s = __ffma2_rn(t2, __ffma2_rn(t2, __ffma2_rn(t2, both(k9), both(-k7)), both(k5)), both(-k3));
  s = __ffma2_rn(t, both(k1), __ffma2_rn(__fmul2_rn(t, t2), s, __fmul2_rn(t, both(k1lo))));
  float2 c = __ffma2_rn(t2, __ffma2_rn(t2, __ffma2_rn(t2, __ffma2_rn(t2, both(-k10), both(k8)),
                                                      both(-k6)), both(k4)), both(-k2));
  c = __ffma2_rn(t2, c, both(1.0f));
  auto place = [](uint32_t q, float co, float si) {  // a quarter turn swaps them, a half negates
    const float a = (q & 1) ? si : co, b = (q & 1) ? co : si;
    return make_float2(__uint_as_float(__float_as_uint(a) ^ (((q + 1) & 2) << 30)),
                       __uint_as_float(__float_as_uint(b) ^ ((q & 2) << 30)));
  };
  first = place(q0, c.x, s.x);
  second = place(q1, c.y, s.y);
}

// Writes 4 rot_dim bytes per position and reads nothing: 200704 positions x 64
// planes 15.9 us, 0.95 of the floor (a thread per plane with 64-bit division
// and conversion 92 us, with running sums 24 us); 32768 positions 4.3 us, of
// which the launch is half.
//
// Thread (column, row lane): two planes of every (rows-per-pass)-th position
// (P = 1, an odd number of planes: one plane of two such positions).  The
// angle's fraction of a turn advances by a whole number of 2^-64 turns per
// step, modulo 2^64, so the running sum is exact.
template <int P>
__global__ void __launch_bounds__(kRopeThreads) table_kernel(const __grid_constant__ TableParams p) {
  // (from shared memory: parameters indexed by lane are read one at a time)
  __shared__ uint64_t turns[kD / 2];
  if (threadIdx.x < p.pairs) turns[threadIdx.x] = p.turns[threadIdx.x];
  __syncthreads();
  const int rows = kRopeThreads / p.cols;  // positions per block and pass
  const int col = threadIdx.x % p.cols, row = threadIdx.x / p.cols;
  grid_dependency_wait();
  grid_launch_dependents();
  if (row >= rows) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  int64_t pos = static_cast<int64_t>(blockIdx.x) * rows + row;
  const uint64_t t0 = turns[col * P], t1 = turns[col * P + P - 1];
  const uint64_t d0 = t0 * static_cast<uint64_t>(step), d1 = t1 * static_cast<uint64_t>(step);
  uint64_t u0 = t0 * static_cast<uint64_t>(pos), u1 = t1 * static_cast<uint64_t>(pos);
  float *out = p.table + (pos * p.pairs + col * P) * 2;
  const int64_t stride = step * p.pairs * 2;
  float2 a, b;
  if (P == 2) {
    for (; pos < p.n_pos; pos += step, out += stride, u0 += d0, u1 += d1) {
      cos_sin_turns(u0, u1, a, b);
      *reinterpret_cast<float4 *>(out) = make_float4(a.x, a.y, b.x, b.y);
    }
  } else {
    for (; pos < p.n_pos; pos += 2 * step, out += 2 * stride, u0 += 2 * d0) {
      cos_sin_turns(u0, u0 + d0, a, b);
      *reinterpret_cast<float2 *>(out) = a;
      if (pos + step < p.n_pos) *reinterpret_cast<float2 *>(out + stride) = b;
    }
  }
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
  int n_heads, pos0, hpw, chunks;  // heads per warp, and such groups in a row
  float sign;
};

constexpr int kAnyHeads = 8;  // heads per warp of the general kernel

// One warp per (row, up to sixteen heads): the angles are read once, and all
// the heads' values are requested before the first is used (up to 4 KB per
// warp in flight).  Bound by HBM: 8191 rows x 40 bf16 heads, 64 interleaved
// dims, 27.6 us, 0.91 of the floor; by lanes of four values 31 us, with one
// head at a time 51 us.  16 rows x 40 heads take 2.0 us, a launch's length.
template <int TI, int TO>
__global__ void __launch_bounds__(kRopeThreads) apply_kernel(const __grid_constant__ ApplyParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int64_t row = item / p.chunks;
  if (row >= p.n_rows) return;
  const int h0 = static_cast<int>(item % p.chunks) * p.hpw;
  const uint8_t *x = p.x + row * p.x_row + h0 * p.x_head;
  uint8_t *y = p.y + row * p.y_row + h0 * p.y_head;
  rotate_heads_eight<TI, TO, 4 / (TI == KVQ_T_F32 ? 2 : 1)>(
      p.rope, x, p.x_head, y, p.y_head, min(p.hpw, p.n_heads - h0), p.sign, lane, [&] {
        return rope_row(p.rope, p.positions ? p.positions[row] : p.pos0 + row, p.err);
      });
}

// Planes that eight lanes cannot hold: one head at a time, 4 values per lane,
// eight heads requested at once.  8191 rows x 40 bf16 heads: interleaved, 6 dims
// 31 us (0.80 of the floor), halves with 40 dims 33 us (0.75); with 20 and 126
// dims (Lanes::kAny) 48 and 49 us (0.52), bound by instruction issue (0.77 per
// scheduler and cycle).
template <int TI, int TO>
__global__ void __launch_bounds__(kRopeThreads)
    apply_any_kernel(const __grid_constant__ ApplyParams p) {
  using Raw = typename RowType<TI>::raw4;
  constexpr int SI = sizeof(typename RowType<TI>::type), SO = sizeof(typename RowType<TO>::type);
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int64_t row = item / p.chunks;
  if (row >= p.n_rows) return;
  const int h0 = static_cast<int>(item % p.chunks) * p.hpw, nh = min(p.hpw, p.n_heads - h0);
  const uint8_t *x = p.x + row * p.x_row + h0 * p.x_head + 4 * lane * SI;
  uint8_t *y = p.y + row * p.y_row + h0 * p.y_head + 4 * lane * SO;
  Raw raw[kAnyHeads];
#pragma unroll
  for (int h = 0; h < kAnyHeads; ++h)
    if (h < nh) raw[h] = *reinterpret_cast<const Raw *>(x + h * p.x_head);
  const int64_t pos = p.positions ? p.positions[row] : p.pos0 + row;
  const LaneAngles a = lane_angles(p.rope, rope_row(p.rope, pos, p.err), lane, p.sign);
  with_lanes(p.rope, [&](auto lanes) {
#pragma unroll
    for (int h = 0; h < kAnyHeads; ++h)
      if (h < nh) {
        float v[4];
        load4<TI>(&raw[h], v);
        rotate_lane<decltype(lanes)::value>(p.rope, a, lane, v);
        store4<TO>(y + h * p.y_head, v);
      }
  });
}

// ------------------------------------------------------------------ shift

struct DeltaParams {
  const int32_t *seq_lens, *evict, *n_evicted;
  int32_t *delta;
  int capacity, max_evict;
};

// Of the block's n items, how many does the predicate hold for (it holds for a
// first part of them), by probing them 256 at a time: one dependent load per
// round, two rounds up to 65536 items.
template <typename Pred>
__device__ __forceinline__ int block_partition(int n, Pred pred) {
  int lo = 0;
  while (n > 0) {
    const int step = (n + kRopeThreads - 1) / kRopeThreads, at = threadIdx.x * step;
    const int k = __syncthreads_count(at < n && pred(lo + at));
    if (k == 0) break;
    if (step == 1) return lo + k;
    lo += (k - 1) * step + 1;  // probe k - 1 holds; the answer lies before probe k
    n = min(step - 1, n - (k - 1) * step - 1);
  }
  return lo;
}

// delta[s][w] = -(evicted tokens before the one that moves to w).  evict[j] - j
// kept tokens lie before evicted token j, a non-decreasing count, so that
// number is the count of j with evict[j] - j <= w.  A block takes 256
// consecutive w: it finds the first of them together, keeps the next 256
// counts in shared memory, and each thread searches those.  (A binary search
// by each thread over 2048 evicted tokens is eleven dependent loads, 6 us.)
__global__ void __launch_bounds__(kRopeThreads) delta_kernel(DeltaParams p) {
  __shared__ int key[kRopeThreads];
  grid_dependency_wait();
  grid_launch_dependents();
  const int s = blockIdx.y;
  const int w0 = blockIdx.x * kRopeThreads, w = w0 + threadIdx.x;
  const int len = min(p.seq_lens[s], p.capacity);
  const int n = max(0, min(p.n_evicted[s], p.max_evict));
  if (w0 >= len - n) return;  // (the whole block)
  const int32_t *e = p.evict + static_cast<int64_t>(s) * p.max_evict;
  const int first = block_partition(n, [&](int j) { return e[j] - j < w0; });
  const int m = min(kRopeThreads, n - first);
  if (threadIdx.x < m) key[threadIdx.x] = e[first + threadIdx.x] - (first + threadIdx.x);
  __syncthreads();
  if (w >= len - n) return;
  int lo = 0, hi = m;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (key[mid] <= w) lo = mid + 1;
    else hi = mid;
  }
  lo += first;
  if (lo == first + kRopeThreads) {  // many evicted tokens in a row: search the rest
    hi = n;
    while (lo < hi) {
      const int mid = lo + ((hi - lo) >> 1);
      if (e[mid] - mid <= w) lo = mid + 1;
      else hi = mid;
    }
  }
  p.delta[static_cast<int64_t>(s) * p.capacity + w] = -lo;
}

struct ShiftParams {
  RopeArgs rope;
  uint8_t *k;
  const int32_t *seq_lens, *delta, *table;
  int32_t *err;
  int n_kv, capacity, pages_per_seq, n_pages;
  int kind;  // quad_kind
};

// One warp per (sequence, 16-token unit, up to kShiftHeads kv heads).  A head's
// unit is copied to shared memory while the one before it is worked on, the
// first ones beside the shifts, which in an eviction's wake are seldom all
// zero; every quad turns and encodes its two rows from there and stores the ones
// that move straight to the unit.
//
// 74k tokens x 8 heads in four sequences, the deltas (2.5 us) included: f16 51
// us, 0.88 of the floor (the next unit in registers 57 us, no look-ahead 74 us),
// bound by HBM; q8_0 58 us and q4_0 67 us, bound by the latency of dependent
// instructions (0.64 issued per scheduler and cycle by its 3.7 warps; 31 and 37
// us at full issue); turbo4 123 us, bound by instruction issue (0.83), most of
// it the encoder's.  Tried for f16, q8_0 and q4_0: both rows encoded before
// either is stored 52, 60, 70 us; rows encoded in the shared copy and the whole
// unit stored 52, 62, 73 us; a third unit in the ring 51, 59, 68 us; a third
// block per SM (80 registers) 56, 63, 72 us; eight heads per warp 52, 55, 66 us,
// but 29 instead of 17 us for 16k tokens in eight sequences (q8_0).  The code of
// a lane's two rows is interleaved but for turbo4 (124 instead of 133 us; q8_0
// 60 instead of 58 us).
constexpr int kShiftHeads = 4;
constexpr int kShiftSlots = 2;  // units in a warp's ring

// ANY: planes that cross lanes (a kernel of its own, so that its registers are
// not the others'): with 40 dims in halves f16 62 us, q8_0 76 us, turbo4 145 us
// (by whole rows, a warp each, f16 166 us).
template <int CODEC, bool ANY>
__global__ void __launch_bounds__(kRopeThreads, 2)
    shift_units_kernel(const __grid_constant__ ShiftParams p) {
  extern __shared__ __align__(16) uint8_t units[];
  grid_dependency_wait();
  __shared__ __align__(16) float copies[ANY ? kRopeWarps : 1][ANY ? kQuadBytes / 4 : 4];
  const int lane = threadIdx.x & 31, g = lane >> 2, w = lane & 3, s = blockIdx.y;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int groups = (p.n_kv + kShiftHeads - 1) / kShiftHeads;
  const int j = static_cast<int>(item / groups);  // unit
  const int h0 = static_cast<int>(item % groups) * kShiftHeads;  // first kv head
  const int len = min(p.seq_lens[s], p.capacity);
  if (j * kUnitTokens >= len) return;
  int64_t unit = (static_cast<int64_t>(s) * p.n_kv + h0) * (p.capacity / kUnitTokens) + j;
  int64_t step = p.capacity / kUnitTokens;
  if (p.table) {
    const int pg = page_of(p.table, p.pages_per_seq, p.n_pages, s, j / kPageUnits);
    if (pg < 0) {
      if (lane == 0) set_err(p.err, KVQ_DEVERR_PAGE);
      return;
    }
    unit = (static_cast<int64_t>(pg) * p.n_kv + h0) * kPageUnits + j % kPageUnits;
    step = kPageUnits;
  }
  constexpr int kBytes = unit_bytes(CODEC);
  uint8_t *u = p.k + unit * kBytes;
  step *= kBytes;
  const int heads = min(kShiftHeads, p.n_kv - h0);
  uint8_t *const ring = units + (threadIdx.x >> 5) * kShiftSlots * kBytes;
  auto fetch = [&](int h) {  // head h's unit (none behind the last: an empty group)
    if (h < heads)
      for (int c = 16 * lane; c < kBytes; c += 512)
        copy_async16(ring + h % kShiftSlots * kBytes + c, u + h * step + c);
    copy_async_commit();
  };
#pragma unroll
  for (int h = 0; h < kShiftSlots - 1; ++h) fetch(h);
  int d[2];
#pragma unroll
  for (int rh = 0; rh < 2; ++rh) {
    const int t = j * kUnitTokens + g + 8 * rh;
    d[rh] = t < len ? p.delta[static_cast<int64_t>(s) * p.capacity + t] : 0;
  }
  if (!__any_sync(0xffffffffu, d[0] != 0 || d[1] != 0)) {
    copy_async_wait<0>();
    return;
  }
  const float *row[2];
#pragma unroll
  for (int rh = 0; rh < 2; ++rh) {
    const int64_t by = d[rh];
    row[rh] = rope_row(p.rope, by < 0 ? -by : by, p.err);
  }
#pragma unroll 1
  for (int h = 0; h < heads; ++h) {
    copy_async_wait<kShiftSlots - 2>();
    __syncwarp();  // every lane's copies of head h have landed, and head h - 1 has left
    fetch(h + kShiftSlots - 1);
    uint8_t *slot = ring + h % kShiftSlots * kBytes;
#pragma unroll (ANY || CODEC == KVQ_TURBO4 ? 1 : 2)
    for (int rh = 0; rh < 2; ++rh) {
      const int by = rh ? d[1] : d[0];
      const float *angles = rh ? row[1] : row[0], sign = by < 0 ? -1.0f : 1.0f;
      float v[8][4];
      QuadCodes<CODEC> q;
      quad_load_row<CODEC>(slot, g + 8 * rh, w, q);
      quad_decode<CODEC>(q, w, v);
      if (ANY)
        quad_rotate_copied<true>(p.rope, angles, lane, sign, copies[ANY ? threadIdx.x >> 5 : 0], v);
      else
        quad_rotate<true>(p.rope, p.kind, angles, w, sign, v);
      quad_encode<CODEC>(v, w, by != 0, q);
      if (by != 0) quad_store_row<CODEC>(u + h * step, g + 8 * rh, w, q);
    }
  }
}

template <int CODEC>
cudaError_t launch_shift(const ShiftParams &p, dim3 grid, cudaStream_t stream) {
  static std::atomic<uint64_t> optin[2]{};
  const bool any = p.kind == kQuadAny;
  const auto kernel = any ? shift_units_kernel<CODEC, true> : shift_units_kernel<CODEC, false>;
  const int bytes = kRopeWarps * kShiftSlots * unit_bytes(CODEC);
  const cudaError_t e = smem_optin(kernel, bytes, optin[any]);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, grid, dim3(kRopeThreads), bytes, stream, p);
}

template <int TI, int TO>
cudaError_t launch_apply_t(ApplyParams &p, cudaStream_t stream) {
  const bool eight = eight_lanes(p.rope);
  p.hpw = eight ? (TI == KVQ_T_F32 ? 8 : 16) : kAnyHeads;
  // few rows: spread the heads over more warps (four are one step of eight lanes)
  const int64_t few = static_cast<int64_t>(device_sms()) * kSmallGrid;
  while (p.hpw > 4 && p.n_rows * ((p.n_heads + p.hpw - 1) / p.hpw) < few) p.hpw /= 2;
  p.chunks = (p.n_heads + p.hpw - 1) / p.hpw;
  const int64_t blocks = (p.n_rows * p.chunks + kRopeWarps - 1) / kRopeWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(eight ? apply_kernel<TI, TO> : apply_any_kernel<TI, TO>,
                    dim3(static_cast<unsigned>(blocks)), dim3(kRopeThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_rope_table(const double *freqs, int rot_dim, int n_pos, float *table,
                              cudaStream_t stream) {
  TableParams p;
  p.table = table;
  p.n_pos = n_pos;
  p.pairs = rot_dim / 2;
  for (int i = 0; i < p.pairs; ++i) p.turns[i] = turns_of(freqs[i]);
  const int planes = p.pairs % 2 == 0 ? 2 : 1;
  p.cols = p.pairs / planes;
  const int rows = kRopeThreads / p.cols;
  const int64_t passes = (p.n_pos + rows - 1) / rows;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int64_t most = static_cast<int64_t>(sms) * kTableBlocks;
  const unsigned grid = static_cast<unsigned>(passes < most ? passes : most);
  return launch_pdl(planes == 2 ? table_kernel<2> : table_kernel<1>, dim3(grid),
                    dim3(kRopeThreads), 0, stream, p);
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
  p.n_kv = L.n_kv_heads;
  p.capacity = L.capacity;
  p.pages_per_seq = L.pages_per_seq;
  p.n_pages = L.n_pages;
  p.kind = quad_kind(p.rope);
  const int64_t items = static_cast<int64_t>(L.capacity / kUnitTokens) *
                        ((L.n_kv_heads + kShiftHeads - 1) / kShiftHeads);
  const int64_t blocks = (items + kRopeWarps - 1) / kRopeWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks), L.n_seqs);
  return L.codec_k == KVQ_F16    ? launch_shift<KVQ_F16>(p, grid, stream)
         : L.codec_k == KVQ_Q8_0 ? launch_shift<KVQ_Q8_0>(p, grid, stream)
         : L.codec_k == KVQ_Q4_0 ? launch_shift<KVQ_Q4_0>(p, grid, stream)
                                 : launch_shift<KVQ_TURBO4>(p, grid, stream);
}

}  // namespace kvq
