// read_rows.cu -- cached rows read back as values (fp16, bf16 or fp32): every
// row decoded exactly and rounded once to the output's type.
//
// A cached row's bytes lie in 16- to 64-byte pieces over its unit, next to those
// of the unit's other rows, so the work is done by units: a block looks 64 rows of the
// call up, once, as runs of rows that follow one another in a unit, and its warps take
// (run, kv head, side) in turn.  A warp reads the unit's codes as it does for a
// fragment, 16 bytes a lane, turns them into values of the output's type in a tile
// of its own in shared memory, and writes the run's rows from there, 16 bytes a lane
// and whole rows at a time.  Small calls go row by row instead, a warp for each.
//
// Codes and their sums stay fp16 pairs, which hold them exactly: |c| <= 128, and
// turbo4's transform sums 128 of at most 8, the order of the stages changing nothing.
// The product with the scale has at most 19 bits (turbo4: 21), exact in fp32 and rounded
// once by the conversion, or by an fp16 multiplication.
//
// Bound: the output's bytes.  98304 tokens x 8 heads of q4_0 to fp16 (516 MB): calls in a
// row 97 us, 5.3 TB/s (the kernel by itself behind a flushed cache 99); row by row, four
// values a lane, 426 us.
#include <cuda_runtime.h>

#include <atomic>

#include "kvq_launch.h"
#include "kvq_packed.cuh"
#include "kvq_rope.cuh"
#include "kvq_row_decode.cuh"

namespace kvq {
namespace {

constexpr int kReadWarps = 8;
constexpr int kReadRows = 64;  // of a block
constexpr int kStarts = 256;   // row_start's sequences that are kept in shared memory
constexpr int kPad = 16;       // bytes behind a tile's row: rows on other banks

struct ReadParams {
  const uint8_t *cache[2];
  uint8_t *out[2];
  int64_t row[2], head[2];  // strides in bytes
  int type[2], codec[2];
  PackedRows rows;
  const int32_t *first, *seq_lens, *table;
  int32_t *err;
  int n_kv, capacity, pages_per_seq, n_pages;
  int side0, items;  // the first side that is read; (side, kv head) pairs
  int per_block;     // of which a block takes this many
  int tile_bytes;    // a warp's
  int head_units;    // units from a kv head to the next
};

struct ReadRun {
  int64_t unit;  // of kv head 0
  int64_t row;   // the call's row
  int r, n;      // rows r .. r + n - 1 of the unit
};

// A unit's values as they are decoded, at their places in the tile.
template <int T>
struct Tile {
  uint8_t *at;
  static constexpr int kBytes = T == KVQ_T_F32 ? 4 : 2;
  static constexpr int kPitch = kD * kBytes + kPad;
  // d (a, b) of dims dim, dim + 1; EXACT16: fp16 holds d and its product is to be
  // rounded to fp16 (not turbo4, whose d is divided by 16)
  template <bool EXACT16>
  static __device__ __forceinline__ uint2 scale(uint32_t c, float d) {
    if (T == KVQ_T_F16 && EXACT16) {
      const __half2 x = __hmul2(*reinterpret_cast<__half2 *>(&c), __float2half2_rn(d));
      return make_uint2(*reinterpret_cast<const uint32_t *>(&x), 0u);
    }
    const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&c));
    const float x = f.x * d, y = f.y * d;
    if (T == KVQ_T_F32) return make_uint2(__float_as_uint(x), __float_as_uint(y));
    if (T == KVQ_T_F16) return make_uint2(pack_half2(x, y), 0u);
    const __nv_bfloat162 z = __floats2bfloat162_rn(x, y);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&z), 0u);
  }
  template <bool EXACT16>
  __device__ __forceinline__ void put2(int row, int dim, uint32_t c, float d) const {
    uint8_t *y = at + row * kPitch + dim * kBytes;
    const uint2 x = scale<EXACT16>(c, d);
    if (T == KVQ_T_F32) *reinterpret_cast<uint2 *>(y) = x;
    else *reinterpret_cast<uint32_t *>(y) = x.x;
  }
  template <bool EXACT16>
  __device__ __forceinline__ void put4(int row, int dim, uint32_t c0, uint32_t c1, float d) const {
    uint8_t *y = at + row * kPitch + dim * kBytes;
    const uint2 a = scale<EXACT16>(c0, d), b = scale<EXACT16>(c1, d);
    if (T == KVQ_T_F32) *reinterpret_cast<uint4 *>(y) = make_uint4(a.x, a.y, b.x, b.y);
    else *reinterpret_cast<uint2 *>(y) = make_uint2(a.x, b.x);
  }
  // values that are fp16 already: their own bits to fp16
  __device__ __forceinline__ void keep2(int row, int dim, uint32_t c) const {
    if (T == KVQ_T_F16) *reinterpret_cast<uint32_t *>(at + row * kPitch + dim * kBytes) = c;
    else put2<false>(row, dim, c, 1.0f);
  }
  __device__ __forceinline__ void keep4(int row, int dim, uint32_t c0, uint32_t c1) const {
    if (T == KVQ_T_F16)
      *reinterpret_cast<uint2 *>(at + row * kPitch + dim * kBytes) = make_uint2(c0, c1);
    else put4<false>(row, dim, c0, c1, 1.0f);
  }
};

__device__ __forceinline__ uint32_t fma_bits(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b),
                            *reinterpret_cast<__half2 *>(&c));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// The transform of a row's 128 codes, 16 pairs in each of four lanes (lane bits 0
// and 1): any order of the dims' bits over pair, register and lane will do.
__device__ __forceinline__ void fwht_pairs(uint32_t (&v)[16], int lane) {
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i & h) == 0) {
        const uint32_t a = v[i], b = v[i + h];
        v[i] = fma_bits(a, 0x3c003c00u, b);
        v[i + h] = hsub2_bits(a, b);
      }
  const uint32_t s1 = (lane & 1) ? 0xbc00bc00u : 0x3c003c00u;
  const uint32_t s2 = (lane & 2) ? 0xbc00bc00u : 0x3c003c00u;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = fma_bits(v[i], 0xbc003c00u, __byte_perm(v[i], v[i], 0x1032));  // (a + b, a - b)
    v[i] = fma_bits(v[i], s1, __shfl_xor_sync(0xffffffffu, v[i], 1));
    v[i] = fma_bits(v[i], s2, __shfl_xor_sync(0xffffffffu, v[i], 2));
  }
}
// A turbo4 row: its transform, and the factor that its values still want.  A scale that is
// no number or infinite (values past fp16's) goes into the sums, as it does by definition.
__device__ __forceinline__ float turbo_pairs(uint32_t (&v)[16], float d, int lane) {
  const bool finite = fabsf(d) <= 65504.0f;
  if (!finite) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __half2 x = __hmul2(*reinterpret_cast<__half2 *>(&v[i]), __float2half2_rn(d));
      v[i] = *reinterpret_cast<const uint32_t *>(&x);
    }
  }
  __syncwarp();
  fwht_pairs(v, lane);
  return finite ? d * 0.0625f : 1.0f;
}
// The sign flips of dims dim, dim + 1 (even) of a pair.
__device__ __forceinline__ uint32_t flip_pair(uint32_t signs, int dim, uint32_t v) {
  const uint32_t s = signs >> (dim & 31);
  return v ^ (((s & 1u) << 15) | ((s & 2u) << 30));
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint4 ld128(const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ float half_of(uint32_t w, int hi) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(hi ? w >> 16 : w)));
}

// A unit of K (all 32 lanes): a lane takes the 16-byte pieces (g, w), which belong to
// rows g and g + 8; the order of g over the lanes keeps eight lanes' stores on
// distinct banks.
template <int CODEC, int T>
__device__ __forceinline__ void unit_k(const uint8_t *u, const Tile<T> &tile, int lane) {
  const int q8 = lane >> 2, w = lane & 3, g = ((q8 & 3) << 1) | (q8 >> 2);
  const uint8_t *src = u + (4 * g + w) * 16;
  if (CODEC == KVQ_F16) {
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ld128(src + i * 512);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = g + 8 * (i & 1), dim = 32 * (i >> 1) + 4 * w;
      tile.keep4(row, dim, x[i].x, x[i].y);
      tile.keep4(row, dim + 16, x[i].z, x[i].w);
    }
  } else if (CODEC == KVQ_Q8_0) {
    const uint4 z = ld128(u + 2048 + g * 16);
    const uint32_t d[4] = {z.x, z.y, z.z, z.w};  // (rh, b >> 1)
    uint4 x[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) x[b] = ld128(src + b * 512);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t y[4] = {x[b].x, x[b].y, x[b].z, x[b].w};  // (rh, h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        s8_quad(y[i], lo, hi);
        tile.template put4<true>(g + 8 * (i >> 1), 32 * b + 16 * (i & 1) + 4 * w, lo, hi,
                                 half_of(d[2 * (i >> 1) + (b >> 1)], b & 1));
      }
    }
  } else {
    const uint4 xa = ld128(src), xb = ld128(src + 512);
    const uint32_t y[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};  // (b, rh)
    if (CODEC == KVQ_Q4_0) {
      const uint4 z = ld128(u + 1024 + g * 16);
      const uint32_t d[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int b = i >> 1, rh = i & 1;
        const float s = half_of(d[2 * rh + (b >> 1)], b & 1);
        uint32_t lo, hi;
        u4_quad(y[i] & 0x0f0f0f0fu, lo, hi);
        tile.template put4<true>(g + 8 * rh, 32 * b + 4 * w, lo, hi, s);
        u4_quad((y[i] >> 4) & 0x0f0f0f0fu, lo, hi);
        tile.template put4<true>(g + 8 * rh, 32 * b + 16 + 4 * w, lo, hi, s);
      }
    } else {
      const uint32_t d = *reinterpret_cast<const uint32_t *>(u + 1024 + g * 4);
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) {
        uint32_t v[16];  // (b, h, pair)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          u4_quad(y[2 * b + rh] & 0x0f0f0f0fu, v[4 * b], v[4 * b + 1]);
          u4_quad((y[2 * b + rh] >> 4) & 0x0f0f0f0fu, v[4 * b + 2], v[4 * b + 3]);
        }
        const float s = turbo_pairs(v, half_of(d, rh), lane);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int dim = 32 * (i >> 2) + 16 * ((i >> 1) & 1) + 4 * w;
          const uint32_t signs = turbo_signs(i >> 2);
          tile.template put4<false>(g + 8 * rh, dim, flip_pair(signs, dim, v[i]),
                                    flip_pair(signs, dim + 2, v[i + 1]), s);
        }
      }
    }
  }
}

// A unit of V: a lane takes the pieces (gq, tig), four tokens of some dims.  Nibbles of
// two tokens share a pair, which a transposition of 8 x 8 pairs' halves turns into two
// dims of one token (token lane / 4 of eight, dims 2 (lane % 4) ..).
template <int CODEC, int T>
__device__ __forceinline__ void unit_v(const uint8_t *u, const Tile<T> &tile, int lane) {
  const int gq = lane >> 2, tig = lane & 3;
  const uint8_t *src = u + (4 * gq + tig) * 16;
  if (CODEC == KVQ_F16) {
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ld128(src + i * 512);
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // (rh, s): tokens 2 tig and 2 tig + 1
      const int dim = 16 * i + 2 * gq;
      tile.keep2(2 * tig, dim, __byte_perm(x[i].x, x[i].y, 0x5410));
      tile.keep2(2 * tig + 1, dim, __byte_perm(x[i].x, x[i].y, 0x7632));
      tile.keep2(2 * tig + 8, dim, __byte_perm(x[i].z, x[i].w, 0x5410));
      tile.keep2(2 * tig + 9, dim, __byte_perm(x[i].z, x[i].w, 0x7632));
    }
  } else if (CODEC == KVQ_Q8_0) {
    const uint4 za = ld128(u + 2048 + tig * 32), zb = ld128(u + 2048 + tig * 32 + 16);
    const uint32_t d[8] = {za.x, za.y, za.z, za.w, zb.x, zb.y, zb.z, zb.w};  // (b, rh)
    uint4 x[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) x[b] = ld128(src + b * 512);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t y[4] = {x[b].x, x[b].y, x[b].z, x[b].w};  // (mt & 1, rh)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rh = i & 1, dim = 32 * b + 16 * (i >> 1) + 2 * gq;
        uint32_t lo, hi;  // of token 2 tig, of the next
        s8_quad(y[i], lo, hi);
        tile.template put2<true>(2 * tig + 8 * rh, dim, lo, half_of(d[2 * b + rh], 0));
        tile.template put2<true>(2 * tig + 8 * rh + 1, dim, hi, half_of(d[2 * b + rh], 1));
      }
    }
  } else {
    const uint4 xa = ld128(src), xb = ld128(src + 512);
    const uint32_t y[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};  // mt; bytes (par, rh)
    const int token = lane >> 2, par = token & 1, dim0 = 2 * (lane & 3);
    uint32_t d[8];  // (b, rh): of token pairs
    if (CODEC == KVQ_Q4_0) {
      const uint8_t *sc = u + 1024 + (token >> 1) * 32;
      const uint4 za = ld128(sc), zb = ld128(sc + 16);
      d[0] = za.x; d[1] = za.y; d[2] = za.z; d[3] = za.w;
      d[4] = zb.x; d[5] = zb.y; d[6] = zb.z; d[7] = zb.w;
    } else {
      const uint2 z = *reinterpret_cast<const uint2 *>(u + 1024 + (token >> 1) * 8);
      d[0] = z.x; d[1] = z.y;
    }
#pragma unroll
    for (int rh = 0; rh < 2; ++rh) {
      uint32_t v[16];  // (mt, nibble)
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        const uint32_t z = rh ? y[mt] >> 8 : y[mt];
        v[2 * mt] = transposed8x8(u4_pair_minus8(z));
        v[2 * mt + 1] = transposed8x8(u4_pair_minus8_hi(z));
      }
      float s = 0.0f;
      if (CODEC == KVQ_TURBO4) s = turbo_pairs(v, half_of(d[rh], par), lane);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int b = i >> 2, dim = 32 * b + 8 * ((i >> 1) & 1) + 16 * (i & 1) + dim0;
        if (CODEC == KVQ_TURBO4)
          tile.template put2<false>(token + 8 * rh, dim, flip_pair(turbo_signs(b), dim, v[i]), s);
        else
          tile.template put2<true>(token + 8 * rh, dim, v[i], half_of(d[2 * b + rh], par));
      }
    }
  }
}

// The unit of row i of sequence s, of kv head 0, and the row's place in it; -1 (and the
// error word) where the row is no token's or its page is none.
__device__ __forceinline__ int64_t unit_of_row(const ReadParams &p, int s, int64_t i, int &place) {
  const int64_t t = (p.first ? p.first[s] : 0) + i, j = t / kUnitTokens;
  place = static_cast<int>(t % kUnitTokens);
  if (t < 0 || t >= p.seq_lens[s] || t >= p.capacity) {
    set_err(p.err, KVQ_DEVERR_SEQLEN);
    return -1;
  }
  if (!p.table) return static_cast<int64_t>(s) * p.n_kv * p.head_units + j;
  const int pg = page_of(p.table, p.pages_per_seq, p.n_pages, s, j / kPageUnits);
  if (pg < 0) {
    set_err(p.err, KVQ_DEVERR_PAGE);
    return -1;
  }
  return static_cast<int64_t>(pg) * p.n_kv * kPageUnits + j % kPageUnits;
}

// One run of one kv head and side: through the warp's tile to the output.
template <int T>
__device__ __forceinline__ void read_run(const ReadParams &p, const ReadRun &run, int h, int side,
                                         uint8_t *buf, int lane) {
  const int codec = p.codec[side];
  const uint8_t *u = p.cache[side] + (run.unit + h * p.head_units) * unit_bytes(codec);
  const Tile<T> tile{buf};
  if (side == 0) {
    if (codec == KVQ_F16) unit_k<KVQ_F16, T>(u, tile, lane);
    else if (codec == KVQ_Q8_0) unit_k<KVQ_Q8_0, T>(u, tile, lane);
    else if (codec == KVQ_Q4_0) unit_k<KVQ_Q4_0, T>(u, tile, lane);
    else unit_k<KVQ_TURBO4, T>(u, tile, lane);
  } else {
    if (codec == KVQ_F16) unit_v<KVQ_F16, T>(u, tile, lane);
    else if (codec == KVQ_Q8_0) unit_v<KVQ_Q8_0, T>(u, tile, lane);
    else if (codec == KVQ_Q4_0) unit_v<KVQ_Q4_0, T>(u, tile, lane);
    else unit_v<KVQ_TURBO4, T>(u, tile, lane);
  }
  __syncwarp();
  constexpr int kLanes = kD * Tile<T>::kBytes / 16;  // of a row
  uint8_t *y = p.out[side] + run.row * p.row[side] + h * p.head[side] + (lane % kLanes) * 16;
  const uint8_t *x = buf + (lane % kLanes) * 16;
#pragma unroll
  for (int i = 0; i < kUnitTokens; i += 32 / kLanes) {
    const int r = i + lane / kLanes;
    if (r >= run.r && r < run.r + run.n)
      *reinterpret_cast<uint4 *>(y + (r - run.r) * p.row[side]) = ld128(x + r * Tile<T>::kPitch);
  }
  __syncwarp();
}

// Row by row: a warp per (row, kv head, side).
__global__ void __launch_bounds__(kReadWarps * 32)
    read_each_kernel(const __grid_constant__ ReadParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0) packed_check(p.rows, p.err);
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5);
  const int64_t row = i / p.items;
  const int item = static_cast<int>(i - row * p.items);
  const int side = p.side0 + (item >= p.n_kv ? 1 : 0), h = item >= p.n_kv ? item - p.n_kv : item;
  if (row >= p.rows.n_rows) return;
  int r, s;
  int64_t at;
  if (!packed_find(p.rows, row, s, at)) return;
  const int64_t unit = unit_of_row(p, s, at, r);
  if (unit < 0) return;
  const int codec = p.codec[side];
  const uint8_t *u = p.cache[side] + (unit + h * p.head_units) * unit_bytes(codec);
  float x[4];
  if (side == 0) decode_row_lane<0>(codec, u, r, lane, x);
  else decode_row_lane<1>(codec, u, r, lane, x);
  uint8_t *y = p.out[side] + row * p.row[side] + h * p.head[side];
  if (p.type[side] == KVQ_T_F32) store4<KVQ_T_F32>(y + 16 * lane, x);
  else if (p.type[side] == KVQ_T_BF16) store4<KVQ_T_BF16>(y + 8 * lane, x);
  else store4<KVQ_T_F16>(y + 8 * lane, x);
}

__global__ void __launch_bounds__(kReadWarps * 32, 3)
    read_rows_kernel(const __grid_constant__ ReadParams p) {
  extern __shared__ __align__(16) uint8_t tiles[];
  __shared__ int32_t starts[kStarts + 1];
  __shared__ ReadRun runs[kReadRows];
  __shared__ int64_t unit_of[kReadRows];  // of kv head 0; -1: none
  __shared__ int place_of[kReadRows], n_runs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0) packed_check(p.rows, p.err);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kReadRows;
  if (tid == 0) n_runs = 0;
  PackedRows rows = p.rows;
  if (rows.row_start && rows.n_seqs <= kStarts) {  // searched in shared memory
    for (int i = tid; i <= rows.n_seqs; i += kReadWarps * 32) starts[i] = rows.row_start[i];
    __syncthreads();
    rows.row_start = starts;
  }
  if (tid < kReadRows) {
    int64_t unit = -1, i;
    int place = 0, s;
    if (row0 + tid < rows.n_rows && packed_find(rows, row0 + tid, s, i))
      unit = unit_of_row(p, s, i, place);
    unit_of[tid] = unit;
    place_of[tid] = place;
  }
  __syncthreads();
  // A run: rows at places that follow one another in a unit (in pages, two sequences'
  // rows may lie in one).
  auto follows = [&](int i) {
    return unit_of[i] == unit_of[i - 1] && place_of[i] == place_of[i - 1] + 1;
  };
  if (tid < kReadRows && unit_of[tid] >= 0 && (tid == 0 || !follows(tid))) {
    int n = 1;
    while (tid + n < kReadRows && follows(tid + n)) ++n;
    runs[atomicAdd(&n_runs, 1)] = {unit_of[tid], row0 + tid, place_of[tid], n};
  }
  __syncthreads();
  const int from = blockIdx.y * p.per_block, items = min(p.per_block, p.items - from);
  for (int i = warp; i < n_runs * items; i += kReadWarps) {
    const int item = from + i % items;
    const int side = p.side0 + (item >= p.n_kv ? 1 : 0), h = item >= p.n_kv ? item - p.n_kv : item;
    const ReadRun run = runs[i / items];
    uint8_t *buf = tiles + warp * p.tile_bytes;
    if (p.type[side] == KVQ_T_F32) read_run<KVQ_T_F32>(p, run, h, side, buf, lane);
    else if (p.type[side] == KVQ_T_BF16) read_run<KVQ_T_BF16>(p, run, h, side, buf, lane);
    else read_run<KVQ_T_F16>(p, run, h, side, buf, lane);
  }
}

}  // namespace

cudaError_t launch_read_rows(const kvq_layer &L, const kvq_rows *k, const kvq_rows *v,
                             int64_t n_rows, const int32_t *n_read, const int32_t *row_start,
                             const int32_t *first, int sms, cudaStream_t stream) {
  ReadParams p;
  p.cache[0] = static_cast<const uint8_t *>(L.k_cache);
  p.cache[1] = static_cast<const uint8_t *>(L.v_cache);
  p.codec[0] = L.codec_k;
  p.codec[1] = L.codec_v;
  const kvq_rows *rows[2] = {k, v};
  int wide = 0;
  for (int i = 0; i < 2; ++i) {
    p.out[i] = rows[i] ? static_cast<uint8_t *>(rows[i]->data) : nullptr;
    p.type[i] = rows[i] ? rows[i]->type : KVQ_T_F16;
    p.row[i] = rows[i] ? rows[i]->row_stride * type_bytes(p.type[i]) : 0;
    p.head[i] = rows[i] ? rows[i]->head_stride * type_bytes(p.type[i]) : 0;
    wide = wide || p.type[i] == KVQ_T_F32;
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
  p.side0 = k ? 0 : 1;
  p.items = (k && v ? 2 : 1) * L.n_kv_heads;
  p.tile_bytes = kUnitTokens * (wide ? Tile<KVQ_T_F32>::kPitch : Tile<KVQ_T_F16>::kPitch);
  p.head_units = p.table ? kPageUnits : L.capacity / kUnitTokens;
  // Row by row while a call is small, where finding the rows and fetching the units'
  // longer code is what counts, or has few rows of each sequence, for which whole units are
  // decoded.  Measured, K q8_0 and V turbo4 to fp32 over 8 heads, by rows and by units: one
  // row of 16 sequences 2.9 and 7.0 us, 64 of 4 3.4 and 5.9, 64 of 16 (16384 items) 7.3
  // and 7.4, 313 of 16 28 and 16, 49152 of 2 437 and 191; 2 rows of 1024 16 and 32, 16 of 512
  // (2 heads) 15 and 13.
  constexpr int64_t kFewItems = 16384;
  if (n_rows * p.items < kFewItems || n_rows < 8 * static_cast<int64_t>(L.n_seqs)) {
    const int64_t blocks = (n_rows * p.items + kReadWarps - 1) / kReadWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(read_each_kernel, dim3(static_cast<unsigned>(blocks)),
                      dim3(kReadWarps * 32), 0, stream, p);
  }
  const int64_t blocks = (n_rows + kReadRows - 1) / kReadRows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  // Fewer rows: their heads and sides over more blocks, until every SM has as many as
  // fit it (313 rows of 16 sequences: 16 us; with twice the blocks 19).
  constexpr int kSmBlocks = 3;
  const int64_t parts = (static_cast<int64_t>(sms) * kSmBlocks + blocks - 1) / blocks;
  const int n_parts = static_cast<int>(parts < p.items ? parts : p.items);
  p.per_block = (p.items + n_parts - 1) / n_parts;
  const dim3 grid(static_cast<unsigned>(blocks),
                  static_cast<unsigned>((p.items + p.per_block - 1) / p.per_block));
  const int smem = kReadWarps * p.tile_bytes;
  constexpr int kMost = kReadWarps * kUnitTokens * Tile<KVQ_T_F32>::kPitch;
  static std::atomic<uint64_t> optin{0};
  const cudaError_t e = smem_optin(read_rows_kernel, kMost, optin);
  if (e != cudaSuccess) return e;
  return launch_pdl(read_rows_kernel, grid, dim3(kReadWarps * 32), smem, stream, p);
}

}  // namespace kvq
