// cross.cu -- attention of packed query rows to every cached key of their
// sequence, without a causal mask: cross attention to an encoder's states, and
// the shared part of a decode step behind a common prefix.
//
// o = softmax(scale q K^T) V over the keys below the sequence's length, query
// head h reading kv head h / G, G = n_q / n_kv.  The G heads of a kv head read the
// same keys, so a sequence's rows are taken as n * G rows per kv head (row R:
// token R / G, head R % G) in tiles of 128, and two tiles (a pair) share every
// key tile that is read; a last odd tile stands alone.
//
// Work.  An item is (sequence, kv head, pair or single tile): a run of steps, one
// per 64 keys.  All items' steps are laid end to end by what they cost, every item's
// start with a cost of its own, and the CTAs (one per SM) take equal contiguous slices:
// whole items, and pieces of at most two more.  The rows of a piece go to a partial slot
// (unnormalised O, max, sum), and a second kernel joins an item's pieces by log-sum-exp
// in a fixed order.  Lengths and row counts are read on the device.
//
// Inside a CTA (20 warps) nothing is written to HBM but the results: codes are
// copied in as they lie in the cache, turned into tensor-core operand tiles in
// shared memory and used there.
//  * Warps 16 (K) and 19 (V) copy the codes of 64 keys at a time into their side's ring
//    (1-D bulk copies).
//  * Warps 8-11 (K) and 12-15 (V) turn them into fp16 operand tiles (two 32 KB
//    buffers a side), a 16-token unit each.  The cache's order is kept where the
//    operands leave the choice, so that 16 bytes of codes become whole 8- or 16-byte
//    pieces of a tile without an exchange between lanes: a key's place in its tile is
//    4 tig + 2 rh + par (include/kvq.h), the same for K's rows and V's columns, and
//    K's dims stand in the order 32 b + 8 w + 4 h + i, as Q's do.  turbo4 stays in its
//    rotated space: Q is rotated, O rotated back.
//  * Warps 17 and 18 issue tcgen05.mma for a pipe each: S = Q K^T into TMEM, O += P V
//    with P read from TMEM.
//  * Warps 0-3 and 4-7 are two softmax pipes, one query row per thread, 32 keys at a
//    time in two score buffers.  In a pair they hold the two tiles; with a single tile
//    they take the first and second half of its every key tile, and each joins and writes
//    half of the dims at the end.
//
// fp16 operands do not hold everything that a cache and fp32 do: a cached value past 65504
// (codes and scales go to 8 * 10^6; fp16 rows reach 65532), a bf16 query or a rotated one
// past it, scores so large (2^22 of an exponent) that a step of fp32 between them is no
// longer small against a weight's range.  The first three give NaN (as two parts: an
// infinity and its opposite), the last is seen in the maximum.  Where a CTA meets a row that
// is NaN it computes that piece of it anew at its end, in fp32, a warp a row, key by key:
// right and slow (2048 rows x 32 heads over 32768 states, one value past 65504 in a head:
// 1.1 -> 570 ms; one such query: 19 ms; a NaN in a query ends it at the first key).
//
// Bound: the tensor cores, where a pair's rows fill its tiles: its 64 keys cost 2050
// cycles of products over split sides (1290 over f16) and take 2500 (4600 by one issuing
// warp for both pipes).  2048 rows x 32 heads over 32768 states, K q8_0 and V q4_0: the
// kernel 1.11 ms at 1.93 GHz, calls in a row 1.12 ms and, once the power limit holds the
// clock down, 1.21; over 8192 the tensor pipe is busy for 78 % of the kernel's 0.31 ms.  turbo4
// keys, which leave no room for pairs: 1.43 ms (values turbo4), 1.48 (q8_0).  Where rows are few
// the codes' conversion, about 1000 cycles for 64 keys of q8_0: 120 beams x 40 heads over 24
// inputs of up to 4096 states, K f16 and V q8_0, the kernel 52 us, calls in a row 55 (24 at
// the copy rate).  One row a sequence: 16 over 1500 states 15 to 18 us a call; attn_decode, which
// reads the codes as its operands, takes 14.5, and half for 64 rows over 4096 (110 and 197 us).
#include <cuda_runtime.h>

#include <algorithm>

#include <math.h>

#include "kvq_launch.h"
#include "kvq_packed.cuh"
#include "kvq_rope.cuh"
#include "kvq_row_decode.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kTile = 128;                        // query rows of a tile
constexpr int kKeys = 64;                         // keys of a step
constexpr int kHalf = kKeys / 2;                  // keys of a score buffer
constexpr int kUnits = kKeys / kUnitTokens;       // units of a step, and of a ring slot
constexpr int kBufs = 2;                          // operand tiles of each side
constexpr int kMaxSlots = 8;                      // of one side
constexpr int kThreads = 640;
// warps 0-3, 4-7: softmax pipes; 8-11, 12-15: tiles of K, of V; 16, 19: copies of K's
// codes, of V's; 17, 18: products of each pipe
constexpr int kTileWarp = 8, kCopyWarp = 16, kMmaWarp = 17, kCopyWarpV = 19;
// K's ring, then V's.  What is in flight is what it holds: 24 beams of f16 and q8_0
// states took 73 us with 64 KB of it and one warp for both sides' copies.
constexpr int kRingBytes = 98304;
constexpr int kSmemBytes = 2 * kBufs * kTileBytes + kRingBytes;
constexpr float kRaise = 8.0f;                    // log2 units, as in the prefill
// Weights are held as 2^(s - m + 6): at most 2^14 in fp16, and 2^6 further from
// its subnormals than 2^(s - m).
constexpr float kLift = 6.0f;
// From here on (log2 units) a maximum is too large for fp16 weights: 2^(s - m + 6 + 8) and
// the steps of s and of m, 1 or more each from 2^24, leave fp16's range.
constexpr float kFar = 0x1p22f;
// A partial tile: O as [32 groups of 4 dims][128 rows], so that a warp's rows are
// written and read as whole lines (row by row the lines' parts took 8000 cycles), then
// (m, l) of every row.
constexpr int kPartFloats = kTile * kD + 2 * kTile;
// Work: what a step of a single tile and of a pair count (cycle counters: 1300 to 1550
// and 1900 to 2900), and what an item counts besides its steps (queries, results, the
// pipeline's fill).  With 8, 12, 16, 20, 24 and 28 for the latter a call took, in us: 24 chats
// behind three prompts 52.1, 50.5, 49.2, 49.6, 48.8, 49.0; 120 beams over f16 and q8_0 states 58.1,
// 54.0, 55.0, 55.1, 55.9, 57.2; 3011 rows of eight targets 107, 97, 89.8, 88.4, 88.2, 88.1; of
// fourteen others none differs by more than 3% from 16 on.
constexpr int kSingle = 2, kPair = 3;
constexpr int kItemCost = 24;

// An item whose pieces are to be joined: n of them, of the CTAs from its first on.
struct __align__(16) JoinItem {
  int64_t first;  // the sequence's first row
  int R, row0;    // its rows per kv head; the block's first
  int kvh, rows;  // kv head; the block's rows
  int n, pad;     // (0: no item)
};

struct CrossParams {
  const uint8_t *cache[2];
  int codec[2];
  const uint8_t *q;
  int64_t q_row, q_head, out_row, out_head;  // strides in bytes
  int q_bf16;                                // q and out: bf16, else fp16
  CrossOut out;
  float *part;  // partial slots [2 per CTA][slot_floats]: a tile or two of kPartFloats
  int slot_floats;
  JoinItem *items;  // [CTAs]: the split item that begins in each one's slice
  PackedRows rows;
  const int32_t *seq_lens, *table;
  int32_t *err;
  int n_q, n_kv, G, capacity, max_len, pages_per_seq, n_pages;
  int slots[2];  // ring slots of K and V codes
  int singles;   // no pairs: the second query tile's place holds the rest of a turbo4 query
  float scale_log2;
};

// ------------------------------------------------------------------ work

// a / b of numbers that are not negative, mostly small.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b))
                              : a / b;
}

// x work as steps of weight w, rounded up.
__device__ __forceinline__ int64_t steps_in(int64_t x, int w) {
  return w == kPair ? (x + kPair - 1) / kPair : (x + kSingle - 1) / kSingle;
}

// One sequence's rows and keys.
struct SeqWork {
  int64_t first;     // first row (token)
  int R;             // rows per kv head: tokens * G
  int len, nt;       // keys, key tiles (0: nothing to do)
  int blocks, full;  // pairs and the single tile if there is one (singles: tiles); weight
  bool odd;          // the last block is a single tile among pairs
  __device__ __forceinline__ int weight(int blk) const {
    return odd && blk == blocks - 1 ? kSingle : full;
  }
  __device__ __forceinline__ int64_t per_head() const {
    return nt == 0 ? 0 : static_cast<int64_t>(nt) * (full * blocks - (odd ? kPair - kSingle : 0)) +
                             static_cast<int64_t>(blocks) * kItemCost;
  }
  // position of block blk of kv head kvh, from the sequence's
  __device__ __forceinline__ int64_t at(int kvh, int blk) const {
    return kvh * per_head() + static_cast<int64_t>(blk) * (full * nt + kItemCost);
  }
};
__device__ __forceinline__ SeqWork seq_work(const CrossParams &p, int s) {
  SeqWork w;
  bool bad;
  const int64_t n = packed_rows(p.rows, s, w.first, bad);
  w.len = max(0, min(p.seq_lens[s], p.max_len));
  w.R = static_cast<int>(n) * p.G;
  w.nt = n > 0 ? (w.len + kKeys - 1) / kKeys : 0;
  const int tiles = (w.R - 1) / kTile + (w.R > 0);
  w.full = p.singles ? kSingle : kPair;
  w.blocks = p.singles ? tiles : (tiles + 1) / 2;
  w.odd = !p.singles && (tiles & 1) != 0;
  return w;
}
// The kv head and block at offset `off` of a sequence's work.
__device__ __forceinline__ void block_at(const SeqWork &w, int64_t off, int &kvh, int &blk) {
  const int64_t head = w.per_head();
  kvh = static_cast<int>(quotient(off, head));
  blk = static_cast<int>(min(quotient(off - kvh * head, w.full * w.nt + kItemCost),
                             static_cast<int64_t>(w.blocks - 1)));
}
// CTAs that get a slice: each of at least four steps of a single tile (of one at least,
// so that every CTA between an item's first and last has a step of it).  With at least two,
// four and eight: a decode step of 64 rows of two kv heads behind 4096 keys 21.3, 19.3 and 21.5
// us, one row of 16 sequences over 1500 15.1, 14.9 and 15.5; where there is more work than that
// for every CTA it makes no difference.
__device__ __forceinline__ int64_t cross_ctas(int64_t W, int grid) {
  return max(static_cast<int64_t>(1), min(static_cast<int64_t>(grid), W / (4 * kSingle)));
}
// The CTA whose slice [W c / P, W (c + 1) / P) holds position x.
__device__ __forceinline__ int64_t owner_of(int64_t x, int64_t W, int64_t P) {
  return quotient((x + 1) * P - 1, W);
}

struct Segment {
  int64_t first;  // the sequence's first row
  int R, row0;    // its rows per kv head; the block's first
  int s, kvh, len, nt, j_lo, j_hi;
  bool pair, inside;  // inside: the item's first step is in this CTA's slice
  int64_t at;         // and its position
};
// A CTA's segments: the pieces of the items that its slice [s0, s1) holds.
struct SegIter {
  int64_t s0, s1, at;  // at: the current item's first position
  SeqWork w;
  int s, kvh, blk;
  __device__ __forceinline__ bool next(const CrossParams &p, Segment &g) {
    while (at < s1) {
      const int wt = w.weight(blk);
      // its steps follow its cost
      const int64_t from = at + kItemCost;
      const int64_t lo = s0 <= from ? 0 : min(static_cast<int64_t>(w.nt), steps_in(s0 - from, wt));
      const int64_t hi = s1 <= from ? 0 : min(static_cast<int64_t>(w.nt), steps_in(s1 - from, wt));
      g.first = w.first;
      g.R = w.R;
      g.row0 = blk * (p.singles ? kTile : 2 * kTile);
      g.s = s;
      g.kvh = kvh;
      g.len = w.len;
      g.nt = w.nt;
      g.j_lo = static_cast<int>(lo);
      g.j_hi = static_cast<int>(hi);
      g.pair = wt == kPair;
      g.inside = from >= s0;
      g.at = from;
      at = from + static_cast<int64_t>(wt) * w.nt;
      if (++blk == w.blocks) {
        blk = 0;
        if (++kvh == p.n_kv) {
          kvh = 0;
          while (++s < p.rows.n_seqs) {
            w = seq_work(p, s);
            if (w.nt > 0) break;
          }
          if (s >= p.rows.n_seqs) at = INT64_MAX;
        }
      }
      if (lo < hi) return true;
    }
    return false;
  }
};
// ------------------------------------------------------------------ codes to operand tiles

__device__ __forceinline__ void sts128(uint8_t *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(a, b, c, d);
}
__device__ __forceinline__ void sts64(uint8_t *p, uint32_t a, uint32_t b) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
}
// c d as hi = RN16(c d) and the rest, which is exact.
struct Parts {
  uint32_t hi, lo;
};
__device__ __forceinline__ Parts scaled(uint32_t c, uint32_t d) {
  const __half2 x = *reinterpret_cast<__half2 *>(&c), y = *reinterpret_cast<__half2 *>(&d);
  const __half2 h = __hmul2(x, y), l = __hfma2(x, y, __hneg2(h));
  return {*reinterpret_cast<const uint32_t *>(&h), *reinterpret_cast<const uint32_t *>(&l)};
}
__device__ __forceinline__ uint32_t twice(uint32_t half) { return half * 0x10001u; }
// Quantized sides are split: x^ = d c has up to 18 bits, an operand 11, so a tile
// holds 64 keys twice, RN16(x^) and the rest.  (Rounded once, 128 keys to a tile,
// outputs over q8_0 sides were 4.1e-4 off, relative to their own rounding of
// 2.1e-4 and that of the weights, 1.7e-4; split they are 2.7e-4 off, as over f16.)
constexpr int kLoRows = 64;  // K: the rests' first row; V: their columns' half

// One unit of K into rows 16 u .. of the tile (all 32 lanes).  A lane takes the
// 16-byte pieces (g, w) of row g and row g + 8; the order of g over the lanes
// keeps loads (pieces 4 g + w) and stores (piece w ^ place of g) of eight lanes on
// distinct banks.
template <int CODEC>
__device__ __forceinline__ void unit_to_k(const uint8_t *u, uint8_t *tile, int row0, int lane) {
  const int q8 = lane >> 2, w = lane & 3;
  const int g = (q8 & 4) | ((0x2130 >> (4 * (q8 & 3))) & 3);
  const int place = row0 + 4 * (g >> 1) + (g & 1);
  uint8_t *row[2] = {tile + place * 128, tile + (place + 2) * 128};
  const int sw[2] = {place & 7, (place + 2) & 7};
  const uint8_t *src = u + (4 * g + w) * 16;
  auto at = [&](int rh, int b) {
    return row[rh] + (b >> 1) * kHalfBytes + (((4 * (b & 1) + w) ^ sw[rh]) << 4);
  };
  if (CODEC == KVQ_F16) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int rh = 0; rh < 2; ++rh)
        *reinterpret_cast<uint4 *>(at(rh, b)) = lds128(src + (2 * b + rh) * 512);
    return;
  }
  uint32_t d[4];  // scales by (row, pair of blocks); turbo4: by row
  if (CODEC == KVQ_TURBO4) {
    const uint32_t x = *reinterpret_cast<const uint32_t *>(u + 1024 + g * 4);
    d[0] = d[1] = twice(x & 0xffffu);
    d[2] = d[3] = twice(x >> 16);
  } else {
    const uint4 x = lds128(u + unit_scale_offset(CODEC) + g * 16);
    d[0] = x.x; d[1] = x.y; d[2] = x.z; d[3] = x.w;
  }
  auto put = [&](int rh, int b, const uint32_t (&c)[4]) {
    const uint32_t z = d[2 * rh + (b >> 1)];
    const uint32_t y = __byte_perm(z, z, (b & 1) ? 0x3232 : 0x1010);
    const Parts a0 = scaled(c[0], y), a1 = scaled(c[1], y);
    const Parts a2 = scaled(c[2], y), a3 = scaled(c[3], y);
    uint8_t *to = at(rh, b);
    sts128(to, a0.hi, a1.hi, a2.hi, a3.hi);
    sts128(to + kLoRows * 128, a0.lo, a1.lo, a2.lo, a3.lo);
  };
  if (CODEC == KVQ_Q8_0) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint4 x = lds128(src + b * 512);
      const uint32_t y[4] = {x.x, x.y, x.z, x.w};  // (rh, h)
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) {
        uint32_t o[4];
        s8_quad(y[2 * rh], o[0], o[1]);
        s8_quad(y[2 * rh + 1], o[2], o[3]);
        put(rh, b, o);
      }
    }
  } else {
#pragma unroll
    for (int bp = 0; bp < 2; ++bp) {
      const uint4 x = lds128(src + bp * 512);
      const uint32_t y[4] = {x.x, x.y, x.z, x.w};  // (b & 1, rh)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[4];
        u4_quad(y[i] & 0x0f0f0f0fu, o[0], o[1]);
        u4_quad((y[i] >> 4) & 0x0f0f0f0fu, o[2], o[3]);
        put(i & 1, 2 * bp + (i >> 1), o);
      }
    }
  }
}

// One unit of V into columns 16 u .. of the tile, whose rows are dims (all 32
// lanes).  A lane takes the pieces (gq, tig): two to eight dims of four tokens,
// eight bytes in each dim's row.  TAIL: of the unit only `live` tokens (any
// number, none and more than 16 included) are the sequence's; the others'
// columns are zeros, whatever lies there.
template <int CODEC, bool TAIL>
__device__ __forceinline__ void unit_to_v(const uint8_t *u, uint8_t *tile, int unit, int live,
                                          int lane) {
  const int q8 = lane >> 2, tig = lane & 3;
  const int gq = nibble_codec(CODEC) ? (0x65217430 >> (4 * q8)) & 7 : q8;
  uint8_t *col = tile + (unit >> 2) * kHalfBytes + (tig & 1) * 8;  // (split: units 0..3)
  const int piece = 2 * (unit & 3) + (tig >> 1);
  uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;  // tokens 2 tig, + 1; + 8, + 9
  if (TAIL) {
    auto mask = [&](int t) {
      return (t < live ? 0x0000ffffu : 0u) | (t + 1 < live ? 0xffff0000u : 0u);
    };
    m0 = mask(2 * tig);
    m1 = mask(2 * tig + 8);
  }
  auto put = [&](int dim, uint32_t a, uint32_t b) {
    if (TAIL) {
      a &= m0;
      b &= m1;
    }
    sts64(col + dim * 128 + ((piece ^ (dim & 7)) << 4), a, b);
  };
  auto put_split = [&](int dim, uint32_t a, uint32_t b, uint2 d) {
    const Parts x = scaled(a, d.x), y = scaled(b, d.y);
    put(dim, x.hi, y.hi);
    col += kHalfBytes;
    put(dim, x.lo, y.lo);
    col -= kHalfBytes;
  };
  const uint8_t *src = u + (4 * gq + tig) * 16;
  if (CODEC == KVQ_F16) {
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      const uint4 x = lds128(src + mt * 512);  // (rh, s)
      put(16 * mt + 2 * gq, x.x, x.z);
      put(16 * mt + 2 * gq + 1, x.y, x.w);
    }
  } else if (CODEC == KVQ_Q8_0) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint2 d = lds64(u + 2048 + tig * 32 + b * 8);
      const uint4 x = lds128(src + b * 512);
      const uint32_t y[4] = {x.x, x.y, x.z, x.w};  // (mt & 1, rh)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int dim = 32 * b + 16 * m + 2 * gq;
        put_split(dim, s8_pair_02(y[2 * m]), s8_pair_02(y[2 * m + 1]), d);
        put_split(dim + 1, s8_pair_13(y[2 * m]), s8_pair_13(y[2 * m + 1]), d);
      }
    }
  } else {
    uint2 d = make_uint2(0u, 0u);
    if (CODEC == KVQ_TURBO4) d = lds64(u + 1024 + tig * 8);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 x = lds128(src + h * 512);
      const uint32_t y[4] = {x.x, x.y, x.z, x.w};  // mt = 4 h + i; bytes (par, rh)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = 2 * h + (i >> 1), dim = 32 * b + 8 * (i & 1) + gq;
        if (CODEC == KVQ_Q4_0 && (i & 1) == 0) d = lds64(u + 1024 + tig * 32 + b * 8);
        const uint32_t z = y[i] >> 8;
        put_split(dim, u4_pair_minus8(y[i]), u4_pair_minus8(z), d);
        put_split(dim + 16, u4_pair_minus8_hi(y[i]), u4_pair_minus8_hi(z), d);
      }
    }
  }
}

__device__ __forceinline__ void unit_to_tile(int side, int codec, const uint8_t *u, uint8_t *tile,
                                             int unit, int live, int lane) {
  if (side == 0) {  // (rows past the length: their scores are masked)
    if (codec == KVQ_F16) unit_to_k<KVQ_F16>(u, tile, 16 * unit, lane);
    else if (codec == KVQ_Q8_0) unit_to_k<KVQ_Q8_0>(u, tile, 16 * unit, lane);
    else if (codec == KVQ_Q4_0) unit_to_k<KVQ_Q4_0>(u, tile, 16 * unit, lane);
    else unit_to_k<KVQ_TURBO4>(u, tile, 16 * unit, lane);
  } else if (live >= kUnitTokens) {
    if (codec == KVQ_F16) unit_to_v<KVQ_F16, false>(u, tile, unit, live, lane);
    else if (codec == KVQ_Q8_0) unit_to_v<KVQ_Q8_0, false>(u, tile, unit, live, lane);
    else if (codec == KVQ_Q4_0) unit_to_v<KVQ_Q4_0, false>(u, tile, unit, live, lane);
    else unit_to_v<KVQ_TURBO4, false>(u, tile, unit, live, lane);
  } else {
    if (codec == KVQ_F16) unit_to_v<KVQ_F16, true>(u, tile, unit, live, lane);
    else if (codec == KVQ_Q8_0) unit_to_v<KVQ_Q8_0, true>(u, tile, unit, live, lane);
    else if (codec == KVQ_Q4_0) unit_to_v<KVQ_Q4_0, true>(u, tile, unit, live, lane);
    else unit_to_v<KVQ_TURBO4, true>(u, tile, unit, live, lane);
  }
}
// The token, within a unit, of column c of a tile (mod 16).
__device__ __forceinline__ constexpr int token_of(int c) {
  return 8 * ((c >> 1) & 1) + 2 * ((c & 15) >> 2) + (c & 1);
}

// ------------------------------------------------------------------ TMEM pieces

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float (&v)[4]) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Unnormalised Sylvester-order FWHT of 32 values in registers.
__device__ __forceinline__ void fwht32(float (&v)[32]) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if ((i & h) == 0) {
        const float a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
}

// The stages across four groups of 32 (v[c]: 8 of group c's), and a factor.
__device__ __forceinline__ void across32(float (&v)[4][8], float f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = v[0][i] + v[1][i], b = v[0][i] - v[1][i];
    const float c = v[2][i] + v[3][i], d = v[2][i] - v[3][i];
    v[0][i] = (a + c) * f;
    v[1][i] = (b + d) * f;
    v[2][i] = (a - c) * f;
    v[3][i] = (b - d) * f;
  }
}

// Where a finished row goes: its place in out (fp16 or bf16, normalised), or
// fp32 (unnormalised) in xo or a partial slot.
struct RowOut {
  uint8_t *half;
  float *full;
  int step;  // floats between groups of 4 dims in full
  float inv;
  int bf16;
  // 8 values at dims d ..
  __device__ __forceinline__ void put(int d, const float (&x)[8]) const {
    if (full) {
      float *y = full + (d >> 2) * step;
      *reinterpret_cast<float4 *>(y) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4 *>(y + step) = make_float4(x[4], x[5], x[6], x[7]);
      return;
    }
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
    if (bf16) store_eight<KVQ_T_BF16>(half + 2 * d, y);
    else store_eight<KVQ_T_F16>(half + 2 * d, y);
  }
};

struct __align__(8) CrossBars {
  uint64_t raw_full[2][kMaxSlots], raw_empty[2][kMaxSlots];
  uint64_t tile_full[2][kBufs], tile_empty[2][kBufs];
  uint64_t sfull[2][2], pfull[2][2];  // by pipe and score buffer
  uint64_t odone[2], segdone[2], qready[2], ofree[2], drain[2];
};

// ------------------------------------------------------------------ attention

__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(x));
  return x != 0;
}
// D += A B with A in TMEM, B's descriptor as its low word and the constant HI.
template <uint32_t HI>
__device__ __forceinline__ void mma_ts_lo(bool leader, uint32_t d_tmem, uint32_t a_tmem,
                                          uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %6, 0;\n"
      " mov.b64 b, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(HI),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}
__device__ __forceinline__ void commit_if(bool leader, uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}

// max(a, b, c), NaN if one of them is.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ------------------------------------------------------------------ rows in fp32

// Where a segment's piece of a row and head lies: its fp32 O (groups of 4 dims `step` floats
// apart) or its 16-bit row, and its (m, l) or lse.
struct Piece {
  float *full;
  int step;
  float2 *ml;
  uint8_t *half;
  float *lse;
};
__device__ __forceinline__ Piece piece_of(const CrossParams &p, const Segment &g, int in) {
  const int R = g.row0 + in, tok = R / p.G, head = g.kvh * p.G + R - tok * p.G;
  const int64_t row = g.first + tok, at = row * p.n_q + head;
  if (g.j_lo > 0 || g.j_hi < g.nt) {
    float *const part = p.part +
                        (2 * static_cast<int64_t>(blockIdx.x) + (g.inside ? 1 : 0)) * p.slot_floats +
                        in / kTile * kPartFloats;
    const int r = in % kTile;
    return {part + 4 * r, 4 * kTile, reinterpret_cast<float2 *>(part + kTile * kD) + r, nullptr, nullptr};
  }
  if (p.out.xo) return {p.out.xo + at * kD, 4, p.out.xml + at, nullptr, nullptr};
  return {nullptr, 0, nullptr, static_cast<uint8_t *>(p.out.out) + row * p.out_row + head * p.out_head,
          p.out.lse ? p.out.lse + at : nullptr};
}

// Whether the piece is NaN somewhere (all 32 lanes).
__device__ __forceinline__ bool piece_is_nan(const CrossParams &p, const Piece &y, int lane) {
  float x[4], l = 0.0f;
  if (y.half) {
    if (p.q_bf16) load4<KVQ_T_BF16>(y.half + 8 * lane, x);
    else load4<KVQ_T_F16>(y.half + 8 * lane, x);
  } else {
    load4<KVQ_T_F32>(y.full + lane * y.step, x);
    l = y.ml->y;
  }
  const float most = fmax3_nan(fmax3_nan(x[0], x[1], x[2]), x[3], l);
  return __any_sync(0xffffffffu, most != most);
}

// A segment's piece of the block's row `in`, by a warp, lane l dims 4 l ..: every key as
// kvq_row_decode.cuh has it, its weight against the running maximum, sums of 256 keys added
// up.  A NaN among the weights ends it: nothing changes it any more.
__device__ __forceinline__ void piece_in_fp32(const CrossParams &p, const Segment &g, int in, int lane) {
  const int R = g.row0 + in, tok = R / p.G, head = g.kvh * p.G + R - tok * p.G;
  const uint8_t *src = p.q + (g.first + tok) * p.q_row + head * p.q_head + 8 * lane;
  float q[4], acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.q_bf16) load4<KVQ_T_BF16>(src, q);
  else load4<KVQ_T_F16>(src, q);
  float m = -INFINITY, l = 0.0f, lp = 0.0f;
  const int t0 = g.j_lo * kKeys, t1 = min(g.len, g.j_hi * kKeys);
  int64_t base = (static_cast<int64_t>(g.s) * p.n_kv + g.kvh) * (p.capacity / kUnitTokens);
#pragma unroll 1
  for (int t = t0; t < t1 && lp == lp; ++t) {
    constexpr int kPageTokens = kPageUnits * kUnitTokens;
    if (t == t0 || t % kPageTokens == 0) {
      const int page = t / kPageTokens;
      if (p.table)  // (an unmapped page: pool page 0, as the copies have it)
        base = (static_cast<int64_t>(max(0, page_of(p.table, p.pages_per_seq, p.n_pages, g.s, page))) *
                    p.n_kv + g.kvh) * kPageUnits - static_cast<int64_t>(page) * kPageUnits;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] += part[i];
        part[i] = 0.0f;
      }
      l += lp;
      lp = 0.0f;
    }
    const int64_t unit = base + t / kUnitTokens;
    float x[4];
    decode_row_lane<0>(p.codec[0], p.cache[0] + unit * unit_bytes(p.codec[0]), t % kUnitTokens, lane, x);
    float z = q[0] * x[0] + q[1] * x[1] + q[2] * x[2] + q[3] * x[3];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    z = __fmul_rn(z, p.scale_log2);  // (rounded: z - m below is then exact near it)
    if (z > m) {
      const float a = fast_exp2(m - z);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] *= a;
        part[i] *= a;
      }
      l *= a;
      lp *= a;
      m = z;
    }
    const float w = z == -INFINITY ? 0.0f : fast_exp2(z - m);
    lp += w;
    decode_row_lane<1>(p.codec[1], p.cache[1] + unit * unit_bytes(p.codec[1]), t % kUnitTokens, lane, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) part[i] = fmaf(w, x[i], part[i]);
  }
  l += lp;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = l != l ? l : acc[i] + part[i];
  if (l != l) m = INFINITY;  // (as above: no join leaves it out)
  const Piece y = piece_of(p, g, in);
  if (y.full) {
    store4<KVQ_T_F32>(y.full + lane * y.step, acc);
    if (lane == 0) *y.ml = make_float2(m, l);
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] *= inv;
  if (p.q_bf16) store4<KVQ_T_BF16>(y.half + 8 * lane, acc);
  else store4<KVQ_T_F16>(y.half + 8 * lane, acc);
  if (y.lse && lane == 0)
    *y.lse = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// The pieces of a CTA's rows that are NaN (all warps, once its results are written).  (A call
// of its own in the kernel costs the loops before it registers: 3011 rows 87 -> 93 us.)
__device__ __forceinline__ void nan_rows_in_fp32(const CrossParams &p, SegIter it, Segment g, int warp,
                                              int lane) {
  do {
    const int rows = min(g.R - g.row0, g.pair ? 2 * kTile : kTile);
    for (int in = warp; in < rows; in += kThreads / 32)
      if (piece_is_nan(p, piece_of(p, g, in), lane)) piece_in_fp32(p, g, in, lane);
  } while (it.next(p, g));
}

// ------------------------------------------------------------------ rows without keys

// Rows times query heads of a sequence without keys that one CTA writes while it looks for its
// slice, about 10 ns each; more of them go over all CTAs (4096 rows of 32 heads beside 64
// rows over 1500 keys: 1430 -> 32 us).
constexpr int64_t kFillRows = 512;
__device__ __forceinline__ void fill_row(const CrossParams &p, int64_t row, int head, int lane) {
  const int64_t at = row * p.n_q + head;
  if (p.out.xo) {
    if (lane == 0) p.out.xml[at] = make_float2(-INFINITY, 0.0f);
  } else {
    reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out.out) + row * p.out_row +
                              head * p.out_head)[lane] = make_uint2(0u, 0u);
    if (p.out.lse && lane == 0) p.out.lse[at] = -INFINITY;
  }
}
// Row i of those of the sequence whose first row is `first`.
__device__ __forceinline__ void fill_row_at(const CrossParams &p, int64_t first, int64_t i, int lane) {
  const int64_t tok = quotient(i, p.n_q);
  fill_row(p, first + tok, static_cast<int>(i - tok * p.n_q), lane);
}
// The n sequences of many rows (noted: the first kManySeqs of them).
constexpr int kManySeqs = 8;
__device__ __forceinline__ void fill_many_rows(const CrossParams &p, int n, const int *noted, int warp,
                                               int lane) {
  const bool all = n > kManySeqs;
#pragma unroll 1
  for (int k = 0; k < (all ? p.rows.n_seqs : n); ++k) {
    const SeqWork w = seq_work(p, all ? k : noted[k]);
    const int64_t end = static_cast<int64_t>(w.R) * p.n_kv;
    if (w.len > 0 || end <= kFillRows) continue;
#pragma unroll 1
    for (int64_t i = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x; i < end;
         i += (kThreads / 32) * static_cast<int64_t>(gridDim.x))
      fill_row_at(p, w.first, i, lane);
  }
}

// Both softmax pipes (256 threads).
__device__ __forceinline__ void pipes_sync() {
  asm volatile("bar.sync 1, 256;\n" ::: "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    cross_attn_kernel(const __grid_constant__ CrossParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ CrossBars bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ SegIter begin;      // the slice, behind its first segment
  __shared__ Segment first_seg;
  __shared__ int have_first;
  __shared__ int many_n, many_seq[kManySeqs];  // sequences without keys that have many rows
  __shared__ int64_t all[2];     // all work, and the CTAs that share it
  __shared__ float2 pipe_ml[2][kTile];  // of a single tile's pipes
  __shared__ int any_nan;               // among the CTA's rows
  uint8_t *tiles = smem, *ring = smem + 2 * kBufs * kTileBytes;  // operand tiles of K, of V; codes
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);  // (uniform)
  const int lane = threadIdx.x & 31;

  // (swizzled tiles lie at multiples of 1024 bytes, as this memory is declared; there is
  // none left to round up in)
  if ((smem_u32(smem) & 1023u) != 0) {
    grid_dependency_wait();
    set_err(p.err, KVQ_DEVERR_TIMEOUT);
    if (threadIdx.x == 0) p.items[blockIdx.x].n = 0;  // nothing to join
    return;
  }

  // What needs no other kernel's results
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_base_sh, 512);
  } else if (warp == kCopyWarp) {
    if (lane == 0) {
      abort_flag = 0;
      any_nan = 0;
      for (int i = 0; i < 2 * kMaxSlots; ++i) {
        mbar_init(&bars.raw_full[0][i], 1);
        mbar_init(&bars.raw_empty[0][i], kUnits);  // one arrival per unit
      }
      for (int i = 0; i < 2 * kBufs; ++i) {
        mbar_init(&bars.tile_full[0][i], kUnits);
        mbar_init(&bars.tile_empty[0][i], 2);  // both pipes' products
      }
      for (int i = 0; i < 2; ++i) {
        for (int b = 0; b < 2; ++b) {
          mbar_init(&bars.sfull[i][b], 1);
          mbar_init(&bars.pfull[i][b], 4);  // one arrival per softmax warp
        }
        mbar_init(&bars.odone[i], 1);
        mbar_init(&bars.segdone[i], 1);
        mbar_init(&bars.qready[i], 4);
        mbar_init(&bars.ofree[i], 4);
        mbar_init(&bars.drain[i], 1);
      }
      fence_mbar_init();
    }
  }
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {  // this CTA's slice, and where it begins
    if (lane == 0) many_n = 0;
    __syncwarp();
    int64_t sum = 0;
    SeqWork mine;  // (of up to 32 sequences: looked up once)
    for (int s = lane; s < p.rows.n_seqs; s += 32) {
      if (blockIdx.x == 0) {
        bool bad;
        int64_t first;
        packed_rows(p.rows, s, first, bad);
        if (bad) set_err(p.err, KVQ_DEVERR_ROWS);
        if (p.seq_lens[s] > p.max_len) set_err(p.err, KVQ_DEVERR_MAXLEN);
      }
      mine = seq_work(p, s);
      sum += mine.per_head() * p.n_kv;
      if (mine.len == 0 && static_cast<int64_t>(mine.R) * p.n_kv > kFillRows) {
        const int k = atomicAdd(&many_n, 1);
        if (k < kManySeqs) many_seq[k] = s;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int64_t W = sum, P = cross_ctas(W, gridDim.x), c = blockIdx.x;
    const int64_t s0 = c < P ? quotient(W * c, P) : W, s1 = c < P ? quotient(W * (c + 1), P) : W;
    if (lane == 0) {
      have_first = 0;
      all[0] = W;
      all[1] = P;
      p.items[blockIdx.x].n = 0;
    }
    __syncwarp();
    if (s0 < s1) {
      int64_t carry = 0;
      for (int base = 0; base < p.rows.n_seqs; base += 32) {
        const int s = base + lane;
        if (p.rows.n_seqs > 32 && s < p.rows.n_seqs) mine = seq_work(p, s);
        const int64_t n = s < p.rows.n_seqs ? mine.per_head() * p.n_kv : 0;
        int64_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        const unsigned past = __ballot_sync(0xffffffffu, carry + incl > s0);
        if (past) {
          if (lane == __ffs(past) - 1) {
            const int64_t seq_at = carry + incl - n;
            SegIter it;
            it.s0 = s0;
            it.s1 = s1;
            it.s = s;
            it.w = mine;
            block_at(mine, s0 - seq_at, it.kvh, it.blk);
            it.at = seq_at + mine.at(it.kvh, it.blk);
            Segment g;
            have_first = it.next(p, g);
            first_seg = g;
            begin = it;
          }
          break;
        }
        carry += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  } else {  // rows of sequences without keys
    for (int s = blockIdx.x; s < p.rows.n_seqs; s += gridDim.x) {
      const SeqWork w = seq_work(p, s);
      const int64_t n = static_cast<int64_t>(w.R) * p.n_kv;  // rows x query heads
      if (w.len > 0 || n > kFillRows) continue;
      for (int64_t i = warp - 1; i < n; i += kThreads / 32 - 1)
        fill_row_at(p, w.first, i, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  if (many_n > 0) fill_many_rows(p, many_n, many_seq, warp, lane);
  if (!have_first) {  // whole CTA: no work
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
    return;
  }
  // columns: each pipe's two score buffers (32 keys each), query tiles, outputs
  const uint32_t tm_s[2] = {tmem, tmem + 64}, tm_q[2] = {tmem + 128, tmem + 192};
  const uint32_t tm_o[2] = {tmem + 256, tmem + 384};
  SegIter it = begin;
  Segment sg = first_seg;
  bool have = true;

  if (warp >= kCopyWarp) {
    if (warp == kCopyWarp || warp == kCopyWarpV) {
      // ---------------- codes into a side's ring, a step at a time
      if (lane == 0) {
        const int side = warp == kCopyWarp ? 0 : 1, slots = p.slots[side];
        const int ub = unit_bytes(p.codec[side]);
        uint8_t *const to = ring + (side ? p.slots[0] * kUnits * unit_bytes(p.codec[0]) : 0);
        int slot = 0;
        uint32_t turn = 0;
        bool ok = true;
        for (; ok && have; have = it.next(p, sg)) {
          const int units = (sg.len + kUnitTokens - 1) / kUnitTokens;
          // the units of the sequence's kv head; in pages, those of the current page
          int64_t base = (static_cast<int64_t>(sg.s) * p.n_kv + sg.kvh) * (p.capacity / kUnitTokens);
          for (int j = sg.j_lo; j < sg.j_hi; ++j) {
            const int u0 = j * kUnits;
            if (p.table && (j == sg.j_lo || u0 % kPageUnits == 0)) {  // (a step lies inside one page)
              int pg = page_of(p.table, p.pages_per_seq, p.n_pages, sg.s, u0 / kPageUnits);
              if (pg < 0) {
                set_err(p.err, KVQ_DEVERR_PAGE);
                pg = 0;  // read pool page 0 in its place
              }
              base = (static_cast<int64_t>(pg) * p.n_kv + sg.kvh) * kPageUnits -
                     u0 / kPageUnits * kPageUnits;
            }
            uint64_t *full = &bars.raw_full[side][slot];
            if (turn > 0 && !mbar_wait_bounded(&bars.raw_empty[side][slot], (turn - 1) & 1u, &abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t bytes = static_cast<uint32_t>(min(kUnits, units - u0) * ub);
            mbar_arrive_expect_tx(full, bytes);
            bulk_copy_g2s(to + slot * kUnits * ub, p.cache[side] + (base + u0) * ub, bytes, full);
            if (++slot == slots) {
              slot = 0;
              ++turn;
            }
          }
        }
        // after an abort, wait (bounded) for the copies still landing in the ring: each
        // slot's last one
        if (!ok || *reinterpret_cast<volatile int *>(&abort_flag))
          for (int i = 0; i < slots; ++i) {
            const uint32_t n = turn + (i < slot ? 1u : 0u);  // copies into it
            if (n > 0)
              mbar_wait_bounded(&bars.raw_full[side][i], (n - 1) & 1u, nullptr, 100000000ull);
          }
      }
    } else {
      // ---------------- MMA issuer of pipe e.  The whole warp walks the steps, so that what an
      // instruction takes is known to be uniform; one elected thread issues.  (By one
      // thread of a diverged warp, with descriptors put together for each, an
      // instruction took about 96 cycles whatever its size; the tensor core takes
      // 16 for 32 keys of K and 64 for 16 keys of V.  Turns, one warp waiting while the
      // other issues, took 8 % longer than both at will.)
      const int e = warp - kMmaWarp;
      const bool leader = elect_one();
      const bool split_k = p.codec[0] != KVQ_F16, split_v = p.codec[1] != KVQ_F16;
      constexpr uint32_t idesc_k = idesc_f16(0, kHalf), idesc_v = idesc_f16(0);
      // A tile's 16 columns kk: 32 bytes on inside 64 columns, then the next half.
      // The low word of the descriptor is all that changes from one to the next.
      constexpr uint32_t kLo = 1u << 16, kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
      const uint32_t tile0 = kLo | ((smem_u32(tiles) & 0x3FFFFu) >> 4);
      auto step = [](int kk) { return ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16; };
      auto wait = [&](uint64_t *bar, int phase) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, static_cast<uint32_t>(phase) & 1u,
                                                         &abort_flag)) != 0;
      };
      // S = Q K^T of half h of K's tile u into score buffer b: split keys add their rests'
      // products, turbo4 those of the rest of Q (at a: the query tile)
      auto qk = [&](uint32_t a, int u, int h, int b) {
        const uint32_t k = tile0 + (u % kBufs) * (kTileBytes / 16) + h * (kHalf * 128 / 16);
        const uint32_t d = tm_s[e] + b * kHalf;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_lo<kHi>(leader, d, a + kk * 8, k + step(kk), idesc_k, kk > 0);
        if (split_k) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_lo<kHi>(leader, d, a + kk * 8, k + kLoRows * 8 + step(kk), idesc_k, 1u);
        }
        if (p.singles) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_lo<kHi>(leader, d, tm_q[1] + kk * 8, k + step(kk), idesc_k, 1u);
        }
        commit_if(leader, &bars.sfull[e][b]);
      };
      // O (+)= P V of half h of V's tile u, P from score buffer b; split values: the
      // same P with the rests, columns 64 .. of V
      auto pv = [&](int u, int h, int b, bool first) {
        const uint32_t v = tile0 + (kBufs + u % kBufs) * (kTileBytes / 16) + h * (kHalf * 2 / 16);
        const uint32_t d = tm_o[e], a = tm_s[e] + b * kHalf;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
          mma_ts_lo<kHi>(leader, d, a + kk * 8, v + step(kk), idesc_v, (!first || kk > 0) ? 1u : 0u);
        if (split_v) {
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            mma_ts_lo<kHi>(leader, d, a + kk * 8, v + step(4 + kk), idesc_v, 1u);
        }
        commit_if(leader, &bars.odone[e]);
      };
      // tiles of a side are numbered over all segments
      auto free_tile = [&](int side, int u) {
        commit_if(leader, &bars.tile_empty[side][u % kBufs]);
      };
      auto have_tile = [&](int side, int u) {
        return wait(&bars.tile_full[side][u % kBufs], u / kBufs);
      };
      // a barrier, and tiles of V and K where they are asked for
      auto wait3 = [&](uint64_t *bar, int phase, bool need_v, int uv, bool need_k, int uk) {
        uint64_t *const v = need_v ? &bars.tile_full[1][uv % kBufs] : bar;
        uint64_t *const x = need_k ? &bars.tile_full[0][uk % kBufs] : bar;
        const int vp = need_v ? uv / kBufs : phase, xp = need_k ? uk / kBufs : phase;
        const bool a = mbar_try_wait(bar, static_cast<uint32_t>(phase) & 1u);
        const bool b = mbar_try_wait(v, static_cast<uint32_t>(vp) & 1u);
        const bool c = mbar_try_wait(x, static_cast<uint32_t>(xp) & 1u);
        if (__all_sync(0xffffffffu, a & b & c)) return true;
        return wait(bar, phase) && wait(v, vp) && wait(x, xp);
      };
      int u0 = 0;  // tiles of earlier segments
      int c0 = 0;  // halves that the pipe has taken in earlier segments
      int k = 0;   // segments
      bool ok = true;
      for (; ok && have; have = it.next(p, sg)) {
        const int n = sg.j_hi - sg.j_lo;
        const bool pair = sg.pair;
        // The pipe's halves i: of a pair both of every tile, of a single tile's the
        // pipe's own of every tile.
        const int cnt = pair ? 2 * n : n;
        const uint32_t q = tm_q[pair ? e : 0];
        auto scores = [&](int i) {  // of half i
          const int t = pair ? i >> 1 : i;
          qk(q, u0 + t, pair ? i & 1 : e, (c0 + i) & 1);
          if (!pair || (i & 1)) free_tile(0, u0 + t);
        };
        ok = wait(&bars.qready[e], k) && have_tile(0, u0) &&
             (pair || cnt == 1 || have_tile(0, u0 + 1)) &&
             (k == 0 || wait(&bars.ofree[e], k - 1));
        if (!ok) break;
        tc_fence_after();
        scores(0);
        if (cnt > 1) scores(1);
        for (int i = 0; i < cnt; ++i) {
          const int t = pair ? i >> 1 : i, b = (c0 + i) & 1;
          // P of half i, V's tile, and K's of half i + 2, asked for together: one wait
          // after the other the tensor core ran dry between them (100 cycles each)
          const int tk = pair ? t + 1 : t + 2;
          const bool fresh = !pair || (i & 1) == 0;  // not asked for with the half before
          ok = wait3(&bars.pfull[e][b], (c0 + i) >> 1, fresh, u0 + t, fresh && tk < n, u0 + tk);
          if (!ok) break;
          tc_fence_after();
          pv(u0 + t, pair ? i & 1 : e, b, i == 0);
          if (!pair || (i & 1)) free_tile(1, u0 + t);
          if (i + 2 < cnt) scores(i + 2);
        }
        if (!ok) break;
        u0 += n;
        c0 += cnt;
        ++k;
        commit_if(leader, &bars.segdone[e]);  // the pipe's O is complete
      }
      if (!ok && lane == 0) {
        set_err(p.err, KVQ_DEVERR_TIMEOUT);
        atomicExch(&abort_flag, 1);
      }
      // drain: every MMA the thread issued has finished (TMEM is freed after it)
      commit_if(leader, &bars.drain[e]);
      mbar_wait_bounded(&bars.drain[e], 0, nullptr, 100000000ull);
    }
  } else if (warp >= kTileWarp) {
    // ---------------- codes into operand tiles: warp w of a side takes unit w of each
    const int side = (warp - kTileWarp) >> 2, unit = warp & 3;
    const int codec = p.codec[side];
    const int slot_bytes = kUnits * unit_bytes(codec), slots = p.slots[side];
    const uint8_t *src = ring + (side ? p.slots[0] * kUnits * unit_bytes(p.codec[0]) : 0) +
                         unit * unit_bytes(codec);
    int u = 0, slot = 0;  // this side's tiles so far; its next ring slot
    uint32_t turn = 0;
    bool ok = true;
    for (; ok && have; have = it.next(p, sg)) {
      const int n = sg.j_hi - sg.j_lo;
      for (int j = 0; j < n; ++j, ++u) {
        const int buf = u % kBufs;
        uint64_t *const raw = &bars.raw_full[side][slot], *const place = &bars.tile_empty[side][buf];
        const uint32_t gone = static_cast<uint32_t>(u / kBufs - 1) & 1u;
        const bool there = mbar_try_wait(raw, turn & 1u);  // asked for together: beams 50.9 -> 49.6 us
        const bool free = u < kBufs || mbar_try_wait(place, gone);
        if (!__all_sync(0xffffffffu, there & free)) {
          ok = mbar_wait_bounded(raw, turn & 1u, &abort_flag) &&
               (u < kBufs || mbar_wait_bounded(place, gone, &abort_flag));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        const int live = sg.len - (sg.j_lo + j) * kKeys - unit * kUnitTokens;
        unit_to_tile(side, codec, src + slot * slot_bytes,
                     tiles + (side * kBufs + buf) * kTileBytes, unit, live, lane);
        fence_proxy_async_smem();  // generic-proxy writes, read by the tensor core
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.raw_empty[side][slot]);
          mbar_arrive(&bars.tile_full[side][buf]);
        }
        if (++slot == slots) {
          slot = 0;
          ++turn;
        }
      }
    }
    if (!ok && lane == 0) {
      set_err(p.err, KVQ_DEVERR_TIMEOUT);
      atomicExch(&abort_flag, 1);
    }
  } else {
    // ---------------- softmax pipe e: thread = query row
    const int e = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tms = tm_s[e] + lane_off, tmo = tm_o[e] + lane_off;
    const bool rot_k = p.codec[0] == KVQ_TURBO4, rot_v = p.codec[1] == KVQ_TURBO4;
    // This pipe's query tile of a segment, a thread its own row, as fp16 in K's order
    // of dims into TMEM, where the products take it from (with both operands in
    // shared memory they took twice as long); then tell the pipe's issuer.  A single
    // tile is pipe 0's, for both issuers.
    auto load_q = [&](const Segment &g) {
      if (e == 1 && !g.pair) return;
      const int R = g.row0 + e * kTile + r;
      const bool have = R < g.R;
      const int tok = have ? R / p.G : 0, head = g.kvh * p.G + (have ? R - tok * p.G : 0);
      const uint8_t *src = p.q + (g.first + tok) * p.q_row + head * p.q_head;
      auto eight = [&](int d) {  // dims d ..
        return have ? *reinterpret_cast<const uint4 *>(src + 2 * d) : make_uint4(0u, 0u, 0u, 0u);
      };
      if (rot_k) {
        // H (s q) / 16 by way of this pipe's columns of O, which are free: the stages
        // inside 32 dims, then those across; two parts, the second in tile 1's place
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float v[32];
          const uint32_t signs = turbo_signs(c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            Eight<KVQ_T_F16> x;
            x.w[0] = eight(32 * c + 8 * k);
            float(&f)[8] = reinterpret_cast<float(&)[8]>(v[8 * k]);
            if (p.q_bf16) eight_values<KVQ_T_BF16>(*reinterpret_cast<Eight<KVQ_T_BF16> *>(&x), f);
            else eight_values<KVQ_T_F16>(x, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (signs >> (8 * k + i)) & 1u ? -f[i] : f[i];
          }
          fwht32(v);
          tmem_st32f(tmo + c * 32, v);
        }
        tmem_wait_st();
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {  // dims 32 c + 4 m .., + 16: columns 16 c + 4 m .. of Q
          float v[4][8];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld4(tmo + c * 32 + 4 * m, reinterpret_cast<float(&)[4]>(v[c][0]));
            tmem_ld4(tmo + c * 32 + 4 * m + 16, reinterpret_cast<float(&)[4]>(v[c][4]));
          }
          tmem_wait_ld();
          across32(v, 0.0625f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              hi[i] = pack_half2(v[c][2 * i], v[c][2 * i + 1]);
              const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi[i]));
              lo[i] = pack_half2(v[c][2 * i] - f.x, v[c][2 * i + 1] - f.y);
            }
            tmem_st4(tm_q[0] + lane_off + 16 * c + 4 * m, hi);
            tmem_st4(tm_q[1] + lane_off + 16 * c + 4 * m, lo);
          }
        }
      } else {
        uint4 two[2][4];  // (two blocks' pieces requested together)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if ((b & 1) == 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) two[k >> 2][k & 3] = eight(32 * b + 8 * k);
          }
          uint4(&x)[4] = two[b & 1];
          if (p.q_bf16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t *y = reinterpret_cast<uint32_t *>(&x[k]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                // (y 0 + y: an infinity, of a value past fp16's, becomes NaN)
                const uint32_t z =
                    pack_half2(__uint_as_float(y[i] << 16), __uint_as_float(y[i] & 0xffff0000u));
                const __half2 h = *reinterpret_cast<const __half2 *>(&z);
                const __half2 v = __hfma2(h, __float2half2_rn(0.0f), h);
                y[i] = *reinterpret_cast<const uint32_t *>(&v);
              }
            }
          }
          const uint32_t w[16] = {x[0].x, x[0].y, x[2].x, x[2].y, x[0].z, x[0].w, x[2].z, x[2].w,
                                  x[1].x, x[1].y, x[3].x, x[3].y, x[1].z, x[1].w, x[3].z, x[3].w};
          tmem_st16(tm_q[e] + lane_off + 16 * b, w);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.qready[e]);
        if (!g.pair) mbar_arrive(&bars.qready[1]);
      }
    };
    int c0 = 0, kseg = 0;  // halves and segments of this pipe so far
    bool ok = true;
    if (have) load_q(sg);
    while (have) {
      const int n = sg.j_hi - sg.j_lo, cnt = sg.pair ? 2 * n : n;
      const int row0 = sg.row0 + (sg.pair ? e * kTile : 0);
      const bool idle = row0 + quad * 32 >= sg.R;  // no row in this warp
      float m = -INFINITY, l = 0.0f, far = 0.0f;
      // After an abort (ok false) the segments still run to the end without waits,
      // so that both pipes meet at the same barriers.
      for (int i = 0; i < cnt && ok; ++i) {
        const int b = (c0 + i) & 1;
        ok = mbar_wait_bounded(&bars.sfull[e][b], static_cast<uint32_t>((c0 + i) >> 1) & 1u,
                               &abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) atomicExch(&abort_flag, 1);
          break;
        }
        tc_fence_after();
        if (!idle) {
          // keys from the half's first on
          const int left = sg.len - (sg.pair ? (2 * sg.j_lo + i) * kHalf
                                             : (2 * (sg.j_lo + i) + e) * kHalf);
          float v[kHalf];
          tmem_ld32(tms + b * kHalf, v);
          tmem_wait_ld();
          if (left < kHalf) {  // places past the length
#pragma unroll
            for (int c = 0; c < kHalf; ++c)
              if ((c & 16) + token_of(c) >= left) v[c] = -INFINITY;
          }
          float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < kHalf; c += 2) mp[(c >> 1) & 3] = fmax3(mp[(c >> 1) & 3], v[c], v[c + 1]);
          const float mx = fmaxf(fmax3(mp[0], mp[1], mp[2]), mp[3]) * p.scale_log2;
          // A row's running maximum is raised only when it grew by more than the
          // threshold; O is rescaled for the whole warp when one of its rows is.
          const bool raise = mx > m + kRaise || m == -INFINITY;
          const float mnew = raise ? fmaxf(mx, m) : m;
          const float a = (raise && m != -INFINITY) ? fast_exp2(m - mnew) : 1.0f;
          if (__any_sync(0xffffffffu, raise && m != -INFINITY)) {
            // every product of the halves before is in O: the one before the last was
            // done before these scores were, the last is waited for
            bool got = mbar_wait_bounded(&bars.odone[e], static_cast<uint32_t>(c0 + i - 1) & 1u,
                                         &abort_flag);
            got = __all_sync(0xffffffffu, got);
            if (!got) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              float x[16];
              tmem_ld16(tmo + c * 16, x);
              tmem_wait_ld();
              uint32_t y[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(x[k] * a);
              tmem_st16(tmo + c * 16, y);
            }
            tmem_wait_st();
          }
          l *= a;
          m = mnew;
          // P = exp2(s * scale_log2 - m + lift) as fp16 pairs over S, and the row's sum.
          const float nm = m == -INFINITY ? 0.0f : kLift - m;
          far = fmaxf(far, fabsf(nm));
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(nm, nm);
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
          uint32_t pk[kHalf / 2];
#pragma unroll
          for (int c = 0; c < kHalf / 2; ++c) {
            const float2 tt = fma2(make_float2(v[2 * c], v[2 * c + 1]), sc2, nm2);
            const float2 x = make_float2(fast_exp2(tt.x), fast_exp2(tt.y));
            sum[c & 1] = add2(sum[c & 1], x);
            pk[c] = pack_half2(x.x, x.y);
          }
          tmem_st16(tms + b * kHalf, pk);
          const float2 s2 = add2(sum[0], sum[1]);
          l += s2.x + s2.y;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.pfull[e][b]);
      }
      c0 += cnt;
      // Once both pipes have read their last scores the query tiles are free, and no
      // pipe is further than that ahead of the other.
      pipes_sync();
      Segment nsg;
      const bool have_next = it.next(p, nsg);
      if (have_next && !rot_k) load_q(nsg);
      if (ok) ok = mbar_wait_bounded(&bars.segdone[e], static_cast<uint32_t>(kseg) & 1u, &abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      ++kseg;
      tc_fence_after();
      if (far >= kFar) l = NAN;
      // The row's place: out (whole items), xo, or this CTA's partial slot.
      const bool whole = sg.j_lo == 0 && sg.j_hi == sg.nt;
      const int R = row0 + r, tok = R / p.G;
      const bool valid = R < sg.R;
      const int head = sg.kvh * p.G + R - tok * p.G;
      const int64_t row = valid ? sg.first + tok : 0, at = row * p.n_q + head;
      RowOut ro;
      ro.half = nullptr;
      ro.full = nullptr;
      ro.bf16 = p.q_bf16;
      float *const slot = p.part +
                          (2 * static_cast<int64_t>(blockIdx.x) + (sg.inside ? 1 : 0)) * p.slot_floats +
                          (sg.pair ? e : 0) * kPartFloats;
      ro.step = whole ? 4 : 4 * kTile;
      if (!whole)
        ro.full = slot + 4 * r;
      else if (p.out.xo)
        ro.full = p.out.xo + at * kD;
      else
        ro.half = static_cast<uint8_t *>(p.out.out) + row * p.out_row + head * p.out_head;
      if (!whole && sg.inside && threadIdx.x == 0) {
        const int64_t last = sg.at + static_cast<int64_t>(sg.nt - 1) * (sg.pair ? kPair : kSingle);
        p.items[blockIdx.x] = {sg.first, sg.R, sg.row0, sg.kvh, sg.pair ? 2 * kTile : kTile,
                               static_cast<int>(owner_of(last, all[0], all[1]) - blockIdx.x + 1), 0};
      }
      // A single tile's O is both pipes' (the same lanes of TMEM), and each writes half
      // of the dims.
      float w0 = 1.0f, w1 = 0.0f;
      if (!sg.pair) {
        pipe_ml[e][r] = make_float2(m, l);
        tc_fence_before();
        pipes_sync();  // both pipes' products are done
        tc_fence_after();
        const float2 x = pipe_ml[0][r], y = pipe_ml[1][r];
        m = fmaxf(x.x, y.x);
        w0 = x.x == -INFINITY ? 0.0f : fast_exp2(x.x - m);
        w1 = y.x == -INFINITY ? 0.0f : fast_exp2(y.x - m);
        l = fmaf(w1, y.y, w0 * x.y);
      }
      const int lo = sg.pair ? 0 : 2 * e, hi = sg.pair ? 4 : lo + 2;
      const uint32_t o0 = (sg.pair ? tm_o[e] : tm_o[0]) + lane_off, o1 = tm_o[1] + lane_off;
      ro.inv = l == 0.0f ? 0.0f : 1.0f / l;
      float nan = l;
#pragma unroll 1
      for (int c = lo; c < hi && !idle; ++c) {
        float v[32];
        tmem_ld32(o0 + c * 32, v);
        tmem_wait_ld();
        if (!sg.pair) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float y[16];
            tmem_ld16(o1 + c * 32 + 16 * h, y);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[16 * h + i] = fmaf(w1, y[i], w0 * v[16 * h + i]);
          }
        }
        if (p.codec[1] != KVQ_F16) {  // (of split values past fp16's range)
#pragma unroll
          for (int i = 0; i < 32; i += 2) nan = fmax3_nan(nan, v[i], v[i + 1]);
        }
        if (rot_v) {  // the stages inside 32 columns
          fwht32(v);
          tmem_st32f(o0 + c * 32, v);
        } else if (valid) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ro.put(c * 32 + 8 * i, reinterpret_cast<const float(&)[8]>(v[8 * i]));
        }
      }
      if (rot_v) {  // the stages across them, and x = s H y / 16
        tmem_wait_st();
        if (!sg.pair) {
          tc_fence_before();
          pipes_sync();
          tc_fence_after();
        }
#pragma unroll 1
        for (int g = lo; g < hi && !idle; ++g) {
          float v[4][8];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld8(o0 + c * 32 + 8 * g, v[c]);
          tmem_wait_ld();
          across32(v, 0.0625f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t signs = turbo_signs(c) >> (8 * g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = (signs >> i) & 1u ? -v[c][i] : v[c][i];
            if (valid) ro.put(c * 32 + 8 * g, v[c]);
          }
        }
      }
      // (fp16 operands hold fp16 queries and keys: a NaN sum of theirs stays)
      if (valid && nan != nan &&
          (l == l || p.codec[0] != KVQ_F16 || p.q_bf16 || far >= kFar))
        any_nan = 1;
      tc_fence_before();  // O read: the next segment's first product may overwrite it
      if (sg.pair) __syncwarp();
      else pipes_sync();
      if (rot_k && have_next) {  // (its way leads through O)
        tc_fence_after();
        load_q(nsg);
        tc_fence_before();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&bars.ofree[e]);
      // Weights were lifted: sums of 2^(s - (m - lift)).  A sum that is no number, where no
      // maximum tells of it, goes with an infinite one, so that no join leaves it out.
      const float ml = l != l ? INFINITY : m == -INFINITY ? m : m - kLift;
      if (valid && (sg.pair || e == 0)) {
        if (!whole)
          reinterpret_cast<float2 *>(slot + kTile * kD)[r] = make_float2(ml, l);
        else if (p.out.xo)
          p.out.xml[at] = make_float2(ml, l);
        else if (p.out.lse)
          p.out.lse[at] = l == 0.0f ? -INFINITY : (ml + log2f(l)) * 0.69314718055994531f;
      }
      sg = nsg;
      have = have_next;
    }
    if (!ok && lane == 0) {
      set_err(p.err, KVQ_DEVERR_TIMEOUT);
      atomicExch(&abort_flag, 1);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (any_nan) nan_rows_in_fp32(p, begin, first_seg, warp, lane);
}

// ------------------------------------------------------------------ joining the pieces

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = kJoinThreads / 16;

// The items that the attention kernel split over several CTAs: o = sum_c
// 2^(m_c - M) o_c over the pieces in order.  Block (c, rows): the item, if any, that
// begins in CTA c's slice and ends in another's; 16 threads per row (8 dims each), a
// warp 16 rows wide, four pieces requested at a time.
__global__ void __launch_bounds__(kJoinThreads, 4)
    cross_join_kernel(const __grid_constant__ CrossParams p) {
  const int tid = threadIdx.x, g8 = tid >> 4;  // dims 8 g8 ..
  grid_dependency_wait();                      // items and partials are complete
  grid_launch_dependents();
  const JoinItem item = p.items[blockIdx.x];
  const int64_t c0 = blockIdx.x;
  const int n = item.n, in = blockIdx.y * kJoinRows + (tid & 15);  // row of the block
  const int R = item.row0 + in;
  if (n == 0 || in >= item.rows || R >= item.R) return;
  const int tok = R / p.G, head = item.kvh * p.G + R - tok * p.G;
  const int64_t row = item.first + tok;
  // the item begins inside its first CTA's slice, and before every other's
  auto part = [&](int j) {
    return p.part + (2 * (c0 + j) + (j == 0 ? 1 : 0)) * p.slot_floats + (in / kTile) * kPartFloats;
  };
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  float M = -INFINITY, L = 0.0f;
  constexpr int kAhead = 4;
  for (int j0 = 0; j0 < n; j0 += kAhead) {
    float4 v[kAhead][2];
    float2 y[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float *pr = part(min(j0 + k, n - 1));
      const int r = in % kTile;
      y[k] = __ldcg(reinterpret_cast<const float2 *>(pr + kTile * kD) + r);
      v[k][0] = __ldcg(reinterpret_cast<const float4 *>(pr) + 2 * g8 * kTile + r);
      v[k][1] = __ldcg(reinterpret_cast<const float4 *>(pr) + (2 * g8 + 1) * kTile + r);
      if (j0 + k >= n) y[k].x = -INFINITY;
    }
    const float top = fmaxf(fmaxf(M, fmaxf(y[0].x, y[1].x)), fmaxf(y[2].x, y[3].x));
    const float f0 = M == -INFINITY ? 0.0f : fast_exp2(M - top);
    L *= f0;
#pragma unroll
    for (int d = 0; d < 8; ++d) acc[d] *= f0;
    M = top;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (y[k].x == -INFINITY) continue;
      const float f = fast_exp2(y[k].x - M);
      L = fmaf(f, y[k].y, L);
      const float z[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                          v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
      for (int d = 0; d < 8; ++d) acc[d] = fmaf(f, z[d], acc[d]);
    }
  }
  const int64_t to = row * p.n_q + head;
  RowOut ro;
  ro.inv = L == 0.0f ? 0.0f : 1.0f / L;
  ro.bf16 = p.q_bf16;
  ro.full = p.out.xo ? p.out.xo + to * kD : nullptr;
  ro.step = 4;
  ro.half = static_cast<uint8_t *>(p.out.out) + row * p.out_row + head * p.out_head;
  ro.put(8 * g8, acc);
  if (g8 == 0) {
    if (p.out.xo) p.out.xml[to] = make_float2(M, L);
    else if (p.out.lse)
      p.out.lse[to] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
  }
}

}  // namespace

// What a call can need: CTAs for the most work that n_rows rows over max_len keys can be
// (cross_ctas of it), and tiles for the most rows that a sequence can have.
CrossPlan plan_cross(const kvq_layer &L, int64_t n_rows, int max_len, int num_sms) {
  CrossPlan pl;
  const int64_t R = n_rows * (L.n_q_heads / L.n_kv_heads);  // per kv head
  pl.tiles = L.codec_k != KVQ_TURBO4 && R > kTile ? 2 : 1;
  // sum ceil(R_s / tile rows) over the sequences with rows
  const int64_t blocks = R / (pl.tiles * kTile) + std::min<int64_t>(L.n_seqs, n_rows);
  const int64_t steps = (max_len + kKeys - 1) / kKeys;
  const int64_t W = L.n_kv_heads * blocks * (steps * (pl.tiles == 2 ? kPair : kSingle) + kItemCost);
  pl.grid = static_cast<int>(std::min<int64_t>(num_sms, std::max<int64_t>(1, W / (4 * kSingle))));
  pl.items_off = 2 * static_cast<int64_t>(pl.grid) * pl.tiles * kPartFloats * 4;
  pl.ws_bytes = pl.items_off + pl.grid * static_cast<int64_t>(sizeof(JoinItem));
  return pl;
}

cudaError_t launch_cross(const kvq_layer &L, const CrossPlan &pl, const kvq_rows &q,
                         int64_t n_rows, const int32_t *n_new, const int32_t *row_start,
                         float scale, const CrossOut &out, int64_t out_row, int64_t out_head,
                         int max_len, void *workspace, cudaStream_t stream) {
  CrossParams p;
  p.cache[0] = static_cast<const uint8_t *>(L.k_cache);
  p.cache[1] = static_cast<const uint8_t *>(L.v_cache);
  p.codec[0] = L.codec_k;
  p.codec[1] = L.codec_v;
  p.q = static_cast<const uint8_t *>(q.data);
  p.q_row = q.row_stride * type_bytes(q.type);
  p.q_head = q.head_stride * type_bytes(q.type);
  p.q_bf16 = q.type == KVQ_T_BF16;
  p.out = out;
  p.out_row = out_row * 2;
  p.out_head = out_head * 2;
  p.part = static_cast<float *>(workspace);
  p.slot_floats = pl.tiles * kPartFloats;
  p.items = reinterpret_cast<JoinItem *>(static_cast<uint8_t *>(workspace) + pl.items_off);
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
  // as many steps of each side as fit, and what is left to the side that it fits
  const int kb = kUnits * unit_bytes(L.codec_k), vb = kUnits * unit_bytes(L.codec_v);
  int n = std::min(kMaxSlots, kRingBytes / (kb + vb)), left = kRingBytes - n * (kb + vb);
  p.slots[0] = p.slots[1] = n;
  for (int side = 1; side >= 0; --side)
    while (p.slots[side] < kMaxSlots && left >= (side ? vb : kb)) {
      ++p.slots[side];
      left -= side ? vb : kb;
    }
  p.singles = L.codec_k == KVQ_TURBO4;
  p.scale_log2 = scale * 1.4426950408889634f;
  static std::atomic<uint64_t> optin{0};
  cudaError_t e = smem_optin(cross_attn_kernel, kSmemBytes, optin);
  if (e != cudaSuccess) return e;
  e = launch_pdl(cross_attn_kernel, dim3(static_cast<unsigned>(pl.grid)), dim3(kThreads), kSmemBytes,
                 stream, p);
  if (e != cudaSuccess || pl.grid < 2) return e;
  // at most this many rows of a block (fewer: short batches need fewer blocks)
  const int64_t rows = std::min<int64_t>(p.singles ? kTile : 2 * kTile, n_rows * p.G);
  return launch_pdl(cross_join_kernel,
                    dim3(static_cast<unsigned>(pl.grid - 1),
                         static_cast<unsigned>((rows + kJoinRows - 1) / kJoinRows)),
                    dim3(kJoinThreads), 0, stream, p);
}

}  // namespace kvq
