// kvq_encode.cuh -- the row encoders of the cache codecs (device code shared
// by the append, re-encode and fused decode-step kernels).
//
// Block codecs of the "Codecs" table of the buun-llama-cpp listing (q8_0 8.5
// and q4_0 4.5 bits per value, 32-value blocks with an fp16 scale) and the
// rotated turbo4 rows, with the fp32 encoder formulas of include/kvq.h,
// evaluated with explicit IEEE round-to-nearest operations so that the bytes
// are reproducible bit for bit.  One warp encodes one 128-value row: lane l
// holds dims 4l..4l+3.  A NaN is left out of a block's maximum and takes the
// code of 0, as an infinity's quotient by the infinite scale does.
#pragma once

#include <cuda_runtime.h>

#include "kvq_device.cuh"

namespace kvq {
namespace {

// The integers the encoders take from the quotients x/d, without a division
// or a float-to-int conversion per value.  t = RN(x * RN(1/d)) lies within
// |x/d| * 3 * 2^-24 of RN(x/d) (two roundings of relative size 2^-24).
// Where t is far enough from the boundary at which the encoder's integer
// changes, t gives the same integer as RN(x/d) (tests below); elsewhere the
// encoder divides exactly.  Integers come from the 1.5 * 2^23 addition: for
// |y| < 2^22, RN(y + 1.5 * 2^23) holds RN-to-nearest-integer(y) in its low
// mantissa bits.  The bytes are those of the exact division.
constexpr float kRoundMagic = 12582912.0f;  // 1.5 * 2^23
constexpr int kRoundMagicBits = 0x4B400000;

// q8_0: q = round-half-away(RN(x/d)) with |x/d| <= 127 (1 + 2^-23), so
// |t - RN(x/d)| < 2^-15.4.  t more than 2^-14 away from every half-integer
// rounds the same way, and there round-half-away equals round-to-nearest.
__device__ __forceinline__ int q8_from_quotient(float x, float d, float rcp) {
  const float t = __fmul_rn(x, rcp);
  const float tm = __fadd_rn(t, kRoundMagic);
  const float dist = fabsf(__fsub_rn(t, __fsub_rn(tm, kRoundMagic)));  // to the nearest integer
  if (fabsf(__fsub_rn(dist, 0.5f)) > 0x1p-14f) return __float_as_int(tm) - kRoundMagicBits;
  return __float2int_rz(roundf(__fdiv_rn(x, d)));  // (NaN: 0)
}

// The 4-bit rule by its division (rare; a call, as its length inline cost the
// callers more: 2048 appended rows of 8 heads into q4_0 13.9 instead of 15.0 us
// with the ties below).  A NaN gives 8.  u >= 0.5 but for the last steps of
// fp32, where d is a rounded m / -8: a negative integer keeps its lowest 4 bits.
__device__ __noinline__ int q4_exact(float x, float d) {
  const float t = __fdiv_rn(x, d);
  return t != t ? 8 : min(__float2int_rz(__fadd_rn(t, 8.5f)), 15) & 15;
}

// q4_0 and turbo4: q = min(15, trunc(RN(RN(x/d) + 8.5))) with |x/d| <= 8 (1 +
// 2^-23): u = RN(t + 8.5) lies within 2^-18.5 of the exact path's value, so
// u more than 2^-17 away from every integer truncates the same way
// (floor(u) = the integer nearest to u - 0.5, which is exact there).
__device__ __forceinline__ int q4_from_quotient(float x, float d, float rcp) {
  const float u = __fadd_rn(__fmul_rn(x, rcp), 8.5f);
  const float fm = __fadd_rn(__fsub_rn(u, 0.5f), kRoundMagic);
  const float fr = __fsub_rn(u, __fsub_rn(fm, kRoundMagic));  // u - floor(u)
  return fr > 0x1p-17f && fr < 1.0f - 0x1p-17f ? min(__float_as_int(fm) - kRoundMagicBits, 15)
                                               : q4_exact(x, d);
}

// The largest magnitude of three values, NaN if one of them is (fmaxf leaves
// NaN out).
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Bytes 0 of a, b, c, d as one word (a in the lowest byte).
__device__ __forceinline__ uint32_t low_bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// Four byte lanes holding 0..16, each clamped to 15 (16 - (16 >> 4)).
__device__ __forceinline__ uint32_t clamp15x4(uint32_t w) { return w - ((w >> 4) & 0x01010101u); }

// The quotient path of q8_from_quotient / q4_from_quotient on one chunk, two
// values per instruction: k[v] gets the fast path's code (its lowest byte;
// q4_0: the level before the clamp), and far collects the chunk's largest
// distance of t (q4_0: of u - 0.5) from the integer next to it, which says
// whether the fast path is the exact one for every value.  Where 1/d is
// infinite (d below 2^-128) the quotients are infinities or NaN and so is
// their distance: far keeps a NaN, and codes_exact refuses it.
template <int DC>
__device__ __forceinline__ void rq_codes_fast(const float (&x)[8], float rcp, uint32_t (&k)[8],
                                              float &far) {
  const float2 r2 = make_float2(rcp, rcp), m2 = make_float2(kRoundMagic, kRoundMagic);
  const float2 nm2 = make_float2(-kRoundMagic, -kRoundMagic), n1 = make_float2(-1.0f, -1.0f);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float2 t = __fmul2_rn(make_float2(x[j], x[j + 1]), r2);
    if (DC != KVQ_Q8_0)  // floor(u) = the integer next to u - 0.5
      t = __fadd2_rn(__fadd2_rn(t, make_float2(8.5f, 8.5f)), make_float2(-0.5f, -0.5f));
    const float2 tm = __fadd2_rn(t, m2);
    const float2 fr = __ffma2_rn(__fadd2_rn(tm, nm2), n1, t);  // t - round(t)
    far = max3_abs_nan(far, fr.x, fr.y);
    k[j] = __float_as_uint(tm.x);
    k[j + 1] = __float_as_uint(tm.y);
  }
}

// Whether the codes that rq_codes_fast gave a block (far over all its chunks)
// are the exact path's.
template <int DC>
__device__ __forceinline__ bool codes_exact(float far) {
  return far < 0.5f - (DC == KVQ_Q8_0 ? 0x1p-14f : 0x1p-17f);
}

// q8_0: amax over the 8 lanes of the block, d = amax/127, q = round(x/d).
__device__ __forceinline__ void encode_q8(const float (&x)[4], int (&q)[4], __half &d16) {
  float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
  a = fmaxf(a, 0.0f);  // (four NaN)
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  const float d = __fdiv_rn(a, 127.0f);
  d16 = __float2half_rn(d);
  const float rcp = d != 0.0f ? __frcp_rn(d) : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = d != 0.0f ? q8_from_quotient(x[i], d, rcp) : 0;
}

// The first of the dims of LANES lanes that hold +-hi, times 2, plus its sign
// (all 32 lanes; 2^20: none).  A call: ties are rare.
template <int LANES>
__device__ __noinline__ int first_of(float x0, float x1, float x2, float x3, float hi, int lane) {
  const float x[4] = {x0, x1, x2, x3};
  int best = 1 << 20;
#pragma unroll
  for (int i = 3; i >= 0; --i)
    if (fabsf(x[i]) == hi) best = (4 * lane + i) * 2 + (__float_as_uint(x[i]) >> 31);
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
  return best;
}

// The signed value of largest magnitude of the rows' groups of LANES lanes,
// the lowest dim on ties, 0 where all are NaN (all 32 lanes).
template <int LANES>
__device__ __forceinline__ float lanes_signed_max(const float (&x)[4], int lane) {
  float hi = -INFINITY, lo = INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi = fmaxf(hi, x[i]);
    lo = fminf(lo, x[i]);
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  const bool tie = hi == -lo;
  if (__any_sync(0xffffffffu, tie)) {
    const int best = first_of<LANES>(x[0], x[1], x[2], x[3], hi, lane);
    if (tie) {  // (+-0 keeps its sign; no dim at all: only NaN)
      const float size = best == 1 << 20 ? 0.0f : fabsf(hi);
      return (best & 1) ? -size : size;
    }
  }
  return hi > -lo ? hi : lo;
}

// q4_0: m = the block's signed value of largest magnitude, d = m/-8,
// q = min(15, trunc(x/d + 8.5)).
__device__ __forceinline__ void encode_q4(const float (&x)[4], int lane, int (&q)[4], __half &d16) {
  const float m = lanes_signed_max<8>(x, lane);
  const float d = __fdiv_rn(m, -8.0f);
  d16 = __float2half_rn(d);
  const float rcp = d != 0.0f ? __frcp_rn(d) : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = d != 0.0f ? q4_from_quotient(x[i], d, rcp) : 8;
}

// turbo4: signs, FWHT and the factor 1/8 (the rotation of the row, exact
// order of the definition), then the q4_0 rule over all 128 rotated values
// (32 lanes, lowest dim wins ties).
__device__ __forceinline__ void encode_turbo4(const float (&x)[4], int lane, int (&q)[4],
                                              __half &d16) {
  float y[4] = {x[0], x[1], x[2], x[3]};
  turbo_flip_lane(y, lane);
  fwht128_warp(y, lane);
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] *= 0.125f;
  const float m = lanes_signed_max<32>(y, lane);
  const float d = __fdiv_rn(m, -8.0f);
  d16 = __float2half_rn(d);
  const float rcp = d != 0.0f ? __frcp_rn(d) : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = d != 0.0f ? q4_from_quotient(y[i], d, rcp) : 8;
}

__device__ __forceinline__ void st_u16(uint8_t *p, uint32_t v) {
  *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(v);
}

// Write one row (token row r of `unit`) from lane-held data.
template <int SIDE>
__device__ __forceinline__ void store_row(int codec, uint8_t *unit, int r, int lane,
                                          const uint2 raw, const int (&q)[4], __half d16) {
  const int g = r & 7, rh = r >> 3, tig = (r & 7) >> 1, par = r & 1;
  const int b = lane >> 3, lb = lane & 7;  // block and lane-in-block
  if (codec == KVQ_F16) {
    if (SIDE == 0) {
      const int h = (lane >> 2) & 1, w = lane & 3;
      *reinterpret_cast<uint2 *>(unit + (2 * b + rh) * 512 + (4 * g + w) * 16 + h * 8) = raw;
    } else {
      const uint16_t v[4] = {static_cast<uint16_t>(raw.x), static_cast<uint16_t>(raw.x >> 16),
                             static_cast<uint16_t>(raw.y), static_cast<uint16_t>(raw.y >> 16)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 4 * lane + i, mt = d >> 4, gq = (d & 15) >> 1, s = d & 1;
        *reinterpret_cast<uint16_t *>(unit + mt * 512 + (4 * gq + tig) * 16 +
                                      (rh * 4 + s * 2 + par) * 2) = v[i];
      }
    }
    return;
  }
  const uint16_t dbits = __half_as_ushort(d16);
  if (codec == KVQ_Q8_0) {
    if (SIDE == 0) {
      const uint32_t word = (q[0] & 0xff) | ((q[1] & 0xff) << 8) | ((q[2] & 0xff) << 16) |
                            (static_cast<uint32_t>(q[3] & 0xff) << 24);
      const int h = lb >> 2, w = lane & 3;
      *reinterpret_cast<uint32_t *>(unit + b * 512 + (4 * g + w) * 16 + (2 * rh + h) * 4) = word;
      if (lb == 0) st_u16(unit + 2048 + g * 16 + rh * 8 + b * 2, dbits);
    } else {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int d = 4 * lane + 2 * p, mt = d >> 4, gq = (d & 15) >> 1;
        st_u16(unit + (mt >> 1) * 512 + (4 * gq + tig) * 16 + ((mt & 1) * 2 + rh) * 4 + par * 2,
               (q[2 * p] & 0xff) | ((q[2 * p + 1] & 0xff) << 8));
      }
      if (lb == 0) st_u16(unit + 2048 + tig * 32 + b * 8 + rh * 4 + par * 2, dbits);
    }
    return;
  }
  // q4_0 and turbo4: canonical byte jc of block (group) b = q[jc] | q[jc+16]
  // << 4; lanes lb<4 hold jc = 4lb..4lb+3 and fetch the high nibbles from
  // lane lb+4 of the same block.
  int hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) hi[i] = __shfl_down_sync(0xffffffffu, q[i], 4);
  if (lb < 4) {
    uint32_t bytes[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bytes[i] = (q[i] & 0xf) | ((hi[i] & 0xf) << 4);
    if (SIDE == 0) {
      const uint32_t word = bytes[0] | (bytes[1] << 8) | (bytes[2] << 16) | (bytes[3] << 24);
      *reinterpret_cast<uint32_t *>(unit + (b >> 1) * 512 + (4 * g + lb) * 16 +
                                    ((b & 1) * 2 + rh) * 4) = word;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int jc = 4 * lb + i, mt = 2 * b + (jc >> 3), gq = jc & 7;
        unit[(mt >> 2) * 512 + (4 * gq + tig) * 16 + (mt & 3) * 4 + par * 2 + rh] =
            static_cast<uint8_t>(bytes[i]);
      }
    }
  }
  if (codec == KVQ_TURBO4) {  // one scale per row
    if (lane == 0)
      st_u16(unit + (SIDE == 0 ? 1024 + g * 4 + rh * 2 : 1024 + tig * 8 + rh * 4 + par * 2),
             dbits);
    return;
  }
  if (lb == 0) {
    const int off = SIDE == 0 ? 1024 + g * 16 + rh * 8 + b * 2
                              : 1024 + tig * 32 + b * 8 + rh * 4 + par * 2;
    st_u16(unit + off, dbits);
  }
}

// Encode one fp32 row (lane l holds its dims 4l..4l+3) with `codec` into token
// row r of `unit` (all 32 lanes of the warp); an f16 target rounds to fp16.
template <int SIDE>
__device__ __forceinline__ void encode_f32_row_into(int codec, const float (&x)[4], uint8_t *unit,
                                                    int r, int lane) {
  int q[4] = {0, 0, 0, 0};
  __half d16 = __float2half_rn(0.0f);
  uint2 raw = make_uint2(0u, 0u);
  if (codec == KVQ_Q8_0) encode_q8(x, q, d16);
  else if (codec == KVQ_Q4_0) encode_q4(x, lane, q, d16);
  else if (codec == KVQ_TURBO4) encode_turbo4(x, lane, q, d16);
  else raw = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
  store_row<SIDE>(codec, unit, r, lane, raw, q, d16);
}

// Encode one fp16 row (lane l holds its dims 4l..4l+3 in `raw`) with
// `codec` into token row r of `unit` (all 32 lanes of the warp).
template <int SIDE>
__device__ __forceinline__ void encode_row_into(int codec, const uint2 raw, uint8_t *unit, int r,
                                                int lane) {
  float x[4];
  {
    const __half2 h01 = *reinterpret_cast<const __half2 *>(&raw.x);
    const __half2 h23 = *reinterpret_cast<const __half2 *>(&raw.y);
    x[0] = __low2float(h01); x[1] = __high2float(h01);
    x[2] = __low2float(h23); x[3] = __high2float(h23);
  }
  int q[4] = {0, 0, 0, 0};
  __half d16 = __float2half_rn(0.0f);
  if (codec == KVQ_Q8_0) encode_q8(x, q, d16);
  else if (codec == KVQ_Q4_0) encode_q4(x, lane, q, d16);
  else if (codec == KVQ_TURBO4) encode_turbo4(x, lane, q, d16);
  store_row<SIDE>(codec, unit, r, lane, raw, q, d16);
}

}  // namespace
}  // namespace kvq
