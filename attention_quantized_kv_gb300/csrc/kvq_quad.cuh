// kvq_quad.cuh -- rows of a K-side unit held by quads of lanes, in the order
// in which the unit stores them (include/kvq.h): lane 4g + w of a warp holds,
// of row g (or g + 8), the dims 16c + 4w + i as v[c][i] (c < 8, i < 4).  In
// every codec those are the bytes of whole 16-byte pieces at 16 * lane of each
// 512 bytes, so a warp loads and stores a unit as contiguous 512-byte pieces,
// with no exchange between lanes but a block's maximum (two shuffles).  The
// planes of a rotation lie inside a lane too, for the interleaved layout and
// for half layouts whose rot_dim is a multiple of 32; otherwise the partners
// are read from the rows in shared memory.
#pragma once

#include "kvq_encode.cuh"
#include "kvq_rope.cuh"

namespace kvq {
namespace {

// 16 bytes from global to shared memory behind the thread's back, in groups.
__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;\n" ::: "memory");
}
template <int N>  // all but the newest N groups have landed (this thread's)
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void copy_async_wait_all() {
  asm volatile("cp.async.wait_all;\n" ::: "memory");
}

// How a rotation's planes lie: kQuadInterleaved, or N = 1..4 for the planes
// ((c, i), (c + N, i)) of a half layout with rot_dim 32 N.
constexpr int kQuadInterleaved = 0;
constexpr int kQuadAny = -1;        // planes cross lanes
constexpr int kQuadPitch = kD + 4;  // floats from row to row of the copy: four banks apart
constexpr int kQuadBytes = 8 * kQuadPitch * 4;  // a warp's copy: one row per quad

inline int quad_kind(const RopeArgs &p) {
  if (p.layout == KVQ_ROPE_INTERLEAVED) return kQuadInterleaved;
  return p.rot % 32 == 0 ? p.rot / 32 : kQuadAny;
}

// PURE: no magnitude (kv_rope_shift); otherwise no sign.
template <bool PURE>
__device__ __forceinline__ void quad_turn(const RopeArgs &p, float &a, float &b, float co, float si,
                                          float sign) {
  if (PURE) turn(a, b, co, sign * si);
  else turn(a, b, __fmul_rn(co, p.magnitude), __fmul_rn(si, p.magnitude));
}

template <int N, bool PURE>
__device__ __forceinline__ void quad_rotate_half(const RopeArgs &p, const float *row, int w,
                                                 float sign, float (&v)[8][4]) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float4 t = *reinterpret_cast<const float4 *>(row + 2 * (16 * c + 4 * w));
    const float4 u = *reinterpret_cast<const float4 *>(row + 2 * (16 * c + 4 * w) + 4);
    const float co[4] = {t.x, t.z, u.x, u.z}, si[4] = {t.y, t.w, u.y, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      quad_turn<PURE>(p, v[c][i], v[c + N][i], co[i], si[i], sign);
  }
}

// Planes anywhere, by the unrotated row: four(d, o) its values d .. d + 3 (d a
// multiple of 4), one(d) its value d.
template <bool PURE, typename Four, typename One>
__device__ __forceinline__ void quad_rotate_any(const RopeArgs &p, const float *row, int w,
                                                float sign, Four four, One one,
                                                float (&v)[8][4]) {
  const int h = p.rot >> 1;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int d0 = 16 * c + 4 * w;
    if (d0 >= p.rot) continue;
    float o[4], co[4], si[4];
    if ((h & 3) == 0) {  // the four values lie in one half, their partners together
      const int e = d0 < h ? d0 : d0 - h;
      four(d0 < h ? d0 + h : e, o);
      const float4 t = *reinterpret_cast<const float4 *>(row + 2 * e);
      const float4 u = *reinterpret_cast<const float4 *>(row + 2 * e + 4);
      co[0] = t.x; co[1] = t.z; co[2] = u.x; co[3] = u.z;
      si[0] = t.y; si[1] = t.w; si[2] = u.y; si[3] = u.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = d0 + i < p.rot ? d0 + i : 0, e = d < h ? d : d - h;
        const float2 t = *reinterpret_cast<const float2 *>(row + 2 * e);
        o[i] = one(d < h ? d + h : e);
        co[i] = t.x;
        si[i] = t.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float cc = PURE ? co[i] : __fmul_rn(co[i], p.magnitude);
      const float ss = PURE ? sign * si[i] : __fmul_rn(si[i], p.magnitude);
      if (d0 + i < p.rot)
        v[c][i] = __fadd_rn(__fmul_rn(v[c][i], cc), __fmul_rn(o[i], d0 + i < h ? -ss : ss));
    }
  }
}

// The same by a copy of the quad's row in shared memory (all 32 lanes).
template <bool PURE>
__device__ __forceinline__ void quad_rotate_copied(const RopeArgs &p, const float *row, int lane,
                                                   float sign, float *copy, float (&v)[8][4]) {
  const int w = lane & 3;
  float *mine = copy + (lane >> 2) * kQuadPitch;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4 *>(mine + 16 * c + 4 * w) =
        make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
  __syncwarp();
  quad_rotate_any<PURE>(
      p, row, w, sign,
      [&](int d, float(&o)[4]) {
        const float4 x = *reinterpret_cast<const float4 *>(mine + d);
        o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
      },
      [&](int d) { return mine[d]; }, v);
  __syncwarp();  // the copy may be written again
}

// Rotate the quad's row by the table row `row` (kind: quad_kind's, not kQuadAny).
template <bool PURE>
__device__ __forceinline__ void quad_rotate(const RopeArgs &p, int kind, const float *row, int w,
                                            float sign, float (&v)[8][4]) {
  if (kind == 4) quad_rotate_half<4, PURE>(p, row, w, sign, v);
  else if (kind == 3) quad_rotate_half<3, PURE>(p, row, w, sign, v);
  else if (kind == 2) quad_rotate_half<2, PURE>(p, row, w, sign, v);
  else if (kind == 1) quad_rotate_half<1, PURE>(p, row, w, sign, v);
  else {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int d = 16 * c + 4 * w;
      if (d >= p.rot) continue;
      float4 t;
      if ((p.rot & 3) == 0) {
        t = *reinterpret_cast<const float4 *>(row + d);
      } else {  // table rows on 8-byte boundaries; the last plane may stand alone
        const float2 a = *reinterpret_cast<const float2 *>(row + d);
        float2 b = make_float2(0.0f, 0.0f);
        if (d + 2 < p.rot) b = *reinterpret_cast<const float2 *>(row + d + 2);
        t = make_float4(a.x, a.y, b.x, b.y);
      }
      quad_turn<PURE>(p, v[c][0], v[c][1], t.x, t.y, sign);
      if (d + 2 < p.rot) quad_turn<PURE>(p, v[c][2], v[c][3], t.z, t.w, sign);
    }
  }
}

// ------------------------------------------------------------- turbo4 rows

__device__ __forceinline__ void quad_signs(float (&v)[8][4], int w) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t bits = turbo_signs(c >> 1) >> (16 * (c & 1) + 4 * w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((bits >> i) & 1u) v[c][i] = -v[c][i];
  }
}

// Unnormalised Sylvester-order FWHT, stages 1, 2 (i), 4, 8 (lanes), 16, 32, 64
// (c), each output one fp32 addition or subtraction, as fwht128_warp's.
__device__ __forceinline__ void quad_fwht(float (&v)[8][4], int w) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float a0 = __fadd_rn(v[c][0], v[c][1]), a1 = __fsub_rn(v[c][0], v[c][1]);
    const float a2 = __fadd_rn(v[c][2], v[c][3]), a3 = __fsub_rn(v[c][2], v[c][3]);
    v[c][0] = __fadd_rn(a0, a2); v[c][2] = __fsub_rn(a0, a2);
    v[c][1] = __fadd_rn(a1, a3); v[c][3] = __fsub_rn(a1, a3);
  }
#pragma unroll
  for (int m = 1; m < 4; m <<= 1) {
    const bool upper = (w & m) != 0;
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float o = __shfl_xor_sync(0xffffffffu, v[c][i], m);
        v[c][i] = upper ? __fsub_rn(o, v[c][i]) : __fadd_rn(v[c][i], o);
      }
  }
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if ((c & h) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = v[c][i], b = v[c + h][i];
          v[c][i] = __fadd_rn(a, b);
          v[c + h][i] = __fsub_rn(a, b);
        }
      }
}

// ------------------------------------------------------------- codes

// A lane's codes of one row: f16 words 2c, 2c + 1 = v[c]; q8_0 word c = v[c];
// nibble codecs word b = levels v[2b] low, v[2b + 1] high.  scale: of block w
// of the row (turbo4: the row's).
template <int CODEC>
struct QuadCodes {
  static constexpr int N = CODEC == KVQ_F16 ? 16 : CODEC == KVQ_Q8_0 ? 8 : 4;
  uint32_t w[N];
  uint16_t scale;
};

// Token row r's codes (this lane's part of them) from a unit.
template <int CODEC>
__device__ __forceinline__ void quad_load_row(const uint8_t *unit, int r, int w,
                                              QuadCodes<CODEC> &q) {
  const int g = r & 7, rh = r >> 3;
  const uint8_t *u = unit + (4 * g + w) * 16;
  if (CODEC == KVQ_F16) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint4 x = *reinterpret_cast<const uint4 *>(u + (2 * b + rh) * 512);
      q.w[4 * b] = x.x; q.w[4 * b + 1] = x.y; q.w[4 * b + 2] = x.z; q.w[4 * b + 3] = x.w;
    }
    return;
  }
  const uint16_t *sc = reinterpret_cast<const uint16_t *>(unit + unit_scale_offset(CODEC));
  q.scale = CODEC == KVQ_TURBO4 ? sc[2 * g + rh] : sc[8 * g + 4 * rh + w];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (CODEC == KVQ_Q8_0) {
      const uint2 x = *reinterpret_cast<const uint2 *>(u + b * 512 + rh * 8);
      q.w[2 * b] = x.x; q.w[2 * b + 1] = x.y;
    } else {
      q.w[b] = *reinterpret_cast<const uint32_t *>(u + (b >> 1) * 512 + ((b & 1) * 2 + rh) * 4);
    }
  }
}

// And back into a unit.
template <int CODEC>
__device__ __forceinline__ void quad_store_row(uint8_t *unit, int r, int w,
                                               const QuadCodes<CODEC> &q) {
  const int g = r & 7, rh = r >> 3;
  uint8_t *u = unit + (4 * g + w) * 16;
  if (CODEC == KVQ_F16) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *reinterpret_cast<uint4 *>(u + (2 * b + rh) * 512) =
          make_uint4(q.w[4 * b], q.w[4 * b + 1], q.w[4 * b + 2], q.w[4 * b + 3]);
    return;
  }
  uint16_t *sc = reinterpret_cast<uint16_t *>(unit + unit_scale_offset(CODEC));
  if (CODEC != KVQ_TURBO4) sc[8 * g + 4 * rh + w] = q.scale;
  else if (w == 0) sc[2 * g + rh] = q.scale;
  if (CODEC == KVQ_Q8_0) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *reinterpret_cast<uint2 *>(u + b * 512 + rh * 8) = make_uint2(q.w[2 * b], q.w[2 * b + 1]);
  } else {
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *reinterpret_cast<uint32_t *>(u + (b >> 1) * 512 + ((b & 1) * 2 + rh) * 4) = q.w[b];
  }
}

__device__ __forceinline__ float half_bits(uint32_t b) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
}

// The row's values, exact in fp32 (all 32 lanes).
template <int CODEC>
__device__ __forceinline__ void quad_decode(const QuadCodes<CODEC> &q, int w, float (&v)[8][4]) {
  if (CODEC == KVQ_F16) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&q.w[2 * c]));
      const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&q.w[2 * c + 1]));
      v[c][0] = a.x; v[c][1] = a.y; v[c][2] = b.x; v[c][3] = b.y;
    }
    return;
  }
  // An unsigned byte or nibble n in the mantissa of 2^23 is 2^23 + n; taking
  // off 2^23 and the code's offset (q8_0: 128, after flipping the sign bit;
  // nibbles: 8) leaves the code exactly.
  const uint32_t magic = 0x4B000000u;
  const float off = CODEC == KVQ_Q8_0 ? -8388736.0f : -8388616.0f;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float d = half_bits(CODEC == KVQ_TURBO4
                                  ? q.scale
                                  : __shfl_sync(0xffffffffu, static_cast<uint32_t>(q.scale), b, 4));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t x;  // four bytes: the codes of v[2b + h]
      if (CODEC == KVQ_Q8_0) x = q.w[2 * b + h] ^ 0x80808080u;
      else x = (h ? q.w[b] >> 4 : q.w[b]) & 0x0f0f0f0fu;
      float *y = v[2 * b + h];
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float2 n = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(x, magic, 0x7440 + i)),
                                                __uint_as_float(__byte_perm(x, magic, 0x7441 + i))),
                                    make_float2(off, off));
        const float2 z = __fmul2_rn(n, make_float2(d, d));
        y[i] = z.x;
        y[i + 1] = z.y;
      }
    }
  }
  if (CODEC == KVQ_TURBO4) {
    quad_fwht(v, w);
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] *= 0.0625f;
    quad_signs(v, w);
  }
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// The codes of 8 values value by value: where rq_codes_fast's distance says
// that one lies too near a rounding boundary (of random values one group of
// eight in 2^10 for q8_0, in 2^13 for 4 bits).  A call, so that its length stays out of the callers.
template <int DC>
__device__ __noinline__ uint2 codes8_exact(float x0, float x1, float x2, float x3, float x4,
                                           float x5, float x6, float x7, float d, float rcp) {
  const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
  uint32_t k[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    k[i] = static_cast<uint32_t>(DC == KVQ_Q8_0 ? q8_from_quotient(x[i], d, rcp)
                                                : q4_from_quotient(x[i], d, rcp));
  return make_uint2(low_bytes4(k[0], k[1], k[2], k[3]), low_bytes4(k[4], k[5], k[6], k[7]));
}

// The codes of 8 values of one block by its scale, as two words of bytes;
// levels of the nibble codecs not yet clamped.  live: they are stored (what a
// place without a row holds is often NaN, and not worth the divisions).
template <int DC>
__device__ __forceinline__ uint2 quad_codes8(const float (&x)[8], float d, float rcp, bool live) {
  uint32_t k[8];
  float far = 0.0f;
  rq_codes_fast<DC>(x, rcp, k, far);
  uint2 c = make_uint2(low_bytes4(k[0], k[1], k[2], k[3]), low_bytes4(k[4], k[5], k[6], k[7]));
  if (d == 0.0f) c = DC == KVQ_Q8_0 ? make_uint2(0u, 0u) : make_uint2(0x08080808u, 0x08080808u);
  else if (live && !codes_exact<DC>(far))
    c = codes8_exact<DC>(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], d, rcp);
  return c;
}

// The scale's numerator for the 4-bit rule over the values of N planes groups
// of the quad: the signed value of largest magnitude, the lowest dim on ties,
// 0 where all are NaN (all 32 lanes; c0 .. c0 + N - 1).
template <int N>
__device__ __forceinline__ float quad_signed_max(const float (&v)[8][4], int c0, int w) {
  float hi = -INFINITY, lo = INFINITY;
#pragma unroll
  for (int c = 0; c < N; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi = fmaxf(hi, v[c0 + c][i]);
      lo = fminf(lo, v[c0 + c][i]);
    }
  hi = quad_max(hi);
  lo = -quad_max(-lo);
  const bool tie = hi == -lo;
  if (__any_sync(0xffffffffu, tie)) {  // the first of the dims that hold +-hi
    int best = 1 << 20;
#pragma unroll
    for (int c = N - 1; c >= 0; --c)
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const float x = v[c0 + c][i];
        if (fabsf(x) == hi) best = (16 * c + 4 * w + i) * 2 + (__float_as_uint(x) >> 31);
      }
    best = min(best, __shfl_xor_sync(0xffffffffu, best, 1));
    best = min(best, __shfl_xor_sync(0xffffffffu, best, 2));
    if (tie) {  // (+-0 keeps its sign; no dim at all: only NaN)
      const float size = best == 1 << 20 ? 0.0f : fabsf(hi);
      return (best & 1) ? -size : size;
    }
  }
  return hi > -lo ? hi : lo;
}

// Encode the quad's row (all 32 lanes; live: its codes are stored).
template <int CODEC>
__device__ __forceinline__ void quad_encode(float (&v)[8][4], int w, bool live,
                                            QuadCodes<CODEC> &q) {
  if (CODEC == KVQ_F16) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      q.w[2 * c] = pack_half2(v[c][0], v[c][1]);
      q.w[2 * c + 1] = pack_half2(v[c][2], v[c][3]);
    }
    return;
  }
  if (CODEC == KVQ_TURBO4) {
    quad_signs(v, w);
    quad_fwht(v, w);
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] *= 0.125f;
  }
  // Lane w takes block w's division (turbo4: all the row's), the quad shares it.
  float num[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (CODEC == KVQ_Q8_0) {
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) a = fmaxf(a, fmaxf(fabsf(v[2 * b][i]), fabsf(v[2 * b + 1][i])));
      num[b] = quad_max(a);
    } else {
      num[b] = CODEC == KVQ_Q4_0 ? quad_signed_max<2>(v, 2 * b, w)
               : b == 0          ? quad_signed_max<8>(v, 0, w)
                                 : num[0];
    }
  }
  const float mine = w == 0 ? num[0] : w == 1 ? num[1] : w == 2 ? num[2] : num[3];
  const float dw = CODEC == KVQ_Q8_0 ? __fdiv_rn(mine, 127.0f) : __fdiv_rn(mine, -8.0f);
  const float rw = dw != 0.0f ? __frcp_rn(dw) : 0.0f;
  q.scale = __half_as_ushort(__float2half_rn(dw));
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float d = __shfl_sync(0xffffffffu, dw, b, 4), rcp = __shfl_sync(0xffffffffu, rw, b, 4);
    const float x[8] = {v[2 * b][0],     v[2 * b][1],     v[2 * b][2],     v[2 * b][3],
                        v[2 * b + 1][0], v[2 * b + 1][1], v[2 * b + 1][2], v[2 * b + 1][3]};
    const uint2 k = quad_codes8<CODEC == KVQ_Q8_0 ? KVQ_Q8_0 : KVQ_Q4_0>(x, d, rcp, live);
    if (CODEC == KVQ_Q8_0) {
      q.w[2 * b] = k.x;
      q.w[2 * b + 1] = k.y;
    } else {
      q.w[b] = clamp15x4(k.x) | (clamp15x4(k.y) << 4);
    }
  }
}

}  // namespace
}  // namespace kvq
