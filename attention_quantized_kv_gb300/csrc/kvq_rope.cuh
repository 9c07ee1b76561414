// kvq_rope.cuh -- the rotation of 128-value rows held by a warp, four values
// per lane (lane l: dims 4l .. 4l + 3, the encoders' order).
//
// y_a = RN(RN(x_a c) - RN(x_b s)), y_b = RN(RN(x_a s) + RN(x_b c)) for the
// planes (a, b) of include/kvq.h.  With s' = -s for element a and +s for
// element b both are RN(RN(x c) + RN(partner s')): negation and the order of
// an addition do not change a rounding.  __fmul_rn / __fadd_rn keep the
// compiler from contracting the sum, so a row's bits do not depend on where
// it is rotated.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kvq_device.cuh"

namespace kvq {

// (a, b) -> (a c - b s, a s + b c), every operation rounded.  (The packed pair
// __fmul2_rn, __fadd2_rn would be shorter, but the compiler contracts it: of
// 8M random sums 46% came out as a fused multiply-add's.)
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
  const float x = __fadd_rn(__fmul_rn(a, c), __fmul_rn(b, -s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// What a kernel needs of kvq_rope.
struct RopeArgs {
  const float *table;
  int n_pos, rot, layout;
  float magnitude;
};

inline RopeArgs rope_args(const kvq_rope &r) {
  return RopeArgs{r.table, r.n_pos, r.rot_dim, r.layout, r.magnitude};
}

// The table row of a position; one outside the table sets KVQ_DEVERR_POS and
// takes the nearest row.
__device__ __forceinline__ const float *rope_row(const RopeArgs &p, int64_t pos, int32_t *err) {
  if (pos < 0 || pos >= p.n_pos) {
    set_err(err, KVQ_DEVERR_POS);
    pos = pos < 0 ? 0 : p.n_pos - 1;
  }
  return p.table + pos * p.rot;  // rot / 2 pairs of floats
}

// A lane's angles: y[i] = x[i] c[i] + partner s[i] for the elements below rot.
struct LaneAngles {
  float c[4], s[4];
};

// sign = -1: the transposed rotation.
__device__ __forceinline__ LaneAngles lane_angles(const RopeArgs &p, const float *row, int lane,
                                                  float sign = 1.0f) {
  LaneAngles a;
  const int h = p.rot >> 1, d0 = 4 * lane;
  float co[4], si[4];
  bool lower[4];
  if (p.layout == KVQ_ROPE_INTERLEAVED) {
    float4 t = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
    if ((p.rot & 3) == 0) {  // rows of the table are 16-byte aligned
      if (d0 < p.rot) t = *reinterpret_cast<const float4 *>(row + d0);
    } else {
      if (d0 < p.rot) {
        const float2 u = *reinterpret_cast<const float2 *>(row + d0);
        t.x = u.x; t.y = u.y;
      }
      if (d0 + 2 < p.rot) {
        const float2 u = *reinterpret_cast<const float2 *>(row + d0 + 2);
        t.z = u.x; t.w = u.y;
      }
    }
    co[0] = co[1] = t.x; si[0] = si[1] = t.y;
    co[2] = co[3] = t.z; si[2] = si[3] = t.w;
    lower[0] = lower[2] = true;
    lower[1] = lower[3] = false;
  } else if ((h & 3) == 0) {  // a lane's four elements lie in one half
    const int e = d0 < h ? d0 : d0 - h;
    float4 t = make_float4(1.0f, 0.0f, 1.0f, 0.0f), u = t;
    if (d0 < p.rot) {
      t = *reinterpret_cast<const float4 *>(row + 2 * e);
      u = *reinterpret_cast<const float4 *>(row + 2 * e + 4);
    }
    co[0] = t.x; si[0] = t.y; co[1] = t.z; si[1] = t.w;
    co[2] = u.x; si[2] = u.y; co[3] = u.z; si[3] = u.w;
    lower[0] = lower[1] = lower[2] = lower[3] = d0 < h;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = d0 + i, e = d < h ? d : d - h;
      float2 t = make_float2(1.0f, 0.0f);
      if (d < p.rot) t = *reinterpret_cast<const float2 *>(row + 2 * e);
      co[i] = t.x; si[i] = t.y;
      lower[i] = d < h;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a.c[i] = __fmul_rn(co[i], p.magnitude);
    const float s = sign * __fmul_rn(si[i], p.magnitude);
    a.s[i] = lower[i] ? -s : s;
  }
  return a;
}

// How a row's partners lie, a kernel's uniform branch outside its loop over
// rows: in the lane, in another lane's same element, or anywhere.
enum class Lanes { kInterleaved, kHalf, kAny };

// Rotate the row that the warp holds (all 32 lanes).
template <Lanes L>
__device__ __forceinline__ void rotate_lane(const RopeArgs &p, const LaneAngles &a, int lane,
                                            float (&x)[4]) {
  const int h = p.rot >> 1, d0 = 4 * lane;
  float o[4];  // the partners
  if (L == Lanes::kInterleaved) {
    o[0] = x[1]; o[1] = x[0]; o[2] = x[3]; o[3] = x[2];
  } else if (L == Lanes::kHalf) {
    const int src = d0 < h ? lane + (h >> 2) : lane - (h >> 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], src & 31);
  } else {  // the partner of a lane's element may be any element of any lane
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = d0 + i, e = (d < h ? d + h : d - h) & (kD - 1);
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = __shfl_sync(0xffffffffu, x[k], e >> 2);
        if ((e & 3) == k) t = v;
      }
      o[i] = t;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (d0 + i < p.rot) x[i] = __fadd_rn(__fmul_rn(x[i], a.c[i]), __fmul_rn(o[i], a.s[i]));
}

// f(the rope's Lanes as a constant).
template <typename F>
__device__ __forceinline__ void with_lanes(const RopeArgs &p, F f) {
  if (p.layout == KVQ_ROPE_INTERLEAVED) f(std::integral_constant<Lanes, Lanes::kInterleaved>());
  else if ((p.rot & 7) == 0) f(std::integral_constant<Lanes, Lanes::kHalf>());
  else f(std::integral_constant<Lanes, Lanes::kAny>());
}

__device__ __forceinline__ void rotate_lane(const RopeArgs &p, const LaneAngles &a, int lane,
                                            float (&x)[4]) {
  with_lanes(p, [&](auto lanes) { rotate_lane<decltype(lanes)::value>(p, a, lane, x); });
}

// ------------------------------------------------------------- row types
// (raw4: four consecutive values as they lie in memory)

template <int T>
struct RowType;
template <>
struct RowType<KVQ_T_F16> { using type = __half; using raw4 = uint2; };
template <>
struct RowType<KVQ_T_BF16> { using type = __nv_bfloat16; using raw4 = uint2; };
template <>
struct RowType<KVQ_T_F32> { using type = float; using raw4 = float4; };

// Four consecutive values as fp32 (p aligned to their size).
template <int T>
__device__ __forceinline__ void load4(const void *p, float (&x)[4]) {
  if (T == KVQ_T_F32) {
    const float4 v = *static_cast<const float4 *>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const uint2 v = *static_cast<const uint2 *>(p);
    if (T == KVQ_T_F16) {
      const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
      const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
      x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    } else {  // bf16: the upper half of an fp32
      x[0] = __uint_as_float(v.x << 16);
      x[1] = __uint_as_float(v.x & 0xffff0000u);
      x[2] = __uint_as_float(v.y << 16);
      x[3] = __uint_as_float(v.y & 0xffff0000u);
    }
  }
}

// One value as fp32.
template <int T>
__device__ __forceinline__ float load1(const void *p) {
  if (T == KVQ_T_F32) return *static_cast<const float *>(p);
  const uint16_t v = *static_cast<const uint16_t *>(p);
  return T == KVQ_T_F16 ? __half2float(__ushort_as_half(v))
                        : __uint_as_float(static_cast<uint32_t>(v) << 16);
}
// Four consecutive values, rounded once to the type.
template <int T>
__device__ __forceinline__ void store4(void *p, const float (&x)[4]) {
  if (T == KVQ_T_F32) {
    *static_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else if (T == KVQ_T_F16) {
    *static_cast<uint2 *>(p) = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *static_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                          *reinterpret_cast<const uint32_t *>(&b));
  }
}

// ------------------------------------------------------------- eight lanes per row
//
// Where the planes allow it a row is held by eight lanes, 16 values each: for
// a half layout lane l takes dims 8l .. and rot/2 + 8l .., both elements of its
// planes, so nothing crosses lanes, loads and stores are 16 bytes and a warp
// moves four heads at once (lanes behind the planes take what passes
// through).  An interleaved layout takes dims 8l .. and 64 + 8l ..

__host__ __device__ inline bool eight_lanes(const RopeArgs &p) {
  return p.layout == KVQ_ROPE_INTERLEAVED ? p.rot % 8 == 0 : p.rot % 16 == 0;
}

struct EightLanes {
  int a, b;           // first dims of the lane's two groups of eight
  bool turn_a, turn_b;  // whether they are rotated (half layouts: together)
};

__device__ __forceinline__ EightLanes eight_lanes_of(const RopeArgs &p, int l) {
  EightLanes m;
  const int h = p.rot >> 1;
  if (p.layout == KVQ_ROPE_INTERLEAVED) {
    m.a = 8 * l;
    m.b = 64 + 8 * l;
    m.turn_a = m.a < p.rot;
    m.turn_b = m.b < p.rot;
  } else {
    m.turn_a = m.turn_b = 8 * l < h;
    m.a = m.turn_a ? 8 * l : p.rot + 16 * (l - (h >> 3));
    m.b = m.turn_a ? h + 8 * l : m.a + 8;
  }
  return m;
}

struct EightAngles {
  float c[8], s[8];
};

__device__ __forceinline__ EightAngles eight_angles(const RopeArgs &p, const EightLanes &m,
                                                    const float *row, int l, float sign = 1.0f) {
  EightAngles a;
  const bool inter = p.layout == KVQ_ROPE_INTERLEAVED;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // half: entries 8l + 2i, + 1; interleaved: 4l + .. of group a, 32 + 4l + .. of b
    const int at = !inter ? 16 * l + 4 * i : i < 2 ? 8 * l + 4 * i : 64 + 8 * l + 4 * (i - 2);
    float4 t = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
    if (inter && i >= 2 ? m.turn_b : m.turn_a) t = *reinterpret_cast<const float4 *>(row + at);
    a.c[2 * i] = __fmul_rn(t.x, p.magnitude);
    a.s[2 * i] = sign * __fmul_rn(t.y, p.magnitude);
    a.c[2 * i + 1] = __fmul_rn(t.z, p.magnitude);
    a.s[2 * i + 1] = sign * __fmul_rn(t.w, p.magnitude);
  }
  return a;
}

// Rotate the lane's groups xa, xb.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate_eight(const EightLanes &m, const EightAngles &g,
                                             float (&xa)[8], float (&xb)[8]) {
  if (INTERLEAVED) {
    if (m.turn_a) {
#pragma unroll
      for (int k = 0; k < 4; ++k) turn(xa[2 * k], xa[2 * k + 1], g.c[k], g.s[k]);
    }
    if (m.turn_b) {
#pragma unroll
      for (int k = 0; k < 4; ++k) turn(xb[2 * k], xb[2 * k + 1], g.c[4 + k], g.s[4 + k]);
    }
  } else if (m.turn_a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(xa[i], xb[i], g.c[i], g.s[i]);
  }
}

// Eight consecutive values as they lie in memory, as fp32, and back.
template <int T>
struct Eight {
  uint4 w[T == KVQ_T_F32 ? 2 : 1];
};
template <int T>
__device__ __forceinline__ Eight<T> load_eight(const uint8_t *p) {
  Eight<T> r;
  r.w[0] = *reinterpret_cast<const uint4 *>(p);
  if (T == KVQ_T_F32) r.w[T == KVQ_T_F32] = *reinterpret_cast<const uint4 *>(p + 16);
  return r;
}
template <int T>
__device__ __forceinline__ void eight_values(const Eight<T> &r, float (&x)[8]) {
  constexpr int kSecond = T == KVQ_T_F32 ? 1 : 0;
  float lo[4], hi[4];
  load4<T>(&r.w[0], lo);
  load4<T>(T == KVQ_T_F32 ? reinterpret_cast<const uint2 *>(&r.w[kSecond])
                          : reinterpret_cast<const uint2 *>(&r.w[0]) + 1,
           hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = lo[i];
    x[4 + i] = hi[i];
  }
}
template <int T>
__device__ __forceinline__ void store_eight(uint8_t *p, const float (&x)[8]) {
  const float lo[4] = {x[0], x[1], x[2], x[3]}, hi[4] = {x[4], x[5], x[6], x[7]};
  uint4 w[T == KVQ_T_F32 ? 2 : 1];
  if (T == KVQ_T_F32) {
    store4<T>(&w[0], lo);
    store4<T>(&w[T == KVQ_T_F32], hi);
    reinterpret_cast<uint4 *>(p)[1] = w[T == KVQ_T_F32];
  } else {
    store4<T>(&w[0], lo);
    store4<T>(reinterpret_cast<uint2 *>(&w[0]) + 1, hi);
  }
  *reinterpret_cast<uint4 *>(p) = w[0];
}

// Heads of one row by one warp, four at a time: x + h * x_head to
// y + h * y_head for h < nh <= 4 * N, all of them requested before the angles.
template <int TI, int TO, int N, typename Row>
__device__ __forceinline__ void rotate_heads_eight(const RopeArgs &p, const uint8_t *x,
                                                   int64_t x_head, uint8_t *y, int64_t y_head,
                                                   int nh, float sign, int lane, Row table_row) {
  constexpr int SI = TI == KVQ_T_F32 ? 4 : 2, SO = TO == KVQ_T_F32 ? 4 : 2;
  const int l = lane & 7, sub = lane >> 3;
  const EightLanes m = eight_lanes_of(p, l);
  Eight<TI> ra[N], rb[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int h = 4 * k + sub;
    if (h < nh) {
      ra[k] = load_eight<TI>(x + h * x_head + m.a * SI);
      rb[k] = load_eight<TI>(x + h * x_head + m.b * SI);
    }
  }
  const float *row = table_row();
  if (!row) return;
  const EightAngles g = eight_angles(p, m, row, l, sign);
  auto all = [&](auto interleaved) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int h = 4 * k + sub;
      if (h < nh) {
        float a[8], b[8];
        eight_values<TI>(ra[k], a);
        eight_values<TI>(rb[k], b);
        rotate_eight<decltype(interleaved)::value>(m, g, a, b);
        store_eight<TO>(y + h * y_head + m.a * SO, a);
        store_eight<TO>(y + h * y_head + m.b * SO, b);
      }
    }
  };
  if (p.layout == KVQ_ROPE_INTERLEAVED) all(std::true_type());
  else all(std::false_type());
}

}  // namespace kvq
