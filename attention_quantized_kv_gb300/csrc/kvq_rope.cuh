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

}  // namespace kvq
