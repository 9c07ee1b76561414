// kvq_row_decode.cuh -- one cached row's values held by a warp, four per lane
// (lane l: dims 4l .. 4l + 3), read from the bytes of its unit by the placement
// formulas of include/kvq.h.  Exact in fp32 for every codec.
#pragma once

#include "kvq_device.cuh"

namespace kvq {

// Token row r of `unit` (all 32 lanes; global or shared memory).
template <int SIDE>
__device__ __forceinline__ void decode_row_lane(int codec, const uint8_t *unit, int r, int lane,
                                                float (&x)[4]) {
  const int g = r & 7, rh = r >> 3, tig = (r & 7) >> 1, par = r & 1;
  const int b = lane >> 3, lb = lane & 7;  // block and lane in it
  if (codec == KVQ_F16) {
    if (SIDE == 0) {
      const uint2 w = *reinterpret_cast<const uint2 *>(
          unit + (2 * b + rh) * 512 + (4 * g + (lane & 3)) * 16 + (lb >> 2) * 8);
      const float2 lo = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
      const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
      x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 4 * lane + i;
        x[i] = __half2float(*reinterpret_cast<const __half *>(
            unit + (d >> 4) * 512 + (4 * ((d & 15) >> 1) + tig) * 16 +
            (rh * 4 + (d & 1) * 2 + par) * 2));
      }
    }
    return;
  }
  if (codec == KVQ_TURBO4) {
    turbo4_row_rotated<SIDE>(unit, r, lane, x);
    turbo_unrotate_lane(x, lane);
    return;
  }
  const float d = __half2float(*reinterpret_cast<const __half *>(
      unit + unit_scale_offset(codec) +
      (SIDE == 0 ? g * 16 + rh * 8 + b * 2 : tig * 32 + b * 8 + rh * 4 + par * 2)));
  if (codec == KVQ_Q8_0) {
    uint32_t w;  // dims 4 lane .. + 3, one byte each
    if (SIDE == 0) {
      w = *reinterpret_cast<const uint32_t *>(unit + b * 512 + (4 * g + (lane & 3)) * 16 +
                                              (2 * rh + (lb >> 2)) * 4);
    } else {
      w = 0;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int at = 4 * lane + 2 * p, mt = at >> 4, gq = (at & 15) >> 1;
        w |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(
                 unit + (mt >> 1) * 512 + (4 * gq + tig) * 16 + ((mt & 1) * 2 + rh) * 4 + par * 2))
             << (16 * p);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = d * static_cast<float>(static_cast<int8_t>((w >> (8 * i)) & 0xffu));
  } else {  // q4_0: lanes 4..7 of a block hold the high nibbles of its bytes
    const int l4 = lb & 3;
    uint32_t w = 0;
    if (SIDE == 0) {
      w = *reinterpret_cast<const uint32_t *>(unit + (b >> 1) * 512 + (4 * g + l4) * 16 +
                                              ((b & 1) * 2 + rh) * 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int jc = 4 * l4 + i, mt = 2 * b + (jc >> 3);
        w |= static_cast<uint32_t>(
                 unit[(mt >> 2) * 512 + (4 * (jc & 7) + tig) * 16 + (mt & 3) * 4 + par * 2 + rh])
             << (8 * i);
      }
    }
    w >>= 4 * (lb >> 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = d * static_cast<float>(static_cast<int>((w >> (8 * i)) & 0xfu) - 8);
  }
}

}  // namespace kvq
