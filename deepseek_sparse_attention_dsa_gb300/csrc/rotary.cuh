// rotary.cuh -- rotation of pairs of columns by position x frequency, as the
// rotary kernel (rotary.cu) and the appends (append.cu) apply it.
//
// A pair (a, b) at angle t becomes (a cos t - b sin t, a sin t + b cos t), in
// fp32.  Angles are exact to the last bit that matters at any position: a table
// holds each pair's frequency (a double) in turns a position as a 64-bit fraction of
// a turn, f = round(2^64 frequency / 2 pi) modulo 2^64, so position * f modulo 2^64
// (what a 64-bit product keeps by itself) is the fraction of a turn with an error of
// at most |position| * 2^-65 turns.  Its nearest quarter goes to the signs and the order of
// sine and cosine, and what is left, at most an eighth of a turn, is converted to
// fp32 with all of its digits.  (position * frequency in fp32 is off by 2^-24 of the
// angle: 0.008 rad at position 131,072.)
#pragma once
#include <stdint.h>

#include "dsa.h"
#include "fp8.cuh"

namespace dsa {

// (cos, sin) of a position's angle for one pair, times the table's amplitude: the
// Taylor sums of sin and cos of pi / 2 x, |x| <= 1/2, to x^9 and x^10, whose remainders
// are below 2^-28 of the result; rounded they are off by 3 half steps at most.  (Some
// 30 instructions; with sincospif they were a quarter of an append's.)
__device__ __forceinline__ float2 rotary_angle(int32_t position, uint64_t turns, float amplitude) {
  const uint64_t part = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns + (uint64_t(1) << 61);
  const uint32_t quarter = static_cast<uint32_t>(part >> 62);
  const int64_t rest = static_cast<int64_t>(part & ((uint64_t(1) << 62) - 1)) - (int64_t(1) << 61);
  const float x = __ll2float_rn(rest) * 0x1p-62f, x2 = x * x;
  float s = fmaf(x2, 1.6044118e-4f, -4.6817541e-3f);      // (pi / 2)^9 / 9!, -(pi / 2)^7 / 7!, ...
  s = fmaf(x2, s, 7.9692626e-2f);
  s = fmaf(x2, s, -6.4596410e-1f);
  s = fmaf(x2, s, 1.5707963f) * x;
  float c = fmaf(x2, -2.5202043e-5f, 9.1926027e-4f);      // -(pi / 2)^10 / 10!, (pi / 2)^8 / 8!, ...
  c = fmaf(x2, c, -2.0863481e-2f);
  c = fmaf(x2, c, 2.5366951e-1f);
  c = fmaf(x2, c, -1.2337006f);
  c = fmaf(x2, c, 1.0f);
  const float cosine = quarter & 1 ? s : c, sine = quarter & 1 ? c : s;
  return make_float2((quarter + 1) & 2 ? -cosine * amplitude : cosine * amplitude, quarter & 2 ? -sine * amplitude : sine * amplitude);
}

// Neighbouring pairs in N columns ("interleaved"); cs: their angles.
template <int N>
__device__ __forceinline__ void rotate_interleaved(float (&v)[N], const float2 *cs) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 w = cs[i];
    const float a = v[2 * i], b = v[2 * i + 1];
    v[2 * i] = fmaf(a, w.x, -b * w.y);
    v[2 * i + 1] = fmaf(a, w.y, b * w.x);
  }
}
// N pairs, the first columns in a, the second in b ("half").
template <int N>
__device__ __forceinline__ void rotate_half(float (&a)[N], float (&b)[N], const float2 *cs) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 w = cs[i];
    const float x = a[i], y = b[i];
    a[i] = fmaf(x, w.x, -y * w.y);
    b[i] = fmaf(y, w.x, x * w.y);
  }
}

// Units of a row of `width` columns whose columns offset .. offset + rot rotate:
// first the rotated ones (eight columns, or twice eight where the layout is half),
// then pieces of up to eight of the columns before and behind them.
__host__ __device__ inline int rotary_units(int rot, int layout) {
  return layout == DSA_ROTARY_HALF ? (rot / 2 + 7) / 8 : (rot + 7) / 8;
}
__host__ __device__ inline int rotary_copies(int width, int offset, int rot) {
  auto pieces = [](int n) { return n / 8 + (n % 8 > 0); };      // (a width may be 2^31 - 1)
  return pieces(offset) + pieces(width - offset - rot);
}
// Angles held for a row: whole units of them, so that a cut unit reads inside its row.
__host__ __device__ inline int rotary_pairs(int rot) { return (rot / 2 + 7) / 8 * 8; }

// Unit u of a row of `src` into `dst` (types and alignment each its own); cs: the
// row's angles, null where nothing rotates (rot 0).
__device__ __forceinline__ void rotary_unit(int u, int rot, int layout, int offset, int width, const float2 *cs,
                                            const void *src, int src_type, bool src_vec, void *dst, int dst_type,
                                            bool dst_vec) {
  const int n = rotary_units(rot, layout);
  float a[8];
  if (u < n) {
    if (layout == DSA_ROTARY_HALF) {
      float b[8];
      const int half = rot / 2, i = u * 8;
      load8(a, src, src_type, offset + i, offset + half, src_vec);
      load8(b, src, src_type, offset + half + i, offset + rot, src_vec);
      rotate_half(a, b, cs + i);
      store8(dst, dst_type, offset + i, offset + half, dst_vec, a);
      store8(dst, dst_type, offset + half + i, offset + rot, dst_vec, b);
    } else {
      load8(a, src, src_type, offset + u * 8, offset + rot, src_vec);
      rotate_interleaved(a, cs + u * 4);
      store8(dst, dst_type, offset + u * 8, offset + rot, dst_vec, a);
    }
    return;
  }
  u -= n;
  const int before = offset / 8 + (offset % 8 > 0);
  const int col = u < before ? u * 8 : offset + rot + (u - before) * 8, end = u < before ? offset : width;
  load8(a, src, src_type, col, end, src_vec);
  store8(dst, dst_type, col, end, dst_vec, a);
}

// Whether every unit's pieces start on 16 bytes when the rows do.
__host__ __device__ inline bool rotary_whole(int offset, int rot, int layout) {
  return offset % 8 == 0 && rot % (layout == DSA_ROTARY_HALF ? 16 : 8) == 0;
}

}  // namespace dsa
