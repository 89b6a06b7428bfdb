// fp8.cuh -- device helpers of the 8-bit operators (rmsnorm.cu,
// quantize_rows.cu, project.cu): eight values of a row at a time from bf16 or
// fp32, and groups of values to e4m3 codes.
//
// Quantisation, as everywhere in the library: a group's scale is amax / 448 in
// fp32 (1 where that is zero: an all-zero group, or one below fp32's range), a
// code is E4M3 of the fp32 quotient by it, rounded to nearest with ties to even, NaN
// being 0x7F and finite values saturating at 448.  The maximum is taken over the bit
// patterns of the magnitudes, which order as the magnitudes do with NaN above
// infinity, so a NaN or an infinity always reaches the scale: such a group has
// the scale NaN or infinity and no finite value comes back out of it.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "dsa.h"

namespace dsa {

// The kernels of these operators are short, so the next one's launch and set-up
// weigh: each lets its successor be launched at once and waits, before it touches
// global memory, until its predecessor is complete and its writes are visible.
// Every CTA waits (also one without work: a kernel that ended before its
// predecessor would let its successor run beside that).  Inputs may be written
// after such a kernel has started, so it does not use read-only (nc) loads.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency() {
  launch_dependents();
  grid_dependency_wait();
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight bf16 values of a 16-byte piece: as floats, and the bits of their
// largest magnitude (as of a float), two at a time.
__device__ __forceinline__ void unpack8(float (&v)[8], uint4 u) {
  v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint32_t amax_bits8(uint4 u) {
  const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                              __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
  return max(m << 16, m & 0xFFFF0000u);
}

// Values col .. col+7 of a row (zero at and after `width`).  `vec`: the row
// starts on 16 bytes, so a whole piece is one or two 16-byte loads.
__device__ __forceinline__ void load8(float (&v)[8], const void *row, int type, int64_t col, int64_t width, bool vec) {
  if (type == DSA_BF16) {
    const uint16_t *p = static_cast<const uint16_t *>(row) + col;
    if (vec && col + 8 <= width) {
      unpack8(v, *reinterpret_cast<const uint4 *>(p));
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < width ? bf16_lo(p[i]) : 0.f;
  } else {
    const float *p = static_cast<const float *>(row) + col;
    if (vec && col + 8 <= width) {
      const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < width ? p[i] : 0.f;
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// The same eight values back, each rounded once to the row's type.
__device__ __forceinline__ void store8(void *row, int type, int64_t col, int64_t width, bool vec, const float (&v)[8]) {
  if (type == DSA_BF16) {
    __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(row) + col;
    if (vec && col + 8 <= width) {
      *reinterpret_cast<uint4 *>(p) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < width) p[i] = __float2bfloat16_rn(v[i]);
  } else {
    float *p = static_cast<float *>(row) + col;
    if (vec && col + 8 <= width) {
      reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < width) p[i] = v[i];
  }
}

// Bits of the largest magnitude of eight values, NaN above everything.
__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

__device__ __forceinline__ float group_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) / 448.f;
  return s == 0.f ? 1.f : s;
}

// A group's scale and its reciprocal, rounded.  Exact quotients by the scale then
// take three instructions (Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990: with r the rounded reciprocal of s,
// q the rounded product x r and e = x - q s, which a fused multiply-add has
// exactly, q + e r rounds to the rounded quotient x / s).  They have to be exact:
// bf16 values over bf16 maxima meet borders between two codes in one value of
// some 600.  e is exact down to x = 2^-102, and below it the quotient by a scale
// of 2^-80 or more is far inside code 0; smaller scales take the division.  The
// negative of e is taken, q s - x, for the sign of a zero: an exact difference is
// +0, so x = -0 gives -(+0) r + -0 = -0, and x = +0 gives -0 + +0 = +0 (with x - q s
// it is +0 for both; x's sign put onto the result instead took 66.5 us for 2048 x
// 65536 bf16 against 63.8).  An infinite scale has r = 0 and q = +-0 for a finite x;
// bounded, s keeps q s a zero, so that the quotient is x's zero as by a division
// (and NaN for an infinite x, whose q is NaN); a NaN scale has r = NaN.
struct GroupScale {
  float scale, r;
  __device__ __forceinline__ explicit GroupScale(uint32_t amax_bits) : scale(group_scale(amax_bits)), r(1.f / scale) {}
  __device__ __forceinline__ GroupScale(float s, float reciprocal) : scale(s), r(reciprocal) {}
  __device__ __forceinline__ float quotient(float x) const {
    const float q = x * r;
    return fmaf(-fmaf(q, fminf(scale, 0x1.fffffep127f), -x), r, q);
  }
};
// Four quotients to four codes, the first in bits 0-7.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Eight values of one group to eight codes.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const GroupScale &g) {
  if (g.scale < 0x1p-80f)
    return make_uint2(e4m3x4(v[0] / g.scale, v[1] / g.scale, v[2] / g.scale, v[3] / g.scale),
                      e4m3x4(v[4] / g.scale, v[5] / g.scale, v[6] / g.scale, v[7] / g.scale));
  return make_uint2(e4m3x4(g.quotient(v[0]), g.quotient(v[1]), g.quotient(v[2]), g.quotient(v[3])),
                    e4m3x4(g.quotient(v[4]), g.quotient(v[5]), g.quotient(v[6]), g.quotient(v[7])));
}

// Codes col .. col+7 of a row.  `vec`: the row starts on 8 bytes.
__device__ __forceinline__ void store_codes8(uint8_t *row, int64_t col, int64_t width, bool vec, uint2 c) {
  if (vec && col + 8 <= width) {
    *reinterpret_cast<uint2 *>(row + col) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < width) row[col + i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
}

// Rows of a call that are not padding: `rows`, or with a capturable plan the
// plan's current row count (device memory) times the rows the call has for
// each of the plan's.
__device__ __forceinline__ int64_t live_rows(int64_t rows, const int32_t *count, int32_t per_row) {
  if (count == nullptr) return rows;
  const int64_t live = static_cast<int64_t>(*count) * per_row;
  return live < rows ? live : rows;
}

}  // namespace dsa
