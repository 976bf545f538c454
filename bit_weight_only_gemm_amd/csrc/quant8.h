// quant8.h -- symmetric 8-bit quantization shared by the 8-bit product and
// the 8-bit cache: a set of values (a row, or the rows of a cache page) is
// held as codes c in [-127, 127] and one fp32 scale s, value c s.
//
//   s = max|x| * fp32(1 / 127),  c = clip(rint(x / s), -127, 127),
//
// every operation in fp32 and rounded once (IEEE division, rint half to
// even), so a result is a function of the values alone, whatever the split of
// the work.  A set that holds an infinity or a NaN has the scale NaN: what it
// reaches is NaN, as it would be without quantization.
#pragma once
#include "common.h"

namespace w4a16 {

constexpr uint32_t kInfBits = 0x7F800000u;

// |x| as an integer: the order of the magnitudes, infinities above every
// finite value and NaN above those.
__device__ __forceinline__ uint32_t mag_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
}

// The scale of a set whose largest magnitude has these bits.
__device__ __forceinline__ float scale_of(uint32_t mag) {
  return mag >= kInfBits ? __builtin_nanf("") : __builtin_bit_cast(float, mag) * (1.0f / 127.0f);
}

// The code of x (s != 0).  A NaN quotient gives a code all the same; its
// scale is NaN then.
__device__ __forceinline__ int code_of(float x, float s) {
  return (int)fminf(fmaxf(rintf(x / s), -127.0f), 127.0f);
}

// The codes of 8 values, code_of's without its divisions: n = rint(x fp32(1/s))
// is the same unless x / s lies within 2^-12 or so of a half-integer, and
// fma(-n, s, x) / s says how far it is from n to far better than that.  Where
// one of the 8 is that near (or s too small for its reciprocal), all are
// divided.
struct Codes8 {
  float s, inv, near;
  __device__ __forceinline__ explicit Codes8(float scale)
      : s(scale), inv(1.0f / scale), near(scale > 1e-30f ? 0.4995f * scale : -1.0f) {}
  __device__ __forceinline__ void operator()(const float (&x)[8], int (&c)[8]) const {
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = rintf(x[i] * inv);
      far = fmaxf(far, fabsf(__builtin_fmaf(-n, s, x[i])));
      c[i] = (int)n;
    }
    if (!(far < near)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = code_of(x[i], s);
    }
  }
};

// Largest magnitude over a group of lanes (offsets below N, a power of two).
template <int N>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

// 8 consecutive 16-bit values as fp32.
template <int DT>
__device__ __forceinline__ void widen8(u32x4_t w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = widen16<DT>((uint16_t)(w[i] & 0xFFFFu));
    f[2 * i + 1] = widen16<DT>((uint16_t)(w[i] >> 16));
  }
}

}  // namespace w4a16
