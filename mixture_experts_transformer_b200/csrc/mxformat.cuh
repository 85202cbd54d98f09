// MXFP8: e4m3 values in groups of 32 along a row with one power-of-two scale
// (e8m0: code c stands for 2^(c - 127), 0xFF for NaN) per group - the OCP
// Microscaling MXFP8 element and scale formats.
//
// The scale of a group is the smallest 2^j >= amax / 448 (j in [-127, 127]),
// so the largest value lands in (224, 448] and nothing saturates; the values
// are v / 2^j - an exact scaling - rounded to e4m3 (nearest, ties to even).
// An all-zero group has scale code 0 and zero codes. A group that holds an
// infinity or a NaN has scale code 0xFF and NaN codes (0x7F): all 32 values
// read back as NaN.
#pragma once

#include "ptx.cuh"

namespace moe {

constexpr int kMxGroup = 32;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Scale code of a group from the largest |v| bit pattern (as integers NaN >
// infinity > finite, so an integer maximum carries a NaN through).
// amax = 1.f * 2^e: 2^j >= amax / (1.75 * 2^8) means j = e - 8, or e - 7 when 1.f > 1.75.
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 0xFFu;
  const int c = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return c < 0 ? 0u : static_cast<uint32_t>(c);
}

// 2^(127 - code): the exact multiplier that scales a group's values (NaN for 0xFF).
__device__ __forceinline__ float mx_inv_scale(uint32_t code) {
  return code == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - code) << 23);
}

// Four e4m3 codes, v0 in the low byte. NaN gives 0x7F (the sign of a NaN is not kept).
__device__ __forceinline__ uint32_t e4m3x4(float v0, float v1, float v2, float v3) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
  return r;
}

// Byte offset of the scale of (row, group c32) in a [ceil(rows/128)][ceil(K/128)][512]
// array of scale atoms: the atom of rows 128a..128a+127 and K range 128b..128b+127
// holds row r, group c (0..3) at byte 16 (r % 32) + 4 (r / 32) + c.
__host__ __device__ __forceinline__ size_t mx_sf_offset(int row, int c32, int kblocks) {
  return (static_cast<size_t>(row >> 7) * kblocks + (c32 >> 2)) * 512 + 16 * (row & 31) + 4 * ((row & 127) >> 5) +
         (c32 & 3);
}

// Quantise one whole group held by one thread: returns the scale code, writes the 32 code bytes.
__device__ __forceinline__ uint32_t mx_group(const float (&v)[32], uint4 (&codes)[2]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, abs_bits(v[i]));
  const uint32_t sc = mx_scale_code(m);
  const float r = mx_inv_scale(sc);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = e4m3x4(v[4 * i] * r, v[4 * i + 1] * r, v[4 * i + 2] * r, v[4 * i + 3] * r);
  codes[0] = make_uint4(w[0], w[1], w[2], w[3]);
  codes[1] = make_uint4(w[4], w[5], w[6], w[7]);
  return sc;
}

// GELU, tanh form, in fp32: z/2 (1 + tanh(u)) = z / (1 + exp(-2u)). Its
// relative error is at most (4.2 |2u| + 5) 2^-23: six roundings of 2u, each
// |2u| 2^-24 in the exponent, __expf's 2 + 1.173 |2u| units, __fdividef's two,
// one more of the sum - 2^-19 at |z| = 1, 2^-17 at z = -4, where the value is
// 1e-4 of z. (1 + tanh(u) in fp32 loses all of its bits there.)
// The MXFP8 quantiser behind it turns an error d of a value into a flipped
// code with probability d / step, so the approximate tanh (absolute error
// 2^-11) would cost up to 2^-11-sized flips of whole e4m3 steps.
__device__ __forceinline__ float gelu_tanh_exact(float z) {
  const float c2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
  const float u2 = c2 * fmaf(0.044715f * z, z * z, z);
  return __fdividef(z, 1.0f + __expf(-u2));
}

}  // namespace moe
