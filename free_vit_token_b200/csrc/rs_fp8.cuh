// rs_fp8.cuh -- 8-bit blocks: e4m3 values with one power-of-two scale (an E8M0 byte) per
// 128 consecutive values along the reduction.
//
// For a block with largest finite magnitude a, e is the least integer with a <= 448 * 2^e
// (448 is e4m3's largest value), at least -127; an all-zero block has e = -127. The stored
// value is RN_e4m3(x * 2^-e), ties to even: x * 2^-e is exact (or a result far below e4m3's
// least value), so a value is rounded once, by at most half an e4m3 step (2^-4 of the value, 2^-10 * 2^e below
// 2^-6 * 2^e). A power of two, not a / 448 itself, because the tensor cores apply E8M0
// scales inside the matrix instruction: the product then needs no pass over its fp32
// accumulators between blocks. Infinities and NaN become e4m3's NaN and do not count for a.
//
// Scale bytes (e + 127) lie as the tensor cores read them, in tiles of 128 rows x 4 blocks
// (512 bytes): row r and block j of an operand with KQ = ceil(K / 512) tiles along K at
//   ((r / 128) KQ + j / 4) 512 + 16 (r % 32) + 4 (r / 32 % 4) + j % 4.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "rs_ptx.cuh"

namespace rs {

// Products of two fp32 pairs (the sums are in rs_ptx.cuh).
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

constexpr int kQBlock = 128;      // values per scale
constexpr int kScaleTile = 512;   // bytes of scales for 128 rows x 4 blocks

__host__ __device__ __forceinline__ int64_t scale_offset(int64_t r, int j, int kq) {
  return ((r >> 7) * kq + (j >> 2)) * kScaleTile + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3);
}

// Scale byte e + 127 of a block whose largest finite magnitude has the fp32 bits `amax`:
// with amax = m 2^k, 1 <= m < 2, e = k - 8 for m <= 1.75 (448 = 1.75 * 2^8), else k - 7;
// adding 0x1FFFFF to the bits carries into the exponent exactly when m > 1.75.
__device__ __forceinline__ uint32_t e8m0_byte(uint32_t amax) {
  const int f = static_cast<int>((amax + 0x1FFFFFu) >> 23) - 8;
  return static_cast<uint32_t>(f > 0 ? f : 0);
}
// 2^-e for a scale byte of e8m0_byte (at most 247, so the exponent field is at least 7).
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// Two values to e4m3 (`lo` in the low byte), round to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// |x| as bits, which order like the magnitudes, NaN above infinity above all finite values.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;
// For blocks that hold infinities or NaN: the magnitude that counts (0 for those values),
// and the value with infinities turned into NaN, which e4m3 can hold.
__device__ __forceinline__ uint32_t finite_abs_bits(float x) {
  const uint32_t b = abs_bits(x);
  return b < kInfBits ? b : 0u;
}
__device__ __forceinline__ float inf_to_nan(float x) {
  return abs_bits(x) < kInfBits ? x : __uint_as_float(0x7FC00000u);
}

// ---------------------------------------------------------------- 16-byte vectors of T
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int E = 8;
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = bf16lo(w[e]);
      f[2 * e + 1] = bf16hi(w[e]);
    }
  }
  static __device__ __forceinline__ void pairs(const uint4& v, uint64_t (&f)[4]) {
    f[0] = bf16x2_to_f2(v.x);
    f[1] = bf16x2_to_f2(v.y);
    f[2] = bf16x2_to_f2(v.z);
    f[3] = bf16x2_to_f2(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Elem<__half> {
  static constexpr int E = 8;
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
      f[2 * e] = t.x;
      f[2 * e + 1] = t.y;
    }
  }
  static __device__ __forceinline__ void pairs(const uint4& v, uint64_t (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
      f[e] = f2pack(t.x, t.y);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 h = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Elem<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ void pairs(const uint4& v, uint64_t (&f)[2]) {
    f[0] = (static_cast<uint64_t>(v.y) << 32) | v.x;
    f[1] = (static_cast<uint64_t>(v.w) << 32) | v.z;
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

}  // namespace rs
