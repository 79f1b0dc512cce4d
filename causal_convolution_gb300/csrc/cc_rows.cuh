// Device helpers of the norm, quantisation and 8-bit product kernels: vectors
// of eight channels, the activation, and e4m3 with a scale per 128 channels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cc {

constexpr int kScaleBlock = 128;             // channels that share a scale
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite, and a block of zeros keeps a scale

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values to e4m3, round to nearest even, beyond +-448 to +-448, NaN kept.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[4 * i + 1]), "f"(f[4 * i]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[4 * i + 3]), "f"(f[4 * i + 2]));
    w[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  return make_uint2(w[0], w[1]);
}

// v * sigmoid(v). 1 + e^-v overflows to infinity below -88, where the quotient
// is 0; the two fast operations are each good to about 2^-22, which the
// rounding to bf16 or e4m3 behind them hides.
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

template <bool SILU>
__device__ __forceinline__ void activate8(float (&f)[8]) {
  if (SILU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = silu(f[e]);
  }
}

// The largest |v| as its bit pattern: patterns of non-negative floats order
// like the floats, with infinity and then NaN on top, so a NaN is not lost as
// it would be in fmaxf.
__device__ __forceinline__ uint32_t absmax8_bits(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7fffffffu);
  return m;
}

// The scale of a block whose largest |v| has these bits. A NaN stays one.
__device__ __forceinline__ float block_scale(uint32_t absmax_bits) {
  const float s = __uint_as_float(absmax_bits) / kE4m3Max;
  return s < kMinScale ? kMinScale : s;
}

// Quantises the eight values of each lane of a half warp, whose 16 lanes hold
// one block of 128 channels (lanes past the row hold zeros). The values are
// multiplied by the scale's correctly rounded reciprocal rather than divided:
// at most two roundings of 2^-24 in front of the one to e4m3 (2^-4).
__device__ __forceinline__ uint2 quantize_block(float (&f)[8], float& scale) {
  uint32_t m = absmax8_bits(f);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  scale = block_scale(m);
  const float inv = 1.f / scale;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= inv;
  return pack8_e4m3(f);
}

}  // namespace cc
