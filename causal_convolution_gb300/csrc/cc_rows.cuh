// Device helpers of the norm, quantisation and 8-bit product kernels: vectors
// of eight channels, the activation, and e4m3 with a scale per 128 channels.
//
// These kernels start while the one in front of them, and through it the one
// before that, may still be writing what they read after their wait. So they
// read with ordinary loads: ld.global.nc is for data that nobody writes while
// the kernel lives, and a line that an earlier kernel's loads left in an SM's
// cache may be what it finds. It was no faster either.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cc_ptx.cuh"

namespace cc {

constexpr int kScaleBlock = 128;             // channels that share a scale
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite, and a block of zeros keeps a scale

// Two fp32 values in one 64-bit register pair: sums, products and fused
// multiply-adds of pairs take one instruction for both, which these passes
// need -- at full memory rate an SM has about 20 issue slots per channel.
typedef uint64_t f32x2;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float lo(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Eight channels.
struct Vec8 {
  f32x2 p[4];
  __device__ __forceinline__ float operator[](int e) const { return (e & 1) ? hi(p[e >> 1]) : lo(p[e >> 1]); }
};

__device__ __forceinline__ Vec8 unpack8(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Vec8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return v;
}

__device__ __forceinline__ Vec8 splat8(float f) {
  Vec8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = pair(f, f);
  return v;
}

__device__ __forceinline__ uint4 pack8(const Vec8& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo(v.p[i]), hi(v.p[i]));
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values to e4m3, round to nearest even, beyond +-448 to +-448, NaN kept.
__device__ __forceinline__ uint2 pack8_e4m3(const Vec8& v) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(hi(v.p[2 * i])), "f"(lo(v.p[2 * i])));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(hi(v.p[2 * i + 1])), "f"(lo(v.p[2 * i + 1])));
    asm("mov.b32 %0, {%1, %2};" : "=r"(w[i]) : "h"(a), "h"(b));
  }
  return make_uint2(w[0], w[1]);
}

// v * sigmoid(v) = v / (1 + 2^(-v log2 e)). The exponential and the reciprocal are
// the hardware's approximations, each good to about 2^-22 (and the exponent's
// rounding to |v| 2^-24), which the rounding to bf16 or e4m3 behind them hides. The reciprocal of a divisor above 2^126 is 0:
// below -87.3 the result is 0, off by less than 2^-119.
template <bool SILU>
__device__ __forceinline__ void activate8(Vec8& v) {
  if (SILU) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 t = mul2(v.p[i], pair(-1.4426950408889634f, -1.4426950408889634f));
      const f32x2 d = add2(pair(ex2_approx(lo(t)), ex2_approx(hi(t))), pair(1.f, 1.f));
      float a, b;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(lo(d)));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(hi(d)));
      v.p[i] = mul2(v.p[i], pair(a, b));
    }
  }
}

// The largest |v|; a NaN among them is the result.
__device__ __forceinline__ float absmax3(float a, float b, float c) {
  float m;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float absmax8(const Vec8& v) {
  float m = absmax3(v[0], v[1], v[2]);
  m = absmax3(m, v[3], v[4]);
  m = absmax3(m, v[5], v[6]);
  return absmax3(m, v[7], 0.f);
}

// The scale of a block with this largest |v|. A NaN stays one.
__device__ __forceinline__ float block_scale(float absmax) {
  const float s = absmax / kE4m3Max;
  return s < kMinScale ? kMinScale : s;
}

// Quantises the eight values of each lane of a half warp, whose 16 lanes hold
// one block of 128 channels (lanes past the row hold zeros). The values are
// multiplied by the scale's reciprocal rather than divided: a few roundings of
// 2^-24 in front of the one to e4m3 (2^-4). EXACT: scale and reciprocal are
// correctly rounded quotients, so that a quantised tensor can be told bit by
// bit; behind a norm, whose values are rounded already, they may be a step of
// 2^-23 off and cost a quarter of the instructions.
template <bool EXACT>
__device__ __forceinline__ uint2 quantize_block(Vec8& v, float& scale) {
  float m = absmax8(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  float inv;
  if (EXACT) {
    scale = block_scale(m);
    inv = 1.f / scale;
  } else {
    scale = m * (1.f / kE4m3Max);
    scale = scale < kMinScale ? kMinScale : scale;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = mul2(v.p[i], pair(inv, inv));
  return pack8_e4m3(v);
}

}  // namespace cc
