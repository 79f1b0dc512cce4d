// Group norm over channels-last instances with an optional SiLU, written as
// bf16 or as e4m3 with a scale per position and block of 128 channels.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cc.h"
#include "cc_host.h"
#include "cc_ptx.cuh"
#include "cc_rows.cuh"

namespace cc {
namespace {

constexpr int kGnThreads = 512;
constexpr int kGnMaxChannels = 8 * kGnThreads;
constexpr int kChunkVecs = 16;  // vectors per thread and statistics chunk

// Mean and sum of squared deviations of `n` values; two of them merge exactly
// (in real arithmetic) into that of their union, without the cancellation
// that sum(x^2) - n mean^2 has when the mean is large.
struct Moments {
  float n, mean, m2;
};

__device__ __forceinline__ void merge(Moments& a, const Moments& b) {
  if (b.n == 0.f) return;
  const float n = a.n + b.n;
  const float d = b.mean - a.mean;
  const float f = b.n / n;
  a.mean = fmaf(d, f, a.mean);
  a.m2 += b.m2 + d * d * a.n * f;
  a.n = n;
}

__device__ __forceinline__ Moments warp_merge(Moments m) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    // the lower lane's moments come first on both sides, so all lanes agree
    Moments b = {__shfl_xor_sync(0xffffffffu, m.n, o), __shfl_xor_sync(0xffffffffu, m.mean, o),
                 __shfl_xor_sync(0xffffffffu, m.m2, o)};
    if ((threadIdx.x & o) != 0) {
      const Moments t = m;
      m = b;
      b = t;
    }
    if (m.n == 0.f) {
      m = b;
    } else {
      merge(m, b);
    }
  }
  return m;
}

struct GnArgs {
  const uint4* x;
  const uint4* gamma;  // nullptr: ones
  const uint4* beta;   // nullptr: zeros
  void* y;
  float* scales;
  float2* part;  // [N][chunks][G]
  float2* stat;  // [N][G] (mean, 1 / standard deviation)
  int p;
  int vecs;   // C / 8
  int slots;  // vecs, rounded up to whole half warps for e4m3
  int groups;
  int cpg;
  int gw;  // channels of a vector part that always share a group: gcd(C / G, 8)
  int chunks;
  int chunk_rows;
  int blocks;
  float eps;
};

// The moments of each group over a CTA's positions, from each thread's sums
// of its eight channels around a pivot of their own.
__device__ __forceinline__ void block_moments(const GnArgs& a, float2* red, float* cnt, const float (&pivot)[8],
                                              const float (&s1)[8], const float (&s2)[8], int n, float2* out) {
  const int tid = threadIdx.x;
  float mean[8], m2[8];
  const float inv = n > 0 ? 1.f / n : 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float d = s1[e] * inv;
    mean[e] = pivot[e] + d;
    m2[e] = s2[e] - s1[e] * d;
    m2[e] = m2[e] < 0.f ? 0.f : m2[e];  // keeps a NaN
  }
  int w = 1;
  float half = 0.5f * n;
#pragma unroll
  for (int l = 1; l < 8; l <<= 1) {
    if (a.gw > l) {  // uniform
#pragma unroll
      for (int e = 0; e < 8; e += 2 * l) {
        const float d = mean[e + l] - mean[e];
        m2[e] += m2[e + l] + d * d * half;
        mean[e] = 0.5f * (mean[e] + mean[e + l]);
      }
      w = 2 * l;
      half *= 2.f;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e % w == 0) red[(e / w) * kGnThreads + tid] = make_float2(mean[e], m2[e]);
  cnt[tid] = static_cast<float>(n * w);
  __syncthreads();
  const int per = a.cpg / a.gw;           // vector parts per group and position
  const int lanes = kGnThreads / a.slots;  // positions side by side
  const int parts = 8 / a.gw;
  for (int g = tid >> 5; g < a.groups; g += kGnThreads / 32) {
    Moments m = {0.f, 0.f, 0.f};
    for (int i = tid & 31; i < per * lanes; i += 32) {
      const int j = g * per + i % per;
      const int t = (i / per) * a.slots + j / parts;
      const float2 v = red[(j % parts) * kGnThreads + t];
      const Moments b = {cnt[t], v.x, v.y};
      if (m.n == 0.f) {
        m = b;
      } else {
        merge(m, b);
      }
    }
    m = warp_merge(m);
    if ((tid & 31) == 0) out[g] = make_float2(m.mean, m.m2);
  }
}

__global__ void __launch_bounds__(kGnThreads) gn_stats_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ float2 red[];
  __shared__ float cnt[kGnThreads];
  const int lanes = kGnThreads / a.slots;
  const int lane = threadIdx.x / a.slots;
  const int v = threadIdx.x - lane * a.slots;
  const int r0 = blockIdx.x * a.chunk_rows;
  const int r1 = min(r0 + a.chunk_rows, a.p);
  const uint4* x = a.x + static_cast<long long>(blockIdx.y) * a.p * a.vecs + v;
  float pivot[8] = {}, s1[8] = {}, s2[8] = {};
  int n = 0;
  if (lane < lanes && v < a.vecs) {
    for (int r = r0 + lane; r < r1; r += lanes) {
      float f[8];
      unpack8(x[static_cast<long long>(r) * a.vecs], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (n == 0) pivot[e] = f[e];
        const float d = f[e] - pivot[e];
        s1[e] += d;
        s2[e] = fmaf(d, d, s2[e]);
      }
      ++n;
    }
  }
  block_moments(a, red, cnt, pivot, s1, s2, n,
                a.part + (static_cast<long long>(blockIdx.y) * a.chunks + blockIdx.x) * a.groups);
}

__global__ void __launch_bounds__(128) gn_finish_kernel(const __grid_constant__ GnArgs a) {
  const int g = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (g >= a.groups) return;
  const long long n = blockIdx.y;
  Moments m = {0.f, 0.f, 0.f};
  for (int i = threadIdx.x & 31; i < a.chunks; i += 32) {
    const float2 v = a.part[(n * a.chunks + i) * a.groups + g];
    const int rows = min(a.chunk_rows, a.p - i * a.chunk_rows);
    const Moments b = {static_cast<float>(rows) * a.cpg, v.x, v.y};
    if (m.n == 0.f) {
      m = b;
    } else {
      merge(m, b);
    }
  }
  m = warp_merge(m);
  if ((threadIdx.x & 31) == 0) a.stat[n * a.groups + g] = make_float2(m.mean, 1.f / sqrtf(m.m2 / m.n + a.eps));
}

template <bool SILU, bool FP8>
__global__ void __launch_bounds__(kGnThreads) gn_apply_kernel(const __grid_constant__ GnArgs a) {
  const int lanes = kGnThreads / a.slots;
  const int lane = threadIdx.x / a.slots;
  const int v = threadIdx.x - lane * a.slots;
  const int r0 = blockIdx.x * a.chunk_rows;
  const int r1 = min(r0 + a.chunk_rows, a.p);
  const bool used = lane < lanes && v < a.vecs;
  // (x - mean) * k + beta, the mean taken off first: folded into beta it would
  // cost digits where it is large against the deviation
  float mean[8], k[8], b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) k[e] = 1.f, b[e] = 0.f, mean[e] = 0.f;
  if (used) {
    if (a.gamma) unpack8(a.gamma[v], k);
    if (a.beta) unpack8(a.beta[v], b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 st = a.stat[static_cast<long long>(blockIdx.y) * a.groups + (8 * v + e) / a.cpg];
      mean[e] = st.x;
      k[e] *= st.y;
    }
  }
  for (int rr = r0; rr < r1; rr += lanes) {
    const int r = rr + lane;
    const bool on = used && r < r1;
    const long long at = (static_cast<long long>(blockIdx.y) * a.p + r) * a.vecs + v;
    float f[8] = {};
    if (on) {
      unpack8(a.x[at], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmaf(f[e] - mean[e], k[e], b[e]);
      activate8<SILU>(f);
    }
    if (FP8) {
      float scale;
      const uint2 q = quantize_block(f, scale);
      if (on) {
        static_cast<uint2*>(a.y)[at] = q;
        if ((v & 15) == 0) a.scales[(static_cast<long long>(blockIdx.y) * a.p + r) * a.blocks + (v >> 4)] = scale;
      }
    } else if (on) {
      static_cast<uint4*>(a.y)[at] = pack8(f);
    }
  }
}

int gn_chunk_rows(int c) { return std::max(1, kGnThreads / (c / 8)) * kChunkVecs; }

size_t gn_bytes(int n, int p, int c, int groups) {
  const size_t chunks = (static_cast<size_t>(p) + gn_chunk_rows(c) - 1) / gn_chunk_rows(c);
  return (chunks + 1) * n * groups * sizeof(float2);
}

cc_status run_group_norm(const char* what, const cc_bf16* x, const cc_bf16* gamma, const cc_bf16* beta, void* y,
                         float* scales, bool fp8, int n, int p, int c, int groups, float eps, int act, void* ws,
                         size_t ws_bytes, void* stream) {
  cc_status st;
  if (empty_request(what, {n, p}, &st)) return st;
  if (!x || !y || (fp8 && !scales)) return fail(CC_ERR_INVALID, "%s: null pointer", what);
  if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(y) || !aligned16(scales) || !aligned16(ws))
    return fail(CC_ERR_INVALID, "%s: pointers must be 16-byte aligned", what);
  if (c <= 0 || groups <= 0 || c % groups != 0)
    return fail(CC_ERR_INVALID, "%s: the groups must divide C (C %d, %d groups)", what, c, groups);
  if (c % 8 != 0) return fail(CC_ERR_UNSUPPORTED, "%s: C must be a multiple of 8 (got %d)", what, c);
  if (c > kGnMaxChannels) return fail(CC_ERR_UNSUPPORTED, "%s: C must be at most %d (got %d)", what, kGnMaxChannels, c);
  if (n > 65535) return fail(CC_ERR_UNSUPPORTED, "%s: at most 65535 instances", what);
  if (p > (1 << 30)) return fail(CC_ERR_UNSUPPORTED, "%s: too many positions", what);
  if (!(eps > 0.f && eps <= 1e30f)) return fail(CC_ERR_INVALID, "%s: eps must be positive and finite", what);
  if (act != CC_ACT_NONE && act != CC_ACT_SILU) return fail(CC_ERR_INVALID, "%s: unknown activation %d", what, act);
  const size_t need = gn_bytes(n, p, c, groups);
  if (!ws || ws_bytes < need)
    return fail(CC_ERR_INVALID, "%s: workspace of %zu bytes needed (got %zu)", what, need, ws ? ws_bytes : 0);
  DeviceInfo di;
  if ((st = device_info(&di)) != CC_OK) return st;
  GnArgs a = {};
  a.x = reinterpret_cast<const uint4*>(x);
  a.gamma = reinterpret_cast<const uint4*>(gamma);
  a.beta = reinterpret_cast<const uint4*>(beta);
  a.y = y;
  a.scales = scales;
  a.p = p;
  a.vecs = c / 8;
  a.groups = groups;
  a.cpg = c / groups;
  a.gw = a.cpg % 8 == 0 ? 8 : a.cpg % 4 == 0 ? 4 : a.cpg % 2 == 0 ? 2 : 1;
  a.chunk_rows = gn_chunk_rows(c);
  a.chunks = (p + a.chunk_rows - 1) / a.chunk_rows;
  a.blocks = (c + kScaleBlock - 1) / kScaleBlock;
  a.eps = eps;
  a.stat = static_cast<float2*>(ws);
  a.part = a.stat + static_cast<size_t>(n) * groups;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.slots = a.vecs;
  gn_stats_kernel<<<dim3(a.chunks, n), kGnThreads, 8 / a.gw * kGnThreads * sizeof(float2), s>>>(a);
  if ((st = launch_status(what)) != CC_OK) return st;
  gn_finish_kernel<<<dim3((groups + 3) / 4, n), 128, 0, s>>>(a);
  if ((st = launch_status(what)) != CC_OK) return st;
  if (fp8) a.slots = (a.vecs + 15) / 16 * 16;
  auto kern = fp8 ? (act == CC_ACT_SILU ? gn_apply_kernel<true, true> : gn_apply_kernel<false, true>)
                  : (act == CC_ACT_SILU ? gn_apply_kernel<true, false> : gn_apply_kernel<false, false>);
  kern<<<dim3(a.chunks, n), kGnThreads, 0, s>>>(a);
  return launch_status(what);
}

}  // namespace
}  // namespace cc

using namespace cc;

extern "C" size_t cc_group_norm_workspace_bytes(int n, int p, int c, int groups) {
  if (n <= 0 || p <= 0 || c < 8 || groups <= 0) return 0;
  return gn_bytes(n, p, c, groups);
}

extern "C" cc_status cc_group_norm_act(const cc_bf16* x, const cc_bf16* gamma, const cc_bf16* beta, cc_bf16* y, int n,
                                       int p, int c, int groups, float eps, int act, void* ws, size_t ws_bytes,
                                       void* stream) {
  return run_group_norm("group_norm_act", x, gamma, beta, y, nullptr, false, n, p, c, groups, eps, act, ws, ws_bytes,
                        stream);
}

extern "C" cc_status cc_group_norm_act_fp8(const cc_bf16* x, const cc_bf16* gamma, const cc_bf16* beta, cc_fp8* y,
                                           float* scales, int n, int p, int c, int groups, float eps, int act,
                                           void* ws, size_t ws_bytes, void* stream) {
  return run_group_norm("group_norm_act_fp8", x, gamma, beta, y, scales, true, n, p, c, groups, eps, act, ws,
                        ws_bytes, stream);
}
