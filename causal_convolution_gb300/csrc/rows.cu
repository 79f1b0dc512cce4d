// Passes over independent rows of channels: RMS norm with an activation, and
// the quantisation of bf16 rows and weights to e4m3 with block scales.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cc.h"
#include "cc_host.h"
#include "cc_ptx.cuh"
#include "cc_rows.cuh"

namespace cc {
namespace {

constexpr int kRowThreads = 256;
constexpr int kMaxRowChannels = 16384;

struct RowArgs {
  const uint4* x;
  const uint4* gamma;  // nullptr: ones
  void* y;
  float* scales;
  long long rows;
  long long ld_x;  // in vectors of eight channels
  int vecs;        // C / 8
  int piece;       // vectors that a warp takes of a row at a time
  int blocks;      // ceil(C / 128)
  float inv_c;
  float eps;
};

// What follows the load: norm factor, activation, output. `on`: the lane has a
// vector of the row. Whole warps call it, with the lanes of a half warp on one
// block of 128 channels.
template <bool NORM, bool SILU, bool FP8>
__device__ __forceinline__ void finish_vector(const RowArgs& a, const uint4& raw, const uint4& gamma, float rs,
                                              long long r, int v, bool on) {
  Vec8 f = unpack8(raw);
  if (NORM) {
    const Vec8 g = unpack8(gamma);
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = mul2(f.p[i], mul2(g.p[i], pair(rs, rs)));
    activate8<SILU>(f);
  }
  if (FP8) {
    float scale;
    const uint2 q = quantize_block<!NORM>(f, scale);  // lanes without a vector hold zeros
    if (on) {
      static_cast<uint2*>(a.y)[r * a.vecs + v] = q;
      if ((threadIdx.x & 15) == 0) a.scales[r * a.blocks + (v >> 4)] = scale;
    }
  } else if (on) {
    static_cast<uint4*>(a.y)[r * a.vecs + v] = pack8(f);
  }
}

__device__ __forceinline__ f32x2 sum_squares(const uint4& raw, f32x2 sum) {
  const Vec8 f = unpack8(raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = fma2(f.p[i], f.p[i], sum);
  return sum;
}

// 1 / sqrt(mean of squares + eps). The reciprocal root (off by at most two units in
// the last place) saves e4m3 outputs 3-9 % (300000 x 128 35.8 -> 33.9 us,
// 94467 x 160 23.3 -> 21.4); with it the bf16 kernel gets its registers dealt
// worse (439296 x 512 145 -> 178), so that one divides.
template <bool FP8>
__device__ __forceinline__ float norm_factor(float sum, const RowArgs& a) {
  const float v = fmaf(sum, a.inv_c, a.eps);
  return FP8 ? rsqrtf(v) : 1.f / sqrtf(v);
}

// CTAs of a row kernel to an SM: three with 80 registers a thread, or four with
// 64. (Some forms of either keep up to 36 bytes a thread in local memory.) In us with three / with four: norm of
// 439296 x 512 to bf16 149 / 145, to e4m3 (100000 rows) 35 / 38; with four
// vectors to a lane (100000 x 1024) the norm takes 67 / 74, quantising 55 / 50,
// and with one (100000 x 256) 14.5 / 17.0.
template <int V, bool NORM, bool FP8>
constexpr int row_ctas() {
  return (V == 4 ? NORM : FP8) ? 3 : 4;
}

// Rows of up to 8 * TPR * V channels, TPR lanes each with V vectors of a row in
// registers, so a row is read once and its sum costs shuffles only. A warp
// loads R rows (about four 16-byte loads a lane) before it uses the first, and
// walks the rows in steps of the grid; gamma stays in registers. Neighbouring
// rows go to different CTAs, so few rows spread over the SMs. Without a norm
// longer rows come in pieces of whole blocks, as blockIdx.y says.
//
// Bound by memory where there are many rows: RMS norm + SiLU of 439296 x 512 in
// 145 us (6.2 TB/s, 0.92 of a copy; a block per row took 1.6 ms), quantising
// 13728 x 1024 in 5.9 us (7.2 TB/s, part of it out of L2) and 60000 x 2048 in 60
// (6.2 TB/s). Few rows cost a launch and a trip to memory: 300 x 1024 2.0 us,
// 5 x 1000 quantised 1.6 us, less than the call on the host. To e4m3 instructions
// bound it: 164068 x 616 takes 79 us for 45 us of bytes, and 97 with SiLU, whose
// exponentials and reciprocals at 16 a clock and SM would take 43 to 53 alone.
template <int TPR, int V, bool NORM, bool SILU, bool FP8>
__global__ void __launch_bounds__(kRowThreads, row_ctas<V, NORM, FP8>()) row_kernel(const __grid_constant__ RowArgs a) {
  constexpr int R = 4 / V;
  const int lane = threadIdx.x % TPR;
  const long long step = static_cast<long long>(gridDim.x) * (kRowThreads / TPR);
  const long long first = static_cast<long long>(threadIdx.x / TPR) * gridDim.x + blockIdx.x;
  const int v0 = NORM ? lane : blockIdx.y * a.piece + lane;
  const int end = NORM ? a.vecs : min(a.vecs, static_cast<int>(blockIdx.y + 1) * a.piece);
  pdl_launch_dependents();
  pdl_wait();
  uint4 gamma[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = v0 + i * TPR;
    gamma[i] = NORM && a.gamma && v < a.vecs ? a.gamma[v]
                                             : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  }
  // every lane of a warp runs the same number of rounds (they share shuffles)
  const long long warp_first = TPR == 32 ? first : static_cast<long long>(threadIdx.x / 32 * 2) * gridDim.x + blockIdx.x;
  for (long long off = 0; warp_first + off < a.rows; off += R * step) {
    uint4 raw[R][V];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const long long r = first + off + j * step;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = v0 + i * TPR;
        raw[j][i] = r < a.rows && v < end ? __ldcs(a.x + r * a.ld_x + v) : make_uint4(0, 0, 0, 0);
      }
    }
    float rs[R];
    if (NORM) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        f32x2 sum = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) sum = sum_squares(raw[j][i], sum);
        rs[j] = lo(sum) + hi(sum);
      }
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int j = 0; j < R; ++j) rs[j] += __shfl_xor_sync(0xffffffffu, rs[j], o);
      }
#pragma unroll
      for (int j = 0; j < R; ++j) rs[j] = norm_factor<FP8>(rs[j], a);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const long long r = first + off + j * step;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = v0 + i * TPR;
        if (V > 2 && v - lane >= end) break;  // the same for the whole warp
        finish_vector<NORM, SILU, FP8>(a, raw[j][i], gamma[i], NORM ? rs[j] : 1.f, r, v, r < a.rows && v < end);
      }
    }
  }
}

// Norms of longer rows: one row per CTA, up to four vectors a thread, with one
// barrier a row for its sum. 60000 x 2048 to e4m3 72 us, to bf16 76; a warp with
// eight vectors a lane took 101 and 86, two vectors a thread take 97 and 96.
template <bool SILU, bool FP8>
__global__ void __launch_bounds__(kMaxRowChannels / 32) long_row_kernel(const __grid_constant__ RowArgs a) {
  __shared__ float red[2][16];
  const int tid = threadIdx.x;
  int turn = 0;
  pdl_launch_dependents();
  pdl_wait();
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
    uint4 raw[4];
    f32x2 sum = pair(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = tid + i * blockDim.x;
      raw[i] = v < a.vecs ? __ldcs(a.x + r * a.ld_x + v) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = sum_squares(raw[i], sum);
    float rs = lo(sum) + hi(sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, o);
    if ((tid & 31) == 0) red[turn][tid >> 5] = rs;
    __syncthreads();  // one per row: the two halves of `red` take turns
    rs = 0.f;
    for (int i = 0; i < blockDim.x / 32; ++i) rs += red[turn][i];
    rs = norm_factor<FP8>(rs, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i * static_cast<int>(blockDim.x) >= a.vecs) break;
      const int v = tid + i * blockDim.x;
      const uint4 gamma =
          a.gamma && v < a.vecs ? a.gamma[v] : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
      finish_vector<true, SILU, FP8>(a, raw[i], gamma, rs, r, v, v < a.vecs);
    }
  }
}

template <bool NORM, bool SILU, bool FP8>
cc_status launch_rows(const char* what, RowArgs& a, int sms, cudaStream_t stream) {
  const int lanes = a.vecs <= 16 ? 16 : 32;
  const int v = (a.vecs + lanes - 1) / lanes;
  void (*kern)(RowArgs);
  int threads = kRowThreads, ctas, pieces = 1;
  if (NORM && v > 4) {
    kern = long_row_kernel<SILU, FP8>;
    threads = (a.vecs + 127) / 128 * 32;
    ctas = 2048 / threads;
  } else {
    kern = lanes == 16 ? row_kernel<16, 1, NORM, SILU, FP8>
           : v == 1    ? row_kernel<32, 1, NORM, SILU, FP8>
           : v == 2    ? row_kernel<32, 2, NORM, SILU, FP8>
                       : row_kernel<32, 4, NORM, SILU, FP8>;
    ctas = v > 2 ? row_ctas<4, NORM, FP8>() : row_ctas<1, NORM, FP8>();
    pieces = (v + 3) / 4;
    a.piece = (v + pieces - 1) / pieces * lanes;
  }
  // as many CTAs as fit, walking the rows
  const long long fit = (static_cast<long long>(sms) * ctas + pieces - 1) / pieces;
  const dim3 grid(static_cast<unsigned>(std::min<long long>(a.rows, fit)), pieces);
  const cudaError_t e = launch_pdl(kern, grid, dim3(threads), 0, stream, a);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: launch: %s", what, cudaGetErrorString(e));
  return launch_status(what);
}

cc_status run_rows(const char* what, bool norm, const cc_bf16* x, const cc_bf16* gamma, void* y, float* scales,
                   int rows, int c, int64_t ld_x, float eps, int act, void* stream) {
  cc_status st;
  if (empty_request(what, {rows}, &st)) return st;
  if (!x || !y) return fail(CC_ERR_INVALID, "%s: null pointer", what);
  if (!aligned16(x) || !aligned16(gamma) || !aligned16(y) || !aligned16(scales))
    return fail(CC_ERR_INVALID, "%s: pointers must be 16-byte aligned", what);
  if (c <= 0) return fail(CC_ERR_INVALID, "%s: channel counts must be positive", what);
  if (c % 8 != 0) return fail(CC_ERR_UNSUPPORTED, "%s: C must be a multiple of 8 (got %d)", what, c);
  if (c > kMaxRowChannels)
    return fail(CC_ERR_UNSUPPORTED, "%s: C must be at most %d (got %d)", what, kMaxRowChannels, c);
  if (ld_x < c || ld_x % 8 != 0)
    return fail(CC_ERR_INVALID, "%s: ld_x must be at least C and a multiple of 8", what);
  if (act != CC_ACT_NONE && act != CC_ACT_SILU) return fail(CC_ERR_INVALID, "%s: unknown activation %d", what, act);
  if (norm && !(eps > 0.f && eps <= 1e30f)) return fail(CC_ERR_INVALID, "%s: eps must be positive and finite", what);
  DeviceInfo di;
  if ((st = device_info(&di)) != CC_OK) return st;
  RowArgs a = {};
  a.x = reinterpret_cast<const uint4*>(x);
  a.gamma = reinterpret_cast<const uint4*>(gamma);
  a.y = y;
  a.scales = scales;
  a.rows = rows;
  a.ld_x = ld_x / 8;
  a.vecs = c / 8;
  a.blocks = (c + kScaleBlock - 1) / kScaleBlock;
  a.inv_c = 1.f / static_cast<float>(c);
  a.eps = eps;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (!norm) return launch_rows<false, false, true>(what, a, di.sm_count, cs);
  if (scales)
    return act == CC_ACT_SILU ? launch_rows<true, true, true>(what, a, di.sm_count, cs)
                              : launch_rows<true, false, true>(what, a, di.sm_count, cs);
  return act == CC_ACT_SILU ? launch_rows<true, true, false>(what, a, di.sm_count, cs)
                            : launch_rows<true, false, false>(what, a, di.sm_count, cs);
}

// One CTA per 128 x 128 block of the weights: the block's largest |w|, then
// its e4m3 values, out of a second reading that finds the block in L1 or L2. Run
// once per layer when weights are loaded: 4096 x 4096 in 7.3 us, 16384 x 16384
// in 164 (119 at the copy rate).
__global__ void __launch_bounds__(256) fp8_weights_kernel(const uint4* __restrict__ w, uint2* __restrict__ wq,
                                                          float* __restrict__ sw, int n, int kv, int kblocks) {
  __shared__ float red[8];
  const int tid = threadIdx.x;
  const int v = blockIdx.x * 16 + (tid & 15);
  const int row0 = blockIdx.y * kScaleBlock + (tid >> 4);
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    if (row < n && v < kv) m = max_nan(m, absmax8(unpack8(w[static_cast<long long>(row) * kv + v])));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, red[i]);
  const float scale = block_scale(m);
  const float inv = 1.f / scale;
  if (tid == 0) sw[static_cast<long long>(blockIdx.y) * kblocks + blockIdx.x] = scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    if (row < n && v < kv) {
      Vec8 f = unpack8(w[static_cast<long long>(row) * kv + v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) f.p[e] = mul2(f.p[e], pair(inv, inv));
      wq[static_cast<long long>(row) * kv + v] = pack8_e4m3(f);
    }
  }
}

}  // namespace
}  // namespace cc

using namespace cc;

extern "C" cc_status cc_rms_norm_act(const cc_bf16* x, const cc_bf16* gamma, cc_bf16* y, int rows, int c,
                                     int64_t ld_x, float eps, int act, void* stream) {
  return run_rows("rms_norm_act", true, x, gamma, y, nullptr, rows, c, ld_x, eps, act, stream);
}

extern "C" cc_status cc_rms_norm_act_fp8(const cc_bf16* x, const cc_bf16* gamma, cc_fp8* y, float* scales, int rows,
                                         int c, int64_t ld_x, float eps, int act, void* stream) {
  cc_status st;
  if (empty_request("rms_norm_act_fp8", {rows}, &st)) return st;
  if (!scales) return fail(CC_ERR_INVALID, "rms_norm_act_fp8: null pointer");
  return run_rows("rms_norm_act_fp8", true, x, gamma, y, scales, rows, c, ld_x, eps, act, stream);
}

extern "C" cc_status cc_fp8_quantize(const cc_bf16* x, cc_fp8* y, float* scales, int rows, int c, int64_t ld_x,
                                     void* stream) {
  cc_status st;
  if (empty_request("fp8_quantize", {rows}, &st)) return st;
  if (!scales) return fail(CC_ERR_INVALID, "fp8_quantize: null pointer");
  return run_rows("fp8_quantize", false, x, nullptr, y, scales, rows, c, ld_x, 1.f, CC_ACT_NONE, stream);
}

extern "C" cc_status cc_gemm_fp8_prepare(const cc_bf16* w, cc_fp8* wq, float* sw, int n, int k, void* stream) {
  if (!w || !wq || !sw) return fail(CC_ERR_INVALID, "gemm_fp8_prepare: null pointer");
  if (!aligned16(w) || !aligned16(wq) || !aligned16(sw))
    return fail(CC_ERR_INVALID, "gemm_fp8_prepare: pointers must be 16-byte aligned");
  if (n <= 0 || k <= 0) return fail(CC_ERR_INVALID, "gemm_fp8_prepare: sizes must be positive");
  if (k % 16 != 0) return fail(CC_ERR_UNSUPPORTED, "gemm_fp8_prepare: K must be a multiple of 16 (got %d)", k);
  const int nb = (n - 1) / kScaleBlock + 1, kb = (k - 1) / kScaleBlock + 1;
  if (nb > 65535 || k > (1 << 24))
    return fail(CC_ERR_UNSUPPORTED, "gemm_fp8_prepare: N must be at most %d and K %d", 65535 * kScaleBlock, 1 << 24);
  DeviceInfo di;
  cc_status st = device_info(&di);
  if (st != CC_OK) return st;
  fp8_weights_kernel<<<dim3(kb, nb), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      reinterpret_cast<const uint4*>(w), reinterpret_cast<uint2*>(wq), sw, n, k / 8, kb);
  return launch_status("gemm_fp8_prepare");
}
