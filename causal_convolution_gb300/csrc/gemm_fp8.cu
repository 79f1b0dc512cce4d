// The 1x1x1 product in 8 bits: e4m3 rows times e4m3 weights with a scale per
// 128 channels of K on both sides, fp32 accumulation, bias, residual.
//
// The tensor core sums the products of one block of 128 channels (four
// kind::f8f6f4 MMAs) into tensor memory; the two scales of the block differ
// from row to row and block to block, so the sum leaves tensor memory before
// the next block's is added: each epilogue thread owns a row, reads its sums
// and adds them, times sa[row][block] * sw[column block][block], to fp32
// accumulators in its registers. Two accumulator buffers in tensor memory let
// the MMAs of one block run while the previous one is read.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cc.h"
#include "cc_host.h"
#include "cc_ptx.cuh"
#include "cc_rows.cuh"

namespace cc {
namespace {

struct Fp8GemmArgs {
  const float* sa;
  const float* sw;
  const uint4* bias;
  const cc_bf16* res;
  cc_bf16* out;
  int m, n, kblocks;
  long long ld_res, ld_out;
  unsigned int* err;
  unsigned long long timeout_ns;
};

constexpr int kTile = 128;
constexpr int kStageBytes = 2 * kTile * kTile;
constexpr int kStages = 6;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 256;
constexpr int kThreads = 192;

__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ Fp8GemmArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int m0 = blockIdx.y * kTile;
  const int n0 = blockIdx.x * kTile;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 4);
    }
    mbar_init(smem_u32(done), 1);
    fence_mbar_init();
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 2 * kTile);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t tlim = args.timeout_ns;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = 0; kb < args.kblocks; ++kb) {
        if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, args.err, tlim)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&full[stage]);
        const uint32_t dst = smem_u32(smem + stage * kStageBytes);
        mbar_arrive_expect_tx(fb, kStageBytes);
        tma_load_2d(dst, &tmA, fb, kb * kTile, m0);
        tma_load_2d(dst + kTile * kTile, &tmB, fb, kb * kTile, n0);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        // copies already issued land before the CTA can exit
        for (int s = 0; s < kStages; ++s)
          (void)mbar_wait(smem_u32(&full[s]), (s < stage) ? phase : (phase ^ 1u), args.err, 200000000ull);
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_e4m3_f32(kTile, kTile);
    int stage = 0;
    uint32_t phase = 0;
    const uint64_t a_desc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t b_desc0 = sdesc_sw128(smem_u32(smem + kTile * kTile), 16, 1024);
    for (int kb = 0; kb < args.kblocks; ++kb) {
      const int acc = kb & 1;
      if (!__all_sync(0xffffffffu,
                      mbar_wait(smem_u32(&tempty[acc]), ((kb >> 1) & 1) ^ 1u, args.err, tlim) &&
                          mbar_wait(smem_u32(&full[stage]), phase, args.err, tlim)))
        break;
      tc_fence_after();
      const uint64_t off = static_cast<uint64_t>(stage) * (kStageBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8(tmem_base + acc * kTile, a_desc0 + off + 2 * k, b_desc0 + off + 2 * k, idesc, k != 0 ? 1u : 0u);
        mma_commit(smem_u32(&empty[stage]));
        mma_commit(smem_u32(&tfull[acc]));
      }
      __syncwarp();
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // no MMA may still be running when tensor memory is released
    if (elect_one()) mma_commit(smem_u32(done));
    __syncwarp();
    (void)mbar_wait(smem_u32(done), 0, args.err, tlim);
  } else {
    const int quarter = warp & 3;
    const int m = m0 + quarter * 32 + lane;
    const bool row_ok = m < args.m;
    const float* sa = args.sa + static_cast<long long>(row_ok ? m : 0) * args.kblocks;
    const float* sw = args.sw + static_cast<long long>(blockIdx.x) * args.kblocks;
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    float acc[kTile];
#pragma unroll
    for (int j = 0; j < kTile; ++j) acc[j] = 0.f;
    bool ok = true;
    for (int kb = 0; kb < args.kblocks; ++kb) {
      const int buf = kb & 1;
      const float s = row_ok ? sa[kb] * sw[kb] : 0.f;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&tfull[buf]), (kb >> 1) & 1, args.err, tlim))) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kTile; c += 32) {
        uint32_t r[32];
        tmem_ld32_wait(tbase + buf * kTile + c, r);
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(__uint_as_float(r[j]), s, acc[c + j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tempty[buf]));
    }
    if (ok && row_ok) {
#pragma unroll
      for (int c = 0; c < kTile; c += 8) {
        const int n = n0 + c;
        if (n < args.n) {
          Vec8 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v.p[e] = pair(acc[c + 2 * e], acc[c + 2 * e + 1]);
          if (args.bias) {
            const Vec8 t = unpack8(args.bias[n >> 3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v.p[e] = add2(v.p[e], t.p[e]);
          }
          if (args.res) {
            const Vec8 t = unpack8(*reinterpret_cast<const uint4*>(args.res + m * args.ld_res + n));
#pragma unroll
            for (int e = 0; e < 4; ++e) v.p[e] = add2(v.p[e], t.p[e]);
          }
          *reinterpret_cast<uint4*>(args.out + m * args.ld_out + n) = pack8(v);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * kTile);
  }
}

}  // namespace
}  // namespace cc

using namespace cc;

extern "C" cc_status cc_gemm_fp8(const cc_fp8* a, const float* sa, const cc_fp8* wq, const float* sw,
                                 const cc_bf16* bias, const cc_bf16* res, cc_bf16* out, int m, int n, int k,
                                 int64_t ld_res, int64_t ld_out, void* stream) {
  const char* what = "gemm_fp8";
  cc_status st;
  if (empty_request(what, {m}, &st)) return st;
  if (!a || !sa || !wq || !sw || !out) return fail(CC_ERR_INVALID, "%s: null pointer", what);
  if (!aligned16(a) || !aligned16(sa) || !aligned16(wq) || !aligned16(sw) || !aligned16(bias) || !aligned16(res) ||
      !aligned16(out))
    return fail(CC_ERR_INVALID, "%s: pointers must be 16-byte aligned", what);
  if (n <= 0 || k <= 0) return fail(CC_ERR_INVALID, "%s: channel counts must be positive", what);
  if (k % 16 != 0) return fail(CC_ERR_UNSUPPORTED, "%s: K must be a multiple of 16 (got %d)", what, k);
  if (n % 8 != 0) return fail(CC_ERR_UNSUPPORTED, "%s: N must be a multiple of 8 (got %d)", what, n);
  if (ld_out < n || ld_out % 8 != 0 || (res && (ld_res < n || ld_res % 8 != 0)))
    return fail(CC_ERR_INVALID, "%s: ld_out and ld_res must be at least N and multiples of 8", what);
  const int m_tiles = (m - 1) / kTile + 1, n_tiles = (n - 1) / kTile + 1;
  if (m_tiles > 65535) return fail(CC_ERR_UNSUPPORTED, "%s: too many output tiles", what);
  DeviceInfo di;
  if ((st = device_info(&di)) != CC_OK) return st;
  CUtensorMap ta, tb;
  if ((st = encode_tiled_2d_u8(&ta, a, k, m, k, kTile, kTile)) != CC_OK) return st;
  if ((st = encode_tiled_2d_u8(&tb, wq, k, n, k, kTile, kTile)) != CC_OK) return st;
  Fp8GemmArgs args = {};
  args.sa = sa;
  args.sw = sw;
  args.bias = reinterpret_cast<const uint4*>(bias);
  args.res = res;
  args.out = out;
  args.m = m;
  args.n = n;
  args.kblocks = (k - 1) / kScaleBlock + 1;
  args.ld_res = ld_res;
  args.ld_out = ld_out;
  args.err = di.err_word;
  args.timeout_ns = kWaitLimitNs;
  cudaError_t e = cudaFuncSetAttribute(fp8_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: shared-memory attribute: %s", what, cudaGetErrorString(e));
  fp8_gemm_kernel<<<dim3(n_tiles, m_tiles), kThreads, kSmemBytes, static_cast<cudaStream_t>(stream)>>>(ta, tb, args);
  return launch_status(what);
}
