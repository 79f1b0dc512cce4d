// Attention with heads for few query rows to a sequence (single tokens, or a few,
// with the query heads of a group): up to 16 rows of a key head at a time. Each
// key and value is used for two products of 16 rows, so the cache's bytes bound
// it, and the kernel is built around reading them without a pause: warp 0 finds
// the CTA's run (cc_heads.cuh) and streams 64 keys and their values at a time with
// TMA, across the borders of items; warps 1-4 take 16 of the 64 keys each, with
// row statistics and a sum of their own, so that nothing but the tiles' arrival
// ties them together. Their sums are joined at an item's end. The products are
// m16n8k16 from registers: a 128-row tile of tcgen05 would be filled to an eighth
// or less, and its way through tensor memory is longer than a tile's reading.
// Weights are taken in two bf16 parts, which costs products that have time.
//
// Two CTAs to an SM, 96 KB of tiles in flight each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cc_heads.cuh"

namespace cc {
namespace {

constexpr int kFrThreads = 160;
constexpr int kFrKeys = 64;
constexpr int kFrBlock = kFrKeys * 128;  // bytes of 64 keys x 64 channels
constexpr float kFrRoom = 8.f;           // powers of two that weights may pass their row's scale by

__device__ __forceinline__ void ldsm4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}

template <int NB, int STAGES>
struct FrSmem {
  static constexpr int kTile = 2 * NB * kFrBlock;  // keys and values
  static constexpr int kSum = NB * 8 * 512;        // a warp's sums, as its lanes hold them
  static constexpr int kBytes = 1024 + STAGES * kTile + kSum + 2 * 4 * 16 * 4 + 512;
};

template <int NB, int STAGES>
__global__ void __launch_bounds__(kFrThreads, 2)
    attn_few_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ AhArgs a) {
  using Sm = FrSmem<NB, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* sSum = reinterpret_cast<float4*>(smem + STAGES * Sm::kTile);
  float* sC = reinterpret_cast<float*>(smem + STAGES * Sm::kTile + Sm::kSum);  // [4][16]
  float* sL = sC + 64;
  AhItem* items = reinterpret_cast<AhItem*>(sL + 64);
  uint64_t* full = reinterpret_cast<uint64_t*>(items + kAhItems);
  uint64_t* empty = full + STAGES;
  uint64_t* item_full = empty + STAGES;
  uint64_t* item_empty = item_full + kAhItems;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 4);
    }
    for (int i = 0; i < kAhItems; ++i) {
      mbar_init(smem_u32(&item_full[i]), 1);
      mbar_init(smem_u32(&item_empty[i]), 4);
    }
    fence_mbar_init();
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();

  int stage = 0, slot = 0;
  uint32_t ph = 0, it_ph = 0;
  if (warp == 0) {
    // -------------------------------------------- run, items and TMA loads --
    Run r;
    const bool any = find_run(a, blockIdx.x, gridDim.x, lane, r);
    bool ok = true;
    if (a.may_split && lane < 2) a.meta[2 * blockIdx.x + lane] = make_int4(0, 0, 0, 0);
    __syncwarp();
    if (any && !r.split && r.t > 0) {  // whole items: from the first one that starts in the run
      r.at += max(1, r.tiles) - r.t;
      next_item(a, r);
    }
    while (ok) {
      const bool more = any && r.at < r.end && r.b < a.plan.seqs;
      ok = warp_wait(&item_empty[slot], it_ph ^ 1u, a);
      if (!ok) break;
      AhItem it = {};
      it.last = !more;
      if (more) it = make_item(a, r, lane);
      if (lane == 0) {
        items[slot] = it;
        mbar_arrive(smem_u32(&item_full[slot]));
      }
      __syncwarp();
      if (++slot == kAhItems) {
        slot = 0;
        it_ph ^= 1u;
      }
      if (!more) break;
      for (int t = it.t_begin; t < it.t_end; ++t) {
        const int boxes = (min(kFrKeys, it.len - t * kFrKeys) + a.box - 1) / a.box;
        int page = it.seq, at = t * kFrKeys + lane * a.box;
        if (lane < boxes && a.plan.page_table) {
          const int n = at / a.plan.page_size;
          at -= n * a.plan.page_size;
          page = a.plan.page_table[static_cast<long long>(it.seq) * a.plan.max_pages + n];
          if (page < 0 || page >= a.plan.pages) {
            atomicOr(a.err, DEVERR_BOUNDS);
            page = a.plan.pages;  // out of the map's range: the box reads as zeros
          }
        }
        ok = warp_wait(&empty[stage], ph ^ 1u, a);
        if (!ok) break;
        const uint32_t bar = smem_u32(&full[stage]);
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * a.box * 128 * 2 * NB));
        __syncwarp();
        if (lane < boxes) {
          const uint32_t dst = smem_u32(smem + stage * Sm::kTile) + static_cast<uint32_t>(lane * a.box) * 128u;
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            tma_load_4d(dst + i * kFrBlock, &tmK, bar, i * 64, it.head, at, page);
            tma_load_4d(dst + (NB + i) * kFrBlock, &tmV, bar, i * 64, it.head, at, page);
          }
        }
        if (++stage == STAGES) {
          stage = 0;
          ph ^= 1u;
        }
      }
      r.at += static_cast<unsigned>(max(1, it.t_end - it.t_begin));
      next_item(a, r);
    }
    if (!ok) {  // copies in flight land before the CTA goes
      for (int i = 0; i < STAGES; ++i)
        (void)mbar_wait(smem_u32(&full[i]), (i < stage) ? ph : (ph ^ 1u), a.err, 200000000ull);
    }
  } else {
    const int w = warp - 1;
    const int steps = a.d / 16;
    const int kb = w * 16;  // this warp's keys of a tile
    // ldmatrix addresses within a tile: keys as rows of the second factor of q k^T, values transposed as that of P v
    const int k_row = kb + (lane >> 4) * 8 + (lane & 7), k_chunk = lane >> 3 & 1;
    const int v_row = kb + (lane >> 3 & 1) * 8 + (lane & 7), v_chunk = lane >> 4;
    bool ok = true;
    while (true) {
      // A warp whose wait ran out goes through the rest of its item without waiting, as the others count on it at
      // the barriers, and all four leave together here.
      if (!named_barrier_and(1, 128, ok && warp_wait(&item_full[slot], it_ph, a))) break;
      const AhItem it = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&item_empty[slot]));
      if (++slot == kAhItems) {
        slot = 0;
        it_ph ^= 1u;
      }
      if (it.last) break;
      const int n = it.t_end - it.t_begin;
      const int rows = it.tokens * a.group;
      // rows lane / 4 and + 8 of the item
      int limit[2];
      long long at_q[2], at_o[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 2) + 8 * i, tok = static_cast<int>(quotient(r, a.inv_group)), h = it.head * a.group + r - tok * a.group;
        limit[i] = r < rows ? key_limit(a, it.fresh, it.len, it.first + tok) : 0;
        at_q[i] = (it.q_row + tok) * a.ld_q + static_cast<long long>(h) * a.d;
        at_o[i] = (it.q_row + tok) * a.ld_o + static_cast<long long>(h) * a.d;
      }
      const bool in[2] = {(lane >> 2) < rows, (lane >> 2) + 8 < rows};
      uint32_t qf[NB * 4][4];
#pragma unroll
      for (int k = 0; k < NB * 4; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i & 1;
          qf[k][i] = k < steps && in[r]
                         ? *reinterpret_cast<const uint32_t*>(a.q + at_q[r] + k * 16 + (i >> 1) * 8 + (lane & 3) * 2)
                         : 0u;
        }
      }
      float acc[NB * 8][4];
#pragma unroll
      for (int j = 0; j < NB * 8; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
      }
      float c[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
      for (int t = it.t_begin; t < it.t_end; ++t) {
        ok = ok && warp_wait(&full[stage], ph, a);
        uint8_t* tile = smem + stage * Sm::kTile;
        const int valid = it.len - t * kFrKeys - kb;  // of this warp's keys
        if (valid < 16) {
          // values behind the sequence's end count 0 times, but 0 * NaN is NaN: they become zeros
          for (int i = max(valid, 0) * 8 + lane; i < 128; i += 32) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
              *reinterpret_cast<uint4*>(tile + (NB + b) * kFrBlock + kb * 128 + i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (valid > 0) {
          const uint32_t kt = smem_u32(tile) + k_row * 128, vt = smem_u32(tile) + NB * kFrBlock + v_row * 128;
          float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int k = 0; k < NB * 4; ++k) {
            if (k < steps) {
              uint32_t b[4];
              ldsm4(kt + (k >> 2) * kFrBlock + ((((k & 3) * 2 + k_chunk) ^ (k_row & 7)) << 4), b);
              mma16816(sc[0], qf[k], b[0], b[1]);
              mma16816(sc[1], qf[k], b[2], b[3]);
            }
          }
          // scores of keys 8 * j + 2 * (lane % 4) + {0, 1}, rows lane / 4 (0, 1) and + 8 (2, 3)
          const int lim0 = limit[0] - t * kFrKeys - kb, lim1 = limit[1] - t * kFrKeys - kb;
          float m[2] = {kNegInf, kNegInf};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = j * 8 + (lane & 3) * 2 + (i & 1);
              sc[j][i] = key < (i < 2 ? lim0 : lim1) ? sc[j][i] * a.kx : kNegInf;
              m[i >> 1] = fmaxf(m[i >> 1], sc[j][i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
            m[i] = ceilf(fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2)));
            m[i] = m[i] > c[i] + (c[i] == kNegInf ? 0.f : kFrRoom) ? m[i] : c[i];
          }
          if (__any_sync(0xffffffffu, m[0] != c[0] || m[1] != c[1])) {
            const float f0 = pow2_diff(c[0], m[0]), f1 = pow2_diff(c[1], m[1]);
#pragma unroll
            for (int j = 0; j < NB * 8; ++j) acc[j][0] *= f0, acc[j][1] *= f0, acc[j][2] *= f1, acc[j][3] *= f1;
            l[0] *= f0, l[1] *= f1;
            c[0] = m[0], c[1] = m[1];
          }
          const float b0 = c[0] == kNegInf ? 0.f : c[0], b1 = c[1] == kNegInf ? 0.f : c[1];
          uint32_t hi[4], lo_[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float p0 = ex2_approx(sc[j][2 * i] - (i ? b1 : b0)), p1 = ex2_approx(sc[j][2 * i + 1] - (i ? b1 : b0));
              l[i] += p0 + p1;
              const uint32_t h = pack_bf16(p0, p1);
              hi[2 * j + i] = h;
              lo_[2 * j + i] = pack_bf16(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u));
            }
          }
#pragma unroll
          for (int j = 0; j < NB * 4; ++j) {
            if (j < steps) {
              uint32_t b[4];
              ldsm4_trans(vt + (j >> 2) * kFrBlock + ((((j & 3) * 2 + v_chunk) ^ (v_row & 7)) << 4), b);
              mma16816(acc[2 * j], hi, b[0], b[1]);
              mma16816(acc[2 * j + 1], hi, b[2], b[3]);
              mma16816(acc[2 * j], lo_, b[0], b[1]);
              mma16816(acc[2 * j + 1], lo_, b[2], b[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&empty[stage]));
        if (++stage == STAGES) {
          stage = 0;
          ph ^= 1u;
        }
      }
      // the four warps' sums on one scale
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if ((lane & 3) == 0) {
          sC[w * 16 + (lane >> 2) + 8 * i] = c[i];
          sL[w * 16 + (lane >> 2) + 8 * i] = l[i];
        }
      }
      named_barrier_sync(1, 128);
      float top[2] = {kNegInf, kNegInf}, sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 2) + 8 * i;
#pragma unroll
        for (int j = 0; j < 4; ++j) top[i] = fmaxf(top[i], sC[j * 16 + r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i] = fmaf(sL[j * 16 + r], pow2_diff(sC[j * 16 + r], top[i]), sum[i]);
      }
      const float f0 = pow2_diff(c[0], top[0]), f1 = pow2_diff(c[1], top[1]);
#pragma unroll
      for (int j = 0; j < NB * 8; ++j) acc[j][0] *= f0, acc[j][1] *= f0, acc[j][2] *= f1, acc[j][3] *= f1;
      // a quarter of the channels at a time; each warp adds up and writes one
      constexpr int Q = NB * 2;
      float4 res[Q];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int j = 0; j < Q; ++j)
          sSum[(w * Q + j) * 32 + lane] =
              make_float4(acc[q * Q + j][0], acc[q * Q + j][1], acc[q * Q + j][2], acc[q * Q + j][3]);
        named_barrier_sync(1, 128);
        if (w == q) {
#pragma unroll
          for (int j = 0; j < Q; ++j) {
            float4 v = sSum[j * 32 + lane];
#pragma unroll
            for (int from = 1; from < 4; ++from) {
              const float4 x = sSum[(from * Q + j) * 32 + lane];
              v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
            res[j] = v;
          }
        }
        named_barrier_sync(1, 128);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!in[i]) continue;
        const bool sees = n > 0 && limit[i] > 0;
        const float inv = 1.f / sum[i];
        const long long at = static_cast<long long>(it.slot) * a.slot_rows + (lane >> 2) + 8 * i;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
          const int col = (w * Q + j) * 8 + (lane & 3) * 2;
          const float x0 = i ? res[j].z : res[j].x, x1 = i ? res[j].w : res[j].y;
          if (col >= a.d) break;
          if (it.slot < 0)
            *reinterpret_cast<uint32_t*>(a.o + at_o[i] + col) = sees ? pack_bf16(x0 * inv, x1 * inv) : 0u;
          else
            *reinterpret_cast<float2*>(a.part + at * a.d + col) = make_float2(x0, x1);
        }
        if (it.slot >= 0 && w == 0 && (lane & 3) == 0) {
          const bool any = limit[i] > it.t_begin * kFrKeys;
          a.part_cl[at] = make_float2(any && top[i] == kNegInf ? kNoScore : top[i], sum[i]);
        }
      }
    }
  }
}

template <int NB, int STAGES>
cc_status launch(const char* what, const CUtensorMap& tk, const CUtensorMap& tv, AhArgs& a, int grid,
                 cudaStream_t stream) {
  auto kern = attn_few_rows_kernel<NB, STAGES>;
  constexpr int kSmem = FrSmem<NB, STAGES>::kBytes;
  static_assert(kSmem <= 115712, "two CTAs to an SM");
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kSmem, a.device, ready);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: shared-memory attribute: %s", what, cudaGetErrorString(e));
  e = launch_pdl(kern, dim3(grid), dim3(kFrThreads), kSmem, stream, tk, tv, a);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: launch: %s", what, cudaGetErrorString(e));
  return launch_status(what);
}

}  // namespace

cc_status launch_few_rows(const char* what, const CUtensorMap& tk, const CUtensorMap& tv, AhArgs& a, int grid,
                          cudaStream_t stream) {
  return a.d > 64 ? launch<2, 3>(what, tk, tv, a, grid, stream) : launch<1, 6>(what, tk, tv, a, grid, stream);
}

}  // namespace cc
