// Attention with heads for few query rows to a sequence (single tokens, or a few,
// with the query heads of a group): up to 8 rows of a key head at a time. Each key
// and value is used for two products with those rows, so the cache's bytes bound
// it, and the kernel is built around reading them without a pause: warp 0 finds
// the CTA's run (cc_heads.cuh) and streams a tile of keys and their values at a
// time with TMA, across the borders of items; warps 1-4 take a quarter of it each, with
// row statistics and a sum of their own, so that nothing but the tiles' arrival
// ties them together. Their sums are joined at an item's end.
//
// The products are m16n8k16 from registers, keys (for k q^T) and channels (for
// v^T p) along m and the rows along n: a 128-row tile of tcgen05 would be filled
// to a sixteenth or less, and its way through tensor memory takes longer than a
// tile's reading. Weights are taken in two bf16 parts, which costs products that
// have time (results are then off from 64 bits by 0.0015 to 0.0017, L2, relative:
// their own rounding).
//
// Two CTAs to an SM, 96 KB of tiles in flight each; a tile is 64 keys of 65 to
// 128 channels or 128 of up to 64 (so that waits and maxima come half as often
// there: 64 streams over 4096 keys of 8 heads of 64 channels 137 -> 121 us, of 32
// 108 -> 82; 94 and 60 since L2 fetches no more than a head's row). Measured:
// single tokens of 64 streams, 100 to 8192 keys each, 32 heads over 8 of 128
// channels: 180 us, 6.0 TB/s or 0.91 of a copy's rate, pages of 16 or 128 alike;
// with the rows along m (16 at least, the keys along n) it was 192.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cc_heads.cuh"

namespace cc {
namespace {

constexpr int kFrThreads = 160;
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

// An 8 x 8 matrix of bf16, two of a row to a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// NB: 64-channel blocks of a head; KG: groups of 16 keys that a warp takes of a tile; STAGES: tiles in flight.
template <int NB, int KG, int STAGES>
struct FrSmem {
  static constexpr int kKeys = 64 * KG;
  static constexpr int kBlock = kKeys * 128;     // bytes of a tile's keys x 64 channels
  static constexpr int kTile = 2 * NB * kBlock;  // keys and values
  static constexpr int kSum = 4 * 3 * NB * 512;    // quarters of sums on their way to the warps that add them up
  static constexpr int kBytes = 1024 + STAGES * kTile + kSum + 4 * 8 * 8 + 512;
};

template <int NB, int KG, int STAGES>
__global__ void __launch_bounds__(kFrThreads, 2)
    attn_few_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ AhArgs a) {
  using Sm = FrSmem<NB, KG, STAGES>;
  constexpr int kKeys = Sm::kKeys, kBlock = Sm::kBlock, kMine = 16 * KG;  // kMine: a warp's keys of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* sSum = reinterpret_cast<float4*>(smem + STAGES * Sm::kTile);
  float2* sCL = reinterpret_cast<float2*>(smem + STAGES * Sm::kTile + Sm::kSum);  // [4][8] (c, l)
  AhItem* items = reinterpret_cast<AhItem*>(sCL + 32);
  uint64_t* full = reinterpret_cast<uint64_t*>(items + kAhItems);
  uint64_t* empty = full + STAGES;
  uint64_t* item_full = empty + STAGES;
  uint64_t* item_empty = item_full + kAhItems;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    if (a.plan.page_size > 0) {  // there are keys, and maps of them
      tma_prefetch_map(&tmK);
      tma_prefetch_map(&tmV);
    }
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
        const int boxes = (min(kKeys, it.len - t * kKeys) + a.box - 1) / a.box;
        int page = it.seq, at = t * kKeys + lane * a.box;
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
            tma_load_4d(dst + i * kBlock, &tmK, bar, i * 64, it.head, at, page);
            tma_load_4d(dst + (NB + i) * kBlock, &tmV, bar, i * 64, it.head, at, page);
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
#pragma unroll 1
      for (int i = 0; i < STAGES; ++i)
        (void)mbar_wait(smem_u32(&full[i]), (i < stage) ? ph : (ph ^ 1u), a.err, 200000000ull);
    }
  } else {
    const int w = warp - 1;
    const int steps = a.d / 16;
    const int kb = w * kMine;  // this warp's keys of a tile
    // ldmatrix addresses within a tile: 16 keys x 16 channels as they are, and values transposed
    const int k_row = kb + (lane >> 3 & 1) * 8 + (lane & 7), k_chunk = lane >> 4;
    const int v_row = kb + (lane >> 4) * 8 + (lane & 7), v_chunk = lane >> 3 & 1;
    const int col = (lane & 3) * 2;  // rows col and col + 1 of the item are this lane's columns of scores and sums
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
      // row lane / 4 is the one whose query this lane holds, two channels of eight
      const int my_row = lane >> 2, my_tok = static_cast<int>(quotient(my_row, a.inv_group));
      const int my_head = it.head * a.group + my_row - my_tok * a.group;
      uint32_t qf[NB * 4][2];
      {
        const __nv_bfloat16* q =
            a.q + (it.q_row + my_tok) * a.ld_q + static_cast<long long>(my_head) * a.d + (lane & 3) * 2;
#pragma unroll
        for (int k = 0; k < NB * 4; ++k) {
          const bool on = k < steps && my_row < rows;
          qf[k][0] = on ? *reinterpret_cast<const uint32_t*>(q + k * 16) : 0u;
          qf[k][1] = on ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8) : 0u;
        }
      }
      int limit[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = static_cast<int>(quotient(col + i, a.inv_group));
        limit[i] = col + i < rows ? key_limit(a, it.fresh, it.len, it.first + tok) : 0;
      }
      float acc[NB * 4][4];  // channels 16 j + lane / 4 (0, 1) and + 8 (2, 3) of rows col and col + 1
#pragma unroll
      for (int j = 0; j < NB * 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
      float c[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
      for (int t = it.t_begin; t < it.t_end; ++t) {
        ok = ok && warp_wait(&full[stage], ph, a);
        uint8_t* tile = smem + stage * Sm::kTile;
        const int valid = it.len - t * kKeys - kb;  // of this warp's keys
        if (valid < kMine) {
          // values behind the sequence's end count 0 times, but 0 * NaN is NaN: they become zeros
          for (int i = max(valid, 0) * 8 + lane; i < 8 * kMine; i += 32) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
              *reinterpret_cast<uint4*>(tile + (NB + b) * kBlock + kb * 128 + i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (valid > 0) {
          const uint32_t kt = smem_u32(tile) + k_row * 128, vt = smem_u32(tile) + NB * kBlock + v_row * 128;
          // scores of each group's keys lane / 4 (0, 1) and + 8 (2, 3) and rows col, col + 1; two chains of products
          float s0[KG][4], s1[KG][4];
#pragma unroll
          for (int g = 0; g < KG; ++g) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s0[g][i] = s1[g][i] = 0.f;
          }
#pragma unroll
          for (int k = 0; k < NB * 4; ++k) {
            if (k < steps) {
#pragma unroll
              for (int g = 0; g < KG; ++g) {
                uint32_t x[4];
                ldsm4(kt + g * 2048 + (k >> 2) * kBlock + ((((k & 3) * 2 + k_chunk) ^ (k_row & 7)) << 4), x);
                mma16816(k & 1 ? s1[g] : s0[g], x, qf[k][0], qf[k][1]);
              }
            }
          }
          float m[2] = {kNegInf, kNegInf};
#pragma unroll
          for (int g = 0; g < KG; ++g) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = t * kKeys + kb + g * 16 + (lane >> 2) + (i >> 1) * 8;
              s0[g][i] = key < limit[i & 1] ? (s0[g][i] + s1[g][i]) * a.kx : kNegInf;
              m[i & 1] = fmaxf(m[i & 1], s0[g][i]);
            }
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
            m[1] = fmaxf(m[1], __shfl_xor_sync(0xffffffffu, m[1], o));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            m[i] = ceilf(m[i]);
            m[i] = m[i] > c[i] + kFrRoom ? m[i] : c[i];
          }
          if (__any_sync(0xffffffffu, m[0] != c[0] || m[1] != c[1])) {
            const float f0 = pow2_diff(c[0], m[0]), f1 = pow2_diff(c[1], m[1]);
#pragma unroll
            for (int j = 0; j < NB * 4; ++j) acc[j][0] *= f0, acc[j][1] *= f1, acc[j][2] *= f0, acc[j][3] *= f1;
            l[0] *= f0, l[1] *= f1;
            c[0] = m[0], c[1] = m[1];
          }
          // weights, and what their rounding leaves, turned into the second factor of v^T p
          uint32_t hi[KG][2], rest[KG][2];
#pragma unroll
          for (int g = 0; g < KG; ++g) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float p0 = ex2_approx(s0[g][2 * i] - (c[0] == kNegInf ? 0.f : c[0]));
              const float p1 = ex2_approx(s0[g][2 * i + 1] - (c[1] == kNegInf ? 0.f : c[1]));
              l[0] += p0;
              l[1] += p1;
              const uint32_t h = pack_bf16(p0, p1);
              rest[g][i] = transpose8(pack_bf16(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u)));
              hi[g][i] = transpose8(h);
            }
          }
#pragma unroll
          for (int j = 0; j < NB * 4; ++j) {
            if (j < steps) {
#pragma unroll
              for (int g = 0; g < KG; ++g) {
                uint32_t x[4];
                ldsm4_trans(vt + g * 2048 + (j >> 2) * kBlock + ((((j & 3) * 2 + v_chunk) ^ (v_row & 7)) << 4), x);
                mma16816(acc[j], x, hi[g][0], hi[g][1]);
                mma16816(acc[j], x, rest[g][0], rest[g][1]);
              }
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
      for (int o = 4; o < 32; o <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
      }
      if (lane < 4) {
        sCL[w * 8 + col] = make_float2(c[0], l[0]);
        sCL[w * 8 + col + 1] = make_float2(c[1], l[1]);
      }
      named_barrier_sync(1, 128);
      float top[2] = {kNegInf, kNegInf}, sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 cl[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) cl[j] = sCL[j * 8 + col + i];
        top[i] = fmaxf(fmaxf(cl[0].x, cl[1].x), fmaxf(cl[2].x, cl[3].x));
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i] = fmaf(cl[j].y, pow2_diff(cl[j].x, top[i]), sum[i]);
      }
      const float f0 = pow2_diff(c[0], top[0]), f1 = pow2_diff(c[1], top[1]);
      // each warp adds up and writes a quarter of the channels; the others' shares come through shared memory
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q == w) continue;
#pragma unroll
        for (int j = 0; j < NB; ++j)
          sSum[((q * 3 + (w < q ? w : w - 1)) * NB + j) * 32 + lane] =
              make_float4(acc[q * NB + j][0] * f0, acc[q * NB + j][1] * f1, acc[q * NB + j][2] * f0, acc[q * NB + j][3] * f1);
      }
      named_barrier_sync(1, 128);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q == w) v = make_float4(acc[q * NB + j][0] * f0, acc[q * NB + j][1] * f1, acc[q * NB + j][2] * f0, acc[q * NB + j][3] * f1);
        }
#pragma unroll
        for (int from = 0; from < 3; ++from) {
          const float4 x = sSum[((w * 3 + from) * NB + j) * 32 + lane];
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        const int ch = (w * NB + j) * 16;
        if (ch >= a.d) break;
        if (it.slot < 0) {
          const bool sees0 = n > 0 && limit[0] > 0, sees1 = n > 0 && limit[1] > 0;
          const float inv0 = 1.f / sum[0], inv1 = 1.f / sum[1];
          const uint32_t x0 = transpose8(pack_bf16(sees0 ? v.x * inv0 : 0.f, sees1 ? v.y * inv1 : 0.f));
          const uint32_t x1 = transpose8(pack_bf16(sees0 ? v.z * inv0 : 0.f, sees1 ? v.w * inv1 : 0.f));
          if (my_row < rows) {
            __nv_bfloat16* o =
                a.o + (it.q_row + my_tok) * a.ld_o + static_cast<long long>(my_head) * a.d + ch + (lane & 3) * 2;
            *reinterpret_cast<uint32_t*>(o) = x0;
            *reinterpret_cast<uint32_t*>(o + 8) = x1;
          }
        } else {
          float* part = a.part + (static_cast<long long>(it.slot) * a.slot_rows + col) * a.d + ch + (lane >> 2);
          if (col < rows) part[0] = v.x, part[8] = v.z;
          if (col + 1 < rows) part[a.d] = v.y, part[a.d + 8] = v.w;
        }
      }
      if (it.slot >= 0 && w == 0 && lane < 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool any = limit[i] > it.t_begin * kKeys;
          if (col + i < rows)
            a.part_cl[static_cast<long long>(it.slot) * a.slot_rows + col + i] =
                make_float2(any && top[i] == kNegInf ? kNoScore : top[i], sum[i]);
        }
      }
    }
  }
}

template <int NB, int KG, int STAGES>
cc_status launch(const char* what, const CUtensorMap& tk, const CUtensorMap& tv, AhArgs& a, int grid,
                 cudaStream_t stream) {
  auto kern = attn_few_rows_kernel<NB, KG, STAGES>;
  constexpr int kSmem = FrSmem<NB, KG, STAGES>::kBytes;
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
  return a.d > 64 ? launch<2, 1, 3>(what, tk, tv, a, grid, stream) : launch<1, 2, 3>(what, tk, tv, a, grid, stream);
}

}  // namespace cc
