// The 1x1x1 product in 8 bits: e4m3 rows times e4m3 weights with a scale per
// 128 channels of K on both sides, fp32 accumulation, bias, residual.
//
// The tensor core sums the products of one block of 128 channels (four
// kind::f8f6f4 MMAs) into tensor memory; the two scales of the block differ
// from row to row and block to block, so the sum leaves tensor memory before
// the next block's is added: each epilogue thread owns a row, reads its sums
// and adds them, times sa[row][block] * sw[column block][block], to fp32
// accumulators in its registers.
//
// Two kernels: CTA pairs with tiles of 256 rows for many rows, and, for few, the
// weights as the tensor core's 128-row side with K split over a cluster.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cc.h"
#include "cc_fp8_shares.h"
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
  int n_tiles, tiles;   // pair kernel
  int kb_split;         // blocks of K per CTA (few rows) or pair (split tiles)
  long long ld_res, ld_out;
  unsigned int* err;
  unsigned long long timeout_ns;
};

// Tile coordinates stay in 32 bits.
constexpr int kMaxRows = 0x7fffffff - 1024;
constexpr int kMaxChannels = 1 << 24;

constexpr int kMaxSmem = 232448;
constexpr int kKBytes = 128;  // bytes of K per stage: one scale block, one swizzle row

// ------------------------------------------------------- CTA pairs, many rows --

// Persistent pairs on tiles of 256 rows (128 of a per CTA) x 256 columns, or x
// 128 where that fills the last round of tiles better. An accumulator holds 128
// columns, one scale block of the weights; the one or two of a tile have four or
// two buffers each in tensor memory (512 columns, all of it), so that the MMAs
// of one run while another is read. An epilogue thread keeps half of the tile's
// columns of its row in registers: with 256 columns half of the register file,
// and eight warps with 128 columns each measured faster than sixteen with 64.
//
// What bounds it: the epilogue. A block of K takes the tensor core 512 cycles,
// and a warp about 620 to read and add its 128 columns (two trips to tensor
// memory, 64 paired multiply-adds that the two warps of a scheduler share, and
// what the loop around them costs); a tile's end takes 2000 more, of which the
// accumulators in reserve hide two blocks. Measured: 16384 x 4096 x 4096 in 180
// us in the first milliseconds (3.0 PFLOP/s; 139 us with the epilogue left out)
// and in 205 once the power limit holds the clock at 1.7 GHz, 13728 x 1024 x 1024
// with bias and residual 19.5 us (16.8 where part of it comes out of L2; without the
// residual 16.8 and 15.4), 439296 x 256 x 512 79 us (5.7 TB/s). A block of K of
// the narrow tile takes 480 cycles of 384 that its 24 KB a CTA take to arrive.
// (As two accumulators of 64 columns it took 580: an MMA with 64 columns takes as
// long as one with 128.)
//
// SPLITS: where there are few tiles, a cluster of two or four pairs takes a narrow
// one, each pair a run of blocks of K. The pairs' sums meet in shared memory and
// are added in the pairs' order, so results do not change from run to run.
constexpr int kPairRows = 128;     // of A, per CTA
constexpr int kAccCols = 128;      // of an accumulator; each CTA loads 64 of its weight rows
constexpr int kEpiWarps = 8;       // one per half of the tile's columns and quarter of the rows
constexpr int kPairThreads = 128 + 32 * kEpiWarps;  // a warpgroup to load and issue, two for the epilogue
// registers a thread: 128 * 72 + 256 * 216 = 384 * 168, what the launch has
constexpr int kIssueRegs = 72, kEpiRegs = 216;

// ACCS: accumulators side by side in a tile, one or two.
template <int ACCS>
struct PairShape {
  static constexpr int kCols = ACCS * kAccCols;
  static constexpr int kEpiCols = kCols / 2;     // of a warp
  static constexpr int kBufs = 512 / kCols;      // of an accumulator: all of tensor memory
  static constexpr int kABytes = kPairRows * kKBytes;
  static constexpr int kBBytes = kAccCols / 2 * kKBytes;  // of an accumulator's weights
  static constexpr int kStageBytes = kABytes + ACCS * kBBytes;
  static constexpr int kStages = ACCS == 2 ? 5 : 8;
  static constexpr int kPieceBytes = 32 * 64 * 2;  // a warp's 32 rows leave in pieces of 64 columns
  static constexpr int kPieces = kEpiCols / 64;
  static constexpr int kOutBytes = kPieces * kPieceBytes;
  static constexpr int kBarBytes = 320;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kEpiWarps * kOutBytes + kBarBytes;
  static_assert(kSmem <= kMaxSmem, "shared memory budget");
  static_assert((2 * kStages + 2 * ACCS * kBufs + kEpiWarps + 1) * 8 + 4 <= kBarBytes, "barriers");
};

// 64 sums of this thread's tensor memory lane, at %33 and on, into t0 .. t63;
// then each pair of them, times %34, added to the accumulators %0 .. %31.
#define CC_LOAD_SUMS \
  ".reg .b32 t<64>, a<4>;\n\t.reg .b64 p<32>;\n\t" \
  "add.u32 a0, %33, 0;\n\t" \
  "add.u32 a1, %33, 16;\n\t" \
  "add.u32 a2, %33, 32;\n\t" \
  "add.u32 a3, %33, 48;\n\t" \
  "tcgen05.ld.sync.aligned.32x32b.x16.b32 {t0, t1, t2, t3, t4, t5, t6, t7, " \
  "t8, t9, t10, t11, t12, t13, t14, t15}, [a0];\n\t" \
  "tcgen05.ld.sync.aligned.32x32b.x16.b32 {t16, t17, t18, t19, t20, t21, t22, t23, " \
  "t24, t25, t26, t27, t28, t29, t30, t31}, [a1];\n\t" \
  "tcgen05.ld.sync.aligned.32x32b.x16.b32 {t32, t33, t34, t35, t36, t37, t38, t39, " \
  "t40, t41, t42, t43, t44, t45, t46, t47}, [a2];\n\t" \
  "tcgen05.ld.sync.aligned.32x32b.x16.b32 {t48, t49, t50, t51, t52, t53, t54, t55, " \
  "t56, t57, t58, t59, t60, t61, t62, t63}, [a3];\n\t" \
  "tcgen05.wait::ld.sync.aligned;\n\t"
#define CC_ADD(k, lo, hi) \
  "mov.b64 p" #k ", {t" #lo ", t" #hi "};\n\tfma.rn.f32x2 %" #k ", p" #k ", %34, %" #k ";\n\t"
#define CC_ADD_SUMS \
  CC_ADD(0, 0, 1) CC_ADD(1, 2, 3) CC_ADD(2, 4, 5) CC_ADD(3, 6, 7) \
  CC_ADD(4, 8, 9) CC_ADD(5, 10, 11) CC_ADD(6, 12, 13) CC_ADD(7, 14, 15) \
  CC_ADD(8, 16, 17) CC_ADD(9, 18, 19) CC_ADD(10, 20, 21) CC_ADD(11, 22, 23) \
  CC_ADD(12, 24, 25) CC_ADD(13, 26, 27) CC_ADD(14, 28, 29) CC_ADD(15, 30, 31) \
  CC_ADD(16, 32, 33) CC_ADD(17, 34, 35) CC_ADD(18, 36, 37) CC_ADD(19, 38, 39) \
  CC_ADD(20, 40, 41) CC_ADD(21, 42, 43) CC_ADD(22, 44, 45) CC_ADD(23, 46, 47) \
  CC_ADD(24, 48, 49) CC_ADD(25, 50, 51) CC_ADD(26, 52, 53) CC_ADD(27, 54, 55) \
  CC_ADD(28, 56, 57) CC_ADD(29, 58, 59) CC_ADD(30, 60, 61) CC_ADD(31, 62, 63)
#define CC_ACCUMULATORS \
  "+l"(acc[0]), "+l"(acc[1]), "+l"(acc[2]), "+l"(acc[3]), \
  "+l"(acc[4]), "+l"(acc[5]), "+l"(acc[6]), "+l"(acc[7]), \
  "+l"(acc[8]), "+l"(acc[9]), "+l"(acc[10]), "+l"(acc[11]), \
  "+l"(acc[12]), "+l"(acc[13]), "+l"(acc[14]), "+l"(acc[15]), \
  "+l"(acc[16]), "+l"(acc[17]), "+l"(acc[18]), "+l"(acc[19]), \
  "+l"(acc[20]), "+l"(acc[21]), "+l"(acc[22]), "+l"(acc[23]), \
  "+l"(acc[24]), "+l"(acc[25]), "+l"(acc[26]), "+l"(acc[27]), \
  "+l"(acc[28]), "+l"(acc[29]), "+l"(acc[30]), "+l"(acc[31])

// acc += 64 sums times `scale`. In one statement, so that the sums are used
// where the load puts them: as separate ones they were moved first, which took
// a third of the time that adding them takes.
__device__ __forceinline__ void add_sums64(uint32_t taddr, f32x2* acc, f32x2 scale) {
  uint32_t unused = 0;
  asm volatile("{\n\t" CC_LOAD_SUMS CC_ADD_SUMS "}"
               : CC_ACCUMULATORS, "+r"(unused)
               : "r"(taddr), "l"(scale)
               : "memory");
}

// The same for the last 64 sums of an accumulator buffer: once they are in
// registers the warp's first lane releases the buffer (`tempty`, in the even
// CTA), and the next buffer's barrier is asked for its phase, both before the
// additions that hide them. Returns whether that phase is complete.
__device__ __forceinline__ bool add_sums64_release(uint32_t taddr, f32x2* acc, f32x2 scale, uint32_t tempty,
                                                   uint32_t first, uint32_t next_bar, uint32_t next_parity) {
  uint32_t ready = 0;
  asm volatile("{\n\t.reg .pred first, ready;\n\t" CC_LOAD_SUMS
               "tcgen05.fence::before_thread_sync;\n\t"
               "bar.warp.sync 0xffffffff;\n\t"
               "setp.ne.b32 first, %36, 0;\n\t"
               "@first mbarrier.arrive.shared::cluster.b64 _, [%35];\n\t"
               "mbarrier.test_wait.parity.shared::cta.b64 ready, [%37], %38;\n\t"
               "selp.u32 %32, 1, 0, ready;\n\t" CC_ADD_SUMS "}"
               : CC_ACCUMULATORS, "+r"(ready)
               : "r"(taddr), "l"(scale), "r"(tempty), "r"(first), "r"(next_bar), "r"(next_parity)
               : "memory");
  return ready != 0;
}
#undef CC_LOAD_SUMS
#undef CC_ADD
#undef CC_ADD_SUMS
#undef CC_ACCUMULATORS

// Four blocks' scales of a row of a, or of a block row of the weights, from
// block kb < kblocks on.
__device__ __forceinline__ float4 load_scales(const float* p, int kb, int kblocks, bool on) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (on) {
    if ((kblocks & 3) == 0) {  // rows of scales start on 16-byte boundaries
      v = *reinterpret_cast<const float4*>(p + kb);
    } else {
      v.x = p[kb];
      if (kb + 1 < kblocks) v.y = p[kb + 1];
      if (kb + 2 < kblocks) v.z = p[kb + 2];
      if (kb + 3 < kblocks) v.w = p[kb + 3];
    }
  }
  return v;
}

template <int ACCS, int SPLITS>
__global__ void __cluster_dims__(2 * SPLITS, 1, 1) __launch_bounds__(kPairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmRes, const __grid_constant__ CUtensorMap tmOut,
                    const __grid_constant__ Fp8GemmArgs args) {
  using S = PairShape<ACCS>;
  constexpr bool SPLIT = SPLITS > 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_out = smem + S::kStages * S::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_out + kEpiWarps * S::kOutBytes);
  uint64_t* empty = full + S::kStages;
  uint64_t* tfull = empty + S::kStages;  // [accumulator][buffer]
  uint64_t* tempty = tfull + ACCS * S::kBufs;
  uint64_t* rfull = tempty + ACCS * S::kBufs;  // [kEpiWarps] residual pieces
  uint64_t* done = rfull + kEpiWarps;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  // split: 128 rows of partial sums, padded so that a warp's stores do not collide
  constexpr int kPartRow = S::kCols + 4;
  static_assert(!SPLIT || (ACCS == 1 && kPairRows * kPartRow * 4 <= S::kStages * S::kStageBytes), "partial sums");
  float* part = reinterpret_cast<float*>(smem);

  // from a shuffle, so that the roles' branches are known to be uniform: without
  // it the whole kernel took a fifth longer
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t cluster_rank = cluster_ctarank();
  const uint32_t rank = SPLIT ? cluster_rank & 1 : cluster_rank;  // in the pair
  const uint32_t even = cluster_rank - rank;                       // the pair's first CTA
  const uint16_t both = static_cast<uint16_t>(0x3 << even);
  const bool leader = rank == 0;
  // split: a cluster for each tile, kbs blocks of K from kb0 for this pair. (Whole
  // tiles read args.kblocks where they use it: kept in a register it cost 1 %.)
  const int pair_id = SPLIT ? blockIdx.x / (2 * SPLITS) : blockIdx.x >> 1;
  const int pairs = SPLIT ? args.tiles : gridDim.x >> 1;
  const int kb0 = SPLIT ? static_cast<int>(cluster_rank >> 1) * args.kb_split : 0;
  const int kbs = SPLIT ? blocks_in_share(args.kblocks, args.kb_split, kb0) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < ACCS * S::kBufs; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 2 * kEpiWarps / ACCS);  // the accumulator's warps in both CTAs
    }
    mbar_init(smem_u32(done), 1);
    for (int i = 0; i < kEpiWarps; ++i) mbar_init(smem_u32(&rfull[i]), 1);
    fence_mbar_init();
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
    tma_prefetch_map(&tmOut);
    if (args.res) tma_prefetch_map(&tmRes);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), ACCS * S::kBufs * kAccCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();
  const uint64_t tlim = args.timeout_ns;

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = pair_id; ok && tile < args.tiles; tile += pairs) {
        const int m0 = (2 * (tile / args.n_tiles) + static_cast<int>(rank)) * kPairRows;
        const int n0 = tile % args.n_tiles * S::kCols + static_cast<int>(rank) * (kAccCols / 2);
        for (int kb = 0; kb < (SPLIT ? kbs : args.kblocks); ++kb) {
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, args.err, tlim)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = smem_u32(&full[stage]);
          const uint32_t fb = mapa_shared(fb_local, even);
          if (leader) mbar_arrive_expect_tx(fb_local, 2 * S::kStageBytes);
          const uint32_t dst = smem_u32(smem + stage * S::kStageBytes);
          tma_load_2d_pair(dst, &tmA, fb, (kb0 + kb) * kKBytes, m0);
#pragma unroll
          for (int h = 0; h < ACCS; ++h)
            tma_load_2d_pair(dst + S::kABytes + h * S::kBBytes, &tmB, fb, (kb0 + kb) * kKBytes, n0 + h * kAccCols);
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) {
        // copies of both CTAs complete on the even CTA's barriers; let the
        // armed ones land (200 ms each at most) before the pair winds down
        for (int s = 0; s < S::kStages; ++s)
          (void)mbar_wait(smem_u32(&full[s]), (s < stage) ? phase : (phase ^ 1u), args.err, 200000000ull);
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------- MMA issuer (even CTA only) --
    if (leader) {
      constexpr uint32_t idesc = idesc_e4m3_f32(2 * kPairRows, kAccCols);
      int stage = 0;
      uint32_t phase = 0;
      int buf = 0;
      uint32_t buf_phase = 0;
      bool ok = true;
      const uint64_t a_desc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t b_desc0 = sdesc_sw128(smem_u32(smem + S::kABytes), 16, 1024);
      for (int tile = pair_id; ok && tile < args.tiles; tile += pairs) {
        for (int kb = 0; ok && kb < (SPLIT ? kbs : args.kblocks); ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[stage]), phase, args.err, tlim))) {
            ok = false;
            break;
          }
          const uint64_t off = static_cast<uint64_t>(stage) * (S::kStageBytes >> 4);
#pragma unroll
          for (int h = 0; h < ACCS; ++h) {
            const int acc = h * S::kBufs + buf;
            if (ok && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&tempty[acc]), buf_phase ^ 1u, args.err, tlim)))
              ok = false;
            if (ok) {
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)  // 32 channels, 32 bytes on inside the swizzle row
                  mma_f8_pair(tmem_base + acc * kAccCols, a_desc0 + off + 2 * k,
                              b_desc0 + off + h * (S::kBBytes >> 4) + 2 * k, idesc, k != 0 ? 1u : 0u);
                mma_commit_pair_both(smem_u32(&tfull[acc]), both);
                if (h == ACCS - 1) mma_commit_pair_both(smem_u32(&empty[stage]), both);
              }
              __syncwarp();
            }
          }
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == S::kBufs) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
      // no MMA may still be running when tensor memory is released
      if (elect_one()) mma_commit_pair_both(smem_u32(done), both);
      __syncwarp();
      (void)mbar_wait(smem_u32(done), 0, args.err, tlim);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------- epilogue (both CTAs) --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int quarter = warp & 3;  // tensor memory lanes this warp may read
    const int half = (warp - 4) >> 2;
    uint8_t* stage_out = s_out + (warp - 4) * S::kOutBytes;
    const uint32_t rbar = smem_u32(&rfull[warp - 4]);
    uint32_t rphase = 0;
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 
                           (ACCS == 2 ? half * S::kBufs * kAccCols : half * S::kEpiCols);
    const int first_buf = ACCS == 2 ? half * S::kBufs : 0;
    const uint32_t tfull0 = smem_u32(&tfull[first_buf]);
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[first_buf]), even);
    uint32_t it = 0;  // blocks of K so far: buffer it % kBufs, its phase it / kBufs & 1
    bool ready = false;
    bool ok = true;
    // The scales come in fours and a group ahead, and are multiplied when their
    // turn comes: a product at once would wait for the loads.
    const float *row_scales, *col_scales;
    bool row_on;
    float4 ahead_a, ahead_w;
    auto scales_of = [&](int tile, int mt, int nt) {
      const int m = (2 * mt + static_cast<int>(rank)) * kPairRows + quarter * 32 + lane;
      const int n = nt * S::kCols + half * S::kEpiCols;
      row_on = tile < args.tiles && m < args.m && n < args.n;
      row_scales = args.sa + static_cast<long long>(row_on ? m : 0) * args.kblocks;
      col_scales = args.sw + static_cast<long long>(row_on ? n / kScaleBlock : 0) * args.kblocks;
    };
    auto load_ahead = [&](int kb) {
      ahead_a = load_scales(row_scales, kb, args.kblocks, row_on);
      ahead_w = load_scales(col_scales, kb, args.kblocks, row_on);
    };
    int mt = pair_id / args.n_tiles, nt = pair_id % args.n_tiles;
    const int mt_step = pairs / args.n_tiles, nt_step = pairs % args.n_tiles;
    scales_of(pair_id, mt, nt);
    // A pair whose share of K is empty asks for the rows' first scales and uses
    // none: at kb0 the rows have ended. (Asking for nothing there took 0.2 us more,
    // 128 x 4096 x 4096 9.16 -> 9.39.)
    load_ahead(SPLIT ? first_request(kbs, kb0) : 0);
    for (int tile = pair_id; ok && tile < args.tiles; tile += pairs) {
      const int m0 = (2 * mt + static_cast<int>(rank)) * kPairRows + quarter * 32;
      const int n0 = nt * S::kCols + half * S::kEpiCols;
      const bool any = m0 < args.m && n0 < args.n;  // uniform
      mt += mt_step;
      nt += nt_step;
      if (nt >= args.n_tiles) {
        nt -= args.n_tiles;
        ++mt;
      }
      f32x2 acc[S::kEpiCols / 2];
#pragma unroll
      for (int j = 0; j < S::kEpiCols / 8; ++j) {
        const bool on = args.bias && kb0 == 0 && n0 + 8 * j < args.n;
        const Vec8 t = unpack8(on ? args.bias[(n0 >> 3) + j] : make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[4 * j + e] = t.p[e];
      }
      float4 now = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int kb = 0; kb < (SPLIT ? kbs : args.kblocks); ++kb) {
        if ((kb & 3) == 0) {
          now = make_float4(ahead_a.x * ahead_w.x, ahead_a.y * ahead_w.y, ahead_a.z * ahead_w.z, ahead_a.w * ahead_w.w);
          if (kb + 4 < (SPLIT ? kbs : args.kblocks)) {
            load_ahead(kb0 + kb + 4);
          } else {
            scales_of(tile + pairs, mt, nt);
            load_ahead(0);
          }
        }
        const uint32_t buf = it % S::kBufs;
        if (!__all_sync(0xffffffffu, ready) &&
            !__all_sync(0xffffffffu, mbar_wait(tfull0 + buf * 8, it / S::kBufs & 1, args.err, tlim))) {
          ok = false;
          break;
        }
        ++it;
        tc_fence_after();
        const f32x2 ss = pair(now.x, now.x);
        now = make_float4(now.y, now.z, now.w, 0.f);
        const uint32_t from = tbase + buf * kAccCols;
        if (ACCS == 2) add_sums64(from, acc, ss);
        constexpr int kLast = S::kEpiCols - 64;
        ready = add_sums64_release(from + kLast, acc + kLast / 2, ss, tempty0 + buf * 8, lane == 0,
                                   tfull0 + it % S::kBufs * 8, it / S::kBufs & 1);
        if (!SPLIT && kb == 0 && args.res && any) {
          // the residual's piece, into staging rows that the previous tile's
          // stores have read by now (at the tile's start they had not)
          if (lane == 0) {
            bulk_wait_read_all();
            mbar_arrive_expect_tx(rbar, S::kOutBytes);
#pragma unroll
            for (int g = 0; g < S::kPieces; ++g)
              tma_load_2d(smem_u32(stage_out + g * S::kPieceBytes), &tmRes, rbar, n0 + 64 * g, m0);
          }
          __syncwarp();
        }
      }
      __syncwarp();
      if (SPLIT) {
        // every MMA has read the stages: this pair's sums go over them
        float* to = part + (quarter * 32 + lane) * kPartRow + half * S::kEpiCols;
#pragma unroll
        for (int j = 0; j < S::kEpiCols / 4; ++j)
          *reinterpret_cast<ulonglong2*>(to + 4 * j) = make_ulonglong2(acc[2 * j], acc[2 * j + 1]);
        break;
      }
      if (!any) continue;
      if (args.res) {
        if (!__all_sync(0xffffffffu, mbar_wait(rbar, rphase, args.err, tlim))) ok = false;
        rphase ^= 1u;
      } else {
        if (lane == 0) bulk_wait_read_all();  // the previous tile's stores have read the staging rows
        __syncwarp();
      }
      if (!ok) break;
      // 64 columns at a time, all loads in front of the first store
#pragma unroll
      for (int g = 0; g < S::kPieces; ++g) {
        uint8_t* row = stage_out + g * S::kPieceBytes + lane * 128;
        if (args.res) {
          uint4 extra[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) extra[j] = *reinterpret_cast<const uint4*>(row + ((j ^ (lane & 7)) << 4));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const Vec8 t = unpack8(extra[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[32 * g + 4 * j + e] = add2(acc[32 * g + 4 * j + e], t.p[e]);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          Vec8 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v.p[e] = acc[32 * g + 4 * j + e];
          *reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4)) = pack8(v);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
#pragma unroll
        for (int g = 0; g < S::kPieces; ++g)
          if (n0 + 64 * g < args.n) tma_store_2d(&tmOut, smem_u32(stage_out + g * S::kPieceBytes), n0 + 64 * g, m0);
        bulk_commit();
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
    if (SPLIT) {
      cluster_sync_all();
      // each pair finishes its share of the tile's rows, a warp to a row, in the pairs' order
      constexpr int share = kPairRows / SPLITS;
      const int r0 = static_cast<int>(cluster_rank >> 1) * share;
      const int m0 = (2 * (pair_id / args.n_tiles) + static_cast<int>(rank)) * kPairRows;
      const int n = pair_id % args.n_tiles * S::kCols + lane * 4;
#pragma unroll 4
      for (int r = r0 + warp - 4; r < r0 + share; r += kEpiWarps) {
        const int m = m0 + r;
        if (m >= args.m || n >= args.n) continue;
        const uint32_t at = smem_u32(part + r * kPartRow + lane * 4);
        float4 of[SPLITS];
#pragma unroll
        for (uint32_t i = 0; i < SPLITS; ++i) of[i] = ld_cluster_f4(mapa_shared(at, 2 * i + rank));
        float4 v = of[0];
#pragma unroll
        for (int i = 1; i < SPLITS; ++i) {
          v.x += of[i].x;
          v.y += of[i].y;
          v.z += of[i].z;
          v.w += of[i].w;
        }
        if (args.res) {
          const uint2 t = *reinterpret_cast<const uint2*>(args.res + m * args.ld_res + n);
          v.x += __uint_as_float(t.x << 16);
          v.y += __uint_as_float(t.x & 0xffff0000u);
          v.z += __uint_as_float(t.y << 16);
          v.w += __uint_as_float(t.y & 0xffff0000u);
        }
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(args.out + m * args.ld_out + n) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      }
      __syncwarp();
    }
  }
  if (SPLIT && warp < 4) {  // (in the branches: here the epilogue's registers are not all warps')
    __syncwarp();
    cluster_sync_all();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peers no longer read this CTA's shared memory or signals its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, ACCS * S::kBufs * kAccCols);
  }
}

// ------------------------------------------------------------------ few rows --

// The weights' 128 rows take the tensor core's M side and up to MT rows of a
// its N side, so a call with one row moves the weights and wastes nothing but
// tensor core time. K is split over the CTAs of a cluster, whose partial sums
// meet in shared memory, in rank order: the weights stream through all SMs
// although there are few output tiles. One row x 4096 x 4096: 4.8 us (3.5 TB/s,
// of which half is the launch and the exchange); 64 rows: 7.3 us.
constexpr int kFewThreads = 192;
constexpr int kFewMax = 64;       // rows
constexpr int kFewScales = 4096;  // staged scales of a: MT x blocks of K per CTA
constexpr int kFewStages = 6;
constexpr int kFewRanks = 8;      // CTAs in a cluster

// Shared memory of a CTA with kb_split blocks of K: stages, over which the
// partial sums go when all are used up, and the scales.
int few_smem(int mt, int kb_split) {
  return 1024 + std::max(std::min(kFewStages, kb_split) * (128 + mt) * kKBytes, mt * 128 * 4) + mt * kb_split * 4 + 256;
}
constexpr int kMaxSmemOfTwo = 112 * 1024;  // of each of two CTAs on an SM
static_assert(kMaxSmem / 2 + 1024 <= 1024 + kFewStages * (128 + 16) * kKBytes + kFewScales * 4 + 256,
              "the most a launch asks for is allowed");

template <int MT>
struct FewShape {
  static constexpr int kWBytes = 128 * kKBytes;
  static constexpr int kABytes = MT * kKBytes;
  static constexpr int kStageBytes = kWBytes + kABytes;
  static constexpr uint32_t kTmemCols = 2 * MT;
  static constexpr int kPartBytes = MT * 128 * 4;  // partial sums, over the stages when all are used up
};

template <int MT>
__global__ void __launch_bounds__(kFewThreads, 2)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ Fp8GemmArgs args, const int stages) {
  using S = FewShape<MT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bars[2 * kFewStages + 5];
  __shared__ uint32_t tmem_slot;
  uint64_t* full = bars;
  uint64_t* empty = bars + kFewStages;
  uint64_t* tfull = empty + kFewStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  float* part = reinterpret_cast<float*>(smem);
  float* ssa = reinterpret_cast<float*>(smem + (stages * S::kStageBytes > S::kPartBytes ? stages * S::kStageBytes
                                                                                        : S::kPartBytes));
  uint32_t ranks;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const uint32_t rank = cluster_ctarank();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nt = blockIdx.x / ranks;
  const int kb0 = rank * args.kb_split;
  const int kbs = blocks_in_share(args.kblocks, args.kb_split, kb0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
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
    tma_prefetch_map(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  pdl_launch_dependents();
  pdl_wait();
  const uint64_t tlim = args.timeout_ns;

  bool ok = true;
  f32x2 acc[MT / 2];
#pragma unroll
  for (int j = 0; j < MT / 2; ++j) acc[j] = 0;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = 0; kb < kbs; ++kb) {
        if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, args.err, tlim)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&full[stage]);
        const uint32_t dst = smem_u32(smem + stage * S::kStageBytes);
        mbar_arrive_expect_tx(fb, S::kStageBytes);
        tma_load_2d(dst, &tmW, fb, (kb0 + kb) * kKBytes, nt * 128);
        tma_load_2d(dst + S::kWBytes, &tmA, fb, (kb0 + kb) * kKBytes, 0);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        // copies already issued land before the CTA can exit
        for (int s = 0; s < stages; ++s)
          (void)mbar_wait(smem_u32(&full[s]), (s < stage) ? phase : (phase ^ 1u), args.err, 200000000ull);
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_e4m3_f32(128, MT);
    int stage = 0;
    uint32_t phase = 0;
    const uint64_t w_desc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t a_desc0 = sdesc_sw128(smem_u32(smem + S::kWBytes), 16, 1024);
    for (int kb = 0; kb < kbs; ++kb) {
      const int buf = kb & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&tempty[buf]), ((kb >> 1) & 1) ^ 1u, args.err, tlim) &&
                                       mbar_wait(smem_u32(&full[stage]), phase, args.err, tlim)))
        break;
      tc_fence_after();
      const uint64_t off = static_cast<uint64_t>(stage) * (S::kStageBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8(tmem_base + buf * MT, w_desc0 + off + 2 * k, a_desc0 + off + 2 * k, idesc, k != 0 ? 1u : 0u);
        mma_commit(smem_u32(&empty[stage]));
        mma_commit(smem_u32(&tfull[buf]));
      }
      __syncwarp();
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (elect_one()) mma_commit(smem_u32(done));
    __syncwarp();
    (void)mbar_wait(smem_u32(done), 0, args.err, tlim);
  } else {
    const int quarter = warp & 3;
    const int tid = threadIdx.x - 64;
    // ssa[kb][row]: the rows' scales times the weights'
    for (int i = tid; i < MT * kbs; i += 128) {
      const int kb = i / MT, r = i % MT;
      ssa[i] = r < args.m ? args.sa[static_cast<long long>(r) * args.kblocks + kb0 + kb] *
                                     args.sw[static_cast<long long>(nt) * args.kblocks + kb0 + kb]
                               : 0.f;
    }
    __syncwarp();
    named_barrier_sync(1, 128);
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    for (int kb = 0; kb < kbs; ++kb) {
      const int buf = kb & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&tfull[buf]), (kb >> 1) & 1, args.err, tlim))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t r[MT / 16][16];  // all loads in front of the first wait
#pragma unroll
      for (int i = 0; i < MT / 16; ++i) tmem_ld16(tbase + buf * MT + 16 * i, r[i]);
#pragma unroll
      for (int i = 0; i < MT / 16; ++i) {
        tmem_wait16(r[i]);
        const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(ssa + kb * MT + 16 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const ulonglong2 s = sc[j];
          f32x2* to = acc + 8 * i + 2 * j;
          to[0] = fma2(pair(__uint_as_float(r[i][4 * j]), __uint_as_float(r[i][4 * j + 1])), s.x, to[0]);
          to[1] = fma2(pair(__uint_as_float(r[i][4 * j + 2]), __uint_as_float(r[i][4 * j + 3])), s.y, to[1]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tempty[buf]));
    }
  }
  // every copy has landed and every MMA has read it before the stages become
  // the partial sums (the MMA warp waited for `done`)
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    // before this CTA waits for others: what holds tensor memory then waits for nobody
    tc_fence_after();
    tmem_dealloc(tmem_base, S::kTmemCols);
  }
  if (warp >= 2) {
    const int n = (warp & 3) * 32 + lane;
#pragma unroll
    for (int j = 0; j < MT / 2; ++j) {
      part[(2 * j) * 128 + n] = lo(acc[j]);
      part[(2 * j + 1) * 128 + n] = hi(acc[j]);
    }
  }
  __syncwarp();
  cluster_sync_all();
  // each rank finishes its share of the rows, two columns to a thread
  const int share = (MT + static_cast<int>(ranks) - 1) / static_cast<int>(ranks);
  for (int i = threadIdx.x; i < share * 64; i += kFewThreads) {
    const int m = static_cast<int>(rank) * share + (i >> 6);
    const int c = (i & 63) * 2;
    const int n = nt * 128 + c;
    if (m < args.m && n < args.n) {
      const uint32_t at = smem_u32(part + m * 128 + c);
      float2 of[kFewRanks];  // all trips to the other CTAs at once
#pragma unroll
      for (uint32_t k = 0; k < kFewRanks; ++k)
        if (k < ranks) of[k] = ld_cluster_f2(mapa_shared(at, k));
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (uint32_t k = 0; k < kFewRanks; ++k) {
        if (k < ranks) {
          v.x += of[k].x;
          v.y += of[k].y;
        }
      }
      if (args.bias) {
        const float2 t = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(args.bias)[n >> 1]);
        v.x += t.x;
        v.y += t.y;
      }
      if (args.res) {
        const float2 t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(args.res + m * args.ld_res + n));
        v.x += t.x;
        v.y += t.y;
      }
      *reinterpret_cast<__nv_bfloat162*>(args.out + m * args.ld_out + n) = __floats2bfloat162_rn(v.x, v.y);
    }
  }
  __syncwarp();
  cluster_sync_all();  // the peers have read this CTA's partial sums
}

// -------------------------------------------------------------------- launch --

// A launch in clusters of `cluster` CTAs that may begin before the previous one ends.
template <typename... Args>
cc_status launch_clusters(const char* what, void (*kern)(Args...), int grid, int cluster, int threads, int smem,
                          int max_smem, cudaStream_t stream, const Args&... args) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: shared-memory attribute: %s", what, cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: launch: %s", what, cudaGetErrorString(e));
  return launch_status(what);
}

template <int MT>
cc_status launch_few(const char* what, Fp8GemmArgs& args, const cc_fp8* a, const cc_fp8* wq, int k, int ranks,
                     int sms, cudaStream_t stream) {
  using S = FewShape<MT>;
  CUtensorMap ta, tw;
  cc_status st;
  if ((st = encode_tiled_2d_u8(&ta, a, k, args.m, k, kKBytes, MT)) != CC_OK) return st;
  if ((st = encode_tiled_2d_u8(&tw, wq, k, args.n, k, kKBytes, 128)) != CC_OK) return st;
  const int stages = std::min(kFewStages, args.kb_split);
  // Shared memory that lets no more CTAs on an SM than it takes to run all of them
  // at once: they are put closer together while SMs are idle otherwise (one row x
  // 4096 x 4096, 256 CTAs: 5.5 -> 4.8 us)
  const int ctas = ((args.n - 1) / 128 + 1) * ranks;
  const int per_sm = ctas <= sms - 4 * ranks ? 1 : ctas <= 2 * sms - 4 * ranks ? 2 : 3;
  const int smem = std::max(few_smem(MT, args.kb_split), kMaxSmem / (per_sm + 1) + 1024);
  return launch_clusters(what, fp8_few_kernel<MT>, ctas, ranks, kFewThreads, smem,
                         few_smem(MT, kFewScales / MT), stream, ta, tw, args, stages);
}

template <int ACCS, int SPLITS>
cc_status launch_pair(const char* what, Fp8GemmArgs& args, const cc_fp8* a, const cc_fp8* wq, int k, int sms,
                      cudaStream_t stream) {
  using S = PairShape<ACCS>;
  CUtensorMap ta, tb, to, tr;
  cc_status st;
  if ((st = encode_tiled_2d_u8(&ta, a, k, args.m, k, kKBytes, kPairRows)) != CC_OK) return st;
  if ((st = encode_tiled_2d_u8(&tb, wq, k, args.n, k, kKBytes, kAccCols / 2)) != CC_OK) return st;
  if ((st = encode_tiled_2d(&to, args.out, args.n, args.m, args.ld_out * 2, 64, 32)) != CC_OK) return st;
  tr = to;
  if (args.res && (st = encode_tiled_2d(&tr, args.res, args.n, args.m, args.ld_res * 2, 64, 32)) != CC_OK) return st;
  const long long m_tiles = (args.m - 1) / (2 * kPairRows) + 1;
  args.n_tiles = (args.n - 1) / S::kCols + 1;
  if (m_tiles * args.n_tiles > 0x7fffffffLL - 1024) return fail(CC_ERR_UNSUPPORTED, "%s: too many output tiles", what);
  args.tiles = static_cast<int>(m_tiles * args.n_tiles);
  return launch_clusters(what, fp8_pair_kernel<ACCS, SPLITS>,
                         2 * (SPLITS > 1 ? args.tiles * SPLITS : std::min(args.tiles, sms / 2)), 2 * SPLITS,
                         kPairThreads, S::kSmem, S::kSmem, stream, ta, tb, tr, to, args);
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
  if (m > kMaxRows || n > kMaxChannels || k > kMaxChannels)
    return fail(CC_ERR_UNSUPPORTED, "%s: too many rows or channels", what);
  if (ld_out < n || ld_out % 8 != 0 || (res && (ld_res < n || ld_res % 8 != 0)))
    return fail(CC_ERR_INVALID, "%s: ld_out and ld_res must be at least N and multiples of 8", what);
  DeviceInfo di;
  if ((st = device_info(&di)) != CC_OK) return st;
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  // Few rows: one N-side tile of the tensor core, K over the CTAs of a cluster
  // while all of them run at once (one to an SM, or two where they are small;
  // clusters of eight do not fill all SMs). Beyond that a second round costs more
  // than the split saves: 64 x 4096 x 16384 takes 18 us on four CTAs each, 29 on
  // eight; 1 x 4096 x 16384 with two to an SM 14.7 on four, 13.7 on eight. 64 x
  // 4096 x 4096 takes 7.3 us, on pairs 9.4; 128 rows take longer than on pairs.
  if (m <= kFewMax) {
    const int mt = m <= 16 ? 16 : m <= 32 ? 32 : 64;
    const long long n_tiles = (n - 1) / 128 + 1;
    int ranks = 1;
    auto split = [&](int r) { return (args.kblocks - 1) / r + 1; };
    auto fits = [&](int r) { return static_cast<long long>(mt) * split(r) <= kFewScales; };
    while (ranks < kFewRanks && 2 * ranks <= args.kblocks) {
      const int next = 2 * ranks;
      const bool two = mt < 64 && fits(next) && few_smem(mt, split(next)) <= kMaxSmemOfTwo;
      if (fits(ranks) && n_tiles * next > (two ? 2 : 1) * di.sm_count - 4 * next) break;
      ranks = next;
    }
    args.kb_split = split(ranks);
    if (fits(ranks)) {
      if (mt == 16) return launch_few<16>(what, args, a, wq, k, ranks, di.sm_count, s);
      if (mt == 32) return launch_few<32>(what, args, a, wq, k, ranks, di.sm_count, s);
      return launch_few<64>(what, args, a, wq, k, ranks, di.sm_count, s);
    }
  }
  // Tiles of 256 columns or of 128: rounds of tiles times what a tile takes, in
  // hundredths of a microsecond a block of K and at its end. In us, wide / narrow:
  // 128 x 4096 x 4096 14.8 / 10.9, 100000 x 128 x 512 20.8 / 17.6 (one round
  // either way, half the columns), 1546 x 3184 x 1264 13.7 / 12.8 (two and three
  // rounds); 1024 x 4096 x 4096 16.4 / 19.9, 13728 x 1024 x 1024 16.9 / 19.2.
  const long long pairs = di.sm_count / 2, m_tiles = (m - 1) / (2 * kPairRows) + 1;
  auto tiles = [&](int cols) { return m_tiles * ((n - 1) / cols + 1); };
  auto cost = [&](int cols, long long block, long long end) {
    return ((tiles(cols) - 1) / pairs + 1) * (args.kblocks * block + end);
  };
  const long long wide = cost(PairShape<2>::kCols, 36, 100), narrow = cost(PairShape<1>::kCols, 25, 50);
  // Few narrow tiles: two or four pairs to each, while all clusters run at once
  // (of eight CTAs fifteen); putting the sums together takes 2 us. 256 x 512 x
  // 16384 takes 32.8 us whole, 19.4 on two and 12.4 on four pairs; 128 x 4096 x
  // 4096 11.1 and 9.7; 128 x 1024 x 1024, eight blocks, 5.3 and 6.0.
  long long best = std::min(wide, narrow);
  int splits = 1;
  for (int next = 2; next <= 4; next *= 2) {
    const int blocks = share_blocks(args.kblocks, next);
    if (tiles(PairShape<1>::kCols) * 2 * next > di.sm_count - 8 * next || blocks * 25 + 250 >= best) continue;
    best = blocks * 25 + 250;
    splits = next;
    args.kb_split = blocks;
  }
  if (splits == 4) return launch_pair<1, 4>(what, args, a, wq, k, di.sm_count, s);
  if (splits == 2) return launch_pair<1, 2>(what, args, a, wq, k, di.sm_count, s);
  if (narrow < wide) return launch_pair<1, 1>(what, args, a, wq, k, di.sm_count, s);
  return launch_pair<2, 1>(what, args, a, wq, k, di.sm_count, s);
}
