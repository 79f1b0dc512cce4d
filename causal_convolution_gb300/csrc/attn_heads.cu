// Attention with heads: the new tokens of several sequences over a paged cache,
// and queries over an encoder's states.
//
//   o_i = sum_{j < limit(i)} softmax_j(scale q_i . k_j) v_j
//
// Work. An item is up to 256 query rows of one sequence and one key head -- two
// halves of 128 rows, a row being a (token, query head of the group) pair, so
// that grouped heads share the keys they read -- and all the 128-key tiles that
// any of its rows sees. The items' tiles, laid end to end (sequence, rows, head),
// are cut into equal runs, one for each CTA of a persistent grid. An item cut by
// a run's end leaves partial sums in the workspace, which a second kernel joins;
// where whole items spread well enough nothing is cut (cc_heads.cuh). The lengths
// are read on the device, so every CTA finds its run by itself. Few rows to a
// sequence go to another kernel (attn_few_rows.cu).
//
// Kernel. Warps 16 and 19 stream q and k, and v, with TMA (a box per page piece,
// so a page of 16 tokens costs eight boxes and 64 channels; with one warp for
// both, 2432 rows of 16 heads over 8192 keys in such pages went from 157 to 201
// us, in pages of 128 they took 156 either way). Warps 17 and 18 issue the
// products of a stream each: S = q k^T (128 x 128, K = D) into tensor memory,
// then O += P v with P read from tensor memory, where it takes the place of S.
// Warps 0-7 and 8-15 are two softmax streams: they turn a tile of S into P =
// bf16(exp2(kx S - c)), half a row to a thread. Items of two halves give each
// stream a half and both the same keys; items of one half give the streams every
// other tile, and their sums are joined at the end. While a stream works on its
// S, the tensor cores run the other's products.
//
// c, the row's scale, is a whole power of two: where it moves, and where streams
// and pieces are joined, sums are multiplied exactly. It begins as 2^0 and moves
// when a row's weights of half a tile come to 2^20, or those of the first keys that
// it sees to less than 2^-10, which their sum tells: no maximum is looked for but
// where that happens (short texts 13.2 -> 11.6 us against a maximum of each item's
// first tile, together with the exchange of a row's sums during its last product).
// fp32 sums of weights up to 2^20 lose nothing that weights up to 1 would keep.
//
// Weights are rounded to bf16, the type of the values that the tensor cores multiply
// them with: off by up to 2^-8 of themselves, on whatever scale. What is divided by is
// the sum of the rounded ones, so only the spread of the roundings is left; against 64
// bits results are off by 0.0020 to 0.0023 (L2, relative) where their own rounding
// alone makes 0.0017. A second part for what is left, as in the kernel for few rows,
// would cost a second product with v, half as much again for the tensor cores. Which
// kernel a row gets, and with it which of the two, follows from the whole call
// (few_rows below).
//
// Bound: long chunks by the streams' chain -- 1024 clocks of products, 1900 of
// softmax with its trips through tensor memory and barriers, where two streams
// would need 2048 in all for the tensor cores alone; tensor memory (512 columns)
// holds no third S beside the sums of 128 channels. 13728 rows of 16 heads of 128
// over 27456 keys in blocks of 3432: 1.58 ms for a single launch (1.59 PFLOP/s, tensor
// pipe 70 % busy), 1.78 to 1.82 ms back to back, under the power limit (1.38 to 1.41
// PFLOP/s; the library product's own rate under it is 1.73). Texts of 512 keys: 60 us
// for 29 of products, as an item's beginning and end come one after the other for both
// streams. What led here, for the chunk back to back: one row to a thread
// with eight softmax warps 2.12 ms; a maximum for every tile 2.17; products of
// both streams issued by two warps as they come 2.24, by one in turns 1.94, by two
// in turns 1.90; 64-key tiles with two S to a stream 2.26; CTAs with the same
// keys in step 1.87 (5.5 -> 3.1 GB from memory); shorter waits 1.84; a tile's
// scores in two halves, so that registers suffice, 1.77.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "cc.h"
#include "cc_heads.cuh"
#include "cc_host.h"

namespace cc {
namespace {

constexpr int kAhTmaWarp = 16;    // behind 16 softmax warps
constexpr int kAhMmaWarp = 17;    // and 18, one for each stream
constexpr int kAhValueWarp = 19;  // the second TMA warp, for values
constexpr int kAhThreads = 640;
constexpr int kAhTileShift = 7;
constexpr int kAhKeys = 1 << kAhTileShift;  // keys per tile, in two halves for the softmax
constexpr int kAhHalf = 128;      // rows per half
constexpr int kAhQBlock = kAhHalf * 128;   // bytes of 128 query rows x 64 channels
constexpr int kAhKvBlock = kAhKeys * 128;  // bytes of 128 keys (or values) x 64 channels
constexpr float kAhRoom = 1048576.f;  // 2^20: what half a tile's weights of a row may come to before its scale moves
constexpr float kAhLeast = 1.f / 1024;  // and to at least, on the scale that a row tries first
constexpr float kAhMove = 8.f;        // and by how many powers of two at least
// What cutting items costs, in tiles, for a run of one item; see find_run. Measured with 6, 12, 16, 24 and 48: 128 rows
// of 8 heads, one key head, over 3000 keys 33 us cut and 45 whole (22 tiles apart), 512 of 16 over 2500 39 and 43 (16),
// over 600 to 1200 28 and 24 (5).
constexpr int kAhSplitCost = 12;

// A value that all lanes hold, said in a way that the compiler keeps it in
// uniform registers.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// A matrix descriptor as sdesc_sw128 makes it, in halves: only the low one, the
// address, changes from product to product.
__device__ __forceinline__ uint32_t sdesc_low(const void* p, uint32_t lbo_bytes) {
  return static_cast<uint32_t>(sdesc_sw128(smem_u32(p), lbo_bytes, 1024));
}
__device__ __forceinline__ uint64_t sdesc_of(uint32_t low) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low), "n"(static_cast<int>(64u | 1u << 14 | 2u << 29)));
  return d;
}

// NB: 64-channel blocks of a head; STAGES: k or v tiles in flight.
template <int NB, int STAGES>
struct AhSmem {
  static constexpr int kTile = NB * kAhKvBlock;
  static constexpr int kQHalf = NB * kAhQBlock;
  static constexpr int kQ = 2 * kQHalf;
  static constexpr int kBytes = 1024 + kQ + STAGES * kTile + 1024 + 2 * kAhHalf * 8 + 8 * kAhHalf * 4;
};

template <int NB, int STAGES>
__global__ void __launch_bounds__(kAhThreads, 1)
    attn_heads_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AhArgs a) {
  using Sm = AhSmem<NB, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = sQ + Sm::kQ;
  float2* sCL = reinterpret_cast<float2*>(sKV + STAGES * Sm::kTile);  // [2][128] stream 1's (c, l) of single halves
  float* sX = reinterpret_cast<float*>(sCL + 2 * kAhHalf);    // [2][4][128] what warps of the same rows exchange: maxima, sums
  AhItem* items = reinterpret_cast<AhItem*>(sX + 8 * kAhHalf);
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + kAhItems);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = kv_full + STAGES;
  uint64_t* item_full = kv_empty + STAGES;
  uint64_t* item_empty = item_full + kAhItems;
  uint64_t* q_full = item_empty + kAhItems;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_ready = q_empty + 1;  // [2] S of a stream complete
  uint64_t* p_ready = s_ready + 2;  // [2] P in its place, and O on its scale
  uint64_t* pv_done = p_ready + 2;  // [2] the item's last product of a stream complete
  uint64_t* o_free = pv_done + 2;   // [2] O of a stream read out
  uint64_t* cl_ready = o_free + 2;
  uint64_t* turns = cl_ready + 1;   // [4] a job of the MMA warps issued
  uint64_t* done = turns + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (warp == kAhTmaWarp && lane == 0) {
    tma_prefetch_map(&tmQ);
    if (a.plan.page_size > 0) {  // there are keys, and maps of them
      tma_prefetch_map(&tmK);
      tma_prefetch_map(&tmV);
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&kv_full[i]), 1);
      mbar_init(smem_u32(&kv_empty[i]), 2);
    }
    for (int i = 0; i < kAhItems; ++i) {
      mbar_init(smem_u32(&item_full[i]), 1);
      mbar_init(smem_u32(&item_empty[i]), 19);
    }
    mbar_init(smem_u32(q_full), 1);
    mbar_init(smem_u32(q_empty), 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_ready[i]), 1);
      mbar_init(smem_u32(&p_ready[i]), 8);
      mbar_init(smem_u32(&pv_done[i]), 1);
      mbar_init(smem_u32(&o_free[i]), 8);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&turns[i]), 1);
    mbar_init(smem_u32(cl_ready), 8);
    mbar_init(smem_u32(done), 2);
    fence_mbar_init();
  }
  if (warp == kAhMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == kAhTmaWarp || warp == kAhValueWarp) {
    // -------------------------------------------- run, items and TMA loads --
    // One warp finds the run, publishes its items and loads q and keys, the other one loads values.
    const bool keys = warp == kAhTmaWarp;
    const CUtensorMap* map = keys ? &tmK : &tmV;
    Run r = {};
    bool ok = true, any = false;
    int stage = 0, slot = 0;
    uint32_t kv_ph = 0, it_ph = 0, q_ph = 0;
    // one tile of keys (or values): a box per piece of a page, a lane to a box
    auto load_tile = [&](int b, int h, int len, int t) {
      const int boxes = (min(kAhKeys, len - t * kAhKeys) + a.box - 1) / a.box;
      int page = b, at = t * kAhKeys + lane * a.box;
      if (lane < boxes && a.plan.page_table) {
        const int n = at / a.plan.page_size;
        at -= n * a.plan.page_size;
        page = a.plan.page_table[static_cast<long long>(b) * a.plan.max_pages + n];
        if (page < 0 || page >= a.plan.pages) {
          atomicOr(a.err, DEVERR_BOUNDS);
          page = a.plan.pages;  // out of the map's range: the box reads as zeros
        }
      }
      if (!warp_wait(&kv_empty[stage], kv_ph ^ 1u, a)) return false;
      const uint32_t full = smem_u32(&kv_full[stage]);
      if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(boxes * a.box * 128 * NB));
      __syncwarp();
      if (lane < boxes) {
        const uint32_t dst = smem_u32(sKV + stage * Sm::kTile) + static_cast<uint32_t>(lane * a.box) * 128u;
#pragma unroll
        for (int i = 0; i < NB; ++i) tma_load_4d(dst + i * kAhKvBlock, map, full, i * 64, h, at, page);
      }
      return true;
    };
    if (keys) {
      any = find_run(a, blockIdx.x, gridDim.x, lane, r);
      if (a.may_split && lane < 2) a.meta[2 * blockIdx.x + lane] = make_int4(0, 0, 0, 0);
      __syncwarp();
      if (any && !r.split && r.t > 0) {  // whole items: from the first one that starts in the run
        r.at += max(1, r.tiles) - r.t;
        next_item(a, r);
      }
    }
    while (ok) {
      ok = warp_wait(keys ? &item_empty[slot] : &item_full[slot], keys ? it_ph ^ 1u : it_ph, a);
      if (!ok) break;
      if (keys) {
        AhItem it = {};
        it.last = !(any && r.at < r.end && r.b < a.plan.seqs);
        if (!it.last) it = make_item(a, r, lane);
        if (lane == 0) {
          items[slot] = it;
          mbar_arrive(smem_u32(&item_full[slot]));  // releases the descriptor
        }
        __syncwarp();
      }
      const int last = uniform(items[slot].last), t_begin = uniform(items[slot].t_begin), seq = uniform(items[slot].seq);
      const int head = uniform(items[slot].head), len = uniform(items[slot].len), from = uniform(items[slot].turn);
      const int n = uniform(items[slot].t_end) - t_begin, q_row = uniform(items[slot].q_row);
      const bool two = uniform(items[slot].tokens) > a.tq;
      __syncwarp();
      if (!keys && lane == 0) mbar_arrive(smem_u32(&item_empty[slot]));
      if (++slot == kAhItems) {
        slot = 0;
        it_ph ^= 1u;
      }
      if (last) break;
      // k of the first tiles, q, then v of each tile with k of the one that far ahead
      const int ahead = two ? 1 : 2;  // a tile of scores ahead in each stream
#pragma unroll 1
      for (int i = 0; ok && n > 0 && i < n + ahead; ++i) {
        if (keys && i == min(ahead, n)) {
          ok = warp_wait(q_empty, q_ph ^ 1u, a);
          if (!ok) break;
          q_ph ^= 1u;
          if (lane == 0) {
            const uint32_t full = smem_u32(q_full);
            mbar_arrive_expect_tx(full, static_cast<uint32_t>((two ? 2 : 1) * NB * a.tq * a.group * 128));
#pragma unroll 1
            for (int s = 0; s < (two ? 2 : 1); ++s)
              for (int b = 0; b < NB; ++b)
                tma_load_4d(smem_u32(sQ + s * Sm::kQHalf + b * kAhQBlock), &tmQ, full, b * 64, head * a.group,
                            q_row + s * a.tq, 0);
          }
          __syncwarp();
        }
#pragma unroll 1
        for (int kind = i >= ahead ? 0 : 1; ok && kind < (i < n ? 2 : 1); ++kind) {  // v, k
          if ((kind != 0) == keys) ok = load_tile(seq, head, len, tile_of(t_begin, n, from, kind ? i : i - ahead));
          if (++stage == STAGES) {
            stage = 0;
            kv_ph ^= 1u;
          }
        }
      }
      if (keys) {
        r.at += static_cast<unsigned>(max(1, n));
        next_item(a, r);
      }
    }
    if (!ok) {  // copies in flight land before the CTA goes
#pragma unroll 1
      for (int i = 0; i < STAGES; ++i)
        (void)mbar_wait(smem_u32(&kv_full[i]), (i < stage) ? kv_ph : (kv_ph ^ 1u), a.err, 200000000ull);
      (void)mbar_wait(smem_u32(q_full), q_ph ^ 1u, a.err, 200000000ull);
    }
  } else if (warp >= kAhMmaWarp) {
    // ------------------------------------------------ MMA, a warp per stream --
    // A product and the stream's next scores are a job. Jobs are issued one after
    // the other, streams in turn, so that a stream is back at its softmax while
    // the other's job runs; the queue holds next to nothing, so a warp that has
    // its turn has done its waiting before. Without turns the streams' products
    // mix and both finish late.
    const int s = uniform(warp - kAhMmaWarp);
    const uint32_t idesc_s = idesc_bf16_f32(kAhHalf, kAhKeys, false);
    const uint32_t idesc_o = idesc_bf16_f32(kAhHalf, a.d, true);
    const int steps = a.d / 16;
    const uint32_t q0 = sdesc_low(sQ, 16), k0 = sdesc_low(sKV, 16), v0 = sdesc_low(sKV, kAhKvBlock);
    const uint32_t s_tmem = tmem + s * 128, o_tmem = tmem + 256 + s * 128;
    int stage = 0, slot = 0;
    uint32_t kv_ph = 0, it_ph = 0, q_ph = 0, p_ph = 0, of_ph = 0;
    uint32_t job = 0;   // number of the item's first job, of both streams
    bool used = false;  // the stream's O was written by an item before
    bool ok = true;
    // waits for the next k or v tile; its stage, -1 where the wait ran out
    auto next_tile = [&]() {
      const int at = stage;
      const bool got = warp_wait(&kv_full[stage], kv_ph, a);
      if (++stage == STAGES) {
        stage = 0;
        kv_ph ^= 1u;
      }
      return got ? at : -1;
    };
    // the other stream's tile
    auto skip_tile = [&]() {
      const int at = next_tile();
      if (lane == 0 && at >= 0) mbar_arrive(smem_u32(&kv_empty[at]));
      __syncwarp();
      return at >= 0;
    };
    // job j waits until the one in front of it has been issued, and says when it has been
    auto turn = [&](uint32_t j) { return j == 0 || warp_wait(&turns[(j - 1) & 3], (j - 1) >> 2 & 1u, a); };
    auto issued = [&](uint32_t j) {
      if (lane == 0) mbar_arrive(smem_u32(&turns[j & 3]));
      __syncwarp();
    };
    auto scores = [&](int half, int at, bool last) {
      const uint32_t ad = q0 + half * (Sm::kQHalf >> 4), bd = k0 + at * (Sm::kTile >> 4);
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < NB * 4; ++k) {
          if (k < steps)
            mma_bf16(s_tmem, sdesc_of(ad + (k >> 2) * (kAhQBlock >> 4) + (k & 3) * 2),
                     sdesc_of(bd + (k >> 2) * (kAhKvBlock >> 4) + (k & 3) * 2), idesc_s, k ? 1u : 0u);
        }
        mma_commit(smem_u32(&s_ready[s]));
        mma_commit(smem_u32(&kv_empty[at]));
        if (last) mma_commit(smem_u32(q_empty));
      }
      __syncwarp();
    };
    while (true) {
      if (!warp_wait(&item_full[slot], it_ph, a)) break;
      const AhItem* it = &items[slot];
      const int last = uniform(it->last), t_begin = uniform(it->t_begin), len = uniform(it->len), from = uniform(it->turn);
      const int n = uniform(it->t_end) - t_begin;
      const bool two = uniform(it->tokens) > a.tq;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&item_empty[slot]));
      if (++slot == kAhItems) {
        slot = 0;
        it_ph ^= 1u;
      }
      if (last) break;
      if (n <= 0) continue;
      const int half = two ? s : 0;
      const int jobs = two ? 2 * n : n;  // of two halves a tile is a job for each stream, of one every other tile
      const int firsts = min(2, jobs);   // in front of them, each stream's first scores
      if (!warp_wait(q_full, q_ph, a)) break;
      q_ph ^= 1u;
      if (s >= jobs && lane == 0) mbar_arrive(smem_u32(q_empty));
      __syncwarp();
      // the tiles come as k of each stream's first, then v of each with k of the one that far ahead
      const int ahead = two ? 1 : 2;
#pragma unroll 1
      for (int i = 0; ok && i < min(ahead, n); ++i) {
        if (!two && i != s) {
          ok = skip_tile();
          continue;
        }
        const int ks = next_tile();
        ok = ks >= 0 && turn(job + s);
        if (!ok) break;
        scores(half, ks, s + 2 >= jobs);
        issued(job + s);
      }
#pragma unroll 1
      for (int i = 0; ok && i < n; ++i) {
        const bool more = i + ahead < n;
        if (!two && (i & 1) != s) {
          ok = skip_tile() && (!more || skip_tile());
          continue;
        }
        const int j = two ? 2 * i + s : i;
        const int vs = next_tile();
        ok = vs >= 0;
        if (!ok) break;
        const int valid = len - tile_of(t_begin, n, from, i) * kAhKeys;
        if (valid < kAhKeys) {
          // values behind the sequence's end count 0 times, but 0 * NaN is NaN: they become zeros
          uint8_t* base = sKV + vs * Sm::kTile;
#pragma unroll 1
          for (int e = lane; e < (kAhKeys - valid) * 8; e += 32) {
#pragma unroll
            for (int blk = 0; blk < NB; ++blk)
              *reinterpret_cast<uint4*>(base + blk * kAhKvBlock + valid * 128 + e * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        int ks = 0;
        if (two && more) ks = next_tile();  // of one half memory sets the pace: no product waits for a tile it does not need
        ok = ks >= 0;
        if (ok && j < 2 && used) {  // the sums of the item before have been read
          ok = warp_wait(&o_free[s], of_ph, a);
          of_ph ^= 1u;
        }
        used = true;
        ok = ok && turn(job + firsts + j) && warp_wait(&p_ready[s], p_ph, a);
        if (!ok) break;
        p_ph ^= 1u;
        const uint32_t bd = v0 + vs * (Sm::kTile >> 4);
        tc_fence_after();
        if (elect_one()) {
          // P of a tile's halves: columns 0-31 and 64-95
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ta(o_tmem, s_tmem + (k >> 2) * 64 + (k & 3) * 8, sdesc_of(bd + k * 128), idesc_o, (j >= 2 || k) ? 1u : 0u);
          if (j + 2 >= jobs) mma_commit(smem_u32(&pv_done[s]));
          mma_commit(smem_u32(&kv_empty[vs]));
        }
        __syncwarp();
        if (more) {
          if (!two) ks = next_tile();
          ok = ks >= 0;
          if (!ok) break;
          scores(half, ks, j + 4 >= jobs);
        }
        issued(job + firsts + j);
      }
      if (!ok) break;
      job += firsts + jobs;
    }
    if (elect_one()) mma_commit(smem_u32(done));
    __syncwarp();
    (void)warp_wait(done, 0, a);
  } else {
    // -------------------------------------------------------------- softmax --
    const int s = warp >> 3;         // stream
    const int hf = (warp >> 2) & 1;  // half of a tile's keys
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + s * 128 + hf * 64, o_col = tmem + lanes + 256 + s * 128;
    const uint32_t mates = 1 + s * 4 + (warp & 3);  // barrier of the two warps that share these rows
    float* my_x = sX + (2 * s + hf) * kAhHalf + row;
    const float* mate_x = sX + (2 * s + 1 - hf) * kAhHalf + row;
    const int row_tok = static_cast<int>(quotient(row, a.inv_group)), row_head = row - row_tok * a.group;
    const f32x2 kx2 = pair(a.kx, a.kx);
    int slot = 0;
    uint32_t it_ph = 0, cl_ph = 0, s_ph = 0, pv_ph = 0;
    bool ok = true;
    while (true) {
      // A warp whose wait ran out goes through the rest of its item without waiting, as its mate counts on it at the
      // barriers, and both leave together here.
      if (!named_barrier_and(mates, 64, ok && warp_wait(&item_full[slot], it_ph, a))) break;
      const AhItem& it = items[slot];
      if (it.last) break;
      auto release = [&]() {  // of the descriptor
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&item_empty[slot]));
        if (++slot == kAhItems) {
          slot = 0;
          it_ph ^= 1u;
        }
      };
      const int t_begin = it.t_begin, n = it.t_end - t_begin, from = it.turn;
      const bool two = it.tokens > a.tq;
      const int tok = (two ? s * a.tq : 0) + row_tok;  // of the item
      const bool row_ok = row < a.tq * a.group && tok < it.tokens;
      const int limit = row_ok ? key_limit(a, it.fresh, it.len, it.first + tok) : 0x7fffffff;
      const bool active = __any_sync(0xffffffffu, row_ok);
      const int mine = two ? n : (n + 1 - s) >> 1;  // tiles of this stream
      float c = 0.f, l = 0.f;
      float least = kAhLeast;  // below 0: the row's scale c is settled
#pragma unroll 1
      for (int i = 0; i < mine; ++i) {
        const int t = tile_of(t_begin, n, from, two ? i : 2 * i + s);
        ok = ok && warp_wait(&s_ready[s], s_ph, a);
        s_ph ^= 1u;
        if (active) {
          tc_fence_after();
          const int lim = limit - t * kAhKeys - hf * 64;
          const bool masked = __any_sync(0xffffffffu, lim < 64);
          // Weights on the scale in hand, which is fine while none is far above 1; their sum tells that without a
          // maximum. Where a row outgrew its scale, or begins far below it, it gets one, and the tile is done again.
          // Scores come in two halves, so that nothing is spilled (chunk 1818 -> 1764 us, texts 69 -> 60.5).
          for (bool again = false;; again = true) {
            uint32_t sv[32];
            if (again) {
              // The scale of the tile's largest score, and l and O with it (O's last product was complete before
              // these scores were). Both warps of a row come here together, and the barrier makes each one's maximum
              // visible to the other. Their scores need none: a warp reads and overwrites its own half's columns only.
              float m0 = kNegInf, m1 = kNegInf;
#pragma unroll 1
              for (int h = 0; h < 64; h += 32) {
                tmem_ld32_wait(s_col + h, sv);
                if (masked) {
#pragma unroll
                  for (int e = 0; e < 32; ++e) sv[e] = e + h < lim ? sv[e] : 0xff800000u;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  m0 = max3(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]), m0);
                  m1 = max3(__uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3]), m1);
                }
              }
              float up = ceilf(fmaxf(m0, m1) * a.kx);
              *my_x = up;
              named_barrier_sync(mates, 64);
              up = fmaxf(up, *mate_x);
              const bool first = least > 0.f;  // l and O are 0 still
              const float top = row_ok && up > (first ? kNegInf : c + kAhMove) ? up : c;
              if (up > kNegInf) least = -1.f;
              if (__any_sync(0xffffffffu, top != c)) {
                const float f = first ? 1.f : pow2_diff(c, top);
                if (i > 0) {
#pragma unroll 1
                  for (int col = hf * 16; col < a.d; col += 32) {
                    uint32_t o[16];
                    tmem_ld16(o_col + col, o);
                    tmem_wait16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st16(o_col + col, o);
                  }
                }
                l *= f;
                c = top;
              }
            }
            const f32x2 nb2 = pair(-c, -c);
            f32x2 sum = pair(0.f, 0.f), sum1 = sum;
            uint32_t pk[32];
            auto weights = [&](int h) {
              if (masked) {
#pragma unroll
                for (int e = 0; e < 32; ++e) sv[e] = e + h < lim ? sv[e] : 0xff800000u;
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const f32x2 x = fma2(pair(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), kx2, nb2);
                const uint32_t w = pack_bf16(ex2_approx(lo(x)), ex2_approx(hi(x)));
                pk[h / 2 + e] = w;
                // the rounded weights are summed, so that they come to 1: a row that one key rules is exact
                const f32x2 p = pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
                if (e & 1)
                  sum1 = add2(sum1, p);
                else
                  sum = add2(sum, p);
              }
            };
            tmem_ld32_wait(s_col, sv);
            weights(0);
            tmem_ld32_wait(s_col + 32, sv);
            weights(32);
            sum = add2(sum, sum1);
            const float total = lo(sum) + hi(sum);
            if (!again) {
              const float need = masked && lim <= 0 ? -1.f : least;
              if (named_barrier_or(mates, 64, row_ok && !(total < kAhRoom && total > need))) continue;
              if (!masked || lim + hf * 64 > 0) least = -1.f;
            }
            tmem_st32(s_col, pk);
            l += total;
            break;
          }
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_ready[s]));
      }
      if (least > 0.f) c = kNegInf;  // the row has seen nothing
      const int other = two ? 0 : n >> 1;  // stream 1's tiles, where stream 0 joins both
      if (!two && s == 1) {
        // hand (c, l) over to stream 0, which reads both sums
        if (mine > 0) {
          ok = ok && warp_wait(&pv_done[s], pv_ph, a);
          pv_ph ^= 1u;
          sCL[hf * kAhHalf + row] = make_float2(c, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(cl_ready));
        }
        release();
        continue;
      }
      float top = c, f0 = 1.f, f1 = 0.f;
      if (n > 0) {
        // the row's whole sum, while the last product runs
        my_x[4 * kAhHalf] = l;
        named_barrier_sync(mates, 64);
        l += mate_x[4 * kAhHalf];
        if (other > 0) {
          // stream 1 arrives after its own last product, so that O of both is complete
          ok = ok && warp_wait(cl_ready, cl_ph, a);
          cl_ph ^= 1u;
          const float c1 = sCL[row].x;
          top = fmaxf(c, c1);
          f0 = pow2_diff(c, top), f1 = pow2_diff(c1, top);
          l = l * f0 + (sCL[row].y + sCL[kAhHalf + row].y) * f1;
        }
        ok = ok && warp_wait(&pv_done[s], pv_ph, a);
        pv_ph ^= 1u;
        tc_fence_after();
      }
      const float sum = l;
      if (active) {
        const bool sees = n > 0 && limit > 0;
        const float inv = 1.f / sum;
        const int r = (two ? s * kAhHalf : 0) + row;
        const bool whole = it.slot < 0;
        const int64_t my_row = whole ? (it.q_row + tok) * a.ld_o + static_cast<int64_t>(it.head * a.group + row_head) * a.d
                                     : (static_cast<int64_t>(it.slot) * a.slot_rows + r) * a.d;
#pragma unroll 1
        for (int col = hf * 16; col < a.d; col += 32) {  // the two warps of a row take turns
          uint32_t o[16];
          float x[16];
          if (n > 0) {
            tmem_ld16(o_col + col, o);
            tmem_wait16(o);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = n > 0 ? __uint_as_float(o[e]) * f0 : 0.f;
          if (other > 0) {
            tmem_ld16(o_col + 128 + col, o);
            tmem_wait16(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = fmaf(__uint_as_float(o[e]), f1, x[e]);
          }
          uint4 v[2];
          if (whole) {
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) pk[e] = sees ? pack_bf16(x[2 * e] * inv, x[2 * e + 1] * inv) : 0u;
            v[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            v[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            if (row_ok) {  // 16 channels: a sector, where rows start on one
              uint4* dst = reinterpret_cast<uint4*>(a.o + my_row + col);
              if (a.o_sectors) {
                st_global_v8(dst, v);
              } else {
                dst[0] = v[0];
                dst[1] = v[1];
              }
            }
          } else if (row_ok) {
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
#pragma unroll
              for (int b = 0; b < 2; ++b)
                v[b] = make_uint4(__float_as_uint(x[e + 4 * b]), __float_as_uint(x[e + 4 * b + 1]),
                                  __float_as_uint(x[e + 4 * b + 2]), __float_as_uint(x[e + 4 * b + 3]));
              uint4* dst = reinterpret_cast<uint4*>(a.part + my_row + col + e);
              if (a.part_sectors) {
                st_global_v8(dst, v);
              } else {
                dst[0] = v[0];
                dst[1] = v[1];
              }
            }
          }
          __syncwarp();
        }
        if (row_ok && it.slot >= 0 && hf == 0) {
          const bool any = limit > it.t_begin * kAhKeys;
          a.part_cl[static_cast<long long>(it.slot) * a.slot_rows + r] =
              make_float2(any && top == kNegInf ? kNoScore : top, sum);
        }
      }
      if (n > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&o_free[s]));
          if (other > 0) mbar_arrive(smem_u32(&o_free[1]));
        }
      }
      release();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kAhMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial sums of cut items: o = sum_p 2^(c_p - c) O_p / sum_p
// 2^(c_p - c) l_p over the pieces p of a row, c = max_p c_p. A CTA reads the
// directory that the runs' CTAs left and shares the cut items out evenly over the
// grid: an item cut at the end of run `first` has its first piece in that run's
// slot 1 and goes on in the slots 0 of the runs behind it. A warp takes four rows
// of an item of two pieces at once, else a row; where pieces are many, or CTAs
// enough, a CTA's warps share a row.
constexpr int kJoinThreads = 256;

__device__ __forceinline__ void join_store(const AhArgs& a, int q_row, int h, int i, int lane, float top, float l, float4 v) {
  const int tok = static_cast<int>(quotient(i, a.inv_group));
  const float inv = 1.f / l;
  const bool sees = top != kNegInf;
  *reinterpret_cast<uint2*>(a.o + static_cast<long long>(q_row + tok) * a.ld_o +
                            static_cast<long long>(h * a.group + i - tok * a.group) * a.d + lane * 4) =
      sees ? make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv)) : make_uint2(0u, 0u);
}

__global__ void __launch_bounds__(kJoinThreads) attn_heads_join_kernel(const __grid_constant__ AhArgs a, int ctas) {
  __shared__ float sO[8][128];
  __shared__ float2 sL[8];  // (c, l)
  constexpr int kWords = (kAhMaxCtas + 31) / 32;
  __shared__ unsigned sCut[kWords], sOn[kWords];  // runs whose last item is cut; runs whose first item goes on behind them
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  for (int w = warp; w < kWords; w += kJoinThreads / 32) {
    const int j = w * 32 + lane;
    const int cut_here = j < ctas ? a.meta[2 * j + 1].x : 0, on_here = j < ctas ? a.meta[2 * j].x : 0;
    const unsigned cut = __ballot_sync(0xffffffffu, cut_here != 0), on = __ballot_sync(0xffffffffu, on_here == 1);
    if (lane == 0) sCut[w] = cut, sOn[w] = on;
  }
  __syncthreads();
  int items = 0;
#pragma unroll
  for (int w = 0; w < kWords; ++w) items += __popc(sCut[w]);
  if (items == 0) return;
  const int share = gridDim.x / items;  // CTAs of an item: at least one, as the grid has as many as there are runs
  const int item = blockIdx.x / share, y = blockIdx.x - item * share;
  if (item >= items) return;
  // the item's first run, and the one that ends it
  int at_word = 0, skip = item;
  while (skip >= __popc(sCut[at_word])) skip -= __popc(sCut[at_word++]);
  unsigned bits = sCut[at_word];
  while (skip-- > 0) bits &= bits - 1;
  const int first = at_word * 32 + __ffs(bits) - 1;
  at_word = (first + 1) >> 5;
  bits = at_word < kWords ? ~sOn[at_word] & ~0u << ((first + 1) & 31) : 1u;
  while (bits == 0 && ++at_word < kWords) bits = ~sOn[at_word];
  const int last = min(ctas - 1, at_word < kWords ? at_word * 32 + __ffs(bits) - 1 : ctas);
  const int pieces = last - first + 1;
  const int4 head = a.meta[2 * first + 1];
  const int q_row = head.y, tokens = head.z, h = head.w;
  const bool two = tokens > a.tq;
  const int rows = tokens * a.group;
  // row i of an item in a piece's slot
  auto slot_of = [&](int p, int i) {
    const int tok = static_cast<int>(quotient(i, a.inv_group));
    const int r = two && tok >= a.tq ? kAhHalf + i - a.tq * a.group : i;
    return static_cast<long long>(p == 0 ? 2 * first + 1 : 2 * (first + p)) * a.slot_rows + r;
  };
  const bool on = lane * 4 < a.d;
  if (pieces <= 2 && share * 8 < rows) {
    for (int i0 = (y * 8 + warp) * 4; i0 < rows; i0 += share * 32) {
      float2 cl[8];
      float4 v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const long long at = slot_of(min(e & 1, pieces - 1), min(i0 + (e >> 1), rows - 1));
        cl[e] = a.part_cl[at];
        v[e] = on ? *reinterpret_cast<const float4*>(a.part + at * a.d + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if (i0 + (e >> 1) >= rows || !on) continue;
        const float top = fmaxf(cl[e].x, cl[e + 1].x);
        const float f0 = pow2_diff(cl[e].x, top), f1 = pieces > 1 ? pow2_diff(cl[e + 1].x, top) : 0.f;
        join_store(a, q_row, h, i0 + (e >> 1), lane, top, fmaf(cl[e].y, f0, cl[e + 1].y * f1),
                   make_float4(fmaf(v[e].x, f0, v[e + 1].x * f1), fmaf(v[e].y, f0, v[e + 1].y * f1),
                               fmaf(v[e].z, f0, v[e + 1].z * f1), fmaf(v[e].w, f0, v[e + 1].w * f1)));
      }
    }
    return;
  }
  // rounds of loads that a row to a warp, and a row to a CTA take
  const int alone = (rows + share * 8 - 1) / (share * 8) * ((pieces + 7) / 8);
  const int together = (rows + share - 1) / share * ((pieces + 63) / 64);
  const bool shared_rows = together <= alone;
  for (int i0 = shared_rows ? y : y * 8; i0 < rows; i0 += shared_rows ? share : share * 8) {
    const int i = shared_rows ? i0 : i0 + warp;
    if (!shared_rows && i >= rows) break;
    float top = kNegInf, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int by = shared_rows ? 8 : 1;
    for (int p0 = shared_rows ? warp : 0; p0 < pieces; p0 += 8 * by) {  // eight pieces in flight
      float2 cl[8];
      float4 v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int p = p0 + e * by;
        const long long at = slot_of(min(p, pieces - 1), i);
        cl[e] = p < pieces ? a.part_cl[at] : make_float2(kNegInf, 0.f);
        v[e] = p < pieces && on ? *reinterpret_cast<const float4*>(a.part + at * a.d + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float up = top;
#pragma unroll
      for (int e = 0; e < 8; ++e) up = fmaxf(up, cl[e].x);
      const float old = pow2_diff(top, up);
      l *= old;
      acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
      top = up;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = pow2_diff(cl[e].x, top);
        l = fmaf(cl[e].y, f, l);
        acc.x = fmaf(v[e].x, f, acc.x);
        acc.y = fmaf(v[e].y, f, acc.y);
        acc.z = fmaf(v[e].z, f, acc.z);
        acc.w = fmaf(v[e].w, f, acc.w);
      }
    }
    if (shared_rows) {
      *reinterpret_cast<float4*>(&sO[warp][lane * 4]) = acc;
      if (lane == 0) sL[warp] = make_float2(top, l);
      __syncthreads();
      if (warp == 0) {
        for (int w = 0; w < 8; ++w) top = fmaxf(top, sL[w].x);
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < 8; ++w) {
          const float f = pow2_diff(sL[w].x, top);
          const float4 v = *reinterpret_cast<const float4*>(&sO[w][lane * 4]);
          acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y), acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
          l = fmaf(sL[w].y, f, l);
        }
      }
      __syncthreads();
    }
    if (on && (!shared_rows || warp == 0)) join_store(a, q_row, h, i, lane, top, l, acc);
  }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kAhMaxHeads = 65536;
constexpr int kAhMaxRows = 1 << 30;
// Every CTA counts all sequences before its first item, while its other warps' waits of two seconds run: so many take
// 0.03 s of one row each, 0.28 of two items each other one, 0.15 where nearly all are empty and one CTA skips them one by
// one, 0.54 of three rows of 128 heads.
constexpr int kAhMaxSeqs = 1 << 20;
constexpr double kAhMaxSpan = 0x1p38;  // elements from an instance's keys to the next one's stay below

cc_status check_attn(const char* what, const void* q, const void* k, const void* v, const void* o, int heads,
                     int kv_heads, int d, int64_t ld_q, int64_t ld_o, float scale) {
  if (!q || !o || !k || !v) return fail(CC_ERR_INVALID, "%s: null pointer", what);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
    return fail(CC_ERR_INVALID, "%s: pointers must be 16-byte aligned", what);
  if (heads <= 0 || kv_heads <= 0 || d <= 0 || heads % kv_heads != 0)
    return fail(CC_ERR_INVALID, "%s: the query heads must be a multiple of the key heads (got %d and %d)", what, heads,
                kv_heads);
  if (d % 16 != 0 || d > 128)
    return fail(CC_ERR_UNSUPPORTED, "%s: D must be a multiple of 16 up to 128 (got %d)", what, d);
  if (heads > kAhMaxHeads || heads / kv_heads > kAhHalf)
    return fail(CC_ERR_UNSUPPORTED, "%s: at most 65536 heads, 128 to a key head", what);
  if (ld_q < (int64_t)heads * d || ld_o < (int64_t)heads * d || ld_q % 8 || ld_o % 8)
    return fail(CC_ERR_INVALID, "%s: row strides must hold the heads and be multiples of 8", what);
  if (ld_q >= (1ll << 38) || ld_o >= (1ll << 38))
    return fail(CC_ERR_UNSUPPORTED, "%s: row strides must be below 2^38 elements", what);
  if (!(scale > 0.f) || !std::isfinite(scale * kLog2e))
    return fail(CC_ERR_INVALID, "%s: scale must be > 0, and finite times log2(e)", what);
  return CC_OK;
}

constexpr int kFewRows = 8;        // query rows of an item of the few-rows kernel: the n of its products
// As above, in its tiles. 64 streams of 100 to 1000 keys: 15.4 us with up to 8, 19.2 with 12; 128 of 50 to 600: 47.5
// and 46.6.
constexpr int kFewSplitCost = 6;

// Its tiles: 128 keys, 64 of heads of more than 64 channels.
int few_tile_shift(int d) { return d > 64 ? 6 : 7; }

// Few rows to a sequence on average: the kernel whose CTAs do little but read the
// cache. (The other one takes 128 rows of a key head at once: 246 us instead of
// 180 for single tokens of 64 streams with four heads to a key head. With more
// rows than fit one item the keys are read again for each eight of them.)
//
// The lengths of a plan are on the device, so the host knows the average alone and a
// call is one kernel's. That holds for steps whose sequences are alike; a prompt beside
// single tokens makes one of the two wait for a kernel that is not its own. Heads of
// 128, in us: 64 tokens over 4096 keys each 170 and 400 rows over 4096 32, together 188;
// 255 tokens over 2048 327 and 1793 rows over 8192 69, together 681 here and 448 with one
// row more in the other kernel; with four heads to a key head 32 tokens over 4096 84 and
// 2000 rows 76, together 199; 64 tokens 172 and 400 rows over 4096 48, together 234. A
// caller that has both kinds can make a call for each.
bool few_rows(int64_t rows, int64_t seqs, int group) { return group <= kFewRows && rows * group <= kFewRows * seqs; }

// Rows that a partial slot holds: those of all tokens where an item (of the
// kernel for few rows) or half of one has room for them.
int slot_rows(bool few, int64_t tokens, int group) {
  const int tq = (few ? kFewRows : kAhHalf) / group;
  return tokens <= tq ? static_cast<int>(tokens) * group : few ? kFewRows : 2 * kAhHalf;
}

// Tokens of an item, see AhArgs.
int item_tokens(bool few, int group) { return few ? kFewRows / group : 2 * (kAhHalf / group); }

// Tiles are counted in 31 bits. tiles: of a sequence, at most
bool too_many_tiles(int64_t rows, int64_t seqs, int item_tokens, int64_t kv_heads, int64_t tiles) {
  return ((rows / item_tokens + seqs) * kv_heads) * (double)tiles >= 0x1p31;
}

size_t part_bytes(int ctas, int rows, int d) { return (size_t)2 * ctas * rows * d * 4; }

size_t workspace_bytes(bool few, int64_t tokens, int group, int d) {
  const int ctas = few ? kAhMaxCtas : kAhMaxCtas / 2, rows = slot_rows(few, tokens, group);
  return part_bytes(ctas, rows, d) + (size_t)2 * ctas * (rows * 8 + 16);
}

struct CacheSide {
  const cc_bf16* p;
  int64_t page, token, head;
};

cc_status encode_side(CUtensorMap* map, const CacheSide& c, const AhArgs& a) {
  const uint64_t dims[4] = {(uint64_t)a.d, (uint64_t)a.kv_heads, (uint64_t)a.plan.page_size, (uint64_t)a.plan.pages};
  const uint64_t strides[3] = {2ull * c.head, 2ull * c.token, 2ull * c.page};
  return encode_tiled_4d(map, c.p, dims, strides, 64, 1, a.box);
}

template <int NB, int STAGES>
cc_status launch_attn(const char* what, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, AhArgs& a,
                      int grid, cudaStream_t stream) {
  auto kern = attn_heads_kernel<NB, STAGES>;
  constexpr int kSmem = AhSmem<NB, STAGES>::kBytes;
  static_assert(kSmem <= 232448, "shared memory budget");
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kSmem, a.device, ready);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: shared-memory attribute: %s", what, cudaGetErrorString(e));
  e = launch_pdl(kern, dim3(grid), dim3(kAhThreads), kSmem, stream, tq, tk, tv, a);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: launch: %s", what, cudaGetErrorString(e));
  return launch_status(what);
}

// keys: no sequence has more; max_tokens: nor new tokens; seqs: sequences that the rows belong to.
cc_status run_attn(const char* what, AhArgs& a, const cc_bf16* q, int64_t ld_q, const CacheSide& k, const CacheSide& v,
                   int64_t keys, int64_t max_tokens, void* ws, size_t ws_bytes, void* stream) {
  a.group = a.heads / a.kv_heads;
  const bool few = few_rows(a.rows, a.plan.seqs, a.group);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.ld_q = ld_q;
  a.o_sectors = reinterpret_cast<uintptr_t>(a.o) % 32 == 0 && a.ld_o % 16 == 0;
  a.tq = (few ? kFewRows : kAhHalf) / a.group;
  a.item_tokens = item_tokens(few, a.group);
  a.tile_shift = few ? few_tile_shift(a.d) : kAhTileShift;
  a.split_cost = few ? kFewSplitCost : kAhSplitCost;
  const int tile = 1 << a.tile_shift;
  a.box = std::min(tile, a.box);
  const int64_t tiles = std::max<int64_t>(1, (keys + tile - 1) / tile);
  if (too_many_tiles(a.rows, a.plan.seqs, a.item_tokens, a.kv_heads, tiles))
    return fail(CC_ERR_UNSUPPORTED, "%s: rows, heads and keys make 2^31 tiles or more", what);
  a.may_split = tiles > a.split_cost;
  a.slot_rows = slot_rows(few, max_tokens, a.group);
  DeviceInfo di;
  cc_status st;
  if (a.may_split) {
    const size_t need = workspace_bytes(few, max_tokens, a.group, a.d);
    if (!ws) return fail(CC_ERR_INVALID, "%s: null workspace", what);
    if (!aligned16(ws)) return fail(CC_ERR_INVALID, "%s: pointers must be 16-byte aligned", what);
    if (ws_bytes < need) return fail(CC_ERR_INVALID, "%s: workspace of %zu bytes, need %zu", what, ws_bytes, need);
    const int ctas = few ? kAhMaxCtas : kAhMaxCtas / 2;
    a.part = static_cast<float*>(ws);
    a.part_sectors = reinterpret_cast<uintptr_t>(ws) % 32 == 0;
    a.part_cl = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + part_bytes(ctas, a.slot_rows, a.d));
    a.meta = reinterpret_cast<int4*>(a.part_cl + (size_t)2 * ctas * a.slot_rows);
  }
  if ((st = device_info(&di)) != CC_OK) return st;
  a.err = di.err_word;
  a.device = di.device;
  CUtensorMap tk = {}, tv = {};
  if (keys > 0 && ((st = encode_side(&tk, k, a)) != CC_OK || (st = encode_side(&tv, v, a)) != CC_OK)) return st;
  const int grid = std::min(kAhMaxCtas, 2 * di.sm_count) / (few ? 1 : 2);
  a.inv_ctas = inverse(grid);
  a.inv_tokens = inverse(a.item_tokens);
  a.inv_block = a.block ? inverse(a.block) : 0;
  a.inv_group = inverse(a.group);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (few) {
    st = launch_few_rows(what, tk, tv, a, grid, cs);
  } else {
    CUtensorMap tq = {};
    const uint64_t qdims[4] = {(uint64_t)a.d, (uint64_t)a.heads, (uint64_t)a.rows, 1};
    const uint64_t qstrides[3] = {2ull * a.d, 2ull * ld_q, 2ull * ld_q};
    if ((st = encode_tiled_4d(&tq, q, qdims, qstrides, 64, a.group, a.tq)) != CC_OK) return st;
    st = a.d > 64 ? launch_attn<2, 4>(what, tq, tk, tv, a, grid, cs) : launch_attn<1, 8>(what, tq, tk, tv, a, grid, cs);
  }
  if (st != CC_OK || !a.may_split) return st;
  // the joining kernel's CTAs: as many as give each of their warps four rows of an item to each run
  const int join = grid * ((a.slot_rows + 31) / 32);
  const cudaError_t e = launch_pdl(attn_heads_join_kernel, dim3(join), dim3(kJoinThreads), 0, cs, a, grid);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: launch: %s", what, cudaGetErrorString(e));
  return launch_status(what);
}

// Sizes that the calls take, as far as a workspace's size depends on them.
bool sizes_ok(int64_t rows, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t d) {
  return rows <= kAhMaxRows && seqs <= kAhMaxSeqs && heads > 0 && heads <= kAhMaxHeads && kv_heads > 0 &&
         heads % kv_heads == 0 && heads / kv_heads <= kAhHalf && d > 0 && d % 16 == 0 && d <= 128;
}

}  // namespace
}  // namespace cc

using namespace cc;

extern "C" size_t cc_attn_paged_workspace_bytes(int rows, int seqs, int heads, int kv_heads, int d) {
  if (rows <= 0 || seqs <= 0 || !sizes_ok(rows, seqs, heads, kv_heads, d)) return 0;
  const int group = heads / kv_heads;
  return workspace_bytes(few_rows(rows, seqs, group), rows, group, d);
}

extern "C" size_t cc_attn_cross_workspace_bytes(int n, int lq, int lk, int heads, int kv_heads, int d) {
  if (n <= 0 || lq <= 0 || !sizes_ok((int64_t)n * lq, n, heads, kv_heads, d)) return 0;
  const int group = heads / kv_heads;
  const bool few = few_rows((int64_t)n * lq, n, group);
  const int shift = few ? few_tile_shift(d) : kAhTileShift;
  if (lk <= (few ? kFewSplitCost : kAhSplitCost) << shift) return 0;  // nothing is cut
  const int64_t tiles = ((int64_t)lk + (1 << shift) - 1) >> shift;
  if (too_many_tiles((int64_t)n * lq, n, item_tokens(few, group), kv_heads, tiles)) return 0;
  if ((double)kv_heads * d * lk >= kAhMaxSpan) return 0;
  return workspace_bytes(few, lq, group, d);
}

extern "C" cc_status cc_attn_paged(const cc_bf16* q, const cc_bf16* k_cache, const cc_bf16* v_cache, cc_bf16* o,
                                   const int32_t* q_offsets, const int32_t* kv_lens, const int32_t* page_table,
                                   int rows, int seqs, int max_pages, int pages, int page_size, int heads,
                                   int kv_heads, int d, int64_t ld_q, int64_t ld_o, int64_t k_page, int64_t k_token,
                                   int64_t k_head, int64_t v_page, int64_t v_token, int64_t v_head, float scale,
                                   int causal_block, void* ws, size_t ws_bytes, void* stream) {
  const char* what = "attn_paged";
  cc_status st;
  if (empty_request(what, {rows, seqs}, &st)) return st;
  if ((st = check_attn(what, q, k_cache, v_cache, o, heads, kv_heads, d, ld_q, ld_o, scale)) != CC_OK) return st;
  if ((st = check_plan(what, q_offsets, kv_lens, page_table, max_pages, pages, page_size)) != CC_OK) return st;
  if ((st = check_cache_strides(what, k_page, k_token, k_head, pages, kv_heads, d)) != CC_OK ||
      (st = check_cache_strides(what, v_page, v_token, v_head, pages, kv_heads, d)) != CC_OK)
    return st;
  if (rows > kAhMaxRows) return fail(CC_ERR_UNSUPPORTED, "%s: at most 2^30 rows", what);
  if (seqs > kAhMaxSeqs) return fail(CC_ERR_UNSUPPORTED, "%s: at most 2^20 sequences", what);
  if (causal_block < 0) return fail(CC_ERR_INVALID, "%s: the causal block must not be negative", what);
  AhArgs a = {};
  a.plan = {q_offsets, kv_lens, page_table, seqs, max_pages, pages, page_size};
  a.rows = rows;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.d = d;
  a.box = page_size & -page_size;
  a.o = reinterpret_cast<__nv_bfloat16*>(o);
  a.ld_o = ld_o;
  a.kx = scale * kLog2e;
  a.block = std::min(causal_block, 1 << 30);
  return run_attn(what, a, q, ld_q, {k_cache, k_page, k_token, k_head}, {v_cache, v_page, v_token, v_head},
                  (int64_t)max_pages * page_size, rows, ws, ws_bytes, stream);
}

extern "C" cc_status cc_attn_cross(const cc_bf16* q, const cc_bf16* k, const cc_bf16* v, cc_bf16* o,
                                   const int32_t* kv_lens, int n, int lq, int lk, int heads, int kv_heads, int d,
                                   int64_t ld_q, int64_t ld_k, int64_t ld_v, int64_t ld_o, float scale, void* ws,
                                   size_t ws_bytes, void* stream) {
  const char* what = "attn_cross";
  cc_status st;
  if (empty_request(what, {n, lq}, &st)) return st;
  if (lk < 0) return fail(CC_ERR_INVALID, "%s: sizes must not be negative", what);
  if ((st = check_attn(what, q, lk ? k : q, lk ? v : q, o, heads, kv_heads, d, ld_q, ld_o, scale)) != CC_OK) return st;
  if (!aligned16(kv_lens)) return fail(CC_ERR_INVALID, "%s: pointers must be 16-byte aligned", what);
  if (ld_k < (int64_t)kv_heads * d || ld_v < (int64_t)kv_heads * d || ld_k % 8 || ld_v % 8)
    return fail(CC_ERR_INVALID, "%s: row strides must hold the heads and be multiples of 8", what);
  if ((int64_t)n * lq > kAhMaxRows) return fail(CC_ERR_UNSUPPORTED, "%s: at most 2^30 rows", what);
  if (n > kAhMaxSeqs) return fail(CC_ERR_UNSUPPORTED, "%s: at most 2^20 instances", what);
  if ((double)ld_k * lk >= kAhMaxSpan || (double)ld_v * lk >= kAhMaxSpan)
    return fail(CC_ERR_UNSUPPORTED, "%s: an instance's keys must lie within 2^38 elements", what);
  AhArgs a = {};
  a.plan = {nullptr, kv_lens, nullptr, n, 1, n, lk};
  a.lq = lq;
  a.rows = n * lq;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.d = d;
  a.box = 1 << 30;
  a.o = reinterpret_cast<__nv_bfloat16*>(o);
  a.ld_o = ld_o;
  a.kx = scale * kLog2e;
  return run_attn(what, a, q, ld_q, {k, ld_k * lk, ld_k, d}, {v, ld_v * lk, ld_v, d}, lk, lq, ws, ws_bytes, stream);
}
