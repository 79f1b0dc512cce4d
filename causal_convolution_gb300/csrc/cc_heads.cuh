// What the attention kernels with heads share: the items of work and how the
// CTAs of a persistent grid divide them, waits, and the arithmetic of partial
// sums.
//
// An item is up to item_tokens new tokens of one sequence, with the query heads
// of one key head, and all the key tiles that any of them sees. The items' tiles,
// laid end to end (sequence, tokens, head), are cut into equal runs, one for each
// CTA. An item cut by a run's end leaves partial sums in the workspace, which a
// second kernel joins; where whole items spread well enough nothing is cut. The
// lengths are read on the device, so every CTA finds its run by itself.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cc_host.h"
#include "cc_paged.cuh"
#include "cc_ptx.cuh"
#include "cc_rows.cuh"

namespace cc {

constexpr int kAhMaxCtas = 304;   // two per SM of a GB300
constexpr int kAhItems = 4;       // item descriptors in flight

struct AhArgs {
  KvPlan plan;      // q_offsets nullptr: sequence b owns rows b * lq .. (b + 1) * lq - 1; page_table nullptr: page b
  int lq;
  int rows, heads, kv_heads, group, d;
  int tq;           // tokens of a half: as many as fit its rows
  int item_tokens;  // of an item: one half or two
  int tile_shift;   // keys of a tile: 2^tile_shift
  int split_cost;   // tiles that cutting items costs a call, on its critical path
  int box;          // slots per TMA box: pieces of this size never cross a page
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  long long ld_q, ld_o;
  int o_sectors, part_sectors;  // rows of o, of partial sums start on 32-byte borders
  float kx;         // scale * log2(e)
  unsigned block;   // causal block, 0: none
  int may_split;
  int slot_rows;    // rows a partial slot holds
  float* part;      // [2 * ctas][slot_rows][d]
  float2* part_cl;  // [2 * ctas][slot_rows] (c, l)
  int4* meta;       // [2 * ctas]: 0 unused, 1 goes on, 2 ends its item; first row, tokens, head
  unsigned int* err;
  int device;
  // ceil(2^64 / divisor) for quotient(): CTAs, tokens of an item, the causal block, heads of a group
  unsigned long long inv_ctas, inv_tokens, inv_block, inv_group;
};

// x / divisor: exact, as x and the divisors are below 2^31. 0 stands for a divisor of 1.
__host__ __device__ constexpr unsigned long long inverse(unsigned divisor) { return divisor == 1 ? 0 : ~0ull / divisor + 1; }
__device__ __forceinline__ unsigned quotient(unsigned x, unsigned long long inv) {
  return inv ? static_cast<unsigned>(__umul64hi(x, inv)) : x;
}

// A piece of an item, as the roles of a CTA pass it on.
struct __align__(16) AhItem {
  int q_row;        // row of the item's first token
  int tokens;       // of the item
  int head;         // key head
  int t_begin, t_end, t_all;  // this piece's key tiles, of all
  int len;          // keys of the sequence
  int first;        // the item's first token among the new ones
  int fresh;        // new tokens of the sequence
  int slot;         // partial slot, -1: the whole item
  int seq;
  int last;         // no item: the CTA is done
  int turn;         // the piece's tiles are taken from t_begin + turn on, around its end
};

struct Seq {
  int begin, n, len, m;  // first row, new tokens, keys, items along the rows
};

__device__ __forceinline__ Seq load_seq(const AhArgs& a, int b) {
  Seq s = {0, 0, 0, 0};
  if (b >= a.plan.seqs) return s;
  if (a.plan.q_offsets) {
    s.begin = a.plan.q_offsets[b];
    const int end = a.plan.q_offsets[b + 1];
    s.len = a.plan.kv_lens[b];
    const long long n = static_cast<long long>(end) - s.begin;
    if (n != 0 && (n < 0 || s.begin < 0 || end > a.rows || s.len < 0 || (a.block && s.len < n) ||
                   s.len > static_cast<long long>(a.plan.max_pages) * a.plan.page_size)) {
      atomicOr(a.err, DEVERR_BOUNDS);
      return {0, 0, 0, 0};
    }
    s.n = static_cast<int>(n);
  } else {
    s.begin = b * a.lq;
    s.n = a.lq;
    s.len = a.plan.page_size;
    if (a.plan.kv_lens) {
      const int len = a.plan.kv_lens[b];
      if (len < 0 || len > s.len) atomicOr(a.err, DEVERR_BOUNDS);
      s.len = max(0, min(len, s.len));
    }
  }
  s.m = static_cast<int>(quotient(s.n + a.item_tokens - 1, a.inv_tokens));
  return s;
}

// How many of a sequence's keys its i-th new token sees.
__device__ __forceinline__ int key_limit(const AhArgs& a, int n, int len, int i) {
  if (a.block == 0) return len;
  const unsigned end = (quotient(i, a.inv_block) + 1) * a.block;
  return len - n + static_cast<int>(min(static_cast<unsigned>(n), end));
}

// Key tiles of the m-th item of a sequence.
__device__ __forceinline__ int item_tiles(const AhArgs& a, const Seq& s, int m) {
  const int lim = key_limit(a, s.n, s.len, min(s.n, (m + 1) * a.item_tokens) - 1);
  return static_cast<int>((static_cast<unsigned>(lim) + (1u << a.tile_shift) - 1) >> a.tile_shift);
}

// Inclusive sums over the lanes.
__device__ __forceinline__ unsigned warp_scan(unsigned v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

__device__ __forceinline__ Seq seq_of_lane(const Seq& s, int src) {
  return {__shfl_sync(0xffffffffu, s.begin, src), __shfl_sync(0xffffffffu, s.n, src),
          __shfl_sync(0xffffffffu, s.len, src), __shfl_sync(0xffffffffu, s.m, src)};
}

// Units of work of lane's sequence over all heads: its tiles, at least one to an
// item. most: the tiles of its largest item, the last one. Whole warps call it: the
// items of a causal sequence are summed by all lanes.
__device__ __forceinline__ unsigned seq_units(const AhArgs& a, const Seq& s, int lane, int& most) {
  most = s.m > 0 ? max(1, item_tiles(a, s, s.m - 1)) : 0;
  unsigned w = static_cast<unsigned>(s.m) * most;
  unsigned todo = __ballot_sync(0xffffffffu, s.m > 1 && a.block != 0);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    const Seq one = seq_of_lane(s, src);
    unsigned sum = 0;
    for (int i = lane; i < one.m; i += 32) sum += max(1, item_tiles(a, one, i));
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == src) w = sum;
  }
  return w * a.kv_heads;
}

// A CTA's run of units [at, end) and where it stands: sequence, item, head and
// tile. All lanes of a warp hold the same values.
struct Run {
  unsigned at, end, start;
  bool split;
  int b;
  Seq s;
  int m, h, t, tiles;  // tiles: of the item
};

// Finds the CTA's run; false if it is empty. (The host has made sure that units
// stay below 2^31. This runs once, on cold instructions, before anything else can
// start: what counts is that it is short.)
__device__ __forceinline__ bool find_run(const AhArgs& a, int cta, int ctas, int lane, Run& r) {
  unsigned w = 0, units = 0, items = 0;
  int most = 0, top = 0;
  Seq s = {};
  r.b = -1;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {  // all sequences' units; then the sequence of the run's first one
    unsigned before = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.plan.seqs; b0 += 32) {
      if (pass == 0 || a.plan.seqs > 32) {  // else the lanes still hold the only ones
        s = load_seq(a, b0 + lane);
        w = seq_units(a, s, lane, most);
      }
      if (pass == 0) {
        units += w;
        items += static_cast<unsigned>(s.m) * a.kv_heads;
        top = max(top, most);
      } else {
        const unsigned upto = before + warp_scan(w, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, r.at < upto);
        if (hit) {
          const int src = __ffs(hit) - 1;
          r.b = b0 + src;
          r.s = seq_of_lane(s, src);
          before = __shfl_sync(0xffffffffu, upto - w, src);
          break;
        }
        before = __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    if (pass == 0) {
      units = __reduce_add_sync(0xffffffffu, units);
      items = __reduce_add_sync(0xffffffffu, items);
      top = __reduce_max_sync(0xffffffffu, top);
      const unsigned per = max(2u, quotient(units + ctas - 1, a.inv_ctas));
      // What the longest run would be with whole items: as many of the average's size as come to a CTA, at least the
      // largest one; where sequences differ, a large item may start behind small ones. Against it cut ones, whose
      // partial sums have to be written, read and joined; where there are as many items as CTAs, a run has two of them,
      // both cut, to begin and to end.
      const float avg = __fdividef(static_cast<float>(units), static_cast<float>(items)), largest = static_cast<float>(top);
      float whole = fmaxf(largest, static_cast<float>(quotient(items + ctas - 1, a.inv_ctas)) * avg);
      if (a.plan.seqs > 1) whole += 0.5f * (largest - avg);
      const float cost = a.split_cost * fminf(2.f, 1.f + __fdividef(static_cast<float>(items), static_cast<float>(ctas)));
      r.split = a.may_split && whole > static_cast<float>(per) + cost;
      r.at = r.start = cta * per;
      r.end = min(units, r.at + per);
      if (r.at >= units) return false;
    } else {
      w = r.at - before;  // into the sequence
    }
  }
  if (r.b < 0) return false;  // lengths that changed meanwhile
  for (int m0 = 0; m0 < r.s.m; m0 += 32) {
    const int m = m0 + lane;
    const int tiles = m < r.s.m ? item_tiles(a, r.s, m) : 0;
    const unsigned size = m < r.s.m ? static_cast<unsigned>(max(1, tiles)) * a.kv_heads : 0;
    const unsigned upto = warp_scan(size, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, w < upto);
    if (hit) {
      const int src = __ffs(hit) - 1;
      r.m = m0 + src;
      r.tiles = __shfl_sync(0xffffffffu, tiles, src);
      w -= __shfl_sync(0xffffffffu, upto - size, src);
      // w / tiles is below 2^16, so a quotient of floats is at most one off
      const int len = max(1, r.tiles);
      r.h = static_cast<int>(__fdividef(static_cast<float>(w), static_cast<float>(len)));
      r.t = static_cast<int>(w) - r.h * len;
      if (r.t < 0) --r.h, r.t += len;
      if (r.t >= len) ++r.h, r.t -= len;
      return true;
    }
    w -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// On to the next item (its units start at r.at).
__device__ __forceinline__ void next_item(const AhArgs& a, Run& r) {
  r.t = 0;
  if (++r.h < a.kv_heads) return;
  r.h = 0;
  if (++r.m >= r.s.m) {
    r.m = 0;
    do {
      r.s = load_seq(a, ++r.b);
    } while (r.s.m == 0 && r.b < a.plan.seqs);
    if (r.s.m == 0) return;
  }
  r.tiles = item_tiles(a, r.s, r.m);
}

// 2^(c - top) for scales c <= top: a power of two, 0 where it would be subnormal
// (or c is -inf), 1 where both are the same infinity.
__device__ __forceinline__ float pow2_diff(float c, float top) {
  if (c == top) return 1.f;
  const float e = c - top;
  return e > -127.f ? __int_as_float((127 + static_cast<int>(e)) << 23) : 0.f;
}

constexpr float kNegInf = -INFINITY;
// c of a row all of whose visible scores are -inf: its sum is 0 and its result NaN
constexpr float kNoScore = -3.0e38f;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

// A whole warp's wait for a phase of an mbarrier, of about two seconds at most.
// There are many of these and the instruction cache is small, so it is a loop of
// few instructions that looks at the low half of the SM's clock alone (a try
// returns within far less than the part of its range that is left).
constexpr uint32_t kAhWaitClocks = 0xf0000000u;
__device__ __forceinline__ uint32_t clock_low() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%clock;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool warp_wait(const uint64_t* bar, uint32_t parity, const AhArgs& a) {
  const uint32_t at = smem_u32(bar), since = clock_low();
#pragma unroll 1
  while (!__all_sync(0xffffffffu, mbar_try_wait(at, parity))) {
    if (__any_sync(0xffffffffu, clock_low() - since > kAhWaitClocks)) {
      atomicOr(a.err, DEVERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The piece of an item at the head of a run; says in the workspace's directory
// where its partial sums go on or end.
__device__ __forceinline__ AhItem make_item(const AhArgs& a, const Run& r, int lane) {
  AhItem it = {};
  it.first = r.m * a.item_tokens;
  it.tokens = min(a.item_tokens, r.s.n - it.first);
  it.q_row = r.s.begin + it.first;
  it.head = r.h;
  it.len = r.s.len;
  it.fresh = r.s.n;
  it.seq = r.b;
  it.t_all = r.tiles;
  it.t_begin = r.t;
  it.t_end = r.split ? min(it.t_all, r.t + static_cast<int>(r.end - r.at)) : it.t_all;
  // CTAs whose items have the same keys take the same tile at about the same time, so that it is read from memory
  // once: each goes on from where its number of tiles so far points to.
  it.turn = 0;
  if (it.t_end > it.t_begin) {
    const unsigned done = r.at - r.start, all = static_cast<unsigned>(it.t_all);
    const int here = static_cast<int>(done % all) - it.t_begin;
    if (here > 0 && here < it.t_end - it.t_begin) it.turn = here;
  }
  it.slot = -1;
  if (it.t_begin > 0 || it.t_end < it.t_all) {
    it.slot = 2 * blockIdx.x + (it.t_begin > 0 ? 0 : 1);
    if (lane == 0) a.meta[it.slot] = make_int4(it.t_end < it.t_all ? 1 : 2, it.q_row, it.tokens, it.head);
  }
  return it;
}

// The tile that a piece takes as its i-th.
__device__ __forceinline__ int tile_of(int t_begin, int n, int turn, int i) {
  const int at = i + turn;
  return t_begin + (at >= n ? at - n : at);
}

// Launches the kernel for few rows to a sequence (attn_few_rows.cu).
cc_status launch_few_rows(const char* what, const CUtensorMap& tk, const CUtensorMap& tv, AhArgs& a, int grid,
                          cudaStream_t stream);

}  // namespace cc
