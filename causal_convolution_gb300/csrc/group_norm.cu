// Group norm over channels-last instances with an optional SiLU, written as
// bf16 or as e4m3 with a scale per position and block of 128 channels.
//
// The channels of an instance are cut into slabs of whole groups (64 channels
// where the groups allow it, so that a position's piece is 128 bytes). A slab
// is independent of the others, and two kernels take it:
//
//  - gn_cluster_kernel: a cluster of up to 16 CTAs holds the slab in its
//    shared memory, exchanges the groups' moments through it and writes the
//    result. x is read once; no workspace.
//  - gn_stream_kernel, for slabs that a cluster cannot hold: CTAs take tiles
//    in an order in which a slab's second reading (to normalise) follows its
//    first (for the moments) closely enough to find the slab in L2.
//
// Both sum a thread's values around a pivot, its first value, so that nothing
// cancels where the mean is large against the deviation, and merge the
// threads' means and squared deviations in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <numeric>

#include "cc.h"
#include "cc_host.h"
#include "cc_ptx.cuh"
#include "cc_rows.cuh"

namespace cc {
namespace {

constexpr int kGnMaxChannels = 4096;

// Mean and sum of squared deviations of `n` values; two of them merge exactly
// (in real arithmetic) into that of their union, without the cancellation
// that sum(x^2) - n mean^2 has when the mean is large.
struct Moments {
  float n, mean, m2;
};

__device__ __forceinline__ void merge(Moments& a, const Moments& b) {
  if (a.n == 0.f) {
    a = b;
  } else if (b.n != 0.f) {
    const float n = a.n + b.n;
    const float d = b.mean - a.mean;
    const float f = __fdividef(b.n, n);
    a.mean = fmaf(d, f, a.mean);
    a.m2 += fmaf(d * d, a.n * f, b.m2);
    a.n = n;
  }
}

__device__ __forceinline__ Moments warp_merge(Moments m) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Moments b = {__shfl_xor_sync(0xffffffffu, m.n, o), __shfl_xor_sync(0xffffffffu, m.mean, o),
                 __shfl_xor_sync(0xffffffffu, m.m2, o)};
    if ((threadIdx.x & o) != 0) {  // the lower lane's moments come first on both sides: all lanes agree
      const Moments t = m;
      m = b;
      b = t;
    }
    merge(m, b);
  }
  return m;
}

struct GnArgs {
  const uint4* x;
  const uint4* gamma;  // nullptr: ones
  const uint4* beta;   // nullptr: zeros
  void* y;
  float* scales;
  int p;
  int vecs;        // C / 8
  int blocks;      // ceil(C / 128)
  int slabs;       // per instance
  int slab_vecs;   // of every slab but, perhaps, the last
  int cpg;         // C / groups
  int gw;          // channels of a vector that always share a group: gcd(C / groups, 8)
  float eps;
  // cluster kernel
  int rows_per_cta;
  int rounds;      // vectors a thread keeps
  int scratch_at, keep_at;  // bytes into shared memory
  // stream kernel
  int tiles;       // per slab
  int lead;        // tiles between a tile's first and second reading, at least `tiles`
  long long all_tiles;
  unsigned long long* ticket;
  unsigned int* done;   // [units] tiles whose moments are written
  unsigned int* ready;  // [units] 1: stat is written
  float2* part;         // [units][tiles][groups of a slab]
  float2* stat;         // [units][groups of a slab]: mean, 1 / deviation
  int slab_groups;
  unsigned int* err;
  unsigned long long timeout_ns;
};

// Where a thread of T stands in its slab: positions `lane`, lane + lanes, ...,
// and vector v of them. For e4m3 the vectors take whole half warps, so that the
// 16 lanes of a block of 128 channels are neighbours.
template <bool FP8, int T>
struct Place {
  int vecs, slots, lanes, lane, v;
  bool on;
  __device__ __forceinline__ Place(const GnArgs& a, int slab) {
    vecs = min(a.slab_vecs, a.vecs - slab * a.slab_vecs);
    slots = FP8 ? (vecs + 15) & ~15 : vecs;
    lanes = T / slots;
    lane = threadIdx.x / slots;
    v = threadIdx.x - lane * slots;
    on = lane < lanes && v < vecs;
  }
  // positions below `rows` that are this thread's
  __device__ __forceinline__ int count(int rows) const { return on && lane < rows ? (rows - lane - 1) / lanes + 1 : 0; }
};

// A thread's sums around its pivots: one for its vector where all eight
// channels share a group (ONE), one for each channel otherwise. `first` is the
// thread's first vector.
template <bool ONE>
struct Sums {
  static constexpr int K = ONE ? 1 : 4;
  f32x2 neg[K], s1[K], s2[K];
  __device__ __forceinline__ void start(const uint4& first) {
    const Vec8 f = unpack8(first);
#pragma unroll
    for (int e = 0; e < K; ++e) {
      neg[e] = ONE ? pair(-f[0], -f[0]) : pair(-f[2 * e], -f[2 * e + 1]);
      s1[e] = s2[e] = pair(0.f, 0.f);
    }
  }
  __device__ __forceinline__ void add(const uint4& raw) {
    const Vec8 f = unpack8(raw);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = ONE ? 0 : e;
      const f32x2 d = add2(f.p[e], neg[k]);
      s1[k] = add2(s1[k], d);
      s2[k] = fma2(d, d, s2[k]);
    }
  }
};

// Shared scratch of block_moments: an entry (moments of each part of a vector,
// count) per thread, or per warp and slot where a warp's lanes of the same
// slot can be merged by shuffles.
__host__ __device__ constexpr bool gn_shuffles(int slots) { return slots <= 16 && (slots & (slots - 1)) == 0; }
__host__ __device__ constexpr int gn_entries(int slots, int threads) {
  return gn_shuffles(slots) ? threads / 32 * slots : threads;
}
__host__ __device__ constexpr int gn_entry_bytes(int gw) { return 8 / gw * 8 + 4; }

// The moments of the slab's groups over the CTA's positions, merged from the
// threads' sums (of n positions each) in a fixed order; `out(group, moments)`
// runs on one lane.
template <bool ONE, bool FP8, int T, typename Out>
__device__ __forceinline__ void block_moments(const GnArgs& a, const Place<FP8, T>& at, const Sums<ONE>& s, int n,
                                              void* scratch, Out out) {
  constexpr int K = ONE ? 1 : 8;
  const int tid = threadIdx.x;
  const int entries = gn_entries(at.slots, T);
  float2* red = static_cast<float2*>(scratch);
  float* cnt = reinterpret_cast<float*>(red + (ONE ? 1 : 8 / a.gw) * entries);
  Moments m[K];
  if (ONE) {
    const float c = 8.f * n, sum = lo(s.s1[0]) + hi(s.s1[0]);
    const float d = n > 0 ? __fdividef(sum, c) : 0.f;
    m[0] = {c, d - lo(s.neg[0]), lo(s.s2[0]) + hi(s.s2[0]) - sum * d};
  } else {
    const float inv = n > 0 ? 1.f / n : 0.f;
#pragma unroll
    for (int e = 0; e < K; ++e) {
      const int k = (e >> 1) % Sums<ONE>::K;
      const float sum = (e & 1) ? hi(s.s1[k]) : lo(s.s1[k]);
      const float d = sum * inv;
      m[e] = {static_cast<float>(n), d - ((e & 1) ? hi(s.neg[k]) : lo(s.neg[k])),
              ((e & 1) ? hi(s.s2[k]) : lo(s.s2[k])) - sum * d};
    }
  }
#pragma unroll
  for (int e = 0; e < K; ++e) m[e].m2 = m[e].m2 < 0.f ? 0.f : m[e].m2;  // keeps a NaN
  int w = 1;
  if (!ONE) {
#pragma unroll
    for (int l = 1; l < 8; l <<= 1) {
      if (a.gw > l) {  // neighbours of the same group
#pragma unroll
        for (int e = 0; e < 8; e += 2 * l) merge(m[e % K], m[(e + l) % K]);
        w = 2 * l;
      }
    }
  }
  int entry = tid;
  bool writes = true;
  if (gn_shuffles(at.slots)) {  // uniform
    for (int o = at.slots; o < 32; o <<= 1) {
#pragma unroll
      for (int e = 0; e < K; ++e) {
        if (e % w == 0) {
          Moments b = {__shfl_xor_sync(0xffffffffu, m[e].n, o), __shfl_xor_sync(0xffffffffu, m[e].mean, o),
                       __shfl_xor_sync(0xffffffffu, m[e].m2, o)};
          merge(m[e], b);  // only the lowest lanes' results are used
        }
      }
    }
    entry = (tid >> 5) * at.slots + (tid & 31);
    writes = (tid & 31) < at.slots;
  }
  if (writes) {
#pragma unroll
    for (int e = 0; e < K; ++e)
      if (e % w == 0) red[(e / w) * entries + entry] = make_float2(m[e].mean, m[e].m2);
    cnt[entry] = m[0].n;
  }
  __syncthreads();
  const int parts = ONE ? 1 : 8 / a.gw;      // of a vector
  const int per = ONE ? a.cpg >> 3 : a.cpg / a.gw;  // parts in a group
  const int side = gn_shuffles(at.slots) ? T / 32 : at.lanes;  // entries of a slot
  for (int g = tid >> 5; g < at.vecs * 8 / a.cpg; g += T / 32) {
    Moments t = {0.f, 0.f, 0.f};
    for (int i = tid & 31; i < per * side; i += 32) {
      const int q = i / per;
      const int j = g * per + (i - q * per);
      const int at_entry = q * at.slots + (ONE ? j : j / parts);
      const float2 v = red[(ONE ? 0 : j % parts) * entries + at_entry];
      merge(t, Moments{cnt[at_entry], v.x, v.y});
    }
    t = warp_merge(t);
    if ((tid & 31) == 0) out(g, t);
  }
}

__device__ __forceinline__ float2 mean_and_factor(const Moments& m, float eps) {
  return make_float2(m.mean, 1.f / sqrtf(m.m2 / m.n + eps));
}

// A thread's eight channels: act((x - mean) * k + beta). The mean is taken off
// first: folded into beta it would cost digits where it is large.
template <bool ONE, bool SILU, bool FP8, int T>
struct Affine {
  f32x2 neg[Sums<ONE>::K];
  Vec8 k, b;
  __device__ __forceinline__ void load_params(const GnArgs& a, const Place<FP8, T>& at, int slab) {
    k = splat8(1.f);
    b = splat8(0.f);
    if (at.on && a.gamma) k = unpack8(__ldg(a.gamma + slab * a.slab_vecs + at.v));
    if (at.on && a.beta) b = unpack8(__ldg(a.beta + slab * a.slab_vecs + at.v));
  }
  template <typename Stat>
  __device__ __forceinline__ void load_stat(const GnArgs& a, const Place<FP8, T>& at, Stat stat) {
    if (ONE) {
      const float2 s = at.on ? stat(8 * at.v / a.cpg) : make_float2(0.f, 0.f);
      neg[0] = pair(-s.x, -s.x);
#pragma unroll
      for (int i = 0; i < 4; ++i) k.p[i] = mul2(k.p[i], pair(s.y, s.y));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 8 * at.v + 2 * i;
        const float2 s = at.on ? stat(c / a.cpg) : make_float2(0.f, 0.f);
        const float2 t = at.on ? stat((c + 1) / a.cpg) : make_float2(0.f, 0.f);
        neg[i % Sums<ONE>::K] = pair(-s.x, -t.x);
        k.p[i] = mul2(k.p[i], pair(s.y, t.y));
      }
    }
  }
  // y and scales: of the vector, and of the row's first block of the slab
  __device__ __forceinline__ void write(const Place<FP8, T>& at, const uint4& raw, void* y, float* scales,
                                        bool on) const {
    Vec8 f = unpack8(raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = fma2(add2(f.p[i], neg[ONE ? 0 : i]), k.p[i], b.p[i]);
    activate8<SILU>(f);
    if (FP8) {
      if (!at.on) f = splat8(0.f);
      float scale;
      const uint2 q = quantize_block(f, scale);
      if (on) {
        *static_cast<uint2*>(y) = q;
        if ((at.v & 15) == 0) scales[at.v >> 4] = scale;
      }
    } else if (on) {
      *static_cast<uint4*>(y) = pack8(f);
    }
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------- on chip --

// One cluster per (instance, slab); its CTAs take the positions in equal runs.
// A thread copies its own vectors to shared memory and is the only one to read
// them back, so the copies need no barrier; they are waited for in quarters,
// the moments of one while the next are on their way.
template <bool ONE, bool SILU, bool FP8, int T>
__global__ void __launch_bounds__(T, 1024 / T) gn_cluster_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint32_t ranks;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const uint32_t rank = cluster_ctarank();
  const int unit = blockIdx.x / ranks;
  const int instance = unit / a.slabs;
  const int slab = unit - instance * a.slabs;
  const Place<FP8, T> at(a, slab);
  float2* mom = reinterpret_cast<float2*>(smem);
  float2* stat = mom + a.slab_groups;
  uint8_t* scratch = smem + a.scratch_at;
  const int stride = at.lanes * at.slots;
  uint4* keep = reinterpret_cast<uint4*>(smem + a.keep_at) + threadIdx.x;
  const int r0 = rank * a.rows_per_cta;
  const int rows = max(0, min(a.rows_per_cta, a.p - r0));
  const int n = at.count(rows);
  const long long row0 = static_cast<long long>(instance) * a.p + r0;
  const uint4* x = a.x + (row0 + at.lane) * a.vecs + slab * a.slab_vecs + at.v;
  const int step = at.lanes * a.vecs;
  const int quarter = (a.rounds + 3) / 4;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int end = min((q + 1) * quarter, n);
    for (int i = q * quarter; i < end; ++i)
      cp_async16(smem_u32(keep + i * stride), x + static_cast<long long>(i) * step);
    cp_async_commit();
  }
  Affine<ONE, SILU, FP8, T> affine;
  affine.load_params(a, at, slab);
  Sums<ONE> sums;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q == 0) cp_async_wait<3>();
    if (q == 1) cp_async_wait<2>();
    if (q == 2) cp_async_wait<1>();
    if (q == 3) cp_async_wait<0>();
    if (q == 0) sums.start(n > 0 ? keep[0] : make_uint4(0, 0, 0, 0));
    const int end = min((q + 1) * quarter, n);
    for (int i = q * quarter; i < end; ++i) sums.add(keep[i * stride]);
  }
  block_moments<ONE>(a, at, sums, n, scratch,
                     [&](int g, const Moments& m) { mom[g] = make_float2(m.mean, m.m2); });
  __syncwarp();
  cluster_sync_all();
  for (int g = threadIdx.x; g < at.vecs * 8 / a.cpg; g += T) {
    Moments m = {0.f, 0.f, 0.f};
    for (uint32_t k = 0; k < ranks; ++k) {
      const float2 v = ld_cluster_f2(mapa_shared(smem_u32(&mom[g]), k));
      const int c = max(0, min(a.rows_per_cta, a.p - static_cast<int>(k) * a.rows_per_cta));
      merge(m, Moments{static_cast<float>(c) * a.cpg, v.x, v.y});
    }
    stat[g] = mean_and_factor(m, a.eps);
  }
  __syncthreads();
  // nobody reads this CTA's moments any more once all have arrived here
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  affine.load_stat(a, at, [&](int g) { return stat[g]; });
  const long long at_y = (row0 + at.lane) * a.vecs + slab * a.slab_vecs + at.v;
  uint8_t* y = static_cast<uint8_t*>(a.y) + at_y * (FP8 ? 8 : 16);
  float* scales = FP8 ? a.scales + (row0 + at.lane) * a.blocks + slab * a.slab_vecs / 16 : nullptr;
  // e4m3: whole warps stay together, for the shuffles
  const int end = FP8 ? (rows + at.lanes - 1) / at.lanes : n;
#pragma unroll 2
  for (int i = 0; i < end; ++i) {
    const bool on = i < n;
    affine.write(at, on ? keep[i * stride] : make_uint4(0, 0, 0, 0), y, scales, on);
    y += static_cast<long long>(step) * (FP8 ? 8 : 16);
    if (FP8) scales += at.lanes * a.blocks;
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// -------------------------------------------------------------- through L2 --

constexpr int kTileVecs = 4;   // vectors a thread has in flight
constexpr int kTileTurns = 2;  // times that makes a tile

__device__ __forceinline__ unsigned int ld_acquire(const unsigned int* p) {
  unsigned int v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(unsigned int* p, unsigned int v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Tiles are numbered through the units (instance, slab) in order. Tickets hand
// out first readings `lead` tiles ahead of second readings and alternate
// between them; a second reading waits until its unit's statistics are there,
// which takes first readings with smaller tickets only, so the smallest open
// ticket never waits for one that nobody holds, however few CTAs run at once.
template <bool ONE, bool SILU, bool FP8, int T>
__global__ void __launch_bounds__(T, 1024 / T) gn_stream_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ unsigned long long next;
  __shared__ unsigned int word;
  const int tid = threadIdx.x;
  if (tid == 0) next = atomicAdd(a.ticket, 1ull);
  __syncthreads();
  for (;;) {
    const long long t = static_cast<long long>(next);
    if (t >= 2 * a.all_tiles) return;
    bool second;
    long long tile;
    if (t < a.lead) {
      second = false, tile = t;
    } else if (t < 2 * a.all_tiles - a.lead) {
      second = (t - a.lead) & 1;
      tile = (t - a.lead) / 2 + (second ? 0 : a.lead);
    } else {
      second = true, tile = t - a.all_tiles;
    }
    const int unit = static_cast<int>(tile / a.tiles);
    const int i0 = static_cast<int>(tile - static_cast<long long>(unit) * a.tiles);
    const int instance = unit / a.slabs;
    const int slab = unit - instance * a.slabs;
    const Place<FP8, T> at(a, slab);
    const int tile_rows = at.lanes * kTileVecs * kTileTurns;
    const int r0 = i0 * tile_rows;
    const int rows = max(0, min(tile_rows, a.p - r0));  // a narrower last slab has fewer tiles than the others
    const int n = at.count(rows);
    const long long row0 = static_cast<long long>(instance) * a.p + r0 + at.lane;
    const uint4* x = a.x + row0 * a.vecs + slab * a.slab_vecs + at.v;
    const int step = at.lanes * a.vecs;
    __syncthreads();  // `next` is read
    if (tid == 0) next = atomicAdd(a.ticket, 1ull);
    uint4 raw[kTileVecs];
    if (!second) {
      Sums<ONE> sums;
#pragma unroll
      for (int turn = 0; turn < kTileTurns; ++turn) {
#pragma unroll
        for (int i = 0; i < kTileVecs; ++i)
          if (turn * kTileVecs + i < n) raw[i] = __ldg(x + static_cast<long long>(turn * kTileVecs + i) * step);
        if (turn == 0) sums.start(n > 0 ? raw[0] : make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int i = 0; i < kTileVecs; ++i)
          if (turn * kTileVecs + i < n) sums.add(raw[i]);
      }
      float2* part = a.part + (static_cast<long long>(unit) * a.tiles + i0) * a.slab_groups;
      block_moments<ONE>(a, at, sums, n, smem, [&](int g, const Moments& m) {
        part[g] = make_float2(m.mean, m.m2);
        __threadfence();
      });
      __syncthreads();
      if (tid == 0) word = atomicAdd(a.done + unit, 1u);
      __syncthreads();
      if (word == static_cast<unsigned int>(a.tiles - 1)) {  // the unit's last: merge in the tiles' order
        __threadfence();
        const float2* all = a.part + static_cast<long long>(unit) * a.tiles * a.slab_groups;
        for (int g = tid >> 5; g < at.vecs * 8 / a.cpg; g += T / 32) {
          Moments m = {0.f, 0.f, 0.f};
#pragma unroll 4
          for (int i = tid & 31; i < a.tiles; i += 32) {
            const float2 v = __ldcg(all + static_cast<long long>(i) * a.slab_groups + g);
            const int c = max(0, min(tile_rows, a.p - i * tile_rows));
            merge(m, Moments{static_cast<float>(c) * a.cpg, v.x, v.y});
          }
          m = warp_merge(m);
          if ((tid & 31) == 0) {
            a.stat[static_cast<long long>(unit) * a.slab_groups + g] = mean_and_factor(m, a.eps);
            __threadfence();
          }
        }
        __syncthreads();
        if (tid == 0) st_release(a.ready + unit, 1u);
      }
    } else {
      Affine<ONE, SILU, FP8, T> affine;
#pragma unroll
      for (int i = 0; i < kTileVecs; ++i) {
        raw[i] = make_uint4(0, 0, 0, 0);
        if (i < n) raw[i] = __ldcs(x + static_cast<long long>(i) * step);
      }
      affine.load_params(a, at, slab);
      if (tid == 0) {
        unsigned int ok = ld_acquire(a.ready + unit);
        if (!ok) {
          const uint64_t t0 = globaltimer_ns();
          while (!ok && globaltimer_ns() - t0 < a.timeout_ns) ok = ld_acquire(a.ready + unit);
          if (!ok) atomicOr(a.err, DEVERR_TIMEOUT);
        }
        word = ok;
      }
      __syncthreads();
      if (!word) return;
      const float2* stat = a.stat + static_cast<long long>(unit) * a.slab_groups;
      affine.load_stat(a, at, [&](int g) { return __ldcg(stat + g); });
      uint8_t* y = static_cast<uint8_t*>(a.y) + (row0 * a.vecs + slab * a.slab_vecs + at.v) * (FP8 ? 8 : 16);
      float* scales = FP8 ? a.scales + row0 * a.blocks + slab * a.slab_vecs / 16 : nullptr;
#pragma unroll
      for (int turn = 0; turn < kTileTurns; ++turn) {
        if (turn > 0) {
#pragma unroll
          for (int i = 0; i < kTileVecs; ++i)
            if (turn * kTileVecs + i < n) raw[i] = __ldcs(x + static_cast<long long>(turn * kTileVecs + i) * step);
        }
#pragma unroll
        for (int i = 0; i < kTileVecs; ++i) {
          const int j = turn * kTileVecs + i;
          affine.write(at, raw[i], y + static_cast<long long>(j) * step * (FP8 ? 8 : 16),
                       FP8 ? scales + static_cast<long long>(j) * at.lanes * a.blocks : nullptr, j < n);
        }
      }
    }
    __syncthreads();  // the next ticket is there, `word` and the scratch are free
  }
}

// -------------------------------------------------------------------- host --

// Channels of a slab: whole groups, whole vectors (whole blocks of 128 for
// e4m3), at least 64 of them. At most 128 groups: below 64 channels the least
// common multiple of C / groups and 8 has 8 groups at most, and that with 128
// has 128.
int slab_channels(int c, int groups, bool fp8) {
  const int unit = std::lcm(c / groups, fp8 ? kScaleBlock : 8);
  if (unit >= c) return c;
  return std::min(c, unit * std::max(1, 64 / unit));
}

struct GnPlan {
  bool cluster;
  int threads;
  int slab_c, slabs, slab_groups, scratch;
  int ranks, rows, rounds, scratch_at, keep_at;  // cluster
  size_t smem;
  int tiles;  // stream
  long long units;
  size_t ws_bytes;
};

constexpr size_t kMaxSmem = 232448;

GnPlan gn_plan(int n, int p, int c, int groups, bool fp8) {
  GnPlan g = {};
  g.slab_c = slab_channels(c, groups, fp8);
  g.slabs = (c + g.slab_c - 1) / g.slab_c;
  g.slab_groups = g.slab_c / (c / groups);
  g.units = static_cast<long long>(n) * g.slabs;
  const int gw = std::gcd(c / groups, 8);
  // the widest slab has the fewest positions side by side
  const int slots = fp8 ? (g.slab_c / 8 + 15) / 16 * 16 : g.slab_c / 8;
  const int last_c = c - (g.slabs - 1) * g.slab_c;
  const int last = fp8 ? (last_c / 8 + 15) / 16 * 16 : last_c / 8;
  g.threads = slots > 256 ? 512 : 256;
  const int lanes = g.threads / slots;
  g.scratch = std::max(gn_entries(slots, g.threads), gn_entries(last, g.threads)) * gn_entry_bytes(gw);
  g.scratch_at = (2 * g.slab_groups * static_cast<int>(sizeof(float2)) + 15) / 16 * 16;
  g.keep_at = g.scratch_at + (g.scratch + 15) / 16 * 16;
  auto cut = [&](int ranks) {
    g.ranks = ranks;
    g.rows = (p + ranks - 1) / ranks;
    g.rounds = (g.rows + lanes - 1) / lanes;
    g.smem = g.keep_at + static_cast<size_t>(g.rows) * slots * 16;
  };
  for (int ranks = 1; ranks <= 16; ranks *= 2) {
    cut(ranks);
    if (g.smem <= kMaxSmem) break;
  }
  g.cluster = g.smem <= kMaxSmem;
  if (g.cluster) {
    // two CTAs to an SM where eight of them hold the slab, and more CTAs while
    // SMs are idle and a thread still has several vectors
    while (g.ranks < 8 && (g.smem > kMaxSmem / 2 - 1024 || (g.units * g.ranks < 152 && g.rounds > 2))) cut(g.ranks * 2);
    return g;
  }
  const int tile_rows = lanes * kTileVecs * kTileTurns;
  g.tiles = (p + tile_rows - 1) / tile_rows;
  g.ws_bytes = 16 + (g.units * 8 + 15) / 16 * 16 +
               static_cast<size_t>(g.units) * (g.tiles + 1) * g.slab_groups * sizeof(float2);
  return g;
}

template <bool ONE, bool SILU, bool FP8, int T>
cc_status launch_group_norm(const char* what, GnArgs& a, const GnPlan& g, int sms, cudaStream_t s) {
  if (g.cluster) {
    auto kern = gn_cluster_kernel<ONE, SILU, FP8, T>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess && g.ranks > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: kernel attributes: %s", what, cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(g.units * g.ranks));
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = g.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = g.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: launch: %s", what, cudaGetErrorString(e));
    return launch_status(what);
  }
  auto kern = gn_stream_kernel<ONE, SILU, FP8, T>;
  const long long grid = std::min<long long>(1024LL / T * sms, 2 * a.all_tiles);
  kern<<<static_cast<unsigned>(grid), T, g.scratch, s>>>(a);
  return launch_status(what);
}

template <bool ONE, bool SILU, bool FP8>
cc_status launch_group_norm(const char* what, GnArgs& a, const GnPlan& g, int sms, cudaStream_t s) {
  return g.threads == 512 ? launch_group_norm<ONE, SILU, FP8, 512>(what, a, g, sms, s)
                          : launch_group_norm<ONE, SILU, FP8, 256>(what, a, g, sms, s);
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
  const GnPlan g = gn_plan(n, p, c, groups, fp8);
  if (g.ws_bytes > 0 && (!ws || ws_bytes < g.ws_bytes))
    return fail(CC_ERR_INVALID, "%s: workspace of %zu bytes needed (got %zu)", what, g.ws_bytes, ws ? ws_bytes : 0);
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
  a.blocks = (c + kScaleBlock - 1) / kScaleBlock;
  a.slabs = g.slabs;
  a.slab_vecs = g.slab_c / 8;
  a.cpg = c / groups;
  a.gw = std::gcd(a.cpg, 8);
  a.eps = eps;
  a.slab_groups = g.slab_groups;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (g.cluster) {
    a.rows_per_cta = g.rows;
    a.rounds = g.rounds;
    a.scratch_at = g.scratch_at;
    a.keep_at = g.keep_at;
  } else {
    a.tiles = g.tiles;
    a.all_tiles = g.units * g.tiles;
    a.lead = static_cast<int>(std::min<long long>(a.all_tiles, g.tiles + std::min(g.tiles, 1200)));
    a.err = di.err_word;
    a.timeout_ns = kWaitLimitNs;
    a.ticket = static_cast<unsigned long long*>(ws);
    a.done = reinterpret_cast<unsigned int*>(static_cast<uint8_t*>(ws) + 16);
    a.ready = a.done + g.units;
    const size_t head = 16 + (g.units * 8 + 15) / 16 * 16;
    a.stat = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + head);
    a.part = a.stat + g.units * a.slab_groups;
    const cudaError_t e = cudaMemsetAsync(ws, 0, head, s);
    if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: workspace: %s", what, cudaGetErrorString(e));
  }
  const bool silu = act == CC_ACT_SILU;
  if (a.gw == 8) {
    if (fp8)
      return silu ? launch_group_norm<true, true, true>(what, a, g, di.sm_count, s)
                  : launch_group_norm<true, false, true>(what, a, g, di.sm_count, s);
    return silu ? launch_group_norm<true, true, false>(what, a, g, di.sm_count, s)
                : launch_group_norm<true, false, false>(what, a, g, di.sm_count, s);
  }
  if (fp8)
    return silu ? launch_group_norm<false, true, true>(what, a, g, di.sm_count, s)
                : launch_group_norm<false, false, true>(what, a, g, di.sm_count, s);
  return silu ? launch_group_norm<false, true, false>(what, a, g, di.sm_count, s)
              : launch_group_norm<false, false, false>(what, a, g, di.sm_count, s);
}

}  // namespace
}  // namespace cc

using namespace cc;

extern "C" size_t cc_group_norm_workspace_bytes(int n, int p, int c, int groups) {
  if (n <= 0 || p <= 0 || c < 8 || c > kGnMaxChannels || c % 8 != 0 || groups <= 0 || c % groups != 0) return 0;
  return std::max(gn_plan(n, p, c, groups, false).ws_bytes, gn_plan(n, p, c, groups, true).ws_bytes);
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
