// Group norm over channels-last instances with an optional SiLU, written as
// bf16 or as e4m3 with a scale per position and block of 128 channels.
//
// The channels of an instance are cut into slabs of whole groups (64 channels
// where the groups allow it, so that a position's piece is 128 bytes). A slab
// is independent of the others, and one of two ways takes it:
//
//  - gn_cluster_kernel: a cluster of up to 8 CTAs keeps the slab in its
//    shared memory, exchanges the groups' moments through it and writes the
//    result. x is read once; no workspace.
//  - gn_moments_kernel, gn_merge_kernel, gn_apply_kernel: x is read twice.
//
// (One kernel that keeps slabs of up to 15 MB on all SMs and meets in global
// memory, and one that reads a slab a second time out of L2, took 1.1 ms for
// 16 frames of 219,648 x 256 where these three take 0.79 ms, the time that
// copying 3 x 1.8 GB takes. Their CTAs spent their time meeting.)
//
// A thread sums its values around a pivot, its first value, so that nothing
// cancels where the mean is large against the deviation. The CTA then adds up
// the threads' sums to the groups' means q, and after that each thread's
// squared deviations from its own mean plus n (mean - q)^2: two plain sums in a
// fixed order, of terms that are not negative in the second.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <mutex>
#include <numeric>

#include "cc.h"
#include "cc_host.h"
#include "cc_ptx.cuh"
#include "cc_rows.cuh"

namespace cc {
namespace {

constexpr int kGnMaxChannels = 4096;
constexpr int kMaxRanks = 8;  // CTAs in a cluster

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
  int slab_vecs;   // of every slab but, perhaps, the last
  int cpg;         // C / groups
  int gw_shift;    // log2 of gw = gcd(C / groups, 8): channels of a vector that always share a group
  int per;         // C / groups / gw: parts of gw channels in a group
  float eps;
  int rows_per_cta;
  int rounds;       // vectors a thread keeps (cluster kernel)
  int slab_groups;  // of the widest slab
  int cols_at, red_at, keep_at;  // bytes into shared memory (cluster kernel)
  int runs;         // per instance (two readings)
  float2* part;     // moments of each CTA's positions (two readings)
  float2* stat;     // mean, 1 / deviation (two readings)
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

// Columns are the parts of gw channels of a position's slab, slots * 8 / gw of
// them. A warp's lanes of the same slot can be added up by shuffles where their
// number divides 32.
__host__ __device__ constexpr bool gn_shuffles(int slots) { return slots <= 16 && (slots & (slots - 1)) == 0; }
// Rows of `red` in block_sums, one value per column each.
__host__ __device__ constexpr int gn_red_rows(int slots, int threads) {
  return gn_shuffles(slots) ? threads / 32 : threads / slots;
}

// The sums over the CTA's positions of val[0 .. parts), each thread's value for
// its parts, added up per group: `of(sum)` of a group's sum goes to all of the
// group's columns in `cols` and to out(group, value). red: [red rows][columns].
template <int K, bool FP8, int T, typename Of, typename Out>
__device__ __forceinline__ void block_sums(const GnArgs& a, const Place<FP8, T>& at, int parts, int groups,
                                           float (&val)[K], float* red, float* cols, Of of, Out out) {
  const int n_cols = at.slots * parts;
  int row = at.lane;
  bool writes = at.lane < at.lanes;
  if (gn_shuffles(at.slots)) {  // the same for every thread
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      if (o >= at.slots) {
#pragma unroll
        for (int e = 0; e < K; ++e) val[e] += __shfl_xor_sync(0xffffffffu, val[e], o);
      }
    }
    row = threadIdx.x >> 5;
    writes = (threadIdx.x & 31) < at.slots;
  }
  if (writes) {
    float* to = red + row * n_cols + at.v * parts;
#pragma unroll
    for (int e = 0; e < K; ++e)
      if (e < parts) to[e] = val[e];
  }
  __syncthreads();
  const int rows = gn_shuffles(at.slots) ? T / 32 : at.lanes;
  for (int c = threadIdx.x; c < n_cols; c += T) {
    float t = 0.f;
#pragma unroll 8
    for (int r = 0; r < rows; ++r) t += red[r * n_cols + c];
    cols[c] = t;
  }
  __syncthreads();
  if (a.per < 32) {  // a thread to a group
    for (int g = threadIdx.x; g < groups; g += T) {
      float t = 0.f;
#pragma unroll 4
      for (int j = 0; j < a.per; ++j) t += cols[g * a.per + j];
      t = of(t);
#pragma unroll 4
      for (int j = 0; j < a.per; ++j) cols[g * a.per + j] = t;
      out(g, t);
    }
  } else {  // a warp to a group
    for (int g = threadIdx.x >> 5; g < groups; g += T / 32) {
      float t = 0.f;
      for (int j = threadIdx.x & 31; j < a.per; j += 32) t += cols[g * a.per + j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      t = of(t);
      for (int j = threadIdx.x & 31; j < a.per; j += 32) cols[g * a.per + j] = t;
      if ((threadIdx.x & 31) == 0) out(g, t);
    }
  }
  __syncthreads();
}

// mom[group] = mean and summed squared deviations over the CTA's `rows`
// positions, of which this thread has n. red, cols: scratch of block_sums.
template <bool ONE, bool FP8, int T>
__device__ __forceinline__ void block_moments(const GnArgs& a, const Place<FP8, T>& at, int groups, const Sums<ONE>& s,
                                              int n, int rows, float* red, float* cols, float2* mom) {
  constexpr int K = ONE ? 1 : 8;
  const int parts = ONE ? 1 : 8 >> a.gw_shift;
  // each part's mean and squared deviations; parts of several channels in
  // their lowest elements
  float mean[K], m2[K], val[K];
  float count = static_cast<float>(ONE ? 8 * n : n);
  const float inv = n > 0 ? __fdividef(1.f, count) : 0.f;
  if (ONE) {
    const float sum = lo(s.s1[0]) + hi(s.s1[0]);
    const float d = sum * inv;
    mean[0] = d - lo(s.neg[0]);
    m2[0] = lo(s.s2[0]) + hi(s.s2[0]) - sum * d;
  } else {
#pragma unroll
    for (int e = 0; e < K; ++e) {
      const int k = (e >> 1) % Sums<ONE>::K;
      const float sum = (e & 1) ? hi(s.s1[k]) : lo(s.s1[k]);
      const float d = sum * inv;
      mean[e] = d - ((e & 1) ? hi(s.neg[k]) : lo(s.neg[k]));
      m2[e] = ((e & 1) ? hi(s.s2[k]) : lo(s.s2[k])) - sum * d;
    }
  }
#pragma unroll
  for (int e = 0; e < K; ++e) m2[e] = m2[e] < 0.f ? 0.f : m2[e];  // keeps a NaN
  if (!ONE) {
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      if (a.gw_shift > l) {  // the same for every thread: neighbours of one group, with equal counts
#pragma unroll
        for (int e = 0; e < (8 >> (l + 1)); ++e) {
          const int u = 2 * e % K, v = (2 * e + 1) % K;
          const float d = mean[v] - mean[u];
          const float q = m2[u] + m2[v] + 0.5f * count * d * d;
          mean[e % K] = mean[u] + 0.5f * d;
          m2[e % K] = q;
        }
        count *= 2.f;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < K; ++e) val[e] = count * mean[e];
  const float all = static_cast<float>(rows) * a.cpg;
  block_sums(a, at, parts, groups, val, red, cols, [&](float t) { return rows > 0 ? t / all : 0.f; },
             [&](int g, float t) { mom[g].x = t; });
#pragma unroll
  for (int e = 0; e < K; ++e) {
    const float d = at.on && e < parts ? mean[e] - cols[at.v * parts + e] : 0.f;
    val[e] = at.on && e < parts ? fmaf(count * d, d, m2[e]) : 0.f;
  }
  __syncthreads();  // the columns' means are read
  block_sums(a, at, parts, groups, val, red, cols, [](float t) { return t; }, [&](int g, float t) { mom[g].y = t; });
}

__device__ __forceinline__ float2 mean_and_factor(const Moments& m, float eps) {
  return make_float2(m.mean, rsqrtf(m.m2 / m.n + eps));
}

// A thread's eight channels: act((x - mean) * k + beta). The mean is taken off
// first: folded into beta it would cost digits where it is large.
template <bool ONE, bool SILU, bool FP8, int T>
struct Affine {
  f32x2 neg[Sums<ONE>::K];
  Vec8 k, b;
  __device__ __forceinline__ void load_params(const GnArgs& a, const Place<FP8, T>& at, int slab) {
    // a thread without a vector computes zeros
    k = splat8(at.on ? 1.f : 0.f);
    b = splat8(0.f);
    if (at.on && a.gamma) k = unpack8(a.gamma[slab * a.slab_vecs + at.v]);
    if (at.on && a.beta) b = unpack8(a.beta[slab * a.slab_vecs + at.v]);
  }
  // stat(e): mean and factor of the thread's channel e
  template <typename Stat>
  __device__ __forceinline__ void load_stat(const Place<FP8, T>& at, Stat stat) {
#pragma unroll
    for (int i = 0; i < Sums<ONE>::K; ++i) {
      const float2 s = at.on ? stat(2 * i) : make_float2(0.f, 0.f);
      const float2 t = ONE ? s : at.on ? stat(2 * i + 1) : make_float2(0.f, 0.f);
      neg[i] = pair(-s.x, -t.x);
#pragma unroll
      for (int j = 0; j < (ONE ? 4 : 1); ++j) k.p[ONE ? j : i] = mul2(k.p[ONE ? j : i], pair(s.y, t.y));
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
      float scale;
      const uint2 q = quantize_block<false>(f, scale);
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

// ---------------------------------------------------------------- on chip --

// One cluster per (instance, slab); its CTAs take the positions in equal runs.
// A thread copies its own vectors to shared memory and is the only one to read
// them back, so the copies need no barrier; they are waited for in quarters,
// the moments of one while the next are on their way.
//
// x is read once, but what bounds it is the SMs: of the 12.8 us that
// 4 x 3432 x 1024 to e4m3 takes (its 43 MB would take 6.3 us at the copy rate),
// traced on an SM, 4 go by on normalising and quantising (about 60
// instructions for eight channels, issued nearly back to back), 3 on the
// loads, 1.5 on the sums that hide behind them, 1.5 on adding them up and 2 on
// the clusters' meeting. 3 x 3555 x 480 (groups of 15 channels, 96 CTAs): 11.5
// us; 2 x 96 x 64: 4.2 us.
template <bool ONE, bool SILU, bool FP8, int T>
__global__ void __launch_bounds__(T, 1024 / T) gn_cluster_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int ranks = gridDim.x, rank = blockIdx.x, slab = blockIdx.y, instance = blockIdx.z;
  const Place<FP8, T> at(a, slab);
  float2* mom = reinterpret_cast<float2*>(smem);
  float* cols = reinterpret_cast<float*>(smem + a.cols_at);  // later the columns' statistics
  float* red = reinterpret_cast<float*>(smem + a.red_at);
  const int stride = at.lanes * at.slots;
  uint4* keep = reinterpret_cast<uint4*>(smem + a.keep_at) + threadIdx.x;
  const int r0 = rank * a.rows_per_cta;
  const int rows = max(0, min(a.rows_per_cta, a.p - r0));
  const int n = at.count(rows);
  const long long row0 = static_cast<long long>(instance) * a.p + r0;
  const uint4* x = a.x + (row0 + at.lane) * a.vecs + slab * a.slab_vecs + at.v;
  const int step = at.lanes * a.vecs;
  const int quarter = (a.rounds + 3) / 4;
  const int parts = ONE ? 1 : 8 >> a.gw_shift;
  const int groups = at.vecs * 8 / a.cpg;
  // set up: the next kernel may be scheduled, the previous one has to be done
  pdl_launch_dependents();
  pdl_wait();
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
  block_moments<ONE>(a, at, groups, sums, n, rows, red, cols, mom);
  __syncwarp();
  cluster_sync_all();
  // The ranks' moments in their order, around the first one's mean (which
  // takes at most three bits if that rank is the odd one out of eight).
  float2* col_stat = reinterpret_cast<float2*>(cols);
  const float count = static_cast<float>(a.p) * a.cpg;
  for (int g = threadIdx.x; g < groups; g += T) {
    float sum = 0.f, m2 = 0.f;
    float2 of[kMaxRanks];  // all trips to the other CTAs at once
#pragma unroll
    for (int k = 0; k < kMaxRanks; ++k)
      if (k < ranks) of[k] = ld_cluster_f2(mapa_shared(smem_u32(&mom[g]), k));
    const float pivot = of[0].x;
#pragma unroll
    for (int k = 0; k < kMaxRanks; ++k) {
      if (k < ranks) {
        const float c = static_cast<float>(max(0, min(a.rows_per_cta, a.p - k * a.rows_per_cta))) * a.cpg;
        const float d = of[k].x - pivot;
        sum = fmaf(c, d, sum);
        m2 += fmaf(c * d, d, of[k].y);
      }
    }
    const float shift = sum / count;
    m2 -= sum * shift;
    m2 = m2 < 0.f ? 0.f : m2;  // keeps a NaN
    // for all of the group's columns, so that a thread finds its own without a division
    const float2 st = mean_and_factor(Moments{count, pivot + shift, m2}, a.eps);
#pragma unroll 4
    for (int j = 0; j < a.per; ++j) col_stat[g * a.per + j] = st;
  }
  __syncthreads();
  __syncwarp();
  // nobody reads this CTA's moments any more once all have arrived here
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  affine.load_stat(at, [&](int e) { return col_stat[at.v * parts + (ONE ? 0 : e >> a.gw_shift)]; });
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

// ------------------------------------------------------------- twice from memory --

// What does not fit on chip: the moments of runs of positions, their merging,
// and a second reading that normalises. All three stream at about the copy
// rate: 16 x 219648 x 256 + SiLU takes 790 us for its three passes over 1.8 GB
// (797 at the copy rate), of which a norm that read x once would save a third.
constexpr int kMergeThreads = 256;

template <bool ONE, int T>
__global__ void __launch_bounds__(T, 1024 / T) gn_moments_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Place<false, T> at(a, 0);
  const int r0 = blockIdx.x * a.rows_per_cta;
  const int rows = min(a.rows_per_cta, a.p - r0);
  const int n = at.count(rows);
  const int step = at.lanes * a.vecs;
  const uint4* x = a.x + (static_cast<long long>(blockIdx.y) * a.p + r0 + at.lane) * a.vecs + at.v;
  pdl_launch_dependents();
  pdl_wait();
  Sums<ONE> sums;
  sums.start(n > 0 ? *x : make_uint4(0, 0, 0, 0));
  int i = 0;
  for (; i + 8 <= n; i += 8) {
    uint4 raw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) raw[j] = x[static_cast<long long>(i + j) * step];
#pragma unroll
    for (int j = 0; j < 8; ++j) sums.add(raw[j]);
  }
  for (; i < n; i += 4) {
    uint4 raw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      raw[j] = i + j < n ? x[static_cast<long long>(i + j) * step] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) sums.add(raw[j]);
  }
  block_moments<ONE>(a, at, at.vecs * 8 / a.cpg, sums, n, rows, reinterpret_cast<float*>(smem),
                     reinterpret_cast<float*>(smem + a.cols_at),
                     a.part + (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * a.slab_groups);
}

// A CTA to a group, so that few trips to memory follow one another.
__global__ void __launch_bounds__(kMergeThreads) gn_merge_kernel(const __grid_constant__ GnArgs a) {
  __shared__ Moments of[kMergeThreads / 32];
  const int g = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const float2* part = a.part + static_cast<long long>(blockIdx.y) * a.runs * a.slab_groups + g;
  Moments m = {0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = threadIdx.x; i < a.runs; i += kMergeThreads) {
    const float2 v = part[static_cast<long long>(i) * a.slab_groups];
    const int c = min(a.rows_per_cta, a.p - i * a.rows_per_cta);
    merge(m, Moments{static_cast<float>(c) * a.cpg, v.x, v.y});
  }
  m = warp_merge(m);
  if ((threadIdx.x & 31) == 0) of[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kMergeThreads / 32; ++i) merge(m, of[i]);
    a.stat[static_cast<long long>(blockIdx.y) * a.slab_groups + g] = mean_and_factor(m, a.eps);
  }
}

template <bool ONE, bool SILU, bool FP8, int T>
__global__ void __launch_bounds__(T, 1024 / T) gn_apply_kernel(const __grid_constant__ GnArgs a) {
  const Place<FP8, T> at(a, 0);
  const int r0 = blockIdx.x * a.rows_per_cta;
  const int rows = min(a.rows_per_cta, a.p - r0);
  const int n = at.count(rows);
  const int step = at.lanes * a.vecs;
  const long long row0 = static_cast<long long>(blockIdx.y) * a.p + r0 + at.lane;
  const uint4* x = a.x + row0 * a.vecs + at.v;
  pdl_launch_dependents();
  pdl_wait();
  uint4 raw[4];
  auto load = [&](int i) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      raw[j] = i + j < n ? __ldcs(x + static_cast<long long>(i + j) * step) : make_uint4(0, 0, 0, 0);
  };
  load(0);  // in front of the statistics, which wait for memory twice
  Affine<ONE, SILU, FP8, T> affine;
  affine.load_params(a, at, 0);
  const float2* stat = a.stat + static_cast<long long>(blockIdx.y) * a.slab_groups;
  affine.load_stat(at, [&](int e) { return stat[(8 * at.v + e) / a.cpg]; });
  uint8_t* y = static_cast<uint8_t*>(a.y) + (row0 * a.vecs + at.v) * (FP8 ? 8 : 16);
  float* scales = FP8 ? a.scales + row0 * a.blocks : nullptr;
  const int end = FP8 ? (rows + at.lanes - 1) / at.lanes : n;
  for (int i = 0; i < end; i += 4) {
    if (i > 0) load(i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j < end)
        affine.write(at, raw[j], y + static_cast<long long>(i + j) * step * (FP8 ? 8 : 16),
                     FP8 ? scales + static_cast<long long>(i + j) * at.lanes * a.blocks : nullptr, i + j < n);
    }
  }
}

// -------------------------------------------------------------------- host --

// Channels of a slab: whole groups, whole vectors (whole blocks of 128 for
// e4m3), at least 64 of them where there are that many.
int slab_channels(int c, int groups, bool fp8) {
  const int unit = std::lcm(c / groups, fp8 ? kScaleBlock : 8);
  if (unit >= c) return c;
  return std::min(c, unit * std::max(1, 64 / unit));
}

struct GnPlan {
  bool cluster;
  int threads;
  int slab_c, slabs, slab_groups;
  int ranks, rows, rounds;
  int cols_at, red_at, keep_at;
  size_t smem;
  int runs;
  long long units;
  size_t ws_bytes;
};

constexpr size_t kMaxSmem = 232448;

int align16(int v) { return (v + 15) / 16 * 16; }

// Clusters of `ranks` CTAs that run at the same time with `k` CTAs to an SM at
// most. On this GPU with one: 15 of eight or seven, 23 of six, 28 of
// five, 36 of four.
struct GnCaps {
  int at_once[kMaxRanks + 1][4];
};

// Dynamic shared memory with which an SM takes `k` CTAs and no more.
constexpr size_t smem_for(int k) { return kMaxSmem / (k + 1) + 1024; }

// `caps` (nullptr: unknown) changes only how a cluster plan is cut.
GnPlan gn_plan(int n, int p, int c, int groups, bool fp8, const GnCaps* caps) {
  GnPlan g = {};
  const int cpg = c / groups;
  const int parts = 8 / std::gcd(cpg, 8);
  g.slab_c = slab_channels(c, groups, fp8);
  g.slabs = (c + g.slab_c - 1) / g.slab_c;
  g.slab_groups = g.slab_c / cpg;
  g.units = static_cast<long long>(n) * g.slabs;
  // the widest slab has the fewest positions side by side
  const int slots = fp8 ? (g.slab_c / 8 + 15) / 16 * 16 : g.slab_c / 8;
  const int last_c = c - (g.slabs - 1) * g.slab_c;
  const int last = fp8 ? (last_c / 8 + 15) / 16 * 16 : last_c / 8;
  auto red_bytes = [&](int sl) { return gn_red_rows(sl, g.threads) * sl * parts * 4; };
  auto cut = [&](int ranks, int threads) {
    g.threads = std::max(threads, slots > 256 ? 512 : 256);
    const int lanes = g.threads / slots;
    g.cols_at = align16(g.slab_groups * 8);
    g.red_at = g.cols_at + align16(slots * parts * 8);
    g.keep_at = g.red_at + align16(std::max(red_bytes(slots), red_bytes(last)));
    g.ranks = ranks;
    g.rows = (p - 1) / ranks + 1;
    g.rounds = (g.rows + lanes - 1) / lanes;
    g.smem = g.keep_at + static_cast<size_t>(g.rows) * slots * 16;
  };
  constexpr size_t kHalf = kMaxSmem / 2 - 1024;  // what leaves room for a second CTA on the SM
  cut(1, 256);
  // two CTAs to an SM where eight of them hold the slab, and more CTAs while
  // SMs are idle and a thread still has several vectors
  while (g.ranks < kMaxRanks && (g.smem > kHalf || (g.units * g.ranks < 152 && g.rounds > 2))) cut(g.ranks * 2, 256);
  // Where the SMs hold one CTA of a cluster each, fifteen clusters of eight run
  // at a time (the sixteenth waits for the first) and nothing fills their waits,
  // and few clusters leave SMs idle: two readings by all SMs are faster once there
  // is enough to read.
  // Clusters against two readings in us (silu):
  //   16 x 12800 x 512, 32 groups   136 / 108   (16 x 7000, two CTAs to an SM: 60 / 64)
  //   16 x 11520 x 64, 2 groups    28.0 / 20.7  (15 instances:              16.1 / 18.5)
  //   1 x 5632 x 64, 2 groups, 22 rounds   8.5 / 7.2   (3840, 15 rounds:      7.2 / 7.2)
  //   4 x 3240 x 208, 1 group, 45 rounds  12.4 / 9.4   (2160, 30 rounds:     10.1 / 8.7)
  //   8 x 3240 x 208                      12.5 / 11.3  (2160:               10.3 / 11.6)
  // (Clusters of 16 CTAs lie between: 3 x 3234 x 168 e4m3 18.5 with 8, 12.9 with
  // 16, 12.5 with two readings; 4 x 17253 x 112 22.7 with 16, 13.4.)
  g.cluster = g.smem <= kMaxSmem && !(g.smem > kHalf && g.units > 15) && g.rounds <= 5 * std::max(4LL, g.units);
  if (g.cluster) {
    // Many clusters, or several of four CTAs or more: as many CTAs as let all
    // clusters run at once, with the fewest rounds of vectors on an SM; a second CTA on it hides
    // some of the first one's waits, so that its rounds count for a part. CTAs
    // are put two to an SM while others are idle unless their shared memory
    // forbids it, so it is asked for: 24 x 1500 x 128 to e4m3 9.7 -> 8.1 us,
    // 20 x 3432 x 64 11.0 -> 8.0 (six CTAs), 12 x 3432 x 64 7.5 -> 7.0,
    // 75 x 1500 x 120 27.1 -> 19.0, 120 x 400 x 64 7.5 -> 6.3 (one CTA each).
    size_t least = 0;
    int per_sm = 0;  // 0: as it comes
    if (caps && (g.ranks >= 4 || g.units > 36)) {
      int best = INT_MAX, ranks = g.ranks;
      for (int r = kMaxRanks; r >= (g.units > 36 ? 1 : 4); --r) {
        cut(r, 256);
        for (int k = 1; k <= 3; ++k) {
          const int cost = g.rounds * (k == 1 ? 10 : k * (fp8 ? 8 : 9));
          if (k * g.threads <= 1024 && k * (g.smem + 1024) <= kMaxSmem + 1024 && g.units <= caps->at_once[r][k] && cost < best)
            best = cost, ranks = r, per_sm = k;
        }
      }
      cut(ranks, 256);
      if (per_sm > 0) least = smem_for(per_sm);
    }
    // 512 threads where each still has eight vectors and only one partial sum
    // to hand over: 4 x 3432 x 1024 (32 groups) takes 12.8 us against 13.5 with
    // 256; with eight partial sums, 3 x 3555 x 480 takes 12.5 against 11.5
    if (parts == 1 && g.rounds >= 16 && per_sm <= 2) {
      const size_t room = g.smem > kHalf ? kMaxSmem : kHalf;
      cut(g.ranks, 512);
      if (g.smem > room) cut(g.ranks, 256);
    }
    g.smem = std::max(g.smem, least);
    return g;
  }
  g.slab_c = c;
  g.slabs = 1;
  g.slab_groups = groups;
  g.units = n;
  g.threads = c > 2048 ? 512 : 256;
  // Runs of 32 vectors a thread: 16 x 219648 x 256 takes 790 us with 32, 794
  // with 64. (Launching a frame at a time, to find it in L2 the second time, took
  // 1.0-1.1 ms.) What is not worth 1.5 rounds of the CTAs that run at a time is
  // cut so that the last round is full, at about four vectors' time for a CTA's
  // start and end: 2 x 21996 x 648 e4m3 57.2 -> 47.7 us, 7 x 14000 x 320 46.8 ->
  // 38.2; from there on it gains nothing (3 x 50000 x 840 148 -> 151). Runs of at
  // least four: 1 x 6192 x 624 e4m3 15.2 us with eight, 13.2 with four, 13.1 with two.
  const int lanes = g.threads / (c / 8);
  const int per = (p - 1) / lanes + 1;
  const int at_once = 608 * 256 / g.threads;  // four CTAs of 256 threads to an SM
  int run = 32;
  if (static_cast<long long>(n) * per < 48LL * at_once) {
    int best = INT_MAX;
    for (int r = 4; r <= 40; ++r) {
      const int cost = ((n * ((per - 1) / r + 1) - 1) / at_once + 1) * (r + 4);
      if (cost < best) best = cost, run = r;
    }
  }
  g.rows = lanes * run;
  g.runs = (p - 1) / g.rows + 1;
  g.cols_at = align16(red_bytes(c / 8));
  // partial sums and columns, at most 16 KB of each: no more than a launch has unasked
  g.smem = g.cols_at + static_cast<size_t>(c / 8) * parts * 4;
  g.ws_bytes = static_cast<size_t>(n) * (g.runs + 1) * groups * sizeof(float2);
  return g;
}

// Asked of the CUDA runtime once per device.
cc_status gn_caps(const char* what, int device, const GnCaps** out) {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static GnCaps known[kMaxDevices];
  static bool ok[kMaxDevices] = {};
  if (device < 0 || device >= kMaxDevices) return fail(CC_ERR_UNSUPPORTED, "%s: device index %d", what, device);
  std::lock_guard<std::mutex> lock(mu);
  if (!ok[device]) {
    auto kern = gn_cluster_kernel<true, false, false, 256>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    GnCaps caps = {};
    for (int r = 1; r <= kMaxRanks; ++r) {
      for (int k = 1; k <= 3; ++k) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = r;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(r);
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = smem_for(k);
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&caps.at_once[r][k], kern, &cfg);
      }
    }
    if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: clusters at a time: %s", what, cudaGetErrorString(e));
    known[device] = caps;
    ok[device] = true;
  }
  *out = &known[device];
  return CC_OK;
}

template <bool ONE, bool SILU, bool FP8, int T>
cc_status launch_cluster(const char* what, GnArgs& a, const GnPlan& g, cudaStream_t s) {
  auto kern = gn_cluster_kernel<ONE, SILU, FP8, T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: kernel attributes: %s", what, cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.ranks, g.slabs, static_cast<unsigned>(g.units / g.slabs));
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = g.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = g.ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: launch: %s", what, cudaGetErrorString(e));
  return launch_status(what);
}

template <bool ONE, bool SILU, bool FP8, int T>
cc_status launch_twice(const char* what, GnArgs& a, const GnPlan& g, int n, cudaStream_t s) {
  auto moments = gn_moments_kernel<ONE, T>;
  cudaError_t e = launch_pdl(moments, dim3(g.runs, n), dim3(T), g.smem, s, a);
  if (e == cudaSuccess) e = launch_pdl(gn_merge_kernel, dim3(a.slab_groups, n), dim3(kMergeThreads), 0, s, a);
  if (e == cudaSuccess) e = launch_pdl(gn_apply_kernel<ONE, SILU, FP8, T>, dim3(g.runs, n), dim3(T), 0, s, a);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: launch: %s", what, cudaGetErrorString(e));
  return launch_status(what);
}

template <bool ONE, bool SILU, bool FP8>
cc_status launch_group_norm(const char* what, GnArgs& a, const GnPlan& g, int n, cudaStream_t s) {
  if (!g.cluster)
    return g.threads == 512 ? launch_twice<ONE, SILU, FP8, 512>(what, a, g, n, s)
                            : launch_twice<ONE, SILU, FP8, 256>(what, a, g, n, s);
  return g.threads == 512 ? launch_cluster<ONE, SILU, FP8, 512>(what, a, g, s)
                          : launch_cluster<ONE, SILU, FP8, 256>(what, a, g, s);
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
  const size_t need = gn_plan(n, p, c, groups, fp8, nullptr).ws_bytes;
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(CC_ERR_INVALID, "%s: workspace of %zu bytes needed (got %zu)", what, need, ws ? ws_bytes : 0);
  DeviceInfo di;
  if ((st = device_info(&di)) != CC_OK) return st;
  const GnCaps* caps;
  if ((st = gn_caps(what, di.device, &caps)) != CC_OK) return st;
  const GnPlan g = gn_plan(n, p, c, groups, fp8, caps);
  GnArgs a = {};
  a.x = reinterpret_cast<const uint4*>(x);
  a.gamma = reinterpret_cast<const uint4*>(gamma);
  a.beta = reinterpret_cast<const uint4*>(beta);
  a.y = y;
  a.scales = scales;
  a.p = p;
  a.vecs = c / 8;
  a.blocks = (c + kScaleBlock - 1) / kScaleBlock;
  a.slab_vecs = g.slab_c / 8;
  a.cpg = c / groups;
  const int gw = std::gcd(a.cpg, 8);
  a.gw_shift = gw == 8 ? 3 : gw == 4 ? 2 : gw == 2 ? 1 : 0;
  a.per = a.cpg / gw;
  a.eps = eps;
  a.slab_groups = g.slab_groups;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.rows_per_cta = g.rows;
  a.rounds = g.rounds;
  a.cols_at = g.cols_at;
  a.red_at = g.red_at;
  a.keep_at = g.keep_at;
  a.runs = g.runs;
  if (!g.cluster) {
    a.stat = static_cast<float2*>(ws);
    a.part = a.stat + static_cast<size_t>(n) * groups;
  }
  const bool silu = act == CC_ACT_SILU;
  if (gw == 8) {
    if (fp8)
      return silu ? launch_group_norm<true, true, true>(what, a, g, n, s)
                  : launch_group_norm<true, false, true>(what, a, g, n, s);
    return silu ? launch_group_norm<true, true, false>(what, a, g, n, s)
                : launch_group_norm<true, false, false>(what, a, g, n, s);
  }
  if (fp8)
    return silu ? launch_group_norm<false, true, true>(what, a, g, n, s)
                : launch_group_norm<false, false, true>(what, a, g, n, s);
  return silu ? launch_group_norm<false, true, false>(what, a, g, n, s)
              : launch_group_norm<false, false, false>(what, a, g, n, s);
}

}  // namespace
}  // namespace cc

using namespace cc;

extern "C" size_t cc_group_norm_workspace_bytes(int n, int p, int c, int groups) {
  if (n <= 0 || n > 65535 || p <= 0 || p > (1 << 30) || c < 8 || c > kGnMaxChannels || c % 8 != 0 || groups <= 0 || c % groups != 0) return 0;
  return std::max(gn_plan(n, p, c, groups, false, nullptr).ws_bytes,
                  gn_plan(n, p, c, groups, true, nullptr).ws_bytes);
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
