// RMS norm of every query and key head with the rotation of its channel pairs
// in the same pass; the keys and values go to rows or into a paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma
//   (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c),  (c, s) = rot[pos][pair]
//
// in fp32, rounded once. A value costs eight operations and is read and written
// once, so memory bounds the pass where there are many rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cc.h"
#include "cc_host.h"
#include "cc_paged.cuh"
#include "cc_ptx.cuh"
#include "cc_rows.cuh"

namespace cc {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeRows = 128;  // most rows of a CTA

struct RopeArgs {
  const uint4 *q, *k, *v;  // v: append only
  const uint4 *gamma_q, *gamma_k;
  const float2* rot;
  const int* pos;
  uint4 *q_out, *k_out, *v_out;
  long long rows;
  int heads, kv_heads;
  int cta_rows;                    // rows of a CTA
  unsigned chunks;                 // groups of heads that CTAs take: of queries, of keys, of values
  int q_chunks, k_chunks;
  int vecs;                        // D / 8
  int rot_vecs;                    // rd / 8
  int positions;
  long long ld_q, ld_k, ld_v, ld_qo;       // vectors of eight channels from here on
  long long ko_row, ko_page, ko_head;      // rows: row stride; cache: token stride
  long long vo_row, vo_page, vo_head;
  KvPlan plan;                             // append only
  float inv_d, eps;
  unsigned int* err;
};

// A CTA takes up to kRopeRows rows and, of each, HC neighbouring heads of one
// kind (queries, keys or, copied as they are, values): its threads first look up
// where the rows belong, one row each, so that the chain of loads behind a place
// (sequence, length, page) is waited for once. Then LPH lanes hold a head, eight
// channels each, and load the next row's heads before they work on this one's; a
// row's rotation factors are loaded once for its HC heads.
//
// Bound by memory where there are many rows: 13728 rows of 16 + 16 heads of 128
// channels take 40 us with pairs, 5.8 TB/s or 0.86 of a copy's rate. On the way
// there, from 56: places looked up for a CTA's rows at once and the next row's
// heads loaded before this one is worked on 47, CTAs of 128 threads (more of
// them, so that their beginnings and ends overlap) 42, two heads to a thread and
// nine CTAs to an SM 40. All of that was measured with pairs. Halves take 59 us
// (0.59 of a copy's rate), and 19.4 instead of 14.8 for three appended chunks of
// 77 to 4001 rows of 10 heads of 96: every channel is exchanged between lanes, so
// that the load-store unit's data pipe is busy for 80 % of the time (pairs 53 %)
// and four times as many warps wait for it, and with eight factors of each kind
// instead of four the 56 registers of nine CTAs do not do (32 to 40 bytes a
// thread are spilled and 40 to 48 read back, with a cache 68 to 76 and 100 to
// 124; pairs spill none). Single tokens are bound by the host's call (11 to 15
// us; on the device 2.2, and 3.8 with a cache, whose place hangs on three loads
// in a row).
template <int LPH, int HC, bool HALVES, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, 9) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ long long s_out[kRopeRows];
  __shared__ int s_pos[kRopeRows];  // -1: the row is left out
  constexpr int kSlots = kRopeThreads / LPH;
  const int lane = threadIdx.x % LPH, group = threadIdx.x / LPH;
  const unsigned mask = LPH == 32 ? 0xffffffffu
                                  : ((1u << (LPH % 32)) - 1u) << (threadIdx.x % 32 / LPH * LPH);
  const bool on = lane < a.vecs;
  const unsigned block = blockIdx.x / a.chunks;  // of rows
  const int chunk = static_cast<int>(blockIdx.x - block * a.chunks);
  const int kind = (chunk >= a.q_chunks) + (chunk >= a.q_chunks + a.k_chunks);
  const int h0 = (chunk - (kind == 0 ? 0 : kind == 1 ? a.q_chunks : a.q_chunks + a.k_chunks)) * HC;
  const int heads = min(HC, (kind == 0 ? a.heads : a.kv_heads) - h0);
  const long long r0 = static_cast<long long>(block) * a.cta_rows;
  const int rows = static_cast<int>(min(static_cast<long long>(a.cta_rows), a.rows - r0));
  const long long ld = kind == 0 ? a.ld_q : kind == 1 ? a.ld_k : a.ld_v;
  const uint4* x = (kind == 0 ? a.q : kind == 1 ? a.k : a.v) + r0 * ld + h0 * a.vecs + lane;
  const long long out_head = kind == 0 ? a.vecs : kind == 1 ? a.ko_head : a.vo_head;
  uint4* y = (kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out) + h0 * out_head + lane;
  const uint4* gamma = kind == 0 ? a.gamma_q : a.gamma_k;
  pdl_launch_dependents();
  pdl_wait();
  auto load = [&](int i, uint4 (&raw)[HC]) {
#pragma unroll
    for (int j = 0; j < HC; ++j)
      raw[j] = on && j < heads ? __ldcs(x + i * ld + j * a.vecs) : make_uint4(0, 0, 0, 0);
  };
  uint4 next[HC];
  if (group < rows) load(group, next);
  const Vec8 g = kind < 2 && on && gamma ? unpack8(gamma[lane]) : splat8(1.f);
  if (threadIdx.x < rows) {
    const long long r = r0 + threadIdx.x;
    long long p = r, out = r * (kind == 0 ? a.ld_qo : a.ko_row);
    bool bad = false, none = false;
    if (APPEND) {
      int page = 0, slot = 0;
      const PlaceResult res = find_place(a.plan, static_cast<int>(r), p, page, slot);
      bad = res == PLACE_BAD;
      none = res == PLACE_NONE;
      if (kind > 0) out = kind == 1 ? page * a.ko_page + slot * a.ko_row : page * a.vo_page + slot * a.vo_row;
    }
    if (a.pos) p = a.pos[r];
    bad = bad || (!none && a.rot_vecs > 0 && (p < 0 || p >= a.positions));
    if (bad) atomicOr(a.err, DEVERR_BOUNDS);
    s_pos[threadIdx.x] = bad || none ? -1 : a.rot_vecs > 0 ? static_cast<int>(p) : 0;
    s_out[threadIdx.x] = out;
  }
  __syncthreads();
  const bool turn = kind < 2 && lane < a.rot_vecs;
  const int half = a.rot_vecs / 2;
  const int other = threadIdx.x % 32 - lane + (turn ? (lane < half ? lane + half : lane - half) : lane);
  for (int i = group; i < rows; i += kSlots) {
    uint4 raw[HC];
#pragma unroll
    for (int j = 0; j < HC; ++j) raw[j] = next[j];
    if (i + kSlots < rows) load(i + kSlots, next);
    const int p = s_pos[i];
    if (p < 0) continue;
    uint4* dst = y + s_out[i];
    if (APPEND && kind == 2) {
#pragma unroll
      for (int j = 0; j < HC; ++j) {
        if (on && j < heads) dst[j * out_head] = raw[j];
      }
      continue;
    }
    // the factors of this lane's channels
    float c[HALVES ? 8 : 4], s[HALVES ? 8 : 4];
    if (turn) {
      const float4* t = reinterpret_cast<const float4*>(a.rot + static_cast<long long>(p) * (a.rot_vecs * 4)) +
                        (HALVES ? (lane < half ? lane : lane - half) * 4 : lane * 2);
#pragma unroll
      for (int e = 0; e < (HALVES ? 4 : 2); ++e) {
        const float4 f = t[e];
        c[2 * e] = f.x, s[2 * e] = f.y, c[2 * e + 1] = f.z, s[2 * e + 1] = f.w;
      }
      if (HALVES && lane < half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = -s[e];
      }
    }
#pragma unroll
    for (int j = 0; j < HC; ++j) {
      if (j >= heads) break;
      Vec8 f = unpack8(raw[j]);
      f32x2 sq = pair(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) sq = fma2(f.p[e], f.p[e], sq);
      float sum = lo(sq) + hi(sq);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
      const float rs = rsqrtf(fmaf(sum, a.inv_d, a.eps));  // off by at most two units in the last place
#pragma unroll
      for (int e = 0; e < 4; ++e) f.p[e] = mul2(g.p[e], mul2(f.p[e], pair(rs, rs)));
      if (HALVES) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = __shfl_sync(mask, f[e], other);
          v[e] = turn ? fmaf(z, s[e], f[e] * c[e]) : f[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) f.p[e] = pair(v[2 * e], v[2 * e + 1]);
      } else if (turn) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x0 = lo(f.p[e]), x1 = hi(f.p[e]);
          f.p[e] = pair(x0 * c[e] - x1 * s[e], x0 * s[e] + x1 * c[e]);
        }
      }
      if (on) dst[j * out_head] = pack8(f);
    }
  }
}

template <int LPH, bool APPEND>
cc_status launch_rope(const char* what, RopeArgs& a, int style, int sms, cudaStream_t stream) {
  constexpr int kSlots = kRopeThreads / LPH, HC = 2;
  a.q_chunks = (a.heads + HC - 1) / HC;
  a.k_chunks = (a.kv_heads + HC - 1) / HC;
  const long long chunks = a.q_chunks + static_cast<long long>(APPEND ? 2 : 1) * a.k_chunks;
  a.chunks = static_cast<unsigned>(chunks);
  // rows of a CTA: as many as leave about 24 CTAs to an SM, whole rounds of its lanes
  const long long want = a.rows * chunks / (sms * 24ll) / kSlots * kSlots;
  a.cta_rows = static_cast<int>(std::max<long long>(kSlots, std::min<long long>(want, kRopeRows)));
  const long long ctas = (a.rows + a.cta_rows - 1) / a.cta_rows * chunks;
  if (ctas > 0x7fffffffLL) return fail(CC_ERR_UNSUPPORTED, "%s: too many rows of heads", what);
  const dim3 grid(static_cast<unsigned>(ctas));
  const cudaError_t e =
      style == CC_ROT_HALVES
          ? launch_pdl(qk_norm_rope_kernel<LPH, HC, true, APPEND>, grid, dim3(kRopeThreads), 0, stream, a)
          : launch_pdl(qk_norm_rope_kernel<LPH, HC, false, APPEND>, grid, dim3(kRopeThreads), 0, stream, a);
  if (e != cudaSuccess) return fail(CC_ERR_CUDA, "%s: launch: %s", what, cudaGetErrorString(e));
  return launch_status(what);
}

template <bool APPEND>
cc_status run_rope(const char* what, RopeArgs& a, int style, void* stream) {
  DeviceInfo di;
  const cc_status st = device_info(&di);
  if (st != CC_OK) return st;
  a.err = di.err_word;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return a.vecs <= 4    ? launch_rope<4, APPEND>(what, a, style, di.sm_count, cs)
         : a.vecs <= 8  ? launch_rope<8, APPEND>(what, a, style, di.sm_count, cs)
         : a.vecs <= 16 ? launch_rope<16, APPEND>(what, a, style, di.sm_count, cs)
                        : launch_rope<32, APPEND>(what, a, style, di.sm_count, cs);
}

// The checks that both entry points share.
cc_status check_heads(const char* what, const void* q, const void* k, const void* gamma_q, const void* gamma_k,
                      const void* rot, const void* q_out, const void* k_out, int heads, int kv_heads, int d, int rd,
                      int positions, int64_t ld_q, int64_t ld_k, int64_t ld_qo, float eps, int style) {
  if (heads < 0 || kv_heads < 0 || d <= 0 || heads + (int64_t)kv_heads == 0)
    return fail(CC_ERR_INVALID, "%s: head counts must not be negative, their sum and D be positive", what);
  if ((heads && (!q || !q_out)) || (kv_heads && (!k || !k_out))) return fail(CC_ERR_INVALID, "%s: null pointer", what);
  if (!aligned16(q) || !aligned16(k) || !aligned16(gamma_q) || !aligned16(gamma_k) || !aligned16(rot) ||
      !aligned16(q_out) || !aligned16(k_out))
    return fail(CC_ERR_INVALID, "%s: pointers must be 16-byte aligned", what);
  if (d % 16 != 0 || d > 256)
    return fail(CC_ERR_UNSUPPORTED, "%s: D must be a multiple of 16 up to 256 (got %d)", what, d);
  if (heads > 65536 || kv_heads > 65536) return fail(CC_ERR_UNSUPPORTED, "%s: at most 65536 heads", what);
  if (rd < 0 || rd > d || rd % 16 != 0)
    return fail(CC_ERR_INVALID, "%s: the rotated channels must be a multiple of 16 up to D (got %d)", what, rd);
  if (rd > 0 && (!rot || positions <= 0)) return fail(CC_ERR_INVALID, "%s: a rotation needs its table", what);
  if ((heads && (ld_q < (int64_t)heads * d || ld_qo < (int64_t)heads * d)) || (kv_heads && ld_k < (int64_t)kv_heads * d) ||
      ld_q % 8 || ld_qo % 8 || ld_k % 8)
    return fail(CC_ERR_INVALID, "%s: row strides must hold the heads and be multiples of 8", what);
  if (!(eps > 0.f && eps <= 1e30f)) return fail(CC_ERR_INVALID, "%s: eps must be positive and finite", what);
  if (style != CC_ROT_PAIRS && style != CC_ROT_HALVES) return fail(CC_ERR_INVALID, "%s: unknown style %d", what, style);
  return CC_OK;
}

RopeArgs rope_args(const cc_bf16* q, const cc_bf16* k, const cc_bf16* gamma_q, const cc_bf16* gamma_k, const float* rot,
                   const int32_t* pos, cc_bf16* q_out, int rows, int heads, int kv_heads, int d, int rd, int positions,
                   int64_t ld_q, int64_t ld_k, int64_t ld_qo, float eps) {
  RopeArgs a = {};
  a.q = reinterpret_cast<const uint4*>(q);
  a.k = reinterpret_cast<const uint4*>(k);
  a.gamma_q = reinterpret_cast<const uint4*>(gamma_q);
  a.gamma_k = reinterpret_cast<const uint4*>(gamma_k);
  a.rot = reinterpret_cast<const float2*>(rot);
  a.pos = pos;
  a.q_out = reinterpret_cast<uint4*>(q_out);
  a.rows = rows;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.vecs = d / 8;
  a.rot_vecs = rd / 8;
  a.positions = positions;
  a.ld_q = ld_q / 8;
  a.ld_k = ld_k / 8;
  a.ld_qo = ld_qo / 8;
  a.inv_d = 1.f / static_cast<float>(d);
  a.eps = eps;
  return a;
}

}  // namespace
}  // namespace cc

using namespace cc;

extern "C" cc_status cc_qk_norm_rope(const cc_bf16* q, const cc_bf16* k, const cc_bf16* gamma_q,
                                     const cc_bf16* gamma_k, const float* rot, const int32_t* pos, cc_bf16* q_out,
                                     cc_bf16* k_out, int rows, int heads, int kv_heads, int d, int rd, int positions,
                                     int64_t ld_q, int64_t ld_k, int64_t ld_qo, int64_t ld_ko, float eps, int style,
                                     void* stream) {
  const char* what = "qk_norm_rope";
  cc_status st;
  if (empty_request(what, {rows}, &st)) return st;
  if ((st = check_heads(what, q, k, gamma_q, gamma_k, rot, q_out, k_out, heads, kv_heads, d, rd, positions, ld_q, ld_k,
                        ld_qo, eps, style)) != CC_OK)
    return st;
  if ((kv_heads && ld_ko < (int64_t)kv_heads * d) || ld_ko % 8)
    return fail(CC_ERR_INVALID, "%s: row strides must hold the heads and be multiples of 8", what);
  if (rd > 0 && !pos && rows > positions)
    return fail(CC_ERR_INVALID, "%s: %d rows without positions need a table of as many (got %d)", what, rows, positions);
  RopeArgs a = rope_args(q, k, gamma_q, gamma_k, rot, pos, q_out, rows, heads, kv_heads, d, rd, positions, ld_q, ld_k,
                         ld_qo, eps);
  a.k_out = reinterpret_cast<uint4*>(k_out);
  a.ko_row = ld_ko / 8;
  a.ko_head = d / 8;
  return run_rope<false>(what, a, style, stream);
}

extern "C" cc_status cc_qk_norm_rope_append(const cc_bf16* q, const cc_bf16* k, const cc_bf16* v,
                                            const cc_bf16* gamma_q, const cc_bf16* gamma_k, const float* rot,
                                            const int32_t* pos, cc_bf16* q_out, cc_bf16* k_cache, cc_bf16* v_cache,
                                            const int32_t* q_offsets, const int32_t* kv_lens,
                                            const int32_t* page_table, int rows, int seqs, int max_pages, int pages,
                                            int page_size, int heads, int kv_heads, int d, int rd, int positions,
                                            int64_t ld_q, int64_t ld_k, int64_t ld_v, int64_t ld_qo, int64_t k_page,
                                            int64_t k_token, int64_t k_head, int64_t v_page, int64_t v_token,
                                            int64_t v_head, float eps, int style, void* stream) {
  const char* what = "qk_norm_rope_append";
  cc_status st;
  if (empty_request(what, {rows, seqs}, &st)) return st;
  if (kv_heads <= 0) return fail(CC_ERR_INVALID, "%s: a cache has at least one head", what);
  if ((st = check_heads(what, q, k, gamma_q, gamma_k, rot, q_out, k_cache, heads, kv_heads, d, rd, positions, ld_q,
                        ld_k, ld_qo, eps, style)) != CC_OK)
    return st;
  if (!v || !v_cache) return fail(CC_ERR_INVALID, "%s: null pointer", what);
  if (!aligned16(v) || !aligned16(v_cache))
    return fail(CC_ERR_INVALID, "%s: pointers must be 16-byte aligned", what);
  if (ld_v < (int64_t)kv_heads * d || ld_v % 8)
    return fail(CC_ERR_INVALID, "%s: row strides must hold the heads and be multiples of 8", what);
  if ((st = check_plan(what, q_offsets, kv_lens, page_table, max_pages, pages, page_size)) != CC_OK) return st;
  if ((st = check_cache_strides(what, k_page, k_token, k_head, pages, kv_heads, d)) != CC_OK ||
      (st = check_cache_strides(what, v_page, v_token, v_head, pages, kv_heads, d)) != CC_OK)
    return st;
  RopeArgs a = rope_args(q, k, gamma_q, gamma_k, rot, pos, q_out, rows, heads, kv_heads, d, rd, positions, ld_q, ld_k,
                         ld_qo, eps);
  a.v = reinterpret_cast<const uint4*>(v);
  a.ld_v = ld_v / 8;
  a.k_out = reinterpret_cast<uint4*>(k_cache);
  a.v_out = reinterpret_cast<uint4*>(v_cache);
  a.ko_page = k_page / 8;
  a.ko_row = k_token / 8;
  a.ko_head = k_head / 8;
  a.vo_page = v_page / 8;
  a.vo_row = v_token / 8;
  a.vo_head = v_head / 8;
  a.plan = {q_offsets, kv_lens, page_table, seqs, max_pages, pages, page_size};
  return run_rope<true>(what, a, style, stream);
}
