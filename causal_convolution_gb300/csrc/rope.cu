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

constexpr int kRopeThreads = 256;

struct RopeArgs {
  const uint4 *q, *k, *v;  // v: append only
  const uint4 *gamma_q, *gamma_k;
  const float2* rot;
  const int* pos;
  uint4 *q_out, *k_out, *v_out;
  long long rows;
  int heads, kv_heads, all_heads;  // all_heads: heads + kv_heads, append: + kv_heads values
  int chunks;                      // ceil(all_heads / HC)
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

// LPH lanes hold a head, eight channels each; they take HC heads of a row, so
// that the rotation's factors are loaded once for them and HC loads of a lane
// are in flight.
template <int LPH, int HC, bool HALVES, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  const int lane = threadIdx.x % LPH;
  const unsigned mask = LPH == 32 ? 0xffffffffu
                                  : ((1u << (LPH % 32)) - 1u) << (threadIdx.x % 32 / LPH * LPH);
  const bool on = lane < a.vecs;
  pdl_launch_dependents();
  pdl_wait();
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  const uint4 gq = on && a.gamma_q ? a.gamma_q[lane] : ones;
  const uint4 gk = on && a.gamma_k ? a.gamma_k[lane] : ones;
  const long long units = a.rows * a.chunks;
  constexpr int kSlots = kRopeThreads / LPH;
  for (long long u = static_cast<long long>(blockIdx.x) * kSlots + threadIdx.x / LPH; u < units;
       u += static_cast<long long>(gridDim.x) * kSlots) {
    const long long r = u / a.chunks;
    const int h0 = static_cast<int>(u - r * a.chunks) * HC;
    uint4 raw[HC];
#pragma unroll
    for (int j = 0; j < HC; ++j) {
      const int h = h0 + j;
      raw[j] = make_uint4(0, 0, 0, 0);
      if (!on || h >= a.all_heads) continue;
      const uint4* src = h < a.heads                    ? a.q + r * a.ld_q + h * a.vecs
                         : h < a.heads + a.kv_heads ? a.k + r * a.ld_k + (h - a.heads) * a.vecs
                                                        : a.v + r * a.ld_v + (h - a.heads - a.kv_heads) * a.vecs;
      raw[j] = __ldcs(src + lane);
    }
    // where the row belongs
    long long p = r, ko = r * a.ko_row, vo = 0;
    if (APPEND) {
      int seq, page, slot;
      const PlaceResult res = find_place<LPH>(a.plan, static_cast<int>(r), lane, mask, p, seq, page, slot);
      if (res != PLACE_OK) {
        if (res == PLACE_BAD && lane == 0) atomicOr(a.err, DEVERR_BOUNDS);
        continue;
      }
      ko = page * a.ko_page + slot * a.ko_row;
      vo = page * a.vo_page + slot * a.vo_row;
    }
    if (a.pos) p = a.pos[r];
    if (a.rot_vecs > 0 && (p < 0 || p >= a.positions)) {
      if (lane == 0) atomicOr(a.err, DEVERR_BOUNDS);
      continue;
    }
    // the factors of this lane's channels
    const bool turn = lane < a.rot_vecs;
    const int half = a.rot_vecs / 2;
    float c[HALVES ? 8 : 4], s[HALVES ? 8 : 4];
    if (turn) {
      const float4* t = reinterpret_cast<const float4*>(a.rot + p * (a.rot_vecs * 4)) +
                        (HALVES ? (lane < half ? lane : lane - half) * 4 : lane * 2);
#pragma unroll
      for (int i = 0; i < (HALVES ? 4 : 2); ++i) {
        const float4 f = t[i];
        c[2 * i] = f.x, s[2 * i] = f.y, c[2 * i + 1] = f.z, s[2 * i + 1] = f.w;
      }
    }
#pragma unroll
    for (int j = 0; j < HC; ++j) {
      const int h = h0 + j;
      if (h >= a.all_heads) break;
      if (APPEND && h >= a.heads + a.kv_heads) {
        if (on) a.v_out[vo + (h - a.heads - a.kv_heads) * a.vo_head + lane] = raw[j];
        continue;
      }
      Vec8 f = unpack8(raw[j]);
      f32x2 sq = pair(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = fma2(f.p[i], f.p[i], sq);
      float sum = lo(sq) + hi(sq);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
      const float rs = 1.f / sqrtf(fmaf(sum, a.inv_d, a.eps));
      const Vec8 g = unpack8(h < a.heads ? gq : gk);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.p[i] = mul2(g.p[i], mul2(f.p[i], pair(rs, rs)));
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = f[i];
      if (HALVES) {
        const int base = threadIdx.x % 32 - lane;
        const int other = base + (turn ? (lane < half ? lane + half : lane - half) : lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float z = __shfl_sync(mask, y[i], other);
          if (turn) y[i] = lane < half ? y[i] * c[i] - z * s[i] : z * s[i] + y[i] * c[i];
        }
      } else if (turn) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = y[2 * i], x1 = y[2 * i + 1];
          y[2 * i] = x0 * c[i] - x1 * s[i];
          y[2 * i + 1] = x0 * s[i] + x1 * c[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) f.p[i] = pair(y[2 * i], y[2 * i + 1]);
      const uint4 res = pack8(f);
      if (!on) continue;
      if (h < a.heads)
        a.q_out[r * a.ld_qo + h * a.vecs + lane] = res;
      else
        a.k_out[ko + (h - a.heads) * a.ko_head + lane] = res;
    }
  }
}

template <int LPH, int HC, bool APPEND>
cc_status launch_rope(const char* what, RopeArgs& a, int style, int sms, cudaStream_t stream) {
  a.chunks = (a.all_heads + HC - 1) / HC;
  const long long units = a.rows * a.chunks;
  constexpr int kSlots = kRopeThreads / LPH;
  const unsigned grid = static_cast<unsigned>(std::min<long long>((units + kSlots - 1) / kSlots, sms * 8ll));
  const cudaError_t e =
      style == CC_ROT_HALVES
          ? launch_pdl(qk_norm_rope_kernel<LPH, HC, true, APPEND>, dim3(grid), dim3(kRopeThreads), 0, stream, a)
          : launch_pdl(qk_norm_rope_kernel<LPH, HC, false, APPEND>, dim3(grid), dim3(kRopeThreads), 0, stream, a);
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
  return a.vecs <= 4    ? launch_rope<4, 4, APPEND>(what, a, style, di.sm_count, cs)
         : a.vecs <= 8  ? launch_rope<8, 4, APPEND>(what, a, style, di.sm_count, cs)
         : a.vecs <= 16 ? launch_rope<16, 4, APPEND>(what, a, style, di.sm_count, cs)
                        : launch_rope<32, 4, APPEND>(what, a, style, di.sm_count, cs);
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
  a.all_heads = heads + kv_heads;
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
  if ((st = check_cache_strides(what, k_page, k_token, k_head, d)) != CC_OK ||
      (st = check_cache_strides(what, v_page, v_token, v_head, d)) != CC_OK)
    return st;
  RopeArgs a = rope_args(q, k, gamma_q, gamma_k, rot, pos, q_out, rows, heads, kv_heads, d, rd, positions, ld_q, ld_k,
                         ld_qo, eps);
  a.v = reinterpret_cast<const uint4*>(v);
  a.ld_v = ld_v / 8;
  a.k_out = reinterpret_cast<uint4*>(k_cache);
  a.v_out = reinterpret_cast<uint4*>(v_cache);
  a.all_heads = heads + 2 * kv_heads;
  a.ko_page = k_page / 8;
  a.ko_row = k_token / 8;
  a.ko_head = k_head / 8;
  a.vo_page = v_page / 8;
  a.vo_row = v_token / 8;
  a.vo_head = v_head / 8;
  a.plan = {q_offsets, kv_lens, page_table, seqs, max_pages, pages, page_size};
  return run_rope<true>(what, a, style, stream);
}
