// Attention with heads: the new tokens of several sequences over a paged cache,
// and queries over an encoder's states.
//
//   o_i = sum_{j < limit(i)} softmax_j(scale q_i . k_j) v_j
//
// Simple form: a warp per query row and head walks the keys 32 at a time with a
// running maximum and sum; a lane takes a key's product, then four channels of
// the weighted sum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "cc.h"
#include "cc_host.h"
#include "cc_paged.cuh"
#include "cc_ptx.cuh"
#include "cc_rows.cuh"

namespace cc {
namespace {

constexpr int kHeadsThreads = 128;

struct HeadsArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  KvPlan plan;      // q_offsets nullptr: sequence b owns rows b * lq .. (b + 1) * lq - 1; page_table nullptr: page b
  int lq;
  long long rows;
  int heads, group, d;
  long long ld_q, ld_o, k_page, k_token, k_head, v_page, v_token, v_head;
  float kx;         // scale * log2(e)
  int block;
  unsigned int* err;
};

__global__ void __launch_bounds__(kHeadsThreads) attn_heads_simple_kernel(const __grid_constant__ HeadsArgs a) {
  __shared__ float sq[kHeadsThreads / 32][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && a.plan.q_offsets) {
    for (int b = threadIdx.x; b < a.plan.seqs; b += kHeadsThreads) {
      if (a.plan.q_offsets[b + 1] < a.plan.q_offsets[b] || a.plan.q_offsets[b + 1] > a.rows)
        atomicOr(a.err, DEVERR_BOUNDS);
    }
  }
  const long long unit = static_cast<long long>(blockIdx.x) * (kHeadsThreads / 32) + warp;
  if (unit >= a.rows * a.heads) return;
  const int r = static_cast<int>(unit / a.heads), h = static_cast<int>(unit % a.heads), hk = h / a.group;
  int seq, begin, end;
  if (a.plan.q_offsets) {
    int lo = 0, hi = a.plan.seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.plan.q_offsets[mid] <= r) lo = mid; else hi = mid;
    }
    seq = lo;
    begin = a.plan.q_offsets[seq];
    end = a.plan.q_offsets[seq + 1];
    if (r < begin || r >= end) return;
  } else {
    seq = r / a.lq;
    begin = seq * a.lq;
    end = begin + a.lq;
  }
  const long long most = static_cast<long long>(a.plan.max_pages) * a.plan.page_size;
  long long len = a.plan.kv_lens ? a.plan.kv_lens[seq] : a.plan.page_size;
  const int n = end - begin;
  if (len < 0 || len > most || (a.block > 0 && len < n)) {
    if (lane == 0) atomicOr(a.err, DEVERR_BOUNDS);
    len = len < 0 ? 0 : len > most ? most : len;
  }
  const int i = r - begin;
  long long limit = len;
  if (a.block > 0) limit = len - n + min(static_cast<long long>(n), (static_cast<long long>(i) / a.block + 1) * a.block);
  for (int c = lane; c < a.d; c += 32) sq[warp][c] = __bfloat162float(a.q[r * a.ld_q + h * a.d + c]);
  __syncwarp();
  float m = __int_as_float(0xff800000u), l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (long long j0 = 0; j0 < limit; j0 += 32) {
    const long long j = j0 + lane;
    float s = __int_as_float(0xff800000u);
    long long vrow = -1;
    if (j < limit) {
      int page = seq, slot = static_cast<int>(j);
      if (a.plan.page_table) {
        const int pg = static_cast<int>(j / a.plan.page_size);
        slot = static_cast<int>(j - static_cast<long long>(pg) * a.plan.page_size);
        page = a.plan.page_table[static_cast<long long>(seq) * a.plan.max_pages + pg];
      }
      if (page < 0 || page >= a.plan.pages) {
        atomicOr(a.err, DEVERR_BOUNDS);
      } else {
        const uint4* kp = reinterpret_cast<const uint4*>(a.k + page * a.k_page + slot * a.k_token + hk * a.k_head);
        vrow = page * a.v_page + slot * a.v_token + hk * a.v_head;
        float dot = 0.f;
        for (int c = 0; c < a.d / 8; ++c) {
          const Vec8 f = unpack8(kp[c]);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(f[e], sq[warp][c * 8 + e], dot);
        }
        s = dot * a.kx;
      }
    }
    float top = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float mn = fmaxf(m, top), base = mn == __int_as_float(0xff800000u) ? 0.f : mn;
    const float f = exp2f(m - base), p = vrow >= 0 ? exp2f(s - base) : 0.f;
    m = mn;
    float sum = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * f + sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= f;
    for (int t = 0; t < 32; ++t) {
      const float w = __shfl_sync(0xffffffffu, p, t);
      const long long at = __shfl_sync(0xffffffffu, vrow, t);
      if (at < 0 || lane * 4 >= a.d) continue;
      const uint2 raw = *reinterpret_cast<const uint2*>(a.v + at + lane * 4);
      acc[0] = fmaf(w, __uint_as_float(raw.x << 16), acc[0]);
      acc[1] = fmaf(w, __uint_as_float(raw.x & 0xffff0000u), acc[1]);
      acc[2] = fmaf(w, __uint_as_float(raw.y << 16), acc[2]);
      acc[3] = fmaf(w, __uint_as_float(raw.y & 0xffff0000u), acc[3]);
    }
  }
  if (lane * 4 < a.d) {
    const float inv = limit > 0 ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      a.o[r * a.ld_o + h * a.d + lane * 4 + e] = __float2bfloat16_rn(limit > 0 ? acc[e] * inv : 0.f);
  }
}

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
  if (heads > 65536 || heads / kv_heads > 128)
    return fail(CC_ERR_UNSUPPORTED, "%s: at most 65536 heads, 128 to a key head", what);
  if (ld_q < (int64_t)heads * d || ld_o < (int64_t)heads * d || ld_q % 8 || ld_o % 8)
    return fail(CC_ERR_INVALID, "%s: row strides must hold the heads and be multiples of 8", what);
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(CC_ERR_INVALID, "%s: scale must be finite and > 0", what);
  return CC_OK;
}

cc_status launch_attn(const char* what, HeadsArgs& a, void* stream) {
  DeviceInfo di;
  const cc_status st = device_info(&di);
  if (st != CC_OK) return st;
  a.err = di.err_word;
  const long long units = a.rows * a.heads, ctas = (units + 3) / 4;
  if (ctas > 0x7fffffffLL) return fail(CC_ERR_UNSUPPORTED, "%s: too many rows", what);
  attn_heads_simple_kernel<<<static_cast<unsigned>(ctas), kHeadsThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launch_status(what);
}

}  // namespace
}  // namespace cc

using namespace cc;

extern "C" size_t cc_attn_paged_workspace_bytes(int rows, int seqs, int heads, int kv_heads, int d) { return 0; }

extern "C" size_t cc_attn_cross_workspace_bytes(int n, int lq, int lk, int heads, int kv_heads, int d) { return 0; }

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
  if ((st = check_cache_strides(what, k_page, k_token, k_head, d)) != CC_OK ||
      (st = check_cache_strides(what, v_page, v_token, v_head, d)) != CC_OK)
    return st;
  if (causal_block < 0) return fail(CC_ERR_INVALID, "%s: the causal block must not be negative", what);
  HeadsArgs a = {};
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.k = reinterpret_cast<const __nv_bfloat16*>(k_cache);
  a.v = reinterpret_cast<const __nv_bfloat16*>(v_cache);
  a.o = reinterpret_cast<__nv_bfloat16*>(o);
  a.plan = {q_offsets, kv_lens, page_table, seqs, max_pages, pages, page_size};
  a.rows = rows;
  a.heads = heads;
  a.group = heads / kv_heads;
  a.d = d;
  a.ld_q = ld_q;
  a.ld_o = ld_o;
  a.k_page = k_page, a.k_token = k_token, a.k_head = k_head;
  a.v_page = v_page, a.v_token = v_token, a.v_head = v_head;
  a.kx = scale * 1.4426950408889634f;
  a.block = causal_block;
  return launch_attn(what, a, stream);
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
  if ((int64_t)n * lq > 0x7fffffffLL) return fail(CC_ERR_UNSUPPORTED, "%s: at most 2^31 - 1 query rows", what);
  HeadsArgs a = {};
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.k = reinterpret_cast<const __nv_bfloat16*>(k);
  a.v = reinterpret_cast<const __nv_bfloat16*>(v);
  a.o = reinterpret_cast<__nv_bfloat16*>(o);
  a.plan = {nullptr, kv_lens, nullptr, n, 1, n, lk};
  a.lq = lq;
  a.rows = static_cast<long long>(n) * lq;
  a.heads = heads;
  a.group = heads / kv_heads;
  a.d = d;
  a.ld_q = ld_q;
  a.ld_o = ld_o;
  a.k_page = ld_k * lk, a.k_token = ld_k, a.k_head = d;
  a.v_page = ld_v * lk, a.v_token = ld_v, a.v_head = d;
  a.kx = scale * 1.4426950408889634f;
  return launch_attn(what, a, stream);
}
