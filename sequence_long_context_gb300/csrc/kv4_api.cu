// C ABI of the 4-bit KV cache: argument checks on the host, then the launch.
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "kv4_host.h"

namespace usp {
namespace {

bool aligned(const void* p, unsigned n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

constexpr int kMaxCapacity = 0x7fffffff - (1 << 20) + 1;

// The checks every call makes of a cache (usp.h, "The 4-bit KV cache").
usp_status_t check_cache(const usp_kv4_cache_t* c) {
  if (!c || c->B < 0 || c->Hkv < 1 || c->capacity < 0 || c->capacity % kv4::kRowAlign != 0)
    return USP_ERR_INVALID_ARG;
  if (c->B > 65535 || c->Hkv > 65535) return USP_ERR_UNSUPPORTED;
  // the kernels count rows in 32 bits, and step past the last by less than 2^20
  if (c->capacity > kMaxCapacity) return USP_ERR_UNSUPPORTED;
  if (c->D != 64 && c->D != 128) return USP_ERR_UNSUPPORTED;
  const float d[] = {c->k_descale, c->v_descale};
  for (float x : d)
    if (!(x > 0.f) || !std::isfinite(x) || !std::isfinite(1.0f / x)) return USP_ERR_INVALID_ARG;
  if (c->B > 0 && (!c->seq_lens || (c->capacity > 0 && (!c->k_codes || !c->k_scales ||
                                                        !c->v_codes || !c->v_scales))))
    return USP_ERR_INVALID_ARG;
  const void* ptrs[] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales, c->key_weight};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return USP_ERR_ALIGNMENT;
  if (!aligned(c->seq_lens, 4)) return USP_ERR_ALIGNMENT;
  return USP_OK;
}

kv4::Cache view(const usp_kv4_cache_t* c) {
  return {static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->k_scales),
          static_cast<uint8_t*>(c->v_codes), static_cast<uint8_t*>(c->v_scales),
          c->key_weight, c->seq_lens, c->B, c->capacity, c->Hkv};
}

// 32-bit row and unit counts in the decode's kernels
bool too_many_rows(int B, int Tq, int Hq, int Hkv) {
  const long long rows = (long long)(Hq / Hkv) * Tq;
  return rows > (1 << 20) || (long long)B * Hkv * ((rows + 7) / 8) > 0x3fffffffLL;
}

bool valid_dtype(usp_dtype_t t) { return t == USP_BF16 || t == USP_FP32; }

// [a, a + na) and [b, b + nb) share a byte
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

}  // namespace
}  // namespace usp

using namespace usp;

extern "C" {

usp_status_t usp_kv4_append(const usp_kv4_cache_t* cache, const void* k, const void* v,
                            const float* new_weight, const int32_t* cu_seqlens, int T,
                            usp_dtype_t dtype, int32_t* seq_lens_out, usp_stream_t stream) {
  usp_status_t r = check_cache(cache);
  if (r != USP_OK) return r;
  if (T < 0 || !valid_dtype(dtype)) return USP_ERR_INVALID_ARG;
  if (cu_seqlens && cache->B < 1) return USP_ERR_INVALID_ARG;
  if (cache->B > 0 && T > 0 && (!k || !v)) return USP_ERR_INVALID_ARG;
  if (new_weight && !cache->key_weight) return USP_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(new_weight, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(seq_lens_out, 4))
    return USP_ERR_ALIGNMENT;
  if (cache->B == 0) return USP_OK;
  return launch_kv4_append(view(cache), cache->D, k, v, new_weight, cu_seqlens, T,
                           dtype == USP_BF16, 1.0f / cache->k_descale, 1.0f / cache->v_descale,
                           seq_lens_out, reinterpret_cast<cudaStream_t>(stream));
}

usp_status_t usp_kv4_read(const usp_kv4_cache_t* cache, const int32_t* start, int T, void* k,
                          void* v, usp_dtype_t dtype, usp_stream_t stream) {
  usp_status_t r = check_cache(cache);
  if (r != USP_OK) return r;
  if (T < 0 || !valid_dtype(dtype)) return USP_ERR_INVALID_ARG;
  if (cache->B > 0 && T > 0 && (!k || !v)) return USP_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4)) return USP_ERR_ALIGNMENT;
  if (cache->B == 0 || T == 0) return USP_OK;
  return launch_kv4_read(view(cache), cache->D, start, T, k, v, dtype == USP_BF16,
                         cache->k_descale, cache->v_descale,
                         reinterpret_cast<cudaStream_t>(stream));
}

size_t usp_attn_decode_kv4_workspace_size(int B, int Tq, int capacity, int Hq, int Hkv, int D,
                                          int accumulate) {
  usp_kv4_cache_t c{};
  c.capacity = capacity;
  c.Hkv = Hkv;
  c.D = D;
  c.k_descale = c.v_descale = 1.f;
  if (check_cache(&c) != USP_OK || B < 0 || B > 65535 || Tq < 1 || Hq < 1 || Hq % Hkv != 0 ||
      too_many_rows(B, Tq, Hq, Hkv))
    return 0;
  return decode_kv4_workspace(B, Tq, capacity, Hq, Hkv, D, accumulate);
}

usp_status_t usp_attn_decode_kv4(const usp_kv4_cache_t* cache, const void* q, void* out,
                                 float* lse, int Tq, int Hq, float softmax_scale, int causal,
                                 int window, int sink_tokens, int accumulate, usp_dtype_t dtype,
                                 void* workspace, size_t workspace_bytes, usp_stream_t stream) {
  usp_status_t r = check_cache(cache);
  if (r != USP_OK) return r;
  if (Tq < 1 || Hq < 1 || Hq % cache->Hkv != 0 || sink_tokens < 0) return USP_ERR_INVALID_ARG;
  if (dtype == USP_FP32) return USP_ERR_UNSUPPORTED;
  if (dtype != USP_BF16) return USP_ERR_INVALID_ARG;
  if (cache->B > 0 && (!q || !out || !lse)) return USP_ERR_INVALID_ARG;
  if (accumulate && cache->B > 0 && cache->capacity > 0 && !cache->key_weight)
    return USP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 16)) return USP_ERR_ALIGNMENT;
  if (!aligned(workspace, 256)) return USP_ERR_ALIGNMENT;
  if (too_many_rows(cache->B, Tq, Hq, cache->Hkv)) return USP_ERR_UNSUPPORTED;
  if (cache->B == 0) return USP_OK;
  if (!workspace || workspace_bytes < decode_kv4_workspace(cache->B, Tq, cache->capacity, Hq,
                                                           cache->Hkv, cache->D, accumulate))
    return USP_ERR_WORKSPACE;
  DecodeKv4Args a{};
  a.c = view(cache);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.Tq = Tq;
  a.Hq = Hq;
  a.D = cache->D;
  a.scale = softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)cache->D);
  a.k_descale = cache->k_descale;
  a.v_descale = cache->v_descale;
  a.causal = causal ? 1 : 0;
  a.window = window > 0 ? window : 0;
  a.sink = sink_tokens;
  a.accumulate = (accumulate && cache->capacity > 0) ? 1 : 0;
  return launch_decode_kv4(a, workspace, reinterpret_cast<cudaStream_t>(stream));
}

usp_status_t usp_kv4_evict(const usp_kv4_cache_t* src, const usp_kv4_cache_t* dst, int32_t* kept,
                           int keep, int recent, int sink_tokens, usp_stream_t stream) {
  usp_status_t r = check_cache(src);
  if (r == USP_OK) r = check_cache(dst);
  if (r != USP_OK) return r;
  if (dst->B != src->B || dst->Hkv != src->Hkv || dst->D != src->D) return USP_ERR_INVALID_ARG;
  if (keep < 1 || recent < 0 || sink_tokens < 0 || (long long)recent + sink_tokens > keep)
    return USP_ERR_INVALID_ARG;
  if (keep > dst->capacity) return USP_ERR_INVALID_ARG;
  if (src->B > 0 && (!kept || (src->capacity > 0 && !src->key_weight))) return USP_ERR_INVALID_ARG;
  if (!aligned(kept, 16)) return USP_ERR_ALIGNMENT;
  if (src->B == 0) return USP_OK;
  // in place (every pointer the same), or nothing shared
  const bool same = src->k_codes == dst->k_codes && src->k_scales == dst->k_scales &&
                    src->v_codes == dst->v_codes && src->v_scales == dst->v_scales &&
                    src->key_weight == dst->key_weight && src->seq_lens == dst->seq_lens &&
                    src->capacity == dst->capacity;
  {  // (in place, `kept` alone may share nothing with the cache)
    const size_t rs = (size_t)src->B * src->Hkv * src->capacity;
    const size_t rd = (size_t)dst->B * dst->Hkv * dst->capacity;
    const size_t code = src->D / 2, scale = src->D / kv4::kBlock;
    const void* sp[] = {src->k_codes, src->v_codes, src->k_scales, src->v_scales,
                        src->key_weight, src->seq_lens};
    const size_t sn[] = {rs * code, rs * code, rs * scale, rs * scale, rs * 4, (size_t)src->B * 4};
    const void* dp[] = {dst->k_codes, dst->v_codes, dst->k_scales, dst->v_scales,
                        dst->key_weight, dst->seq_lens, kept};
    const size_t dn[] = {rd * code, rd * code, rd * scale, rd * scale, rd * 4, (size_t)dst->B * 4,
                         (size_t)src->B * src->Hkv * keep * 4};
    for (int i = 0; i < 6; ++i)
      for (int j = same ? 6 : 0; j < 7; ++j)
        if (overlap(sp[i], sn[i], dp[j], dn[j])) return USP_ERR_INVALID_ARG;
  }
  return launch_kv4_evict(view(src), view(dst), src->D, kept, keep, recent, sink_tokens,
                          reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
