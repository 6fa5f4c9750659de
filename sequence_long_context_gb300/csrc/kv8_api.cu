// C ABI of the rotation of positions and the paged 8-bit KV cache: argument checks
// on the host, then the launch.
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "kv8_host.h"
#include "kv8_mask.h"

namespace usp {
namespace {

bool aligned(const void* p, unsigned n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}
bool valid_dtype(usp_dtype_t t) { return t == USP_BF16 || t == USP_FP32; }

using kv8::kMaxRows;

// The checks every call makes of a cache (usp.h, "The paged 8-bit KV cache").
usp_status_t check_cache(const usp_kv8_cache_t* c) {
  if (!c || c->B < 0 || c->Hkv < 1 || c->max_pages < 0 || c->num_pages < 0 || c->page_size < 1)
    return USP_ERR_INVALID_ARG;
  if (c->B > 65535 || c->Hkv > 65535) return USP_ERR_UNSUPPORTED;
  if (c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return USP_ERR_UNSUPPORTED;
  if (c->D != 64 && c->D != 128) return USP_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * c->page_size > kMaxRows) return USP_ERR_UNSUPPORTED;
  if ((long long)c->num_pages * c->Hkv > 0x7fffffffLL) return USP_ERR_UNSUPPORTED;
  if (c->B > 0 && !c->seq_lens) return USP_ERR_INVALID_ARG;
  if (c->B > 0 && c->max_pages > 0 && !c->page_table) return USP_ERR_INVALID_ARG;
  if (c->num_pages > 0 && (!c->k_codes || !c->k_exps || !c->v_codes || !c->v_exps))
    return USP_ERR_INVALID_ARG;
  const void* ptrs[] = {c->k_codes, c->k_exps, c->v_codes, c->v_exps};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return USP_ERR_ALIGNMENT;
  if (!aligned(c->seq_lens, 4) || !aligned(c->page_table, 4)) return USP_ERR_ALIGNMENT;
  return USP_OK;
}

kv8::Cache view(const usp_kv8_cache_t* c) {
  kv8::Cache v{};
  v.kc = static_cast<uint8_t*>(c->k_codes);
  v.ke = c->k_exps;
  v.vc = static_cast<uint8_t*>(c->v_codes);
  v.ve = c->v_exps;
  v.table = c->page_table;
  v.lens = c->seq_lens;
  v.B = c->B;
  v.mp = c->max_pages;
  v.np = c->num_pages;
  v.ps = c->page_size;
  v.H = c->Hkv;
  v.cap = c->max_pages * c->page_size;
  v.ps_log2 = c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  return v;
}

// A table of `rows` positions that turns the first rotary_dim of D channels, or none.
usp_status_t check_rope(const float* table, int rows, int rotary_dim, int D) {
  if (!table) return USP_OK;
  if (rows < 1 || rotary_dim < 16 || rotary_dim > D || rotary_dim % 16 != 0)
    return USP_ERR_INVALID_ARG;
  return aligned(table, 16) ? USP_OK : USP_ERR_ALIGNMENT;
}

// [a, a + na) and [b, b + nb) share a byte
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// 32-bit row and unit counts of the attention's kernels
bool too_many_rows(int B, int max_new, int Hq, int Hkv) {
  const long long rows = (long long)(Hq / Hkv) * max_new;
  return rows > (1 << 26) || (long long)B * Hkv * ((rows + 7) / 8) > 0x3ffffffLL;
}

}  // namespace
}  // namespace usp

using namespace usp;

extern "C" {

usp_status_t usp_rope(const void* x, void* y, const float* table, int table_rows, int rotary_dim,
                      int interleaved, int inverse, int B, int S, int H, int D,
                      const int32_t* cu_seqlens, int cp_size, usp_layout_t layout,
                      usp_dtype_t dtype, usp_stream_t stream) {
  if (B < 0 || S < 0 || H < 1 || cp_size < 1 || !table || !valid_dtype(dtype))
    return USP_ERR_INVALID_ARG;
  if (layout != USP_LAYOUT_CONTIGUOUS && layout != USP_LAYOUT_ZIGZAG && layout != USP_LAYOUT_STRIPE)
    return USP_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return USP_ERR_UNSUPPORTED;
  if (S % cp_size != 0 || (layout == USP_LAYOUT_ZIGZAG && S % (2LL * cp_size) != 0))
    return USP_ERR_INVALID_ARG;
  if (cu_seqlens && B < 1) return USP_ERR_INVALID_ARG;
  usp_status_t r = check_rope(table, table_rows, rotary_dim, D);
  if (r != USP_OK) return r;
  if (S > table_rows) return USP_ERR_INVALID_ARG;
  const long long batch = cu_seqlens ? 1 : B;
  const long long tokens = batch * S;
  if (tokens > 0 && (!x || !y)) return USP_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(cu_seqlens, 4)) return USP_ERR_ALIGNMENT;
  const size_t bytes = (size_t)tokens * H * D * (dtype == USP_BF16 ? 2 : 4);
  if (x != y && overlap(x, bytes, y, bytes)) return USP_ERR_INVALID_ARG;
  if (tokens == 0) return USP_OK;
  const kv8::Rope rope{table, table_rows, rotary_dim, interleaved ? 1 : 0};
  return launch_rope(x, y, rope, inverse ? 1 : 0, (int)batch, S, H, D, cu_seqlens, B, cp_size,
                     (int)layout, dtype == USP_BF16, reinterpret_cast<cudaStream_t>(stream));
}

usp_status_t usp_kv8_append(const usp_kv8_cache_t* cache, const void* k, const void* v,
                            const void* q, void* q_out, int Hq, const float* table, int table_rows,
                            int rotary_dim, int interleaved, const int32_t* positions,
                            const int32_t* cu_seqlens, int T, usp_dtype_t dtype,
                            int32_t* seq_lens_out, usp_stream_t stream) {
  usp_status_t r = check_cache(cache);
  if (r != USP_OK) return r;
  if (T < 0 || !valid_dtype(dtype)) return USP_ERR_INVALID_ARG;
  if (T > kMaxRows) return USP_ERR_UNSUPPORTED;
  r = check_rope(table, table_rows, rotary_dim, cache->D);
  if (r != USP_OK) return r;
  // the positions of the cache's rows, all of them in the table (without tokens there are none,
  // and an empty tensor of positions is a null pointer)
  if (T > 0 && table && !positions && (long long)cache->max_pages * cache->page_size > table_rows)
    return USP_ERR_INVALID_ARG;
  if (cu_seqlens && cache->B < 1) return USP_ERR_INVALID_ARG;
  if (cache->B > 0 && T > 0 && (!k || !v)) return USP_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_out != nullptr) || (q && (Hq < 1 || Hq > 65535)))
    return USP_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) ||
      !aligned(positions, 4) || !aligned(cu_seqlens, 4) || !aligned(seq_lens_out, 4))
    return USP_ERR_ALIGNMENT;
  if (cache->B == 0) return USP_OK;
  {
    const size_t el = dtype == USP_BF16 ? 2 : 4;
    const size_t tokens = cu_seqlens ? (size_t)T : (size_t)T * cache->B;
    const size_t nq = tokens * Hq * cache->D * el, nk = tokens * cache->Hkv * cache->D * el;
    if (q && q != q_out && overlap(q, nq, q_out, nq)) return USP_ERR_INVALID_ARG;
    if (q && (overlap(q_out, nq, k, nk) || overlap(q_out, nq, v, nk))) return USP_ERR_INVALID_ARG;
  }
  Kv8AppendArgs a{};
  a.c = view(cache);
  a.rope = kv8::Rope{table, table_rows, rotary_dim, interleaved ? 1 : 0};
  a.k = k;
  a.v = v;
  a.q = q;
  a.q_out = q_out;
  a.positions = positions;
  a.cu = cu_seqlens;
  a.lens_out = seq_lens_out;
  a.T = T;
  a.Hq = Hq;
  a.D = cache->D;
  a.bf16 = dtype == USP_BF16;
  return launch_kv8_append(a, reinterpret_cast<cudaStream_t>(stream));
}

usp_status_t usp_kv8_read(const usp_kv8_cache_t* cache, const int32_t* start, int T, void* k,
                          void* v, usp_dtype_t dtype, usp_stream_t stream) {
  usp_status_t r = check_cache(cache);
  if (r != USP_OK) return r;
  if (T < 0 || !valid_dtype(dtype)) return USP_ERR_INVALID_ARG;
  if (cache->B > 0 && T > 0 && (!k || !v)) return USP_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4)) return USP_ERR_ALIGNMENT;
  if (cache->B == 0 || T == 0) return USP_OK;
  return launch_kv8_read(view(cache), cache->D, start, T, k, v, dtype == USP_BF16,
                         reinterpret_cast<cudaStream_t>(stream));
}

size_t usp_attn_kv8_workspace_size(int B, int T, int max_new, int packed, int capacity, int Hq,
                                   int Hkv, int D) {
  if (B < 0 || B > 65535 || T < 1 || capacity < 0 || capacity > kMaxRows || Hq < 1 || Hkv < 1 ||
      Hkv > 65535 || Hq % Hkv != 0 || (D != 64 && D != 128))
    return 0;
  if (!packed || max_new < 1 || max_new > T) max_new = T;
  if (too_many_rows(B, max_new, Hq, Hkv)) return 0;
  return attn_kv8_workspace(B, max_new, capacity, Hq, Hkv, D);
}

usp_status_t usp_attn_kv8(const usp_kv8_cache_t* cache, const void* q, void* out, float* lse,
                          const int32_t* cu_seqlens, int T, int max_new, int Hq,
                          float softmax_scale, int causal, int window, int sink_tokens,
                          usp_dtype_t dtype, void* workspace, size_t workspace_bytes,
                          usp_stream_t stream) {
  usp_status_t r = check_cache(cache);
  if (r != USP_OK) return r;
  if (T < 1 || Hq < 1 || Hq % cache->Hkv != 0 || sink_tokens < 0) return USP_ERR_INVALID_ARG;
  if (dtype == USP_FP32) return USP_ERR_UNSUPPORTED;
  if (dtype != USP_BF16) return USP_ERR_INVALID_ARG;
  if (cu_seqlens && cache->B < 1) return USP_ERR_INVALID_ARG;
  if (cache->B > 0 && (!q || !out || !lse)) return USP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 16)) return USP_ERR_ALIGNMENT;
  if (!aligned(cu_seqlens, 4) || !aligned(workspace, 256)) return USP_ERR_ALIGNMENT;
  if (!cu_seqlens || max_new < 1 || max_new > T) max_new = T;
  if (T > kMaxRows || (!cu_seqlens && (long long)T * cache->B > 0x7fffffffLL) ||
      too_many_rows(cache->B, max_new, Hq, cache->Hkv))
    return USP_ERR_UNSUPPORTED;
  if (cache->B == 0) return USP_OK;
  const size_t need =
      attn_kv8_workspace(cache->B, max_new, (long long)cache->max_pages * cache->page_size, Hq,
                         cache->Hkv, cache->D);
  if (need > 0 && (!workspace || workspace_bytes < need)) return USP_ERR_WORKSPACE;
  AttnKv8Args a{};
  a.c = view(cache);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.cu = cu_seqlens;
  a.T = T;
  a.max_new = max_new;
  a.Hq = Hq;
  a.D = cache->D;
  a.scale = softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)cache->D);
  a.causal = causal ? 1 : 0;
  a.window = kv8::window_of(window);  // (the kernels subtract it from positions)
  a.sink = sink_tokens;
  return launch_attn_kv8(a, workspace, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
