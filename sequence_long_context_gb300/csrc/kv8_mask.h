// Which keys a query of the attention to the paged 8-bit cache sees, 32 at a time. Plain
// C++ too, so that a test can go over it on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define USP_KV8_FN __host__ __device__ __forceinline__
#else
#define USP_KV8_FN inline
#endif

namespace usp {
namespace kv8 {

// Rows of a sequence, and tokens of a call: positions lie between -kMaxRows and
// kMaxRows, so that a sum or difference of two of them has room in 32 bits.
constexpr int kMaxRows = 1 << 30;

// A window as the kernels take it: 0 none, and no more than there can be rows.
USP_KV8_FN int window_of(int window) {
  return window <= 0 ? 0 : window < kMaxRows ? window : kMaxRows;
}

// The query at position i of len keys: keys lo .. hi and 0 .. sink_hi (a window of
// window_of alone). i < 0: none.
struct RowKeys {
  int lo, hi, sink_hi;
};
USP_KV8_FN RowKeys row_keys(int i, int len, int causal, int window, int sink) {
  RowKeys r;
  r.hi = i < 0 ? -1 : causal && i < len - 1 ? i : len - 1;
  r.lo = window > 0 && i >= window ? i - window + 1 : 0;
  r.sink_hi = window <= 0 ? -1 : sink - 1 < r.hi ? sink - 1 : r.hi;
  return r;
}

// Columns [lo, hi] (relative to a block's first key) as bits.
USP_KV8_FN uint32_t col_bits(int lo, int hi) {
  if (hi < 0 || lo > 31 || hi < lo) return 0;
  const uint32_t a = lo <= 0 ? ~0u : ~0u << lo;
  return hi >= 31 ? a : a & ((2u << hi) - 1);
}
// The keys [k, k + 32) that are seen.
USP_KV8_FN uint32_t key_bits(const RowKeys& r, int k) {
  return col_bits(r.lo - k, r.hi - k) | col_bits(-k, r.sink_hi - k);
}

}  // namespace kv8
}  // namespace usp
