// The paged 8-bit KV cache's number format and its arrays, and the rotation of
// positions, as the kernels see them.
//
// A code is an E4M3 number; a block of 32 tokens of a head has one exponent e
// (int8, [-40, 40]) and stands for code * 2^e. A power of two costs E4M3 nothing:
// while e is not clamped, the largest element of a block becomes a code of more than
// 224, and every element down to 2^-13 of it keeps 4 significant bits (codes below 2^-6
// are subnormal); a block whose exponent rises keeps its older values but for those that
// become subnormal. Codes are exact in fp16, and their products with 2^e in bf16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace usp {
namespace kv8 {

constexpr int kBlock = 32;  // tokens per exponent
constexpr int kExpMin = -40, kExpMax = 40;

struct Cache {
  uint8_t* kc;
  int8_t* ke;
  uint8_t* vc;
  int8_t* ve;
  const int* table;  // [B][mp] pages of the sequences
  int* lens;
  int B, mp, np, ps, H;  // sequences, pages of each, pages in all, page size, KV heads
  int cap;               // mp * ps
  int ps_log2;
};

__device__ __forceinline__ int clamp_len(int len, int C) { return min(max(len, 0), C); }

// Page that holds row `row` of sequence b, or -1 (an entry that names none).
__device__ __forceinline__ int page_of(const Cache& c, int b, int row) {
  const int p = __ldg(c.table + (long long)b * c.mp + (row >> c.ps_log2));
  return static_cast<unsigned>(p) < static_cast<unsigned>(c.np) ? p : -1;
}
// Rows before (page, head)'s first; times D for codes, / 32 for exponents.
__device__ __forceinline__ long long head_rows(const Cache& c, int page, int h) {
  return ((long long)page * c.H + h) << c.ps_log2;
}
__device__ __forceinline__ int clamp_exp(int e) { return min(max(e, kExpMin), kExpMax); }
__device__ __forceinline__ float exp2i(int e) {  // 2^e, e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// Smallest e >= kExpMin with amax <= 448 * 2^e, at most kExpMax (amax >= 0, no
// NaN). 448 = 1.75 * 2^8.
__device__ __forceinline__ int exponent_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return clamp_exp(e);
}

// Two E4M3 bytes (low byte first) as an fp16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two_bytes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(two_bytes)));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two_bytes) {
  const uint32_t h = e4m3x2_to_h2(two_bytes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // (aligned: the warp is together)
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// ------------------------------------------------------------------ rotation
struct Rope {
  const float* table;  // [rows][R]: cos of R/2 frequencies, sin of them; or nullptr
  int rows, R;
  int inter;           // pairs (2i, 2i+1) instead of (i, i + R/2)
};

// A row's D channels are D / (2 V) items of two vectors of V channels: the two
// sides of V pairs, or (channels R and up) two vectors that stay as they are.
template <int V>
struct Item {
  int a, b;   // first channels of the two vectors
  int f;      // first frequency, < 0: not rotated
};
template <int V>
__device__ __forceinline__ Item<V> item_of(const Rope& r, int j) {
  if (!r.table || 2 * V * j >= r.R) return {2 * V * j, 2 * V * j + V, -1};
  if (r.inter) return {2 * V * j, 2 * V * j + V, V * j};
  return {V * j, r.R / 2 + V * j, V * j};
}
// cos and sin of the item's V frequencies at a position.
template <int V>
__device__ __forceinline__ void load_turn(const Rope& r, const Item<V>& it, int pos,
                                          float (&c)[V], float (&s)[V]) {
  if (it.f < 0) return;
  const float* t = r.table + (long long)min(max(pos, 0), r.rows - 1) * r.R + it.f;
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(t + i));
    const float4 y = __ldg(reinterpret_cast<const float4*>(t + r.R / 2 + i));
    c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
    s[i] = y.x; s[i + 1] = y.y; s[i + 2] = y.z; s[i + 3] = y.w;
  }
}
// The definition's arithmetic: both products and their sum rounded to fp32 (no
// fused multiply-add, so that every build gives the same bits).
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}
template <int V>
__device__ __forceinline__ void rotate(const Item<V>& it, bool inter, const float (&c)[V],
                                       const float (&s)[V], float (&a)[V], float (&b)[V]) {
  if (it.f < 0) return;
  if (inter) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) turn(a[2 * i], a[2 * i + 1], c[i], s[i]);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) turn(b[2 * i], b[2 * i + 1], c[V / 2 + i], s[V / 2 + i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) turn(a[i], b[i], c[i], s[i]);
  }
}

// 16 bytes of bf16 or fp32 as floats, and back (rounded to nearest even).
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);
__device__ __forceinline__ void unpack(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& r, float (&x)[4]) {
  x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
  x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}

}  // namespace kv8
}  // namespace usp
