// The 4-bit KV cache's number format and its arrays, as the kernels see them.
//
// A block of 32 channels is stored as 32 nibbles u = c + 8 (c in [-7, 7]) and
// one E4M3 scale s; it stands for c * s * descale. |c| has 3 significant bits
// and s has 4, so c * s has at most 7: exact in bf16 (8) and in fp16 (11, and
// e4m3's range of 2^-9 .. 448 times 7 is inside fp16's). The kernels decode
// to c * s without any rounding and apply descale in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace usp {
namespace kv4 {

constexpr int kBlock = 32;     // channels per scale
constexpr int kRowAlign = 16;  // capacities are multiples of this

struct Cache {
  uint8_t* kc;
  uint8_t* ks;
  uint8_t* vc;
  uint8_t* vs;
  float* w;      // key weights or nullptr
  int* lens;
  int B, C, H;
};

// Rows before (b, h)'s first: rows of D/2 codes, D/32 scales, one weight.
__host__ __device__ __forceinline__ long long head_row(const Cache& c, int b, int h) {
  return ((long long)b * c.H + h) * c.C;
}

__device__ __forceinline__ int clamp_len(int len, int C) { return min(max(len, 0), C); }

// Two E4M3 bytes (low byte first) as an fp16 pair, exactly.
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t two_bytes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(two_bytes)));
  return *reinterpret_cast<__half2*>(&r);
}
__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  return __low2float(e4m3x2_to_half2(byte & 0xffu));
}

}  // namespace kv4
}  // namespace usp
