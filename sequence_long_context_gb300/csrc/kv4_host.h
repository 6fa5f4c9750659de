// Host-side declarations of the 4-bit KV cache's launchers.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "../../include/usp.h"
#include "kv4.cuh"

namespace usp {

// A kernel's limit of dynamic shared memory, set once per device (the call
// takes about a microsecond).
struct SmemAttr {
  std::atomic<unsigned long long> done{0};
  template <typename K>
  cudaError_t set(K kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
};

// kv4_cache.cu
usp_status_t launch_kv4_append(const kv4::Cache& c, int D, const void* k, const void* v,
                               const float* new_w, const int* cu, int T, int bf16, float k_inv,
                               float v_inv, int* lens_out, cudaStream_t st);
usp_status_t launch_kv4_read(const kv4::Cache& c, int D, const int* start, int T, void* k, void* v,
                             int bf16, float k_descale, float v_descale, cudaStream_t st);

// kv4_evict.cu
usp_status_t launch_kv4_evict(const kv4::Cache& src, const kv4::Cache& dst, int D, int* kept,
                              int keep, int recent, int sink, cudaStream_t st);

// decode_kv4.cu
struct DecodeKv4Args {
  kv4::Cache c;
  const void* q;
  void* out;
  float* lse;
  int Tq, Hq, D;
  float scale, k_descale, v_descale;
  int causal, window, sink, accumulate;
};
// Bytes of the workspace (0 never: the partials are always needed), and the
// launch that carves them from it.
size_t decode_kv4_workspace(int B, int Tq, int C, int Hq, int Hkv, int D, int accumulate);
usp_status_t launch_decode_kv4(const DecodeKv4Args& a, void* workspace, cudaStream_t st);
int read_clear_decode_kv4_status();  // -1 on a CUDA error

}  // namespace usp
