// Host-side declarations of the 4-bit KV cache's launchers.
#pragma once

#include <cuda_runtime.h>

#include "../../include/usp.h"
#include "kv4.cuh"

namespace usp {

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
