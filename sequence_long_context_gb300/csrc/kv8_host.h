// Host-side declarations of the paged 8-bit KV cache's launchers.
#pragma once

#include <cuda_runtime.h>

#include "../../include/usp.h"
#include "kv8.cuh"

namespace usp {

// rope.cu
usp_status_t launch_rope(const void* x, void* y, const kv8::Rope& r, int inverse, int B, int S,
                         int H, int D, const int* cu, int nseq, int cp, int layout, int bf16,
                         cudaStream_t st);

// kv8_cache.cu
struct Kv8AppendArgs {
  kv8::Cache c;
  kv8::Rope rope;
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  const int* positions;
  const int* cu;
  int* lens_out;
  int T, Hq, D, bf16;
};
usp_status_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t st);
usp_status_t launch_kv8_read(const kv8::Cache& c, int D, const int* start, int T, void* k, void* v,
                             int bf16, cudaStream_t st);

// attn_kv8.cu
struct AttnKv8Args {
  kv8::Cache c;
  const void* q;
  void* out;
  float* lse;
  const int* cu;
  int T, max_new;  // tokens of a sequence (packed: in all); most of a sequence
  int Hq, D;
  float scale;
  int causal, window, sink;
};
size_t attn_kv8_workspace(int B, int max_new, long long cap, int Hq, int Hkv, int D);
usp_status_t launch_attn_kv8(const AttnKv8Args& a, void* workspace, cudaStream_t st);
int read_clear_attn_kv8_status();  // -1 on a CUDA error

// attn_kv8_tc.cu (many query rows per KV head), from launch_attn_kv8
size_t attn_kv8_tc_workspace(int D);
usp_status_t launch_attn_kv8_tc(const AttnKv8Args& a, void* workspace, cudaStream_t st);
int read_clear_attn_kv8_tc_status();  // -1 on a CUDA error

}  // namespace usp
