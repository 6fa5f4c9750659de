// Filling the 4-bit KV cache and reading it back.
//
// Both are copies with a few operations per element: bound by HBM for prompts
// and by launch latency for single tokens.
//
// Append. A warp takes one tensor (K or V) of one KV head and eight tokens
// that follow one another, so its writes are contiguous rows of the head. A
// lane holds eight channels (16 bytes of bf16), four lanes a block of 32: the
// block's maximum takes two shuffles, and the codes of eight channels are one
// word. The quotients are true divisions: max|y| / 7 rounds to a tie of E4M3,
// and y / s to a tie of the integers, only where the exact quotient is one
// (numerators have at most 24 significant bits, the ties times the divisor at
// most 8), so the codes are those of the definition whatever the inputs.
//
// Read. A lane decodes eight channels of one row and writes them as 16 (bf16)
// or 32 (fp32) bytes; the lanes run over the output in its own order.
#include "internal.h"
#include "kv4.cuh"
#include "kv4_host.h"
#include "tc_ptx.cuh"

namespace usp {
namespace {

using namespace kv4;

constexpr int kGroup = 8;          // tokens per warp of the append
constexpr int kAppendThreads = 256;

struct AppendParams {
  Cache c;
  const void* k;
  const void* v;
  const float* new_w;
  const int* cu;
  int* lens_out;
  int T;           // tokens per sequence; packed: in all
  float k_inv, v_inv;
};

template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* src, float (&x)[8]) {
  const uint4 r = __ldg(reinterpret_cast<const uint4*>(src));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* src, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(src));
  const float4 b = __ldg(reinterpret_cast<const float4*>(src) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// New tokens of sequence b, given its boundaries (packed) or T.
__device__ __forceinline__ int new_tokens(const AppendParams& P, int b) {
  return P.cu ? max(0, __ldg(P.cu + b + 1) - __ldg(P.cu + b)) : P.T;
}

// One warp's item: tensor `which` (0: K, 1: V), KV head h, tokens
// [tok0, tok0 + kGroup) of the input's rows (all sequences in a row), those
// below `end`. seq: the sequence they belong to, or -1: look each one up.
template <typename T, int D>
__device__ __forceinline__ void append_item(const AppendParams& P, int which, int h,
                                            long long tok0, long long end, int seq) {
  constexpr int kLanes = D / 8;          // lanes per row
  constexpr int kRows = 32 / kLanes;     // rows per pass
  const int lane = threadIdx.x & 31;
  const int lr = lane / kLanes, lc = lane % kLanes;
  const T* src = static_cast<const T*>(which ? P.v : P.k);
  uint8_t* codes = which ? P.c.vc : P.c.kc;
  uint8_t* scales = which ? P.c.vs : P.c.ks;
  const float inv = which ? P.v_inv : P.k_inv;
  float x[kGroup / kRows][8];
#pragma unroll
  for (int i = 0; i < kGroup / kRows; ++i) {
    const long long tok = tok0 + i * kRows + lr;
    if (tok < end) load8<T>(src + (tok * P.c.H + h) * D + lc * 8, x[i]);
  }
#pragma unroll
  for (int i = 0; i < kGroup / kRows; ++i) {
    const long long tok = tok0 + i * kRows + lr;
    const bool in = tok < end;
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float y = in ? x[i][e] * inv : 0.f;
      if (isnan(y)) y = 0.f;
      x[i][e] = y;
      amax = fmaxf(amax, fabsf(y));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t sbyte = tc::pack_e4m3(__fdiv_rn(amax, 7.f), 0.f) & 0xffu;
    const float s = e4m3_to_float(sbyte);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float c = s > 0.f ? rintf(__fdiv_rn(x[i][e], s)) : 0.f;
      c = fminf(fmaxf(c, -7.f), 7.f);
      word |= static_cast<uint32_t>(static_cast<int>(c) + 8) << (4 * e);
    }
    if (!in) continue;
    int b = seq;
    long long t;
    if (P.cu) {
      if (b < 0) b = seg_of(P.cu, P.c.B, (int)tok);
      t = tok - __ldg(P.cu + b);
    } else {
      if (b < 0) b = (int)(tok / P.T);
      t = tok - (long long)b * P.T;
    }
    const long long pos = clamp_len(P.c.lens[b], P.c.C) + t;
    if (t < 0 || pos >= P.c.C) continue;  // no room (or malformed boundaries)
    const long long row = head_row(P.c, b, h) + pos;
    *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + lc * 4) = word;
    if ((lc & 3) == 0) scales[row * (D / kBlock) + (lc >> 2)] = (uint8_t)sbyte;
    if (which == 0 && lc == 0 && P.c.w != nullptr) {
      float w = 0.f;
      if (P.new_w)
        w = P.cu ? P.new_w[(long long)h * P.T + tok]
                 : P.new_w[((long long)b * P.c.H + h) * P.T + t];
      P.c.w[row] = w;
    }
  }
}

// One block per sequence, which also writes the sequence's new length.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) append_seq_kernel(const AppendParams P) {
  const int b = blockIdx.x;
  const long long first = (long long)b * P.T;
  const int groups = (P.T + kGroup - 1) / kGroup;
  for (int it = threadIdx.x >> 5; it < 2 * P.c.H * groups; it += kAppendThreads / 32) {
    const int which = it & 1, h = (it >> 1) % P.c.H, g = (it >> 1) / P.c.H;
    append_item<T, D>(P, which, h, first + (long long)g * kGroup, first + P.T, b);
  }
  __syncthreads();  // every warp has read the old length
  if (threadIdx.x == 0 && P.lens_out)
    P.lens_out[b] = (int)min((long long)P.c.C, (long long)clamp_len(P.c.lens[b], P.c.C) + P.T);
}

// Warps over (group of tokens, head, tensor); the lengths are written by a
// launch of their own behind this one.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads)
append_kernel(const AppendParams P, long long tokens, long long items) {
  const long long it = (long long)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  if (it >= items) return;
  const int which = (int)(it & 1), h = (int)((it >> 1) % P.c.H);
  const long long g = (it >> 1) / P.c.H;
  append_item<T, D>(P, which, h, g * kGroup, min(tokens, (g + 1) * kGroup), -1);
}

__global__ void append_lens_kernel(const AppendParams P) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < P.c.B)
    P.lens_out[b] =
        (int)min((long long)P.c.C, (long long)clamp_len(P.c.lens[b], P.c.C) + new_tokens(P, b));
}

template <typename T, int D>
usp_status_t launch_append_t(const AppendParams& P, cudaStream_t st) {
  const long long tokens = P.cu ? P.T : (long long)P.c.B * P.T;
  const long long groups = (tokens + kGroup - 1) / kGroup;
  // Few tokens per sequence: one launch, whose blocks own their sequences'
  // lengths. Else the items are spread over the whole GPU and a second,
  // one-block launch (about 2 us) updates the lengths in stream order.
  if (!P.cu && (long long)P.T * P.c.H <= 64) {
    {
      ProfScope ps(st, "kv4_append");
      append_seq_kernel<T, D><<<P.c.B, kAppendThreads, 0, st>>>(P);
    }
    note_launch();
    return check_launch();
  }
  const long long items = groups * P.c.H * 2;
  const long long blocks = (items + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  if (blocks > 0x7fffffffLL) return USP_ERR_UNSUPPORTED;
  if (blocks > 0) {
    {
      ProfScope ps(st, "kv4_append");
      append_kernel<T, D><<<(unsigned)blocks, kAppendThreads, 0, st>>>(P, tokens, items);
    }
    note_launch();
    usp_status_t r = check_launch();
    if (r != USP_OK) return r;
  }
  if (P.lens_out == nullptr) return USP_OK;
  {
    ProfScope ps(st, "kv4_append_lens");
    append_lens_kernel<<<(P.c.B + 255) / 256, 256, 0, st>>>(P);
  }
  note_launch();
  return check_launch();
}

struct ReadParams {
  Cache c;
  const int* start;
  void* k;
  void* v;
  int T;
  float k_descale, v_descale;
};

template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* dst, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(dst) = make_uint4(tc::pack_bf16(x[0], x[1]), tc::pack_bf16(x[2], x[3]),
                                              tc::pack_bf16(x[4], x[5]), tc::pack_bf16(x[6], x[7]));
}
template <>
__device__ __forceinline__ void store8<float>(float* dst, const float (&x)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// grid (chunks of the sequence's T * H * D/8 outputs, tensor, sequence)
template <typename T, int D>
__global__ void __launch_bounds__(256) read_kernel(const ReadParams P) {
  const int b = blockIdx.z, which = blockIdx.y;
  const long long n8 = (long long)P.T * P.c.H * (D / 8);
  const uint8_t* codes = which ? P.c.vc : P.c.kc;
  const uint8_t* scales = which ? P.c.vs : P.c.ks;
  T* out = static_cast<T*>(which ? P.v : P.k) + (long long)b * n8 * 8;
  const float descale = which ? P.v_descale : P.k_descale;
  const int len = clamp_len(__ldg(P.c.lens + b), P.c.C);
  const long long start = P.start ? __ldg(P.start + b) : 0;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n8; i += (long long)gridDim.x * 256) {
    const int lc = (int)(i % (D / 8));
    const long long th = i / (D / 8);
    const int h = (int)(th % P.c.H);
    const long long pos = start + th / P.c.H;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (pos >= 0 && pos < len) {
      const long long row = head_row(P.c, b, h) + pos;
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + row * (D / 2)) + lc);
      const float s = e4m3_to_float(__ldg(scales + row * (D / kBlock) + (lc >> 2)));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = (static_cast<float>(static_cast<int>((w >> (4 * e)) & 15u) - 8) * s) * descale;
    }
    store8<T>(out + i * 8, x);
  }
}

template <typename T, int D>
usp_status_t launch_read_t(const ReadParams& P, cudaStream_t st) {
  const long long n8 = (long long)P.T * P.c.H * (D / 8);
  long long blocks = (n8 + 255) / 256;
  if (blocks > 152 * 16) blocks = 152 * 16;
  {
    ProfScope ps(st, "kv4_read");
    read_kernel<T, D><<<dim3((unsigned)blocks, 2, P.c.B), 256, 0, st>>>(P);
  }
  note_launch();
  return check_launch();
}

}  // namespace

usp_status_t launch_kv4_append(const Cache& c, int D, const void* k, const void* v,
                               const float* new_w, const int* cu, int T, int bf16, float k_inv,
                               float v_inv, int* lens_out, cudaStream_t st) {
  AppendParams P{c, k, v, new_w, cu, lens_out, T, k_inv, v_inv};
  if (bf16)
    return D == 128 ? launch_append_t<__nv_bfloat16, 128>(P, st)
                    : launch_append_t<__nv_bfloat16, 64>(P, st);
  return D == 128 ? launch_append_t<float, 128>(P, st) : launch_append_t<float, 64>(P, st);
}

usp_status_t launch_kv4_read(const Cache& c, int D, const int* start, int T, void* k, void* v,
                             int bf16, float k_descale, float v_descale, cudaStream_t st) {
  ReadParams P{c, start, k, v, T, k_descale, v_descale};
  if (bf16)
    return D == 128 ? launch_read_t<__nv_bfloat16, 128>(P, st)
                    : launch_read_t<__nv_bfloat16, 64>(P, st);
  return D == 128 ? launch_read_t<float, 128>(P, st) : launch_read_t<float, 64>(P, st);
}

}  // namespace usp
