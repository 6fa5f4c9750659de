// Filling the 4-bit KV cache and reading it back.
//
// Both are copies with a few operations per element. 32K tokens of 8 heads of 128,
// bf16 (170 MB): the append takes 44 us, 3.9 TB/s, bound by instruction issue
// (87 % of all slots, about 20 instructions per channel); the read 29 us, 5.8
// TB/s. Single tokens are bound by launch latency (3.9 us). An append with a
// descale of 1 leaves out the multiplications by 1 (44 us instead of 51), and a
// read in bf16 with powers of two makes two values per packed multiply-add, exactly
// (29 instead of 34); every bit is the same either way.
//
// A warp takes one tensor (K or V) of one KV head and eight tokens that follow
// one another, so that its side of the cache is one contiguous run. A lane
// holds eight channels of a row: 16 bytes of bf16, one word of codes; four
// lanes share a block of 32, whose maximum takes two shuffles.
//
// The codes are those of the definition for every input, although no true
// division is made. For a quotient y / s, with r within an ulp or two of 1 / s,
//     t = y r,   e = y - t s,   t' = t + e r
// leaves t' = y / s (1 + 2^-43) before its one rounding (t s has 28 bits and e
// cancels to a few, so e is exact). t' then rounds to an integer, and ties are
// what matters. Exact tie y = (h + 1/2) s: t' is h + 1/2, exactly. Not a tie:
// y is at least one ulp(y) from (h + 1/2) s, and ulp(y) / s exceeds half an ulp
// of h + 1/2 by the factor 2 / sigma >= 16/15, sigma <= 15/8 the significand
// of s (4 bits), so t' does not round onto the tie. The same holds for
// max|y| / 7 against E4M3's ties (sigma = 7/4).
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "kv4.cuh"
#include "kv4_host.h"
#include "tc_ptx.cuh"

namespace usp {
namespace {

using namespace kv4;

constexpr int kGroup = 8;  // tokens per warp
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// a / d for the roundings above (finite a); r: about 1 / d.
__device__ __forceinline__ float quotient(float a, float d, float r) {
  const float t = a * r;
  return fmaf(fmaf(-t, d, a), r, t);
}

// Eight channels of a row as loaded, their largest magnitude (not a NaN's;
// `odd`: there may be one), and as floats.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float amax(bool& odd) const {
    // magnitudes as 16-bit integers, which order like the numbers; a NaN's is
    // above infinity's
    const uint32_t m = 0x7fff7fffu;
    const uint32_t x = __vmaxu2(__vmaxu2(r.x & m, r.y & m), __vmaxu2(r.z & m, r.w & m));
    const uint32_t y = max(x >> 16, x & 0xffffu);
    odd = y > 0x7f80u;
    return __uint_as_float(y << 16);
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float amax(bool& odd) const {
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    odd = m > 0x7f800000u;
    return __uint_as_float(m);
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

// The codes' word and the block's scale byte of a lane's eight channels.
// kOne: the descale, and so inv, is 1.
template <typename T, bool kOne>
__device__ __forceinline__ uint32_t encode(const Raw<T>& raw, float inv, uint32_t& sbyte) {
  bool odd;
  // rounding is monotonic, so the largest |x| gives the largest |x inv|
  float amax = raw.amax(odd);
  float y[8];
  raw.floats(y);
  if constexpr (!kOne) {
    amax *= inv;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= inv;
  }
  if (odd) {  // a NaN counts as 0
    amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (isnan(y[e])) y[e] = 0.f;
      amax = fmaxf(amax, fabsf(y[e]));
    }
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  amax = fminf(amax, 1e38f);  // infinite: saturates like this
  sbyte = tc::pack_e4m3(quotient(amax, 7.f, 1.f / 7.f), 0.f) & 0xffu;
  const float s = e4m3_to_float(sbyte);
  // The sum with 1.5 2^23 + 8 rounds to an integer, half to even, and leaves
  // c + 8 in the low bits of 0x4B400000; the constants, shifted like the codes,
  // are taken off the word at the end (modulo 2^32).
  constexpr float kMagic = 12582912.f + 8.f;
  constexpr uint32_t kBits = 0x4B400000u * 0x11111111u;
  uint32_t word = 0u - kBits;
  if (sbyte >= 8u && sbyte < 0x7Eu) {
    // a normal scale is within 2^-4 of max / 7: |y / s| < 7.5, no clamp
    const float r = rcp_approx(s);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      word += __float_as_uint(quotient(y[e], s, r) + kMagic) << (4 * e);
  } else {
    const float r = s > 0.f ? rcp_approx(s) : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // far outside (or infinite): no remainder needed
      const float t = fminf(fmaxf(y[e] * r, -8.f), 8.f);
      const float q = fabsf(t) == 8.f ? t : fmaf(fmaf(-t, s, y[e]), r, t);
      word += __float_as_uint(fminf(fmaxf(q, -7.f), 7.f) + kMagic) << (4 * e);
    }
  }
  return word;
}

// One warp's item: tensor `which` (0: K, 1: V), KV head h, tokens [t0, t0 +
// kGroup) below P.T of sequence b (b < 0: of the packed batch, each token's
// sequence is looked up).
template <typename T, int D, bool kOne>
__device__ __forceinline__ void append_item(const AppendParams& P, int which, int h, int b, int t0) {
  constexpr int kLanes = D / 8;          // lanes per row
  constexpr int kRows = 32 / kLanes;     // rows per pass
  constexpr int kPasses = kGroup / kRows;
  const int lane = threadIdx.x & 31;
  const int lr = lane / kLanes, lc = lane % kLanes;
  const float inv = which ? P.v_inv : P.k_inv;
  const int n = P.T - t0 - lr;           // rows i kRows < n are there
  const long long hd = (long long)P.c.H * D;  // between tokens
  const T* src = static_cast<const T*>(which ? P.v : P.k) +
                 ((b < 0 ? 0 : (long long)b * P.T) + t0 + lr) * hd + h * D + lc * 8;
  Raw<T> raw[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    if (i * kRows < n) raw[i].load(src + i * kRows * hd);
    else raw[i].zero();
  }
  // the lane's first row in the cache, if all are of one sequence
  int pos0 = 0;
  long long row0 = 0;
  if (b >= 0) {
    pos0 = clamp_len(P.c.lens[b], P.c.C);
    row0 = head_row(P.c, b, h);
  }
  uint8_t* codes = which ? P.c.vc : P.c.kc;
  uint8_t* scales = which ? P.c.vs : P.c.ks;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    uint32_t sbyte;
    const uint32_t word = encode<T, kOne>(raw[i], inv, sbyte);
    if (i * kRows >= n) continue;
    const int tok = t0 + lr + i * kRows;
    int bb = b, t = tok;
    if (b < 0) {
      bb = seg_of(P.cu, P.c.B, tok);
      t = tok - __ldg(P.cu + bb);
      if (tok >= __ldg(P.cu + bb + 1)) continue;  // behind the last boundary
      pos0 = clamp_len(P.c.lens[bb], P.c.C);
      row0 = head_row(P.c, bb, h);
    }
    if (t < 0 || t >= P.c.C - pos0) continue;  // no room (or malformed boundaries)
    const long long row = row0 + pos0 + t;
    *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + lc * 4) = word;
    if ((lc & 3) == 0) scales[row * (D / kBlock) + (lc >> 2)] = (uint8_t)sbyte;
    if (which == 0 && lc == 0 && P.c.w != nullptr) {
      float w = 0.f;
      if (P.new_w)
        w = P.cu ? P.new_w[(long long)h * P.T + tok]
                 : P.new_w[((long long)bb * P.c.H + h) * P.T + t];
      P.c.w[row] = w;
    }
  }
}

// One block per sequence, which also writes the sequence's new length.
template <typename T, int D, bool kOne>
__global__ void __launch_bounds__(kThreads) append_seq_kernel(const AppendParams P) {
  const int b = blockIdx.x;
  const int groups = (P.T + kGroup - 1) / kGroup;
  for (int it = threadIdx.x >> 5; it < 2 * P.c.H * groups; it += kWarps) {
    const int g = it / (2 * P.c.H), x = it - g * 2 * P.c.H;
    append_item<T, D, kOne>(P, x & 1, x >> 1, b, g * kGroup);
  }
  __syncthreads();  // every warp has read the old length
  if (threadIdx.x == 0 && P.lens_out)
    P.lens_out[b] = (int)min((long long)P.c.C, (long long)clamp_len(P.c.lens[b], P.c.C) + P.T);
}

// grid (items, sequences; packed: 1): warps over (group of tokens, head,
// tensor). The lengths are written by a launch of their own behind this one.
template <typename T, int D, bool kOne>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams P, unsigned items) {
  const unsigned it = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (it >= items) return;
  const unsigned g = it / (2 * P.c.H), x = it - g * 2 * P.c.H;
  append_item<T, D, kOne>(P, x & 1, x >> 1, P.cu ? -1 : (int)blockIdx.y, (int)(g * kGroup));
}

__global__ void append_lens_kernel(const AppendParams P) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= P.c.B) return;
  const long long n = P.cu ? max(0, __ldg(P.cu + b + 1) - __ldg(P.cu + b)) : P.T;
  P.lens_out[b] = (int)min((long long)P.c.C, clamp_len(P.c.lens[b], P.c.C) + n);
}

// Items of one sequence's (packed: the batch's) T tokens, 0 if too many.
long long items_of(int T, int H) {
  const long long n = ((long long)T + kGroup - 1) / kGroup * H * 2;
  return n / kWarps < 0x7fffffffLL - 1 && n < 0xffffffffLL ? n : -1;
}

template <typename T, int D, bool kOne>
usp_status_t launch_append_t(const AppendParams& P, cudaStream_t st) {
  // Few tokens per sequence: one launch, whose blocks own their sequences'
  // lengths. Else the items are spread over the whole GPU and a second, small
  // launch updates the lengths in stream order. On the GPU both take 3.5 to 3.9
  // us up to 8 tokens of 8 heads, and one launch saves its caller about 2 us; for
  // 16 tokens one takes 6.1 us and two 3.9, for 32 10.9 and 3.8.
  if (!P.cu && (long long)P.T * P.c.H <= 64) {
    {
      ProfScope ps(st, "kv4_append");
      append_seq_kernel<T, D, kOne><<<P.c.B, kThreads, 0, st>>>(P);
    }
    note_launch();
    return check_launch();
  }
  const long long items = items_of(P.T, P.c.H);
  if (items < 0) return USP_ERR_UNSUPPORTED;
  if (items > 0) {
    const dim3 grid((unsigned)((items + kWarps - 1) / kWarps), P.cu ? 1 : P.c.B);
    {
      ProfScope ps(st, "kv4_append");
      append_kernel<T, D, kOne><<<grid, kThreads, 0, st>>>(P, (unsigned)items);
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

// The eight values c s descale of a word of codes (nibble e: channel e), as
// they are written. kExact: bf16, and c s descale is exact in bf16 (a descale
// that is a power of two): the nibbles go into the mantissa of 16 and one
// packed FMA by (s, -24 s), s being scaled already, gives two values.
template <typename T, bool kExact>
__device__ __forceinline__ void store_values(T* dst, uint32_t w, uint32_t sbyte, float descale) {
  const float s = e4m3_to_float(sbyte);
  if constexpr (kExact) {
    const float sd = s * descale;
    const uint32_t s2 = tc::pack_bf16(sd, sd), z2 = tc::pack_bf16(-24.f * sd, -24.f * sd);
    uint32_t v[4];  // nibbles j and j + 4
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = j == 0 ? w << 3 : j == 1 ? w >> 1 : j == 2 ? w >> 5 : w >> 9;
      const uint32_t u = (x & 0x00780078u) | 0x41804180u;
      asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[j]) : "r"(u), "r"(s2), "r"(z2));
    }
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                   __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
  } else {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      y[e] = (static_cast<float>(static_cast<int>((w >> (4 * e)) & 15u) - 8) * s) * descale;
    store8<T>(dst, y);
  }
}

// grid (items, sequences), as the append
template <typename T, int D, bool kExact>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams P, unsigned items) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kPasses = kGroup / kRows;
  const unsigned it = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (it >= items) return;
  const unsigned g = it / (2 * P.c.H), x = it - g * 2 * P.c.H;
  const int b = blockIdx.y, which = x & 1, h = x >> 1;
  const int lane = threadIdx.x & 31, lr = lane / kLanes, lc = lane % kLanes;
  const float descale = which ? P.v_descale : P.k_descale;
  const int len = clamp_len(__ldg(P.c.lens + b), P.c.C);
  const int t0 = (int)(g * kGroup) + lr;
  const long long p0 = (P.start ? (long long)__ldg(P.start + b) : 0) + t0;
  const long long row = head_row(P.c, b, h) + p0;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(which ? P.c.vc : P.c.kc) +
                          row * (D / 8) + lc;
  const uint8_t* scales = (which ? P.c.vs : P.c.ks) + row * (D / kBlock) + (lc >> 2);
  uint32_t w[kPasses], sb[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const long long pos = p0 + i * kRows;
    w[i] = 0x88888888u;  // zeros
    sb[i] = 0;
    if (pos >= 0 && pos < len) {
      w[i] = __ldg(codes + i * kRows * (D / 8));
      sb[i] = __ldg(scales + i * kRows * (D / kBlock));
    }
  }
  const long long hd = (long long)P.c.H * D;
  T* out = static_cast<T*>(which ? P.v : P.k) + ((long long)b * P.T + t0) * hd + h * D + lc * 8;
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    if (i * kRows < P.T - t0) store_values<T, kExact>(out + i * kRows * hd, w[i], sb[i], descale);
}

template <typename T, int D, bool kExact>
usp_status_t launch_read_t(const ReadParams& P, cudaStream_t st) {
  const long long items = items_of(P.T, P.c.H);
  if (items < 0) return USP_ERR_UNSUPPORTED;
  {
    ProfScope ps(st, "kv4_read");
    read_kernel<T, D, kExact>
        <<<dim3((unsigned)((items + kWarps - 1) / kWarps), P.c.B), kThreads, 0, st>>>(
            P, (unsigned)items);
  }
  note_launch();
  return check_launch();
}

// a power of two that keeps every c s descale a normal bf16
bool exact_descale(float x) {
  int e;
  return std::frexp(x, &e) == 0.5f && e > -64 && e < 64;
}

}  // namespace

usp_status_t launch_kv4_append(const Cache& c, int D, const void* k, const void* v,
                               const float* new_w, const int* cu, int T, int bf16, float k_inv,
                               float v_inv, int* lens_out, cudaStream_t st) {
  AppendParams P{c, k, v, new_w, cu, lens_out, T, k_inv, v_inv};
  const bool one = k_inv == 1.f && v_inv == 1.f;
  auto go = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    if (bf16)
      return one ? launch_append_t<__nv_bfloat16, kD, true>(P, st)
                 : launch_append_t<__nv_bfloat16, kD, false>(P, st);
    return one ? launch_append_t<float, kD, true>(P, st) : launch_append_t<float, kD, false>(P, st);
  };
  return D == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
}

usp_status_t launch_kv4_read(const Cache& c, int D, const int* start, int T, void* k, void* v,
                             int bf16, float k_descale, float v_descale, cudaStream_t st) {
  ReadParams P{c, start, k, v, T, k_descale, v_descale};
  const bool exact = exact_descale(k_descale) && exact_descale(v_descale);
  auto go = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    if (!bf16) return launch_read_t<float, kD, false>(P, st);
    return exact ? launch_read_t<__nv_bfloat16, kD, true>(P, st)
                 : launch_read_t<__nv_bfloat16, kD, false>(P, st);
  };
  return D == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
}

}  // namespace usp
