// Eviction from the 4-bit KV cache by accumulated attention weight.
//
// Select: one block per (sequence, KV head) finds the rank-th largest weight
// of the keys between the sinks and the recent ones by four 8-bit radix
// passes over order-preserving 32-bit keys, then writes the kept rows'
// indices in ascending order. Move: the kept rows are copied to their places.
#include "internal.h"
#include "kv4.cuh"
#include "kv4_host.h"

namespace usp {
namespace {

using namespace kv4;

constexpr int kThreads = 1024;

// Larger float <=> larger key; +0 and -0 alike; a NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (isnan(x)) return 0xffffffffu;
  if (x == 0.f) return 0x80000000u;
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictParams {
  Cache src, dst;
  int* kept;
  int keep, recent, sink;
};

__global__ void __launch_bounds__(kThreads) select_kernel(const EvictParams P) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_need;
  __shared__ uint32_t warp_tie[32], warp_keep[32];
  const int h = blockIdx.x, b = blockIdx.y;
  const int L = clamp_len(P.src.lens[b], P.src.C);
  int* kept = P.kept + ((long long)b * P.src.H + h) * P.keep;
  if (L <= P.keep) {
    for (int i = threadIdx.x; i < P.keep; i += kThreads) kept[i] = i < L ? i : -1;
    return;
  }
  const float* w = P.src.w + head_row(P.src, b, h);
  const int lo = P.sink, hi = L - P.recent;  // candidates [lo, hi)
  uint32_t need = (uint32_t)(P.keep - P.sink - P.recent);
  uint32_t prefix = 0;  // the threshold's bits found so far
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int j = lo + threadIdx.x; j < hi; j += kThreads) {
        const uint32_t key = order_key(w[j]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t left = need;
        int bin = 255;
        while (bin > 0 && hist[bin] < left) left -= hist[bin--];
        s_prefix = prefix | ((uint32_t)bin << shift);
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
  }
  // keys above `prefix` are kept, and the first `need` equal to it
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool any = P.keep - P.sink - P.recent > 0;
  uint32_t ties = 0, out = 0;  // so far, the same in every thread
  for (int base = 0; base < L; base += kThreads) {
    const int j = base + threadIdx.x;
    bool above = false, tie = false;
    if (j < L) {
      if (j < lo || j >= hi) {
        above = true;
      } else if (any) {
        const uint32_t key = order_key(w[j]);
        above = key > prefix;
        tie = key == prefix;
      }
    }
    const uint32_t tb = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) warp_tie[warp] = __popc(tb);
    __syncthreads();
    uint32_t before = ties, all = ties;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) before += warp_tie[i];
      all += warp_tie[i];
    }
    before += __popc(tb & ((1u << lane) - 1u));
    const bool take = above || (tie && before < need);
    const uint32_t kb = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_keep[warp] = __popc(kb);
    __syncthreads();
    uint32_t at = out, total = out;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) at += warp_keep[i];
      total += warp_keep[i];
    }
    at += __popc(kb & ((1u << lane) - 1u));
    if (take && at < (uint32_t)P.keep) kept[at] = j;
    ties = all;
    out = total;
    __syncthreads();
  }
}

// One block per (sequence, KV head), in rounds of kRows rows: every row of a
// round is in registers before any is written, and rows only move towards
// the front, so dst may be src.
constexpr int kRows = 256;

template <int D>
__global__ void __launch_bounds__(kThreads) move_kernel(const EvictParams P) {
  constexpr int kChunks = D / 32;               // 16-byte pieces of one tensor's row
  constexpr int kPieces = kRows * 2 * kChunks;  // of a round
  constexpr int kPer = (kPieces + kThreads - 1) / kThreads;
  const int h = blockIdx.x, b = blockIdx.y;
  const int* kept = P.kept + ((long long)b * P.src.H + h) * P.keep;
  const long long s0 = head_row(P.src, b, h), d0 = head_row(P.dst, b, h);
  for (int r0 = 0; r0 < P.keep; r0 += kRows) {
    uint4 buf[kPer];
    uint32_t sc = 0;
    float w = 0.f;
    int from[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = threadIdx.x + i * kThreads;
      const int r = r0 + p / (2 * kChunks), c = p % (2 * kChunks);
      from[i] = (p < kPieces && r < P.keep) ? kept[r] : -1;
      if (from[i] >= 0) {
        const uint8_t* t = c < kChunks ? P.src.kc : P.src.vc;
        buf[i] = *reinterpret_cast<const uint4*>(t + (s0 + from[i]) * (D / 2) + (c % kChunks) * 16);
      }
    }
    // threads 0 .. kRows-1: K scales and weights; kRows .. 2 kRows - 1: V scales
    const int sr = r0 + (threadIdx.x % kRows), st = threadIdx.x / kRows;
    const int sfrom = (st < 2 && sr < P.keep) ? kept[sr] : -1;
    if (sfrom >= 0) {
      const uint8_t* t = (st ? P.src.vs : P.src.ks) + (s0 + sfrom) * (D / 32);
      sc = D == 128 ? *reinterpret_cast<const uint32_t*>(t) : *reinterpret_cast<const uint16_t*>(t);
      if (st == 0) w = P.src.w[s0 + sfrom];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = threadIdx.x + i * kThreads;
      const int r = r0 + p / (2 * kChunks), c = p % (2 * kChunks);
      if (from[i] >= 0) {
        uint8_t* t = c < kChunks ? P.dst.kc : P.dst.vc;
        *reinterpret_cast<uint4*>(t + (d0 + r) * (D / 2) + (c % kChunks) * 16) = buf[i];
      }
    }
    if (sfrom >= 0) {
      uint8_t* t = (st ? P.dst.vs : P.dst.ks) + (d0 + sr) * (D / 32);
      if (D == 128) *reinterpret_cast<uint32_t*>(t) = sc;
      else *reinterpret_cast<uint16_t*>(t) = (uint16_t)sc;
      if (st == 0) {
        if (P.dst.w) P.dst.w[d0 + sr] = w;
        // the last kept row tells the new length
        if (h == 0 && (sr + 1 == P.keep || kept[sr + 1] < 0)) P.dst.lens[b] = sr + 1;
      }
    }
    __syncthreads();
  }
  if (h == 0 && threadIdx.x == 0 && kept[0] < 0) P.dst.lens[b] = 0;
}

}  // namespace

usp_status_t launch_kv4_evict(const Cache& src, const Cache& dst, int D, int* kept, int keep,
                              int recent, int sink, cudaStream_t st) {
  EvictParams P{src, dst, kept, keep, recent, sink};
  {
    ProfScope ps(st, "kv4_evict_select");
    select_kernel<<<dim3(src.H, src.B), kThreads, 0, st>>>(P);
  }
  note_launch();
  usp_status_t r = check_launch();
  if (r != USP_OK) return r;
  {
    ProfScope ps(st, "kv4_evict_move");
    if (D == 128)
      move_kernel<128><<<dim3(src.H, src.B), kThreads, 0, st>>>(P);
    else
      move_kernel<64><<<dim3(src.H, src.B), kThreads, 0, st>>>(P);
  }
  note_launch();
  return check_launch();
}

}  // namespace usp
