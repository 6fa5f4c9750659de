// Eviction from the 4-bit KV cache by accumulated attention weight.
//
// A cluster of CTAs owns one (sequence, KV head). Every CTA takes an equal,
// contiguous part of the head's weights, brings it into shared memory once as
// order-preserving 32-bit keys, and the cluster finds the n-th largest key by
// three radix passes (11, 10 and 11 bits): each CTA counts its part into its
// own histogram, also in groups of 32 bins; after one cluster barrier every CTA
// adds up the cluster's groups through distributed shared memory, and then the
// bins of the one group that matters (3 KB read from the others; all of their
// histograms would be 64 KB), so that all reach the same bin with no further
// exchange. One more barrier gives every CTA how many keys are kept before its
// part, and it writes their rows in ascending order; after another the cluster
// copies the kept rows' codes, scales and weights.
//
// Bound by latency: a cluster takes about 20 us to choose (of which the weights'
// load 3.5, each pass 2, the barriers 1 each) and 9 to move 8192 rows, at HBM's
// rate, and 36 clusters of eight fit the GPU at once. 64 heads of up to 128K
// tokens, 8192 kept: 68 us, 2.5 TB/s (45 with 256 kept; 153 with clusters of four,
// 232 of two: choosing is as long as a CTA's part). 64 heads of 1088, 1024 kept:
// 14 us replayed from a graph, of which launch and barriers are most. In place: 75
// and 16 us. Rows only move towards the front,
// so in place the copy goes in rounds: every row of a round is in registers
// before a barrier, and written after it; later rounds read behind every row that
// earlier ones write.
#include <type_traits>

#include "internal.h"
#include "kv4.cuh"
#include "kv4_host.h"
#include "tc_ptx.cuh"

namespace usp {
namespace {

using namespace kv4;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
// Keys of a CTA's part in shared memory; longer parts (beyond 8 x 16K tokens) are
// read again from L2 in each pass. Two CTAs of this size leave 92 KB of the SM to
// L1, where the moved rows' gathers in flight are held: with 60 KB the 128K prompt
// below took 78 us, with 28 KB 108. Twenty thousand keys: 150 us instead of 146
// for 64 heads of 160K tokens, 123 instead of 97 for 32 of 256K, but 52 instead of
// 59 for 16 of 160K.
constexpr int kKeysInSmem = 16384;
// Where key i (a multiple of 4) of a warp's part stands: the 16-byte pieces of
// 32 keys change places with the row, so that both ways of reading them (a warp
// 128 in a row, or each lane 32 of its own) meet all banks.
__device__ __forceinline__ int place(int i) { return i ^ (i >> 3 & 28); }

// Larger float <=> larger key; +0 and -0 alike; a NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (isnan(x)) return 0xffffffffu;
  if (x == 0.f) return 0x80000000u;
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The 32-bit word at this CTA's shared address `p`, of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t peer_load(const uint32_t* p, uint32_t rank) {
  uint32_t a, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// A lane lists its kept keys by itself up to this many (about 10 instructions
// each, one after the other; the 32 steps of the warp together take as long as
// 12 of them).
constexpr int kSparse = 12;

struct EvictParams {
  Cache src, dst;
  int* kept;
  int keep, recent, sink;
  int in_place;
  int cluster;  // CTAs per (sequence, KV head)
};

constexpr int kGroups = kBins / 32;
struct __align__(16) EvictSmem {
  __device__ __forceinline__ uint32_t* bins(int pass) { return pass == 1 ? hist1 : hist; }
  uint32_t hist[kBins];                 // of the first and the third pass
  uint32_t hist1[kBins / 2];            // of the second
  uint32_t groups[3][kGroups];          // sums of 32 bins
  uint32_t sums[kGroups];               // of the cluster
  uint32_t above[kWarps], tie[kWarps];  // of each warp's part
  uint32_t total[2];                    // kept for sure and ties of this CTA
};

// Of 32 counts, lane l's being that of item 31 - l: which item holds the
// need-th one from the top; leaves in `need` how many of that item are needed.
__device__ __forceinline__ int item_of(uint32_t count, uint32_t& need) {
  const int lane = threadIdx.x & 31;
  uint32_t inc = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  const int l = __ffs(__ballot_sync(0xffffffffu, inc >= need)) - 1;
  need -= __shfl_sync(0xffffffffu, inc - count, l);
  return 31 - l;
}

// The bin (from the top) in which the cluster's need-th key lies; `need`
// becomes how many of the bin are needed. Every warp finds it for itself.
__device__ __forceinline__ uint32_t find_bin(EvictSmem& s, int pass, int cluster, uint32_t& need) {
  const int lane = threadIdx.x & 31;
  const int item = threadIdx.x >> 3, r = threadIdx.x & 7;  // eight lanes: one per CTA
  static_assert(kThreads == 8 * kGroups && kMaxCluster == 8, "a group per eight threads");
  uint32_t x = r < cluster ? peer_load(&s.groups[pass][item], r) : 0u;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (r == 0) s.sums[item] = x;
  __syncthreads();
  const uint32_t hi = s.sums[kGroups - 1 - 2 * lane], lo = s.sums[kGroups - 2 - 2 * lane];
  const int pair = item_of(hi + lo, need);  // groups 2 pair + 1 and 2 pair
  const uint32_t top = __shfl_sync(0xffffffffu, hi, 31 - pair);
  int group = 2 * pair + 1;
  if (need > top) {
    need -= top;
    group = 2 * pair;
  }
  __syncthreads();
  if (item < 32) {  // (whole warps)
    x = r < cluster ? peer_load(&s.bins(pass)[32 * group + item], r) : 0u;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (r == 0) s.sums[item] = x;
  }
  __syncthreads();
  return 32 * group + item_of(s.sums[31 - lane], need);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const EvictParams P) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  EvictSmem& s = *reinterpret_cast<EvictSmem*>(smem_raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem_raw + sizeof(EvictSmem));
  const int rank = (int)cluster_rank();
  const int h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int L = clamp_len(P.src.lens[b], P.src.C);
  const int n_out = min(L, P.keep);
  int* kept = P.kept + ((long long)b * P.src.H + h) * P.keep;
  const long long s0 = head_row(P.src, b, h), d0 = head_row(P.dst, b, h);
  const float* w = P.src.w + s0;

  if (L <= P.keep) {
    for (int i = rank * kThreads + threadIdx.x; i < P.keep; i += P.cluster * kThreads)
      kept[i] = i < L ? i : -1;
    if (P.in_place) return;  // (the whole cluster)
  } else {
    const int lo = P.sink, hi = L - P.recent;  // candidates [lo, hi)
    uint32_t need = (uint32_t)(P.keep - P.sink - P.recent);
    // this warp's part: `per` keys from `first` on
    const int per = ((L + P.cluster * kWarps - 1) / (P.cluster * kWarps) + 127) / 128 * 128;
    const long long first = (long long)(rank * kWarps + warp) * per;
    const int n = (int)max(0LL, min((long long)per, L - first));
    const bool in_smem = per * kWarps <= kKeysInSmem;
    uint32_t* mine = keys + warp * per;
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      s.hist[i] = 0;
      if (i < kBins / 2) s.hist1[i] = 0;
    }
    if (in_smem) {
      // 16 bytes per lane (the rows before a head are a multiple of 16); a
      // read behind L stays inside the capacity
#pragma unroll 4
      for (int i = 4 * lane; i < n; i += 128) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(w + first + i));
        *reinterpret_cast<uint4*>(mine + place(i)) =
            make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
      }
    }
    __syncthreads();
    // keys i .. i + 3 of the warp's part (i a multiple of 4)
    auto keys_at = [&](int i) {
      if (in_smem) return *reinterpret_cast<const uint4*>(mine + place(i));
      const float4 x = __ldg(reinterpret_cast<const float4*>(w + first + i));
      return make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
    };
    // which of them: not behind the part (n) and, relative to it, in [lo, hi)
    const int c_lo = (int)max(0LL, min((long long)n, lo - first));
    const int c_hi = (int)max((long long)c_lo, min((long long)n, hi - first));
    uint32_t prefix = 0;  // the n-th largest key's bits found so far
    if (need > 0) {
      constexpr int kShift[3] = {21, 11, 0};
      constexpr uint32_t kMask[3] = {0u, 0xffe00000u, 0xfffff800u};
#pragma unroll
      for (int pass = 0; pass < 3; ++pass) {
        const uint32_t bin_mask = pass == 1 ? 1023u : 2047u;
        // several keys per lane at a time, so that their latencies overlap
        auto count = [&](auto vectors, int i0) {
          constexpr int kV = decltype(vectors)::value, kN = 4 * kV;
          uint32_t key[kN];
#pragma unroll
          for (int u = 0; u < kV; ++u) {
            const int i = i0 + 128 * u + 4 * lane;
            uint4 k = make_uint4(0, 0, 0, 0);
            if (i < c_hi) k = keys_at(i);
            key[4 * u] = k.x; key[4 * u + 1] = k.y; key[4 * u + 2] = k.z; key[4 * u + 3] = k.w;
          }
          constexpr uint32_t kAll = (1u << kN) - 1u;
          uint32_t in = 0;
#pragma unroll
          for (int e = 0; e < kN; ++e) in |= ((key[e] & kMask[pass]) == prefix ? 1u : 0u) << e;
          if (i0 < c_lo || i0 + 128 * kV > c_hi) {  // an end of the candidates
#pragma unroll
            for (int e = 0; e < kN; ++e) {
              const int i = i0 + 128 * (e >> 2) + 4 * lane + (e & 3);
              if (i < c_lo || i >= c_hi) in &= ~(1u << e);
            }
          }
          if (!__any_sync(0xffffffffu, in != 0)) return;
          bool alike = in == kAll;
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            key[e] = (key[e] >> kShift[pass]) & bin_mask;
            alike = alike && key[e] == key[0];
          }
          // one addition where the whole warp agrees (runs of equal weights)
          if (__all_sync(0xffffffffu, alike) &&
              __all_sync(0xffffffffu, key[0] == __shfl_sync(0xffffffffu, key[0], 0))) {
            if (lane == 0) atomicAdd(&s.bins(pass)[key[0]], 32u * kN);
          } else {
#pragma unroll
            for (int e = 0; e < kN; ++e)
              if ((in >> e) & 1u) atomicAdd(&s.bins(pass)[key[e]], 1u);
          }
        };
        int i0 = c_lo / 128 * 128;
        for (; i0 + 384 < c_hi; i0 += 512) count(std::integral_constant<int, 4>{}, i0);
        for (; i0 < c_hi; i0 += 128) count(std::integral_constant<int, 1>{}, i0);
        __syncthreads();
        {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (pass != 1 || threadIdx.x < kThreads / 2)
            x = reinterpret_cast<const uint4*>(s.bins(pass))[threadIdx.x];
          uint32_t sum = x.x + x.y + x.z + x.w;
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if ((threadIdx.x & 7) == 0) s.groups[pass][threadIdx.x >> 3] = sum;
        }
        cluster_sync();
        if (pass == 1)  // no CTA reads the first pass's counts any more
          for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[i] = 0;
        prefix |= find_bin(s, pass, P.cluster, need) << kShift[pass];
      }
    }
    const bool any = P.keep - P.sink - P.recent > 0;
    // Of the lane's 32 keys from i0 + 32 lane on: those kept for sure (sinks,
    // recent, above the n-th largest), and those equal to it.
    auto masks_at = [&](int i0, uint32_t& sure, uint32_t& tied) {
      const int at = i0 + 32 * lane;
      auto bits = [&](int lo, int hi) {  // of [lo, hi)
        const int x = min(max(lo - at, 0), 32), y = min(max(hi - at, x), 32);
        return static_cast<uint32_t>((1ull << y) - (1ull << x));
      };
      const uint32_t free = any ? bits(c_lo, c_hi) : 0u;
      sure = bits(0, c_lo) | bits(c_hi, n);
      tied = 0;
      if (free == 0) return;
      uint32_t above = 0;
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        uint4 k = make_uint4(0, 0, 0, 0);
        if (at + 4 * v < n) k = keys_at(at + 4 * v);
        const uint32_t key[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          above |= (key[e] > prefix ? 1u : 0u) << (4 * v + e);
          tied |= (key[e] == prefix ? 1u : 0u) << (4 * v + e);
        }
      }
      sure |= above & free;
      tied &= free;
    };
    uint32_t above = 0, tie = 0, sure = 0, tied = 0;
    for (int i0 = 0; i0 < n; i0 += 1024) {
      masks_at(i0, sure, tied);
      above += __popc(sure);
      tie += __popc(tied);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      above += __shfl_xor_sync(0xffffffffu, above, o);
      tie += __shfl_xor_sync(0xffffffffu, tie, o);
    }
    if (lane == 0) {
      s.above[warp] = above;
      s.tie[warp] = tie;
    }
    __syncthreads();
    uint32_t a_before = 0, t_before = 0;
    {
      const uint32_t x = lane < kWarps ? s.above[lane] : 0u, y = lane < kWarps ? s.tie[lane] : 0u;
      uint32_t xi = x, yi = y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t xo = __shfl_up_sync(0xffffffffu, xi, o);
        const uint32_t yo = __shfl_up_sync(0xffffffffu, yi, o);
        if (lane >= o) {
          xi += xo;
          yi += yo;
        }
      }
      a_before = __shfl_sync(0xffffffffu, xi - x, warp);
      t_before = __shfl_sync(0xffffffffu, yi - y, warp);
      if (warp == 0 && lane == 31) {
        s.total[0] = xi;
        s.total[1] = yi;
      }
    }
    cluster_sync();
    {
      // of the CTAs before this one
      uint32_t x = lane < rank ? peer_load(&s.total[0], lane) : 0u;
      uint32_t y = lane < rank ? peer_load(&s.total[1], lane) : 0u;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
      }
      a_before += x;
      t_before += y;
    }
    for (int i0 = 0; i0 < n; i0 += 1024) {
      if (n > 1024) masks_at(i0, sure, tied);  // (else they are still there)
      uint32_t ai = __popc(sure), ti = __popc(tied);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t ao = __shfl_up_sync(0xffffffffu, ai, o);
        const uint32_t to = __shfl_up_sync(0xffffffffu, ti, o);
        if (lane >= o) {
          ai += ao;
          ti += to;
        }
      }
      const uint32_t t = t_before + ti - __popc(tied);  // ties before the lane's
      uint32_t out = a_before + ai - __popc(sure) + min(t, need);
      a_before += __shfl_sync(0xffffffffu, ai, 31);
      t_before += __shfl_sync(0xffffffffu, ti, 31);
      // the first `need` ties of all are kept
      uint32_t ties = tied;
      for (uint32_t left = __popc(tied), k = t < need ? need - t : 0u; left > k; --left)
        ties &= ~(0x80000000u >> __clz(ties));
      uint32_t word = sure | ties;
      const int key0 = (int)first + i0 + 32 * lane;
      if (__reduce_max_sync(0xffffffffu, __popc(word)) > kSparse) {
        // lane by lane, the warp together
#pragma unroll 4
        for (int l = 0; l < 32; ++l) {
          const uint32_t w = __shfl_sync(0xffffffffu, word, l);
          const uint32_t at = __shfl_sync(0xffffffffu, out, l) + __popc(w & ((1u << lane) - 1u));
          if (((w >> lane) & 1u) && at < (uint32_t)P.keep)
            kept[at] = (int)first + i0 + 32 * l + lane;
        }
      } else {
        for (; word != 0; word &= word - 1, ++out)
          if (out < (uint32_t)P.keep) kept[out] = key0 + __ffs(word) - 1;
      }
    }
  }
  cluster_sync();  // the list is complete; no CTA needs another's memory any more

  // ------------------------------------------------------------------ move
  constexpr int kChunks = D / 16;  // 16-byte pieces of a row's K and V codes
  constexpr int kPer = D / 16;     // pieces in a thread's registers: 512 rows per CTA and round
  constexpr int kRows = kThreads * kPer / kChunks;
  static_assert(kRows == kThreads, "a row per thread");
  const int c = threadIdx.x % kChunks;
  const uint8_t* from_codes = (c < kChunks / 2 ? P.src.kc : P.src.vc) + (c % (kChunks / 2)) * 16;
  uint8_t* to_codes = (c < kChunks / 2 ? P.dst.kc : P.dst.vc) + (c % (kChunks / 2)) * 16;
  for (int r0 = rank * kRows; r0 - rank * kRows < n_out; r0 += P.cluster * kRows) {
    uint4 buf[kPer];
    int from[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = r0 + threadIdx.x / kChunks + i * (kThreads / kChunks);
      from[i] = r < n_out ? kept[r] : -1;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (from[i] >= 0)
        buf[i] = *reinterpret_cast<const uint4*>(from_codes + (s0 + from[i]) * (D / 2));
    // scales and weights: a thread per row
    const int sr = r0 + threadIdx.x;
    const int sfrom = threadIdx.x < kRows && sr < n_out ? kept[sr] : -1;
    uint32_t sk = 0, sv = 0;
    float sw = 0.f;
    if (sfrom >= 0) {
      const uint8_t* ks = P.src.ks + (s0 + sfrom) * (D / kBlock);
      const uint8_t* vs = P.src.vs + (s0 + sfrom) * (D / kBlock);
      if constexpr (D == 128) {
        sk = *reinterpret_cast<const uint32_t*>(ks);
        sv = *reinterpret_cast<const uint32_t*>(vs);
      } else {
        sk = *reinterpret_cast<const uint16_t*>(ks);
        sv = *reinterpret_cast<const uint16_t*>(vs);
      }
      sw = w[sfrom];
    }
    if (P.in_place) cluster_sync();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = r0 + threadIdx.x / kChunks + i * (kThreads / kChunks);
      if (from[i] >= 0) *reinterpret_cast<uint4*>(to_codes + (d0 + r) * (D / 2)) = buf[i];
    }
    if (sfrom >= 0) {
      uint8_t* ks = P.dst.ks + (d0 + sr) * (D / kBlock);
      uint8_t* vs = P.dst.vs + (d0 + sr) * (D / kBlock);
      if constexpr (D == 128) {
        *reinterpret_cast<uint32_t*>(ks) = sk;
        *reinterpret_cast<uint32_t*>(vs) = sv;
      } else {
        *reinterpret_cast<uint16_t*>(ks) = (uint16_t)sk;
        *reinterpret_cast<uint16_t*>(vs) = (uint16_t)sv;
      }
      if (P.dst.w) P.dst.w[d0 + sr] = sw;
    }
  }
  // In place, other clusters may still have to read the old length: a launch
  // behind this one writes the new one.
  if (!P.in_place && h == 0 && rank == 0 && threadIdx.x == 0) P.dst.lens[b] = n_out;
}

__global__ void evict_lens_kernel(const EvictParams P) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < P.src.B) P.dst.lens[b] = min(clamp_len(P.src.lens[b], P.src.C), P.keep);
}

template <int D>
usp_status_t launch_d(const EvictParams& P, cudaStream_t st) {
  const int per = ((P.src.C + P.cluster * kWarps - 1) / (P.cluster * kWarps) + 127) / 128 * 128;
  const int n = per * kWarps <= kKeysInSmem ? per * kWarps : kKeysInSmem;
  const size_t smem = sizeof(EvictSmem) + (size_t)n * 4;
  static SmemAttr smem_attr;
  cudaError_t e = smem_attr.set(evict_kernel<D>, (int)(sizeof(EvictSmem) + kKeysInSmem * 4));
  if (e != cudaSuccess) return fail_cuda("cudaFuncSetAttribute(smem)", e);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(P.cluster, P.src.H, P.src.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = P.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  {
    ProfScope ps(st, "kv4_evict");
    e = cudaLaunchKernelEx(&cfg, evict_kernel<D>, P);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail_cuda("kernel launch", e);
  }
  note_launch();
  return USP_OK;
}

}  // namespace

usp_status_t launch_kv4_evict(const Cache& src, const Cache& dst, int D, int* kept, int keep,
                              int recent, int sink, cudaStream_t st) {
  EvictParams P{src, dst, kept, keep, recent, sink, src.kc == dst.kc && src.C > 0, 1};
  // a CTA per 4K tokens (one radix pass takes a warp 128 keys), at most eight
  while (P.cluster < kMaxCluster && (long long)P.cluster * 4096 < src.C) P.cluster *= 2;
  usp_status_t r = D == 128 ? launch_d<128>(P, st) : launch_d<64>(P, st);
  if (r != USP_OK || !P.in_place) return r;
  {
    ProfScope ps(st, "kv4_evict_lens");
    evict_lens_kernel<<<(src.B + 255) / 256, 256, 0, st>>>(P);
  }
  note_launch();
  return check_launch();
}

}  // namespace usp
