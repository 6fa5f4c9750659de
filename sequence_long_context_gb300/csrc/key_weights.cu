// How much each key of a prompt was attended: column sums of the attention
// matrix, from the forward's q, k and LSE.
//
//     weight[g][j] = sum over query heads h of group g and observed queries i
//                    that see key j of exp(scale <q_i,h, k_j> - LSE_i,h)
// ("Long Context Attention" notes, "Motivation": the LSE is what the forward
// keeps; with it a probability needs no second pass over its row.)
//
// Tensor-core kernel (bf16). One CTA owns 256 keys (two tiles of 128) of one
// KV head and takes the query tiles of 64 that may see them, for some of the
// group's query heads and a segment of the queries: S^T = K Q^T, keys on the
// 128 TMEM lanes, so that a softmax thread owns a key and the column sum is a
// register. Nothing is normalised or rescaled, and nothing goes back to the
// tensor core. The keys are the A operand and stay in tensor memory, put there
// by the threads that own them: from shared memory the products would read
// 6 KB in the 32 clocks of a 128 x 64 x 16 product, where 4 KB is what it can
// give (measured: 57 clocks each). So only Q (2 KB per product) passes through
// shared memory. The products of a 128 x 64 tile (D = 128) take 256 clocks,
// its exponentials (32 per clock and SM) as many. A key tile has one 64-column
// buffer of scores: the softmax takes it into registers at once, and while it
// works the other products run. What then limits is the MMA warp, whose
// products are issued no faster than they run and which waits between them:
// so two CTAs per SM, each with its own, and as few barriers for it as can be
// (512 keys in one CTA: 2400 clocks per 512 x 64 scores).
// Roles (320 threads):
//   warps 0-7  softmax: warp w owns keys [32 w, 32 w + 32)
//   warp 8     producer: finds the query tiles that can see the keys (32 at a
//              time, one per lane), loads Q (five slots) and, with all lanes,
//              the tile's LSE (asked for one tile ahead) and positions
//   warp 9     MMA issuer, owner of tensor memory: K of key tile a in columns
//              [a D/2, + D/2), its S^T in [D + 64 a, + 64)
// Positions are read per query from shared memory, so a tile may cross chunk
// and shard boundaries: any layout and any length has this kernel.
//
// The partial sums of several heads or segments go to the workspace and are
// added in a fixed order by a second kernel.
//
// CUDA-core kernel (fp32 inputs, and as a cross-check): 64 x 64 tiles.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdio>

#include "internal.h"
#include "tc_ptx.cuh"
#include "tile_sched.cuh"

namespace usp {
namespace {

using namespace tc;

__device__ int g_key_weights_status = 0;

constexpr int kQT = 64;             // queries per tile
constexpr int kKT = 2;              // key tiles per CTA
constexpr int kKeys = kKT * kTile;  // keys per CTA
constexpr int kSoftWarps = 4 * kKT;
constexpr int kProducerWarp = kSoftWarps;
constexpr int kMmaWarp = kProducerWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kSlots = 5;           // Q tiles
constexpr int kRing = 8;           // entries of query statistics
constexpr int kEnd = -1;
constexpr int kNowhere = -(1 << 30);  // position of a row that is not observed
constexpr float kLog2e = 1.4426950408889634f;

// True in one lane of the warp, the same every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

struct WeightParams {
  AttnParams P;
  float* part;   // [parts][Bt][Hkv][S]
  int observe;   // 0: all
  int hpi;       // query heads per CTA
  int nseg;      // segments of query tiles
  int tps;       // query tiles per segment
  int nkb;       // key blocks
  int q0;        // first row of tile 0: where the observed rows begin, if they
                 // are one run to the end; else 0
  int ntiles;    // query tiles
};

template <int D>
struct WSmem {
  // A ring entry is written for tile x once the products of tile x - kSlots
  // are done; the softmax is then past the scores of tile x - kSlots - 1, so
  // past the statistics of tile x - kSlots - 2.
  static_assert(kRing >= kSlots + 2, "a statistics entry is free");
  static constexpr int kHalves = D / 64;
  static constexpr int kQHalf = kQT * 128;              // 64 channels of a Q tile
  static constexpr int kQTile = kQHalf * kHalves;
  static constexpr int kQ = 0;
  static constexpr int kStat = kQ + kSlots * kQTile;    // kRing x (-lse2[64], pos[64])
  static constexpr int kStatBytes = 2 * kQT * 4;
  static constexpr int kSched = kStat + kRing * kStatBytes;  // kRing ints
  static constexpr int kBar = kSched + kRing * 4;
  static constexpr int kKReady = 0, kQFull = kKReady + kKT, kQFree = kQFull + kSlots,
                       kSFull = kQFree + kSlots, kSFree = kSFull + kKT,
                       kStatFull = kSFree + kKT, kMmaDone = kStatFull + kRing,
                       kNumBars = kMmaDone + 1;
  static constexpr int kTmemS = kKT * D / 2;            // columns
  static constexpr int kTmem = 256;
  static_assert(kTmemS + kQT * kKT <= kTmem, "tensor memory");
  static constexpr int kMisc = (kBar + 8 * kNumBars + 15) / 16 * 16;
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 113 * 1024, "two CTAs per SM");
  static_assert(kBar % 8 == 0 && kStat % 16 == 0, "alignment");
};

// The queries that see the key at natural position j, as positions [lo, hi].
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen seen_by(const AttnParams& P, int j) {
  int s = 0, e = P.S;
  if (P.cu != nullptr) {
    const int n = seg_of(P.cu, P.nseq, j);
    s = __ldg(P.cu + n);
    e = __ldg(P.cu + n + 1);
  }
  Seen r;
  r.lo = P.causal ? j : s;
  r.hi = e - 1;
  if (P.window > 0 && j - s >= P.sink) r.hi = min(r.hi, j + P.window - 1);
  return r;
}

// Natural position of the query at rank-major row p if it is observed.
__device__ __forceinline__ int observed_pos(const WeightParams& W, int p) {
  const AttnParams& P = W.P;
  if (p >= P.S) return kNowhere;
  const int i = nat_pos(P, p);
  if (W.observe > 0) {
    int e = P.S;
    if (P.cu != nullptr) e = __ldg(P.cu + seg_of(P.cu, P.nseq, i) + 1);
    if (i < e - W.observe) return kNowhere;
  }
  return i;
}

// Bounds of the natural positions of rank-major rows [p0, p0 + n) (clipped to
// S); exact where the rows are one run of a chunk, else row by row.
__device__ __forceinline__ PosRange row_bounds(const AttnParams& P, int p0, int n) {
  PosRange r{1, 0};
  const int p1 = min(p0 + n, P.S) - 1;
  if (p1 < p0) return r;
  const int run = P.layout == kZigzag ? P.chunk : P.shard;
  if (p0 / run == p1 / run) {
    r.lo = nat_pos(P, p0);
    r.hi = nat_pos(P, p1);
    return r;
  }
  if (P.layout == kContiguous) {
    r.lo = p0;
    r.hi = p1;
    return r;
  }
  r.lo = P.S;
  r.hi = -1;
  for (int p = p0; p <= p1; ++p) {
    const int i = nat_pos(P, p);
    r.lo = min(r.lo, i);
    r.hi = max(r.hi, i);
  }
  return r;
}

struct KeyBlock {
  PosRange k;     // natural positions of the keys
  PosRange q;     // of the queries that may see one of them
  int seg0, seg1; // packed sequences of the first and last key
};
__device__ __forceinline__ KeyBlock key_block(const AttnParams& P, int key0) {
  KeyBlock b;
  b.k = row_bounds(P, key0, kKeys);
  int s0 = 0, e1 = P.S;
  b.seg0 = b.seg1 = 0;
  if (P.cu != nullptr) {
    b.seg0 = seg_of(P.cu, P.nseq, b.k.lo);
    b.seg1 = seg_of(P.cu, P.nseq, b.k.hi);
    s0 = __ldg(P.cu + b.seg0);
    e1 = __ldg(P.cu + b.seg1 + 1);
  }
  const bool sinks = P.sink > 0 && (b.seg0 != b.seg1 || b.k.lo < s0 + P.sink);
  b.q.lo = P.causal ? b.k.lo : s0;
  b.q.hi = (P.window > 0 && !sinks) ? min(e1 - 1, b.k.hi + P.window - 1) : e1 - 1;
  return b;
}

// empty / full / masked for the queries of tile qt against the key block.
__device__ __forceinline__ int classify_tile(const WeightParams& W, int qt, const KeyBlock& b) {
  const AttnParams& P = W.P;
  const int p0 = W.q0 + qt * kQT;
  const PosRange q = row_bounds(P, p0, kQT);
  if (q.lo > q.hi || q.hi < b.q.lo || q.lo > b.q.hi) return kClsEmpty;
  bool all = true;  // rows behind S are zeros with LSE = inf: no mask needed
  if (W.observe > 0) {
    if (P.cu == nullptr) {
      if (q.hi < P.S - W.observe) return kClsEmpty;
      all = all && q.lo >= P.S - W.observe;
    } else {
      // the last `observe` of some sequence between q.lo's and q.hi's
      const int n = seg_of(P.cu, P.nseq, q.lo);
      const int e = __ldg(P.cu + n + 1);
      if (q.hi < e - W.observe) return kClsEmpty;
      all = all && q.lo >= e - W.observe;
    }
  }
  if (P.cu != nullptr) {
    const int s0 = seg_of(P.cu, P.nseq, q.lo), s1 = seg_of(P.cu, P.nseq, q.hi);
    if (s0 != s1 || b.seg0 != b.seg1 || s0 != b.seg0) return kClsMasked;
  }
  if (P.causal && b.k.hi > q.lo) all = false;
  if (P.window > 0 && q.hi - b.k.lo >= P.window) all = false;
  return all ? kClsFull : kClsMasked;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
key_weights_tc_kernel(const WeightParams W, const __grid_constant__ CUtensorMap tm_q) {
  using L = WSmem<D>;
  const AttnParams& P = W.P;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(sm);
  auto bar = [&](int i) { return sbase + L::kBar + 8 * i; };
  volatile int* sched = reinterpret_cast<volatile int*>(sm + L::kSched);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  int* status = &g_key_weights_status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // key blocks outermost: with a causal mask the heaviest (first) start first
  const int groups = P.G / W.hpi;  // CTAs per KV head and segment
  int idx = blockIdx.x;
  const int part = idx % (groups * W.nseg);
  idx /= groups * W.nseg;
  const int g = idx % P.Hkv;
  idx /= P.Hkv;
  const int bt = idx % P.Bt, kb = idx / P.Bt;
  const int seg = part / groups, h0 = g * P.G + (part % groups) * W.hpi;
  const int key0 = kb * kKeys;
  const int ktiles = min(kKT, (P.S - key0 + kTile - 1) / kTile);  // with keys in them

  if (warp == kProducerWarp && lane == 0) {
    // the four warps of a key tile: its keys are in tensor memory
    for (int a = 0; a < kKT; ++a) mbar_init(bar(L::kKReady + a), 4);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(L::kQFull + s), 1);
      mbar_init(bar(L::kQFree + s), 1);
    }
    for (int s = 0; s < kKT; ++s) {
      mbar_init(bar(L::kSFull + s), 1);
      mbar_init(bar(L::kSFree + s), 4);  // the four warps of a key tile
    }
    for (int s = 0; s < kRing; ++s) mbar_init(bar(L::kStatFull + s), 1);
    mbar_init(bar(L::kMmaDone), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch(&tm_q);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sbase + L::kMisc, L::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    const KeyBlock blk = key_block(P, key0);
    int first = seg * W.tps, last = min(W.ntiles, first + W.tps);
    if (P.layout == kContiguous) {  // rank-major order is natural order
      first = max(first, (blk.q.lo - W.q0) / kQT);  // (towards 0: an extra tile is skipped)
      last = blk.q.hi < W.q0 ? 0 : min(last, (blk.q.hi - W.q0) / kQT + 1);
    }
    // The next (tile, head), its rows' positions and LSE. This runs once per
    // tile in one warp, so it is kept short: what takes divisions is found for
    // 32 tiles at a time, one per lane.
    struct Item {
      int row, cls, h, pos[kQT / 32];  // row: the tile's first
      float lse[kQT / 32];
    };
    const float* lse_head = P.lse + lse_index(P, bt, h0, 0);
    const int step = P.layout == kStripe ? P.cp : 1;
    const int run = P.layout == kZigzag ? P.chunk : P.shard;
    int base = first - 32, cls_mine = kClsEmpty, lo_mine = 0, hh = 0;
    unsigned todo = 0;
    Item nx{};
    bool more = true;
    auto fetch = [&]() {
      if (hh == 0) {  // a new tile
        while (todo == 0 && (base += 32) < last) {
          const int t = base + lane;
          cls_mine = t < last ? classify_tile(W, t, blk) : kClsEmpty;
          todo = __ballot_sync(0xffffffffu, cls_mine != kClsEmpty);
          // first position, or -1: the rows are not one run of a chunk, or
          // which are observed depends on the sequence
          lo_mine = -1;
          if (cls_mine != kClsEmpty && (W.observe == 0 || P.cu == nullptr)) {
            const int p0 = W.q0 + t * kQT, p1 = min(p0 + kQT, P.S) - 1;
            if (p0 / run == p1 / run || P.layout == kContiguous) lo_mine = nat_pos(P, p0);
          }
        }
        if (todo == 0) {
          more = false;
          return;
        }
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        nx.row = W.q0 + (base + src) * kQT;
        nx.cls = __shfl_sync(0xffffffffu, cls_mine, src);
        const int lo = __shfl_sync(0xffffffffu, lo_mine, src);
        const int from = W.observe > 0 ? P.S - W.observe : 0;
#pragma unroll
        for (int e = 0; e < kQT / 32; ++e) {
          const int r = lane + 32 * e;
          if (lo >= 0) {
            const int i = lo + r * step;
            nx.pos[e] = nx.row + r < P.S && i >= from ? i : kNowhere;
          } else {
            nx.pos[e] = observed_pos(W, nx.row + r);
          }
        }
      }
      nx.h = h0 + hh;
      const float* src_lse = lse_head + hh * P.lse_sh + nx.row + lane;
#pragma unroll
      for (int e = 0; e < kQT / 32; ++e) nx.lse[e] = nx.pos[e] >= 0 ? __ldg(src_lse + 32 * e) : 0.f;
      if (++hh == W.hpi) hh = 0;
    };
    fetch();
    int n = 0, slot = 0, phase = 1;  // (the first waits on a free slot pass)
    bool ok = true;
    while (more) {
      const Item it = nx;
      fetch();  // its loads are on their way during this tile's waits
      if (n >= kSlots) {  // the slot's previous tile has been multiplied
        ok = mbar_wait(bar(L::kQFree + slot), phase, abort_flag, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
      }
      const int ring = n & (kRing - 1);
      float* st = reinterpret_cast<float*>(sm + L::kStat + ring * L::kStatBytes);
#pragma unroll
      for (int e = 0; e < kQT / 32; ++e) {
        const float x = it.lse[e] * kLog2e;
        // a row that sees nothing adds nothing
        const bool none = it.pos[e] < 0 || x == -INFINITY;
        st[lane + 32 * e] = none ? -INFINITY : -x;
        reinterpret_cast<int*>(st)[kQT + lane + 32 * e] = it.pos[e];
      }
      if (lane == 0) sched[ring] = it.cls;
      __syncwarp();
      if (lane == 0) {
        // (the MMA warp reads the entry's class behind the Q tile's barrier)
        mbar_expect_tx(bar(L::kQFull + slot), L::kQTile);
        for (int hf = 0; hf < L::kHalves; ++hf)
          tma_load_4d(sbase + L::kQ + slot * L::kQTile + hf * L::kQHalf, &tm_q,
                      bar(L::kQFull + slot), hf * 64, it.h, it.row, bt);
        mbar_arrive(bar(L::kStatFull + ring));
      }
      ++n;
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1;
      }
    }
    if (lane == 0) {
      if (ok && (n < kSlots || mbar_wait(bar(L::kQFree + slot), phase, abort_flag, status))) {
        sched[n & (kRing - 1)] = kEnd;
        mbar_arrive(bar(L::kStatFull + (n & (kRing - 1))));
        mbar_arrive(bar(L::kQFull + slot));
      }
      // aborted: the copies in flight land before the CTA ends
      if (*abort_flag)
        for (int i = n > kSlots ? n - kSlots : 0; i < n; ++i)
          mbar_wait_drain(bar(L::kQFull + i % kSlots), (i / kSlots) & 1);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // Every lane runs the loop and one elected lane issues: the descriptors
    // then are uniform values, which the issue takes as they are. (In a loop
    // of one lane alone each of its operands is first moved to a uniform
    // register, 76 clocks per 32-clock product.)
    constexpr uint32_t kId = idesc_bf16_f32(kTile, kQT, 0, 0);
    const uint64_t dq = sdesc_sw128(sbase + L::kQ, 16, 1024);
    const uint32_t t0 = __shfl_sync(0xffffffffu, tmem, 0);
    bool ok = true;
    int slot = 0, phase = 0;
    for (int n = 0; ok; ++n) {
      const int ring = n & (kRing - 1);
      ok = mbar_wait(bar(L::kQFull + slot), phase, abort_flag, status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (__shfl_sync(0xffffffffu, sched[ring], 0) == kEnd) break;
#pragma unroll
      for (int a = 0; a < kKT; ++a) {
        if (a >= ktiles) break;
        if (n == 0) ok = mbar_wait(bar(L::kKReady + a), 0, abort_flag, status);
        // the previous scores have been read
        if (n >= 1) ok = mbar_wait(bar(L::kSFree + a), (n - 1) & 1, abort_flag, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t d = t0 + L::kTmemS + 64 * a, ka = t0 + a * (D / 2);
        const uint64_t db = sdesc_add(dq, slot * L::kQTile);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts(d, ka + 8 * kk, sdesc_add(db, (kk >> 2) * L::kQHalf + (kk & 3) * 32), kId,
                   kk > 0 ? 1u : 0u);
          mma_commit(bar(L::kSFull + a));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) mma_commit(bar(L::kQFree + slot));
      __syncwarp();
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1;
      }
    }
    if (elect_one()) mma_commit(bar(L::kMmaDone));
    mbar_wait_drain(bar(L::kMmaDone), 0);
  } else if ((warp >> 2) < ktiles) {
    // ------------------------------------------------------------ softmax
    const int a = warp >> 2;  // key tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int kp = key0 + warp * 32 + lane;
    {
      // the key's row into tensor memory: lane, channels 2c and 2c + 1 in column c
      const uint4* row = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(P.k) + (((long long)bt * P.S + kp) * P.Hkv + g) * D);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t x[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = kp < P.S ? __ldg(row + 8 * c + i) : make_uint4(0, 0, 0, 0);
          x[4 * i] = v.x;
          x[4 * i + 1] = v.y;
          x[4 * i + 2] = v.z;
          x[4 * i + 3] = v.w;
        }
        tmem_st32(tmem + lane_off + a * (D / 2) + 32 * c, x);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kKReady + a));
    }
    Seen vis{1, 0};
    if (kp < P.S) vis = seen_by(P, nat_pos(P, kp));
    const uint64_t sc2 = f2_pack(P.scale_log2, P.scale_log2);
    uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
    bool ok = true;
    for (int n = 0;; ++n) {
      const int ring = n & (kRing - 1);
      ok = mbar_wait(bar(L::kStatFull + ring), (n / kRing) & 1, abort_flag, status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int cls = sched[ring];
      if (cls == kEnd) break;
      ok = mbar_wait(bar(L::kSFull + a), n & 1, abort_flag, status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc_fence_after();
      uint32_t v[2][32];
      tmem_ld32(tmem + lane_off + L::kTmemS + 64 * a, v[0]);
      tmem_ld32(tmem + lane_off + L::kTmemS + 64 * a + 32, v[1]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kSFree + a));
      const float4* nlse = reinterpret_cast<const float4*>(sm + L::kStat + ring * L::kStatBytes);
      const int4* pos = reinterpret_cast<const int4*>(nlse + kQT / 4);
      if (cls == kClsFull) {
#pragma unroll
        for (int k = 0; k < kQT / 4; ++k) {
          const float4 l = nlse[k];
          const uint32_t* s = &v[k >> 3][4 * (k & 7)];
          const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[0]), __uint_as_float(s[1])), sc2,
                                    f2_pack(l.x, l.y));
          const uint64_t y = f2_fma(f2_pack(__uint_as_float(s[2]), __uint_as_float(s[3])), sc2,
                                    f2_pack(l.z, l.w));
          float x0, x1, y0, y1;
          f2_unpack(x, x0, x1);
          f2_unpack(y, y0, y1);
          sum[(2 * k) & 3] = f2_add(sum[(2 * k) & 3], f2_pack(ex2(x0), ex2(x1)));
          sum[(2 * k + 1) & 3] = f2_add(sum[(2 * k + 1) & 3], f2_pack(ex2(y0), ex2(y1)));
        }
      } else {
#pragma unroll
        for (int k = 0; k < kQT / 4; ++k) {
          const float4 l = nlse[k];
          const int4 i = pos[k];
          const uint32_t* s = &v[k >> 3][4 * (k & 7)];
          auto one = [&](uint32_t sv, float lv, int iv) {
            const float p = ex2(fmaf(__uint_as_float(sv), P.scale_log2, lv));
            return iv >= vis.lo && iv <= vis.hi ? p : 0.f;
          };
          sum[0] = f2_add(sum[0], f2_pack(one(s[0], l.x, i.x), one(s[1], l.y, i.y)));
          sum[1] = f2_add(sum[1], f2_pack(one(s[2], l.z, i.z), one(s[3], l.w, i.w)));
        }
      }
    }
    if (ok && kp < P.S) {
      float x, y;
      f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), x, y);
      W.part[(((long long)part * P.Bt + bt) * P.Hkv + g) * P.S + kp] = x + y;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, L::kTmem);
}

// weight[i] = the parts' sum, in order.
__global__ void __launch_bounds__(256)
key_weights_sum_kernel(const float* __restrict__ part, float* __restrict__ weight, long long n,
                       int parts) {
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    float s = 0.f;
    for (int p = 0; p < parts; ++p) s += __ldg(part + p * n + i);
    weight[i] = s;
  }
}

// CUDA cores: 64 keys per block, query tiles of 64 in 32-channel slices;
// thread (ty, tx) of 16 x 16 owns 4 keys x 4 queries.
template <typename T, int D>
__global__ void __launch_bounds__(256) key_weights_simt_kernel(const WeightParams W, float* weight) {
  constexpr int kT = 64, kC = 32;
  __shared__ float ks[kC][kT + 4], qs[kC][kT + 4];
  __shared__ float red[16][kT + 1];
  const AttnParams& P = W.P;
  const int g = blockIdx.y, bt = blockIdx.z, key0 = blockIdx.x * kT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const T* k = static_cast<const T*>(P.k) + ((long long)bt * P.S * P.Hkv + g) * D;
  Seen vis[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int kp = key0 + 4 * ty + a;
    vis[a] = kp < P.S ? seen_by(P, nat_pos(P, kp)) : Seen{1, 0};
  }
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int q0 = 0; q0 < P.S; q0 += kT) {
    int pos[4];
    bool any = false;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      pos[c] = observed_pos(W, q0 + 4 * tx + c);
#pragma unroll
      for (int a = 0; a < 4; ++a) any |= pos[c] >= vis[a].lo && pos[c] <= vis[a].hi;
    }
    if (!__syncthreads_or(any)) continue;
    for (int h = g * P.G; h < (g + 1) * P.G; ++h) {
      const T* q = static_cast<const T*>(P.q) + ((long long)bt * P.S * P.Hq + h) * D;
      float acc[4][4] = {};
      for (int d0 = 0; d0 < D; d0 += kC) {
        __syncthreads();
        for (int i = threadIdx.x; i < kT * kC / 4; i += 256) {
          const int r = i / (kC / 4), c = (i % (kC / 4)) * 4;
          float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
          if (key0 + r < P.S) load_row<T, 4>(k + (long long)(key0 + r) * P.Hkv * D + d0 + c, x);
          if (q0 + r < P.S) load_row<T, 4>(q + (long long)(q0 + r) * P.Hq * D + d0 + c, y);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ks[c + e][r] = x[e];
            qs[c + e][r] = y[e];
          }
        }
        __syncthreads();
#pragma unroll 8
        for (int d = 0; d < kC; ++d) {
          const float4 x = *reinterpret_cast<const float4*>(&ks[d][4 * ty]);
          const float4 y = *reinterpret_cast<const float4*>(&qs[d][4 * tx]);
          const float xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[a][c] = fmaf(xa[a], ya[c], acc[a][c]);
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (pos[c] < 0) continue;
        const float lse = __ldg(P.lse + lse_index(P, bt, h, q0 + 4 * tx + c));
        if (lse == -INFINITY) continue;
#pragma unroll
        for (int a = 0; a < 4; ++a)
          if (pos[c] >= vis[a].lo && pos[c] <= vis[a].hi)
            sum[a] += exp2f((acc[a][c] * P.scale - lse) * kLog2e);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < 4; ++a) red[tx][4 * ty + a] = sum[a];
  __syncthreads();
  if (threadIdx.x < kT && key0 + threadIdx.x < P.S) {
    float s = 0.f;
    for (int i = 0; i < 16; ++i) s += red[i][threadIdx.x];
    weight[((long long)bt * P.Hkv + g) * P.S + key0 + threadIdx.x] = s;
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// [Bt][S][H][D] bf16 -> 4-D map (D, H, S, Bt), box (64, 1, rows, 1), 128-byte
// swizzle; rows behind S read as zeros.
bool make_map(CUtensorMap* m, const void* base, int Bt, int S, int H, int D, int rows) {
  auto fn = encode_fn();
  if (!fn) {
    fail_cuda_msg("cuTensorMapEncodeTiled", "driver entry point not found");
    return false;
  }
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)Bt};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2, (cuuint64_t)S * H * D * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)rows, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                  box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    char msg[64];
    std::snprintf(msg, sizeof(msg), "CUresult %d", (int)r);
    fail_cuda_msg("cuTensorMapEncodeTiled", msg);
    return false;
  }
  return true;
}

// How the problem is cut (host side, from the shapes alone).
struct Cut {
  int hpi, nseg, tps, nkb, q0, ntiles, parts;
};
// tail: the observed queries are the last rows (natural order, one sequence).
Cut cut_of(int B, int S, int Hq, int Hkv, int observe, bool tail) {
  Cut c{};
  const int G = Hq / Hkv;
  if (observe >= S) observe = 0;
  c.q0 = observe > 0 && tail ? S - observe : 0;
  c.ntiles = (S - c.q0 + kQT - 1) / kQT;
  // query tiles that a key block meets at most, of one sequence
  const int all = (S + kQT - 1) / kQT;
  const int tiles = observe > 0 ? std::min((observe + kQT - 1) / kQT + 1, all) : all;
  c.nkb = (S + kKeys - 1) / kKeys;
  c.hpi = G;
  c.nseg = 1;
  const long long blocks = (long long)c.nkb * Hkv * B;
  const long long want = 8LL * 304;  // CTAs that even out what the masks leave
  if (blocks < want && tiles >= 16) {  // (each CTA loads its keys anew)
    c.hpi = 1;
    const long long have = blocks * G;
    if (have < want && observe == 0) {
      long long n = (want + have - 1) / have;
      const long long most = (tiles + 15) / 16;  // at least 16 tiles each
      if (n > most) n = most;
      if (n > 16) n = 16;
      c.nseg = (int)n;
    }
  }
  c.tps = (c.ntiles + c.nseg - 1) / c.nseg;
  c.parts = (G / c.hpi) * c.nseg;
  return c;
}

template <int D>
usp_status_t launch_tc(const WeightParams& W, cudaStream_t st) {
  const AttnParams& P = W.P;
  using L = WSmem<D>;
  CUtensorMap mq;
  if (!make_map(&mq, P.q, P.Bt, P.S, P.Hq, D, kQT)) return USP_ERR_CUDA;
  const int smem = L::kAlloc;
  cudaError_t e = cudaFuncSetAttribute(key_weights_tc_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return fail_cuda("cudaFuncSetAttribute(smem)", e);
  const long long blocks = (long long)W.nkb * P.Bt * P.Hkv * (P.G / W.hpi) * W.nseg;
  if (blocks > 0x7fffffffLL) return USP_ERR_UNSUPPORTED;
  {
    ProfScope ps(st, "attn_key_weights");
    key_weights_tc_kernel<D><<<(unsigned)blocks, kThreads, smem, st>>>(W, mq);
  }
  note_launch();
  return check_launch();
}

}  // namespace

size_t key_weights_workspace(int B, int S, int Hq, int Hkv, int observe) {
  const Cut c = cut_of(B, S, Hq, Hkv, observe, false);  // (parts do not depend on `tail`)
  return c.parts > 1 ? (size_t)c.parts * B * Hkv * S * 4 : 0;
}

usp_status_t launch_key_weights_tc(const AttnParams& P, float* weight, int observe,
                                   void* workspace, cudaStream_t st) {
  const Cut c = cut_of(P.Bt, P.S, P.Hq, P.Hkv, observe, P.layout == kContiguous && !P.cu);
  WeightParams W{P, c.parts > 1 ? static_cast<float*>(workspace) : weight,
                 observe < P.S ? observe : 0, c.hpi, c.nseg, c.tps, c.nkb, c.q0, c.ntiles};
  usp_status_t r = P.D == 128 ? launch_tc<128>(W, st) : launch_tc<64>(W, st);
  if (r != USP_OK || c.parts == 1) return r;
  const long long n = (long long)P.Bt * P.Hkv * P.S;
  const long long blocks = (n + 255) / 256;
  {
    ProfScope ps(st, "attn_key_weights_sum");
    key_weights_sum_kernel<<<(unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), 256, 0, st>>>(
        W.part, weight, n, c.parts);
  }
  note_launch();
  return check_launch();
}

usp_status_t launch_key_weights_simt(const AttnParams& P, float* weight, int observe, int bf16,
                                     cudaStream_t st) {
  WeightParams W{P, nullptr, observe, P.G, 1, 0, 0, 0};
  const dim3 grid((P.S + 63) / 64, P.Hkv, P.Bt);
  {
    ProfScope ps(st, "attn_key_weights_simt");
    if (bf16) {
      if (P.D == 128) key_weights_simt_kernel<__nv_bfloat16, 128><<<grid, 256, 0, st>>>(W, weight);
      else key_weights_simt_kernel<__nv_bfloat16, 64><<<grid, 256, 0, st>>>(W, weight);
    } else {
      if (P.D == 128) key_weights_simt_kernel<float, 128><<<grid, 256, 0, st>>>(W, weight);
      else key_weights_simt_kernel<float, 64><<<grid, 256, 0, st>>>(W, weight);
    }
  }
  note_launch();
  return check_launch();
}

int read_clear_key_weights_status() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_key_weights_status, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0) cudaMemcpyToSymbol(g_key_weights_status, &z, sizeof(int));
  return v;
}

}  // namespace usp
