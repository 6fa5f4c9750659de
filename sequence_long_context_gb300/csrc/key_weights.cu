// How much each key of a prompt was attended: column sums of the attention
// matrix, from the forward's q, k and LSE.
//
//     weight[g][j] = sum over query heads h of group g and observed queries i
//                    that see key j of exp(scale <q_i,h, k_j> - LSE_i,h)
// ("Long Context Attention" notes, "Motivation": the LSE is what the forward
// keeps; with it a probability needs no second pass over its row.)
//
// Tensor-core kernel (bf16). S^T = K Q^T, keys on the 128 TMEM lanes, so that a
// softmax thread owns a key and the column sum is a register. Nothing is
// normalised or rescaled, and nothing goes back to the tensor core. An item of
// work is 256 keys (two tiles of 128) of one KV head with the query tiles of
// 128 that may see them, for some of the group's query heads and a segment of
// the queries; one CTA per SM takes items in turn, and its roles run ahead of
// one another across items. Where an item's query tiles fit beside the keys
// (few observed queries) they stay, and an item is a run of key blocks: 64
// observed queries of a 32K prompt, 32 heads of 8, take 27 us called one by one (23
// replayed from a graph, 3.0 TB/s), and 36 with their queries and statistics
// prepared anew for every 256 keys.
// What bounds it: per 128 x 128 tile (D = 128) the products take 512 clocks
// (616 with both operands from shared memory, 64 KB), the exponentials (32 per
// clock and SM) 512, and what a tile needs besides, waits on barriers and
// tensor memory's latency, about 1500 per buffer of scores. So scores have
// four 128-column buffers (all of tensor memory) and each key tile two groups
// of softmax warps, which take its query tiles in turn: fewer or smaller
// buffers left the tensor core and the exponentials idle two thirds of the
// time (8K prompt, zigzag ring of 8, 32 heads of 8: 262 us, 1.05 PFLOP/s; 314
// with one buffer per key tile of 512 keys, 320 with keys in tensor memory and
// 64 columns). A 128 x 256 tile now takes 1.15 us, the exponentials half of it:
// a warp that reads its next scores ahead needs code that is slower (below).
// Roles (640 threads):
//   warps 0-15 softmax: warp w takes keys [32 (w & 7), + 32) and every other
//              query tile (w >> 3: which), from a score buffer that its four
//              warps have to themselves
//   warp 16    items and keys: counts the query tiles that can see an item's
//              keys (32 at a time, one per lane), publishes the item and loads
//              its K (a ring of two to four tiles, the next block's ahead of time)
//   warp 17    queries: loads an item's Q tiles (two to four slots) and, with all
//              lanes, their LSE (asked for one tile ahead) and positions. (One
//              warp for 16 and 17 took 4.2 us per item, which with few
//              queries was all the time there is.)
//   warps 18, 19  MMA issuers, one per key tile (what a warp waits between its
//              products the other fills); 18 owns tensor memory
// Positions are read per query from shared memory, so a tile may cross chunk
// and shard boundaries: any layout and any length has this kernel. (Where chunks are
// no multiple of 128 the bounds of a tile are found row by row: a zigzag ring of 8
// over 7760 tokens, chunks of 485, takes 734 us, the same prompt in natural order
// 231.)
//
// The partial sums of several heads or segments go to the workspace and are
// added in a fixed order by a second kernel.
//
// CUDA-core kernel (fp32 inputs, and as a cross-check): 64 x 64 tiles. 8K tokens, 32
// heads of 8: 11.6 ms; 64 observed queries of 32K: 3.8 ms (every query tile is
// looked at).
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdio>

#include "internal.h"
#include "kv4_host.h"
#include "tc_ptx.cuh"
#include "tile_sched.cuh"

namespace usp {
namespace {

using namespace tc;

__device__ int g_key_weights_status = 0;

constexpr int kQT = 128;            // queries per tile
constexpr int kKT = 2;              // key tiles per block of keys
constexpr int kKeys = kKT * kTile;  // keys per block
constexpr int kSoftWarps = 8 * kKT; // two groups of four per key tile
constexpr int kKeyWarp = kSoftWarps;
constexpr int kQueryWarp = kKeyWarp + 1;
constexpr int kMmaWarp = kQueryWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + kKT);
// Tiles of K and Q in shared memory: three each; where no item has more than two
// query tiles two of Q and four of K, and where none has more than four, four of
// Q and two of K. An item's query tiles then stay while a run of key blocks
// passes, if they are the same tiles for all of them.
constexpr int kTileSlots = 6;
constexpr int kSlots = 4;           // Q tiles, at most
constexpr int kKSlots = 4;          // K tiles, at most
constexpr int kSBufs = 2 * kKT;     // score buffers of 128 columns: one per softmax group
constexpr int kRing = 16;           // entries of query statistics
constexpr int kCtas = 152;          // one per SM
constexpr int kRecords = 4;         // items that the roles may be apart
constexpr int kJoins = 2;           // key blocks that the softmax groups may be apart
constexpr int kDiag = 1 << 16;
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
  int hpi;       // query heads per item
  int groups;    // items per KV head, key block and segment: G / hpi
  int nseg;      // segments: which of a key block's query tiles, in turn
  int nkb;       // key blocks
  int q0;        // first row of tile 0: where the observed rows begin, if they
                 // are one run to the end; else 0
  int ntiles;    // query tiles
  int pair;      // 2: one tile of at most 64 rows, two heads share the 128; else 1
  int qslots, kslots;
  int run;       // key blocks per item
  int items;
};

template <int D>
struct WSmem {
  // A ring entry is written for tile x once both MMA warps have released tile
  // y = x - kSlots (or later) in the last block of its item. One that multiplied it
  // there had its two buffers emptied of all but the tile before, which is y - 1 or
  // of y's item; one without keys there has waited until both were empty. So the
  // softmax groups use no entry before y's item, nor, in an item of one block,
  // before y - 1; and an item of several blocks has at most kSlots tiles.
  static_assert(kRing > 2 * kSlots, "a statistics entry is free");
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = kTile * 128;             // 64 channels of a K or Q tile
  static constexpr int kTileBytes = kHalf * kHalves;
  static constexpr int kK = 0;                          // kslots tiles of K, then Q
  static constexpr int kStat = kTileSlots * kTileBytes;  // kRing x (-lse2[128], pos[128])
  static constexpr int kStatBytes = 2 * kQT * 4;
  static constexpr int kJoin = kStat + kRing * kStatBytes;  // [kJoins][kKeys] sums of group 0
  static constexpr int kSched = kJoin + kJoins * kKeys * 4;  // kRing ints: class | rows << 8 | kDiag
  static constexpr int kItem = kSched + kRing * 4;      // [kRecords] ItemRecord
  static constexpr int kBar = kItem + kRecords * 16;
  static constexpr int kKFull = 0, kKFree = kKFull + kKSlots, kQFull = kKFree + kKSlots,
                       kQFree = kQFull + kSlots, kSFull = kQFree + kSlots,
                       kSFree = kSFull + kSBufs, kItemFull = kSFree + kSBufs, kItemFree = kItemFull + kRecords,
                       kJoinFull = kItemFree + kRecords /* [kJoins][kKT] */,
                       kJoinFree = kJoinFull + kJoins * kKT,
                       kMmaDone = kJoinFree + kJoins * kKT,
                       kNumBars = kMmaDone + kKT;
  static constexpr int kMisc = (kBar + 8 * kNumBars + 15) / 16 * 16;
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "exceeds the per-CTA shared memory limit");
  static_assert(kBar % 8 == 0 && kStat % 16 == 0 && kItem % 16 == 0, "alignment");
};

// What the roles know of an item: the number of (query tile, head) pairs, or
// kEnd, and which item it is.
struct ItemRecord {
  int count, item, pad[2];
};
struct ItemPos {
  int part, g, bt, key0, h0, seg;
  int blocks;  // of keys
};
// Key tiles of the block at key0 with keys in them.
__device__ __forceinline__ int ktiles_of(const AttnParams& P, int key0) {
  return min(kKT, (P.S - key0 + kTile - 1) / kTile);
}
__device__ __forceinline__ ItemPos item_pos(const WeightParams& W, int item) {
  const AttnParams& P = W.P;
  // key blocks outermost: with a causal mask the heaviest (first) start first
  const int groups = W.groups;
  ItemPos r;
  r.part = r.g = r.bt = 0;
  if (groups * W.nseg > 1) {
    r.part = item % (groups * W.nseg);
    item /= groups * W.nseg;
  }
  if (P.Hkv > 1) {
    r.g = item % P.Hkv;
    item /= P.Hkv;
  }
  if (P.Bt > 1) {
    r.bt = item % P.Bt;
    item /= P.Bt;
  }
  // ... in natural order, where a block of keys is one
  r.key0 = item * W.run * kKeys;
  r.blocks = min(W.run, W.nkb - item * W.run);
  if (P.layout == kZigzag && P.chunk % kKeys == 0) r.key0 = permuted_of(P, r.key0);
  r.seg = r.part / groups;
  r.h0 = r.g * P.G + (r.part - r.seg * groups) * W.hpi;
  return r;
}

// The queries that see the key at natural position j, as positions [lo, hi]; none
// where a packed batch has no sequence there.
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen seen_by(const AttnParams& P, int j) {
  int s = 0, e = P.S;
  if (P.cu != nullptr) {
    const int n = seg_of(P.cu, P.nseq, j);
    s = __ldg(P.cu + n);
    e = __ldg(P.cu + n + 1);
    if (j < s || j >= e) return Seen{1, 0};
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
  if (P.layout == kContiguous) {
    r.lo = p0;
    r.hi = p1;
    return r;
  }
  const int run = P.layout == kZigzag ? P.chunk : P.shard;
  if (p0 / run == p1 / run) {
    r.lo = nat_pos(P, p0);
    r.hi = nat_pos(P, p1);
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
  int begin, end; // of them
};
__device__ __forceinline__ KeyBlock key_block(const AttnParams& P, int key0, int blocks) {
  KeyBlock b;
  b.k = row_bounds(P, key0, blocks * kKeys);
  int s0 = 0, e1 = P.S;
  b.seg0 = b.seg1 = 0;
  if (P.cu != nullptr) {
    b.seg0 = seg_of(P.cu, P.nseq, b.k.lo);
    b.seg1 = seg_of(P.cu, P.nseq, b.k.hi);
    s0 = __ldg(P.cu + b.seg0);
    e1 = __ldg(P.cu + b.seg1 + 1);
  }
  b.begin = s0;
  b.end = e1;
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
  bool all = true;  // rows behind S have no position, which the query warp sees
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
    // (rows outside the boundaries count as the first or last sequence's)
    if (min(q.lo, b.k.lo) < b.begin || max(q.hi, b.k.hi) >= b.end) return kClsMasked;
  }
  if (P.causal && b.k.hi > q.lo) all = false;
  if (P.window > 0 && q.hi - b.k.lo >= P.window) all = false;
  return all ? kClsFull : kClsMasked;
}

// 20 warps: five share a 16K-register sub-partition, so <= 102 each (96 in the
// allocation's steps of 8).
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
key_weights_tc_kernel(const WeightParams W, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k) {
  using L = WSmem<D>;
  const AttnParams& P = W.P;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(sm);
  auto bar = [&](int i) { return sbase + L::kBar + 8 * i; };
  volatile int* sched = reinterpret_cast<volatile int*>(sm + L::kSched);
  volatile ItemRecord* record = reinterpret_cast<volatile ItemRecord*>(sm + L::kItem);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  int* status = &g_key_weights_status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qslots = W.qslots, kslots = W.kslots;
  const uint32_t q_at = sbase + kslots * L::kTileBytes;  // the Q tiles

  if (warp == kKeyWarp && lane == 0) {
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(bar(L::kKFull + s), 1);
      mbar_init(bar(L::kKFree + s), kKT);  // both MMA warps
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(L::kQFull + s), 1);
      mbar_init(bar(L::kQFree + s), kKT);  // both MMA warps
    }
    for (int s = 0; s < kSBufs; ++s) {
      // the products' commit, and the MMA warp's own arrival: it has seen the
      // tile's statistics (behind the Q tile's barrier), so the softmax may
      mbar_init(bar(L::kSFull + s), 2);
      mbar_init(bar(L::kSFree + s), 4);  // the four warps that take it
    }
    for (int s = 0; s < kRecords; ++s) {
      mbar_init(bar(L::kItemFull + s), 1);
      mbar_init(bar(L::kItemFree + s), kSoftWarps + kKT + 1);  // MMA, queries
    }
    for (int s = 0; s < kJoins * kKT; ++s) {
      mbar_init(bar(L::kJoinFull + s), 4);
      mbar_init(bar(L::kJoinFree + s), 4);
    }
    for (int a = 0; a < kKT; ++a) mbar_init(bar(L::kMmaDone + a), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch(&tm_q);
    tma_prefetch(&tm_k);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sbase + L::kMisc, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  // query tiles first, first + nseg .. < last of an item's segment may see its keys
  auto tiles_of = [&](const ItemPos& ip, const KeyBlock& blk, int& first, int& last) {
    first = 0;
    last = W.ntiles;
    if (P.layout == kContiguous) {  // rank-major order is natural order
      first = max(0, (blk.q.lo - W.q0) / kQT);  // (towards 0: an extra tile is skipped)
      last = blk.q.hi < W.q0 ? 0 : min(last, (blk.q.hi - W.q0) / kQT + 1);
    }
    first += ip.seg;
  };
  if (warp == kKeyWarp) {
    // ------------------------------------------------------- items and keys
    bool ok = true;
    int kn = 0, kslot = 0, kphase = 1;  // K tiles (the first waits are skipped)
    for (int it = 0; ok; ++it) {
      // the items are sorted by their work as far as the mask goes: there and
      // back, every CTA gets its share
      const long long at = (long long)it * gridDim.x +
                           ((it & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      const int item = (int)at;
      const bool end = at >= W.items;
      const ItemPos ip = item_pos(W, end ? 0 : item);
      const KeyBlock blk = key_block(P, ip.key0, ip.blocks);
      int first, last;
      tiles_of(ip, blk, first, last);
      int tiles = 0;
      for (int base = first; base < last; base += 32 * W.nseg) {
        const int t = base + lane * W.nseg;
        tiles += __popc(__ballot_sync(
            0xffffffffu, t < last && classify_tile(W, t, blk) != kClsEmpty));
      }
      const int rec = it % kRecords;
      if (it >= kRecords) {  // every role is done with the record's previous item
        ok = mbar_wait(bar(L::kItemFree + rec), (it / kRecords - 1) & 1, abort_flag, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
      }
      if (lane == 0) {
        record[rec].count = end ? kEnd : tiles * (W.hpi / W.pair);
        record[rec].item = item;
        mbar_arrive(bar(L::kItemFull + rec));
      }
      if (end) break;
      if (tiles == 0) continue;
      for (int x = 0; ok && x < ip.blocks; ++x) {
        const int key0 = ip.key0 + x * kKeys, ktiles = ktiles_of(P, key0);
        for (int a = 0; ok && a < ktiles; ++a) {
          if (kn >= kslots) {  // the slot's previous keys have been multiplied
            ok = mbar_wait(bar(L::kKFree + kslot), kphase, abort_flag, status);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
          }
          if (lane == 0) {
            mbar_expect_tx(bar(L::kKFull + kslot), L::kTileBytes);
            for (int hf = 0; hf < L::kHalves; ++hf)
              tma_load_4d(sbase + L::kK + kslot * L::kTileBytes + hf * L::kHalf, &tm_k,
                          bar(L::kKFull + kslot), hf * 64, ip.g, key0 + a * kTile, ip.bt);
          }
          ++kn;
          if (++kslot == kslots) {
            kslot = 0;
            kphase ^= 1;
          }
        }
      }
    }
    // aborted: the copies in flight land before the CTA ends
    if (lane == 0 && *abort_flag)
      for (int i = kn > kslots ? kn - kslots : 0; i < kn; ++i)
        mbar_wait_drain(bar(L::kKFull + i % kslots), (i / kslots) & 1);
  } else if (warp == kQueryWarp) {
    // ------------------------------------------------------------- queries
    bool ok = true;
    int n = 0, slot = 0, phase = 1;  // Q tiles (the first waits are skipped)
    const int step = P.layout == kStripe ? P.cp : 1;
    const int run = P.layout == kZigzag ? P.chunk : P.shard;
    const int from = W.observe > 0 ? P.S - W.observe : 0;
    for (int it = 0; ok; ++it) {
      const int rec = it % kRecords;
      ok = mbar_wait(bar(L::kItemFull + rec), (it / kRecords) & 1, abort_flag, status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int count = record[rec].count;
      const ItemPos ip = item_pos(W, record[rec].item);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kItemFree + rec));  // the record has been read
      if (count == kEnd) break;
      if (count == 0) continue;
      const KeyBlock blk = key_block(P, ip.key0, ip.blocks);
      int first, last;
      tiles_of(ip, blk, first, last);
      // The next (tile, head), its rows' positions and LSE. This runs once per
      // tile in one warp, so it is kept short: what takes divisions is found
      // for 32 tiles at a time, one per lane.
      struct Next {
        int row, cls, h, pos[kQT / 32];  // row: the tile's first
        float lse[kQT / 32];
      };
      const float* lse_head = P.lse + lse_index(P, ip.bt, ip.h0, 0);
      int base = first - 32 * W.nseg, cls_mine = kClsEmpty, lo_mine = 0, hh = 0;
      unsigned todo = 0;
      Next nx{};
      bool more = true;
      auto fetch = [&]() {
        if (hh == 0) {  // a new tile
          while (todo == 0 && (base += 32 * W.nseg) < last) {
            const int t = base + lane * W.nseg;
            cls_mine = t < last ? classify_tile(W, t, blk) : kClsEmpty;
            todo = __ballot_sync(0xffffffffu, cls_mine != kClsEmpty);
            // first position, or -1: the rows are not one run of a chunk, or
            // which are observed depends on the sequence
            lo_mine = -1;
            if (cls_mine != kClsEmpty && (W.observe == 0 || P.cu == nullptr)) {
              const int p0 = W.q0 + t * kQT, p1 = min(p0 + kQT, P.S) - 1;
              if (P.layout == kContiguous || p0 / run == p1 / run) lo_mine = nat_pos(P, p0);
            }
          }
          if (todo == 0) {
            more = false;
            return;
          }
          const int src = __ffs(todo) - 1;
          todo &= todo - 1;
          nx.row = W.q0 + (base + src * W.nseg) * kQT;
          nx.cls = __shfl_sync(0xffffffffu, cls_mine, src);
          const int lo = __shfl_sync(0xffffffffu, lo_mine, src);
#pragma unroll
          for (int e = 0; e < kQT / 32; ++e) {
            const int r = W.pair == 2 ? lane + 32 * (e & 1) : lane + 32 * e;
            if (lo >= 0) {
              const int i = lo + r * step;
              nx.pos[e] = nx.row + r < P.S && i >= from ? i : kNowhere;
            } else {
              nx.pos[e] = observed_pos(W, nx.row + r);
            }
          }
        }
        nx.h = ip.h0 + hh;
        const float* src_lse = lse_head + hh * P.lse_sh + nx.row + lane;
#pragma unroll
        for (int e = 0; e < kQT / 32; ++e) {
          const float* at = W.pair == 2 ? src_lse + (e >> 1) * P.lse_sh + 32 * (e & 1) : src_lse + 32 * e;
          nx.lse[e] = nx.pos[e] >= 0 ? __ldg(at) : 0.f;
        }
        hh += W.pair;
        if (hh == W.hpi) hh = 0;
      };
      fetch();
      while (more) {
        const Next cur = nx;
        fetch();  // its loads are on their way during this tile's waits
        if (n >= qslots) {  // the slot's previous tile has been multiplied
          ok = mbar_wait(bar(L::kQFree + slot), phase, abort_flag, status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        const int ring = n & (kRing - 1), rows = W.pair == 2 ? kQT : min(kQT, P.S - cur.row);
        float* st = reinterpret_cast<float*>(sm + L::kStat + ring * L::kStatBytes);
        bool skips = false;
#pragma unroll
        for (int e = 0; e < kQT / 32; ++e) {
          const float x = cur.lse[e] * kLog2e;
          // a row that sees nothing adds nothing, whatever it holds: its
          // position is nowhere, and the tile's positions are looked at
          const bool none = cur.pos[e] < 0 || x == -INFINITY;
          skips |= cur.pos[e] >= 0 && none;
          st[lane + 32 * e] = none ? -INFINITY : -x;
          reinterpret_cast<int*>(st)[kQT + lane + 32 * e] = none ? kNowhere : cur.pos[e];
        }
        skips = __any_sync(0xffffffffu, skips);
        // where causality alone hides keys, of a run's last blocks only
        const bool diag = !skips && W.run > 1 && P.causal && P.window == 0;
        if (lane == 0)
          sched[ring] = (skips ? kClsMasked : cur.cls) | rows << 8 | (diag ? kDiag : 0);
        __syncwarp();
        if (lane == 0) {
          // 64 rows at a time; the barrier stands for the ring's entry too
          const int boxes = rows > 64 ? 2 : 1;
          mbar_expect_tx(bar(L::kQFull + slot), L::kTileBytes / 2 * boxes);
          for (int r = 0; r < boxes; ++r)
            for (int hf = 0; hf < L::kHalves; ++hf)
              tma_load_4d(q_at + slot * L::kTileBytes + hf * L::kHalf + r * (L::kHalf / 2),
                          &tm_q, bar(L::kQFull + slot), hf * 64,
                          W.pair == 2 ? cur.h + r : cur.h, W.pair == 2 ? cur.row : cur.row + 64 * r,
                          ip.bt);
        }
        ++n;
        if (++slot == qslots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    // aborted: the copies in flight land before the CTA ends
    if (lane == 0 && *abort_flag)
      for (int i = n > qslots ? n - qslots : 0; i < n; ++i)
        mbar_wait_drain(bar(L::kQFull + i % qslots), (i / qslots) & 1);
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------ MMA issuers
    // Every lane runs the loop and one elected lane issues: the descriptors
    // then are uniform values, which the issue takes as they are. (In a loop
    // of one lane alone each of its operands is first moved to a uniform
    // register, 76 clocks per product.)
    constexpr uint32_t kId128 = idesc_bf16_f32(kTile, 128, 0, 0);
    constexpr uint32_t kId64 = idesc_bf16_f32(kTile, 64, 0, 0);
    const uint64_t dk = sdesc_sw128(sbase + L::kK, 16, 1024);
    const uint64_t dq = sdesc_sw128(q_at, 16, 1024);
    const uint32_t t0 = __shfl_sync(0xffffffffu, tmem, 0);
    const int a = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0);  // key tile
    bool ok = true;
    // Score buffer a + kKT g is written by this warp and read by key tile a's
    // softmax group g alone, so each side sees every one of its phases (a parity
    // cannot tell a phase from the one two before it). The groups take the tiles in
    // turn, over the ends of blocks and items.
    int n = 0, slot = 0, phase = 0, kn = 0, pairs = 0, used0 = 0, used1 = 0;
    for (int it = 0; ok; ++it) {
      const int rec = it % kRecords;
      ok = mbar_wait(bar(L::kItemFull + rec), (it / kRecords) & 1, abort_flag, status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int count = __shfl_sync(0xffffffffu, record[rec].count, 0);
      const int item = __shfl_sync(0xffffffffu, record[rec].item, 0);
      if (count == kEnd) break;
      const ItemPos ip = item_pos(W, item);
      const int slot0 = slot, phase0 = phase;
      for (int x = 0; x < ip.blocks && count > 0 && ok; ++x) {
        const int ktiles = ktiles_of(P, ip.key0 + x * kKeys);
        const bool last = x + 1 == ip.blocks;
        slot = slot0;
        phase = phase0;
        // The ring's slots go from one key tile to the other: this warp sees and
        // frees the other tile too (it has landed by the time that its own has, or
        // been multiplied by), so that it knows every phase of every slot.
        auto pass_tile = [&](int other) {
          const int ks = (kn + other) % kslots;
          ok = mbar_wait(bar(L::kKFull + ks), ((kn + other) / kslots) & 1, abort_flag, status);
          ok = __all_sync(0xffffffffu, ok);
          if (ok && lane == 0) mbar_arrive(bar(L::kKFree + ks));
        };
        if (a > 0) pass_tile(0);
        // A warp without keys in this block releases the queries as fast as they
        // come, and the statistics ring with them: its groups first take out what
        // they were given before.
        if (ok && a >= ktiles) {
          if (used0 > 0)
            ok = mbar_wait(bar(L::kSFree + a), (used0 - 1) & 1, abort_flag, status);
          if (ok && used1 > 0)
            ok = mbar_wait(bar(L::kSFree + a + kKT), (used1 - 1) & 1, abort_flag, status);
          ok = __all_sync(0xffffffffu, ok);
        }
        for (int j = 0; j < count && ok; ++j) {
          ok = mbar_wait(bar(L::kQFull + slot), phase, abort_flag, status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          const int rows = __shfl_sync(0xffffffffu, sched[(n + j) & (kRing - 1)], 0) >> 8 & 255;
          const uint32_t id = rows > 64 ? kId128 : kId64;
          if (a < ktiles) {
            const int g = (pairs + j) & 1, used = g ? used1 : used0;
            const int ks = (kn + a) % kslots, buf = a + kKT * g;
            if (j == 0) ok = mbar_wait(bar(L::kKFull + ks), ((kn + a) / kslots) & 1, abort_flag, status);
            // the buffer's previous scores have been taken out
            if (ok && used > 0)
              ok = mbar_wait(bar(L::kSFree + buf), (used - 1) & 1, abort_flag, status);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            if (g) ++used1;
            else ++used0;
            if (lane == 0) mbar_arrive(bar(L::kSFull + buf));
            tc_fence_after();
            const uint64_t da = sdesc_add(dk, ks * L::kTileBytes);
            const uint64_t db = sdesc_add(dq, slot * L::kTileBytes);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * L::kHalf + (kk & 3) * 32;
                mma_ss(t0 + 128 * buf, sdesc_add(da, off), sdesc_add(db, off), id, kk > 0 ? 1u : 0u);
              }
              mma_commit(bar(L::kSFull + buf));
              if (j + 1 == count) mma_commit(bar(L::kKFree + ks));
              if (last) mma_commit(bar(L::kQFree + slot));
            }
          } else if (last && elect_one()) {
            // no such key tile, but products of the blocks before may still read
            // the slot: it is free once those of this thread are done
            mma_commit(bar(L::kQFree + slot));
          }
          __syncwarp();
          if (++slot == qslots) {
            slot = 0;
            phase ^= 1;
          }
        }
        if (ok && a + 1 < ktiles) pass_tile(a + 1);
        kn += ktiles;
        pairs += count;
      }
      n += count;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kItemFree + rec));
    }
    if (elect_one()) mma_commit(bar(L::kMmaDone + a));
    mbar_wait_drain(bar(L::kMmaDone + a), 0);
  } else {
    // ------------------------------------------------------------ softmax
    const int a = (warp >> 2) & 1, group = warp >> 3;  // key tile, which of its groups
    const int buf = a + kKT * group;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint64_t sc2 = f2_pack(P.scale_log2, P.scale_log2);
    bool ok = true;
    int n = 0, pairs = 0, used = 0, joins = 0;
    for (int it = 0; ok; ++it) {
      const int rec = it % kRecords;
      ok = mbar_wait(bar(L::kItemFull + rec), (it / kRecords) & 1, abort_flag, status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int count = record[rec].count, item = record[rec].item;
      if (count == kEnd) break;
      const ItemPos ip = item_pos(W, item);
      for (int x = 0; x < ip.blocks; ++x) {
        const int key0 = ip.key0 + x * kKeys, ktiles = ktiles_of(P, key0);
        if (a < ktiles) {
          const int kp = key0 + (warp & 7) * 32 + lane;
          Seen vis{1, 0};
          if (kp < P.S) vis = seen_by(P, nat_pos(P, kp));
          uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
          for (int j = (pairs ^ group) & 1; j < count; j += 2, ++used) {
            const int ring = (n + j) & (kRing - 1);
            ok = mbar_wait(bar(L::kSFull + buf), used & 1, abort_flag, status);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            const uint32_t t_s = tmem + lane_off + 128 * buf;
            const float4* nlse = reinterpret_cast<const float4*>(sm + L::kStat + ring * L::kStatBytes);
            const int entry = sched[ring], rows = entry >> 8 & 255;
            int cls = entry & 255;
            if ((entry & kDiag) && key0 + kKeys - 1 <= reinterpret_cast<const int*>(nlse)[kQT])
              cls = kClsFull;  // before the tile's first query
            auto add = [&](const uint32_t(&v)[32], const float4* nl) {
              if (cls == kClsFull) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float4 l = nl[k];
                  const uint32_t* s = &v[4 * k];
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
                const int4* pos = reinterpret_cast<const int4*>(nl + kQT / 4);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float4 l = nl[k];
                  const int4 i = pos[k];
                  const uint32_t* s = &v[4 * k];
                  auto one = [&](uint32_t sv, float lv, int iv) {
                    const float p = ex2(fmaf(__uint_as_float(sv), P.scale_log2, lv));
                    return iv >= vis.lo && iv <= vis.hi ? p : 0.f;
                  };
                  sum[0] = f2_add(sum[0], f2_pack(one(s[0], l.x, i.x), one(s[1], l.y, i.y)));
                  sum[1] = f2_add(sum[1], f2_pack(one(s[2], l.z, i.z), one(s[3], l.w, i.w)));
                }
              }
            };
            // 32 columns at a time, one copy of the code. (With the next columns
            // loaded ahead it spills, and takes 1.25 to 1.5 times as long; 16
            // columns ahead of 16 do not spill, and take 1.05 times as long: the
            // other warps fill the time.)
            uint32_t v[32];
#pragma unroll 1
            for (int c = 0; c < rows; c += 32) {
              tmem_ld32(t_s + c, v);
              tmem_wait_ld();
              if (c + 32 >= rows) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kSFree + buf));
              }
              add(v, nlse + c / 4);
            }
          }
          if (!ok) break;
          // the two groups' sums, which the second adds: where the first takes the
          // first of an even number of tiles it is done first, and goes on without a wait (`joins`
          // counts this key tile's blocks, alike in both groups)
          float u, w;
          f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), u, w);
          const int jb = joins % kJoins * kKT + a;
          float* join = reinterpret_cast<float*>(sm + L::kJoin) + joins % kJoins * kKeys;
          const int at = (warp & 7) * 32 + lane;
          if (group == 0) {
            if (joins >= kJoins)  // the sums before have been read
              ok = mbar_wait(bar(L::kJoinFree + jb), (joins / kJoins - 1) & 1, abort_flag, status);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            join[at] = u + w;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kJoinFull + jb));
          } else {
            ok = mbar_wait(bar(L::kJoinFull + jb), (joins / kJoins) & 1, abort_flag, status);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const float other = join[at];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kJoinFree + jb));
            if (kp < P.S)
              W.part[(((long long)ip.part * P.Bt + ip.bt) * P.Hkv + ip.g) * P.S + kp] = u + w + other;
          }
          ++joins;
        }
        pairs += count;
      }
      if (!ok) break;
      n += count;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kItemFree + rec));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
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

// Query tiles of a segment, about, at least (4 packed sequences of 5003 tokens, 8
// heads: 48 us uncut, 35 with 16, 40 with 8, 36 with 4; 4K tokens, 8 heads: 29,
// 34, 38 with 16, 8, 4; 2K tokens: 27, 20, 19; a zigzag ring of 4 over 4K: 32, 39,
// 43; and 3 to 4 us for the sum of the segments, where there are any).
constexpr int kMinTiles = 16;
// Pairs of a query tile and a head in an item, at most: a pair takes 1.2 us, and
// roles wait for up to an item's time, so 0.3 s where a wait gives up after 2.
constexpr long long kMaxPairs = 1 << 18;
// How the problem is cut (host side, from the shapes alone).
struct Cut {
  int hpi, nseg, nkb, q0, ntiles, parts;
};
// tail: the observed queries are the last rows (natural order, one sequence).
// nseq: packed sequences, or 0. A key block meets the queries of its own
// sequences alone; a long one is taken to be twice the mean.
Cut cut_of(int B, int S, int Hq, int Hkv, int observe, bool tail, int nseq) {
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
  const long long want = 4LL * kCtas;  // items that even out what the masks leave
  if (blocks < want && tiles >= 8) {  // (each item loads its keys anew)
    c.hpi = 1;
    const long long have = blocks * G;
    if (have < want && observe == 0) {
      long long n = (want + have - 1) / have;
      const int met = nseq > 1 ? std::min(tiles, 2 * tiles / nseq) : tiles;
      const long long most = std::max((met + kMinTiles - 1) / kMinTiles, 1);
      if (n > most) n = most;
      if (n > 16) n = 16;
      c.nseg = (int)n;
    }
  }
  const long long cuts = ((long long)tiles * c.hpi + kMaxPairs - 1) / kMaxPairs;
  if (c.nseg < cuts) c.nseg = (int)cuts;
  c.parts = (G / c.hpi) * c.nseg;
  return c;
}

// Key blocks per item where an item's queries stay in shared memory: the fewest
// steps of the busiest CTA, an item costing about as much besides as two blocks.
int run_of(int nkb, long long heads) {
  int best = 1;
  long long least = -1;
  for (int r = 1; r <= nkb && r <= 64; ++r) {
    const long long items = (nkb + r - 1) / r * heads;
    const long long t = (items + kCtas - 1) / kCtas * (r + 2);
    if (least < 0 || t < least) {
      least = t;
      best = r;
    }
  }
  return best;
}

template <int D>
usp_status_t launch_tc(const WeightParams& W, cudaStream_t st) {
  const AttnParams& P = W.P;
  using L = WSmem<D>;
  CUtensorMap mq, mk;
  if (!make_map(&mq, P.q, P.Bt, P.S, P.Hq, D, 64) || !make_map(&mk, P.k, P.Bt, P.S, P.Hkv, D, kTile))
    return USP_ERR_CUDA;
  const int smem = L::kAlloc;
  static SmemAttr attr;
  cudaError_t e = attr.set(key_weights_tc_kernel<D>, smem);
  if (e != cudaSuccess) return fail_cuda("cudaFuncSetAttribute(smem)", e);
  const int blocks = W.items < kCtas ? W.items : kCtas;
  {
    ProfScope ps(st, "attn_key_weights");
    key_weights_tc_kernel<D><<<blocks, kThreads, smem, st>>>(W, mq, mk);
  }
  note_launch();
  return check_launch();
}

}  // namespace

size_t key_weights_workspace(int B, int S, int Hq, int Hkv, int observe) {
  const Cut c = cut_of(B, S, Hq, Hkv, observe, false, 0);  // (no more parts if `tail` or packed)
  return c.parts > 1 ? (size_t)c.parts * B * Hkv * S * 4 : 0;
}

usp_status_t launch_key_weights_tc(const AttnParams& P, float* weight, int observe,
                                   void* workspace, cudaStream_t st) {
  const Cut c = cut_of(P.Bt, P.S, P.Hq, P.Hkv, observe, P.layout == kContiguous && !P.cu,
                       P.cu ? P.nseq : 0);
  WeightParams W{P, c.parts > 1 ? static_cast<float*>(workspace) : weight,
                 observe < P.S ? observe : 0, c.hpi, P.G / c.hpi, c.nseg, c.nkb, c.q0, c.ntiles, 1, 3, 3, 1, 0};
  if (c.ntiles == 1 && P.S - c.q0 <= 64 && c.hpi % 2 == 0) W.pair = 2;
  const bool straight = P.layout == kContiguous && !P.cu;
  const long long most = (long long)c.ntiles * (c.hpi / W.pair);  // query tiles of an item
  if (most <= 2) {
    W.qslots = 2;
    W.kslots = 4;
  } else if (most <= kSlots && straight) {
    W.qslots = kSlots;
    W.kslots = kTileSlots - kSlots;
  }
  const long long heads = (long long)P.Bt * P.Hkv * W.groups * c.nseg;
  if (most <= W.qslots && straight) W.run = run_of(c.nkb, heads);
  const long long items = (c.nkb + W.run - 1) / W.run * heads;
  if (items > 0x3fffffffLL) return USP_ERR_UNSUPPORTED;
  W.items = (int)items;
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
  WeightParams W{P, nullptr, observe, P.G, 1, 1, 0, 0};
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
