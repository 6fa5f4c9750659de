// Attention of the newest tokens to the paged 8-bit KV cache, few rows per KV head.
//
// "Long Context Attention" notes, "Ring Attention" (flash decoding is ring
// attention at inference time) and "Tree Attention" (log-sum-exp partials
// combine in any order): 2 D + 2/32 bytes per key and KV head are read once per
// block of up to 16 query rows.
//
// Division of the work. A unit is one (sequence, KV head, block of 8 NT query
// rows); a step is 32 of its keys, which share one exponent each for K and V and
// lie in one page. All steps of all units, in unit order and each unit followed by
// a few that stand for the cost of its end, are one line of length T that the
// warps of the GPU share in equal runs, whatever the lengths (read on the
// device). Warp c takes [T c / N, T (c+1) / N); it leaves one partial (m, l, O) per
// unit of which it has steps, in slot c + unit (between two consecutive partials
// either c or the unit grows), and the second kernel merges a unit's partials,
// which are consecutive, in order. Neighbouring runs go to different SMs, so that
// a short problem uses all of them. Where few units have few keys (own_cluster below) a
// cluster of CTAs takes each instead, and that is the only kernel.
//
// One warp. It is on its own: its own ring of stages (32 keys and values each,
// 4 D / 128 KB, brought in by TMA with the swizzle that makes its reads free of bank
// conflicts), its own barriers and its own online softmax; no barrier of the CTA.
// The pages and exponents of the next 32 steps are fetched by its lanes at once.
// The keys and channels are the M side of the matrix products and the query rows
// the N side (8 rows per product, where 16 would be padding for most head groups):
//   S^T [keys x rows]  = K [keys x D] Q^T      (fp16 m16n8k16, fp32 sums)
//   O^T [D x rows]    += V^T [D x keys] P^T
// The K index of a product may be any permutation of the channels (keys) that
// both operands share. Thread (g, t) = (lane / 4, lane % 4) owns channels
// [t D/4, ..) of key rows g and g + 8 for K, and channels [g D/8, ..) of keys
// 2t, 2t+1, 2t+8, 2t+9 for V: vector loads, one conversion per two elements.
//
// Numbers. Codes are exact in fp16. q is scaled by a power of two per row, exactly,
// to a largest element of 64 .. 128 (elements below 2^-23 of it lose bits). A
// block's exponents never touch the codes: K's multiplies the scores, V's is
// added to them in log2 units, so p = 2^(score + e_v - m) belongs to the codes of V,
// and the row's sum takes p 2^-e_v back. The reference m starts 2^7 below the
// running maximum of score + e_v and moves when that exceeds it by 2^15, so p uses
// fp16's range: a p of down to 2^-21 of the largest contribution keeps all 11 bits
// (its rounding, 2^-12, is the only one of the products), and below that its error is at
// most 2^-32 of it, so many small keys beside a sink still count.
//
// Bound by HBM where the keys are many: 8 sequences of 128K keys, 8 KV heads, D = 128 and 4
// rows each, 2.15 GB in 319 us (6.7 TB/s) and the merge, 328 in all; of the issue slots 34 % are
// taken. Windows of 1000 keys of 16 sequences and 32 KV heads: 134 MB in 30 us, of which the
// start, the ends of 512 units and the merge are some 10. One sequence of 1024 keys: 7 us,
// a chain of dependent loads (lengths, pages, keys) and the launch.
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "internal.h"
#include "kv4_host.h"
#include "kv8.cuh"
#include "kv8_attn.cuh"
#include "kv8_host.h"
#include "tc_ptx.cuh"

namespace usp {
namespace {

using namespace kv8;
using namespace tc;

__device__ int g_attn_kv8_status = 0;

constexpr int kStep = kBlock;   // keys per step
constexpr int kSms = 152;
constexpr int kWarps = 8;       // of a CTA, one CTA per SM
constexpr int kThreads = 32 * kWarps;
constexpr int kRuns = kSms * kWarps;
// Of a unit's end, in steps (4 x 32K keys and 12 rows: 41.7 us with 1, 40.2 with 3, 38.8
// with 5, 39.5 with 8; 512 units of 33 steps: 30.9, 30.0, 30.0, 30.7).
constexpr int kUnitCost = 5;
constexpr float kBelow = 7.f, kAbove = 15.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  Cache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  float* o_part;    // [slots][8 NT][D]
  float2* ml_part;  // [slots][8 NT]: (m, l), m the reference in log2 units
  int2* span;       // [units]: first and last slot (units that have steps)
  const int* cu;    // packed: boundaries of the tokens, T in all
  int T, max_new;
  int Hq, G, nrb;   // most blocks of rows of a KV head
  int slots;
  float score_mul;  // softmax scale * log2(e)
  int causal, window, sink;
};

// A sequence as the kernels see it.
struct Seq {
  int len, n;          // cached tokens, new ones among them
  int first;           // of its tokens in q (dense: b T)
  int R, nrb;          // rows per KV head, blocks of them
  int steps;           // of a unit: key step s (s < sinks) or s + skip
  int sinks, skip;
};
template <int NT>
__device__ __forceinline__ Seq seq_of(const Params& P, int b) {
  Seq q;
  q.len = clamp_len(__ldg(P.c.lens + b), P.c.cap);
  if (P.cu) {
    q.first = min(max(__ldg(P.cu + b), 0), P.T);
    q.n = min(max(__ldg(P.cu + b + 1), q.first), P.T) - q.first;
  } else {
    q.first = b * P.T;
    q.n = P.T;
  }
  q.R = min(q.n, P.max_new) * P.G;
  q.nrb = (q.R + 8 * NT - 1) / (8 * NT);
  q.steps = (q.len + kStep - 1) / kStep;
  q.sinks = q.skip = 0;
  if (P.window > 0) {
    const int i0 = max(0, q.len - q.n);  // first query position
    const int first = max(0, i0 - P.window + 1) / kStep;
    q.sinks = min((min(P.sink, q.len) + kStep - 1) / kStep, first);
    q.skip = first - q.sinks;
    q.steps -= q.skip;
  }
  if (q.nrb == 0) q.steps = 0;
  return q;
}
// Length of a unit of n steps on the line that the warps share.
__device__ __forceinline__ int line_len(int n) { return n > 0 ? n + kUnitCost : 0; }

// The sequences [b0, b0 + 32) on the line, one per lane: where each ends.
template <int NT>
__device__ __forceinline__ long long line_ends(const Params& P, int b0) {
  const int b = b0 + (threadIdx.x & 31);
  long long inc = 0;
  if (b < P.c.B) {
    const Seq q = seq_of<NT>(P, b);
    inc = (long long)line_len(q.steps) * q.nrb * P.c.H;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if ((threadIdx.x & 31) >= o) inc += x;
  }
  return inc;
}
__device__ __forceinline__ long long scaled(long long T, unsigned c, unsigned N) {  // T c / N
  if (T <= 0xffffffffLL / kRuns) return (unsigned)T * c / N;  // (a 64-bit division is slow)
  return T * c / N;
}

__device__ __forceinline__ void grid_dependency_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A walk over the steps of a run: the current unit's steps [s, end).
struct Walk {
  int b, hr;        // sequence, KV head * its blocks + row block
  int s, end;       // of the unit
  Seq q;
  long long left;   // of the run's part of the line, behind this unit
};
template <int NT>
__device__ __forceinline__ bool next_unit(const Params& P, Walk& w) {
  if (w.left <= 0) return false;
  if (++w.hr >= P.c.H * w.q.nrb) {
    w.hr = 0;
    do {
      if (++w.b >= P.c.B) return false;
      w.q = seq_of<NT>(P, w.b);
    } while (w.q.steps == 0);
  }
  w.s = 0;
  w.end = (int)min((long long)w.q.steps, w.left);
  w.left -= line_len(w.q.steps);
  return true;
}

constexpr int kMeta = 64;  // steps whose page and exponents are kept, a power of two
template <int D>
struct Smem {
  static constexpr int kTile = kStep * D;        // bytes of K (or V) of a step
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kWarpBytes = kStages * 2 * kTile;
  static constexpr int kMetaAt = kWarps * kWarpBytes;             // [kWarps][kMeta] int2
  static constexpr int kBar = kMetaAt + kWarps * kMeta * 8;       // [kWarps][kStages]
  static constexpr int kMisc = kBar + kWarps * kStages * 8;       // abort
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 227 * 1024, "one CTA per SM");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
  return x;
}

// kOwn: a cluster of `cl` CTAs has a unit to itself; its warps take equal parts of the
// steps, and their partials are joined in order over (distributed) shared memory: no
// workspace, no second kernel.
template <int D, int NT, bool kOwn>
__global__ void __launch_bounds__(kThreads, 1)
attn_kv8_kernel(const Params P, int cl, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v) {
  using L = Smem<D>;
  constexpr int kStages = L::kStages;
  constexpr int kRows = 8 * NT;
  constexpr int kCK = D / 64;      // 16-byte chunks a thread has per K row
  constexpr int kMT = D / 16;      // 16-channel tiles of O^T
  constexpr int kWV = D / 32;      // 32-bit words of codes a thread has per V row
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t sbase = smem_u32(sm);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kMisc);
  int2* meta = reinterpret_cast<int2*>(sm + L::kMetaAt) + warp * kMeta;
  auto full = [&](int st) { return sbase + L::kBar + 8 * (warp * kStages + st); };

  if constexpr (kOwn) grid_dependency_launch();  // (no merge behind it)
  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(full(st), 1);
    fence_barrier_init();
    if (warp == 0) {
      *abort_flag = 0;
      if (P.c.np > 0) {
        tma_prefetch(&tm_k);
        tma_prefetch(&tm_v);
      }
    }
  }
  __syncthreads();  // no warp waits for another from here to the end of its steps
  grid_dependency_wait();  // (this kernel's launch overlaps the end of what came before it)
  // The merge may start from here on, when all that came before is complete: it reads lengths
  // and boundaries ahead of its own wait. (A wait of the merge's first instead, with the trigger
  // at the start: 0.7 us more, 30.3 -> 31.0 us for the windows.)
  if constexpr (!kOwn) grid_dependency_launch();

  // ------------------------------------------------------- this warp's run
  const unsigned run = warp * kSms + blockIdx.x;
  const unsigned rank = kOwn ? blockIdx.x % cl : 0;
  Walk cur;
  bool more = true;
  if constexpr (kOwn) {
    if (P.cu) {  // zeros for the tokens outside the sequences, by all clusters
      const int e0 = min(max(__ldg(P.cu), 0), P.T), e1 = max(e0, min(max(__ldg(P.cu + P.c.B), 0), P.T));
      for (int i = blockIdx.x; i < e0 + P.T - e1; i += gridDim.x) {
        const long long tok = i < e0 ? i : e1 + (i - e0);
        uint2* r = reinterpret_cast<uint2*>(P.out + tok * P.Hq * D);
        for (int u = threadIdx.x; u < P.Hq * D / 4; u += kThreads) r[u] = make_uint2(0, 0);
        for (int u = threadIdx.x; u < P.Hq; u += kThreads) P.lse[tok * P.Hq + u] = -INFINITY;
      }
    }
    const int unit = blockIdx.x / cl, bh = unit / P.nrb, rb = unit - bh * P.nrb;
    if (bh >= P.c.B * P.c.H) return;  // a cluster for such tokens alone
    cur.b = bh / P.c.H;
    cur.q = seq_of<NT>(P, cur.b);
    const int n = rb < cur.q.nrb ? cur.q.steps : 0;
    cur.q.nrb = max(cur.q.nrb, 1);
    cur.hr = (bh - cur.b * P.c.H) * cur.q.nrb + (rb < cur.q.nrb ? rb : 0);
    // equal parts of the steps; neighbouring ones to different CTAs (no products that pass
    // 32 bits: a unit has kOwnSteps * W steps at most)
    const int w = warp * cl + rank, W = kWarps * cl;
    cur.s = n * w / W;
    cur.end = n * (w + 1) / W;
    cur.left = 0;
    more = cur.end > cur.s;
  } else {
    long long ends = line_ends<NT>(P, 0);
    long long T = __shfl_sync(0xffffffffu, ends, 31);
    for (int b = 32; b < P.c.B; b += 32)
      T += __shfl_sync(0xffffffffu, line_ends<NT>(P, b), 31);
    const unsigned N = (unsigned)min(T, (long long)kRuns);
    if (run >= N) return;
    const long long first = scaled(T, run, N), count = scaled(T, run + 1, N) - first;
    if (count == 0) return;
    // the sequence that holds `first`
    int b0 = 0;
    long long before = 0;
    for (;;) {
      const unsigned over = __ballot_sync(0xffffffffu, before + ends > first);
      if (over) {
        const int src = __ffs(over) - 1;
        if (src > 0) before += __shfl_sync(0xffffffffu, ends, src - 1);
        b0 += src;
        break;
      }
      before += __shfl_sync(0xffffffffu, ends, 31);
      b0 += 32;
      if (b0 >= P.c.B) return;  // not reached: first < T
      ends = line_ends<NT>(P, b0);
    }
    cur.b = b0;
    cur.q = seq_of<NT>(P, b0);
    const int n = cur.q.steps, ln = line_len(n);
    const long long in = first - before;
    cur.hr = in <= 0xffffffffLL ? (int)((unsigned)in / ln) : (int)(in / ln);
    const int at = (int)(in - (long long)cur.hr * ln);
    cur.s = at;
    cur.end = (int)min((long long)n, at + count);
    cur.left = count - (ln - at);
    // the run may begin behind a unit's last step, and end there too
    if (at >= n && !next_unit<NT>(P, cur)) return;
  }

  // ------------------------------------------------- copies, kStages ahead
  Walk pre = cur;
  unsigned issued = 0, known = 0, used = 0;  // steps: copied, with a page, taken
  const uint32_t ring = sbase + warp * L::kWarpBytes;
  // Exponents of the steps whose pages came last, on their way: nothing needs them before
  // the keys are there, so the copies do not wait for them.
  unsigned exps_at = 0;
  bool exps_due = false;
  int ke = 0, ve = 0;
  auto put_exps = [&]() {
    meta[(exps_at + lane) & (kMeta - 1)].y = (clamp_exp(ke) & 0xffff) | (clamp_exp(ve) << 16);
    __syncwarp();
    exps_due = false;
  };
  auto issue = [&]() {
    if (issued == known) {
      if (exps_due) put_exps();
      // pages and exponents of the unit's next 32 steps, one per lane
      const int s = pre.s + lane;
      int page = -1;
      ke = ve = 0;
      if (s < pre.end) {
        const int row = (s < pre.q.sinks ? s : s + pre.q.skip) * kStep;
        page = page_of(P.c, pre.b, row);
        if (page >= 0) {
          const long long blk =
              (head_rows(P.c, page, pre.hr / pre.q.nrb) + (row & (P.c.ps - 1))) / kBlock;
          ke = P.c.ke[blk];
          ve = P.c.ve[blk];
        }
      }
      // (the entries of the last kStages steps and of these 32 are in use: kMeta has room)
      meta[(known + lane) & (kMeta - 1)].x = page;
      __syncwarp();
      exps_at = known;
      exps_due = true;
      known += min(32, pre.end - pre.s);
    }
    if (lane == 0) {
      const int st = issued % kStages;
      const int page = meta[issued & (kMeta - 1)].x;
      if (page >= 0) {
        const int key = (pre.s < pre.q.sinks ? pre.s : pre.s + pre.q.skip) * kStep;
        const int hp = page * P.c.H + pre.hr / pre.q.nrb;
        const uint32_t dst = ring + st * (2 * L::kTile);
        mbar_expect_tx(full(st), 2 * L::kTile);
        tma_load_3d(dst, &tm_k, full(st), 0, key & (P.c.ps - 1), hp);
        tma_load_3d(dst + L::kTile, &tm_v, full(st), 0, key & (P.c.ps - 1), hp);
      } else {
        mbar_arrive(full(st));
      }
    }
    ++issued;
    if (++pre.s >= pre.end) more = next_unit<NT>(P, pre);
  };
#pragma unroll
  for (int st = 0; st < kStages; ++st)
    if (more) issue();

  bool ok = true;
  for (;;) {
    // ---------------------------------------------------------------- a unit
    const Seq sq = cur.q;
    const int h = cur.hr / sq.nrb, rb = kOwn ? (int)(blockIdx.x / cl) % P.nrb : cur.hr - h * sq.nrb;
    const int len = sq.len, i_first = len - sq.n;
    // Q^T fragments: product kk = 4 j + w takes channels 4 w .. 4 w + 3 of chunk j of
    // the thread's run of D/4
    uint32_t qf[NT][4 * kCK][2];
    float mul[NT][2];  // of rows 2t, 2t + 1: products to log2 units
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = rb * kRows + nt * 8 + g;
      const __nv_bfloat16* src = nullptr;
      if (r < sq.R) {
        const int tok = r / P.G, hh = r - tok * P.G;
        src = P.q + ((long long)(sq.first + tok) * P.Hq + h * P.G + hh) * D + t * (D / 4);
      }
      uint4 x[2 * kCK];
      float big = 0.f;
#pragma unroll
      for (int w = 0; w < 2 * kCK; ++w) {
        x[w] = src ? __ldg(reinterpret_cast<const uint4*>(src) + w) : make_uint4(0, 0, 0, 0);
        const uint32_t e[4] = {x[w].x, x[w].y, x[w].z, x[w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          big = fmaxf(big, fmaxf(fabsf(__uint_as_float(e[i] << 16)),
                                 fabsf(__uint_as_float(e[i] & 0xffff0000u))));
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // 2^ex times a largest element in [1, 2) is brought to [64, 128)
      const int ex = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -120), 127);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 6 - ex) << 23);
#pragma unroll
      for (int w = 0; w < 2 * kCK; ++w) {
        const uint32_t e[4] = {x[w].x, x[w].y, x[w].z, x[w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qf[nt][2 * w + i / 2][i & 1] = half2_bits(__floats2half2_rn(
              __uint_as_float(e[i] << 16) * up, __uint_as_float(e[i] & 0xffff0000u) * up));
      }
      // not 0 or infinite, with a block's exponent too, which a masked key's -inf or a
      // score of 0 would make NaN
      const float row_mul = fminf(fmaxf(ldexpf(P.score_mul, ex - 6), FLT_MIN * 0x1p41f),
                                  FLT_MAX * 0x1p-41f);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        mul[nt][e] = __shfl_sync(0xffffffffu, row_mul, 4 * (2 * t + e));
    }
    float o[NT][kMT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    for (int s = cur.s; s < cur.end; ++s) {
      const int st = used % kStages;
      if (exps_due) put_exps();
      ok = mbar_wait(full(st), (used / kStages) & 1, abort_flag, &g_attn_kv8_status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int2 mt = meta[used & (kMeta - 1)];
      ++used;
      const int key0 = (s < sq.sinks ? s : s + sq.skip) * kStep;
      if (mt.x >= 0) {
        const uint8_t* kt = sm + warp * L::kWarpBytes + st * (2 * L::kTile);
        const uint8_t* vt = kt + L::kTile;
        const float kx = exp2i(static_cast<int16_t>(mt.y & 0xffff));
        const int ve = mt.y >> 16;
        // does the mask (or the sequence's end) hide any of the step's keys?
        const int last = key0 + kStep - 1;
        const bool masked = last >= len || i_first < 0 || (P.causal && last > i_first) ||
                            (P.window > 0 && len - 1 - key0 >= P.window);
        // ------------------------------------------------------------ scores
        float sc[NT][2][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nt][half][e] = 0.f;
          const int r0 = 16 * half + g;
#pragma unroll
          for (int j = 0; j < kCK; ++j) {
            const uint4 a = *reinterpret_cast<const uint4*>(kt + tile_at<D>(r0, kCK * t + j));
            const uint4 c = *reinterpret_cast<const uint4*>(kt + tile_at<D>(r0 + 8, kCK * t + j));
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t f[4] = {e4m3x2_to_h2(aw[w] & 0xffffu), e4m3x2_to_h2(cw[w] & 0xffffu),
                                     e4m3x2_to_h2(aw[w] >> 16), e4m3x2_to_h2(cw[w] >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(sc[nt][half], f, qf[nt][4 * j + w][0], qf[nt][4 * j + w][1]);
            }
          }
        }
        // ----------------------------------------------------------- softmax
        if (masked) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = key0 + 16 * half + g + 8 * (e >> 1);
                const int i = i_first + (rb * kRows + nt * 8 + 2 * t + (e & 1)) / P.G;
                const bool see = j < len && i >= 0 && (!P.causal || j <= i) &&
                                 (P.window <= 0 || i - j < P.window || j < P.sink);
                if (!see) sc[nt][half][e] = -INFINITY;
              }
        }
        bool grow = false;
        float mx[NT][2], ms[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ms[nt][e] = mul[nt][e] * kx;
            mx[nt][e] = fmaf(ms[nt][e], fmaxf(fmaxf(sc[nt][0][e], sc[nt][0][e + 2]),
                                              fmaxf(sc[nt][1][e], sc[nt][1][e + 2])),
                             static_cast<float>(ve));
            grow |= mx[nt][e] > m[nt][e] + kAbove;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = mx[nt][e];
#pragma unroll
              for (int off = 4; off < 32; off <<= 1)
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
              x = fmaxf(x - kBelow, m[nt][e]);
              a[e] = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - x);
              m[nt][e] = x;
              l[nt][e] *= a[e];
            }
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
              o[nt][i][0] *= a[0];
              o[nt][i][1] *= a[1];
              o[nt][i][2] *= a[0];
              o[nt][i][3] *= a[1];
            }
          }
        }
        uint32_t pf[NT][2][2];  // P^T fragments: [half][keys 0-7, 8-15]
        const float back = exp2i(-ve);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float v = static_cast<float>(ve);
          const float m0 = m[nt][0] == -INFINITY ? 0.f : v - m[nt][0];
          const float m1 = m[nt][1] == -INFINITY ? 0.f : v - m[nt][1];
          float ls[2] = {0.f, 0.f};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = ex2(fmaf(sc[nt][half][e], ms[nt][e & 1], (e & 1) ? m1 : m0));
            ls[0] += p[0] + p[2];
            ls[1] += p[1] + p[3];
            pf[nt][half][0] = movmatrix_t(half2_bits(__floats2half2_rn(p[0], p[1])));
            pf[nt][half][1] = movmatrix_t(half2_bits(__floats2half2_rn(p[2], p[3])));
          }
          l[nt][0] = fmaf(ls[0], back, l[nt][0]);
          l[nt][1] = fmaf(ls[1], back, l[nt][1]);
        }
        // -------------------------------------------------------------- P V
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t vw[4][kWV];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 16 * half + 2 * t + (i & 1) + 8 * (i >> 1);
            if constexpr (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(vt + tile_at<D>(key, g));
              vw[i][0] = x.x; vw[i][1] = x.y; vw[i][2] = x.z; vw[i][3] = x.w;
            } else {
              const uint2 x =
                  *reinterpret_cast<const uint2*>(vt + tile_at<D>(key, g >> 1) + 8 * (g & 1));
              vw[i][0] = x.x; vw[i][1] = x.y;
            }
            // rows behind the sequence hold anything: 0, so that 0 * it is 0
            if (masked && key0 + key >= len) {
#pragma unroll
              for (int w = 0; w < kWV; ++w) vw[i][w] = 0;
            }
          }
#pragma unroll
          for (int w = 0; w < kWV; ++w)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              // channels 4 w + 2 u and the next of keys (2t, 2t + 1) and (.. + 8)
              const uint32_t x = __byte_perm(vw[0][w], vw[1][w], u ? 0x7362 : 0x5140);
              const uint32_t y = __byte_perm(vw[2][w], vw[3][w], u ? 0x7362 : 0x5140);
              const uint32_t f[4] = {e4m3x2_to_h2(x & 0xffffu), e4m3x2_to_h2(x >> 16),
                                     e4m3x2_to_h2(y & 0xffffu), e4m3x2_to_h2(y >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[nt][2 * w + u], f, pf[nt][half][0], pf[nt][half][1]);
            }
        }
      }
      __syncwarp();  // the stage has been read
      if (more) issue();
    }
    if constexpr (kOwn) {
      // the warp's partial where its tiles stood, then the CTA's, then the cluster's
      if (!ok)  // (aborted: the copies in flight land first)
        for (; used < issued; ++used) mbar_wait_drain(full(used % kStages), (used / kStages) & 1);
      __syncwarp();
      float* mine = reinterpret_cast<float*>(sm + warp * L::kWarpBytes);  // [rows][D], then m, l
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = l[nt][e];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
          const int r = nt * 8 + 2 * t + e;
          if (g == 0) {
            mine[kRows * D + 2 * r] = m[nt][e];
            mine[kRows * D + 2 * r + 1] = x;
          }
          float4* dst = reinterpret_cast<float4*>(mine + r * D + g * (D / 8));
#pragma unroll
          for (int i = 0; i < kMT; i += 2)
            dst[i / 2] =
                make_float4(o[nt][i][e], o[nt][i][e + 2], o[nt][i + 1][e], o[nt][i + 1][e + 2]);
        }
      __syncthreads();
      const int rows = min(kRows, sq.R - rb * kRows);  // that exist
      constexpr int kPart = L::kWarpBytes / 4;         // floats from one warp's to the next's
      const float* parts = reinterpret_cast<const float*>(sm);
      float* cta = reinterpret_cast<float*>(sm) + kRows * D + 2 * kRows;  // the CTA's, behind warp 0's
      static_assert(2 * (kRows * D + 2 * kRows) <= kPart, "a warp's tiles hold two partials");
      for (int x = threadIdx.x; x < rows * D; x += kThreads) {
        const int r = x / D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, parts[w * kPart + kRows * D + 2 * r]);
        float os = 0.f, ls = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = parts[w * kPart + kRows * D + 2 * r];
          const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
          ls += parts[w * kPart + kRows * D + 2 * r + 1] * f;
          os += parts[w * kPart + x] * f;
        }
        cta[x] = os;
        if (x == r * D) {
          cta[kRows * D + 2 * r] = M;
          cta[kRows * D + 2 * r + 1] = ls;
        }
      }
      cluster_sync();
      const uint32_t at = smem_u32(cta);
      for (int x = rank * kThreads + threadIdx.x; x < rows * D; x += cl * kThreads) {
        const int r = x / D, row = rb * kRows + r;
        float M = -INFINITY, os = 0.f, ls = 0.f;
        for (int c = 0; c < cl; ++c) M = fmaxf(M, ld_cluster(at + 4 * (kRows * D + 2 * r), c));
        for (int c = 0; c < cl; ++c) {
          const float mc = ld_cluster(at + 4 * (kRows * D + 2 * r), c);
          const float f = mc == -INFINITY ? 0.f : ex2(mc - M);
          ls += ld_cluster(at + 4 * (kRows * D + 2 * r + 1), c) * f;
          os += ld_cluster(at + 4 * x, c) * f;
        }
        const int tok = row / P.G, hh = row - tok * P.G;
        const long long o_row = (long long)(sq.first + tok) * P.Hq + h * P.G + hh;
        const bool none = ls == 0.f;  // no visible key (a NaN score makes ls NaN)
        P.out[o_row * D + x - r * D] = __float2bfloat16_rn(none ? 0.f : os * (1.f / ls));
        if (x == r * D) P.lse[o_row] = none ? -INFINITY : (M + log2f(ls)) * kLn2;
      }
      cluster_sync();  // (no CTA ends while another reads its memory)
      return;
    }
    if (!ok) break;
    // ------------------------------------------------- the unit's partial
    const int unit = (cur.b * P.c.H + h) * P.nrb + rb;
    const long long slot = (long long)run + unit;
    if (lane == 0) {
      if (cur.s == 0) P.span[unit].x = (int)slot;
      if (cur.end == sq.steps) P.span[unit].y = (int)slot;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        const int r = nt * 8 + 2 * t + e;
        if (rb * kRows + r >= sq.R) continue;
        if (g == 0) P.ml_part[slot * kRows + r] = make_float2(m[nt][e], x);
        // o[i][e], o[i][e + 2]: channels 2 i, 2 i + 1 of the thread's run of D/8
        float4* dst = reinterpret_cast<float4*>(P.o_part + (slot * kRows + r) * D + g * (D / 8));
#pragma unroll
        for (int i = 0; i < kMT; i += 2)
          dst[i / 2] = make_float4(o[nt][i][e], o[nt][i][e + 2], o[nt][i + 1][e], o[nt][i + 1][e + 2]);
      }
    if (!next_unit<NT>(P, cur)) break;
  }
  // aborted: the copies in flight land before the CTA ends
  if (!ok && lane == 0)
    for (; used < issued; ++used) mbar_wait_drain(full(used % kStages), (used / kStages) & 1);
}

constexpr int kMergeThreads = 256;

// A unit's first and last slot. Where a wait of the kernel before gave up (which
// usp_device_status reports), they may never have been written: whatever stands
// there, only slots that exist are read.
__device__ __forceinline__ int2 span_of(const Params& P, int unit) {
  const int2 s = P.span[unit];
  return make_int2(max(s.x, 0), min(s.y, P.slots - 1));
}

// D / 4 threads take every kParts-th partial of a row (they stand in consecutive slots);
// a block kMaxParts / kParts rows. Blocks behind the rows (packed): zeros for the
// tokens outside the sequences. Launched while the kernel above still runs, but only once that
// has waited for what came before it: lengths and boundaries are read ahead of the wait, nothing
// that the kernel above writes is.
template <int D>
constexpr int kMaxParts = kMergeThreads / (D / 4);
template <int D, int NT, int kParts>
__global__ void __launch_bounds__(kMergeThreads) attn_kv8_merge_kernel(const Params P, int pads) {
  constexpr int kRows = 8 * NT, kLanes = D / 4, kPer = kMaxParts<D> / kParts;
  __shared__ float4 s_o[kParts > 1 ? kParts : 1][kLanes];
  __shared__ float2 s_ml[kParts];
  const int rows = P.c.B * P.c.H * P.nrb * kRows, blocks = (rows + kPer - 1) / kPer;
  if ((int)blockIdx.x >= blocks) {
    const int e0 = min(max(__ldg(P.cu), 0), P.T), e1 = max(e0, min(max(__ldg(P.cu + P.c.B), 0), P.T));
    grid_dependency_wait();
    for (int i = blockIdx.x - blocks; i < e0 + P.T - e1; i += pads) {
      const long long tok = i < e0 ? i : e1 + (i - e0);
      uint2* r = reinterpret_cast<uint2*>(P.out + tok * P.Hq * D);
      for (int u = threadIdx.x; u < P.Hq * D / 4; u += kMergeThreads) r[u] = make_uint2(0, 0);
      for (int u = threadIdx.x; u < P.Hq; u += kMergeThreads) P.lse[tok * P.Hq + u] = -INFINITY;
    }
    return;
  }
  const int group = threadIdx.x / kLanes, d = threadIdx.x - group * kLanes;
  const int part = group % kParts, x = blockIdx.x * kPer + group / kParts;
  if (x >= rows) return;  // (kParts > 1: all of a block's threads, kPer being 1)
  const int unit = x / kRows, r = x % kRows;  // r: row within the block
  const int bh = unit / P.nrb, rb = unit - bh * P.nrb;
  const int b = bh / P.c.H, h = bh - b * P.c.H;
  const int row = rb * kRows + r;
  const Seq q = seq_of<NT>(P, b);
  if (row >= q.R) return;
  int2 span = make_int2(0, -1);  // no steps, no partials
  grid_dependency_wait();
  if (q.steps > 0) span = span_of(P, unit);
  float M = -INFINITY, ls = 0.f;
  float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (long long s = span.x + part; s <= span.y; s += kParts) {
    const float2 a = P.ml_part[s * kRows + r];
    const float4 y = reinterpret_cast<const float4*>(P.o_part + (s * kRows + r) * D)[d];
    const float Mn = fmaxf(M, a.x);
    const float f0 = M == -INFINITY ? 0.f : ex2(M - Mn);
    const float f1 = a.x == -INFINITY ? 0.f : ex2(a.x - Mn);
    os.x = os.x * f0 + y.x * f1;
    os.y = os.y * f0 + y.y * f1;
    os.z = os.z * f0 + y.z * f1;
    os.w = os.w * f0 + y.w * f1;
    ls = ls * f0 + a.y * f1;
    M = Mn;
  }
  if constexpr (kParts > 1) {
    s_o[part][d] = os;
    if (d == 0) s_ml[part] = make_float2(M, ls);
    __syncthreads();
    if (part != 0) return;
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kParts; ++i) M = fmaxf(M, s_ml[i].x);
    ls = 0.f;
    os = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const float f = s_ml[i].x == -INFINITY ? 0.f : ex2(s_ml[i].x - M);
      ls += s_ml[i].y * f;
      os.x += s_o[i][d].x * f;
      os.y += s_o[i][d].y * f;
      os.z += s_o[i][d].z * f;
      os.w += s_o[i][d].w * f;
    }
  }
  const int tok = row / P.G, hh = row - tok * P.G;
  const long long o_row = (long long)(q.first + tok) * P.Hq + h * P.G + hh;
  const bool none = ls == 0.f;  // no visible key (a NaN score makes ls NaN)
  const float inv = none ? 0.f : 1.f / ls;
  if (none) os = make_float4(0.f, 0.f, 0.f, 0.f);
  reinterpret_cast<uint2*>(P.out + o_row * D)[d] =
      make_uint2(pack_bf16(os.x * inv, os.y * inv), pack_bf16(os.z * inv, os.w * inv));
  if (d == 0) P.lse[o_row] = none ? -INFINITY : (M + log2f(ls)) * kLn2;
}

// ------------------------------------------------------------------- host
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Ws {
  long long nrb, slots;
  int rows;
  size_t o, ml, span, total;
};
Ws layout(int B, int max_new, int Hq, int Hkv, int D) {
  Ws w{};
  const long long R = (long long)(Hq / Hkv) * max_new;
  w.rows = R <= 8 ? 8 : 16;
  w.nrb = (R + w.rows - 1) / w.rows;
  w.slots = (long long)B * Hkv * w.nrb + kRuns;
  w.ml = up256((size_t)w.slots * w.rows * D * 4);
  w.span = w.ml + up256((size_t)w.slots * w.rows * 8);
  w.total = w.span + up256((size_t)B * Hkv * w.nrb * 8);
  return w;
}

// Which kernel: this one reads the keys once per 16 rows, the tcgen05 kernel (its 128
// rows cost the same however many there are) once per 128 or 256. 4 x 64K keys, 8 KV heads:
// 32 rows 166 us here and 215 there, 48 rows 243 and 217. Where the keys are few the
// ends count: 16 x 1024 keys, 32 rows 29 us and 39, 64 rows 35 and 41, 128 rows 45
// and 44; 8192 keys of one sequence, 64 rows 26 and 43. `rows` of a KV head; `keys` of all
// heads and sequences that the cache has room for.
constexpr long long kRowsHere = 32, kRowsFewKeys = 64, kFewKeys = 1 << 18;
bool many_rows(long long rows, long long keys) {
  return rows > (keys <= kFewKeys ? kRowsFewKeys : kRowsHere);
}

// The CTAs of a unit's cluster, where units have clusters of their own; else 0. One launch
// and no workspace, 4.5 us less for the host of a call (23.6 -> 19), and on the GPU (8 KV
// heads, 4 heads each, sequences of one length): 1 x 4096 keys 10.2 us on one line and 8.3
// in clusters, 4 x 1024 8.0 and 7.0, 4 x 8192 18.3 and 17.4, 16 x 2048 19.3 and 17.6; 1 x
// 32768 21.6 and 24.4. But a short sequence's cluster does not help with a long one's
// keys, so it stays below kOwnSteps steps of a warp, where the host's time is the longer
// even then. The sizes are those of which a GB300 holds as many at once as there are units
// (15 clusters of 8, 23 of 6, 46 of 3, 76 of 2, with one CTA per SM: 2 x 8 units in
// clusters of 8, of which one waits for the others' end, took 15.6 us instead of 10.8).
constexpr int kOwnSteps = 8;  // of a warp at most
int own_cluster(long long units, long long cap) {
  if (units < 1 || units > kSms) return 0;
  const int u = (int)units;
  const int cl = u <= 15 ? 8 : u <= 46 ? min(6, 138 / u) : u <= 76 ? 2 : 1;
  return (cap + kStep - 1) / kStep <= (long long)kOwnSteps * kWarps * cl ? cl : 0;
}

template <int D, int NT>
usp_status_t launch_own(const Params& P, int cl, cudaStream_t st) {
  CUtensorMap mk{}, mv{};
  if (P.c.np > 0 && (!make_map(&mk, P.c.kc, P.c, D) || !make_map(&mv, P.c.vc, P.c, D)))
    return USP_ERR_CUDA;
  const int smem = Smem<D>::kAlloc;
  static SmemAttr attr;
  cudaError_t e = attr.set(attn_kv8_kernel<D, NT, true>, smem);
  if (e != cudaSuccess) return fail_cuda("cudaFuncSetAttribute(smem)", e);
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  int clusters = P.c.B * P.c.H * P.nrb;
  if (P.cu && P.T > kSms) clusters = max(clusters, kSms / cl);  // many tokens to clear, perhaps
  cfg.gridDim = dim3((unsigned)(clusters * cl));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = cl;
  a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 2;
  {
    ProfScope ps(st, "attn_kv8");
    e = cudaLaunchKernelEx(&cfg, attn_kv8_kernel<D, NT, true>, P, cl, mk, mv);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail_cuda("kernel launch", e);
  }
  note_launch();
  return USP_OK;
}

template <int D, int NT>
usp_status_t launch_t(const Params& P, cudaStream_t st) {
  CUtensorMap mk{}, mv{};  // (without pages, nothing is loaded through them)
  if (P.c.np > 0 && (!make_map(&mk, P.c.kc, P.c, D) || !make_map(&mv, P.c.vc, P.c, D))) return USP_ERR_CUDA;
  const int smem = Smem<D>::kAlloc;
  static SmemAttr attr;
  cudaError_t e = attr.set(attn_kv8_kernel<D, NT, false>, smem);
  if (e != cudaSuccess) return fail_cuda("cudaFuncSetAttribute(smem)", e);
  // A row's partials are merged by a block where a unit has many, else by a few threads:
  // of units spread over kRuns warps, each has about kRuns / units + 1.
  const long long units = (long long)P.c.B * P.c.H * P.nrb, rows = units * 8 * NT;
  const bool one = units * 4 > kRuns;
  const int per = one ? kMaxParts<D> : 1;
  const int pads = P.cu ? 64 : 0;
  const long long blocks = (rows + per - 1) / per + pads;
  if (blocks > 0x7fffffffLL) return USP_ERR_UNSUPPORTED;
  // each kernel's launch and set-up overlap the end of the one before it
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(kSms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  {
    ProfScope ps(st, "attn_kv8");
    e = cudaLaunchKernelEx(&cfg, attn_kv8_kernel<D, NT, false>, P, 1, mk, mv);
  }
  if (e == cudaSuccess) {
    note_launch();
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    ProfScope ps(st, "attn_kv8_merge");
    e = one ? cudaLaunchKernelEx(&cfg, attn_kv8_merge_kernel<D, NT, 1>, P, pads)
            : cudaLaunchKernelEx(&cfg, attn_kv8_merge_kernel<D, NT, kMaxParts<D>>, P, pads);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail_cuda("kernel launch", e);
  }
  note_launch();
  return USP_OK;
}

}  // namespace

size_t attn_kv8_workspace(int B, int max_new, long long cap, int Hq, int Hkv, int D) {
  const long long rows = (long long)(Hq / Hkv) * max_new;
  if (many_rows(rows, (long long)B * Hkv * cap)) return attn_kv8_tc_workspace(D);
  const Ws w = layout(B, max_new, Hq, Hkv, D);
  return own_cluster((long long)B * Hkv * w.nrb, cap) ? 0 : w.total;
}

usp_status_t launch_attn_kv8(const AttnKv8Args& a, void* workspace, cudaStream_t st) {
  if (many_rows((long long)(a.Hq / a.c.H) * a.max_new, (long long)a.c.B * a.c.H * a.c.cap))
    return launch_attn_kv8_tc(a, workspace, st);
  const Ws w = layout(a.c.B, a.max_new, a.Hq, a.c.H, a.D);
  char* base = static_cast<char*>(workspace);
  Params P{};
  P.c = a.c;
  P.q = static_cast<const __nv_bfloat16*>(a.q);
  P.out = static_cast<__nv_bfloat16*>(a.out);
  P.lse = a.lse;
  P.o_part = reinterpret_cast<float*>(base);
  P.ml_part = reinterpret_cast<float2*>(base + w.ml);
  P.span = reinterpret_cast<int2*>(base + w.span);
  P.cu = a.cu;
  P.T = a.T;
  P.max_new = a.max_new;
  P.Hq = a.Hq;
  P.G = a.Hq / a.c.H;
  P.nrb = (int)w.nrb;
  P.slots = (int)w.slots;
  P.score_mul = a.scale * kLog2e;
  P.causal = a.causal;
  P.window = a.window;
  P.sink = a.sink;
  if (const int cl = own_cluster((long long)a.c.B * a.c.H * w.nrb, a.c.cap)) {
    if (a.D == 128)
      return w.rows == 8 ? launch_own<128, 1>(P, cl, st) : launch_own<128, 2>(P, cl, st);
    return w.rows == 8 ? launch_own<64, 1>(P, cl, st) : launch_own<64, 2>(P, cl, st);
  }
  if (a.D == 128) return w.rows == 8 ? launch_t<128, 1>(P, st) : launch_t<128, 2>(P, st);
  return w.rows == 8 ? launch_t<64, 1>(P, st) : launch_t<64, 2>(P, st);
}

int read_clear_attn_kv8_status() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_kv8_status, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0) cudaMemcpyToSymbol(g_attn_kv8_status, &z, sizeof(int));
  return v;
}

}  // namespace usp
