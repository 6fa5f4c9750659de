// Decode-step attention over the 4-bit KV cache.
//
// "Long Context Attention" notes, "Ring Attention" (flash decoding is ring
// attention at inference time) and "Tree Attention" (log-sum-exp partials
// combine in any order): the newest Tq tokens of every sequence attend to its
// cached keys, D (1 + 1/16) bytes per key and KV head.
//
// 8 x 128K keys, 32 query heads over 8, D = 128: 236 us, 4.8 TB/s, 0.71 of the
// measured copy rate; bound by instruction issue (64 % of all slots, 660
// instructions of a warp per 32 keys, 16 warps per SM) more than by HBM. 16
// windows of 1000 keys and 32 heads: 30 us, of which rounds of keys 15, the start
// 4, the ends of units the rest. 3 new tokens (12 rows) over 4 x 32K: 57 us. 16
// and 32 rows per KV head over 8 x 128K: 357 and 702 us (a block of 16 rows reads
// the keys anew); one row with its weights accumulated 318 (the scores, 134 MB,
// are written and read once).
//
// Division of the work. A unit is one (sequence, KV head, block of up to 8 NT
// query rows); a step is 32 of its keys. All steps of all units, in unit
// order and each unit followed by a few that stand for the cost of its end, are
// one line of length T that the CTAs share in equal runs, whatever the lengths
// (read on the device). CTA c takes [T c / N, T (c+1) / N) of N = min(grid, T / 8)
// CTAs; a run may cover the end of one unit and the start of others. It leaves
// one partial (m, l, O) per unit of which it has steps, in slot c + unit:
// between two consecutive partials either c or the unit grows, so the slots
// differ, and a unit's partials are consecutive. The CTAs that hold a unit's
// first and last step leave those two slots for the merge kernel.
//
// One CTA. A round is one step for each warp; its codes and scales are one
// contiguous piece of each array (two where the sinks end), brought in by
// untiled bulk copies two or three rounds ahead, which the warps issue in
// turn. Every warp has its own online softmax; the warps meet only at the end
// of a unit. The keys and
// channels are the M side of the matrix products and the query rows the N
// side (8 rows per product, where 16 would be padding for most head groups):
//   S^T [keys x rows]  = K [keys x D] Q^T      (fp16 m16n8k16, fp32 sums)
//   O^T [D x rows]    += V^T [D x keys] P^T
// The K index of a product may be any permutation of the channels (keys) that
// both operands share. Thread (g, t) = (lane / 4, lane % 4) owns channels
// [t D/4, ..) of key rows g and g + 8 for K, and channels [g D/8, ..) of keys
// 2t, 2t+1, 2t+8, 2t+9 for V: vector loads, and one scale per key (D/4 and
// D/8 divide a block of 32 or are one).
//
// 4 bits to 16. The products take u s with the nibble u = c + 8 >= 0, and the
// bias 8 s is taken off by one more product per 16 keys:
//   S^T: sum_d q_d (u_d - 8) s_d = sum_d q_d u_d s_d + sum_blocks s_blk (-8 sum_{d in blk} q_d)
//   O^T: sum_j p_j (u_j - 8) s_j = sum_j p_j u_j s_j - 8 sum_j p_j s_j
// u s has at most 8 significant bits, so it is exact in fp16, and costs half an
// instruction per element and half a multiply-add: a nibble in bits [3:0] of an
// fp16 whose constant is 1024 stands for 1024 + u, in bits [7:4] under 64 for
// 64 + u, and (B + u) s - B s needs B s to be exact only, which a power of two
// always is. Two of a word's four nibble pairs are in place, the other two
// after one shift. (With the bias inside, (B + 8) s must be exact, which takes
// smaller constants and a shift for every pair: 425 instructions per 16 keys
// instead of 330, and the integer pipe at its limit.) The scale is 2^-4 s, so
// that 1024 s stays in range. q is scaled by a power of two per row, exactly,
// to a largest element of 64 .. 128 (elements below 2^-23 of it lose bits),
// and -8 sum q is given as three fp16 parts. The rounding of p to fp16
// (2^-11; bf16 would have 2^-8) is the only one of the products, and is the
// same in both of O's sums. p is taken against a reference that starts 2^7 below
// the running maximum, and so uses fp16's range up to 2^15: a p of down to 2^-21 of
// the maximum keeps all 11 bits, and below that its error is at most 2^-32 of it
// (against the maximum itself, keys below 2^-25 of a sink were 0 in O and still
// counted in l). O's bias is taken off at the end of every step (32
// multiply-adds of a thread's 700 instructions at D = 128; 8 x 128K keys took 241 us
// with it and 243 without in one session): taken off once at the end, the sums'
// roundings were 0.33 % of O at 128K keys per head and 3.3 % at 1M, where bf16's
// own are 0.17 %.
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "internal.h"
#include "kv4.cuh"
#include "kv4_host.h"
#include "tc_ptx.cuh"

namespace usp {
namespace {

using namespace kv4;
using namespace tc;

__device__ int g_decode_kv4_status = 0;

constexpr int kStep = 32;                 // keys per step
constexpr int kGridMax = 304;             // 152 SMs x 2 resident CTAs
// Up to eight query rows: two CTAs of eight warps per SM at 128 registers;
// sixteen: one CTA (at D = 128, with ten or twelve warps at 168 registers and Q^T in
// shared memory, it spills: 63 and 69 us instead of 51 for 4 x 32K keys and 12 rows;
// D = 64 has the same form, and was not tried with more warps).
// Rows 9..16 as two blocks of eight read and decode every key twice: 76 us
// instead of 61 for 4 x 32K keys, 459 instead of 352 for 8 x 128K (12.3 instead
// of 14.7 for 2K keys of one sequence, which no rule is made for).
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// What a unit costs besides its steps, in steps: its last round is half empty on
// average, and the combination and the next queries take 2.8 us, a round of
// eight steps 2. (16 x 32 units of at most 33 steps: 37.2 us without it, 33.4
// with 8, 32.3 with 12, 33.1 with 16.)
constexpr int kUnitCost = 12;
// p = 2^(score - m), m the reference: set 2^kBelow below the running maximum, and
// moved when a score exceeds it by 2^kAbove (fp16 ends at 2^16).
constexpr float kBelow = 7.f, kAbove = 15.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  Cache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  float* o_part;    // [slots][8 NT][D], columns in the kernel's order
  float2* ml_part;  // [slots][8 NT]: (m, l), m the reference in log2 units
  int2* span;       // [units]: first and last slot (units that have steps)
  float2* scores;   // accumulate: [B][H][Rs / 2][C] log2-scaled scores of two rows
  int Tq, Hq, G, R, Rs, nrb;  // R = G Tq rows per KV head, nrb blocks of them
  int grid;
  int slots;                  // of partials
  float score_mul;            // times 2^score_exp: softmax scale * log2(e) * k_descale
  int score_exp;
  float v_descale;
  int causal, window, sink;
};

// What a sequence of L cached tokens has to visit: steps [0, sinks) and
// [first, ..), `n` in all.
struct SeqSteps {
  int n, sinks, skip;  // step s is key step s (s < sinks) or s + skip
};
__device__ __forceinline__ SeqSteps seq_steps(const Params& P, int L) {
  SeqSteps r{0, 0, 0};
  if (L <= 0) return r;
  const int all = (L + kStep - 1) / kStep;
  if (P.window > 0) {
    const int i0 = max(0, L - P.Tq);                 // first query position
    const int first = max(0, i0 - P.window + 1) / kStep;
    r.sinks = min((min(P.sink, L) + kStep - 1) / kStep, first);
    r.skip = first - r.sinks;
  }
  r.n = all - r.skip;
  return r;
}
__device__ __forceinline__ int seq_len(const Params& P, int b) {
  return clamp_len(__ldg(P.c.lens + b), P.c.C);
}

// Length of a unit of n steps on the line that the CTAs share.
__device__ __forceinline__ int line_len(int n) { return n > 0 ? n + kUnitCost : 0; }

// The sequences [b0, b0 + 32) on the line, one per lane: where each ends.
__device__ __forceinline__ long long line_ends(const Params& P, int b0, int per_seq) {
  const int b = b0 + (threadIdx.x & 31);
  long long inc = b < P.c.B ? (long long)line_len(seq_steps(P, seq_len(P, b)).n) * per_seq : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if ((threadIdx.x & 31) >= o) inc += x;
  }
  return inc;
}
__device__ __forceinline__ long long scaled(long long T, unsigned c, unsigned N) {  // T c / N
  if (T <= 0xffffffffLL / kGridMax) return (unsigned)T * c / N;  // (a 64-bit division is slow)
  return T * c / N;
}

// The launch of the dependent kernel may proceed; and, in that one: the kernel
// before it has ended and its writes are visible.
__device__ __forceinline__ void grid_dependency_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A walk over the steps of a CTA's run: the current unit's steps [s, end).
struct Walk {
  int b, hr;        // sequence, KV head * nrb + row block
  int s, end;       // of the unit
  int len;          // of the sequence
  SeqSteps q;
  long long row;    // before the head's first
  long long left;   // of the run's part of the line, behind this unit
};
__device__ __forceinline__ void enter_seq(const Params& P, Walk& w) {
  w.len = seq_len(P, w.b);
  w.q = seq_steps(P, w.len);
}
__device__ __forceinline__ bool next_unit(const Params& P, Walk& w) {
  if (w.left <= 0) return false;
  if (++w.hr == P.c.H * P.nrb) {
    w.hr = 0;
    do {
      if (++w.b >= P.c.B) return false;
      enter_seq(P, w);
    } while (w.q.n == 0);
  }
  w.row = head_row(P.c, w.b, w.hr / P.nrb);
  w.s = 0;
  w.end = (int)min((long long)w.q.n, w.left);
  w.left -= line_len(w.q.n);
  return true;
}

template <int D, int NT>
struct Smem {
  static constexpr int kKeys = kWarps * kStep;  // of a round
  // a stage: one round's codes and scales
  static constexpr int kCodes = kKeys * D / 2, kScales = kKeys * D / kBlock;
  static constexpr int kKC = 0, kVC = kCodes, kKS = 2 * kCodes, kVS = 2 * kCodes + kScales;
  static constexpr int kStageBytes = 2 * kCodes + 2 * kScales;
  static constexpr int kStages = D == 64 ? 4 : NT == 1 ? 2 : 3;
  static constexpr int kRedStride = D + 4;
  static constexpr int kRed = kStages * kStageBytes;              // [kWarps][8][D + 4]
  static constexpr int kML = kRed + kWarps * 8 * kRedStride * 4;  // [kWarps][8] float2
  static constexpr int kBar = kML + kWarps * 8 * 8;
  static constexpr int kMisc = kBar + 2 * kStages * 8;            // abort, run
  static constexpr int kBytes = kMisc + 64;
  static_assert(kBytes <= (NT == 1 ? 113 : 227) * 1024, "residency");
  static_assert(kRed % 16 == 0 && kML % 16 == 0 && kBar % 8 == 0 &&
                    kMisc % 16 == 0 && kStageBytes % 128 == 0,
                "alignment");
  static_assert(kStages <= kWarps, "a warp has at most one round's copies in flight");
};

__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// (x & mask) | base
template <uint32_t kMask, uint32_t kBase>
__device__ __forceinline__ uint32_t and_or(uint32_t x) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "n"(kMask), "n"(kBase));
  return d;
}
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

// Row of a 16-key tile that stands at index i (0..15) of the products' M (K)
// or K (V) side: neighbouring rows go to indices whose threads read together,
// so that a quarter (V: half) of a warp spreads over both halves of the banks.
__device__ __forceinline__ int tile_key(int i) { return i ^ ((i >> 1) & 1); }

// The four pairs (nibbles j and j + 4, j = 0..3) of a word of codes times a pair
// of scales: a[j] = u s. zb = -1024 s, zs = -64 s.
__device__ __forceinline__ void expand(uint32_t x, uint32_t s, uint32_t zb, uint32_t zs,
                                       uint32_t (&a)[4]) {
  const uint32_t y = x >> 8;
  a[0] = h2_fma(and_or<0x000F000Fu, 0x64006400u>(x), s, zb);
  a[1] = h2_fma(and_or<0x00F000F0u, 0x54005400u>(x), s, zs);
  a[2] = h2_fma(and_or<0x000F000Fu, 0x64006400u>(y), s, zb);
  a[3] = h2_fma(and_or<0x00F000F0u, 0x54005400u>(y), s, zs);
}

// Asks for a unit's query rows to be brought into L2, by one warp.
template <int D, int NT>
__device__ __forceinline__ void want_q(const Params& P, const Walk& w) {
  constexpr int kLines = D / 64;  // of 128 bytes
  const int h = w.hr / P.nrb, rb = w.hr - h * P.nrb;
  const int x = threadIdx.x & 31, r = rb * 8 * NT + x / kLines;
  static_assert(8 * NT * kLines <= 32, "a line per lane");
  if (x < 8 * NT * kLines && r < P.R) {
    const int hh = r / P.Tq, tok = r - hh * P.Tq;
    const __nv_bfloat16* p = P.q + (((long long)w.b * P.Tq + tok) * P.Hq + h * P.G + hh) * D +
                             x % kLines * 64;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
  }
}

// Starts the copies of the round that begins at w.s into a stage.
template <int D, int NT>
__device__ __forceinline__ void load_round(const Params& P, const Walk& w, uint32_t stage,
                                           uint32_t bar) {
  using L = Smem<D, NT>;
  const int s1 = min(w.s + kWarps, w.end), sp = min(max(w.q.sinks, w.s), s1);
  // rows of steps [a, e): whole 16-row groups that hold cached keys (the
  // capacity is a multiple of 16)
  auto rows_of = [&](int a, int e, int key0) {
    return min((e - a) * kStep, (w.len - key0 + kRowAlign - 1) / kRowAlign * kRowAlign);
  };
  // steps before the window's skip, and behind it
  const int k0 = w.s * kStep, k1 = (sp + w.q.skip) * kStep;
  const int n0 = sp > w.s ? rows_of(w.s, sp, k0) : 0, n1 = s1 > sp ? rows_of(sp, s1, k1) : 0;
  mbar_expect_tx(bar, static_cast<uint32_t>(n0 + n1) * 2 * (D / 2 + D / kBlock));
  auto piece = [&](int at, int key0, int n) {
    const long long row = w.row + key0;
    const uint32_t cb = n * (D / 2), sb = n * (D / kBlock);
    bulk_load(stage + L::kKC + at * (D / 2), P.c.kc + row * (D / 2), cb, bar);
    bulk_load(stage + L::kKS + at * (D / kBlock), P.c.ks + row * (D / kBlock), sb, bar);
    bulk_load(stage + L::kVC + at * (D / 2), P.c.vc + row * (D / 2), cb, bar);
    bulk_load(stage + L::kVS + at * (D / kBlock), P.c.vs + row * (D / kBlock), sb, bar);
  };
  if (n0 > 0) piece(0, k0, n0);
  if (n1 > 0) piece((sp - w.s) * kStep, k1, n1);
}

template <int D, int NT, bool SC>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1)
decode_kv4_kernel(const Params P) {
  using L = Smem<D, NT>;
  constexpr int kStages = L::kStages;
  constexpr int kRows = 8 * NT;
  constexpr int kWK = D / 32;      // 32-bit words of codes a thread has per K row
  constexpr int kWV = D / 64;      // and per V row
  constexpr int kMT = D / 16;      // 16-channel tiles of O^T
  extern __shared__ __align__(128) uint8_t sm[];
  const uint32_t sbase = smem_u32(sm);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kMisc);
  long long* run = reinterpret_cast<long long*>(sm + L::kMisc + 16);  // first step, count, ..
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  auto full = [&](int st) { return sbase + L::kBar + 8 * st; };
  auto empty = [&](int st) { return sbase + L::kBar + 8 * (kStages + st); };

  grid_dependency_launch();
  if (threadIdx.x == 32) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(full(st), 1);
      mbar_init(empty(st), kWarps);
    }
    fence_barrier_init();
  }
  if (warp == 0) {
    const int per_seq = P.c.H * P.nrb;
    long long ends = line_ends(P, 0, per_seq);
    long long T = __shfl_sync(0xffffffffu, ends, 31);
    for (int b = 32; b < P.c.B; b += 32)
      T += __shfl_sync(0xffffffffu, line_ends(P, b, per_seq), 31);
    const long long want = (T + kWarps - 1) / kWarps;
    const unsigned N = (unsigned)min(want, (long long)P.grid);
    long long first = 0, count = 0;
    if (blockIdx.x < N) {
      first = scaled(T, blockIdx.x, N);
      count = scaled(T, blockIdx.x + 1, N) - first;
    }
    // the sequence that holds `first`
    int b0 = 0;
    long long before = 0;
    if (count > 0) {
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
        if (b0 >= P.c.B) {  // not reached: first < T
          count = 0;
          break;
        }
        ends = line_ends(P, b0, per_seq);
      }
    }
    if (lane == 0) {
      run[0] = first - before;  // within sequence b0
      run[1] = count;
      run[2] = b0;
      *abort_flag = 0;
    }
  }
  __syncthreads();
  if (run[1] == 0) return;
  Walk cur;
  {
    cur.b = (int)run[2];
    enter_seq(P, cur);
    const int n = cur.q.n, ln = line_len(n);
    cur.hr = run[0] <= 0xffffffffLL ? (int)((unsigned)run[0] / ln) : (int)(run[0] / ln);
    const int at = (int)(run[0] - (long long)cur.hr * ln);
    cur.row = head_row(P.c, cur.b, cur.hr / P.nrb);
    cur.s = at;
    cur.end = (int)min((long long)n, at + run[1]);
    cur.left = run[1] - (ln - at);
    // the run may begin behind a unit's last step, and end there too
    if (at >= n && !next_unit(P, cur)) return;
  }
  // Q is fetched ahead of use, and here ahead of the copies that it would
  // otherwise queue behind (2 us)
  if (warp == 0) want_q<D, NT>(P, cur);
  // the copies run kStages rounds ahead of the computation, over the ends of
  // units; the warps issue them in turn
  Walk pre = cur;
  bool more = true;
  int issued = 0, used = 0, mine = -1;  // rounds; the last one this warp issued
  auto issue = [&]() {
    if (warp == issued % kWarps) {
      mine = issued;
      const int st = issued % kStages;
      if (lane == 0)
        load_round<D, NT>(P, pre, sbase + st * L::kStageBytes, full(st));
    }
    ++issued;
    pre.s += kWarps;
    if (pre.s >= pre.end) {
      more = next_unit(P, pre);
      if (more && warp == issued % kWarps) want_q<D, NT>(P, pre);
    }
  };
#pragma unroll
  for (int st = 0; st < kStages; ++st)
    if (more) issue();

  const __half2 k2m4 = __float2half2_rn(0.0625f);
  const __half2 m1024 = __float2half2_rn(-1024.f), m64 = __float2half2_rn(-64.f);
  bool ok = true;
  for (;;) {
    // ---------------------------------------------------------------- a unit
    const int b = cur.b, h = cur.hr / P.nrb, rb = cur.hr - h * P.nrb;
    const int len = cur.len;
    const SeqSteps steps = cur.q;
    // Q^T fragments: product kk = 2w + jj takes channels (8w + 2jj, + 4) and
    // (8w + 2jj + 1, + 4) of the thread's run of D/4; qb: -8 times the run's
    // (its block's part's) sum in three parts
    uint32_t qf[NT][2 * kWK][2], qb[NT][2];
    float mul[NT][2];  // of rows 2t, 2t + 1: scores to log2 units
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = rb * kRows + nt * 8 + g;
      const __nv_bfloat16* src = nullptr;
      if (r < P.R) {
        const int hh = r / P.Tq, tok = r - hh * P.Tq;
        src = P.q + (((long long)b * P.Tq + tok) * P.Hq + h * P.G + hh) * D + t * (D / 4);
      }
      uint4 x[kWK];
      float big = 0.f;
#pragma unroll
      for (int w = 0; w < kWK; ++w) {
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
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWK; ++w) {
        const uint32_t e[4] = {x[w].x, x[w].y, x[w].z, x[w].w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = __uint_as_float(e[i] << 16) * up;
          f[2 * i + 1] = __uint_as_float(e[i] & 0xffff0000u) * up;
        }
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __half2 p = __floats2half2_rn(f[2 * jj + i], f[2 * jj + i + 4]);
            qf[nt][2 * w + jj][i] = half2_bits(p);
            const float2 back = __half22float2(p);
            sum += back.x + back.y;
          }
      }
      sum *= -8.f;
      const __half hi = __float2half_rn(sum);
      const float rest = sum - __half2float(hi);
      const __half mid = __float2half_rn(rest);
      qb[nt][0] = half2_bits(__halves2half2(hi, mid));
      qb[nt][1] = half2_bits(__floats2half2_rn(rest - __half2float(mid), 0.f));
      // 2^4 for the scale's 2^-4; not 0 or infinite, which a masked key's -inf or a
      // score of 0 would make NaN
      const float row_mul =
          fminf(fmaxf(ldexpf(P.score_mul, P.score_exp + ex - 6 + 4), FLT_MIN), FLT_MAX);
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
    const int i_first = len - P.Tq;  // position of token 0
    for (int s0 = cur.s; s0 < cur.end; s0 += kWarps) {
     const int st = used % kStages, s = s0 + warp;
     // A warp without a step in the unit's last round waits for the copies too:
     // they are issued once every warp has released the stage's round before, so
     // its arrival on `empty` below cannot count for that round, in place of a
     // warp that still reads it.
     if (!mbar_wait(full(st), (used / kStages) & 1, abort_flag, &g_decode_kv4_status)) ok = false;
     if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
     if (s < cur.end) {
      const uint8_t* stp = sm + st * L::kStageBytes;
      const uint8_t* kcodes = stp + L::kKC + warp * (kStep * D / 2);
      const uint8_t* vcodes = stp + L::kVC + warp * (kStep * D / 2);
      const uint8_t* kscales = stp + L::kKS + warp * (kStep * D / kBlock);
      const uint8_t* vscales = stp + L::kVS + warp * (kStep * D / kBlock);
      const int key0 = (s < steps.sinks ? s : s + steps.skip) * kStep;
      // does the mask (or the sequence's end) hide any of the step's keys?
      const int last = key0 + kStep - 1;
      const bool masked = last >= len || i_first < 0 || (P.causal && last > i_first) ||
                          (P.window > 0 && len - 1 - key0 >= P.window);
      // ------------------------------------------------------------ scores
      float sc[NT][2][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r0 = 16 * half + tile_key(g), r1 = r0 + 8;
        uint32_t k0[kWK], k1[kWK];
        const uint8_t* kc = kcodes + t * (D / 8);
        if constexpr (D == 128) {
          const uint4 a = *reinterpret_cast<const uint4*>(kc + r0 * (D / 2));
          const uint4 c = *reinterpret_cast<const uint4*>(kc + r1 * (D / 2));
          k0[0] = a.x; k0[1] = a.y; k0[2] = a.z; k0[3] = a.w;
          k1[0] = c.x; k1[1] = c.y; k1[2] = c.z; k1[3] = c.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(kc + r0 * (D / 2));
          const uint2 c = *reinterpret_cast<const uint2*>(kc + r1 * (D / 2));
          k0[0] = a.x; k0[1] = a.y;
          k1[0] = c.x; k1[1] = c.y;
        }
        const uint8_t* ks = kscales + (t * (D / 4)) / kBlock;
        const __half2 ss = __hmul2(
            e4m3x2_to_half2(ks[r0 * (D / kBlock)] | (ks[r1 * (D / kBlock)] << 8)), k2m4);
        const uint32_t s0 = half2_bits(__low2half2(ss)), s1 = half2_bits(__high2half2(ss));
        const __half2 zb = __hmul2(ss, m1024), zs = __hmul2(ss, m64);
        const uint32_t zb0 = half2_bits(__low2half2(zb)), zb1 = half2_bits(__high2half2(zb));
        const uint32_t zs0 = half2_bits(__low2half2(zs)), zs1 = half2_bits(__high2half2(zs));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][half][e] = 0.f;
          // the bias: thread t's K indices stand for its block (D = 64: its
          // half of the block)
          const uint32_t a[4] = {s0, s1, s0, s1};
          mma_f16(sc[nt][half], a, qb[nt][0], qb[nt][1]);
        }
#pragma unroll
        for (int w = 0; w < kWK; ++w) {
          // nibbles j and j + 4 of a word: channels 8w + j, 8w + 4 + j
          uint32_t p0[4], p1[4];
          expand(k0[w], s0, zb0, zs0, p0);
          expand(k1[w], s1, zb1, zs1, p1);
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const uint32_t a[4] = {p0[2 * jj], p1[2 * jj], p0[2 * jj + 1], p1[2 * jj + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(sc[nt][half], a, qf[nt][2 * w + jj][0], qf[nt][2 * w + jj][1]);
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
              const int j = key0 + 16 * half + tile_key(g) + 8 * (e >> 1);
              const int tok = (rb * kRows + nt * 8 + 2 * t + (e & 1)) % P.Tq;
              const int i = i_first + tok;
              const bool see = j < len && i >= 0 && (!P.causal || j <= i) &&
                               (P.window <= 0 || i - j < P.window || j < P.sink);
              if (!see) sc[nt][half][e] = -INFINITY;
            }
      }
      bool grow = false;
      float mx[NT][2];  // in log2 units (the factor is positive)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nt][e] = mul[nt][e] * fmaxf(fmaxf(sc[nt][0][e], sc[nt][0][e + 2]),
                                         fmaxf(sc[nt][1][e], sc[nt][1][e + 2]));
          grow |= mx[nt][e] > m[nt][e] + kAbove;
        }
      if constexpr (SC) {
        // the weights need every score once the whole row's sum is known
        float2* dst = P.scores + head_row(P.c, b, h) * (P.Rs / 2);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = rb * kRows + nt * 8 + 2 * t;
          if (r >= P.Rs) continue;
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const int j = key0 + 16 * half + tile_key(g) + 8 * (e >> 1);
              if (j < len)
                dst[(long long)(r / 2) * P.c.C + j] =
                    make_float2(sc[nt][half][e] * mul[nt][0], sc[nt][half][e + 1] * mul[nt][1]);
            }
        }
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
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -INFINITY ? 0.f : -m[nt][0];
        const float m1 = m[nt][1] == -INFINITY ? 0.f : -m[nt][1];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[e] = ex2(fmaf(sc[nt][half][e], mul[nt][e & 1], (e & 1) ? m1 : m0));
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
          pf[nt][half][0] = movmatrix_t(half2_bits(__floats2half2_rn(p[0], p[1])));
          pf[nt][half][1] = movmatrix_t(half2_bits(__floats2half2_rn(p[2], p[3])));
        }
      }
      // -------------------------------------------------------------- P V
      float ob[NT][4];  // sum_j p_j s_j of the step
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) ob[nt][e] = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int ka = 16 * half + tile_key(2 * t), kb = 16 * half + tile_key(2 * t + 1);
        const int keys[4] = {ka, kb, ka + 8, kb + 8};
        uint32_t vw[4][kWV], sb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* vc = vcodes + keys[i] * (D / 2) + g * (D / 16);
          if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(vc);
            vw[i][0] = x.x;
            vw[i][1] = x.y;
          } else {
            vw[i][0] = *reinterpret_cast<const uint32_t*>(vc);
          }
          sb[i] = vscales[keys[i] * (D / kBlock) + (g * (D / 8)) / kBlock];
          // rows behind the sequence hold anything: 0, so that 0 * it is 0
          if (masked && key0 + keys[i] >= len) sb[i] = 0;
        }
        const __half2 sab = __hmul2(e4m3x2_to_half2(sb[0] | (sb[1] << 8)), k2m4);
        const __half2 scd = __hmul2(e4m3x2_to_half2(sb[2] | (sb[3] << 8)), k2m4);
        const uint32_t s0 = half2_bits(sab), s1 = half2_bits(scd);
        const uint32_t zb0 = half2_bits(__hmul2(sab, m1024)), zs0 = half2_bits(__hmul2(sab, m64));
        const uint32_t zb1 = half2_bits(__hmul2(scd, m1024)), zs1 = half2_bits(__hmul2(scd, m64));
        // row g of the bias product is the scale of the thread's own channels
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t a[4] = {s0, 0u, s1, 0u};
          mma_f16(ob[nt], a, pf[nt][half][0], pf[nt][half][1]);
        }
#pragma unroll
        for (int w = 0; w < kWV; ++w) {
          // channels 8w + 0..3 (low halves) and 8w + 4..7 of both keys
          uint32_t xl[4], xh[4], yl[4], yh[4];
          expand(__byte_perm(vw[0][w], vw[1][w], 0x5410), s0, zb0, zs0, xl);
          expand(__byte_perm(vw[0][w], vw[1][w], 0x7632), s0, zb0, zs0, xh);
          expand(__byte_perm(vw[2][w], vw[3][w], 0x5410), s1, zb1, zs1, yl);
          expand(__byte_perm(vw[2][w], vw[3][w], 0x7632), s1, zb1, zs1, yh);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a[4] = {xl[j], xh[j], yl[j], yh[j]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(o[nt][4 * w + j], a, pf[nt][half][0], pf[nt][half][1]);
          }
        }
      }
      // the bias comes off in every step: with it, the sum outgrows O by the
      // number of keys over its root, and the products' roundings go with the sum
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][i][e] = fmaf(-8.f, ob[nt][e & 1], o[nt][i][e]);
     }
      __syncwarp();  // the stage has been read
      if (lane == 0) mbar_arrive(empty(st));
      if (more) {
        // the round after the next ones goes where this one was, once every
        // warp is done with it
        if (warp == issued % kWarps) {
          ok = mbar_wait(empty(st), (used / kStages) & 1, abort_flag, &g_decode_kv4_status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        issue();
      }
      ++used;
    }
    // ------------------------------------------------- the unit's partial
    // O in the order (tile i, half, g): element 16 i + 8 half + g of a row is
    // channel g D/8 + 8 (i / 4) + i % 4 + 4 half
    const int unit = b * P.c.H * P.nrb + cur.hr;
    const long long slot = (long long)blockIdx.x + unit;
    if (threadIdx.x == 0) {
      if (cur.s == 0) P.span[unit].x = (int)slot;
      if (cur.end == steps.n) P.span[unit].y = (int)slot;
    }
    float* red = reinterpret_cast<float*>(sm + L::kRed);
    float2* ml = reinterpret_cast<float2*>(sm + L::kML);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rows = min(8, P.R - rb * kRows - nt * 8);  // that exist
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (g == 0) ml[warp * 8 + 2 * t + e] = make_float2(m[nt][e], x);
      }
      float* mine = red + (warp * 8 + 2 * t) * L::kRedStride + g;
      if (2 * t < rows) {
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
          mine[16 * i] = o[nt][i][0];
          mine[L::kRedStride + 16 * i] = o[nt][i][1];
          mine[16 * i + 8] = o[nt][i][2];
          mine[L::kRedStride + 16 * i + 8] = o[nt][i][3];
        }
      }
      __syncthreads();
      for (int x = threadIdx.x; x < rows * D; x += kThreads) {
        const int r = x / D, d = x - r * D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * 8 + r].x);
        float os = 0.f, ls = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 a = ml[w * 8 + r];
          const float f = a.x == -INFINITY ? 0.f : ex2(a.x - M);
          ls += a.y * f;
          os += red[(w * 8 + r) * L::kRedStride + d] * f;
        }
        P.o_part[(slot * kRows + nt * 8 + r) * D + d] = os;
        if (d == 0) P.ml_part[slot * kRows + nt * 8 + r] = make_float2(M, ls);
      }
      __syncthreads();
    }
    if (*abort_flag) break;
    if (!next_unit(P, cur)) break;
  }
  // aborted: the copies that this warp has in flight land before the CTA ends
  if (lane == 0 && *abort_flag && mine >= 0)
    mbar_wait_drain(full(mine % kStages), (mine / kStages) & 1);
}

constexpr int kMergeThreads = 256;
// Keys per thread at a time, and, with the six pairs of rows unrolled, scores in
// flight (4 x 32K keys, 12 rows, 50 MB of scores in L2: 24 us; with two pairs 29,
// with two keys in twice as many blocks 23 to 27, with one key 31).
constexpr int kWeightKeys = 4;
constexpr int kMaxWeightRows = 64;  // (m, 1 / l) kept at a time

// A unit's first and last slot. Where a wait of the kernel before gave up (which
// usp_device_status reports), they may never have been written: whatever stands
// there, only slots that exist are read.
__device__ __forceinline__ int2 span_of(const Params& P, int unit) {
  const int2 s = P.span[unit];
  return make_int2(max(s.x, 0), min(s.y, P.slots - 1));
}

// Block x < units * 8 NT: a row of a unit, whose partials (consecutive slots)
// are merged in key order by D threads per part of them. Blocks behind those
// (accumulate): a piece of the keys of a (sequence, KV head):
//   key_weight[j] += sum over the rows of 2^(score - m) / l.
// Launched while the kernel above still runs; nothing it writes is read before
// the wait.
template <int D, int NT, bool SC>
__global__ void __launch_bounds__(kMergeThreads) merge_kv4_kernel(const Params P, int pieces) {
  constexpr int kRows = 8 * NT;
  constexpr int kParts = kMergeThreads / D;
  __shared__ float s_o[kParts][D];
  __shared__ float2 s_ml[SC && kMaxWeightRows > kParts ? kMaxWeightRows : kParts];
  const int per_seq = P.c.H * P.nrb;
  const int merges = P.c.B * per_seq * kRows;
  if (!SC || (int)blockIdx.x < merges) {
    const int unit = blockIdx.x / kRows, r = blockIdx.x % kRows;  // r: row within the block
    const int b = unit / per_seq, hr = unit - b * per_seq;
    const int h = hr / P.nrb, rb = hr - h * P.nrb;
    const int row = rb * kRows + r;
    if (row >= P.R) return;
    int2 span = make_int2(0, -1);  // no steps, no partials
    const bool some = seq_steps(P, seq_len(P, b)).n > 0;
    grid_dependency_wait();
    if (some) span = span_of(P, unit);
    const int part = threadIdx.x / D, d = threadIdx.x - part * D;
    float M = -INFINITY, ls = 0.f, os = 0.f;
    #pragma unroll 2
    for (long long s = span.x + part; s <= span.y; s += kParts) {
      const float2 a = P.ml_part[s * kRows + r];
      const float x = P.o_part[(s * kRows + r) * D + d];
      const float Mn = fmaxf(M, a.x);
      const float f0 = M == -INFINITY ? 0.f : ex2(M - Mn);
      const float f1 = a.x == -INFINITY ? 0.f : ex2(a.x - Mn);
      os = os * f0 + x * f1;
      ls = ls * f0 + a.y * f1;
      M = Mn;
    }
    s_o[part][d] = os;
    if (d == 0) s_ml[part] = make_float2(M, ls);
    __syncthreads();
    if (part != 0) return;
    float Mt = -INFINITY;
#pragma unroll
    for (int i = 0; i < kParts; ++i) Mt = fmaxf(Mt, s_ml[i].x);
    float lt = 0.f, ot = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const float f = s_ml[i].x == -INFINITY ? 0.f : ex2(s_ml[i].x - Mt);
      lt += s_ml[i].y * f;
      ot += s_o[i][d] * f;
    }
    const int hh = row / P.Tq, tok = row - hh * P.Tq;
    const long long o_row = ((long long)b * P.Tq + tok) * P.Hq + h * P.G + hh;
    const bool none = lt == 0.f;  // no visible key (a NaN score makes lt NaN)
    const float inv = none ? 0.f : 1.f / lt;
    const int i = d >> 4, half = (d >> 3) & 1, g = d & 7;
    const int ch = g * (D / 8) + 8 * (i >> 2) + (i & 3) + 4 * half;
    // (the kernel's V is 2^-4 of the cache's)
    P.out[o_row * D + ch] = __float2bfloat16_rn(none ? 0.f : ot * inv * 16.f * P.v_descale);
    if (d == 0) P.lse[o_row] = none ? -INFINITY : (Mt + log2f(lt)) * kLn2;
    return;
  }
  if constexpr (SC) {
    const int x = blockIdx.x - merges, piece = x % pieces, bh = x / pieces;
    const int b = bh / P.c.H, h = bh - b * P.c.H;
    const int len = seq_len(P, b);
    const SeqSteps q = seq_steps(P, len);
    const long long head = head_row(P.c, b, h);
    const int keys = q.n * kStep;
    int k0 = piece * (kWeightKeys * kMergeThreads);
    if (k0 >= keys) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    for (; k0 < keys; k0 += pieces * (kWeightKeys * kMergeThreads)) {
      int j[kWeightKeys];
      float old[kWeightKeys], w[kWeightKeys];  // (the step's sum is added at once)
#pragma unroll
      for (int u = 0; u < kWeightKeys; ++u) {
        const int i = k0 + u * kMergeThreads + threadIdx.x, s = i / kStep;
        j[u] = (s < q.sinks ? s : s + q.skip) * kStep + i % kStep;
        if (i >= keys || j[u] >= len) j[u] = -1;
        old[u] = j[u] >= 0 ? P.c.w[head + j[u]] : 0.f;
        w[u] = 0.f;
      }
      for (int r0 = 0; r0 < P.R; r0 += kMaxWeightRows) {
        const int n = min(kMaxWeightRows, P.Rs - r0);
        __syncthreads();
        for (int r = warp; r < n; r += kMergeThreads / 32) {  // a warp per row
          const int rb = (r0 + r) / kRows, rr = r0 + r - rb * kRows;
          const int2 span = span_of(P, b * per_seq + h * P.nrb + rb);
          float M = -INFINITY, l = 0.f;
          for (long long i = span.x + lane; i <= span.y; i += 32)
            M = fmaxf(M, P.ml_part[i * kRows + rr].x);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
          for (long long i = span.x + lane; i <= span.y; i += 32) {
            const float2 a = P.ml_part[i * kRows + rr];
            l += a.y * (a.x == -INFINITY ? 0.f : ex2(a.x - M));
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          const bool none = l == 0.f || r0 + r >= P.R;
          if (lane == 0) s_ml[r] = make_float2(none ? 0.f : M, none ? 0.f : 1.f / l);
        }
        __syncthreads();
        const float2* sc = P.scores + head * (P.Rs / 2) + (long long)(r0 / 2) * P.c.C;
#pragma unroll 6
        for (int r = 0; r < n; r += 2) {
          const float2 a0 = s_ml[r], a1 = s_ml[r + 1];
          const bool odd = r0 + r + 1 >= P.R;  // the last row's partner was never written
#pragma unroll
          for (int u = 0; u < kWeightKeys; ++u) {
            if (j[u] < 0) continue;
            const float2 v = sc[(long long)(r / 2) * P.c.C + j[u]];
            w[u] += ex2(v.x - a0.x) * a0.y;
            if (!odd) w[u] += ex2(v.y - a1.x) * a1.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kWeightKeys; ++u)
        if (j[u] >= 0) P.c.w[head + j[u]] = old[u] + w[u];
    }
  }
}

// ------------------------------------------------------------------- host
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Ws {
  size_t o, ml, span, scores, total;
};
int tiles_for(int R) { return R <= 8 ? 1 : 2; }

Ws layout(int B, int Tq, int C, int Hq, int Hkv, int D, int accumulate) {
  const long long R = (long long)(Hq / Hkv) * Tq;
  const int rows = 8 * tiles_for((int)(R < 16 ? R : 16));
  const long long nrb = (R + rows - 1) / rows;
  const long long slots = (long long)B * Hkv * nrb + kGridMax;
  const long long Rs = (R + 1) / 2 * 2;
  Ws w{};
  size_t at = 0;
  w.o = at;
  at += up256((size_t)slots * rows * D * 4);
  w.ml = at;
  at += up256((size_t)slots * rows * 8);
  w.span = at;
  at += up256((size_t)B * Hkv * nrb * 8);
  if (accumulate) {
    w.scores = at;
    at += up256((size_t)B * Hkv * C * Rs * 4);
  }
  w.total = at;
  return w;
}

template <int D, int NT, bool SC>
usp_status_t launch_t(const Params& P, cudaStream_t st) {
  const int smem = Smem<D, NT>::kBytes;
  static SmemAttr attr;
  cudaError_t e = attr.set(decode_kv4_kernel<D, NT, SC>, smem);
  if (e != cudaSuccess) return fail_cuda("cudaFuncSetAttribute(smem)", e);
  long long blocks = (long long)P.c.B * P.c.H * P.nrb * 8 * NT;
  int pieces = 0;
  if constexpr (SC) {
    const int most = (P.c.C + kWeightKeys * kMergeThreads - 1) / (kWeightKeys * kMergeThreads);
    const int want = 152 * 6 / (P.c.B * P.c.H) + 1;  // most of the GPU's warps, over the heads
    pieces = most < want ? most : want;
    blocks += (long long)P.c.B * P.c.H * pieces;
  }
  if (blocks > 0x7fffffffLL) return USP_ERR_UNSUPPORTED;
  {
    ProfScope ps(st, "attn_decode_kv4");
    decode_kv4_kernel<D, NT, SC><<<P.grid, kThreads, smem, st>>>(P);
  }
  note_launch();
  usp_status_t r = check_launch();
  if (r != USP_OK) return r;
  // the merge's launch and set-up overlap the end of the kernel before it
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  {
    ProfScope ps(st, "attn_decode_kv4_merge");
    e = cudaLaunchKernelEx(&cfg, merge_kv4_kernel<D, NT, SC>, P, pieces);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail_cuda("kernel launch", e);
  }
  note_launch();
  return USP_OK;
}

template <int D>
usp_status_t launch_d(const Params& P, int nt, cudaStream_t st) {
  if (P.scores) return nt == 1 ? launch_t<D, 1, true>(P, st) : launch_t<D, 2, true>(P, st);
  return nt == 1 ? launch_t<D, 1, false>(P, st) : launch_t<D, 2, false>(P, st);
}

}  // namespace

size_t decode_kv4_workspace(int B, int Tq, int C, int Hq, int Hkv, int D, int accumulate) {
  return layout(B, Tq, C, Hq, Hkv, D, accumulate).total;
}

usp_status_t launch_decode_kv4(const DecodeKv4Args& a, void* workspace, cudaStream_t st) {
  const Ws w = layout(a.c.B, a.Tq, a.c.C, a.Hq, a.c.H, a.D, a.accumulate);
  char* base = static_cast<char*>(workspace);
  Params P{};
  P.c = a.c;
  P.q = static_cast<const __nv_bfloat16*>(a.q);
  P.out = static_cast<__nv_bfloat16*>(a.out);
  P.lse = a.lse;
  P.o_part = reinterpret_cast<float*>(base + w.o);
  P.ml_part = reinterpret_cast<float2*>(base + w.ml);
  P.span = reinterpret_cast<int2*>(base + w.span);
  if (a.accumulate) {
    P.scores = reinterpret_cast<float2*>(base + w.scores);
  }
  P.Tq = a.Tq;
  P.Hq = a.Hq;
  P.G = a.Hq / a.c.H;
  P.R = P.G * a.Tq;
  P.Rs = (P.R + 1) / 2 * 2;
  const int nt = tiles_for(P.R);
  P.nrb = (P.R + 8 * nt - 1) / (8 * nt);
  P.grid = nt == 1 ? kGridMax : kGridMax / 2;
  P.slots = P.c.B * P.c.H * P.nrb + kGridMax;  // as layout() has them
  // (the product alone may be beyond fp32)
  P.score_mul = (float)std::frexp((double)a.scale * kLog2e * a.k_descale, &P.score_exp);
  P.v_descale = a.v_descale;
  P.causal = a.causal;
  P.window = a.window;
  P.sink = a.sink;
  return a.D == 128 ? launch_d<128>(P, nt, st) : launch_d<64>(P, nt, st);
}

int read_clear_decode_kv4_status() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_decode_kv4_status, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0) cudaMemcpyToSymbol(g_decode_kv4_status, &z, sizeof(int));
  return v;
}

}  // namespace usp
