// Attention of the newest tokens to the paged 8-bit KV cache on the 5th-generation
// tensor cores (tcgen05): chunks of a prompt, many query rows per KV head.
//
// A unit is 256 query rows of one (sequence, KV head), in two halves of 128; a step
// is 128 of its keys. The rows of a KV head are its tokens' query heads, token by
// token, so a half covers 128 / G neighbouring tokens and every K and V row that is
// read serves all of them. All steps of all units are one line that the CTAs share
// in equal runs (as in attn_kv8.cu), so ragged batches and causal triangles are
// balanced; a unit that lies in one run is written at once, the others' partials
// (m, l, O) go through the workspace to a second kernel.
//
// One persistent CTA per SM, 16 warps:
//   warps 0-3, 4-7  softmax of half A and B, one query row per thread: scores from
//                   tensor memory, p = 2^(score + e_v - m) back over them as fp16
//   warps 8-11      converters: E4M3 codes to fp16 tiles in shared memory, once for
//                   both halves (exact; the products need both operands of one type)
//   warp 12         producer: pages and exponents of the tiles, TMA of the codes
//   warps 13, 14    MMA issuers of half A and B (one thread each); 13 owns the tensor memory
// Tensor memory, for each half: scores of 64 keys in two places of 64 columns (P over
// them as fp16), and O. So the products of one place, P V of its keys and then Q K of the
// next step's, run while the softmax works on the other; the halves share the tiles
// and nothing else.
//
// 4096 tokens at the end of 16K keys, 32 query heads over 8, D = 128 (0.96 TFLOP): 805 us,
// 0.64 of the measured bf16 rate; 512 tokens at 32K: 244 us; a packed batch of single
// tokens and chunks: 141 us. What bounds it is the chain from one role to the next more
// than any unit: of a step's 4100 clocks the tensor core is busy 2560 (its products of 64
// keys with both operands in shared memory take 48 clocks for 32 of arithmetic), shared
// memory about 3000, a tile's conversion 1000 for K and 1000 for V, each hand-over 200 to
// 300. At 822 us the conversions left out saved 4 %, the exponentials and the maximum 2 %,
// most of the products 6 %. Copies of the next step but one into L2 gave 1 %, a path
// without the test of rows for whole tiles 1 %. Also measured, at 822 us: scores of 128 keys
// in one place 983 us; one place for both halves 1062; P apart from the scores, which then
// come a part ahead, 977; one half per CTA with 128 keys in two places and K's codes
// as they are (q as the sum of two E4M3 numbers) 1010; two such CTAs per SM with one
// place 1032. Units of at most 128 rows with both halves on the same rows and every other
// tile each: no faster (4 x 64K keys, 128 rows 214 us; the converters' chain of hand-overs
// bounds them), and 10 % slower for the others by spills.
// The numbers are attn_kv8.cu's: q scaled to fp16 by a power of two per row, K's
// exponent a factor of the block's scores, V's added to them, p against a reference
// 2^7 to 2^15 below the running maximum of score + e_v, the row's sum over p 2^-e_v.
#include <cuda_fp16.h>

#include <cfloat>
#include <type_traits>

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

__device__ int g_attn_kv8_tc_status = 0;

constexpr int kBM = 128;                 // rows of a half
constexpr int kUnitRows = 2 * kBM;
constexpr int kBN = 128;                 // keys of a step
constexpr int kBlocks = kBN / kBlock;    // exponents of a step
constexpr int kSub = 64;                 // keys whose scores are made at once
constexpr int kGrid = 152;
constexpr int kThreads = 512;
constexpr int kConvWarp = 8, kConvWarps = 4, kProducerWarp = 12, kMmaWarp = 13;
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;  // 2 x 128 x (184 + 72) = 512 x 128
// What a unit costs besides its steps, in steps (its queries, its end; the packed batch
// takes 168 us with 1, 158 with 2, 149 with 4 and 6, 151 with 8), and the fewest steps that
// are worth a run of their own.
constexpr int kUnitCost = 6;
constexpr int kRunMin = 3;
constexpr int kInfo = 8;                 // steps whose description is kept
constexpr float kBelow = 7.f, kAbove = 15.f;
constexpr float kLn2 = 0.6931471805599453f;

// A step as the producer describes it.
constexpr int kHasB = 1, kFirst = 2, kLast = 4, kEnd = 8;
struct Info {
  int key0;
  int flags;        // k*; bits 8..: blocks that hold no key; bits 16..: keys below len
  uint32_t ke, ve;  // exponents of the blocks, int8
};

struct TcParams {
  Cache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  float* o_part;    // [2 kGrid][D / 4][256] of four channels
  float2* ml_part;  // [2 kGrid][256]
  int4* rec;        // [2 kGrid]: 1 a partial, 3 its unit's last; b, rt, h
  const int* cu;
  int T, max_new, Hq, G;
  float score_mul;
  int causal, window, sink;
};

struct Seq {
  int len, n, first, R, nt;
};
__device__ __forceinline__ Seq seq_of(const TcParams& P, int b) {
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
  q.nt = (q.R + kUnitRows - 1) / kUnitRows;
  return q;
}
// Steps of a unit: key tile s (s < sinks) or s + skip.
struct Steps {
  int n, sinks, skip;
};
__device__ __forceinline__ Steps steps_of(const TcParams& P, const Seq& q, int rt) {
  Steps r{0, 0, 0};
  const int t0 = rt * kUnitRows / P.G, t1 = (min(q.R, (rt + 1) * kUnitRows) - 1) / P.G;
  const int i0 = max(0, q.len - q.n + t0), i1 = q.len - q.n + t1;
  if (q.len <= 0 || i1 < 0) return r;
  const int last = (P.causal ? min(i1, q.len - 1) : q.len - 1) / kBN;
  int first = 0;
  if (P.window > 0) {
    first = max(0, i0 - P.window + 1) / kBN;
    r.sinks = min((min(P.sink, q.len) + kBN - 1) / kBN, first);
    r.skip = first - r.sinks;
  }
  r.n = last + 1 - r.skip;
  return r;
}
__device__ __forceinline__ int line_len(int n) { return n + kUnitCost; }

// A walk over the steps of a CTA's run: the current unit's steps [s, end).
struct Walk {
  int b, rt, h;
  Seq q;
  Steps st;
  int s, end;
  long long left;
};
__device__ __forceinline__ bool next_unit(const TcParams& P, Walk& w) {
  if (w.left <= 0) return false;
  if (++w.h == P.c.H) {
    w.h = 0;
    if (++w.rt >= w.q.nt) {
      w.rt = 0;
      do {
        if (++w.b >= P.c.B) return false;
        w.q = seq_of(P, w.b);
      } while (w.q.nt == 0);
    }
    w.st = steps_of(P, w.q, w.rt);
  }
  w.s = 0;
  w.end = (int)min((long long)w.st.n, w.left);
  w.left -= line_len(w.st.n);
  return true;
}

// Length on the line of a sequence's units of one head, by a warp.
__device__ __forceinline__ long long seq_line(const TcParams& P, const Seq& q) {
  long long x = 0;
  for (int rt = threadIdx.x & 31; rt < q.nt; rt += 32) x += line_len(steps_of(P, q, rt).n);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ long long scan32(long long x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}
// The sequences [b0, b0 + 32) on the line, one per lane: where each ends.
__device__ __forceinline__ long long line_ends(const TcParams& P, int b0) {
  const int lane = threadIdx.x & 31, b = b0 + lane;
  Seq q{};
  if (b < P.c.B) q = seq_of(P, b);
  long long x = 0;
  if (!__any_sync(0xffffffffu, q.nt > 4)) {
    for (int rt = 0; rt < q.nt; ++rt) x += line_len(steps_of(P, q, rt).n);
  } else {
    for (int i = 0; i < 32 && b0 + i < P.c.B; ++i) {
      const long long y = seq_line(P, seq_of(P, b0 + i));
      if (lane == i) x = y;
    }
  }
  return scan32(x * P.c.H);
}

// This CTA's run, found by one warp. left == 0: none.
__device__ __forceinline__ Walk find_run(const TcParams& P) {
  Walk w{};
  const int lane = threadIdx.x & 31;
  long long ends = line_ends(P, 0);
  long long T = __shfl_sync(0xffffffffu, ends, 31);
  for (int b = 32; b < P.c.B; b += 32) T += __shfl_sync(0xffffffffu, line_ends(P, b), 31);
  const long long N = min((T + kRunMin - 1) / kRunMin, (long long)gridDim.x);
  if (blockIdx.x >= N) return w;
  const long long first = T * blockIdx.x / N, count = T * (blockIdx.x + 1) / N - first;
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
    if (b0 >= P.c.B) return w;  // not reached: first < T
    ends = line_ends(P, b0);
  }
  w.b = b0;
  w.q = seq_of(P, b0);
  for (int rt0 = 0;; rt0 += 32) {
    const int rt = rt0 + lane;
    const long long x =
        scan32(rt < w.q.nt ? (long long)line_len(steps_of(P, w.q, rt).n) * P.c.H : 0);
    const unsigned over = __ballot_sync(0xffffffffu, before + x > first);
    if (over) {
      const int src = __ffs(over) - 1;
      if (src > 0) before += __shfl_sync(0xffffffffu, x, src - 1);
      w.rt = rt0 + src;
      break;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
    if (rt0 >= w.q.nt) return w;  // not reached
  }
  w.st = steps_of(P, w.q, w.rt);
  const int ln = line_len(w.st.n);
  w.h = (int)((first - before) / ln);
  const int at = (int)(first - before - (long long)w.h * ln);
  w.s = at;
  w.end = (int)min((long long)w.st.n, at + count);
  w.left = count - (ln - at);
  // the run may begin behind a unit's last step, and end there too: `end` is then no
  // larger than `s`, and the unit (written by the run before) is passed over
  if (at >= w.st.n && at > 0) {
    w.end = 0;
    if (!next_unit(P, w)) w.b = -1;
  }
  if (count == 0) w.b = -1;
  return w;
}

template <int D>
struct Smem {
  static constexpr int kHalfBytes = kBN * 128;    // of an fp16 tile
  static constexpr int kTile = kBN * D * 2;       // an fp16 tile
  static constexpr int kCodes = kBN * D;
  static constexpr int kQ = 0;                    // A, B
  static constexpr int kK = kQ + 2 * kTile;       // two slots
  static constexpr int kV = kK + 2 * kTile;
  static constexpr int kKC = kV + 2 * kTile;      // codes, one slot each
  static constexpr int kVC = kKC + kCodes;
  static constexpr int kInfoAt = kVC + kCodes;
  static constexpr int kBar = kInfoAt + kInfo * 16;
  enum { kKcFull, kKcEmpty, kVcFull, kVcEmpty, kKFull, kKEmpty = kKFull + 2, kVFull = kKEmpty + 2,
         kVEmpty = kVFull + 2, kQFull = kVEmpty + 2, kSFull = kQFull + 2, kPFull = kSFull + 4, kOFull = kPFull + 4,
         kODone = kOFull + 2, kInfoFull = kODone + 2, kMmaDone = kInfoFull + kInfo, kNumBars = kMmaDone + 2 };
  static constexpr int kWalk = (kBar + 8 * kNumBars + 15) / 16 * 16;
  static constexpr int kMisc = kWalk + ((1 + kConvWarp) * sizeof(Walk) + 15) / 16 * 16;  // tmem base, abort
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 227 * 1024, "one CTA per SM");
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn_major) {
  return idesc_bf16_f32(M, N, 0, b_mn_major) & ~((1u << 7) | (1u << 10));  // A, B format: f16
}

template <int kRegs>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_kv8_tc_kernel(const TcParams P, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(sm);
  auto bar = [&](int i) { return sbase + L::kBar + 8 * i; };
  volatile Info* infos = reinterpret_cast<volatile Info*>(sm + L::kInfoAt);
  Walk* start = reinterpret_cast<Walk*>(sm + L::kWalk);  // the run's; the softmax warps'
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  int* status = &g_attn_kv8_tc_status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == kProducerWarp && lane == 0) {
    const int one[] = {L::kKcFull, L::kVcFull, L::kSFull, L::kSFull + 1, L::kSFull + 2,
                       L::kSFull + 3, L::kOFull, L::kOFull + 1, L::kODone,
                       L::kODone + 1, L::kMmaDone, L::kMmaDone + 1};
    for (int i : one) mbar_init(bar(i), 1);
    const int two[] = {L::kKEmpty, L::kKEmpty + 1, L::kVEmpty, L::kVEmpty + 1};
    for (int i : two) mbar_init(bar(i), 2);  // both halves
    const int conv[] = {L::kKcEmpty, L::kVcEmpty, L::kKFull, L::kKFull + 1, L::kVFull,
                        L::kVFull + 1};
    for (int i : conv) mbar_init(bar(i), kConvWarps);
    const int soft[] = {L::kQFull, L::kQFull + 1, L::kPFull, L::kPFull + 1, L::kPFull + 2,
                        L::kPFull + 3};
    for (int i : soft) mbar_init(bar(i), kBM / 32);
    for (int i = 0; i < kInfo; ++i) mbar_init(bar(L::kInfoFull + i), 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (P.c.np > 0) {
      tma_prefetch(&tm_k);
      tma_prefetch(&tm_v);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sbase + L::kMisc, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the launch overlaps what came before)
  if (warp == 0) {
    const Walk w = find_run(P);
    if (lane == 0) *start = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const bool any = start->b >= 0 && start->q.nt > 0;

  if (warp >= kConvWarp) {
    reg_dec<kOtherRegs>();
    if (warp < kConvWarp + kConvWarps) {
      // -------------------------------------------------------- converters
      // lanes 0-7 take eight rows' same chunk: reads and writes then touch every
      // bank once
      const int cw = warp - kConvWarp, r8 = lane & 7, c4 = lane >> 3;
      bool ok = any;
      auto rows_of = [&](const uint8_t* src, uint8_t* dst, int valid, auto all) {
#pragma unroll
        for (int i = 0; i < kBN / (8 * kConvWarps); ++i) {
          const int row = 32 * cw + 8 * i + r8;
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const int c = 4 * j + c4;
            uint4 x = *reinterpret_cast<const uint4*>(src + tile_at<D>(row, c));
            if (!all && row >= valid) x = make_uint4(0, 0, 0, 0);
            uint8_t* d = dst + (c >> 2) * L::kHalfBytes + row * 128;
            const int c8 = 2 * (c & 3);
            *reinterpret_cast<uint4*>(d + ((c8 ^ r8) << 4)) =
                make_uint4(e4m3x2_to_h2(x.x & 0xffffu), e4m3x2_to_h2(x.x >> 16),
                           e4m3x2_to_h2(x.y & 0xffffu), e4m3x2_to_h2(x.y >> 16));
            *reinterpret_cast<uint4*>(d + (((c8 + 1) ^ r8) << 4)) =
                make_uint4(e4m3x2_to_h2(x.z & 0xffffu), e4m3x2_to_h2(x.z >> 16),
                           e4m3x2_to_h2(x.w & 0xffffu), e4m3x2_to_h2(x.w >> 16));
          }
        }
      };
      // rows that hold no key hold anything: 0, so that 0 * it is 0
      auto convert = [&](const uint8_t* src, uint8_t* dst, int valid, int none) {
        if ((none >> cw) & 1) valid = 0;
        if (valid >= kBN) rows_of(src, dst, valid, std::true_type{});
        else rows_of(src, dst, valid, std::false_type{});
        fence_proxy_async_smem();  // read next by the tensor core
        __syncwarp();
      };
      for (int n = 0; ok; ++n) {
        const int sl = n & 1;
        ok = mbar_wait(bar(L::kInfoFull + n % kInfo), (n / kInfo) & 1, abort_flag, status) &&
             mbar_wait(bar(L::kKcFull), n & 1, abort_flag, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const int fl = infos[n % kInfo].flags;
        if (fl & kEnd) break;
        if (n >= 2) {
          ok = mbar_wait(bar(L::kKEmpty + sl), ((n >> 1) + 1) & 1, abort_flag, status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        convert(sm + L::kKC, sm + L::kK + sl * L::kTile, fl >> 16, (fl >> 8) & 15);
        if (lane == 0) {
          mbar_arrive(bar(L::kKFull + sl));
          mbar_arrive(bar(L::kKcEmpty));
        }
        ok = mbar_wait(bar(L::kVcFull), n & 1, abort_flag, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (n >= 2) {
          ok = mbar_wait(bar(L::kVEmpty + sl), ((n >> 1) + 1) & 1, abort_flag, status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        convert(sm + L::kVC, sm + L::kV + sl * L::kTile, fl >> 16, (fl >> 8) & 15);
        if (lane == 0) {
          mbar_arrive(bar(L::kVFull + sl));
          mbar_arrive(bar(L::kVcEmpty));
        }
      }
    } else if (warp == kProducerWarp && any) {
      // ---------------------------------------------------------- producer
      Walk w = *start;
      int n = 0, nk = 0, nv = 0;  // steps described, K and V copies issued
      bool ok = true, more = true, begins = true;
      if (w.s >= w.end) {  // units without steps
        do more = next_unit(P, w);
        while (more && w.s >= w.end);
      }
      while (more && ok) {
        // eight steps of the unit at a time: a lane per block
        const int s8 = w.s + (lane >> 2);
        int page = -1, ke = 0, ve = 0;
        const int kt = s8 < w.st.sinks ? s8 : s8 + w.st.skip;
        const int row = kt * kBN + (lane & 3) * kBlock;
        if (s8 < w.end && row < w.q.len) {
          page = page_of(P.c, w.b, row);
          if (page >= 0) {
            const long long blk = (head_rows(P.c, page, w.h) + (row & (P.c.ps - 1))) / kBlock;
            ke = P.c.ke[blk];  // (in flight: the copies do not wait for them)
            ve = P.c.ve[blk];
          }
        }
        const unsigned none = __ballot_sync(0xffffffffu, page < 0);
        const int cnt = min(8, w.end - w.s);
        const bool has_b = w.q.R - w.rt * kUnitRows > kBM;
        uint32_t ke4 = 0, ve4 = 0;
        for (int i = 0; i < cnt; ++i, ++n) {
          const int src = 4 * i;
          const int key0 = (w.s + i < w.st.sinks ? w.s + i : w.s + i + w.st.skip) * kBN;
          const int none4 = (none >> src) & 15;
          const uint32_t bytes = (kBlocks - __popc(none4)) * kBlock * D;
          const bool mine = (lane >> 2) == i && page >= 0;
          const int at = (lane & 3) * kBlock, hp = page * P.c.H + w.h;
          ok = n < 1 || mbar_wait(bar(L::kKcEmpty), (n - 1) & 1, abort_flag, status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (lane == 0) {
            if (bytes) mbar_expect_tx(bar(L::kKcFull), bytes);
            else mbar_arrive(bar(L::kKcFull));
          }
          __syncwarp();
          if (mine)
            tma_load_3d(sbase + L::kKC + at * D, &tm_k, bar(L::kKcFull), 0,
                        (key0 + at) & (P.c.ps - 1), hp);
          ++nk;
          if (i == 0) {  // four lanes' exponents as bytes (the first copy is on its way)
            ke4 = (clamp_exp(ke) & 0xff) << (8 * (lane & 3));
            ve4 = (clamp_exp(ve) & 0xff) << (8 * (lane & 3));
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
              ke4 |= __shfl_xor_sync(0xffffffffu, ke4, o);
              ve4 |= __shfl_xor_sync(0xffffffffu, ve4, o);
            }
          }
          const uint32_t k4 = __shfl_sync(0xffffffffu, ke4, src);
          const uint32_t v4 = __shfl_sync(0xffffffffu, ve4, src);
          if (lane == 0) {
            volatile Info* x = infos + n % kInfo;
            x->key0 = key0;
            x->flags = (has_b ? kHasB : 0) | (i == 0 && begins ? kFirst : 0) |
                       (w.s + i + 1 == w.end ? kLast : 0) | none4 << 8 |
                       min(kBN, w.q.len - key0) << 16;
            x->ke = k4;
            x->ve = v4;
            mbar_arrive(bar(L::kInfoFull + n % kInfo));
          }
          ok = n < 1 || mbar_wait(bar(L::kVcEmpty), (n - 1) & 1, abort_flag, status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (lane == 0) {
            if (bytes) mbar_expect_tx(bar(L::kVcFull), bytes);
            else mbar_arrive(bar(L::kVcFull));
          }
          __syncwarp();
          if (mine)
            tma_load_3d(sbase + L::kVC + at * D, &tm_v, bar(L::kVcFull), 0,
                        (key0 + at) & (P.c.ps - 1), hp);
          ++nv;
          // the next copies but one come from L2
          if ((lane >> 2) == i + 2 && page >= 0) {
            tma_prefetch_3d(&tm_k, 0, row & (P.c.ps - 1), hp);
            tma_prefetch_3d(&tm_v, 0, row & (P.c.ps - 1), hp);
          }
        }
        w.s += cnt;
        begins = w.s >= w.end;
        while (more && w.s >= w.end) more = next_unit(P, w);
      }
      if (ok && n >= 1) ok = mbar_wait(bar(L::kKcEmpty), (n - 1) & 1, abort_flag, status);
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0) {
        if (ok) {
          infos[n % kInfo].flags = kEnd;
          mbar_arrive(bar(L::kInfoFull + n % kInfo));
          mbar_arrive(bar(L::kKcFull));
        } else {
          // aborted: the copies in flight land before the CTA ends
          if (nk > 0) mbar_wait_drain(bar(L::kKcFull), (nk - 1) & 1);
          if (nv > 0) mbar_wait_drain(bar(L::kVcFull), (nv - 1) & 1);
        }
      }
    } else if ((warp == kMmaWarp || warp == kMmaWarp + 1) && any) {
      // -------------------------------------------------- MMA issuer of a half
      if (lane == 0) {
        const int hf = warp - kMmaWarp;
        constexpr uint32_t kIdQK = idesc_f16_f32(kBM, kSub, 0);
        constexpr uint32_t kIdPV = idesc_f16_f32(kBM, D, 1);
        const uint32_t s_tm = tmem + hf * kBN, o_tm = tmem + 2 * kBN + hf * D;
        const uint64_t dq0 = sdesc_sw128(sbase + L::kQ + hf * L::kTile, 16, 1024);
        const uint64_t dk0 = sdesc_sw128(sbase + L::kK, 16, 1024);
        const uint64_t dv0 = sdesc_sw128(sbase + L::kV, L::kHalfBytes, 1024);
        auto wait = [&](int b, unsigned parity) {
          return mbar_wait(bar(b), parity & 1, abort_flag, status);
        };
        unsigned th = 0, uh = 0;  // steps and units of this half
        // scores of 64 keys of step n into one of two places
        auto qk = [&](int n, int sub) {
          const uint64_t dk = sdesc_add(dk0, (n & 1) * L::kTile + sub * (kSub * 128));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * L::kHalfBytes + (kk & 3) * 32;
            mma_ss(s_tm + sub * kSub, sdesc_add(dq0, off), sdesc_add(dk, off), kIdQK, kk > 0);
          }
          mma_commit(bar(L::kSFull + 2 * hf + sub));
          if (sub == 1) mma_commit(bar(L::kKEmpty + (n & 1)));
        };
        int n = 0;  // steps of the run
        bool ok = wait(L::kInfoFull, 0);
        while (ok) {
          int fl = infos[n % kInfo].flags;
          if (fl & kEnd) break;
          if (!(ok = wait(L::kKFull + (n & 1), n >> 1))) break;
          if (hf == 1 && !(fl & kHasB)) {  // no rows in this half
            mbar_arrive(bar(L::kKEmpty + (n & 1)));
            if (!(ok = wait(L::kVFull + (n & 1), n >> 1))) break;
            mbar_arrive(bar(L::kVEmpty + (n & 1)));
            ++n;
            ok = wait(L::kInfoFull + n % kInfo, n / kInfo);
            continue;
          }
          if (!(ok = wait(L::kQFull + hf, uh++))) break;
          tc_fence_after();
          qk(n, 0);
          qk(n, 1);
          for (;;) {  // a unit's steps
            const uint64_t dv = sdesc_add(dv0, (n & 1) * L::kTile);
            const bool last = fl & kLast;
            if (!(ok = wait(L::kVFull + (n & 1), n >> 1))) break;
#pragma unroll 1
            for (int sub = 0; sub < 2; ++sub) {
              if (!(ok = wait(L::kPFull + 2 * hf + sub, th))) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < kSub / 16; ++kk)
                mma_ts(o_tm, s_tm + sub * kSub + kk * 8,
                       sdesc_add(dv, sub * (kSub * 128) + kk * 2048), kIdPV,
                       !(fl & kFirst) || sub > 0 || kk > 0);
              mma_commit(bar(L::kOFull + hf));
              if (sub == 1) mma_commit(bar(L::kVEmpty + (n & 1)));
              if (sub == 1 && last) mma_commit(bar(L::kODone + hf));
              if (!last) {
                if (sub == 0 && !(ok = wait(L::kKFull + ((n + 1) & 1), (n + 1) >> 1))) break;
                tc_fence_after();
                qk(n + 1, sub);
              }
            }
            if (!ok) break;
            ++th;
            ++n;
            if (!(ok = wait(L::kInfoFull + n % kInfo, n / kInfo))) break;
            if (last) break;
            fl = infos[n % kInfo].flags;
          }
        }
        // nothing of ours may still run on the tensor core when TMEM is freed
        mma_commit(bar(L::kMmaDone + hf));
        mbar_wait_drain(bar(L::kMmaDone + hf), 0);
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    reg_inc<kSoftmaxRegs>();
    // the walk stands in shared memory: no room for it in registers
    Walk& w = start[1 + warp];
    if (lane == 0) w = start[0];
    __syncwarp();
    const int hf = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the half = lane of the tensor memory
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + hf * kBN, o_tm = tmem + lane_off + 2 * kBN + hf * D;
    if (threadIdx.x == 0)
      P.rec[2 * blockIdx.x] = P.rec[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    int n = 0;              // steps of the run
    unsigned th = 0, to = 0, uh = 0;  // this half's steps, parts of them, units
    bool ok = any, more = any;
    // This thread's query row of the unit in w, or null. The next unit's is asked for
    // before the end of the one before it.
    auto q_row = [&]() -> const uint4* {
      const int row = w.rt * kUnitRows + hf * kBM + r, tok = row / P.G;
      if (w.end <= w.s || row >= w.q.R) return nullptr;
      return reinterpret_cast<const uint4*>(
          P.q + ((long long)(w.q.first + tok) * P.Hq + w.h * P.G + row - tok * P.G) * D);
    };
    while (more) {  // a unit
      const int steps = max(0, w.end - w.s), R = w.q.R, first = w.q.first, h = w.h;
      const int row0 = w.rt * kUnitRows + hf * kBM, row = row0 + r;
      const bool whole = w.s == 0 && w.end == w.st.n;
      const int part = 2 * blockIdx.x + (w.s == 0 ? 1 : 0);
      if (!whole && threadIdx.x == 0)
        P.rec[part] = make_int4(w.end == w.st.n ? 3 : 1, w.b, w.rt, w.h);
      float m_run = -INFINITY, l_run = 0.f;
      if (row0 < R) {
        const int i = w.q.len - w.q.n + row / P.G;  // position
        if (steps > 0) {
          // ------------------------------------------------------ queries
          // (every product with the rows that stood here has completed: its scores
          // have been read)
          float row_mul;
          {
            const uint4* src = q_row();
            uint4 x[D / 8];
            float big = 0.f;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              x[c] = src ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
              const uint32_t e[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                big = fmaxf(big, fmaxf(fabsf(__uint_as_float(e[j] << 16)),
                                       fabsf(__uint_as_float(e[j] & 0xffff0000u))));
            }
            // 2^ex times a largest element in [1, 2) is brought to [64, 128)
            const int ex = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -120), 127);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 6 - ex) << 23);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint32_t e[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
              uint32_t f[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                f[j] = pack_f16(__uint_as_float(e[j] << 16) * up,
                                __uint_as_float(e[j] & 0xffff0000u) * up);
              *reinterpret_cast<uint4*>(sm + L::kQ + hf * L::kTile + (c >> 3) * L::kHalfBytes +
                                        r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                  make_uint4(f[0], f[1], f[2], f[3]);
            }
            // not 0 or infinite, with a block's exponent too, which a masked key's -inf
            // or a score of 0 would make NaN
            row_mul = fminf(fmaxf(ldexpf(P.score_mul, ex - 6), FLT_MIN * 0x1p41f),
                            FLT_MAX * 0x1p-41f);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kQFull + hf));
          }
          // the half's positions
          const int i_lo = w.q.len - w.q.n + row0 / P.G;
          const int i_hi = w.q.len - w.q.n + (min(w.q.R, row0 + kBM) - 1) / P.G;
          const RowKeys seen = row_keys(i, w.q.len, P.causal, P.window, P.sink);
          for (int s = 0; s < steps; ++s) {
            const int ns = n + s;
            Info inf{};
            bool masked = false;
#pragma unroll 1
            for (int sub = 0; sub < 2; ++sub, ++to) {
              // The scores first: a half that had no part in the units before may be more
              // than kInfo steps ahead, where the description's barrier is still two phases
              // back and would pass at once. Once the scores are there, so is it.
              ok = mbar_wait(bar(L::kSFull + 2 * hf + sub), th & 1, abort_flag, status) &&
                   (sub == 1 || mbar_wait(bar(L::kInfoFull + ns % kInfo), (ns / kInfo) & 1,
                                          abort_flag, status));
              if (!(ok = __all_sync(0xffffffffu, ok))) break;
              tc_fence_after();
              uint32_t sr[2][32];
              tmem_ld32(s_tm + sub * kSub, sr[0]);
              tmem_ld32(s_tm + sub * kSub + 32, sr[1]);
              if (sub == 0) {
                const volatile Info* x = infos + ns % kInfo;
                inf.key0 = x->key0;
                inf.flags = x->flags;
                inf.ke = x->ke;
                inf.ve = x->ve;
                masked = (inf.flags & 0xf00) || (inf.flags >> 16) < kBN || i_lo < 0 ||
                         (P.causal && inf.key0 + kBN - 1 > i_lo) ||
                         (P.window > 0 && i_hi - inf.key0 >= P.window);
              } else {
                inf.ke >>= 16;
                inf.ve >>= 16;
              }
              float mul[2], ev[2], mx = -INFINITY;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                mul[c] = row_mul * exp2i(static_cast<int8_t>(inf.ke >> (8 * c)));
                ev[c] = static_cast<float>(static_cast<int8_t>(inf.ve >> (8 * c)));
              }
              tmem_wait_ld();
              if (masked) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  uint32_t vis = key_bits(seen, inf.key0 + sub * kSub + 32 * c);
                  if ((inf.flags >> (8 + 2 * sub + c)) & 1) vis = 0;
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (!((vis >> j) & 1u)) sr[c][j] = __float_as_uint(-INFINITY);
                }
              }
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float a[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) a[j] = __uint_as_float(sr[c][j]);
#pragma unroll
                for (int j = 4; j < 28; j += 8)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    a[e] = fmaxf(fmaxf(a[e], __uint_as_float(sr[c][j + e])),
                                 __uint_as_float(sr[c][j + 4 + e]));
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = fmaxf(a[e], __uint_as_float(sr[c][28 + e]));
                mx = fmaxf(mx, fmaf(mul[c], fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])), ev[c]));
              }
              // the reference moves when p would leave fp16's range
              const bool need = mx > m_run + kAbove;
              float alpha = 1.f;
              if (need) {
                const float x = mx - kBelow;
                alpha = m_run == -INFINITY ? 0.f : ex2(m_run - x);
                m_run = x;
                l_run *= alpha;
              }
              const float msub = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float a = ev[c] - msub;
                const uint64_t mul2 = f2_pack(mul[c], mul[c]), add2 = f2_pack(a, a);
                uint64_t ls[2] = {0, 0};
                uint32_t pk[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  float x0, x1;
                  f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c][2 * j]),
                                           __uint_as_float(sr[c][2 * j + 1])), mul2, add2), x0, x1);
                  const float p0 = ex2(x0), p1 = ex2(x1);
                  ls[j & 1] = f2_add(ls[j & 1], f2_pack(p0, p1));
                  pk[j] = pack_f16(p0, p1);
                }
                float a0, a1, b0, b1;
                f2_unpack(ls[0], a0, a1);
                f2_unpack(ls[1], b0, b1);
                l_run = fmaf((a0 + a1) + (b0 + b1),
                             exp2i(-static_cast<int8_t>(inf.ve >> (8 * c))), l_run);
                tmem_st16(s_tm + sub * kSub + 16 * c, pk);
              }
              // O holds the keys before; it follows the reference before P V adds to it.
              // (The P V before the last one has completed, as these scores came behind it:
              // the phase waited for is the next to end.)
              if (__any_sync(0xffffffffu, need && (s > 0 || sub > 0))) {
                ok = mbar_wait(bar(L::kOFull + hf), (to - 1) & 1, abort_flag, status);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
#pragma unroll 1
                for (int oc = 0; oc < D / 32; ++oc) {
                  uint32_t o[32];
                  tmem_ld32(o_tm + 32 * oc, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                  tmem_st32(o_tm + 32 * oc, o);
                }
              }
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(L::kPFull + 2 * hf + sub));
            }
            if (!ok) break;
            ++th;
          }
          if (!ok) break;
        }
      }
      n += steps;
      __syncwarp();
      if (lane == 0) more = next_unit(P, w);
      more = __shfl_sync(0xffffffffu, more, 0);
      __syncwarp();
      if (const uint4* src = more ? q_row() : nullptr) {
#pragma unroll
        for (int l = 0; l < D / 64; ++l)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 8 * l));
      }
      // ------------------------------------------------------------- the end
      if (row0 >= R) continue;
      if (steps > 0) {
        ok = mbar_wait(bar(L::kODone + hf), uh & 1, abort_flag, status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        ++uh;
        tc_fence_after();
      }
      const bool none = l_run == 0.f;  // no visible key (a NaN score makes it NaN)
      const float inv = none ? 0.f : 1.f / l_run;
      // Rows of O go out through the queries' places (free: every product with them has
      // completed), a warp's own 32, so that neighbouring lanes write neighbouring bytes.
      uint8_t* stage = sm + L::kQ + hf * L::kTile;
      auto place = [&](int row, int c) {  // of 8 channels of a row of the half
        return reinterpret_cast<uint4*>(stage + (c >> 3) * L::kHalfBytes + row * 128 +
                                        (((c & 7) ^ (row & 7)) << 4));
      };
#pragma unroll 1
      for (int oc = 0; oc < D / 32; ++oc) {
        uint32_t o[32];
        if (steps > 0) {
          tmem_ld32(o_tm + 32 * oc, o);
          tmem_wait_ld();
        }
        if (whole) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            o[j] = none ? 0u : __float_as_uint(__uint_as_float(o[j]) * inv);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              f[e] = pack_bf16(__uint_as_float(o[8 * j + 2 * e]),
                               __uint_as_float(o[8 * j + 2 * e + 1]));
            *place(r, 4 * oc + j) = make_uint4(f[0], f[1], f[2], f[3]);
          }
        } else if (row < R) {  // (four channels of all rows stand together)
          uint4* dst = reinterpret_cast<uint4*>(P.o_part) +
                       ((long long)part * (D / 4) + 8 * oc) * kUnitRows + hf * kBM + r;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[j * kUnitRows] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      }
      auto o_row = [&](int row) {
        const int tok = row / P.G;
        return (long long)(first + tok) * P.Hq + h * P.G + row - tok * P.G;
      };
      if (whole) {
        __syncwarp();
#pragma unroll 4
        for (int e = lane; e < 32 * (D / 8); e += 32) {
          const int rr = quarter * 32 + e / (D / 8), c = e % (D / 8);
          if (row0 + rr < R)
            reinterpret_cast<uint4*>(P.out + o_row(row0 + rr) * D)[c] = *place(rr, c);
        }
        __syncwarp();  // (before the next queries)
        if (row < R) P.lse[o_row(row)] = none ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
      } else if (row < R) {
        P.ml_part[(long long)part * kUnitRows + hf * kBM + r] = make_float2(m_run, l_run);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

constexpr int kPads = 64;           // blocks that clear padding
constexpr int kMergeRows = 32;      // of a block: a row per lane, 8 channels per warp
template <int D>
constexpr int kMergeThreads = 32 * (D / 8);

// Block (x, y): rows [32 y, ..) of the x-th unit that lies in several runs. Its
// first partial stands behind the run j that it begins in, the others before the runs
// behind j. Blocks x >= heads (packed): zeros for the tokens outside the sequences.
template <int D>
__global__ void __launch_bounds__(kMergeThreads<D>)
attn_kv8_tc_merge_kernel(const TcParams P, int heads) {
  __shared__ int s_run[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x >= heads) {
    const int i0 = (blockIdx.x - heads) * gridDim.y + blockIdx.y;
    const int step = (gridDim.x - heads) * gridDim.y;
    const int e0 = min(max(__ldg(P.cu), 0), P.T), e1 = max(e0, min(max(__ldg(P.cu + P.c.B), 0), P.T));
    for (int i = i0; i < e0 + P.T - e1; i += step) {
      const long long tok = i < e0 ? i : e1 + (i - e0);
      uint2* r = reinterpret_cast<uint2*>(P.out + tok * P.Hq * D);
      for (int u = threadIdx.x; u < P.Hq * D / 4; u += kMergeThreads<D>) r[u] = make_uint2(0, 0);
      for (int u = threadIdx.x; u < P.Hq; u += kMergeThreads<D>) P.lse[tok * P.Hq + u] = -INFINITY;
    }
    return;
  }
  if (threadIdx.x < 32) {  // run j, and the one with the unit's last steps
    int left = blockIdx.x, j = -1, last = -1;
    for (int j0 = 0; j0 < kGrid && last < 0; j0 += 32) {
      const int k = j0 + (threadIdx.x & 31);
      const int tail = k < kGrid ? P.rec[2 * k].x : 0, head = k < kGrid ? P.rec[2 * k + 1].x : 0;
      // the ends of units behind run j (their first parts' runs come before them)
      unsigned ends = __ballot_sync(0xffffffffu, tail == 3);
      unsigned begins = __ballot_sync(0xffffffffu, head == 1);
      if (j < 0) {
        const int here = __popc(begins);
        if (left >= here) {
          left -= here;
          continue;
        }
        for (; left > 0; --left) begins &= begins - 1;
        const int at = __ffs(begins) - 1;
        j = j0 + at;
        ends &= at == 31 ? 0u : ~0u << (at + 1);
      }
      if (ends) last = j0 + __ffs(ends) - 1;
    }
    if (threadIdx.x == 0) {
      s_run[0] = last < 0 ? -1 : j;
      s_run[1] = last;
    }
  }
  __syncthreads();
  const int j = s_run[0], last = s_run[1];
  if (j < 0) return;  // fewer such units
  const int4 rec = P.rec[2 * j + 1];
  const Seq q = seq_of(P, rec.y);
  const int c8 = threadIdx.x >> 5, rr = blockIdx.y * kMergeRows + (threadIdx.x & 31);
  const int row = rec.z * kUnitRows + rr;
  if (row >= q.R) return;
  float M = -INFINITY, ls = 0.f, os[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = j; k <= last; ++k) {
    const long long slot = k == j ? 2 * j + 1 : 2 * k;
    const float2 a = P.ml_part[slot * kUnitRows + rr];
    const float4* o = reinterpret_cast<const float4*>(P.o_part) +
                      (slot * (D / 4) + 2 * c8) * kUnitRows + rr;
    const float4 x = o[0], y = o[kUnitRows];
    const float Mn = fmaxf(M, a.x);
    const float f0 = M == -INFINITY ? 0.f : ex2(M - Mn);
    const float f1 = a.x == -INFINITY ? 0.f : ex2(a.x - Mn);
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) os[e] = os[e] * f0 + v[e] * f1;
    ls = ls * f0 + a.y * f1;
    M = Mn;
  }
  const int tok = row / P.G, hh = row - tok * P.G;
  const long long o_row = (long long)(q.first + tok) * P.Hq + rec.w * P.G + hh;
  const bool none = ls == 0.f;
  const float inv = none ? 0.f : 1.f / ls;
  uint32_t f[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    f[e] = none ? 0u : pack_bf16(os[2 * e] * inv, os[2 * e + 1] * inv);
  reinterpret_cast<uint4*>(P.out + o_row * D)[c8] = make_uint4(f[0], f[1], f[2], f[3]);
  if (c8 == 0) P.lse[o_row] = none ? -INFINITY : (M + log2f(ls)) * kLn2;
}

// ------------------------------------------------------------------- host
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Ws {
  size_t ml, rec, total;
};
Ws layout(int D) {
  Ws w{};
  w.ml = up256((size_t)2 * kGrid * kUnitRows * D * 4);
  w.rec = w.ml + up256((size_t)2 * kGrid * kUnitRows * 8);
  w.total = w.rec + up256((size_t)2 * kGrid * 16);
  return w;
}

template <int D>
usp_status_t launch_t(const TcParams& P, cudaStream_t st) {
  CUtensorMap mk{}, mv{};  // (without pages, nothing is loaded through them)
  if (P.c.np > 0 && (!make_map(&mk, P.c.kc, P.c, D) || !make_map(&mv, P.c.vc, P.c, D)))
    return USP_ERR_CUDA;
  const int smem = Smem<D>::kAlloc;
  static SmemAttr attr;
  cudaError_t e = attr.set(attn_kv8_tc_kernel<D>, smem);
  if (e != cudaSuccess) return fail_cuda("cudaFuncSetAttribute(smem)", e);
  // each kernel's launch and set-up overlap the end of the one before it
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(kGrid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  {
    ProfScope ps(st, "attn_kv8_tc");
    e = cudaLaunchKernelEx(&cfg, attn_kv8_tc_kernel<D>, P, mk, mv);
  }
  if (e == cudaSuccess) {
    note_launch();
    // at most one unit in several runs per run's end, and no more than there are units
    const long long tiles = ((long long)P.max_new * P.G + kUnitRows - 1) / kUnitRows;
    const long long units = (long long)P.c.B * P.c.H * tiles;
    const int heads = units < kGrid - 1 ? (int)units : kGrid - 1;
    const int slices = kUnitRows / kMergeRows;
    cfg.gridDim = dim3(heads + (P.cu ? kPads / slices : 0), slices);
    cfg.blockDim = dim3(kMergeThreads<D>);
    cfg.dynamicSmemBytes = 0;
    ProfScope ps(st, "attn_kv8_tc_merge");
    e = cudaLaunchKernelEx(&cfg, attn_kv8_tc_merge_kernel<D>, P, heads);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail_cuda("kernel launch", e);
  }
  note_launch();
  return USP_OK;
}

}  // namespace

size_t attn_kv8_tc_workspace(int D) { return layout(D).total; }

usp_status_t launch_attn_kv8_tc(const AttnKv8Args& a, void* workspace, cudaStream_t st) {
  const Ws w = layout(a.D);
  char* base = static_cast<char*>(workspace);
  TcParams P{};
  P.c = a.c;
  P.q = static_cast<const __nv_bfloat16*>(a.q);
  P.out = static_cast<__nv_bfloat16*>(a.out);
  P.lse = a.lse;
  P.o_part = reinterpret_cast<float*>(base);
  P.ml_part = reinterpret_cast<float2*>(base + w.ml);
  P.rec = reinterpret_cast<int4*>(base + w.rec);
  P.cu = a.cu;
  P.T = a.T;
  P.max_new = a.max_new;
  P.Hq = a.Hq;
  P.G = a.Hq / a.c.H;
  P.score_mul = a.scale * 1.4426950408889634f;
  P.causal = a.causal;
  P.window = a.window;
  P.sink = a.sink;
  return a.D == 128 ? launch_t<128>(P, st) : launch_t<64>(P, st);
}

int read_clear_attn_kv8_tc_status() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_kv8_tc_status, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0) cudaMemcpyToSymbol(g_attn_kv8_tc_status, &z, sizeof(int));
  return v;
}

}  // namespace usp
