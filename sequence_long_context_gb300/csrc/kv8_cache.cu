// Filling the paged 8-bit KV cache, with the rotation of positions on the way, and
// reading it back.
//
// A block of 32 rows of one head and tensor shares an exponent, so the block's
// maximum is known before its first code is written. A CTA of four warps takes
// one block of a sequence: each warp eight rows, each lane one item (two vectors
// of 16 bytes of the input) of a row, in kPass passes. Cos and sin of a lane's
// rows stay in registers while the CTA passes over the heads of K and V, and the next
// head's rows are loaded before the present one's are used. A prompt's blocks are
// shared out among CTAs by heads too where there are few. Queries are a copy with a
// rotation: warps of other CTAs of the same launch take a token each, eight rows in
// flight (with the keys' and values' blocks they were 134 us for 32K tokens).
//
// Bound by HBM: 32K tokens of 8 KV and 32 query heads, D = 128, bf16 (738 MB with the codes)
// take 123 us, 6.0 TB/s; their reading (201 MB, some of which stays in L2) 32 to 36 us; one
// token of 8 sequences 6.1 us for both calls.
//
// Rows that the block held before the call keep their codes unless the exponent
// rises; then they are rounded once more. Every block belongs to one CTA for a
// given head, so nothing is read that another CTA writes.
#include "internal.h"
#include "kv8.cuh"
#include "kv8_host.h"
#include "tc_ptx.cuh"

namespace usp {
namespace {

using namespace kv8;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerWarp = kBlock / kWarps;

struct AppendParams {
  Kv8AppendArgs a;
  int splits;     // CTAs that share a block's heads
  int slots;      // blocks per sequence (dense), or in all (packed)
  int seq_form;   // a cluster of `splits` CTAs takes a whole sequence
  int kv_blocks;  // CTAs behind these rotate queries (other form)
};

// Tokens of sequence b: the first and how many. Boundaries are trusted, but no
// index leaves [0, T).
struct Tokens {
  long long first;
  int n;
};
__device__ __forceinline__ Tokens tokens_of(const int* cu, int T, int b) {
  if (!cu) return {(long long)b * T, T};
  const int a = min(max(__ldg(cu + b), 0), T), e = min(max(__ldg(cu + b + 1), a), T);
  return {a, e - a};
}

// Eight (four) floats as E4M3 codes of x * up: nearest even, saturating, NaN as 0.
template <int V>
__device__ __forceinline__ void encode(const float (&x)[V], float up, uint32_t (&w)[V / 4]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i)
    w[i] = tc::pack_e4m3(x[4 * i] * up, x[4 * i + 1] * up) |
           (tc::pack_e4m3(x[4 * i + 2] * up, x[4 * i + 3] * up) << 16);
}
template <int V>
__device__ __forceinline__ void recode(uint32_t (&w)[V / 4], float up) {
  float x[V];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const float2 lo = e4m3x2_to_float2(w[i] & 0xffffu), hi = e4m3x2_to_float2(w[i] >> 16);
    x[4 * i] = lo.x; x[4 * i + 1] = lo.y; x[4 * i + 2] = hi.x; x[4 * i + 3] = hi.y;
  }
  encode(x, up, w);
}
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[2]) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  w[0] = x.x; w[1] = x.y;
}
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[1]) {
  w[0] = *reinterpret_cast<const uint32_t*>(p);
}
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[2]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[1]) {
  *reinterpret_cast<uint32_t*>(p) = w[0];
}

// One block of a sequence: rows [blk * 32, ..) of which [lo, hi) are new, token
// t0 + (row - lo) each; this CTA's share of the heads.
template <typename T, int D>
__device__ __forceinline__ void append_block(const AppendParams& P, int b, int blk, int start,
                                             const Tokens& tok, int split, float (*s_max)[kWarps],
                                             int& turn_no) {
  constexpr int V = kVec<T>, kItems = D / (2 * V);
  constexpr int kRowsAtOnce = 32 / kItems, kPass = kRowsPerWarp / kRowsAtOnce;
  const Kv8AppendArgs& A = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = lane % kItems;
  const Item<V> it = item_of<V>(A.rope, item);
  const int base = blk * kBlock;
  const int lo = max(start, base) - base;                        // first new row
  const int hi = (int)min((long long)start + tok.n, (long long)base + kBlock) - base;
  const bool room = base < A.c.cap;
  const int page = room ? page_of(A.c, b, base) : -1;
  int row[kPass];
  long long token[kPass];
  bool fresh[kPass];
  float c[kPass][V], s[kPass][V];
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    row[p] = warp * kRowsPerWarp + p * kRowsAtOnce + lane / kItems;
    fresh[p] = row[p] >= lo && row[p] < hi;
    token[p] = tok.first + (base + row[p] - start);
    if (fresh[p] && it.f >= 0)
      load_turn(A.rope, it, A.positions ? __ldg(A.positions + token[p]) : base + row[p], c[p], s[p]);
  }
  const int H = A.c.H;
  if (page < 0) return;
  uint4 xa[kPass], xb[kPass];
  auto load = [&](int j) {  // K heads, then V heads
    const T* src = static_cast<const T*>(j < H ? A.k : A.v);
    const int h = j < H ? j : j - H;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      xa[p] = xb[p] = make_uint4(0, 0, 0, 0);
      if (fresh[p]) {
        const T* r = src + (token[p] * H + h) * D;
        // V is not rotated: its items are the two vectors of a rotated one all the same
        xa[p] = *reinterpret_cast<const uint4*>(r + it.a);
        xb[p] = *reinterpret_cast<const uint4*>(r + it.b);
      }
    }
  };
  int j = split;
  if (j < 2 * H) load(j);
  for (; j < 2 * H; j += P.splits) {
    const bool isk = j < H;
    float fa[kPass][V], fb[kPass][V];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      unpack(xa[p], fa[p]);
      unpack(xb[p], fb[p]);
    }
    if (j + P.splits < 2 * H) load(j + P.splits);
    if (isk) {
#pragma unroll
      for (int p = 0; p < kPass; ++p)
        if (fresh[p]) rotate(it, A.rope.inter != 0, c[p], s[p], fa[p], fb[p]);
    }
    const int h = isk ? j : j - H;
    int8_t* ex = (isk ? A.c.ke : A.c.ve) +
                 (head_rows(A.c, page, h) + (base & (A.c.ps - 1))) / kBlock;
    uint8_t* codes = (isk ? A.c.kc : A.c.vc) + (head_rows(A.c, page, h) + (base & (A.c.ps - 1))) * D;
    const int old = lo > 0 ? clamp_exp(*ex) : kExpMin;
    float amax = 0.f;
#pragma unroll
    for (int p = 0; p < kPass; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        fa[p][i] = isnan(fa[p][i]) ? 0.f : fa[p][i];
        fb[p][i] = isnan(fb[p][i]) ? 0.f : fb[p][i];
        if (fresh[p]) amax = fmaxf(amax, fmaxf(fabsf(fa[p][i]), fabsf(fb[p][i])));
      }
    amax = warp_max(amax);
    float* sm = s_max[turn_no & 1];  // two, so that one barrier per head is enough
    ++turn_no;
    if (lane == 0) sm[warp] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const int e = max(old, exponent_of(amax));
    const float up = exp2i(-e);
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      uint8_t* r = codes + row[p] * D;
      uint32_t wa[V / 4], wb[V / 4];
      if (fresh[p]) {
        encode(fa[p], up, wa);
        encode(fb[p], up, wb);
      } else if (row[p] < lo && e > old) {  // held before, and the exponent has risen
        load_codes(r + it.a, wa);
        load_codes(r + it.b, wb);
        const float down = exp2i(old - e);
        recode<V>(wa, down);
        recode<V>(wb, down);
      } else {
        continue;
      }
      store_codes(r + it.a, wa);
      store_codes(r + it.b, wb);
    }
    if (threadIdx.x == 0) *ex = static_cast<int8_t>(e);
  }
}

// Rotates `chunk` heads of a token from head h0 on, by a warp.
template <typename T, int D>
__device__ __forceinline__ void rotate_q(const Kv8AppendArgs& A, long long token, int pos, int h0,
                                         int chunk) {
  constexpr int V = kVec<T>, kItems = D / (2 * V), kHeads = 32 / kItems, kFlight = 8;
  const int lane = threadIdx.x & 31;
  const Item<V> it = item_of<V>(A.rope, lane % kItems);
  float c[V], s[V];
  load_turn(A.rope, it, pos, c, s);
  const T* x = static_cast<const T*>(A.q) + token * A.Hq * D;
  T* y = static_cast<T*>(A.q_out) + token * A.Hq * D;
  const int end = min(h0 + chunk, A.Hq);
  for (int h = h0 + lane / kItems; h < end; h += kFlight * kHeads) {
    uint4 a[kFlight], b[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
      if (h + i * kHeads < end) {
        a[i] = *reinterpret_cast<const uint4*>(x + (h + i * kHeads) * D + it.a);
        b[i] = *reinterpret_cast<const uint4*>(x + (h + i * kHeads) * D + it.b);
      }
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
      if (h + i * kHeads < end) {
        if (it.f >= 0) {
          float fa[V], fb[V];
          unpack(a[i], fa);
          unpack(b[i], fb);
          rotate(it, A.rope.inter != 0, c, s, fa, fb);
          a[i] = pack(fa);
          b[i] = pack(fb);
        }
        *reinterpret_cast<uint4*>(y + (h + i * kHeads) * D + it.a) = a[i];
        *reinterpret_cast<uint4*>(y + (h + i * kHeads) * D + it.b) = b[i];
      }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams P) {
  __shared__ float s_max[2][kWarps];
  const Kv8AppendArgs& A = P.a;
  int turn_no = 0;
  const int split = blockIdx.x % P.splits, x = blockIdx.x / P.splits;
  const int warp = threadIdx.x >> 5;
  if (A.cu && A.q && (P.seq_form || (int)blockIdx.x >= P.kv_blocks)) {  // q of padding: zeros
    const int i0 = P.seq_form ? 0 : P.kv_blocks;
    const int e0 = min(max(__ldg(A.cu), 0), A.T), e1 = min(max(__ldg(A.cu + A.c.B), 0), A.T);
    const int pad = e0 + A.T - max(e0, e1);
    const int vecs = A.Hq * D / kVec<T>;
    for (int i = blockIdx.x - i0; i < pad; i += gridDim.x - i0) {
      const long long t = i < e0 ? i : (long long)max(e0, e1) + (i - e0);
      uint4* r = reinterpret_cast<uint4*>(static_cast<T*>(A.q_out) + t * A.Hq * D);
      for (int u = threadIdx.x; u < vecs; u += kThreads) r[u] = make_uint4(0, 0, 0, 0);
    }
  }
  if (P.seq_form) {
    const int b = x;
    const Tokens tok = tokens_of(A.cu, A.T, b);
    const int start = clamp_len(A.c.lens[b], A.c.cap);
    if (tok.n > 0) {
      const int last = (int)(((long long)start + tok.n - 1) / kBlock);
      for (int blk = start / kBlock; blk <= last; ++blk)
        append_block<T, D>(P, b, blk, start, tok, split, s_max, turn_no);
    }
    if (A.q) {  // few heads of a token per warp
      constexpr int kChunk = 32 / (D / (2 * kVec<T>));
      const int slices = (A.Hq + kChunk - 1) / kChunk;
      for (int i = split * kWarps + warp; i < tok.n * slices; i += P.splits * kWarps) {
        const int t = i / slices;
        rotate_q<T, D>(A, tok.first + t,
                       A.positions ? __ldg(A.positions + tok.first + t) : start + t,
                       (i - t * slices) * kChunk, kChunk);
      }
    }
    if (A.lens_out) {
      cluster_sync();  // every CTA of the sequence has read its length
      if (split == 0 && threadIdx.x == 0)
        A.lens_out[b] = (int)min((long long)A.c.cap, (long long)start + tok.n);
    }
    return;
  }
  if ((int)blockIdx.x >= P.kv_blocks) {  // queries: a token per warp
    const long long tokens = A.cu ? A.T : (long long)A.c.B * A.T;
    const long long step = (long long)(gridDim.x - P.kv_blocks) * kWarps;
    for (long long t = (long long)(blockIdx.x - P.kv_blocks) * kWarps + warp; t < tokens; t += step) {
      const int b = A.cu ? seg_of(A.cu, A.c.B, (int)t) : (int)(t / A.T);
      const Tokens tok = tokens_of(A.cu, A.T, b);
      if (t < tok.first || t >= tok.first + tok.n) continue;
      const int pos = A.positions ? __ldg(A.positions + t)
                                  : clamp_len(A.c.lens[b], A.c.cap) + (int)(t - tok.first);
      rotate_q<T, D>(A, t, pos, 0, A.Hq);
    }
    return;
  }
  int b, at;
  if (A.cu) {
    // slot cu[b] / 32 + 2 b is sequence b's first: it has at most n / 32 + 2 blocks
    int l = 0, r = A.c.B - 1;
    while (l < r) {
      const int m = (l + r + 1) >> 1;
      if (tokens_of(A.cu, A.T, m).first / kBlock + 2 * m <= x) l = m; else r = m - 1;
    }
    b = l;
    at = x - (int)(tokens_of(A.cu, A.T, b).first / kBlock + 2 * b);
  } else {
    b = x / P.slots;
    at = x - b * P.slots;
  }
  const Tokens tok = tokens_of(A.cu, A.T, b);
  const int start = clamp_len(A.c.lens[b], A.c.cap);
  if (at == 0 && split == 0 && threadIdx.x == 0 && A.lens_out && A.lens_out != A.c.lens)
    A.lens_out[b] = (int)min((long long)A.c.cap, (long long)start + tok.n);
  const int blk = start / kBlock + at;
  if (at < 0 || tok.n == 0 || (long long)blk * kBlock >= (long long)start + tok.n) return;
  append_block<T, D>(P, b, blk, start, tok, split, s_max, turn_no);
}

// The lengths after an append into the cache's own, once it has read them.
__global__ void append_lens_kernel(const AppendParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= P.a.c.B) return;
  const int start = clamp_len(P.a.c.lens[b], P.a.c.cap);
  P.a.lens_out[b] = (int)min((long long)P.a.c.cap,
                             (long long)start + tokens_of(P.a.cu, P.a.T, b).n);
}

template <typename T, int D>
usp_status_t launch_append(AppendParams& P, cudaStream_t st) {
  const Kv8AppendArgs& A = P.a;
  const int jobs = 2 * A.c.H;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  cfg.attrs = at;
  P.seq_form = A.T <= 2 * kBlock;
  long long blocks;
  if (P.seq_form) {
    P.splits = 1;
    while (P.splits < 8 && P.splits < jobs) P.splits *= 2;
    blocks = (long long)A.c.B * P.splits;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = P.splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
  } else {
    P.slots = A.cu ? 0 : (int)(((long long)A.T + 2 * kBlock - 2) / kBlock);
    blocks = A.cu ? (long long)A.T / kBlock + 2LL * A.c.B : (long long)A.c.B * P.slots;
    const long long want = 5LL * sm_count();  // resident CTAs
    long long n = (want + blocks - 1) / blocks;
    P.splits = (int)(n < 1 ? 1 : n > jobs ? jobs : n);
    blocks *= P.splits;
    if (blocks > 0x7fffffffLL) return USP_ERR_UNSUPPORTED;
    P.kv_blocks = (int)blocks;
    if (A.q) {
      const long long warps = A.cu ? A.T : (long long)A.c.B * A.T;
      const long long need = (warps + kWarps - 1) / kWarps, most = 16LL * sm_count();
      blocks += need < most ? need : most;
    }
  }
  if (blocks > 0x7fffffffLL) return USP_ERR_UNSUPPORTED;
  cfg.gridDim = dim3((unsigned)blocks);
  cudaError_t e;
  {
    ProfScope ps(st, "kv8_append");
    e = cudaLaunchKernelEx(&cfg, append_kernel<T, D>, P);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail_cuda("kernel launch", e);
  }
  note_launch();
  if (P.seq_form || A.lens_out != A.c.lens) return USP_OK;
  cfg.gridDim = dim3((A.c.B + 127) / 128);
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  {
    ProfScope ps(st, "kv8_append_lens");
    e = cudaLaunchKernelEx(&cfg, append_lens_kernel, P);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail_cuda("kernel launch", e);
  }
  note_launch();
  return USP_OK;
}

// ------------------------------------------------------------------- reading
struct ReadParams {
  Cache c;
  const int* start;
  int T;
  void* k;
  void* v;
};
constexpr int kReadThreads = 256;

// A thread takes as many channels of a row of K and of V as make 16 bytes of output, so
// that a warp's loads and stores are each one run. It steps over the rows of one
// sequence (blockIdx.y) without a division.
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadParams P) {
  constexpr int V = kVec<T>, kPer = D / V;
  const int b = blockIdx.y;
  const unsigned per_row = P.c.H * kPer;  // of all heads
  const unsigned step = gridDim.x * kReadThreads, step_t = step / per_row, step_x = step % per_row;
  const unsigned i0 = blockIdx.x * kReadThreads + threadIdx.x;
  unsigned t = i0 / per_row, x = i0 % per_row;
  const int first = P.start ? __ldg(P.start + b) : 0;
  const int len = clamp_len(__ldg(P.c.lens + b), P.c.cap);
  T* k = static_cast<T*>(P.k) + (long long)b * P.T * P.c.H * D;
  T* v = static_cast<T*>(P.v) + (long long)b * P.T * P.c.H * D;
  for (; t < (unsigned)P.T; t += step_t, x += step_x) {
    if (x >= per_row) {
      x -= per_row;
      if (++t >= (unsigned)P.T) break;
    }
    const long long row = (long long)first + t;
    uint32_t kw[V / 4], vw[V / 4];
    float ks = 0.f, vs = 0.f;
#pragma unroll
    for (int e = 0; e < V / 4; ++e) kw[e] = vw[e] = 0;
    if (row >= 0 && row < len) {
      const int page = page_of(P.c, b, (int)row);
      if (page >= 0) {
        const long long at = head_rows(P.c, page, x / kPer) + ((int)row & (P.c.ps - 1));
        load_codes(P.c.kc + at * D + (x % kPer) * V, kw);
        load_codes(P.c.vc + at * D + (x % kPer) * V, vw);
        ks = exp2i(clamp_exp(P.c.ke[at / kBlock]));
        vs = exp2i(clamp_exp(P.c.ve[at / kBlock]));
      }
    }
    float kf[V], vf[V];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      const float2 a = e4m3x2_to_float2(e & 1 ? kw[e / 2] >> 16 : kw[e / 2] & 0xffffu);
      const float2 c = e4m3x2_to_float2(e & 1 ? vw[e / 2] >> 16 : vw[e / 2] & 0xffffu);
      kf[2 * e] = a.x * ks;
      kf[2 * e + 1] = a.y * ks;
      vf[2 * e] = c.x * vs;
      vf[2 * e + 1] = c.y * vs;
    }
    const long long at = ((long long)t * per_row + x) * V;
    *reinterpret_cast<uint4*>(k + at) = pack(kf);
    *reinterpret_cast<uint4*>(v + at) = pack(vf);
  }
}

template <typename T, int D>
usp_status_t launch_read(const ReadParams& P, cudaStream_t st) {
  const long long n = (long long)P.T * P.c.H * (D / kVec<T>);  // of a sequence
  long long cap = (16LL * sm_count() + P.c.B - 1) / P.c.B;
  // (a thread's first row and column in 32 bits)
  if (cap > 0x7fffffff / kReadThreads / 2) cap = 0x7fffffff / kReadThreads / 2;
  const long long need = (n + kReadThreads - 1) / kReadThreads;
  {
    ProfScope ps(st, "kv8_read");
    read_kernel<T, D><<<dim3((unsigned)(need < cap ? need : cap), P.c.B), kReadThreads, 0, st>>>(P);
  }
  note_launch();
  return check_launch();
}

}  // namespace

usp_status_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t st) {
  AppendParams P{};
  P.a = a;
  if (a.T == 0) {  // no tokens: the lengths alone
    if (!a.lens_out) return USP_OK;
    {
      ProfScope ps(st, "kv8_append_lens");
      append_lens_kernel<<<(a.c.B + 127) / 128, 128, 0, st>>>(P);
    }
    note_launch();
    return check_launch();
  }
  if (a.bf16)
    return a.D == 128 ? launch_append<__nv_bfloat16, 128>(P, st)
                      : launch_append<__nv_bfloat16, 64>(P, st);
  return a.D == 128 ? launch_append<float, 128>(P, st) : launch_append<float, 64>(P, st);
}

usp_status_t launch_kv8_read(const Cache& c, int D, const int* start, int T, void* k, void* v,
                             int bf16, cudaStream_t st) {
  ReadParams P{c, start, T, k, v};
  if (bf16)
    return D == 128 ? launch_read<__nv_bfloat16, 128>(P, st) : launch_read<__nv_bfloat16, 64>(P, st);
  return D == 128 ? launch_read<float, 128>(P, st) : launch_read<float, 64>(P, st);
}

}  // namespace usp
