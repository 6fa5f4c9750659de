// Rotation of positions (usp_rope): y = x with every pair of channels turned by
// its token's angles, or back by them (the gradient).
//
// A copy with six operations per pair: bound by HBM. Queries of 2 x 8192 tokens
// and 32 heads of 128, bf16, zigzag (268 MB): 38.7 us, 6.9 TB/s.
//
// A warp takes tokens; a lane one item (two vectors of 16 bytes) of a row, whose
// cos and sin it keeps in registers while it passes over the token's heads, so
// the table is read once per token. Where a token has fewer heads than lanes
// could take, the warp takes several tokens at once.
#include "internal.h"
#include "kv8.cuh"
#include "kv8_host.h"

namespace usp {
namespace {

using namespace kv8;

constexpr int kThreads = 256;

struct RopeParams {
  const void* x;
  void* y;
  Rope r;
  int inverse;
  int B, S, H;        // batch rows (1: packed), tokens of each, heads
  const int* cu;
  int nseq;
  int layout, cp, shard, chunk;
  int heads_at_once;  // of a token, a power of two
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams P) {
  constexpr int V = kVec<T>, kItems = D / (2 * V), kFlight = 4;
  const int lane = threadIdx.x & 31;
  const int item = lane % kItems, slot = lane / kItems;
  const int hp = P.heads_at_once, tw = 32 / (kItems * hp);  // tokens of a warp
  const int h0 = slot % hp;
  const Item<V> it = item_of<V>(P.r, item);
  const long long tokens = (long long)P.B * P.S;
  const long long step = (long long)gridDim.x * (kThreads / 32) * tw;
  const T* x = static_cast<const T*>(P.x);
  T* y = static_cast<T*>(P.y);
  for (long long t = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * tw + slot / hp;
       t < tokens; t += step) {
    int pos = nat_pos((int)(t % P.S), P.layout, P.cp, P.shard, P.chunk);
    Item<V> mine = it;
    if (P.cu) {
      const int n = seg_of(P.cu, P.nseq, pos), first = __ldg(P.cu + n);
      // padding outside the sequences stays as it is
      if (pos < first || pos >= __ldg(P.cu + n + 1)) mine.f = -1, mine.a = 2 * V * item,
                                                     mine.b = 2 * V * item + V;
      pos -= first;
    }
    float c[V], s[V];
    load_turn(P.r, mine, pos, c, s);
    if (P.inverse && mine.f >= 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = -s[i];
    }
    const long long row = t * P.H;
    for (int h = h0; h < P.H; h += kFlight * hp) {
      uint4 a[kFlight], b[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (h + i * hp < P.H) {
          const T* src = x + (row + h + i * hp) * D;
          a[i] = *reinterpret_cast<const uint4*>(src + mine.a);
          b[i] = *reinterpret_cast<const uint4*>(src + mine.b);
        }
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (h + i * hp < P.H) {
          T* dst = y + (row + h + i * hp) * D;
          if (mine.f >= 0) {
            float fa[V], fb[V];
            unpack(a[i], fa);
            unpack(b[i], fb);
            rotate(mine, P.r.inter != 0, c, s, fa, fb);
            a[i] = pack(fa);
            b[i] = pack(fb);
          }
          *reinterpret_cast<uint4*>(dst + mine.a) = a[i];
          *reinterpret_cast<uint4*>(dst + mine.b) = b[i];
        }
    }
  }
}

template <typename T, int D>
usp_status_t launch(RopeParams& P, cudaStream_t st) {
  constexpr int kItems = D / (2 * kVec<T>);
  int hp = 1;
  while (hp < P.H && hp * kItems < 32) hp *= 2;
  P.heads_at_once = hp;
  const long long warps = ((long long)P.B * P.S + 32 / (kItems * hp) - 1) / (32 / (kItems * hp));
  const long long need = (warps + kThreads / 32 - 1) / (kThreads / 32);
  const long long cap = (long long)sm_count() * 8;
  {
    ProfScope ps(st, "rope");
    rope_kernel<T, D><<<(unsigned)(need < cap ? need : cap), kThreads, 0, st>>>(P);
  }
  note_launch();
  return check_launch();
}

}  // namespace

usp_status_t launch_rope(const void* x, void* y, const Rope& r, int inverse, int B, int S, int H,
                         int D, const int* cu, int nseq, int cp, int layout, int bf16,
                         cudaStream_t st) {
  RopeParams P{};
  P.x = x;
  P.y = y;
  P.r = r;
  P.inverse = inverse;
  P.B = B;
  P.S = S;
  P.H = H;
  P.cu = cu;
  P.nseq = nseq;
  P.layout = layout;
  P.cp = cp;
  P.shard = S / cp;
  P.chunk = S / (2 * cp);
  if (bf16) return D == 128 ? launch<__nv_bfloat16, 128>(P, st) : launch<__nv_bfloat16, 64>(P, st);
  return D == 128 ? launch<float, 128>(P, st) : launch<float, 64>(P, st);
}

}  // namespace usp
