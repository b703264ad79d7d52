// What the selective scan's forward and backward kernels share.
#pragma once

#include "block.cuh"

namespace ttt {
namespace scan {

constexpr int kNB = 16;    // states a warp holds
constexpr int kPart = 32;  // tokens staged at once: one 32-bit mask

// A warp holds 16 states of 16 channels: a lane has 4 states of 2 channels, a
// pair of fp32 being one state of both.
constexpr int kCh = 16;
constexpr int kPiece = kNB * kCh;  // a warp's states in memory: two float4 a lane
// (float4 q of a lane: states 4*(lane&3) + 2q, +1, each with its two channels)
constexpr int tiles_per_block(int warps) { return warps >= 3 ? 1 : 4 / warps; }

// How a call's channels and states are laid over blocks: channel tiles of one
// head beside one another, each with a warp for every 16 states.
struct Grid {
  int warps, tpb;   // 16-state warps a channel tile, channel tiles a block
  int per_head;     // blocks a head
  int64_t blocks;   // of the call: batch rows, heads
  __host__ __device__ int wpb() const { return warps * tpb; }
  __host__ __device__ int cw() const { return tpb * kCh; }  // channels a block
};
inline Grid grid_of(const ScanArgs& a) {
  Grid g;
  g.warps = (a.N + kNB - 1) / kNB;
  g.tpb = tiles_per_block(g.warps);
  g.per_head = (a.d + g.cw() - 1) / g.cw();
  g.blocks = (int64_t)a.B * a.H * g.per_head;
  return g;
}

// Where a token stands in its sequence.
struct TokenAt {
  int seq, lo, hi;
  bool live;
};
__device__ __forceinline__ TokenAt token_at(const Seqs& q, int b, int T, int t, int* status) {
  if (!q.cu) return {b, 0, T, t < T};
  TokenAt r = {first_seq_behind(q.cu, q.S, t), 0, 0, false};
  if (t < T && r.seq < q.S) {
    packed_seq(q.cu, r.seq, T, status, &r.lo, &r.hi);
    r.live = t >= r.lo && t < r.hi;
  }
  return r;
}

// Step size from its raw value.
__device__ __forceinline__ float step_of(float raw, int softplus) {
  return softplus ? softplus_f(raw) : raw;
}

// Which sequence events fall on a part's tokens.
struct Marks {
  uint32_t live, begin, end;
};

// What a block's threads know of their place.
struct Place {
  int tid, lane, warp, wt, wn;  // wt: the warp's channel tile in the block, wn: its 16 states
  int sg, cg;                   // the lane's states 4 sg .. and channels 2 cg ..
  int h, b, c0, g;              // head, batch row, first channel of the block, group
  int64_t ch0;                  // h * d + c0
};
template <int W>
__device__ __forceinline__ Place place(const ScanArgs& a, int per_head) {
  constexpr int cw = tiles_per_block(W) * kCh;
  Place q;
  q.tid = threadIdx.x;
  q.lane = q.tid & 31;
  q.warp = q.tid >> 5;
  q.wt = q.warp / W;
  q.wn = q.warp % W;
  q.sg = q.lane & 3;
  q.cg = q.lane >> 2;
  const int64_t blk = blockIdx.x;
  q.c0 = (int)(blk % per_head) * cw;
  q.h = (int)(blk / per_head % a.H);
  q.b = (int)(blk / per_head / a.H);
  q.g = q.h / (a.H / a.G);
  q.ch0 = (int64_t)q.h * a.d + q.c0;
  return q;
}

// Marks of the nt tokens at tb; *seq gets the lane's token's sequence.
__device__ __forceinline__ Marks marks(const ScanArgs& a, const Place& q, int tb, int nt, int* seq) {
  Marks m;
  if (!a.seqs.cu) {
    m.live = nt < 32 ? (1u << nt) - 1 : 0xffffffffu;
    m.begin = tb == 0;
    m.end = tb + nt == a.T ? 1u << (nt - 1) : 0;
    *seq = q.b;
    return m;
  }
  const TokenAt at = token_at(a.seqs, q.b, a.T, tb + q.lane, a.status);
  const bool in = q.lane < nt && at.live;
  m.live = __ballot_sync(0xffffffffu, in);
  m.begin = __ballot_sync(0xffffffffu, in && tb + q.lane == at.lo);
  m.end = __ballot_sync(0xffffffffu, in && tb + q.lane == at.hi - 1);
  *seq = at.seq;
  return m;
}

// A token tensor's piece of a block (kPart rows of kWidth elements from p, of
// which `left` exist) on its way into shared memory; dead rows become zeros.
template <typename T, int kWidth, int kThreads>
__device__ __forceinline__ void copy_part(T* dst, const T* p, int64_t stride, int left, uint32_t live, int tid,
                                          bool wide) {
  constexpr int V = Vec<T>::n, per = kWidth / V;
#pragma unroll
  for (int i0 = 0; i0 < kPart * per; i0 += kThreads) {
    const int i = i0 + tid, row = i / per, c = i % per * V;
    if (kPart * per % kThreads == 0 || i < kPart * per)
      copy_async(dst + i * V, p + row * stride + c, live >> row & 1 ? left - c : 0, wide);
  }
}

// A staged part of B or C (kPart rows of kWidth states) to fp32, each value
// twice: a packed operation takes two channels with one state.
template <typename T, int kWidth, int kThreads>
__device__ __forceinline__ void spread_part(float* dst, const T* src, int tid) {
  constexpr int n = kPart * kWidth / 2;
#pragma unroll
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    if (n % kThreads == 0 || i < n) {
      const float x = to_f32(src[2 * i]), y = to_f32(src[2 * i + 1]);
      reinterpret_cast<float4*>(dst)[i] = make_float4(x, x, y, y);
    }
  }
}

// Element (channel c of the block, state n) of a [H,d,N] array whose rows begin
// at `row`; 0 where there is none. The read itself is always made (in bounds):
// reads behind a choice would wait for one another.
__device__ __forceinline__ float state_at(const ScanArgs& a, const Place& q, const float* p, int64_t row, int n, int c) {
  const int cc = min(q.c0 + c, a.d - 1) - q.c0, nn = min(n, a.N - 1);
  const float v = p[(row + q.ch0 + cc) * a.N + nn];
  return nn == n && cc == c ? v : 0.f;
}

// The lane's decay rates, in powers of two.
__device__ __forceinline__ void rates(const ScanArgs& a, const Place& q, f2 (&A2)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = q.wn * kNB + q.sg * 4 + k, c = q.wt * kCh + q.cg * 2 + i;
      r[i] = state_at(a, q, a.A, 0, n, c) * kLog2e;
    }
    A2[k] = mk2(r[0], r[1]);
  }
}

// The lane's elements of a [S,H,d,N] tensor's row `seq` (zeros for null).
__device__ __forceinline__ void seq_state(const ScanArgs& a, const Place& q, const float* p, int seq,
                                          f2 (&s)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = q.wn * kNB + q.sg * 4 + k, c = q.wt * kCh + q.cg * 2 + i;
      r[i] = p ? state_at(a, q, p, (int64_t)seq * a.H * a.d, n, c) : 0.f;
    }
    s[k] = mk2(r[0], r[1]);
  }
}
__device__ __forceinline__ void put_state(const ScanArgs& a, const Place& q, float* p, int seq,
                                          const f2 (&s)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float r[2];
    un2(s[k], r[0], r[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = q.wn * kNB + q.sg * 4 + k, c = q.wt * kCh + q.cg * 2 + i;
      if (n < a.N && q.c0 + c < a.d) p[((int64_t)seq * a.H * a.d + q.ch0 + c) * a.N + n] = r[i];
    }
  }
}

// A warp's states as a piece of memory.
__device__ __forceinline__ void load_piece(const float* p, int lane, f2 (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const ulonglong2 v = reinterpret_cast<const ulonglong2*>(p)[i * 32 + lane];
    s[2 * i] = v.x;
    s[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void store_piece(float* p, int lane, const f2 (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<ulonglong2*>(p)[i * 32 + lane] = make_ulonglong2(s[2 * i], s[2 * i + 1]);
}
// Four states' values (each twice) of a token in shared memory.
__device__ __forceinline__ void four(const float* s, f2 (&v)[4]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(s), b = *reinterpret_cast<const ulonglong2*>(s + 4);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// f(integral constant) for the 16-state warps a tile has.
template <typename F>
cudaError_t for_warps(int warps, F f) {
  switch (warps) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
  }
  return cudaErrorInvalidValue;
}

// Where element e of [blocks][warps a block][piece] stands.
struct PieceAt {
  int64_t blk;
  int n, cb;  // state, channel in the block
};
__host__ __device__ __forceinline__ PieceAt piece_at(int64_t e, const Grid& g) {
  const int in = (int)(e % kPiece), lane = in % 128 / 4, k = in / 128 * 2 + in % 4 / 2, i = in % 2;
  const int warp = (int)(e / kPiece % g.wpb());
  PieceAt r;
  r.blk = e / kPiece / g.wpb();
  r.n = warp % g.warps * kNB + (lane & 3) * 4 + k;
  r.cb = warp / g.warps * kCh + (lane >> 2) * 2 + i;
  return r;
}

// dst (may be null) = src (zeros where null) for every sequence without a
// token: the states and their gradients that no kernel of the scan reaches. It
// also sees every offset of a packed call and reports the ones out of order.
cudaError_t copy_empty_states(const Seqs& q, int T, int64_t n, const float* src, float* dst,
                              int* status, cudaStream_t s);

}  // namespace scan
}  // namespace ttt
