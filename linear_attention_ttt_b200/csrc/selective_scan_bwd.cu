// Selective scan, backward (selective_scan_bwd of include/ttt.h).
//
// A warp holds 16 states of 16 channels (a lane: 4 states of 2 channels), a
// block up to four warps: channel tiles of one head beside one another, or the
// 16-state parts of one tile. The tokens are worked in parts of 32:
//   - forward through the part, keeping the state before every fourth token in
//     shared memory;
//   - backward through its blocks of four tokens: each is run forward once
//     more from its kept state with the decays and states in registers, then
//     backward, carrying g; y, which the gate's gradient needs, comes along.
// So a part takes two exponentials per (channel, state, token), and states
// never travel token by token through memory.
//
// The sequence is cut into chunks of several parts so that every SM has work.
// A first pass (one exponential) finds each part's start state from a zero
// start of its chunk, the chunk's decay exp(A sum D_t), and the gradient that
// the chunk sends to the state before it; a small kernel joins the chunks in
// both directions; the main pass then starts every chunk, and every part, from
// true states. Sums over channels (dB, dC) and over tokens (dA, dD, ddt_bias)
// leave a block as partial sums that a second kernel adds in order.
//
// What bounds it: three exponentials and about 21 fp32 operations per
// (channel, state, token) in both passes together, and the sums over channels:
// every token leaves 32 sums over 16 channels a warp, which cost about as many
// instructions as the recurrence. B2 T2048 d2048 N16 takes 369 us; in a
// profile the main pass is 273 (two blocks an SM by registers and shared memory,
// 40 % of the issue slots used) and the first pass 70. At the special-function
// unit's rate alone both together would be 101 us.
#include "scan.cuh"

namespace ttt {
namespace scan {
namespace {

constexpr int kBlk = 4;     // tokens held in registers

constexpr int kMostChunks = 8192;

struct Plan : Grid {
  int parts, chunk, chunks;  // parts in all, parts a chunk, chunks
};
Plan plan(const ScanArgs& a) {
  Plan p;
  static_cast<Grid&>(p) = grid_of(a);
  p.parts = (a.T + kPart - 1) / kPart;
  // Blocks run two an SM; a chunk costs its parts and about 0.6 of one for
  // itself (rates, sums, the join), the last round of blocks 0.8 of a chunk.
  // Measured (N 16, bf16, gated) in chunks of 1, 2, 4, 8, 64 parts: B4 T2048 d4096
  // 1319, 1278, 1244, 1229, 1449 us; B1 T8192 d2048 734, 672, 653, 673, 1370;
  // B1 T200 d512 55, 58, 90, 129, 129.
  const double slots = 148 * 2;
  double best = 0;
  p.chunk = 1;
  for (int c = 1; c <= p.parts && c <= 1024; ++c) {
    const double rounds = (double)p.blocks * ((p.parts + c - 1) / c) / slots;
    const double cost = ((rounds > 1 ? rounds : 1) + 0.8) * (c + 0.6);
    if ((p.parts + c - 1) / c <= kMostChunks && (best == 0 || cost < best)) {
      best = cost;
      p.chunk = c;
    }
  }
  if (best == 0 && p.parts > 0) p.chunk = (p.parts + kMostChunks - 1) / kMostChunks;
  p.chunks = (p.parts + p.chunk - 1) / p.chunk;
  return p;
}

// Workspace, in floats.
struct Ws {
  float *start, *sums;      // [parts][blocks][warps a block][kPiece], [parts][blocks][channels]
  float *hin, *gin, *total; // [chunks][blocks]... likewise; total: sum of D_t over a chunk
  float* sums_of;           // [chunks * B][cols]: a batch row's partial sums of dA, then of dD and ddt_bias
  int64_t cols;
  float *dBC;               // [blocks][T][2][states padded]
  int64_t floats;
};
Ws carve(const ScanArgs& a, const Plan& p, float* base) {
  Ws w;
  const int64_t wpb = (int64_t)p.tpb * p.warps, ch = (int64_t)p.tpb * kCh;
  int64_t at = 0;
  auto take = [&](int64_t n) {
    float* r = base ? base + at : nullptr;
    at += (n + 3) / 4 * 4;
    return r;
  };
  w.start = take(p.parts * p.blocks * wpb * kPiece);
  w.sums = take(p.parts * p.blocks * ch);
  w.hin = take(p.chunks * p.blocks * wpb * kPiece);
  w.gin = take(p.chunks * p.blocks * wpb * kPiece);
  w.total = take(p.chunks * p.blocks * ch);
  w.cols = p.blocks / a.B * (wpb * kPiece + 2 * ch);
  w.sums_of = take(p.chunks * (int64_t)a.B * w.cols);
  w.dBC = take(p.blocks * a.T * 2 * p.warps * kNB);
  w.floats = at;
  return w;
}

// Shared memory of a block.
template <int W, bool kPre>
struct Shared {
  static constexpr int tpb = tiles_per_block(W), wpb = W * tpb, threads = 32 * wpb;
  static constexpr int cw = tpb * kCh, ns = W * kNB;
  static constexpr int kBlocks = kPart / kBlk;
  float dt[kPart * cw], u[kPart * cw], e[kPart * cw];  // D_t, D_t x_t, e_t [token][channel]
  float b[kPart * 2 * ns], c[kPart * 2 * ns];          // [token][state], each value twice
  // A warp's sums over its states of g B, g A exp(DA) h and C h [token][channel].
  // With one warp a tile the last two take the places of u and e, token by token.
  float q[kPre ? 4 : wpb * kPart * kCh];
  float ry[kPre || W == 1 ? 4 : 2 * wpb * kPart * kCh];
  // A warp's states before every block but the last; a block's dB, dC [4][32]
  // take the place of its states, the last block's have room of their own.
  float keep[kPre ? 4 : wpb * ((kBlocks - 1) * kPiece + kBlk * 32)];
  float red[kPre ? 4 : wpb * kBlk * 256];              // a block's dB, dC on their way over lanes
  int seq[kPart];
};

// Stages a part: D_t, D_t x_t and e_t (the gradient of y_t) of the block's
// channels, B and C of its states. Dead tokens are zeros, so that nothing of
// theirs enters a sum.
template <bool kWhole, typename T, typename S>
__device__ __forceinline__ void stage_as(const ScanArgs& a, const TokView& dy, const Place& q, int tb, uint32_t live,
                                      const float (&bias)[4], S& s) {
  constexpr int kGroups = S::cw / 4, dr = S::threads / kGroups;
  const int vc = q.tid % kGroups * 4, vn = a.d - q.c0 - vc;
  constexpr int kTurns = (kPart + dr - 1) / dr;
  const T* xp = static_cast<const T*>(a.x.p) + q.b * a.x.sb + q.h * a.x.sh + q.c0 + vc;
  const T* dp = static_cast<const T*>(a.dt.p) + q.b * a.dt.sb + q.h * a.dt.sh + q.c0 + vc;
  const T* gp = static_cast<const T*>(dy.p) + q.b * dy.sb + q.h * dy.sh + q.c0 + vc;
  // without a gate the gradient stands in its place and is not used
  const bool gate = a.z.p != nullptr;
  const T* zp = gate ? static_cast<const T*>(a.z.p) + q.b * a.z.sb + q.h * a.z.sh + q.c0 + vc : gp;
  const int64_t zs = gate ? a.z.st : dy.st;
  using R = typename Raw<T>::type;
  R rx[kTurns], rd[kTurns], re[kTurns], rz[kTurns];
#pragma unroll
  for (int pass = 0; pass < (kWhole ? 1 : 2); ++pass) {
    if (pass == 1 && a.wide && (vn >= kV || vn <= 0)) break;  // no ragged piece
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int row = min(i * dr + q.tid / kGroups, kPart - 1);
      const int n = kWhole || live >> row & 1 ? vn : 0;
      const bool whole = kWhole || (a.wide && n >= kV);
      const int64_t t = tb + row;
      if (pass == 0) {
        rx[i] = raw_whole<T>(xp + t * a.x.st, whole);
        rd[i] = raw_whole<T>(dp + t * a.dt.st, whole);
        re[i] = raw_whole<T>(gp + t * dy.st, whole);
        rz[i] = raw_whole<T>(zp + t * zs, whole);
      } else {
        raw_rest<T>(rx[i], xp + t * a.x.st, n, a.wide);
        raw_rest<T>(rd[i], dp + t * a.dt.st, n, a.wide);
        raw_rest<T>(re[i], gp + t * dy.st, n, a.wide);
        raw_rest<T>(rz[i], zp + t * zs, n, a.wide);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int row = i * dr + q.tid / kGroups;
    if (kPart % dr != 0 && row >= kPart) break;
    const bool on = kWhole || live >> row & 1;
    float x[4], d[4], e[4], z[4];
    floats_of(rx[i], x);
    floats_of(rd[i], d);
    floats_of(re[i], e);
    floats_of(rz[i], z);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[j] += bias[j];
      if (a.softplus) d[j] = softplus_f(d[j]);
      if (gate) e[j] *= silu_f(z[j]);
      if (!on) d[j] = 0.f;
    }
    const int o = row * S::cw + vc;
    *reinterpret_cast<float4*>(s.dt + o) = make_float4(d[0], d[1], d[2], d[3]);
    *reinterpret_cast<float4*>(s.u + o) = make_float4(d[0] * x[0], d[1] * x[1], d[2] * x[2], d[3] * x[3]);
    *reinterpret_cast<float4*>(s.e + o) = make_float4(e[0], e[1], e[2], e[3]);
  }
  constexpr int per = S::ns / 2;  // two states a turn: consecutive threads write consecutive 16 bytes
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const TokView& v = w ? a.Cm : a.Bm;
    const T* p = static_cast<const T*>(v.p) + q.b * v.sb + q.g * v.sh;
#pragma unroll
    for (int i0 = 0; i0 < kPart * per; i0 += S::threads) {
      const int i = i0 + q.tid, row = i / per, n0 = i % per * 2;
      if (kPart * per % S::threads != 0 && i >= kPart * per) break;
      // the reads are always made, in bounds; what is not there becomes zero
      const bool on = kWhole || live >> row & 1;
      const T* at = p + (int64_t)min(tb + row, a.T - 1) * v.st;
      const float v0 = to_f32(at[min(n0, a.N - 1)]), v1 = to_f32(at[min(n0 + 1, a.N - 1)]);
      const float f0 = on && n0 < a.N ? v0 : 0.f, f1 = on && n0 + 1 < a.N ? v1 : 0.f;
      reinterpret_cast<float4*>(w ? s.c : s.b)[i] = make_float4(f0, f0, f1, f1);
    }
  }
}

// Whether a part is whole: every token live, every channel there, rows aligned.
template <typename S>
__device__ __forceinline__ bool is_whole(const ScanArgs& a, const Place& q, uint32_t live) {
  return a.wide && live == 0xffffffffu && q.c0 + S::cw <= a.d;
}
template <typename T, typename S>
__device__ __forceinline__ void stage(const ScanArgs& a, const TokView& dy, const Place& q, int tb, uint32_t live,
                                      const float (&bias)[4], S& s) {
  if (is_whole<S>(a, q, live)) stage_as<true, T>(a, dy, q, tb, live, bias, s);
  else stage_as<false, T>(a, dy, q, tb, live, bias, s);
}

// Four parameters of the channels from c on (head h), zeros for null.
__device__ __forceinline__ void four_of(const float* p, const ScanArgs& a, int h, int c, float (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = p ? p[(int64_t)h * a.d + min(c + j, a.d - 1)] : 0.f;
}

// First pass over a chunk: start states of its parts from a zero start, sums
// of D_t before each part and over the chunk, the chunk's end state (to hin of
// the chunk itself, joined later), and the gradient it sends back (to gin).
template <typename T, int W>
__global__ void __launch_bounds__(128, 4) pre_kernel(ScanBwdArgs ga, Plan p, Ws ws) {
  using S = Shared<W, true>;
  extern __shared__ __align__(16) unsigned char raw[];
  S& s = *reinterpret_cast<S*>(raw);
  const ScanArgs& a = ga.f;
  const Place q = place<W>(a, p.per_head);
  const int chunk = blockIdx.y;
  f2 A2[4], hs[4] = {0, 0, 0, 0}, gs[4] = {0, 0, 0, 0}, P[4];
  rates(a, q, A2);
#pragma unroll
  for (int k = 0; k < 4; ++k) P[k] = mk2(1.f, 1.f);
  f2 sum = 0;
  float bias[4];
  {
    const int vc = q.tid % (S::cw / 4) * 4;
    four_of(a.dt_bias, a, q.h, q.c0 + vc, bias);
  }
  bool open = true;  // the sequence that enters the chunk has not ended
  pdl_trigger();     // the join may be launched now, and waits
  const int lane_c = q.wt * kCh + q.cg * 2, lane_s = q.wn * 2 * kNB + q.sg * 8;
  const int part1 = min(p.parts, (chunk + 1) * p.chunk);
  for (int part = chunk * p.chunk; part < part1; ++part) {
    const int64_t at = (int64_t)part * p.blocks + blockIdx.x;
    if (part > chunk * p.chunk) {
      store_piece(ws.start + (at * S::wpb + q.warp) * kPiece, q.lane, hs);
      if (q.wn == 0 && q.sg == 0) *reinterpret_cast<f2*>(ws.sums + at * S::cw + lane_c) = sum;
    }
    const int tb = part * kPart, nt = min(kPart, a.T - tb);
    int seq;
    const Marks m = marks(a, q, tb, nt, &seq);
    if (q.warp == 0) s.seq[q.lane] = seq;
    stage<T>(a, ga.dy, q, tb, m.live, bias, s);
    __syncthreads();
    auto token = [&](int t, bool events) {
      if (events && (m.begin >> t & 1)) {
        seq_state(a, q, a.h0, s.seq[t], hs);
        if (tb + t != chunk * p.chunk * kPart) open = false;
      }
      const f2 dt = *reinterpret_cast<const f2*>(s.dt + t * S::cw + lane_c);
      const f2 u = *reinterpret_cast<const f2*>(s.u + t * S::cw + lane_c);
      const f2 e = *reinterpret_cast<const f2*>(s.e + t * S::cw + lane_c);
      f2 bb[4], cc[4], dec[4];
      four(s.b + t * 2 * S::ns + lane_s, bb);
      four(s.c + t * 2 * S::ns + lane_s, cc);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dec[k] = ex2_pair(mul2(dt, A2[k]));
        hs[k] = fma2(dec[k], hs[k], mul2(u, bb[k]));
      }
      sum = add2(sum, dt);
      if (events && !open) return;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        P[k] = mul2(P[k], dec[k]);
        gs[k] = fma2(P[k], mul2(e, cc[k]), gs[k]);
      }
      if (events && (m.end >> t & 1)) {
        open = false;
        f2 df[4];
        seq_state(a, q, ga.dh_final, s.seq[t], df);
#pragma unroll
        for (int k = 0; k < 4; ++k) gs[k] = fma2(P[k], df[k], gs[k]);
      }
    };
#pragma unroll 1
    for (int t4 = 0; t4 < nt; t4 += 4) {
      if (open && t4 + 4 <= nt && !((m.begin | m.end) >> t4 & 15)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) token(t4 + i, false);
      } else {
#pragma unroll 1
        for (int t = t4; t < min(t4 + 4, nt); ++t) token(t, true);
      }
    }
    __syncthreads();
  }
  const int64_t at = (int64_t)chunk * p.blocks + blockIdx.x;
  store_piece(ws.hin + (at * S::wpb + q.warp) * kPiece, q.lane, hs);
  store_piece(ws.gin + (at * S::wpb + q.warp) * kPiece, q.lane, gs);
  if (q.wn == 0 && q.sg == 0) *reinterpret_cast<f2*>(ws.total + at * S::cw + lane_c) = sum;
}

constexpr int kAhead = 8;  // chunks read before their use

// Joins the chunks: hin becomes the state before each chunk, gin the gradient
// that reaches the state behind it. An element a thread. A chunk in which a
// sequence begins (or ends) passes nothing through, and nothing crosses a
// border at which one begins.
__global__ void join_kernel(ScanArgs a, Plan p, Ws ws) {
  // packed sequences: bit 0 the sequence at a chunk's first token was there
  // before it, bit 1 and before the chunk in front of it, bit 2 and it goes on
  // behind the chunk
  __shared__ uint8_t border[kMostChunks];
  if (a.seqs.cu) {
    const int span = p.chunk * kPart;
    for (int i = threadIdx.x; i < p.chunks; i += blockDim.x) {
      const TokenAt at = token_at(a.seqs, 0, a.T, i * span, a.status);
      const bool on = at.live && at.lo < i * span;
      border[i] = on | (on && at.lo < (i - 1) * span) << 1 | (on && at.hi > (i + 1) * span) << 2;
    }
    __syncthreads();
  }
  const int64_t per = p.blocks * p.wpb() * kPiece, e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= per) return;
  const PieceAt at = piece_at(e, p);
  const int n = at.n, cb = at.cb;
  const int64_t blk = at.blk;
  const int c = (int)(blk % p.per_head) * p.cw() + cb, h = (int)(blk / p.per_head % a.H);
  const float A2 = n < a.N && c < a.d ? a.A[((int64_t)h * a.d + c) * a.N + n] * kLog2e : 0.f;
  const int64_t row = p.blocks * p.cw();
  const float* total = ws.total + blk * p.cw() + cb;
  pdl_trigger();
  pdl_wait();
  for (int way = 0; way < 2; ++way) {  // forward: states, backward: gradients
    float* x = (way ? ws.gin : ws.hin) + e;
    float carry = 0.f;
    for (int i0 = 0; i0 < p.chunks; i0 += kAhead) {
      float local[kAhead], dec[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int k = min(i0 + j, p.chunks - 1);
        const int64_t i = way ? p.chunks - 1 - k : k;
        local[j] = x[i * per];
        dec[j] = ex2(A2 * total[i * row]);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (i0 + j >= p.chunks) break;
        const int i = way ? p.chunks - 1 - (i0 + j) : i0 + j;
        x[i * per] = carry;
        bool through = way ? i + 1 < p.chunks : i > 0, on = true;
        if (a.seqs.cu) {
          const int mark = border[way ? i : min(i + 1, p.chunks - 1)];
          on = mark & 1;
          through = way ? mark & 4 : mark & 2;
        }
        carry = !on ? 0.f : through ? fmaf(dec[j], carry, local[j]) : local[j];
      }
    }
  }
}

// Where a warp's sums go: [token * stride + channel], and its kept states.
struct WarpMem {
  float *q, *r, *y, *keep, *red;
};
struct BackRegs {
  f2 hs[4], gs[4], dA[4];
};

// One block of tokens: forward from its kept state hs with the decays and
// states in registers, then backward, carrying gs. kEvents: sequences may begin
// or end in the block, or the tokens end.
template <int W, bool kEvents>
__device__ __forceinline__ void back_block(const ScanBwdArgs& ga, Shared<W, false>& s, const Place& q, const Marks& m,
                                           int nt, int blk, const f2 (&A2)[4], BackRegs& g_, const WarpMem& mem) {
  using S = Shared<W, false>;
  constexpr int cw = S::cw, ns = S::ns, qs = W == 1 ? cw : kCh;
  const ScanArgs& a = ga.f;
  const int lane_c = q.wt * kCh + q.cg * 2, lane_s = q.wn * 2 * kNB + q.sg * 8;
  f2(&hs)[4] = g_.hs;
  f2(&gs)[4] = g_.gs;
  f2(&dA)[4] = g_.dA;
  float *keep = mem.keep, *red = mem.red, *sq = mem.q, *sr = mem.r, *sy = mem.y;
  f2 dec[kBlk][4], st[kBlk][4];  // the decays, and the decayed states exp(D A) h_{t-1}
#pragma unroll
  for (int i = 0; i < kBlk; ++i) {
    const int t = blk * kBlk + i;
    if (kEvents && t >= nt) continue;
    if (kEvents && (m.begin >> t & 1)) seq_state(a, q, a.h0, s.seq[t], hs);
    const f2 dt = *reinterpret_cast<const f2*>(s.dt + t * cw + lane_c);
    const f2 u = *reinterpret_cast<const f2*>(s.u + t * cw + lane_c);
    f2 bb[4];
    four(s.b + t * 2 * ns + lane_s, bb);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dec[i][k] = ex2_pair(mul2(dt, A2[k]));
      st[i][k] = mul2(dec[i][k], hs[k]);
      hs[k] = fma2(u, bb[k], st[i][k]);
    }
  }
  f2 vq[kBlk], vr[kBlk], vy[kBlk];
  float* out = keep + (blk < S::kBlocks - 1 ? blk * kPiece : (S::kBlocks - 1) * kPiece);
#pragma unroll
  for (int i = kBlk - 1; i >= 0; --i) {
    const int t = blk * kBlk + i;
    vq[i] = vr[i] = vy[i] = 0;
    if (kEvents && t >= nt) continue;
    if (kEvents && (m.end >> t & 1)) seq_state(a, q, ga.dh_final, s.seq[t], gs);
    const f2 dt = *reinterpret_cast<const f2*>(s.dt + t * cw + lane_c);
    const f2 u = *reinterpret_cast<const f2*>(s.u + t * cw + lane_c);
    const f2 e = *reinterpret_cast<const f2*>(s.e + t * cw + lane_c);
    f2 bb[4], cc[4];
    float dB[4], dC[4];
    four(s.b + t * 2 * ns + lane_s, bb);
    four(s.c + t * 2 * ns + lane_s, cc);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f2 g = fma2(e, cc[k], gs[k]), h = fma2(u, bb[k], st[i][k]);
      vq[i] = fma2(g, bb[k], vq[i]);
      vy[i] = fma2(h, cc[k], vy[i]);
      const f2 gh = mul2(g, st[i][k]);
      vr[i] = fma2(gh, A2[k], vr[i]);
      dA[k] = fma2(gh, dt, dA[k]);
      gs[k] = mul2(dec[i][k], g);
      float lo, hi;
      un2(mul2(g, u), lo, hi);
      dB[k] = lo + hi;
      un2(mul2(e, h), lo, hi);
      dC[k] = lo + hi;
    }
    if (kEvents && (m.begin >> t & 1) && ga.dh0) put_state(a, q, ga.dh0, s.seq[t], gs);
    // dB, dC on their way over the warp's 8 channel lanes
    *reinterpret_cast<float4*>(red + i * 256 + q.cg * 32 + q.sg * 4) = make_float4(dB[0], dB[1], dB[2], dB[3]);
    *reinterpret_cast<float4*>(red + i * 256 + q.cg * 32 + 16 + q.sg * 4) = make_float4(dC[0], dC[1], dC[2], dC[3]);
  }
  // a value a lane of every token: which = lane / 16 of state lane % 16
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kBlk; ++i) {
    if (kEvents && blk * kBlk + i >= nt) continue;
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = red[i * 256 + c * 32 + q.lane];
    out[i * 32 + q.lane] = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
  }
  __syncwarp();
  // the four tokens' sums over the tile's state lanes: halve twice, a token a lane is left
  const bool up = q.sg & 1, up2 = q.sg & 2;
  const int t = blk * kBlk + (up ? 2 : 0) + (up2 ? 1 : 0);
  auto join = [&](const f2 (&v)[kBlk]) {
    const f2 v0 = add2(up ? v[2] : v[0], __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 1));
    const f2 v1 = add2(up ? v[3] : v[1], __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 1));
    return add2(up2 ? v1 : v0, __shfl_xor_sync(0xffffffffu, up2 ? v0 : v1, 2));
  };
  *reinterpret_cast<f2*>(sq + t * qs + q.cg * 2) = join(vq);
  *reinterpret_cast<f2*>(sr + t * qs + q.cg * 2) = join(vr);
  *reinterpret_cast<f2*>(sy + t * qs + q.cg * 2) = join(vy);
}
// The rare form stays out of the other's registers.
template <int W>
__device__ __noinline__ void back_block_events(const ScanBwdArgs& ga, Shared<W, false>& s, const Place& q,
                                               const Marks& m, int nt, int blk, const BackRegs& rate, BackRegs& g_,
                                               const WarpMem& mem) {
  back_block<W, true>(ga, s, q, m, nt, blk, rate.hs, g_, mem);
}

template <typename T, int W>
__global__ void __launch_bounds__(128, 2) main_kernel(const __grid_constant__ ScanBwdArgs ga, Plan p, Ws ws) {
  using S = Shared<W, false>;
  constexpr int cw = S::cw, ns = S::ns, wpb = S::wpb;
  constexpr int kGroups = cw / 4, dr = S::threads / kGroups;
  extern __shared__ __align__(16) unsigned char raw[];
  S& s = *reinterpret_cast<S*>(raw);
  const ScanArgs& a = ga.f;
  const Place q = place<W>(a, p.per_head);
  const int chunk = blockIdx.y;
  const int64_t chat = (int64_t)chunk * p.blocks + blockIdx.x;
  f2 A2[4];
  BackRegs regs;
#pragma unroll
  for (int k = 0; k < 4; ++k) regs.dA[k] = 0;
  rates(a, q, A2);
  if (p.chunks > 1) {
    pdl_wait();  // launched before the joined states were there
    load_piece(ws.gin + (chat * wpb + q.warp) * kPiece, q.lane, regs.gs);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) regs.gs[k] = 0;
  }
  const int vc = q.tid % kGroups * 4, vn = a.d - q.c0 - vc;
  float bias[4], sD[4] = {0.f, 0.f, 0.f, 0.f}, sbias[4] = {0.f, 0.f, 0.f, 0.f};
  float dskip[4];
  four_of(a.dt_bias, a, q.h, q.c0 + vc, bias);
  four_of(a.D, a, q.h, q.c0 + vc, dskip);
  const float ln2 = 0.6931471805599453f;
  const int lane_c = q.wt * kCh + q.cg * 2, lane_s = q.wn * 2 * kNB + q.sg * 8;
  WarpMem mem;
  mem.q = s.q + (W == 1 ? q.wt * kCh : q.warp * kPart * kCh);
  mem.r = W == 1 ? s.u + q.wt * kCh : s.ry + q.warp * kPart * kCh;
  mem.y = W == 1 ? s.e + q.wt * kCh : s.ry + (wpb + q.warp) * kPart * kCh;
  mem.keep = s.keep + q.warp * ((S::kBlocks - 1) * kPiece + kBlk * 32);
  mem.red = s.red + q.warp * kBlk * 256;

  const int part0 = chunk * p.chunk, part1 = min(p.parts, part0 + p.chunk);
  for (int part = part1 - 1; part >= part0; --part) {
    const int tb = part * kPart, nt = min(kPart, a.T - tb), last = (nt - 1) / kBlk;
    int seq;
    const Marks m = marks(a, q, tb, nt, &seq);
    if (q.warp == 0) s.seq[q.lane] = seq;
    stage<T>(a, ga.dy, q, tb, m.live, bias, s);
    // the state before the part
    f2(&hs)[4] = regs.hs;
    if (p.chunks > 1) {
      load_piece(ws.hin + (chat * wpb + q.warp) * kPiece, q.lane, hs);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) hs[k] = 0;
    }
    if (part > part0) {
      const int64_t at = (int64_t)part * p.blocks + blockIdx.x;
      f2 local[4];
      load_piece(ws.start + (at * wpb + q.warp) * kPiece, q.lane, local);
      const TokenAt here = token_at(a.seqs, q.b, a.T, tb, a.status);
      const bool entered = here.live && here.lo < part0 * kPart;  // its sequence was there before the chunk
      const f2 sum = *reinterpret_cast<const f2*>(ws.sums + at * cw + lane_c);
#pragma unroll
      for (int k = 0; k < 4; ++k) hs[k] = entered ? fma2(ex2_pair(mul2(sum, A2[k])), hs[k], local[k]) : local[k];
    }
    __syncthreads();
    // whether block blk is whole and no sequence begins or ends in it
    auto plain = [&](int blk) {
      return blk * kBlk + kBlk <= nt && !((m.begin | m.end) >> (blk * kBlk) & ((1u << kBlk) - 1));
    };
    // forward, keeping the state before every block; hs ends before the last one
    auto step = [&](int t, bool events) {
      if (events && (m.begin >> t & 1)) seq_state(a, q, a.h0, s.seq[t], hs);
      const f2 dt = *reinterpret_cast<const f2*>(s.dt + t * cw + lane_c);
      const f2 u = *reinterpret_cast<const f2*>(s.u + t * cw + lane_c);
      f2 bb[4];
      four(s.b + t * 2 * ns + lane_s, bb);
#pragma unroll
      for (int k = 0; k < 4; ++k) hs[k] = fma2(ex2_pair(mul2(dt, A2[k])), hs[k], mul2(u, bb[k]));
    };
#pragma unroll 1
    for (int blk = 0; blk < last; ++blk) {
      store_piece(mem.keep + blk * kPiece, q.lane, hs);
      if (plain(blk)) {
#pragma unroll
        for (int i = 0; i < kBlk; ++i) step(blk * kBlk + i, false);
      } else {
#pragma unroll 1
        for (int i = 0; i < kBlk; ++i) step(blk * kBlk + i, true);
      }
    }
    // backward, block by block
#pragma unroll 1
    for (int blk = last; blk >= 0; --blk) {
      if (blk < last) {
        load_piece(mem.keep + blk * kPiece, q.lane, hs);
        __syncwarp();  // read by every lane before the block's dB, dC go there
      }
      if (plain(blk)) {
        back_block<W, false>(ga, s, q, m, nt, blk, A2, regs, mem);
      } else {
        BackRegs rate, copy = regs;
#pragma unroll
        for (int k = 0; k < 4; ++k) rate.hs[k] = A2[k];
        const Place qc = q;
        const Marks mc = m;
        const WarpMem memc = mem;
        back_block_events<W>(ga, s, qc, mc, nt, blk, rate, copy, memc);
        regs = copy;
      }
    }
    __syncthreads();
    // dx, ddt, dz, and the channels' sums
    const float* q0 = s.q;
    const float* r0 = W == 1 ? s.u : s.ry;
    const float* y0 = W == 1 ? s.e : s.ry + wpb * kPart * kCh;
    auto finish = [&](auto whole) {
      constexpr bool kWhole = decltype(whole)::value;
      constexpr int kTurns = (kPart + dr - 1) / dr;
      const int64_t t0 = tb;
      const T* xp = static_cast<const T*>(a.x.p) + q.b * a.x.sb + q.h * a.x.sh + q.c0 + vc;
      const T* dp = static_cast<const T*>(a.dt.p) + q.b * a.dt.sb + q.h * a.dt.sh + q.c0 + vc;
      const T* gp = static_cast<const T*>(ga.dy.p) + q.b * ga.dy.sb + q.h * ga.dy.sh + q.c0 + vc;
      // without a gate the gradient stands in its place and is not used
      const bool gate = a.z.p != nullptr;
      const T* zp = gate ? static_cast<const T*>(a.z.p) + q.b * a.z.sb + q.h * a.z.sh + q.c0 + vc : gp;
      const int64_t zs = gate ? a.z.st : ga.dy.st;
      using R = typename Raw<T>::type;
      R rx[kTurns], rd[kTurns], re[kTurns], rz[kTurns];
#pragma unroll
      for (int pass = 0; pass < (kWhole ? 1 : 2); ++pass) {
        if (pass == 1 && a.wide && (vn >= kV || vn <= 0)) break;  // no ragged piece
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
          const int row = min(i * dr + q.tid / kGroups, kPart - 1);
          const int n = kWhole || m.live >> row & 1 ? vn : 0;
          const bool whole = kWhole || (a.wide && n >= kV);
          const int64_t t = t0 + row;
          if (pass == 0) {
            rx[i] = raw_whole<T>(xp + t * a.x.st, whole);
            rd[i] = raw_whole<T>(dp + t * a.dt.st, whole);
            re[i] = raw_whole<T>(gp + t * ga.dy.st, whole);
            rz[i] = raw_whole<T>(zp + t * zs, whole);
          } else {
            raw_rest<T>(rx[i], xp + t * a.x.st, n, a.wide);
            raw_rest<T>(rd[i], dp + t * a.dt.st, n, a.wide);
            raw_rest<T>(re[i], gp + t * ga.dy.st, n, a.wide);
            raw_rest<T>(rz[i], zp + t * zs, n, a.wide);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const int row = i * dr + q.tid / kGroups;
        if (kPart % dr != 0 && row >= kPart) break;
        if (!kWhole && (!(m.live >> row & 1) || vn <= 0)) continue;
        const int64_t t = t0 + row;
        auto joined = [&](const float* base, float (&v)[4]) {  // over a tile's warps
          const float* at = W == 1 ? base + row * cw + vc : base + (vc / kCh * W * kPart + row) * kCh + vc % kCh;
          float4 f = *reinterpret_cast<const float4*>(at);
#pragma unroll
          for (int k = 1; k < W; ++k) {
            const float4 o = *reinterpret_cast<const float4*>(at + k * kPart * kCh);
            f.x += o.x, f.y += o.y, f.z += o.z, f.w += o.w;
          }
          v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        };
        float x[4], w[4], e[4], z[4], gb[4], gr[4], y[4], o[4];
        floats_of(rx[i], x);
        floats_of(rd[i], w);
        floats_of(re[i], e);
        floats_of(rz[i], z);
        joined(q0, gb);
        joined(r0, gr);
        if (gate) {
          joined(y0, y);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[j] = e[j] * fmaf(dskip[j], x[j], y[j]) * dsilu_f(z[j]);
            e[j] *= silu_f(z[j]);
          }
          write_row<kWhole, T, 4>(static_cast<T*>(ga.dz.p) + q.b * ga.dz.sb + q.h * ga.dz.sh + q.c0 + vc + t * ga.dz.st, vn,
                                  a.wide, o);
        }
        const float4 d = *reinterpret_cast<const float4*>(s.dt + row * cw + vc);
        o[0] = fmaf(dskip[0], e[0], d.x * gb[0]), o[1] = fmaf(dskip[1], e[1], d.y * gb[1]);
        o[2] = fmaf(dskip[2], e[2], d.z * gb[2]), o[3] = fmaf(dskip[3], e[3], d.w * gb[3]);
        write_row<kWhole, T, 4>(static_cast<T*>(ga.dx.p) + q.b * ga.dx.sb + q.h * ga.dx.sh + q.c0 + vc + t * ga.dx.st, vn,
                                a.wide, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[j] = fmaf(x[j], gb[j], gr[j] * ln2);  // the rates are in powers of two
          if (a.softplus) o[j] *= sigmoid_f(w[j] + bias[j]);
          sD[j] = fmaf(e[j], x[j], sD[j]);
          sbias[j] += o[j];
        }
        write_row<kWhole, T, 4>(static_cast<T*>(ga.ddt.p) + q.b * ga.ddt.sb + q.h * ga.ddt.sh + q.c0 + vc + t * ga.ddt.st, vn,
                                a.wide, o);
      }
    };
    if (is_whole<S>(a, q, m.live)) finish(std::true_type());
    else finish(std::false_type());
    // dB, dC over the block's channel tiles, to the block's slab
    for (int i = q.tid; i < nt * 2 * ns; i += S::threads) {
      const int t = i / (2 * ns), which = i / ns % 2, n = i % ns;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < S::tpb; ++w)
        v += s.keep[(w * W + n / kNB) * ((S::kBlocks - 1) * kPiece + kBlk * 32) + t / kBlk * kPiece + t % kBlk * 32 +
                    which * 16 + n % kNB];
      ws.dBC[(((int64_t)blockIdx.x * a.T + tb + t) * 2 + which) * ns + n] = v;
    }
    __syncthreads();
  }
  const int64_t heads = (int64_t)a.H * p.per_head, in = blockIdx.x % heads;  // the block's place in its batch row
  float* sums = ws.sums_of + ((int64_t)chunk * a.B + q.b) * ws.cols;
  store_piece(sums + (in * wpb + q.warp) * kPiece, q.lane, regs.dA);
  // the threads' channel sums: rows of threads that share channels, in order
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float* sh = s.dt;  // [dr][cw]
#pragma unroll
    for (int j = 0; j < 4; ++j) sh[q.tid / kGroups * cw + vc + j] = w ? sbias[j] : sD[j];
    __syncthreads();
    for (int c = q.tid; c < cw; c += S::threads) {
      float v = 0.f;
      for (int i = 0; i < dr; ++i) v += sh[i * cw + c];
      sums[heads * wpb * kPiece + (in * 2 + w) * cw + c] = v;
    }
    __syncthreads();
  }
}

// Destinations of the ordered sums over batch rows and chunks.
struct PutSums {
  float *dA, *dD, *dbias;
  int d, N;
  Grid g;
  int64_t first;  // columns of dA
  __device__ void operator()(int64_t col, float v) const {
    if (col < first) {
      const PieceAt at = piece_at(col, g);
      const int64_t h = at.blk / g.per_head;
      const int c = (int)(at.blk % g.per_head) * g.cw() + at.cb;
      if (at.n < N && c < d) dA[(h * d + c) * N + at.n] = v;
    } else {
      const int64_t i = col - first, blk = i / (2 * g.cw()), h = blk / g.per_head;
      const int c = (int)(blk % g.per_head) * g.cw() + (int)(i % g.cw());
      float* p = i / g.cw() % 2 ? dbias : dD;
      if (p && c < d) p[h * d + c] = v;
    }
  }
};

// dB, dC of a group: its heads' channel blocks in order.
template <typename T>
__global__ void put_bc_kernel(ScanBwdArgs ga, Plan p, const float* __restrict__ dBC) {
  const ScanArgs& a = ga.f;
  const int states = p.warps * kNB;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t row = (int64_t)a.T * 2 * states;
  if (i >= row * a.B * a.G) return;
  const int64_t in = i % row;
  const int g = (int)(i / row % a.G), b = (int)(i / row / a.G);
  const int n = (int)(in % states), which = (int)(in / states % 2), t = (int)(in / states / 2);
  if (n >= a.N) return;
  const TokenAt at = token_at(a.seqs, b, a.T, t, a.status);
  if (!at.live) return;
  const int per_group = a.H / a.G;
  const int64_t first = ((int64_t)b * a.H + (int64_t)g * per_group) * p.per_head;
  const int64_t count = (int64_t)per_group * p.per_head;
  float v = 0.f;
#pragma unroll 8
  for (int64_t k = 0; k < count; ++k) v += dBC[(first + k) * row + in];
  const TokViewMut& o = which ? ga.dCm : ga.dBm;
  static_cast<T*>(o.p)[b * o.sb + g * o.sh + (int64_t)t * o.st + n] = from_f32<T>(v);
}

template <typename T>
cudaError_t bwd(const ScanBwdArgs& ga, cudaStream_t s) {
  const ScanArgs& a = ga.f;
  const Plan p = plan(a);
  const Ws ws = carve(a, p, ga.ws);
  cudaError_t e =
      copy_empty_states(a.seqs, a.T, (int64_t)a.H * a.d * a.N, ga.dh_final, ga.dh0, a.status, s);
  if (e != cudaSuccess) return e;
  const int nw = p.wpb();
  const int64_t heads = (int64_t)a.H * p.per_head;  // channel blocks of a batch row
  if (a.T > 0) {
    e = for_warps(p.warps, [&](auto w) {
      constexpr int W = decltype(w)::value;
      using First = Shared<W, true>;
      using All = Shared<W, false>;
      cudaError_t r = cudaFuncSetAttribute(pre_kernel<T, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(First));
      if (r != cudaSuccess) return r;
      r = cudaFuncSetAttribute(main_kernel<T, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(All));
      if (r != cudaSuccess) return r;
      const dim3 grid((unsigned)p.blocks, p.chunks);
      // one chunk enters with nothing and passes nothing on; its first part
      // starts from its own beginning
      if (p.parts > 1) pre_kernel<T, W><<<grid, 32 * nw, sizeof(First), s>>>(ga, p, ws);
      const int64_t n = p.blocks * nw * kPiece;
      r = cudaGetLastError();
      if (r != cudaSuccess) return r;
      if (p.chunks > 1) {
        r = launch_pdl(join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a, p, ws);
        if (r != cudaSuccess) return r;
        r = launch_pdl(main_kernel<T, W>, grid, dim3(32 * nw), sizeof(All), s, ga, p, ws);
        if (r != cudaSuccess) return r;
      } else {
        main_kernel<T, W><<<grid, 32 * nw, sizeof(All), s>>>(ga, p, ws);
      }
      const int64_t bc = (int64_t)a.B * a.G * a.T * 2 * p.warps * kNB;
      put_bc_kernel<T><<<(unsigned)((bc + 255) / 256), 256, 0, s>>>(ga, p, ws.dBC);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
  }
  return sum_parts(ws.sums_of, (int64_t)p.chunks * a.B, ws.cols,
                   PutSums{ga.dA, ga.dD, ga.ddt_bias, a.d, a.N, p, heads * nw * kPiece}, s);
}

}  // namespace
}  // namespace scan

size_t selective_scan_bwd_workspace(const ScanBwdArgs& a) {
  return (size_t)scan::carve(a.f, scan::plan(a.f), nullptr).floats * sizeof(float);
}
cudaError_t launch_selective_scan_bwd(const ScanBwdArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? scan::bwd<__nv_bfloat16>(a, s) : scan::bwd<float>(a, s);
}

}  // namespace ttt
