// Selective scan, backward (selective_scan_bwd of include/ttt.h).
//
// A warp holds 16 states of 16 channels (a lane: 4 states of 2 channels), a
// block up to four warps: channel tiles of one head beside one another, or the
// 16-state parts of one tile. The tokens are worked in parts of 32:
//   - forward through the part, keeping the state before every fourth token in
//     shared memory (and y, which the gate's gradient needs);
//   - backward through its blocks of four tokens: each is run forward once
//     more from its kept state with the decays and states in registers, then
//     backward, carrying g.
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
// (channel, state, token) in both passes together.
#include "scan.cuh"

namespace ttt {
namespace scan {
namespace {

constexpr int kBlk = 4;     // tokens held in registers

struct Plan : Grid {
  int parts, chunk, chunks;  // parts in all, parts a chunk, chunks
};
Plan plan(const ScanArgs& a) {
  Plan p;
  static_cast<Grid&>(p) = grid_of(a);
  p.parts = (a.T + kPart - 1) / kPart;
  // eight rounds of three blocks an SM; a chunk of one part costs the most
  // join traffic, a long one leaves SMs idle at the end
  const int64_t want = 148 * 3 * 8, c = (want + p.blocks - 1) / p.blocks;
  p.chunk = (int)(c >= p.parts ? 1 : (p.parts + c - 1) / c);
  if (p.chunk < 1) p.chunk = 1;
  p.chunks = (p.parts + p.chunk - 1) / p.chunk;
  return p;
}

// Workspace, in floats.
struct Ws {
  float *start, *sums;      // [parts][blocks][warps a block][kPiece], [parts][blocks][channels]
  float *hin, *gin, *total; // [chunks][blocks]... likewise; total: sum of D_t over a chunk
  float *dA, *dD;           // [B*chunks][...] partial sums; dD: dD then ddt_bias
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
  w.dA = take(p.chunks * p.blocks * wpb * kPiece);
  w.dD = take(p.chunks * p.blocks * ch * 2);
  w.dBC = take(p.blocks * a.T * 2 * p.warps * kNB);
  w.floats = at;
  return w;
}

template <typename T, int W>
struct Kernel {
  static constexpr int V = Vec<T>::n, tpb = tiles_per_block(W), nw = W * tpb;
  static constexpr int cw = tpb * kCh, states = W * kNB;

  // Stages a part: D_t, D_t x_t and e_t (the gradient of y_t) of the block's
  // channels [token][channel], B and C of its states [token][state], each
  // value twice. Dead tokens and channels are zeros.
  static __device__ __forceinline__ void stage(const ScanArgs& a, const TokView& dy, const Place& q, int tb, uint32_t live, float* s_dt, float* s_u,
                                               float* s_e, float* s_b, float* s_c) {
    constexpr int lpr = cw / V;
#pragma unroll
    for (int i = q.tid; i < kPart * lpr; i += 32 * nw) {
      const int row = i / lpr, vc = i % lpr * V;
      const int n = live >> row & 1 ? a.d - q.c0 - vc : 0;
      const int64_t t = tb + row;
      const T* xp = static_cast<const T*>(a.x.p) + q.b * a.x.sb + q.h * a.x.sh + q.c0 + vc + t * a.x.st;
      const T* dp = static_cast<const T*>(a.dt.p) + q.b * a.dt.sb + q.h * a.dt.sh + q.c0 + vc + t * a.dt.st;
      const T* gp = static_cast<const T*>(dy.p) + q.b * dy.sb + q.h * dy.sh + q.c0 + vc + t * dy.st;
      const Vec<T> xv = load_vec(xp, n, a.wide), dv = load_vec(dp, n, a.wide), gv = load_vec(gp, n, a.wide);
      float x[V], d[V], e[V], u[V];
      unpack<T>(xv, x);
      unpack<T>(dv, d);
      unpack<T>(gv, e);
      if (a.z.p) {
        const T* zp = static_cast<const T*>(a.z.p) + q.b * a.z.sb + q.h * a.z.sh + q.c0 + vc + t * a.z.st;
        float z[V];
        unpack<T>(load_vec(zp, n, a.wide), z);
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] *= silu_f(z[j]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float bias = a.dt_bias && j < n ? a.dt_bias[q.ch0 + vc + j] : 0.f;
        d[j] = j < n ? step_of(d[j] + bias, a.softplus) : 0.f;
        u[j] = d[j] * x[j];
      }
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const int o = row * cw + vc + j;
        *reinterpret_cast<float4*>(s_dt + o) = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
        *reinterpret_cast<float4*>(s_u + o) = make_float4(u[j], u[j + 1], u[j + 2], u[j + 3]);
        *reinterpret_cast<float4*>(s_e + o) = make_float4(e[j], e[j + 1], e[j + 2], e[j + 3]);
      }
    }
    constexpr int spr = states / V;
    for (int i = q.tid; i < kPart * spr * 2; i += 32 * nw) {
      const int m = i / (kPart * spr), row = i / spr % kPart, n0 = i % spr * V;
      const int n = live >> row & 1 ? a.N - n0 : 0;
      const TokView& w = m ? a.Cm : a.Bm;
      const T* p = static_cast<const T*>(w.p) + q.b * w.sb + q.g * w.sh + (int64_t)(tb + row) * w.st + n0;
      float f[V];
      unpack<T>(load_vec(p, n, a.wide), f);
      float* s = (m ? s_c : s_b) + 2 * (row * states + n0);
#pragma unroll
      for (int j = 0; j < V; j += 2)
        *reinterpret_cast<float4*>(s + 2 * j) = make_float4(f[j], f[j], f[j + 1], f[j + 1]);
    }
  }
};

struct Shared {
  float *dt, *u, *e, *b, *c;  // [32][cw], [32][2 * states]
  float *y, *r;          // a warp's: [32][ystride]; r takes the place of u where a tile has one warp
  float* keep;           // a warp's kept states: [8][kPiece], later its dB, dC [32][32]
};
template <int W>
__device__ __forceinline__ Shared shared_of(float* sm, const Place& q) {
  constexpr int tpb = tiles_per_block(W), cw = tpb * kCh, states = W * kNB, nw = W * tpb;
  Shared s;
  s.dt = sm;
  s.u = s.dt + kPart * cw;
  s.e = s.u + kPart * cw;
  s.b = s.e + kPart * cw;
  s.c = s.b + kPart * 2 * states;
  float* next = s.c + kPart * 2 * states;
  if (W == 1) {
    s.y = next + q.wt * kCh;
    s.r = s.u + q.wt * kCh;
    next += kPart * cw;
  } else {
    s.y = next + q.warp * kPart * kCh;
    s.r = s.y + nw * kPart * kCh;
    next += 2 * nw * kPart * kCh;
  }
  s.keep = next + q.warp * (kPart / kBlk) * kPiece;
  return s;
}
size_t smem_bytes(const Plan& p, bool pre) {
  const int cw = p.tpb * kCh, nw = p.tpb * p.warps;
  int64_t n = 3 * kPart * cw + 2 * kPart * 2 * p.warps * kNB;
  if (!pre) n += (p.warps == 1 ? kPart * cw : 2 * nw * kPart * kCh) + nw * (kPart / kBlk) * kPiece;
  return (size_t)n * sizeof(float);
}

// First pass over a chunk: start states of its parts from a zero start, sums
// of D_t before each part and over the chunk, the chunk's end state (to hin of
// the chunk itself, joined later), and the gradient it sends back (to gin).
template <typename T, int W>
__global__ void __launch_bounds__(128) pre_kernel(ScanBwdArgs ga, Plan p, Ws ws) {
  using K = Kernel<T, W>;
  extern __shared__ __align__(16) float sm[];
  __shared__ int s_seq[kPart];
  const ScanArgs& a = ga.f;
  const Place q = place<W>(a, p.per_head);
  const Shared s = shared_of<W>(sm, q);
  constexpr int nw = K::nw;
  const int chunk = blockIdx.y;
  f2 A2[4], hs[4] = {0, 0, 0, 0}, gs[4] = {0, 0, 0, 0}, P[4];
  rates(a, q, A2);
  const f2 one = mk2(1.f, 1.f);
#pragma unroll
  for (int k = 0; k < 4; ++k) P[k] = one;
  f2 sum = 0;
  bool open = true;  // the sequence that enters the chunk has not ended
  const int part1 = min(p.parts, (chunk + 1) * p.chunk);
  for (int part = chunk * p.chunk; part < part1; ++part) {
    const int64_t at = (int64_t)part * p.blocks + blockIdx.x;
    if (part > chunk * p.chunk) {
      store_piece(ws.start + (at * nw + q.warp) * kPiece, q.lane, hs);
      if (q.wn == 0 && q.sg == 0)
        *reinterpret_cast<f2*>(ws.sums + at * K::cw + q.wt * kCh + q.cg * 2) = sum;
    }
    const int tb = part * kPart, nt = min(kPart, a.T - tb);
    int seq;
    const Marks m = marks(a, q, tb, nt, &seq);
    if (q.warp == 0) s_seq[q.lane] = seq;
    K::stage(a, ga.dy, q, tb, m.live, s.dt, s.u, s.e, s.b, s.c);
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      if (m.begin >> t & 1) {
        seq_state(a, q, a.h0, s_seq[t], hs);
        if (tb + t != chunk * p.chunk * kPart) open = false;
      }
      const int o = t * K::cw + q.wt * kCh + q.cg * 2;
      const f2 dt = *reinterpret_cast<const f2*>(s.dt + o), u = *reinterpret_cast<const f2*>(s.u + o);
      f2 bb[4], cc[4], dec[4];
      four(s.b + t * 2 * K::states + q.wn * 2 * kNB + q.sg * 8, bb);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dec[k] = ex2_pair(mul2(dt, A2[k]));
        hs[k] = fma2(dec[k], hs[k], mul2(u, bb[k]));
      }
      sum = add2(sum, dt);
      if (open) {
        const f2 e = *reinterpret_cast<const f2*>(s.e + o);
        four(s.c + t * 2 * K::states + q.wn * 2 * kNB + q.sg * 8, cc);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          P[k] = mul2(P[k], dec[k]);
          gs[k] = fma2(P[k], mul2(e, cc[k]), gs[k]);
        }
        if (m.end >> t & 1) {
          open = false;
          f2 df[4];
          seq_state(a, q, ga.dh_final, s_seq[t], df);
#pragma unroll
          for (int k = 0; k < 4; ++k) gs[k] = fma2(P[k], df[k], gs[k]);
        }
      }
    }
    __syncthreads();
  }
  const int64_t at = (int64_t)chunk * p.blocks + blockIdx.x;
  store_piece(ws.hin + (at * nw + q.warp) * kPiece, q.lane, hs);
  store_piece(ws.gin + (at * nw + q.warp) * kPiece, q.lane, gs);
  if (q.wn == 0 && q.sg == 0) *reinterpret_cast<f2*>(ws.total + at * K::cw + q.wt * kCh + q.cg * 2) = sum;
}

constexpr int kAhead = 8;  // chunks read before their use

// Joins the chunks: hin becomes the state before each chunk, gin the gradient
// that reaches the state behind it. An element a thread. A chunk in which a
// sequence begins (or ends) passes nothing through, and nothing crosses a
// border at which one begins.
__global__ void join_kernel(ScanArgs a, Plan p, Ws ws) {
  const int64_t per = p.blocks * p.wpb() * kPiece, e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= per) return;
  const PieceAt at = piece_at(e, p);
  const int n = at.n, cb = at.cb;
  const int64_t blk = at.blk;
  const int c = (int)(blk % p.per_head) * p.cw() + cb, h = (int)(blk / p.per_head % a.H);
  const int b = (int)(blk / p.per_head / a.H);
  const float A2 = n < a.N && c < a.d ? a.A[((int64_t)h * a.d + c) * a.N + n] * kLog2e : 0.f;
  const int span = p.chunk * kPart;
  const int64_t row = p.blocks * p.cw();
  const float* total = ws.total + blk * p.cw() + cb;
  for (int way = 0; way < 2; ++way) {  // forward: states, backward: gradients
    float* x = (way ? ws.gin : ws.hin) + e;
    float carry = 0.f;
    for (int i0 = 0; i0 < p.chunks; i0 += kAhead) {
      float local[kAhead], dec[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t i = way ? p.chunks - 1 - (i0 + j) : i0 + j;
        const bool in = i0 + j < p.chunks;
        local[j] = in ? x[i * per] : 0.f;
        dec[j] = in ? ex2(A2 * total[i * row]) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (i0 + j >= p.chunks) break;
        const int i = way ? p.chunks - 1 - (i0 + j) : i0 + j;
        x[i * per] = carry;
        bool through = way ? i + 1 < p.chunks : i > 0, on = true;
        if (a.seqs.cu) {
          // the token behind the border that the carry crosses, and its sequence
          const int border = way ? i * span : (i + 1) * span;
          const TokenAt at = token_at(a.seqs, b, a.T, border, a.status);
          on = at.live && at.lo < border;
          through = on && (way ? at.hi > (i + 1) * span : at.lo < i * span);
        }
        carry = !on ? 0.f : through ? fmaf(dec[j], carry, local[j]) : local[j];
      }
    }
  }
}

template <typename T, int W>
__global__ void __launch_bounds__(128, 3) main_kernel(ScanBwdArgs ga, Plan p, Ws ws) {
  using K = Kernel<T, W>;
  constexpr int V = K::V, lpr = K::cw / V;
  extern __shared__ __align__(16) float sm[];
  __shared__ int s_seq[kPart];
  const ScanArgs& a = ga.f;
  const Place q = place<W>(a, p.per_head);
  const Shared s = shared_of<W>(sm, q);
  constexpr int nw = K::nw;
  const int chunk = blockIdx.y;
  const int64_t chat = (int64_t)chunk * p.blocks + blockIdx.x;
  f2 A2[4], h_in[4], gs[4], dA[4] = {0, 0, 0, 0};
  rates(a, q, A2);
  load_piece(ws.hin + (chat * nw + q.warp) * kPiece, q.lane, h_in);
  load_piece(ws.gin + (chat * nw + q.warp) * kPiece, q.lane, gs);
  // channel sums of the thread's vectors: their channels are the same in every turn
  constexpr int ystride = W == 1 ? K::cw : kCh;
  const int vc = q.tid % lpr * V, vn = a.d - q.c0 - vc;
  float sD[V], sbias[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sD[j] = sbias[j] = 0.f;
  const float ln2 = 0.6931471805599453f;

  const int part0 = chunk * p.chunk, part1 = min(p.parts, part0 + p.chunk);
  for (int part = part1 - 1; part >= part0; --part) {
    const int tb = part * kPart, nt = min(kPart, a.T - tb);
    int seq;
    const Marks m = marks(a, q, tb, nt, &seq);
    if (q.warp == 0) s_seq[q.lane] = seq;
    K::stage(a, ga.dy, q, tb, m.live, s.dt, s.u, s.e, s.b, s.c);
    // the state before the part
    f2 hs[4];
    if (part == part0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) hs[k] = h_in[k];
    } else {
      const int64_t at = (int64_t)part * p.blocks + blockIdx.x;
      load_piece(ws.start + (at * nw + q.warp) * kPiece, q.lane, hs);
      const TokenAt here = token_at(a.seqs, q.b, a.T, tb, a.status);
      if (here.live && here.lo < part0 * kPart) {  // its sequence entered the chunk from before
        const f2 sum = *reinterpret_cast<const f2*>(ws.sums + at * K::cw + q.wt * kCh + q.cg * 2);
#pragma unroll
        for (int k = 0; k < 4; ++k) hs[k] = fma2(ex2_pair(mul2(sum, A2[k])), h_in[k], hs[k]);
      }
    }
    __syncthreads();
    const int lane_o = q.wt * kCh + q.cg * 2, lane_s = q.wn * 2 * kNB + q.sg * 8;
    // forward, keeping the state before every block
    for (int t = 0; t < nt; ++t) {
      if (t % kBlk == 0) store_piece(s.keep + t / kBlk * kPiece, q.lane, hs);
      if (m.begin >> t & 1) seq_state(a, q, a.h0, s_seq[t], hs);
      const f2 dt = *reinterpret_cast<const f2*>(s.dt + t * K::cw + lane_o);
      const f2 u = *reinterpret_cast<const f2*>(s.u + t * K::cw + lane_o);
      f2 bb[4], cc[4], y = 0;
      four(s.b + t * 2 * K::states + lane_s, bb);
#pragma unroll
      for (int k = 0; k < 4; ++k) hs[k] = fma2(ex2_pair(mul2(dt, A2[k])), hs[k], mul2(u, bb[k]));
      if (a.z.p) {
        four(s.c + t * 2 * K::states + lane_s, cc);
#pragma unroll
        for (int k = 0; k < 4; ++k) y = fma2(hs[k], cc[k], y);
        float y0, y1;
        un2(y, y0, y1);
        const bool up = q.sg & 1;
        const float o = __shfl_xor_sync(0xffffffffu, up ? y0 : y1, 1);
        float v = (up ? y1 : y0) + o;
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if (q.sg < 2) s.y[t * ystride + q.cg * 2 + up] = v;
      }
    }
    const float* ysm = s.y - (W == 1 ? q.wt * kCh : q.warp * kPart * kCh);
    const float* rsm = s.r - (W == 1 ? q.wt * kCh : q.warp * kPart * kCh);
    // the sum over a tile's warps of y or r, at a token and channel of the block
    auto joined = [&](const float* base, int row, int c) {
      if (W == 1) return base[row * K::cw + c];
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += base[((c / kCh * W + w) * kPart + row) * kCh + c % kCh];
      return v;
    };
    if (a.z.p) {  // dz = dy y silu'(z)
      __syncthreads();
      for (int i = q.tid; i < kPart * lpr; i += blockDim.x) {
        const int row = i / lpr;
        if (!(m.live >> row & 1) || vn <= 0) continue;
        const int64_t t = tb + row;
        float x[V], z[V], g[V];
        unpack<T>(load_vec(static_cast<const T*>(a.x.p) + q.b * a.x.sb + q.h * a.x.sh + q.c0 + vc + t * a.x.st, vn, a.wide), x);
        unpack<T>(load_vec(static_cast<const T*>(a.z.p) + q.b * a.z.sb + q.h * a.z.sh + q.c0 + vc + t * a.z.st, vn, a.wide), z);
        unpack<T>(load_vec(static_cast<const T*>(ga.dy.p) + q.b * ga.dy.sb + q.h * ga.dy.sh + q.c0 + vc + t * ga.dy.st, vn, a.wide), g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float dskip = a.D && j < vn ? a.D[q.ch0 + vc + j] : 0.f;
          g[j] *= fmaf(dskip, x[j], joined(ysm, row, vc + j)) * dsilu_f(z[j]);
        }
        store_vec<T>(static_cast<T*>(ga.dz.p) + q.b * ga.dz.sb + q.h * ga.dz.sh + q.c0 + vc + t * ga.dz.st, vn, a.wide, g);
      }
      __syncthreads();
    }
    // backward, block by block
    for (int blk = (nt - 1) / kBlk; blk >= 0; --blk) {
      f2 dec[kBlk][4], st[kBlk][4];  // the decays, and the decayed states exp(D A) h_{t-1}
      f2 h[4];
      load_piece(s.keep + blk * kPiece, q.lane, h);
#pragma unroll
      for (int i = 0; i < kBlk; ++i) {
        const int t = blk * kBlk + i;
        if (t < nt) {
          if (m.begin >> t & 1) seq_state(a, q, a.h0, s_seq[t], h);
          const f2 dt = *reinterpret_cast<const f2*>(s.dt + t * K::cw + lane_o);
          const f2 u = *reinterpret_cast<const f2*>(s.u + t * K::cw + lane_o);
          f2 bb[4];
          four(s.b + t * 2 * K::states + lane_s, bb);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            dec[i][k] = ex2_pair(mul2(dt, A2[k]));
            st[i][k] = mul2(dec[i][k], h[k]);
            h[k] = fma2(u, bb[k], st[i][k]);
          }
        }
      }
      __syncwarp();  // keep[blk] is read by every lane before the block's dB, dC go there
#pragma unroll
      for (int i = kBlk - 1; i >= 0; --i) {
        const int t = blk * kBlk + i;
        if (t < nt) {
          if (m.end >> t & 1) seq_state(a, q, ga.dh_final, s_seq[t], gs);
          const f2 dt = *reinterpret_cast<const f2*>(s.dt + t * K::cw + lane_o);
          const f2 u = *reinterpret_cast<const f2*>(s.u + t * K::cw + lane_o);
          const f2 e = *reinterpret_cast<const f2*>(s.e + t * K::cw + lane_o);
          f2 bb[4], cc[4], sq = 0, sr = 0, dB[4], dC[4];
          four(s.b + t * 2 * K::states + lane_s, bb);
          four(s.c + t * 2 * K::states + lane_s, cc);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const f2 g = fma2(e, cc[k], gs[k]);
            sq = fma2(g, bb[k], sq);
            dB[k] = mul2(g, u);
            dC[k] = mul2(e, fma2(u, bb[k], st[i][k]));
            const f2 gh = mul2(g, st[i][k]);
            sr = fma2(gh, A2[k], sr);
            dA[k] = fma2(gh, dt, dA[k]);
            gs[k] = mul2(dec[i][k], g);
          }
          if ((m.begin >> t & 1) && ga.dh0) put_state(a, q, ga.dh0, s_seq[t], gs);
          // <g, B> and <g, A exp(DA) h> of two channels over the tile's four state lanes
          float v[4];
          un2(sq, v[0], v[1]);
          un2(sr, v[2], v[3]);
          const bool up = q.sg & 1, up2 = q.sg & 2;
          const float p0 = __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 1);
          const float p1 = __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 1);
          const float w0 = (up ? v[2] : v[0]) + p0, w1 = (up ? v[3] : v[1]) + p1;
          const float r0 = __shfl_xor_sync(0xffffffffu, up2 ? w0 : w1, 2);
          const float w = (up2 ? w1 : w0) + r0;
          (up ? s.r : s.y)[t * ystride + q.cg * 2 + (up2 ? 1 : 0)] = up ? w * ln2 : w;
          // dB, dC of four states over the warp's 16 channels: pairs, then 8 lanes
          float f[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float lo, hi;
            un2(dB[k], lo, hi);
            f[k] = lo + hi;
            un2(dC[k], lo, hi);
            f[4 + k] = lo + hi;
          }
          const bool b0 = q.cg & 1, b1 = q.cg & 2, b2 = q.cg & 4;
          float f4[4], f2_[2];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            f4[k] = (b0 ? f[4 + k] : f[k]) + __shfl_xor_sync(0xffffffffu, b0 ? f[k] : f[4 + k], 4);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            f2_[k] = (b1 ? f4[2 + k] : f4[k]) + __shfl_xor_sync(0xffffffffu, b1 ? f4[k] : f4[2 + k], 8);
          const float fin = (b2 ? f2_[1] : f2_[0]) + __shfl_xor_sync(0xffffffffu, b2 ? f2_[0] : f2_[1], 16);
          // dB (b0 = 0) or dC of state 4 sg + 2 b1 + b2: into the block's used-up kept states
          s.keep[blk * kPiece + i * 32 + (b0 ? 16 : 0) + q.sg * 4 + (b1 ? 2 : 0) + (b2 ? 1 : 0)] = fin;
        }
      }
    }
    __syncthreads();
    // dx, ddt, and the channels' sums
    for (int i = q.tid; i < kPart * lpr; i += blockDim.x) {
      const int row = i / lpr;
      if (!(m.live >> row & 1) || vn <= 0) continue;
      const int64_t t = tb + row;
      float x[V], raw[V], dx[V], dd[V];
      unpack<T>(load_vec(static_cast<const T*>(a.x.p) + q.b * a.x.sb + q.h * a.x.sh + q.c0 + vc + t * a.x.st, vn, a.wide), x);
      unpack<T>(load_vec(static_cast<const T*>(a.dt.p) + q.b * a.dt.sb + q.h * a.dt.sh + q.c0 + vc + t * a.dt.st, vn, a.wide), raw);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float dskip = a.D && j < vn ? a.D[q.ch0 + vc + j] : 0.f;
        const float bias = a.dt_bias && j < vn ? a.dt_bias[q.ch0 + vc + j] : 0.f;
        const int o = row * K::cw + vc + j;
        const float gb = joined(ysm, row, vc + j), ga_ = joined(rsm, row, vc + j), e = s.e[o];
        dx[j] = fmaf(dskip, e, s.dt[o] * gb);
        dd[j] = fmaf(x[j], gb, ga_);
        if (a.softplus) dd[j] *= sigmoid_f(raw[j] + bias);
        sD[j] = fmaf(e, x[j], sD[j]);
        sbias[j] += dd[j];
      }
      store_vec<T>(static_cast<T*>(ga.dx.p) + q.b * ga.dx.sb + q.h * ga.dx.sh + q.c0 + vc + t * ga.dx.st, vn, a.wide, dx);
      store_vec<T>(static_cast<T*>(ga.ddt.p) + q.b * ga.ddt.sb + q.h * ga.ddt.sh + q.c0 + vc + t * ga.ddt.st, vn, a.wide, dd);
    }
    // dB, dC over the block's channel tiles, to the block's slab
    const float* keep0 = s.keep - q.warp * (kPart / kBlk) * kPiece;
    for (int i = q.tid; i < nt * 2 * K::states; i += blockDim.x) {
      const int t = i / (2 * K::states), which = i / K::states % 2, n = i % K::states;
      float v = 0.f;
      for (int w = 0; w < K::tpb; ++w)
        v += keep0[((w * W + n / kNB) * (kPart / kBlk) + t / kBlk) * kPiece + t % kBlk * 32 + which * 16 + n % kNB];
      ws.dBC[(((int64_t)blockIdx.x * a.T + tb + t) * 2 + which) * K::states + n] = v;
    }
    __syncthreads();
  }
  store_piece(ws.dA + (chat * nw + q.warp) * kPiece, q.lane, dA);
  // the threads' channel sums: rows of threads that share a vector, in order
  for (int w = 0; w < 2; ++w) {
    float* sh = s.dt;  // [threads / lpr][cw]: within the three staged tensors
#pragma unroll
    for (int j = 0; j < V; ++j) sh[q.tid / lpr * K::cw + vc + j] = w ? sbias[j] : sD[j];
    __syncthreads();
    for (int c = q.tid; c < K::cw; c += blockDim.x) {
      float v = 0.f;
      for (int i = 0; i < (int)blockDim.x / lpr; ++i) v += sh[i * K::cw + c];
      ws.dD[(chat * 2 + w) * K::cw + c] = v;
    }
    __syncthreads();
  }
}

// Destinations of the ordered sums over batch rows and chunks. A column is an
// element of the block's layout for one (head, channel block).
struct PutA {
  float* dA;
  int d, N;
  Grid g;
  __device__ void operator()(int64_t col, float v) const {
    const PieceAt at = piece_at(col, g);
    const int64_t h = at.blk / g.per_head;
    const int c = (int)(at.blk % g.per_head) * g.cw() + at.cb;
    if (at.n < N && c < d) dA[(h * d + c) * N + at.n] = v;
  }
};
struct PutD {
  float *dD, *dbias;
  int d, per_head, cw;
  __device__ void operator()(int64_t col, float v) const {
    const int c = (int)(col % cw), which = (int)(col / cw % 2);
    const int64_t blk = col / cw / 2, h = blk / per_head;
    const int ch = (int)(blk % per_head) * cw + c;
    float* p = which ? dbias : dD;
    if (p && ch < d) p[h * d + ch] = v;
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
  const int nw = p.tpb * p.warps, cw = p.tpb * kCh;
  const int64_t heads = (int64_t)a.H * p.per_head;  // channel blocks of a batch row
  if (a.T > 0) {
    e = for_warps(p.warps, [&](auto w) {
      constexpr int W = decltype(w)::value;
      const size_t sh = smem_bytes(p, false);
      const cudaError_t r =
          cudaFuncSetAttribute(main_kernel<T, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sh);
      if (r != cudaSuccess) return r;
      const dim3 grid((unsigned)p.blocks, p.chunks);
      pre_kernel<T, W><<<grid, 32 * nw, smem_bytes(p, true), s>>>(ga, p, ws);
      const int64_t n = p.blocks * nw * kPiece;
      join_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, p, ws);
      main_kernel<T, W><<<grid, 32 * nw, sh, s>>>(ga, p, ws);
      const int64_t bc = (int64_t)a.B * a.G * a.T * 2 * p.warps * kNB;
      put_bc_kernel<T><<<(unsigned)((bc + 255) / 256), 256, 0, s>>>(ga, p, ws.dBC);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
  }
  // [chunk][batch row][head block]: parts are (chunk, batch row) pairs
  const int64_t parts = (int64_t)p.chunks * a.B;
  e = sum_parts(ws.dA, parts, heads * nw * kPiece, PutA{ga.dA, a.d, a.N, p}, s);
  if (e != cudaSuccess || (!ga.dD && !ga.ddt_bias)) return e;
  return sum_parts(ws.dD, parts, heads * 2 * cw, PutD{ga.dD, ga.ddt_bias, a.d, p.per_head, cw}, s);
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
