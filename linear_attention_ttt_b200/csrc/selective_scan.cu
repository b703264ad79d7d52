// Selective scan, forward for prompts and single tokens (selective_scan_fwd,
// selective_scan_step of include/ttt.h).
//
// A warp holds 16 states of 16 channels: a lane has 4 states of 2 channels, so
// the sum over states takes two shuffles a token and the inputs of a token are
// a few wide reads of shared memory. N > 16 gives a channel tile a warp per 16
// states, which add their parts of y through shared memory. The tokens of a
// part (32) are staged once: softplus, the products D_t x_t and the gate are
// computed once per element, from 16-byte loads.
//
// What bounds it: one exponential and four fp32 operations per (channel,
// state, token). The special-function unit gives 16 exponentials a clock and
// SM, which at N = 16 takes three times as long as the memory traffic does.
//
// Where B x channels give too few warps, the tokens are split into chunks: a
// first pass computes each chunk's end state from a zero start and its sum of
// D_t, a small kernel joins the chunks (the decay over a chunk is
// exp(A sum D_t)), and the main pass starts every chunk from its true state.
#include "scan.cuh"

namespace ttt {
namespace scan {
namespace {

struct Plan : Grid {
  int chunks, len;  // len: tokens, a multiple of kPart
};
Plan plan(const ScanArgs& a) {
  Plan p;
  static_cast<Grid&>(p) = grid_of(a);
  const int64_t have = p.blocks * p.wpb(), want = 148 * 16;
  int64_t c = (want + have - 1) / have;
  const int64_t most = (a.T + 63) / 64;
  c = c < most ? c : most;
  c = c < 1 ? 1 : c;
  p.len = (int)(((a.T + c - 1) / c + kPart - 1) / kPart * kPart);
  if (p.len < kPart) p.len = kPart;
  p.chunks = a.T > 0 ? (a.T + p.len - 1) / p.len : 0;
  return p;
}

// Shared memory: D_t, D_t x_t [token][channel], B, C [token][state] (each value
// twice), and y of the block's warps where a tile has several.
size_t smem_bytes(const Grid& g, bool pre) {
  const int states = g.warps * kNB;
  return (size_t)kPart * (2 * g.cw() + (pre ? 2 : 4) * states + (g.warps > 1 && !pre ? g.wpb() * kCh : 0)) *
         sizeof(float);
}

// kPre: the first pass over a chunk (its end state and sum of D_t); otherwise
// the outputs. A part's rows are loaded while the part before is scanned.
template <typename T, int W, bool kPre>
__global__ void __launch_bounds__(128, sizeof(T) == 2 ? 4 : 3)
    scan_kernel(ScanArgs a, Plan p, float* states, float* sums, int* cuts) {
  constexpr int V = Vec<T>::n, tpb = tiles_per_block(W), wpb = W * tpb;
  constexpr int cw = tpb * kCh, ns = W * kNB, lpr = cw / V, spr = ns / V;
  constexpr int dr = 32 * wpb / lpr, bdr = 32 * wpb / spr;  // rows between a thread's vectors
  constexpr int kRows = (kPart + dr - 1) / dr, kBC = (kPart + bdr - 1) / bdr;
  extern __shared__ __align__(16) float sm[];
  __shared__ int s_seq[kPart];
  const Place q = place<W>(a, p.per_head);
  const int chunk = blockIdx.y;
  float* s_dt = sm;
  float* s_u = s_dt + kPart * cw;
  float* s_b = s_u + kPart * cw;
  float* s_c = s_b + kPart * 2 * ns;
  // one warp a tile: y takes the place of u, token by token
  constexpr int ys = W == 1 ? cw : kCh;
  float* s_y = W == 1 ? s_u + q.wt * kCh : s_c + kPart * 2 * ns + q.warp * kPart * kCh;
  const int t0 = chunk * p.len, t1 = min(a.T, t0 + p.len);

  f2 A2[4], hs[4] = {0, 0, 0, 0}, sum = 0;
  rates(a, q, A2);
  const int64_t piece = ((int64_t)chunk * p.blocks + blockIdx.x) * wpb + q.warp;
  if (!kPre && chunk > 0) load4(states + piece * kPiece, q.lane, hs);

  // what the thread stages: channels vc .. of rows row0, row0 + dr, ..; states
  // n0 .. of B's and C's rows
  const int vc = q.tid % lpr * V, vn = a.d - q.c0 - vc, row0 = q.tid / lpr;
  const int n0 = q.tid % spr * V, nn = a.N - n0, brow0 = q.tid / spr;
  const T* xp = static_cast<const T*>(a.x.p) + q.b * a.x.sb + q.h * a.x.sh + q.c0 + vc;
  const T* dp = static_cast<const T*>(a.dt.p) + q.b * a.dt.sb + q.h * a.dt.sh + q.c0 + vc;
  const T* zp = !kPre && a.z.p ? static_cast<const T*>(a.z.p) + q.b * a.z.sb + q.h * a.z.sh + q.c0 + vc : nullptr;
  const T* bp = static_cast<const T*>(a.Bm.p) + q.b * a.Bm.sb + q.g * a.Bm.sh + n0;
  const T* cp = static_cast<const T*>(a.Cm.p) + q.b * a.Cm.sb + q.g * a.Cm.sh + n0;

  Vec<T> xv[kRows], dv[kRows], zv[kRows], bv[kBC], cv[kBC];
  Marks m;
  int seq;
  auto fetch = [&](int tb) {
    m = marks(a, q, tb, min(kPart, t1 - tb), &seq);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = row0 + i * dr;
      const int n = row < kPart && m.live >> row & 1 ? vn : 0;
      const int64_t t = tb + row;
      xv[i] = load_vec(xp + t * a.x.st, n, a.wide);
      dv[i] = load_vec(dp + t * a.dt.st, n, a.wide);
      if (zp) zv[i] = load_vec(zp + t * a.z.st, n, a.wide);
    }
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int row = brow0 + i * bdr;
      const int n = row < kPart && m.live >> row & 1 ? nn : 0;
      bv[i] = load_vec(bp + (int64_t)(tb + row) * a.Bm.st, n, a.wide);
      if (!kPre) cv[i] = load_vec(cp + (int64_t)(tb + row) * a.Cm.st, n, a.wide);
    }
  };
  const int lane_c = q.wt * kCh + q.cg * 2, lane_s = q.wn * 2 * kNB + q.sg * 8;
  bool cut = false;  // a sequence began in this chunk

  fetch(t0);
  for (int tb = t0; tb < t1; tb += kPart) {
    const int nt = min(kPart, t1 - tb);
    const Marks now = m;
    // stage the part
    Vec<T> xk[kRows], zk[kRows];  // for the outputs
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = row0 + i * dr;
      if (row >= kPart) break;
      float x[V], d[V], u[V];
      unpack<T>(xv[i], x);
      unpack<T>(dv[i], d);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float bias = a.dt_bias && j < vn ? a.dt_bias[q.ch0 + vc + j] : 0.f;
        d[j] = step_of(d[j] + bias, a.softplus);
        u[j] = d[j] * x[j];
      }
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        *reinterpret_cast<float4*>(s_dt + row * cw + vc + j) = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
        *reinterpret_cast<float4*>(s_u + row * cw + vc + j) = make_float4(u[j], u[j + 1], u[j + 2], u[j + 3]);
      }
      xk[i] = xv[i];
      if (zp) zk[i] = zv[i];
    }
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int row = brow0 + i * bdr;
      if (row >= kPart) break;
#pragma unroll
      for (int w = 0; w < (kPre ? 1 : 2); ++w) {
        float f[V];
        unpack<T>(w ? cv[i] : bv[i], f);
        float* s = (w ? s_c : s_b) + 2 * (row * ns + n0);
#pragma unroll
        for (int j = 0; j < V; j += 2) *reinterpret_cast<float4*>(s + 2 * j) = make_float4(f[j], f[j], f[j + 1], f[j + 1]);
      }
    }
    if (q.warp == 0) s_seq[q.lane] = seq;
    __syncthreads();
    if (tb + kPart < t1) fetch(tb + kPart);

    auto token = [&](int t, bool events) {
      if (events && (now.begin >> t & 1)) {
        cut = true;
        seq_state(a, q, a.h0, s_seq[t], hs);
      }
      const f2 dt = *reinterpret_cast<const f2*>(s_dt + t * cw + lane_c);
      const f2 u = *reinterpret_cast<const f2*>(s_u + t * cw + lane_c);
      f2 bb[4];
      four(s_b + t * 2 * ns + lane_s, bb);
#pragma unroll
      for (int k = 0; k < 4; ++k) hs[k] = fma2(ex2_pair(mul2(dt, A2[k])), hs[k], mul2(u, bb[k]));
      if (kPre) {
        sum = add2(sum, dt);
      } else {
        f2 cc[4];
        four(s_c + t * 2 * ns + lane_s, cc);
        f2 y = mul2(hs[0], cc[0]);
#pragma unroll
        for (int k = 1; k < 4; ++k) y = fma2(hs[k], cc[k], y);
        // two channels over four lanes
        float y0, y1;
        un2(y, y0, y1);
        const bool up = q.sg & 1;
        float v = (up ? y1 : y0) + __shfl_xor_sync(0xffffffffu, up ? y0 : y1, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if (q.sg < 2) s_y[t * ys + q.cg * 2 + up] = v;
        if (events && (now.end >> t & 1) && a.h_final) put_state(a, q, a.h_final, s_seq[t], hs);
      }
    };
    if (nt == kPart && !(now.begin | now.end)) {
#pragma unroll 4
      for (int t = 0; t < kPart; ++t) token(t, false);
    } else {
      for (int t = 0; t < nt; ++t) token(t, true);
    }
    __syncthreads();
    if (!kPre) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int row = row0 + i * dr;
        if (row >= kPart) break;
        if (!(now.live >> row & 1)) continue;
        float x[V], z[V], y[V];
        unpack<T>(xk[i], x);
        if (zp) unpack<T>(zk[i], z);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float v;
          if (W == 1) {
            v = s_u[row * cw + vc + j];
          } else {
            const float* base = s_c + kPart * 2 * ns + ((vc + j) / kCh * W * kPart + row) * kCh + (vc + j) % kCh;
            v = base[0];
#pragma unroll
            for (int w = 1; w < W; ++w) v += base[w * kPart * kCh];
          }
          const float dskip = a.D && j < vn ? a.D[q.ch0 + vc + j] : 0.f;
          v = fmaf(dskip, x[j], v);
          y[j] = zp ? v * silu_f(z[j]) : v;
        }
        store_vec<T>(static_cast<T*>(a.out.p) + q.b * a.out.sb + q.h * a.out.sh + q.c0 + vc + (int64_t)(tb + row) * a.out.st,
                     vn, a.wide, y);
      }
      __syncthreads();
    }
  }
  if (kPre) {
    store4(states + piece * kPiece, q.lane, hs);
    if (q.wn == 0 && q.sg == 0)
      *reinterpret_cast<f2*>(sums + ((int64_t)chunk * p.blocks + blockIdx.x) * cw + lane_c) = sum;
    if (blockIdx.x == 0 && q.tid == 0) cuts[chunk] = cut;
  }
}

// states[c] (a chunk's end from zero) -> the state before chunk c: an element
// a thread, over the chunks in order, eight loads ahead.
constexpr int kAhead = 8;
__global__ void join_kernel(ScanArgs a, Plan p, float* states, const float* __restrict__ sums,
                            const int* __restrict__ cuts) {
  const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t per = p.blocks * p.wpb() * kPiece, row = p.blocks * p.cw();
  if (e >= per) return;
  const PieceAt at = piece_at(e, p);
  const int c = (int)(at.blk % p.per_head) * p.cw() + at.cb, h = (int)(at.blk / p.per_head % a.H);
  const float A2 = at.n < a.N && c < a.d ? a.A[((int64_t)h * a.d + c) * a.N + at.n] * kLog2e : 0.f;
  const float* sum = sums + at.blk * p.cw() + at.cb;
  float carry = 0.f;
  for (int i0 = 0; i0 < p.chunks; i0 += kAhead) {
    float local[kAhead], dec[kAhead];
    bool cut[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const bool in = i0 + j + 1 < p.chunks;  // the last chunk passes nothing on
      local[j] = in ? states[(i0 + j) * per + e] : 0.f;
      dec[j] = in ? ex2(A2 * sum[(i0 + j) * row]) : 0.f;
      cut[j] = in && cuts[i0 + j];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j >= p.chunks) break;
      states[(i0 + j) * per + e] = carry;
      carry = cut[j] ? local[j] : fmaf(dec[j], carry, local[j]);
    }
  }
}

template <typename T>
cudaError_t fwd(const ScanArgs& a, cudaStream_t s) {
  const Plan p = plan(a);
  cudaError_t e = copy_empty_states(a.seqs, a.T, (int64_t)a.H * a.d * a.N, a.h0, a.h_final, a.status, s);
  if (e != cudaSuccess || a.T == 0) return e;
  float* states = a.ws;
  float* sums = states + (int64_t)p.chunks * p.blocks * p.wpb() * kPiece;
  int* cuts = reinterpret_cast<int*>(sums + (int64_t)p.chunks * p.blocks * p.cw());
  const int threads = 32 * p.wpb();
  return for_warps(p.warps, [&](auto w) {
    constexpr int W = decltype(w)::value;
    const dim3 first((unsigned)p.blocks, p.chunks - 1), all((unsigned)p.blocks, p.chunks);
    if (p.chunks > 1) {
      scan_kernel<T, W, true><<<first, threads, smem_bytes(p, true), s>>>(a, p, states, sums, cuts);
      const int64_t n = p.blocks * p.wpb() * kPiece;
      join_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, p, states, sums, cuts);
    }
    scan_kernel<T, W, false><<<all, threads, smem_bytes(p, false), s>>>(a, p, states, sums, cuts);
    return cudaGetLastError();
  });
}

__global__ void copy_empty_kernel(Seqs q, int T, int64_t n, const float* src, float* dst, int* status) {
  int lo = 0, hi = T;
  if (q.cu) packed_seq(q.cu, blockIdx.x, T, status, &lo, &hi);
  if (hi > lo || !dst) return;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
    dst[blockIdx.x * n + i] = src ? src[blockIdx.x * n + i] : 0.f;
}

// One token: a lane has four states of a channel, and a channel has 2^k lanes.
// Bound by memory: the states are read and written once, in 16-byte pieces.
constexpr int kStepThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kStepThreads) step_kernel(ScanStepArgs a, int lanes, int cts) {
  SlotRows rows;
  if (!rows.begin(a.slots, blockIdx.y, a.B, a.S, a.status)) return;
  const int per = kStepThreads / lanes, n0 = threadIdx.x % lanes * 4;
  const int h = blockIdx.x / cts, c = blockIdx.x % cts * per + threadIdx.x / lanes;
  const bool live = c < a.d;
  const int64_t ch = (int64_t)h * a.d + (live ? c : 0);
  const int left = live ? a.N - n0 : 0;
  const bool whole = a.wide && left >= 4 && a.N % 4 == 0;
  float A[4], s[4];
  float* sp = a.state + ((int64_t)rows.slot * a.H * a.d + ch) * a.N + n0;
  const float* ap = a.A + ch * a.N + n0;
  if (whole) {
    const float4 v = *reinterpret_cast<const float4*>(sp), w = *reinterpret_cast<const float4*>(ap);
    s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
    A[0] = w.x, A[1] = w.y, A[2] = w.z, A[3] = w.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s[k] = k < left ? sp[k] : 0.f;
      A[k] = k < left ? ap[k] : 0.f;
    }
  }
  const float bias = a.dt_bias && live ? a.dt_bias[ch] : 0.f;
  const float dskip = a.D && live ? a.D[ch] : 0.f;
  const int g = h / (a.H / a.G);
  do {
    float x = 0.f, raw = 0.f, z = 0.f, y = 0.f;
    if (live) {
      x = to_f32(static_cast<const T*>(a.x.p)[rows.b * a.x.sb + h * a.x.sh + c]);
      raw = to_f32(static_cast<const T*>(a.dt.p)[rows.b * a.dt.sb + h * a.dt.sh + c]);
      if (a.z.p) z = to_f32(static_cast<const T*>(a.z.p)[rows.b * a.z.sb + h * a.z.sh + c]);
    }
    const T* bp = static_cast<const T*>(a.Bm.p) + rows.b * a.Bm.sb + g * a.Bm.sh + n0;
    const T* cp = static_cast<const T*>(a.Cm.p) + rows.b * a.Cm.sb + g * a.Cm.sh + n0;
    const float dt = step_of(raw + bias, a.softplus);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= left) break;
      s[k] = fmaf(ex2(dt * (A[k] * kLog2e)), s[k], dt * x * to_f32(bp[k]));
      y = fmaf(s[k], to_f32(cp[k]), y);
    }
    for (int o = lanes / 2; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (live && n0 == 0) {
      y = fmaf(dskip, x, y);
      if (a.z.p) y *= silu_f(z);
      static_cast<T*>(a.out.p)[rows.b * a.out.sb + h * a.out.sh + c] = from_f32<T>(y);
    }
  } while (rows.next_row());
  if (whole) {
    *reinterpret_cast<float4*>(sp) = make_float4(s[0], s[1], s[2], s[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) sp[k] = s[k];
  }
}

template <typename T>
cudaError_t step(const ScanStepArgs& a, cudaStream_t s) {
  int lanes = 1;
  while (lanes * 4 < a.N) lanes *= 2;
  const int per = kStepThreads / lanes, cts = (a.d + per - 1) / per;
  step_kernel<T><<<dim3((unsigned)(a.H * cts), a.B), kStepThreads, 0, s>>>(a, lanes, cts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t copy_empty_states(const Seqs& q, int T, int64_t n, const float* src, float* dst, int* status,
                              cudaStream_t s) {
  if (!q.cu && (T > 0 || !dst)) return cudaSuccess;
  copy_empty_kernel<<<q.S, 256, 0, s>>>(q, T, n, src, dst, status);
  return cudaGetLastError();
}

}  // namespace scan

size_t selective_scan_workspace(const ScanArgs& a) {
  const scan::Plan p = scan::plan(a);
  if (p.chunks <= 1) return 0;
  return (size_t)p.chunks * (p.blocks * (p.wpb() * scan::kPiece + p.cw()) + 1) * sizeof(float);
}
cudaError_t launch_selective_scan_fwd(const ScanArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? scan::fwd<__nv_bfloat16>(a, s) : scan::fwd<float>(a, s);
}
cudaError_t launch_selective_scan_step(const ScanStepArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? scan::step<__nv_bfloat16>(a, s) : scan::step<float>(a, s);
}

}  // namespace ttt
