// Selective scan, forward for prompts and single tokens (selective_scan_fwd,
// selective_scan_step of include/ttt.h).
//
// A warp holds 16 states of 32 channels: a lane has 4 states of 4 channels,
// so the sum over states takes three shuffles a token and the inputs of a
// token are four 16-byte reads of shared memory. N > 16 gives a channel tile
// a warp per 16 states, which add their parts of y through shared memory.
// The tokens of a tile (16) are staged once: softplus, the products D_t x_t
// and the gate are computed once per element, from 16-byte loads.
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

constexpr int kCh = 32;    // channels a tile
constexpr int kTile = 16;  // tokens staged at once

// A warp's piece of the joined states: 512 floats, 16 a lane, as four float4
// (state 4*(lane&3) + k, channels 4*(lane>>2) .. +3).
constexpr int kPiece = kNB * kCh;

struct Plan {
  int warps;      // 16-state warps a channel tile
  int64_t tiles;  // channel tiles of the call (batch rows, heads)
  int chunks, len;
};
Plan plan(const ScanArgs& a) {
  Plan p;
  p.warps = (a.N + kNB - 1) / kNB;
  p.tiles = (int64_t)a.B * a.H * ((a.d + kCh - 1) / kCh);
  const int64_t have = p.tiles * p.warps, want = 148 * 16;
  int64_t c = (want + have - 1) / have;
  const int64_t most = (a.T + 63) / 64;
  c = c < most ? c : most;
  c = c < 1 ? 1 : c;
  p.len = (int)(((a.T + c - 1) / c + kTile - 1) / kTile * kTile);
  if (p.len < kTile) p.len = kTile;
  p.chunks = a.T > 0 ? (a.T + p.len - 1) / p.len : 0;
  return p;
}

// kPre: the first pass over a chunk (its end state and sum of D_t); otherwise
// the outputs.
template <typename T, bool kPre>
__global__ void __launch_bounds__(128)
    scan_kernel(ScanArgs a, int len, int64_t tiles, float* states, float* sums, int* cuts) {
  constexpr int V = Vec<T>::n, LPR = kCh / V, MAXV = kTile * LPR / 32;
  extern __shared__ __align__(16) float sm[];
  __shared__ int s_seq[kTile];
  const int tid = threadIdx.x, lane = tid & 31, wb = tid >> 5, nw = blockDim.x >> 5;
  const int sg = lane & 3, cg = lane >> 2;
  float* s_dt = sm;
  float* s_u = s_dt + kTile * kCh;
  float* s_b = s_u + kTile * kCh + wb * 2 * kTile * 2 * kNB;  // each value twice
  float* s_c = s_b + kTile * 2 * kNB;
  // one warp: y takes the place of u, token by token
  float* s_y0 = nw == 1 ? s_u : s_u + kTile * kCh + nw * 2 * kTile * 2 * kNB;
  float* s_y = s_y0 + wb * kTile * kCh;

  const int cts = (a.d + kCh - 1) / kCh;
  const int64_t tile = blockIdx.x;
  const int ct = (int)(tile % cts), h = (int)(tile / cts % a.H), b = (int)(tile / cts / a.H);
  const int c0 = ct * kCh, g = h / (a.H / a.G);
  const int chunk = blockIdx.y, t0 = chunk * len, t1 = min(a.T, t0 + len);

  // decay rates of the lane's states and channels, in powers of two
  f2 A2[4][2], hs[4][2];
  const int64_t ch0 = (int64_t)h * a.d + c0;
  {
    float r[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = wb * kNB + sg * 4 + k, cc = cg * 4 + c;
        r[k][c] = n < a.N && c0 + cc < a.d ? a.A[(ch0 + cc) * a.N + n] * kLog2e : 0.f;
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        A2[k][p] = mk2(r[k][2 * p], r[k][2 * p + 1]);
        hs[k][p] = 0;
      }
  }
  const int64_t piece = ((int64_t)chunk * tiles + tile) * nw + wb;
  if (!kPre && chunk > 0) {
    const float4* in = reinterpret_cast<const float4*>(states + piece * kPiece);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = in[k * 32 + lane];
      hs[k][0] = mk2(v.x, v.y);
      hs[k][1] = mk2(v.z, v.w);
    }
  }

  // the channels a thread stages and writes: vc .. vc+V-1 of every row it has
  const int vc = tid % LPR * V, vn = a.d - c0 - vc;
  float bias[V], dskip[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    bias[j] = a.dt_bias && j < vn ? a.dt_bias[ch0 + vc + j] : 0.f;
    dskip[j] = !kPre && a.D && j < vn ? a.D[ch0 + vc + j] : 0.f;
  }
  const T* xp = static_cast<const T*>(a.x.p) + b * a.x.sb + h * a.x.sh + c0 + vc;
  const T* dp = static_cast<const T*>(a.dt.p) + b * a.dt.sb + h * a.dt.sh + c0 + vc;
  const T* zp = a.z.p ? static_cast<const T*>(a.z.p) + b * a.z.sb + h * a.z.sh + c0 + vc : nullptr;
  const int bt = lane >> 1, bn = (lane & 1) * 8;  // token and first state a lane stages of B and C
  const int bleft = a.N - wb * kNB - bn;
  const T* bp = static_cast<const T*>(a.Bm.p) + b * a.Bm.sb + g * a.Bm.sh + wb * kNB + bn;
  const T* cp = static_cast<const T*>(a.Cm.p) + b * a.Cm.sb + g * a.Cm.sh + wb * kNB + bn;
  T* op = kPre ? nullptr : static_cast<T*>(a.out.p) + b * a.out.sb + h * a.out.sh + c0 + vc;

  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  bool cut = false;  // a sequence began in this chunk
  const int stride = blockDim.x / LPR;  // rows between a thread's vectors

  for (int tb = t0; tb < t1; tb += kTile) {
    const int nt = min(kTile, t1 - tb);
    // which of the tile's tokens are somebody's, begin or end a sequence
    uint32_t live, begin, end;
    if (a.seqs.cu) {
      const TokenAt at = token_at(a.seqs, b, a.T, tb + (lane & (kTile - 1)), a.status);
      const bool in = lane < nt && at.live;
      live = __ballot_sync(0xffffffffu, in);
      begin = __ballot_sync(0xffffffffu, in && tb + lane == at.lo);
      end = __ballot_sync(0xffffffffu, in && tb + lane == at.hi - 1);
      if (wb == 0 && lane < kTile) s_seq[lane] = at.seq;
    } else {
      live = (1u << nt) - 1;
      begin = tb == 0;
      end = tb + nt == a.T ? 1u << (nt - 1) : 0;
      if (tid == 0) s_seq[0] = s_seq[nt - 1] = b;
    }
    // stage the tile: D_t, D_t x_t, B and C
    Vec<T> xv[MAXV], zv[MAXV];
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
      const int row = tid / LPR + i * stride;
      if (row >= kTile) break;
      const int n = live >> row & 1 ? vn : 0;
      xv[i] = load_vec(xp + (tb + row) * a.x.st, n, a.wide);
      const Vec<T> dv = load_vec(dp + (tb + row) * a.dt.st, n, a.wide);
      if (!kPre && zp) zv[i] = load_vec(zp + (tb + row) * a.z.st, n, a.wide);
      float x[V], d[V], u[V];
      unpack<T>(xv[i], x);
      unpack<T>(dv, d);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        d[j] = j < n ? step_of(d[j] + bias[j], a.softplus) : 0.f;
        u[j] = d[j] * x[j];
      }
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        *reinterpret_cast<float4*>(s_dt + row * kCh + vc + j) = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
        *reinterpret_cast<float4*>(s_u + row * kCh + vc + j) = make_float4(u[j], u[j + 1], u[j + 2], u[j + 3]);
      }
    }
    {
      const int n = live >> bt & 1 ? bleft : 0;
#pragma unroll
      for (int m = 0; m < (kPre ? 1 : 2); ++m) {
        const T* p = m ? cp + (tb + bt) * a.Cm.st : bp + (tb + bt) * a.Bm.st;
        float* s = (m ? s_c : s_b) + bt * 2 * kNB + 2 * bn;
#pragma unroll
        for (int v = 0; v < 8; v += V) {
          float f[V];
          unpack<T>(load_vec(p + v, n - v, a.wide), f);
#pragma unroll
          for (int j = 0; j < V; j += 2)
            *reinterpret_cast<float4*>(s + 2 * (v + j)) = make_float4(f[j], f[j], f[j + 1], f[j + 1]);
        }
      }
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      if (begin >> t & 1) {
        cut = true;
        const int64_t row = (int64_t)s_seq[t] * a.H * a.d + ch0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int n = wb * kNB + sg * 4 + k, cc = cg * 4 + c;
            v[c] = a.h0 && n < a.N && c0 + cc < a.d ? a.h0[(row + cc) * a.N + n] : 0.f;
          }
          hs[k][0] = mk2(v[0], v[1]);
          hs[k][1] = mk2(v[2], v[3]);
        }
      }
      const ulonglong2 dt = *reinterpret_cast<const ulonglong2*>(s_dt + t * kCh + cg * 4);
      const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(s_u + t * kCh + cg * 4);
      f2 bb[4], y[2] = {0, 0};
      {
        const ulonglong2 v0 = *reinterpret_cast<const ulonglong2*>(s_b + t * 2 * kNB + sg * 8);
        const ulonglong2 v1 = *reinterpret_cast<const ulonglong2*>(s_b + t * 2 * kNB + sg * 8 + 4);
        bb[0] = v0.x, bb[1] = v0.y, bb[2] = v1.x, bb[3] = v1.y;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        hs[k][0] = fma2(ex2_pair(mul2(dt.x, A2[k][0])), hs[k][0], mul2(u.x, bb[k]));
        hs[k][1] = fma2(ex2_pair(mul2(dt.y, A2[k][1])), hs[k][1], mul2(u.y, bb[k]));
      }
      if (kPre) {
        float d0, d1, d2, d3;
        un2(dt.x, d0, d1);
        un2(dt.y, d2, d3);
        sum[0] += d0, sum[1] += d1, sum[2] += d2, sum[3] += d3;
      } else {
        const ulonglong2 v0 = *reinterpret_cast<const ulonglong2*>(s_c + t * 2 * kNB + sg * 8);
        const ulonglong2 v1 = *reinterpret_cast<const ulonglong2*>(s_c + t * 2 * kNB + sg * 8 + 4);
        const f2 cc[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[0] = fma2(hs[k][0], cc[k], y[0]);
          y[1] = fma2(hs[k][1], cc[k], y[1]);
        }
        // four channels over four lanes: halve twice, a channel a lane is left
        float y0, y1, y2, y3;
        un2(y[0], y0, y1);
        un2(y[1], y2, y3);
        const bool up = sg & 1;
        const float p0 = __shfl_xor_sync(0xffffffffu, up ? y0 : y2, 1);
        const float p1 = __shfl_xor_sync(0xffffffffu, up ? y1 : y3, 1);
        const float q0 = (up ? y2 : y0) + p0, q1 = (up ? y3 : y1) + p1;
        const bool up2 = sg & 2;
        const float r = __shfl_xor_sync(0xffffffffu, up2 ? q0 : q1, 2);
        s_y[t * kCh + cg * 4 + (up ? 2 : 0) + (up2 ? 1 : 0)] = (up2 ? q1 : q0) + r;
        if ((end >> t & 1) && a.h_final) {
          const int64_t row = (int64_t)s_seq[t] * a.H * a.d + ch0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float v[4];
            un2(hs[k][0], v[0], v[1]);
            un2(hs[k][1], v[2], v[3]);
            const int n = wb * kNB + sg * 4 + k;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (n < a.N && c0 + cg * 4 + c < a.d) a.h_final[(row + cg * 4 + c) * a.N + n] = v[c];
          }
        }
      }
    }
    __syncthreads();
    if (!kPre) {
#pragma unroll
      for (int i = 0; i < MAXV; ++i) {
        const int row = tid / LPR + i * stride;
        if (row >= kTile) break;
        if (!(live >> row & 1)) continue;
        float x[V], z[V], y[V];
        unpack<T>(xv[i], x);
        if (zp) unpack<T>(zv[i], z);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float v = s_y0[row * kCh + vc + j];
          for (int w = 1; w < nw; ++w) v += s_y0[(w * kTile + row) * kCh + vc + j];
          v = fmaf(dskip[j], x[j], v);
          y[j] = zp ? v * silu_f(z[j]) : v;
        }
        store_vec<T>(op + (tb + row) * a.out.st, vn, a.wide, y);
      }
      __syncthreads();
    }
  }
  if (kPre) {
    float4* o = reinterpret_cast<float4*>(states + piece * kPiece);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float4 v;
      un2(hs[k][0], v.x, v.y);
      un2(hs[k][1], v.z, v.w);
      o[k * 32 + lane] = v;
    }
    if (wb == 0 && sg == 0)
      *reinterpret_cast<float4*>(sums + ((int64_t)chunk * tiles + tile) * kCh + cg * 4) =
          make_float4(sum[0], sum[1], sum[2], sum[3]);
    if (tile == 0 && tid == 0) cuts[chunk] = cut;
  }
}

// states[c] (a chunk's end from zero) -> the state before chunk c: an element
// a thread, over the chunks in order.
__global__ void join_kernel(ScanArgs a, int chunks, int64_t tiles, int nw, float* states,
                            const float* sums, const int* cuts) {
  const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t per = tiles * nw * kPiece;
  if (e >= per) return;
  const int in = (int)(e % kPiece), k = in / 128, lane = in % 128 / 4, c = (lane >> 2) * 4 + in % 4;
  const int64_t w = e / kPiece, tile = w / nw;
  const int n = (int)(w % nw) * kNB + (lane & 3) * 4 + k;
  const int cts = (a.d + kCh - 1) / kCh;
  const int ch = (int)(tile % cts) * kCh + c, h = (int)(tile / cts % a.H);
  const bool in_range = n < a.N && ch < a.d;
  const float A2 = in_range ? a.A[((int64_t)h * a.d + ch) * a.N + n] * kLog2e : 0.f;
  float carry = 0.f;
#pragma unroll 4
  for (int i = 0; i < chunks; ++i) {
    float* p = states + i * per + e;
    const float local = i + 1 < chunks ? *p : 0.f;
    const float dec = i + 1 < chunks ? ex2(A2 * sums[(i * tiles + tile) * kCh + c]) : 0.f;
    *p = carry;
    carry = (i + 1 < chunks && cuts[i]) ? local : fmaf(dec, carry, local);
  }
}

size_t smem_bytes(int nw, bool pre) {
  return (size_t)(2 * kTile * kCh + nw * 2 * kTile * 2 * kNB + (nw > 1 && !pre ? nw * kTile * kCh : 0)) *
         sizeof(float);
}

template <typename T>
cudaError_t fwd(const ScanArgs& a, cudaStream_t s) {
  const Plan p = plan(a);
  cudaError_t e = copy_empty_states(a.seqs, a.T, (int64_t)a.H * a.d * a.N, a.h0, a.h_final, a.status, s);
  if (e != cudaSuccess || a.T == 0) return e;
  float* states = a.ws;
  float* sums = states + (int64_t)p.chunks * p.tiles * p.warps * kPiece;
  int* cuts = reinterpret_cast<int*>(sums + (int64_t)p.chunks * p.tiles * kCh);
  if (p.chunks > 1) {
    scan_kernel<T, true><<<dim3((unsigned)p.tiles, p.chunks - 1), 32 * p.warps, smem_bytes(p.warps, true), s>>>(
        a, p.len, p.tiles, states, sums, cuts);
    const int64_t n = p.tiles * p.warps * kPiece;
    join_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, p.chunks, p.tiles, p.warps, states, sums, cuts);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const size_t sh = smem_bytes(p.warps, false);
  scan_kernel<T, false><<<dim3((unsigned)p.tiles, p.chunks), 32 * p.warps, sh, s>>>(a, p.len, p.tiles, states,
                                                                                   sums, cuts);
  return cudaGetLastError();
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
  return (size_t)p.chunks * (p.tiles * (p.warps * scan::kPiece + scan::kCh) + 1) * sizeof(float);
}
cudaError_t launch_selective_scan_fwd(const ScanArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? scan::fwd<__nv_bfloat16>(a, s) : scan::fwd<float>(a, s);
}
cudaError_t launch_selective_scan_step(const ScanStepArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? scan::step<__nv_bfloat16>(a, s) : scan::step<float>(a, s);
}

}  // namespace ttt
