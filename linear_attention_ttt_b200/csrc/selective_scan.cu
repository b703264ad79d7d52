// Selective scan, forward for prompts and single tokens (selective_scan_fwd,
// selective_scan_step of include/ttt.h).
//
// A warp holds 16 states of 16 channels: a lane has 4 states of 2 channels, so
// the sums over states cross four lanes only, and the inputs of a token are a
// few wide reads of shared memory. N > 16 gives a channel tile a warp per 16
// states, which add their parts of y through shared memory. The tokens of a
// part (32) are staged once: softplus, the products D_t x_t and the gate are
// computed once per element, from 16-byte loads.
//
// What bounds it: one exponential and four fp32 operations per (channel,
// state, token), and four special functions per element beside them. The
// special-function unit gives 16 a clock and SM: at N = 16 that is 3.5 times the
// memory traffic's time. B16 T1024 d4096 takes 483 us, 290 of them the unit's own
// (60 % busy); B4 T4096 d4096, with two warps a scheduler and nothing to hide
// their latencies behind, 648 (50 %).
//
// The raw rows of a part arrive by asynchronous copies while the part before is
// scanned; a token's decays are computed while the token before is; the sums
// over states leave four tokens at a time. Whole pieces have paths of their
// own: loads behind a choice wait for one another.
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
// Chunks cost a second pass, which only idle SMs pay for. Measured at N = 16,
// bf16, gated: from 1024 warps on one chunk wins (B4 T4096 d4096: 648 us in one
// chunk, 759 in 4, 775 in 16; B16 T1024 d4096: 483, 733, 844), with 256 and fewer
// about 4096 warps in all do (B1 T4096 d4096: 475 us in one, 217 in 16, 221 in 32;
// B1 T16384 d2048: 1861 in one, 472 in 16, 416 in 32). Chunks below 64 tokens gain
// nothing.
Plan plan(const ScanArgs& a) {
  Plan p;
  static_cast<Grid&>(p) = grid_of(a);
  const int64_t warps = p.blocks * p.wpb(), most = (a.T + 63) / 64;
  int64_t c = warps >= 640 || warps == 0 ? 1 : 4096 / warps;
  c = c < most ? c : most;
  c = c < 1 ? 1 : c;
  p.len = (int)(((a.T + c - 1) / c + kPart - 1) / kPart * kPart);
  if (p.len < kPart) p.len = kPart;
  p.chunks = a.T > 0 ? (a.T + p.len - 1) / p.len : 0;
  return p;
}

// Shared memory of a block. The raw rows of the next part arrive while the
// present one is scanned: x, dt, B and C are used up when a part is staged, z
// when its outputs are written.
template <typename T, int W, bool kPre>
struct Shared {
  static constexpr int tpb = tiles_per_block(W), wpb = W * tpb, threads = 32 * wpb;
  static constexpr int cw = tpb * kCh, ns = W * kNB;
  float dt[kPart * cw], u[kPart * cw];            // D_t, D_t x_t [token][channel]
  float b[kPart * 2 * ns], c[kPre ? 4 : kPart * 2 * ns];  // [token][state], each value twice
  float y[kPre ? 4 : wpb * kPart * kCh];          // a warp's sums over its states [token][channel]
  T rx[kPart * cw], rdt[kPart * cw], rz[kPre ? 8 : kPart * cw];
  T rb[kPart * ns], rc[kPre ? 8 : kPart * ns];
  int seq[kPart];
};

// kPre: the first pass over a chunk (its end state and sum of D_t); otherwise
// the outputs.
template <typename T, int W, bool kPre>
__global__ void __launch_bounds__(128, sizeof(T) == 2 ? 4 : 3)
    scan_kernel(ScanArgs a, Plan p, float* states, float* sums, int* cuts) {
  using S = Shared<T, W, kPre>;
  constexpr int cw = S::cw, ns = S::ns, threads = S::threads;
  constexpr int kGroups = cw / 4, dr = threads / kGroups;  // a thread has 4 channels of every dr-th row
  extern __shared__ __align__(16) unsigned char raw[];
  S& s = *reinterpret_cast<S*>(raw);
  const Place q = place<W>(a, p.per_head);
  const int chunk = blockIdx.y, t0 = chunk * p.len, t1 = min(a.T, t0 + p.len);

  f2 A2[4], hs[4] = {0, 0, 0, 0}, sum = 0;
  rates(a, q, A2);
  const int64_t piece = ((int64_t)chunk * p.blocks + blockIdx.x) * S::wpb + q.warp;

  const int vc = q.tid % kGroups * 4, vn = a.d - q.c0 - vc, row0 = q.tid / kGroups;
  float bias[4], skip[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t c = (int64_t)q.h * a.d + min(q.c0 + vc + j, a.d - 1);
    bias[j] = a.dt_bias ? a.dt_bias[c] : 0.f;
    skip[j] = !kPre && a.D ? a.D[c] : 0.f;
  }
  const T* xp = static_cast<const T*>(a.x.p) + q.b * a.x.sb + q.h * a.x.sh + q.c0;
  const T* dp = static_cast<const T*>(a.dt.p) + q.b * a.dt.sb + q.h * a.dt.sh + q.c0;
  const T* zp = !kPre && a.z.p ? static_cast<const T*>(a.z.p) + q.b * a.z.sb + q.h * a.z.sh + q.c0 : nullptr;
  const T* bp = static_cast<const T*>(a.Bm.p) + q.b * a.Bm.sb + q.g * a.Bm.sh;
  const T* cp = static_cast<const T*>(a.Cm.p) + q.b * a.Cm.sb + q.g * a.Cm.sh;
  T* op = kPre ? nullptr : static_cast<T*>(a.out.p) + q.b * a.out.sb + q.h * a.out.sh + q.c0 + vc;

  Marks next;
  int seq;
  auto fetch = [&](int tb) {
    next = marks(a, q, tb, min(kPart, t1 - tb), &seq);
    const int64_t t = tb;
    copy_part<T, cw, threads>(s.rx, xp + t * a.x.st, a.x.st, a.d - q.c0, next.live, q.tid, a.wide);
    copy_part<T, cw, threads>(s.rdt, dp + t * a.dt.st, a.dt.st, a.d - q.c0, next.live, q.tid, a.wide);
    copy_part<T, ns, threads>(s.rb, bp + t * a.Bm.st, a.Bm.st, a.N, next.live, q.tid, a.wide);
    if (!kPre) copy_part<T, ns, threads>(s.rc, cp + t * a.Cm.st, a.Cm.st, a.N, next.live, q.tid, a.wide);
    copy_commit();
  };
  auto fetch_z = [&](int tb, uint32_t live) {
    if (zp) copy_part<T, cw, threads>(s.rz, zp + (int64_t)tb * a.z.st, a.z.st, a.d - q.c0, live, q.tid, a.wide);
    copy_commit();
  };
  const int lane_c = q.wt * kCh + q.cg * 2, lane_s = q.wn * 2 * kNB + q.sg * 8;
  float* ys = s.y + q.warp * kPart * kCh;
  bool cut = false;  // a sequence began in this chunk

  fetch(t0);
  if (!kPre) fetch_z(t0, next.live);
  // the join may be launched now, and waits; the main pass may have been launched
  // before the joined states were there
  if (kPre) pdl_trigger();
  if (!kPre && p.chunks > 1) {
    pdl_wait();
    if (chunk > 0) load_piece(states + piece * kPiece, q.lane, hs);
  }
  for (int tb = t0; tb < t1; tb += kPart) {
    const int nt = min(kPart, t1 - tb);
    const Marks now = next;
    copy_wait<kPre ? 0 : 1>();
    __syncthreads();
    // Every warp has left the part before: the first pass has no barrier at a
    // part's end, and a warp behind still reads the old sequences there.
    if (q.warp == 0) s.seq[q.lane] = seq;
    // stage the part: step sizes, inputs, and D x where y is summed up
#pragma unroll
    for (int r = 0; r < kPart; r += dr) {
      const int row = r + row0;
      if (kPart % dr != 0 && row >= kPart) break;
      float x[4], d[4];
      load_row<T, 4>(s.rx + row * cw + vc, 4, true, x);
      load_row<T, 4>(s.rdt + row * cw + vc, 4, true, d);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] += bias[j];
      if (a.softplus) {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = softplus_f(d[j]);
      }
      *reinterpret_cast<float4*>(s.dt + row * cw + vc) = make_float4(d[0], d[1], d[2], d[3]);
      *reinterpret_cast<float4*>(s.u + row * cw + vc) = make_float4(d[0] * x[0], d[1] * x[1], d[2] * x[2], d[3] * x[3]);
      if (!kPre)
        *reinterpret_cast<float4*>(s.y + (vc / kCh * W * kPart + row) * kCh + vc % kCh) =
            make_float4(skip[0] * x[0], skip[1] * x[1], skip[2] * x[2], skip[3] * x[3]);
    }
    spread_part<T, ns, threads>(s.b, s.rb, q.tid);
    if (!kPre) spread_part<T, ns, threads>(s.c, s.rc, q.tid);
    __syncthreads();
    if (tb + kPart < t1) fetch(tb + kPart);
    else if (!kPre) copy_commit();  // the groups stay in step

    // A token's decays are computed while the token before it is scanned, and
    // the sums over states leave four tokens at a time, one block later: the
    // exponentials run beside everything else.
    f2 dec[4], y[4] = {0, 0, 0, 0};
    {
      const f2 dt = *reinterpret_cast<const f2*>(s.dt + lane_c);
#pragma unroll
      for (int k = 0; k < 4; ++k) dec[k] = ex2_pair(mul2(dt, A2[k]));
      sum = add2(sum, dt);
    }
    auto sums_of = [&](int t4) {
      // over the tile's four state lanes: halve twice, a token a lane is left
      const bool up = q.sg & 1, up2 = q.sg & 2;
      const f2 v0 = add2(up ? y[2] : y[0], __shfl_xor_sync(0xffffffffu, up ? y[0] : y[2], 1));
      const f2 v1 = add2(up ? y[3] : y[1], __shfl_xor_sync(0xffffffffu, up ? y[1] : y[3], 1));
      f2 w = add2(up2 ? v1 : v0, __shfl_xor_sync(0xffffffffu, up2 ? v0 : v1, 2));
      f2* at = reinterpret_cast<f2*>(ys + (t4 + (up ? 2 : 0) + (up2 ? 1 : 0)) * kCh + q.cg * 2);
      if (W == 1 || q.wn == 0) w = add2(w, *at);
      *at = w;
    };
    auto block = [&](int t4, bool events) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t4 + i, tn = (t + 1) % kPart;
        const f2 dtn = *reinterpret_cast<const f2*>(s.dt + tn * cw + lane_c);
        const f2 u = *reinterpret_cast<const f2*>(s.u + t * cw + lane_c);
        f2 bb[4], cc[4], decn[4];
        four(s.b + t * 2 * ns + lane_s, bb);
        if (!kPre) four(s.c + t * 2 * ns + lane_s, cc);
#pragma unroll
        for (int k = 0; k < 4; ++k) decn[k] = ex2_pair(mul2(dtn, A2[k]));
        if (!kPre && i == 0 && t4 > 0) sums_of(t4 - 4);
        if (events && (now.begin >> t & 1)) {
          cut = true;
          seq_state(a, q, a.h0, s.seq[t], hs);
        }
        if (!events || t < nt) {
#pragma unroll
          for (int k = 0; k < 4; ++k) hs[k] = fma2(dec[k], hs[k], mul2(u, bb[k]));
        }
        if (kPre) {
          if (events ? t + 1 < nt : tn > 0) sum = add2(sum, dtn);
        } else {
          y[i] = mul2(hs[0], cc[0]);
#pragma unroll
          for (int k = 1; k < 4; ++k) y[i] = fma2(hs[k], cc[k], y[i]);
          if (events && (now.end >> t & 1) && a.h_final) put_state(a, q, a.h_final, s.seq[t], hs);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) dec[k] = decn[k];
      }
    };
    if (nt == kPart && !(now.begin | now.end)) {
#pragma unroll 4
      for (int t = 0; t < kPart; t += 4) block(t, false);
    } else {
#pragma unroll 1
      for (int t = 0; t < nt; t += 4) block(t, true);
    }
    if (!kPre) {
      sums_of((nt - 1) / 4 * 4);
      copy_wait<1>();
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kPart; r += dr) {
        const int row = r + row0;
        if (kPart % dr != 0 && row >= kPart) break;
        if (!(now.live >> row & 1)) continue;
        const float* base = s.y + (vc / kCh * W * kPart + row) * kCh + vc % kCh;
        float4 v = *reinterpret_cast<const float4*>(base);
#pragma unroll
        for (int w = 1; w < W; ++w) {
          const float4 o = *reinterpret_cast<const float4*>(base + w * kPart * kCh);
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        float o[4] = {v.x, v.y, v.z, v.w};
        if (zp) {
          float z[4];
          load_row<T, 4>(s.rz + row * cw + vc, 4, true, z);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] *= silu_f(z[j]);
        }
        store_row<T, 4>(op + (int64_t)(tb + row) * a.out.st, vn, a.wide, o);
      }
      __syncthreads();
      if (tb + kPart < t1) fetch_z(tb + kPart, next.live);
    }
  }
  if (kPre) {
    store_piece(states + piece * kPiece, q.lane, hs);
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
  pdl_trigger();
  pdl_wait();
  for (int i0 = 0; i0 < p.chunks; i0 += kAhead) {
    float local[kAhead], dec[kAhead];
    bool cut[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      // the last chunk passes nothing on; its place reads the one before
      const int i = min(i0 + j, p.chunks - 2);
      local[j] = states[i * per + e];
      dec[j] = ex2(A2 * sum[i * row]);
      cut[j] = cuts[i];
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
    using First = Shared<T, W, true>;
    using All = Shared<T, W, false>;
    cudaError_t r = cudaFuncSetAttribute(scan_kernel<T, W, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(First));
    if (r != cudaSuccess) return r;
    r = cudaFuncSetAttribute(scan_kernel<T, W, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(All));
    if (r != cudaSuccess) return r;
    if (p.chunks > 1) {
      scan_kernel<T, W, true><<<first, threads, sizeof(First), s>>>(a, p, states, sums, cuts);
      const int64_t n = p.blocks * p.wpb() * kPiece;
      r = cudaGetLastError();
      if (r != cudaSuccess) return r;
      r = launch_pdl(join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a, p, states, (const float*)sums, (const int*)cuts);
      if (r != cudaSuccess) return r;
      return launch_pdl(scan_kernel<T, W, false>, all, dim3(threads), sizeof(All), s, a, p, states, sums, cuts);
    }
    scan_kernel<T, W, false><<<all, threads, sizeof(All), s>>>(a, p, states, sums, cuts);
    return cudaGetLastError();
  });
}

__global__ void copy_empty_kernel(Seqs q, int T, int64_t n, const float* src, float* dst, int* status) {
  int lo = 0, hi = T;
  if (q.cu) packed_seq(q.cu, blockIdx.x, T, status, &lo, &hi);
  if (hi > lo || !dst) return;
  for (int64_t i = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.y * blockDim.x)
    dst[blockIdx.x * n + i] = src ? src[blockIdx.x * n + i] : 0.f;
}

// One token. A channel's states lie on 2^k lanes, four a lane, and a lane has
// them of four channels: places and slots are found once for 16 states. What a
// channel needs once (its step size, the gate) one of its lanes computes for
// the others. The states are read and written once, in 16-byte pieces:
// 64 sequences, d4096 N16 bf16, take 9.3 us a call (5.5 at the measured copy
// rate), waiting on their loads.
constexpr int kStepThreads = 128, kStepCh = 4;

// kWhole: N is 4 kLanes, the block's channels all exist and every row is
// aligned (see read_row).
template <typename T, int kLanes, bool kWhole>
__device__ __forceinline__ void step_rows(const ScanStepArgs& a, SlotRows& rows, int h, int first) {
  constexpr int groups = kStepThreads / kLanes;
  constexpr int kOwn = kLanes >= kStepCh ? 1 : kStepCh / kLanes;  // channels a lane computes for the others
  const int me = threadIdx.x % kLanes, n0 = me * 4, c0 = first + threadIdx.x / kLanes;
  const int64_t ch0 = (int64_t)h * a.d;
  const int left = a.N - n0, g = h / (a.H / a.G), base = threadIdx.x & 31 & ~(kLanes - 1);
  const bool whole = a.wide && a.N % 4 == 0;
  float A[kStepCh][4], s[kStepCh][4], bias[kOwn], D[kOwn];
  int own[kOwn];
  float* sp = a.state + ((int64_t)rows.slot * a.H * a.d + ch0) * a.N + n0;
#pragma unroll
  for (int i = 0; i < kStepCh; ++i) {
    const int c = c0 + i * groups, n = c < a.d ? left : 0;
    read_row<kWhole, float, 4>(sp + (int64_t)c * a.N, n, whole, s[i]);
    read_row<kWhole, float, 4>(a.A + (ch0 + c) * a.N + n0, n, whole, A[i]);
  }
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    own[j] = c0 + ((me & (kStepCh - 1)) + j * kLanes) * groups;
    bias[j] = a.dt_bias && (kWhole || own[j] < a.d) ? a.dt_bias[ch0 + own[j]] : 0.f;
    D[j] = a.D && (kWhole || own[j] < a.d) ? a.D[ch0 + own[j]] : 0.f;
  }
  do {
    const T* xp = static_cast<const T*>(a.x.p) + rows.b * a.x.sb + h * a.x.sh;
    const T* dp = static_cast<const T*>(a.dt.p) + rows.b * a.dt.sb + h * a.dt.sh;
    // without a gate the input stands in its place and is not used
    const T* zp = a.z.p ? static_cast<const T*>(a.z.p) + rows.b * a.z.sb + h * a.z.sh : xp;
    float Bv[4], Cv[4], x[kOwn], dt[kOwn], z[kOwn], y[kOwn];
    read_row<kWhole, T, 4>(static_cast<const T*>(a.Bm.p) + rows.b * a.Bm.sb + g * a.Bm.sh + n0, left, a.rows_wide, Bv);
    read_row<kWhole, T, 4>(static_cast<const T*>(a.Cm.p) + rows.b * a.Cm.sb + g * a.Cm.sh + n0, left, a.rows_wide, Cv);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const bool in = kWhole || own[j] < a.d;
      x[j] = in ? to_f32(xp[own[j]]) : 0.f;
      dt[j] = in ? to_f32(dp[own[j]]) : 0.f;
      z[j] = in ? to_f32(zp[own[j]]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kOwn; ++j) dt[j] = step_of(dt[j] + bias[j], a.softplus);
#pragma unroll
    for (int i = 0; i < kStepCh; ++i) {
      constexpr int kDiv = kLanes < kStepCh ? kLanes : kStepCh;
      const int from = base + i % kDiv, j = kOwn == 1 ? 0 : i / kLanes;
      const float d = __shfl_sync(0xffffffffu, dt[j], from);
      const float u = __shfl_sync(0xffffffffu, dt[j] * x[j], from);
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[i][k] = fmaf(ex2(d * (A[i][k] * kLog2e)), s[i][k], u * Bv[k]);
        v = fmaf(s[i][k], Cv[k], v);
      }
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (me % kDiv == i % kDiv) y[j] = v;
    }
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      y[j] = fmaf(D[j], x[j], y[j]);
      if (a.z.p) y[j] *= silu_f(z[j]);
      if ((kLanes <= kStepCh || me < kStepCh) && (kWhole || own[j] < a.d))
        static_cast<T*>(a.out.p)[rows.b * a.out.sb + h * a.out.sh + own[j]] = from_f32<T>(y[j]);
    }
  } while (rows.next_row());
#pragma unroll
  for (int i = 0; i < kStepCh; ++i) {
    const int c = c0 + i * groups;
    if (kWhole || c < a.d) write_row<kWhole, float, 4>(sp + (int64_t)c * a.N, left, whole, s[i]);
  }
}

template <typename T, int kLanes>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const __grid_constant__ ScanStepArgs a, int cts) {
  constexpr int per = kStepThreads / kLanes * kStepCh;
  SlotRows rows;
  if (!rows.begin(a.slots, blockIdx.y, a.B, a.S, a.status)) return;
  const int h = blockIdx.x / cts, first = blockIdx.x % cts * per;
  if (a.wide && a.rows_wide && a.N == 4 * kLanes && first + per <= a.d) step_rows<T, kLanes, true>(a, rows, h, first);
  else step_rows<T, kLanes, false>(a, rows, h, first);
}

template <typename T, int kLanes>
cudaError_t step_as(const ScanStepArgs& a, cudaStream_t s) {
  constexpr int per = kStepThreads / kLanes * kStepCh;
  const int cts = (a.d + per - 1) / per;
  step_kernel<T, kLanes><<<dim3((unsigned)(a.H * cts), a.B), kStepThreads, 0, s>>>(a, cts);
  return cudaGetLastError();
}
template <typename T>
cudaError_t step(const ScanStepArgs& a, cudaStream_t s) {
  if (a.N <= 4) return step_as<T, 1>(a, s);
  if (a.N <= 8) return step_as<T, 2>(a, s);
  if (a.N <= 16) return step_as<T, 4>(a, s);
  if (a.N <= 32) return step_as<T, 8>(a, s);
  return step_as<T, 16>(a, s);
}

}  // namespace

cudaError_t copy_empty_states(const Seqs& q, int T, int64_t n, const float* src, float* dst, int* status,
                              cudaStream_t s) {
  if (!q.cu && (T > 0 || !dst)) return cudaSuccess;
  // mostly there is nothing to copy: a block for 2048 values, up to 16 a sequence
  const int64_t rows = (n + 2047) / 2048;
  const dim3 g(q.S, (unsigned)(!dst || rows < 1 ? 1 : rows < 16 ? rows : 16));
  copy_empty_kernel<<<g, 256, 0, s>>>(q, T, n, src, dst, status);
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
