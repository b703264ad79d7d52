// Short causal depthwise convolution: prompts, backward, single tokens
// (causal_conv_fwd, causal_conv_bwd, causal_conv_step of include/ttt.h).
//
// A thread owns four neighbouring channels and walks a run of tokens with the
// last K inputs in registers as packed fp32 pairs, so every input is read once
// (plus K-1 rows where a run begins) in row-contiguous pieces, a batch of rows
// ahead of their use, and nothing passes through shared memory.
//
// Forward, K 4, bf16, B4 T4096 d4096: 57 us, 4.7 TB/s (41 us at the measured copy
// rate); the special-function unit, which the activation asks twice an element,
// is 59 % busy. Backward, B2: 70 us against 31 at the copy rate: 167
// registers leave 12 warps an SM, which issue in half of the slots; dp is computed
// from the window again, and K+1 sums are kept per channel.
#include "block.cuh"

namespace ttt {
namespace {

constexpr int kThreads = 128;

// Which channels and tokens a thread has.
struct Run {
  int h, c, n;    // head, first channel, channels that exist (of V)
  int b, r0, r1;  // batch row, tokens [r0, r1)
  bool live;
};
template <int V>
__device__ __forceinline__ Run run_of(int64_t i, int B, int H, int T, int d, int len) {
  const int per_head = (d + V - 1) / V, runs = (T + len - 1) / len;
  const int64_t nv = (int64_t)H * per_head;
  const int64_t row = i / nv, v = i % nv;
  Run r;
  r.h = (int)(v / per_head);
  r.c = (int)(v % per_head) * V;
  r.n = d - r.c;
  r.live = row < (int64_t)B * runs;
  r.b = (int)(row / runs);
  r.r0 = (int)(row % runs) * len;
  r.r1 = min(T, r.r0 + len);
  return r;
}

// The sequence at hand: its state's row and its tokens [lo, hi).
struct Piece {
  int seq, lo, hi;
};
// First piece of a run, and the next one; false when the run is done.
__device__ __forceinline__ bool first_piece(const Seqs& q, const Run& r, int T, int* status, Piece* p) {
  if (!q.cu) {
    *p = {r.b, 0, T};
    return true;
  }
  p->seq = first_seq_behind(q.cu, q.S, r.r0) - 1;
  p->lo = p->hi = 0;
  for (++p->seq; p->seq < q.S; ++p->seq) {
    packed_seq(q.cu, p->seq, T, status, &p->lo, &p->hi);
    if (p->lo >= r.r1) return false;
    if (p->hi > p->lo && p->hi > r.r0) return true;
  }
  return false;
}
__device__ __forceinline__ bool next_piece(const Seqs& q, const Run& r, int T, int* status, Piece* p) {
  if (!q.cu) return false;
  for (++p->seq; p->seq < q.S; ++p->seq) {
    packed_seq(q.cu, p->seq, T, status, &p->lo, &p->hi);
    if (p->lo >= r.r1) return false;
    if (p->hi > p->lo && p->hi > r.r0) return true;
  }
  return false;
}

// win[i] = the input K-1-i tokens before t (i < K-1), from the sequence or the
// state before it.
template <typename T, int K, bool kWhole>
__device__ __forceinline__ void fill_window(const T* x, int64_t st, const TokView& state0, const Run& r,
                                            const Piece& p, int t, bool wide, f2 (&win)[K][2]) {
#pragma unroll
  for (int i = 0; i < K - 1; ++i)  // tokens that are not there read the first
    pairs_of(raw_row<kWhole, T>(x + max(t - (K - 1) + i, p.lo) * st, r.n, wide), win[i]);
  if (t - (K - 1) >= p.lo) return;
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int src = t - (K - 1) + i;
    if (src >= p.lo) continue;
    float f[kV] = {0.f, 0.f, 0.f, 0.f};
    if (state0.p) {
      const T* s0 = static_cast<const T*>(state0.p) + p.seq * state0.sb + r.h * state0.sh + r.c;
      load_row<T, kV>(s0 + (int64_t)(K - 1 + src - p.lo) * state0.st, r.n, wide, f);
    }
    pairs_of(f, win[i]);
  }
}

template <int K>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, int d, const Run& r, f2 (&taps)[K][2],
                                          f2 (&b)[2]) {
  float f[kV], g[K][kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    // channels behind the row's end read its last: nothing of theirs is kept
    const int64_t c = (int64_t)r.h * d + min(r.c + j, d - 1);
    f[j] = bias ? bias[c] : 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) g[i][j] = w[c * K + i];
  }
  pairs_of(f, b);
#pragma unroll
  for (int i = 0; i < K; ++i) pairs_of(g[i], taps[i]);
}
template <int K>
__device__ __forceinline__ void shift(f2 (&win)[K][2]) {
#pragma unroll
  for (int k = 0; k < K - 1; ++k) win[k][0] = win[k + 1][0], win[k][1] = win[k + 1][1];
}
template <int K>
__device__ __forceinline__ void convolve(const f2 (&taps)[K][2], const f2 (&win)[K][2], const f2 (&bias)[2],
                                         float (&y)[kV]) {
  f2 v[2] = {bias[0], bias[1]};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[0] = fma2(taps[k][0], win[k][0], v[0]);
    v[1] = fma2(taps[k][1], win[k][1], v[1]);
  }
  floats_of(v, y);
}

// Rows a thread has in flight: while one batch is computed the next arrives.
template <typename T>
constexpr int kBatch = sizeof(T) == 2 ? 8 : 4;

template <typename T, int K, bool kWhole>
__device__ __forceinline__ void conv_run(const ConvArgs& a, const Run& r) {
  f2 taps[K][2], bias[2];
  load_taps<K>(a.w, a.bias, a.d, r, taps, bias);
  const T* x = static_cast<const T*>(a.x.p) + r.b * a.x.sb + r.h * a.x.sh + r.c;
  T* out = static_cast<T*>(a.out.p) + r.b * a.out.sb + r.h * a.out.sh + r.c;
  Piece p;
  if (!first_piece(a.seqs, r, a.T, a.status, &p)) return;
  do {
    const int t0 = max(p.lo, r.r0), t1 = min(p.hi, r.r1);
    f2 win[K][2];
    fill_window<T, K, kWhole>(x, a.x.st, a.state0, r, p, t0, a.wide, win);
    auto row = [&](int t, typename Raw<T>::type in) {
      float y[kV];
      pairs_of(in, win[K - 1]);
      convolve<K>(taps, win, bias, y);
      if (a.silu) {
#pragma unroll
        for (int j = 0; j < kV; ++j) y[j] = silu_f(y[j]);
      }
      write_row<kWhole, T, kV>(out + t * a.out.st, r.n, a.wide, y);
      shift<K>(win);
    };
    constexpr int n = kBatch<T>;
    int t = t0;
    typename Raw<T>::type in[n], ahead[n];
    if (t + n <= t1) {
#pragma unroll
      for (int i = 0; i < n; ++i) in[i] = raw_row<kWhole, T>(x + (t + i) * a.x.st, r.n, a.wide);
    }
#pragma unroll 1
    for (; t + n <= t1; t += n) {
      const int64_t next = t + 2 * n <= t1 ? t + n : t;  // the last batch reads itself again
#pragma unroll
      for (int i = 0; i < n; ++i) ahead[i] = raw_row<kWhole, T>(x + (next + i) * a.x.st, r.n, a.wide);
#pragma unroll
      for (int i = 0; i < n; ++i) row(t + i, in[i]);
#pragma unroll
      for (int i = 0; i < n; ++i) in[i] = ahead[i];
    }
    if (t < t1) {
#pragma unroll
      for (int i = 0; i < n; ++i) in[i] = raw_row<kWhole, T>(x + min(t + i, t1 - 1) * a.x.st, r.n, a.wide);
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (t + i < t1) row(t + i, in[i]);
    }
    if (a.fin.p && t1 == p.hi) {
      T* f = static_cast<T*>(a.fin.p) + p.seq * a.fin.sb + r.h * a.fin.sh + r.c;
#pragma unroll
      for (int k = 0; k < K - 1; ++k) {
        float v[kV];
        floats_of(win[k], v);
        store_row<T, kV>(f + k * a.fin.st, r.n, a.wide, v);
      }
    }
  } while (next_piece(a.seqs, r, a.T, a.status, &p));
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads, K <= 4 ? 5 : 3) conv_fwd_kernel(const __grid_constant__ ConvArgs a, int len) {
  const Run r = run_of<kV>((int64_t)blockIdx.x * kThreads + threadIdx.x, a.B, a.H, a.T, a.d, len);
  if (!r.live) return;
  if (a.wide && r.n >= kV) conv_run<T, K, true>(a, r);
  else conv_run<T, K, false>(a, r);
}

// dst[i] (dst may be null) = src[i] (zeros where src is null) for every sequence
// without a token; every offset of a packed call is seen here, and reported if
// out of order.
template <typename T>
__global__ void conv_empty_kernel(Seqs q, int T_, int H, int d, int rows, TokView src, RowsView dst,
                                  int* status) {
  const int seq = blockIdx.x;
  int lo = 0, hi = T_;
  if (q.cu) packed_seq(q.cu, seq, T_, status, &lo, &hi);
  if (hi > lo || !dst.p) return;
  const T* s = static_cast<const T*>(src.p);
  T* o = static_cast<T*>(dst.p);
  const int64_t n = (int64_t)H * rows * d;
  for (int64_t i = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.y * blockDim.x) {
    const int c = (int)(i % d), k = (int)(i / d % rows), h = (int)(i / d / rows);
    o[seq * dst.sb + h * dst.sh + k * dst.st + c] =
        s ? s[seq * src.sb + h * src.sh + k * src.st + c] : from_f32<T>(0.f);
  }
}

template <typename T>
cudaError_t copy_empty(const Seqs& q, int T_, int H, int d, int K, const TokView& src, const RowsView& dst,
                       int* status, cudaStream_t s) {
  if (!q.cu && (T_ > 0 || !dst.p)) return cudaSuccess;
  // mostly there is nothing to copy: a block for 1024 values, up to 16 a sequence
  const int64_t n = (int64_t)H * (K - 1) * d, rows = (n + 1023) / 1024;
  const dim3 g(q.S, (unsigned)(!dst.p || rows < 1 ? 1 : rows < 16 ? rows : 16));
  conv_empty_kernel<T><<<g, 256, 0, s>>>(q, T_, H, d, K - 1, src, dst, status);
  return cudaGetLastError();
}

// Gradients of one run. The walk goes K-1 tokens past the run's end: dx_s
// needs dp up to s+K-1, and dp is computed again there rather than exchanged.
// dp of tokens behind the sequence is zero. The run's shares of dweight and
// dbias go to ws[run][K+1][channels].
template <typename T>
constexpr int kBwdBatch = sizeof(T) == 2 ? 4 : 2;
template <typename T, int K, bool kWhole>
__device__ __forceinline__ void conv_back(const ConvBwdArgs& a, const Run& r, float* dst, int64_t cols) {
  f2 taps[K][2], bias[2], dw[K][2], db[2] = {0, 0};
  load_taps<K>(a.w, a.bias, a.d, r, taps, bias);
#pragma unroll
  for (int k = 0; k < K; ++k) dw[k][0] = dw[k][1] = 0;
  const T* x = static_cast<const T*>(a.x.p) + r.b * a.x.sb + r.h * a.x.sh + r.c;
  const T* dy = static_cast<const T*>(a.dy.p) + r.b * a.dy.sb + r.h * a.dy.sh + r.c;
  T* dx = static_cast<T*>(a.dx.p) + r.b * a.dx.sb + r.h * a.dx.sh + r.c;
  Piece p;
  if (first_piece(a.seqs, r, a.T, a.status, &p)) do {
    const int t0 = max(p.lo, r.r0), t1 = min(p.hi, r.r1);
    const int first = t0 == p.lo ? p.lo - (K - 1) : t0;  // the state's inputs belong to the first run
    f2 win[K][2], dp[K][2];  // dp[k] = dp of token t-K+1+k
    fill_window<T, K, kWhole>(x, a.x.st, a.state0, r, p, t0, a.wide, win);
#pragma unroll
    for (int k = 0; k < K; ++k) dp[k][0] = dp[k][1] = 0;
    // dp of token t from its rows; own: the token is the run's
    auto token = [&](typename Raw<T>::type xr, typename Raw<T>::type gr, bool own) {
      pairs_of(xr, win[K - 1]);
      pairs_of(gr, dp[K - 1]);
      if (a.silu) {
        float y[kV];
        convolve<K>(taps, win, bias, y);
#pragma unroll
        for (int j = 0; j < kV; ++j) y[j] = dsilu_f(y[j]);
        f2 v[2];
        pairs_of(y, v);
        dp[K - 1][0] = mul2(dp[K - 1][0], v[0]);
        dp[K - 1][1] = mul2(dp[K - 1][1], v[1]);
      }
      if (own) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          db[i] = add2(db[i], dp[K - 1][i]);
#pragma unroll
          for (int k = 0; k < K; ++k) dw[k][i] = fma2(dp[K - 1][i], win[k][i], dw[k][i]);
        }
      }
      shift<K>(win);
    };
    // dx of the token K-1 before the last dp
    auto gradient = [&](float (&o)[kV]) {
      f2 v[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[0] = fma2(taps[k][0], dp[K - 1 - k][0], v[0]);
        v[1] = fma2(taps[k][1], dp[K - 1 - k][1], v[1]);
      }
      floats_of(v, o);
    };
    // The walk goes in batches, the rows of the next one on their way. A batch
    // of the run's own tokens whose dx are all the run's and the sequence's own
    // (none of those is state_final's) needs no further look at its tokens.
    constexpr int n = kBwdBatch<T>;
    typename Raw<T>::type xr[n], gr[n], xa[n], ga[n];
    auto fetch = [&](int t) {  // tokens behind the sequence read its last
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const int64_t at = min(t + i, p.hi - 1);
        xa[i] = raw_row<kWhole, T>(x + at * a.x.st, r.n, a.wide);
        ga[i] = raw_row<kWhole, T>(dy + at * a.dy.st, r.n, a.wide);
      }
    };
    fetch(t0);
#pragma unroll 1
    for (int t = t0; t < t1 + K - 1; t += n) {
#pragma unroll
      for (int i = 0; i < n; ++i) xr[i] = xa[i], gr[i] = ga[i];
      fetch(t + n);
      if (t + n <= t1 && t - (K - 1) >= max(first, p.lo)) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
          shift<K>(dp);
          token(xr[i], gr[i], true);
          float o[kV];
          gradient(o);
          write_row<kWhole, T, kV>(dx + (t + i - (K - 1)) * a.dx.st, r.n, a.wide, o);
        }
        continue;
      }
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const int ti = t + i, s = ti - (K - 1);
        if (ti >= t1 + K - 1) break;
        shift<K>(dp);
        if (ti < p.hi) token(xr[i], gr[i], ti < t1);
        else dp[K - 1][0] = dp[K - 1][1] = 0;
        if (s < first || s >= t1) continue;
        float o[kV];
        gradient(o);
        if (a.dfin.p && s >= p.hi - (K - 1)) {  // state_final holds this input
          float f[kV];
          const T* df = static_cast<const T*>(a.dfin.p) + p.seq * a.dfin.sb + r.h * a.dfin.sh + r.c;
          load_row<T, kV>(df + (int64_t)(K - 1 + s - p.hi) * a.dfin.st, r.n, a.wide, f);
#pragma unroll
          for (int j = 0; j < kV; ++j) o[j] += f[j];
        }
        if (s >= p.lo) {
          write_row<kWhole, T, kV>(dx + s * a.dx.st, r.n, a.wide, o);
        } else if (a.dstate0.p) {
          T* d0 = static_cast<T*>(a.dstate0.p) + p.seq * a.dstate0.sb + r.h * a.dstate0.sh + r.c;
          store_row<T, kV>(d0 + (int64_t)(K - 1 + s - p.lo) * a.dstate0.st, r.n, a.wide, o);
        }
      }
    }
  } while (next_piece(a.seqs, r, a.T, a.status, &p));
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    float f[kV];
    if (k < K) floats_of(dw[k < K ? k : 0], f);
    else floats_of(db, f);
    *reinterpret_cast<float4*>(dst + k * cols) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads, K > 4 ? 2 : 3)
    conv_bwd_kernel(const __grid_constant__ ConvBwdArgs a, int len, int64_t cols) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const Run r = run_of<kV>(id, a.B, a.H, a.T, a.d, len);
  if (!r.live) return;
  const int64_t nv = cols / kV;
  float* dst = a.ws + (id / nv) * (K + 1) * cols + (id % nv) * kV;
  if (a.wide && r.n >= kV) conv_back<T, K, true>(a, r, dst, cols);
  else conv_back<T, K, false>(a, r, dst, cols);
}

struct ConvDw {
  float *dw, *db;
  int64_t cols;
  int per_head, d, K;  // per_head: padded channels of a head
  __device__ void operator()(int64_t col, float v) const {
    const int k = (int)(col / cols);
    const int64_t i = col % cols, h = i / per_head;
    const int c = (int)(i % per_head);
    if (c >= d) return;
    if (k < K) dw[(h * d + c) * K + k] = v;
    else if (db) db[h * d + c] = v;
  }
};

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStepArgs a) {
  SlotRows rows;
  if (!rows.begin(a.slots, blockIdx.y, a.B, a.S, a.status)) return;
  Run r = run_of<kV>((int64_t)blockIdx.x * kThreads + threadIdx.x, 1, a.H, 1, a.d, 1);
  if (!r.live) r.n = 0, r.h = 0, r.c = 0;  // stays for the block's barriers
  f2 taps[K][2], bias[2], win[K][2];
  T* st = static_cast<T*>(a.state.p) + rows.slot * a.state.sb + r.h * a.state.sh + r.c;
#pragma unroll
  for (int k = 0; k < K - 1; ++k) {
    float f[kV];
    load_row<T, kV>(st + k * a.state.st, r.n, a.wide, f);
    pairs_of(f, win[k]);
  }
  load_taps<K>(a.w, a.bias, a.d, r, taps, bias);
  do {
    const T* x = static_cast<const T*>(a.x.p) + rows.b * a.x.sb + r.h * a.x.sh + r.c;
    T* out = static_cast<T*>(a.out.p) + rows.b * a.out.sb + r.h * a.out.sh + r.c;
    float y[kV];
    load_row<T, kV>(x, r.n, a.wide, y);
    pairs_of(y, win[K - 1]);
    convolve<K>(taps, win, bias, y);
    if (a.silu) {
#pragma unroll
      for (int j = 0; j < kV; ++j) y[j] = silu_f(y[j]);
    }
    shift<K>(win);
    store_row<T, kV>(out, r.n, a.wide, y);
  } while (rows.next_row());
#pragma unroll
  for (int k = 0; k < K - 1; ++k) {
    float f[kV];
    floats_of(win[k], f);
    store_row<T, kV>(st + k * a.state.st, r.n, a.wide, f);
  }
}

// f(integral constant K) for the call's K.
template <typename F>
cudaError_t for_taps(int K, F f) {
  switch (K) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    case 8: return f(std::integral_constant<int, 8>());
  }
  return cudaErrorInvalidValue;
}

// Tokens a thread walks: as many as leave `want` threads, to make the rows read
// twice (K-1 a run, and in the backward pass computed twice, with K+1 partial
// sums a run) cheap; beyond 64 the SMs have too few threads. B2 T4096 d4096 K4
// bf16 backward: 80 us in runs of 32, 70 in 64, 77 in 128.
int run_length(int64_t vecs, int B, int T, int64_t want, int least, int most) {
  int len = most;
  while (len > least && vecs * B * ((T + len - 1) / len) < want) len /= 2;
  return len;
}

int fwd_run(const ConvArgs& a) {
  return run_length((int64_t)a.H * ((a.d + kV - 1) / kV), a.B, a.T, 148 * 1024, 8, 64);
}
int bwd_run(const ConvBwdArgs& a) {
  return run_length((int64_t)a.H * ((a.d + kV - 1) / kV), a.B, a.T, 148 * 256, 16, 64);
}
int64_t bwd_cols(const ConvBwdArgs& a) { return (int64_t)a.H * ((a.d + kV - 1) / kV) * kV; }
int64_t bwd_runs(const ConvBwdArgs& a) {
  const int len = bwd_run(a);
  return (int64_t)a.B * ((a.T + len - 1) / len);
}

template <typename T>
cudaError_t fwd(const ConvArgs& a, cudaStream_t s) {
  cudaError_t e = copy_empty<T>(a.seqs, a.T, a.H, a.d, a.K, a.state0, a.fin, a.status, s);
  if (e != cudaSuccess || a.T == 0) return e;
  const int len = fwd_run(a);
  const int64_t n = (int64_t)a.H * ((a.d + kV - 1) / kV) * a.B * ((a.T + len - 1) / len);
  const int64_t blocks = (n + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return for_taps(a.K, [&](auto k) {
    conv_fwd_kernel<T, decltype(k)::value><<<(unsigned)blocks, kThreads, 0, s>>>(a, len);
    return cudaGetLastError();
  });
}

template <typename T>
cudaError_t bwd(const ConvBwdArgs& a, cudaStream_t s) {
  const RowsView d0 = {a.dstate0.p, a.dstate0.sb, a.dstate0.sh, a.dstate0.st};
  cudaError_t e = copy_empty<T>(a.seqs, a.T, a.H, a.d, a.K, a.dfin, d0, a.status, s);
  if (e != cudaSuccess) return e;
  const int len = bwd_run(a);
  const int64_t cols = bwd_cols(a), runs = bwd_runs(a);
  const int64_t blocks = (cols / kV * runs + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (runs > 0) {
    e = for_taps(a.K, [&](auto k) {
      conv_bwd_kernel<T, decltype(k)::value><<<(unsigned)blocks, kThreads, 0, s>>>(a, len, cols);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
  }
  const int per_head = (a.d + kV - 1) / kV * kV;
  return sum_parts(a.ws, runs, (a.K + 1) * cols, ConvDw{a.dw, a.dbias, cols, per_head, a.d, a.K}, s);
}

template <typename T>
cudaError_t step(const ConvStepArgs& a, cudaStream_t s) {
  const int64_t n = (int64_t)a.H * ((a.d + kV - 1) / kV);
  if (a.B > 65535) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)((n + kThreads - 1) / kThreads), a.B);
  return for_taps(a.K, [&](auto k) {
    conv_step_kernel<T, decltype(k)::value><<<g, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_causal_conv_fwd(const ConvArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? fwd<__nv_bfloat16>(a, s) : fwd<float>(a, s);
}
size_t causal_conv_bwd_workspace(const ConvBwdArgs& a, bool) {
  return (size_t)(bwd_runs(a) * (a.K + 1) * bwd_cols(a)) * sizeof(float);
}
cudaError_t launch_causal_conv_bwd(const ConvBwdArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? bwd<__nv_bfloat16>(a, s) : bwd<float>(a, s);
}
cudaError_t launch_causal_conv_step(const ConvStepArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? step<__nv_bfloat16>(a, s) : step<float>(a, s);
}

}  // namespace ttt
