// Short causal depthwise convolution: prompts, backward, single tokens
// (causal_conv_fwd, causal_conv_bwd, causal_conv_step of include/ttt.h).
//
// Bound by memory. A thread owns a few neighbouring channels and walks a run
// of tokens with the last K inputs in registers, so every input is read once
// (plus K-1 rows where a run begins) in row-contiguous vectors, and nothing
// passes through shared memory.
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
template <typename T, int K, int V>
__device__ __forceinline__ void fill_window(const T* x, int64_t st, const TokView& state0, const Run& r,
                                            const Piece& p, int t, bool wide, float (&win)[K][V]) {
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int src = t - (K - 1) + i;
    if (src >= p.lo) {
      load_row<T, V>(x + src * st, r.n, wide, win[i]);
    } else if (state0.p) {
      const T* s0 = static_cast<const T*>(state0.p) + p.seq * state0.sb + r.h * state0.sh + r.c;
      load_row<T, V>(s0 + (int64_t)(K - 1 + src - p.lo) * state0.st, r.n, wide, win[i]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) win[i][j] = 0.f;
    }
  }
}

template <int K, int V>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, int d, const Run& r,
                                          float (&taps)[K][V], float (&b)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t c = (int64_t)r.h * d + r.c + j;
    const bool in = j < r.n;
    b[j] = in && bias ? bias[c] : 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) taps[i][j] = in ? w[c * K + i] : 0.f;
  }
}

constexpr int kBatch = 4;  // rows loaded ahead of their use

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a, int len) {
  constexpr int V = Vec<T>::n;
  const Run r = run_of<V>((int64_t)blockIdx.x * kThreads + threadIdx.x, a.B, a.H, a.T, a.d, len);
  if (!r.live) return;
  float taps[K][V], bias[V];
  load_taps<K, V>(a.w, a.bias, a.d, r, taps, bias);
  const T* x = static_cast<const T*>(a.x.p) + r.b * a.x.sb + r.h * a.x.sh + r.c;
  T* out = static_cast<T*>(a.out.p) + r.b * a.out.sb + r.h * a.out.sh + r.c;
  Piece p;
  if (!first_piece(a.seqs, r, a.T, a.status, &p)) return;
  do {
    const int t0 = max(p.lo, r.r0), t1 = min(p.hi, r.r1);
    float win[K][V];
    fill_window<T, K, V>(x, a.x.st, a.state0, r, p, t0, a.wide, win);
    for (int tb = t0; tb < t1; tb += kBatch) {
      Vec<T> in[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (tb + i < t1) in[i] = load_vec(x + (tb + i) * a.x.st, r.n, a.wide);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (tb + i >= t1) break;
        unpack<T>(in[i], win[K - 1]);
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          y[j] = bias[j];
#pragma unroll
          for (int k = 0; k < K; ++k) y[j] = fmaf(taps[k][j], win[k][j], y[j]);
          if (a.silu) y[j] = silu_f(y[j]);
#pragma unroll
          for (int k = 0; k < K - 1; ++k) win[k][j] = win[k + 1][j];
        }
        store_vec<T>(out + (tb + i) * a.out.st, r.n, a.wide, y);
      }
    }
    if (a.fin.p && t1 == p.hi) {
      T* f = static_cast<T*>(a.fin.p) + p.seq * a.fin.sb + r.h * a.fin.sh + r.c;
#pragma unroll
      for (int k = 0; k < K - 1; ++k) store_vec<T>(f + k * a.fin.st, r.n, a.wide, win[k]);
    }
  } while (next_piece(a.seqs, r, a.T, a.status, &p));
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
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    const int c = (int)(i % d), k = (int)(i / d % rows), h = (int)(i / d / rows);
    o[seq * dst.sb + h * dst.sh + k * dst.st + c] =
        s ? s[seq * src.sb + h * src.sh + k * src.st + c] : from_f32<T>(0.f);
  }
}

template <typename T>
cudaError_t copy_empty(const Seqs& q, int T_, int H, int d, int K, const TokView& src, const RowsView& dst,
                       int* status, cudaStream_t s) {
  if (!q.cu && (T_ > 0 || !dst.p)) return cudaSuccess;
  conv_empty_kernel<T><<<q.S, 256, 0, s>>>(q, T_, H, d, K - 1, src, dst, status);
  return cudaGetLastError();
}

// Gradients of one run. The walk goes K-1 tokens past the run's end: dx_s
// needs dp up to s+K-1, and dp is computed again there rather than exchanged.
// dp of tokens behind the sequence is zero. The run's shares of dweight and
// dbias go to ws[run][K+1][channels].
constexpr int kBwdV = 4;
template <typename T, int K>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvBwdArgs a, int len, int64_t cols) {
  constexpr int V = kBwdV;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const Run r = run_of<V>(id, a.B, a.H, a.T, a.d, len);
  if (!r.live) return;
  float taps[K][V], bias[V], dw[K][V], db[V];
  load_taps<K, V>(a.w, a.bias, a.d, r, taps, bias);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    db[j] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k][j] = 0.f;
  }
  const T* x = static_cast<const T*>(a.x.p) + r.b * a.x.sb + r.h * a.x.sh + r.c;
  const T* dy = static_cast<const T*>(a.dy.p) + r.b * a.dy.sb + r.h * a.dy.sh + r.c;
  T* dx = static_cast<T*>(a.dx.p) + r.b * a.dx.sb + r.h * a.dx.sh + r.c;
  Piece p;
  if (first_piece(a.seqs, r, a.T, a.status, &p)) do {
    const int t0 = max(p.lo, r.r0), t1 = min(p.hi, r.r1);
    const int first = t0 == p.lo ? p.lo - (K - 1) : t0;  // the state's inputs belong to the first run
    float win[K][V], dp[K][V];
    fill_window<T, K, V>(x, a.x.st, a.state0, r, p, t0, a.wide, win);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) dp[k][j] = 0.f;
    for (int t = t0; t < t1 + K - 1; ++t) {
      // dp[k] = dp of token t-K+1+k
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) dp[k][j] = dp[k + 1][j];
      if (t < p.hi) {
        float g[V];
        load_row<T, V>(x + t * a.x.st, r.n, a.wide, win[K - 1]);
        load_row<T, V>(dy + t * a.dy.st, r.n, a.wide, g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (a.silu) {
            float y = bias[j];
#pragma unroll
            for (int k = 0; k < K; ++k) y = fmaf(taps[k][j], win[k][j], y);
            g[j] *= dsilu_f(y);
          }
          dp[K - 1][j] = g[j];
          if (t < t1) {
            db[j] += g[j];
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][j] = fmaf(g[j], win[k][j], dw[k][j]);
          }
#pragma unroll
          for (int k = 0; k < K - 1; ++k) win[k][j] = win[k + 1][j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) dp[K - 1][j] = 0.f;
      }
      const int s = t - (K - 1);
      if (s < first || s >= t1) continue;
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        o[j] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) o[j] = fmaf(taps[k][j], dp[K - 1 - k][j], o[j]);
      }
      if (a.dfin.p && s >= p.hi - (K - 1)) {  // state_final holds this input
        float f[V];
        const T* df = static_cast<const T*>(a.dfin.p) + p.seq * a.dfin.sb + r.h * a.dfin.sh + r.c;
        load_row<T, V>(df + (int64_t)(K - 1 + s - p.hi) * a.dfin.st, r.n, a.wide, f);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] += f[j];
      }
      if (s >= p.lo) {
        store_row<T, V>(dx + s * a.dx.st, r.n, a.wide, o);
      } else if (a.dstate0.p) {
        T* d0 = static_cast<T*>(a.dstate0.p) + p.seq * a.dstate0.sb + r.h * a.dstate0.sh + r.c;
        store_row<T, V>(d0 + (int64_t)(K - 1 + s - p.lo) * a.dstate0.st, r.n, a.wide, o);
      }
    }
  } while (next_piece(a.seqs, r, a.T, a.status, &p));
  const int64_t nv = cols / V;
  float* dst = a.ws + (id / nv) * (K + 1) * cols + (id % nv) * V;
#pragma unroll
  for (int k = 0; k <= K; ++k)
    *reinterpret_cast<float4*>(dst + k * cols) =
        k < K ? make_float4(dw[k < K ? k : 0][0], dw[k < K ? k : 0][1], dw[k < K ? k : 0][2], dw[k < K ? k : 0][3])
              : make_float4(db[0], db[1], db[2], db[3]);
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
  constexpr int V = Vec<T>::n;
  SlotRows rows;
  if (!rows.begin(a.slots, blockIdx.y, a.B, a.S, a.status)) return;
  Run r = run_of<V>((int64_t)blockIdx.x * kThreads + threadIdx.x, 1, a.H, 1, a.d, 1);
  if (!r.live) r.n = 0, r.h = 0, r.c = 0;  // stays for the block's barriers
  float taps[K][V], bias[V];
  load_taps<K, V>(a.w, a.bias, a.d, r, taps, bias);
  T* st = static_cast<T*>(a.state.p) + rows.slot * a.state.sb + r.h * a.state.sh + r.c;
  float win[K][V];
#pragma unroll
  for (int k = 0; k < K - 1; ++k) load_row<T, V>(st + k * a.state.st, r.n, a.wide, win[k]);
  do {
    const T* x = static_cast<const T*>(a.x.p) + rows.b * a.x.sb + r.h * a.x.sh + r.c;
    T* out = static_cast<T*>(a.out.p) + rows.b * a.out.sb + r.h * a.out.sh + r.c;
    load_row<T, V>(x, r.n, a.wide, win[K - 1]);
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      y[j] = bias[j];
#pragma unroll
      for (int k = 0; k < K; ++k) y[j] = fmaf(taps[k][j], win[k][j], y[j]);
      if (a.silu) y[j] = silu_f(y[j]);
#pragma unroll
      for (int k = 0; k < K - 1; ++k) win[k][j] = win[k + 1][j];
    }
    store_row<T, V>(out, r.n, a.wide, y);
  } while (rows.next_row());
#pragma unroll
  for (int k = 0; k < K - 1; ++k) store_row<T, V>(st + k * a.state.st, r.n, a.wide, win[k]);
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

// Tokens a thread walks: long enough to make the K-1 rows read twice cheap,
// short enough to give every SM 1024 threads.
int run_length(int64_t vecs, int B, int T, int least, int most) {
  const int64_t want = (int64_t)148 * 1024;
  int len = most;
  while (len > least && vecs * B * ((T + len - 1) / len) < want) len /= 2;
  return len;
}

int fwd_run(const ConvArgs& a, int V) {
  return run_length((int64_t)a.H * ((a.d + V - 1) / V), a.B, a.T, 8, 64);
}
int bwd_run(const ConvBwdArgs& a) {
  return run_length((int64_t)a.H * ((a.d + kBwdV - 1) / kBwdV), a.B, a.T, 16, 128);
}
int64_t bwd_cols(const ConvBwdArgs& a) { return (int64_t)a.H * ((a.d + kBwdV - 1) / kBwdV) * kBwdV; }
int64_t bwd_runs(const ConvBwdArgs& a) {
  const int len = bwd_run(a);
  return (int64_t)a.B * ((a.T + len - 1) / len);
}

template <typename T>
cudaError_t fwd(const ConvArgs& a, cudaStream_t s) {
  cudaError_t e = copy_empty<T>(a.seqs, a.T, a.H, a.d, a.K, a.state0, a.fin, a.status, s);
  if (e != cudaSuccess || a.T == 0) return e;
  constexpr int V = Vec<T>::n;
  const int len = fwd_run(a, V);
  const int64_t n = (int64_t)a.H * ((a.d + V - 1) / V) * a.B * ((a.T + len - 1) / len);
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
  const int64_t blocks = (cols / kBwdV * runs + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (runs > 0) {
    e = for_taps(a.K, [&](auto k) {
      conv_bwd_kernel<T, decltype(k)::value><<<(unsigned)blocks, kThreads, 0, s>>>(a, len, cols);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
  }
  const int per_head = (a.d + kBwdV - 1) / kBwdV * kBwdV;
  return sum_parts(a.ws, runs, (a.K + 1) * cols, ConvDw{a.dw, a.dbias, cols, per_head, a.d, a.K}, s);
}

template <typename T>
cudaError_t step(const ConvStepArgs& a, cudaStream_t s) {
  constexpr int V = Vec<T>::n;
  const int64_t n = (int64_t)a.H * ((a.d + V - 1) / V);
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
