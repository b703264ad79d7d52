// RMS norm with the residual's addition and an 8-bit output, and its backward
// (rms_norm_fwd, rms_norm_bwd of include/ttt.h).
//
// Bound by memory: a row is read once into registers (16-byte loads), summed
// in fp32 and written once. A row belongs to a power of two of lanes where it
// has at most 32 vectors (q/k heads of 64: 8 lanes, four rows a warp), to one
// warp up to kVpt * 32 vectors, and to a block of its own above that.
#include <cuda_fp8.h>

#include "block.cuh"

namespace ttt {
namespace {

constexpr int kThreads = 256;   // of a block that holds several rows
constexpr int kVpt = 4;         // vectors a lane holds where a warp has a row
constexpr int kMaxThreads = 512;  // a block of one row; 128 registers a thread

// How a row of d elements is laid over threads.
struct RowPlan {
  int lanes;   // threads a row: a power of two <= 32, or a multiple of 32
  int vpt;     // vectors a thread: 1, 2, 4, or 8 (fp32 only: as many values as 4 of bf16)
  int block;   // threads a block
};
template <typename T>
RowPlan plan_rows(int d) {
  const int nv = (d + Vec<T>::n - 1) / Vec<T>::n;
  RowPlan p;
  if (nv <= 32) {
    p.lanes = 1;
    while (p.lanes < nv) p.lanes *= 2;
    p.vpt = 1;
    p.block = kThreads;
  } else if (nv <= 32 * kVpt) {
    p.lanes = 32;
    p.vpt = nv <= 64 ? 2 : 4;
    p.block = kThreads;
  } else {
    // two vectors a thread keep enough loads in flight without needing many
    // registers; more where 512 threads would not reach
    p.vpt = nv <= 1024 ? 2 : nv <= 2048 ? 4 : 8;
    p.lanes = ((nv + p.vpt - 1) / p.vpt + 31) / 32 * 32;
    p.block = p.lanes;
  }
  return p;
}

// Sum (or maximum, kMax) of v over the `lanes` threads of a row, to all of
// them. `red` holds a value a warp; blocks of one row only. The maximum
// keeps NaN.
template <bool kMax>
__device__ __forceinline__ float join(float a, float b) {
  if (!kMax) return a + b;
  return a > b || a != a ? a : b;
}
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v, int lanes, float* red) {
  for (int o = min(lanes, 32) / 2; o; o >>= 1) v = join<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (lanes > 32) {
    __syncthreads();  // the last use of `red` is over
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < lanes / 32; ++i) v = join<kMax>(v, red[i]);
  }
  return v;
}

struct RowAt {
  int b, h, t;
};
__device__ __forceinline__ RowAt row_at(int64_t r, int H, int T) {
  const int64_t bh = r / T;
  return {(int)(bh / H), (int)(bh % H), (int)(r % T)};
}

// (mean + eps)^(-1/2); a row of zeros with eps = 0 has nothing to scale.
__device__ __forceinline__ float inv_rms(float sumsq, int d, float eps) {
  const float m = sumsq / (float)d + eps;
  return m > 0.f || m != m ? rsqrtf(m) : 0.f;
}

__device__ __forceinline__ void store_e4m3(uint8_t* p, int n, bool wide, const float* y, int count) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    if (i >= count) break;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[i], y[i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(y[i + 2], y[i + 3]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t w = lo | hi << 16;
    if (wide && i + 4 <= n) {
      *reinterpret_cast<uint32_t*>(p + i) = w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < n) p[i + k] = (uint8_t)(w >> (8 * k));
    }
  }
}

template <typename T, int VPT>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(NormArgs a, int lanes) {
  constexpr int V = Vec<T>::n;
  __shared__ float red[32];
  const int lane = threadIdx.x % lanes;
  const int64_t rows = (int64_t)a.B * a.H * a.T;
  const int64_t r = (int64_t)blockIdx.x * (blockDim.x / lanes) + threadIdx.x / lanes;
  const bool live = r < rows;
  const RowAt at = row_at(live ? r : rows - 1, a.H, a.T);
  const T* x = static_cast<const T*>(a.x.p) + at.b * a.x.sb + at.h * a.x.sh + at.t * a.x.st;
  const float* w = a.w + at.h * a.w_sh;
  float s[VPT][V];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) unpack<T>(load_vec(x + (i * lanes + lane) * V, a.d - (i * lanes + lane) * V, a.wide), s[i]);
  if (a.r.p) {
    const T* res = static_cast<const T*>(a.r.p) + at.b * a.r.sb + at.h * a.r.sh + at.t * a.r.st;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * lanes + lane) * V;
      float f[V];
      unpack<T>(load_vec(res + c, a.d - c, a.wide), f);
#pragma unroll
      for (int j = 0; j < V; ++j) s[i][j] += f[j];
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) sum = fmaf(s[i][j], s[i][j], sum);
  if (a.rout.p && live) {
    T* ro = static_cast<T*>(a.rout.p) + at.b * a.rout.sb + at.h * a.rout.sh + at.t * a.rout.st;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * lanes + lane) * V;
      store_vec<T>(ro + c, a.d - c, a.wide, s[i]);
    }
  }
  const float rs = inv_rms(row_reduce<false>(sum, lanes, red), a.d, a.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * lanes + lane) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) s[i][j] = c + j < a.d ? s[i][j] * rs * w[c + j] : 0.f;
  }
  if (!a.scale) {
    if (!live) return;
    T* o = static_cast<T*>(a.out.p) + at.b * a.out.sb + at.h * a.out.sh + at.t * a.out.st;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * lanes + lane) * V;
      store_vec<T>(o + c, a.d - c, a.wide, s[i]);
    }
    return;
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) top = join<true>(top, fabsf(s[i][j]));
  top = row_reduce<true>(top, lanes, red);
  if (!live) return;
  const float scale = top / 448.f;
  if (lane == 0) a.scale[at.b * a.sc_sb + at.h * a.sc_sh + at.t * a.sc_st] = scale;
  const float by = scale == 0.f ? 1.f : scale;
  uint8_t* o = static_cast<uint8_t*>(a.out.p) + at.b * a.out.sb + at.h * a.out.sh + at.t * a.out.st;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * lanes + lane) * V;
    float q[8];
#pragma unroll
    for (int j = 0; j < V; ++j) q[j] = s[i][j] / by;
    store_e4m3(o + c, a.d - c, a.wide, q, V);
  }
}

// Rows of one weight: all of them, or those of head blockIdx.y. Every block
// walks rows worker, worker + workers, ... and keeps its share of dweight in
// registers; the shares go to ws[block][d padded to the row's vectors].
template <typename T, int VPT>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(NormBwdArgs a, int lanes, int64_t rows, int cols) {
  constexpr int V = Vec<T>::n;
  extern __shared__ float share[];  // [rows a block][cols]
  __shared__ float red[32];
  const int lane = threadIdx.x % lanes, sub = threadIdx.x / lanes, subs = blockDim.x / lanes;
  const int64_t workers = (int64_t)gridDim.x * subs;
  const int head = blockIdx.y;
  const float* w = a.w + head * a.w_sh;
  float dw[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
  // every thread of a block makes the same number of turns (row_reduce synchronises)
  const int64_t turns = (rows + workers - 1) / workers;
  for (int64_t k = 0; k < turns; ++k) {
    const int64_t r = k * workers + (int64_t)blockIdx.x * subs + sub;
    const bool live = r < rows;
    RowAt at = {0, 0, 0};
    if (live) {
      if (a.w_sh) {
        at = {(int)(r / a.T), head, (int)(r % a.T)};
      } else {
        at = row_at(r, a.H, a.T);
      }
    }
    const T* hp = static_cast<const T*>(a.h.p) + at.b * a.h.sb + at.h * a.h.sh + at.t * a.h.st;
    const T* gp = static_cast<const T*>(a.dy.p) + at.b * a.dy.sb + at.h * a.dy.sh + at.t * a.dy.st;
    Vec<T> hv[VPT], gv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * lanes + lane) * V;
      hv[i] = load_vec(hp + c, live ? a.d - c : 0, a.wide);
      gv[i] = load_vec(gp + c, live ? a.d - c : 0, a.wide);
    }
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * lanes + lane) * V;
      float h[V], g[V];
      unpack<T>(hv[i], h);
      unpack<T>(gv[i], g);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sum = fmaf(h[j], h[j], sum);
        dot = fmaf(c + j < a.d ? g[j] * w[c + j] : 0.f, h[j], dot);
      }
    }
    const float rs = inv_rms(row_reduce<false>(sum, lanes, red), a.d, a.eps);
    const float m = row_reduce<false>(dot, lanes, red) / (float)a.d * rs * rs;
    if (!live) continue;  // the block's last turn
    const T* rp = a.dres.p ? static_cast<const T*>(a.dres.p) + at.b * a.dres.sb + at.h * a.dres.sh + at.t * a.dres.st
                           : nullptr;
    T* op = static_cast<T*>(a.dh.p) + at.b * a.dh.sb + at.h * a.dh.sh + at.t * a.dh.st;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * lanes + lane) * V;
      float h[V], g[V], o[V];
      unpack<T>(hv[i], h);
      unpack<T>(gv[i], g);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        dw[i][j] = fmaf(g[j], h[j] * rs, dw[i][j]);
        o[j] = rs * ((c + j < a.d ? g[j] * w[c + j] : 0.f) - h[j] * m);
      }
      if (rp) {
        float f[V];
        unpack<T>(load_vec(rp + c, a.d - c, a.wide), f);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] += f[j];
      }
      store_vec<T>(op + c, a.d - c, a.wide, o);
    }
  }
  float* dst = a.ws + ((int64_t)blockIdx.x * gridDim.y + head) * cols;
  if (subs == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) dst[(i * lanes + lane) * V + j] = dw[i][j];
    return;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) share[sub * cols + (i * lanes + lane) * V + j] = dw[i][j];
  __syncthreads();
  for (int c = threadIdx.x; c < cols; c += blockDim.x) {
    float s = share[c];
    for (int k = 1; k < subs; ++k) s += share[k * cols + c];
    dst[c] = s;
  }
}

struct NormDw {
  float* dw;
  int cols, d;
  __device__ void operator()(int64_t col, float v) const {
    const int64_t h = col / cols;
    const int c = (int)(col % cols);
    if (c < d) dw[h * d + c] = v;
  }
};

// Blocks along a weight's rows: enough to fill the GPU several times over,
// few enough that the shares of dweight stay small beside the rows.
template <typename T>
int bwd_blocks(const NormBwdArgs& a) {
  const RowPlan p = plan_rows<T>(a.d);
  const int64_t rows = (int64_t)a.B * a.T * (a.w_sh ? 1 : a.H);
  const int subs = p.block / p.lanes;
  const int64_t want = (rows + subs - 1) / subs;
  const int64_t cap = (int64_t)148 * (2048 / p.block) / (a.w_sh ? a.H : 1);
  return (int)(want < 1 ? 1 : want < cap ? want : cap < 1 ? 1 : cap);
}

template <typename T>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
  const RowPlan p = plan_rows<T>(a.d);
  const int64_t rows = (int64_t)a.B * a.H * a.T, per = p.block / p.lanes;
  const int64_t blocks = (rows + per - 1) / per;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)blocks), b(p.block);
  if (p.vpt == 1) norm_fwd_kernel<T, 1><<<g, b, 0, s>>>(a, p.lanes);
  else if (p.vpt == 2) norm_fwd_kernel<T, 2><<<g, b, 0, s>>>(a, p.lanes);
  else if (p.vpt == 4) norm_fwd_kernel<T, 4><<<g, b, 0, s>>>(a, p.lanes);
  else if constexpr (Vec<T>::n == 4) norm_fwd_kernel<T, 8><<<g, b, 0, s>>>(a, p.lanes);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t s) {
  const RowPlan p = plan_rows<T>(a.d);
  const int cols = p.lanes * p.vpt * Vec<T>::n, heads = a.w_sh ? a.H : 1;
  const int64_t rows = (int64_t)a.B * a.T * (a.w_sh ? 1 : a.H);
  const int subs = p.block / p.lanes, blocks = bwd_blocks<T>(a);
  const dim3 g(blocks, heads), b(p.block);
  const size_t sh = subs > 1 ? (size_t)subs * cols * 4 : 0;
  if (p.vpt == 1) norm_bwd_kernel<T, 1><<<g, b, sh, s>>>(a, p.lanes, rows, cols);
  else if (p.vpt == 2) norm_bwd_kernel<T, 2><<<g, b, sh, s>>>(a, p.lanes, rows, cols);
  else if (p.vpt == 4) norm_bwd_kernel<T, 4><<<g, b, sh, s>>>(a, p.lanes, rows, cols);
  else if constexpr (Vec<T>::n == 4) norm_bwd_kernel<T, 8><<<g, b, sh, s>>>(a, p.lanes, rows, cols);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return sum_parts(a.ws, blocks, (int64_t)heads * cols, NormDw{a.dw, cols, a.d}, s);
}

}  // namespace

cudaError_t launch_rms_norm_fwd(const NormArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? fwd<__nv_bfloat16>(a, s) : fwd<float>(a, s);
}

size_t rms_norm_bwd_workspace(const NormBwdArgs& a, bool bf16) {
  const RowPlan p = bf16 ? plan_rows<__nv_bfloat16>(a.d) : plan_rows<float>(a.d);
  const int blocks = bf16 ? bwd_blocks<__nv_bfloat16>(a) : bwd_blocks<float>(a);
  return (size_t)blocks * (a.w_sh ? a.H : 1) * p.lanes * p.vpt * (bf16 ? 8 : 4) * sizeof(float);
}

cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? bwd<__nv_bfloat16>(a, s) : bwd<float>(a, s);
}

}  // namespace ttt
