// RMS norm with the residual's addition and an 8-bit output, and its backward
// (rms_norm_fwd, rms_norm_bwd of include/ttt.h).
//
// Bound by memory: a row is read once into registers (16-byte loads), summed
// in fp32 and written once. A row belongs to a power of two of lanes where it
// has at most 32 vectors (q/k heads of 64: 8 lanes, four rows a warp), to one
// warp up to 256 vectors (128 in the backward pass), and to a block of its own
// above that.
//
// B4 T4096 d2048 bf16: forward with residual and 8-bit output 43 us (36 at the
// measured copy rate), backward 64 us (41) with the ordered sum of
// dweight's shares; 16 heads of 64, B8 T2048: 20 us (10), waiting on its loads
// with 5 blocks an SM.
#include <cuda_fp8.h>

#include "block.cuh"

namespace ttt {
namespace {

constexpr int kThreads = 128;   // of a block that holds several rows
constexpr int kVpt = 4;         // vectors a lane holds where a warp has a row
constexpr int kMaxThreads = 512;  // a block of one row; 128 registers a thread

// How a row of d elements is laid over threads.
struct RowPlan {
  int lanes;   // threads a row: a power of two <= 32, or a multiple of 32
  int vpt;     // vectors a thread: 1, 2, 4 or 8
  int block;   // threads a block
};
template <typename T>
RowPlan plan_rows(int d, int warp_vecs = kVpt) {
  const int nv = (d + Vec<T>::n - 1) / Vec<T>::n;
  RowPlan p;
  if (nv <= 32) {
    p.lanes = 1;
    while (p.lanes < nv) p.lanes *= 2;
    p.vpt = 1;
    p.block = kThreads;
  } else if (nv <= 32 * warp_vecs) {
    p.lanes = 32;
    p.vpt = nv <= 64 ? 2 : nv <= 128 ? 4 : 8;
    p.block = p.vpt == 8 ? 32 : kThreads;
  } else {
    // two vectors a thread keep enough loads in flight without needing many
    // registers; more where 512 threads would not reach
    p.vpt = nv <= 1024 ? 2 : nv <= 2048 ? 4 : 8;
    p.lanes = ((nv + p.vpt - 1) / p.vpt + 31) / 32 * 32;
    p.block = p.lanes;
  }
  return p;
}

// Sums (or maxima, kMax) of v[0..n) over the `lanes` threads of a row, to all of
// them. `red` holds n values a warp; blocks of one row only. The maximum keeps NaN.
template <bool kMax>
__device__ __forceinline__ float join(float a, float b) {
  if (!kMax) return a + b;
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <bool kMax, int n>
__device__ __forceinline__ void row_reduce(float (&v)[n], int lanes, float* red) {
  for (int o = min(lanes, 32) / 2; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = join<kMax>(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
  if (lanes > 32) {
    __syncthreads();  // the last use of `red` is over
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < n; ++i) red[(threadIdx.x >> 5) * n + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < n; ++i) {
      v[i] = red[i];
      for (int k = 1; k < lanes / 32; ++k) v[i] = join<kMax>(v[i], red[k * n + i]);
    }
  }
}

struct RowAt {
  int b, h, t;
};
__device__ __forceinline__ RowAt row_at(int64_t r, int H, int T) {
  if (r < 0x7fffffff) {  // the common case, without 64-bit division
    const unsigned bh = (unsigned)r / (unsigned)T;
    return {(int)(bh / H), (int)(bh % H), (int)((unsigned)r - bh * T)};
  }
  const int64_t bh = r / T;
  return {(int)(bh / H), (int)(bh % H), (int)(r % T)};
}

// (mean + eps)^(-1/2); a row of zeros with eps = 0 has nothing to scale.
__device__ __forceinline__ float inv_rms(float m) { return m > 0.f || m != m ? rsqrtf(m) : 0.f; }

// Whether a row's mean square (with eps) overflowed, or is so small that squares
// may have been lost: below 2^-90 they come near fp32's smallest number.
__device__ __forceinline__ bool lost_squares(float m) { return !(m >= 0x1p-90f && m < INFINITY); }
// The power of two that brings such a row's largest magnitude, or the root of eps,
// near 1; 1 for a row that has none (infinities, NaN).
__device__ __forceinline__ float row_scale(float top, float eps) {
  if (!(top < INFINITY)) return 1.f;
  auto exponent = [](float x) { return (int)(__float_as_uint(x) >> 23) - 127; };
  const int k = max(exponent(top), eps > 0.f ? exponent(eps) / 2 : -126);
  return __uint_as_float((uint32_t)(127 - min(max(k, -126), 126)) << 23);
}

// V quotients as 8-bit values, n of them to memory.
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t* p, int n, bool wide, const float (&y)[8]) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  if (wide && n >= V) {
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (k < n) p[k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
  }
}

// A thread's vectors of a row. Whole ones are read by predicated instructions,
// all of them before any value is looked at; the rest (the row's last elements,
// rows that are not aligned) follows one element after another.
template <typename T, int VPT, bool kWhole>
__device__ __forceinline__ void read_vecs(const T* row, int lane, int lanes, int d, bool wide, Vec<T> (&v)[VPT]) {
  constexpr int V = Vec<T>::n;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * lanes + lane) * V;
    if constexpr (kWhole) {
      v[i].v = *reinterpret_cast<const uint4*>(row + c);
    } else {
      v[i].v = make_uint4(0, 0, 0, 0);
      asm volatile(
          "{\n .reg .pred p;\n setp.ne.s32 p, %5, 0;\n @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
          : "+r"(v[i].v.x), "+r"(v[i].v.y), "+r"(v[i].v.z), "+r"(v[i].v.w)
          : "l"(row + c), "r"((int)(wide && c + V <= d)));
    }
  }
  if (!kWhole && (!wide || d % V != 0)) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * lanes + lane) * V;
      if (c < d && !(wide && c + V <= d)) v[i] = load_vec(row + c, d - c, false);
    }
  }
}

// V weights of a row's piece at column c.
template <bool kWhole, int V>
__device__ __forceinline__ void weights(const float* w, int c, int d, float (&f)[V]) {
  if constexpr (kWhole) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(w + c + j);
      f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = w[min(c + j, d - 1)];  // nothing behind the row's end is kept
  }
}

// R tokens of a head beside one another, each by the same threads. kWhole:
// every vector of every thread is a whole one of the row's (see read_row).
template <typename T, int VPT, int R, bool kWhole>
__device__ __forceinline__ void norm_rows(const NormArgs& a, int lanes, float* red) {
  constexpr int V = Vec<T>::n;
  const int lane = threadIdx.x % lanes, groups = (a.T + R - 1) / R;
  const int64_t all = (int64_t)a.B * a.H * groups;
  const int64_t g = (int64_t)blockIdx.x * (blockDim.x / lanes) + threadIdx.x / lanes;
  const RowAt at = row_at(min(g, all - 1), a.H, groups);
  const int t0 = at.t * R, n = g < all ? min(R, a.T - t0) : 0;  // tokens that are this thread's
  const T* x = static_cast<const T*>(a.x.p) + at.b * a.x.sb + at.h * a.x.sh;
  const float* w = a.w + at.h * a.w_sh;
  float s[R][VPT][V];
  Vec<T> xv[R][VPT];
#pragma unroll
  for (int k = 0; k < R; ++k)
    read_vecs<T, VPT, kWhole>(x + min(t0 + k, a.T - 1) * a.x.st, lane, lanes, a.d, a.wide, xv[k]);
  if (a.r.p) {
    const T* res = static_cast<const T*>(a.r.p) + at.b * a.r.sb + at.h * a.r.sh;
    Vec<T> rv[R][VPT];
#pragma unroll
    for (int k = 0; k < R; ++k)
      read_vecs<T, VPT, kWhole>(res + min(t0 + k, a.T - 1) * a.r.st, lane, lanes, a.d, a.wide, rv[k]);
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float q[V];
        unpack<T>(xv[k][i], s[k][i]);
        unpack<T>(rv[k][i], q);
#pragma unroll
        for (int j = 0; j < V; ++j) s[k][i][j] += q[j];
      }
  } else {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < VPT; ++i) unpack<T>(xv[k][i], s[k][i]);
  }
  float sum[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    sum[k] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) sum[k] = fmaf(s[k][i][j], s[k][i][j], sum[k]);
  }
  if (a.rout.p) {
    T* ro = static_cast<T*>(a.rout.p) + at.b * a.rout.sb + at.h * a.rout.sh;
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * lanes + lane) * V;
        if (k < n) write_row<kWhole, T, V>(ro + (t0 + k) * a.rout.st + c, a.d - c, a.wide, s[k][i]);
      }
  }
  row_reduce<false>(sum, lanes, red);
  float m[R];  // mean square and eps
  bool lost = false;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    m[k] = sum[k] / (float)a.d + a.eps;
    lost |= lost_squares(m[k]);
  }
  if (__any_sync(0xffffffffu, lost)) {  // rare; a row's threads agree
    float top[R], by[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      top[k] = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) top[k] = join<true>(top[k], fabsf(s[k][i][j]));
    }
    row_reduce<true>(top, lanes, red);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      by[k] = lost_squares(m[k]) ? row_scale(top[k], a.eps) : 1.f;
      sum[k] = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          s[k][i][j] *= by[k];
          sum[k] = fmaf(s[k][i][j], s[k][i][j], sum[k]);
        }
    }
    row_reduce<false>(sum, lanes, red);
#pragma unroll
    for (int k = 0; k < R; ++k) m[k] = sum[k] / (float)a.d + a.eps * by[k] * by[k];
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float f[V];
    weights<kWhole, V>(w, (i * lanes + lane) * V, a.d, f);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float rs = inv_rms(m[k]);
#pragma unroll
      for (int j = 0; j < V; ++j) s[k][i][j] = s[k][i][j] * rs * f[j];
    }
  }
  if (!a.scale) {
    T* o = static_cast<T*>(a.out.p) + at.b * a.out.sb + at.h * a.out.sh;
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * lanes + lane) * V;
        if (k < n) write_row<kWhole, T, V>(o + (t0 + k) * a.out.st + c, a.d - c, a.wide, s[k][i]);
      }
    return;
  }
  float top[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    top[k] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) top[k] = join<true>(top[k], fabsf(s[k][i][j]));
  }
  row_reduce<true>(top, lanes, red);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (k >= n) break;
    const float scale = top[k] / 448.f;
    if (lane == 0) a.scale[at.b * a.sc_sb + at.h * a.sc_sh + (t0 + k) * a.sc_st] = scale;
    // The fp32 quotient, as a division rounds it: s / scale by the reciprocal is an
    // fp32 step off at times, and next to the middle between two 8-bit values that
    // step decides; the remainder (exact in an fma) puts it right. Scales whose
    // remainders would leave fp32's range keep the division.
    const float inv = 1.f / scale;
    const bool divide = !(scale >= 1e-28f && scale < INFINITY);
    uint8_t* o = static_cast<uint8_t*>(a.out.p) + at.b * a.out.sb + at.h * a.out.sh + (t0 + k) * a.out.st;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * lanes + lane) * V;
      float y[8];
      if (divide) {
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = scale == 0.f ? s[k][i][j] : s[k][i][j] / scale;
      } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const f2 v = mk2(s[k][i][j], s[k][i][j + 1]), q = mul2(v, mk2(inv, inv));
          un2(fma2(fma2(q, mk2(-scale, -scale), v), mk2(inv, inv), q), y[j], y[j + 1]);
        }
      }
      store_e4m3<V>(o + c, kWhole ? V : a.d - c, kWhole || a.wide, y);
    }
  }
}

// Whether every thread's vectors are whole ones of the row's.
template <typename T>
__host__ __device__ __forceinline__ bool whole_rows(bool wide, int d, int lanes, int vpt) {
  return wide && d == lanes * vpt * Vec<T>::n;
}

template <typename T, int VPT, int R>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_fwd_kernel(const __grid_constant__ NormArgs a, int lanes) {
  __shared__ float red[32];
  if (whole_rows<T>(a.wide, a.d, lanes, VPT)) norm_rows<T, VPT, R, true>(a, lanes, red);
  else norm_rows<T, VPT, R, false>(a, lanes, red);
}

// Rows of one weight: all of them, or those of head blockIdx.y. Every block
// walks rows worker, worker + workers, ... , reading the next row while it works
// on one, and keeps its share of dweight in registers; the shares go to
// ws[block][d padded to the row's vectors].
template <typename T, int VPT, bool kWhole>
__device__ __forceinline__ void norm_back(const NormBwdArgs& a, int lanes, int64_t rows, int cols, float* share,
                                          float* red) {
  constexpr int V = Vec<T>::n;
  const int lane = threadIdx.x % lanes, sub = threadIdx.x / lanes, subs = blockDim.x / lanes;
  const int64_t workers = (int64_t)gridDim.x * subs;
  const int head = blockIdx.y;
  // long rows leave no registers for the weights and the next row
  constexpr bool kAhead = VPT * V <= 16;
  const float* wp = a.w + head * a.w_sh;
  float w[kAhead ? VPT : 1][V], dw[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (kAhead) weights<kWhole, V>(wp, (i * lanes + lane) * V, a.d, w[kAhead ? i : 0]);
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
  }
  // every thread of a block makes the same number of turns (row_reduce synchronises)
  const int64_t turns = (rows + workers - 1) / workers;
  Vec<T> hv[VPT], gv[VPT], rv[VPT];
  RowAt at = {0, 0, 0}, ahead = {0, 0, 0};
  auto fetch = [&](int64_t k) {
    const int64_t r = min(k * workers + (int64_t)blockIdx.x * subs + sub, rows - 1);
    if (a.w_sh) {
      ahead = row_at(r, 1, a.T);
      ahead.h = head;
    } else {
      ahead = row_at(r, a.H, a.T);
    }
    const T* hp = static_cast<const T*>(a.h.p) + ahead.b * a.h.sb + ahead.h * a.h.sh + ahead.t * a.h.st;
    const T* gp = static_cast<const T*>(a.dy.p) + ahead.b * a.dy.sb + ahead.h * a.dy.sh + ahead.t * a.dy.st;
    // without it the gradient stands in its place and is not used
    const T* rp = a.dres.p ? static_cast<const T*>(a.dres.p) + ahead.b * a.dres.sb + ahead.h * a.dres.sh + ahead.t * a.dres.st
                           : gp;
    read_vecs<T, VPT, kWhole>(hp, lane, lanes, a.d, a.wide, hv);
    read_vecs<T, VPT, kWhole>(gp, lane, lanes, a.d, a.wide, gv);
    read_vecs<T, VPT, kWhole>(rp, lane, lanes, a.d, a.wide, rv);
  };
  if (kAhead && turns > 0) fetch(0);
  for (int64_t k = 0; k < turns; ++k) {
    const bool live = k * workers + (int64_t)blockIdx.x * subs + sub < rows;
    if (!kAhead) fetch(k);
    at = ahead;
    float h[VPT][V], g[VPT][V];
    Vec<T> res[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack<T>(hv[i], h[i]);
      unpack<T>(gv[i], g[i]);
      res[i] = rv[i];
    }
    if (kAhead && k + 1 < turns) fetch(k + 1);
    float sums[2] = {0.f, 0.f};  // of h^2 and of dy w h
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float(&f)[V] = w[kAhead ? i : 0];
      if (!kAhead) weights<kWhole, V>(wp, (i * lanes + lane) * V, a.d, f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sums[0] = fmaf(h[i][j], h[i][j], sums[0]);
        sums[1] = fmaf(g[i][j] * f[j], h[i][j], sums[1]);
      }
    }
    row_reduce<false>(sums, lanes, red);
    float ms = sums[0] / (float)a.d + a.eps, by = 1.f;  // mean square; what the row is multiplied with
    if (__any_sync(0xffffffffu, lost_squares(ms))) {  // rare; a row's threads agree
      float top[1] = {0.f};
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) top[0] = join<true>(top[0], fabsf(h[i][j]));
      row_reduce<true>(top, lanes, red);
      if (lost_squares(ms)) by = row_scale(top[0], a.eps);
      sums[0] = sums[1] = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float(&f)[V] = w[kAhead ? i : 0];
        if (!kAhead) weights<kWhole, V>(wp, (i * lanes + lane) * V, a.d, f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          h[i][j] *= by;
          sums[0] = fmaf(h[i][j], h[i][j], sums[0]);
          sums[1] = fmaf(g[i][j] * f[j], h[i][j], sums[1]);
        }
      }
      row_reduce<false>(sums, lanes, red);
      ms = sums[0] / (float)a.d + a.eps * by * by;
    }
    const float rn = inv_rms(ms), rs = rn * by;  // of the row in registers, of h
    const float m = sums[1] / (float)a.d * rn * rn;
    if (!live) continue;  // the block's last turn
    T* op = static_cast<T*>(a.dh.p) + at.b * a.dh.sb + at.h * a.dh.sh + at.t * a.dh.st;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * lanes + lane) * V;
      float(&f)[V] = w[kAhead ? i : 0];
      if (!kAhead) weights<kWhole, V>(wp, c, a.d, f);
      float o[V];
      unpack<T>(res[i], o);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        dw[i][j] = fmaf(g[i][j], h[i][j] * rn, dw[i][j]);
        o[j] = fmaf(rs, fmaf(g[i][j], f[j], -h[i][j] * m), a.dres.p ? o[j] : 0.f);
      }
      write_row<kWhole, T, V>(op + c, a.d - c, a.wide, o);
    }
  }
  float* dst = a.ws + ((int64_t)blockIdx.x * gridDim.y + head) * cols;
  if (subs == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < V; j += 4)
        *reinterpret_cast<float4*>(dst + (i * lanes + lane) * V + j) =
            make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
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

template <typename T, int VPT>
__global__ void __launch_bounds__(kMaxThreads, 1)
    norm_bwd_kernel(const __grid_constant__ NormBwdArgs a, int lanes, int64_t rows, int cols) {
  extern __shared__ float share[];  // [rows a block][cols]
  __shared__ float red[32];
  if (whole_rows<T>(a.wide, a.d, lanes, VPT)) norm_back<T, VPT, true>(a, lanes, rows, cols, share, red);
  else norm_back<T, VPT, false>(a, lanes, rows, cols, share, red);
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
  const int64_t cap = (int64_t)148 * (512 / p.block) / (a.w_sh ? a.H : 1);
  return (int)(want < 1 ? 1 : want < cap ? want : cap < 1 ? 1 : cap);
}

// Short rows (a vector a thread) go four tokens a thread: their places and
// weights are found once, and four loads are in flight.
constexpr int kShortRows = 4;
// A warp a row, without barriers, up to 256 vectors: B4 T4096 d2048 with 8-bit
// output takes 43 us (5.4 TB/s), a block of 128 threads a row 59 us. Wider rows do not fit
// a warp's registers and take a block each: as many elements in rows of 4096 68 us, in rows
// of 8192 100 us. The backward pass has no registers for it beside its share of dweight.
constexpr int kFwdVpt = 8;

template <typename T>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
  const RowPlan p = plan_rows<T>(a.d, kFwdVpt);
  const int R = p.vpt == 1 && a.T >= kShortRows ? kShortRows : 1;
  const int64_t groups = (int64_t)a.B * a.H * ((a.T + R - 1) / R), per = p.block / p.lanes;
  const int64_t blocks = (groups + per - 1) / per;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)blocks), b(p.block);
  if (R > 1) norm_fwd_kernel<T, 1, kShortRows><<<g, b, 0, s>>>(a, p.lanes);
  else if (p.vpt == 1) norm_fwd_kernel<T, 1, 1><<<g, b, 0, s>>>(a, p.lanes);
  else if (p.vpt == 2) norm_fwd_kernel<T, 2, 1><<<g, b, 0, s>>>(a, p.lanes);
  else if (p.vpt == 4) norm_fwd_kernel<T, 4, 1><<<g, b, 0, s>>>(a, p.lanes);
  else norm_fwd_kernel<T, 8, 1><<<g, b, 0, s>>>(a, p.lanes);
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
