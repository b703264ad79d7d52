// Arguments and shared device code of the recurrent block's operators: RMS
// norm, short causal convolution, selective scan (see include/ttt.h).
#pragma once

#include "common.cuh"

namespace ttt {

// ---- host-side arguments ------------------------------------------------------

struct RowsView {  // like TokView, also for 8-bit elements
  void* p;
  int64_t sb, sh, st;
};

struct NormArgs {
  TokView x, r;            // r.p null: no residual
  const float* w;
  int64_t w_sh;            // 0: one weight for all heads
  float eps;
  RowsView out, rout;      // rout.p null: the sum is not wanted
  float* scale;            // non-null: out is e4m3
  int64_t sc_sb, sc_sh, sc_st;
  int B, H, T, d;
  bool wide;               // token rows are 16-byte aligned, and so is the weight's every row
};
cudaError_t launch_rms_norm_fwd(const NormArgs& a, bool bf16, cudaStream_t s);

struct NormBwdArgs {
  TokView h, dy, dres;     // dres.p null: none
  const float* w;
  int64_t w_sh;
  float eps;
  TokViewMut dh;
  float* dw;
  float* ws;
  int B, H, T, d;
  bool wide;
};
size_t rms_norm_bwd_workspace(const NormBwdArgs& a, bool bf16);
cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, bool bf16, cudaStream_t s);

// A call's sequences: S packed ones (cu non-null, B = 1), or B of T tokens.
struct Seqs {
  const int32_t* cu;
  int S;
};

struct ConvArgs {
  TokView x, state0;       // state0.p null: zeros
  const float *w, *bias;   // bias may be null
  Seqs seqs;
  RowsView out, fin;       // fin.p null: not wanted
  int B, H, T, d, K, silu;
  bool wide;
  int* status;
};
cudaError_t launch_causal_conv_fwd(const ConvArgs& a, bool bf16, cudaStream_t s);

struct ConvBwdArgs {
  TokView x, state0, dy, dfin;
  const float *w, *bias;
  Seqs seqs;
  TokViewMut dx, dstate0;  // dstate0.p null: not wanted
  float *dw, *dbias;       // dbias may be null
  float* ws;
  int B, H, T, d, K, silu;
  bool wide;
  int* status;
};
size_t causal_conv_bwd_workspace(const ConvBwdArgs& a, bool bf16);
cudaError_t launch_causal_conv_bwd(const ConvBwdArgs& a, bool bf16, cudaStream_t s);

struct ConvStepArgs {
  TokView x;
  TokViewMut state, out;
  const int32_t* slots;    // may be null
  const float *w, *bias;
  int B, S, H, d, K, silu;
  bool wide;
  int* status;
};
cudaError_t launch_causal_conv_step(const ConvStepArgs& a, bool bf16, cudaStream_t s);

struct ScanArgs {
  TokView x, dt, z, Bm, Cm;   // z.p may be null; Bm, Cm: sh is the group stride
  const float *A, *D, *dt_bias, *h0;   // D, dt_bias, h0 may be null
  Seqs seqs;
  TokViewMut out;
  float* h_final;          // may be null
  float* ws;
  int B, H, T, d, N, G, softplus;
  bool wide;
  int* status;
};
size_t selective_scan_workspace(const ScanArgs& a);
cudaError_t launch_selective_scan_fwd(const ScanArgs& a, bool bf16, cudaStream_t s);

struct ScanBwdArgs {
  ScanArgs f;              // the forward's inputs (out, h_final, ws unused)
  TokView dy;
  const float* dh_final;   // may be null
  TokViewMut dx, ddt, dz, dBm, dCm;   // dz.p may be null
  float *dA, *dD, *ddt_bias, *dh0;    // all but dA may be null
  float* ws;
};
size_t selective_scan_bwd_workspace(const ScanBwdArgs& a);
cudaError_t launch_selective_scan_bwd(const ScanBwdArgs& a, bool bf16, cudaStream_t s);

struct ScanStepArgs {
  TokView x, dt, z, Bm, Cm;
  const float *A, *D, *dt_bias;
  float* state;
  const int32_t* slots;
  TokViewMut out;
  int B, S, H, d, N, G, softplus;
  bool wide;               // state and A are 16-byte aligned
  bool rows_wide;          // and so are the token rows
  int* status;
};
cudaError_t launch_selective_scan_step(const ScanStepArgs& a, bool bf16, cudaStream_t s);

// ---- device code --------------------------------------------------------------

// 16 bytes of a token row: 8 bf16 or 4 fp32 channels.
template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
  uint4 v;
};

template <typename T>
__device__ __forceinline__ void unpack(const Vec<T>& a, float (&f)[Vec<T>::n]);
template <>
__device__ __forceinline__ void unpack<float>(const Vec<float>& a, float (&f)[4]) {
  f[0] = __uint_as_float(a.v.x);
  f[1] = __uint_as_float(a.v.y);
  f[2] = __uint_as_float(a.v.z);
  f[3] = __uint_as_float(a.v.w);
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const Vec<__nv_bfloat16>& a, float (&f)[8]) {
  const uint32_t w[4] = {a.v.x, a.v.y, a.v.z, a.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its fp32
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ Vec<T> pack(const float (&f)[Vec<T>::n]);
template <>
__device__ __forceinline__ Vec<float> pack<float>(const float (&f)[4]) {
  return {make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3]))};
}
template <>
__device__ __forceinline__ Vec<__nv_bfloat16> pack<__nv_bfloat16>(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return {make_uint4(w[0], w[1], w[2], w[3])};
}

// The first `n` elements (n may be <= 0) of the row piece at p; the rest reads
// as zero. A piece that ends inside the vector is read element by element, so
// that nothing behind the row's end is touched, and so is every piece where
// the call's rows are not all 16-byte aligned (wide is false).
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p, int n, bool wide) {
  Vec<T> r;
  if (wide && n >= Vec<T>::n) {
    r.v = *reinterpret_cast<const uint4*>(p);
  } else {
    float f[Vec<T>::n];
#pragma unroll
    for (int i = 0; i < Vec<T>::n; ++i) f[i] = i < n ? to_f32(p[i]) : 0.f;
    r = pack<T>(f);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, int n, bool wide, const float (&f)[Vec<T>::n]) {
  if (wide && n >= Vec<T>::n) {
    *reinterpret_cast<uint4*>(p) = pack<T>(f).v;
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::n; ++i)
      if (i < n) p[i] = from_f32<T>(f[i]);
  }
}

// V channels of a token row, in fp32: 16 bytes of bf16 (V = 8) or fp32 (V = 4),
// or 8 bytes of bf16 (V = 4).
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* p, int n, bool wide, float (&f)[V]) {
  if constexpr (V * sizeof(T) == 16) {
    unpack<T>(load_vec(p, n, wide), f);
  } else {
    if (wide && n >= V) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      f[0] = __uint_as_float(v.x << 16);
      f[1] = __uint_as_float(v.x & 0xffff0000u);
      f[2] = __uint_as_float(v.y << 16);
      f[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = i < n ? to_f32(p[i]) : 0.f;
    }
  }
}
// kWhole: the piece is known to be aligned and whole. Loads without a choice
// stay in flight beside one another; behind a choice each is waited for where
// its two ways meet. Kernels choose once for all of a block's loads.
template <bool kWhole, typename T, int V>
__device__ __forceinline__ void read_row(const T* p, int n, bool wide, float (&f)[V]) {
  if constexpr (kWhole) load_row<T, V>(p, V, true, f);
  else load_row<T, V>(p, n, wide, f);
}
template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, int n, bool wide, const float (&f)[V]) {
  if constexpr (V * sizeof(T) == 16) {
    store_vec<T>(p, n, wide, f);
  } else {
    if (wide && n >= V) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
      *reinterpret_cast<uint2*>(p) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) p[i] = from_f32<T>(f[i]);
    }
  }
}

template <bool kWhole, typename T, int V>
__device__ __forceinline__ void write_row(T* p, int n, bool wide, const float (&f)[V]) {
  if constexpr (kWhole) store_row<T, V>(p, V, true, f);
  else store_row<T, V>(p, n, wide, f);
}

// Asynchronous copy of a row piece of 16 bytes into shared memory: the first n
// elements, zeros behind them (n <= 0: zeros, nothing is read). Rows that are
// not 16-byte aligned are copied at once, element by element.
template <typename T>
__device__ __forceinline__ void copy_async(T* dst, const T* src, int n, bool wide) {
  constexpr int V = Vec<T>::n;
  n = n < 0 ? 0 : n > V ? V : n;
  if (wide) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"((int)(n * sizeof(T)))
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) dst[i] = i < n ? src[i] : from_f32<T>(0.f);
  }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last kLeft groups of this thread's copies have arrived.
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// 2^x and 1/x by the special-function unit (2^-22 relative); denormal results
// are 0, 1/inf is 0, NaN stays NaN.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_f(float x) { return rcp(1.f + ex2(-kLog2e * x)); }
__device__ __forceinline__ float silu_f(float x) { return x * sigmoid_f(x); }
// d silu / dx = s (1 + x (1 - s)); right of 88 it is 1 in fp32 (inf * 0 is avoided).
__device__ __forceinline__ float dsilu_f(float x) {
  const float s = sigmoid_f(x);
  return x > 88.f ? 1.f : s * fmaf(x, 1.f - s, 1.f);
}
// log(1 + exp(x)) = max(x, 0) + log1p(t), t = exp(-|x|), and log1p(t) = 2 atanh(v)
// with v = t / (2 + t) <= 1/3: an odd series, here its best polynomial of degree 4
// in v^2 (4e-9 relative). Small steps (very negative x) keep their relative
// accuracy, which log(1 + t) would lose.
__device__ __forceinline__ float softplus_f(float x) {
  const float t = ex2(-kLog2e * fabsf(x));
  const float v = t * rcp(2.f + t), w = v * v;
  float p = fmaf(w, 0.14095773f, 0.13978833f);
  p = fmaf(w, p, 0.20012557f);
  p = fmaf(w, p, 0.33333155f);
  p = fmaf(w, p, 1.f);
  return fmaf(v + v, p, fmaxf(x, 0.f));
}

// ---- two fp32 in one 64-bit register (the packed fp32 instructions of sm_100
// do two operations an issue slot) -------------------------------------------

using f2 = unsigned long long;
__device__ __forceinline__ f2 mk2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void un2(f2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 ex2_pair(f2 x) {
  float a, b;
  un2(x, a, b);
  return mk2(ex2(a), ex2(b));
}

// Four channels of a token row as they lie in memory, and as two fp32 pairs.
constexpr int kV = 4;
template <typename T>
struct Raw {
  using type = uint2;
};
template <>
struct Raw<float> {
  using type = uint4;
};
// kWhole: all four exist and are aligned (see read_row).
template <bool kWhole, typename T>
__device__ __forceinline__ typename Raw<T>::type raw_row(const T* p, int n, bool wide) {
  if constexpr (kWhole) {
    return *reinterpret_cast<const typename Raw<T>::type*>(p);
  } else {
    float f[kV];
    load_row<T, kV>(p, n, wide, f);
    if constexpr (sizeof(T) == 4) {
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {  // exact: the values came from bf16
      return make_uint2(__float_as_uint(f[0]) >> 16 | (__float_as_uint(f[1]) & 0xffff0000u),
                        __float_as_uint(f[2]) >> 16 | (__float_as_uint(f[3]) & 0xffff0000u));
    }
  }
}
__device__ __forceinline__ void pairs_of(uint4 r, f2 (&v)[2]) {
  v[0] = mk2(__uint_as_float(r.x), __uint_as_float(r.y));
  v[1] = mk2(__uint_as_float(r.z), __uint_as_float(r.w));
}
__device__ __forceinline__ void pairs_of(uint2 r, f2 (&v)[2]) {
  v[0] = mk2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
  v[1] = mk2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ void floats_of(const f2 (&v)[2], float (&f)[kV]) {
  un2(v[0], f[0], f[1]);
  un2(v[1], f[2], f[3]);
}
__device__ __forceinline__ void pairs_of(const float (&f)[kV], f2 (&v)[2]) {
  v[0] = mk2(f[0], f[1]);
  v[1] = mk2(f[2], f[3]);
}

// The same where a piece may be missing or ragged: first all of a thread's
// reads by predicated instructions (whole: the piece is whole and aligned), so
// that they are in flight together; then raw_rest() for each, which reads the
// pieces that are neither whole nor empty one element after another.
template <typename T>
__device__ __forceinline__ typename Raw<T>::type raw_whole(const T* p, bool whole) {
  typename Raw<T>::type r;
  if constexpr (sizeof(T) == 2) {
    r = make_uint2(0, 0);
    asm volatile("{\n .reg .pred p;\n setp.ne.s32 p, %3, 0;\n @p ld.global.v2.u32 {%0, %1}, [%2];\n}\n"
                 : "+r"(r.x), "+r"(r.y)
                 : "l"(p), "r"((int)whole));
  } else {
    r = make_uint4(0, 0, 0, 0);
    asm volatile("{\n .reg .pred p;\n setp.ne.s32 p, %5, 0;\n @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
                 : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
                 : "l"(p), "r"((int)whole));
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void raw_rest(typename Raw<T>::type& r, const T* p, int n, bool wide) {
  if (n > 0 && !(wide && n >= kV)) r = raw_row<false, T>(p, n, false);
}
__device__ __forceinline__ void floats_of(uint2 r, float (&f)[kV]) {
  f[0] = __uint_as_float(r.x << 16);
  f[1] = __uint_as_float(r.x & 0xffff0000u);
  f[2] = __uint_as_float(r.y << 16);
  f[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void floats_of(uint4 r, float (&f)[kV]) {
  f[0] = __uint_as_float(r.x);
  f[1] = __uint_as_float(r.y);
  f[2] = __uint_as_float(r.z);
  f[3] = __uint_as_float(r.w);
}

// Sequence i of a packed call, its offsets clamped into [0, T]; empty (lo =
// hi) where they decrease or leave the range, which is recorded.
__device__ __forceinline__ void packed_seq(const int32_t* cu, int i, int T, int* status, int* lo,
                                           int* hi) {
  int a = cu[i], b = cu[i + 1];
  if (a < 0 || b < a || b > T) {
    record_error(status, DEV_BOUNDS);
    a = b = 0;
  }
  *lo = a;
  *hi = b;
}

// The first sequence whose end lies behind token t (S if none).
__device__ __forceinline__ int first_seq_behind(const int32_t* cu, int S, int t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// A row's place in a pool of states (slots null: row b has place b), for a
// block that works on row b alone. False: nothing to do here. Rows that name
// one place are all done by the block of the first of them, in row order: it
// calls next_row() after each row until that returns false.
struct SlotRows {
  const int32_t* slots;
  int b, B, slot;
  bool more;
  __device__ __forceinline__ bool begin(const int32_t* s, int row, int rows, int S, int* status) {
    slots = s;
    b = row;
    B = rows;
    slot = s ? s[row] : row;
    more = false;
    if (slot < 0 || slot >= S) {
      if (slot != -1 && threadIdx.x == 0) record_error(status, DEV_BOUNDS);
      return false;
    }
    if (!s) return true;
    int earlier = 0, later = 0;
    for (int i = threadIdx.x; i < B; i += blockDim.x)
      if (s[i] == slot) {
        earlier |= i < b;
        later |= i > b;
      }
    if (__syncthreads_or(earlier)) return false;
    more = __syncthreads_or(later);
    return true;
  }
  __device__ __forceinline__ bool next_row() {
    if (!more) return false;
    __shared__ int s_next;
    __syncthreads();
    if (threadIdx.x == 0) s_next = B;
    __syncthreads();
    for (int i = b + 1 + threadIdx.x; i < B; i += blockDim.x)
      if (slots[i] == slot) {
        atomicMin(&s_next, i);
        break;
      }
    __syncthreads();
    b = s_next;
    return b < B;
  }
};

// out(col, sum over p of ws[p * cols + col]): kRows threads a column, each
// summing every kRows-th part in order, then a fixed tree: the result does not
// depend on scheduling. Few columns go 8 a block (a sector of memory) with 64
// threads each, many (from 16384, where 8 a block would leave blocks too short)
// 32 with 16.
template <int kCols, int kRows, typename Out>
__global__ void __launch_bounds__(kCols * kRows)
    sum_parts_kernel(const float* __restrict__ ws, int64_t parts, int64_t cols, Out out) {
  __shared__ float part[kRows][kCols];
  const int c = threadIdx.x % kCols, r = threadIdx.x / kCols;
  const int64_t col = (int64_t)blockIdx.x * kCols + c;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int64_t p = r; p < parts; p += kRows) s += ws[p * cols + col];
  }
  part[r][c] = s;
  for (int h = kRows / 2; h; h /= 2) {
    __syncthreads();
    if (r < h) part[r][c] += part[r + h][c];
  }
  if (r == 0 && col < cols) out(col, part[0][c]);
}
template <typename Out>
cudaError_t sum_parts(const float* ws, int64_t parts, int64_t cols, Out out, cudaStream_t s) {
  if (cols < 16384)
    sum_parts_kernel<8, 64><<<(unsigned)((cols + 7) / 8), 512, 0, s>>>(ws, parts, cols, out);
  else
    sum_parts_kernel<32, 16><<<(unsigned)((cols + 31) / 32), 512, 0, s>>>(ws, parts, cols, out);
  return cudaGetLastError();
}

}  // namespace ttt
