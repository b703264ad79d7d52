// What the selective scan's forward and backward kernels share.
#pragma once

#include "block.cuh"

namespace ttt {
namespace scan {

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
// 2^x; denormal results are 0.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f2 ex2_pair(f2 x) {
  float a, b;
  un2(x, a, b);
  return mk2(ex2(a), ex2(b));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kNB = 16;  // states a warp holds

// Step size from its raw value, and the derivative of the one by the other.
__device__ __forceinline__ float step_of(float raw, int softplus) {
  return softplus ? softplus_f(raw) : raw;
}

// Where a token stands in its sequence.
struct TokenAt {
  int seq, lo, hi;
  bool live;
};
__device__ __forceinline__ TokenAt token_at(const Seqs& q, int b, int T, int t, int* status) {
  if (!q.cu) return {b, 0, T, t < T};
  TokenAt r = {first_seq_behind(q.cu, q.S, t), 0, 0, false};
  if (t < T && r.seq < q.S) {
    packed_seq(q.cu, r.seq, T, status, &r.lo, &r.hi);
    r.live = t >= r.lo && t < r.hi;
  }
  return r;
}

// dst (may be null) = src (zeros where null) for every sequence without a
// token: the states and their gradients that no kernel of the scan reaches. It
// also sees every offset of a packed call and reports the ones out of order.
cudaError_t copy_empty_states(const Seqs& q, int T, int64_t n, const float* src, float* dst,
                              int* status, cudaStream_t s);

}  // namespace scan
}  // namespace ttt
