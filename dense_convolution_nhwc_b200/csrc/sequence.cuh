// sequence.cuh -- what the sequence operators (causal conv1d, selective scan)
// share: where a call's sequences lie, vector loads of any alignment, and the
// logistic functions in fp32.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace b200conv {

constexpr float kLog2e = 1.4426950408889634f;

// Row range of sequence `seq` in a packed call.  Offsets come from device memory
// and are not trusted: both ends are clamped to [0, rows], so a bad list gives
// unspecified rows and never an access outside the tensors.
__device__ __forceinline__ void packed_range(const int* offsets, int seq, int rows, int* lo, int* hi) {
  const int a = min(max(__ldg(offsets + seq), 0), rows);
  const int b = min(max(__ldg(offsets + seq + 1), a), rows);
  *lo = a;
  *hi = b;
}

// The cache slot of sequence `seq`, or -1 for a sequence to leave out.
__device__ __forceinline__ int slot_of(const int* slots, int seq, int state_slots) {
  if (!slots) return seq;
  const int v = __ldg(slots + seq);
  return (unsigned)v < (unsigned)state_slots ? v : -1;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int N>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src));
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst)), "l"(src), "n"(N));
}

// V elements as fp32.  VEC: one aligned access of V * sizeof(T) bytes (16 at
// most); else V accesses of one element.
template <typename T, int V, bool VEC>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[V]) {
  if constexpr (VEC && V * sizeof(T) == 16) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = Store<T>::to_f32(e[i]);
  } else if constexpr (VEC && V * sizeof(T) == 8) {
    const uint2 raw = *reinterpret_cast<const uint2*>(p);
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = Store<T>::to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = Store<T>::to_f32(p[i]);
  }
}

template <typename T, int V, bool VEC>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[V]) {
  if constexpr (VEC && sizeof(T) == 2 && V == 8) {
    uint4 raw;
    raw.x = pack2<T>(v[0], v[1]);
    raw.y = pack2<T>(v[2], v[3]);
    raw.z = pack2<T>(v[4], v[5]);
    raw.w = pack2<T>(v[6], v[7]);
    *reinterpret_cast<uint4*>(p) = raw;
  } else if constexpr (VEC && sizeof(T) == 2 && V == 4) {
    uint2 raw;
    raw.x = pack2<T>(v[0], v[1]);
    raw.y = pack2<T>(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = raw;
  } else if constexpr (VEC && sizeof(T) == 4 && V == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = Store<T>::from_f32(v[i]);
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// ex2's results lie 0.1 to 0.4 u (u = 2^-24) below the true values on average for
// arguments in (-1, 0), as measured over 65536 arguments a decade.  Over the many
// tokens a slowly decaying state remembers that adds up where roundings to both
// sides do not, so decays are taken at an argument 0.3 u / ln 2 higher.
constexpr float kEx2Bias = 0.3f / 16777216.0f * kLog2e;
// exp(a delta), one of the two times log2(e).
__device__ __forceinline__ float decay(float a, float delta) { return ex2(fmaf(a, delta, kEx2Bias)); }
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// v / (1 + exp(-v)); -inf gives NaN as the quotient does.  From v = -87.3 down the reciprocal
// and then exp(-v) leave fp32's range while the quotient is in it (a normal number to
// -91.9).  So the exponential comes as the square of that of half the argument, and is
// added to 1 as 2^-32 of itself, which keeps the reciprocal in range down to -109.  The
// sigmoid itself is then below 2^-126 and a multiple of 2^-149: the result is off by up to
// |v| 2^-150 more.  (A test for low values in its place: scans of 16 sequences of 512
// tokens 246 us, 240 so.)
__device__ __forceinline__ float silu(float v) {
  const float h = ex2(-0.5f * kLog2e * v);
  return v * (rcp(fmaf(h * 0x1p-32f, h, 0x1p-32f)) * 0x1p-32f);
}
// Of two values, the arithmetic between the special functions packed.
__device__ __forceinline__ float2 silu(float2 v) {
  auto c = [](float k) { return make_float2(k, k); };
  const float2 arg = __fmul2_rn(v, c(-0.5f * kLog2e));
  const float2 h = make_float2(ex2(arg.x), ex2(arg.y));
  const float2 low = __ffma2_rn(__fmul2_rn(h, c(0x1p-32f)), h, c(0x1p-32f));
  return __fmul2_rn(v, __fmul2_rn(make_float2(rcp(low.x), rcp(low.y)), c(0x1p-32f)));
}

// The same above kFar alone, for a kernel bound by the way from a sum to its output: it
// looks for sums further out with `lowest` and puts those outputs right afterwards with
// silu_far.  There 1 + exp(-v) is exp(-v) to 2^-115 and the quotient v exp(v), its
// exponential taken 2^32 times as large so that only the last product is below 2^-126.
// (A convolution of 50 us takes 56 with the form above, or with a test before the store;
// one by single elements, 4096 rows of 4092, 28 in place of 26.)
constexpr float kFar = -80.0f;
__device__ __forceinline__ float silu_far(float v) { return v * ex2(fmaf(v, kLog2e, 32.0f)) * 0x1p-32f; }
__device__ __forceinline__ float silu_near(float v) { return v * rcp(1.0f + ex2(-kLog2e * v)); }
__device__ __forceinline__ float2 silu_near(float2 v) {
  const float2 arg = __fmul2_rn(v, make_float2(-kLog2e, -kLog2e));
  const float2 low = __fadd2_rn(make_float2(ex2(arg.x), ex2(arg.y)), make_float2(1.0f, 1.0f));
  return __fmul2_rn(v, make_float2(rcp(low.x), rcp(low.y)));
}
template <int V>
__device__ __forceinline__ float lowest(const float (&v)[V], float so_far) {
#pragma unroll
  for (int i = 0; i < V; ++i) so_far = fminf(so_far, v[i]);
  return so_far;
}

// log(1 + exp(v)) = max(v, 0) + log1p(t), t = exp(-|v|) in (0, 1].  A logarithm of
// 1 + t would lose t's low bits where the result is small (v << 0, the usual
// case), so log1p(t) = 2 artanh(s), s = t / (2 + t) <= 1/3, and artanh(s) / s is a
// polynomial in s^2, fitted over [0, 1/9] for the least largest relative error
// (8e-9 with its coefficients in fp32; its Taylor series takes three terms more).
// Results below 2^-126 (v < -87.3) are zero.
__device__ __forceinline__ float2 softplus(float2 v) {
  const float2 t = make_float2(ex2(-kLog2e * fabsf(v.x)), ex2(-kLog2e * fabsf(v.y)));
  const float2 low = __fadd2_rn(t, make_float2(2.0f, 2.0f));
  const float2 s = __fmul2_rn(t, make_float2(rcp(low.x), rcp(low.y)));
  const float2 q = __fmul2_rn(s, s);
  auto c = [](float k) { return make_float2(k, k); };
  float2 r = __ffma2_rn(q, c(0.14089164f), c(0.13980296f));
  r = __ffma2_rn(q, r, c(0.20012456f));
  r = __ffma2_rn(q, r, c(0.33333158f));
  r = __ffma2_rn(q, r, c(1.0f));
  // fmaxf drops a NaN; t carries it
  return __ffma2_rn(__fadd2_rn(s, s), r, make_float2(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
}
__device__ __forceinline__ float softplus(float v) { return softplus(make_float2(v, v)).x; }

}  // namespace b200conv
