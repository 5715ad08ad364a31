// tbe_two.cuh -- two-wide fp32 arithmetic and approximate functions, for the
// kernels that are bound by the number of instructions they issue.
#pragma once

#include <stdint.h>

namespace tbe {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float root(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inv_root(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger one, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two fp32 numbers in one register pair: one instruction for both.
struct Two {
  float2 v;
};
__device__ __forceinline__ Two two(float a, float b) { return Two{make_float2(a, b)}; }
__device__ __forceinline__ Two two(float a) { return two(a, a); }
__device__ __forceinline__ float lo(Two t) { return t.v.x; }
__device__ __forceinline__ float hi(Two t) { return t.v.y; }
__device__ __forceinline__ Two operator*(Two a, Two b) { return Two{__fmul2_rn(a.v, b.v)}; }
__device__ __forceinline__ Two operator+(Two a, Two b) { return Two{__fadd2_rn(a.v, b.v)}; }
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) { return Two{__ffma2_rn(a.v, b.v, c.v)}; }
__device__ __forceinline__ Two ex2(Two a) { return two(ex2(lo(a)), ex2(hi(a))); }
__device__ __forceinline__ Two rcp(Two a) { return two(rcp(lo(a)), rcp(hi(a))); }
__device__ __forceinline__ Two root(Two a) { return two(root(lo(a)), root(hi(a))); }
__device__ __forceinline__ Two inv_root(Two a) { return two(inv_root(lo(a)), inv_root(hi(a))); }
__device__ __forceinline__ Two negative(Two t) { return two(-lo(t), -hi(t)); }

// A constant made once per thread: two-wide instructions take their operands
// from registers only, and the compiler would otherwise move a constant there
// again at each use.
__device__ __forceinline__ Two keep(float f) {
  Two t = two(f);
  asm volatile("" : "+f"(t.v.x), "+f"(t.v.y));
  return t;
}

}  // namespace tbe
