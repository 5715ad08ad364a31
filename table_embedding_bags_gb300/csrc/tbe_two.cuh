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

// Two fp32 numbers in one register pair: one instruction for both.
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two t;
  asm("mov.b64 %0, {%1, %2};" : "=l"(t.v) : "f"(a), "f"(b));
  return t;
}
__device__ __forceinline__ Two two(float a) { return two(a, a); }
__device__ __forceinline__ float lo(Two t) {
  return __uint_as_float((uint32_t)t.v);
}
__device__ __forceinline__ float hi(Two t) {
  return __uint_as_float((uint32_t)(t.v >> 32));
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  Two t;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t.v) : "l"(a.v), "l"(b.v));
  return t;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two t;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(t.v) : "l"(a.v), "l"(b.v));
  return t;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two t;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return t;
}
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
  asm volatile("" : "+l"(t.v));
  return t;
}

}  // namespace tbe
