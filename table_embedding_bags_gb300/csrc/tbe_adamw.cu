// tbe_adamw.cu -- one AdamW step over a list of dense tensors in one launch.
//
//   m <- beta1 m + (1 - beta1) g            v <- beta2 v + (1 - beta2) g^2
//   w <- (1 - lr wd) w - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
//
// States live in one flat buffer per moment, cut into blocks of 256 elements;
// every tensor's states start on a block.  A warp owns a block at a time, so
// a block's largest magnitude (the scale of its 8-bit codes) is one warp
// reduction and nothing is shared between warps.
//
// 8-bit states: m = sign(q) (q / 127)^2 s, v = (q / 255)^4 s with s the
// block's largest magnitude.  Both put the codes evenly in the root of what
// the step uses (m and sqrt(v)), so that small moments keep relative
// precision: 0.8 % at the top, 16,000 : 1 between the largest and the
// smallest.  A moment takes the code whose root is nearest; a second moment
// that is not zero keeps a code of at least 1, because the step divides by it.
// The moments are computed with one rounding per operation (no contraction
// into fused multiply-adds), so that codes do not depend on how the compiler
// groups operations.
//
// What bounds it: 32-bit states, memory: 200 M half-precision parameters and
// gradients, 22 bytes each, 632 us (7.0 TB/s).  8-bit states, instructions: 64
// M elements, 10 bytes each, 136 us (4.3 TB/s, 60 instructions per element at
// 73 % of issue slots; with fp32 parameters and gradients, 16 bytes, 1.4 times
// that); the states' values written out 94 us (6.2 TB/s).  A list of small
// tensors, the launch: 4.9 us.
#include "tbe_internal.cuh"
#include "tbe_two.cuh"

#include <cmath>
#include <cstring>
#include <new>

namespace tbe {
namespace {

constexpr int kBlock = TBE_ADAMW_BLOCK;  // elements of a state block
constexpr int kPer = kBlock / 32;        // elements of a block per lane
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kTiny = 1.17549435e-38f;  // smallest normal fp32

struct __align__(16) TensorMeta {
  void* p;
  const void* g;
  int64_t numel;
  int32_t block0;  // first state block
  uint8_t pdt, gdt;
  uint8_t vec;  // parameters and gradients may be read and written eight elements at a time
  uint8_t pad;
};
static_assert(sizeof(TensorMeta) == 32, "TensorMeta must stay 32 bytes");

struct StepArgs {
  const TensorMeta* meta;      // [n + 1], the last one a sentinel
  const int32_t* tile_tensor;  // first tensor of each thread block's part
  int32_t blocks;
  int32_t per_warp;  // state blocks of a warp
  void* m;
  void* v;
  float* ms;
  float* vs;
  const float* grad_scale;
  const int32_t* skip;
  float b1, c1, b2, c2, root_scale, eps, decay, size;
};

// Where a code begins, in the block's own scale: half-way between two codes'
// roots.  Entry 0 is never consulted.
struct Levels {
  float m[128], v[256];
  constexpr Levels() : m(), v() {
    for (int k = 1; k < 128; ++k) m[k] = (float)(((k - 0.5) / 127) * ((k - 0.5) / 127));
    for (int k = 1; k < 256; ++k) {
      const double r = (k - 0.5) / 255;
      v[k] = (float)((r * r) * (r * r));
    }
  }
};
__device__ const Levels kLevels = Levels();

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm volatile("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Eight consecutive 32-bit words: one 32-byte access.
__device__ __forceinline__ void ld8(const void* p, uint32_t* r) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ void st8(void* p, const uint32_t* r) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void ld4(const void* p, uint32_t* r) {
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "l"(p));
}
__device__ __forceinline__ void ld2(const void* p, uint32_t* r) {
  asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p));
}

__device__ __forceinline__ float half_bits(int dt, uint32_t h) {
  if (dt == TBE_BF16) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half((unsigned short)h));
}
__device__ __forceinline__ uint32_t to_half_bits(int dt, float f) {
  if (dt == TBE_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
  return __half_as_ushort(__float2half_rn(f));
}

// A lane's eight elements of a block as loaded.  VEC: elements 8 l .. 8 l + 7
// in one access.  Otherwise element 32 j + l at step j, each on its own
// (tensors that are not aligned, and a tensor's last block): still whole
// lines per access.
template <bool VEC>
__device__ __forceinline__ int elem(int lane, int j) {
  return VEC ? lane * kPer + j : j * 32 + lane;
}

template <bool VEC>
__device__ __forceinline__ void load_raw(int dt, const void* base, int64_t at, int lane, int count, uint32_t* raw) {
  if (VEC) {
    if (dt == TBE_F32) ld8(static_cast<const float*>(base) + at + lane * kPer, raw);
    else ld4(static_cast<const uint16_t*>(base) + at + lane * kPer, raw);
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = elem<VEC>(lane, j);
      raw[j] = 0;
      if (e < count) {
        if (dt == TBE_F32) raw[j] = static_cast<const uint32_t*>(base)[at + e];
        else raw[j] = static_cast<const uint16_t*>(base)[at + e];
      }
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void unpack(int dt, const uint32_t* raw, float* f) {
  if (dt == TBE_F32) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) f[j] = __uint_as_float(raw[j]);
  } else if (VEC) {
    if (dt == TBE_BF16) {
#pragma unroll
      for (int j = 0; j < kPer / 2; ++j) {
        f[2 * j] = __uint_as_float(raw[j] << 16);
        f[2 * j + 1] = __uint_as_float(raw[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer / 2; ++j) {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&raw[j]));
        f[2 * j] = h.x;
        f[2 * j + 1] = h.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) f[j] = half_bits(dt, raw[j]);
  }
}

template <bool VEC>
__device__ __forceinline__ void store(int dt, void* base, int64_t at, int lane, int count, const float* f) {
  if (VEC) {
    if (dt == TBE_F32) {
      st8(static_cast<float*>(base) + at + lane * kPer, reinterpret_cast<const uint32_t*>(f));
    } else if (dt == TBE_F16) {
      store_out(static_cast<__half*>(base) + at + lane * kPer, f, kPer, true);
    } else {
      store_out(static_cast<__nv_bfloat16*>(base) + at + lane * kPer, f, kPer, true);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = elem<VEC>(lane, j);
      if (e < count) {
        if (dt == TBE_F32) static_cast<float*>(base)[at + e] = f[j];
        else static_cast<uint16_t*>(base)[at + e] = (uint16_t)to_half_bits(dt, f[j]);
      }
    }
  }
}

// Codes as floats: a byte's bits under the exponent of 2^17 (2^16) are
// 2^17 + byte / 64 (2^16 + byte / 128).  A code of a first moment counts in
// units of 1/64, one of a second moment in units of 1/128, so that a block's
// scale is multiplied by 64^2 / 127^2 = 0.25 (128^4 / 255^4 = 0.06): by 1 / 127^2
// (1 / 255^4) a scale below 2e-34 (5e-29) would leave the normal numbers, and
// with them its precision, before the codes are multiplied in.
constexpr float kUnitM = (float)(64.0 * 64.0 / (127.0 * 127.0));
constexpr float kUnitV = (float)(128.0 * 128.0 * 128.0 * 128.0 / (255.0 * 255.0 * 255.0 * 255.0));
constexpr float kBaseM = 131072.f + 2.f, kBaseV = 65536.f;  // 2: a first moment's code comes plus 128
__device__ __forceinline__ float byte_m(uint32_t w, int b) { return __uint_as_float(__byte_perm(w, 0x48000000u, 0x7640 + b)); }
__device__ __forceinline__ float byte_v(uint32_t w, int b) { return __uint_as_float(__byte_perm(w, 0x47800000u, 0x7640 + b)); }
__device__ __forceinline__ float code_m(uint32_t w, int b) { return byte_m(w ^ 0x80808080u, b) - kBaseM; }
__device__ __forceinline__ float code_v(uint32_t w, int b) { return byte_v(w, b) - kBaseV; }

// The scale that divides a block whose largest magnitude is `top`: its
// inverse, or 0 where there is nothing to divide by: a block below the
// smallest normal number is held as 0, one with an infinite or NaN moment as
// NaN (any code times a NaN scale).
__device__ __forceinline__ float block_inverse(float top, float* scale) {
  const bool finite = top <= 3.402823466e38f;
  *scale = finite ? (top < kTiny ? 0.f : top) : __uint_as_float(0x7fffffffu);
  return finite && top >= kTiny ? __fdiv_rn(1.f, top) : 0.f;
}

// The code whose root is nearest to y's: f = y's root in codes, from an
// approximate square root (2^-23 of it; of 255 codes and twice: below 7e-5).  Where f is that
// near to the middle between two codes, the exact level decides.
constexpr float kNearLevel = 0.49992f;
__device__ __forceinline__ int nearest_code(float f, float y, const float* level) {
  const float r = rintf(f);
  int q = (int)r;
  if (fabsf(f - r) > kNearLevel) {
    const int k = (int)floorf(f) + 1;
    q = y >= __ldg(level + k) ? k : k - 1;
  }
  return q;
}

template <int BITS, bool VEC>
__device__ __forceinline__ void update_block(const StepArgs& a, const TensorMeta& t, int64_t block, int64_t at,
                                             int count, int lane, float gscale) {
  uint32_t rp[kPer], rg[kPer], rm[kPer], rv[kPer];
  float sm = 0.f, sv = 0.f;
  load_raw<VEC>(t.gdt, t.g, at, lane, count, rg);
  load_raw<VEC>(t.pdt, t.p, at, lane, count, rp);
  const int64_t s0 = block * kBlock;
  if (BITS == 32) {
    load_raw<VEC>(TBE_F32, a.m, s0, lane, count, rm);
    load_raw<VEC>(TBE_F32, a.v, s0, lane, count, rv);
  } else {
    if (VEC) {
      ld2(static_cast<const uint8_t*>(a.m) + s0 + lane * kPer, rm);
      ld2(static_cast<const uint8_t*>(a.v) + s0 + lane * kPer, rv);
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int e = elem<VEC>(lane, j);
        rm[j] = e < count ? static_cast<const uint8_t*>(a.m)[s0 + e] : 0;
        rv[j] = e < count ? static_cast<const uint8_t*>(a.v)[s0 + e] : 0;
      }
    }
    sm = a.ms[block];
    sv = a.vs[block];
  }
  float g[kPer], p[kPer], m[kPer], v[kPer];
  unpack<VEC>(t.gdt, rg, g);
  unpack<VEC>(t.pdt, rp, p);
  if (BITS == 32) {
    unpack<VEC>(TBE_F32, rm, m);
    unpack<VEC>(TBE_F32, rv, v);
  } else {
    const float cm = __fmul_rn(sm, kUnitM), cv = __fmul_rn(sv, kUnitV);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t wm = VEC ? rm[j / 4] : rm[j], wv = VEC ? rv[j / 4] : rv[j];
      const float q = code_m(wm, VEC ? j % 4 : 0);
      m[j] = __fmul_rn(q * fabsf(q), cm);
      const float z = code_v(wv, VEC ? j % 4 : 0);
      const float z2 = z * z;
      v[j] = __fmul_rn(__fmul_rn(z2, z2), cv);
    }
  }
  float top_m = 0.f, top_v = 0.f;
  uint32_t bits_m = 0, bits_v = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    g[j] = __fmul_rn(g[j], gscale);
    m[j] = __fadd_rn(__fmul_rn(m[j], a.b1), __fmul_rn(g[j], a.c1));
    v[j] = __fadd_rn(__fmul_rn(v[j], a.b2), __fmul_rn(__fmul_rn(g[j], g[j]), a.c2));
    const float bottom = fmaf(sqrt_approx(v[j]), a.root_scale, a.eps);
    // the whole change first: the weight itself is rounded once
    p[j] -= fmaf(a.size, m[j] * rcp(bottom), p[j] * a.decay);
    if (BITS == 8 && (VEC || elem<VEC>(lane, j) < count)) {
      // magnitudes order like their bits, NaN above infinity
      bits_m = max(bits_m, __float_as_uint(m[j]) & 0x7fffffffu);
      bits_v = max(bits_v, __float_as_uint(v[j]) & 0x7fffffffu);
    }
  }
  store<VEC>(t.pdt, t.p, at, lane, count, p);
  if (BITS == 32) {
    store<VEC>(TBE_F32, a.m, s0, lane, count, m);
    store<VEC>(TBE_F32, a.v, s0, lane, count, v);
    return;
  }
  top_m = __uint_as_float(__reduce_max_sync(kFull, bits_m));
  top_v = __uint_as_float(__reduce_max_sync(kFull, bits_v));
  float scale_m, scale_v;
  const float inv_m = block_inverse(top_m, &scale_m), inv_v = block_inverse(top_v, &scale_v);
  uint32_t qm[2] = {0, 0}, qv[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float ym = fminf(__fmul_rn(fabsf(m[j]), inv_m), 1.f);
    int q = nearest_code(127.f * root(ym), ym, kLevels.m);
    if (m[j] < 0.f) q = -q;
    const float yv = fminf(__fmul_rn(v[j], inv_v), 1.f);
    int z = nearest_code(255.f * root(root(yv)), yv, kLevels.v);
    if (yv > 0.f) z = max(z, 1);
    if (VEC) {
      qm[j / 4] |= (uint32_t)(q & 0xff) << (8 * (j % 4));
      qv[j / 4] |= (uint32_t)z << (8 * (j % 4));
    } else {
      const int e = elem<VEC>(lane, j);
      if (e < count) {
        static_cast<int8_t*>(a.m)[s0 + e] = (int8_t)q;
        static_cast<uint8_t*>(a.v)[s0 + e] = (uint8_t)z;
      }
    }
  }
  if (VEC) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + s0 + lane * kPer) = make_uint2(qm[0], qm[1]);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + s0 + lane * kPer) = make_uint2(qv[0], qv[1]);
  }
  if (lane == 0) {
    a.ms[block] = scale_m;
    a.vs[block] = scale_v;
  }
}

// Whole, aligned blocks of one tensor with 8-bit states: the same arithmetic
// two elements at a time.  This case is bound by instructions, not by its 10
// to 16 bytes an element, so codes are rounded by adding 1.5 * 2^23 (the code
// is then the sum's low byte, in two's complement) and nearness to a level is
// tested once for the lane's eight elements.  Blocks to come are copied into
// a ring of the warp's own in shared memory while one is worked on.
template <int PDT, int GDT>
struct Ring8 {
  static constexpr int kP = PDT == TBE_F32 ? 4 : 2, kG = GDT == TBE_F32 ? 4 : 2;  // bytes of an element
  // a slot: weights, gradients, codes, scales
  static constexpr int kGradAt = kBlock * kP, kMAt = kGradAt + kBlock * kG, kVAt = kMAt + kBlock, kScaleAt = kVAt + kBlock;
  static constexpr int kSlot = kScaleAt + 16;
  static constexpr int kSlots = kP + kG == 4 ? 3 : 2;  // at most 41 KB a block of eight warps
  static constexpr int kBytes = kSlots * kSlot;
  const uint8_t* mem;
  uint32_t base;
  int read, write, lane;
  __device__ __forceinline__ Ring8(const uint8_t* m, int l) : mem(m), base(smem_u32(m)), read(0), write(0), lane(l) {}
  static __device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  }
  // Asks for the next block (`more`: there is one); pp and gp: the lane's elements of it.
  __device__ __forceinline__ void fill(const StepArgs& a, const uint8_t* pp, const uint8_t* gp, int64_t block, bool more) {
    if (more) {
      const uint32_t to = base + write;
#pragma unroll
      for (int i = 0; i < kG / 2; ++i) copy16(to + kGradAt + lane * kPer * kG + 16 * i, gp + 16 * i);
#pragma unroll
      for (int i = 0; i < kP / 2; ++i) copy16(to + lane * kPer * kP + 16 * i, pp + 16 * i);
      cp_async8(to + kMAt + lane * kPer, static_cast<const uint8_t*>(a.m) + block * kBlock + lane * kPer);
      cp_async8(to + kVAt + lane * kPer, static_cast<const uint8_t*>(a.v) + block * kBlock + lane * kPer);
      if (lane < 2) cp_async4(to + kScaleAt + lane * 4, (lane ? a.vs : a.ms) + block);
    }
    cp_commit();
    write = write + kSlot == kBytes ? 0 : write + kSlot;
  }
  __device__ __forceinline__ void ready() const {
    cp_wait<kSlots - 1>();
    __syncwarp();
  }
  __device__ __forceinline__ void done() {
    __syncwarp();
    read = read + kSlot == kBytes ? 0 : read + kSlot;
  }
};
// A lane's share of a block, as read.
template <int PDT, int GDT>
struct Raw8 {
  uint32_t p[PDT == TBE_F32 ? 8 : 4], g[GDT == TBE_F32 ? 8 : 4], m[2], v[2];
  float sm, sv;
  __device__ __forceinline__ Raw8(const Ring8<PDT, GDT>& r) {
    using R = Ring8<PDT, GDT>;
    const uint8_t* s = r.mem + r.read;
#pragma unroll
    for (int i = 0; i < R::kP / 2; ++i)
      *reinterpret_cast<uint4*>(p + 4 * i) = *reinterpret_cast<const uint4*>(s + r.lane * kPer * R::kP + 16 * i);
#pragma unroll
    for (int i = 0; i < R::kG / 2; ++i)
      *reinterpret_cast<uint4*>(g + 4 * i) = *reinterpret_cast<const uint4*>(s + R::kGradAt + r.lane * kPer * R::kG + 16 * i);
    *reinterpret_cast<uint2*>(m) = *reinterpret_cast<const uint2*>(s + R::kMAt + r.lane * kPer);
    *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(s + R::kVAt + r.lane * kPer);
    sm = *reinterpret_cast<const float*>(s + R::kScaleAt);
    sv = *reinterpret_cast<const float*>(s + R::kScaleAt + 4);
  }
};
template <int DT>
__device__ __forceinline__ Two raw_pair(const uint32_t* r, int j) {
  if (DT == TBE_F32) return two(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
  if (DT == TBE_BF16) return two(__uint_as_float(r[j] << 16), __uint_as_float(r[j] & 0xffff0000u));
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&r[j]));
  return two(h.x, h.y);
}
// The sum of two products, each rounded, and the sum rounded: two-wide
// multiplies and adds would be contracted.
__device__ __forceinline__ Two rounded_sum(Two a, Two b) {
  return two(__fadd_rn(lo(a), lo(b)), __fadd_rn(hi(a), hi(b)));
}
__device__ __forceinline__ uint32_t pack4(const uint32_t* c) {
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

template <int PDT, int GDT>
__device__ __forceinline__ void step_8(const StepArgs& a, const Raw8<PDT, GDT>& x, uint8_t* pp, int64_t block, int lane,
                                       Two gscale) {
  const Two cm = two(__fmul_rn(x.sm, kUnitM)), cv = two(__fmul_rn(x.sv, kUnitV));
  Two m[kPer / 2], v[kPer / 2];
  float top_m = 0.f, top_v = 0.f;
#pragma unroll
  for (int j = 0; j < kPer / 2; ++j) {
    const uint32_t wm = x.m[j / 2] ^ 0x80808080u, wv = x.v[j / 2];  // the signed codes plus 128
    const int b = 2 * j % 4;
    const Two q = two(byte_m(wm, b), byte_m(wm, b + 1)) + two(-kBaseM);
    const Two z = two(byte_v(wv, b), byte_v(wv, b + 1)) + two(-kBaseV);
    const Two z2 = z * z;
    const Two g = raw_pair<GDT>(x.g, j) * gscale;
    m[j] = rounded_sum(two(lo(q) * fabsf(lo(q)), hi(q) * fabsf(hi(q))) * cm * two(a.b1), g * two(a.c1));
    v[j] = rounded_sum(z2 * z2 * cv * two(a.b2), g * g * two(a.c2));
    top_m = max_nan(max_nan(top_m, fabsf(lo(m[j]))), fabsf(hi(m[j])));
    top_v = max_nan(max_nan(top_v, lo(v[j])), hi(v[j]));
  }
  // magnitudes order like their bits, NaN above infinity
  top_m = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top_m)));
  top_v = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top_v)));
  // With an eps of at least 1e-10, the root of a v below the normal numbers
  // (under 1.1e-19) does not show beside it, and may count as 0.
  Two w[kPer / 2];
  if (a.eps >= 1e-10f) {
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) w[j] = root(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) w[j] = two(sqrt_approx(lo(v[j])), sqrt_approx(hi(v[j])));
  }
#pragma unroll
  for (int j = 0; j < kPer / 2; ++j) {
    const Two bottom = fma2(w[j], two(a.root_scale), two(a.eps));
    const Two p = raw_pair<PDT>(x.p, j);
    // the whole change first: the weight itself is rounded once
    w[j] = p + negative(fma2(two(a.size), m[j] * rcp(bottom), p * two(a.decay)));
  }
  float f[kPer];
#pragma unroll
  for (int j = 0; j < kPer / 2; ++j) f[2 * j] = lo(w[j]), f[2 * j + 1] = hi(w[j]);
  if (PDT == TBE_F32) st8(pp, reinterpret_cast<const uint32_t*>(f));
  else if (PDT == TBE_F16) store_out(reinterpret_cast<__half*>(pp), f, kPer, true);
  else store_out(reinterpret_cast<__nv_bfloat16*>(pp), f, kPer, true);
  float scale_m, scale_v;
  const float inv_m = block_inverse(top_m, &scale_m), inv_v = block_inverse(top_v, &scale_v);
  // Roots in codes: the codes' number goes under the root with the scale.  For
  // a largest magnitude below 2^-114 (m) or 2^-96 (v) that factor is infinite
  // and distances below are NaN, which max_nan keeps: every code then comes
  // from the division that follows.
  const Two km = two(inv_m * 16129.f), kv = two(inv_v * 4228250625.f);
  const Two magic = two(12582912.f), back = two(-12582912.f);
  uint32_t cq[kPer], cz[kPer];
  float off = 0.f;
#pragma unroll
  for (int j = 0; j < kPer / 2; ++j) {
    const Two ym = m[j] * km, yv = v[j] * kv;
    Two c = two(copysignf(root(fabsf(lo(ym))), lo(ym)), copysignf(root(fabsf(hi(ym))), hi(ym)));
    Two r = c + magic;
    Two d = c + negative(r + back);
    off = max_nan(max_nan(off, fabsf(lo(d))), fabsf(hi(d)));
    cq[2 * j] = __float_as_uint(lo(r));
    cq[2 * j + 1] = __float_as_uint(hi(r));
    c = root(root(yv));
    // at least 1 for what is not 0
    c = two(fmaxf(lo(c), __saturatef(lo(c) * 1e30f)), fmaxf(hi(c), __saturatef(hi(c) * 1e30f)));
    r = c + magic;
    d = c + negative(r + back);
    off = max_nan(max_nan(off, fabsf(lo(d))), fabsf(hi(d)));
    cz[2 * j] = __float_as_uint(lo(r));
    cz[2 * j + 1] = __float_as_uint(hi(r));
  }
  if (!(off <= kNearLevel)) {  // some code is close to its neighbour: its level decides
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float mj = j & 1 ? hi(m[j / 2]) : lo(m[j / 2]), vj = j & 1 ? hi(v[j / 2]) : lo(v[j / 2]);
      const float ym = fminf(__fmul_rn(fabsf(mj), inv_m), 1.f), yv = fminf(__fmul_rn(vj, inv_v), 1.f);
      const int q = nearest_code(127.f * root(ym), ym, kLevels.m);
      const int z = nearest_code(255.f * root(root(yv)), yv, kLevels.v);
      cq[j] = mj < 0.f ? -q : q;
      cz[j] = yv > 0.f ? max(z, 1) : z;
    }
  }
  const int64_t s0 = block * kBlock + lane * kPer;
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + s0) = make_uint2(pack4(cq), pack4(cq + 4));
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + s0) = make_uint2(pack4(cz), pack4(cz + 4));
  if (lane == 0) {
    a.ms[block] = scale_m;
    a.vs[block] = scale_v;
  }
}

// `count` whole blocks from `block` on, at element `at` of the tensor.
template <int PDT, int GDT>
__device__ __forceinline__ void whole_blocks_8(const StepArgs& a, const TensorMeta& t, int64_t block, int64_t at, int count,
                                               int lane, Two gscale, const uint8_t* mem) {
  using R = Ring8<PDT, GDT>;
  uint8_t* pp = static_cast<uint8_t*>(t.p) + (at + lane * kPer) * R::kP;
  const uint8_t* from_p = pp;
  const uint8_t* from_g = static_cast<const uint8_t*>(t.g) + (at + lane * kPer) * R::kG;
  R ring(mem, lane);
  int asked = 0;
  auto ask = [&] {
    ring.fill(a, from_p, from_g, block + asked, asked < count);
    ++asked;
    from_p += kBlock * R::kP;
    from_g += kBlock * R::kG;
  };
#pragma unroll
  for (int i = 0; i < R::kSlots; ++i) ask();
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    ring.ready();
    const Raw8<PDT, GDT> x(ring);
    ring.done();
    ask();
    step_8<PDT, GDT>(a, x, pp, block + i, lane, gscale);
    pp += kBlock * R::kP;
  }
  cp_wait<0>();
}

// One launch for the whole list.  PDT, GDT: the types of every tensor, or
// kMixed: looked up at each one.  (8-bit states: the 64 registers that leave
// room for four blocks on an SM make all but two of the nine typed variants
// spill 16 or 24 bytes a thread, the mixed one 52.)
constexpr int kMixed = -1;
template <int BITS, int PDT, int GDT>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 4 : 3) adamw_kernel(StepArgs a) {
  if (a.skip && *a.skip != 0) return;
  const float gscale = a.grad_scale ? *a.grad_scale : 1.f;
  constexpr bool kRing = BITS == 8 && PDT != kMixed;
  __shared__ __align__(16) uint8_t mem[kRing ? kWarps * Ring8<PDT, GDT>::kBytes : 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int t = a.tile_tensor[blockIdx.x];
  // a warp takes neighbouring blocks
  int64_t block = ((int64_t)blockIdx.x * kWarps + warp) * a.per_warp;
  const int64_t end = block + a.per_warp < a.blocks ? block + a.per_warp : a.blocks;
  while (block < end) {
    while (a.meta[t + 1].block0 <= block) ++t;  // the sentinel's is above every block
    TensorMeta tm = a.meta[t];
    if constexpr (PDT != kMixed) tm.pdt = PDT, tm.gdt = GDT;
    const int64_t at = (block - tm.block0) * kBlock;
    const int64_t left = tm.numel - at;
    if (kRing && tm.vec && left >= kBlock) {
      const int64_t whole = left / kBlock;
      const int count = (int)(whole < end - block ? whole : end - block);
      if constexpr (kRing)
        whole_blocks_8<PDT, GDT>(a, tm, block, at, count, lane, two(gscale), mem + warp * Ring8<PDT, GDT>::kBytes);
      block += count;
    } else {
      if ((BITS == 32 || PDT == kMixed) && tm.vec && left >= kBlock)
        update_block<BITS, true>(a, tm, block, at, kBlock, lane, gscale);
      else
        update_block<BITS, false>(a, tm, block, at, left < kBlock ? (int)left : kBlock, lane, gscale);
      ++block;
    }
  }
}

template <int BITS, int PDT>
void launch_step(int gdt, int tiles, const StepArgs& a, cudaStream_t s) {
  if (gdt == TBE_F32) adamw_kernel<BITS, PDT, TBE_F32><<<tiles, kThreads, 0, s>>>(a);
  else if (gdt == TBE_F16) adamw_kernel<BITS, PDT, TBE_F16><<<tiles, kThreads, 0, s>>>(a);
  else adamw_kernel<BITS, PDT, TBE_BF16><<<tiles, kThreads, 0, s>>>(a);
}
template <int BITS>
void launch_step(int pdt, int gdt, int tiles, const StepArgs& a, cudaStream_t s) {
  if (pdt == kMixed) adamw_kernel<BITS, kMixed, kMixed><<<tiles, kThreads, 0, s>>>(a);
  else if (pdt == TBE_F32) launch_step<BITS, TBE_F32>(gdt, tiles, a, s);
  else if (pdt == TBE_F16) launch_step<BITS, TBE_F16>(gdt, tiles, a, s);
  else launch_step<BITS, TBE_BF16>(gdt, tiles, a, s);
}

// 8-bit states as the values they stand for: eight elements per thread.
__global__ void __launch_bounds__(kThreads)
    adamw_state_kernel(const uint8_t* m, const uint8_t* v, const float* ms, const float* vs, float* mo, float* vo,
                       int64_t groups) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= groups) return;
  uint32_t rm[2], rv[2];
  ld2(m + i * 8, rm);
  ld2(v + i * 8, rv);
  const int64_t block = i / (kBlock / 8);
  const float cm = __fmul_rn(__ldg(ms + block), kUnitM), cv = __fmul_rn(__ldg(vs + block), kUnitV);
  float fm[8], fv[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = code_m(rm[j / 4], j % 4);
    fm[j] = __fmul_rn(q * fabsf(q), cm);
    const float z = code_v(rv[j / 4], j % 4);
    const float z2 = z * z;
    fv[j] = __fmul_rn(__fmul_rn(z2, z2), cv);
  }
  st8(mo + i * 8, reinterpret_cast<const uint32_t*>(fm));
  st8(vo + i * 8, reinterpret_cast<const uint32_t*>(fv));
}

struct AdamWPlan {
  int32_t n;
  int32_t bits;
  int32_t blocks;
  int32_t tiles;
  int32_t per_warp;
  int32_t device;
  int32_t pdt, gdt;  // of every tensor, or kMixed
  const TensorMeta* dmeta;
  const int32_t* dtile;
};

bool aligned_to(const void* p, size_t b) { return ((uintptr_t)p & (b - 1)) == 0; }

// Total state blocks of n tensors, or -1 where a size is out of range.
int64_t count_blocks(int32_t n, const int64_t* numel) {
  if (n < 1 || n > TBE_ADAMW_MAX_TENSORS || !numel) return -1;
  int64_t blocks = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] >= (int64_t(1) << 40)) return -1;
    blocks += (numel[i] + kBlock - 1) / kBlock;
    if (blocks >= (int64_t(1) << 31) - (1 << 20)) return -1;
  }
  return blocks;
}

size_t meta_bytes(int32_t n) { return ((size_t)(n + 1) * sizeof(TensorMeta) + 255) / 256 * 256; }

// State blocks per warp.  8-bit steps fill a warp's ring once for all its
// blocks, but more of them than four leave the last warps alone: 64 M
// elements, step and states read back, 293.6, 232.4, 233.7 and 235.5 us with 1,
// 4, 8 and 52 (one wave); 16 M 78.9, 66.2, 68.3 us (1, 4, 8).  Steps that fit
// one wave take as few as that needs (1 M: 8.9 us, with four 11.0 us).  32-bit
// steps have no ring: 1 M elements 5.6, 5.2, 5.8 us with 1, 2, 4 blocks, 64 M
// 218, 208, 207 us.
int32_t blocks_per_warp(int64_t blocks, int32_t bits) {
  if (bits == 32) return 2;
  const int64_t warps = (int64_t)sm_count() * 4 * kWarps;
  const int64_t n = (blocks + warps - 1) / warps;
  return n < 1 ? 1 : (n > 4 ? 4 : (int32_t)n);
}
int32_t tile_count(int64_t blocks, int32_t bits) {
  const int64_t tile = (int64_t)blocks_per_warp(blocks, bits) * kWarps;
  return (int32_t)((blocks + tile - 1) / tile);
}

}  // namespace
}  // namespace tbe

using namespace tbe;

struct tbe_adamw_plan : public tbe::AdamWPlan {};

extern "C" {

int64_t tbe_adamw_state_blocks(int32_t n, const int64_t* numel) { return count_blocks(n, numel); }

size_t tbe_adamw_plan_device_bytes(int32_t n, const int64_t* numel, int32_t state_bits) {
  const int64_t blocks = count_blocks(n, numel);
  if (blocks < 0 || (state_bits != 8 && state_bits != 32)) return 0;
  return meta_bytes(n) + ((size_t)tile_count(blocks, state_bits) * 4 + 255) / 256 * 256;
}

int tbe_adamw_plan_create(const tbe_adamw_tensors* L, void* dev_meta, size_t dev_meta_bytes, void* stream,
                          tbe_adamw_plan** plan_out) {
  if (!L || !dev_meta || !plan_out || !L->numel || !L->params || !L->grads || !L->param_dtype || !L->grad_dtype)
    return TBE_ERR_INVALID_ARG;
  if (L->state_bits != 8 && L->state_bits != 32) return TBE_ERR_INVALID_ARG;
  const int64_t blocks = count_blocks(L->n, L->numel);
  if (blocks < 0) return TBE_ERR_INVALID_ARG;
  if (!aligned_to(dev_meta, 16)) return TBE_ERR_UNSUPPORTED;
  const size_t need = tbe_adamw_plan_device_bytes(L->n, L->numel, L->state_bits);
  if (dev_meta_bytes < need) return TBE_ERR_WORKSPACE;
  const size_t mb = meta_bytes(L->n);
  uint8_t* host = new (std::nothrow) uint8_t[need];
  tbe_adamw_plan* p = new (std::nothrow) tbe_adamw_plan();
  if (!host || !p) {
    delete[] host;
    delete p;
    return TBE_ERR_INVALID_ARG;
  }
  std::memset(host, 0, need);
  TensorMeta* meta = reinterpret_cast<TensorMeta*>(host);
  int32_t* tile = reinterpret_cast<int32_t*>(host + mb);
  int st = TBE_OK;
  const int64_t tile_blocks = (int64_t)blocks_per_warp(blocks, L->state_bits) * kWarps;
  int64_t at = 0, next_tile = 0;
  for (int32_t i = 0; i < L->n && st == TBE_OK; ++i) {
    const int32_t pd = L->param_dtype[i], gd = L->grad_dtype[i];
    if (pd < TBE_F32 || pd > TBE_BF16 || gd < TBE_F32 || gd > TBE_BF16) st = TBE_ERR_INVALID_ARG;
    else if (L->numel[i] > 0 && (!L->params[i] || !L->grads[i])) st = TBE_ERR_INVALID_ARG;
    else if (!aligned_to(L->params[i], pd == TBE_F32 ? 4 : 2) || !aligned_to(L->grads[i], gd == TBE_F32 ? 4 : 2))
      st = TBE_ERR_UNSUPPORTED;
    TensorMeta& m = meta[i];
    m.p = L->params[i];
    m.g = L->grads[i];
    m.numel = L->numel[i];
    m.block0 = (int32_t)at;
    m.pdt = (uint8_t)pd;
    m.gdt = (uint8_t)gd;
    m.vec = aligned_to(m.p, pd == TBE_F32 ? 32 : 16) && aligned_to(m.g, gd == TBE_F32 ? 32 : 16);
    const int64_t end = at + (m.numel + kBlock - 1) / kBlock;
    while (next_tile * tile_blocks < end) tile[next_tile++] = i;
    at = end;
  }
  meta[L->n].block0 = 0x7fffffff;
  if (st == TBE_OK) {
    p->n = L->n;
    p->bits = L->state_bits;
    p->blocks = (int32_t)blocks;
    p->tiles = tile_count(blocks, L->state_bits);
    p->per_warp = blocks_per_warp(blocks, L->state_bits);
    p->pdt = L->param_dtype[0];
    p->gdt = L->grad_dtype[0];
    for (int32_t i = 1; i < L->n; ++i)
      if (L->param_dtype[i] != p->pdt || L->grad_dtype[i] != p->gdt) {
        p->pdt = p->gdt = kMixed;
        break;
      }
    cudaGetDevice(&p->device);
    p->dmeta = reinterpret_cast<const TensorMeta*>(dev_meta);
    p->dtile = reinterpret_cast<const int32_t*>(static_cast<uint8_t*>(dev_meta) + mb);
    // pageable memory: the copy has left the host buffer when the call returns
    if (cudaMemcpyAsync(dev_meta, host, need, cudaMemcpyHostToDevice, (cudaStream_t)stream) != cudaSuccess)
      st = TBE_ERR_CUDA;
  }
  delete[] host;
  if (st != TBE_OK) {
    delete p;
    return st;
  }
  *plan_out = p;
  return TBE_OK;
}

void tbe_adamw_plan_destroy(tbe_adamw_plan* plan) { delete plan; }

int tbe_adamw_step(const tbe_adamw_plan* plan, const tbe_adamw* opt, void* exp_avg, void* exp_avg_sq,
                   float* exp_avg_scale, float* exp_avg_sq_scale, const float* grad_scale, const int32_t* skip,
                   void* stream) {
  if (!plan || !opt) return TBE_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return TBE_ERR_CUDA;
  if (dev != plan->device) return TBE_ERR_INVALID_ARG;
  const tbe_adamw& o = *opt;
  if (o.step < 1 || !std::isfinite(o.learning_rate) || !std::isfinite(o.weight_decay) || !std::isfinite(o.eps) ||
      o.eps < 0 || !(o.beta1 >= 0 && o.beta1 < 1) || !(o.beta2 >= 0 && o.beta2 < 1))
    return TBE_ERR_INVALID_ARG;
  if (plan->blocks == 0) return TBE_OK;
  if (!exp_avg || !exp_avg_sq) return TBE_ERR_INVALID_ARG;
  if (!aligned_to(exp_avg, 32) || !aligned_to(exp_avg_sq, 32)) return TBE_ERR_UNSUPPORTED;
  if (plan->bits == 8 && (!exp_avg_scale || !exp_avg_sq_scale)) return TBE_ERR_INVALID_ARG;
  StepArgs a;
  a.meta = plan->dmeta;
  a.tile_tensor = plan->dtile;
  a.blocks = plan->blocks;
  a.per_warp = plan->per_warp;
  a.m = exp_avg;
  a.v = exp_avg_sq;
  a.ms = exp_avg_scale;
  a.vs = exp_avg_sq_scale;
  a.grad_scale = grad_scale;
  a.skip = skip;
  // the constants in 64 bits, each rounded once
  a.b1 = (float)o.beta1;
  a.c1 = (float)(1.0 - o.beta1);
  a.b2 = (float)o.beta2;
  a.c2 = (float)(1.0 - o.beta2);
  a.root_scale = (float)(1.0 / std::sqrt(1.0 - std::pow(o.beta2, (double)o.step)));
  a.eps = (float)o.eps;
  a.decay = (float)(o.learning_rate * o.weight_decay);
  a.size = (float)(o.learning_rate / (1.0 - std::pow(o.beta1, (double)o.step)));
  cudaStream_t s = (cudaStream_t)stream;
  trace_begin(s);
  if (plan->bits == 8) launch_step<8>(plan->pdt, plan->gdt, plan->tiles, a, s);
  else launch_step<32>(plan->pdt, plan->gdt, plan->tiles, a, s);
  const int st = check_launch();
  trace_mark(s, "adamw");
  return st;
}

int tbe_adamw_state(const tbe_adamw_plan* plan, const void* exp_avg, const void* exp_avg_sq,
                    const float* exp_avg_scale, const float* exp_avg_sq_scale, float* exp_avg_out,
                    float* exp_avg_sq_out, void* stream) {
  if (!plan || plan->bits != 8) return TBE_ERR_INVALID_ARG;
  if (plan->blocks == 0) return TBE_OK;
  if (!exp_avg || !exp_avg_sq || !exp_avg_scale || !exp_avg_sq_scale || !exp_avg_out || !exp_avg_sq_out)
    return TBE_ERR_INVALID_ARG;
  if (!aligned_to(exp_avg, 32) || !aligned_to(exp_avg_sq, 32) || !aligned_to(exp_avg_out, 32) ||
      !aligned_to(exp_avg_sq_out, 32))
    return TBE_ERR_UNSUPPORTED;
  const int64_t groups = (int64_t)plan->blocks * (kBlock / 8);
  adamw_state_kernel<<<(unsigned)((groups + kThreads - 1) / kThreads), kThreads, 0, (cudaStream_t)stream>>>(
      static_cast<const uint8_t*>(exp_avg), static_cast<const uint8_t*>(exp_avg_sq), exp_avg_scale, exp_avg_sq_scale,
      exp_avg_out, exp_avg_sq_out, groups);
  return check_launch();
}

}  // extern "C"
