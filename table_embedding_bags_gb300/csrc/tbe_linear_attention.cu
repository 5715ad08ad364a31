// tbe_linear_attention.cu -- causal linear attention with a decay for each
// head over jagged sequences, its backward pass and its form for single
// tokens.
//
//   S_t = gamma S_{t-1} + k_t v_t^T      o_t = scale q_t^T S_t      gamma = exp(-decay[head])
//
// In tiles of 64 tokens: within a tile a masked product, o += (q k^T . gamma^
// distance) v, and across tiles the state, o += gamma^(place + 1) q S and S =
// gamma^64 S + sum gamma^(63 - place) k v^T.  Tiles cut the token axis, not
// the sequences: one tile may hold many short sequences, whose products the
// mask keeps apart, so the work goes by tokens whatever the lengths are.
//
// A block takes a run of tiles of one head and up to 64 value columns.  The
// state that a run finds comes from the runs before it: a first kernel sums
// what each run adds to the state of the sequence that leaves it, a second
// one joins those along the runs, in order; sequences that end inside their
// run cost neither anything.  No block waits for another inside a kernel and
// no sum depends on timing.
//
// The backward needs nothing new.  With G_t = scale q_t do_t^T + gamma G_{t+1},
//   dq_t = scale S_t do_t     is the same recurrence of (do, v, k) with S^T,
//   dk_t = G_t v_t, dv_t = G_t^T k_t  are it from the last token to the first,
// of (v, do, q) and (k, q, do), where the decay comes behind the read.  Its
// three passes go side by side in the launches of one.
//
// Numbers.  Products of inputs are exact and summed in fp32; the state is
// held in fp32.  Two operands are rounded to the inputs' type: the weighted
// products of a tile and the state as it is read, both half a step of the
// type that the output is rounded to as well.  What is added to the state
// must not be: gamma^n k goes in as the sum of as many numbers of the type as
// hold its 24 bits (three of bf16, two of fp16).  fp16 lacks fp32's range, so
// there each of the three is first moved by a power of two that its largest
// value names: products by row, the state by block, keys by warp.
#include "tbe_internal.cuh"

#include <algorithm>
#include <cmath>

namespace tbe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 64;     // tokens
constexpr int kThreads = 128; // four warps: 16 rows of a tile each
constexpr int kPowers = kTile + 2;
constexpr int kMaxPasses = 3;

__device__ __forceinline__ void wait_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One recurrence.  Heads and tokens are `h*` and `s*` elements apart.
struct Pass {
  const uint16_t *q, *k, *v;
  int64_t sq, sk, sv, hq, hk, hv;
  uint16_t* o;
  int64_t so, ho;
  const float* in;     // [sequences, heads, d, d] or null
  float* out;          // likewise
  int32_t in_turned;   // `in` holds the transposes
  int32_t back;        // from the last token to the first, decay behind the read
  int32_t piece;       // bytes that rows are read by,
  int32_t piece_o;     //   and written by
  float scale_tile, scale_add, scale_read;
  float* carry;        // [heads, runs, DK, DK]: what each run leaves to the next
  int32_t* kind;       // [runs]
};
struct Args {
  Pass pass[kMaxPasses];
  const float* decay;
  IdxPtr offsets;
  int64_t N;
  int32_t S, H, d;
  int32_t tiles;   // of a run
  int32_t runs;
  int32_t parts;   // of the value columns
  int32_t* status;
};
// What a run leaves: nothing, the state of a sequence that began in it, or
// one that came in at its start and goes on behind it.
enum Kind : int32_t { kNothing, kBegan, kThrough };

// The sequences' first positions, counted from the end that the pass begins at.
struct Starts {
  IdxPtr p;
  int64_t N;
  int32_t S;
  bool back;
  __device__ __forceinline__ int64_t at(int64_t i) const { return back ? N - p.ldg(S - i) : p.ldg(i); }
  __device__ __forceinline__ int32_t sequence(int64_t i) const { return (int32_t)(back ? S - 1 - i : i); }
  // the first i with at(i) >= x, of all or of lo .. hi
  __device__ int64_t first(int64_t x) const { return first_from(x, 0, (int64_t)S + 1); }
  __device__ int64_t first_from(int64_t x, int64_t lo, int64_t hi) const {
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (at(mid) >= x) hi = mid; else lo = mid + 1;
    }
    return lo;
  }
};

__device__ __forceinline__ float power(float decay, int64_t n) { return n == 0 ? 1.f : exp2f(-(float)n * decay * kLog2e); }

// ---------------------------------------------------------------------------
// fragments
// ---------------------------------------------------------------------------

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (DT == TBE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if (DT == TBE_BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <int DT>
__device__ __forceinline__ float to_float(uint16_t u) {
  return unpack2<DT>(u).x;
}

template <int DT>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (DT == TBE_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b alone.
template <int DT>
__device__ __forceinline__ void mma_first(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (DT == TBE_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void ldsm(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Powers of two for fp16: what brings values of magnitude `top` to 2^14 or
// just below, as an exponent (kept where fp32 stays normal).
__device__ __forceinline__ int room_for(float top) {
  const int e = (int)(__float_as_uint(top) >> 23 & 255) - 127;  // 128 for infinities and NaN
  return max(-100, min(60, 13 - e));
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// ---------------------------------------------------------------------------
// a block's shared memory
// ---------------------------------------------------------------------------

// Rows are padded by 16 bytes: eight rows of a fragment then lie in different banks.
template <int DK>
struct Shape {
  static constexpr int DV = DK < 64 ? DK : 64;
  static constexpr int LK = DK + 8, LV = DV + 8;
  // the state over the warps: MT x NT pieces of 16 x 8 each
  static constexpr int MT = DK / 64 > 0 ? DK / 64 : 1;
  static constexpr int NT = DK >= 64 ? DV / 8 : DV / 16;
  static constexpr int NO = DV / 8;  // pieces of 8 columns of the outputs
  static constexpr int KS = DK / 16;
};
template <int DK>
struct Shared {
  using D = Shape<DK>;
  uint16_t q[kTile * D::LK], k[kTile * D::LK], v[kTile * D::LV], s[DK * D::LV];
  float pow[kPowers];
  unsigned long long starts;  // places of the tile where a sequence starts
  int32_t sequence[kTile];    // and which
  int32_t closes;             // a sequence ends at the tile's end
  int64_t next_at;            // the first start behind it
  uint32_t top[3];            // largest magnitudes of the state, in turn
};

// The kTile rows of one head from position p on, COLS of their columns, to
// shared memory; zeros behind the last row (n) and column.
template <int COLS, int LD>
__device__ __forceinline__ void load_rows(uint16_t* dst, const uint16_t* src, int64_t stride, int64_t p, int n, int cols,
                                          int64_t N, bool back, int piece) {
  const int64_t first = back ? N - 1 - p : p, step = back ? -stride : stride;  // row r is first * stride + r * step
  if (piece == 16) {
    constexpr int kPerRow = COLS / 8, kRowsAtOnce = kThreads / kPerRow;
    const int r0 = threadIdx.x / kPerRow, c = threadIdx.x % kPerRow * 8;
    const uint16_t* from = src + first * stride + r0 * step + c;
    uint32_t to = smem_u32(dst + r0 * LD + c);
    const int rows = c < cols ? n - r0 : 0;  // this thread's row k * kRowsAtOnce is there where that is below
#pragma unroll
    for (int k = 0; k < kTile / kRowsAtOnce; ++k) {
      const bool in = k * kRowsAtOnce < rows;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(in ? from : src), "r"(in ? 16 : 0)
                   : "memory");
      from += kRowsAtOnce * step;
      to += kRowsAtOnce * LD * 2;
    }
    return;
  }
  const int each = piece / 2, per_row = COLS / each;
  for (int i = threadIdx.x; i < kTile * per_row; i += kThreads) {
    const int r = i / per_row, c = (i - r * per_row) * each;
    const bool in = r < n && c < cols;
    const uint16_t* from = in ? src + first * stride + r * step + c : src;
    uint16_t* to = dst + r * LD + c;
    const uint32_t bytes = in ? piece : 0;
    if (piece == 8)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(bytes) : "memory");
    else if (piece == 4)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(bytes) : "memory");
    else
      *to = in ? __ldg(from) : 0;
  }
}

// ---------------------------------------------------------------------------
// the state of a block, in registers
// ---------------------------------------------------------------------------

template <int DT, int DK>
struct State {
  using D = Shape<DK>;
  float s[D::MT][D::NT][4];
  int m0, n0;  // the warp's first key row and value column

  __device__ __forceinline__ void place(int warp) {
    if (DK >= 64) {
      m0 = warp * D::MT * 16;
      n0 = 0;
    } else {
      m0 = warp % 2 * 16;
      n0 = warp / 2 * (DK / 2);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < D::MT; ++m)
#pragma unroll
      for (int n = 0; n < D::NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][n][e] = 0.f;
  }
  // Calls f(value, key row, value column) for each element held.
  template <typename F>
  __device__ __forceinline__ void each(int lane, F f) {
#pragma unroll
    for (int m = 0; m < D::MT; ++m)
#pragma unroll
      for (int n = 0; n < D::NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f(s[m][n][e], m0 + m * 16 + lane / 4 + (e >> 1) * 8, n0 + n * 8 + lane % 4 * 2 + (e & 1));
  }
  // A [d, d] matrix, or its transpose; `first` is the block's first value column.
  __device__ __forceinline__ void read(const float* p, int d, int first, bool turned, int lane) {
    each(lane, [&](float& x, int i, int j) {
      j += first;
      x = i < d && j < d ? __ldg(p + (turned ? (int64_t)j * d + i : (int64_t)i * d + j)) : 0.f;
    });
  }
  __device__ __forceinline__ void write(float* p, int d, int first, int lane) {
    each(lane, [&](float& x, int i, int j) {
      j += first;
      if (i < d && j < d) p[(int64_t)i * d + j] = x;
    });
  }
  __device__ __forceinline__ float largest() const {
    float t = 0.f;
#pragma unroll
    for (int m = 0; m < D::MT; ++m)
#pragma unroll
      for (int n = 0; n < D::NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) t = fmaxf(t, fabsf(s[m][n][e]));
    return t;
  }
  // To shared memory in the inputs' type, times 2^up.
  __device__ __forceinline__ void publish(Shared<DK>& sh, int lane, int up) const {
    const float f = DT == TBE_F16 ? pow2(up) : 1.f;
#pragma unroll
    for (int m = 0; m < D::MT; ++m)
#pragma unroll
      for (int n = 0; n < D::NT; ++n) {
        uint16_t* at = sh.s + (m0 + m * 16 + lane / 4) * D::LV + n0 + n * 8 + lane % 4 * 2;
        *reinterpret_cast<uint32_t*>(at) = pack2<DT>(s[m][n][0] * f, s[m][n][1] * f);
        *reinterpret_cast<uint32_t*>(at + 8 * D::LV) = pack2<DT>(s[m][n][2] * f, s[m][n][3] * f);
      }
  }

  // S = gamma^(b - a) S + sum over rows a..b-1 of scale gamma^(b - 1 - row + late) k v^T.
  // EXACT: a state that is a result.  One that is only read, rounded to 16
  // bits, takes two terms of bf16 (16 bits) and the tensor cores' own sums.
  template <bool EXACT>
  __device__ __forceinline__ void add(const Shared<DK>& sh, int a, int b, int late, float scale, int lane) {
    const uint32_t keys = smem_u32(sh.k) + ((lane % 8 + lane / 16 * 8) * D::LK + m0 + lane / 8 % 2 * 8) * 2;
    const uint32_t values = smem_u32(sh.v) + ((lane % 8 + lane / 8 % 2 * 8) * D::LV + n0 + lane / 16 * 8) * 2;
    const int k0 = a / 16, k1 = (b + 15) / 16;
    int up = 0;
    if (DT == TBE_F16) {
      // the largest key of this warp's rows, decayed or not
      __half2 top = __half2half2(__ushort_as_half(0));
      for (int ks = k0; ks < k1; ++ks)
#pragma unroll
        for (int m = 0; m < D::MT; ++m) {
          uint32_t r[4];
          ldsm_t(r, keys + (ks * 16 * D::LK + m * 16) * 2);
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(*reinterpret_cast<const __half2*>(&r[e])));
        }
      const float2 t = __half22float2(top);
      float most = fmaxf(t.x, t.y) * fabsf(scale);
#pragma unroll
      for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
      up = room_for(most);
    }
    const float down = DT == TBE_F16 ? pow2(-up) : 1.f;
    // (not EXACT: the sum itself is moved, and moved back)
    const float by = sh.pow[b - a] * (DT == TBE_F16 && !EXACT ? pow2(up) : 1.f);
    each(lane, [&](float& x, int, int) { x *= by; });
    const float weigh = scale * (DT == TBE_F16 ? pow2(up) : 1.f);
    const bool cut = (a | b) & 15;  // some step of 16 has rows of others
    for (int ks = k0; ks < k1; ++ks) {
      // weights of the four tokens whose keys and values this lane holds
      float w[4];
      uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
      const int t0 = ks * 16 + lane % 4 * 2;
      if (cut) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = t0 + h * 8;
          const bool in0 = t >= a && t < b, in1 = t + 1 >= a && t + 1 < b;
          w[2 * h] = in0 ? sh.pow[b - 1 - t + late] * weigh : 0.f;
          w[2 * h + 1] = in1 ? sh.pow[b - 2 - t + late] * weigh : 0.f;
          keep[h] = (in0 ? 0xffffu : 0u) | (in1 ? 0xffff0000u : 0u);
        }
      } else {
        const float* pw = sh.pow + (b - 1 - t0 + late);
        w[0] = pw[0] * weigh;
        w[1] = pw[-1] * weigh;
        w[2] = pw[-8] * weigh;
        w[3] = pw[-9] * weigh;
      }
      constexpr int kTerms = DT == TBE_BF16 && EXACT ? 3 : 2;
      uint32_t f[D::MT][kTerms][4];
#pragma unroll
      for (int m = 0; m < D::MT; ++m) {
        uint32_t r[4];
        ldsm_t(r, keys + (ks * 16 * D::LK + m * 16) * 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (what stands in rows of other sequences is left out before it is multiplied)
          float2 x = unpack2<DT>(r[e] & keep[e >> 1]);
          x.x *= w[e >> 1 << 1];
          x.y *= w[(e >> 1 << 1) + 1];
#pragma unroll
          for (int t = 0; t < kTerms; ++t) {
            if (DT == TBE_BF16 && t < kTerms - 1) {  // cut off: its two halves are the numbers' upper ones
              f[m][t][e] = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
              x.x -= __uint_as_float(__float_as_uint(x.x) & 0xffff0000u);
              x.y -= __uint_as_float(__float_as_uint(x.y) & 0xffff0000u);
            } else {
              f[m][t][e] = pack2<DT>(x.x, x.y);
              if (t < kTerms - 1) {
                const float2 y = unpack2<DT>(f[m][t][e]);
                x.x -= y.x;
                x.y -= y.y;
              }
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < D::NT; n += 2) {
        uint32_t r[4];
        ldsm_t(r, values + (ks * 16 * D::LV + n * 8) * 2);
        if (cut) {
#pragma unroll
          for (int e = 0; e < 4; ++e) r[e] &= keep[e & 1];
        }
#pragma unroll
        for (int m = 0; m < D::MT; ++m)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (EXACT) {
              // added up apart: the tensor cores cut sums off, which a long sum would feel
              float c[4];
              mma_first<DT>(c, f[m][kTerms - 1], r[2 * u], r[2 * u + 1]);
#pragma unroll
              for (int t = kTerms - 2; t >= 0; --t) mma<DT>(c, f[m][t], r[2 * u], r[2 * u + 1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) s[m][n + u][e] = DT == TBE_F16 ? fmaf(c[e], down, s[m][n + u][e]) : s[m][n + u][e] + c[e];
            } else {
#pragma unroll
              for (int t = kTerms - 1; t >= 0; --t) mma<DT>(s[m][n + u], f[m][t], r[2 * u], r[2 * u + 1]);
            }
          }
      }
    }
    if (DT == TBE_F16 && !EXACT) each(lane, [&](float& x, int, int) { x *= down; });
  }
};

// ---------------------------------------------------------------------------
// where sequences start in a tile
// ---------------------------------------------------------------------------

// A tile's sequences.
struct Marks {
  unsigned long long starts;  // places where one starts
  int n;                      // places taken
  bool closes;                // a sequence ends at its end
};
// Notes the starts below p + n, n at most kTile, in shared memory, and moves
// `next`, the first start not yet passed (at next_at), on.  Where the tile
// need not reach its end (`may_cut`) and its last sequence neither ends there
// nor fills it, the tile ends where that sequence starts: short sequences are
// then never cut, and need no state.  All threads call it.
template <int DK>
__device__ __forceinline__ Marks mark_starts(Shared<DK>& sh, const Starts& st, int64_t p, int n, bool may_cut, int64_t& next,
                                             int64_t& next_at) {
  Marks m = {0, n, false};
  if (next_at >= p + n) {  // none
    m.closes = next_at == p + n;
    return m;
  }
  if (threadIdx.x == 0) {
    sh.starts = 0;
    sh.closes = 0;
  }
  if (threadIdx.x < kTile) sh.sequence[threadIdx.x] = -1;
  __syncthreads();
  const int64_t before = next;
  int64_t i, x;
  int c;
  for (;;) {
    i = next + threadIdx.x;
    x = i <= st.S ? st.at(i) : INT64_MAX;
    const bool below = x < p + n;
    if (below && x >= p && i < st.S) {
      atomicOr(&sh.starts, 1ull << (x - p));
      atomicMax(&sh.sequence[x - p], (int32_t)i);  // empty sequences start there too: the last one has the tokens
    }
    if (x == p + n) sh.closes = 1;
    c = __syncthreads_count(below);
    if (c < kThreads) break;
    next += c;
  }
  m.starts = sh.starts;
  m.closes = sh.closes != 0;
  const int last = m.starts ? 63 - __clzll((long long)m.starts) : 0;
  if (may_cut && !m.closes && last > 0) {
    m.n = last;
    m.starts &= ~(1ull << last);
    m.closes = true;
    c = __syncthreads_count(x < p + last);
    if (c == 0 && next > before) {  // (more empty sequences than threads: back to the first that starts there)
      next = st.first_from(p + last, before, next);
      next_at = p + last;
      return m;
    }
  }
  if (threadIdx.x == c) sh.next_at = x;  // the first that is not below
  next += c;
  __syncthreads();
  next_at = sh.next_at;
  return m;
}

// ---------------------------------------------------------------------------
// what runs leave
// ---------------------------------------------------------------------------

template <int DT, int DK>
__global__ void __launch_bounds__(kThreads) carry_kernel(const __grid_constant__ Args a) {
  using D = Shape<DK>;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared<DK>& sh = *reinterpret_cast<Shared<DK>*>(raw);
  const Pass& ps = a.pass[blockIdx.y];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % a.parts, head = blockIdx.x / a.parts % a.H, run = blockIdx.x / (a.parts * a.H);
  const int64_t p0 = (int64_t)run * a.tiles * kTile, p1 = p0 + (int64_t)a.tiles * kTile;  // (the last run is not asked)
  const Starts st = {a.offsets, a.N, a.S, ps.back != 0};
  const int64_t next = st.first(p1);  // first start at or behind the run's end
  const bool goes_on = next <= a.S && st.at(next) > p1 && next > 0;
  const int64_t begin = goes_on ? st.at(next - 1) : p1;
  const int32_t kind = !goes_on ? kNothing : begin >= p0 ? kBegan : kThrough;
  if (threadIdx.x == 0 && part == 0 && head == 0) ps.kind[run] = kind;
  if (kind == kNothing) return;
  const float decay = a.decay[head];
  for (int k = threadIdx.x; k < kPowers; k += kThreads) sh.pow[k] = power(decay, k);
  State<DT, DK> state;
  state.place(warp);
  if (kind == kBegan && ps.in)
    state.read(ps.in + ((int64_t)st.sequence(next - 1) * a.H + head) * a.d * a.d, a.d, part * D::DV, ps.in_turned, lane);
  else state.clear();
  const int64_t from = max(begin, p0);
  for (int64_t p = from / kTile * kTile; p < p1; p += kTile) {
    __syncthreads();
    load_rows<DK, D::LK>(sh.k, ps.k + head * ps.hk, ps.sk, p, kTile, a.d, a.N, ps.back, ps.piece);
    load_rows<D::DV, D::LV>(sh.v, ps.v + head * ps.hv + part * D::DV, ps.sv, p, kTile, a.d - part * D::DV, a.N, ps.back,
                            ps.piece);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    const int a0 = (int)max(from - p, (int64_t)0);
    if (ps.out) state.template add<true>(sh, a0, kTile, ps.back, ps.scale_add, lane);
    else state.template add<false>(sh, a0, kTile, ps.back, ps.scale_add, lane);
  }
  float* out = ps.carry + ((int64_t)head * a.runs + run) * DK * DK;
  state.each(lane, [&](float& x, int i, int j) { out[i * DK + part * D::DV + j] = x; });
}

// carry[run] = what run `run` leaves, with what came through it.
template <int DK>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a) {
  wait_predecessor();
  const Pass& ps = a.pass[blockIdx.y];
  constexpr int kPerHead = DK * DK / 256;
  const int head = blockIdx.x / kPerHead, at = blockIdx.x % kPerHead * 256 + threadIdx.x;
  const float through = power(a.decay[head], (int64_t)a.tiles * kTile);
  float* c = ps.carry + (int64_t)head * a.runs * DK * DK + at;
  float s = 0.f;
  constexpr int kAhead = 16;
  for (int r = 0; r < a.runs - 1; r += kAhead) {
    float x[kAhead];
    int32_t kind[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {  // (what is not there to be read is not used either)
      const int at_run = min(r + k, a.runs - 2);
      kind[k] = __ldcg(ps.kind + at_run);
      x[k] = __ldcg(c + (int64_t)at_run * DK * DK);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (r + k >= a.runs - 1) break;
      if (kind[k] == kThrough) {
        s = fmaf(through, s, x[k]);
        c[(int64_t)(r + k) * DK * DK] = s;
      } else {
        s = x[k];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the outputs
// ---------------------------------------------------------------------------

// Resident blocks of an SM.
template <int DK>
constexpr int kBlocks = DK == 128 ? 3 : 4;

// Whether any of the tile's values is an infinity or a NaN.
template <int DT, int DK>
__device__ __forceinline__ bool not_finite(const Shared<DK>& sh) {
  using D = Shape<DK>;
  constexpr uint32_t kInf = DT == TBE_BF16 ? 0x7f80u : 0x7c00u;
  bool bad = false;
  for (int i = threadIdx.x; i < kTile * D::DV / 8; i += kThreads) {
    const uint4 u = *reinterpret_cast<const uint4*>(sh.v + i / (D::DV / 8) * D::LV + i % (D::DV / 8) * 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t x = (&u.x)[e];
      bad |= (x & kInf) == kInf || (x >> 16 & kInf) == kInf;
    }
  }
  return bad;
}

template <int DT, int DK>
__global__ void __launch_bounds__(kThreads, kBlocks<DK>) output_kernel(const __grid_constant__ Args a) {
  using D = Shape<DK>;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared<DK>& sh = *reinterpret_cast<Shared<DK>*>(raw);
  const Pass& ps = a.pass[blockIdx.y];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % a.parts, head = blockIdx.x / a.parts % a.H, run = blockIdx.x / (a.parts * a.H);
  const int64_t p0 = (int64_t)run * a.tiles * kTile, p1 = min(a.N, p0 + (int64_t)a.tiles * kTile);
  const Starts st = {a.offsets, a.N, a.S, ps.back != 0};
  const int first_col = part * D::DV;
  const int late = ps.back;
  wait_predecessor();
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // broken offsets are reported
    bool bad = false;
    for (int64_t i = threadIdx.x; i < a.S; i += kThreads) bad |= a.offsets.ldg(i) > a.offsets.ldg(i + 1);
    if (threadIdx.x == 0) bad |= a.offsets.ldg(0) != 0 || a.offsets.ldg(a.S) != a.N;
    if (bad) report(a.status, TBE_DEV_BAD_OFFSETS);
  }
  const float decay = a.decay[head];
  for (int k = threadIdx.x; k < kPowers; k += kThreads) sh.pow[k] = power(decay, k);
  if (threadIdx.x < 3) sh.top[threadIdx.x] = 0;
  int64_t next = st.first(p0);
  int64_t next_at = next <= a.S ? st.at(next) : INT64_MAX;

  State<DT, DK> state;
  state.place(warp);
  state.clear();
  bool live = false;      // there is a state, in registers and in shared memory
  uint32_t turn = 0;      // of sh.top
  float read_scale = 0.f; // what the state in shared memory is to be multiplied by
  // All threads: the state's registers to shared memory (after a barrier
  // behind which nobody reads the old one; a barrier must follow).
  auto note_top = [&] {
    if (DT == TBE_F16) {
      float t = state.largest();
#pragma unroll
      for (int o = 16; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, o));
      if (lane == 0) atomicMax(&sh.top[turn % 3], __float_as_uint(t));
    }
  };
  auto publish = [&] {
    int up = 0;
    if (DT == TBE_F16) {
      up = room_for(__uint_as_float(sh.top[turn % 3]));
      if (threadIdx.x == 0) sh.top[(turn + 2) % 3] = 0;
      ++turn;
    }
    state.publish(sh, lane, up);
    read_scale = ps.scale_read * (DT == TBE_F16 ? pow2(-up) : 1.f);
  };
  __syncthreads();
  if (next_at > p0 && run > 0) {
    const float* c = ps.carry + ((int64_t)head * a.runs + run - 1) * DK * DK;
    state.each(lane, [&](float& x, int i, int j) { x = __ldcg(c + i * DK + first_col + j); });
    live = true;
    note_top();
    __syncthreads();
    publish();
  }

  const uint32_t queries = smem_u32(sh.q) + ((warp * 16 + lane % 16) * D::LK + lane / 16 * 8) * 2;
  const uint32_t keys = smem_u32(sh.k) + ((lane % 8 + lane / 16 * 8) * D::LK + lane / 8 % 2 * 8) * 2;
  const uint32_t values = smem_u32(sh.v) + ((lane % 8 + lane / 8 % 2 * 8) * D::LV + lane / 16 * 8) * 2;
  const uint32_t stored = smem_u32(sh.s) + ((lane % 8 + lane / 8 % 2 * 8) * D::LV + lane / 16 * 8) * 2;
  const int row0 = warp * 16 + lane / 4;  // this lane's rows are row0 and row0 + 8

  // what the products of a row and a column of another 16 are multiplied by has a part for each
  float by_col[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) by_col[e] = sh.pow[15 - (lane % 4 * 2 + (e & 1) + (e >> 1) * 8)] * ps.scale_tile;

  for (int64_t p = p0; p < p1;) {
    const int most = (int)min((int64_t)kTile, p1 - p);
    const int64_t came = next - 1;  // the sequence that comes in, where there is one
    load_rows<DK, D::LK>(sh.q, ps.q + head * ps.hq, ps.sq, p, most, a.d, a.N, ps.back, ps.piece);
    load_rows<DK, D::LK>(sh.k, ps.k + head * ps.hk, ps.sk, p, most, a.d, a.N, ps.back, ps.piece);
    load_rows<D::DV, D::LV>(sh.v, ps.v + head * ps.hv + first_col, ps.sv, p, most, a.d - first_col, a.N, ps.back, ps.piece);
    cp_commit();
    const Marks mk = mark_starts(sh, st, p, most, p + most < p1, next, next_at);
    const unsigned long long starts = mk.starts;
    const int n = mk.n;
    const bool closes = mk.closes, last_tile = p + n >= p1;
    const bool whole = (starts & ~1ull) == 0;  // one sequence has all of the tile
    cp_wait<0>();
    __syncthreads();

    float o[D::NO][4];
#pragma unroll
    for (int j = 0; j < D::NO; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    uint32_t qf[D::KS][4];
#pragma unroll
    for (int k = 0; k < D::KS; ++k) ldsm(qf[k], queries + k * 32);

    // the state's part, sequence by sequence
    for (int at = 0; at < n;) {
      const bool begins = starts >> at & 1;
      const unsigned long long later = at < 63 ? starts >> (at + 1) << (at + 1) : 0;
      const int end = later ? __ffsll((long long)later) - 1 : n;
      const int64_t which = begins ? sh.sequence[at] : came;
      const bool known = which >= 0 && which < a.S;  // (always, unless offsets are broken)
      const bool ends = end < n || closes;
      const int64_t matrix = ((int64_t)st.sequence(which) * a.H + head) * a.d * a.d;
      if (begins) {
        live = ps.in != nullptr;
        if (live) {
          state.read(ps.in + matrix, a.d, first_col, ps.in_turned, lane);
          note_top();
          __syncthreads();  // the state before it has been read
          publish();
          __syncthreads();
        } else {
          state.clear();
        }
      }
      if (live) {
        float f[2];
        bool mine[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = row0 + half * 8;
          mine[half] = row >= at && row < end;
          f[half] = mine[half] ? sh.pow[row - at + 1 - late] * read_scale : 0.f;
        }
#pragma unroll
        for (int j0 = 0; j0 < D::NO; j0 += 4) {
          float r[4][4];
#pragma unroll
          for (int k = 0; k < D::KS; ++k)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              uint32_t b[4];
              ldsm_t(b, stored + (k * 16 * D::LV + (j0 + j) * 8) * 2);
              if (k == 0) {
                mma_first<DT>(r[j], qf[k], b[0], b[1]);
                mma_first<DT>(r[j + 1], qf[k], b[2], b[3]);
              } else {
                mma<DT>(r[j], qf[k], b[0], b[1]);
                mma<DT>(r[j + 1], qf[k], b[2], b[3]);
              }
            }
          // (chosen by row, not added up: what the state holds stays in its sequence)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j0 + j][e] = mine[e >> 1] ? r[j][e] * f[e >> 1] : o[j0 + j][e];
        }
      }
      if (ends ? ps.out != nullptr && known : !last_tile) {
        if (ps.out) state.template add<true>(sh, at, end, late, ps.scale_add, lane);
        else state.template add<false>(sh, at, end, late, ps.scale_add, lane);
        live = true;
        if (ends) state.write(ps.out + matrix, a.d, first_col, lane);
      }
      if (ends) live = false;
      at = end;
    }

    // the tile's own part: 16 rows of keys at a time
    // (rows of other sequences, and those behind a tile that was cut, are multiplied by 0)
    const bool apart = !(whole && n == most) && __syncthreads_or(not_finite<DT, DK>(sh));
    // first row of each of this lane's rows' sequences
    int from[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const unsigned long long upto = starts << (63 - (row0 + half * 8));
      from[half] = upto ? row0 + half * 8 - __clzll((long long)upto) : 0;
    }
    int up[2] = {0, 0};  // fp16: what the rows' outputs are held multiplied by, as exponents
    for (int j = 0; j <= warp; ++j) {
      float c[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) c[0][e] = c[1][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D::KS; ++k) {
        uint32_t b[4];
        ldsm(b, keys + (j * 16 * D::LK + k * 16) * 2);
        mma<DT>(c[0], qf[k], b[0], b[1]);
        mma<DT>(c[1], qf[k], b[2], b[3]);
      }
      if (j < warp) {
        const float by_row[2] = {sh.pow[row0 - j * 16 - 15], sh.pow[row0 + 8 - j * 16 - 15]};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[t][e] *= by_row[e >> 1] * by_col[t * 2 + (e & 1)];
        if (!whole) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j * 16 + t * 8 + lane % 4 * 2 + (e & 1) < from[e >> 1]) c[t][e] = 0.f;
        }
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int half = e >> 1, s = j * 16 + t * 8 + lane % 4 * 2 + (e & 1), away = row0 + half * 8 - s;
            c[t][e] = away >= 0 && s >= from[half] ? c[t][e] * (sh.pow[away & 63] * ps.scale_tile) : 0.f;
          }
      }
      float top[2];
#pragma unroll
      for (int half = 0; half < 2; ++half)
        top[half] = fmaxf(fmaxf(fabsf(c[0][2 * half]), fabsf(c[0][2 * half + 1])),
                          fmaxf(fabsf(c[1][2 * half]), fabsf(c[1][2 * half + 1])));
      if (DT == TBE_F16) {
        bool moves = j == 0;
        int want[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          top[half] = fmaxf(top[half], __shfl_xor_sync(kFull, top[half], 1));
          top[half] = fmaxf(top[half], __shfl_xor_sync(kFull, top[half], 2));
          // outputs so far are moved too: no further up than by 2^24
          want[half] = min(24, room_for(top[half]));
          moves |= want[half] < up[half];
        }
        if (__any_sync(kFull, moves)) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int to = j == 0 ? want[half] : min(want[half], up[half]);
            const float f = pow2(to - up[half]);
#pragma unroll
            for (int i = 0; i < D::NO; ++i) {
              o[i][2 * half] *= f;
              o[i][2 * half + 1] *= f;
            }
            up[half] = to;
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[t][e] *= pow2(up[e >> 1]);
      }
      const uint32_t w[4] = {pack2<DT>(c[0][0], c[0][1]), pack2<DT>(c[0][2], c[0][3]), pack2<DT>(c[1][0], c[1][1]),
                             pack2<DT>(c[1][2], c[1][3])};
      if (!apart) {
#pragma unroll
        for (int i = 0; i < D::NO; i += 2) {
          uint32_t b[4];
          ldsm_t(b, values + (j * 16 * D::LV + i * 8) * 2);
          mma<DT>(o[i], w, b[0], b[1]);
          mma<DT>(o[i + 1], w, b[2], b[3]);
        }
      } else {
        // some value is no number: each sequence's rows take its own values only, so that it stays in its sequence
        for (int at = 0; at < n;) {
          const unsigned long long later = at < 63 ? starts >> (at + 1) << (at + 1) : 0;
          const int end = later ? __ffsll((long long)later) - 1 : n;
          uint32_t keep[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = j * 16 + lane % 4 * 2 + h * 8;
            keep[h] = (t >= at && t < end ? 0xffffu : 0u) | (t + 1 >= at && t + 1 < end ? 0xffff0000u : 0u);
          }
          const bool mine[2] = {row0 >= at && row0 < end, row0 + 8 >= at && row0 + 8 < end};
#pragma unroll
          for (int i = 0; i < D::NO; i += 2) {
            uint32_t b[4];
            ldsm_t(b, values + (j * 16 * D::LV + i * 8) * 2);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float r[4] = {o[i + u][0], o[i + u][1], o[i + u][2], o[i + u][3]};
              mma<DT>(r, w, b[2 * u] & keep[0], b[2 * u + 1] & keep[1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i + u][e] = mine[e >> 1] ? r[e] : o[i + u][e];
            }
          }
          at = end;
        }
      }
    }
    // this warp's rows go out through its own rows of the queries, which only it read
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float f = DT == TBE_F16 ? pow2(-up[half]) : 1.f;
#pragma unroll
      for (int j = 0; j < D::NO; ++j)
        *reinterpret_cast<uint32_t*>(sh.q + (row0 + half * 8) * D::LK + j * 8 + lane % 4 * 2) =
            pack2<DT>(o[j][2 * half] * f, o[j][2 * half + 1] * f);
    }
    __syncwarp();
    {
      const int cols = min(D::DV, a.d - first_col), each = ps.piece_o / 2, per_row = (cols + each - 1) / each;
      for (int i = lane; i < 16 * per_row; i += 32) {
        const int r = warp * 16 + i / per_row, c = i % per_row * each;
        if (r >= n) break;
        const int64_t token = ps.back ? a.N - 1 - (p + r) : p + r;
        uint16_t* to = ps.o + token * ps.so + head * ps.ho + first_col + c;
        const uint16_t* src = sh.q + r * D::LK + c;
        if (each == 8) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(src);
        else if (each == 4) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(src);
        else if (each == 2) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(src);
        else *to = *src;
      }
    }
    const bool keep_state = live && !last_tile;
    if (keep_state) note_top();
    __syncthreads();  // the tile and the state in shared memory have been read
    if (keep_state) publish();
    p += n;
  }
}

// States of sequences without tokens are handed on.
__global__ void __launch_bounds__(256) empty_kernel(const __grid_constant__ Args a) {
  wait_predecessor();
  const Pass& ps = a.pass[blockIdx.y];
  const int64_t s = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (s >= a.S || a.offsets.ldg(s) < a.offsets.ldg(s + 1)) return;
  const int64_t n = (int64_t)a.H * a.d * a.d;
  for (int64_t k = threadIdx.x & 31; k < n; k += 32) ps.out[s * n + k] = ps.in ? ps.in[s * n + k] : 0.f;
}

// ---------------------------------------------------------------------------
// single tokens
// ---------------------------------------------------------------------------

struct StepArgs {
  const uint16_t *q, *k, *v;
  int64_t sq, sk, sv, hq, hk, hv;
  uint16_t* o;
  int64_t so, ho;
  const float* decay;
  float* state;
  float scale;
  int32_t H, d;
};

constexpr int kStepThreads = 256;

// A block per sequence and head; VEC columns of the state to a lane.
template <int DT, int VEC>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const StepArgs a) {
  __shared__ float q[128], k[128], part[kStepThreads / 32][128];
  const int64_t s = blockIdx.x / a.H;
  const int head = (int)(blockIdx.x % a.H), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d = a.d;
  for (int i = threadIdx.x; i < d; i += kStepThreads) {
    q[i] = to_float<DT>(a.q[s * a.sq + head * a.hq + i]) * a.scale;
    k[i] = to_float<DT>(a.k[s * a.sk + head * a.hk + i]);
  }
  const float gamma = power(a.decay[head], 1);
  __syncthreads();
  float* m = a.state + (int64_t)blockIdx.x * d * d;
  for (int c = lane * VEC; c < d; c += 32 * VEC) {
    float v[VEC], o[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[e] = to_float<DT>(a.v[s * a.sv + head * a.hv + c + e]);
      o[e] = 0.f;
    }
#pragma unroll 8
    for (int i = warp; i < d; i += kStepThreads / 32) {
      float x[VEC];
      float* at = m + (int64_t)i * d + c;
      if (VEC == 4) {
        const float4 y = *reinterpret_cast<const float4*>(at);
        x[0] = y.x;
        x[1 % VEC] = y.y;
        x[2 % VEC] = y.z;
        x[3 % VEC] = y.w;
      } else {
        x[0] = *at;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[e] = fmaf(k[i], v[e], gamma * x[e]);
        o[e] = fmaf(q[i], x[e], o[e]);
      }
      if (VEC == 4) *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1 % VEC], x[2 % VEC], x[3 % VEC]);
      else *at = x[0];
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[warp][c + e] = o[e];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += kStepThreads) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kStepThreads / 32; ++w) o += part[w][c];
    a.o[s * a.so + head * a.ho + c] = (uint16_t)pack2<DT>(o, 0.f);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int width_of(int32_t d) { return d <= 32 ? 32 : d <= 64 ? 64 : 128; }
int parts_of(int32_t d) { return width_of(d) == 128 ? (d + 63) / 64 : 1; }

// Runs: as many blocks as the GPU holds at once.
struct Split {
  int32_t tiles, runs;
};
Split split_of(int64_t N, int32_t H, int32_t d, int passes) {
  const int64_t all = (N + kTile - 1) / kTile, want = std::max<int64_t>(1, (width_of(d) == 128 ? kBlocks<128> : kBlocks<64>) * (int64_t)sm_count() / ((int64_t)H * parts_of(d) * passes));
  Split s;
  s.tiles = (int32_t)std::max<int64_t>(1, (all + want - 1) / want);
  s.runs = (int32_t)std::max<int64_t>(1, (all + s.tiles - 1) / s.tiles);
  return s;
}
struct Layout {
  size_t carry, kind, bytes;  // of a pass
};
Layout layout(int64_t N, int32_t H, int32_t d, int passes) {
  const Split sp = split_of(N, H, d, passes);
  Layout w = {0, 0, 0};
  if (sp.runs > 1) {
    const size_t dk = width_of(d);
    w.kind = round256(sizeof(float) * (size_t)H * sp.runs * dk * dk);
    w.bytes = w.kind + round256(sizeof(int32_t) * (size_t)sp.runs);
  }
  return w;
}

int start(const void* kernel, dim3 grid, int threads, size_t smem, bool after, cudaStream_t s, const Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  void* args[] = {const_cast<Args*>(&a)};
  return cudaLaunchKernelExC(&cfg, kernel, args) == cudaSuccess ? check_launch() : TBE_ERR_CUDA;
}

template <int DT, int DK>
int launch(const Args& a, int passes, cudaStream_t s) {
  constexpr size_t smem = sizeof(Shared<DK>);
  const void *carry = (const void*)carry_kernel<DT, DK>, *output = (const void*)output_kernel<DT, DK>;
  static bool allowed[64] = {};  // once per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !allowed[dev]) {
    for (const void* f : {carry, output})
      if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return TBE_ERR_CUDA;
    if (dev >= 0 && dev < 64) allowed[dev] = true;
  }
  const unsigned per_run = (unsigned)(a.H * a.parts);
  bool after = false;
  int st;
  if (a.N > 0) {
    if (a.runs > 1) {
      if ((st = start(carry, dim3((unsigned)(a.runs - 1) * per_run, passes), kThreads, smem, false, s, a)) != TBE_OK) return st;
      trace_mark(s, "linear_attention_carry");
      const unsigned blocks = (unsigned)a.H * (DK * DK / 256);
      if ((st = start((const void*)join_kernel<DK>, dim3(blocks, passes), 256, 0, true, s, a)) != TBE_OK) return st;
      trace_mark(s, "linear_attention_join");
      after = true;
    }
    if ((st = start(output, dim3((unsigned)a.runs * per_run, passes), kThreads, smem, after, s, a)) != TBE_OK) return st;
    trace_mark(s, "linear_attention_output");
    after = true;
  }
  return TBE_OK;
}

template <int DT>
int dispatch(const Args& a, int passes, cudaStream_t s) {
  const int w = width_of(a.d);
  return w == 32 ? launch<DT, 32>(a, passes, s) : w == 64 ? launch<DT, 64>(a, passes, s) : launch<DT, 128>(a, passes, s);
}

// Bytes (2 to 16) that rows of d elements can be moved by.
int piece_of(const void* p, int64_t stride, int64_t head, int32_t d) {
  int n = 16;
  while (n > 2 && (((uintptr_t)p | (uintptr_t)(stride * 2) | (uintptr_t)(head * 2) | (uintptr_t)(d * 2)) & (n - 1))) n >>= 1;
  return n;
}

struct Rows {
  const void* p;
  int64_t stride, head;
};
bool fits(const Rows& r, int64_t N, int32_t H, int32_t d) {
  // heads of a token must not overlap, nor tokens; the two orders that do that
  return r.head >= d && r.stride >= d && (r.stride >= r.head * (H - 1) + d || (N <= 1) || r.head >= r.stride * (N - 1) + d);
}

int check(const tbe_linear_attention_inputs* in, bool jagged) {
  if (!in || in->dtype < TBE_F32 || in->dtype > TBE_BF16) return TBE_ERR_INVALID_ARG;
  if (in->tokens < 0 || in->sequences < 0 || in->heads < 1 || in->head_dim < 1 || !std::isfinite(in->scale))
    return TBE_ERR_INVALID_ARG;
  if (in->dtype == TBE_F32 || in->head_dim > TBE_LINEAR_MAX_HEAD_DIM || in->heads > (1 << 16) ||
      in->tokens >= (int64_t(1) << 36))
    return TBE_ERR_UNSUPPORTED;
  if (!in->decay || (in->tokens > 0 && (!in->q || !in->k || !in->v))) return TBE_ERR_INVALID_ARG;
  const Rows r[3] = {{in->q, in->q_stride, in->q_head_stride}, {in->k, in->k_stride, in->k_head_stride},
                     {in->v, in->v_stride, in->v_head_stride}};
  for (const Rows& x : r) {
    if (!fits(x, in->tokens, in->heads, in->head_dim)) return TBE_ERR_INVALID_ARG;
    if ((uintptr_t)x.p & 1) return TBE_ERR_UNSUPPORTED;
  }
  if (jagged && (!in->offsets || (in->tokens > 0 && in->sequences == 0))) return TBE_ERR_INVALID_ARG;
  if (((uintptr_t)in->s0 | (uintptr_t)in->decay) & 3) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

Args args_of(const tbe_linear_attention_inputs* in, int passes, int32_t* status) {
  Args a = {};
  a.decay = in->decay;
  a.offsets = IdxPtr{in->offsets, in->offsets_i32 != 0};
  a.N = in->tokens;
  a.S = in->sequences;
  a.H = in->heads;
  a.d = in->head_dim;
  const Split sp = split_of(a.N, a.H, a.d, passes);
  a.tiles = sp.tiles;
  a.runs = sp.runs;
  a.parts = parts_of(a.d);
  a.status = status;
  return a;
}

void set_rows(Pass& p, const Rows& q, const Rows& k, const Rows& v, const Rows& o, int32_t d) {
  p.q = static_cast<const uint16_t*>(q.p);
  p.sq = q.stride;
  p.hq = q.head;
  p.k = static_cast<const uint16_t*>(k.p);
  p.sk = k.stride;
  p.hk = k.head;
  p.v = static_cast<const uint16_t*>(v.p);
  p.sv = v.stride;
  p.hv = v.head;
  p.o = static_cast<uint16_t*>(const_cast<void*>(o.p));
  p.so = o.stride;
  p.ho = o.head;
  p.piece = std::min({piece_of(q.p, q.stride, q.head, d), piece_of(k.p, k.stride, k.head, d), piece_of(v.p, v.stride, v.head, d)});
  p.piece_o = piece_of(o.p, o.stride, o.head, d);
}

// Whether two [sequences, heads, d, d] states share memory: blocks read the
// one while others write the other.
bool overlap(const tbe_linear_attention_inputs* in, const float* p, const float* q) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  const size_t bytes = sizeof(float) * (size_t)in->sequences * in->heads * in->head_dim * in->head_dim;
  return p && q && a < b + bytes && b < a + bytes;
}

int go(Args& a, int passes, int32_t dtype, void* workspace, size_t bytes, cudaStream_t s) {
  const Layout w = layout(a.N, a.H, a.d, passes);
  if (bytes < passes * w.bytes) return TBE_ERR_WORKSPACE;
  if (w.bytes) {
    if (!workspace) return TBE_ERR_INVALID_ARG;
    if ((uintptr_t)workspace & 255) return TBE_ERR_UNSUPPORTED;
    for (int p = 0; p < passes; ++p) {
      uint8_t* at = static_cast<uint8_t*>(workspace) + p * w.bytes;
      a.pass[p].carry = reinterpret_cast<float*>(at);
      a.pass[p].kind = reinterpret_cast<int32_t*>(at + w.kind);
    }
  }
  if ((int64_t)a.runs * a.H * a.parts >= (int64_t(1) << 31)) return TBE_ERR_UNSUPPORTED;
  trace_begin(s);
  const int st = dtype == TBE_F16 ? dispatch<TBE_F16>(a, passes, s) : dispatch<TBE_BF16>(a, passes, s);
  if (st != TBE_OK) return st;
  for (int p = 0; p < passes; ++p)
    if (a.pass[p].out) {  // one at most
      Args e = a;
      e.pass[0] = a.pass[p];
      const int rc = start((const void*)empty_kernel, dim3((unsigned)((a.S + 7) / 8)), 256, 0, a.N > 0, s, e);
      trace_mark(s, "linear_attention_empty");
      return rc;
    }
  return TBE_OK;
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" {

size_t tbe_linear_attention_workspace_bytes(int64_t tokens, int32_t heads, int32_t head_dim, int32_t backward) {
  if (tokens < 0 || heads < 1 || head_dim < 1 || head_dim > TBE_LINEAR_MAX_HEAD_DIM) return 0;
  const int passes = backward ? 3 : 1;
  return passes * layout(tokens, heads, head_dim, passes).bytes;
}

int tbe_linear_attention(const tbe_linear_attention_inputs* in, void* o, int64_t o_stride, int64_t o_head_stride,
                         float* s_last, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  int st = check(in, true);
  if (st != TBE_OK) return st;
  const Rows out = {o, o_stride, o_head_stride};
  if ((in->tokens > 0 && !o) || !fits(out, in->tokens, in->heads, in->head_dim)) return TBE_ERR_INVALID_ARG;
  if (((uintptr_t)o & 1) || ((uintptr_t)s_last & 3)) return TBE_ERR_UNSUPPORTED;
  if (overlap(in, in->s0, s_last)) return TBE_ERR_INVALID_ARG;
  if (in->sequences == 0) return TBE_OK;
  Args a = args_of(in, 1, dev_status);
  Pass& p = a.pass[0];
  set_rows(p, {in->q, in->q_stride, in->q_head_stride}, {in->k, in->k_stride, in->k_head_stride},
           {in->v, in->v_stride, in->v_head_stride}, out, a.d);
  p.in = in->s0;
  p.out = s_last;
  p.scale_tile = p.scale_read = in->scale;
  p.scale_add = 1.f;
  return go(a, 1, in->dtype, workspace, workspace_bytes, (cudaStream_t)stream);
}

int tbe_linear_attention_backward(const tbe_linear_attention_inputs* in, const void* dout, int64_t do_stride,
                                  int64_t do_head_stride, const float* ds_last, const tbe_linear_attention_grads* g,
                                  void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  int st = check(in, true);
  if (st != TBE_OK) return st;
  if (!g || (in->tokens > 0 && (!dout || !g->dq || !g->dk || !g->dv))) return TBE_ERR_INVALID_ARG;
  const Rows q = {in->q, in->q_stride, in->q_head_stride}, k = {in->k, in->k_stride, in->k_head_stride},
             v = {in->v, in->v_stride, in->v_head_stride}, d = {dout, do_stride, do_head_stride},
             dq = {g->dq, g->dq_stride, g->dq_head_stride}, dk = {g->dk, g->dk_stride, g->dk_head_stride},
             dv = {g->dv, g->dv_stride, g->dv_head_stride};
  for (const Rows* r : {&d, &dq, &dk, &dv}) {
    if (!fits(*r, in->tokens, in->heads, in->head_dim)) return TBE_ERR_INVALID_ARG;
    if ((uintptr_t)r->p & 1) return TBE_ERR_UNSUPPORTED;
  }
  if (((uintptr_t)ds_last | (uintptr_t)g->ds0) & 3) return TBE_ERR_UNSUPPORTED;
  if (overlap(in, ds_last, g->ds0) || overlap(in, in->s0, g->ds0)) return TBE_ERR_INVALID_ARG;
  if (in->sequences == 0) return TBE_OK;
  Args a = args_of(in, 3, dev_status);
  set_rows(a.pass[0], d, v, k, dq, a.d);
  a.pass[0].in = in->s0;
  a.pass[0].in_turned = 1;
  a.pass[0].scale_tile = a.pass[0].scale_read = in->scale;
  a.pass[0].scale_add = 1.f;
  set_rows(a.pass[1], v, d, q, dk, a.d);
  a.pass[1].in_turned = 1;
  set_rows(a.pass[2], k, q, d, dv, a.d);
  a.pass[2].out = g->ds0;
  for (int i = 1; i < 3; ++i) {
    a.pass[i].in = ds_last;
    a.pass[i].back = 1;
    a.pass[i].scale_tile = a.pass[i].scale_add = in->scale;
    a.pass[i].scale_read = 1.f;
  }
  return go(a, 3, in->dtype, workspace, workspace_bytes, (cudaStream_t)stream);
}

int tbe_linear_attention_step(const tbe_linear_attention_inputs* in, float* state, void* o, int64_t o_stride,
                              int64_t o_head_stride, void* stream) {
  const int st = check(in, false);
  if (st != TBE_OK) return st;
  if (in->tokens != in->sequences || in->s0) return TBE_ERR_INVALID_ARG;
  if (in->sequences == 0) return TBE_OK;
  const Rows out = {o, o_stride, o_head_stride};
  if (!state || !o || !fits(out, in->tokens, in->heads, in->head_dim)) return TBE_ERR_INVALID_ARG;
  if (((uintptr_t)o & 1) || ((uintptr_t)state & 3)) return TBE_ERR_UNSUPPORTED;
  const int64_t blocks = (int64_t)in->sequences * in->heads;
  if (blocks >= (int64_t(1) << 31)) return TBE_ERR_UNSUPPORTED;
  StepArgs a = {};
  a.q = static_cast<const uint16_t*>(in->q);
  a.k = static_cast<const uint16_t*>(in->k);
  a.v = static_cast<const uint16_t*>(in->v);
  a.sq = in->q_stride;
  a.sk = in->k_stride;
  a.sv = in->v_stride;
  a.hq = in->q_head_stride;
  a.hk = in->k_head_stride;
  a.hv = in->v_head_stride;
  a.o = static_cast<uint16_t*>(o);
  a.so = o_stride;
  a.ho = o_head_stride;
  a.decay = in->decay;
  a.state = state;
  a.scale = in->scale;
  a.H = in->heads;
  a.d = in->head_dim;
  cudaStream_t s = (cudaStream_t)stream;
  trace_begin(s);
  const bool vec = a.d % 4 == 0 && ((uintptr_t)state & 15) == 0;
  const unsigned grid = (unsigned)blocks;
  if (in->dtype == TBE_F16) {
    if (vec) step_kernel<TBE_F16, 4><<<grid, kStepThreads, 0, s>>>(a);
    else step_kernel<TBE_F16, 1><<<grid, kStepThreads, 0, s>>>(a);
  } else {
    if (vec) step_kernel<TBE_BF16, 4><<<grid, kStepThreads, 0, s>>>(a);
    else step_kernel<TBE_BF16, 1><<<grid, kStepThreads, 0, s>>>(a);
  }
  const int rc = check_launch();
  trace_mark(s, "linear_attention_step");
  return rc;
}

}  // extern "C"
