// tbe_gated_scan.cu -- gated linear recurrence over jagged sequences, its
// backward pass and its form for single tokens.
//
//   u_t = sharpness * softplus(decay) * sigmoid(recur_t)      a_t = exp(-u_t)
//   h_t = a_t h_{t-1} + beta_t sigmoid(gate_t) x_t            beta_t = sqrt(1 - a_t^2)
//
// per channel, over every sequence of the jagged batch.  The sequences are
// scanned as one axis of N tokens: at a sequence's first token the recurrence
// is cut (its state enters as a term of its own), so the work splits into
// equal tiles of the token axis whatever the lengths are.
//
// A thread block takes a tile of kTile tokens x 32 lanes' channels: each warp
// a run of kStep tokens, each lane one or two neighbouring channels whose
// tokens it holds in registers.  h over a run is the linear map
// h_out = A h_in + B; the runs' maps are joined in shared memory, and the
// tiles' maps through one 8-byte word per (tile, channel) in the workspace.
// A tile's incoming state is always joined from the same maps in the same
// order -- the tiles before it in its group of kGroup, the groups before it
// in its row of kGroup groups, the last row's end -- so results do not
// depend on timing.  Every input is read once and every output written once.
//
// A map that contains a sequence start has no h_in; it is kept apart from
// A = 0 (which long decays reach by underflow) by A = -1, so that a NaN in
// one sequence never reaches the next.
#include "tbe_internal.cuh"

#include <cmath>

namespace tbe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kStep = 8;              // tokens per thread
constexpr int kTile = TBE_SCAN_TILE;  // tokens per thread block (and between saved states)
constexpr int kWarps = kTile / kStep;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 16;  // tiles joined by one group word, groups joined by one row word
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kEmpty = 0xffffffffu;  // a word nobody has written (the workspace is filled with it)
constexpr int kPolls = 1 << 20;  // of one thread, over all its waits

struct ScanArgs {
  const void* x;
  const void* r;
  const void* g;
  int64_t sx, sr, sg;  // elements between tokens
  const float* decay;
  float sharpness;
  IdxPtr offsets;
  int64_t N;
  int32_t S;
  int32_t C;
  int32_t tiles;     // along the tokens
  int32_t cblocks;   // along the channels
  const float* h0;   // [S, C] or null
  // forward
  void* h;           // [N, C]
  int64_t sh;
  float* h_last;     // [S, C]
  float* states;     // [tiles, C]: the state each tile starts from, or null
  // backward
  const void* dh;
  int64_t sdh;
  const float* dh_last;
  void* dx;
  void* dr;
  void* dg;
  int64_t sdx, sdr, sdg;
  float* dh0;
  float* partial;    // [tiles, C]: each tile's share of the decay's gradient
  // joining the tiles
  uint2* tile_word;   // [tiles, C]
  uint2* group_word;  // [groups, C]
  uint32_t* row_word; // [rows, C]
  uint32_t* ticket;
  int32_t* status;
};

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
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// a = exp(-u) and 1 - a^2 for u >= 0, both to a few units of their own
// size.  Below 1/4, m = a - 1 from its series (the next term is under 5e-8 of
// the sum): near a = 1 its rounding is relative to 1 - a, which is what
// decides how long a state lives, and 1 - a^2 = -m (2 + m) keeps it.
struct Decay {
  float a, q;
};
__device__ __forceinline__ Decay decay_of(float u) {
  float p = fmaf(u, 1.f / 720.f, -1.f / 120.f);
  p = fmaf(u, p, 1.f / 24.f);
  p = fmaf(u, p, -1.f / 6.f);
  p = fmaf(u, p, 0.5f);
  p = fmaf(u, p, -1.f);
  const float e = ex2(-kLog2e * u);
  const bool near = u < 0.25f;
  const float m = near ? u * p : e - 1.f;
  Decay d;
  d.a = near ? 1.f + m : e;
  d.q = -m * (2.f + m);
  return d;
}

// softplus of the decay parameter, once per thread
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
// sharpness * softplus; below the normal numbers, where fp32 keeps no
// relative precision, it counts as 0 (the channel keeps its state)
__device__ __forceinline__ float speed_of(const ScanArgs& a, int64_t c) {
  const float sp = softplus(a.decay[c]);
  return sp < 1.17549435e-38f ? 0.f : a.sharpness * sp;
}

// VEC neighbouring elements as raw bits and as floats.
template <int DT, int VEC>
struct Elems {
  static_assert(DT != TBE_F32 || VEC == 1, "fp32 takes one channel per lane");
  static constexpr int kBytes = (DT == TBE_F32 ? 4 : 2) * VEC;
  __device__ __forceinline__ static uint32_t load(const void* p) {
    uint32_t v;
    if (kBytes == 4) {
      asm volatile("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p));
    } else {
      uint16_t h;
      asm volatile("ld.global.nc.L1::no_allocate.b16 %0, [%1];" : "=h"(h) : "l"(p));
      v = h;
    }
    return v;
  }
  __device__ __forceinline__ static void unpack(uint32_t v, float* f) {
    if (DT == TBE_F32) {
      f[0] = __uint_as_float(v);
    } else if (DT == TBE_BF16) {
      f[0] = __uint_as_float(v << 16);
      if (VEC == 2) f[VEC - 1] = __uint_as_float(v & 0xffff0000u);
    } else {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&v));
      f[0] = h.x;
      if (VEC == 2) f[VEC - 1] = h.y;
    }
  }
  __device__ __forceinline__ static void store(void* p, const float* f) {
    if (DT == TBE_F32) {
      *static_cast<float*>(p) = f[0];
    } else if (DT == TBE_BF16) {
      if (VEC == 2) *static_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[VEC - 1]);
      else *static_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(f[0]);
    } else {
      if (VEC == 2) *static_cast<__half2*>(p) = __floats2half2_rn(f[0], f[VEC - 1]);
      else *static_cast<__half*>(p) = __float2half_rn(f[0]);
    }
  }
};

template <int DT>
__device__ __forceinline__ const uint8_t* at(const void* p, int64_t e) {
  return static_cast<const uint8_t*>(p) + e * (DT == TBE_F32 ? 4 : 2);
}
template <int DT>
__device__ __forceinline__ uint8_t* at(void* p, int64_t e) {
  return static_cast<uint8_t*>(p) + e * (DT == TBE_F32 ? 4 : 2);
}

// The linear map of a run of tokens; A < 0: it does not depend on what comes in.
struct Map {
  float A, B;
};
// `next` after `prev`
__device__ __forceinline__ Map join(Map prev, Map next) {
  Map m;
  m.A = next.A < 0.f || prev.A < 0.f ? -1.f : next.A * prev.A;
  m.B = next.A < 0.f ? next.B : fmaf(next.A, prev.B, next.B);
  return m;
}
__device__ __forceinline__ float apply(Map m, float in) { return m.A < 0.f ? m.B : fmaf(m.A, in, m.B); }

// Words between tiles.  A written word never looks empty: that bit pattern
// is a NaN, and another NaN is written in its place.
__device__ __forceinline__ uint32_t word_of(float f) {
  const uint32_t b = __float_as_uint(f);
  return b == kEmpty ? 0x7fffffffu : b;
}
__device__ __forceinline__ void publish(uint2* p, Map m) {
  const uint64_t v = (uint64_t)word_of(m.B) << 32 | word_of(m.A);
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ void publish(uint32_t* p, float f) {
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(word_of(f)) : "memory");
}
__device__ __forceinline__ uint64_t peek(const uint2* p) {
  uint64_t v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t peek(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// The join of `count` words base[0], base[stride], ... in that order.  All
// are requested at once; the ones that are not written yet are polled.
__device__ __forceinline__ Map join_words(const uint2* base, int64_t stride, int count, bool on, int& left,
                                          int32_t* status) {
  Map m{1.f, 0.f};
  uint64_t w[kGroup];
#pragma unroll
  for (int j = 0; j < kGroup; ++j) w[j] = on && j < count ? peek(base + j * stride) : 0;
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    if (j < count) {
      while ((uint32_t)w[j] == kEmpty && left > 0) {
        if (--left < kPolls - 64) __nanosleep(40);
        w[j] = peek(base + j * stride);
      }
      if ((uint32_t)w[j] == kEmpty) report(status, TBE_DEV_TIMEOUT);
      const Map n{__uint_as_float((uint32_t)w[j]), __uint_as_float((uint32_t)(w[j] >> 32))};
      m = on ? join(m, n) : m;
    }
  }
  return m;
}
__device__ __forceinline__ float wait_word(const uint32_t* p, bool on, int& left, int32_t* status) {
  if (!on) return 0.f;
  uint32_t w = peek(p);
  while (w == kEmpty && left > 0) {
    if (--left < kPolls - 64) __nanosleep(40);
    w = peek(p);
  }
  if (w == kEmpty) report(status, TBE_DEV_TIMEOUT);
  return __uint_as_float(w);
}

// The state that reaches tile k (counted in scan order) from the tiles
// before it, given the tile's own map `own`; writes the tile's, its group's
// and its row's words.  One warp calls this, each lane for its channels.
template <int VEC>
__device__ __forceinline__ void join_tiles(const ScanArgs& a, int k, int64_t c, const Map* own, float* in) {
  const int64_t C = a.C;
  int left = kPolls;
  const int group = k / kGroup, row = group / kGroup;
  const bool last_in_group = k % kGroup == kGroup - 1, last_in_row = group % kGroup == kGroup - 1;
#pragma unroll
  for (int v = 0; v < VEC; ++v)
    if (c + v < C && k + 1 < a.tiles) publish(a.tile_word + (int64_t)k * C + c + v, own[v]);
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const bool on = c + v < C;
    const Map tiles = join_words(a.tile_word + (int64_t)group * kGroup * C + c + v, C, k % kGroup, on, left, a.status);
    Map group_own = join(tiles, own[v]);
    if (on && last_in_group && k + 1 < a.tiles) publish(a.group_word + (int64_t)group * C + c + v, group_own);
    const Map groups =
        join_words(a.group_word + (int64_t)row * kGroup * C + c + v, C, group % kGroup, on, left, a.status);
    const Map before = join(groups, tiles);
    // nothing comes in where a sequence starts on the way
    const float base = row > 0 && before.A >= 0.f ? wait_word(a.row_word + (int64_t)(row - 1) * C + c + v, on, left, a.status)
                                                  : 0.f;
    in[v] = apply(before, base);
    if (on && last_in_group && last_in_row && k + 1 < a.tiles)
      publish(a.row_word + (int64_t)row * C + c + v, apply(own[v], in[v]));
  }
}

// First s in [0, S] with offsets[s] >= t, or S + 1; one warp, 32 pivots a step.
__device__ __forceinline__ int64_t first_at(const IdxPtr& o, int64_t S, int64_t t, int lane) {
  int64_t lo = 0, n = S + 1;  // the answer lies in [lo, lo + n]
  while (n > 0) {
    const int64_t step = (n + 31) / 32;
    const int64_t i = lo + lane * step;
    const bool less = i < lo + n && o.ldg(i) < t;
    const int below = __popc(__ballot_sync(kFull, less));  // pivots are increasing: a prefix of the lanes
    if (below == 0) return lo;
    const int64_t from = lo + (below - 1) * step + 1;  // after the last pivot below t
    const int64_t to = lo + below * step < lo + n ? lo + below * step : lo + n;
    lo = from;
    n = to > from ? to - from : 0;
  }
  return lo;
}

// What a tile has to know of the sequences: where they start and end, and which they are.
struct TileSeqs {
  uint32_t start[kTile / 32 + 1];  // bit t: a sequence starts at the tile's token t
  uint32_t end[kTile / 32 + 1];    // bit t: the tile's token t is its sequence's last
  int32_t start_of[kTile];         // the sequence that starts at token t
  int32_t end_of[kTile];           // the sequence that ends with token t
};

// Fills `q` for tile k (called by every thread; ends with a barrier) and
// calls empty(s) for each empty sequence that lies in the tile.
template <typename F>
__device__ __forceinline__ void find_sequences(const ScanArgs& a, int k, TileSeqs& q, int64_t* s_first, F&& empty) {
  const int64_t t0 = (int64_t)k * kTile;
  const int64_t t1 = k + 1 == a.tiles ? INT64_MAX : t0 + kTile;
  for (int i = threadIdx.x; i < kTile / 32 + 1; i += kThreads) q.start[i] = q.end[i] = 0;
  if (threadIdx.x < 32) {
    const int64_t s = first_at(a.offsets, a.S, t0, threadIdx.x);
    if (threadIdx.x == 0) *s_first = s;
  }
  __syncthreads();
  // the sequence before the first start may end in this tile
  const int64_t from = *s_first > 0 ? *s_first - 1 : 0;
  for (int64_t base = from; base < a.S; base += kThreads) {
    const int64_t s = base + threadIdx.x;
    const bool in = s < a.S;
    const int64_t o = in ? a.offsets.ldg(s) : INT64_MAX;
    if (in && o < t1) {
      const int64_t e = a.offsets.ldg(s + 1);
      if (e > o) {
        if (o >= t0 && o - t0 < kTile) {
          q.start_of[o - t0] = (int32_t)s;
          atomicOr(&q.start[(o - t0) >> 5], 1u << ((o - t0) & 31));
        }
        const int64_t l = e - 1 - t0;
        if (l >= 0 && l < kTile) {
          q.end_of[l] = (int32_t)s;
          atomicOr(&q.end[l >> 5], 1u << (l & 31));
        }
      } else if (o >= t0) {
        empty(s);
      }
    }
    if (__syncthreads_or(o >= t1)) break;
  }
  __syncthreads();
}

// Reports offsets that do not start at 0, end at N or that decrease; the
// tiles of the first channel block share the work.
__device__ __forceinline__ void check_offsets(const ScanArgs& a, int k) {
  const int64_t per = (a.S + a.tiles) / a.tiles;
  const int64_t lo = (int64_t)k * per, hi = lo + per < (int64_t)a.S + 1 ? lo + per : (int64_t)a.S + 1;
  bool bad = false;
  for (int64_t s = lo + threadIdx.x; s < hi; s += kThreads) {
    const int64_t o = a.offsets.ldg(s);
    if (s == 0) bad |= o != 0;
    if (s == a.S) bad |= o != a.N;
    else bad |= a.offsets.ldg(s + 1) < o;
  }
  if (bad) report(a.status, TBE_DEV_BAD_OFFSETS);
}

// The block's tile: tickets follow the scan order, so a tile only waits for
// tiles whose blocks have started.
__device__ __forceinline__ uint32_t take_ticket(const ScanArgs& a, uint32_t* shared) {
  if (a.tiles == 1) return blockIdx.x;
  if (threadIdx.x == 0) *shared = atomicAdd(a.ticket, 1u) + 1u;  // the counter starts at 2^32 - 1
  __syncthreads();
  return *shared;
}

template <int DT, int VEC>
__global__ void __launch_bounds__(kThreads, 2) scan_forward_kernel(ScanArgs a) {
  using E = Elems<DT, VEC>;
  __shared__ TileSeqs q;
  __shared__ Map runs[kWarps][32 * VEC];
  __shared__ float carry[32 * VEC];
  __shared__ int64_t s_first;
  __shared__ uint32_t s_ticket;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t id = take_ticket(a, &s_ticket);
  const int k = id / a.cblocks;
  const int64_t cb = (int64_t)(id % a.cblocks) * 32 * VEC, c = cb + lane * VEC;
  const bool on = c < a.C;
  const int64_t t0 = (int64_t)k * kTile + warp * kStep;
  const int count = t0 >= a.N ? 0 : (a.N - t0 < kStep ? (int)(a.N - t0) : kStep);

  uint32_t rx[kStep], rr[kStep], rg[kStep];
#pragma unroll
  for (int j = 0; j < kStep; ++j) {
    const bool ok = on && j < count;
    rr[j] = ok ? E::load(at<DT>(a.r, (t0 + j) * a.sr + c)) : 0;
    rg[j] = ok ? E::load(at<DT>(a.g, (t0 + j) * a.sg + c)) : 0;
    rx[j] = ok ? E::load(at<DT>(a.x, (t0 + j) * a.sx + c)) : 0;
  }
  if (cb == 0) check_offsets(a, k);
  find_sequences(a, k, q, &s_first, [&](int64_t s) {  // an empty sequence hands its state on
    for (int64_t e = cb; e < cb + 32 * VEC && e < a.C; ++e)
      a.h_last[s * a.C + e] = a.h0 ? a.h0[s * a.C + e] : 0.f;
  });
  float speed[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) speed[v] = on ? speed_of(a, c + v) : 0.f;
  const uint32_t starts = q.start[warp * kStep / 32] >> (warp * kStep % 32) & ((1u << kStep) - 1);
  const uint32_t ends = q.end[warp * kStep / 32] >> (warp * kStep % 32) & ((1u << kStep) - 1);

  float A[kStep][VEC], B[kStep][VEC];
  Map own[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) own[v] = Map{1.f, 0.f};
#pragma unroll
  for (int j = 0; j < kStep; ++j) {
    float x[VEC], r[VEC], g[VEC], first[VEC];
    E::unpack(rx[j], x);
    E::unpack(rr[j], r);
    E::unpack(rg[j], g);
    const bool start = starts >> j & 1;
    if (start) {
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        first[v] = a.h0 && on ? a.h0[(int64_t)q.start_of[warp * kStep + j] * a.C + c + v] : 0.f;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const Decay d = decay_of(speed[v] * sigmoid(r[v]));
      A[j][v] = d.a;
      B[j][v] = root(d.q) * sigmoid(g[v]) * x[v];
      if (start) {
        B[j][v] = fmaf(A[j][v], first[v], B[j][v]);
        A[j][v] = -1.f;
      }
      own[v] = join(own[v], Map{A[j][v], B[j][v]});
    }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) runs[warp][lane * VEC + v] = own[v];
  __syncthreads();
  if (warp == 0) {
    Map tile[VEC];
    float in[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      tile[v] = runs[0][lane * VEC + v];
      for (int w = 1; w < kWarps; ++w) tile[v] = join(tile[v], runs[w][lane * VEC + v]);
      in[v] = 0.f;
    }
    if (a.tiles > 1) join_tiles<VEC>(a, k, c, tile, in);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      carry[lane * VEC + v] = in[v];
      if (a.states && c + v < a.C) a.states[(int64_t)k * a.C + c + v] = in[v];
    }
  }
  __syncthreads();
  float h[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    h[v] = carry[lane * VEC + v];
    for (int w = 0; w < warp; ++w) h[v] = apply(runs[w][lane * VEC + v], h[v]);
  }
  if (!on) return;
#pragma unroll
  for (int j = 0; j < kStep; ++j) {
    if (j >= count) break;
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = apply(Map{A[j][v], B[j][v]}, h[v]);
    E::store(at<DT>(a.h, (t0 + j) * a.sh + c), h);
    if (ends >> j & 1) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) a.h_last[(int64_t)q.end_of[warp * kStep + j] * a.C + c + v] = h[v];
    }
  }
}

// Backward: the tiles in reverse.  What runs from token to token is
// a_t G_t, with G_t = dh_t + a_{t+1} G_{t+1} inside a sequence and
// dh_t + dh_last at its end.  The states h_{t-1} are made again from each
// tile's saved first state, in 32 bits, so h itself is not read.
template <int DT, int VEC>
__global__ void __launch_bounds__(kThreads) scan_backward_kernel(ScanArgs a) {
  using E = Elems<DT, VEC>;
  __shared__ TileSeqs q;
  __shared__ Map runs[kWarps][32 * VEC];  // forward maps of the runs
  __shared__ Map back[kWarps][32 * VEC];  // and the backward ones
  __shared__ float carry[32 * VEC];
  __shared__ int64_t s_first;
  __shared__ uint32_t s_ticket;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t id = take_ticket(a, &s_ticket);
  const int order = id / a.cblocks;  // in scan order
  const int k = a.tiles - 1 - order;
  const int64_t cb = (int64_t)(id % a.cblocks) * 32 * VEC, c = cb + lane * VEC;
  const bool on = c < a.C;
  const int64_t t0 = (int64_t)k * kTile + warp * kStep;
  const int count = t0 >= a.N ? 0 : (a.N - t0 < kStep ? (int)(a.N - t0) : kStep);

  uint32_t rx[kStep], rr[kStep], rg[kStep], rd[kStep];
#pragma unroll
  for (int j = 0; j < kStep; ++j) {
    const bool ok = on && j < count;
    rr[j] = ok ? E::load(at<DT>(a.r, (t0 + j) * a.sr + c)) : 0;
    rg[j] = ok ? E::load(at<DT>(a.g, (t0 + j) * a.sg + c)) : 0;
    rx[j] = ok ? E::load(at<DT>(a.x, (t0 + j) * a.sx + c)) : 0;
    rd[j] = ok ? E::load(at<DT>(a.dh, (t0 + j) * a.sdh + c)) : 0;
  }
  if (cb == 0) check_offsets(a, k);
  find_sequences(a, k, q, &s_first, [&](int64_t s) {
    if (a.dh0)
      for (int64_t e = cb; e < cb + 32 * VEC && e < a.C; ++e)
        a.dh0[s * a.C + e] = a.dh_last ? a.dh_last[s * a.C + e] : 0.f;
  });
  float speed[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) speed[v] = on ? speed_of(a, c + v) : 0.f;
  const uint32_t starts = q.start[warp * kStep / 32] >> (warp * kStep % 32) & ((1u << kStep) - 1);
  const uint32_t ends = q.end[warp * kStep / 32] >> (warp * kStep % 32) & ((1u << kStep) - 1);

  float sr[kStep][VEC], sg[kStep][VEC], A[kStep][VEC], D[kStep][VEC];
  Map own[VEC], rev[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) own[v] = rev[v] = Map{1.f, 0.f};
#pragma unroll
  for (int j = 0; j < kStep; ++j) {
    float x[VEC], r[VEC], g[VEC];
    E::unpack(rx[j], x);
    E::unpack(rr[j], r);
    E::unpack(rg[j], g);
    E::unpack(rd[j], D[j]);
    const bool start = starts >> j & 1, end = ends >> j & 1;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      sr[j][v] = sigmoid(r[v]);
      sg[j][v] = sigmoid(g[v]);
      const Decay d = decay_of(speed[v] * sr[j][v]);
      A[j][v] = d.a;
      float b = root(d.q) * sg[j][v] * x[v];
      if (start) {
        const float first = a.h0 && on ? a.h0[(int64_t)q.start_of[warp * kStep + j] * a.C + c + v] : 0.f;
        b = fmaf(A[j][v], first, b);
        own[v] = Map{-1.f, b};
      } else {
        own[v] = join(own[v], Map{A[j][v], b});
      }
      if (end && a.dh_last && on) D[j][v] += a.dh_last[(int64_t)q.end_of[warp * kStep + j] * a.C + c + v];
    }
  }
#pragma unroll
  for (int j = kStep - 1; j >= 0; --j) {
    const bool end = ends >> j & 1;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      // a_t G_t = a_t in + a_t dh_t; nothing comes in behind a sequence's end
      const Map t{end ? -1.f : A[j][v], A[j][v] * D[j][v]};
      rev[v] = join(rev[v], t);
    }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    runs[warp][lane * VEC + v] = own[v];
    back[warp][lane * VEC + v] = rev[v];
  }
  __syncthreads();
  if (warp == 0) {
    Map tile[VEC];
    float in[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      tile[v] = back[kWarps - 1][lane * VEC + v];
      for (int w = kWarps - 2; w >= 0; --w) tile[v] = join(tile[v], back[w][lane * VEC + v]);
      in[v] = 0.f;
    }
    if (a.tiles > 1) join_tiles<VEC>(a, order, c, tile, in);
#pragma unroll
    for (int v = 0; v < VEC; ++v) carry[lane * VEC + v] = in[v];
  }
  // the states that the run's tokens find
  float before[kStep][VEC], h[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    h[v] = on ? a.states[(int64_t)k * a.C + c + v] : 0.f;
    for (int w = 0; w < warp; ++w) h[v] = apply(runs[w][lane * VEC + v], h[v]);
  }
#pragma unroll
  for (int j = 0; j < kStep; ++j) {
    float x[VEC];
    E::unpack(rx[j], x);
    const bool start = starts >> j & 1;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      if (start) h[v] = a.h0 && on ? a.h0[(int64_t)q.start_of[warp * kStep + j] * a.C + c + v] : 0.f;
      before[j][v] = h[v];
      h[v] = fmaf(A[j][v], h[v], root(decay_of(speed[v] * sr[j][v]).q) * sg[j][v] * x[v]);
    }
  }
  __syncthreads();
  float G_in[VEC], share[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    G_in[v] = carry[lane * VEC + v];
    for (int w = kWarps - 1; w > warp; --w) G_in[v] = apply(back[w][lane * VEC + v], G_in[v]);
    share[v] = 0.f;
  }
#pragma unroll
  for (int j = kStep - 1; j >= 0; --j) {
    if (j < count && on) {
      float x[VEC], dx[VEC], dr[VEC], dg[VEC];
      E::unpack(rx[j], x);
      const bool start = starts >> j & 1, end = ends >> j & 1;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float G = end ? D[j][v] : D[j][v] + G_in[v];
        const float u = speed[v] * sr[j][v];
        const float qq = decay_of(u).q;
        const float inv = rsqrtf(qq);
        const float beta = qq > 0.f ? qq * inv : 0.f;
        const float slope = qq > 0.f ? u * A[j][v] * A[j][v] * inv : 0.f;  // u d beta / d u
        const float w = G * (slope * sg[j][v] * x[v] - u * A[j][v] * before[j][v]);
        dx[v] = G * beta * sg[j][v];
        dg[v] = dx[v] * x[v] * (1.f - sg[j][v]);
        dr[v] = w * (1.f - sr[j][v]);
        share[v] += w;
        G_in[v] = A[j][v] * G;
        if (start && a.dh0) a.dh0[(int64_t)q.start_of[warp * kStep + j] * a.C + c + v] = G_in[v];
      }
      E::store(at<DT>(a.dx, (t0 + j) * a.sdx + c), dx);
      E::store(at<DT>(a.dr, (t0 + j) * a.sdr + c), dr);
      E::store(at<DT>(a.dg, (t0 + j) * a.sdg + c), dg);
    }
  }
  // the tile's share of the decay's gradient: the warps' sums, in order
  float* sums = reinterpret_cast<float*>(runs);
  __syncthreads();
#pragma unroll
  for (int v = 0; v < VEC; ++v) sums[warp * 32 * VEC + lane * VEC + v] = share[v];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * VEC; i += kThreads) {
    float t = 0.f;
    for (int w = 0; w < kWarps; ++w) t += sums[w * 32 * VEC + i];
    if (cb + i < a.C) a.partial[(int64_t)k * a.C + cb + i] = t;
  }
}

// ddecay = sigmoid(decay) / softplus(decay) * sum over the tiles, 32 channels
// per block, its warps each a share of the tiles.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32)
    decay_grad_kernel(const float* partial, const float* decay, float* ddecay, int32_t tiles, int32_t C) {
  __shared__ float part[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < C)
    for (int64_t k = warp; k < tiles; k += kSumWarps) s += partial[k * C + c];
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < C) {
    for (int w = 1; w < kSumWarps; ++w) s += part[w][lane];
    const float d = decay[c], sp = softplus(d);
    // far below zero softplus(d) = sigmoid(d) = exp(d): the ratio is 1
    ddecay[c] = d < -16.f ? s : s * (1.f / (1.f + expf(-d))) / sp;
  }
}

// One token of each of S sequences: the state moves on in place.
template <int DT, int VEC>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs a) {
  using E = Elems<DT, VEC>;
  const int64_t per_row = (a.C + VEC - 1) / VEC;
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (i >= per_row * a.S) return;
  const int64_t s = i / per_row, c = (i - s * per_row) * VEC;
  float x[VEC], r[VEC], g[VEC], h[VEC];
  float* state = a.h_last + s * a.C + c;
  E::unpack(E::load(at<DT>(a.x, s * a.sx + c)), x);
  E::unpack(E::load(at<DT>(a.r, s * a.sr + c)), r);
  E::unpack(E::load(at<DT>(a.g, s * a.sg + c)), g);
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const Decay d = decay_of(speed_of(a, c + v) * sigmoid(r[v]));
    h[v] = fmaf(d.a, state[v], root(d.q) * sigmoid(g[v]) * x[v]);
    state[v] = h[v];
  }
  E::store(at<DT>(a.h, s * a.sh + c), h);
}

int32_t tile_count(int64_t N) { return N <= 0 ? 1 : (int32_t)((N + kTile - 1) / kTile); }
int32_t groups_of(int32_t n) { return (n + kGroup - 1) / kGroup; }
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// The workspace: the ticket, the words of rows, groups and tiles (filled with
// kEmpty before each use), then the backward's partial sums.
struct Workspace {
  size_t row, group, tile, words_end, partial, bytes;
};
Workspace layout(int64_t N, int32_t C, bool backward) {
  const int32_t tiles = tile_count(N);
  Workspace w;
  size_t at = 256;
  w.row = at;
  at += round256((size_t)groups_of(groups_of(tiles)) * C * 4);
  w.group = at;
  at += round256((size_t)groups_of(tiles) * C * 8);
  w.tile = at;
  at += round256((size_t)tiles * C * 8);
  if (tiles == 1) at = w.row = w.group = w.tile = 0;
  w.words_end = at;
  w.partial = at;
  if (backward) at += round256((size_t)tiles * C * 4);
  w.bytes = at;
  return w;
}

bool even4(const void* p, int64_t stride) { return ((uintptr_t)p & 3) == 0 && stride % 2 == 0; }

// Two channels per lane where every row of every half-precision array starts
// on 4 bytes.
bool pairs(const ScanArgs& a, int32_t dtype) {
  if (dtype == TBE_F32 || a.C % 2 != 0) return false;
  bool ok = even4(a.x, a.sx) && even4(a.r, a.sr) && even4(a.g, a.sg);
  if (a.h) ok = ok && even4(a.h, a.sh);
  if (a.dh) ok = ok && even4(a.dh, a.sdh) && even4(a.dx, a.sdx) && even4(a.dr, a.sdr) && even4(a.dg, a.sdg);
  return ok;
}

enum { kForward, kBackward, kOne };

template <int DT, int VEC>
int launch(ScanArgs& a, int what, cudaStream_t s) {
  a.cblocks = (a.C + 32 * VEC - 1) / (32 * VEC);
  if (what == kOne) {
    const int64_t n = (int64_t)a.S * ((a.C + VEC - 1) / VEC);
    scan_step_kernel<DT, VEC><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(a);
    return check_launch();
  }
  const unsigned grid = (unsigned)a.tiles * (unsigned)a.cblocks;
  if (what == kForward) scan_forward_kernel<DT, VEC><<<grid, kThreads, 0, s>>>(a);
  else scan_backward_kernel<DT, VEC><<<grid, kThreads, 0, s>>>(a);
  return check_launch();
}

int dispatch(ScanArgs& a, int32_t dtype, int what, cudaStream_t s) {
  const bool two = pairs(a, dtype);
  if (dtype == TBE_F32) return launch<TBE_F32, 1>(a, what, s);
  if (dtype == TBE_F16) return two ? launch<TBE_F16, 2>(a, what, s) : launch<TBE_F16, 1>(a, what, s);
  return two ? launch<TBE_BF16, 2>(a, what, s) : launch<TBE_BF16, 1>(a, what, s);
}

bool aligned_for(const void* p, int32_t dtype) { return ((uintptr_t)p & (dtype == TBE_F32 ? 3 : 1)) == 0; }

// Checks shared by the entry points.
int check(const tbe_scan_inputs* in) {
  if (!in) return TBE_ERR_INVALID_ARG;
  if (in->dtype < TBE_F32 || in->dtype > TBE_BF16) return TBE_ERR_INVALID_ARG;
  if (in->tokens < 0 || in->sequences < 0 || in->channels < 1 || !std::isfinite(in->sharpness) || in->sharpness < 0)
    return TBE_ERR_INVALID_ARG;
  if (in->tokens >= (int64_t(1) << 38) || in->channels > (1 << 20)) return TBE_ERR_UNSUPPORTED;
  if (!in->decay) return TBE_ERR_INVALID_ARG;
  if (in->tokens > 0 && (!in->x || !in->recur || !in->gate)) return TBE_ERR_INVALID_ARG;
  if (in->x_stride < in->channels || in->recur_stride < in->channels || in->gate_stride < in->channels)
    return TBE_ERR_INVALID_ARG;
  if (!aligned_for(in->x, in->dtype) || !aligned_for(in->recur, in->dtype) || !aligned_for(in->gate, in->dtype))
    return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

ScanArgs args_of(const tbe_scan_inputs* in) {
  ScanArgs a = {};
  a.x = in->x;
  a.r = in->recur;
  a.g = in->gate;
  a.sx = in->x_stride;
  a.sr = in->recur_stride;
  a.sg = in->gate_stride;
  a.decay = in->decay;
  a.sharpness = in->sharpness;
  a.offsets = IdxPtr{in->offsets, in->offsets_i32 != 0};
  a.N = in->tokens;
  a.S = in->sequences;
  a.C = in->channels;
  a.tiles = tile_count(in->tokens);
  a.h0 = in->h0;
  return a;
}

int check_jagged(const tbe_scan_inputs* in) {
  const int st = check(in);
  if (st != TBE_OK) return st;
  if (!in->offsets || (in->tokens > 0 && in->sequences == 0)) return TBE_ERR_INVALID_ARG;
  if ((int64_t)tile_count(in->tokens) * ((in->channels + 31) / 32) >= (int64_t(1) << 31)) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

// Points the words into the workspace and empties them.
int use_workspace(ScanArgs& a, bool backward, void* workspace, size_t bytes, cudaStream_t s) {
  const Workspace w = layout(a.N, a.C, backward);
  if (bytes < w.bytes) return TBE_ERR_WORKSPACE;
  if (w.bytes == 0) return TBE_OK;
  if (!workspace) return TBE_ERR_INVALID_ARG;
  if ((uintptr_t)workspace & 255) return TBE_ERR_UNSUPPORTED;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  a.ticket = reinterpret_cast<uint32_t*>(p);
  a.row_word = reinterpret_cast<uint32_t*>(p + w.row);
  a.group_word = reinterpret_cast<uint2*>(p + w.group);
  a.tile_word = reinterpret_cast<uint2*>(p + w.tile);
  a.partial = reinterpret_cast<float*>(p + w.partial);
  if (w.words_end > 0 && cudaMemsetAsync(p, 0xff, w.words_end, s) != cudaSuccess) return TBE_ERR_CUDA;
  return TBE_OK;
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" {

int64_t tbe_gated_scan_states(int64_t tokens) { return tokens < 0 ? 0 : tile_count(tokens); }

size_t tbe_gated_scan_workspace_bytes(int64_t tokens, int32_t channels, int32_t backward) {
  if (tokens < 0 || channels < 1) return 0;
  return layout(tokens, channels, backward != 0).bytes;
}

int tbe_gated_scan(const tbe_scan_inputs* in, void* h, int64_t h_stride, float* h_last, float* states,
                   void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  int st = check_jagged(in);
  if (st != TBE_OK) return st;
  if (in->sequences == 0) return TBE_OK;
  if ((in->tokens > 0 && !h) || !h_last || h_stride < in->channels) return TBE_ERR_INVALID_ARG;
  if (!aligned_for(h, in->dtype)) return TBE_ERR_UNSUPPORTED;
  ScanArgs a = args_of(in);
  a.h = h;
  a.sh = h_stride;
  a.h_last = h_last;
  a.states = states;
  a.status = dev_status;
  cudaStream_t s = (cudaStream_t)stream;
  trace_begin(s);
  st = use_workspace(a, false, workspace, workspace_bytes, s);
  if (st != TBE_OK) return st;
  st = dispatch(a, in->dtype, kForward, s);
  trace_mark(s, "gated_scan");
  return st;
}

int tbe_gated_scan_backward(const tbe_scan_inputs* in, const void* dh, int64_t dh_stride, const float* dh_last,
                            const float* states, const tbe_scan_grads* out, void* workspace, size_t workspace_bytes,
                            int32_t* dev_status, void* stream) {
  int st = check_jagged(in);
  if (st != TBE_OK) return st;
  if (!out || !out->ddecay) return TBE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (in->sequences == 0)
    return cudaMemsetAsync(out->ddecay, 0, sizeof(float) * (size_t)in->channels, s) == cudaSuccess ? TBE_OK : TBE_ERR_CUDA;
  if (!states || dh_stride < in->channels || out->dx_stride < in->channels || out->drecur_stride < in->channels ||
      out->dgate_stride < in->channels)
    return TBE_ERR_INVALID_ARG;
  if (in->tokens > 0 && (!dh || !out->dx || !out->drecur || !out->dgate)) return TBE_ERR_INVALID_ARG;
  if (!aligned_for(dh, in->dtype) || !aligned_for(out->dx, in->dtype) || !aligned_for(out->drecur, in->dtype) ||
      !aligned_for(out->dgate, in->dtype))
    return TBE_ERR_UNSUPPORTED;
  ScanArgs a = args_of(in);
  a.dh = dh;
  a.sdh = dh_stride;
  a.dh_last = dh_last;
  a.states = const_cast<float*>(states);  // only read
  a.dx = out->dx;
  a.dr = out->drecur;
  a.dg = out->dgate;
  a.sdx = out->dx_stride;
  a.sdr = out->drecur_stride;
  a.sdg = out->dgate_stride;
  a.dh0 = out->dh0;
  a.status = dev_status;
  trace_begin(s);
  st = use_workspace(a, true, workspace, workspace_bytes, s);
  if (st != TBE_OK) return st;
  st = dispatch(a, in->dtype, kBackward, s);
  if (st != TBE_OK) return st;
  trace_mark(s, "gated_scan_backward");
  decay_grad_kernel<<<(unsigned)((a.C + 31) / 32), kSumWarps * 32, 0, s>>>(a.partial, a.decay, out->ddecay, a.tiles, a.C);
  st = check_launch();
  trace_mark(s, "decay_grad");
  return st;
}

int tbe_gated_scan_step(const tbe_scan_inputs* in, float* state, void* h, int64_t h_stride, void* stream) {
  const int st = check(in);
  if (st != TBE_OK) return st;
  if (in->tokens != in->sequences || in->h0) return TBE_ERR_INVALID_ARG;
  if (in->sequences == 0) return TBE_OK;
  if (!state || !h || h_stride < in->channels) return TBE_ERR_INVALID_ARG;
  if (!aligned_for(h, in->dtype)) return TBE_ERR_UNSUPPORTED;
  if ((int64_t)in->sequences * in->channels >= (int64_t(1) << 37)) return TBE_ERR_UNSUPPORTED;
  ScanArgs a = args_of(in);
  a.h_last = state;
  a.h = h;
  a.sh = h_stride;
  cudaStream_t s = (cudaStream_t)stream;
  trace_begin(s);
  const int rc = dispatch(a, in->dtype, kOne, s);
  trace_mark(s, "gated_scan_step");
  return rc;
}

}  // extern "C"
