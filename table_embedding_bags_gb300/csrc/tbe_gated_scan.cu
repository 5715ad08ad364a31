// tbe_gated_scan.cu -- gated linear recurrence over jagged sequences, its
// backward pass and its form for single tokens.
//
//   u_t = sharpness * softplus(decay) * sigmoid(recur_t)      a_t = exp(-u_t)
//   h_t = a_t h_{t-1} + beta_t sigmoid(gate_t) x_t            beta_t = sqrt(1 - a_t^2)
//
// per channel, over every sequence of the jagged batch.  The sequences are
// scanned as one axis of N tokens: at a sequence's first token the recurrence
// is cut (its state enters as a term of its own), so the work splits into
// equal runs of the token axis whatever the lengths are.
//
// A warp takes a run of tokens and 128 bytes of channels (a lane one fp32 or
// two half-precision ones); a block's warps take neighbouring runs.  h over a
// run is the linear map h_out = A h_in + B, so two passes do it:
//  - maps: each run's map (only from the last start in it on, if there is
//    one), joined over the block;
//  - apply: each block joins the maps of the blocks before it, back to the
//    nearest one that holds a sequence start, each warp those of the warps
//    before it, and then walks its run token by token.
// No block waits for another one inside a kernel, and maps are always joined
// in the same order, so results do not depend on timing.  A batch of one
// block's tokens takes both passes in one kernel.
//
// Both passes stream a warp's tokens through a ring of shared-memory slots of
// its own (kStep tokens each), filled by asynchronous copies some steps
// ahead: the warps of a block meet only where maps are joined.
//
// A map that contains a sequence start has no h_in; it is kept apart from
// A = 0 (which long decays reach by underflow) by A = -1, so that a NaN in
// one sequence never reaches the next.
//
// The backward walks the runs in reverse: from token to token goes a_t G_t,
// with G_t = dh_t + a_{t+1} G_{t+1} inside a sequence and dh_t + dh_last at
// its end.  The states h_{t-1} of a step are made again from the state it
// started from, which the forward saved in 32 bits, so h itself is not read.
#include "tbe_internal.cuh"

#include <cmath>

namespace tbe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kStep = TBE_SCAN_STEP;  // tokens per step (and between saved states)
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlocksPerSm = 2;
constexpr int kRow = 128;            // bytes of a warp's row
constexpr int kBox = kStep * kRow;   // one input's bytes of a step
constexpr float kLog2e = 1.4426950408889634f;

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
  int32_t run;      // tokens per warp, a multiple of kStep
  int32_t blocks;   // along the tokens
  int32_t cblocks;  // along the channels
  int32_t pairs;    // half precision: every row of every array starts on 4 bytes
  int32_t copy;     // bytes per asynchronous copy: 16, 4, or 0 (plain loads)
  int64_t Cp;       // channels filled up to whole warps
  const float* h0;  // [S, C] or null
  // forward
  void* h;          // [N, C]
  int64_t sh;
  float* h_last;    // [S, C]
  float* states;    // [ceil(N / kStep), C]: the state each step starts from, or null
  // backward
  const void* dh;
  int64_t sdh;
  const float* dh_last;
  void* dx;
  void* dr;
  void* dg;
  int64_t sdx, sdr, sdg;
  float* dh0;
  float* partial;    // [blocks * kWarps, C]: each run's share of the decay's gradient
  float2* warp_map;  // [blocks * kWarps, Cp]
  float2* block_map; // [blocks, Cp]
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
__device__ __forceinline__ float inv_root(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

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

// a = exp(-u) and 1 - a^2 for u >= 0, both to a few units of their own
// size.  Below 1/4, n = 1 - a from its series (the next term is under 5e-8 of
// the sum): near a = 1 its rounding is relative to 1 - a, which is what
// decides how long a state lives, and 1 - a^2 = n (2 - n) keeps it.
constexpr float kNear = 0.25f;
template <typename T>
struct Decay {
  T a, q;
};
__device__ __forceinline__ Decay<Two> decay_near(Two u) {
  Two p = fma2(u, two(-1.f / 720.f), two(1.f / 120.f));
  p = fma2(u, p, two(-1.f / 24.f));
  p = fma2(u, p, two(1.f / 6.f));
  p = fma2(u, p, two(-0.5f));
  p = fma2(u, p, two(1.f));
  const Two n = u * p;
  Decay<Two> d;
  d.a = fma2(n, two(-1.f), two(1.f));
  d.q = n * fma2(n, two(-1.f), two(2.f));
  return d;
}
__device__ __forceinline__ Decay<float> decay_of(float u) {
  float p = fmaf(u, -1.f / 720.f, 1.f / 120.f);
  p = fmaf(u, p, -1.f / 24.f);
  p = fmaf(u, p, 1.f / 6.f);
  p = fmaf(u, p, -0.5f);
  p = fmaf(u, p, 1.f);
  const float e = ex2(-kLog2e * u);
  const bool near = u < kNear;
  const float n = near ? u * p : 1.f - e;
  Decay<float> d;
  d.a = near ? 1.f - n : e;
  d.q = n * (2.f - n);
  return d;
}
__device__ __forceinline__ Decay<Two> decay_any(Two u) {
  const Decay<float> a = decay_of(lo(u)), b = decay_of(hi(u));
  return Decay<Two>{two(a.a, b.a), two(a.q, b.q)};
}

// softplus of the decay parameter
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
// sharpness * softplus; below the normal numbers, where fp32 keeps no
// relative precision, it counts as 0 (the channel keeps its state)
__device__ __forceinline__ float speed_of(const ScanArgs& a, int64_t c) {
  const float sp = softplus(a.decay[c]);
  return sp < 1.17549435e-38f ? 0.f : a.sharpness * sp;
}

// Both sigmoids of a token from one reciprocal, 1 / ((1 + e^-r)(1 + e^-g)).
// `top` gathers the products: above kTop (an input below about -40) one of
// the factors may not be told apart from infinity, and the run is done again
// by gates_any.
constexpr float kTop = 1e36f;
__device__ __forceinline__ void gates_near(Two r, Two g, Two& sr, Two& sg, float& top) {
  const Two pr = ex2(r * two(-kLog2e)) + two(1.f), pg = ex2(g * two(-kLog2e)) + two(1.f);
  const Two product = pr * pg, inv = rcp(product);
  sr = inv * pg;
  sg = inv * pr;
  top = fmaxf(top, fmaxf(lo(product), hi(product)));
}
__device__ __forceinline__ void gates_any(Two r, Two g, Two& sr, Two& sg) {
  sr = two(sigmoid(lo(r)), sigmoid(hi(r)));
  sg = two(sigmoid(lo(g)), sigmoid(hi(g)));
}

// A lane's channels: one fp32 or two half-precision ones, 4 bytes.  A Pair is
// what two-wide arithmetic works on: a token's two channels, or two
// neighbouring tokens of one fp32 channel.
template <int DT>
struct Lane {
  static constexpr int kVec = DT == TBE_F32 ? 1 : 2;
  static constexpr int kSize = DT == TBE_F32 ? 4 : 2;
  static constexpr int kPairs = kStep * kVec / 2;  // of a step
  static constexpr int kChannels = 32 * kVec;      // of a warp
};
template <int DT>
__device__ __forceinline__ float2 halves(uint32_t v) {
  if (DT == TBE_BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// Token j, channel v of an array of pairs.
template <int DT>
__device__ __forceinline__ float element(const Two* t, int j, int v) {
  if (DT == TBE_F32) return j & 1 ? hi(t[j >> 1]) : lo(t[j >> 1]);
  return v ? hi(t[j]) : lo(t[j]);
}

template <int DT>
__device__ __forceinline__ const uint8_t* at(const void* p, int64_t e) {
  return static_cast<const uint8_t*>(p) + e * Lane<DT>::kSize;
}
template <int DT>
__device__ __forceinline__ uint8_t* at(void* p, int64_t e) {
  return static_cast<uint8_t*>(p) + e * Lane<DT>::kSize;
}

// A lane's word of a token straight from memory, for arrays that TMA cannot
// read (not on 16 bytes): in one piece, or half by half.
template <int DT>
__device__ __forceinline__ uint32_t load_word(const uint8_t* p, bool pairs, int left) {
  if (DT == TBE_F32) return left > 0 ? *reinterpret_cast<const uint32_t*>(p) : 0;
  if (pairs && left > 1) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t v = left > 0 ? *reinterpret_cast<const uint16_t*>(p) : 0;
  if (left > 1) v |= (uint32_t) * reinterpret_cast<const uint16_t*>(p + 2) << 16;
  return v;
}
// Stores a token's channels (`left` of them lie inside the array).
template <int DT>
__device__ __forceinline__ void store_word(uint8_t* p, bool pairs, int left, float a, float b) {
  if (DT == TBE_F32) {
    if (left > 0) *reinterpret_cast<float*>(p) = a;
    return;
  }
  uint32_t v;
  if (DT == TBE_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    v = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    v = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (pairs && left > 1) {
    *reinterpret_cast<uint32_t*>(p) = v;
  } else {
    if (left > 0) *reinterpret_cast<uint16_t*>(p) = (uint16_t)v;
    if (left > 1) *reinterpret_cast<uint16_t*>(p + 2) = (uint16_t)(v >> 16);
  }
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


// Where sequences start and end.  The cursor holds 32 neighbouring offsets,
// one per lane, and is moved by a search where it does not reach.
struct Cursor {
  const ScanArgs& a;
  int64_t base, off;
  int lane;
  __device__ __forceinline__ Cursor(const ScanArgs& args, int lane_) : a(args), base(0), off(0), lane(lane_) {
    load(0);
  }
  __device__ __forceinline__ void load(int64_t from) {
    base = from;
    off = base + lane <= a.S ? a.offsets.ldg(base + lane) : INT64_MAX;
  }
  // The sequence that token t belongs to, and its first token and end.
  __device__ __forceinline__ int64_t owner(int64_t t, bool down, int64_t& first, int64_t& end) {
    int below = __popc(__ballot_sync(kFull, off <= t));
    if (below == 0 || below == 32) {
      int64_t s = first_at(a.offsets, a.S, t + 1, lane) - 1;
      s = s < 0 ? 0 : (s >= a.S ? a.S - 1 : s);
      load(down ? (s > 30 ? s - 30 : 0) : s);
      below = __popc(__ballot_sync(kFull, off <= t));
    }
    // broken offsets must not lead outside the arrays
    int l = below - 1 < 0 ? 0 : (below - 1 > 30 ? 30 : below - 1);
    if (base + l >= a.S) l = (int)(a.S - 1 - base) < 0 ? 0 : (int)(a.S - 1 - base);
    first = __shfl_sync(kFull, off, l);
    end = __shfl_sync(kFull, off, l + 1);
    return base + l;
  }
};

// The starts and ends among the tokens t .. t + count - 1 of a step: a bit
// per token, and in lane j the sequence of token j.  Nothing is looked up
// while the step lies inside the sequence of the step before.
struct Events {
  uint32_t starts, ends;
  int32_t s;
  int64_t first, end;  // of the sequence looked up last
  int32_t owner;
  __device__ __forceinline__ Events() : starts(0), ends(0), s(0), first(0), end(-1), owner(0) {}
  __device__ __forceinline__ void find(Cursor& cur, int64_t t, int count, bool down, int lane) {
    starts = ends = 0;
    s = owner;
    if (first < t && t + count < end) return;
    for (int j = 0; j < count;) {
      const int64_t at = t + j;
      owner = (int32_t)cur.owner(at, down, first, end);
      int64_t stop = end - t;
      if (stop <= j) stop = j + 1;
      const int next = stop < count ? (int)stop : count;
      if (first == at) starts |= 1u << j;
      if (end == t + next) ends |= 1u << (next - 1);
      if (lane >= j && lane < next) s = owner;
      j = next;
    }
    if (down && count > 0) owner = (int32_t)cur.owner(t, true, first, end);  // goes on below
  }
  __device__ __forceinline__ int64_t sequence(int j) const { return __shfl_sync(kFull, s, j); }
};

// A warp's ring.  Slot layout: kBox bytes per input, then (backward) the
// states of the step's start.
template <int DT, int INPUTS, int SLOTS, bool STATES>
struct Ring {
  static constexpr int kSlot = INPUTS * kBox + (STATES ? 256 : 0);
  static constexpr int kBytes = SLOTS * kSlot;
  uint8_t* mem;
  const void* in[INPUTS];
  int64_t stride[INPUTS];
  const ScanArgs& a;
  int64_t cb;  // the warp's first channel
  int lane;

  __device__ __forceinline__ Ring(const ScanArgs& args, uint8_t* m, int64_t c, int l) : mem(m), a(args), cb(c), lane(l) {}

  static __device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  }
  static __device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  }

  // Asks for the step of tokens t .. t + count - 1 (count may be 0: nothing
  // is read).  Tokens and channels outside the batch read as 0.
  __device__ __forceinline__ void fill(int slot, int64_t t, int count) {
    constexpr int kSize = Lane<DT>::kSize;
    uint8_t* to = mem + slot * kSlot;
    const int left = (int)((a.C - cb) * kSize < kRow ? (a.C - cb) * kSize : kRow);  // bytes of a row
#pragma unroll
    for (int i = 0; i < INPUTS; ++i) {
      const uint8_t* p = at<DT>(in[i], t * stride[i] + cb);
      const int64_t row_bytes = stride[i] * kSize;
      if (a.copy == 16) {
#pragma unroll
        for (int k = 0; k < kStep / 4; ++k) {
          const int row = k * 4 + (lane >> 3), col = (lane & 7) * 16;
          const int n = row < count ? (left - col < 0 ? 0 : (left - col < 16 ? left - col : 16)) : 0;
          copy16(smem_u32(to + i * kBox + row * kRow + col), n > 0 ? p + row * row_bytes + col : in[i], n);
        }
      } else if (a.copy == 4) {
#pragma unroll
        for (int row = 0; row < kStep; ++row) {
          const int col = lane * 4;
          const int n = row < count ? (left - col < 0 ? 0 : (left - col < 4 ? left - col : 4)) : 0;
          copy4(smem_u32(to + i * kBox + row * kRow + col), n > 0 ? p + row * row_bytes + col : in[i], n);
        }
      } else {
        uint32_t w[kStep];
#pragma unroll
        for (int row = 0; row < kStep; ++row)
          w[row] = row < count ? load_word<DT>(p + row * row_bytes + lane * 4, false, (left - lane * 4) / kSize) : 0;
#pragma unroll
        for (int row = 0; row < kStep; ++row) *reinterpret_cast<uint32_t*>(to + i * kBox + row * kRow + lane * 4) = w[row];
      }
    }
    if (STATES) {
#pragma unroll
      for (int v = 0; v < Lane<DT>::kVec; ++v) {
        const int64_t c = cb + v * 32 + lane;
        const bool ok = count > 0 && c < a.C;
        copy4(smem_u32(to + INPUTS * kBox + (v * 32 + lane) * 4), ok ? a.states + t / kStep * a.C + c : a.states, ok ? 4 : 0);
      }
    }
    cp_commit();
  }
  // All but the SLOTS - 1 newest steps have landed, for the whole warp.
  __device__ __forceinline__ void ready() const {
    cp_wait<SLOTS - 1>();
    __syncwarp();
  }
  // The slot has been read by the whole warp.
  __device__ __forceinline__ void done() const { __syncwarp(); }
  __device__ __forceinline__ uint32_t word(int slot, int i, int j) const {
    return *reinterpret_cast<const uint32_t*>(mem + slot * kSlot + i * kBox + j * kRow + lane * 4);
  }
  // `again`: read anew where it was read before, so that nothing made from
  // it the first time is kept in registers for the second
  __device__ __forceinline__ Two pair(int slot, int i, int p, bool again = false) const {
    uint32_t w = DT == TBE_F32 ? word(slot, i, 2 * p) : word(slot, i, p), w1 = DT == TBE_F32 ? word(slot, i, 2 * p + 1) : 0;
    if (again) asm volatile("" : "+r"(w), "+r"(w1));
    if (DT == TBE_F32) return two(__uint_as_float(w), __uint_as_float(w1));
    const float2 f = halves<DT>(w);
    return two(f.x, f.y);
  }
  __device__ __forceinline__ float state(int slot, int v) const {
    return *reinterpret_cast<const float*>(mem + slot * kSlot + INPUTS * kBox + (lane * Lane<DT>::kVec + v) * 4);
  }
};
constexpr int kX = 2, kR = 0, kG = 1, kD = 3;  // inputs of the rings that hold them all

// A warp's place: its run of tokens and its lanes' channels.
struct Place {
  int64_t t0, t1, c, cb;
  int left;  // channels of the lane inside the array
};
template <int DT>
__device__ __forceinline__ Place place_of(const ScanArgs& a, int warp, int lane) {
  Place p;
  const int64_t k = blockIdx.x / a.cblocks;
  p.cb = (int64_t)(blockIdx.x % a.cblocks) * Lane<DT>::kChannels;
  p.c = p.cb + lane * Lane<DT>::kVec;
  p.t0 = (k * kWarps + warp) * a.run;
  p.t1 = p.t0 + a.run < a.N ? p.t0 + a.run : a.N;
  if (p.t0 > p.t1) p.t0 = p.t1;
  p.left = p.c >= a.C ? 0 : (a.C - p.c < 2 ? 1 : 2);
  return p;
}

// The lane's decay rates; `near`: whether the whole warp's stay where the
// series holds (at most kNear, as sigmoids do not pass 1).
template <int DT>
__device__ __forceinline__ Two speeds(const ScanArgs& a, const Place& p, bool& near) {
  const float s0 = p.left > 0 ? speed_of(a, p.c) : 0.f;
  const float s1 = DT == TBE_F32 ? s0 : (p.left > 1 ? speed_of(a, p.c + 1) : 0.f);
  near = __all_sync(kFull, s0 < kNear && s1 < kNear);
  return two(s0, s1);
}

// Sigmoids, decays a and 1 - a^2 of a step.
template <int DT, typename RING>
__device__ __forceinline__ void step_gates(const RING& ring, int slot, Two speed, bool near, Two* sr, Two* sg, Two* A,
                                           Two* Q) {
  constexpr int kP = Lane<DT>::kPairs;
  float top = 0.f;
  if (near) {
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      gates_near(ring.pair(slot, kR, p), ring.pair(slot, kG, p), sr[p], sg[p], top);
      const Decay<Two> d = decay_near(speed * sr[p]);
      A[p] = d.a;
      Q[p] = d.q;
    }
  }
  if (!__all_sync(kFull, near && top < kTop)) {
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      gates_any(ring.pair(slot, kR, p, true), ring.pair(slot, kG, p, true), sr[p], sg[p]);
      const Decay<Two> d = decay_any(speed * sr[p]);
      A[p] = d.a;
      Q[p] = d.q;
    }
  }
}

constexpr int kForwardSlots = 4, kBackwardSlots = 3, kBackMapSlots = 6;
template <int DT>
using ForwardRing = Ring<DT, 3, kForwardSlots, false>;
template <int DT>
using BackwardRing = Ring<DT, 4, kBackwardSlots, true>;
template <int DT>
using BackMapRing = Ring<DT, 2, kBackMapSlots, false>;

// The map of a run, forward: h at its end from h at its start.  Only the
// tokens from the run's last start on count.
template <int DT>
__device__ __forceinline__ void run_map(const ScanArgs& a, const Place& p, uint8_t* mem, Two speed, bool near, int lane,
                                        Map* m) {
  constexpr int VEC = Lane<DT>::kVec, kP = Lane<DT>::kPairs;
#pragma unroll
  for (int v = 0; v < VEC; ++v) m[v] = Map{1.f, 0.f};
  if (p.t0 >= p.t1) return;
  Cursor cur(a, lane);
  int64_t first, end;
  const int64_t s = cur.owner(p.t1 - 1, true, first, end);
  const bool cut = first >= p.t0 && first < p.t1;
  if (cut) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) m[v].B = a.h0 && v < p.left ? a.h0[s * a.C + p.c + v] : 0.f;
  }
  ForwardRing<DT> ring(a, mem, p.cb, lane);
  ring.in[kX] = a.x, ring.in[kR] = a.r, ring.in[kG] = a.g;
  ring.stride[kX] = a.sx, ring.stride[kR] = a.sr, ring.stride[kG] = a.sg;
  const int64_t from = cut ? first : p.t0;
  auto count = [&](int64_t t) { return t >= p.t1 ? 0 : (p.t1 - t < kStep ? (int)(p.t1 - t) : kStep); };
#pragma unroll
  for (int i = 0; i < kForwardSlots; ++i) ring.fill(i, from + i * kStep, count(from + i * kStep));
  int slot = 0;
  for (int64_t t = from; t < p.t1; t += kStep) {
    ring.ready();
    Two sr[kP], sg[kP], A[kP], B[kP];
    step_gates<DT>(ring, slot, speed, near, sr, sg, A, B);
#pragma unroll
    for (int q = 0; q < kP; ++q) B[q] = root(B[q]) * sg[q] * ring.pair(slot, kX, q);
    ring.done();
    ring.fill(slot, t + kForwardSlots * kStep, count(t + kForwardSlots * kStep));
    slot = slot + 1 == kForwardSlots ? 0 : slot + 1;
    const int n = count(t);
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      if (j < n) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const float A_ = element<DT>(A, j, v);
          m[v].B = fmaf(A_, m[v].B, element<DT>(B, j, v));
          m[v].A *= A_;
        }
      }
    }
  }
  cp_wait<0>();
  if (cut) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) m[v].A = -1.f;
  }
}

// The map of a run, backward: a G at its start from a G behind its end.
// Only the tokens up to the run's first end count.
template <int DT>
__device__ __forceinline__ void run_map_back(const ScanArgs& a, const Place& p, uint8_t* mem, Two speed, bool near,
                                             int lane, Map* m) {
  constexpr int VEC = Lane<DT>::kVec, kP = Lane<DT>::kPairs;
#pragma unroll
  for (int v = 0; v < VEC; ++v) m[v] = Map{1.f, 0.f};
  if (p.t0 >= p.t1) return;
  Cursor cur(a, lane);
  int64_t first, end;
  const int64_t s = cur.owner(p.t0, false, first, end);
  const bool cut = end > p.t0 && end <= p.t1;
  const int64_t stop = cut ? end : p.t1;
  BackMapRing<DT> ring(a, mem, p.cb, lane);
  ring.in[kR] = a.r, ring.in[1] = a.dh;
  ring.stride[kR] = a.sr, ring.stride[1] = a.sdh;
  auto count = [&](int64_t t) { return t >= stop ? 0 : (stop - t < kStep ? (int)(stop - t) : kStep); };
#pragma unroll
  for (int i = 0; i < kBackMapSlots; ++i) ring.fill(i, p.t0 + i * kStep, count(p.t0 + i * kStep));
  int slot = 0;
  for (int64_t t = p.t0; t < stop; t += kStep) {
    ring.ready();
    Two A[kP], D[kP];
    if (near) {
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        const Two e = ex2(ring.pair(slot, kR, q) * two(-kLog2e)) + two(1.f);
        A[q] = decay_near(speed * rcp(e)).a;
      }
    } else {
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        const Two r = ring.pair(slot, kR, q);
        A[q] = decay_any(speed * two(sigmoid(lo(r)), sigmoid(hi(r)))).a;
      }
    }
#pragma unroll
    for (int q = 0; q < kP; ++q) D[q] = ring.pair(slot, 1, q);
    ring.done();
    ring.fill(slot, t + kBackMapSlots * kStep, count(t + kBackMapSlots * kStep));
    slot = slot + 1 == kBackMapSlots ? 0 : slot + 1;
    const int n = count(t);
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      if (j < n) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          float d = element<DT>(D, j, v);
          if (cut && t + j == stop - 1 && a.dh_last && v < p.left) d += a.dh_last[s * a.C + p.c + v];
          m[v].A *= element<DT>(A, j, v);
          m[v].B = fmaf(m[v].A, d, m[v].B);
        }
      }
    }
  }
  cp_wait<0>();
  if (cut) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) m[v].A = -1.f;
  }
}

__device__ __forceinline__ float2 word_of(Map m) { return make_float2(m.A, m.B); }
__device__ __forceinline__ Map map_of(float2 w) { return Map{w.x, w.y}; }

// The maps of every run and every block (scan order: BACK counts from the
// last run down).
template <int DT, bool BACK>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) maps_kernel(ScanArgs a) {
  constexpr int VEC = Lane<DT>::kVec;
  extern __shared__ __align__(128) uint8_t mem[];
  __shared__ Map runs[kWarps][64];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of<DT>(a, warp, lane);
  bool near;
  const Two speed = speeds<DT>(a, p, near);
  Map m[VEC];
  if (BACK) run_map_back<DT>(a, p, mem + warp * BackMapRing<DT>::kBytes, speed, near, lane, m);
  else run_map<DT>(a, p, mem + warp * ForwardRing<DT>::kBytes, speed, near, lane, m);
  const int64_t k = blockIdx.x / a.cblocks;
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    runs[warp][lane * VEC + v] = m[v];
    a.warp_map[(k * kWarps + warp) * a.Cp + p.c + v] = word_of(m[v]);
  }
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      Map all = runs[BACK ? kWarps - 1 : 0][lane * VEC + v];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) all = join(all, runs[BACK ? kWarps - 1 - w : w][lane * VEC + v]);
      a.block_map[k * a.Cp + p.c + v] = word_of(all);
    }
  }
}

// What reaches a warp's run: the blocks before this one, in rounds of 64 from
// the nearest on (eight to a warp), until nothing further back matters; then
// the warps before this one.  Every thread of the block calls this.
template <int DT, bool BACK>
__device__ __forceinline__ void reach(const ScanArgs& a, const Place& p, int warp, int lane, float* in) {
  constexpr int VEC = Lane<DT>::kVec;
  __shared__ Map part[kWarps][64];
  const int64_t k = blockIdx.x / a.cblocks;
  const int64_t before = BACK ? a.blocks - 1 - k : k;  // blocks before this one in scan order
  Map all[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) all[v] = Map{1.f, 0.f};
  for (int64_t done = 0; done < before && !(all[0].A < 0.f); done += 8 * kWarps) {
    // this warp's eight, farthest first, `done + 8 * warp` blocks away at least
    Map m[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) m[v] = Map{1.f, 0.f};
    float2 w[8][VEC];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t away = done + 8 * warp + 8 - j;  // 1: the neighbour
      const int64_t b = BACK ? k + away : k - away;
#pragma unroll
      for (int v = 0; v < VEC; ++v) w[j][v] = away <= before ? __ldcg(a.block_map + b * a.Cp + p.c + v) : make_float2(1.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int v = 0; v < VEC; ++v) m[v] = join(m[v], map_of(w[j][v]));
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VEC; ++v) part[warp][lane * VEC + v] = m[v];
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      Map round = part[kWarps - 1][lane * VEC + v];
#pragma unroll
      for (int j = kWarps - 2; j >= 0; --j) round = join(round, part[j][lane * VEC + v]);
      all[v] = join(round, all[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) in[v] = apply(all[v], 0.f);
  float2 w[kWarps - 1][VEC];
#pragma unroll
  for (int j = 0; j < kWarps - 1; ++j) {
    const int r = BACK ? kWarps - 1 - j : j;  // in scan order
    const bool mine = BACK ? r > warp : r < warp;
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      w[j][v] = mine ? __ldcg(a.warp_map + (k * kWarps + r) * a.Cp + p.c + v) : make_float2(1.f, 0.f);
  }
#pragma unroll
  for (int j = 0; j < kWarps - 1; ++j)
#pragma unroll
    for (int v = 0; v < VEC; ++v) in[v] = apply(map_of(w[j][v]), in[v]);
}

// The same where one block holds all tokens: the warps' maps are made here.
template <int DT, bool BACK>
__device__ __forceinline__ void reach_alone(const Map* m, int warp, int lane, float* in) {
  constexpr int VEC = Lane<DT>::kVec;
  __shared__ Map runs[kWarps][64];
#pragma unroll
  for (int v = 0; v < VEC; ++v) runs[warp][lane * VEC + v] = m[v];
  __syncthreads();
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    in[v] = 0.f;
    for (int j = BACK ? kWarps - 1 : 0; j != warp; j += BACK ? -1 : 1) in[v] = apply(runs[j][lane * VEC + v], in[v]);
  }
}

// Empty sequences hand their states on (to[s] = from[s], 0 where there is no
// `from`; nothing where there is no `to`), and broken offsets are reported:
// ones that do not start at 0, end at N, or that decrease.  The blocks share
// the sequences.
__device__ __forceinline__ void empty_sequences(const ScanArgs& a, const float* from, float* to) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kWarps, me = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  bool bad = false;
  for (int64_t base = me * 32; base <= a.S; base += warps * 32) {
    const int64_t s = base + lane;
    int64_t o = 0, e = 0;
    if (s <= a.S) {
      o = a.offsets.ldg(s);
      if (s == 0) bad |= o != 0;
      if (s == a.S) bad |= o != a.N;
      else e = a.offsets.ldg(s + 1);
      if (s < a.S) bad |= e < o;
    }
    uint32_t empty = __ballot_sync(kFull, s < a.S && e == o);
    if (to == nullptr) empty = 0;
    for (; empty; empty &= empty - 1) {
      const int64_t row = (base + __ffs(empty) - 1) * a.C;
      for (int64_t c = lane; c < a.C; c += 32) to[row + c] = from ? from[row + c] : 0.f;
    }
  }
  if (bad) report(a.status, TBE_DEV_BAD_OFFSETS);
}

// ALONE: the batch is one block's tokens, no maps kernel ran.
template <int DT, bool ALONE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) forward_kernel(ScanArgs a) {
  constexpr int VEC = Lane<DT>::kVec, kP = Lane<DT>::kPairs;
  extern __shared__ __align__(128) uint8_t mem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of<DT>(a, warp, lane);
  bool near;
  const Two speed = speeds<DT>(a, p, near);
  float h[VEC];
  if (ALONE) {
    Map m[VEC];
    run_map<DT>(a, p, mem + warp * ForwardRing<DT>::kBytes, speed, near, lane, m);
    reach_alone<DT, false>(m, warp, lane, h);
    __syncwarp();
  }
  ForwardRing<DT> ring(a, mem + warp * ForwardRing<DT>::kBytes, p.cb, lane);
  ring.in[kX] = a.x, ring.in[kR] = a.r, ring.in[kG] = a.g;
  ring.stride[kX] = a.sx, ring.stride[kR] = a.sr, ring.stride[kG] = a.sg;
  auto count = [&](int64_t t) { return t >= p.t1 ? 0 : (p.t1 - t < kStep ? (int)(p.t1 - t) : kStep); };
#pragma unroll
  for (int i = 0; i < kForwardSlots; ++i) ring.fill(i, p.t0 + i * kStep, count(p.t0 + i * kStep));
  empty_sequences(a, a.h0, a.h_last);
  if (!ALONE) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    reach<DT, false>(a, p, warp, lane, h);
  }
  Cursor cur(a, lane);
  Events ev;
  int slot = 0;
  for (int64_t t = p.t0; t < p.t1; t += kStep) {
    const int n = count(t);
    ev.find(cur, t, n, false, lane);
    ring.ready();
    Two sr[kP], sg[kP], A[kP], B[kP];
    step_gates<DT>(ring, slot, speed, near, sr, sg, A, B);
#pragma unroll
    for (int q = 0; q < kP; ++q) B[q] = root(B[q]) * sg[q] * ring.pair(slot, kX, q);
    ring.done();
    ring.fill(slot, t + kForwardSlots * kStep, count(t + kForwardSlots * kStep));
    slot = slot + 1 == kForwardSlots ? 0 : slot + 1;
    if (a.states) {
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if (v < p.left) a.states[t / kStep * a.C + p.c + v] = h[v];
    }
    uint8_t* to = at<DT>(a.h, t * a.sh + p.c);
    const int64_t row = a.sh * Lane<DT>::kSize;
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      if (ev.starts >> j & 1) {
        const int64_t s = ev.sequence(j);
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = a.h0 && v < p.left ? a.h0[s * a.C + p.c + v] : 0.f;
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) h[v] = fmaf(element<DT>(A, j, v), h[v], element<DT>(B, j, v));
      if (j < n) store_word<DT>(to + j * row, a.pairs, p.left, h[0], h[VEC - 1]);
      if (ev.ends >> j & 1) {
        const int64_t s = ev.sequence(j);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if (v < p.left) a.h_last[s * a.C + p.c + v] = h[v];
      }
    }
  }
  cp_wait<0>();
}

template <int DT, bool ALONE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) backward_kernel(ScanArgs a) {
  constexpr int VEC = Lane<DT>::kVec, kP = Lane<DT>::kPairs;
  extern __shared__ __align__(128) uint8_t mem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of<DT>(a, warp, lane);
  bool near;
  const Two speed = speeds<DT>(a, p, near);
  float c[VEC], share[VEC];
  if (ALONE) {
    Map m[VEC];
    run_map_back<DT>(a, p, mem + warp * BackwardRing<DT>::kBytes, speed, near, lane, m);
    reach_alone<DT, true>(m, warp, lane, c);
    __syncwarp();
  }
  BackwardRing<DT> ring(a, mem + warp * BackwardRing<DT>::kBytes, p.cb, lane);
  ring.in[kX] = a.x, ring.in[kR] = a.r, ring.in[kG] = a.g, ring.in[kD] = a.dh;
  ring.stride[kX] = a.sx, ring.stride[kR] = a.sr, ring.stride[kG] = a.sg, ring.stride[kD] = a.sdh;
  // steps from the run's last one down
  const int64_t last = p.t0 < p.t1 ? p.t0 + (p.t1 - 1 - p.t0) / kStep * kStep : p.t0;
  auto count = [&](int64_t t) { return t < p.t0 || t >= p.t1 ? 0 : (p.t1 - t < kStep ? (int)(p.t1 - t) : kStep); };
#pragma unroll
  for (int i = 0; i < kBackwardSlots; ++i) {
    const int64_t t = last - (int64_t)i * kStep;
    ring.fill(i, t < p.t0 ? p.t0 : t, count(t));
  }
  empty_sequences(a, a.dh_last, a.dh0);
  if (!ALONE) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    reach<DT, true>(a, p, warp, lane, c);
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) share[v] = 0.f;
  Cursor cur(a, lane);
  Events ev;
  int slot = 0;
  if (p.t0 < p.t1) {
    for (int64_t t = last; t >= p.t0; t -= kStep) {
      const int n = count(t);
      ev.find(cur, t, n, true, lane);
      ring.ready();
      Two sr[kP], sg[kP], A[kP], inv[kP], beta[kP];
      step_gates<DT>(ring, slot, speed, near, sr, sg, A, beta);
      // the states that the step's tokens find
      float before[kStep][VEC], h[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) h[v] = ring.state(slot, v);
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        // where 1 - a^2 is 0 the token takes nothing in, and its gate's slope
        // u d beta / d u = u a^2 / beta goes to 0 with u
        const Two safe = two(fmaxf(lo(beta[q]), 1e-37f), fmaxf(hi(beta[q]), 1e-37f));
        inv[q] = inv_root(safe);
        beta[q] = beta[q] * inv[q];
        const Two b = beta[q] * sg[q] * ring.pair(slot, kX, q);
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // the pair's tokens, or its channels
          const int j = DT == TBE_F32 ? 2 * q + e : q, v = DT == TBE_F32 ? 0 : e;
          if (ev.starts >> j & 1) {
            const int64_t s = ev.sequence(j);
            h[v] = a.h0 && v < p.left ? a.h0[s * a.C + p.c + v] : 0.f;
          }
          before[j][v] = h[v];
          h[v] = fmaf(e ? hi(A[q]) : lo(A[q]), h[v], e ? hi(b) : lo(b));
        }
      }
#pragma unroll
      for (int q = kP - 1; q >= 0; --q) {
        const Two x = ring.pair(slot, kX, q, true), dh = ring.pair(slot, kD, q);
        float G[2];
#pragma unroll
        for (int e = 1; e >= 0; --e) {
          const int j = DT == TBE_F32 ? 2 * q + e : q, v = DT == TBE_F32 ? 0 : e;
          G[e] = e ? hi(dh) : lo(dh);
          if (ev.ends >> j & 1) {
            const int64_t s = ev.sequence(j);
            if (a.dh_last && v < p.left) G[e] += a.dh_last[s * a.C + p.c + v];
          } else if (j < n) {
            G[e] += c[v];
          }
          if (j < n) c[v] = (e ? hi(A[q]) : lo(A[q])) * G[e];
          if (ev.starts >> j & 1) {
            const int64_t s = ev.sequence(j);
            if (a.dh0 && v < p.left) a.dh0[s * a.C + p.c + v] = c[v];
          }
        }
        const Two g2 = two(G[0], G[1]), minus = two(-1.f), one = two(1.f);
        const Two ua = speed * sr[q] * A[q], sx = sg[q] * x;
        const Two found = DT == TBE_F32 ? two(before[2 * q & 7][0], before[(2 * q + 1) & 7][0])
                                        : two(before[q & 7][0], before[q & 7][VEC - 1]);
        const Two w = g2 * ua * fma2(A[q] * inv[q], sx, minus * found);
        const Two dx = g2 * beta[q] * sg[q], dg = dx * x * fma2(sg[q], minus, one), dr = w * fma2(sr[q], minus, one);
#pragma unroll
        for (int e = 0; e < (DT == TBE_F32 ? 2 : 1); ++e) {
          const int j = DT == TBE_F32 ? 2 * q + e : q;
          if (j < n) {
            const int64_t tj = t + j;
            store_word<DT>(at<DT>(a.dx, tj * a.sdx + p.c), a.pairs, p.left, e ? hi(dx) : lo(dx), hi(dx));
            store_word<DT>(at<DT>(a.dr, tj * a.sdr + p.c), a.pairs, p.left, e ? hi(dr) : lo(dr), hi(dr));
            store_word<DT>(at<DT>(a.dg, tj * a.sdg + p.c), a.pairs, p.left, e ? hi(dg) : lo(dg), hi(dg));
            if (DT == TBE_F32) {
              share[0] += e ? hi(w) : lo(w);
            } else {
              share[0] += lo(w);
              share[VEC - 1] += hi(w);
            }
          }
        }
      }
      ring.done();
      const int64_t next = t - kBackwardSlots * kStep;
      ring.fill(slot, next < p.t0 ? p.t0 : next, count(next));
      slot = slot + 1 == kBackwardSlots ? 0 : slot + 1;
    }
  }
  cp_wait<0>();
#pragma unroll
  for (int v = 0; v < VEC; ++v)
    if (v < p.left) a.partial[((int64_t)(blockIdx.x / a.cblocks) * kWarps + warp) * a.C + p.c + v] = share[v];
}

// ddecay = sigmoid(decay) / softplus(decay) * sum over the runs, 32 channels
// per block, its warps each a share of the runs.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32)
    decay_grad_kernel(const float* partial, const float* decay, float* ddecay, int32_t rows, int32_t C) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float part[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < C)
    for (int64_t k = warp; k < rows; k += kSumWarps) s += partial[k * C + c];
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
template <int DT>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs a) {
  constexpr int VEC = Lane<DT>::kVec;
  const int64_t per_row = (a.C + VEC - 1) / VEC;
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (i >= per_row * a.S) return;
  const int64_t s = i / per_row, c = (i - s * per_row) * VEC;
  const int left = a.C - c < 2 ? 1 : 2;
  const uint32_t x = load_word<DT>(at<DT>(a.x, s * a.sx + c), a.pairs, left);
  const uint32_t r = load_word<DT>(at<DT>(a.r, s * a.sr + c), a.pairs, left);
  const uint32_t g = load_word<DT>(at<DT>(a.g, s * a.sg + c), a.pairs, left);
  float* state = a.h_last + s * a.C + c;
  float h[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    h[v] = 0.f;
    if (v < left) {
      auto of = [&](uint32_t w) {
        if (DT == TBE_F32) return __uint_as_float(w);
        const float2 f = halves<DT>(w);
        return v ? f.y : f.x;
      };
      const Decay<float> d = decay_of(speed_of(a, c + v) * sigmoid(of(r)));
      h[v] = fmaf(d.a, state[v], root(d.q) * sigmoid(of(g)) * of(x));
      state[v] = h[v];
    }
  }
  store_word<DT>(at<DT>(a.h, s * a.sh + c), a.pairs, left, h[0], h[VEC - 1]);
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int64_t whole_channels(int32_t C) { return ((int64_t)C + 63) / 64 * 64; }
int32_t channel_blocks(int32_t C, int32_t dtype) { return dtype == TBE_F32 ? (C + 31) / 32 : (C + 63) / 64; }

// Tokens per warp: as many as give every warp that fits on the GPU one run,
// in whole steps.  Up to kAlone tokens one block takes the whole batch (both
// passes in one kernel, no second launch).
constexpr int64_t kAlone = 256;
struct Split {
  int32_t run, blocks;
};
Split split_of(int64_t N, int32_t cblocks) {
  const int64_t warps = (int64_t)sm_count() * kBlocksPerSm * kWarps / cblocks;
  const int64_t parts = N <= kAlone || warps < kWarps ? kWarps : warps / kWarps * kWarps;
  int64_t run = ((N + parts - 1) / parts + kStep - 1) / kStep * kStep;
  if (run < kStep) run = kStep;
  Split s;
  s.run = (int32_t)run;
  s.blocks = (int32_t)((N + run * kWarps - 1) / (run * kWarps));
  if (s.blocks < 1) s.blocks = 1;
  return s;
}

// The workspace: maps of blocks and runs, then the backward's partial sums.
struct Workspace {
  size_t block, warp, partial, bytes;
};
Workspace layout(int64_t N, int32_t C, int32_t dtype, bool backward) {
  const Split sp = split_of(N, channel_blocks(C, dtype));
  const size_t Cp = (size_t)whole_channels(C);
  Workspace w;
  size_t at = 0;
  w.block = w.warp = 0;
  if (sp.blocks > 1) {
    at += round256((size_t)sp.blocks * Cp * sizeof(float2));
    w.warp = at;
    at += round256((size_t)sp.blocks * kWarps * Cp * sizeof(float2));
  }
  w.partial = at;
  if (backward) at += round256((size_t)sp.blocks * kWarps * C * 4);
  w.bytes = at;
  return w;
}

bool aligned_to(const void* p, int64_t stride_bytes, int n) { return ((uintptr_t)p & (n - 1)) == 0 && stride_bytes % n == 0; }

// How rows may be read and written: bytes per asynchronous copy of an input,
// and whether two half-precision channels can be stored at once.
void choose_access(ScanArgs& a, int32_t dtype) {
  const int size = dtype == TBE_F32 ? 4 : 2;
  auto all = [&](int n) {
    return aligned_to(a.x, a.sx * size, n) && aligned_to(a.r, a.sr * size, n) && aligned_to(a.g, a.sg * size, n) &&
           (!a.dh || aligned_to(a.dh, a.sdh * size, n));
  };
  a.copy = all(16) ? 16 : all(4) ? 4 : 0;
  a.pairs = a.copy != 0;  // the step kernel reads pairs too
  if (dtype != TBE_F32 && a.h) a.pairs = a.pairs && aligned_to(a.h, a.sh * size, 4);
  if (dtype != TBE_F32 && a.dh)
    a.pairs = a.pairs && aligned_to(a.dx, a.sdx * size, 4) && aligned_to(a.dr, a.sdr * size, 4) && aligned_to(a.dg, a.sdg * size, 4);
}

template <typename K>
int start(K kernel, unsigned grid, unsigned threads, size_t smem, bool after, cudaStream_t s, const ScanArgs& a) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return TBE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;  // may start while the kernel before it ends
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? check_launch() : TBE_ERR_CUDA;
}

template <int DT, bool BACK>
int launch_scan(const ScanArgs& a, cudaStream_t s) {
  constexpr size_t ring = kWarps * (size_t)(BACK ? BackwardRing<DT>::kBytes : ForwardRing<DT>::kBytes);
  constexpr size_t map_ring = kWarps * (size_t)(BACK ? BackMapRing<DT>::kBytes : ForwardRing<DT>::kBytes);
  static_assert(!BACK || ring >= map_ring, "the maps of a lone block use the same ring");
  const unsigned grid = (unsigned)a.blocks * (unsigned)a.cblocks;
  if (a.blocks == 1) {
    if constexpr (BACK) return start(backward_kernel<DT, true>, grid, kThreads, ring, false, s, a);
    else return start(forward_kernel<DT, true>, grid, kThreads, ring, false, s, a);
  }
  const int st = start(maps_kernel<DT, BACK>, grid, kThreads, map_ring, false, s, a);
  if (st != TBE_OK) return st;
  trace_mark(s, BACK ? "gated_scan_maps_back" : "gated_scan_maps");
  if constexpr (BACK) return start(backward_kernel<DT, false>, grid, kThreads, ring, true, s, a);
  else return start(forward_kernel<DT, false>, grid, kThreads, ring, true, s, a);
}

template <int DT>
int launch_step(const ScanArgs& a, cudaStream_t s) {
  const int64_t n = (int64_t)a.S * ((a.C + Lane<DT>::kVec - 1) / Lane<DT>::kVec);
  scan_step_kernel<DT><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(a);
  return check_launch();
}

enum { kForward, kBackward, kOne };

template <int DT>
int launch(ScanArgs& a, int what, cudaStream_t s) {
  if (what == kOne) return launch_step<DT>(a, s);
  return what == kForward ? launch_scan<DT, false>(a, s) : launch_scan<DT, true>(a, s);
}

int dispatch(ScanArgs& a, int32_t dtype, int what, cudaStream_t s) {
  choose_access(a, dtype);
  if (dtype == TBE_F32) return launch<TBE_F32>(a, what, s);
  if (dtype == TBE_F16) return launch<TBE_F16>(a, what, s);
  return launch<TBE_BF16>(a, what, s);
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
  a.h0 = in->h0;
  a.cblocks = channel_blocks(in->channels, in->dtype);
  const Split sp = split_of(in->tokens, a.cblocks);
  a.run = sp.run;
  a.blocks = sp.blocks;
  a.Cp = whole_channels(in->channels);
  return a;
}

int check_jagged(const tbe_scan_inputs* in) {
  const int st = check(in);
  if (st != TBE_OK) return st;
  if (!in->offsets || (in->tokens > 0 && in->sequences == 0)) return TBE_ERR_INVALID_ARG;
  return TBE_OK;
}

int use_workspace(ScanArgs& a, int32_t dtype, bool backward, void* workspace, size_t bytes) {
  const Workspace w = layout(a.N, a.C, dtype, backward);
  if (bytes < w.bytes) return TBE_ERR_WORKSPACE;
  if (w.bytes == 0) return TBE_OK;
  if (!workspace) return TBE_ERR_INVALID_ARG;
  if ((uintptr_t)workspace & 255) return TBE_ERR_UNSUPPORTED;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  a.block_map = reinterpret_cast<float2*>(p + w.block);
  a.warp_map = reinterpret_cast<float2*>(p + w.warp);
  a.partial = reinterpret_cast<float*>(p + w.partial);
  return TBE_OK;
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" {

int64_t tbe_gated_scan_states(int64_t tokens) { return tokens < 1 ? 1 : (tokens + kStep - 1) / kStep; }

size_t tbe_gated_scan_workspace_bytes(int64_t tokens, int32_t channels, int32_t dtype, int32_t backward) {
  if (tokens < 0 || channels < 1) return 0;
  return layout(tokens, channels, dtype, backward != 0).bytes;
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
  st = use_workspace(a, in->dtype, false, workspace, workspace_bytes);
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
  st = use_workspace(a, in->dtype, true, workspace, workspace_bytes);
  if (st != TBE_OK) return st;
  st = dispatch(a, in->dtype, kBackward, s);
  if (st != TBE_OK) return st;
  trace_mark(s, "gated_scan_backward");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.C + 31) / 32));
  cfg.blockDim = dim3(kSumWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, decay_grad_kernel, (const float*)a.partial, a.decay, out->ddecay, a.blocks * kWarps,
                         a.C) != cudaSuccess)
    return TBE_ERR_CUDA;
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
