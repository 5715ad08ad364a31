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
// A warp takes a run of tokens and 32 channels, a block's warps neighbouring
// runs.  h over a run is the linear map h_out = A h_in + B, so two passes do
// it:
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
#include "tbe_two.cuh"

#include <cmath>

namespace tbe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kStep = TBE_SCAN_STEP;  // tokens per step (and between saved states)
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// blocks that stay resident on an SM: the forward fits 80 registers, the
// backward would spill there
template <bool BACK>
constexpr int kBlocksPerSm = BACK ? 2 : 3;
constexpr int kPairs = kStep / 2;  // neighbouring tokens of a step, two at a time
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
  int32_t run;      // tokens per warp, whole slots of the rings
  int32_t blocks;   // along the tokens
  int32_t cblocks;  // along the channels
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
  float* partial;    // [blocks, C]: each block's share of the decay's gradient
  float* ddecay;
  uint32_t* arrived; // [cblocks]: blocks that have written their share
  float2* warp_map;  // [blocks * kWarps, Cp]
  float2* block_map; // [blocks, Cp]
  int32_t* status;
};

__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// a = exp(-u) and 1 - a^2 for u >= 0, both to a few units of their own
// size.  Below 1/4, n = 1 - a from its series (the next term is under 5e-8 of
// the sum): near a = 1 its rounding is relative to 1 - a, which is what
// decides how long a state lives, and 1 - a^2 = n (2 - n) keeps it.
constexpr float kNear = 0.25f;
template <typename T>
struct Decay {
  T a, q;
};
// The constants of two-wide arithmetic, made once per thread: an instruction
// takes them from registers only, and the compiler would otherwise move them
// there again at each use.
struct Constants {
  Two one, minus_log2e, c5, c4, c3, c2, c1, c0;
  __device__ __forceinline__ Constants()
      : one(keep(1.f)), minus_log2e(keep(-kLog2e)), c5(keep(1.f / 720.f)), c4(keep(-1.f / 120.f)), c3(keep(1.f / 24.f)),
        c2(keep(-1.f / 6.f)), c1(keep(0.5f)), c0(keep(-1.f)) {}
};
__device__ __forceinline__ Decay<Two> decay_near(Two u, const Constants& k) {
  Two p = fma2(u, k.c5, k.c4);
  p = fma2(u, p, k.c3);
  p = fma2(u, p, k.c2);
  p = fma2(u, p, k.c1);
  p = fma2(u, p, k.c0);
  const Two m = u * p;  // a - 1
  Decay<Two> d;
  d.a = m + k.one;
  d.q = negative(m) * (d.a + k.one);
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
__device__ __forceinline__ void gates_near(Two r, Two g, const Constants& k, Two& sr, Two& sg, float& top) {
  const Two pr = ex2(r * k.minus_log2e) + k.one, pg = ex2(g * k.minus_log2e) + k.one;
  const Two product = pr * pg, inv = rcp(product);
  sr = inv * pg;
  sg = inv * pr;
  top = fmaxf(fmaxf(top, lo(product)), hi(product));
}
__device__ __forceinline__ void gates_any(Two r, Two g, Two& sr, Two& sg) {
  sr = two(sigmoid(lo(r)), sigmoid(hi(r)));
  sg = two(sigmoid(lo(g)), sigmoid(hi(g)));
}

template <int DT>
constexpr int kSize = DT == TBE_F32 ? 4 : 2;
template <int DT>
__device__ __forceinline__ const uint8_t* at(const void* p, int64_t e) {
  return static_cast<const uint8_t*>(p) + e * kSize<DT>;
}
template <int DT>
__device__ __forceinline__ uint8_t* at(void* p, int64_t e) {
  return static_cast<uint8_t*>(p) + e * kSize<DT>;
}
// An element's bits, and as a number.
template <int DT>
__device__ __forceinline__ uint32_t load_bits(const uint8_t* p) {
  if (DT == TBE_F32) return *reinterpret_cast<const uint32_t*>(p);
  return *reinterpret_cast<const uint16_t*>(p);
}
template <int DT>
__device__ __forceinline__ float number(uint32_t b) {
  if (DT == TBE_F32) return __uint_as_float(b);
  if (DT == TBE_BF16) return __uint_as_float(b << 16);
  return __half2float(__ushort_as_half((unsigned short)b));
}
// Stores a pair's two tokens; `both`: the second lies inside the batch.
template <int DT>
__device__ __forceinline__ void store_pair(uint8_t* p, int64_t row, float a, float b, bool one, bool both) {
  if (DT == TBE_F32) {
    if (one) *reinterpret_cast<float*>(p) = a;
    if (both) *reinterpret_cast<float*>(p + row) = b;
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
  if (one) *reinterpret_cast<uint16_t*>(p) = (uint16_t)v;
  if (both) *reinterpret_cast<uint16_t*>(p + row) = (uint16_t)(v >> 16);
}
__device__ __forceinline__ float element(const Two* t, int j) { return j & 1 ? hi(t[j >> 1]) : lo(t[j >> 1]); }

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
  int32_t quiet;  // steps to come that lie inside it
  __device__ __forceinline__ Events() : starts(0), ends(0), s(0), first(0), end(-1), owner(0), quiet(0) {}
  __device__ __forceinline__ void find(Cursor& cur, int64_t t, int count, bool down, int lane) {
    starts = ends = 0;
    if (quiet > 0) {
      --quiet;
      return;
    }
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
    if (down) cur.owner(t, true, first, end);  // the sequence that goes on below
    // later steps t' with t' + kStep < end (downwards: first < t')
    const int64_t room = down ? (t - first - 1) / kStep : (end - t - kStep - 1) / kStep;
    quiet = room < 0 ? 0 : (room < (1 << 30) ? (int)room : 1 << 30);
  }
  __device__ __forceinline__ int64_t sequence(int j) const { return __shfl_sync(kFull, s, j); }
};

// A warp's ring.  A slot holds kTokens<DT> tokens of 32 channels of each input,
// then (DOWN) the states that its steps start from.  Slots are filled upwards,
// or downwards, from where the ring was set until the run's tokens are all
// asked for.  WIDE: rows start
// on 16 bytes and channels come in whole 16-byte pieces; otherwise a copy is
// of 4 bytes, or (half precision at odd places) an element at a time.
template <int DT>
constexpr int kTokens = DT == TBE_F32 ? kStep : 2 * kStep;
template <int DT, int INPUTS, int SLOTS, bool DOWN, bool WIDE>
struct Ring {
  static constexpr int kTok = kTokens<DT>;
  static constexpr int kRow = 32 * kSize<DT>, kBox = kTok * kRow;
  static constexpr int kSlot = INPUTS * kBox + (DOWN ? kTok / kStep * 128 : 0);
  static constexpr int kBytes = SLOTS * kSlot;
  static constexpr int kLanes = kRow / 16;  // of a row, 16 bytes each
  const uint8_t* mem;
  const uint8_t* now;
  const uint8_t* src[INPUTS];  // this lane's first piece of the next step
  int64_t row[INPUTS];         // bytes between tokens
  const float* state;
  const ScanArgs& a;
  uint32_t base;  // of slot 0, in shared memory
  int bytes;      // of a lane's piece inside the array
  bool on;        // the lane's channel lies inside the array
  int lane;
  int read, write;  // bytes from slot 0: the oldest slot, the next to be filled
  int left;         // tokens of the run that are not asked for yet

  // `tokens`: of the run; downwards the first slot takes what does not fill one
  __device__ __forceinline__ Ring(const ScanArgs& args, uint8_t* m, int64_t cb, int l, int tokens)
      : mem(m), now(m), state(nullptr), a(args), base(smem_u32(m)), lane(l), read(0), write(0), left(tokens) {
    const int left = (int)((a.C - cb) * kSize<DT> < kRow ? (a.C - cb) * kSize<DT> : kRow);
    const int piece = WIDE ? 16 : a.copy == 4 ? 4 : kSize<DT>;
    const int b = left - col();
    bytes = b < 0 ? 0 : (b < piece ? b : piece);
    on = cb + l < a.C;
  }
  // the lane's place in a row, and the first row it copies
  __device__ __forceinline__ int col() const {
    return WIDE ? lane % kLanes * 16 : a.copy == 4 ? lane % (kRow / 4) * 4 : lane * kSize<DT>;
  }
  __device__ __forceinline__ int first_row() const { return WIDE ? lane / kLanes : a.copy == 4 ? lane / (kRow / 4) : 0; }
  __device__ __forceinline__ void input(int i, const void* p, int64_t stride, int64_t t, int64_t cb) {
    row[i] = stride * kSize<DT>;
    src[i] = at<DT>(p, t * stride + cb) + first_row() * row[i] + col();
  }
  static __device__ __forceinline__ void copy16(uint32_t dst, const void* from, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(n) : "memory");
  }
  static __device__ __forceinline__ void copy4(uint32_t dst, const void* from, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(from), "r"(n) : "memory");
  }
  // A slot of `count` tokens, by any kind of copy.  What lies outside the run
  // (in the batch's last one), or outside the channels, reads as 0.
  __device__ __forceinline__ void fill_part(int count) {
    const uint32_t to = base + write;
#pragma unroll
    for (int i = 0; i < INPUTS; ++i) {
      const uint8_t* from = src[i];
      if (WIDE) {
        constexpr int kRows = 32 / kLanes;
#pragma unroll
        for (int k = 0; k < kTok / kRows; ++k) {
          const int n = k * kRows + first_row() < count ? bytes : 0;
          copy16(to + i * kBox + k * 512 + lane * 16, n ? from : a.x, n);
          from += kRows * row[i];
        }
      } else if (a.copy == 4) {
        constexpr int kRows = 128 / kRow;
#pragma unroll
        for (int k = 0; k < kTok / kRows; ++k) {
          const int n = k * kRows + first_row() < count ? bytes : 0;
          copy4(to + i * kBox + k * 128 + lane * 4, n ? from : a.x, n);
          from += kRows * row[i];
        }
      } else {
        uint32_t w[kTok];
#pragma unroll
        for (int k = 0; k < kTok; ++k) w[k] = k < count && bytes ? load_bits<DT>(from + k * row[i]) : 0;
#pragma unroll
        for (int k = 0; k < kTok; ++k)
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + i * kBox + k * kRow + lane * 2), "h"((uint16_t)w[k]) : "memory");
      }
      src[i] += (DOWN ? -kTok : kTok) * row[i];
    }
    if (DOWN) {
#pragma unroll
      for (int u = 0; u < kTok / kStep; ++u) {
        const int n = u * kStep < count && on ? 4 : 0;
        copy4(to + INPUTS * kBox + u * 128 + lane * 4, n ? (const void*)(state + (int64_t)u * a.C) : a.x, n);
      }
      state -= (int64_t)(kTok / kStep) * a.C;
    }
  }
  // The next slot.
  __device__ __forceinline__ void fill() {
    int count = left < kTok ? left : kTok;
    if (DOWN && left > kTok && left % kTok) count = left % kTok;
    left -= count;
    if (WIDE && count == kTok) {
      const uint32_t to = base + write + lane * 16;
      constexpr int kRows = 32 / kLanes;
#pragma unroll
      for (int i = 0; i < INPUTS; ++i) {
#pragma unroll
        for (int k = 0; k < kTok / kRows; ++k) copy16(to + i * kBox + k * 512, src[i] + k * kRows * row[i], bytes);
        src[i] += (DOWN ? -kTok : kTok) * row[i];
      }
      if (DOWN) {
#pragma unroll
        for (int u = 0; u < kTok / kStep; ++u)
          copy4(base + write + lane * 4 + INPUTS * kBox + u * 128, state + (int64_t)u * a.C, on ? 4 : 0);
        state -= (int64_t)(kTok / kStep) * a.C;
      }
    } else {
      fill_part(count);
    }
    cp_commit();
    write = write + kSlot == kBytes ? 0 : write + kSlot;
  }
  // The oldest slot has landed, for the whole warp.
  __device__ __forceinline__ void ready() const {
    cp_wait<SLOTS - 1>();
    __syncwarp();
  }
  // It has been read by the whole warp and takes other tokens.
  __device__ __forceinline__ void done() {
    __syncwarp();
    fill();
    read = write;
  }
  // step u of the slot, of which the next reads are
  __device__ __forceinline__ void step(int u) { now = mem + read + u * (kStep * kRow) + lane * kSize<DT>; }
  __device__ __forceinline__ uint32_t bits(int i, int j) const { return load_bits<DT>(now + (i * kBox + j * kRow)); }
  // `again`: read anew where it was read before, so that nothing made from
  // it the first time is kept in registers for the second
  __device__ __forceinline__ Two pair(int i, int p, bool again = false) const {
    uint32_t w0 = bits(i, 2 * p), w1 = bits(i, 2 * p + 1);
    if (again) asm volatile("" : "+r"(w0), "+r"(w1));
    return two(number<DT>(w0), number<DT>(w1));
  }
  __device__ __forceinline__ float first_state(int u) const {
    return *reinterpret_cast<const float*>(mem + read + INPUTS * kBox + u * 128 + lane * 4);
  }
};

// One output of a warp, a step at a time.  WIDE: gathered in shared memory and
// written 16 bytes to a lane; otherwise each element on its own.
template <int DT, bool DOWN, bool WIDE>
struct Out {
  static constexpr int kRow = 32 * kSize<DT>, kLanes = kRow / 16, kRows = 32 / kLanes;
  uint8_t* to;    // this lane's first piece of the step
  uint8_t* room;  // kStep rows of shared memory (WIDE)
  int64_t row;
  int lane;
  bool on;
  __device__ __forceinline__ Out(void* p, int64_t stride, int64_t t, int64_t cb, int32_t C, uint8_t* m, int l)
      : room(m), row(stride * kSize<DT>), lane(l) {
    const int col = WIDE ? l % kLanes * 16 : l * kSize<DT>;
    on = cb * kSize<DT> + col < (int64_t)C * kSize<DT>;
    to = at<DT>(p, t * stride + cb) + col + (WIDE ? l / kLanes * row : 0);
  }
  // pair q of the step (`n` tokens of it lie inside the batch)
  __device__ __forceinline__ void put(int q, float a, float b, int n) {
    if (WIDE) store_pair<DT>(room + lane * kSize<DT> + 2 * q * kRow, kRow, a, b, true, true);
    else store_pair<DT>(to + 2 * q * row, row, a, b, on && 2 * q < n, on && 2 * q + 1 < n);
  }
  // the step is complete (the caller puts a __syncwarp before and after)
  __device__ __forceinline__ void flush(int n) {
    if (WIDE) {
#pragma unroll
      for (int k = 0; k < kStep / kRows; ++k)
        if (on && (n == kStep || k * kRows + lane / kLanes < n))
          *reinterpret_cast<uint4*>(to + k * kRows * row) = *reinterpret_cast<const uint4*>(room + k * 512 + lane * 16);
    }
    to += (DOWN ? -kStep : kStep) * row;
  }
};
constexpr int kR = 0, kG = 1, kX = 2, kD = 3;  // inputs of the rings that hold them all

// A warp's place: its run of tokens and its lanes' channels.
struct Place {
  int64_t t0, t1, c, cb;
  bool on;  // the lane's channel lies inside the array
};
__device__ __forceinline__ Place place_of(const ScanArgs& a, int warp, int lane) {
  Place p;
  const int64_t k = blockIdx.x / a.cblocks;
  p.cb = (int64_t)(blockIdx.x % a.cblocks) * 32;
  p.c = p.cb + lane;
  p.t0 = (k * kWarps + warp) * a.run;
  p.t1 = p.t0 + a.run < a.N ? p.t0 + a.run : a.N;
  if (p.t0 > p.t1) p.t0 = p.t1;
  p.on = p.c < a.C;
  return p;
}

// The lane's decay rate; `near`: whether the whole warp's stay where the
// series holds (at most kNear, as sigmoids do not pass 1).
__device__ __forceinline__ Two speed_at(const ScanArgs& a, const Place& p, bool& near) {
  const float s = p.on ? speed_of(a, p.c) : 0.f;
  near = __all_sync(kFull, s < kNear);
  return two(s);
}

// Sigmoids, decays a and 1 - a^2 of a step.
template <typename RING>
__device__ __forceinline__ void step_gates(const RING& ring, const Constants& k, Two speed, bool near, Two* sr, Two* sg,
                                           Two* A, Two* Q) {
  float top = 0.f;
  if (near) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      gates_near(ring.pair(kR, p), ring.pair(kG, p), k, sr[p], sg[p], top);
      const Decay<Two> d = decay_near(speed * sr[p], k);
      A[p] = d.a;
      Q[p] = d.q;
    }
  }
  if (!__all_sync(kFull, near && top < kTop)) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      gates_any(ring.pair(kR, p, true), ring.pair(kG, p, true), sr[p], sg[p]);
      const Decay<Two> d = decay_any(speed * sr[p]);
      A[p] = d.a;
      Q[p] = d.q;
    }
  }
}

// Slots: as many as leave room for those blocks (at most 72 KB a block
// forward, 108 KB backward).
constexpr int kForwardSlots = 2;
constexpr int kBackwardSlots = 2;
template <int DT>
constexpr int kBackMapSlots = DT == TBE_F32 ? 4 : 3;
template <int DT, bool WIDE>
using ForwardRing = Ring<DT, 3, kForwardSlots, false, WIDE>;
template <int DT, bool WIDE>
using BackwardRing = Ring<DT, 4, kBackwardSlots, true, WIDE>;
template <int DT, bool WIDE>
using BackMapRing = Ring<DT, 2, kBackMapSlots<DT>, false, WIDE>;
// shared memory of a warp, with room for its outputs
template <int DT>
constexpr int kForwardBytes = ForwardRing<DT, true>::kBytes + kStep * 32 * kSize<DT>;
template <int DT>
constexpr int kBackwardBytes = BackwardRing<DT, true>::kBytes + 3 * kStep * 32 * kSize<DT>;
template <int DT>
constexpr int kMapBytes(bool back) {
  return back ? BackMapRing<DT, true>::kBytes : ForwardRing<DT, true>::kBytes;
}

// The map of a run, forward: h at its end from h at its start.  Only the
// tokens from the run's last start on count.
template <int DT, bool WIDE>
__device__ __forceinline__ Map run_map(const ScanArgs& a, const Place& p, uint8_t* mem, Two speed, bool near, int lane) {
  Map m{1.f, 0.f};
  if (p.t0 >= p.t1) return m;
  Cursor cur(a, lane);
  int64_t first, end;
  const int64_t s = cur.owner(p.t1 - 1, true, first, end);
  const bool cut = first >= p.t0 && first < p.t1;
  if (cut && a.h0 && p.on) m.B = a.h0[s * a.C + p.c];
  const int64_t from = cut ? first : p.t0;
  int left = (int)(p.t1 - from);
  ForwardRing<DT, WIDE> ring(a, mem, p.cb, lane, left);
  const Constants k;
  ring.input(kR, a.r, a.sr, from, p.cb);
  ring.input(kG, a.g, a.sg, from, p.cb);
  ring.input(kX, a.x, a.sx, from, p.cb);
#pragma unroll
  for (int i = 0; i < kForwardSlots; ++i) ring.fill();
  while (left > 0) {
    ring.ready();
#pragma unroll 1
    for (int u = 0; u < kTokens<DT> / kStep && left > 0; ++u, left -= kStep) {
      ring.step(u);
      Two sr[kPairs], sg[kPairs], A[kPairs], B[kPairs];
      step_gates(ring, k, speed, near, sr, sg, A, B);
#pragma unroll
      for (int q = 0; q < kPairs; ++q) B[q] = root(B[q]) * sg[q] * ring.pair(kX, q);
      if (left < kStep) {  // tokens outside the run change nothing
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {
          A[q] = two(2 * q < left ? lo(A[q]) : 1.f, 2 * q + 1 < left ? hi(A[q]) : 1.f);
          B[q] = two(2 * q < left ? lo(B[q]) : 0.f, 2 * q + 1 < left ? hi(B[q]) : 0.f);
        }
      }
#pragma unroll
      for (int j = 0; j < kStep; ++j) m.B = fmaf(element(A, j), m.B, element(B, j));
      const Two P = A[0] * A[1] * (A[2] * A[3]);
      m.A *= lo(P) * hi(P);
    }
    ring.done();
  }
  cp_wait<0>();
  if (cut) m.A = -1.f;
  return m;
}

// The map of a run, backward: a G at its start from a G behind its end.
// Only the tokens up to the run's first end count.
template <int DT, bool WIDE>
__device__ __forceinline__ Map run_map_back(const ScanArgs& a, const Place& p, uint8_t* mem, Two speed, bool near, int lane) {
  Map m{1.f, 0.f};
  if (p.t0 >= p.t1) return m;
  Cursor cur(a, lane);
  int64_t first, end;
  const int64_t s = cur.owner(p.t0, false, first, end);
  const bool cut = end > p.t0 && end <= p.t1;
  int left = (int)((cut ? end : p.t1) - p.t0);
  const float last = cut && a.dh_last && p.on ? a.dh_last[s * a.C + p.c] : 0.f;
  BackMapRing<DT, WIDE> ring(a, mem, p.cb, lane, left);
  const Constants k;
  ring.input(0, a.r, a.sr, p.t0, p.cb);
  ring.input(1, a.dh, a.sdh, p.t0, p.cb);
#pragma unroll
  for (int i = 0; i < kBackMapSlots<DT>; ++i) ring.fill();
  while (left > 0) {
    ring.ready();
#pragma unroll 1
    for (int u = 0; u < kTokens<DT> / kStep && left > 0; ++u, left -= kStep) {
      ring.step(u);
      Two A[kPairs], D[kPairs];
      if (near) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
          A[i] = decay_near(speed * rcp(ex2(ring.pair(0, i) * k.minus_log2e) + k.one), k).a;
      } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const Two r = ring.pair(0, i);
          A[i] = decay_any(speed * two(sigmoid(lo(r)), sigmoid(hi(r)))).a;
        }
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i) D[i] = ring.pair(1, i);
      if (left <= kStep) {  // the run's last token, and those outside it
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          A[i] = two(2 * i < left ? lo(A[i]) : 1.f, 2 * i + 1 < left ? hi(A[i]) : 1.f);
          D[i] = D[i] + two(2 * i + 1 == left ? last : 0.f, 2 * i + 2 == left ? last : 0.f);
        }
      }
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        m.A *= element(A, j);
        m.B = fmaf(m.A, element(D, j), m.B);
      }
    }
    ring.done();
  }
  cp_wait<0>();
  if (cut) m.A = -1.f;
  return m;
}

__device__ __forceinline__ float2 word_of(Map m) { return make_float2(m.A, m.B); }
__device__ __forceinline__ Map map_of(float2 w) { return Map{w.x, w.y}; }

// The maps of every run and every block (scan order: BACK counts from the
// last run down).
template <int DT, bool BACK, bool WIDE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<BACK>) maps_kernel(ScanArgs a) {
  extern __shared__ __align__(128) uint8_t mem[];
  __shared__ Map runs[kWarps][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of(a, warp, lane);
  bool near;
  const Two speed = speed_at(a, p, near);
  uint8_t* mine = mem + warp * kMapBytes<DT>(BACK);
  const Map m = BACK ? run_map_back<DT, WIDE>(a, p, mine, speed, near, lane) : run_map<DT, WIDE>(a, p, mine, speed, near, lane);
  const int64_t k = blockIdx.x / a.cblocks;
  if (BACK && k == 0 && threadIdx.x == 0) a.arrived[blockIdx.x] = 0;  // for the backward kernel, which waits for this one
  runs[warp][lane] = m;
  a.warp_map[(k * kWarps + warp) * a.Cp + p.c] = word_of(m);
  __syncthreads();
  if (warp == 0) {
    Map all = runs[BACK ? kWarps - 1 : 0][lane];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) all = join(all, runs[BACK ? kWarps - 1 - w : w][lane]);
    a.block_map[k * a.Cp + p.c] = word_of(all);
  }
}

// What reaches a warp's run: the blocks before this one, in rounds of 128
// from the nearest on (sixteen to a warp), until nothing further back
// matters; then the warps before this one.  Every thread of the block calls
// this.
template <bool BACK>
__device__ __forceinline__ float reach(const ScanArgs& a, const Place& p, int warp, int lane) {
  constexpr int kEach = 16;
  __shared__ Map part[kWarps][32];
  const int64_t k = blockIdx.x / a.cblocks;
  const int64_t before = BACK ? a.blocks - 1 - k : k;  // blocks before this one in scan order
  float2 own[kWarps - 1];
#pragma unroll
  for (int j = 0; j < kWarps - 1; ++j) {
    const int r = BACK ? kWarps - 1 - j : j;  // in scan order
    const bool mine = BACK ? r > warp : r < warp;
    own[j] = mine ? __ldcg(a.warp_map + (k * kWarps + r) * a.Cp + p.c) : make_float2(1.f, 0.f);
  }
  Map all{1.f, 0.f};
  for (int64_t done = 0; done < before && !(all.A < 0.f); done += kEach * kWarps) {
    // this warp's share, farthest first
    Map m{1.f, 0.f};
    float2 w[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int64_t away = done + kEach * warp + kEach - j;  // 1: the neighbour
      const int64_t b = BACK ? k + away : k - away;
      w[j] = away <= before ? __ldcg(a.block_map + b * a.Cp + p.c) : make_float2(1.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) m = join(m, map_of(w[j]));
    __syncthreads();
    part[warp][lane] = m;
    __syncthreads();
    Map round = part[kWarps - 1][lane];
#pragma unroll
    for (int j = kWarps - 2; j >= 0; --j) round = join(round, part[j][lane]);
    all = join(round, all);
  }
  float in = apply(all, 0.f);
#pragma unroll
  for (int j = 0; j < kWarps - 1; ++j) in = apply(map_of(own[j]), in);
  return in;
}

// The same where one block holds all tokens: the warps' maps are made here.
template <bool BACK>
__device__ __forceinline__ float reach_alone(Map m, int warp, int lane) {
  __shared__ Map runs[kWarps][32];
  runs[warp][lane] = m;
  __syncthreads();
  float in = 0.f;
  for (int j = BACK ? kWarps - 1 : 0; j != warp; j += BACK ? -1 : 1) in = apply(runs[j][lane], in);
  return in;
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
template <int DT, bool ALONE, bool WIDE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<false>) forward_kernel(ScanArgs a) {
  extern __shared__ __align__(128) uint8_t mem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of(a, warp, lane);
  bool near;
  const Two speed = speed_at(a, p, near);
  uint8_t* mine = mem + warp * kForwardBytes<DT>;
  float h = 0.f;
  if (ALONE) h = reach_alone<false>(run_map<DT, WIDE>(a, p, mine, speed, near, lane), warp, lane);
  int left = (int)(p.t1 - p.t0);
  ForwardRing<DT, WIDE> ring(a, mine, p.cb, lane, left);
  ring.input(kR, a.r, a.sr, p.t0, p.cb);
  ring.input(kG, a.g, a.sg, p.t0, p.cb);
  ring.input(kX, a.x, a.sx, p.t0, p.cb);
#pragma unroll
  for (int i = 0; i < kForwardSlots; ++i) ring.fill();
  empty_sequences(a, a.h0, a.h_last);
  if (!ALONE) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    h = reach<false>(a, p, warp, lane);
  }
  Cursor cur(a, lane);
  Events ev;
  const Constants k;
  Out<DT, false, WIDE> to(a.h, a.sh, p.t0, p.cb, a.C, mine + ForwardRing<DT, WIDE>::kBytes, lane);
  float* state = a.states ? a.states + p.t0 / kStep * a.C + p.c : nullptr;
  int64_t t = p.t0;
  while (left > 0) {
    ring.ready();
#pragma unroll 1
    for (int u = 0; u < kTokens<DT> / kStep && left > 0; ++u, left -= kStep, t += kStep) {
      const int n = left < kStep ? left : kStep;
      ev.find(cur, t, n, false, lane);
      ring.step(u);
      Two sr[kPairs], sg[kPairs], A[kPairs], B[kPairs];
      step_gates(ring, k, speed, near, sr, sg, A, B);
#pragma unroll
      for (int q = 0; q < kPairs; ++q) B[q] = root(B[q]) * sg[q] * ring.pair(kX, q);
      if (state) {
        if (p.on) *state = h;
        state += a.C;
      }
      float out[kStep];
      if ((ev.starts | ev.ends) == 0) {
#pragma unroll
        for (int j = 0; j < kStep; ++j) out[j] = h = fmaf(element(A, j), h, element(B, j));
      } else {
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
          if (ev.starts >> j & 1) {
            const int64_t s = ev.sequence(j);
            h = a.h0 && p.on ? a.h0[s * a.C + p.c] : 0.f;
          }
          out[j] = h = fmaf(element(A, j), h, element(B, j));
          if (ev.ends >> j & 1) {
            const int64_t s = ev.sequence(j);
            if (p.on) a.h_last[s * a.C + p.c] = h;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < kPairs; ++q) to.put(q, out[2 * q], out[2 * q + 1], n);
      __syncwarp();
      to.flush(n);
      __syncwarp();
    }
    ring.done();
  }
  cp_wait<0>();
}

template <int DT, bool ALONE, bool WIDE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<true>) backward_kernel(ScanArgs a) {
  extern __shared__ __align__(128) uint8_t mem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of(a, warp, lane);
  bool near;
  const Two speed = speed_at(a, p, near);
  uint8_t* mine = mem + warp * kBackwardBytes<DT>;
  float c = 0.f;
  Two sum = two(0.f);
  if (ALONE) c = reach_alone<true>(run_map_back<DT, WIDE>(a, p, mine, speed, near, lane), warp, lane);
  // slots from the run's last one down
  const int tokens = (int)(p.t1 - p.t0);
  const int slots = (tokens + kTokens<DT> - 1) / kTokens<DT>;
  const int64_t last = p.t0 + (int64_t)(slots > 0 ? slots - 1 : 0) * kTokens<DT>;
  BackwardRing<DT, WIDE> ring(a, mine, p.cb, lane, tokens);
  ring.input(kR, a.r, a.sr, last, p.cb);
  ring.input(kG, a.g, a.sg, last, p.cb);
  ring.input(kX, a.x, a.sx, last, p.cb);
  ring.input(kD, a.dh, a.sdh, last, p.cb);
  ring.state = a.states + last / kStep * a.C + p.c;
#pragma unroll
  for (int i = 0; i < kBackwardSlots; ++i) ring.fill();
  empty_sequences(a, a.dh_last, a.dh0);
  if (!ALONE) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    c = reach<true>(a, p, warp, lane);
  }
  Cursor cur(a, lane);
  Events ev;
  uint8_t* room = mine + BackwardRing<DT, WIDE>::kBytes;
  constexpr int kBox = kStep * 32 * kSize<DT>;
  const int64_t top = tokens > 0 ? p.t0 + (tokens - 1) / kStep * kStep : p.t0;  // the run's last step
  Out<DT, true, WIDE> px(a.dx, a.sdx, top, p.cb, a.C, room, lane);
  Out<DT, true, WIDE> pr(a.dr, a.sdr, top, p.cb, a.C, room + kBox, lane);
  Out<DT, true, WIDE> pg(a.dg, a.sdg, top, p.cb, a.C, room + 2 * kBox, lane);
  const Constants k;
  int64_t t = top;
  int n = tokens - (int)(top - p.t0);  // of the last step; the others are whole
  for (int left = slots; left > 0; --left) {
    ring.ready();
#pragma unroll 1
    for (int u = (int)(t - p.t0) / kStep % (kTokens<DT> / kStep); u >= 0; --u, t -= kStep, n = kStep) {
      ev.find(cur, t, n, true, lane);
      ring.step(u);
      Two sr[kPairs], sg[kPairs], A[kPairs], inv[kPairs], beta[kPairs], found[kPairs], G[kPairs];
      step_gates(ring, k, speed, near, sr, sg, A, beta);
      const bool plain = (ev.starts | ev.ends) == 0 && n == kStep;
      // the states that the step's tokens find
      float h = ring.first_state(u);
#pragma unroll
      for (int q = 0; q < kPairs; ++q) {
        // where 1 - a^2 is 0 the token takes nothing in, and its gate's slope
        // u d beta / d u = u a^2 / beta goes to 0 with u
        const Two safe = two(fmaxf(lo(beta[q]), 1e-37f), fmaxf(hi(beta[q]), 1e-37f));
        inv[q] = inv_root(safe);
        beta[q] = beta[q] * inv[q];
        const Two b = beta[q] * sg[q] * ring.pair(kX, q);
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!plain && (ev.starts >> (2 * q + e) & 1)) {
            const int64_t s = ev.sequence(2 * q + e);
            h = a.h0 && p.on ? a.h0[s * a.C + p.c] : 0.f;
          }
          f[e] = h;
          h = fmaf(e ? hi(A[q]) : lo(A[q]), h, e ? hi(b) : lo(b));
        }
        found[q] = two(f[0], f[1]);
        G[q] = ring.pair(kD, q);
      }
      if (plain) {
#pragma unroll
        for (int q = kPairs - 1; q >= 0; --q) {
          const float g1 = hi(G[q]) + c, g0 = fmaf(hi(A[q]), g1, lo(G[q]));
          c = lo(A[q]) * g0;
          G[q] = two(g0, g1);
        }
      } else {
#pragma unroll
        for (int j = kStep - 1; j >= 0; --j) {
          float g = element(G, j);
          if (j < n) {
            if (ev.ends >> j & 1) {
              const int64_t s = ev.sequence(j);
              if (a.dh_last && p.on) g += a.dh_last[s * a.C + p.c];
            } else {
              g += c;
            }
            c = element(A, j) * g;
            if (ev.starts >> j & 1) {
              const int64_t s = ev.sequence(j);
              if (a.dh0 && p.on) a.dh0[s * a.C + p.c] = c;
            }
          }
          G[j >> 1] = j & 1 ? two(lo(G[j >> 1]), g) : two(g, hi(G[j >> 1]));
        }
      }
#pragma unroll
      for (int q = 0; q < kPairs; ++q) {
        const Two x = ring.pair(kX, q, true);
        const Two w = G[q] * (speed * sr[q]) * A[q] * fma2(A[q] * inv[q], sg[q] * x, negative(found[q]));
        const Two dx = G[q] * beta[q] * sg[q], dg = dx * x * (k.one + negative(sg[q])), dr = w * (k.one + negative(sr[q]));
        px.put(q, lo(dx), hi(dx), n);
        pr.put(q, lo(dr), hi(dr), n);
        pg.put(q, lo(dg), hi(dg), n);
        sum = sum + w;  // 0 behind the batch, where dh reads as 0
      }
      __syncwarp();
      px.flush(n);
      pr.flush(n);
      pg.flush(n);
      __syncwarp();
    }
    ring.done();
  }
  cp_wait<0>();

  // The decay's gradient: the warps' shares, then the blocks', always added in
  // the same order, the blocks' by the last of them to finish.
  __shared__ float shares[kWarps][32];
  __shared__ bool s_last;
  const int64_t block = blockIdx.x / a.cblocks;
  shares[warp][lane] = lo(sum) + hi(sum);
  __syncthreads();
  float total = 0.f;
  if (warp == 0) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += shares[w][lane];
  }
  if (!ALONE) {
    if (warp == 0) {
      if (p.on) a.partial[block * a.C + p.c] = total;
      __threadfence();
      __syncwarp();
      if (lane == 0) s_last = atomicAdd(a.arrived + blockIdx.x % a.cblocks, 1u) == (uint32_t)a.blocks - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    total = 0.f;
    if (p.on) {
#pragma unroll 8
      for (int64_t k = warp; k < a.blocks; k += kWarps) total += __ldcg(a.partial + k * a.C + p.c);
    }
    shares[warp][lane] = total;
    __syncthreads();
    total = 0.f;
    if (warp == 0) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) total += shares[w][lane];
    }
  }
  if (warp == 0 && p.on) {
    const float d = a.decay[p.c], sp = softplus(d);
    // ddecay = sigmoid(decay) / softplus(decay) * total; far below zero both
    // are exp(decay) and the ratio is 1
    a.ddecay[p.c] = d < -16.f ? total : total * (1.f / (1.f + expf(-d))) / sp;
  }
}

// One token of each of S sequences: the state moves on in place.
template <int DT>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (i >= (int64_t)a.S * a.C) return;
  const int64_t s = i / a.C, c = i - s * a.C;
  const float x = number<DT>(load_bits<DT>(at<DT>(a.x, s * a.sx + c)));
  const float r = number<DT>(load_bits<DT>(at<DT>(a.r, s * a.sr + c)));
  const float g = number<DT>(load_bits<DT>(at<DT>(a.g, s * a.sg + c)));
  const Decay<float> d = decay_of(speed_of(a, c) * sigmoid(r));
  const float h = fmaf(d.a, a.h_last[i], root(d.q) * sigmoid(g) * x);
  a.h_last[i] = h;
  store_pair<DT>(at<DT>(a.h, s * a.sh + c), 0, h, h, true, false);
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int32_t channel_blocks(int32_t C) { return (C + 31) / 32; }

// Tokens per warp: as many as give every warp that fits on the GPU one run,
// in whole steps.  Up to kAlone tokens one block takes the whole batch (both
// passes in one kernel, no second launch).
constexpr int64_t kAlone = 256;
struct Split {
  int32_t run, blocks;
};
Split split_of(int64_t N, int32_t cblocks, bool back) {
  const int64_t warps = (int64_t)sm_count() * (back ? kBlocksPerSm<true> : kBlocksPerSm<false>) * kWarps / cblocks;
  const int64_t parts = N <= kAlone || warps < kWarps ? kWarps : warps / kWarps * kWarps;
  constexpr int kUnit = 2 * kStep;  // whole slots of every type
  int64_t run = ((N + parts - 1) / parts + kUnit - 1) / kUnit * kUnit;
  if (run < kUnit) run = kUnit;
  Split s;
  s.run = (int32_t)run;
  s.blocks = (int32_t)((N + run * kWarps - 1) / (run * kWarps));
  if (s.blocks < 1) s.blocks = 1;
  return s;
}

// The workspace: maps of blocks and runs, then the backward's partial sums
// and counters.  A batch of one block needs none.
struct Workspace {
  size_t block, warp, partial, arrived, bytes;
};
Workspace layout(int64_t N, int32_t C, bool backward) {
  const Split sp = split_of(N, channel_blocks(C), backward);
  const size_t Cp = (size_t)channel_blocks(C) * 32;
  Workspace w;
  size_t at = 0;
  w.block = w.warp = w.arrived = 0;
  if (sp.blocks > 1) {
    at += round256((size_t)sp.blocks * Cp * sizeof(float2));
    w.warp = at;
    at += round256((size_t)sp.blocks * kWarps * Cp * sizeof(float2));
  }
  w.partial = at;
  if (backward && sp.blocks > 1) {
    at += round256((size_t)sp.blocks * C * 4);
    w.arrived = at;
    at += round256((size_t)channel_blocks(C) * 4);
  }
  w.bytes = at;
  return w;
}

bool aligned_to(const void* p, int64_t stride_bytes, int n) { return ((uintptr_t)p & (n - 1)) == 0 && stride_bytes % n == 0; }

// How rows may be read: bytes per asynchronous copy of an input.
void choose_access(ScanArgs& a, int32_t dtype) {
  const int size = dtype == TBE_F32 ? 4 : 2;
  auto all = [&](int n) {
    return aligned_to(a.x, a.sx * size, n) && aligned_to(a.r, a.sr * size, n) && aligned_to(a.g, a.sg * size, n) &&
           (!a.dh || aligned_to(a.dh, a.sdh * size, n));
  };
  auto out = [&](const void* p, int64_t stride) { return !p || aligned_to(p, stride * size, 16); };
  a.copy = all(16) && a.C * size % 16 == 0 && out(a.h, a.sh) && out(a.dx, a.sdx) && out(a.dr, a.sdr) && out(a.dg, a.sdg)
               ? 16
               : all(4) ? 4 : 0;
}

// Launches KERNEL; `after`: it may start while the kernel before it ends.
template <auto KERNEL>
int start(unsigned grid, size_t smem, bool after, cudaStream_t s, const ScanArgs& a) {
  if (smem > 40 * 1024) {  // beyond the default once the static slots are counted
    static bool allowed[64] = {};  // once per device
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !allowed[dev]) {
      if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return TBE_ERR_CUDA;
      if (dev >= 0 && dev < 64) allowed[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, KERNEL, a) == cudaSuccess ? check_launch() : TBE_ERR_CUDA;
}

template <int DT, bool BACK, bool WIDE>
int launch_passes(const ScanArgs& a, cudaStream_t s) {
  constexpr size_t bytes = kWarps * (size_t)(BACK ? kBackwardBytes<DT> : kForwardBytes<DT>);
  constexpr size_t map_bytes = kWarps * (size_t)kMapBytes<DT>(BACK);
  static_assert(bytes >= map_bytes, "the maps of a lone block use the same memory");
  const unsigned grid = (unsigned)a.blocks * (unsigned)a.cblocks;
  if (a.blocks == 1) {
    if constexpr (BACK) return start<backward_kernel<DT, true, WIDE>>(grid, bytes, false, s, a);
    else return start<forward_kernel<DT, true, WIDE>>(grid, bytes, false, s, a);
  }
  const int st = start<maps_kernel<DT, BACK, WIDE>>(grid, map_bytes, false, s, a);
  if (st != TBE_OK) return st;
  trace_mark(s, BACK ? "gated_scan_maps_back" : "gated_scan_maps");
  if constexpr (BACK) return start<backward_kernel<DT, false, WIDE>>(grid, bytes, true, s, a);
  else return start<forward_kernel<DT, false, WIDE>>(grid, bytes, true, s, a);
}
template <int DT, bool BACK>
int launch_scan(const ScanArgs& a, cudaStream_t s) {
  return a.copy == 16 ? launch_passes<DT, BACK, true>(a, s) : launch_passes<DT, BACK, false>(a, s);
}

template <int DT>
int launch_step(const ScanArgs& a, cudaStream_t s) {
  scan_step_kernel<DT><<<(unsigned)(((int64_t)a.S * a.C + 127) / 128), 128, 0, s>>>(a);
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
  a.cblocks = channel_blocks(in->channels);
  a.Cp = (int64_t)a.cblocks * 32;
  return a;
}

int check_jagged(const tbe_scan_inputs* in) {
  const int st = check(in);
  if (st != TBE_OK) return st;
  if (!in->offsets || (in->tokens > 0 && in->sequences == 0)) return TBE_ERR_INVALID_ARG;
  return TBE_OK;
}

int use_workspace(ScanArgs& a, bool backward, void* workspace, size_t bytes) {
  const Split sp = split_of(a.N, a.cblocks, backward);
  a.run = sp.run;
  a.blocks = sp.blocks;
  const Workspace w = layout(a.N, a.C, backward);
  if (bytes < w.bytes) return TBE_ERR_WORKSPACE;
  if (w.bytes == 0) return TBE_OK;
  if (!workspace) return TBE_ERR_INVALID_ARG;
  if ((uintptr_t)workspace & 255) return TBE_ERR_UNSUPPORTED;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  a.block_map = reinterpret_cast<float2*>(p + w.block);
  a.warp_map = reinterpret_cast<float2*>(p + w.warp);
  a.partial = reinterpret_cast<float*>(p + w.partial);
  a.arrived = reinterpret_cast<uint32_t*>(p + w.arrived);
  return TBE_OK;
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" {

int64_t tbe_gated_scan_states(int64_t tokens) { return tokens < 1 ? 1 : (tokens + kStep - 1) / kStep; }

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
  st = use_workspace(a, false, workspace, workspace_bytes);
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
  a.ddecay = out->ddecay;
  a.status = dev_status;
  trace_begin(s);
  st = use_workspace(a, true, workspace, workspace_bytes);
  if (st != TBE_OK) return st;
  st = dispatch(a, in->dtype, kBackward, s);
  trace_mark(s, "gated_scan_backward");
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
