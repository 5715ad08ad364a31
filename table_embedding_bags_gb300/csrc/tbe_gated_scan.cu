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
// A warp takes a run of tokens and 32 or 64 channels, a block's warps
// neighbouring runs.  h over a run is the linear map h_out = A h_in + B, so two
// passes do it:
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
//
// What bounds it: the issue of instructions and memory, close together.  A
// training pass of 65,537 tokens x 1,024 channels bf16 (2 sequences, 408 us):
//   maps      24 instructions per element, 64 % of issue slots, 6.0 TB/s, 67 us
//   forward   28, 60 %, 5.9 TB/s, 89 us
//   maps back 21, 62 %, 4.3 TB/s, 61 us
//   backward  69, 67 %, 5.0 TB/s, 187 us
// Two passes read the inputs twice (1.6 times the bytes that one pass would),
// but one pass that waits for its neighbours' words ran them one after another.
// Short sequences in short batches (2,048 of them, 40,960 tokens x 128 bf16,
// 57 us) pay for the runs' starts: 9 steps to a run, with addresses, offsets
// and joined maps before them, in each of four launches.
#include "tbe_internal.cuh"
#include "tbe_two.cuh"

#include <cmath>

namespace tbe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kStep = TBE_SCAN_STEP;  // tokens per step (and between saved states)
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// Blocks that stay resident on an SM.  Three, with the forward at 80
// registers, spill in its loop: prefill of 100,003 x 512 f16 132.8 us against
// 124.5 us, training pass of 65,537 x 1,024 bf16 417.7 us against 407.9 us.
constexpr int kBlocksPerSm = 2;
// Channels of a lane: VEC.  Arithmetic goes by pairs: a token's two channels (2),
// or two neighbouring tokens of the one channel (1).  The forward takes two
// half-precision channels, which halves what a step costs beside its
// elements; the backward would need more registers than there are.
template <int DT, bool BACK>
constexpr int kVec = DT == TBE_F32 || BACK ? 1 : 2;
template <int VEC>
constexpr int kPairs = kStep * VEC / 2;  // of a step
template <int VEC>
constexpr int kChannels = 32 * VEC;  // of a warp
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
  int32_t run;      // tokens per warp, whole steps
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
// by gates_any.  NaN in one input makes both sigmoids NaN.  The forward may
// leave it so, as h is NaN from that token on either way; the backward (BACK)
// may not, as the gate has no part in a, which carries G to earlier tokens: a
// lane that meets NaN does the step again.
constexpr float kTop = 1e36f;
template <bool BACK>
__device__ __forceinline__ void gates_near(Two r, Two g, const Constants& k, Two& sr, Two& sg, float& top) {
  const Two pr = ex2(r * k.minus_log2e) + k.one, pg = ex2(g * k.minus_log2e) + k.one;
  const Two product = pr * pg, inv = rcp(product);
  sr = inv * pg;
  sg = inv * pr;
  top = BACK ? max_nan(max_nan(top, lo(product)), hi(product)) : fmaxf(fmaxf(top, lo(product)), hi(product));
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
template <int DT>
__device__ __forceinline__ float number(uint32_t b) {
  if (DT == TBE_F32) return __uint_as_float(b);
  if (DT == TBE_BF16) return __uint_as_float(b << 16);
  return __half2float(__ushort_as_half((unsigned short)b));
}
// Both halves of a word.
template <int DT>
__device__ __forceinline__ Two halves(uint32_t w) {
  if (DT == TBE_BF16) return two(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return two(f.x, f.y);
}
template <int DT>
__device__ __forceinline__ uint32_t to_halves(Two v) {
  if (DT == TBE_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo(v), hi(v));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo(v), hi(v));
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int DT>
__device__ __forceinline__ float load_element(const uint8_t* p) {
  if (DT == TBE_F32) return *reinterpret_cast<const float*>(p);
  return number<DT>(*reinterpret_cast<const uint16_t*>(p));
}
// Token j, channel v of an array of a step's pairs.
template <int VEC>
__device__ __forceinline__ float element(const Two* t, int j, int v) {
  if (VEC == 1) return j & 1 ? hi(t[j >> 1]) : lo(t[j >> 1]);
  return v ? hi(t[j]) : lo(t[j]);
}
// The token and channel of component e of pair q.
template <int VEC>
__device__ __forceinline__ constexpr int token_of(int q, int e) {
  return VEC == 1 ? 2 * q + e : q;
}
template <int VEC>
__device__ __forceinline__ constexpr int channel_of(int e) {
  return VEC == 1 ? 0 : e;
}
// The pair with the components of tokens from `n` on replaced.
template <int VEC>
__device__ __forceinline__ Two upto(Two t, int q, int n, float other) {
  return two(token_of<VEC>(q, 0) < n ? lo(t) : other, token_of<VEC>(q, 1) < n ? hi(t) : other);
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
// one per lane, and is moved where it does not reach: to where the token would
// lie if all sequences were equally long, give or take 128 sequences (two
// dependent loads), else by a search.  (A training pass over 2,048 sequences
// and 40,960 tokens: 60.0 us with the search alone, 56.8 us so.)
struct Cursor {
  const ScanArgs& a;
  int64_t base, off;
  int lane;
  __device__ __forceinline__ Cursor(const ScanArgs& args, int lane_) : a(args), base(0), off(INT64_MAX), lane(lane_) {}
  __device__ __forceinline__ int64_t at_index(int64_t i) const { return i <= a.S ? a.offsets.ldg(i) : INT64_MAX; }
  __device__ __forceinline__ int load(int64_t from, int64_t t) {
    base = from < 0 ? 0 : from;
    off = at_index(base + lane);
    return __popc(__ballot_sync(kFull, off <= t));
  }
  // The sequence that token t belongs to, and its first token and end.
  __device__ __forceinline__ int64_t owner(int64_t t, bool down, int64_t& first, int64_t& end) {
    int below = __popc(__ballot_sync(kFull, off <= t));
    if (below == 0 || below == 32) {
      int64_t from = 0;
      if (a.S >= 32) {
        from = (int64_t)((float)t / (float)a.N * (float)a.S) - 128;
        if (from > a.S - 256) from = a.S - 256;
        if (from < 0) from = 0;
        const int pivots = __popc(__ballot_sync(kFull, at_index(from + 8 * lane) <= t));
        from += 8 * (pivots > 0 ? pivots - 1 : 0) - (down ? 16 : 0);
      }
      below = load(from, t);
      if (below == 0 || below == 32) {
        const int64_t s = first_at(a.offsets, a.S, t + 1, lane) - 1;
        below = load(down ? s - 30 : s, t);
      }
    }
    // broken offsets must not lead outside the arrays
    int l = below < 1 ? 0 : (below > 31 ? 30 : below - 1);
    if (base > a.S - 1) base = a.S - 1, l = 0;
    if (base + l > a.S - 1) l = (int)(a.S - 1 - base);
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

// A warp's ring.  A slot holds a step of each input, then (DOWN) the states
// that the step starts from.  Slots are filled upwards, or downwards, from
// where the ring was set until the run's tokens are all asked for.  WIDE: rows
// start on 16 bytes and channels come in whole 16-byte pieces; otherwise a copy
// is of 4 bytes, or (half precision at odd places) an element at a time.
template <int DT, int VEC, int INPUTS, int SLOTS, bool DOWN, bool WIDE>
struct Ring {
  static constexpr int kRow = 32 * VEC * kSize<DT>, kBox = kStep * kRow;
  static constexpr int kSlot = INPUTS * kBox + (DOWN ? kChannels<VEC> * 4 : 0);
  static constexpr int kBytes = SLOTS * kSlot;
  static constexpr int kLanes = kRow / 16, kRows = 32 / kLanes;  // 16-byte pieces of a row, rows of a copy
  const uint8_t* mem;
  const uint8_t* src[INPUTS];  // this lane's first piece of the next step
  int64_t row[INPUTS];         // bytes between tokens
  const float* state;          // of the warp's first channel
  const ScanArgs& a;
  uint32_t base;   // of slot 0, in shared memory
  int left_bytes;  // of a row inside the array
  int piece;       // bytes of a row that the lane copies at once
  int lane;
  int read, write;  // bytes from slot 0: the oldest slot, the next to be filled
  int left;         // tokens of the run that are not asked for yet

  // `tokens`: of the run; downwards the first slot takes what does not fill one
  __device__ __forceinline__ Ring(const ScanArgs& args, uint8_t* m, int64_t cb, int l, int tokens)
      : mem(m), state(nullptr), a(args), base(smem_u32(m)), lane(l), read(0), write(0), left(tokens) {
    left_bytes = (int)((a.C - cb) * kSize<DT> < kRow ? (a.C - cb) * kSize<DT> : kRow);
    const int b = left_bytes - (WIDE ? col() : lane % (kRow / 4) * 4), most = WIDE ? 16 : 4;
    piece = b < 0 ? 0 : (b < most ? b : most);
  }
  // the lane's place in a row, and the first row it copies (WIDE)
  __device__ __forceinline__ int col() const { return WIDE ? lane % kLanes * 16 : 0; }
  __device__ __forceinline__ int first_row() const { return WIDE ? lane / kLanes : 0; }
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
  // The next slot.  What lies outside the run (in the batch's last one), or
  // outside the channels, reads as 0: a copy of 0 bytes reads nothing.
  __device__ __forceinline__ void fill() {
    int count = left < kStep ? left : kStep;
    if (DOWN && left > kStep && left % kStep) count = left % kStep;
    left -= count;
    const uint32_t to = base + write;
    if (WIDE) {
#pragma unroll
      for (int k = 0; k < kStep; k += kRows) {
        const int n = k + first_row() < count ? piece : 0;
#pragma unroll
        for (int i = 0; i < INPUTS; ++i) copy16(to + i * kBox + k * kRow + lane * 16, src[i] + k * row[i], n);
      }
    } else if (a.copy == 4) {
      constexpr int kPieces = kRow / 4;  // of a row
#pragma unroll
      for (int k = 0; k < kStep; k += 32 / kPieces) {
        const int r = k + lane / kPieces, n = r < count ? piece : 0;
#pragma unroll
        for (int i = 0; i < INPUTS; ++i)
          copy4(to + i * kBox + k * kRow + lane * 4, src[i] + r * row[i] + lane % kPieces * 4, n);
      }
    } else {
#pragma unroll 4
      for (int k = 0; k < kStep; ++k)
#pragma unroll
        for (int i = 0; i < INPUTS; ++i)
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            const int c = (v * 32 + lane) * 2;
            const uint16_t w = k < count && c < left_bytes ? *reinterpret_cast<const uint16_t*>(src[i] + k * row[i] + c) : 0;
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + i * kBox + k * kRow + c), "h"(w) : "memory");
          }
    }
#pragma unroll
    for (int i = 0; i < INPUTS; ++i) src[i] += (DOWN ? -kStep : kStep) * row[i];
    if (DOWN) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const bool ok = count > 0 && (v * 32 + lane) * kSize<DT> < left_bytes;
        copy4(to + INPUTS * kBox + (v * 32 + lane) * 4, state + v * 32 + lane, ok ? 4 : 0);
      }
      state -= a.C;
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
  // a token's channels of the lane
  __device__ __forceinline__ uint32_t word(int i, int j) const {
    const uint8_t* p = mem + read + lane * (VEC * kSize<DT>) + (i * kBox + j * kRow);
    return VEC * kSize<DT> == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
  }
  // `again`: read anew where it was read before, so that nothing made from
  // it the first time is kept in registers for the second
  __device__ __forceinline__ Two pair(int i, int q, bool again = false) const {
    if (VEC == 1) {
      uint32_t w0 = word(i, 2 * q), w1 = word(i, 2 * q + 1);
      if (again) asm volatile("" : "+r"(w0), "+r"(w1));
      return two(number<DT>(w0), number<DT>(w1));
    }
    uint32_t w = word(i, q);
    if (again) asm volatile("" : "+r"(w));
    return halves<DT>(w);
  }
  __device__ __forceinline__ float first_state(int v) const {
    return *reinterpret_cast<const float*>(mem + read + INPUTS * kBox + (lane * VEC + v) * 4);
  }
};

// One output of a warp, a step at a time.  WIDE: gathered in shared memory and
// written 16 bytes to a lane; otherwise each element on its own.
template <int DT, int VEC, bool DOWN, bool WIDE>
struct Out {
  static constexpr int kRow = 32 * VEC * kSize<DT>, kLanes = kRow / 16, kRows = 32 / kLanes;
  uint8_t* to;    // this lane's first piece of the step
  uint8_t* room;  // a step's rows in shared memory (WIDE)
  int64_t row;
  int lane;
  int on;  // channels (WIDE: 16-byte pieces) of the lane inside the array
  __device__ __forceinline__ Out(void* p, int64_t stride, int64_t t, int64_t cb, int32_t C, uint8_t* m, int l)
      : room(m), row(stride * kSize<DT>), lane(l) {
    const int64_t left = WIDE ? (C - cb) * kSize<DT> - l % kLanes * 16 : C - cb - l * VEC;
    on = left <= 0 ? 0 : (WIDE || left < VEC ? 1 : VEC);
    to = at<DT>(p, t * stride + cb) + (WIDE ? l % kLanes * 16 + l / kLanes * row : l * VEC * kSize<DT>);
  }
  __device__ __forceinline__ void element_out(uint8_t* q, float f) {
    if (DT == TBE_F32) *reinterpret_cast<float*>(q) = f;
    else if (DT == TBE_F16) *reinterpret_cast<__half*>(q) = __float2half_rn(f);
    else *reinterpret_cast<__nv_bfloat16*>(q) = __float2bfloat16_rn(f);
  }
  // pair q of the step (`n` tokens of it lie inside the batch)
  __device__ __forceinline__ void put(int q, Two v, int n) {
    if (WIDE) {
      uint8_t* r = room + lane * (VEC * kSize<DT>) + token_of<VEC>(q, 0) * kRow;
      if (DT == TBE_F32) {
        *reinterpret_cast<float*>(r) = lo(v);
        *reinterpret_cast<float*>(r + kRow) = hi(v);
      } else {
        const uint32_t w = to_halves<DT>(v);
        if (VEC == 2) {
          *reinterpret_cast<uint32_t*>(r) = w;
        } else {
          *reinterpret_cast<uint16_t*>(r) = (uint16_t)w;
          *reinterpret_cast<uint16_t*>(r + kRow) = (uint16_t)(w >> 16);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (token_of<VEC>(q, e) < n && channel_of<VEC>(e) < on)
          element_out(to + token_of<VEC>(q, e) * row + channel_of<VEC>(e) * kSize<DT>, e ? hi(v) : lo(v));
    }
  }
  // the step is complete (the caller puts a __syncwarp before and after)
  __device__ __forceinline__ void flush(int n) {
    if (WIDE) {
#pragma unroll
      for (int k = 0; k < kStep; k += kRows) {
        const uint4 a = *reinterpret_cast<const uint4*>(room + k * kRow + lane * 16);
        if (on && (n == kStep || k + lane / kLanes < n)) *reinterpret_cast<uint4*>(to + k * row) = a;
      }
    }
    to += (DOWN ? -kStep : kStep) * row;
  }
};
constexpr int kR = 0, kG = 1, kX = 2, kD = 3;  // inputs of the rings that hold them all

// A warp's place: its run of tokens and its lanes' channels.
struct Place {
  int64_t t0, t1, c, cb;
  int on;  // channels of the lane inside the array
};
template <int VEC>
__device__ __forceinline__ Place place_of(const ScanArgs& a, int warp, int lane) {
  Place p;
  const int64_t k = blockIdx.x / a.cblocks;
  p.cb = (int64_t)(blockIdx.x % a.cblocks) * kChannels<VEC>;
  p.c = p.cb + lane * VEC;
  p.t0 = (k * kWarps + warp) * a.run;
  p.t1 = p.t0 + a.run < a.N ? p.t0 + a.run : a.N;
  if (p.t0 > p.t1) p.t0 = p.t1;
  p.on = p.c >= a.C ? 0 : (p.c + VEC <= a.C ? VEC : 1);
  return p;
}

// The lane's decay rates; `near`: whether the whole warp's stay where the
// series holds (at most kNear, as sigmoids do not pass 1).  A single channel
// that forgets faster sends its warp down the other branch, which takes each
// sigmoid and decay by itself.  With one such channel in 64, or all of them:
// training pass of 65,537 x 1,024 bf16 438 us, 410 us without; of 40,960 x 128
// bf16 in 2,048 sequences 59.5 and 55.6 us; prefill of 100,003 x 512 f16 140 and
// 125 us.
template <int VEC>
__device__ __forceinline__ Two speed_at(const ScanArgs& a, const Place& p, bool& near) {
  const float s0 = p.on > 0 ? speed_of(a, p.c) : 0.f;
  const float s1 = VEC == 1 ? s0 : (p.on > 1 ? speed_of(a, p.c + 1) : 0.f);
  near = __all_sync(kFull, s0 < kNear && s1 < kNear);
  return two(s0, s1);
}

// Sigmoids, decays a and 1 - a^2 of a step.
template <int VEC, typename RING>
__device__ __forceinline__ void step_gates(const RING& ring, const Constants& k, Two speed, bool near, Two* sr, Two* sg,
                                           Two* A, Two* Q) {
  float top = 0.f;
  if (near) {
#pragma unroll
    for (int p = 0; p < kPairs<VEC>; ++p) {
      gates_near<true>(ring.pair(kR, p), ring.pair(kG, p), k, sr[p], sg[p], top);
      const Decay<Two> d = decay_near(speed * sr[p], k);
      A[p] = d.a;
      Q[p] = d.q;
    }
  }
  // (the vote keeps the usual step free of a divergent branch: training pass
  // of 65,537 x 1,024 bf16 408.4 us with it, 410.6 us without)
  const bool again = !(near && top < kTop);
  if (__any_sync(kFull, again) && again) {
#pragma unroll
    for (int p = 0; p < kPairs<VEC>; ++p) {
      gates_any(ring.pair(kR, p, true), ring.pair(kG, p, true), sr[p], sg[p]);
      const Decay<Two> d = decay_any(speed * sr[p]);
      A[p] = d.a;
      Q[p] = d.q;
    }
  }
}
// Decays a and inputs b of a step.
template <int VEC, typename RING>
__device__ __forceinline__ void step_inputs(const RING& ring, const Constants& k, Two speed, bool near, Two* A, Two* B) {
  float top = 0.f;
  if (near) {
#pragma unroll
    for (int p = 0; p < kPairs<VEC>; ++p) {
      Two sr, sg;
      gates_near<false>(ring.pair(kR, p), ring.pair(kG, p), k, sr, sg, top);
      const Decay<Two> d = decay_near(speed * sr, k);
      A[p] = d.a;
      B[p] = root(d.q) * sg * ring.pair(kX, p);
    }
  }
  if (!__all_sync(kFull, near && top < kTop)) {
#pragma unroll
    for (int p = 0; p < kPairs<VEC>; ++p) {
      Two sr, sg;
      gates_any(ring.pair(kR, p, true), ring.pair(kG, p, true), sr, sg);
      const Decay<Two> d = decay_any(speed * sr);
      A[p] = d.a;
      B[p] = root(d.q) * sg * ring.pair(kX, p, true);
    }
  }
}
// One pair's step of the recurrence; returns the states.
template <int VEC>
__device__ __forceinline__ Two advance(Two A, Two B, float* h) {
  if (VEC == 1) {
    const float h0 = fmaf(lo(A), h[0], lo(B));
    h[0] = fmaf(hi(A), h0, hi(B));
    return two(h0, h[0]);
  }
  const Two t = fma2(A, two(h[0], h[VEC - 1]), B);
  h[0] = lo(t);
  h[VEC - 1] = hi(t);
  return t;
}

// Slots: what fits two blocks on an SM (forward with 3 or 4 of them, prefill
// of 100,003 x 512 f16: 124.5 and 125.8 us).
constexpr int kForwardSlots = 3;
template <int DT>
constexpr int kBackwardSlots = DT == TBE_F32 ? 2 : 4;
template <int DT>
constexpr int kBackMapSlots = DT == TBE_F32 ? 3 : 6;
template <int DT, bool WIDE>
using ForwardRing = Ring<DT, kVec<DT, false>, 3, kForwardSlots, false, WIDE>;
template <int DT, bool WIDE>
using BackwardRing = Ring<DT, kVec<DT, true>, 4, kBackwardSlots<DT>, true, WIDE>;
template <int DT, bool WIDE>
using BackMapRing = Ring<DT, kVec<DT, true>, 2, kBackMapSlots<DT>, false, WIDE>;
// shared memory of a warp, with room for its outputs
template <int DT>
constexpr int kForwardBytes = ForwardRing<DT, true>::kBytes + ForwardRing<DT, true>::kBox;
template <int DT>
constexpr int kBackwardBytes = BackwardRing<DT, true>::kBytes + 3 * BackwardRing<DT, true>::kBox;
template <int DT>
constexpr int kMapBytes(bool back) {
  return back ? BackMapRing<DT, true>::kBytes : ForwardRing<DT, true>::kBytes;
}

// The maps of a run, forward: h at its end from h at its start.  Only the
// tokens from the run's last start on count.
template <int DT, bool WIDE>
__device__ __forceinline__ void run_map(const ScanArgs& a, const Place& p, uint8_t* mem, Two speed, bool near, int lane,
                                        Map* m) {
  constexpr int VEC = kVec<DT, false>;
#pragma unroll
  for (int v = 0; v < VEC; ++v) m[v] = Map{1.f, 0.f};
  if (p.t0 >= p.t1) return;
  Cursor cur(a, lane);
  int64_t first, end;
  const int64_t s = cur.owner(p.t1 - 1, true, first, end);
  const bool cut = first >= p.t0 && first < p.t1;
  float h[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) h[v] = cut && a.h0 && v < p.on ? a.h0[s * a.C + p.c + v] : 0.f;
  const int64_t from = cut ? first : p.t0;
  int left = (int)(p.t1 - from);
  ForwardRing<DT, WIDE> ring(a, mem, p.cb, lane, left);
  const Constants k;
  ring.input(kR, a.r, a.sr, from, p.cb);
  ring.input(kG, a.g, a.sg, from, p.cb);
  ring.input(kX, a.x, a.sx, from, p.cb);
#pragma unroll
  for (int i = 0; i < kForwardSlots; ++i) ring.fill();
  Two product = two(1.f);
  for (; left > 0; left -= kStep) {
    ring.ready();
    Two A[kPairs<VEC>], B[kPairs<VEC>];
    step_inputs<VEC>(ring, k, speed, near, A, B);
    if (left < kStep) {  // tokens outside the run change nothing
#pragma unroll
      for (int q = 0; q < kPairs<VEC>; ++q) {
        A[q] = upto<VEC>(A[q], q, left, 1.f);
        B[q] = upto<VEC>(B[q], q, left, 0.f);
      }
    }
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) {
      advance<VEC>(A[q], B[q], h);
      product = product * A[q];
    }
    ring.done();
  }
  cp_wait<0>();
  m[0] = Map{cut ? -1.f : (VEC == 1 ? lo(product) * hi(product) : lo(product)), h[0]};
  if (VEC == 2) m[VEC - 1] = Map{cut ? -1.f : hi(product), h[VEC - 1]};
}

// The maps of a run, backward: a G at its start from a G behind its end.
// Only the tokens up to the run's first end count.
template <int DT, bool WIDE>
__device__ __forceinline__ void run_map_back(const ScanArgs& a, const Place& p, uint8_t* mem, Two speed, bool near, int lane,
                                             Map* m) {
  constexpr int VEC = kVec<DT, true>;
#pragma unroll
  for (int v = 0; v < VEC; ++v) m[v] = Map{1.f, 0.f};
  if (p.t0 >= p.t1) return;
  Cursor cur(a, lane);
  int64_t first, end;
  const int64_t s = cur.owner(p.t0, false, first, end);
  const bool cut = end > p.t0 && end <= p.t1;
  int left = (int)((cut ? end : p.t1) - p.t0);
  float last[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) last[v] = cut && a.dh_last && v < p.on ? a.dh_last[s * a.C + p.c + v] : 0.f;
  BackMapRing<DT, WIDE> ring(a, mem, p.cb, lane, left);
  const Constants k;
  ring.input(0, a.r, a.sr, p.t0, p.cb);
  ring.input(1, a.dh, a.sdh, p.t0, p.cb);
#pragma unroll
  for (int i = 0; i < kBackMapSlots<DT>; ++i) ring.fill();
  for (; left > 0; left -= kStep) {
    ring.ready();
#pragma unroll
    for (int q = 0; q < kPairs<VEC>; ++q) {
      const Two r = ring.pair(0, q);
      Two A = near ? decay_near(speed * rcp(ex2(r * k.minus_log2e) + k.one), k).a
                   : decay_any(speed * two(sigmoid(lo(r)), sigmoid(hi(r)))).a;
      Two D = ring.pair(1, q);
      if (left <= kStep) {  // the run's last token, and those outside it
        A = upto<VEC>(A, q, left, 1.f);
        D = D + two(token_of<VEC>(q, 0) + 1 == left ? last[0] : 0.f, token_of<VEC>(q, 1) + 1 == left ? last[VEC - 1] : 0.f);
      }
      if (VEC == 1) {
        m[0].A *= lo(A);
        m[0].B = fmaf(m[0].A, lo(D), m[0].B);
        m[0].A *= hi(A);
        m[0].B = fmaf(m[0].A, hi(D), m[0].B);
      } else {
        const Two P = two(m[0].A, m[VEC - 1].A) * A, B = fma2(P, D, two(m[0].B, m[VEC - 1].B));
        m[0] = Map{lo(P), lo(B)};
        m[VEC - 1] = Map{hi(P), hi(B)};
      }
    }
    ring.done();
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
template <int DT, bool BACK, bool WIDE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) maps_kernel(ScanArgs a) {
  constexpr int VEC = kVec<DT, BACK>;
  extern __shared__ __align__(128) uint8_t mem[];
  __shared__ Map runs[kWarps][64];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of<VEC>(a, warp, lane);
  bool near;
  const Two speed = speed_at<VEC>(a, p, near);
  uint8_t* mine = mem + warp * kMapBytes<DT>(BACK);
  Map m[VEC];
  if (BACK) run_map_back<DT, WIDE>(a, p, mine, speed, near, lane, m);
  else run_map<DT, WIDE>(a, p, mine, speed, near, lane, m);
  const int64_t k = blockIdx.x / a.cblocks;
  if (BACK && k == 0 && threadIdx.x == 0) a.arrived[blockIdx.x] = 0;  // for the backward kernel, which waits for this one
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    runs[warp][lane * VEC + v] = m[v];
    a.warp_map[(k * kWarps + warp) * a.Cp + p.c + v] = word_of(m[v]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kChannels<VEC>; i += kThreads) {
    Map all = runs[BACK ? kWarps - 1 : 0][i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) all = join(all, runs[BACK ? kWarps - 1 - w : w][i]);
    a.block_map[k * a.Cp + p.cb + i] = word_of(all);
  }
}

// What reaches a warp's run: the blocks before this one, in rounds of 128 or 64
// from the nearest on (sixteen or eight to a warp), until nothing further back
// matters; then the warps before this one.  Every thread of the block calls
// this.
template <int VEC, bool BACK>
__device__ __forceinline__ void reach(const ScanArgs& a, const Place& p, int warp, int lane, float* in) {
  constexpr int kEach = 16 / VEC;
  __shared__ Map part[kWarps][64];
  const int64_t k = blockIdx.x / a.cblocks;
  const int64_t before = BACK ? a.blocks - 1 - k : k;  // blocks before this one in scan order
  float2 own[kWarps - 1][VEC];
#pragma unroll
  for (int j = 0; j < kWarps - 1; ++j) {
    const int r = BACK ? kWarps - 1 - j : j;  // in scan order
    const bool mine = BACK ? r > warp : r < warp;
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      own[j][v] = mine ? __ldcg(a.warp_map + (k * kWarps + r) * a.Cp + p.c + v) : make_float2(1.f, 0.f);
  }
  Map all[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) all[v] = Map{1.f, 0.f};
  for (int64_t done = 0; done < before && !(all[0].A < 0.f); done += kEach * kWarps) {
    // this warp's share, farthest first
    Map m[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) m[v] = Map{1.f, 0.f};
    float2 w[kEach][VEC];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int64_t away = done + kEach * warp + kEach - j;  // 1: the neighbour
      const int64_t b = BACK ? k + away : k - away;
#pragma unroll
      for (int v = 0; v < VEC; ++v) w[j][v] = away <= before ? __ldcg(a.block_map + b * a.Cp + p.c + v) : make_float2(1.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
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
  for (int v = 0; v < VEC; ++v) {
    in[v] = apply(all[v], 0.f);
#pragma unroll
    for (int j = 0; j < kWarps - 1; ++j) in[v] = apply(map_of(own[j][v]), in[v]);
  }
}

// The same where one block holds all tokens: the warps' maps are made here.
template <int VEC, bool BACK>
__device__ __forceinline__ void reach_alone(const Map* m, int warp, int lane, float* in) {
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
template <int DT, bool ALONE, bool WIDE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) forward_kernel(ScanArgs a) {
  constexpr int VEC = kVec<DT, false>;
  extern __shared__ __align__(128) uint8_t mem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of<VEC>(a, warp, lane);
  bool near;
  const Two speed = speed_at<VEC>(a, p, near);
  uint8_t* mine = mem + warp * kForwardBytes<DT>;
  float h[VEC];
  if (ALONE) {
    Map m[VEC];
    run_map<DT, WIDE>(a, p, mine, speed, near, lane, m);
    reach_alone<VEC, false>(m, warp, lane, h);
  }
  int left = (int)(p.t1 - p.t0);
  ForwardRing<DT, WIDE> ring(a, mine, p.cb, lane, left);
  ring.input(kR, a.r, a.sr, p.t0, p.cb);
  ring.input(kG, a.g, a.sg, p.t0, p.cb);
  ring.input(kX, a.x, a.sx, p.t0, p.cb);
#pragma unroll
  for (int i = 0; i < kForwardSlots; ++i) ring.fill();
  empty_sequences(a, a.h0, a.h_last);
  Cursor cur(a, lane);
  Events ev;
  if (left > 0) ev.find(cur, p.t0, left < kStep ? left : kStep, false, lane);
  if (!ALONE) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    reach<VEC, false>(a, p, warp, lane, h);
  }
  const Constants k;
  Out<DT, VEC, false, WIDE> out(a.h, a.sh, p.t0, p.cb, a.C, mine + ForwardRing<DT, WIDE>::kBytes, lane);
  float* state = a.states ? a.states + p.t0 / kStep * a.C + p.c : nullptr;
  for (int64_t t = p.t0; left > 0; left -= kStep) {
    const int n = left < kStep ? left : kStep;
    ring.ready();
    if (state) {
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if (v < p.on) state[v] = h[v];
      state += a.C;
    }
    Two A[kPairs<VEC>], B[kPairs<VEC>];
    step_inputs<VEC>(ring, k, speed, near, A, B);
    if ((ev.starts | ev.ends) == 0) {
#pragma unroll
      for (int q = 0; q < kPairs<VEC>; ++q) out.put(q, advance<VEC>(A[q], B[q], h), n);
    } else {
#pragma unroll
      for (int q = 0; q < kPairs<VEC>; ++q) {
        float o[2];
#pragma unroll
        for (int e = 0; e < 3 - VEC; ++e) {  // the pair's tokens
          const int j = token_of<VEC>(q, e);
          if (ev.starts >> j & 1) {
            const int64_t s = ev.sequence(j);
#pragma unroll
            for (int v = 0; v < VEC; ++v) h[v] = a.h0 && v < p.on ? a.h0[s * a.C + p.c + v] : 0.f;
          }
#pragma unroll
          for (int v = 0; v < VEC; ++v) o[e + v] = h[v] = fmaf(element<VEC>(A, j, v), h[v], element<VEC>(B, j, v));
          if (ev.ends >> j & 1) {
            const int64_t s = ev.sequence(j);
#pragma unroll
            for (int v = 0; v < VEC; ++v)
              if (v < p.on) a.h_last[s * a.C + p.c + v] = h[v];
          }
        }
        out.put(q, two(o[0], o[1]), n);
      }
    }
    ring.done();  // keeps the warp together: the step's outputs are complete
    out.flush(n);
    t += kStep;
    if (left > kStep) ev.find(cur, t, left - kStep < kStep ? left - kStep : kStep, false, lane);
  }
  cp_wait<0>();
}

template <int DT, bool ALONE, bool WIDE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) backward_kernel(ScanArgs a) {
  constexpr int VEC = kVec<DT, true>, kP = kPairs<VEC>;
  static_assert(VEC == 1, "a lane takes one channel");
  extern __shared__ __align__(128) uint8_t mem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of<VEC>(a, warp, lane);
  bool near;
  const Two speed = speed_at<VEC>(a, p, near);
  uint8_t* mine = mem + warp * kBackwardBytes<DT>;
  float c[VEC];
  Two sum = two(0.f);
  if (ALONE) {
    Map m[VEC];
    run_map_back<DT, WIDE>(a, p, mine, speed, near, lane, m);
    reach_alone<VEC, true>(m, warp, lane, c);
  }
  // steps from the run's last one down
  const int tokens = (int)(p.t1 - p.t0);
  const int steps = (tokens + kStep - 1) / kStep;
  int64_t t = p.t0 + (int64_t)(steps > 0 ? steps - 1 : 0) * kStep;
  int n = tokens - (steps - 1) * kStep;  // of the last step; the others are whole
  BackwardRing<DT, WIDE> ring(a, mine, p.cb, lane, tokens);
  ring.input(kR, a.r, a.sr, t, p.cb);
  ring.input(kG, a.g, a.sg, t, p.cb);
  ring.input(kX, a.x, a.sx, t, p.cb);
  ring.input(kD, a.dh, a.sdh, t, p.cb);
  ring.state = a.states + t / kStep * a.C + p.cb;
#pragma unroll
  for (int i = 0; i < kBackwardSlots<DT>; ++i) ring.fill();
  empty_sequences(a, a.dh_last, a.dh0);
  Cursor cur(a, lane);
  Events ev;
  if (steps > 0) ev.find(cur, t, n, true, lane);
  if (!ALONE) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    reach<VEC, true>(a, p, warp, lane, c);
  }
  uint8_t* room = mine + BackwardRing<DT, WIDE>::kBytes;
  constexpr int kBox = BackwardRing<DT, WIDE>::kBox;
  Out<DT, VEC, true, WIDE> px(a.dx, a.sdx, t, p.cb, a.C, room, lane);
  Out<DT, VEC, true, WIDE> pr(a.dr, a.sdr, t, p.cb, a.C, room + kBox, lane);
  Out<DT, VEC, true, WIDE> pg(a.dg, a.sdg, t, p.cb, a.C, room + 2 * kBox, lane);
  const Constants k;
  for (int left = steps; left > 0; --left) {
    ring.ready();
    Two sr[kP], sg[kP], A[kP], inv[kP], beta[kP], found[kP], G[kP];
    step_gates<VEC>(ring, k, speed, near, sr, sg, A, beta);
    const bool plain = (ev.starts | ev.ends) == 0 && n == kStep;
    // the states that the step's tokens find
    float h = ring.first_state(0);
#pragma unroll
    for (int q = 0; q < kP; ++q) {
      // where 1 - a^2 is 0 the token takes nothing in, and its gate's slope
      // u d beta / d u = u a^2 / beta goes to 0 with u
      inv[q] = inv_root(two(fmaxf(lo(beta[q]), 1e-37f), fmaxf(hi(beta[q]), 1e-37f)));
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
      for (int q = kP - 1; q >= 0; --q) {
        const float g1 = hi(G[q]) + c[0], g0 = fmaf(hi(A[q]), g1, lo(G[q]));
        c[0] = lo(A[q]) * g0;
        G[q] = two(g0, g1);
      }
    } else {
#pragma unroll
      for (int j = kStep - 1; j >= 0; --j) {
        float g = element<VEC>(G, j, 0);
        if (j < n) {
          if (ev.ends >> j & 1) {
            const int64_t s = ev.sequence(j);
            if (a.dh_last && p.on) g += a.dh_last[s * a.C + p.c];
          } else {
            g += c[0];
          }
          c[0] = element<VEC>(A, j, 0) * g;
          if (ev.starts >> j & 1) {
            const int64_t s = ev.sequence(j);
            if (a.dh0 && p.on) a.dh0[s * a.C + p.c] = c[0];
          }
        }
        G[j >> 1] = j & 1 ? two(lo(G[j >> 1]), g) : two(g, hi(G[j >> 1]));
      }
    }
#pragma unroll
    for (int q = 0; q < kP; ++q) {
      const Two x = ring.pair(kX, q, true);
      const Two w = G[q] * (speed * sr[q]) * A[q] * fma2(A[q] * inv[q], sg[q] * x, negative(found[q]));
      const Two dx = G[q] * beta[q] * sg[q];
      px.put(q, dx, n);
      pr.put(q, w * (k.one + negative(sr[q])), n);
      pg.put(q, dx * x * (k.one + negative(sg[q])), n);
      sum = sum + w;  // 0 behind the batch, where dh reads as 0
    }
    const int wrote = n;
    n = kStep;
    ring.done();  // keeps the warp together: the step's outputs are complete
    px.flush(wrote);
    pr.flush(wrote);
    pg.flush(wrote);
    t -= kStep;
    if (left > 1) ev.find(cur, t, kStep, true, lane);
  }
  cp_wait<0>();

  // The decay's gradient: the warps' shares, then the blocks', always added in
  // the same order, the blocks' by the last of them to finish.
  __shared__ float shares[kWarps][32];
  __shared__ bool s_last;
  const int64_t block = blockIdx.x / a.cblocks;
  shares[warp][lane] = lo(sum) + hi(sum);
  __syncthreads();
  const int i = threadIdx.x;
  const bool mine_to_sum = i < kChannels<VEC>, on = mine_to_sum && p.cb + i < a.C;
  float total = 0.f;
  if (mine_to_sum) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += shares[w][i];
  }
  if (!ALONE) {
    if (on) a.partial[block * a.C + p.cb + i] = total;
    __threadfence();
    __syncthreads();
    if (i == 0) s_last = atomicAdd(a.arrived + blockIdx.x % a.cblocks, 1u) == (uint32_t)a.blocks - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      float part = 0.f;
      if (v < p.on) {
#pragma unroll 8
        for (int64_t b = warp; b < a.blocks; b += kWarps) part += __ldcg(a.partial + b * a.C + p.c + v);
      }
      shares[warp][lane * VEC + v] = part;
    }
    __syncthreads();
    total = 0.f;
    if (mine_to_sum) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) total += shares[w][i];
    }
  }
  if (on) {
    const float d = a.decay[p.cb + i], sp = softplus(d);
    // ddecay = sigmoid(decay) / softplus(decay) * total; far below zero both
    // are exp(decay) and the ratio is 1
    a.ddecay[p.cb + i] = d < -16.f ? total : total * (1.f / (1.f + expf(-d))) / sp;
  }
}

// One token of each of S sequences: the state moves on in place.  A thread
// per element; bound by its launch (64 sequences x 256 channels: 2.2 us).
template <int DT>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (i >= (int64_t)a.S * a.C) return;
  const int64_t s = i / a.C, c = i - s * a.C;
  const float x = load_element<DT>(at<DT>(a.x, s * a.sx + c));
  const float r = load_element<DT>(at<DT>(a.r, s * a.sr + c));
  const float g = load_element<DT>(at<DT>(a.g, s * a.sg + c));
  const Decay<float> d = decay_of(speed_of(a, c) * sigmoid(r));
  const float h = fmaf(d.a, a.h_last[i], root(d.q) * sigmoid(g) * x);
  a.h_last[i] = h;
  if (DT == TBE_F32) static_cast<float*>(a.h)[s * a.sh + c] = h;
  else if (DT == TBE_F16) static_cast<__half*>(a.h)[s * a.sh + c] = __float2half_rn(h);
  else static_cast<__nv_bfloat16*>(a.h)[s * a.sh + c] = __float2bfloat16_rn(h);
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int32_t channel_blocks(int32_t C, int32_t dtype, bool back) {
  const int32_t each = dtype == TBE_F32 || back ? 32 : 64;
  return (C + each - 1) / each;
}
int64_t whole_channels(int32_t C) { return ((int64_t)C + 63) / 64 * 64; }

// Tokens per warp: as many as give every warp that fits on the GPU one run,
// in whole steps (two waves: training pass over 2,048 sequences and 40,960
// tokens 81 us instead of 63; 65,537 x 1,024 406 instead of 408 us).  Up to
// kAlone tokens one block takes the whole batch, both passes in one kernel:
// 4 sequences x 256 channels, training pass of 96 tokens 14.9 us against 15.4
// with two, 192 tokens 18.8 against 15.5 us.
constexpr int64_t kAlone = 128;
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

// The workspace: maps of blocks and runs, then the backward's partial sums
// and counters.  A batch of one block needs none.
struct Workspace {
  size_t block, warp, partial, arrived, bytes;
};
Workspace layout(int64_t N, int32_t C, int32_t dtype, bool backward) {
  const int32_t cblocks = channel_blocks(C, dtype, backward);
  const Split sp = split_of(N, cblocks);
  const size_t Cp = (size_t)whole_channels(C);
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
    at += round256((size_t)cblocks * 4);
  }
  w.bytes = at;
  return w;
}

bool aligned_to(const void* p, int64_t stride_bytes, int n) { return ((uintptr_t)p & (n - 1)) == 0 && stride_bytes % n == 0; }

// How rows may be read: bytes per asynchronous copy of an input.  Training
// passes with 16, 4 and 0: 65,537 tokens x 1,024, 1,022, 1,021 channels bf16
// 404, 713, 920 us; 40,960 tokens x 128, 126, 125 channels 57, 82, 98 us.
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

// Whether two [sequences, channels] states share memory: what a block writes
// of one would race with what another block reads of the other.
bool overlap(const tbe_scan_inputs* in, const float* p, const float* q) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  const size_t bytes = sizeof(float) * (size_t)in->sequences * (size_t)in->channels;
  return p && q && a < b + bytes && b < a + bytes;
}

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
  a.cblocks = channel_blocks(a.C, dtype, backward);
  const Split sp = split_of(a.N, a.cblocks);
  a.run = sp.run;
  a.blocks = sp.blocks;
  const Workspace w = layout(a.N, a.C, dtype, backward);
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
  if (overlap(in, in->h0, h_last)) return TBE_ERR_INVALID_ARG;
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
  if (overlap(in, dh_last, out->dh0)) return TBE_ERR_INVALID_ARG;
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
  st = use_workspace(a, in->dtype, true, workspace, workspace_bytes);
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
