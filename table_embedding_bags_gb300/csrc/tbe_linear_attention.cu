// tbe_linear_attention.cu -- causal linear attention with a decay for each
// head over jagged sequences, its backward pass and its form for single
// tokens.
//
//   S_t = gamma S_{t-1} + k_t v_t^T      o_t = scale q_t^T S_t      gamma = exp(-decay[head])
//
// In tiles of up to 128 tokens: within a tile a masked product, o += (q k^T .
// gamma^distance) v, and across tiles the state, o += gamma^(place + 1) q S
// and S = gamma^n S + sum gamma^(n - 1 - place) k v^T.  A tile may hold many
// short sequences, whose products the mask keeps apart; it ends where its
// last sequence starts if that one goes on behind it, so short sequences need
// no state at all.  (Where states come in or go out, a tile has one sequence.)
//
// A block takes a run of the token axis of one head.  The state that a run
// finds comes from the runs before it: the same kernel first sums what each
// run adds to the state of the sequence that leaves it, a second one joins
// those along the runs, in order; sequences that end inside their run cost
// neither anything.  No block waits for another inside a kernel and no sum
// depends on timing.
//
// The four products of a tile go to the tensor cores (tcgen05), each with 128
// rows: q k^T and q S, then the weighted (q k^T) from TMEM times v, and the
// weighted keys times v.  One warp finds the tiles, starts the copies and
// issues the products; eight warps weigh what comes out of one product before
// it goes into the next, hold the state in registers and write the outputs.
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
// type that the output is rounded to as well.  What is added to the state is
// not: gamma^n k goes in as the sum of two numbers of the type (16 bits of
// bf16, 22 of fp16), or three of bf16 where the state is a result.  A tile's
// sum begins at 0 and is added to the state in registers, because the tensor
// cores cut sums off.  fp16 lacks fp32's range, so there each of the three is
// first moved by a power of two that its largest value names: products by
// row, the state and the keys by tile.
//
// Values that are no numbers.  The mask's zeros do not stop them inside a tile:
// 0 times a NaN is one.  A tile's values are looked over while the products of
// queries and keys go on.  Those of other sequences are set to 0, and the tile is
// cut to its first sequence; for those of its own the product with the values is
// taken again without the last of them and what follows, for the outputs before
// it, and so on: tokens keep theirs up to such a value.
//
// What bounds it: the latency of a tile's chain, with one block of 128-wide
// heads to an SM (its operands take 194 KB) or two of 64-wide ones.  In cycles,
// 128 wide: copies 1,900, q k^T 1,100, weights 1,500-2,100, keys 2,100, products
// of the values and keys 1,700, state 300, outputs 2,200 beside the next copies:
// 9,000 a tile, where its bytes alone would take 5,600.  Under ncu the outputs of
// 40,000 x 4 x 128 bf16 read DRAM at 28 % of its rate with 15 % of the tensor
// cores' cycles and 27 % of the issue slots in use; 64 wide, fp16: 26, 13, 45 %.
// Prefill of 100,003 x 4 x 128 bf16 188 us (its bytes: 60 us), training pass of
// 65,537 x 16 x 64 f16 with states 1,202 us (159), of 2,048 sequences, 40,960 x
// 8 x 64 bf16 225 us (50), prefill of 257 sequences with states, 8,191 x 5 x 100
// f16, 200 us (20).  The same recurrences in tiles of 64 with mma.sync, four warps
// to a block, took 418, 1,466, 358 and 201 us.
#include "tbe_overlap.cuh"
#include "tbe_tensor.cuh"

#include <algorithm>
#include <cmath>

namespace tbe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 128;         // tokens
constexpr int kWarps = 8;          // that work on what the products give
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kPowers = kTile + 2;
constexpr int kMaxPasses = 3;
constexpr int kMaxMaps = 4;

__device__ __forceinline__ void wait_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One recurrence.  Heads and tokens are `h*` and `s*` elements apart.
struct Pass {
  const uint16_t *q, *k, *v;
  int64_t sq, sk, sv, hq, hk, hv;
  int32_t mq, mk, mv;  // their tensor maps
  uint16_t* o;
  int64_t so, ho;
  const float* in;     // [sequences, heads, d, d] or null
  float* out;          // likewise
  int32_t in_turned;   // `in` holds the transposes
  int32_t back;        // from the last token to the first, decay behind the read
  int32_t piece_o;     // bytes that rows are written by
  float scale_tile, scale_add, scale_read;
  float* carry;        // [heads, runs, W, W]: what each run leaves to the next
  int32_t* kind;       // [runs]
};
struct Args {
  CUtensorMap map[kMaxMaps];
  Pass pass[kMaxPasses];
  const float* decay;
  IdxPtr offsets;
  int64_t N;
  int32_t S, H, d;
  int32_t run;     // tokens of a run
  int32_t runs;
  int32_t piece;   // bytes that rows are read by, 0 for tensor copies
  int32_t terms;   // of the weighted keys that there is room for
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
  __device__ __forceinline__ int64_t at_or_end(int64_t i) const { return i <= S ? at(i) : INT64_MAX; }
  __device__ __forceinline__ int64_t sequence(int64_t i) const { return back ? S - 1 - i : i; }
  // the first i with at(i) >= x
  __device__ int64_t first(int64_t x) const {
    int64_t lo = 0, hi = (int64_t)S + 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (at(mid) >= x) hi = mid; else lo = mid + 1;
    }
    return lo;
  }
};

__device__ __forceinline__ float power(float decay, int64_t n) { return n == 0 ? 1.f : exp2f(-(float)n * decay * kLog2e); }

// 2^x to 2^-22 of its size, 0 for the lowest.
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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

// Powers of two for fp16: what brings values of magnitude `top` to 2^14 or
// just below, as an exponent (kept where fp32 stays normal).  For states and
// keys the finite values decide: moved down by an infinity's power, they would
// all become 0.  (x 0 + x is NaN for an infinity, which a maximum passes over.)
__device__ __forceinline__ int room_for(float top) {
  const int e = (int)(__float_as_uint(top) >> 23 & 255) - 127;  // 128 for infinities and NaN
  return max(-100, min(60, 13 - e));
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// ---------------------------------------------------------------------------
// a block's shared memory
// ---------------------------------------------------------------------------

// Operands lie in blocks of 64 columns, [128 rows x 128 bytes] with the
// 128-byte swizzle, as tensor copies write them: element (row, col) in the
// 16-byte chunk (col / 8) ^ (row & 7) of its row.
constexpr int kBlock = kTile * 128;
template <int W>
struct Room {  // W: columns of a head, filled up
  static constexpr int operand = W / 64 * kBlock;
  static constexpr int state = W * W * 2;
  static constexpr int q = 0, k = operand, v = 2 * operand, s = 3 * operand, rest = 3 * operand + state;  // behind the terms
  static constexpr int bytes(int n_terms) { return rest + n_terms * operand; }
  // columns of TMEM: the products of a tile, whose weighted form in 16 bits takes the first and the last quarter of
  // theirs; the two parts of the outputs; the sum that goes to the state (between those quarters, where that is enough)
  static constexpr int cols = W == 64 ? 256 : 512;
  static constexpr int tp = 0, to = kTile, ts = kTile + W, ta = W == 64 ? 32 : kTile + 2 * W;
  static constexpr int weighted(int part) { return tp + (part < 4 ? part * 8 : 64 + part * 8); }  // of 16 columns each
};

// What is known of a tile.
struct Tile {
  int64_t p;          // its first position, -1 behind the last tile
  uint32_t starts[4]; // places where a sequence starts
  int32_t n;          // positions taken
  int32_t e0;         // where its first sequence ends
  int32_t begins;     // a sequence starts at its first place
  int32_t live;       // its first sequence has a state
  int32_t adds;       // it adds to the state,
  int32_t leaves;     //   which goes on behind it
  int32_t mixed;      // rows of other sequences have been copied with it
  int64_t sequence;   // its first sequence
};
struct Control {
  uint64_t known[2], full, products, weighted, keys, out_done, add_done, add_read, out_read, state_ready, exchange, again_done, again_read, row_max[4];
  Tile tile[2];
  float pow[kPowers];
  alignas(16) float by_col[16];  // powers over 16 neighbouring columns
  float top_row[2][kTile];
  uint32_t top[3];
  int32_t bad[2];          // some value of the tile is an infinity or a NaN:
  int32_t again;           //   outputs before this place are made again (0: no more)
  uint32_t passes[kWarps]; //   times that a warp has waited for that
  uint32_t tmem;
  int32_t dead;
};

// A bounded wait: false (and the others give up too) after four seconds.
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int32_t* dead) {
  uint64_t begin, now;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(begin));
  for (;;) {
    if (mbar_wait(bar, parity, 64)) return true;
    if (*dead) return false;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
    if (now - begin > 4000000000ull) {
      *dead = 1;
      return false;
    }
  }
}
// (whole warps)
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Control& c) {
  return __all_sync(kFull, mbar_wait(bar, parity & 1, 1) || wait_long(bar, parity & 1, &c.dead));
}
__device__ __forceinline__ void to_products() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------------------
// which positions make a tile (all lanes of one warp)
// ---------------------------------------------------------------------------

struct Marker {
  Starts st;
  bool one;         // a tile has one sequence
  bool copied;      // rows behind the last token are zeros
  int64_t next;     // the first start not yet passed
  int64_t x;        // at(next + lane), read ahead

  __device__ __forceinline__ void seek(int64_t p, int lane) {
    next = st.first(p);
    x = st.at_or_end(next + lane);
  }
  // The tile at p, of up to `most` positions; live: a state comes in.
  __device__ __forceinline__ void mark(Tile& t, int64_t p, int64_t p1, bool live, bool has_in, bool has_out, int lane) {
    const int most = (int)min((int64_t)kTile, p1 - p);
    const int64_t before = next;
    uint32_t starts[4] = {0, 0, 0, 0};
    int64_t upto = next;  // starts at or below p
    bool closes = false;
    int c;
    for (;;) {
      const bool in = x >= p && x < p + most && next + lane < st.S;
      const int place = in ? (int)(x - p) : 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) starts[w] |= __reduce_or_sync(kFull, in && place >> 5 == w ? 1u << (place & 31) : 0u);
      closes |= __any_sync(kFull, x == p + most);
      upto += __popc(__ballot_sync(kFull, x <= p));
      c = __popc(__ballot_sync(kFull, x < p + most));
      if (c < 32) break;
      next += 32;
      x = st.at_or_end(next + lane);
    }
    t.p = p;
    t.n = most;
    t.begins = starts[0] & 1;
    // the first sequence that starts behind the first place, and the last one
    int first = kTile, last = 0;
#pragma unroll
    for (int w = 3; w >= 0; --w) {
      const uint32_t u = w == 0 ? starts[0] & ~1u : starts[w];
      if (u) {
        first = w * 32 + __ffs((int)u) - 1;
        if (last == 0) last = w * 32 + 31 - __clz((int)u);
      }
    }
    int cut = kTile;
    if (one) cut = first;
    else if (p + most < p1 && !closes && last > 0) cut = last;
    if (cut < most) {
      t.n = cut;
      closes = true;
      if (next == before) {
        c = __popc(__ballot_sync(kFull, x < p + cut));
      } else {  // (more starts than lanes)
        next = st.first(p + cut);
        c = 0;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w)
        starts[w] &= cut >= w * 32 + 32 ? ~0u : cut > w * 32 ? (1u << (cut - w * 32)) - 1 : 0u;
    }
    next += c;
#pragma unroll
    for (int w = 0; w < 4; ++w) t.starts[w] = starts[w];
    t.e0 = min(first, t.n);
    const bool whole = t.e0 == t.n, last_tile = p + t.n >= p1;
    // (its first sequence is always known, unless offsets are broken)
    t.sequence = t.begins ? upto - 1 : before - 1;
    const bool known = t.sequence >= 0 && t.sequence < st.S;
    t.sequence = known ? st.sequence(t.sequence) : 0;
    t.live = t.begins ? has_in : live;
    const bool goes_on = whole && !closes && !last_tile;
    t.adds = goes_on || (has_out && known && whole && closes);
    t.leaves = goes_on;
    t.mixed = !(whole && (t.n == kTile || (p + t.n == st.N && copied)));
    x = st.at_or_end(next + lane);
  }
};

// ---------------------------------------------------------------------------
// the kernel: outputs, or (SUMS) what each run leaves
// ---------------------------------------------------------------------------

// One head's rows of a tile to an operand, where tensor copies cannot: rows
// r0 .. r1 - 1, of which the first is token `first`'s.  Columns behind d and
// rows outside keep what they hold: zeros, or rows of tiles before.
template <int W>
__device__ __forceinline__ void load_rows(uint8_t* dst, const uint16_t* src, int64_t stride, int64_t first, int r0, int r1,
                                          int d, int piece, int thread) {
  const int each = piece / 2, per_row = d / each;
  // a warp takes a row at a time, and parts of two where they are short
  const int at_once = per_row <= 16 ? 16 : 32;
  const int lane = thread % at_once, step = 32 * kWarps / at_once;
#pragma unroll 1
  for (int c0 = lane; c0 < per_row; c0 += at_once) {
    const int c = c0 * each;
    uint8_t* column = dst + c / 64 * kBlock + c % 8 * 2;
    const int chunk = c % 64 / 8;
    const uint16_t* from = src + (first + thread / at_once) * stride + c;
#pragma unroll 4
    for (int r = r0 + thread / at_once; r < r1; r += step, from += step * stride) {
      const uint32_t to = smem_u32(column + r * 128 + ((chunk ^ (r & 7)) * 16));
      if (piece == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
      else if (piece == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
      else if (piece == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
      else asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(__ldg(from)) : "memory");
    }
  }
}

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int32_t col, int32_t head, int32_t row,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(col), "r"(head), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_ahead3(const CUtensorMap* map, int32_t col, int32_t head, int32_t row) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map), "r"(col), "r"(head), "r"(row)
               : "memory");
}

// Where tile i's values lie: without queries their place takes those of every
// other tile, so that a tile's copies go on beside the products of the one
// before (prefill of 100,003 x 4 x 128 bf16 202 -> 187 us).
template <int W, bool SUMS>
__device__ __forceinline__ int values_at(int piece, uint32_t i) {
  return SUMS && piece == 0 && (i & 1) ? Room<W>::q : Room<W>::v;
}

// Descriptor of an operand whose next 64 rows (along M or N) are `apart` bytes on.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, uint32_t apart) {
  return (tc_desc(addr) & ~(0x3fffull << 16)) | ((uint64_t)(apart >> 4) << 16);
}
__device__ __forceinline__ void tc_mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Whether 16 bytes of values hold an infinity or a NaN: 0 times them, added to `sum`, is NaN then.
template <int DT>
__device__ __forceinline__ void look_at(const uint4& u, uint32_t& sum) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (DT == TBE_BF16) {
      const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&(&u.x)[e]),
                                       __bfloat162bfloat162(__ushort_as_bfloat16(0)), *reinterpret_cast<const __nv_bfloat162*>(&sum));
      sum = *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&(&u.x)[e]), __half2half2(__ushort_as_half(0)),
                                *reinterpret_cast<const __half2*>(&sum));
      sum = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}
// The last place marked before place n, or 0.
__device__ __forceinline__ int last_before(const uint32_t (&at)[4], int n) {
  int last = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t u = n >= w * 32 + 32 ? at[w] : n > w * 32 ? at[w] & ((1u << (n - w * 32)) - 1) : 0u;
    if (u) last = w * 32 + 31 - __clz((int)u);
  }
  return last;
}
template <int DT>
__device__ __forceinline__ bool seen(uint32_t sum) {
  const float2 x = unpack2<DT>(sum);
  return !(x.x + x.y == x.x + x.y);
}
// The same of all values of a tile, by STEP threads.
template <int DT, int W, int STEP>
__device__ __forceinline__ bool not_finite(const uint8_t* values, int thread) {
  constexpr int kPieces = Room<W>::operand / 16 / STEP;
  static_assert(kPieces % 4 == 0, "four at a time");
  uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll 2
  for (int i = 0; i < kPieces; i += 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      look_at<DT>(*reinterpret_cast<const uint4*>(values + (i + k) * STEP * 16 + thread * 16), sum[k]);
  }
  return seen<DT>(sum[0]) || seen<DT>(sum[1]) || seen<DT>(sum[2]) || seen<DT>(sum[3]);
}

template <int DT, int W, bool SUMS>
struct Worker {
  static constexpr int kCols = W / 2;  // of the state and the outputs, to a thread
  static constexpr int kChunks = Room<W>::operand / 16 / (32 * kWarps);  // 16-byte pieces of an operand, to a thread
  const Args& a;
  const Pass& ps;
  Control& c;
  uint8_t *terms, *room;
  uint32_t tmem;
  int warp, lane, quarter, half, row;
  int head;
  float s[kCols];         // the state: row `row`, columns half * kCols ..
  float slope;            // -log2 gamma, at most 1e30 (times 0 it is 0)
  float read_scale = 0.f; // what the state in shared memory is to be multiplied by
  uint32_t exchanges = 0;

  __device__ __forceinline__ uint32_t lanes() const { return (uint32_t)(quarter * 32) << 16; }
  __device__ __forceinline__ bool holds() const { return row < W; }  // (else nothing of the state)
  __device__ __forceinline__ void arrive(uint64_t* bar) {
    __syncwarp();
    if (lane == 0) bar_arrive(bar);
  }
  // All of the eight warps meet.  c.top has a word for each meeting in turn.
  __device__ __forceinline__ bool meet() {
    arrive(&c.exchange);
    if (!wait(&c.exchange, exchanges, c)) return false;
    if (warp == 0 && lane == 0) c.top[(exchanges + 2) % 3] = 0;
    ++exchanges;
    return true;
  }
  // The largest of all threads' values (not negative).
  __device__ __forceinline__ bool largest(float& t) {
#pragma unroll
    for (int o = 16; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, o));
    uint32_t* top = &c.top[exchanges % 3];
    if (lane == 0) atomicMax(top, __float_as_uint(t));
    if (!meet()) return false;
    t = __uint_as_float(*(volatile uint32_t*)top);
    return true;
  }

  // The state from, or to, a [d, d] matrix (or its transpose), or a [W, W] one.
  __device__ __forceinline__ void read(const float* p, int d, bool turned) {
    if (!turned && d % 4 == 0 && ((uintptr_t)p & 15) == 0) {
#pragma unroll
      for (int j = 0; j < kCols; j += 4) {
        const int col = half * kCols + j;
        const float4 x = row < d && col < d ? __ldg(reinterpret_cast<const float4*>(p + (int64_t)row * d + col))
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
        s[j] = x.x;
        s[j + 1] = x.y;
        s[j + 2] = x.z;
        s[j + 3] = x.w;
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      const int col = half * kCols + j;
      s[j] = row < d && col < d ? __ldg(p + (turned ? (int64_t)col * d + row : (int64_t)row * d + col)) : 0.f;
    }
  }
  __device__ __forceinline__ void write(float* p, int d) const {
    if (row >= d) return;
    float* to = p + (int64_t)row * d + half * kCols;
    if (d % 4 == 0 && ((uintptr_t)p & 15) == 0) {
#pragma unroll
      for (int j = 0; j < kCols; j += 4)
        if (half * kCols + j < d) *reinterpret_cast<float4*>(to + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (half * kCols + j < d) to[j] = s[j];
    }
  }
  // The state to shared memory in the inputs' type, as the operand [key rows, value columns].
  __device__ __forceinline__ bool publish() {
    float f = 1.f;
    if (DT == TBE_F16) {
      float t = 0.f;
      if (holds()) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) t = fmaxf(t, fabsf(fmaf(s[j], 0.f, s[j])));  // (room_for: finite values)
      }
      if (!largest(t)) return false;
      const int up = room_for(t);
      f = pow2(up);
      read_scale = ps.scale_read * pow2(-up);
    } else {
      read_scale = ps.scale_read;
    }
    if (holds()) {
#pragma unroll
      for (int j = 0; j < kCols; j += 8) {
        const int col = half * kCols + j;
        uint4 u;
        u.x = pack2<DT>(s[j] * f, s[j + 1] * f);
        u.y = pack2<DT>(s[j + 2] * f, s[j + 3] * f);
        u.z = pack2<DT>(s[j + 4] * f, s[j + 5] * f);
        u.w = pack2<DT>(s[j + 6] * f, s[j + 7] * f);
        *reinterpret_cast<uint4*>(room + Room<W>::s + col / 64 * (W * 128) + row * 128 + ((col % 64 / 8) ^ (row & 7)) * 16) = u;
      }
    }
    to_products();
    arrive(&c.state_ready);
    return true;
  }

  // A place's distance from the tile's first position, in the pass's direction.
  __device__ __forceinline__ int place(int r) const { return ps.back ? kTile - 1 - r : r; }

  // fp16: the power of two that the weighted keys are moved by.
  __device__ __forceinline__ bool room_for_keys(int n, int& up) {
    const __half2 none = __half2half2(__ushort_as_half(0));
    __half2 top = none;
#pragma unroll 2
    for (int i = 0; i < kChunks; ++i) {
      const int at = i * 32 * kWarps * 16 + (warp * 32 + lane) * 16;
      const uint4 u = *reinterpret_cast<const uint4*>(room + Room<W>::k + at);
      if (place(at / 128 % kTile) < n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 x = reinterpret_cast<const __half2*>(&u)[e];
          top = __hmax2(top, __habs2(__hfma2(x, none, x)));
        }
      }
    }
    const float2 t = __half22float2(top);
    float most = fmaxf(t.x, t.y) * fabsf(ps.scale_add);
    if (!largest(most)) return false;
    up = room_for(most);
    return true;
  }
  // The keys times 2^up scale_add gamma^(n - 1 - place + late), as a sum of
  // terms; the weight is 0 behind the tile.
  __device__ __forceinline__ void weigh_keys(int n, int n_terms, int up) {
    const int own = (warp * 32 + lane) * 16;
    const float scale = ps.scale_add * (DT == TBE_F16 ? pow2(up) : 1.f);
    const bool all = n == kTile;
#pragma unroll 2
    for (int i = 0; i < kChunks; ++i) {
      const int at = i * 32 * kWarps * 16 + own, far = place(at / 128 % kTile);
      const uint4 u = *reinterpret_cast<const uint4*>(room + Room<W>::k + at);
      const float w = exp2_of(-slope * (float)(n - 1 - far + ps.back)) * scale;
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = unpack2<DT>((&u.x)[e]);
        x[2 * e] = y.x * w;
        x[2 * e + 1] = y.y * w;
      }
      if (!all && far >= n) {  // (whatever stands there)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
      }
      uint8_t* to = terms + at;
      if (DT == TBE_BF16) {
        for (int t = 1; t < n_terms; ++t, to += Room<W>::operand) {  // cut off: the upper halves of the numbers
          uint4 r;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            (&r.x)[e] = __byte_perm(__float_as_uint(x[2 * e]), __float_as_uint(x[2 * e + 1]), 0x7632);
            x[2 * e] -= __uint_as_float(__float_as_uint(x[2 * e]) & 0xffff0000u);
            x[2 * e + 1] -= __uint_as_float(__float_as_uint(x[2 * e + 1]) & 0xffff0000u);
          }
          *reinterpret_cast<uint4*>(to) = r;
        }
      } else {
        uint4 r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          (&r.x)[e] = pack2<DT>(x[2 * e], x[2 * e + 1]);
          const float2 y = unpack2<DT>((&r.x)[e]);
          x[2 * e] -= y.x;
          x[2 * e + 1] -= y.y;
        }
        *reinterpret_cast<uint4*>(to) = r;
        to += Room<W>::operand;
      }
      uint4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) (&r.x)[e] = pack2<DT>(x[2 * e], x[2 * e + 1]);
      *reinterpret_cast<uint4*>(to) = r;
    }
    to_products();
    arrive(&c.keys);
  }

  // S = gamma^n S + the tile's sum.
  __device__ __forceinline__ void add(int n, float down) {
    const float by = c.pow[n];
    if (quarter * 32 < W) {
      float x[kCols];
#pragma unroll
      for (int j = 0; j < kCols; j += 32) tc_ld32(tmem + Room<W>::ta + half * kCols + j + lanes(), x + j);
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < kCols; ++e) s[e] = fmaf(s[e], by, DT == TBE_F16 ? x[e] * down : x[e]);
    }
    tc_before_sync();
    arrive(&c.add_read);
  }

  // The products of row `row` with 64 of the columns, weighted, to TMEM in
  // 16 bits.  fp16: multiplied by 2^up, up by row.
  __device__ __forceinline__ bool weigh_products(const Tile& t, int n, uint32_t turn, int& up) {
    const int far = place(row);
    int from = 0;  // first place of this row's sequence
    const bool whole = t.e0 >= n;
    const int place0 = ps.back ? kTile - 32 - quarter * 32 : quarter * 32, place31 = place0 + 31;  // of this warp's rows
    if (!whole) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t u = far >= w * 32 + 31 ? t.starts[w] : far >= w * 32 ? t.starts[w] & ((2u << (far - w * 32)) - 1) : 0u;
        if (u) from = w * 32 + 31 - __clz((int)u);
      }
    }
    const uint32_t span = (uint32_t)(far - from);  // places from .. far take part
    // 16 columns at a time, in a loop that stays a loop: the code of a tile is run through once a tile by every warp,
    // and what does not stay in the instruction caches costs more than it computes (with the loops below unrolled
    // over 64 columns a warp's own 32 took 3,500 cycles, in a loop over two times 32 1,500).
    const int step = ps.back ? -1 : 1;
    float scale = ps.scale_tile;
    up = 0;
    if (DT == TBE_F16) {
      // the row's largest product that takes part, before its weight (at most the scale)
      float top = 0.f;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int col = half * 64 + k * 16, near = place(col), last = place(col + 15);
        if (min(near, last) > place31) continue;  // all behind this warp's rows
        float x[16];
        tc_ld16(tmem + Room<W>::tp + col + lanes(), x);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int at = near + step * e;
          top = fmaxf(top, at <= far && at >= from ? fabsf(x[e]) : 0.f);
        }
      }
      c.top_row[half][row] = top;
      arrive(&c.row_max[quarter]);
      if (!wait(&c.row_max[quarter], turn, c)) return false;
      up = room_for(fmaxf(top, *(volatile float*)&c.top_row[half ^ 1][row]) * fabsf(scale));
      scale *= pow2(up);
    }
    // Each half of the columns is written over what its own warps have read: the first from its first columns on, the
    // second from its last.
    const float away0 = (float)far;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const int part = half ? 3 - k : k, col = half * 64 + part * 16, near = place(col), last = place(col + 15);
      float x[16];
      if (min(near, last) > place31) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.f;
      } else {
        tc_ld16(tmem + Room<W>::tp + col + lanes(), x);
        tc_wait_ld();
        if (whole && max(near, last) < place0) {
          // gamma^distance in two parts: to the nearest of these columns, and among them
          const float by = exp2_of(-slope * (float)(far - max(near, last))) * scale;
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            float4 w = *reinterpret_cast<const float4*>(c.by_col + e);
            mul2(w.x, w.y, by);
            mul2(w.z, w.w, by);
            x[e] *= w.x;
            x[e + 1] *= w.y;
            x[e + 2] *= w.z;
            x[e + 3] *= w.w;
          }
        } else {
          const float at = away0 - (float)near, sign = (float)step;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float away = fmaf(sign, -(float)e, at);  // (exact)
            const float y = x[e] * (exp2_of(-slope * away) * scale);
            x[e] = (uint32_t)(near - from + step * e) <= span ? y : 0.f;
          }
        }
      }
      uint32_t packed[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) packed[e] = pack2<DT>(x[2 * e], x[2 * e + 1]);
      tc_st8(tmem + half * 96 + part * 8 + lanes(), packed);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    tc_before_sync();
    arrive(&c.weighted);
    return true;
  }

  // o = the tile's part and the state's, rounded once.
  __device__ __forceinline__ void write_outputs(const Tile& t, int n, int up, float read_scale, uint64_t* out_read) {
    const int far = place(row);
    const bool live = t.live && far < t.e0;
    const float of_state = live ? c.pow[far + 1 - ps.back] * read_scale : 0.f, of_tile = DT == TBE_F16 ? pow2(-up) : 1.f;
    const int64_t token = ps.back ? a.N - t.p - kTile + row : t.p + row;
    uint16_t* to = ps.o + token * ps.so + head * ps.ho + half * kCols;
#pragma unroll 1
    for (int j = 0; j < kCols; j += 16) {
      float x[16];
      tc_ld16(tmem + Room<W>::to + half * kCols + j + lanes(), x);
      if (t.live) {
        float y[16];
        tc_ld16(tmem + Room<W>::ts + half * kCols + j + lanes(), y);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (DT == TBE_F16) x[e] *= of_tile;
          x[e] = live ? fmaf(y[e], of_state, x[e]) : x[e];
        }
      } else {
        tc_wait_ld();
        if (DT == TBE_F16) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] *= of_tile;
        }
      }
      if (j + 16 >= kCols) {
        tc_before_sync();
        arrive(out_read);
      }
      const int cols = a.d - half * kCols - j;
      if (far >= n || cols <= 0) continue;
      uint32_t u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = pack2<DT>(x[2 * e], x[2 * e + 1]);
      if (cols >= 16 && ps.piece_o == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + j), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                     "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                     : "memory");
      } else if (ps.piece_o >= 8) {
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          if (2 * e < cols) *reinterpret_cast<uint2*>(to + j + 2 * e) = make_uint2(u[e], u[e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (2 * e < cols) to[j + 2 * e] = (uint16_t)u[e];
          if (2 * e + 1 < cols) to[j + 2 * e + 1] = (uint16_t)(u[e] >> 16);
        }
      }
    }
  }
};

// Blocks of an SM: what their registers, shared memory and TMEM leave room for.
template <int W>
constexpr int kBlocks = W == 64 ? 2 : 1;

template <int DT, int W, bool SUMS>
__global__ void __launch_bounds__(kThreads, kBlocks<W>) attention_kernel(const __grid_constant__ Args a) {
  using R = Room<W>;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* room = raw + a.terms * R::operand;
  const Pass& ps = a.pass[blockIdx.y];
  const int terms = DT == TBE_BF16 && ps.out ? 3 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = blockIdx.x % a.H, run = blockIdx.x / a.H;
  const int64_t p0 = (int64_t)run * a.run, p1 = min(a.N, p0 + a.run);
  const Starts st = {a.offsets, a.N, a.S, ps.back != 0};
  Control& c = *reinterpret_cast<Control*>(room + R::rest);

  // what a run leaves is asked of all but the last
  int64_t begin = p0;
  bool began = false;
  int64_t sequence = 0;
  if (SUMS) {
    const int64_t next = st.first(p1);  // first start at or behind the run's end
    const bool goes_on = next > 0 && next <= a.S && st.at(next) > p1;
    begin = goes_on ? st.at(next - 1) : p1;
    const int32_t kind = !goes_on ? kNothing : begin >= p0 ? kBegan : kThrough;
    if (threadIdx.x == 0 && head == 0) ps.kind[run] = kind;
    if (kind == kNothing) return;
    began = kind == kBegan;
    begin = max(begin, p0);
    sequence = st.sequence(next - 1);
  }

  if (threadIdx.x == 0) {
    for (int k = 0; k < 2; ++k) bar_init(&c.known[k], 1);
    bar_init(&c.full, a.piece ? kWarps : 1);
    bar_init(&c.products, 1);
    bar_init(&c.weighted, kWarps);
    bar_init(&c.keys, kWarps);
    bar_init(&c.out_done, 1);
    bar_init(&c.add_done, 1);
    bar_init(&c.add_read, kWarps);
    bar_init(&c.out_read, kWarps);
    bar_init(&c.state_ready, kWarps);
    bar_init(&c.exchange, kWarps);
    bar_init(&c.again_done, 2);
    bar_init(&c.again_read, kWarps);
    for (int k = 0; k < 4; ++k) bar_init(&c.row_max[k], 2);
    for (int k = 0; k < 3; ++k) c.top[k] = 0;
    c.bad[0] = c.bad[1] = 0;
    for (int k = 0; k < kWarps; ++k) c.passes[k] = 0;
    c.dead = 0;
    bars_visible();
  }
  const float decay = a.decay[head];
  for (int k = threadIdx.x; k < kPowers; k += kThreads) c.pow[k] = power(decay, k);
  if (a.piece) {  // columns and rows that no copy fills
    for (int k = threadIdx.x; k < R::s / 16; k += kThreads) reinterpret_cast<uint4*>(room)[k] = make_uint4(0, 0, 0, 0);
    to_products();
  }
  if (threadIdx.x < 16) c.by_col[threadIdx.x] = power(decay, ps.back ? threadIdx.x : 15 - threadIdx.x);
  if (warp == kWarps) tc_alloc(&c.tmem, R::cols);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = c.tmem;
  wait_predecessor();
  if (!SUMS && blockIdx.x == 0 && blockIdx.y == 0) {  // broken offsets are reported
    bool bad = false;
    for (int64_t i = threadIdx.x; i < a.S; i += kThreads) bad |= a.offsets.ldg(i) > a.offsets.ldg(i + 1);
    if (threadIdx.x == 0) bad |= a.offsets.ldg(0) != 0 || a.offsets.ldg(a.S) != a.N;
    if (bad) report(a.status, TBE_DEV_BAD_OFFSETS);
  }

  if (warp == kWarps) {
    // finds the tiles, starts the copies, issues the products
    Marker m = {st, ps.in != nullptr || ps.out != nullptr, a.piece == 0, 0, 0};
    if (!SUMS) m.seek(p0, lane);
    const bool live = !SUMS && run > 0 && __shfl_sync(kFull, m.x, 0) > p0;  // (m.x of lane 0: the first start)
    uint32_t states = 0, adds = 0, copies = 0, reads = 0;
    bool added = false;  // by the tile before
    const uint32_t room0 = smem_u32(room), terms0 = smem_u32(raw);
    const uint32_t format = DT == TBE_BF16;
    auto find = [&](int64_t at, bool live) {
      Tile t = {};
      if (at >= p1) {
        t.p = -1;
      } else if (SUMS) {
        t.p = at;
        t.n = (int)min((int64_t)kTile, p1 - at);
        t.e0 = t.n;
        t.adds = 1;
        t.mixed = t.n < kTile;
      } else {
        m.mark(t, at, p1, live, ps.in != nullptr, ps.out != nullptr, lane);
      }
      return t;
    };
    Tile following = find(begin, live);
    // The values from place n on are set to 0.
    auto drop = [&](int n, int values) {
#pragma unroll 1
      for (int i = lane; i < R::operand / 16; i += 32) {
        const int r = i / 8 % kTile;
        if ((ps.back ? kTile - 1 - r : r) >= n) *reinterpret_cast<uint4*>(room + values + i * 16) = make_uint4(0, 0, 0, 0);
      }
      to_products();
      __syncwarp();
    };
    // The places of the tile's values that hold one.
    auto where = [&](uint32_t (&places)[4], int values) {
#pragma unroll 1
      for (int i = lane; i < R::operand / 16; i += 32) {
        uint32_t sum = 0;
        look_at<DT>(*reinterpret_cast<const uint4*>(room + values + i * 16), sum);
        const int r = i / 8 % kTile, place = ps.back ? kTile - 1 - r : r;
#pragma unroll
        for (int w = 0; w < 4; ++w) places[w] |= seen<DT>(sum) && place >> 5 == w ? 1u << (place & 31) : 0u;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) places[w] = __reduce_or_sync(kFull, places[w]);
    };
    // The weighted products times the values.
    auto multiply = [&](int values, uint64_t* done) {
      if (lane == 0) {
        const uint32_t idesc = tc_idesc(format, 0, 1, kTile, W);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          tc_mma_tmem(tmem + R::to, tmem + R::weighted(k), desc_of(room0 + values + k * 2048, kBlock), idesc, k > 0);
        tc_commit(done);
      }
      __syncwarp();
    };
    // A tile's rows on their way to the L2.
    auto ahead = [&](const Tile& t) {
      if (t.p < 0 || a.piece || lane != 0) return;
      const int32_t first = (int32_t)(ps.back ? a.N - t.p - kTile : t.p);
#pragma unroll
      for (int b = 0; b < W / 64; ++b) {
        tma_ahead3(&a.map[ps.mk], b * 64, head, first);
        tma_ahead3(&a.map[ps.mq], b * 64, head, first);
        tma_ahead3(&a.map[ps.mv], b * 64, head, first);
      }
    };
    auto load = [&](const Tile& t, uint32_t i) {
      if (t.p < 0 || a.piece) return;
      ++copies;
      if (lane != 0) return;
      bar_expect(&c.full, (SUMS ? 2 : 3) * R::operand);
      const int32_t first = (int32_t)(ps.back ? a.N - t.p - kTile : t.p);
#pragma unroll
      for (int b = 0; b < W / 64; ++b) {
        tma_load3(room0 + R::k + b * kBlock, &a.map[ps.mk], b * 64, head, first, &c.full);
        if (!SUMS) tma_load3(room0 + R::q + b * kBlock, &a.map[ps.mq], b * 64, head, first, &c.full);
        tma_load3(room0 + values_at<W, SUMS>(a.piece, i) + b * kBlock, &a.map[ps.mv], b * 64, head, first, &c.full);
      }
    };
    for (uint32_t i = 0;; ++i) {
      const Tile t = following;
      bool bad = false;
      const int values = values_at<W, SUMS>(a.piece, i);
      // (the products and copies of the tile before are through)
      if (lane == 0) {
        c.tile[i & 1] = t;
        c.bad[i & 1] = 0;
        bar_arrive(&c.known[i & 1]);
      }
      if (!SUMS || i == 0) load(t, i);
      __syncwarp();
      if (t.p < 0) break;
      if (!wait(&c.full, i, c)) break;
      // the sum for the state lies where these products go (64 columns), or has its own place
      if (added && !wait(&c.add_read, adds - 1, c)) break;
      tc_after_sync();
      if (!SUMS) {
        if (lane == 0) {
          const uint32_t idesc = tc_idesc(format, 0, 0, kTile, kTile);
#pragma unroll
          for (int k = 0; k < W / 16; ++k)
            tc_mma(tmem + R::tp, tc_desc(room0 + R::q + k / 4 * kBlock + k % 4 * 32),
                   tc_desc(room0 + R::k + k / 4 * kBlock + k % 4 * 32), idesc, k > 0);
          tc_commit(&c.products);
        }
        __syncwarp();
        if (i > 0 && !wait(&c.out_read, i - 1, c)) break;
        if (t.live) {
          if (!wait(&c.state_ready, states++, c)) break;
          tc_after_sync();
          if (lane == 0) {
            const uint32_t idesc = tc_idesc(format, 0, 1, kTile, W);
#pragma unroll
            for (int k = 0; k < W / 16; ++k)
              tc_mma(tmem + R::ts, tc_desc(room0 + R::q + k / 4 * kBlock + k % 4 * 32), desc_of(room0 + R::s + k * 2048, W * 128),
                     idesc, k > 0);
          }
          __syncwarp();
        }
        following = find(t.p + t.n, t.leaves);  // (while these products go on and are weighted)
        ahead(following);
        if (!wait(&c.weighted, i, c)) break;
        tc_after_sync();
        bad = *(volatile int32_t*)&c.bad[i & 1];
        if (bad && t.mixed) drop(t.e0, values);
        multiply(values, &c.out_done);
      }
      if (t.adds) {
        if (!wait(&c.keys, adds, c)) break;
        tc_after_sync();
        if (SUMS) {
          if (t.mixed && *(volatile int32_t*)&c.bad[i & 1]) drop(t.n, values);
          following = find(t.p + t.n, false);
          load(following, i + 1);  // the keys have been read, and the values go elsewhere
          __syncwarp();
        }
        if (lane == 0) {
          // (64 columns: the products' other 64 rows, of what follows in memory, are not looked at)
          const uint32_t idesc = tc_idesc(format, 1, 1, kTile, W);
          for (int x = terms - 1; x >= 0; --x)
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              tc_mma(tmem + R::ta, desc_of(terms0 + x * R::operand + k * 2048, kBlock),
                     desc_of(room0 + values + k * 2048, kBlock), idesc, x < terms - 1 || k > 0);
          tc_commit(&c.add_done);
        }
        __syncwarp();
        ++adds;
      }
      added = t.adds;
      if (!SUMS && t.mixed && bad && t.e0 < t.n) {
        m.seek(t.p + t.e0, lane);  // the others were told by the same word that the tile ends there
        following = find(t.p + t.e0, false);
      }
      if (!SUMS && !wait(&c.out_done, i, c)) break;
      if (t.adds && !wait(&c.add_done, adds - 1, c)) break;
      if (!SUMS && __builtin_expect(bad, 0)) {  // outputs before such a value again, without it and what follows
        uint32_t places[4] = {0, 0, 0, 0};
        where(places, values);
        if (!wait(&c.out_read, i, c)) break;
        bool ok = true;
        for (int n = t.mixed ? t.e0 : t.n; ok && n > 0;) {
          n = last_before(places, n);
          tc_after_sync();
          if (n > 0) drop(n, values);
          if (lane == 0) {
            c.again = n;
            bar_arrive(&c.again_done);
            if (n == 0) bar_arrive(&c.again_done);
          }
          if (n > 0) {
            multiply(values, &c.again_done);
            ok = wait(&c.again_read, reads++, c);
          }
        }
        if (!ok) break;
      }
    }
    // (after a wait that gave up, copies in flight have time to land)
    if (*(volatile int32_t*)&c.dead && copies) mbar_wait(&c.full, (copies - 1) & 1, 1 << 16);
  } else {
    Worker<DT, W, SUMS> w = {a, ps, c, raw, room, tmem, warp, lane, warp & 3, warp >> 2, (warp & 3) * 32 + lane, head};
    w.slope = decay * kLog2e > 1e30f ? 1e30f : decay * kLog2e;
#pragma unroll
    for (int j = 0; j < w.kCols; ++j) w.s[j] = 0.f;
    const float* carried = ps.carry + ((int64_t)head * a.runs + run - 1) * W * W;
    const int64_t matrix = (int64_t)a.d * a.d;
    if (SUMS && began && ps.in) w.read(ps.in + (sequence * a.H + head) * matrix, a.d, ps.in_turned);
    uint32_t adds = 0;
    for (uint32_t i = 0;; ++i) {
      if (!wait(&c.known[i & 1], i >> 1, c)) break;
      const Tile& t = c.tile[i & 1];
      if (t.p < 0) break;
      if (a.piece) {
        // rows of the tile's own places
        const int r0 = ps.back ? kTile - t.n : 0, r1 = r0 + t.n, thread = warp * 32 + lane;
        const int64_t first = ps.back ? a.N - t.p - t.n : t.p;
        load_rows<W>(room + R::k, ps.k + head * ps.hk, ps.sk, first, r0, r1, a.d, a.piece, thread);
        if (!SUMS) load_rows<W>(room + R::q, ps.q + head * ps.hq, ps.sq, first, r0, r1, a.d, a.piece, thread);
        load_rows<W>(room + R::v, ps.v + head * ps.hv, ps.sv, first, r0, r1, a.d, a.piece, thread);
        cp_commit();
        cp_wait<0>();
        to_products();
        w.arrive(&c.full);
      }
      const bool fresh = !SUMS && t.live && (t.begins || i == 0);  // a state comes from memory
      if (!SUMS) {
        if (t.begins) {
          if (ps.in) w.read(ps.in + (t.sequence * a.H + head) * matrix, a.d, ps.in_turned);
          else {
#pragma unroll
            for (int j = 0; j < w.kCols; ++j) w.s[j] = 0.f;
          }
        } else if (i == 0 && t.live) {
#pragma unroll
          for (int j = 0; j < w.kCols; ++j) w.s[j] = w.holds() ? __ldcg(carried + (int64_t)w.row * W + w.half * w.kCols + j) : 0.f;
        }
      }
      int n = t.n;
      // (sums take all values of their own places)
      if (!SUMS || t.mixed || t.adds) {
        if (!wait(&c.full, i, c)) break;
      }
      if ((!SUMS || t.mixed) &&
          __any_sync(kFull, not_finite<DT, W, 32 * kWarps>(room + values_at<W, SUMS>(a.piece, i), warp * 32 + lane)) && lane == 0)
        c.bad[i & 1] = 1;
      int up_keys = 0, up = 0;
      if (DT == TBE_F16 && t.adds && !w.room_for_keys(n, up_keys)) break;
      if (!SUMS) {
        if (!wait(&c.products, i, c)) break;
        tc_after_sync();
        if (!w.weigh_products(t, n, i, up)) break;
        if (fresh && !w.publish()) break;  // (its loads have had time)
      }
      // (while the products of the values go on)
      if (t.adds) w.weigh_keys(n, terms, up_keys);
      const float read_scale = w.read_scale;
      if (t.adds) {
        if (!wait(&c.add_done, adds++, c)) break;
        tc_after_sync();
        w.add(n, DT == TBE_F16 ? pow2(-up_keys) : 1.f);
        if (t.leaves) {
          if (!w.publish()) break;
        } else if (!SUMS) {
          w.write(ps.out + (t.sequence * a.H + head) * matrix, a.d);
        }
      }
      if (!SUMS) {
        if (!wait(&c.out_done, i, c)) break;
        tc_after_sync();
        const bool bad = *(volatile int32_t*)&c.bad[i & 1];
        if (t.mixed && bad) n = t.e0;
        w.write_outputs(t, n, up, read_scale, &c.out_read);
        if (__builtin_expect(bad, 0)) {  // again, as often as the product is taken
          uint32_t passes = c.passes[warp];
          bool ok;
          while ((ok = wait(&c.again_done, passes++, c)) && (n = *(volatile int32_t*)&c.again) > 0) {
            tc_after_sync();
            w.write_outputs(t, n, up, read_scale, &c.again_read);
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) c.passes[warp] = passes;
          __syncwarp();
        }
      }
    }
    if (SUMS && w.holds()) w.write(ps.carry + ((int64_t)head * a.runs + run) * W * W, W);
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (threadIdx.x == 0 && c.dead) report(a.status, TBE_DEV_TIMEOUT);
  if (warp == kWarps) tc_free(tmem, R::cols);
}

// carry[run] = what run `run` leaves, with what came through it.
template <int W>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a) {
  wait_predecessor();
  const Pass ps = a.pass[blockIdx.y];
  constexpr int kPerHead = W * W / 256;
  const int head = blockIdx.x / kPerHead, at = blockIdx.x % kPerHead * 256 + threadIdx.x;
  const float through = power(a.decay[head], a.run);
  float* c = ps.carry + (int64_t)head * a.runs * W * W + at;
  float s = 0.f;
  constexpr int kAhead = 16;
#pragma unroll 1
  for (int r = 0; r < a.runs - 1; r += kAhead) {
    // All loads are under way before the first is used.  The kinds come through the L1: every warp of the kernel reads
    // the same few, and past it they would all queue at one slice of the L2 (20 us for 36 runs).
    float x[kAhead];
    int32_t kind[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {  // what is not there is read from the last run, and not used
      const int64_t at_run = min(r + k, a.runs - 2);
      asm volatile("ld.global.ca.s32 %0, [%1];" : "=r"(kind[k]) : "l"(ps.kind + at_run));
      asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(x[k]) : "l"(c + at_run * (W * W)));
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool through_it = kind[k] == kThrough;
      s = through_it ? fmaf(through, s, x[k]) : x[k];
      if (through_it && r + k < a.runs - 1) c[(int64_t)(r + k) * (W * W)] = s;
    }
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
constexpr int kStepCols = 64;  // of a block

// A block per sequence, head and 64 value columns, 16 lanes to a row of them
// and the rows in turn to 16 half-warps.  Bound by memory: the state is read
// and written once.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const StepArgs a) {
  constexpr int kRows = kStepThreads / 16;
  __shared__ float q[128], k[128];
  __shared__ float4 part[kRows][16];
  const int parts = (a.d + kStepCols - 1) / kStepCols;
  const int64_t matrix = blockIdx.x / parts, s = matrix / a.H;
  const int head = (int)(matrix % a.H), c = blockIdx.x % parts * kStepCols + threadIdx.x % 16 * 4, r0 = threadIdx.x / 16;
  const int d = a.d;
  for (int i = threadIdx.x; i < d; i += kStepThreads) {
    q[i] = to_float<DT>(a.q[s * a.sq + head * a.hq + i]) * a.scale;
    k[i] = to_float<DT>(a.k[s * a.sk + head * a.hk + i]);
  }
  const float gamma = power(a.decay[head], 1);
  float* m = a.state + matrix * d * d;
  float v[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = c + e < d ? to_float<DT>(a.v[s * a.sv + head * a.hv + c + e]) : 0.f;
  float x[128 / kRows][4];  // this lane's part of the state
#pragma unroll
  for (int n = 0; n < 128 / kRows; ++n) {
    const int i = r0 + n * kRows;
    const float* at = m + (int64_t)i * d + c;
    if (VEC) {
      const float4 y = i < d && c < d ? *reinterpret_cast<const float4*>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[n][0] = y.x;
      x[n][1] = y.y;
      x[n][2] = y.z;
      x[n][3] = y.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] = i < d && c + e < d ? at[e] : 0.f;
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < 128 / kRows; ++n) {
    const int i = r0 + n * kRows;
    if (i >= d) break;
    float* at = m + (int64_t)i * d + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[n][e] = fmaf(k[i], v[e], gamma * x[n][e]);
      o[e] = fmaf(q[i], x[n][e], o[e]);
    }
    if (VEC) {
      if (c < d) *reinterpret_cast<float4*>(at) = make_float4(x[n][0], x[n][1], x[n][2], x[n][3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < d) at[e] = x[n][e];
    }
  }
  part[r0][threadIdx.x % 16] = make_float4(o[0], o[1], o[2], o[3]);
  __syncthreads();
  const int col = blockIdx.x % parts * kStepCols + threadIdx.x;
  if (threadIdx.x < kStepCols && col < d) {
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) sum += reinterpret_cast<const float*>(part[r])[threadIdx.x];
    a.o[s * a.so + head * a.ho + col] = (uint16_t)pack2<DT>(sum, 0.f);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int width_of(int32_t d) { return d <= 64 ? 64 : 128; }

// Runs: as many blocks as the GPU holds at once.
struct Split {
  int32_t run, runs;
};
Split split_of(int64_t N, int32_t H, int32_t d, int passes) {
  const int64_t tiles = (N + kTile - 1) / kTile;
  const int64_t want = std::max<int64_t>(1, (width_of(d) == 64 ? kBlocks<64> : kBlocks<128>) * (int64_t)sm_count() / ((int64_t)H * passes));
  const int64_t each = std::max<int64_t>(1, (tiles + want - 1) / want);
  Split s;
  s.run = (int32_t)std::min<int64_t>(each * kTile, 1 << 30);
  s.runs = (int32_t)std::max<int64_t>(1, (N + s.run - 1) / s.run);
  return s;
}
struct Layout {
  size_t carry, kind, bytes;  // of a pass
};
Layout layout(int64_t N, int32_t H, int32_t d, int passes) {
  const Split sp = split_of(N, H, d, passes);
  Layout w = {0, 0, 0};
  if (sp.runs > 1) {
    const size_t wide = width_of(d);
    w.kind = round256(sizeof(float) * (size_t)H * sp.runs * wide * wide);
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

template <int DT, int W>
int launch(Args& a, int passes, cudaStream_t s) {
  const void *sums = (const void*)attention_kernel<DT, W, true>, *outputs = (const void*)attention_kernel<DT, W, false>;
  a.terms = 2;
  for (int p = 0; p < passes; ++p)
    if (DT == TBE_BF16 && a.pass[p].out) a.terms = 3;
  const size_t smem = Room<W>::bytes(a.terms) + sizeof(Control);
  static_assert(Room<W>::bytes(3) + sizeof(Control) <= 227 * 1024 / kBlocks<W> - (kBlocks<W> > 1 ? 1024 : 0), "fits an SM");
  static bool allowed[64] = {};  // once per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !allowed[dev]) {
    for (const void* f : {sums, outputs})
      if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, Room<W>::bytes(3) + (int)sizeof(Control)) != cudaSuccess)
        return TBE_ERR_CUDA;
    if (dev >= 0 && dev < 64) allowed[dev] = true;
  }
  int st;
  if (a.runs > 1) {
    if ((st = start(sums, dim3((unsigned)(a.runs - 1) * a.H, passes), kThreads, smem, false, s, a)) != TBE_OK) return st;
    trace_mark(s, "linear_attention_sums");
    if ((st = start((const void*)join_kernel<W>, dim3((unsigned)a.H * (W * W / 256), passes), 256, 0, true, s, a)) != TBE_OK) return st;
    trace_mark(s, "linear_attention_join");
  }
  st = start(outputs, dim3((unsigned)a.runs * a.H, passes), kThreads, smem, a.runs > 1, s, a);
  trace_mark(s, "linear_attention_output");
  return st;
}

template <int DT>
int dispatch(Args& a, int passes, cudaStream_t s) {
  return width_of(a.d) == 64 ? launch<DT, 64>(a, passes, s) : launch<DT, 128>(a, passes, s);
}

// Bytes (2 to `most`) that rows of d elements can be moved by.
int piece_of(const void* p, int64_t stride, int64_t head, int32_t d, int most) {
  int n = most;
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
  a.run = sp.run;
  a.runs = sp.runs;
  a.status = status;
  return a;
}

// The tensor maps of up to kMaxMaps row sets; where one cannot be copied so
// (its rows must start on 16 bytes), none is.
struct Maps {
  Rows r[kMaxMaps];
  int n = 0;
  int of(const Rows& x) {
    r[n] = x;
    return n++;
  }
  // (a stride that nothing is reached by need not be one that tensor copies take)
  static int64_t token_stride(const Args& a, const Rows& x) { return a.N > 1 ? x.stride : 128; }
  static int64_t head_stride(const Args& a, const Rows& x) { return a.H > 1 ? x.head : 128; }
  int fill(Args& a, int32_t dtype) const {
    a.piece = 16;
    bool copies = a.N < (int64_t(1) << 31) - kTile;
    for (int i = 0; i < n; ++i) {
      copies &= piece_of(r[i].p, token_stride(a, r[i]), head_stride(a, r[i]), 8, 16) == 16;
      a.piece = std::min(a.piece, piece_of(r[i].p, r[i].stride, r[i].head, a.d, 16));
    }
    if (!copies) return TBE_OK;
    a.piece = 0;
    for (int i = 0; i < n; ++i) {
      const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.H, (cuuint64_t)a.N};
      const cuuint64_t strides[2] = {(cuuint64_t)head_stride(a, r[i]) * 2, (cuuint64_t)token_stride(a, r[i]) * 2};
      const cuuint32_t box[3] = {64, 1, kTile}, one[3] = {1, 1, 1};
      if (!encode_map(&a.map[i], dtype, 3, r[i].p, dims, strides, box, one)) return TBE_ERR_CUDA;
    }
    return TBE_OK;
  }
};
void set_rows(Pass& p, const Maps& m, int q, int k, int v, const Rows& o, int32_t d) {
  p.q = static_cast<const uint16_t*>(m.r[q].p);
  p.sq = m.r[q].stride;
  p.hq = m.r[q].head;
  p.mq = q;
  p.k = static_cast<const uint16_t*>(m.r[k].p);
  p.sk = m.r[k].stride;
  p.hk = m.r[k].head;
  p.mk = k;
  p.v = static_cast<const uint16_t*>(m.r[v].p);
  p.sv = m.r[v].stride;
  p.hv = m.r[v].head;
  p.mv = v;
  p.o = static_cast<uint16_t*>(const_cast<void*>(o.p));
  p.so = o.stride;
  p.ho = o.head;
  p.piece_o = piece_of(o.p, o.stride, o.head, d, 32);
}

// The memory of rows, by tokens of heads or heads of tokens.
Region region_of(const Rows& r, const tbe_linear_attention_inputs* in) {
  const int64_t N = in->tokens, H = in->heads, d = in->head_dim;
  const Region tokens = {(intptr_t)r.p, 2 * d, N, 2 * r.stride, H, 2 * r.head};
  const Region heads = {(intptr_t)r.p, 2 * d, H, 2 * r.head, N, 2 * r.stride};
  return N <= 1 || (H > 1 && r.stride < r.head * (H - 1) + d) ? heads : tokens;
}
Region states_of(const float* p, const tbe_linear_attention_inputs* in) {
  return bytes_of(p, (int64_t)sizeof(float) * in->sequences * in->heads * in->head_dim * in->head_dim);
}
// Whether an output shares memory with an input (`more` of them beside those of `in`) or another output: blocks read
// the one while others write the other.
bool overlap(const tbe_linear_attention_inputs* in, const Region* more, int inputs, const Region* out, int outputs) {
  const int64_t entry = in->offsets_i32 ? 4 : 8;
  const Region own[6] = {region_of({in->q, in->q_stride, in->q_head_stride}, in),
                         region_of({in->k, in->k_stride, in->k_head_stride}, in),
                         region_of({in->v, in->v_stride, in->v_head_stride}, in),
                         bytes_of(in->decay, (int64_t)sizeof(float) * in->heads),
                         bytes_of(in->offsets, in->offsets ? entry * ((int64_t)in->sequences + 1) : 0),
                         states_of(in->s0, in)};
  for (int i = 0; i < outputs; ++i) {
    for (const Region& r : own)
      if (share(out[i], r)) return true;
    for (int k = 0; k < inputs; ++k)
      if (share(out[i], more[k])) return true;
    for (int k = 0; k < i; ++k)
      if (share(out[i], out[k])) return true;
  }
  return false;
}

int go(Args& a, const Maps& maps, int passes, int32_t dtype, void* workspace, size_t bytes, cudaStream_t s) {
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
  if ((int64_t)a.runs * a.H >= (int64_t(1) << 31)) return TBE_ERR_UNSUPPORTED;
  trace_begin(s);
  if (a.N > 0) {
    int st = maps.fill(a, dtype);
    if (st == TBE_OK) st = dtype == TBE_F16 ? dispatch<TBE_F16>(a, passes, s) : dispatch<TBE_BF16>(a, passes, s);
    if (st != TBE_OK) return st;
  }
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
  const Region written[2] = {region_of(out, in), states_of(s_last, in)};
  if (overlap(in, nullptr, 0, written, 2)) return TBE_ERR_INVALID_ARG;
  if (in->sequences == 0) return TBE_OK;
  Args a = args_of(in, 1, dev_status);
  Pass& p = a.pass[0];
  Maps maps;
  const int q = maps.of({in->q, in->q_stride, in->q_head_stride}), k = maps.of({in->k, in->k_stride, in->k_head_stride}),
            v = maps.of({in->v, in->v_stride, in->v_head_stride});
  set_rows(p, maps, q, k, v, out, a.d);
  p.in = in->s0;
  p.out = s_last;
  p.scale_tile = p.scale_read = in->scale;
  p.scale_add = 1.f;
  return go(a, maps, 1, in->dtype, workspace, workspace_bytes, (cudaStream_t)stream);
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
  const Region read[2] = {region_of(d, in), states_of(ds_last, in)};
  const Region written[4] = {region_of(dq, in), region_of(dk, in), region_of(dv, in), states_of(g->ds0, in)};
  if (overlap(in, read, 2, written, 4)) return TBE_ERR_INVALID_ARG;
  if (in->sequences == 0) return TBE_OK;
  Args a = args_of(in, 3, dev_status);
  Maps maps;
  const int mq = maps.of(q), mk = maps.of(k), mv = maps.of(v), md = maps.of(d);
  set_rows(a.pass[0], maps, md, mv, mk, dq, a.d);
  a.pass[0].in = in->s0;
  a.pass[0].in_turned = 1;
  a.pass[0].scale_tile = a.pass[0].scale_read = in->scale;
  a.pass[0].scale_add = 1.f;
  set_rows(a.pass[1], maps, mv, md, mq, dk, a.d);
  a.pass[1].in_turned = 1;
  set_rows(a.pass[2], maps, mk, mq, md, dv, a.d);
  a.pass[2].out = g->ds0;
  for (int i = 1; i < 3; ++i) {
    a.pass[i].in = ds_last;
    a.pass[i].back = 1;
    a.pass[i].scale_tile = a.pass[i].scale_add = in->scale;
    a.pass[i].scale_read = 1.f;
  }
  return go(a, maps, 3, in->dtype, workspace, workspace_bytes, (cudaStream_t)stream);
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
  const Region written[2] = {region_of(out, in), states_of(state, in)};
  tbe_linear_attention_inputs read = *in;  // (offsets are not)
  read.offsets = nullptr;
  if (overlap(&read, nullptr, 0, written, 2)) return TBE_ERR_INVALID_ARG;
  const int64_t blocks = (int64_t)in->sequences * in->heads * ((in->head_dim + kStepCols - 1) / kStepCols);
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
    if (vec) step_kernel<TBE_F16, true><<<grid, kStepThreads, 0, s>>>(a);
    else step_kernel<TBE_F16, false><<<grid, kStepThreads, 0, s>>>(a);
  } else {
    if (vec) step_kernel<TBE_BF16, true><<<grid, kStepThreads, 0, s>>>(a);
    else step_kernel<TBE_BF16, false><<<grid, kStepThreads, 0, s>>>(a);
  }
  const int rc = check_launch();
  trace_mark(s, "linear_attention_step");
  return rc;
}

}  // extern "C"
