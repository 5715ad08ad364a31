// tbe_catalogue.cu -- softmax cross entropy of hidden rows over every row of
// a catalogue's table, with both gradients, without keeping the logits.
//
//   x[n, v] = logit_scale (hidden_n . weights_v)      lse_n = log sum_v exp(x[n, v])
//   loss    = mean over taken tokens of lse_n - x[n, y_n]
//   g[n, v] = exp(x[n, v] - lse_n) - [v = y_n]
//   dhidden = f g weights      dweights = f g^T hidden      f = grad_scale logit_scale / taken
//
// Four products of tokens x vocab x width, all on the tensor cores: the
// logits twice (for the log-sums, then for g) and one for each gradient.  g
// goes through memory in 16 bits, a piece of the vocabulary at a time, in two
// buffers in turn: one launch makes the g of a piece and multiplies the piece
// before it, so that its long tiles and its short ones fill each other's gaps.
// The logits themselves never leave the chip.
//
// Tokens without a label are left out first: the rows of the others are
// copied together, in order, so that neither their products nor what stands
// in their rows takes part.
//
// g is rounded to the operands' type before the second products (half a step,
// 2^-9 of each term for bf16, 2^-12 for fp16, where it is held 2^14 times
// larger so that probabilities down to 4e-9 are normal numbers).  The label's
// entry is exp(-loss) - 1, made from the token's loss: where a token is nearly
// learnt, a difference of 1 and a probability would keep little of it.  Products are exact and
// summed in fp32; dhidden is summed over the pieces in fp32.
//
// What bounds it: the tensor cores where the width is 512 or more (64 % of
// their cycles under ncu), the exponentials and what stands around them below
// (a tile of 256 x 256 costs 3,900 cycles beside its products, 2,050 of them the
// rate of ex2).  8,192 x 100,000 x 512 bf16, 9 in 10 tokens taken: 2,250 us with
// gradients, 1,341 TFLOP/s over the four products (a library's product of 8192^3
// 1,938); every token taken, the loss alone 554 us, 1,514 TFLOP/s.  On the way
// there: 128 x 256 tiles, 4 stages, 4,087 us; 256 x 256 tiles to a pair of blocks
// 3,372; one copy of 16 KB where there were two of 8, and arrivals that order
// nothing, 2,560; tiles given out by a thread of their own, when they are wanted,
// 2,384; larger pieces 2,291; jobs in shared memory 2,262.
// 64 rows over 1,000,003 x 128 take 71 us where the table's bytes take 38: with
// the table's rows as the product's every warp has exponentials to take, and a
// tile's 64 KB wait for its 512 cycles of products and the copies' latency.
#include "tbe_overlap.cuh"
#include "tbe_tensor.cuh"

#include <algorithm>
#include <cmath>

namespace tbe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMost = 3.4028235e38f;  // offsets of exponentials stay finite: that of a logit of +inf is then +inf

__device__ __forceinline__ void wait_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------------------
// which tokens take part
// ---------------------------------------------------------------------------

constexpr int kPickThreads = 1024;

struct PickArgs {
  const int64_t* labels;
  int64_t N;
  int64_t Np;      // N in whole tiles
  int32_t V;
  int32_t* rows;   // [N] token of each row taken
  int32_t* label;  // [Np] its label, -1 behind the last
  float* lse2;     // [Np] set to +inf (nothing) behind the last
  int32_t* count;
  uint32_t* zero;  // counters of the launches that follow
  int32_t zeros;
  float* token_loss;  // [N] 0 for tokens not taken, or null
  float* lse;         // [N], or null
  float* loss;        // 0 where no token is taken, or null
  const float* given;  // [N] the log-sums of an earlier call (lse2 is made from them), or null
  const float* given_loss;  // [N] its losses (own is made from them), or null
  float* own;               // [Np]
  int32_t* status;
};

// The label's entry of g, p - 1, from the token's loss: with p near 1 the difference would keep little of it.
__device__ __forceinline__ float own_of(float loss) { return expm1f(-loss); }

__device__ __forceinline__ bool taken(int64_t y, int32_t V) { return y >= 0 && y < V; }

// One block: each warp counts a stretch of tokens, then writes its rows behind
// those of the warps before it.  The order is the tokens', so sums are the
// same in every run.
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const PickArgs a) {
  __shared__ int32_t sum[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t each = (a.N + 1023) / 1024 * 32, begin = min(a.N, each * warp), end = min(a.N, begin + each);
  int32_t mine = 0;
  bool bad = false;
  for (int64_t n = begin; n < end; n += 32) {
    const int64_t y = n + lane < end ? a.labels[n + lane] : -1;
    mine += __popc(__ballot_sync(kFull, taken(y, a.V)));
    bad |= y >= a.V;
  }
  if (bad) report(a.status, TBE_DEV_BAD_INDEX);
  if (lane == 0) sum[warp] = mine;
  __syncthreads();
  int32_t at = 0, total = 0;
  for (int w = 0; w < 32; ++w) {
    at += w < warp ? sum[w] : 0;
    total += sum[w];
  }
  for (int64_t n = begin; n < end; n += 32) {
    const int64_t i = n + lane, y = i < end ? a.labels[i] : -1;
    const bool in = taken(y, a.V);
    const unsigned m = __ballot_sync(kFull, in);
    if (in) {
      const int32_t k = at + __popc(m & ((1u << lane) - 1));
      a.rows[k] = (int32_t)i;
      a.label[k] = (int32_t)y;
      if (a.given) a.lse2[k] = a.given[i] * kLog2e;
      if (a.given_loss) a.own[k] = own_of(a.given_loss[i]);
    } else if (i < end && a.lse) {
      a.lse[i] = 0.f;
      a.token_loss[i] = 0.f;
    }
    at += __popc(m);
  }
  for (int64_t k = total + threadIdx.x; k < a.Np; k += kPickThreads) {
    a.label[k] = -1;
    a.lse2[k] = INFINITY;
  }
  for (int k = threadIdx.x; k < a.zeros; k += kPickThreads) a.zero[k] = 0;
  if (threadIdx.x == 0) {
    *a.count = total;
    if (a.loss && total == 0) *a.loss = 0.f;
  }
}

// ---------------------------------------------------------------------------
// rows copied together
// ---------------------------------------------------------------------------

struct CopyArgs {
  const uint16_t* src;
  int64_t src_stride;
  const int32_t* rows;   // row of each destination row, or null (the same)
  const int32_t* count;  // rows there are on the device, or null (N)
  uint16_t* dst;         // [whole tiles, Dp], zero behind the last row and column
  int64_t N, Np;
  int32_t D, Dp;
  int32_t vec;           // elements per load
  // gradients of tokens that take no part
  uint16_t* zero;
  int64_t zero_stride;
  const int64_t* labels;
  int32_t V;
};

// A warp's row: from src, or zeros.
__device__ __forceinline__ void copy_row(const CopyArgs& a, int64_t k, const uint16_t* src, int lane) {
  uint16_t* dst = a.dst + k * a.Dp;
  if (a.vec == 8) {
    for (int c = lane * 8; c < a.Dp; c += 256) {
      const uint4 v = src && c < a.D ? __ldg(reinterpret_cast<const uint4*>(src + c)) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(dst + c) = v;
    }
  } else {
    for (int c = lane * 2; c < a.Dp; c += 64) {
      const uint32_t lo = src && c < a.D ? __ldg(src + c) : 0, hi = src && c + 1 < a.D ? __ldg(src + c + 1) : 0;
      *reinterpret_cast<uint32_t*>(dst + c) = lo | hi << 16;
    }
  }
}
__device__ __forceinline__ void clear_row(const CopyArgs& a, int64_t n, int lane) {
  for (int c = lane; c < a.D; c += 32) a.zero[n * a.zero_stride + c] = 0;
}

__global__ void __launch_bounds__(256) copy_kernel(const CopyArgs a) {
  wait_predecessor();
  const int lane = threadIdx.x & 31;
  const int64_t k = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (k < a.N && a.zero && !taken(a.labels[k], a.V)) clear_row(a, k, lane);
  const int64_t count = a.count ? *a.count : a.N;
  if (k >= min(a.Np, (count + 255) / 256 * 256)) return;
  copy_row(a, k, k < count ? a.src + (a.rows ? (int64_t)a.rows[k] : k) * a.src_stride : nullptr, lane);
}

// Both steps in one launch, for batches whose labels every block can look at.
// In one and in two, the loss alone over 1,000 rows of 64 bf16: 8 tokens 16.4 and
// 18.4 us, 512 16.5 and 18.5, 2,048 18.5 and 20.5; with gradients over 10,000 rows
// 37.7 and 38.5, 46.1 and 48.2, 69.7 and 70.8 (a mask of 2,048 tokens is what a
// block keeps; past it its reading of all labels would be what takes the time).
constexpr int kFewTokens = 2048;
struct FewArgs {
  PickArgs p;
  CopyArgs c;
};
__global__ void __launch_bounds__(256) pick_copy_kernel(const FewArgs a) {
  __shared__ uint32_t mask[kFewTokens / 32];       // which of 32 tokens take part
  __shared__ int32_t first[kFewTokens / 32 + 1];   // the row of the first of them
  static_assert(kFewTokens / 32 == 64, "two groups to a lane");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int N = (int)a.p.N, groups = (N + 31) / 32;
  bool bad = false;
  for (int g = warp; g < 64; g += 8) {
    const int n = g * 32 + lane;
    const int64_t y = n < N ? a.p.labels[n] : -1;
    const uint32_t m = __ballot_sync(kFull, taken(y, a.p.V));
    bad |= y >= a.p.V;
    if (lane == 0) mask[g] = m;
  }
  if (bad && blockIdx.x == 0) report(a.p.status, TBE_DEV_BAD_INDEX);
  __syncthreads();
  if (warp == 0) {
    const int c0 = __popc(mask[2 * lane]), c1 = __popc(mask[2 * lane + 1]);
    int sum = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int below = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += below;
    }
    first[2 * lane] = sum - c0 - c1;
    first[2 * lane + 1] = sum - c1;
    if (lane == 31) first[64] = sum;
  }
  __syncthreads();
  const int total = first[64];
  if (blockIdx.x == 0) {
    for (int g = warp; g < groups; g += 8) {
      const int n = g * 32 + lane;
      if (mask[g] >> lane & 1) {
        const int k = first[g] + __popc(mask[g] & ((1u << lane) - 1));
        a.p.rows[k] = n;
        a.p.label[k] = (int32_t)a.p.labels[n];
        if (a.p.given) a.p.lse2[k] = a.p.given[n] * kLog2e;
        if (a.p.given_loss) a.p.own[k] = own_of(a.p.given_loss[n]);
      } else if (n < N && a.p.lse) {
        a.p.lse[n] = 0.f;
        a.p.token_loss[n] = 0.f;
      }
    }
    for (int k = total + threadIdx.x; k < (int)a.p.Np; k += 256) {
      a.p.label[k] = -1;
      a.p.lse2[k] = INFINITY;
    }
    for (int k = threadIdx.x; k < a.p.zeros; k += 256) a.p.zero[k] = 0;
    if (threadIdx.x == 0) {
      *a.p.count = total;
      if (a.p.loss && total == 0) *a.p.loss = 0.f;
    }
  }
  const int k = blockIdx.x * 8 + warp;
  if (k < N && a.c.zero && !(mask[k / 32] >> (k % 32) & 1)) clear_row(a.c, k, lane);
  if (k >= min((int)a.p.Np, (total + 255) / 256 * 256)) return;
  const uint16_t* src = nullptr;
  if (k < total) {
    // the group whose first row is the last one at or before k, and the token of its (k - first)th bit
    const int g = __popc(__ballot_sync(kFull, first[lane] <= k)) + __popc(__ballot_sync(kFull, first[32 + lane] <= k)) - 1;
    src = a.c.src + (int64_t)(g * 32 + (int)__fns(mask[g], 0, k - first[g] + 1)) * a.c.src_stride;
  }
  copy_row(a.c, k, src, lane);
}

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------

// What a tile multiplies and what becomes of it.
enum Mode : int32_t {
  kSums,    // logits -> their row's maximum and sum of exponentials over the tile
  kProbs,   // logits -> g of a piece
  kTable,   // g^T hidden -> rows of dweights
  kHidden,  // g weights -> fp32 sums of dhidden
};
struct Job {
  int32_t mode;
  int32_t v0, v1;   // its part of the vocabulary
  int32_t buffer;   // of g
  int32_t splits;   // kHidden: parts of the vocabulary summed apart,
  int32_t steps;    //   each of so many steps of K
  int32_t first;    // kHidden: stores instead of adding
};
constexpr int kMaxJobs = 3;

// A pair of blocks (on neighbouring SMs) takes a tile of 256 x 256: each
// holds 128 rows of A and of the accumulators, and half of B's columns, which
// the tensor cores of both read.  Against a tile of 128 x 256 to a block that
// is two thirds of the copies, which are what bounds the products here.
constexpr int kRowsM = 128;  // of a block
constexpr int kTileM = 2 * kRowsM, kTileN = 256, kTileK = 64;
constexpr int kHalfN = kTileN / 2;
constexpr int kStages = 6;
constexpr int kStageBytes = (kRowsM + kHalfN) / 64 * kBlockBytes;
constexpr int kTiles = 4;  // tiles known at once
constexpr int kAsk = 6;    // steps before the end of a tile's copies at which the next one is asked for
constexpr int kThreads = 384;
constexpr int kEpilogueWarps = 8;
constexpr uint16_t kBoth = 3;  // blocks of a pair, as a mask
constexpr int kFewRows = 64;

struct GemmArgs {
  // hidden [Np, Dp], weights [V, D] and g [2 Np, vc]: 128 rows by 64 columns (operands along K), and 64 rows by two
  // blocks of 64 columns (along M or N)
  CUtensorMap h, w, p, ht, wt, pt;
  CUtensorMap few;    // hidden in boxes of 64 rows by 64 columns
  Job job[kMaxJobs];
  int32_t jobs;
  int32_t V, D, Dp;
  int32_t half;       // blocks of 64 columns of the gradients that a block of a pair reads
  int64_t Np;
  const int32_t* count;
  uint32_t* next;     // tiles given out
  float scale2;       // logit_scale in units of log 2
  const int32_t* label;
  const float* lse2;
  const float* own;   // the label's entry of g, or null: exp(x - lse) - 1
  float* mine;        // kSums: the label's product, not scaled
  float2* part;       // kSums: [tiles along the vocabulary, Np]
  uint16_t* g;
  int32_t vc;
  uint16_t* dw;
  int64_t dw_stride;
  int32_t dw_piece;   // bytes that its rows can be written by
  float factor;       // grad_scale logit_scale / what g is multiplied by
  float* acc;         // [splits, Np, Dp]
  int32_t* status;
};

// A tile's place.
struct alignas(16) Tile {
  int32_t mode;      // -1 behind the last
  int32_t job;
  int32_t rb;        // block of kTileM rows of the product
  int32_t col;       // first column
  int32_t blocks;    // columns / 64, in whole pairs
  int32_t split, k0, steps;
};
struct Shared {
  uint64_t full[kStages], empty[kStages];   // operands
  uint64_t done[2], drained[2];             // accumulators
  uint64_t known[kTiles], forgotten[kTiles];  // tiles
  uint64_t combine[2][4];
  uint64_t ask;                             // the next tile is wanted
  Tile tile[kTiles];
  Job job[kMaxJobs];  // (a parameter's, with an index, would take hundreds of cycles to load)
  uint32_t tmem;
  int32_t dead;
  float2 half[2][kRowsM];
};

__device__ __forceinline__ int32_t column_tiles(int32_t D, int32_t half) { return (D + 128 * half - 1) / (128 * half); }
__device__ __forceinline__ int32_t tiles_of(const Job& j, int32_t mt, int32_t D, int32_t half) {
  const int32_t v = j.v1 - j.v0;
  if (j.mode <= kProbs) return mt * ((v + kTileN - 1) / kTileN);
  if (j.mode == kTable) return (v + kTileM - 1) / kTileM * column_tiles(D, half);
  return j.splits * mt * column_tiles(D, half);
}
__device__ __forceinline__ Tile tile_of(const GemmArgs& g, const Job* job, int32_t t, int32_t count) {
  const int32_t mt = (count + kTileM - 1) / kTileM;
  Tile r;
  r.job = 0;
  for (; r.job < g.jobs - 1; ++r.job) {
    const int32_t n = tiles_of(job[r.job], mt, g.D, g.half);
    if (t < n) break;
    t -= n;
  }
  const Job& j = job[r.job];
  r.mode = j.mode;
  r.split = 0;
  r.k0 = 0;
  if (r.mode <= kProbs) {
    // the rows of a column tile first: what a wave of tiles reads of the table is then little
    r.rb = t % mt;
    r.col = j.v0 + t / mt * kTileN;
    r.blocks = kTileN / 64;
    r.steps = (g.D + kTileK - 1) / kTileK;
    return r;
  }
  const int32_t ct = column_tiles(g.D, g.half);
  r.col = t % ct * (128 * g.half);
  r.blocks = 2 * g.half;
  t /= ct;
  if (r.mode == kTable) {
    r.rb = t;
    r.steps = (count + kTileK - 1) / kTileK;
  } else {
    r.rb = t % mt;
    r.split = t / mt;
    r.k0 = r.split * j.steps;
    r.steps = max(0, min(j.steps, (j.v1 - j.v0 + kTileK - 1) / kTileK - r.k0));
  }
  return r;
}

// A bounded wait: false (and the others give up too) after four seconds.
template <bool PAIR>
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int32_t* dead) {
  uint64_t begin, now;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(begin));
  for (;;) {
    if (PAIR ? pair_wait(bar, parity, 64) : mbar_wait(bar, parity, 64)) return true;
    if (*dead) return false;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
    if (now - begin > 4000000000ull) {
      *dead = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Shared& s) {
  return mbar_wait(bar, parity, 4) || wait_long<false>(bar, parity, &s.dead);
}
// (for what the other block wrote)
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, Shared& s) {
  return pair_wait(bar, parity, 4) || wait_long<true>(bar, parity, &s.dead);
}

__device__ __forceinline__ uint32_t pack2(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store32(void* p, const uint32_t* u) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
               "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}
// 32 values as 16-bit elements, the first n of them, by pieces of `piece` bytes.
template <int DT>
__device__ __forceinline__ void store_row(uint16_t* p, const float* v, int n, int piece) {
  uint32_t u[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) u[k] = pack2(v[2 * k], v[2 * k + 1], DT == TBE_BF16);
  if (n >= 32 && piece == 32) {
    store32(p, u);
    store32(p + 16, u + 8);
    return;
  }
  if (n >= 32 && piece == 16) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      reinterpret_cast<uint4*>(p)[k] = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    if (piece >= 4 && 2 * k + 1 < n) {
      reinterpret_cast<uint32_t*>(p)[k] = u[k];
    } else {
      if (2 * k < n) p[2 * k] = (uint16_t)u[k];
      if (2 * k + 1 < n) p[2 * k + 1] = (uint16_t)(u[k] >> 16);
    }
  }
}

// What g is multiplied by, as a power of two.
template <int DT>
constexpr int kUp = DT == TBE_F16 ? 14 : 0;

// (a, b) * s + c
__device__ __forceinline__ void fma2(float& a, float& b, float s, float c) {
  asm("{\n\t.reg .b64 p, q, r;\n\t"
      "mov.b64 p, {%0, %1};\n\t"
      "mov.b64 q, {%2, %2};\n\t"
      "mov.b64 r, {%3, %3};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(s), "f"(c));
}
// 2^x to 2^-22 of its size, 0 for the lowest.
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// v[0 .. 31] = 2^(v s + c)
__device__ __forceinline__ void exps(float (&v)[32], float s, float c) {
#pragma unroll
  for (int k = 0; k < 32; k += 2) fma2(v[k], v[k + 1], s, c);
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = exp2_of(v[k]);
}

// A thread's columns of the accumulators, 32 at a time (64 is a divisor of
// their number), the next 32 on their way while these are worked on: calls
// f(values, first column).
template <typename F>
__device__ __forceinline__ void each_chunk(uint32_t tmem, int begin, int end, F& f) {
  if (begin >= end) return;
  float a[32], b[32];
  tc_ld32(tmem + begin, a);
#pragma unroll 1
  for (int c = begin; c < end; c += 64) {
    tc_wait_ld();
    tc_ld32(tmem + c + 32, b);
    f(a, c);
    tc_wait_ld();
    if (c + 64 < end) tc_ld32(tmem + c + 64, a);
    f(b, c + 32);
  }
}

// What becomes of 32 columns of a row, by the tile's mode.
struct SumsOf {
  const GemmArgs& g;
  const Tile& t;
  int64_t r;
  int32_t label;
  bool edge, down;
  float m, l;
  __device__ __forceinline__ void operator()(float (&v)[32], int c) {
    const int32_t col = t.col + c;
    const bool own = (uint32_t)(label - col) < 32u;
    if (own) {
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < 32; ++k) x = k == label - col ? v[k] : x;
      g.mine[r] = x;
    }
    if (edge) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (col + k >= g.V) v[k] = down ? INFINITY : -INFINITY;
    }
    float top = v[0];
    if (down) {
#pragma unroll
      for (int k = 1; k < 32; ++k) top = fminf(top, v[k]);
    } else {
#pragma unroll
      for (int k = 1; k < 32; ++k) top = fmaxf(top, v[k]);
    }
    top = fmaxf(m, g.scale2 == 0.f ? 0.f : fminf(top * g.scale2, kMost));
    const float to = top == -INFINITY ? 0.f : top;
    l *= exp2_of(m - to);
    exps(v, g.scale2, -to);
    if (edge) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (col + k >= g.V) v[k] = 0.f;
    }
    if (own) {  // (row_kernel adds the label's)
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = k == label - col ? 0.f : v[k];
    }
    float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      add2(add[0], add[1], v[k], v[k + 1]);
      add2(add[2], add[3], v[k + 2], v[k + 3]);
    }
    l += (add[0] + add[1]) + (add[2] + add[3]);
    m = top;
  }
};
template <int DT>
struct ProbsOf {
  const GemmArgs& g;
  const Tile& t;
  int32_t label, v0;
  bool there, edge;
  float less;
  const float* own;
  uint16_t* dst;
  __device__ __forceinline__ void operator()(float (&v)[32], int c) {
    const int32_t col = t.col + c;
    exps(v, g.scale2, less);
    if ((uint32_t)(label - col) < 32u) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (k == label - col) v[k] = own ? *own * (float)(1 << kUp<DT>) : v[k] - (float)(1 << kUp<DT>);
    }
    if (!there || edge) {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = there && col + k < g.V ? v[k] : 0.f;
    }
    store_row<DT>(dst + (col - v0), v, 32, 32);
  }
};
template <int DT>
struct TableOf {
  const GemmArgs& g;
  const Tile& t;
  uint16_t* dst;  // or null
  float f;
  __device__ __forceinline__ void operator()(float (&v)[32], int c) {
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = t.steps > 0 ? v[k] * f : 0.f;
    const int32_t col = t.col + c;
    if (dst && col < g.D) store_row<DT>(dst + col, v, g.D - col, g.dw_piece);
  }
};
struct HiddenOf {
  const Tile& t;
  float* dst;
  bool first;
  __device__ __forceinline__ void operator()(float (&v)[32], int c) {
    if (t.steps == 0) {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = 0.f;
    }
    if (first) {
#pragma unroll
      for (int k = 0; k < 32; k += 8) {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(v[k + e]);
        store32(dst + c + k, u);
      }
    } else {  // no other tile adds to these: the order of the sums is that of the launches
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        asm volatile("red.global.add.v4.f32 [%0], {%1,%2,%3,%4};" ::"l"(dst + c + k), "f"(v[k]), "f"(v[k + 1]),
                     "f"(v[k + 2]), "f"(v[k + 3])
                     : "memory");
    }
  }
};

template <int DT>
__device__ __forceinline__ bool epilogue(const GemmArgs& g, Shared& s, const Tile& t, uint32_t tmem, int32_t count,
                                         int half, int row, uint32_t rank, uint32_t& turn) {
  const Job& j = s.job[t.job];
  const int64_t r = (int64_t)t.rb * kTileM + rank * kRowsM + row;
  const int begin = half * kHalfN, end = min(begin + kHalfN, t.blocks * 64);
  const bool edge = t.col + kTileN > g.V;
  // Rows behind the last need no log-sum, and no g but those that a step of K takes with the last.
  const int64_t warp_r = r - (row & 31);
  if (t.mode == kSums) {
    if (warp_r >= count) return true;
    SumsOf f = {g, t, r, g.label[r], edge, g.scale2 < 0.f, -INFINITY, 0.f};
    each_chunk(tmem, begin, end, f);
    // the two halves of the columns meet
    if (half == 1) {
      s.half[turn & 1][row] = make_float2(f.m, f.l);
      __syncwarp();
      if ((row & 31) == 0) bar_arrive(&s.combine[turn & 1][row / 32]);
      ++turn;
      return true;
    }
    if (!wait(&s.combine[turn & 1][row / 32], turn >> 1 & 1, s)) return false;
    const float2 o = s.half[turn & 1][row];
    ++turn;
    const float top = fmaxf(f.m, o.x), to = top == -INFINITY ? 0.f : top;
    if (r < count) g.part[(int64_t)((t.col - j.v0) / kTileN) * g.Np + r] =
        make_float2(top, f.l * exp2_of(f.m - to) + o.y * exp2_of(o.x - to));
  } else if (t.mode == kProbs) {
    if (warp_r >= (count + kTileK - 1) / kTileK * kTileK) return true;
    ProbsOf<DT> f = {g, t, g.label[r], j.v0, r < count, edge, (float)kUp<DT> - g.lse2[r],
                     g.own ? g.own + r : nullptr, g.g + ((int64_t)j.buffer * g.Np + r) * g.vc};
    each_chunk(tmem, begin, end, f);
  } else if (t.mode == kTable) {
    const int64_t row_v = j.v0 + r;
    TableOf<DT> f = {g, t, row_v < j.v1 ? g.dw + row_v * g.dw_stride : nullptr, g.factor / (float)max(count, 1)};
    each_chunk(tmem, begin, end, f);
  } else if (t.steps > 0 || j.first) {
    HiddenOf f = {t, g.acc + ((int64_t)t.split * g.Np + r) * g.Dp + t.col, j.first != 0};
    each_chunk(tmem, begin, min(end, g.Dp - t.col), f);
  }
  return true;
}

// Few tokens over many rows: the table's rows are the product's rows and the
// tokens its columns, 32 to a thread, which keeps their log-sums over all of
// its tiles: a tile of 256 rows of hidden would be mostly empty.
// (kFewRows are one block of the pair's; the other's columns are empty.)
struct FewSums {
  float m[32], l[32];
  int32_t label;  // of token first + lane, or -1
  int first;

  __device__ __forceinline__ void begin(const GemmArgs& g, int32_t count, int half, int lane) {
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      m[k] = -3e38f;  // (finite: a product of -inf adds nothing to it)
      l[k] = 0.f;
    }
    first = half * 32;
    label = first + lane < count ? g.label[first + lane] : -1;
  }
  // One row of the table, row_v, and its products.
  __device__ __forceinline__ void add(const GemmArgs& g, float (&v)[32], int64_t row_v, int32_t tile) {
    uint32_t hit = __ballot_sync(kFull, label >= 0 && label / kTileM == tile);
    while (hit) {
      const int k = __ffs((int)hit) - 1;
      hit &= hit - 1;
      if (__shfl_sync(kFull, label, k) == row_v) {
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          x = e == k ? v[e] : x;
          v[e] = e == k ? (g.scale2 < 0.f ? INFINITY : -INFINITY) : v[e];  // (row_kernel adds the label's; no scale of 0 here)
        }
        g.mine[first + k] = x;
      }
    }
    if (row_v >= g.V) return;
    float most = -INFINITY;
#pragma unroll
    for (int k = 0; k < 32; ++k) most = fmaxf(most, fmaf(v[k], g.scale2, -m[k]));
    if (most < 16.f) {  // m need not be the largest: sums of 2^16 lose nothing
#pragma unroll
      for (int k = 0; k < 32; ++k) l[k] += exp2_of(fmaf(v[k], g.scale2, -m[k]));
      return;
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float x = v[k] * g.scale2;
      if (x > m[k]) {
        const float top = fminf(x, kMost);
        l[k] = fmaf(l[k], exp2_of(m[k] - top), exp2_of(fmaf(v[k], g.scale2, -top)));
        m[k] = top;
      } else {
        l[k] += exp2_of(fmaf(v[k], g.scale2, -m[k]));
      }
    }
  }
  __device__ __forceinline__ void end(const GemmArgs& g, int32_t count, int64_t part, int lane) {
#pragma unroll 1
    for (int o = 16; o; o >>= 1) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float m2 = __shfl_xor_sync(kFull, m[k], o), l2 = __shfl_xor_sync(kFull, l[k], o);
        const float top = fmaxf(m[k], m2);
        l[k] = l[k] * exp2_of(m[k] - top) + l2 * exp2_of(m2 - top);
        m[k] = top;
      }
    }
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (lane == 0 && first + k < count) g.part[part * g.Np + first + k] = make_float2(m[k], l[k]);
  }
};

// Its tiles are all alike, and each pair takes every so manieth.
__device__ __forceinline__ Tile few_tile(const GemmArgs& g, uint32_t n, int32_t count) {
  const int32_t now = (int32_t)(blockIdx.x >> 1) + (int32_t)n * (int32_t)(gridDim.x >> 1);
  const bool there = count > 0 && now < (g.V + kTileM - 1) / kTileM;
  return Tile{there ? (int32_t)kSums : -1, 0, now, 0, 2 * kFewRows / 64, 0, 0, (g.D + kTileK - 1) / kTileK};
}

// Persistent pairs of blocks.  In each block one thread starts its copies and
// eight warps work on its finished accumulators, of which there are two; the
// first block's threads also take the tiles and issue the products of both.
template <int DT, bool FEW>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ GemmArgs g) {
  extern __shared__ __align__(1024) uint8_t raw[];
  __shared__ Shared s;
  uint8_t* ring = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = pair_rank();
  if (threadIdx.x == 0) {
    for (int k = 0; k < kStages; ++k) {
      bar_init(&s.full[k], 1);
      bar_init(&s.empty[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      bar_init(&s.done[k], 1);
      bar_init(&s.drained[k], 2 * kEpilogueWarps);
      for (int q = 0; q < 4; ++q) bar_init(&s.combine[k][q], 1);
    }
    bar_init(&s.ask, 1);
    for (int k = 0; k < kTiles; ++k) {
      bar_init(&s.known[k], 1);
      // the copier and the epilogue warps of a block, and in the first one the issuer and the other block
      bar_init(&s.forgotten[k], rank == 0 ? 3 + kEpilogueWarps : 1 + kEpilogueWarps);
    }
    s.dead = 0;
    for (int k = 0; k < kMaxJobs; ++k) s.job[k] = g.job[k];
    bars_visible();
  }
  if (warp == 2) pair_alloc(&s.tmem, 512);
  tc_before_sync();
  __syncthreads();
  pair_sync();
  tc_after_sync();
  const uint32_t tmem = s.tmem;
  wait_predecessor();
  const int32_t count = *g.count;

  if (warp == 0 && lane == 0) {
    asm volatile("fence.proxy.async;" ::: "memory");  // rows and g were written by ordinary stores
    const uint32_t full0 = pair_addr(&s.full[0], 0), ring0 = smem_u32(ring);
    uint32_t step = 0;  // steps of K so far
    for (uint32_t n = 0;; ++n) {
      if (!FEW && !wait_pair(&s.known[n % kTiles], (n / kTiles) & 1, s)) break;
      const Tile t = FEW ? few_tile(g, n, count) : s.tile[n % kTiles];
      if (t.mode < 0) break;
      if (!FEW) bar_arrive(&s.forgotten[n % kTiles]);
      const Job& j = s.job[t.job];
      const int32_t row0 = t.rb * kTileM + (int32_t)rank * kRowsM;
      const int32_t mine = t.blocks / 2;                       // B's blocks of this block
      const int32_t b_col = t.col + (int32_t)rank * mine * 64;  // its first column
      const uint32_t bytes = 2 * (2 + mine) * kBlockBytes;
      // where A and B lie along K, a step of it is 64 columns on; else 64 rows
      const bool a_along_m = t.mode == kTable, b_along_n = t.mode >= kTable;
      const CUtensorMap* a = FEW ? &g.w : a_along_m ? &g.pt : t.mode == kHidden ? &g.p : &g.h;
      const CUtensorMap* b = FEW ? &g.few : t.mode == kTable ? &g.ht : t.mode == kHidden ? &g.wt : &g.w;
      const int32_t g_row = (int32_t)(j.buffer * g.Np), a_row = t.mode == kHidden ? g_row + row0 : row0;
      const int32_t b_first = t.mode == kHidden ? j.v0 : 0;
      bool ok = true;
      const int ask_at = max(0, t.steps - kAsk);
      if (!FEW && rank == 0 && t.steps == 0) bar_arrive(&s.ask);
      for (int k = 0; k < t.steps; ++k, ++step) {
        const uint32_t at = step % kStages;
        if (!FEW && rank == 0 && k == ask_at) bar_arrive(&s.ask);
        if (step >= kStages && !(ok = wait(&s.empty[at], (step / kStages - 1) & 1, s))) break;
        if (rank == 0) bar_expect(&s.full[at], bytes);
        const uint32_t bar = full0 + at * 8, dst = ring0 + at * kStageBytes;
        const int32_t kk = (t.k0 + k) * kTileK;
        if (a_along_m) pair_load3(dst, a, g_row + kk, row0 / 64, bar);
        else pair_load(dst, a, kk, a_row, bar);
        if (b_along_n) pair_load3(dst + 2 * kBlockBytes, b, b_first + kk, b_col / 64, bar);
        else pair_load(dst + 2 * kBlockBytes, b, kk, b_col, bar);
      }
      if (!ok) break;
    }
    if (*(volatile int32_t*)&s.dead && rank == 0)  // copies in flight land before the blocks end
      for (uint32_t k = step > kStages ? step - kStages : 0; k < step; ++k)
        pair_wait(&s.full[k % kStages], (k / kStages) & 1, 1 << 14);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    uint32_t step = 0;
    for (uint32_t n = 0;; ++n) {
      if (!FEW && !wait_pair(&s.known[n % kTiles], (n / kTiles) & 1, s)) break;
      const Tile t = FEW ? few_tile(g, n, count) : s.tile[n % kTiles];
      if (t.mode < 0) break;
      if (!FEW) bar_arrive(&s.forgotten[n % kTiles]);
      if (n >= 2 && !wait(&s.drained[n & 1], (n / 2 - 1) & 1, s)) break;
      tc_after_sync();
      const uint32_t along_m = t.mode == kTable, along_n = t.mode >= kTable;
      const uint32_t idesc = tc_idesc(DT == TBE_BF16, along_m, along_n, kTileM, t.blocks * 64);
      const uint32_t a_step = (along_m ? 2048 : 32) >> 4, b_step = (along_n ? 2048 : 32) >> 4;
      bool ok = true;
      for (int k = 0; k < t.steps; ++k, ++step) {
        const uint32_t at = step % kStages;
        if (!(ok = wait(&s.full[at], (step / kStages) & 1, s))) break;
        tc_after_sync();
        const uint32_t src = smem_u32(ring) + at * kStageBytes;
        const uint64_t a = tc_desc(src), b = tc_desc(src + 2 * kBlockBytes);
#pragma unroll
        for (int i = 0; i < kTileK / 16; ++i)
          pair_mma(tmem + (n & 1) * kTileN, a + i * a_step, b + i * b_step, idesc, k > 0 || i > 0);
        pair_commit(&s.empty[at], kBoth);
      }
      if (!ok) break;
      pair_commit(&s.done[n & 1], kBoth);
    }
  } else if (!FEW && warp == 3 && lane == 0 && rank == 0) {
    // gives out tiles, to both blocks
    int32_t total = 0;
    for (int k = 0; k < g.jobs; ++k) total += tiles_of(s.job[k], (count + kTileM - 1) / kTileM, g.D, g.half);
    int32_t now = blockIdx.x >> 1;
    for (uint32_t n = 0;; ++n) {
      const uint32_t slot = n % kTiles;
      alignas(16) Tile t = {};
      t.mode = -1;
      if (n > 0) {  // (not asked for before it is wanted: the long tiles would go to few)
        if (!wait(&s.ask, (n - 1) & 1, s)) break;
        now = (int32_t)((gridDim.x >> 1) + atomicAdd(g.next, 1u));
      }
      if (now < total) t = tile_of(g, s.job, now, count);
      if (n >= kTiles && !wait_pair(&s.forgotten[slot], (n / kTiles - 1) & 1, s)) break;
      s.tile[slot] = t;
      const uint32_t other = pair_addr(&s.tile[slot], 1);
#pragma unroll
      for (int k = 0; k < 2; ++k) pair_store16(other + 16 * k, reinterpret_cast<const uint4*>(&t)[k]);
      bar_arrive(&s.known[slot]);
      pair_arrive(pair_addr(&s.known[slot], 1));
      if (now >= total) break;
    }
  } else if (!FEW && warp == 3 && lane == 0) {
    // Tells the first block what this one has read.  An arrival there that orders its reads would wait for the outputs
    // that an epilogue warp has on their way; this thread has none.
    const uint32_t forgotten0 = pair_addr(&s.forgotten[0], 0);
    for (uint32_t n = 0;; ++n) {
      const uint32_t slot = n % kTiles;
      if (!wait_pair(&s.known[slot], (n / kTiles) & 1, s) || s.tile[slot].mode < 0) break;
      if (!wait(&s.forgotten[slot], (n / kTiles) & 1, s)) break;
      pair_arrive(forgotten0 + slot * 8);
    }
  } else if (warp >= 4) {
    const int half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    uint32_t turn = 0;  // tiles of kSums that this warp had rows of
    FewSums few;
    if (FEW) few.begin(g, count, half, lane);
    for (uint32_t n = 0;; ++n) {
      if (!FEW && !wait_pair(&s.known[n % kTiles], (n / kTiles) & 1, s)) break;
      const Tile t = FEW ? few_tile(g, n, count) : s.tile[n % kTiles];
      __syncwarp();
      if (t.mode < 0) break;
      if (!FEW && lane == 0) bar_arrive(&s.forgotten[n % kTiles]);
      if (!wait(&s.done[n & 1], (n / 2) & 1, s)) break;
      tc_after_sync();
      if (FEW) {
        float v[32];
        tc_ld32(tmem + (n & 1) * kTileN + ((uint32_t)(warp & 3) * 32 << 16) + half * 32, v);
        tc_wait_ld();
        tc_before_sync();
        __syncwarp();
        if (lane == 0) pair_arrive_relaxed(pair_addr(&s.drained[n & 1], 0));
        if (half * 32 < count) few.add(g, v, (int64_t)t.rb * kTileM + rank * kRowsM + row, t.rb);
        continue;
      }
      const bool ok = epilogue<DT>(g, s, t, tmem + (n & 1) * kTileN + ((uint32_t)(warp & 3) * 32 << 16), count, half, row,
                                   rank, turn);
      if (!__all_sync(kFull, ok)) break;
      tc_before_sync();
      __syncwarp();
      if (lane == 0) pair_arrive_relaxed(pair_addr(&s.drained[n & 1], 0));
    }
    if (FEW) few.end(g, count, (int64_t)blockIdx.x * 4 + (warp & 3), lane);
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  pair_sync();  // neither leaves while the other's products, copies or arrivals are under way
  tc_after_sync();
  if (threadIdx.x == 0 && s.dead) report(g.status, TBE_DEV_TIMEOUT);
  if (warp == 2) pair_free(tmem, 512);
}

// ---------------------------------------------------------------------------
// the rows' log-sums and losses
// ---------------------------------------------------------------------------

constexpr int kRowThreads = 1024;
constexpr int kRows = 8;  // rows of a block, kRowThreads / kRows threads to each

struct RowArgs {
  const float2* part;
  int32_t parts;
  int64_t Np;
  const int32_t* count;
  const int32_t* rows;
  const float* mine;
  float scale2;
  float* lse2;
  float* own;
  float* token_loss;
  float* lse;
  float* loss;
  float* block_sum;
  uint32_t* arrived;
};

__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2), to = top == -INFINITY ? 0.f : top;
  l = l * exp2f(m - to) + l2 * exp2f(m2 - to);
  m = top;
}

__global__ void __launch_bounds__(kRowThreads) row_kernel(const RowArgs a) {
  wait_predecessor();
  __shared__ float2 part[32][kRows];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t count = *a.count;
  const int64_t row = (int64_t)blockIdx.x * kRows + (threadIdx.x & (kRows - 1));
  if ((int64_t)blockIdx.x * kRows >= count) return;
  float m = -INFINITY, l = 0.f;
  if (row < count) {
#pragma unroll 4
    for (int k = threadIdx.x / kRows; k < a.parts; k += kRowThreads / kRows) {
      const float2 p = a.part[k * a.Np + row];
      join(m, l, p.x, p.y);
    }
  }
#pragma unroll
  for (int o = 16; o >= kRows; o >>= 1) join(m, l, __shfl_xor_sync(kFull, m, o), __shfl_xor_sync(kFull, l, o));
  if (lane < kRows) part[warp][lane] = make_float2(m, l);
  __syncthreads();
  float mine = 0.f;
  if (threadIdx.x < kRows && row < count) {
    const int warps = min(32, (a.parts * kRows + 31) / 32);  // that had any
    for (int w = 1; w < warps; ++w) join(m, l, part[w][threadIdx.x].x, part[w][threadIdx.x].y);
    // The label's own term is not in l, which therefore keeps its digits where that logit stands out and the loss,
    // log(1 + l 2^-d), is close to 0.  d is how far the label's logit lies above m.
    const int32_t n = a.rows[row];
    const float x = a.mine[row], own = x * a.scale2, d = fmaf(x, a.scale2, -m);
    mine = d > -64.f ? log1pf(l * exp2f(-d)) : (log2f(l) - d) * kLn2;
    float log_sum = m + (d <= 0.f ? log2f(l + exp2f(d)) : d + log1pf(l * exp2f(-d)) * kLog2e);
    if (l == 0.f) log_sum = own;  // there is no other row, or none that reaches 2^-126 of the label's
    if (own == INFINITY) {
      mine = NAN;           // (inf - inf)
      log_sum = l + own;    // (a NaN stays one)
    }
    a.lse2[row] = log_sum;
    a.lse[n] = log_sum * kLn2;
    a.own[row] = own_of(mine);
    a.token_loss[n] = mine;
  }
  if (warp != 0) return;
  mine = warp_sum(lane < kRows ? mine : 0.f);
  const uint32_t blocks = (uint32_t)((count + kRows - 1) / kRows);
  if (lane == 0) {
    a.block_sum[blockIdx.x] = mine;
    __threadfence();
    last = atomicAdd(a.arrived, 1u) == blocks - 1;
  }
  __syncwarp();
  if (!last) return;
  __threadfence();
  float all = 0.f;
  for (uint32_t b = lane; b < blocks; b += 32) all += __ldcg(a.block_sum + b);
  all = warp_sum(all);
  if (lane == 0) *a.loss = all / (float)count;
}

// ---------------------------------------------------------------------------
// dhidden
// ---------------------------------------------------------------------------

struct SpreadArgs {
  const float* acc;
  int32_t splits;
  int64_t Np;
  int32_t D, Dp;
  const int32_t* count;
  const int32_t* rows;
  float factor;
  uint16_t* out;
  int64_t stride;
  int32_t pairs;  // rows can be written by pairs
};

template <int DT>
__global__ void __launch_bounds__(256) spread_kernel(const SpreadArgs a) {
  wait_predecessor();
  const int lane = threadIdx.x & 31;
  const int64_t k = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int32_t count = *a.count;
  if (k >= count) return;
  const float f = a.factor / (float)count;
  uint16_t* out = a.out + (int64_t)a.rows[k] * a.stride;
  for (int c = lane * 2; c < a.D; c += 64) {
    float2 sum = make_float2(0.f, 0.f);
    for (int p = 0; p < a.splits; ++p) {
      const float2 v = __ldg(reinterpret_cast<const float2*>(a.acc + ((int64_t)p * a.Np + k) * a.Dp + c));
      sum.x += v.x;
      sum.y += v.y;
    }
    const uint32_t u = pack2(sum.x * f, sum.y * f, DT == TBE_BF16);
    if (a.pairs && c + 1 < a.D) {
      *reinterpret_cast<uint32_t*>(out + c) = u;
    } else {
      out[c] = (uint16_t)u;
      if (c + 1 < a.D) out[c + 1] = (uint16_t)(u >> 16);
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int64_t whole(int64_t n, int64_t of) { return (n + of - 1) / of * of; }

// Elements of a piece's g.  With 2^24, 2^25, 2^26 and 2^27: 8,192 x 100,000 x
// 512 bf16 with gradients 3,115, 2,384, 2,291, 2,249 us; 4,001 x 10,007 x 256 156,
// 144, 127, 126 us; 512 x 150,000 x 128 205, 197, 207, 186 us.  Two buffers of 128
// MB each, that is; 2^27 would take as much memory again for 1 to 10 %.
constexpr int64_t kPiece = 1 << 26;
constexpr int64_t kMaxTokens = 1 << 24;
// The table's rows as the product's, from so many on: the loss alone over 10,000,
// 20,000, 40,000, 100,000 and 400,000 rows, so and with the tokens as rows:
//   1 token, width 64:    18.6 18.6 18.6 20.6 28.9   16.2 18.5 20.7 27.6 61.1 us
//   64 tokens, width 128: 20.6 20.6 20.7 24.7 39.4   16.6 18.9 21.0 28.5 61.6
//   16 tokens, width 512: 20.6 22.7 24.9 35.3 78.9   18.6 22.6 24.7 36.5 83.7
constexpr int32_t kFewFrom = 1 << 15;

// Whether the log-sums take the table's rows for the product's.
bool few_rows(const tbe_catalogue_inputs& in) {
  return in.tokens <= kFewRows && in.vocab >= kFewFrom && in.logit_scale * kLog2e != 0.f;
}

struct Layout {
  int64_t Np;
  int32_t Dp, vc, pieces, splits, steps, vt;
  size_t rows, label, lse2, mine, own, count, next, block_sum, arrived, hidden, part, weights, g, acc, bytes;
};
// Tensor copies want rows that start on 16 bytes and, by blocks of 64 columns,
// whole ones; other tables are copied.
bool off_pieces(const void* p, int64_t stride) { return ((uintptr_t)p & 15) || stride % 8; }
bool copied(const tbe_catalogue_inputs& in, bool grad) {
  return off_pieces(in.weights, in.weights_stride) || (grad && in.width % 64);
}

Layout layout(const tbe_catalogue_inputs& in, bool grad) {
  const int64_t N = in.tokens;
  const int32_t V = in.vocab, D = in.width;
  Layout w;
  w.Np = whole(N, kTileM);  // (whole tiles)
  w.Dp = (int32_t)whole(D, 64);
  w.vt = (V + kTileN - 1) / kTileN;
  w.vc = (int32_t)std::min<int64_t>(whole(V, kTileN), std::max<int64_t>(kTileN, kPiece / w.Np / kTileN * kTileN));
  w.pieces = (V + w.vc - 1) / w.vc;
  // dhidden's tiles: as many as there are SMs, where there are few rows, of at least 8 steps each
  const int64_t tiles = w.Np / kTileM * 2 * ((D + kTileN - 1) / kTileN), steps = (w.vc + kTileK - 1) / kTileK;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>({(sm_count() + tiles - 1) / tiles, steps / 8, 32}));
  w.steps = (int32_t)((steps + want - 1) / want);
  w.splits = (int32_t)((steps + w.steps - 1) / w.steps);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  w.rows = take(4 * (size_t)N);
  w.label = take(4 * (size_t)w.Np);
  w.lse2 = take(4 * (size_t)w.Np);
  w.mine = take(4 * (size_t)w.Np);
  w.own = take(4 * (size_t)w.Np);
  w.count = take(4);
  w.next = take(4 * (size_t)(w.pieces + 3));  // of the log-sums, the pieces and what follows the last; arrived
  w.arrived = w.next + 4 * (size_t)(w.pieces + 2);
  w.block_sum = take(4 * (size_t)(w.Np / kRows));
  w.hidden = take(2 * (size_t)w.Np * w.Dp);
  w.weights = take(copied(in, grad) ? 2 * (size_t)V * w.Dp : 0);
  // the log-sums' parts are through before the first piece
  const size_t parts = sizeof(float2) * (size_t)(few_rows(in) ? 4 * (sm_count() + 1) : w.vt) * w.Np;
  const size_t gs = grad ? 2 * 2 * (size_t)w.Np * w.vc : 0;
  w.part = w.g = take(std::max(parts, gs));
  w.acc = take(grad ? 4 * (size_t)w.splits * w.Np * w.Dp : 0);
  w.bytes = at;
  return w;
}

// [rows, cols] of 16-bit elements, `stride` elements from row to row.
bool map_of(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t stride, int32_t dtype, uint32_t high = kRowsM) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, high}, one[2] = {1, 1};
  return encode_map(m, dtype, 2, p, dims, strides, box, one);
}
// The same as blocks of 64 columns (which cols is a multiple of).
bool blocks_of(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t stride, int32_t blocks, int32_t dtype) {
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)cols / 64}, strides[2] = {(cuuint64_t)stride * 2, 128};
  const cuuint32_t box[3] = {64, kTileK, (cuuint32_t)blocks}, one[3] = {1, 1, 1};
  return encode_map(m, dtype, 3, p, dims, strides, box, one);
}

// Launches `kernel`; `after`: it may start while the kernel before it ends.
template <typename A>
int start(void (*kernel)(A), int64_t grid, int threads, size_t smem, bool after, cudaStream_t s, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? check_launch() : TBE_ERR_CUDA;
}

constexpr size_t kProductBytes = (size_t)kStages * kStageBytes + 1024;

template <int DT, bool FEW = false>
int start_products(const GemmArgs& g, int64_t tiles, cudaStream_t s) {  // tiles: at most so many
  static bool allowed[64] = {};  // once per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !allowed[dev]) {
    if (cudaFuncSetAttribute(product_kernel<DT, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kProductBytes) !=
        cudaSuccess)
      return TBE_ERR_CUDA;
    if (dev >= 0 && dev < 64) allowed[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)std::max<int64_t>(1, std::min<int64_t>(sm_count() / 2, tiles)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kProductBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, product_kernel<DT, FEW>, g) == cudaSuccess ? check_launch() : TBE_ERR_CUDA;
}

struct Call {
  const tbe_catalogue_inputs* in;
  float *loss, *token_loss, *lse;  // the forward's outputs, or null
  const float* given;              // the log-sums of an earlier call, or null
  const float* given_loss;         // its losses, or null
  void* dhidden;
  int64_t dhidden_stride;
  void* dweights;
  int64_t dweights_stride;
  float grad_scale;
  uint8_t* ws;
  int32_t* status;
};

template <typename T>
T* at(uint8_t* p, size_t offset) {
  return reinterpret_cast<T*>(p + offset);
}
int piece_of(const void* p, int64_t stride, int most) {
  while (most > 2 && (((uintptr_t)p | (uintptr_t)(stride * 2)) & (most - 1))) most >>= 1;
  return most;
}

template <int DT>
int run(const Call& c, cudaStream_t s) {
  const tbe_catalogue_inputs& in = *c.in;
  const bool grad = c.dhidden != nullptr, copy = copied(in, grad);
  const int64_t N = in.tokens;
  const Layout w = layout(in, grad);
  uint8_t* ws = c.ws;

  PickArgs p = {};
  p.labels = in.labels;
  p.N = N;
  p.Np = w.Np;
  p.V = in.vocab;
  p.rows = at<int32_t>(ws, w.rows);
  p.label = at<int32_t>(ws, w.label);
  p.lse2 = at<float>(ws, w.lse2);
  p.count = at<int32_t>(ws, w.count);
  p.zero = at<uint32_t>(ws, w.next);
  p.zeros = w.pieces + 3;
  p.token_loss = c.token_loss;
  p.lse = c.lse;
  p.loss = c.loss;
  p.given = c.given;
  p.given_loss = c.given_loss;
  p.own = at<float>(ws, w.own);
  p.status = c.status;
  CopyArgs k = {};
  k.src = static_cast<const uint16_t*>(in.hidden);
  k.src_stride = in.hidden_stride;
  k.rows = p.rows;
  k.count = p.count;
  k.dst = at<uint16_t>(ws, w.hidden);
  k.N = N;
  k.Np = w.Np;
  k.D = in.width;
  k.Dp = w.Dp;
  k.vec = in.width % 8 == 0 && !off_pieces(in.hidden, in.hidden_stride) ? 8 : 1;
  k.zero = static_cast<uint16_t*>(c.dhidden);
  k.zero_stride = c.dhidden_stride;
  k.labels = in.labels;
  k.V = in.vocab;
  int st;
  if (N <= kFewTokens) {
    st = start(pick_copy_kernel, w.Np / 8, 256, 0, false, s, FewArgs{p, k});
  } else {
    if ((st = start(pick_kernel, 1, kPickThreads, 0, false, s, p)) != TBE_OK) return st;
    trace_mark(s, "catalogue_pick");
    st = start(copy_kernel, w.Np / 8, 256, 0, true, s, k);
  }
  if (st != TBE_OK) return st;
  trace_mark(s, "catalogue_rows");
  const void* table = in.weights;
  int64_t table_stride = in.weights_stride;
  if (copy) {
    CopyArgs t = {};
    t.src = static_cast<const uint16_t*>(in.weights);
    t.src_stride = in.weights_stride;
    t.dst = at<uint16_t>(ws, w.weights);
    t.N = t.Np = in.vocab;
    t.D = in.width;
    t.Dp = w.Dp;
    t.vec = 1;
    st = start(copy_kernel, ((int64_t)in.vocab + 7) / 8, 256, 0, true, s, t);
    if (st != TBE_OK) return st;
    trace_mark(s, "catalogue_table");
    table = t.dst;
    table_stride = w.Dp;
  }

  GemmArgs g = {};
  const int64_t table_cols = copy ? w.Dp : in.width;
  g.half = w.Dp <= 128 ? 1 : 2;
  if (!map_of(&g.h, k.dst, w.Np, w.Dp, w.Dp, DT) || !map_of(&g.w, table, in.vocab, table_cols, table_stride, DT))
    return TBE_ERR_CUDA;
  if (grad) {
    const uint16_t* gs = at<uint16_t>(ws, w.g);
    if (!map_of(&g.p, gs, 2 * w.Np, w.vc, w.vc, DT) || !blocks_of(&g.pt, gs, 2 * w.Np, w.vc, w.vc, kRowsM / 64, DT) ||
        !blocks_of(&g.ht, k.dst, w.Np, w.Dp, w.Dp, g.half, DT) ||
        !blocks_of(&g.wt, table, in.vocab, table_cols, table_stride, g.half, DT))
      return TBE_ERR_CUDA;
  }
  g.V = in.vocab;
  g.D = in.width;
  g.Dp = w.Dp;
  g.Np = w.Np;
  g.count = p.count;
  g.scale2 = in.logit_scale * kLog2e;
  g.label = p.label;
  g.lse2 = p.lse2;
  g.own = c.loss || c.given_loss ? p.own : nullptr;
  g.mine = at<float>(ws, w.mine);
  g.part = at<float2>(ws, w.part);
  g.g = at<uint16_t>(ws, w.g);
  g.vc = w.vc;
  g.dw = static_cast<uint16_t*>(c.dweights);
  g.dw_stride = c.dweights_stride;
  g.dw_piece = piece_of(c.dweights, c.dweights_stride, 32);
  g.factor = (float)((double)c.grad_scale * in.logit_scale * std::ldexp(1.0, -kUp<DT>));
  g.acc = at<float>(ws, w.acc);
  g.status = c.status;
  if (c.loss) {
    g.jobs = 1;
    g.job[0] = Job{kSums, 0, in.vocab, 0, 0, 0, 0};
    g.next = p.zero;
    const bool few = few_rows(in);
    if (few && !map_of(&g.few, k.dst, w.Np, w.Dp, w.Dp, DT, kFewRows)) return TBE_ERR_CUDA;
    const int64_t pairs = std::min<int64_t>(sm_count() / 2, w.vt);
    st = few ? start_products<DT, true>(g, w.vt, s) : start_products<DT>(g, w.Np / kTileM * w.vt, s);
    if (st != TBE_OK) return st;
    trace_mark(s, "catalogue_sums");
    RowArgs r = {};
    r.part = g.part;
    r.parts = few ? (int32_t)(8 * std::max<int64_t>(1, pairs)) : w.vt;
    r.Np = w.Np;
    r.count = p.count;
    r.rows = p.rows;
    r.mine = g.mine;
    r.scale2 = g.scale2;
    r.lse2 = p.lse2;
    r.own = p.own;
    r.token_loss = c.token_loss;
    r.lse = c.lse;
    r.loss = c.loss;
    r.block_sum = at<float>(ws, w.block_sum);
    r.arrived = at<uint32_t>(ws, w.arrived);
    st = start(row_kernel, w.Np / kRows, kRowThreads, 0, true, s, r);
    if (st != TBE_OK) return st;
    trace_mark(s, "catalogue_loss");
  }
  if (!grad) return TBE_OK;
  const int64_t row_tiles = w.Np / kTileM, column_tiles = (in.width + 128 * g.half - 1) / (128 * g.half);
  for (int i = 0; i <= w.pieces; ++i) {
    int64_t tiles = 0;
    g.jobs = 0;
    if (i > 0) {  // the long tiles first
      const int32_t v0 = (i - 1) * w.vc, v1 = (int32_t)std::min<int64_t>(in.vocab, (int64_t)v0 + w.vc);
      g.job[g.jobs++] = Job{kTable, v0, v1, (i - 1) & 1, 0, 0, 0};
      g.job[g.jobs++] = Job{kHidden, v0, v1, (i - 1) & 1, w.splits, w.steps, i == 1};
      tiles += ((v1 - v0 + kTileM - 1) / kTileM + w.splits * row_tiles) * column_tiles;
    }
    if (i < w.pieces) {
      const int32_t v0 = i * w.vc, v1 = (int32_t)std::min<int64_t>(in.vocab, (int64_t)v0 + w.vc);
      g.job[g.jobs++] = Job{kProbs, v0, v1, i & 1, 0, 0, 0};
      tiles += row_tiles * ((v1 - v0 + kTileN - 1) / kTileN);
    }
    g.next = p.zero + 1 + i;
    if ((st = start_products<DT>(g, tiles, s)) != TBE_OK) return st;
  }
  trace_mark(s, "catalogue_gradients");
  SpreadArgs d = {};
  d.acc = g.acc;
  d.splits = w.splits;
  d.Np = w.Np;
  d.D = in.width;
  d.Dp = w.Dp;
  d.count = p.count;
  d.rows = p.rows;
  d.factor = g.factor;
  d.out = static_cast<uint16_t*>(c.dhidden);
  d.stride = c.dhidden_stride;
  d.pairs = piece_of(c.dhidden, c.dhidden_stride, 4) == 4;
  st = start(spread_kernel<DT>, w.Np / 8, 256, 0, true, s, d);
  trace_mark(s, "catalogue_dhidden");
  return st;
}

int check(const tbe_catalogue_inputs* in) {
  if (!in || (in->dtype != TBE_F16 && in->dtype != TBE_BF16 && in->dtype != TBE_F32)) return TBE_ERR_INVALID_ARG;
  if (in->dtype == TBE_F32) return TBE_ERR_UNSUPPORTED;
  if (in->tokens < 1 || in->vocab < 1 || in->width < 1 || !std::isfinite(in->logit_scale)) return TBE_ERR_INVALID_ARG;
  if (!in->hidden || !in->weights || !in->labels || in->hidden_stride < in->width || in->weights_stride < in->width)
    return TBE_ERR_INVALID_ARG;
  if (in->tokens > kMaxTokens || in->vocab > (1 << 30) || in->width > (1 << 16)) return TBE_ERR_UNSUPPORTED;
  if (whole(in->tokens, kTileM) / kTileM * (whole(in->vocab, kTileN) / kTileN) >= (int64_t(1) << 31))
    return TBE_ERR_UNSUPPORTED;  // tiles are counted in 32 bits
  if (((uintptr_t)in->hidden | (uintptr_t)in->weights) & 1 || ((uintptr_t)in->labels & 7)) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

int dispatch(const Call& c, void* workspace, size_t bytes, void* stream) {
  const tbe_catalogue_inputs& in = *c.in;
  if (!workspace) return TBE_ERR_INVALID_ARG;
  if ((uintptr_t)workspace & 255) return TBE_ERR_UNSUPPORTED;
  if ((c.dhidden != nullptr) != (c.dweights != nullptr)) return TBE_ERR_INVALID_ARG;
  if (c.dhidden) {
    if (c.dhidden_stride < in.width || c.dweights_stride < in.width || !std::isfinite(c.grad_scale))
      return TBE_ERR_INVALID_ARG;
    if (((uintptr_t)c.dhidden | (uintptr_t)c.dweights) & 1) return TBE_ERR_UNSUPPORTED;
    // inputs are read again after the first results are written
    const int64_t wide = 2 * (int64_t)in.width, each = sizeof(float) * in.tokens;
    const Region read[5] = {rows_of(in.hidden, in.tokens, 2 * in.hidden_stride, wide),
                            rows_of(in.weights, in.vocab, 2 * in.weights_stride, wide),
                            bytes_of(in.labels, (int64_t)sizeof(int64_t) * in.tokens), bytes_of(c.given, each),
                            bytes_of(c.given_loss, each)};
    const Region dh = rows_of(c.dhidden, in.tokens, 2 * c.dhidden_stride, wide),
                 dw = rows_of(c.dweights, in.vocab, 2 * c.dweights_stride, wide);
    for (const Region& r : read)
      if (share(dh, r) || share(dw, r)) return TBE_ERR_INVALID_ARG;
    if (share(dh, dw)) return TBE_ERR_INVALID_ARG;
  }
  const Layout w = layout(in, c.dhidden != nullptr);
  if (bytes < w.bytes) return TBE_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  trace_begin(s);
  return in.dtype == TBE_F16 ? run<TBE_F16>(c, s) : run<TBE_BF16>(c, s);
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" {

size_t tbe_catalogue_workspace_bytes(const tbe_catalogue_inputs* in, int32_t grad) {
  if (check(in) != TBE_OK) return 0;
  return layout(*in, grad != 0).bytes;
}

int tbe_catalogue_loss(const tbe_catalogue_inputs* in, float* loss, float* token_loss, float* lse, void* dhidden,
                       int64_t dhidden_stride, void* dweights, int64_t dweights_stride, float grad_scale,
                       void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int st = check(in);
  if (st != TBE_OK) return st;
  if (!loss || !token_loss || !lse) return TBE_ERR_INVALID_ARG;
  const Call c = {in,       loss, token_loss, lse, nullptr, nullptr, dhidden, dhidden_stride, dweights, dweights_stride, grad_scale,
                  static_cast<uint8_t*>(workspace), dev_status};
  return dispatch(c, workspace, workspace_bytes, stream);
}

int tbe_catalogue_loss_backward(const tbe_catalogue_inputs* in, const float* lse, void* dhidden, int64_t dhidden_stride,
                                void* dweights, int64_t dweights_stride, float grad_scale, void* workspace,
                                size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return tbe_catalogue_loss_backward_full(in, lse, nullptr, dhidden, dhidden_stride, dweights, dweights_stride, grad_scale,
                                          workspace, workspace_bytes, dev_status, stream);
}

int tbe_catalogue_loss_backward_full(const tbe_catalogue_inputs* in, const float* lse, const float* token_loss, void* dhidden,
                                     int64_t dhidden_stride, void* dweights, int64_t dweights_stride, float grad_scale,
                                     void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int st = check(in);
  if (st != TBE_OK) return st;
  if (!lse || !dhidden || !dweights) return TBE_ERR_INVALID_ARG;
  const Call c = {in,      nullptr, nullptr, nullptr, lse, token_loss, dhidden, dhidden_stride, dweights, dweights_stride,
                  grad_scale, static_cast<uint8_t*>(workspace), dev_status};
  return dispatch(c, workspace, workspace_bytes, stream);
}

}  // extern "C"
