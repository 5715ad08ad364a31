// tbe_preference.cu -- a paired-log-ratio preference loss over catalogue
// logits, with its gradient.
//
//   lp_n  = logit[n, y_n] - lse_n            lse_n = log sum_v exp(logit[n, v])
//   s(q)  = sum of lp_n over sequence q's tokens
//   d_b   = beta ((s(0, b) - ref(0, b)) - (s(1, b) - ref(1, b)))
//   loss  = mean_b (1 - e) log(1 + exp(-d_b)) + e log(1 + exp(d_b))
//   dlogit[n, v] = coef_n ([v = y_n] - exp(logit[n, v] - lse_n))
// lse_n is held as two fp32 numbers, its rounded value and what the rounding
// left: a row's probabilities would otherwise share an error of 2^-24 |lse|,
// all of log(V) for a row of nothing but the type's lowest value.
// with coef_n = +- beta / P ((e - 1) / (1 + exp(d_b)) + e / (1 + exp(-d_b))),
// + for a preferred token, - for a rejected one.  Sequences are the bags of
// two features (0 preferred, 1 rejected) in the feature-major layout.
//
// Three kernels: the rows' log-sums (one pass over the logits with a running
// maximum and sum per thread; a long row is cut over several thread blocks
// where there are few rows), the pairs, and the gradient, each started while
// the one before it ends.  A small batch goes through one kernel.
//
// A large batch is bound by memory: the logits are read twice and the gradient
// written once.  3,840 rows of 100,000 bf16 logits take 372 us: the log-sums
// 130 us (5.9 TB/s; with an exponential per element, whose rate alone would
// take 83 us), the gradient 232 us (6.6 TB/s), the pairs the rest.  The second
// reading finds nothing in the 129 MB L2, because the whole batch lies between
// the two: a pair's coefficient needs both its sequences' sums.
#include "tbe_internal.cuh"

#include <cmath>

namespace tbe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;
// A warp takes a row of at most this length where one cluster has the batch
// (loss and gradient of 80 rows of 1,000: 8.5 us, with blocks to them 18.0 us).
constexpr int kWarpRow = 1024;

struct PrefArgs {
  const void* logits;
  int64_t stride;
  const int64_t* labels;
  const int64_t* offsets;
  const float* ref;
  int64_t N;
  int32_t V;
  int32_t P;
  int32_t splits;
  float beta, smoothing, scale;
  float* loss;
  float* logps;
  float* margins;
  float* lse;
  float* low;        // what the rounding of lse left, or null (the gradient alone): 0
  float* coef;
  void* dlogits;
  int64_t dstride;
  float2* part;      // [N, splits] running maximum and sum
  float* lp;         // [N]
  float* block_loss; // one per block of the pairs' kernel, or per pair
  uint32_t* arrived;
  int32_t* status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Running maximum and sum of exp(x - maximum).  The maximum starts at the
// lowest finite value: entries of -inf add exp(-inf) = 0, and a row of
// nothing else keeps the sum 0.
struct Run {
  float m, s;
};
__device__ __forceinline__ Run merge(Run a, Run b) {
  Run r;
  r.m = fmaxf(a.m, b.m);
  r.s = a.s * ex2((a.m - r.m) * kLog2e) + b.s * ex2((b.m - r.m) * kLog2e);
  return r;
}

template <int DT>
struct Vec {
  static constexpr int kElems = Chunk<DT>::kElems;
  static constexpr int kSize = DT == TBE_F32 ? 4 : 2;
};

template <int DT>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if (DT == TBE_F32) return static_cast<const float*>(p)[i];
  if (DT == TBE_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store_one(void* p, int64_t i, float f) {
  if (DT == TBE_F32) static_cast<float*>(p)[i] = f;
  else if (DT == TBE_F16) static_cast<__half*>(p)[i] = __float2half_rn(f);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f);
}
template <int DT>
__device__ __forceinline__ const uint8_t* elem_ptr(const void* p, int64_t i) {
  return static_cast<const uint8_t*>(p) + i * Vec<DT>::kSize;
}
template <int DT>
__device__ __forceinline__ uint8_t* elem_ptr(void* p, int64_t i) {
  return static_cast<uint8_t*>(p) + i * Vec<DT>::kSize;
}

__device__ __forceinline__ uint4 ld_plain16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// A run of n elements from p on, read by `workers` threads of which this is
// number `me`: elements before the first 16-byte boundary and after the last
// one on their own, the rest in 16-byte pieces, four in flight per thread (2,
// 3, 4, 6, 8: 380, 381, 374, 401, 403 us for 3,840 rows of 100,000 bf16).
template <int DT>
__device__ __forceinline__ Run sum_row(const uint8_t* p, int64_t n, int me, int workers) {
  constexpr int kE = Vec<DT>::kElems, kS = Vec<DT>::kSize, kFlight = 4;
  Run r{kLowest, 0.f};
  int64_t head = (16 - ((uintptr_t)p & 15)) % 16 / kS;
  if (head > n) head = n;
  const int64_t pieces = (n - head) / kE, tail = head + pieces * kE;
  auto one = [&](float x) {
    const float m = fmaxf(r.m, x);
    r.s = r.s * ex2((r.m - m) * kLog2e) + ex2((x - m) * kLog2e);
    r.m = m;
  };
  for (int64_t i = me; i < head; i += workers) one(load_one<DT>(p, i));
  for (int64_t i = tail + me; i < n; i += workers) one(load_one<DT>(p, i));
  const uint8_t* body = p + head * kS;
  for (int64_t i = me; i < pieces; i += (int64_t)workers * kFlight) {
    uint4 raw[kFlight];
    bool in[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      in[k] = i + (int64_t)k * workers < pieces;
      if (in[k]) raw[k] = ld_plain16(body + (i + (int64_t)k * workers) * 16);
    }
    float x[kFlight][kE], top = r.m;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (in[k]) {
        Chunk<DT>::to_float(raw[k], x[k]);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) x[k][e] = -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) top = fmaxf(top, x[k][e]);
    }
    float s = r.s * ex2((r.m - top) * kLog2e);
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
#pragma unroll
      for (int e = 0; e < kE; ++e) s += ex2((x[k][e] - top) * kLog2e);
    r.m = top;
    r.s = s;
  }
  return r;
}

__device__ __forceinline__ Run warp_merge(Run r) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Run n;
    n.m = __shfl_xor_sync(kFull, r.m, o);
    n.s = __shfl_xor_sync(kFull, r.s, o);
    r = merge(r, n);
  }
  return r;
}

// The label of row n, or -1 where the row takes no part.
__device__ __forceinline__ int64_t label_of(const PrefArgs& a, int64_t n) {
  const int64_t y = a.labels[n];
  if (y >= a.V) {
    report(a.status, TBE_DEV_BAD_INDEX);
    return -1;
  }
  return y < 0 ? -1 : y;
}

// A row's label, and the label's logit.
struct Label {
  int64_t y;
  float logit;
};
template <int DT>
__device__ __forceinline__ Label read_label(const PrefArgs& a, int64_t n) {
  const int64_t y = label_of(a, n);
  return Label{y, y >= 0 ? load_one<DT>(a.logits, n * a.stride + y) : 0.f};
}
// A row's log-sum and its label's log-probability (returned).  A row of which
// every entry is -inf has nothing to choose from: it takes no part (lse = -inf).
__device__ __forceinline__ float finish_row(const PrefArgs& a, int64_t n, Run r, Label l) {
  const float log_s = logf(r.s);
  if (r.s == 0.f) {
    a.lse[n] = -INFINITY;
    a.low[n] = 0.f;
    return 0.f;
  }
  // the sum of the maximum and log_s, and exactly what its rounding leaves
  const float lse = __fadd_rn(r.m, log_s), got = __fsub_rn(lse, r.m);
  a.lse[n] = lse;
  a.low[n] = __fadd_rn(__fsub_rn(r.m, __fsub_rn(lse, got)), __fsub_rn(log_s, got));
  return l.y >= 0 ? (l.logit - r.m) - log_s : 0.f;
}

// LANES threads to a row: a warp (blocks of kWarps rows), or a block of that
// many threads to a piece of a row.
template <int LANES>
constexpr int kBlockThreads = LANES == 32 ? kThreads : LANES;
template <int DT, int LANES>
__global__ void __launch_bounds__(kBlockThreads<LANES>) rows_kernel(PrefArgs a) {
  constexpr int kRowWarps = LANES / 32;
  __shared__ Run s_run[kRowWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.arrived = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (LANES == 32) {
    const int64_t n = (int64_t)blockIdx.x * kWarps + warp;
    if (n >= a.N) return;
    const Run r = warp_merge(sum_row<DT>(elem_ptr<DT>(a.logits, n * a.stride), a.V, lane, 32));
    if (lane == 0) {
      a.lp[n] = finish_row(a, n, r, read_label<DT>(a, n));
      a.coef[n] = 0.f;
    }
    return;
  }
  const int64_t n = blockIdx.x / a.splits, part = blockIdx.x % a.splits;
  const int64_t lo = a.V * part / a.splits, hi = a.V * (part + 1) / a.splits;
  Run r = warp_merge(sum_row<DT>(elem_ptr<DT>(a.logits, n * a.stride + lo), hi - lo, threadIdx.x, LANES));
  if (lane == 0) s_run[warp] = r;
  __syncthreads();
  if (warp == 0) {
    r = lane < kRowWarps ? s_run[lane] : Run{kLowest, 0.f};
    r = warp_merge(r);
    if (lane == 0) {
      if (a.splits == 1) a.lp[n] = finish_row(a, n, r, read_label<DT>(a, n));
      else a.part[n * a.splits + part] = make_float2(r.m, r.s);
      if (part == 0) a.coef[n] = 0.f;
    }
  }
}

// Pair b, by two neighbouring warps, one to a sequence: the sequences' sums,
// the margin, the loss (returned to the first lane of the first warp, 0 to
// the others) and the tokens' coefficients.  Every thread of the block calls
// this; `logps` has room for its warps.  (A warp to both sequences, one after
// the other: 1,300 rows of 10,007 f16 logits 25.1 us, so 23.4 us;
// 6 rows of 100,000 fp32 13.3, so 10.7 us.)  A warp walks its sequence however
// long it is, twice: 8,000 rows of 100 fp32 logits take 13 us as a hundred pairs
// and 88 us as one.
template <int DT>
__device__ __forceinline__ float pair_loss(const PrefArgs& a, int64_t b, int warp, int lane, float* logps) {
  const int t = warp & 1;
  const bool on = b < a.P;
  const int64_t q = (int64_t)t * a.P + b;
  int64_t lo = 0, hi = 0;
  float ref[2] = {0.f, 0.f};
  if (on) {
    lo = a.offsets[q];
    hi = a.offsets[q + 1];
    ref[0] = a.ref[b];
    ref[1] = a.ref[a.P + b];
    const bool bad = lo < 0 || hi < lo || hi > a.N || (q == 0 && lo != 0) || (q == 2 * (int64_t)a.P - 1 && hi != a.N);
    if (bad && lane == 0) report(a.status, TBE_DEV_BAD_OFFSETS);
    if (lo < 0) lo = 0;
    if (hi > a.N) hi = a.N;
  }
  // of this lane's first row
  const bool have = lo + lane < hi;
  int64_t y = -1;
  float lse = -INFINITY;
  float s = 0.f;
  if (a.splits == 1) {
    if (have) {
      y = a.labels[lo + lane];
      lse = __ldcg(a.lse + lo + lane);
    }
    for (int64_t n = lo + lane; n < hi; n += 32) s += __ldcg(a.lp + n);
  } else {
    // 32 / each lanes to a row's pieces, so that few rows do not leave the
    // loads to few lanes
    const int64_t rows = hi - lo;
    const int each = rows >= 32 ? 32 : (rows >= 16 ? 16 : (rows >= 8 ? 8 : 4)), lanes = 32 / each, sub = lane % lanes;
    for (int64_t i = lane / lanes; i < (rows + each - 1) / each * each; i += each) {
      const int64_t n = lo + i;
      const bool in = i < rows;
      const Label l = in && sub == 0 ? read_label<DT>(a, n) : Label{-1, 0.f};
      Run r{kLowest, 0.f};
#pragma unroll 8
      for (int p = in ? sub : a.splits; p < a.splits; p += lanes) {
        const float2 v = __ldcg(a.part + n * a.splits + p);
        r = merge(r, Run{v.x, v.y});
      }
      for (int o = lanes >> 1; o; o >>= 1) {
        Run other;
        other.m = __shfl_xor_sync(kFull, r.m, o);
        other.s = __shfl_xor_sync(kFull, r.s, o);
        r = merge(r, other);
      }
      if (in && sub == 0) s += finish_row(a, n, r, l);
    }
    __syncwarp();  // the rows' log-sums are read by other lanes
    if (have) {
      y = a.labels[lo + lane];
      lse = __ldcg(a.lse + lo + lane);
    }
  }
  s = warp_sum(s);
  if (lane == 0) {
    logps[warp] = s;
    if (on) a.logps[q] = s;
  }
  __syncthreads();
  const float d = a.beta * ((logps[warp & ~1] - ref[0]) - (logps[warp | 1] - ref[1]));
  // log(1 + exp(-d)) and log(1 + exp(d)) without overflow
  const float l = log1pf(expf(-fabsf(d)));
  // A term of weight 0 counts as 0: d is infinite where a label's logit is
  // -inf, and the other term is then the whole loss.
  float loss = 0.f;
  if (a.smoothing != 1.f) loss = (1.f - a.smoothing) * (fmaxf(-d, 0.f) + l);
  if (a.smoothing != 0.f) loss += a.smoothing * (fmaxf(d, 0.f) + l);
  const float up = 1.f / (1.f + expf(-d)), down = 1.f / (1.f + expf(d));
  const float both = a.beta / (float)a.P * (a.smoothing * up - (1.f - a.smoothing) * down), c = t == 0 ? both : -both;
  if (on && t == 0 && lane == 0) a.margins[b] = d;
  if (have) a.coef[lo + lane] = y < 0 || y >= a.V || lse == -INFINITY ? 0.f : c;
  for (int64_t n = lo + lane + 32; n < hi; n += 32) {
    const int64_t label = a.labels[n];
    a.coef[n] = label < 0 || label >= a.V || __ldcg(a.lse + n) == -INFINITY ? 0.f : c;
  }
  return on && t == 0 && lane == 0 ? loss : 0.f;
}

// Two warps per pair.
template <int DT>
__global__ void __launch_bounds__(kThreads) pairs_kernel(PrefArgs a) {
  __shared__ float s_logps[kWarps], s_loss[kWarps];
  __shared__ bool s_last;
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float loss = pair_loss<DT>(a, (int64_t)blockIdx.x * (kWarps / 2) + warp / 2, warp, lane, s_logps);
  if (lane == 0) s_loss[warp] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w) s += s_loss[w];
    a.block_loss[blockIdx.x] = s;
    __threadfence();
    s_last = atomicAdd(a.arrived, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last || warp != 0) return;
  // the last block to finish adds the blocks' sums, always in the same order
  __threadfence();
  float s = 0.f;
  for (unsigned i = lane; i < gridDim.x; i += 32) s += __ldcg(a.block_loss + i);
  s = warp_sum(s);
  if (lane == 0) *a.loss = s / (float)a.P;
}

template <int DT>
__device__ __forceinline__ uint4 pack(const float* f);
template <>
__device__ __forceinline__ uint4 pack<TBE_F32>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack<TBE_F16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 h = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack<TBE_BF16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// dlogit over n elements, y the label's place among them (or outside).
template <int DT>
__device__ __forceinline__ void grad_row(const uint8_t* p, uint8_t* o, int64_t n, int64_t y, float coef, float lse,
                                         float low, int me, int workers) {
  constexpr int kE = Vec<DT>::kElems, kS = Vec<DT>::kSize, kFlight = 4;
  // both rows in 16-byte pieces only where they lie alike
  int64_t head = (16 - ((uintptr_t)p & 15)) % 16 / kS;
  if (head > n || (((uintptr_t)p ^ (uintptr_t)o) & 15) != 0) head = n;
  const int64_t pieces = (n - head) / kE, tail = head + pieces * kE;
  const float shift = -low * kLog2e;
  auto value = [&](float x, bool label) {
    const float e = -coef * ex2(fmaf(x - lse, kLog2e, shift));
    return label ? e + coef : e;
  };
  for (int64_t i = me; i < head; i += workers)
    store_one<DT>(o, i, coef == 0.f ? 0.f : value(load_one<DT>(p, i), i == y));
  for (int64_t i = tail + me; i < n; i += workers)
    store_one<DT>(o, i, coef == 0.f ? 0.f : value(load_one<DT>(p, i), i == y));
  const uint8_t* pb = p + head * kS;
  uint8_t* ob = o + head * kS;
  if (coef == 0.f) {  // a row that takes no part is not read
    for (int64_t i = me; i < pieces; i += workers) *reinterpret_cast<uint4*>(ob + i * 16) = make_uint4(0, 0, 0, 0);
    return;
  }
  for (int64_t i = me; i < pieces; i += (int64_t)workers * kFlight) {
    uint4 raw[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (i + (int64_t)k * workers < pieces) raw[k] = ld_plain16(pb + (i + (int64_t)k * workers) * 16);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int64_t at = i + (int64_t)k * workers;
      if (at < pieces) {
        float x[kE];
        Chunk<DT>::to_float(raw[k], x);
        const int64_t first = head + at * kE;
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = value(x[e], first + e == y);
        *reinterpret_cast<uint4*>(ob + at * 16) = pack<DT>(x);
      }
    }
  }
}

template <int DT, int LANES>
__global__ void __launch_bounds__(kBlockThreads<LANES>) grad_kernel(PrefArgs a) {
  constexpr bool WARP = LANES == 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = WARP ? (int64_t)blockIdx.x * kWarps + warp : blockIdx.x / a.splits;
  if (n >= a.N) return;
  const int64_t part = WARP ? 0 : blockIdx.x % a.splits, splits = WARP ? 1 : a.splits;
  const int64_t lo = a.V * part / splits, hi = a.V * (part + 1) / splits;
  const float coef = a.coef[n] * a.scale;
  grad_row<DT>(elem_ptr<DT>(a.logits, n * a.stride + lo), elem_ptr<DT>(a.dlogits, n * a.dstride + lo), hi - lo,
               a.labels[n] - lo, coef, a.lse[n], a.low ? a.low[n] : 0.f, WARP ? lane : threadIdx.x, LANES);
}

// Small batches in one launch: one cluster of kSmallBlocks thread blocks goes
// through the three steps, its barrier between them.  A warp takes a short
// row, a block a long one; long rows are cut over blocks where there are fewer
// of them than blocks.  There are no more rows, or pieces of rows, than that
// (is_small).
constexpr int kSmallBlocks = 16, kSmallThreads = 512, kSmallWarps = kSmallThreads / 32;
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int DT>
__global__ void __launch_bounds__(kSmallThreads) small_kernel(PrefArgs a) {
  __shared__ Run s_run[kSmallWarps];
  __shared__ float s_logps[kSmallWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int me = blockIdx.x * kSmallWarps + warp;  // the grid is one cluster
  const bool by_warp = a.V <= kWarpRow;
  if (by_warp) {
    const int64_t n = me;
    if (n < a.N) {
      const Run r = warp_merge(sum_row<DT>(elem_ptr<DT>(a.logits, n * a.stride), a.V, lane, 32));
      if (lane == 0) {
        a.lp[n] = finish_row(a, n, r, read_label<DT>(a, n));
        a.coef[n] = 0.f;
      }
    }
  } else {
    const int64_t u = blockIdx.x;
    if (u < a.N * a.splits) {
      const int64_t n = u / a.splits, part = u % a.splits;
      const int64_t lo = a.V * part / a.splits, hi = a.V * (part + 1) / a.splits;
      Run r = warp_merge(sum_row<DT>(elem_ptr<DT>(a.logits, n * a.stride + lo), hi - lo, threadIdx.x, kSmallThreads));
      if (lane == 0) s_run[warp] = r;
      __syncthreads();
      if (warp == 0) {
        r = warp_merge(lane < kSmallWarps ? s_run[lane] : Run{kLowest, 0.f});
        if (lane == 0) {
          if (a.splits == 1) a.lp[n] = finish_row(a, n, r, read_label<DT>(a, n));
          else a.part[u] = make_float2(r.m, r.s);
          if (part == 0) a.coef[n] = 0.f;
        }
      }
    }
  }
  cluster_sync();
  constexpr int kPairs = kSmallWarps / 2;  // of a block at a time
  for (int64_t b0 = blockIdx.x * kPairs; b0 < a.P; b0 += kSmallBlocks * kPairs) {
    const int64_t b = b0 + warp / 2;
    const float loss = pair_loss<DT>(a, b, warp, lane, s_logps);
    if (b < a.P && lane == 0 && warp % 2 == 0) a.block_loss[b] = loss;
    __syncthreads();  // s_logps is free again
  }
  cluster_sync();
  if (me == 0) {
    float s = 0.f;
    for (int64_t b = lane; b < a.P; b += 32) s += __ldcg(a.block_loss + b);
    s = warp_sum(s);
    if (lane == 0) *a.loss = s / (float)a.P;
  }
  if (!a.dlogits) return;
  const int64_t u = by_warp ? me : blockIdx.x;
  if (u < a.N * a.splits) {
    const int64_t n = u / a.splits, part = u % a.splits;
    const int64_t lo = a.V * part / a.splits, hi = a.V * (part + 1) / a.splits;
    grad_row<DT>(elem_ptr<DT>(a.logits, n * a.stride + lo), elem_ptr<DT>(a.dlogits, n * a.dstride + lo), hi - lo,
                 a.labels[n] - lo, __ldcg(a.coef + n) * a.scale, __ldcg(a.lse + n), __ldcg(a.low + n),
                 by_warp ? lane : threadIdx.x, by_warp ? 32 : kSmallThreads);
  }
}


// Batches that one cluster takes in one round, a warp to a short row or a block
// to a long one, and that are at most this many bytes of logits, go through it:
// its single launch is what they pay for.  Loss and gradient in a row, the
// GPU's time and that of calls in a row: 64 rows of 1,000 fp32 logits 8.1 and
// 10.4 us against 8.1 and 11.4 us of the three kernels; 256 rows of 60 7.1 and
// 8.5 against 6.7 and 12.2 us; 384 rows of 60 9.9 and 12.5 against 7.2 and 12.3
// us, 4,096 rows 48 against 9 us.  Rows of 4,000: 16 of them 7.5 and 10.4
// against 7.2 and 11.7 us, 64 17.1 and 18.6 against 8.6 and 12 us.  Two rows of
// 100,000 (0.8 MB) 9.7 against 11.0 us, four 12.0 against 11.3, six 15.6 against
// 10.7 us.
constexpr int64_t kSmallBytes = 1 << 20;
bool is_small(int64_t N, int32_t V, int32_t P, int32_t dtype) {
  return N <= (V <= kWarpRow ? kSmallBlocks * kSmallWarps : kSmallBlocks) && P <= kSmallBlocks * kSmallWarps &&
         N * (int64_t)V * (dtype == TBE_F32 ? 4 : 2) <= kSmallBytes;
}

// Blocks per row: where there are at most two rows to an SM, long rows are
// cut, to four pieces an SM of at least 2048 entries each (512 or 8,192 make no
// difference).  40 rows of 100,000 bf16 logits: 17.4 us against 21.0 us with a
// block per row; 160 rows 28.0 against 34.3 us; 400 rows 56.1 against 53.3 us.
// (One cluster: as many as it has blocks.)
// Threads to a row in the kernels of larger batches.  Loss and gradient with
// 32, 128 and 256 threads to a row: 3,000 rows of 2,000 half-precision logits
// 15.4, 19.6, 28.1 us; of 8,000: 36.2, 31.2, 35.4 us; 1,300 rows of 10,007:
// 29.0, 25.2, 26.8 us; 3,840 rows of 100,000: 394, 385, 374 us.
int lanes_of(int32_t V) { return V <= 2048 ? 32 : (V <= 16384 ? 128 : kThreads); }
int32_t splits_of(int64_t N, int32_t V, int32_t P, int32_t dtype) {
  if (is_small(N, V, P, dtype)) {
    if (V <= kWarpRow || N < 1) return 1;
    const int64_t want = kSmallBlocks / N, most = V / 2048;
    const int64_t s = want < most ? want : most;
    return s < 1 ? 1 : (int32_t)s;
  }
  if (N <= 0 || N > 2 * sm_count() || lanes_of(V) == 32) return 1;
  const int64_t want = (4 * (int64_t)sm_count() + N - 1) / N, most = V / 2048;
  const int64_t s = want < most ? want : most;
  return s < 1 ? 1 : (int32_t)s;
}

// The workspace: what the rounding of the log-sums left (first, as callers
// find it there), the arrival counter, and what passes between the kernels.
struct Workspace {
  size_t arrived, part, lp, block_loss, bytes;
};
size_t round256(size_t b) { return (b + 255) / 256 * 256; }
Workspace layout(int64_t N, int32_t V, int32_t P, int32_t dtype) {
  Workspace w;
  size_t at = round256((size_t)N * 4);
  w.arrived = at;
  at += 256;
  w.part = at;
  const int32_t s = splits_of(N, V, P, dtype);
  if (s > 1) at += round256((size_t)N * s * sizeof(float2));
  w.lp = at;
  at += round256((size_t)N * 4);
  w.block_loss = at;
  at += round256((size_t)P * 4);
  w.bytes = at;
  return w;
}

// A launch that may start while the kernel before it ends (`after`).
template <typename K>
int start(K kernel, int64_t grid, int threads, bool after, cudaStream_t s, const PrefArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? check_launch() : TBE_ERR_CUDA;
}

template <int DT>
int launch_rows(const PrefArgs& a, cudaStream_t s) {
  const int lanes = lanes_of(a.V);
  if (lanes == 32) return start(rows_kernel<DT, 32>, (a.N + kWarps - 1) / kWarps, kThreads, false, s, a);
  if (lanes == 128) return start(rows_kernel<DT, 128>, a.N * a.splits, 128, false, s, a);
  return start(rows_kernel<DT, kThreads>, a.N * a.splits, kThreads, false, s, a);
}

template <int DT>
int launch_grad(const PrefArgs& a, bool after, cudaStream_t s) {
  // (a small batch's rows may be cut finer here than a block needs: still right)
  const int lanes = lanes_of(a.V);
  if (lanes == 32) return start(grad_kernel<DT, 32>, (a.N + kWarps - 1) / kWarps, kThreads, after, s, a);
  if (lanes == 128) return start(grad_kernel<DT, 128>, a.N * a.splits, 128, after, s, a);
  return start(grad_kernel<DT, kThreads>, a.N * a.splits, kThreads, after, s, a);
}

template <int DT>
int launch_small(const PrefArgs& a, cudaStream_t s) {
  static bool allowed[64] = {};  // once per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !allowed[dev]) {
    if (cudaFuncSetAttribute(small_kernel<DT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return TBE_ERR_CUDA;
    if (dev >= 0 && dev < 64) allowed[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSmallBlocks);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSmallBlocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, small_kernel<DT>, a) == cudaSuccess ? check_launch() : TBE_ERR_CUDA;
}

template <int DT>
int launch_loss(const PrefArgs& a, int32_t dtype, cudaStream_t s) {
  if (is_small(a.N, a.V, a.P, dtype)) {
    const int st = launch_small<DT>(a, s);
    trace_mark(s, "preference_small");
    return st;
  }
  int st = launch_rows<DT>(a, s);
  if (st != TBE_OK) return st;
  trace_mark(s, "preference_rows");
  st = start(pairs_kernel<DT>, ((int64_t)a.P + kWarps / 2 - 1) / (kWarps / 2), kThreads, true, s, a);
  if (st != TBE_OK) return st;
  trace_mark(s, "preference_pairs");
  if (a.dlogits) {
    st = launch_grad<DT>(a, true, s);
    trace_mark(s, "preference_grad");
  }
  return st;
}

bool aligned_for(const void* p, int32_t dtype) { return ((uintptr_t)p & (dtype == TBE_F32 ? 3 : 1)) == 0; }

int check(const tbe_preference_inputs* in) {
  if (!in) return TBE_ERR_INVALID_ARG;
  if (in->dtype < TBE_F32 || in->dtype > TBE_BF16) return TBE_ERR_INVALID_ARG;
  if (in->tokens < 1 || in->vocab < 1 || in->pairs < 1 || in->logits_stride < in->vocab) return TBE_ERR_INVALID_ARG;
  if (!std::isfinite(in->beta) || !(in->label_smoothing >= 0.f && in->label_smoothing <= 1.f)) return TBE_ERR_INVALID_ARG;
  if (!in->logits || !in->labels || !in->offsets || !in->ref_logps) return TBE_ERR_INVALID_ARG;
  if (!aligned_for(in->logits, in->dtype)) return TBE_ERR_UNSUPPORTED;
  if (in->tokens * (int64_t)splits_of(in->tokens, in->vocab, in->pairs, in->dtype) >= (int64_t(1) << 31) ||
      in->pairs >= (1 << 30))
    return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

PrefArgs args_of(const tbe_preference_inputs* in) {
  PrefArgs a = {};
  a.logits = in->logits;
  a.stride = in->logits_stride;
  a.labels = in->labels;
  a.offsets = in->offsets;
  a.ref = in->ref_logps;
  a.N = in->tokens;
  a.V = in->vocab;
  a.P = in->pairs;
  a.beta = in->beta;
  a.smoothing = in->label_smoothing;
  a.splits = splits_of(in->tokens, in->vocab, in->pairs, in->dtype);
  return a;
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" {

size_t tbe_preference_workspace_bytes(int64_t tokens, int32_t vocab, int32_t pairs, int32_t dtype) {
  if (tokens < 1 || vocab < 1 || pairs < 1) return 0;
  return layout(tokens, vocab, pairs, dtype).bytes;
}

int tbe_preference_loss(const tbe_preference_inputs* in, float* loss, float* seq_logps, float* margins, float* lse,
                        float* coef, void* dlogits, int64_t dlogits_stride, float grad_scale, void* workspace,
                        size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int st = check(in);
  if (st != TBE_OK) return st;
  if (!loss || !seq_logps || !margins || !lse || !coef || !workspace) return TBE_ERR_INVALID_ARG;
  if (dlogits && (dlogits_stride < in->vocab || !std::isfinite(grad_scale))) return TBE_ERR_INVALID_ARG;
  if (!aligned_for(dlogits, in->dtype) || ((uintptr_t)workspace & 255)) return TBE_ERR_UNSUPPORTED;
  const Workspace w = layout(in->tokens, in->vocab, in->pairs, in->dtype);
  if (workspace_bytes < w.bytes) return TBE_ERR_WORKSPACE;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  PrefArgs a = args_of(in);
  a.loss = loss;
  a.logps = seq_logps;
  a.margins = margins;
  a.lse = lse;
  a.coef = coef;
  a.dlogits = dlogits;
  a.dstride = dlogits_stride;
  a.scale = grad_scale;
  a.low = reinterpret_cast<float*>(p);
  a.arrived = reinterpret_cast<uint32_t*>(p + w.arrived);
  a.part = reinterpret_cast<float2*>(p + w.part);
  a.lp = reinterpret_cast<float*>(p + w.lp);
  a.block_loss = reinterpret_cast<float*>(p + w.block_loss);
  a.status = dev_status;
  cudaStream_t s = (cudaStream_t)stream;
  trace_begin(s);
  if (in->dtype == TBE_F32) return launch_loss<TBE_F32>(a, in->dtype, s);
  if (in->dtype == TBE_F16) return launch_loss<TBE_F16>(a, in->dtype, s);
  return launch_loss<TBE_BF16>(a, in->dtype, s);
}

int tbe_preference_loss_backward(const tbe_preference_inputs* in, const float* lse, const float* coef,
                                 float grad_scale, void* dlogits, int64_t dlogits_stride, void* stream) {
  return tbe_preference_loss_backward_low(in, lse, nullptr, coef, grad_scale, dlogits, dlogits_stride, stream);
}

int tbe_preference_loss_backward_low(const tbe_preference_inputs* in, const float* lse, const float* lse_low,
                                     const float* coef, float grad_scale, void* dlogits, int64_t dlogits_stride,
                                     void* stream) {
  const int st = check(in);
  if (st != TBE_OK) return st;
  if (!lse || !coef || !dlogits || dlogits_stride < in->vocab || !std::isfinite(grad_scale)) return TBE_ERR_INVALID_ARG;
  if (!aligned_for(dlogits, in->dtype)) return TBE_ERR_UNSUPPORTED;
  PrefArgs a = args_of(in);
  a.lse = const_cast<float*>(lse);      // only read
  a.low = const_cast<float*>(lse_low);  // only read
  a.coef = const_cast<float*>(coef);    // only read
  a.dlogits = dlogits;
  a.dstride = dlogits_stride;
  a.scale = grad_scale;
  cudaStream_t s = (cudaStream_t)stream;
  trace_begin(s);
  const int rc = in->dtype == TBE_F32   ? launch_grad<TBE_F32>(a, false, s)
                 : in->dtype == TBE_F16 ? launch_grad<TBE_F16>(a, false, s)
                                        : launch_grad<TBE_BF16>(a, false, s);
  trace_mark(s, "preference_grad");
  return rc;
}

}  // extern "C"
