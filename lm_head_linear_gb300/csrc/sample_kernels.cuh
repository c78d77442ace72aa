// Drawing tokens from logits: temperature, top-k, top-p and min-p with given random numbers.
//
// Of a row's logits l (best first, equal ones by their index), w_i = e^((l_i - max) / temperature):
//   top-k keeps the first k, top-p of those the shortest prefix whose weights reach p of their
//   sum, min-p those with w_i >= min_p; the token is the first in vocabulary order whose
//   cumulative kept weight exceeds u times their sum.
// What is kept is then all l > t and the first n, by index, of l == t: a threshold is searched
// for, and nothing is sorted but a short list of candidates.
//
// The answer is a whole number that turns on comparisons of long sums, so weights are integers
// in units of 2^-44 or less (2^-46 up to 131,071 words): their sums are exact, in whatever order they are formed, and
// the sum that the search compares is the one that the drawing walks through.  A weight itself
// (table-driven exponential after Tang, 1989) is good to 2^-28.6 of it, 2^-31 in the mean (root mean square
// over all table entries), and half a unit.  A draw from 250,000 words with normal logits then falls on the other side of
// a border once in two million at a deviation of 2, five times in a million at 3, and top-p ends a word off in
// eight rows of a million at most (worked out from the weights on the CPU).  Words with the same logit are off by the same factor;
// two values whose errors are opposite could shift a border by 2^-29.6 of the sum, where a word is 2^-18 of it.
//
// A row belongs to a cluster of CTAs, each with its part in shared memory: the logits are
// read once.  The CTAs agree on maximum, sums and thresholds by pushing a few words into each
// other's shared memory and a cluster barrier.  The ways through the kernel:
//   no filter, min-p alone   maximum; weights of every lane's stretch; the draw
//   top-k up to about 1000   the k-th largest of 2048 groups' maxima bounds the k-th logit from
//                            below; what is above it is listed on one CTA, which does the rest
//   top-p of bf16            logits counted by their value, each value weighed once; then only the CTA
//                            that holds the drawn word goes through its part again
//   other top-p, larger k    logits counted in steps of 1/32 octave of their weight; a prefix
//                            that surely ends within 2048 logits is listed; a longer one ends
//                            within a few steps: these are counted again by value, and everything
//                            is weighed once
//
// Bound: not by memory (the floor is 18.7 us for the 127 MB of 256 x 124,160 fp32).  67 instructions are
// issued for each logit there, of which a weight is 25 to 35 (what the others are was not taken apart; the issue slots
// are 54 to 66 % taken), and every step that the CTAs agree on 2 to 3 us of barrier and skew, which two or three CTAs on an SM hide
// in part.  One row of 248,320 bf16 logits with top-k 50 and top-p: 12.4 us, of which the load takes
// 2.4, the maximum 2, bound and list 6, the rest 2.  256 x 124,160 as they are: fp32 86 us, bf16 55.  93 x 248,320
// bf16 top-p: 91 us (173 by steps of 1/32 octave, of whose 55 us a row weighing every logit took 19 and thresholds
// 15; 105 with all CTAs in the draw).  fp32 rows, and top-k of more than about 1000 words, go by steps: 93 x 248,320
// fp32 top-p 384 us, top-k 3000 and top-p 398 (bf16 189).  777 x 32,001 with settings for each row: 83 us (122 by steps).
// Counted by value, top-k above 256 took 83 us there as well, and made top-p 5 us slower.  44 KB instead of 64 of a row on
// each CTA, in clusters up to 16: 256 x 124,160 fp32 145 instead of 86 us, 93 x 248,320 top-p 139 instead of 91; 127 KB:
// 102 and 110.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "vec8.cuh"

namespace flce {
namespace sample {

using U64 = unsigned long long;

constexpr int kMaxCtas = 16;       // of a cluster
constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMostUnit = 46;      // weights are whole multiples of 2^-unit
constexpr int kTable = 32;         // steps of an octave
constexpr int kBins = 1536;        // of -32 log2(weight), rounded
constexpr int kLive = kMostUnit * kTable + kTable + 1;  // from this bin on weights are 0
constexpr int kList = 2048;        // candidates that are sorted
constexpr int kFewer = 128;        // up to which they are compared each with each
constexpr int kGroups = 2048;      // whose largest logits bound the k-th largest from below
constexpr uint32_t kAll = 0x7fffffffu;
constexpr int kValues = 4096;      // bf16 values that have a weight, for a row to be counted by value
constexpr uint32_t kPositive = 0xbb80u, kNegative = 0x447fu;  // leading 16 bits of the keys of 2^-8 and -2^-8
static_assert(kLive <= kBins && kBins % kMaxThreads == 0, "bins");

struct Params {
  const void* logits;
  const float* u;
  const float* temperature;  // [T], or nullptr: temperature_all (as the three below)
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  double temperature_all, top_p_all, log_min_p_all;
  float c_hi_all, c_lo_all;  // log2(e) / temperature_all
  float temperature_like, top_p_like, min_p_like;  // numbers that compare as those do with 0 and 1
  int64_t top_k_all;
  int64_t ldl, ignore_index;
  int64_t* tokens;
  float* logp;     // or nullptr
  int32_t V;
  int32_t ctas;    // of a cluster
  int32_t chunk;   // 16-byte pieces of a CTA
  int32_t unit;    // weights are multiples of 2^-unit: V 2^unit < 2^63
};

// round(2^(30 + j / 32))
__device__ constexpr uint32_t kPow2[kTable] = {
    1073741824u, 1097253708u, 1121280436u, 1145833280u, 1170923762u, 1196563654u, 1222764986u, 1249540052u,
    1276901417u, 1304861917u, 1333434672u, 1362633090u, 1392470869u, 1422962010u, 1454120821u, 1485961921u,
    1518500250u, 1551751076u, 1585730000u, 1620452965u, 1655936265u, 1692196547u, 1729250827u, 1767116489u,
    1805811301u, 1845353420u, 1885761398u, 1927054196u, 1969251188u, 2012372174u, 2056437387u, 2101467502u};

// Floats in an order of unsigned numbers (-0 and 0 the same).
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t key) {
  return __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kMinusZero = 0x7fffffffu;  // no key: float_of() of it compares like 0, the key above it
__device__ __forceinline__ uint32_t next_below(uint32_t key) { return key - 1 == kMinusZero ? key - 2 : key - 1; }

// A row's way from a logit to its weight: w = 2^-z, z = top - (l - zero) (c_hi + c_lo), the product
// with what it rounds off.  `zero` is 0 and `top` the largest logit's product, rounded up to
// whole 1/32.  Where that passes 2^13 (a tiny temperature), `zero` is the largest
// logit and `top` 0: logits that have a weight are then so close to it that the difference is
// exact.  (A row whose largest logit is infinite is rewritten first.)
struct Scale {
  float zero, c_hi, c_lo;
  float magic;   // kMagic - top
  float least;   // top - 64: products below count as that, the weight 0; NaN (of -inf) as well
  int unit;
};
constexpr float kMagic = 393216.0f;  // 1.5 2^18: sums with it round to whole multiples of 1/32
constexpr float kMostTop = 8192.0f;

__device__ __forceinline__ Scale scale_of(float max, float c_hi, float c_lo, int unit, float* top) {
  const float y = max * c_hi;
  const bool far = !(fabsf(y) <= kMostTop);
  float up = (y + kMagic) - kMagic;
  if (up < y) up += 1.0f / kTable;
  if (far) up = 0.0f;
  *top = up;
  return Scale{far ? max : 0.0f, c_hi, c_lo, kMagic - up, up - 64.0f, unit};
}

// A logit's weight in units (at most 2^unit and a little), rounded to nearest; n = round(32 z) below.
// `lane_table`: this lane's column of the table of powers, which is there once for every
// lane so that no two lanes meet in a bank.
//
// Packed pairs of fp32 with the sum kept as two fp32 numbers, which saves the 64-bit shift and
// addition, took a tenth longer: their constants need two registers each.
__device__ __forceinline__ U64 weight(float l, const Scale& s, const uint2* lane_table) {
  const float a = l - s.zero;
  const float y = a * s.c_hi;
  const float rest = fmaf(a, s.c_lo, fmaf(a, s.c_hi, -y));
  const float yy = fmaxf(y, s.least);
  const float t = yy + s.magic;
  // |r| <= 1/64 and the rest (below 2^-10, where products are near 2^13); exact but for that; NaN where l is infinite
  const float r = (yy - (t - s.magic)) + rest;
  // 2^r - 1: a polynomial fitted to it (least largest error on |r| <= 1/64: 2^-32.8, 2^-32 with the rest), off by
  // 2^-29.7 as it is worked out here
  const float p = r * fmaf(r, fmaf(r, 0.05550457f, 0.24022846f), 0.6931472f);
  const int up = __float_as_int(kMagic) + (kTable - 1) - __float_as_int(t);  // n + 31
  const uint2 power = lane_table[(up & (kTable - 1)) * 32];
  // 2^30 of its octave, below 2^31, and half a unit where units are cut off
  const int drop = (up >> 5) + 30 - s.unit;
  uint32_t half;
  asm("shl.b32 %0, 1, %1;" : "=r"(half) : "r"(drop - 1));  // 0 for amounts that are negative or 32 and more
  const uint32_t w = power.x + static_cast<uint32_t>(__float2int_rn(__uint_as_float(power.y) * p)) + half;
  U64 out;
  asm("shr.u64 %0, %1, %2;" : "=l"(out) : "l"(static_cast<U64>(w) << 32), "r"(drop + 32));  // 0 from 64 on
  return out;
}

// A logit's bin, round(32 z) with z from the rounded product alone.
__device__ __forceinline__ int bin_of(float l, const Scale& s) {
  const float t = fmaxf((l - s.zero) * s.c_hi, s.least) + s.magic;
  return __float_as_int(kMagic) - __float_as_int(t);
}
// The lowest logit of bins up to b (bins fall as logits rise), not -inf; all lanes of a warp, 32 keys
// at a time.
__device__ __forceinline__ float lowest_in(int b, float max, const Scale& s) {
  uint32_t lo = 0x00800000u;                 // the lowest number
  const uint32_t hi = key_of(max);           // b is its bin or one behind it
#pragma unroll 1
  for (int digit = 27; digit >= 0; digit -= digit == 2 ? 2 : 5) {
    const U64 last = static_cast<U64>(lo) + (static_cast<U64>((threadIdx.x & 31) + 1) << digit) - 1;  // of this lane's share
    const bool reaches = last >= hi || bin_of(float_of(static_cast<uint32_t>(last)), s) <= b;
    lo += static_cast<uint32_t>(__ffs(__ballot_sync(0xffffffffu, reaches)) - 1) << digit;
    if (digit == 0) break;
  }
  return float_of(lo);
}

// ------------------------------------------------------------------ 16-byte pieces
template <typename E>
__device__ __forceinline__ E lowest() {  // -inf
  if constexpr (sizeof(E) == 4) return -INFINITY;
  else return 0xff80u;
}
template <typename E>
struct Piece {
  static constexpr int kPer = 16 / static_cast<int>(sizeof(E));
  float v[kPer];
};
template <typename E>
__device__ __forceinline__ Piece<E> unpack(const uint4& a) {
  Piece<E> r;
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 4) {
      r.v[i] = __uint_as_float(w[i]);
    } else {
      r.v[2 * i] = __uint_as_float(w[i] << 16);
      r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  return r;
}

// The one value of a key's leading 16 bits (bf16), or of a key.
template <typename E>
__device__ __forceinline__ float value_of(uint32_t k) {
  if constexpr (sizeof(E) == 4) return float_of(k);
  else return float_of(k << 16 | (k & 0x8000u ? 0u : 0xffffu));
}
__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// The larger of `best` and a piece's logits; `nan` if one of them is none (best is then unknown).
template <typename E>
__device__ __forceinline__ void largest(const uint4& a, float& best, bool& nan) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  float m;
  if constexpr (sizeof(E) == 4) {
    float x, y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(__uint_as_float(w[0])), "f"(__uint_as_float(w[1])));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(__uint_as_float(w[2])), "f"(__uint_as_float(w[3])));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
  } else {
    uint32_t x, y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w[0]), "r"(w[1]));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w[2]), "r"(w[3]));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(y));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(__uint_as_float(x << 16)), "f"(__uint_as_float(x & 0xffff0000u)));
  }
  nan = nan || m != m;
  best = fmaxf(best, m);
}

// ------------------------------------------------------------------ the cluster
struct Two {
  U64 a, b;
};
struct Sum {
  static __device__ __forceinline__ Two of(Two x, Two y) { return Two{x.a + y.a, x.b + y.b}; }
  static constexpr Two kNone{0, 0};
};
struct MaxMin {
  static __device__ __forceinline__ Two of(Two x, Two y) { return Two{x.a > y.a ? x.a : y.a, x.b < y.b ? x.b : y.b}; }
  static constexpr Two kNone{0, ~0ull};
};

struct Plan {  // what the first CTA finds out and tells the others
  U64 mass;
  uint32_t a, b, c, d;
};

struct Shared {
  Two part[kMaxWarps];
  Two from[2][kMaxCtas];
  Plan plan[2];
  double log_min;
  U64 need;
  float c_hi, c_lo, min_logit;
  uint32_t listed, found[3];
  U64 before;
};

template <typename T>
__device__ __forceinline__ T* peer(T* p, int rank) {
  uint64_t r;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<T*>(r);
}

struct Cluster {
  int ctas, rank;
  Shared* s;
  int turn, plans;
  __device__ __forceinline__ void sync() const {
    __syncwarp();
    if (ctas == 1)
      __syncthreads();
    else
      ptx::cluster_sync();
  }
  // Every warp's value, in part[] after a barrier.
  template <typename Op>
  __device__ __forceinline__ void sum_warps(Two v) const {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      v = Op::of(v, Two{__shfl_xor_sync(0xffffffffu, v.a, d), __shfl_xor_sync(0xffffffffu, v.b, d)});
    if ((threadIdx.x & 31) == 0) s->part[threadIdx.x >> 5] = v;
  }
  // Every CTA's value, in from[], for all threads of all CTAs.
  template <typename Op>
  __device__ __forceinline__ const Two* gather(Two v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    sum_warps<Op>(v);
    __syncthreads();
    if (warp == 0) {
      v = lane < warps ? s->part[lane] : Op::kNone;
#pragma unroll
      for (int d = 8; d > 0; d >>= 1)
        v = Op::of(v, Two{__shfl_xor_sync(0xffffffffu, v.a, d), __shfl_xor_sync(0xffffffffu, v.b, d)});
      v = Two{__shfl_sync(0xffffffffu, v.a, 0), __shfl_sync(0xffffffffu, v.b, 0)};
      if (lane < ctas) *peer(&s->from[turn][rank], lane) = v;
    }
    sync();
    const Two* r = s->from[turn];
    turn ^= 1;  // the next one but one writes here: every thread has read it by the barrier between
    return r;
  }
  __device__ __forceinline__ const Two* last() const { return s->from[turn ^ 1]; }  // what it returned
  template <typename Op>
  __device__ __forceinline__ Two all(Two v) {
    const Two* f = gather<Op>(v);
    v = f[0];
    for (int i = 1; i < ctas; ++i) v = Op::of(v, f[i]);
    return v;
  }
  // The first CTA's plan, given by all its threads, to all.
  __device__ __forceinline__ Plan tell(const Plan& plan) {
    Plan* at = s->plan + plans;
    if (rank == 0 && threadIdx.x < ctas) *peer(at, threadIdx.x) = plan;
    sync();
    plans ^= 1;  // as turn
    return *at;
  }
};

// Exclusive prefix sums over the block's threads.
__device__ __forceinline__ Two block_before(Two v, Shared* s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Two incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Two o{__shfl_up_sync(0xffffffffu, incl.a, d), __shfl_up_sync(0xffffffffu, incl.b, d)};
    if (lane >= d) incl = Sum::of(incl, o);
  }
  __syncthreads();
  if (lane == 31) s->part[warp] = incl;
  __syncthreads();
  Two before{incl.a - v.a, incl.b - v.b};
  for (int i = 0; i < warp; ++i) before = Sum::of(before, s->part[i]);
  return before;
}
__device__ __forceinline__ U64 block_before(U64 v, Shared* s) { return block_before(Two{v, 0}, s).a; }

// The least whole number that is f m or more, the product rounded to 53 bits: 0.9 of 4000 equal
// weights are 3600 of them, although the number nearest to 0.9 is a little more.
__device__ __forceinline__ U64 share_up(double f, U64 m) { return __double2ull_ru(f * __ull2double_rn(m)); }
// floor(f m) for f in [0, 1) as a whole multiple of 2^-63.
__device__ __forceinline__ U64 share_down(U64 f, U64 m) { return __umul64hi(f, m) << 1 | (f * m) >> 63; }

// ------------------------------------------------------------------ sorting
// A bitonic sort of `size` numbers (a power of two, R * 32 and more), the largest first; all
// threads of a CTA.  Steps within stretches of R * 32 are a warp's, in registers (R numbers to a
// lane); only steps between stretches go through shared memory and the block's barrier.
template <int R>
__device__ __forceinline__ void merge_stretch(U64 (&v)[R], int base, int k, int j0, int lane) {
  for (int j = j0; j > 0; j /= 2) {
    if (j >= 32) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int step = 1; step < R; step *= 2)
          if (step * 32 == j && !(r & step)) {
            const bool first_largest = ((base + r * 32) & k) == 0;
            const U64 x = v[r], y = v[r | step];
            if ((x < y) == first_largest) v[r] = y, v[r | step] = x;
          }
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const U64 other = __shfl_xor_sync(0xffffffffu, v[r], j);
        const bool largest = ((lane & j) == 0) == (((base + r * 32 + lane) & k) == 0);
        if ((other > v[r]) == largest) v[r] = other;
      }
    }
  }
}
template <int R>
__device__ __forceinline__ void sort_stretches(U64* a, int size) {
  constexpr int kStretch = R * 32;
  const int tid = threadIdx.x, lane = tid & 31;
  for (int k = kStretch; k <= size; k *= 2) {
    for (int j = k / 2; j >= kStretch; j /= 2) {
      for (int i = tid; i < size / 2; i += blockDim.x) {
        const int x = 2 * i - (i & (j - 1)), y = x + j;
        const U64 vx = a[x], vy = a[y];
        if ((vx < vy) == ((x & k) == 0)) a[x] = vy, a[y] = vx;
      }
      __syncthreads();
    }
    for (int base = (tid >> 5) * kStretch; base < size; base += static_cast<int>(blockDim.x >> 5) * kStretch) {
      U64 v[R];
#pragma unroll
      for (int r = 0; r < R; ++r) v[r] = a[base + r * 32 + lane];
      if (k == kStretch) {
        for (int kk = 2; kk < kStretch; kk *= 2) merge_stretch(v, base, kk, kk / 2, lane);
      }
      merge_stretch(v, base, k, kStretch / 2, lane);
#pragma unroll
      for (int r = 0; r < R; ++r) a[base + r * 32 + lane] = v[r];
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ the kernel
// The pieces of a CTA's part of a row: 16 bytes as they lie in memory; what a piece holds before
// or behind the row counts as -inf.  A warp has a stretch of its own and a lane a stretch of
// that, so that sums of lanes are sums of the vocabulary's order; pieces are swizzled (place_of)
// so that the lanes of a load meet few banks twice.
__device__ __forceinline__ int place_of(int piece) { return piece ^ ((piece >> 3) & 7); }
__host__ __device__ constexpr size_t piece_bytes(int chunk) { return static_cast<size_t>((chunk + 7) / 8 * 8) * 16; }  // whole eights

// SEARCH: some row may have top-k or top-p.  Without, nothing is counted or listed, and three CTAs fit on
// an SM instead of two (256 x 124,160 fp32: 86 us, 97 in the other form).
template <typename E, bool SEARCH>
__global__ void __launch_bounds__(kMaxThreads, SEARCH ? 2 : 3) sample_kernel(const Params p) {
  constexpr int kPer = Piece<E>::kPer;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  uint4* const pieces = reinterpret_cast<uint4*>(smem);
  uint2* const table = reinterpret_cast<uint2*>(smem + piece_bytes(p.chunk));
  uint32_t* const bins = reinterpret_cast<uint32_t*>(table + kTable * 32);
  U64* const list = reinterpret_cast<U64*>(bins + kBins);
  U64* const mass_of = list + kList;                               // sums of the sorted list's weights
  uint32_t* const group_max = reinterpret_cast<uint32_t*>(mass_of);  // before that: of every group of the row

  const int threads = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Cluster cl{p.ctas, static_cast<int>(blockIdx.x % p.ctas), &sh, 0, 0};
  if (p.ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // for the wait below
  const int64_t row = blockIdx.x / p.ctas;
  const uint2* const lane_table = table + lane;

  for (int i = tid; i < kTable * 32; i += threads) {  // entry m: 2^((31 - m) / 32), for n + 31 = m modulo 32
    const uint32_t t = kPow2[kTable - 1 - i / 32];
    table[i] = make_uint2(t, __float_as_uint(static_cast<float>(t)));
  }
  ptx::launch_dependents();
  ptx::wait_prerequisites();

  const E* const logits = static_cast<const E*>(p.logits) + row * p.ldl;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(logits) & 15) / static_cast<int>(sizeof(E));
  const int first = cl.rank * p.chunk;
  const int mine = max(0, min(p.chunk, (off + p.V + kPer - 1) / kPer - first));
  const int whole0 = first == 0 && off ? 1 : 0, whole1 = min(mine, (off + p.V) / kPer - first);  // pieces that the row fills
  const int run = (p.chunk + threads - 1) / threads;  // of a lane
  const int w0 = warp * 32 * run, w1 = min(w0 + 32 * run, mine);
  const int l0 = min(w0 + lane * run, w1), l1 = min(l0 + run, w1);
  {
    const uint8_t* from = reinterpret_cast<const uint8_t*>(logits - off) + 16 * static_cast<int64_t>(first + w0 + lane);
    const uint32_t to = ptx::smem_u32(pieces);
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32, from += 512) {
      if (i >= whole0 && i < whole1) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * place_of(i)), "l"(from) : "memory");
      } else {
        const int at = (first + i) * kPer - off;  // the piece's first logit
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          reinterpret_cast<E*>(pieces + place_of(i))[e] = at + e >= 0 && at + e < p.V ? logits[at + e] : lowest<E>();
      }
    }
  }
  // In 32 bits what every thread needs; 64-bit arithmetic, of which an SM does two a cycle, is
  // one thread's (256 x 124,160 fp32: 20 us less).
  const float temperature = p.temperature ? p.temperature[row] : p.temperature_like;
  const int64_t top_k = p.top_k ? p.top_k[row] : p.top_k_all;
  const float top_p = p.top_p ? p.top_p[row] : p.top_p_like;
  const float min_p = p.min_p ? p.min_p[row] : p.min_p_like;
  const float u = p.u[row];
  const bool greedy = !(temperature > 0.0f) || top_k == 1 || top_p <= 0.0f;
  const bool by_k = SEARCH && top_k > 0, by_p = SEARCH && top_p < 1.0f, by_min = min_p > 0.0f;
  if (tid == 0) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;  // log2(e)
    if (greedy) {
      sh.c_hi = 1.0f, sh.c_lo = 0.0f;
    } else if (!p.temperature) {
      sh.c_hi = p.c_hi_all, sh.c_lo = p.c_lo_all;
    } else {
      const float c = fminf(kHi / temperature, 1e37f);
      sh.c_hi = c;
      sh.c_lo = c < 1e37f && temperature < INFINITY ? (fmaf(-c, temperature, kHi) + kLo) / temperature : 0.0f;
    }
    sh.log_min = 0.0;
    if (by_min && !greedy)  // at an infinite temperature every weight is 1, which none of up to 1 cuts off
      sh.log_min = temperature == INFINITY && min_p <= 1.0f ? -INFINITY : (p.temperature ? static_cast<double>(temperature) : p.temperature_all) *
                   (p.min_p ? log(static_cast<double>(min_p)) : p.log_min_p_all);
    sh.listed = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  float quarter[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // the largest of every fourth piece
  bool nan = false;
  for (int i = l0; i < l1; i += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < l1) largest<E>(pieces[place_of(i + j)], quarter[j], nan);
  }
  if (__any_sync(0xffffffffu, nan)) {  // never drawn
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      quarter[j] = -INFINITY;
      for (int i = l0 + j; i < l1; i += 4) {
        const Piece<E> l = unpack<E>(pieces[place_of(i)]);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (l.v[e] != l.v[e]) reinterpret_cast<E*>(pieces + place_of(i))[e] = lowest<E>();
          quarter[j] = fmaxf(quarter[j], l.v[e]);
        }
      }
    }
  }
  const float best = fmaxf(fmaxf(quarter[0], quarter[1]), fmaxf(quarter[2], quarter[3]));
  if (p.ctas > 1) {  // the others' shared memory is there
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  // The largest logits of up to 2048 groups of the row, to every CTA: at least k logits are no
  // smaller than the k-th largest of them.  With k above half of the groups that bound lets too many pass.
  const int groups = min(4 * threads, kGroups / p.ctas);  // of a CTA
  const bool short_k = !greedy && by_k && top_k <= groups * p.ctas / 2 + 128;
  if (short_k) {
    if (groups >= threads) {  // 1, 2 or 4 to a thread
      const int each_thread = groups / threads;
      for (int r = 0; r < p.ctas; ++r) {
        uint32_t* to = peer(group_max, r) + cl.rank * groups + tid;
        if (each_thread == 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) to[j * threads] = key_of(quarter[j]);
        } else if (each_thread == 2) {
          to[0] = key_of(fmaxf(quarter[0], quarter[1])), to[threads] = key_of(fmaxf(quarter[2], quarter[3]));
        } else {
          to[0] = key_of(best);
        }
      }
    } else {
      float g = best;
      const int lanes = threads / groups;  // a power of two
      for (int d = lanes / 2; d > 0; d >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
      for (int r = tid & (lanes - 1); r < p.ctas; r += lanes) peer(group_max, r)[cl.rank * groups + tid / lanes] = key_of(g);
    }
  }
  float row_max = float_of(static_cast<uint32_t>(cl.all<MaxMin>(Two{key_of(best), ~0ull}).a));
  const float real_max = row_max;
  if (row_max == -INFINITY) {  // nothing to draw
    if (cl.rank == 0 && tid == 0) {
      p.tokens[row] = p.ignore_index;
      if (p.logp) p.logp[row] = 0.0f;
    }
    return;
  }
  if (row_max == INFINITY) {  // the infinite ones alone, as equals
    for (int i = l0; i < l1; ++i) {
      const Piece<E> l = unpack<E>(pieces[place_of(i)]);
#pragma unroll
      for (int e = 0; e < kPer; ++e) reinterpret_cast<E*>(pieces + place_of(i))[e] = l.v[e] == INFINITY ? static_cast<E>(0) : lowest<E>();
    }
    row_max = 0.0f;
  }
  float top;
  const Scale sc = scale_of(row_max, sh.c_hi, sh.c_lo, p.unit, &top);
  float least = -INFINITY;  // of min-p
  if (by_min) {
    if (tid == 0) sh.min_logit = fminf(__double2float_ru(static_cast<double>(row_max) + sh.log_min), row_max);
    __syncthreads();
    least = sh.min_logit;
  }
  const auto each_piece = [&](auto f) {
    for (int i = l0; i < l1; ++i) f(unpack<E>(pieces[place_of(i)]));
  };
  const auto write = [&](int64_t token, U64 total) {  // one thread: the token, and log(its weight / total)
    p.tokens[row] = token;
    if (!p.logp) return;
    const float drawn = as_float(logits[token]), l = drawn == INFINITY ? 0.0f : drawn;
    const U64 w = weight(l, sc, lane_table);
    // Pairs of fp32 numbers: 64-bit arithmetic took 5 us longer for each row.
    const auto pair_of = [](U64 v) {
      const float hi = __ull2float_rz(v);
      return Twofold{hi, static_cast<float>(v - static_cast<U64>(hi))};
    };
    float log_p;
    if (w > total - w) {  // -log1p(others / this one): keeps its digits near 0
      const Twofold a = pair_of(total - w), b = pair_of(w);
      const float q = a.hi / b.hi, rest = (fmaf(-q, b.hi, a.hi) + (a.lo - q * b.lo)) / b.hi;
      log_p = -(log1pf(q) + rest / (1.0f + q));
    } else {  // log 2 (y - top - the total's exponent) - log(its leading digits), y from the logit
      constexpr float kHi = 0.693147182f, kLo = -1.90465421e-9f;  // log 2
      const int exponent = 63 - __clzll(total);
      const Twofold lead = pair_of(total << (63 - exponent));
      const float a = l - sc.zero, y = a * sc.c_hi;
      const Twofold v = Twofold{y, fmaf(a, sc.c_lo, fmaf(a, sc.c_hi, -y))} + Twofold{-top, 0.0f} +
                        Twofold{static_cast<float>(p.unit - exponent), 0.0f};
      const float m = v.hi * kHi;
      const Twofold sum = Twofold{m, fmaf(v.hi, kHi, -m) + fmaf(v.hi, kLo, v.lo * kHi)} +
                          Twofold{-logf(lead.hi * 0x1p-63f), -lead.lo / lead.hi};
      log_p = sum.hi + sum.lo;
    }
    p.logp[row] = greedy ? 0.0f : log_p;
  };
  const U64 u_share = u > 0.0f ? static_cast<U64>(fminf(u, 0x1.fffffep-1f) * 0x1p63f) : 0;

  // ---- the list: logits from `low` to `high`, unsorted, on the first CTA.  Returns how many there are.
  // With `sums` also the weights of all.
  const auto gather_list = [&](float low, float high, bool sums = false, U64* total = nullptr) -> U64 {
    const auto hits_of = [&](const Piece<E>& l) {
      uint32_t hits = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) hits |= l.v[e] >= low && l.v[e] <= high ? 1u << e : 0u;
      return hits;
    };
    U64 sum = 0;
    int count = 0;  // of this lane; then one addition for the warp finds them their places
    each_piece([&](const Piece<E>& l) {
      count += __popc(hits_of(l));
      if (sums) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) sum += weight(l.v[e], sc, lane_table);
      }
    });
    int incl = count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    uint32_t at = 0;
    if (lane == 31 && incl) at = atomicAdd(peer(&sh.listed, 0), static_cast<uint32_t>(incl));
    at = __shfl_sync(0xffffffffu, at, 31) + incl - count;
    if (count) {
      U64* const to = peer(list, 0);
      for (int i = l0; i < l1; ++i) {
        const Piece<E> l = unpack<E>(pieces[place_of(i)]);
        const uint32_t hits = hits_of(l);
        if (!hits) continue;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (hits >> e & 1u) {
            if (at < kList)
              to[at] = static_cast<U64>(key_of(l.v[e])) << 32 | (0xffffffffu - static_cast<uint32_t>((first + i) * kPer + e - off));
            ++at;
          }
      }
    }
    const Two all = cl.all<Sum>(Two{static_cast<U64>(count), sum});
    if (sums) *total = all.b;
    return all.a;
  };
  const auto listed = [&](U64 count) { return static_cast<int>(count < kList ? count : kList); };
  const auto key_in_list = [&](int i) { return float_of(static_cast<uint32_t>(list[i] >> 32)); };
  // Sorts m numbers, the largest first; all threads of a CTA.
  const auto sort = [&](U64* a, int m) {
    int size = 64;
    while (size < m) size *= 2;
    for (int i = m + tid; i < size; i += threads) a[i] = 0;
    __syncthreads();
    if (size == 64) sort_stretches<2>(a, size);
    else sort_stretches<4>(a, size);
  };
  // The sums of the sorted list's weights up to each.
  const auto sum_list = [&](int m) {
    const int per = (m + threads - 1) / threads, a = min(tid * per, m), b = min(a + per, m);
    U64 sum = 0;
    for (int i = a; i < b; ++i) sum += weight(key_in_list(i), sc, lane_table);
    U64 run = block_before(sum, &sh);
    for (int i = a; i < b; ++i) mass_of[i] = run += weight(key_in_list(i), sc, lane_table);
    __syncthreads();
  };
  const auto share_of = [&](U64 total) {  // p of it; one thread
    return share_up(p.top_p ? static_cast<double>(top_p) : p.top_p_all, total);
  };
  // How many of the first m of the list it takes for weights of `wanted`.
  const auto prefix_of = [&](int m, U64 wanted) -> int {  // 0: p of their sum
    __syncthreads();
    if (tid == 0) sh.found[0] = static_cast<uint32_t>(m), sh.need = wanted ? wanted : share_of(mass_of[m - 1]);
    __syncthreads();
    const U64 need = sh.need;
    for (int i = tid; i < m; i += threads)
      if (mass_of[i] >= need && (i == 0 || mass_of[i - 1] < need)) sh.found[0] = static_cast<uint32_t>(i) + 1;
    __syncthreads();
    return static_cast<int>(sh.found[0]);
  };
  // The first CTA: top-k (k > 0), top-p (need > 0: the weights wanted; all of top_p otherwise) and
  // min-p on the list of m, which holds all of them, and the draw.
  const auto draw_from_list = [&](int m, int64_t k, U64 need) {
    if (m <= kFewer) {
      // Every one against every other, `share` threads to one: its place and the weights up to it,
      // and then the kept weights up to it in the vocabulary.  Four barriers instead of two sorts'.
      const int share = m <= threads / 16 ? 16 : m <= threads / 8 ? 8 : m <= threads / 4 ? 4 : m <= threads / 2 ? 2 : 1;
      const int mine_at = tid / share, part = tid % share;
      const bool live = mine_at < m;
      __syncthreads();
      for (int i = tid; i < m; i += threads) mass_of[i] = weight(key_in_list(i), sc, lane_table);
      __syncthreads();
      const U64 self = live ? list[mine_at] : 0, w = live ? mass_of[mine_at] : 0;
      U64 up_to = 0;
      int place = 0;
      for (int j = part; j < m; j += share) {
        const U64 other = list[j], w_j = mass_of[j];
        up_to += other >= self ? w_j : 0;
        place += other > self ? 1 : 0;
      }
      for (int d = share / 2; d > 0; d >>= 1) up_to += __shfl_xor_sync(0xffffffffu, up_to, d), place += __shfl_xor_sync(0xffffffffu, place, d);
      const int many = k > 0 && k < m ? static_cast<int>(k) : m;
      if (live && part == 0 && place == many - 1) sh.need = !by_p ? ~0ull : need ? need : share_of(up_to);
      __syncthreads();
      const bool keep = live && place < many && up_to - w < sh.need && float_of(static_cast<uint32_t>(self >> 32)) >= least;
      if (live && part == 0) mass_of[mine_at] = keep ? w : 0;
      __syncthreads();
      U64 total = 0, before = 0;
      const uint32_t self_index = static_cast<uint32_t>(self);  // ~index
      for (int j = part; j < m; j += share) {
        const U64 w_j = mass_of[j];
        total += w_j;
        before += static_cast<uint32_t>(list[j]) > self_index ? w_j : 0;
      }
      for (int d = share / 2; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d), before += __shfl_xor_sync(0xffffffffu, before, d);
      const U64 target = share_down(u_share, total);
      if (keep && part == 0 && before <= target && target < before + w) write(static_cast<int64_t>(0xffffffffu - self_index), total);
      return;
    }
    sort(list, m);
    sum_list(m);
    if (k > 0 && k < m) m = static_cast<int>(k);
    if (by_p) m = prefix_of(m, need);
    if (by_min) {  // a prefix as well
      __syncthreads();
      if (tid == 0) sh.found[0] = static_cast<uint32_t>(m);
      __syncthreads();
      for (int i = tid; i < m; i += threads)
        if (key_in_list(i) < least && (i == 0 || key_in_list(i - 1) >= least)) sh.found[0] = static_cast<uint32_t>(i);
      __syncthreads();
      m = static_cast<int>(sh.found[0]);
    }
    const U64 total = mass_of[m - 1], target = share_down(u_share, total);
    // by index, the first first, each with its weight behind it: 63 - unit and unit + 1 bits
    const int weight_bits = p.unit + 1;
    __syncthreads();
    for (int i = tid; i < m; i += threads) {
      const U64 w = mass_of[i] - (i ? mass_of[i - 1] : 0);
      list[i] = list[i] << weight_bits | w;  // of ~index
    }
    sort(list, m);
    const int per = (m + threads - 1) / threads, a = min(tid * per, m), b = min(a + per, m);
    const U64 weights_only = (1ull << weight_bits) - 1;
    U64 sum = 0;
    for (int i = a; i < b; ++i) sum += list[i] & weights_only;
    U64 run = block_before(sum, &sh);
    for (int i = a; i < b; ++i) {
      const U64 next = run + (list[i] & weights_only);
      if (run <= target && target < next) write(static_cast<int64_t>(~(list[i] >> weight_bits) & ((1ull << (64 - weight_bits)) - 1)), total);
      run = next;
    }
  };

  // ---- what is kept: l > t, and the first n of l == t.  `own`: this thread's weights of l > sure,
  // known already (sure: +inf if none).
  float t = -INFINITY, sure = INFINITY;
  uint32_t n = 0;
  Two own{0, 0};
  uint32_t last_step = 0;  // not 0: list[i] is the weight of the value of key (bf16: of leading 16 bits) last_step - i,
  uint32_t skipped = 0;    // or for keys up to kNegative last_step - skipped - i, and none is there between them and kPositive
  if (greedy) t = row_max, n = 1;

  // top-p of bf16 logits, by value.  Few thousand values have a weight (128 to an octave of the logit;
  // those within 2^-8 of 0, of which there are endless octaves, are weighed where they are met): the
  // logits of each are counted, each CTA adds up and weighs its share of the values, and where p of the sum
  // is reached among them is the end.  Rows of much fewer words than there are values are listed instead
  // (p = 0.95, normal logits of deviation 2, temperature 1: 256 x 1000 34 us listed, 21 counted; 256 x 4096 50 and 19;
  // 256 x 100 18 and 24.  Temperature 0.3, nuclei of some words: 256 x 1000 17 and 19, 2000 x 1000 65 and 72;
  // 0.1, fewer values: 17 and 10, 64 and 38.  How long the nucleus is, which would tell, is known after counting.)
  bool counted = false, alone = false;
  if constexpr (sizeof(E) == 2) {
    if (!greedy && by_p && !by_k) {
      const uint32_t top_key = key_of(row_max) >> 16, low_key = key_of(lowest_in(kLive - 1, row_max, sc)) >> 16;
      const uint32_t gap = top_key >= kPositive ? kPositive - kNegative - 1 : 0;
      const auto middle = [&](uint32_t k) { return k < kPositive && k > kNegative; };
      const auto index_of = [&](uint32_t k) { return top_key - k - (k <= kNegative ? gap : 0); };
      const int above = gap ? static_cast<int>(top_key - kPositive) + 1 : 0;  // values before the middle
      const int values = middle(low_key) ? above : static_cast<int>(index_of(low_key)) + 1;
      const auto key_at = [&](int i) { return top_key - i - (i >= above ? gap : 0); };
      if (!middle(top_key) && values <= kValues && values <= 4 * p.V) {
        uint32_t* const counts = reinterpret_cast<uint32_t*>(mass_of);      // of this CTA
        uint32_t* const row_counts = reinterpret_cast<uint32_t*>(list);     // of the row, its share
        __syncthreads();
        for (int i = tid; i < values; i += threads) counts[i] = 0;
        __syncthreads();
        U64 mid = 0;
        each_piece([&](const Piece<E>& l) {
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const uint32_t k = key_of(l.v[e]) >> 16;
            const uint32_t i = index_of(k);
            if (middle(k)) mid += weight(l.v[e], sc, lane_table);
            else if (i < static_cast<uint32_t>(values)) atomicAdd(counts + i, 1u);
          }
        });
        cl.sync();
        const int each = (values + p.ctas - 1) / p.ctas, v0 = min(cl.rank * each, values), v1 = min(v0 + each, values);
        const int per = (each + threads - 1) / threads, a = min(v0 + tid * per, v1), b = min(a + per, v1);
        U64 here = 0;
        for (int i = a; i < b; ++i) {
          uint32_t c = 0;
          for (int r = 0; r < p.ctas; ++r) c += *peer(counts + i, r);
          row_counts[i] = c;
          here += c * weight(value_of<E>(key_at(i)), sc, lane_table);
        }
        const Two* from = cl.gather<Sum>(Two{here, mid});
        U64 run = 0, sum = 0, mids = 0;
        for (int r = 0; r < p.ctas; ++r) {
          if (r == cl.rank) run = sum;
          sum += from[r].a, mids += from[r].b;
        }
        __syncthreads();
        if (tid == 0) sh.need = share_up(p.top_p ? static_cast<double>(top_p) : p.top_p_all, sum + mids);
        run += block_before(here, &sh);
        const U64 need = sh.need;
        Two end{0, 0};
        for (int i = a; i < b; ++i) {
          const U64 w = weight(value_of<E>(key_at(i)), sc, lane_table), before = run + (i >= above && gap ? mids : 0);
          if (before < need && before + row_counts[i] * w >= need)
            end = Two{(need - before + w - 1) / w, static_cast<U64>(key_at(i)) + 1};
          run += row_counts[i] * w;
        }
        __syncthreads();  // the sums before are read
        end = cl.all<Sum>(end);
        counted = end.b != 0;  // else it ends in the middle
        if (counted) {
          const uint32_t key = static_cast<uint32_t>(end.b) - 1;
          t = value_of<E>(key), n = static_cast<uint32_t>(end.a);
          sure = row_max, last_step = top_key, skipped = key <= kNegative ? gap : 0;
          if (p.ctas > 1 && !by_min) {  // the CTA that the draw falls to goes on alone
            const int last = static_cast<int>(index_of(key));
            Two own_kept{skipped ? mid : 0, tid == 0 ? counts[last] : 0u};
            for (int i = tid; i < last; i += threads)
              if (counts[i]) own_kept.a += counts[i] * weight(value_of<E>(key_at(i)), sc, lane_table);
            const Two* kept_by = cl.gather<Sum>(own_kept);
            const U64 w_t = weight(t, sc, lane_table);
            const auto up_to = [&](const Two& v) { return v.a + (v.b < n ? v.b : static_cast<U64>(n)) * w_t; };
            Two before{0, 0}, all{0, 0};
            for (int r = 0; r < p.ctas; ++r) {
              if (r == cl.rank) before = all;
              all = Sum::of(all, kept_by[r]);
            }
            const U64 target = share_down(u_share, up_to(all));
            if (!(up_to(before) <= target && target < up_to(Sum::of(before, kept_by[cl.rank])))) return;
            alone = true;
          }
          for (int i = tid; i < static_cast<int>(index_of(key)); i += threads) list[i] = weight(value_of<E>(key_at(i)), sc, lane_table);
          __syncthreads();
        }
      }
    }
  }

  if (!counted && !greedy && (by_k || by_p)) {
    if (short_k && real_max < INFINITY) {
      // Every CTA finds the same bound.
      for (int i = tid; i < kBins; i += threads) bins[i] = 0;
      __syncthreads();
      for (int i = tid; i < groups * p.ctas; i += threads) {
        const float l = float_of(group_max[i]);
        const int b = bin_of(l, sc);
        if (static_cast<uint32_t>(b) < kLive) atomicAdd(bins + b, 1u);
      }
      const int per = kBins / threads;
      __syncthreads();
      U64 count = 0;
      for (int i = tid * per; i < (tid + 1) * per; ++i) count += bins[i];
      U64 run = block_before(count, &sh);
      if (tid == 0) sh.found[0] = kBins;
      __syncthreads();
      if (run < static_cast<U64>(top_k) && run + count >= static_cast<U64>(top_k))
        for (int i = tid * per; i < (tid + 1) * per; ++i) {
          if (run < static_cast<U64>(top_k) && run + bins[i] >= static_cast<U64>(top_k)) sh.found[0] = i;
          run += bins[i];
        }
      __syncthreads();
      const int b = static_cast<int>(sh.found[0]);
      if (b < kBins) {
        const U64 m = gather_list(lowest_in(b, row_max, sc), INFINITY);
        if (m <= kList) {
          if (cl.rank == 0) draw_from_list(listed(m), top_k, 0);
          return;
        }
        __syncthreads();
        if (tid == 0) sh.listed = 0;  // seen by the others after the next barrier
      }
    }
    // How many logits fall into each bin.
    __syncthreads();
    for (int i = tid; i < kBins; i += threads) bins[i] = 0;
    __syncthreads();
    each_piece([&](const Piece<E>& l) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int b = bin_of(l.v[e], sc);
        if (static_cast<uint32_t>(b) < kLive) atomicAdd(bins + b, 1u);
      }
    });
    cl.sync();
    // The first CTA adds up the bins of all: bins[b] = how many lie in bins up to b.
    const int per = kBins / threads;
    if (cl.rank == 0) {
      uint32_t count = 0;
      for (int i = tid * per; i < (tid + 1) * per; ++i) {
        uint32_t c = bins[i];
        for (int r = 1; r < p.ctas; ++r) c += *peer(bins + i, r);
        bins[i] = c;
        count += c;
      }
      uint32_t run = static_cast<uint32_t>(block_before(count, &sh));
      for (int i = tid * per; i < (tid + 1) * per; ++i) bins[i] = run += bins[i];
      __syncthreads();
    }
    // Bins [a, b] that hold the end of the shortest prefix with `of` logits, or with p of the
    // weights `of` (0: of all, which the bins bound); how many lie up to b (c) and above a (d); and
    // in all, or what p of the weights `of` is.
    const auto bracket = [&](bool mass, U64 of) {
      Plan plan{};
      if (cl.rank == 0) {
        __syncthreads();
        if (tid == 0) {
          sh.found[0] = sh.found[1] = kLive - 1;  // not behind: nothing has been counted there
          sh.need = mass && of ? share_of(of) : of;
        }
        __syncthreads();
        U64 need = sh.need;
        if (!mass) {
          for (int i = tid; i < kBins; i += threads)
            if (bins[i] >= need && (i == 0 || bins[i - 1] < need)) sh.found[0] = sh.found[1] = i;
        } else {  // between the bounds of their weights
          // A bin is that of the rounded product, a weight that of the product with its rest, which is below
          // 2^-23 + 2^-26 of it (what it rounds off, and c_lo): 2^-10 where it is near 2^13.
          const float unit_f = __uint_as_float(static_cast<uint32_t>(127 + p.unit) << 23);
          const float half = 0.5f / kTable + 0x1p-22f * fmaxf(fabsf(sc.least), fabsf(sc.least + 64.0f));
          const auto bounds = [&](int i) {
            const U64 c = bins[i] - (i ? bins[i - 1] : 0u);
            const float y = static_cast<float>(-i) * (1.0f / kTable);
            const U64 lower = static_cast<U64>(ptx::ex2(y - half) * (1.0f - 0x1p-15f) * unit_f);
            return Two{c * (static_cast<U64>(ptx::ex2(y + half) * (1.0f + 0x1p-15f) * unit_f) + 2), c * (lower ? lower - 1 : 0)};
          };
          Two here{0, 0};
          for (int i = tid * per; i < (tid + 1) * per; ++i) here = Sum::of(here, bounds(i));
          Two run = block_before(here, &sh);
          U64 most = need;
          if (!of) {  // p of the least and of the most that all may weigh
            __syncthreads();
            if (tid == threads - 1) sh.need = share_of(run.b + here.b), sh.before = share_of(run.a + here.a);
            __syncthreads();
            need = sh.need, most = sh.before;
          }
          for (int i = tid * per; i < (tid + 1) * per; ++i) {
            const Two next = Sum::of(run, bounds(i));
            if (run.a < need && next.a >= need) sh.found[0] = i;
            if (run.b < most && next.b >= most) sh.found[1] = i;
            run = next;
          }
        }
        __syncthreads();
        plan = Plan{mass ? sh.need : bins[kBins - 1], sh.found[0], sh.found[1], bins[sh.found[1]], sh.found[0] ? bins[sh.found[0] - 1] : 0u};
      }
      return cl.tell(plan);
    };
    // The end of that prefix, where more logits share its bins than can be sorted: they are counted
    // again by their values, in steps as fine as the bins allow, until a step holds one value (bf16:
    // nearly always at once) or few enough logits to sort.  The end has to lie in the bins given: weights above them
    // are less than wanted, and with theirs enough.  Returns the threshold, how many of
    // its equals (b), and the prefix's weight.
    const auto narrow = [&](bool by_mass, U64 need, const Plan& in) {  // need 0: p of all weights
      uint32_t* const steps = group_max;  // kBins of them
      uint32_t lo = key_of(lowest_in(static_cast<int>(in.b), row_max, sc));
      uint32_t hi = in.d ? next_below(key_of(lowest_in(static_cast<int>(in.a) - 1, row_max, sc))) : key_of(row_max);
      U64 above = 0, above_n = in.d;  // weights and number of logits above hi
      sure = INFINITY, own = Two{0, 0};
      Plan plan{};
      while (true) {
        int shift = sizeof(E) == 2 ? 16 : 0;
        while ((hi >> shift) - (lo >> shift) >= kBins) ++shift;
        const bool single = shift == (sizeof(E) == 2 ? 16 : 0);  // a step is one value
        for (int i = tid; i < kBins; i += threads) steps[i] = 0;
        __syncthreads();
        const float low = float_of(lo), high = float_of(hi), known = sure;
        const uint32_t last = hi >> shift;
        U64 sum = 0, total = 0;
        const bool want_total = by_mass && !need;
        if (known == INFINITY) {  // the first round: most of the row
          each_piece([&](const Piece<E>& l) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const U64 w = weight(l.v[e], sc, lane_table);
              total += w;
              if (l.v[e] > high) sum += w;
              else if (l.v[e] >= low) atomicAdd(steps + (last - (key_of(l.v[e]) >> shift)), 1u);
            }
          });
        } else {
          each_piece([&](const Piece<E>& l) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              if (l.v[e] > high && l.v[e] <= known) sum += weight(l.v[e], sc, lane_table);
              else if (l.v[e] >= low && l.v[e] <= high) atomicAdd(steps + (last - (key_of(l.v[e]) >> shift)), 1u);
            }
          });
        }
        own.a += sum, sure = high;
        const Two sums = cl.all<Sum>(Two{sum, total});
        above += sums.a;
        if (want_total && cl.rank == 0) {
          if (tid == 0) sh.need = share_of(sums.b);
          __syncthreads();
          need = sh.need;
        }
        if (cl.rank == 0) {
          // The sums up to a step, least and most: weights (or numbers).
          const auto bounds = [&](int i) {
            const U64 c = steps[i];
            if (!by_mass) return Two{c, c};
            if (!c) return Two{0, 0};
            const uint32_t k = last - i;
            if (single) {
              const U64 w = weight(value_of<E>(k), sc, lane_table);
              return Two{c * w, c * w};
            }
            // Weights fall back by 2^-29 of them at most where logits rise (from one table entry to the next,
            // close to 0, where numbers lie that near to each other).
            const uint32_t k0 = max(k << shift, lo), k1 = min((k << shift) | ((1u << shift) - 1u), hi);
            const U64 w0 = weight(float_of(k0), sc, lane_table), w1 = weight(float_of(k1), sc, lane_table);
            return Two{c * (w1 + (w1 >> 28) + 2), c * (w0 - min(w0, (w0 >> 28) + 2))};
          };
          uint32_t count = 0;
          for (int i = tid * per; i < (tid + 1) * per; ++i) {
            for (int r = 1; r < p.ctas; ++r) steps[i] += *peer(steps + i, r);
            count += steps[i];
          }
          Two here{0, 0};
          for (int i = tid * per; i < (tid + 1) * per; ++i) here = Sum::of(here, bounds(i));
          if (tid == 0) sh.found[0] = 0, sh.found[1] = last - (lo >> shift);
          Two run = block_before(here, &sh);
          const U64 so_far = by_mass ? above : above_n;
          run.a += so_far, run.b += so_far;
          uint32_t run_n = static_cast<uint32_t>(block_before(static_cast<U64>(count), &sh));
          for (int i = tid * per; i < (tid + 1) * per; ++i) {
            const Two next = Sum::of(run, bounds(i));
            if (run.a < need && next.a >= need) {
              sh.found[0] = i, sh.found[2] = run_n;
              sh.before = run.a;  // single: the prefix without this step
            }
            if (run.b < need && next.b >= need) sh.found[1] = i;
            run = next, run_n += steps[i];
          }
          __syncthreads();
          const uint32_t j0 = sh.found[0], j1 = max(sh.found[1], j0);
          if (single) {
            const uint32_t k = key_of(value_of<E>(last - j0));
            const U64 w = weight(float_of(k), sc, lane_table), before = sh.before;
            U64 equal = by_mass ? (w ? (need - before + w - 1) / w : 1) : need - before;
            equal = equal < 1 ? 1 : equal > steps[j0] ? steps[j0] : equal;
            U64 mass = before + equal * w;
            if (!by_mass) {  // of the steps before
              U64 part = 0;
              for (int i = tid; i < static_cast<int>(j0); i += threads)
                if (steps[i]) part += steps[i] * weight(value_of<E>(last - i), sc, lane_table);
              const U64 sum_before = block_before(part, &sh) + part;
              if (tid == threads - 1) sh.before = above + sum_before + equal * w;
              __syncthreads();
              mass = sh.before;
            }
            plan = Plan{mass, k, static_cast<uint32_t>(equal), 0, 0};
          } else {
            uint32_t c = 0;
            for (int i = static_cast<int>(j0) + tid; i <= static_cast<int>(j1); i += threads) c += steps[i];
            const U64 n_before = block_before(static_cast<U64>(c), &sh) + c;
            if (tid == threads - 1) sh.found[0] = static_cast<uint32_t>(n_before);
            __syncthreads();
            // the steps' keys, how many they are, and how many lie above them here
            plan = Plan{need, max((last - j1) << shift, lo), min(((last - j0) << shift) | ((1u << shift) - 1u), hi), sh.found[0], sh.found[2]};
          }
        }
        plan = cl.tell(plan);
        if (single) {
          // The draw needs the weights of the steps above the threshold: by value, once.
          for (int i = tid; i <= static_cast<int>(last - (plan.a >> shift)); i += threads) list[i] = weight(value_of<E>(last - i), sc, lane_table);
          last_step = last;
          __syncthreads();
          return plan;
        }
        need = plan.mass;
        const uint32_t before = hi - lo;
        lo = plan.a, hi = plan.b, above_n += plan.d;
        if (lo == kMinusZero) ++lo;
        if (hi == kMinusZero) --hi;
        if (plan.c <= kList) break;
        if (hi - lo > before / 2) {  // weights of nearly 0, which the bounds do not tell apart: halves, by exact sums
          uint32_t mid = lo + (hi - lo) / 2;  // (mid, hi] or [lo, mid]
          if (mid == kMinusZero) --mid;
          const float f_hi = float_of(hi), f_mid = float_of(mid), f_sure = sure;
          U64 over = 0;
          Two top{0, 0};
          each_piece([&](const Piece<E>& l) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
              if (l.v[e] > f_mid && l.v[e] <= f_sure) {
                const U64 w = weight(l.v[e], sc, lane_table);
                if (l.v[e] > f_hi) over += w;
                else top.a += w, ++top.b;
              }
          });
          own.a += over, sure = f_hi;
          above += cl.all<Sum>(Two{over, 0}).a;
          const Two all_top = cl.all<Sum>(top);
          if ((by_mass ? above + all_top.a : above_n + all_top.b) >= need) {
            lo = mid + 1;
            if (lo == kMinusZero) ++lo;
          } else {
            above += all_top.a, above_n += all_top.b, own.a += top.a, sure = f_mid;
            hi = mid;
          }
        }
      }
      // The few: sorted, with the weights of those above.
      last_step = 0;
      const float high = float_of(hi), known = sure;
      U64 sum = 0;
      each_piece([&](const Piece<E>& l) {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (l.v[e] > high && l.v[e] <= known) sum += weight(l.v[e], sc, lane_table);
      });
      own.a += sum, sure = high;
      above += cl.all<Sum>(Two{sum, 0}).a;
      const int m = listed(gather_list(float_of(lo), high));
      if (cl.rank == 0) {
        sort(list, m);
        sum_list(m);
        const int end = by_mass ? prefix_of(m, need - above) : min(m, static_cast<int>(need - above_n));
        const uint32_t key = static_cast<uint32_t>(list[end - 1] >> 32);
        if (tid == 0) sh.found[1] = 0, sh.listed = 0;
        __syncthreads();
        uint32_t equal = 0;
        for (int i = tid; i < end; i += threads) equal += static_cast<uint32_t>(list[i] >> 32) == key ? 1u : 0u;
        if (equal) atomicAdd(&sh.found[1], equal);
        __syncthreads();
        plan = Plan{above + mass_of[end - 1], key, sh.found[1], 0, 0};
      }
      return cl.tell(plan);
    };

    Plan end{};
    bool found = false;
    U64 total = 0;  // the weights that top-p is of; 0: all
    if (by_k) {
      const Plan in = bracket(false, static_cast<U64>(top_k));
      if (static_cast<U64>(top_k) < in.mass) {  // else all that have a weight
        if (in.c <= kList) {
          const U64 m = gather_list(lowest_in(static_cast<int>(in.b), row_max, sc), INFINITY);
          if (cl.rank == 0) draw_from_list(listed(m), top_k, 0);
          return;
        }
        end = narrow(false, static_cast<U64>(top_k), in);
        total = end.mass;
        found = true;
      }
    }
    if (by_p) {
      const Plan in = bracket(true, total);
      if (in.c <= kList) {
        U64 all = 0;
        const U64 m = gather_list(lowest_in(static_cast<int>(in.b), row_max, sc), INFINITY, total == 0, &all);
        if (cl.rank == 0) {
          __syncthreads();
          if (tid == 0) sh.need = total ? in.mass : share_of(all);
          __syncthreads();
          draw_from_list(listed(m), 0, sh.need);
        }
        return;
      }
      end = narrow(true, total ? in.mass : 0, in);
      found = true;
    }
    if (found) t = float_of(end.a), n = end.b;
  }
  if (!greedy && by_min && least > t) t = least, n = kAll;

  // The kept weights of a piece, but those of l > sure, and how many are equal to t.
  const bool everything = t == -INFINITY && sure == INFINITY;
  const auto kept_of = [&](const Piece<E>& l, float known) {
    Two v{0, 0};
    if (everything) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) v.a += weight(l.v[e], sc, lane_table);
    } else {
      bool any = false;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        any = any || (l.v[e] > t && l.v[e] <= known);
        v.b += l.v[e] == t ? 1 : 0;
      }
      if (any && known < INFINITY && last_step) {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (l.v[e] > t && l.v[e] <= known) {
            const uint32_t k = key_of(l.v[e]) >> (sizeof(E) == 2 ? 16 : 0);
            if (skipped && k > kNegative && k < kPositive) v.a += weight(l.v[e], sc, lane_table);
            else v.a += list[last_step - k - (k <= kNegative ? skipped : 0)];
          }
      } else if (any) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const U64 w = weight(l.v[e], sc, lane_table);
          if (l.v[e] > t && l.v[e] <= known) v.a += w;
        }
      }
    }
    return v;
  };
  if (t > sure) sure = INFINITY, own = Two{0, 0};  // min-p cut into what was known
  own.b = 0;
  if (everything) {
    U64 sum = 0;
    each_piece([&](const Piece<E>& l) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) sum += weight(l.v[e], sc, lane_table);
    });
    own.a = sum;
  } else {
    each_piece([&](const Piece<E>& l) { own = Sum::of(own, kept_of(l, sure)); });
  }
  const Two* from;
  if (alone) {  // the CTAs' sums were gathered last
    cl.sum_warps<Sum>(own);
    __syncthreads();
    from = cl.last();
  } else {
    from = cl.gather<Sum>(own);
  }
  const U64 w_t = n ? weight(t, sc, lane_table) : 0;
  const auto kept = [&](const Two& s) { return s.a + (s.b < n ? s.b : static_cast<U64>(n)) * w_t; };
  Two before{0, 0}, all{0, 0};
  for (int i = 0; i < p.ctas; ++i) {
    if (i == cl.rank) before = all;
    all = Sum::of(all, from[i]);
  }
  const U64 total = kept(all), target = share_down(u_share, total);
  for (int i = 0; i < warp; ++i) before = Sum::of(before, sh.part[i]);
  const Two here = Sum::of(before, sh.part[warp]);
  if (!(kept(before) <= target && target < kept(here))) return;  // another warp's stretch
  // the lane's, from the sums that it has
  Two incl = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Two o{__shfl_up_sync(0xffffffffu, incl.a, d), __shfl_up_sync(0xffffffffu, incl.b, d)};
    if (lane >= d) incl = Sum::of(incl, o);
  }
  const int owner = __ffs(__ballot_sync(0xffffffffu, kept(Sum::of(before, incl)) > target)) - 1;
  before = Sum::of(before, Two{__shfl_sync(0xffffffffu, incl.a - own.a, owner), __shfl_sync(0xffffffffu, incl.b - own.b, owner)});
  // and that lane's logits, one to each lane at a time
  const int from_piece = min(w0 + owner * run, w1), count = (min(from_piece + run, w1) - from_piece) * kPer;
  for (int q0 = 0; q0 < count; q0 += 32) {
    const int q = q0 + lane;
    Two v{0, 0};
    if (q < count) {
      const float l = as_float(reinterpret_cast<const E*>(pieces + place_of(from_piece + q / kPer))[q % kPer]);
      if (l > t) v.a = weight(l, sc, lane_table);
      else if (l == t) v.b = 1;  // (t = -inf: n is 0)
    }
    Two sums = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Two o{__shfl_up_sync(0xffffffffu, sums.a, d), __shfl_up_sync(0xffffffffu, sums.b, d)};
      if (lane >= d) sums = Sum::of(sums, o);
    }
    const unsigned past = __ballot_sync(0xffffffffu, kept(Sum::of(before, sums)) > target);
    if (past) {
      if (lane == __ffs(past) - 1) write(static_cast<int64_t>(first + from_piece) * kPer + q - off, total);
      return;
    }
    before = Sum::of(before, Two{__shfl_sync(0xffffffffu, sums.a, 31), __shfl_sync(0xffffffffu, sums.b, 31)});
  }
}

inline size_t shared_bytes(int chunk, bool search) {
  return piece_bytes(chunk) + sizeof(uint2) * kTable * 32 + (search ? sizeof(uint32_t) * kBins + 2 * sizeof(U64) * kList : 0);
}

}  // namespace sample
}  // namespace flce
