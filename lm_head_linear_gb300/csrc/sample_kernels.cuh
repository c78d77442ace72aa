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
// in units of 2^-44 of the largest: their sums are exact, in whatever order they are formed, and
// the sum that the search compares is the one that the drawing walks through.  A weight itself
// is good to 2^-31 of it and 2^-44 (table-driven exponential after Tang, 1989): a draw among 250,000
// equally likely words then falls on the other side of a border about once in a million.
//
// A row belongs to a cluster of CTAs, each with its part in shared memory: the logits are
// read once.  The CTAs agree on maximum, sums and thresholds by pushing a few words into each
// other's shared memory and a cluster barrier.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace flce {
namespace sample {

using U64 = unsigned long long;

constexpr int kMaxCtas = 16;       // of a cluster
constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kUnit = 44;          // weights are whole multiples of 2^-44: their sum stays below 2^63
constexpr int kTable = 32;         // steps of an octave
constexpr int kBins = 1536;        // of -32 log2(weight), rounded
constexpr int kLive = (kUnit + 1) * kTable + 1;  // from this bin on weights are 0
constexpr int kList = 1024;        // candidates that are sorted
constexpr int kGroups = 1024;      // whose largest logits bound the k-th largest from below
constexpr uint32_t kAll = 0x7fffffffu;
static_assert(kLive <= kBins && kBins % kMaxThreads == 0, "bins");

struct Params {
  const void* logits;
  const float* u;
  const float* temperature;  // [T], or nullptr: temperature_all (as the three below)
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  double temperature_all, top_p_all, min_p_all;
  float temperature_like, top_p_like, min_p_like;  // numbers that compare as those do with 0 and 1
  int64_t top_k_all;
  int64_t ldl, ignore_index;
  int64_t* tokens;
  float* logp;     // or nullptr
  int32_t V;
  int32_t ctas;    // of a cluster
  int32_t chunk;   // 16-byte pieces of a CTA
};

// round(2^(31 + j / 32))
__device__ constexpr uint32_t kPow2[kTable] = {
    2147483648u, 2194507417u, 2242560872u, 2291666561u, 2341847524u, 2393127307u, 2445529972u, 2499080105u,
    2553802834u, 2609723834u, 2666869345u, 2725266179u, 2784941738u, 2845924021u, 2908241642u, 2971923842u,
    3037000500u, 3103502151u, 3171459999u, 3240905930u, 3311872529u, 3384393094u, 3458501653u, 3534232978u,
    3611622603u, 3690706840u, 3771522796u, 3854108391u, 3938502376u, 4024744348u, 4112874773u, 4202935003u};

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

// A row's way from a logit to its weight: w = 2^-z, z = (l / 2 - max / 2) (-c_hi - c_lo).  Halves:
// the difference of two fp32 numbers need not be one.  (A row whose largest logit is
// infinite is rewritten first, so max is finite.)  Differences below `least` count as that: z = 64,
// the weight 0, also of l = -inf.  Where c is so small that no finite difference gets there,
// the row is flat(), and -inf has to be told from the others by its value.
struct Scale {
  float half_max, c_hi, c_lo, least;
  __device__ __forceinline__ bool flat() const { return c_hi < 2.0e-37f; }
};
constexpr float kMagic = 393216.0f;  // 1.5 2^18: sums with it round to whole multiples of 1/32

// A logit's weight in units of 2^-44, and its bin, n = round(32 z).  `lane_table`: this lane's
// column of the table of powers, which is there once for every lane so that no two lanes meet
// in a bank.
//
// 30 cycles of a lane for bf16, 40 for fp32 (1.9 GHz, two logits' worth of registers in flight).  Packed
// pairs of fp32 with the sum kept as two fp32 numbers, which saves the 64-bit shift and
// addition, took 33 and 42: their constants need two registers each.
struct Weight {
  U64 w;
  int n;
};
template <typename E>
__device__ __forceinline__ Weight weigh(float l, const Scale& s, const uint2* lane_table) {
  const float d = fmaf(l, 0.5f, -s.half_max), dd = fmaxf(d, s.least);
  const float z = dd * -s.c_hi;
  float rest = fmaf(dd, s.c_lo, fmaf(dd, s.c_hi, z));
  if constexpr (sizeof(E) == 4) {  // what d rounds off; bf16 logits lose nothing that counts
    const float h = 0.5f * l, b = d - h;
    const float off = ((h - (d - b)) + (-s.half_max - b)) * s.c_hi;
    rest += fmaxf(off, -1.0f);  // far below 1; NaN where l is infinite
  }
  const float t = kMagic - z;
  const float r = ((kMagic - t) - z) + rest;  // |r| <= 1/64, exact but for the rest
  // 2^r - 1, off by less than 2^-32.8: a polynomial fitted to it (least largest error on |r| <= 1/64)
  const float p = r * fmaf(r, fmaf(r, 0.05550457f, 0.24022846f), 0.6931472f);
  const int up = __float_as_int(kMagic) + (kTable - 1) - __float_as_int(t);  // n + 31
  const uint2 power = lane_table[(up & (kTable - 1)) * 32];
  const uint32_t w = power.x + static_cast<uint32_t>(__float2int_rn(__uint_as_float(power.y) * p));  // 2^31 of its octave
  Weight out;
  out.n = up - (kTable - 1);
  asm("shr.u64 %0, %1, %2;" : "=l"(out.w) : "l"(static_cast<U64>(w) << 32), "r"((up >> 5) + (63 - kUnit)));  // 0 from 64 on
  return out;
}
template <typename E>
__device__ __forceinline__ U64 weight(float l, const Scale& s, const uint2* lane_table) {
  return weigh<E>(l, s, lane_table).w;
}

// The same bin on its own.
__device__ __forceinline__ int bin_of(float l, const Scale& s) {
  const float z = fmaxf(fmaf(l, 0.5f, -s.half_max), s.least) * -s.c_hi;
  return __float_as_int(kMagic) - __float_as_int(kMagic - z);
}
// The lowest logit of bins up to b (bins fall as logits rise), not -inf.
__device__ __forceinline__ float lowest_in(int b, const Scale& s) {
  uint32_t lo = 0x00800000u, hi = key_of(2.0f * s.half_max);  // the lowest number, the largest logit: bin 0
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (bin_of(float_of(mid), s) <= b) hi = mid;
    else lo = mid + 1;
  }
  return float_of(hi);
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
  U64 mass;          // of a prefix; of a bracket: how many logits have a weight
  uint32_t a, b, c;  // threshold's key, its equals; of a bracket: bins a .. b, logits up to b
};

struct Shared {
  Two part[kMaxWarps];
  Two from[2][kMaxCtas];
  Plan plan[2];
  double inv_t, log_min;
  U64 need;
  float c_hi, c_lo, least, min_logit;
  uint32_t listed, found[3];
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
  // Every CTA's value, in from[], for all threads of all CTAs.
  template <typename Op>
  __device__ __forceinline__ const Two* gather(Two v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      v = Op::of(v, Two{__shfl_xor_sync(0xffffffffu, v.a, d), __shfl_xor_sync(0xffffffffu, v.b, d)});
    if (lane == 0) s->part[warp] = v;
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

// Exclusive prefix sum over the block's threads.
__device__ __forceinline__ U64 block_before(U64 v, Shared* s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  U64 incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const U64 o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  __syncthreads();
  if (lane == 31) s->part[warp].a = incl;
  __syncthreads();
  U64 before = incl - v;
  for (int i = 0; i < warp; ++i) before += s->part[i].a;
  return before;
}

// The least whole number that is f m or more, the product rounded to 53 bits: 0.9 of 4000 equal
// weights are 3600 of them, although the number nearest to 0.9 is a little more.
__device__ __forceinline__ U64 share_up(double f, U64 m) { return __double2ull_ru(f * __ull2double_rn(m)); }
// floor(f m) for f in [0, 1) as a whole multiple of 2^-63.
__device__ __forceinline__ U64 share_down(U64 f, U64 m) { return __umul64hi(f, m) << 1 | (f * m) >> 63; }

// ------------------------------------------------------------------ the kernel
// The pieces of a CTA's part of a row: 16 bytes as they lie in memory; what a piece holds before
// or behind the row counts as -inf.  A warp has a stretch of its own, and its lanes read back
// what they have copied themselves.
template <typename E>
__global__ void __launch_bounds__(kMaxThreads, 2) sample_kernel(const Params p) {
  constexpr int kPer = Piece<E>::kPer;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  uint4* const pieces = reinterpret_cast<uint4*>(smem);
  uint2* const table = reinterpret_cast<uint2*>(smem + static_cast<size_t>(p.chunk) * 16);
  uint32_t* const bins = reinterpret_cast<uint32_t*>(table + kTable * 32);
  U64* const list = reinterpret_cast<U64*>(bins + kBins);
  U64* const mass_of = list + kList;                               // sums of the sorted list's weights
  uint32_t* const group_max = reinterpret_cast<uint32_t*>(mass_of);  // before that: of every group of the row

  const int threads = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = threads >> 5;
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
  const int all_pieces = (off + p.V + kPer - 1) / kPer;
  const int first = cl.rank * p.chunk;
  const int mine = max(0, min(p.chunk, all_pieces - first));
  const int stretch = ((p.chunk + warps - 1) / warps + 31) / 32 * 32;
  const int w0 = warp * stretch, w1 = min(w0 + stretch, mine);
  for (int i = w0 + lane; i < w1; i += 32) {
    const int64_t at = static_cast<int64_t>(first + i) * kPer - off;  // the piece's first logit
    if (at >= 0 && at + kPer <= p.V) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(pieces + i)), "l"(logits + at) : "memory");
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        reinterpret_cast<E*>(pieces + i)[e] = at + e >= 0 && at + e < p.V ? logits[at + e] : lowest<E>();
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
  const bool by_k = top_k > 0, by_p = top_p < 1.0f, by_min = min_p > 0.0f;
  if (tid == 0) {
    const double t = p.temperature ? static_cast<double>(temperature) : p.temperature_all;
    const double inv = greedy ? 1.0 : fmin(1.0 / t, 1e37);
    const double c = inv * (2.0 * 1.4426950408889634);
    sh.inv_t = inv;
    sh.c_hi = static_cast<float>(c);
    sh.c_lo = static_cast<float>(c - static_cast<double>(sh.c_hi));
    sh.least = fmaxf(-64.0f / sh.c_hi, -3.4028234e38f);
    sh.log_min = by_min && !greedy ? t * log(p.min_p ? static_cast<double>(min_p) : p.min_p_all) : 0.0;
    sh.listed = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  float best = -INFINITY;
  bool nan = false;
  for (int i = w0 + lane; i < w1; i += 32) largest<E>(pieces[i], best, nan);
  if (__any_sync(0xffffffffu, nan)) {  // never drawn
    best = -INFINITY;
    for (int i = w0 + lane; i < w1; i += 32) {
      const Piece<E> l = unpack<E>(pieces[i]);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (l.v[e] != l.v[e]) reinterpret_cast<E*>(pieces + i)[e] = lowest<E>();
        best = fmaxf(best, l.v[e]);
      }
    }
  }
  if (p.ctas > 1) {  // the others' shared memory is there
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  // The largest logits of up to 1024 groups of the row, to every CTA: at least k logits are no
  // smaller than the k-th largest of them.
  const int groups = min(threads, kGroups / p.ctas);  // of a CTA
  const bool short_k = !greedy && by_k && top_k <= groups * p.ctas;
  if (short_k) {
    float g = best;
    const int lanes = threads / groups;  // a power of two
    for (int d = lanes / 2; d > 0; d >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
    for (int r = tid & (lanes - 1); r < p.ctas; r += lanes) peer(group_max, r)[cl.rank * groups + tid / lanes] = key_of(g);
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
    for (int i = w0 + lane; i < w1; i += 32) {
      const Piece<E> l = unpack<E>(pieces[i]);
#pragma unroll
      for (int e = 0; e < kPer; ++e) reinterpret_cast<E*>(pieces + i)[e] = l.v[e] == INFINITY ? static_cast<E>(0) : lowest<E>();
    }
    row_max = 0.0f;
  }
  const Scale sc{0.5f * row_max, sh.c_hi, sh.c_lo, sh.least};
  float least = -INFINITY;  // of min-p
  if (by_min) {
    if (tid == 0) sh.min_logit = fminf(__double2float_ru(static_cast<double>(row_max) + sh.log_min), row_max);
    __syncthreads();
    least = sh.min_logit;
  }
  const auto each = [&](auto f) {  // every logit of this thread's and its number
    for (int i = w0 + lane; i < w1; i += 32) {
      const Piece<E> l = unpack<E>(pieces[i]);
#pragma unroll
      for (int e = 0; e < kPer; ++e) f(l.v[e], (first + i) * kPer + e - off);
    }
  };
  const auto each_piece = [&](auto f) {
    for (int i = w0 + lane; i < w1; i += 32) f(unpack<E>(pieces[i]));
  };
  const auto write = [&](int64_t token, U64 total) {  // one thread: the token, and log(its weight / total)
    p.tokens[row] = token;
    if (!p.logp) return;
    // the weight's from the logit; of the total the exponent, the leading 24 bits, and the rest apart
    const int top = 63 - __clzll(total);
    const U64 bits = total << (63 - top);
    const float lead = __ull2float_rz(bits);
    const float rest = static_cast<float>(bits - static_cast<U64>(lead)) / lead;
    const float drawn = as_float(logits[token]);
    const double d = drawn == real_max ? 0.0 : static_cast<double>(drawn) - static_cast<double>(real_max);
    const double log_total = static_cast<double>(top - kUnit) * 0.6931471805599453 + (static_cast<double>(logf(lead * 0x1p-63f)) + rest);
    p.logp[row] = greedy ? 0.0f : static_cast<float>(d * sh.inv_t - log_total);
  };
  const U64 u_share = u > 0.0f ? static_cast<U64>(fminf(u, 0x1.fffffep-1f) * 0x1p63f) : 0;

  // ---- the list: logits from `low` on, unsorted, on the first CTA.  Returns how many there are.
  const auto gather_list = [&](float low, float high) -> U64 {
    U64 count = 0;
    each([&](float l, int index) {
      if (l >= low && l <= high) {
        const uint32_t at = atomicAdd(peer(&sh.listed, 0), 1u);
        if (at < kList) *peer(list + at, 0) = static_cast<U64>(key_of(l)) << 32 | (0xffffffffu - static_cast<uint32_t>(index));
        ++count;
      }
    });
    return cl.all<Sum>(Two{count, 0}).a;
  };
  const auto listed = [&](U64 count) { return static_cast<int>(count < kList ? count : kList); };
  const auto key_in_list = [&](int i) { return float_of(static_cast<uint32_t>(list[i] >> 32)); };
  // Sorts m numbers, the largest first; all threads of a CTA.
  const auto sort = [&](U64* a, int m) {
    int size = 32;
    while (size < m) size *= 2;
    for (int i = m + tid; i < size; i += threads) a[i] = 0;
    __syncthreads();
    const bool one_warp = size <= 128;  // without block barriers
    const int step = one_warp ? 32 : threads;
    if (!one_warp || warp == 0) {
      for (int k = 2; k <= size; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
          for (int i = tid; i < size / 2; i += step) {
            const int x = 2 * i - (i & (j - 1)), y = x + j;
            const U64 vx = a[x], vy = a[y];
            if ((vx < vy) == ((x & k) == 0)) a[x] = vy, a[y] = vx;
          }
          if (one_warp) __syncwarp();
          else __syncthreads();
        }
    }
    __syncthreads();
  };
  // The sums of the sorted list's weights up to each.
  const auto sum_list = [&](int m) {
    const int per = (m + threads - 1) / threads, a = min(tid * per, m), b = min(a + per, m);
    U64 sum = 0;
    for (int i = a; i < b; ++i) sum += weight<E>(key_in_list(i), sc, lane_table);
    U64 run = block_before(sum, &sh);
    for (int i = a; i < b; ++i) mass_of[i] = run += weight<E>(key_in_list(i), sc, lane_table);
    __syncthreads();
  };
  // How many of the first m of the list it takes for weights of `need`.
  const auto share_of = [&](U64 total) {  // p of it; one thread
    return share_up(p.top_p ? static_cast<double>(top_p) : p.top_p_all, total);
  };
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
    // by index, the first first, each with its weight behind it: 19 and 45 bits
    __syncthreads();
    for (int i = tid; i < m; i += threads) {
      const U64 w = mass_of[i] - (i ? mass_of[i - 1] : 0);
      list[i] = list[i] << 45 | w;  // of ~index
    }
    sort(list, m);
    const int per = (m + threads - 1) / threads, a = min(tid * per, m), b = min(a + per, m);
    constexpr U64 kWeight = (1ull << 45) - 1;
    U64 sum = 0;
    for (int i = a; i < b; ++i) sum += list[i] & kWeight;
    U64 run = block_before(sum, &sh);
    for (int i = a; i < b; ++i) {
      const U64 next = run + (list[i] & kWeight);
      if (run <= target && target < next) write(static_cast<int64_t>(~(list[i] >> 45) & 0x7ffffu), total);
      run = next;
    }
  };

  // ---- what is kept: l > t, and the first n of l == t.  `own`: this thread's weights of l > sure,
  // known already (sure: +inf if none).
  float t = -INFINITY, sure = INFINITY;
  uint32_t n = 0;
  Two own{0, 0};
  if (greedy) t = row_max, n = 1;

  if (!greedy && (by_k || by_p)) {
    if (short_k && row_max == real_max) {
      // Every CTA finds the same bound.
      for (int i = tid; i < kBins; i += threads) bins[i] = 0;
      __syncthreads();
      for (int i = tid; i < groups * p.ctas; i += threads) {
        const float l = float_of(group_max[i]);
        const int b = bin_of(l, sc);
        if (l > -INFINITY && static_cast<uint32_t>(b) < kLive) atomicAdd(bins + b, 1u);
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
        const U64 m = gather_list(lowest_in(b, sc), INFINITY);
        if (m <= kList) {
          if (cl.rank == 0) draw_from_list(listed(m), top_k, 0);
          return;
        }
        __syncthreads();
        if (tid == 0) sh.listed = 0;  // seen by the others after the next barrier
      }
    }
    // How many logits fall into each bin, and the sum of weights.
    __syncthreads();
    for (int i = tid; i < kBins; i += threads) bins[i] = 0;
    __syncthreads();
    U64 sum = 0;
    if (!sc.flat()) {
      each_piece([&](const Piece<E>& l) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const Weight w = weigh<E>(l.v[e], sc, lane_table);
          if (static_cast<uint32_t>(w.n) < kLive) atomicAdd(bins + w.n, 1u);
          sum += w.w;
        }
      });
    } else {
      each([&](float l, int) {
        const int b = bin_of(l, sc);
        if (l > -INFINITY && static_cast<uint32_t>(b) < kLive) atomicAdd(bins + b, 1u), sum += weight<E>(l, sc, lane_table);
      });
    }
    U64 total = cl.all<Sum>(Two{sum, 0}).a;  // with top-k: of the first k, later
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
    // weights `of`; how many lie up to b; and in all, or what p of the weights is.
    const auto bracket = [&](bool mass, U64 of) {
      Plan plan{0, 0, 0, 0};
      if (cl.rank == 0) {
        __syncthreads();
        if (tid == 0) {
          sh.found[0] = sh.found[1] = kLive - 1;  // not behind: nothing has been counted there
          sh.need = mass ? share_of(of) : of;
        }
        __syncthreads();
        const U64 need = sh.need;
        if (!mass) {
          for (int i = tid; i < kBins; i += threads)
            if (bins[i] >= need && (i == 0 || bins[i - 1] < need)) sh.found[0] = sh.found[1] = i;
        } else {  // between the bounds of their weights
          for (int side = 0; side < 2; ++side) {
            const auto bound = [&](int i) -> U64 {
              const uint32_t c = bins[i] - (i ? bins[i - 1] : 0u);
              const float w = ptx::ex2((static_cast<float>(-i - side) + 0.5f) * (1.0f / kTable)) * (side ? 1.0f - 0x1p-15f : 1.0f + 0x1p-15f);
              const U64 one = static_cast<U64>(w * 0x1p44f);
              return c * (side ? (one ? one - 1 : 0) : one + 2);
            };
            U64 here = 0;
            for (int i = tid * per; i < (tid + 1) * per; ++i) here += bound(i);
            U64 run = block_before(here, &sh);
            if (run < need && run + here >= need)
              for (int i = tid * per; i < (tid + 1) * per; ++i) {
                const U64 next = run + bound(i);
                if (run < need && next >= need) sh.found[side] = i;
                run = next;
              }
          }
        }
        __syncthreads();
        plan = Plan{mass ? need : bins[kBins - 1], sh.found[0], sh.found[1], bins[sh.found[1]]};
      }
      return cl.tell(plan);
    };
    // The end of that prefix, where more logits share its bins than can be sorted: bisection of
    // their values.  Returns the threshold, how many of its equals, and the prefix's weight.
    const auto bisect = [&](bool by_mass, U64 need, const Plan& in) {
      const float low = lowest_in(static_cast<int>(in.b), sc);
      const uint32_t top_key = in.a ? key_of(lowest_in(static_cast<int>(in.a) - 1, sc)) : 0xffffffffu;  // above the bracket
      sure = in.a ? float_of(next_below(top_key)) : INFINITY;
      own = Two{0, 0};
      U64 count = 0;
      Two range{0, ~0ull};
      const float over = sure;
      each_piece([&](const Piece<E>& l) {
        bool any = false;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          any = any || l.v[e] > over;
          if (l.v[e] >= low && l.v[e] <= over) {
            ++count;
            const U64 k = key_of(l.v[e]);
            range = MaxMin::of(range, Two{k, k});
          }
        }
        if (any) {
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const U64 w = weight<E>(l.v[e], sc, lane_table);
            if (l.v[e] > over) own.a += w, ++own.b;
          }
        }
      });
      Two above = cl.all<Sum>(own);
      count = cl.all<Sum>(Two{count, 0}).a;
      range = cl.all<MaxMin>(range);
      uint32_t hi = static_cast<uint32_t>(range.a), lo = static_cast<uint32_t>(range.b);
      while (count > kList && lo < hi) {
        uint32_t mid = lo + (hi - lo) / 2;  // (mid, hi] or [lo, mid]
        if (mid == kMinusZero) --mid;
        const float a = float_of(mid), b = float_of(hi);
        Two here{0, 0};
        each([&](float l, int) {
          if (l > a && l <= b) here.a += weight<E>(l, sc, lane_table), ++here.b;
        });
        const Two top = cl.all<Sum>(here);
        if ((by_mass ? above.a + top.a : above.b + top.b) >= need) {
          lo = mid + 1, count = top.b;
          if (lo == kMinusZero) ++lo;
        } else {
          hi = mid, count -= top.b, above = Sum::of(above, top);
          own = Sum::of(own, here), sure = a;
        }
      }
      if (lo >= hi) {  // equal ones
        const U64 w = weight<E>(float_of(hi), sc, lane_table);
        U64 equal = by_mass ? (w ? (need - above.a + w - 1) / w : 1) : need - above.b;
        equal = equal < 1 ? 1 : equal > count ? count : equal;
        return Plan{above.a + equal * w, hi, static_cast<uint32_t>(equal), 0};
      }
      const int m = listed(gather_list(float_of(lo), float_of(hi)));
      Plan plan{0, 0, 0, 0};
      if (cl.rank == 0) {
        sort(list, m);
        sum_list(m);
        const int end = by_mass ? prefix_of(m, need - above.a) : min(m, static_cast<int>(need - above.b));
        const uint32_t last = static_cast<uint32_t>(list[end - 1] >> 32);
        if (tid == 0) sh.found[1] = 0, sh.listed = 0;
        __syncthreads();
        uint32_t equal = 0;
        for (int i = tid; i < end; i += threads) equal += static_cast<uint32_t>(list[i] >> 32) == last ? 1u : 0u;
        if (equal) atomicAdd(&sh.found[1], equal);
        __syncthreads();
        plan = Plan{above.a + mass_of[end - 1], last, sh.found[1], 0};
      }
      return cl.tell(plan);
    };

    Plan end{0, 0, 0, 0};
    bool found = false;
    if (by_k) {
      const Plan in = bracket(false, static_cast<U64>(top_k));
      if (static_cast<U64>(top_k) < in.mass) {  // else all that have a weight
        if (in.c <= kList) {
          const U64 m = gather_list(lowest_in(static_cast<int>(in.b), sc), INFINITY);
          if (cl.rank == 0) draw_from_list(listed(m), top_k, 0);
          return;
        }
        end = bisect(false, static_cast<U64>(top_k), in);
        total = end.mass;
        found = true;
      }
    }
    if (by_p) {
      const Plan in = bracket(true, total);
      const U64 need = in.mass;
      if (in.c <= kList) {
        const U64 m = gather_list(lowest_in(static_cast<int>(in.b), sc), INFINITY);
        if (cl.rank == 0) draw_from_list(listed(m), 0, need);
        return;
      }
      end = bisect(true, need, in);
      found = true;
    }
    if (found) t = float_of(end.a), n = end.b;
  }
  if (!greedy && by_min && least > t) t = least, n = kAll;

  // The kept weights of a piece, but those of l > sure, and how many are equal to t.
  const bool everything = t == -INFINITY && sure == INFINITY && !sc.flat();
  const auto kept_of = [&](const Piece<E>& l, float known) {
    Two v{0, 0};
    if (everything) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) v.a += weight<E>(l.v[e], sc, lane_table);
    } else {
      bool any = false;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        any = any || (l.v[e] > t && l.v[e] <= known);
        v.b += l.v[e] == t ? 1 : 0;
      }
      if (any) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const U64 w = weight<E>(l.v[e], sc, lane_table);
          if (l.v[e] > t && l.v[e] <= known) v.a += w;
        }
      }
    }
    return v;
  };
  if (t > sure) sure = INFINITY, own = Two{0, 0};  // min-p cut into what was known
  own.b = 0;
  each_piece([&](const Piece<E>& l) { own = Sum::of(own, kept_of(l, sure)); });
  const Two* from = cl.gather<Sum>(own);
  const U64 w_t = n ? weight<E>(t, sc, lane_table) : 0;
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
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    Two v{0, 0};
    Piece<E> l;
    if (i < w1) {
      l = unpack<E>(pieces[i]);
      v = kept_of(l, INFINITY);
    }
    Two incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Two o{__shfl_up_sync(0xffffffffu, incl.a, d), __shfl_up_sync(0xffffffffu, incl.b, d)};
      if (lane >= d) incl = Sum::of(incl, o);
    }
    const unsigned past = __ballot_sync(0xffffffffu, kept(Sum::of(before, incl)) > target);
    if (past) {
      if (lane == __ffs(past) - 1) {
        Two run{before.a + incl.a - v.a, before.b + incl.b - v.b};
        int e_drawn = -1;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (l.v[e] > t) run.a += weight<E>(l.v[e], sc, lane_table);
          else if (l.v[e] == t) ++run.b;  // (t = -inf: n is 0)
          if (e_drawn < 0 && kept(run) > target) e_drawn = e;
        }
        write(static_cast<int64_t>(first + i) * kPer + e_drawn - off, total);
      }
      return;
    }
    before = Sum::of(before, Two{__shfl_sync(0xffffffffu, incl.a, 31), __shfl_sync(0xffffffffu, incl.b, 31)});
  }
}

inline size_t shared_bytes(int chunk) {
  return static_cast<size_t>(chunk) * 16 + sizeof(uint2) * kTable * 32 + sizeof(uint32_t) * kBins + 2 * sizeof(U64) * kList;
}

}  // namespace sample
}  // namespace flce
