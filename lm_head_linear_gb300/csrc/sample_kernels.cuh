// Drawing tokens from logits: temperature, top-k, top-p and min-p with given random numbers.
//
// Of a row's logits l (best first, equal ones by their index), w_i = e^((l_i - max) / temperature):
//   top-k keeps the first k, top-p of those the shortest prefix whose weights reach p of their
//   sum, min-p those with w_i >= min_p; the token is the first in vocabulary order whose
//   cumulative kept weight exceeds u times their sum.
// What is kept is then all l > t and the first n, by index, of l == t: a threshold is searched
// for, and nothing is sorted but a short list around it.
//
// The answer is a whole number that turns on comparisons of long sums, so weights are integers
// in units of 2^-44 of the largest: their sums are exact, in whatever order they are formed, and
// the sum that the search compares is the one that the drawing walks through.  A weight itself
// is good to 2^-31 (table-driven exponential after Tang, 1989): a draw among 250,000
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
constexpr int kBins = 2048;        // of -log2(weight), 0 .. 45
constexpr float kLeast = -45.0f;   // weights below 2^-45 are 0
constexpr float kBinsPerOctave = kBins / 45.0f;
constexpr int kList = 1024;        // candidates that are sorted
constexpr int kTable = 32;
constexpr uint32_t kAll = 0x7fffffffu;

struct Params {
  const void* logits;
  const float* u;
  const float* temperature;  // [T], or nullptr: temperature_all (as the three below)
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  double temperature_all, top_p_all, min_p_all;
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

// A row's way from a logit to its weight: w = 2^y, y = (l / 2 - max / 2) (c_hi + c_lo).  Halves:
// the difference of two fp32 numbers need not be one.
struct Scale {
  float half_max, c_hi, c_lo;
};

// y, not below -64; -inf (whatever l is infinitely below max) and NaN give -64.
__device__ __forceinline__ float log2_weight(float l, const Scale& s, float& d) {
  d = fminf(fmaf(l, 0.5f, -s.half_max), 0.0f);  // NaN where both are infinite: 0, the weight 1
  return fmaxf(d * s.c_hi, -64.0f);
}

// The weight in units of 2^-44.  `lane_table`: this lane's column of the table, which is there
// once for every lane so that no two lanes meet in a bank.
template <typename E>
__device__ __forceinline__ U64 weight(float l, const Scale& s, const uint2* lane_table) {
  constexpr float kMagic = 393216.0f;  // 1.5 2^18: sums round to whole multiples of 1/32
  float d;
  const float y = log2_weight(l, s, d);
  const float yh = d * s.c_hi;
  float lo = fmaf(d, s.c_lo, fmaf(d, s.c_hi, -yh));
  if constexpr (sizeof(E) == 4) {  // what l - max rounds off; bf16 logits lose nothing that counts
    const float h = 0.5f * l, b = d - h;
    lo = fmaf((h - (d - b)) + (-s.half_max - b), s.c_hi, lo);
  }
  const float t = y + kMagic;
  const float r = (y - (t - kMagic)) + lo;  // |r| <= 1/64 (the difference is exact); NaN where l or max is infinite
  const int bits = __float_as_int(t);
  const uint2 entry = lane_table[(bits & (kTable - 1)) * 32];
  // 2^r - 1, off by less than 2^-32.8: a polynomial fitted to it (least largest error on |r| <= 1/64)
  const float p = r * fmaf(r, fmaf(r, 0.05550457f, 0.24022846f), 0.6931472f);
  const uint32_t w = entry.x + static_cast<uint32_t>(__float2int_rn(__uint_as_float(entry.y) * p));
  const int shift = (__float_as_int(kMagic) - bits + kTable - 1) >> 5;  // whole octaves below 1: 0 .. 64
  return (static_cast<U64>(w) << (kUnit - 31)) >> min(shift, 63);
}

// Its bin, kBins and more where it is 0.
__device__ __forceinline__ int bin_of(float l, const Scale& s) {
  float d;
  const float y = log2_weight(l, s, d);
  return y > kLeast ? min(static_cast<int>(-y * kBinsPerOctave), kBins - 1) : kBins;
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
  double inv_t, least;
  float c_hi, c_lo;
  uint32_t listed, found[3];
  U64 found_mass;
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
template <typename E>
__global__ void __launch_bounds__(kMaxThreads) sample_kernel(const Params p) {
  constexpr int kPer = Piece<E>::kPer;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  uint4* const pieces = reinterpret_cast<uint4*>(smem);
  uint2* const table = reinterpret_cast<uint2*>(smem + static_cast<size_t>(p.chunk) * 16);
  uint32_t* const bins = reinterpret_cast<uint32_t*>(table + kTable * 32);
  U64* const list = reinterpret_cast<U64*>(bins + kBins);
  U64* const mass_of = list + kList;

  const int threads = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = threads >> 5;
  Cluster cl{p.ctas, static_cast<int>(blockIdx.x % p.ctas), &sh, 0, 0};
  const int64_t row = blockIdx.x / p.ctas;
  const uint2* const lane_table = table + lane;

  for (int i = tid; i < kTable * 32; i += threads) {
    const uint32_t t = kPow2[i / 32];
    table[i] = make_uint2(t, __float_as_uint(static_cast<float>(t)));
  }
  ptx::launch_dependents();
  ptx::wait_prerequisites();

  // This CTA's part of the row: pieces of 16 bytes as they lie in memory; what a piece holds
  // before or behind the row counts as -inf.  A warp has a stretch of its own, and its lanes
  // read back what they have copied themselves.
  const E* const logits = static_cast<const E*>(p.logits) + row * p.ldl;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(logits) & 15) / static_cast<int>(sizeof(E));
  const int all_pieces = (off + p.V + kPer - 1) / kPer;
  const int first = cl.rank * p.chunk;
  const int mine = max(0, min(p.chunk, all_pieces - first));
  const int stretch = ((p.chunk + warps - 1) / warps + 31) / 32 * 32;
  const int w0 = warp * stretch, w1 = min(w0 + stretch, mine);
  const E* const aligned = logits - off;
  for (int i = w0 + lane; i < w1; i += 32) {
    const int64_t at = static_cast<int64_t>(first + i) * kPer - off;  // the piece's first logit
    if (at >= 0 && at + kPer <= p.V) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(pieces + i)), "l"(aligned + at + off)
                   : "memory");
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        reinterpret_cast<E*>(pieces + i)[e] =
            at + e >= 0 && at + e < p.V ? logits[at + e] : lowest<E>();
    }
  }
  const double temperature = p.temperature ? p.temperature[row] : p.temperature_all;
  const int64_t top_k = p.top_k ? p.top_k[row] : p.top_k_all;
  const double top_p = p.top_p ? p.top_p[row] : p.top_p_all;
  const double min_p = p.min_p ? p.min_p[row] : p.min_p_all;
  const bool greedy = !(temperature > 0.0) || top_k == 1 || top_p <= 0.0;
  const bool by_k = top_k > 0, by_p = top_p < 1.0, by_min = min_p > 0.0;
  if (tid == 0) {
    const double inv = temperature > 0.0 ? fmin(1.0 / temperature, 1e37) : 1.0;
    const double c = inv * (2.0 * 1.4426950408889634);
    sh.inv_t = inv;
    sh.c_hi = static_cast<float>(c);
    sh.c_lo = static_cast<float>(c - static_cast<double>(sh.c_hi));
    sh.least = by_min && !greedy ? temperature * log(min_p) : 0.0;
    sh.listed = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  float best = -INFINITY;
  for (int i = w0 + lane; i < w1; i += 32) {
    const Piece<E> l = unpack<E>(pieces[i]);
    bool nan = false;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      best = fmaxf(best, l.v[e]);
      nan = nan || l.v[e] != l.v[e];
    }
    if (nan) {  // never drawn
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (l.v[e] != l.v[e]) reinterpret_cast<E*>(pieces + i)[e] = lowest<E>();
    }
  }
  cl.sync();  // the others' shared memory is there
  const float row_max = float_of(static_cast<uint32_t>(cl.all<MaxMin>(Two{key_of(best), ~0ull}).a));
  if (row_max == -INFINITY) {  // nothing to draw
    if (cl.rank == 0 && tid == 0) {
      p.tokens[row] = p.ignore_index;
      if (p.logp) p.logp[row] = 0.0f;
    }
    return;
  }
  const Scale sc{0.5f * row_max, sh.c_hi, sh.c_lo};
  const auto each = [&](auto f) {  // every logit of this thread's and its piece's number
    for (int i = w0 + lane; i < w1; i += 32) {
      const Piece<E> l = unpack<E>(pieces[i]);
#pragma unroll
      for (int e = 0; e < kPer; ++e) f(l.v[e], (first + i) * kPer + e - off);
    }
  };

  // What is kept: l > t, and the first n of l == t.
  float t = -INFINITY;
  uint32_t n = 0;
  if (greedy) t = row_max, n = 1;

  // The candidates' list, best first, on the first CTA: the elements `in` selects, `m` of them.
  const auto gather_list = [&](auto in) {
    each([&](float l, int index) {
      if (in(l)) {
        const uint32_t at = atomicAdd(peer(&sh.listed, 0), 1u);
        if (at < kList) *peer(list + at, 0) = static_cast<U64>(key_of(l)) << 32 | (0xffffffffu - static_cast<uint32_t>(index));
      }
    });
    cl.sync();
  };
  // On the first CTA: sorts the list and gives mass_of[] the sums of its weights up to each.
  const auto sort_list = [&]() -> int {
    const int m = min(static_cast<int>(sh.listed), kList);
    int size = 32;
    while (size < m) size *= 2;
    for (int i = m + tid; i < size; i += threads) list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int i = tid; i < size / 2; i += threads) {
          const int a = (i / j) * 2 * j + i % j, b = a + j;
          const U64 x = list[a], y = list[b];
          if ((x < y) == ((a & k) == 0)) list[a] = y, list[b] = x;
        }
        __syncthreads();
      }
    const int per = (m + threads - 1) / threads;
    U64 sum = 0;
    for (int i = tid * per; i < min((tid + 1) * per, m); ++i) sum += weight<E>(float_of(static_cast<uint32_t>(list[i] >> 32)), sc, lane_table);
    U64 run = block_before(sum, &sh);
    for (int i = tid * per; i < min((tid + 1) * per, m); ++i)
      mass_of[i] = run += weight<E>(float_of(static_cast<uint32_t>(list[i] >> 32)), sc, lane_table);
    if (tid == 0) sh.listed = 0, sh.found[0] = static_cast<uint32_t>(m);
    __syncthreads();
    return m;
  };
  // The shortest prefix of the first m of the list whose weights reach `need`.
  const auto prefix_of = [&](int m, U64 need) -> int {
    __syncthreads();
    if (tid == 0) sh.found[0] = static_cast<uint32_t>(m);
    __syncthreads();
    for (int i = tid; i < m; i += threads)
      if (mass_of[i] >= need && (i == 0 || mass_of[i - 1] < need)) sh.found[0] = static_cast<uint32_t>(i) + 1;
    __syncthreads();
    return static_cast<int>(sh.found[0]);
  };
  // The first `m` of the list as a threshold: every thread of the first CTA has it.
  const auto plan_of = [&](int m, U64 mass) {
    const uint32_t last = static_cast<uint32_t>(list[m - 1] >> 32);
    __syncthreads();
    if (tid == 0) sh.found[1] = 0;
    __syncthreads();
    uint32_t equal = 0;
    for (int i = tid; i < m; i += threads) equal += static_cast<uint32_t>(list[i] >> 32) == last ? 1u : 0u;
    if (equal) atomicAdd(&sh.found[1], equal);
    __syncthreads();
    return Plan{mass, last, sh.found[1], 0};
  };

  if (!greedy && (by_k || by_p)) {
    // How many logits fall into each of 2048 bins of log2(weight), and the sum of weights.
    for (int i = tid; i < kBins; i += threads) bins[i] = 0;
    __syncthreads();
    U64 sum = 0;
    each([&](float l, int) {
      const int b = bin_of(l, sc);
      if (b < kBins) atomicAdd(bins + b, 1u);
      if (!by_k) sum += weight<E>(l, sc, lane_table);
    });
    U64 total = cl.all<Sum>(Two{sum, 0}).a;  // everything that has a weight; with top-k: of the first k, later
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
    // Bins [a, b] that hold the end of the shortest prefix with `need` logits, or weights, and
    // how many lie up to b.
    const auto bracket = [&](bool mass, U64 need) {
      Plan plan{0, 0, 0, 0};
      if (cl.rank == 0) {
        if (tid == 0) sh.found[0] = sh.found[1] = kBins - 1;
        __syncthreads();
        if (!mass) {
          for (int i = tid; i < kBins; i += threads)
            if (bins[i] >= need && (i == 0 || bins[i - 1] < need)) sh.found[0] = sh.found[1] = i;
        } else {  // between the bounds of their weights
          for (int side = 0; side < 2; ++side) {
            const auto bound = [&](int i) -> U64 {
              const uint32_t c = bins[i] - (i ? bins[i - 1] : 0u);
              const float w = ptx::ex2(static_cast<float>(-i - side) * (1.0f / kBinsPerOctave)) * (side ? 1.0f - 0x1p-15f : 1.0f + 0x1p-15f);
              const U64 each_one = static_cast<U64>(w * 0x1p44f);
              return c * (side ? (each_one ? each_one - 1 : 0) : each_one + 2);
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
        plan = Plan{bins[kBins - 1], sh.found[0], sh.found[1], bins[sh.found[1]]};
      }
      return cl.tell(plan);
    };
    // The end of that prefix, where more logits share its bins than can be sorted: bisection of
    // their values.  Returns the threshold, how many of its equals, and the prefix's weight.
    const auto bisect = [&](bool by_mass, U64 need, const Plan& in) {
      const int b1 = static_cast<int>(in.a), b2 = static_cast<int>(in.b);
      Two above{0, 0}, range{0, ~0ull};
      U64 count = 0;
      each([&](float l, int) {
        const int b = bin_of(l, sc);
        if (b < b1) {
          above.a += weight<E>(l, sc, lane_table), ++above.b;
        } else if (b <= b2) {
          ++count;
          const U64 k = key_of(l);
          range = MaxMin::of(range, Two{k, k});
        }
      });
      above = cl.all<Sum>(above);
      count = cl.all<Sum>(Two{count, 0}).a;
      range = cl.all<MaxMin>(range);
      uint32_t hi = static_cast<uint32_t>(range.a), lo = static_cast<uint32_t>(range.b);
      while (count > kList && lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;  // (mid, hi] or [lo, mid]
        Two top{0, 0};
        each([&](float l, int) {
          const uint32_t k = key_of(l);
          if (k > mid && k <= hi) top.a += weight<E>(l, sc, lane_table), ++top.b;
        });
        top = cl.all<Sum>(top);
        if ((by_mass ? above.a + top.a : above.b + top.b) >= need)
          lo = mid + 1, count = top.b;
        else
          hi = mid, count -= top.b, above = Sum::of(above, top);
      }
      Plan plan{0, 0, 0, 0};
      if (lo >= hi) {  // equal ones
        const U64 w = weight<E>(float_of(hi), sc, lane_table);
        U64 equal = by_mass ? (w ? (need - above.a + w - 1) / w : 1) : need - above.b;
        equal = equal < 1 ? 1 : equal > count ? count : equal;
        return Plan{above.a + equal * w, hi, static_cast<uint32_t>(equal), 0};
      }
      gather_list([&](float l) {
        const uint32_t k = key_of(l);
        return k >= lo && k <= hi;
      });
      if (cl.rank == 0) {
        const int m = sort_list();
        const int end = by_mass ? prefix_of(m, need - above.a) : min(m, static_cast<int>(need - above.b));
        plan = plan_of(end, above.a + mass_of[end - 1]);
      }
      return cl.tell(plan);
    };

    Plan end{0, 0, 0, 0};
    bool found = false, done = !by_p;
    if (by_k) {
      const Plan in = bracket(false, static_cast<U64>(top_k));
      if (static_cast<U64>(top_k) >= in.mass) {  // all that have a weight
        if (by_p) {
          sum = 0;
          each([&](float l, int) { sum += weight<E>(l, sc, lane_table); });
          total = cl.all<Sum>(Two{sum, 0}).a;
        }
      } else if (in.c <= kList) {  // top-p with it
        gather_list([&](float l) { return bin_of(l, sc) <= static_cast<int>(in.b); });
        Plan plan{0, 0, 0, 0};
        if (cl.rank == 0) {
          sort_list();
          int m = static_cast<int>(top_k);
          if (by_p) m = prefix_of(m, share_up(top_p, mass_of[m - 1]));
          plan = plan_of(m, mass_of[m - 1]);
        }
        end = cl.tell(plan);
        found = done = true;
      } else {
        end = bisect(false, static_cast<U64>(top_k), in);
        total = end.mass;
        found = true;
      }
    }
    if (!done) {
      const U64 need = share_up(top_p, total);
      const Plan in = bracket(true, need);
      if (in.c <= kList) {
        gather_list([&](float l) { return bin_of(l, sc) <= static_cast<int>(in.b); });
        Plan plan{0, 0, 0, 0};
        if (cl.rank == 0) {
          const int m = prefix_of(sort_list(), need);
          plan = plan_of(m, mass_of[m - 1]);
        }
        end = cl.tell(plan);
      } else {
        end = bisect(true, need, in);
      }
      found = true;
    }
    if (found) t = float_of(end.a), n = end.b;
  }
  if (!greedy && by_min) {
    const float least = fminf(__double2float_ru(static_cast<double>(row_max) + sh.least), row_max);
    if (least > t) t = least, n = kAll;
  }

  // The kept weights of every warp's stretch, and the draw.
  Two own{0, 0};
  for (int i = w0 + lane; i < w1; i += 32) {
    const Piece<E> l = unpack<E>(pieces[i]);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (l.v[e] > t)
        own.a += weight<E>(l.v[e], sc, lane_table);
      else if (l.v[e] == t)
        ++own.b;
    }
  }
  const Two* from = cl.gather<Sum>(own);
  const U64 w_t = n ? weight<E>(t, sc, lane_table) : 0;
  const auto kept = [&](const Two& s) { return s.a + (s.b < n ? s.b : static_cast<U64>(n)) * w_t; };
  Two before{0, 0}, all{0, 0};
  for (int i = 0; i < p.ctas; ++i) {
    if (i == cl.rank) before = all;
    all = Sum::of(all, from[i]);
  }
  const U64 total = kept(all);
  const float u = p.u[row];
  const U64 target = share_down(u > 0.0f ? static_cast<U64>(fminf(u, 0x1.fffffep-1f) * 0x1p63f) : 0, total);
  for (int i = 0; i < warp; ++i) before = Sum::of(before, sh.part[i]);
  const Two here = Sum::of(before, sh.part[warp]);
  if (!(kept(before) <= target && target < kept(here))) return;  // another warp's stretch
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    Two v{0, 0};
    Piece<E> l;
    if (i < w1) {
      l = unpack<E>(pieces[i]);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (l.v[e] > t)
          v.a += weight<E>(l.v[e], sc, lane_table);
        else if (l.v[e] == t)
          ++v.b;
      }
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
        float drawn = 0.0f;
        int e_drawn = -1;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (l.v[e] > t)
            run.a += weight<E>(l.v[e], sc, lane_table);
          else if (l.v[e] == t)
            ++run.b;
          if (e_drawn < 0 && kept(run) > target) e_drawn = e, drawn = l.v[e];
        }
        p.tokens[row] = static_cast<int64_t>(first + i) * kPer + e_drawn - off;
        if (p.logp) {
          // log(weight / total): of the total the exponent, the leading 24 bits, and the rest apart
          const int top = 63 - __clzll(total);
          const U64 bits = total << (63 - top);
          const float lead = __ull2float_rz(bits);
          const float rest = static_cast<float>(bits - static_cast<U64>(lead)) / lead;
          const double d = drawn == row_max ? 0.0 : static_cast<double>(drawn) - static_cast<double>(row_max);
          const double log_total =
              static_cast<double>(top - kUnit) * 0.6931471805599453 + (static_cast<double>(logf(lead * 0x1p-63f)) + rest);
          p.logp[row] = greedy ? 0.0f : static_cast<float>(d * sh.inv_t - log_total);
        }
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
