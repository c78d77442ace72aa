// Objectives on per-token log-probabilities: the clipped policy loss with a KL
// term, and the preference loss on paired log ratios.  Each returns its loss and
// the gradient on logp (what flce_backward_logp takes) from one reading of its
// inputs.
//
// Bound: bytes (28 and 20 per token, a few operations each), and below about a
// million tokens latency: launches and the reduction's steps.
//
// Sums, all in a fixed order.  Policy: fp32 over the tokens of one warp (four of each
// thread; beyond 2 M tokens several steps of four), 64 bits across warps and blocks.
// Preference, where log ratios cancel: fp32 with what it rounds off over a warp, 64
// bits from there on.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "vec8.cuh"

namespace flce {
namespace loss {

constexpr float kMaxLogRatio = 20.0f;  // log ratios are clamped here before exp()
constexpr int kStatusSequences = 8;    // FLCE_ERR_SEQUENCES

enum Reduction : int { kNone = 0, kMean = 1, kSum = 2, kSequenceMean = 3 };
enum Kl : int { kK1 = 1, kK2 = 2, kK3 = 3 };
enum Preference : int { kSigmoid = 0, kHinge = 1, kIpo = 2 };

// Keeps NaN (fminf / fmaxf would drop it).
__device__ __forceinline__ float clamp_ratio(float v) {
  return v > kMaxLogRatio ? kMaxLogRatio : (v < -kMaxLogRatio ? -kMaxLogRatio : v);
}

// e^v - 1 - v from v and em = expm1f(v).  Their difference cancels where v is small (at
// 10^-6, where kl is 5 10^-13, all but three bits of it), so below 1/2 the power series is
// summed: v^2 (1/2! + v/3! + .. + v^7/9!), the next term below 3 10^-9 of the first.
__device__ __forceinline__ float exp_above_line(float v, float em) {
  const float v2 = v * v;  // pairs of terms in v^2: a shorter chain than one after the other
  const float a = fmaf(1.0f / 6.0f, v, 0.5f), b = fmaf(1.0f / 120.0f, v, 1.0f / 24.0f);
  const float c = fmaf(1.0f / 5040.0f, v, 1.0f / 720.0f), d = fmaf(1.0f / 362880.0f, v, 1.0f / 40320.0f);
  return fabsf(v) < 0.5f ? v2 * fmaf(fmaf(fmaf(d, v2, c), v2, b), v2, a) : em - v;
}

// ------------------------------------------------------------------ policy loss
struct PolicyParams {
  const float* dloss;    // [1] or [T] (NONE), nullptr: ones
  const float* logp;
  const float* old_logp;
  const float* ref;      // or nullptr
  const float* adv;      // [T] or [S]
  const int64_t* targets;
  const int64_t* cu;     // [S + 1] or nullptr
  float* loss;           // or nullptr
  float* dlogp;          // or nullptr
  float* stats;          // or nullptr
  int64_t* n_valid;      // or nullptr
  int64_t ignore_index;
  int32_t T, S;
  int32_t adv_per_seq, reduction, kl_kind;
  float log_hi, log_lo, ratio_hi, ratio_lo;
  float log_dual, dual;  // log_dual = +inf when there is no dual clip
  float kl_coef;
  // workspace
  int32_t* status;
  int32_t* ticket;       // CTAs of the main launch that are done
  int32_t* nonempty;     // sequences with a valid token (many sequences)
  int32_t* seq_count;    // [S] valid tokens of each sequence (the one-cluster form)
  int32_t* block_count;  // [blocks] valid tokens of a block of `chunk` tokens
  int32_t* block_bad;    // [blocks]
  uint2* words;          // [ceil(T / 32)] mask of 32 tokens, valid tokens of the block before them
  double* block_sum;     // [CTAs of the main launch][5]
  int32_t blocks;        // blocks of the first launch, or CTAs of the one cluster
  int32_t chunk;         // tokens of a block
  int32_t vec;           // every per-token array is 16-byte aligned
};

struct PolicyTerm {
  float loss, grad, kl, cut, d, rho;
};

// One token: value and derivative in logp.
__device__ __forceinline__ PolicyTerm policy_token(const PolicyParams& p, float lp, float old, float ref, float A) {
  PolicyTerm o;
  const float raw = lp - old;
  o.d = clamp_ratio(raw);
  o.rho = expf(o.d);
  // Clipped where the clipped product is the smaller one: by the sign of A.  The
  // test is on the log ratio (exp is monotone), so it does not depend on exp's rounding.
  float ratio = o.rho;
  bool cut = false;
  if (A > 0.0f && o.d > p.log_hi) ratio = p.ratio_hi, cut = true;
  if (A < 0.0f && o.d < p.log_lo) ratio = p.ratio_lo, cut = true;
  if (A < 0.0f && o.d > p.log_dual) ratio = p.dual, cut = true;
  o.cut = cut ? 1.0f : 0.0f;
  o.loss = -A * ratio;
  o.grad = cut || fabsf(raw) > kMaxLogRatio ? 0.0f : -A * o.rho;
  o.kl = 0.0f;
  if (p.ref) {
    const float e = ref - lp;
    float dkl;
    if (p.kl_kind == kK1) {
      o.kl = -e, dkl = 1.0f;
    } else if (p.kl_kind == kK2) {
      o.kl = 0.5f * e * e, dkl = -e;
    } else {
      const float ec = clamp_ratio(e), em = expm1f(ec);
      o.kl = exp_above_line(ec, em);
      dkl = fabsf(e) > kMaxLogRatio ? 0.0f : -em;
    }
    o.loss = fmaf(p.kl_coef, o.kl, o.loss);
    o.grad = fmaf(p.kl_coef, dkl, o.grad);
  }
  return o;
}

constexpr int kSums = 5;          // loss, kl, cut, log ratio, ratio

// Sum over the block in a fixed order; the result on thread 0.
template <typename E, int THREADS>
__device__ __forceinline__ E block_sum(E v, E* sh) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int warp = threadIdx.x >> 5;
  __syncthreads();  // sh may still be read from the sum before
  if ((threadIdx.x & 31) == 0) sh[warp] = v;
  __syncthreads();
  E s = 0;
  if (threadIdx.x == 0)
    for (int i = 0; i < THREADS / 32; ++i) s += sh[i];
  return s;
}

// ------------------------------------------------------------------ policy loss in one launch
// Up to 16 * 512 * 4 = 32,768 tokens: one cluster of CTAs.  A token's loss and
// gradient do not depend on how many tokens count; only the common weight does.
// So every thread reads its four tokens once and keeps the unscaled gradients in
// registers while the counts go round the cluster through distributed shared
// memory (or, per sequence, through integer atomics in the workspace), and scales
// and stores them after one cluster barrier.  No second launch, no second reading:
// 32,768 tokens take 6.7 us, whose bytes (0.9 MB) would take 0.1 us; the rest is the
// launch, one round of loads, the barrier and the tree of the sums.
// Beyond that the 16 SMs of a cluster are too few (131,072 tokens in 61 sequences: 25.5
// us with four such steps a thread), and the two launches further down take over.
constexpr int kClusterCtas = 16;
constexpr int kClusterThreads = 512;
constexpr int kGroup = 4;            // consecutive tokens of a thread and step
constexpr int kCuShared = 4096;      // sequence offsets kept in shared memory
constexpr int kWalk = 4;             // sequences stepped over one by one

__device__ __forceinline__ float4 load4(const float* p, int64_t t, int n, bool vec) {
  if (vec) return __ldg(reinterpret_cast<const float4*>(p + t));
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (n > 0) v.x = __ldg(p + t);
  if (n > 1) v.y = __ldg(p + t + 1);
  if (n > 2) v.z = __ldg(p + t + 2);
  if (n > 3) v.w = __ldg(p + t + 3);
  return v;
}

__device__ __forceinline__ void store4(float* p, int64_t t, int n, bool vec, const float (&v)[kGroup]) {
  if (vec) {
    *reinterpret_cast<float4*>(p + t) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (j < n) p[t + j] = v[j];
}

// Bit j: token t + j counts by its target.
__device__ __forceinline__ uint32_t valid4(const int64_t* y, int64_t ignore, int64_t t, int n, bool vec) {
  if (vec) {
    const longlong2 a = __ldg(reinterpret_cast<const longlong2*>(y + t));
    const longlong2 b = __ldg(reinterpret_cast<const longlong2*>(y + t + 2));
    return (a.x != ignore ? 1u : 0u) | (a.y != ignore ? 2u : 0u) | (b.x != ignore ? 4u : 0u) | (b.y != ignore ? 8u : 0u);
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (j < n && __ldg(y + t + j) != ignore) m |= 1u << j;
  return m;
}

__device__ __forceinline__ float lane4(const float4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The two halves of the cluster barrier; every thread of the warp together.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The offsets of the sequences: from shared memory where they fit, else from global.
struct Offsets {
  const int32_t* sh;
  const int64_t* cu;
  int n;       // sequences
  __device__ __forceinline__ int64_t at(int i) const { return sh ? sh[i] : __ldg(cu + i); }
  // Index s with cu[s] <= t < cu[s + 1], or -1 when t lies in none.  Any contents of cu
  // give an index in [-1, n - 1].
  __device__ __forceinline__ int find(int64_t t) const {
    int lo = 0, hi = n + 1;  // the first index with cu[index] > t lies in [lo, hi]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (at(mid) > t) hi = mid;
      else lo = mid + 1;
    }
    return lo > n ? -1 : lo - 1;  // lo == 0: before the first sequence; n + 1: after the last
  }
  // The sequence of token t from the one of an earlier token: that one or one of the
  // next few.  Any number of empty sequences may lie between two tokens (walking past
  // 2,000,000 took 0.8 s), so beyond a few it is searched for.
  __device__ __forceinline__ int step(int s, int64_t t) const {
    if (s < 0) return find(t);
    const int most = min(s + kWalk, n);
    while (s < most && at(s + 1) <= t) ++s;
    return s < most ? s : find(t);
  }
};

// Four tokens of a thread: their inputs, and what does not depend on the counts.
struct Tokens4 {
  float4 lp, old, ref, adv;
  uint32_t mask;               // bit j: token t + j counts
  int seq0;                    // sequence of the first token that counts
  float grad[kGroup], val[kGroup];
};

__device__ __forceinline__ void load_tokens(const PolicyParams& p, int64_t t, int left, bool vec, Tokens4& q) {
  q.mask = valid4(p.targets, p.ignore_index, t, left, vec);
  q.lp = load4(p.logp, t, left, vec);
  q.old = load4(p.old_logp, t, left, vec);
  if (p.ref) q.ref = load4(p.ref, t, left, vec);
  if (!p.adv_per_seq) q.adv = load4(p.adv, t, left, vec);
}

// [first, end): the tokens that lie in a sequence.
__device__ __forceinline__ void eval_tokens(const PolicyParams& p, const Offsets& off, bool by_seq, int64_t first,
                                            int64_t end, int64_t t, Tokens4& q, float (&sum)[kSums], int& n) {
  uint32_t m = q.mask;
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (t + j < first || t + j >= end) m &= ~(1u << j);
  int s = -1;
  float A_seq = 0.0f;
  if (by_seq && m) {
    s = off.find(t + __ffs(m) - 1);
    if (s < 0) m = 0;
    else if (p.adv_per_seq) A_seq = __ldg(p.adv + s);
  }
  q.seq0 = s;
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    q.grad[j] = q.val[j] = 0.0f;
    if (!(m >> j & 1u)) continue;
    float A = lane4(q.adv, j);
    if (by_seq) {
      const int was = s;
      s = off.step(s, t + j);
      if (s < 0) {  // only where cu is not in order
        m &= ~(1u << j);
        continue;
      }
      if (p.adv_per_seq) {
        if (s != was) A_seq = __ldg(p.adv + s);
        A = A_seq;
      }
    }
    const PolicyTerm o = policy_token(p, lane4(q.lp, j), lane4(q.old, j), lane4(q.ref, j), A);
    q.grad[j] = o.grad;
    q.val[j] = o.loss;
    sum[0] += o.loss, sum[1] += o.kl, sum[2] += o.cut, sum[3] += o.d, sum[4] += o.rho;
    ++n;
  }
  q.mask = m;
}

// SEQUENCE_MEAN: every token's weight from its sequence's count; the weighted loss is returned.
template <typename Count>
__device__ __forceinline__ float weigh_tokens(const Offsets& off, int64_t t, float scale, Tokens4& q, Count count) {
  float total = 0.0f;
  int s = q.seq0;
  float w = q.mask ? scale / static_cast<float>(count(s)) : 0.0f;
#pragma unroll
  for (int j = 0; j < kGroup; ++j)
    if (q.mask >> j & 1u) {
      const int was = s;
      s = off.step(s, t + j);
      if (s != was) w = scale / static_cast<float>(count(s));
      q.grad[j] *= w;
      total = fmaf(q.val[j], w, total);
    }
  return total;
}

__device__ __forceinline__ void store_tokens(const PolicyParams& p, int64_t t, int left, bool vec, float scale, Tokens4& q) {
  if (p.dlogp) {
    const float up = p.dloss && p.reduction != kNone ? __ldg(p.dloss) : 1.0f;
    float4 u = make_float4(up, up, up, up);
    if (p.reduction == kNone && p.dloss) u = load4(p.dloss, t, left, vec);
#pragma unroll
    for (int j = 0; j < kGroup; ++j) q.grad[j] = q.mask >> j & 1u ? q.grad[j] * scale * lane4(u, j) : 0.0f;
    store4(p.dlogp, t, left, vec, q.grad);
  }
  if (p.loss && p.reduction == kNone) store4(p.loss, t, left, vec, q.val);
}

// The scalar outputs from the summed terms: thread i < kSums holds sum i.
__device__ __forceinline__ void store_scalars(const PolicyParams& p, int i, double v, int64_t valid) {
  const double inv = valid > 0 ? 1.0 / static_cast<double>(valid) : 0.0;
  if (i == 0) {
    if (p.loss && p.reduction != kNone) p.loss[0] = static_cast<float>(p.reduction == kMean ? v * inv : v);
    if (p.n_valid) *p.n_valid = valid;
  } else if (p.stats) {
    p.stats[i - 1] = static_cast<float>(v * inv);
  }
}

__global__ void __launch_bounds__(kClusterThreads) policy_cluster_kernel(const PolicyParams p) {
  constexpr int kWarps = kClusterThreads / 32;
  __shared__ int32_t cu_sh[kCuShared];
  __shared__ float warp_sum[kWarps][kSums];
  __shared__ int warp_n[kWarps];
  __shared__ int cta_n[kClusterCtas];              // written by the cluster's CTAs
  __shared__ double cta_sum[kClusterCtas][kSums];  // CTA 0's: written by all
  __shared__ int total;
  const int rank = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = p.blocks;
  const bool seq_mean = p.reduction == kSequenceMean;
  const bool by_seq = seq_mean || p.adv_per_seq;
  const int64_t t = static_cast<int64_t>(kGroup) * (rank * kClusterThreads + tid);
  const int left = static_cast<int>(min(max(p.T - t, int64_t(0)), int64_t(kGroup)));
  const bool vec = p.vec && left == kGroup;
  Tokens4 q{};
  if (left > 0) load_tokens(p, t, left, vec, q);

  if (seq_mean)
    for (int i = rank * kClusterThreads + tid; i < p.S; i += ctas * kClusterThreads) p.seq_count[i] = 0;
  Offsets off{by_seq && p.S < kCuShared ? cu_sh : nullptr, p.cu, p.S};
  bool bad = false;
  if (p.cu) {
    // every CTA reads what it keeps; otherwise the CTAs share the check
    const int first = off.sh ? tid : rank * kClusterThreads + tid;
    const int step = off.sh ? kClusterThreads : ctas * kClusterThreads;
    for (int i = first; i <= p.S; i += step) {
      const int64_t a = i ? p.cu[i - 1] : 0, b = p.cu[i];
      bad = bad || b < a || b > p.T;
      if (off.sh) cu_sh[i] = static_cast<int32_t>(min(max(b, int64_t(0)), int64_t(p.T)));
    }
  }
  const int64_t first_tok = p.cu ? p.cu[0] : 0, end_tok = p.cu ? p.cu[p.S] : p.T;
  bad = __syncthreads_or(bad);
  if (rank == 0 && tid == 0) *p.status = 0;
  cluster_arrive();  // zeroed counts, and: every CTA of the cluster is running

  float sum[kSums] = {};
  int n = 0;
  if (left > 0) eval_tokens(p, off, by_seq, first_tok, end_tok, t, q, sum, n);

  cluster_wait();
  if (seq_mean) {
    // valid tokens of each sequence: one atomic for a warp whose tokens lie in one
    // sequence, else one for each run of a thread's tokens
    int s = q.seq0;
    bool one = true;
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (q.mask >> j & 1u) {
        s = off.step(s, t + j);
        one = one && s == q.seq0;
      }
    const unsigned has = __ballot_sync(0xffffffffu, q.mask != 0);
    if (has) {
      const int lead = __shfl_sync(0xffffffffu, q.seq0, __ffs(has) - 1);
      const bool same = q.mask == 0 || (one && q.seq0 == lead);
      if (__all_sync(0xffffffffu, same)) {
        const int c = __reduce_add_sync(0xffffffffu, __popc(q.mask));
        if (lane == 0) atomicAdd(p.seq_count + lead, c);
      } else if (q.mask) {
        int run = 0, last = q.seq0;
        s = last;
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
          if (q.mask >> j & 1u) {
            s = off.step(s, t + j);
            if (s != last) {
              atomicAdd(p.seq_count + last, run);
              run = 0, last = s;
            }
            ++run;
          }
        atomicAdd(p.seq_count + last, run);
      }
    }
    cluster_arrive();
    cluster_wait();
    // sequences with a valid token, counted by every CTA
    int c = 0;
    for (int i = tid; i < p.S; i += kClusterThreads) c += __ldcg(p.seq_count + i) > 0;
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) warp_n[warp] = c;
    __syncthreads();
    if (tid == 0) {
      int a = 0;
      for (int i = 0; i < kWarps; ++i) a += warp_n[i];
      total = a;
    }
    __syncthreads();
    sum[0] = weigh_tokens(off, t, 1.0f / fmaxf(static_cast<float>(total), 1.0f), q,
                          [&](int i) { return __ldcg(p.seq_count + i); });
  }

  // this CTA's sums: fp32 in a warp, 64 bits across warps; one thread per sum pushes them
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    const float v = warp_total(sum[i]);
    if (lane == 0) warp_sum[warp][i] = v;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  __syncthreads();  // warp_n may still be read above
  if (lane == 0) warp_n[warp] = n;
  __syncthreads();
  if (tid < kSums) {
    double v = 0.0;
    for (int i = 0; i < kWarps; ++i) v += static_cast<double>(warp_sum[i][tid]);
    const uint32_t to = ptx::mapa(ptx::smem_u32(&cta_sum[rank][tid]), 0);
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(v) : "memory");
  } else if (tid >= 32 && tid < 32 + ctas) {
    int a = 0;
    for (int i = 0; i < kWarps; ++i) a += warp_n[i];
    ptx::st_shared_cluster_u32(ptx::mapa(ptx::smem_u32(&cta_n[rank]), tid - 32), static_cast<uint32_t>(a));
  }
  cluster_arrive();
  cluster_wait();

  int valid = 0;
  for (int i = 0; i < ctas; ++i) valid += cta_n[i];
  if (left > 0)
    store_tokens(p, t, left, vec, p.reduction == kMean ? 1.0f / fmaxf(static_cast<float>(valid), 1.0f) : 1.0f, q);
  if (rank == 0 && tid < kSums) {
    double v = 0.0;
    for (int i = 0; i < ctas; ++i) v += cta_sum[i][tid];
    store_scalars(p, tid, v, valid);
  }
  if (bad && tid == 0) atomicCAS(p.status, 0, kStatusSequences);
}

// ------------------------------------------------------------------ policy loss in two launches
// More tokens: first the counts alone, from the targets, then everything else with
// the weights known.  The counts are kept so that the number of valid tokens before
// any token is three loads: a prefix over blocks (each CTA of the second launch adds
// up the at most 1024 block counts), one within the block for every 32 tokens, and
// their mask.  A sequence's count is the difference of two, without atomics or an
// array to clear.  The second launch is dispatched while the first still runs and
// loads its tokens before it waits for it; its last CTA adds up the sums in order.
// Those early loads are safe because the count launch is an ordinary one: whatever wrote
// the inputs is complete before it starts.  It must not be dispatched early itself.
// 131,072 tokens in 61 sequences (3.1 MB, 0.5 us): 11.8 us, latency again, of two launches.
constexpr int kManyThreads = 256;
constexpr int kMaxBlocks = 1024;
constexpr int kStep = kManyThreads * kGroup;  // tokens a CTA takes at a time

__global__ void __launch_bounds__(kManyThreads) policy_count_kernel(const PolicyParams p) {
  constexpr int kWarps = kManyThreads / 32;
  __shared__ int warp_n[kWarps];
  ptx::launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t first = p.cu ? p.cu[0] : 0, end = p.cu ? p.cu[p.S] : p.T;
  const int64_t b0 = static_cast<int64_t>(blockIdx.x) * p.chunk, b1 = min(b0 + p.chunk, int64_t(p.T));
  int before = 0;  // valid tokens of the block so far
  for (int64_t base = b0; base < b1; base += kStep) {
    const int64_t t = base + kGroup * tid;
    const int left = static_cast<int>(min(max(b1 - t, int64_t(0)), int64_t(kGroup)));
    uint32_t m = left > 0 ? valid4(p.targets, p.ignore_index, t, left, p.vec && left == kGroup) : 0;
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (t + j < first || t + j >= end) m &= ~(1u << j);
    // eight threads make a word of 32 tokens
    uint32_t word = m << (4 * (lane & 7));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, d);
    const int c = __popc(m);
    const int all = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    if (lane == 0) warp_n[warp] = all;
    __syncthreads();
    int at = before;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) at += warp_n[i];
      before += warp_n[i];
    }
    // words of this warp before this one
    const int w = __popc(word);
    const int w0 = __shfl_sync(0xffffffffu, w, 0), w1 = __shfl_sync(0xffffffffu, w, 8), w2 = __shfl_sync(0xffffffffu, w, 16);
    at += (lane >= 8 ? w0 : 0) + (lane >= 16 ? w1 : 0) + (lane >= 24 ? w2 : 0);
    if ((lane & 7) == 0 && t < b1) p.words[t / 32] = make_uint2(word, static_cast<uint32_t>(at));
  }
  bool bad = false;
  if (p.cu)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kManyThreads + tid; i <= p.S;
         i += static_cast<int64_t>(gridDim.x) * kManyThreads) {
      const int64_t a = i ? p.cu[i - 1] : 0, b = p.cu[i];
      bad = bad || b < a || b > p.T;
    }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    p.block_count[blockIdx.x] = before;
    p.block_bad[blockIdx.x] = bad;
    if (blockIdx.x == 0) *p.ticket = 0, *p.nonempty = 0;
  }
}

// Valid tokens before each block into prefix[0 .. kMaxBlocks], the last one their total.
__device__ __forceinline__ void block_prefix(const PolicyParams& p, int* prefix, int* warp_n) {
  constexpr int kEach = kMaxBlocks / kManyThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int c[kEach], mine = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * kEach + i;
    c[i] = b < p.blocks ? __ldcg(p.block_count + b) : 0;
    mine += c[i];
  }
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_n[warp] = inc;
  __syncthreads();
  int at = inc - mine;
  for (int i = 0; i < warp; ++i) at += warp_n[i];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    prefix[tid * kEach + i] = at;
    at += c[i];
  }
  if (tid == kManyThreads - 1) prefix[kMaxBlocks] = at;
  __syncthreads();
}

// Valid tokens before token i, 0 <= i <= T; and of sequence s.
__device__ __forceinline__ int tokens_before(const PolicyParams& p, const int* prefix, int64_t i) {
  if (i >= p.T) return prefix[kMaxBlocks];
  const uint2 w = __ldcg(p.words + i / 32);
  return prefix[i / p.chunk] + static_cast<int>(w.y) + __popc(w.x & ((1u << (i & 31)) - 1u));
}
__device__ __forceinline__ int tokens_of(const PolicyParams& p, const int* prefix, const Offsets& off, int s) {
  const int64_t a = min(max(off.at(s), int64_t(0)), int64_t(p.T)), b = min(max(off.at(s + 1), int64_t(0)), int64_t(p.T));
  return tokens_before(p, prefix, b) - tokens_before(p, prefix, a);
}

// SEQUENCE_MEAN with many sequences: how many have a valid token, counted once
// instead of by every CTA of the main launch.
__global__ void __launch_bounds__(kManyThreads) policy_nonempty_kernel(const PolicyParams p) {
  __shared__ int prefix[kMaxBlocks + 1];
  __shared__ int warp_n[kManyThreads / 32];
  ptx::launch_dependents();
  block_prefix(p, prefix, warp_n);
  const Offsets off{nullptr, p.cu, p.S};
  int c = 0;
  for (int s = blockIdx.x * kManyThreads + threadIdx.x; s < p.S; s += gridDim.x * kManyThreads)
    c += tokens_of(p, prefix, off, s) > 0;
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0 && c) atomicAdd(p.nonempty, c);
}

__global__ void __launch_bounds__(kManyThreads) policy_main_kernel(const PolicyParams p) {
  constexpr int kWarps = kManyThreads / 32;
  __shared__ int32_t cu_sh[kCuShared];
  __shared__ int prefix[kMaxBlocks + 1];  // valid tokens before each block
  __shared__ float warp_sum[kWarps][kSums];
  __shared__ int warp_n[kWarps];
  __shared__ int last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool seq_mean = p.reduction == kSequenceMean;
  const bool by_seq = seq_mean || p.adv_per_seq;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kStep;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kStep + kGroup * tid;
  int left = static_cast<int>(min(max(p.T - t, int64_t(0)), int64_t(kGroup)));
  Tokens4 q{};
  if (left > 0) load_tokens(p, t, left, p.vec && left == kGroup, q);
  Offsets off{by_seq && p.S < kCuShared ? cu_sh : nullptr, p.cu, p.S};
  if (off.sh)
    for (int i = tid; i <= p.S; i += kManyThreads)
      cu_sh[i] = static_cast<int32_t>(min(max(p.cu[i], int64_t(0)), int64_t(p.T)));
  const int64_t first = p.cu ? p.cu[0] : 0, end = p.cu ? p.cu[p.S] : p.T;

  ptx::wait_prerequisites();
  block_prefix(p, prefix, warp_n);
  const int valid = prefix[kMaxBlocks];
  const auto count = [&](int i) { return tokens_of(p, prefix, off, i); };
  float scale = p.reduction == kMean ? 1.0f / fmaxf(static_cast<float>(valid), 1.0f) : 1.0f;
  if (seq_mean && !off.sh) {
    scale = 1.0f / fmaxf(static_cast<float>(__ldcg(p.nonempty)), 1.0f);
  } else if (seq_mean) {
    int c = 0;
    for (int i = tid; i < p.S; i += kManyThreads) c += count(i) > 0;
    c = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    if (lane == 0) warp_n[warp] = c;
    __syncthreads();
    c = 0;
    for (int i = 0; i < kWarps; ++i) c += warp_n[i];
    scale = 1.0f / fmaxf(static_cast<float>(c), 1.0f);
  }

  float sum[kSums] = {};
  while (left > 0) {
    const bool vec = p.vec && left == kGroup;
    int n = 0;
    const float old_total = sum[0];
    eval_tokens(p, off, by_seq, first, end, t, q, sum, n);
    if (seq_mean) sum[0] = old_total + weigh_tokens(off, t, scale, q, count);
    store_tokens(p, t, left, vec, seq_mean ? 1.0f : scale, q);
    t += stride;
    left = static_cast<int>(min(max(p.T - t, int64_t(0)), int64_t(kGroup)));
    if (left > 0) load_tokens(p, t, left, p.vec && left == kGroup, q);
  }
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    const float v = warp_total(sum[i]);
    if (lane == 0) warp_sum[warp][i] = v;
  }
  __syncthreads();
  if (tid < kSums) {
    double v = 0.0;
    for (int i = 0; i < kWarps; ++i) v += static_cast<double>(warp_sum[i][tid]);
    p.block_sum[static_cast<int64_t>(blockIdx.x) * kSums + tid] = v;
    __threadfence();
  }
  __syncthreads();
  if (tid == 0) last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!last) return;
  // the last CTA: all sums are in memory; warp i adds up sum i, 32 CTAs at a time in order
  __threadfence();
  if (warp < kSums) {
    double v = 0.0;
    for (int b = lane; b < static_cast<int>(gridDim.x); b += 32) v += __ldcg(p.block_sum + static_cast<int64_t>(b) * kSums + warp);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (lane == 0) store_scalars(p, warp, v, valid);
  } else if (warp == kSums) {
    int bad = 0;
    for (int b = lane; b < p.blocks; b += 32) bad |= __ldcg(p.block_bad + b);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) *p.status = bad ? kStatusSequences : 0;
  }
}

// ------------------------------------------------------------------ preference loss
struct PreferenceParams {
  const float* dloss;    // [1] or [P] (NONE), nullptr: ones
  const float* logp;
  const float* ref;      // or nullptr
  const int64_t* targets;
  const int64_t* cu;     // [2 P + 1]
  float* loss;           // [1], [P] (NONE) or nullptr
  float* dlogp;          // [T] or nullptr
  float* chosen;         // [P] or nullptr
  float* rejected;       // [P] or nullptr
  int64_t ignore_index;
  int64_t T;
  int32_t P;
  int32_t reduction, kind, normalize;
  float beta, smoothing, margin, inv_2beta;
  int32_t* status;
  int32_t* pair_bad;     // [P]
  double* pair_loss;     // [P]
  int32_t ctas;          // CTAs of a cluster
  int32_t vec;           // every per-token array is 16-byte aligned
};

__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }
__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// Value and derivative of one pair's loss in D = S_chosen - S_rejected.
__device__ __forceinline__ void pair_loss(const PreferenceParams& p, float D, float* value, float* slope) {
  const float h = p.beta * D - p.margin;
  if (p.kind == kSigmoid) {
    *value = (1.0f - p.smoothing) * softplus(-h) + p.smoothing * softplus(h);
    *slope = p.beta * (p.smoothing * sigmoid(h) - (1.0f - p.smoothing) * sigmoid(-h));
  } else if (p.kind == kHinge) {
    *value = h < 1.0f ? 1.0f - h : (h >= 1.0f ? 0.0f : h);  // NaN stays NaN
    *slope = h < 1.0f ? -p.beta : 0.0f;
  } else {
    const float m = D - p.inv_2beta;
    *value = m * m;
    *slope = 2.0f * m;
  }
}

constexpr int kPairThreads = 512;    // 256 for the chosen answer, 256 for the rejected one
constexpr int kSide = kPairThreads / 2;
constexpr int kSideWarps = kSide / 32;
constexpr int kKept = 8;             // steps whose mask bits a thread keeps for the second pass
constexpr int kPairCtas = 16;

// Log ratios cancel in the sums, so these keep what fp32 additions round off, within
// a thread and a warp, and are 64 bits wide from there on.
//
// Both answers of a pair at once, one per half of the CTA.  One reading gives the
// sums; the gradient is one number per sequence, so the second pass only stores
// (the mask bits of the first 8 x 1024 tokens stay in a register).
//   SOLO   one cluster holds every pair, one to a CTA (the last CTAs may have none); the
//          scalar loss is summed through distributed shared memory: one launch.
//   else   one cluster per pair, whose CTAs share the pair's tokens and exchange
//          their sums; preference_reduce_kernel adds the pairs' losses.
// 16 pairs of 2 x 200 tokens take 5.3 us.  128 of 2 x 4096 (21 MB, 3.1 us at the copy's
// rate) take 10.4 us, most of it here: a step's loads are used before the next step's are
// issued, and a ragged batch waits for its longest answer's three or four steps.  The
// second reading comes from L2.
template <bool SOLO>
__global__ void __launch_bounds__(kPairThreads) preference_kernel(const PreferenceParams p) {
  __shared__ double warp_s[kPairThreads / 32];
  __shared__ int warp_n[kPairThreads / 32];
  __shared__ double cta_s[2][kPairCtas];  // by CTA of the cluster: sums of the two answers; SOLO: [0] the losses
  __shared__ int cta_n[2][kPairCtas];     // counts; SOLO: [0] malformed pairs
  __shared__ float slope_of[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int side = tid / kSide, i = tid - side * kSide;
  const int ctas = p.ctas;                // of a cluster
  const int rank = blockIdx.x % ctas;
  const int share = SOLO ? 1 : ctas;      // CTAs working on one pair
  const int part = SOLO ? 0 : rank;
  if (!SOLO) ptx::launch_dependents();
  cluster_arrive();  // matched by the wait before the first access to another CTA
  bool arrived = true;
  double loss_sum = 0.0;
  int bad_sum = 0;
  const int pair = SOLO ? rank : blockIdx.x / ctas;
  if (pair < p.P) {
    int64_t at[3];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int64_t v = p.cu[2 * static_cast<int64_t>(pair) + k];
      at[k] = min(max(v, int64_t(0)), p.T);  // no access outside [0, T) whatever cu holds
      bad = bad || v != at[k];
    }
    bad = bad || at[1] < at[0] || at[2] < at[1];
    const int64_t lo = side ? at[1] : at[0], hi = side ? at[2] : at[1];
    const int64_t g0 = lo & ~int64_t(kGroup - 1);
    const int64_t stride = static_cast<int64_t>(kGroup) * kSide * share;
    Twofold sum{0.0f, 0.0f};
    int n = 0, step = 0;
    uint32_t kept = 0;
    for (int64_t t = g0 + static_cast<int64_t>(kGroup) * (part * kSide + i); t < hi; t += stride, ++step) {
      const int left = static_cast<int>(min(p.T - t, int64_t(kGroup)));
      const bool vec = p.vec && left == kGroup;
      uint32_t m = valid4(p.targets, p.ignore_index, t, left, vec);
      const float4 lp = load4(p.logp, t, left, vec);
      float4 ref = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.ref) ref = load4(p.ref, t, left, vec);
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        if (t + j < lo || t + j >= hi) m &= ~(1u << j);
        if (m >> j & 1u) {  // the sum, and what it rounds off
          const float d = lane4(lp, j) - lane4(ref, j), s = sum.hi + d, b = s - sum.hi;
          sum.lo += (sum.hi - (s - b)) + (d - b);
          sum.hi = s;
        }
      }
      n += __popc(m);
      if (step < kKept) kept |= m << (4 * step);
    }
    const Twofold all = warp_sum_twofold(sum);
    // (the low part of an infinite sum is NaN)
    const double ws = isfinite(all.hi) ? static_cast<double>(all.hi) + static_cast<double>(all.lo) : all.hi;
    const int wn = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) warp_s[warp] = ws, warp_n[warp] = wn;
    __syncthreads();
    if (warp == 0) {
      // lanes 0 .. 7: the chosen answer's warps, 8 .. 15 the rejected one's
      double S = lane < 2 * kSideWarps ? warp_s[lane] : 0.0;
      int c = lane < 2 * kSideWarps ? warp_n[lane] : 0;
#pragma unroll
      for (int d = kSideWarps / 2; d > 0; d >>= 1) {
        S += __shfl_xor_sync(0xffffffffu, S, d);
        c += __shfl_xor_sync(0xffffffffu, c, d);
      }
      double S0 = __shfl_sync(0xffffffffu, S, 0), S1 = __shfl_sync(0xffffffffu, S, kSideWarps);
      int c0 = __shfl_sync(0xffffffffu, c, 0), c1 = __shfl_sync(0xffffffffu, c, kSideWarps);
      if (!SOLO && ctas > 1) {
        cluster_wait();
        arrived = false;
        if (lane < ctas) {
          asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(ptx::mapa(ptx::smem_u32(&cta_s[0][rank]), lane)), "d"(S0)
                       : "memory");
          asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(ptx::mapa(ptx::smem_u32(&cta_s[1][rank]), lane)), "d"(S1)
                       : "memory");
          ptx::st_shared_cluster_u32(ptx::mapa(ptx::smem_u32(&cta_n[0][rank]), lane), static_cast<uint32_t>(c0));
          ptx::st_shared_cluster_u32(ptx::mapa(ptx::smem_u32(&cta_n[1][rank]), lane), static_cast<uint32_t>(c1));
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        S0 = S1 = 0.0, c0 = c1 = 0;
        for (int r = 0; r < ctas; ++r) S0 += cta_s[0][r], S1 += cta_s[1][r], c0 += cta_n[0][r], c1 += cta_n[1][r];
      }
      if (lane == 0) {
        if (p.normalize) S0 /= max(c0, 1), S1 /= max(c1, 1);
        float value, slope;
        pair_loss(p, static_cast<float>(S0 - S1), &value, &slope);
        const float up = p.dloss ? p.dloss[p.reduction == kNone ? pair : 0] : 1.0f;
        slope *= p.reduction == kMean ? up / static_cast<float>(p.P) : up;
        slope_of[0] = p.normalize ? slope / static_cast<float>(max(c0, 1)) : slope;
        slope_of[1] = p.normalize ? -slope / static_cast<float>(max(c1, 1)) : -slope;
        if (part == 0) {
          if (p.chosen) p.chosen[pair] = static_cast<float>(p.beta * S0);
          if (p.rejected) p.rejected[pair] = static_cast<float>(p.beta * S1);
          if (p.loss && p.reduction == kNone) p.loss[pair] = value;
          if (!SOLO) p.pair_loss[pair] = value, p.pair_bad[pair] = bad;
        }
        loss_sum = value;
        bad_sum = bad;
      }
    } else if (!SOLO && ctas > 1) {
      cluster_wait();
      arrived = false;
      cluster_arrive();
      cluster_wait();
    }
    __syncthreads();
    if (p.dlogp) {
      const float g = slope_of[side];
      step = 0;
      for (int64_t t = g0 + static_cast<int64_t>(kGroup) * (part * kSide + i); t < hi; t += stride, ++step) {
        const int left = static_cast<int>(min(p.T - t, int64_t(kGroup)));
        const bool vec = p.vec && left == kGroup;
        const uint32_t m = step < kKept ? kept >> (4 * step) : valid4(p.targets, p.ignore_index, t, left, vec);
        float v[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j) v[j] = m >> j & 1u ? g : 0.0f;
        if (t >= lo && t + kGroup <= hi) {
          store4(p.dlogp, t, kGroup, p.vec, v);
        } else {  // the first and last group hold tokens of other sequences
#pragma unroll
          for (int j = 0; j < kGroup; ++j)
            if (t + j >= lo && t + j < hi) p.dlogp[t + j] = v[j];
        }
      }
      // tokens of no sequence: before the first and after the last
      if (pair == 0)
        for (int64_t t = part * kPairThreads + tid; t < at[0]; t += share * kPairThreads) p.dlogp[t] = 0.0f;
      if (pair == p.P - 1)
        for (int64_t t = at[2] + part * kPairThreads + tid; t < p.T; t += share * kPairThreads) p.dlogp[t] = 0.0f;
    }
  }
  if (arrived) cluster_wait();
  if constexpr (SOLO) {
    if (tid == 0) {
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(ptx::mapa(ptx::smem_u32(&cta_s[0][rank]), 0)), "d"(loss_sum)
                   : "memory");
      ptx::st_shared_cluster_u32(ptx::mapa(ptx::smem_u32(&cta_n[0][rank]), 0), static_cast<uint32_t>(bad_sum));
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank == 0 && tid == 0) {
      double s = 0.0;
      int b = 0;
      for (int r = 0; r < ctas; ++r) s += cta_s[0][r], b += cta_n[0][r];
      if (p.loss && p.reduction != kNone) p.loss[0] = static_cast<float>(p.reduction == kMean ? s / p.P : s);
      *p.status = b ? kStatusSequences : 0;
    }
  }
}

constexpr int kReduceThreads = 256;

__global__ void __launch_bounds__(kReduceThreads) preference_reduce_kernel(const PreferenceParams p) {
  ptx::wait_prerequisites();
  __shared__ double sh[kReduceThreads / 32];
  __shared__ int sh_n[kReduceThreads / 32];
  double s = 0.0;
  int bad = 0;
  for (int i = threadIdx.x; i < p.P; i += kReduceThreads) s += __ldcg(p.pair_loss + i), bad += __ldcg(p.pair_bad + i);
  s = block_sum<double, kReduceThreads>(s, sh);
  bad = block_sum<int, kReduceThreads>(bad, sh_n);
  if (threadIdx.x != 0) return;
  if (p.loss && p.reduction != kNone) p.loss[0] = static_cast<float>(p.reduction == kMean ? s / p.P : s);
  *p.status = bad ? kStatusSequences : 0;
}

}  // namespace loss
}  // namespace flce
