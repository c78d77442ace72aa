// Objectives on per-token log-probabilities: the clipped policy loss with a KL
// term, and the preference loss on paired log ratios.  Each returns its loss and
// the gradient on logp (what flce_backward_logp takes) from one reading of its
// inputs.
//
// Bound: bytes (28 and 20 per token, a few operations each), and below about a
// million tokens latency: launches and the reduction's steps.
//
// Sums: fp32 over the few tokens of one thread, 64 bits across threads and
// blocks, in a fixed order.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

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

// ------------------------------------------------------------------ sequences
// Index s with cu[s] <= t < cu[s + 1] over cu [n + 1], or -1 when t lies in none.
// Any contents of cu give an index in [-1, n - 1].
__device__ __forceinline__ int find_sequence(const int64_t* cu, int n, int64_t t) {
  int lo = 0, hi = n + 1;  // the first index with cu[index] > t lies in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo > n ? -1 : lo - 1;  // lo == 0: before the first sequence; lo == n + 1: after the last
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
  int32_t* seq_count;    // [S] valid tokens of each sequence (SEQUENCE_MEAN)
  int32_t* block_count;  // [blocks]
  double* block_sum;     // [blocks][5]
  int32_t blocks;
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
      // e^e - 1 - e through expm1: exact to rounding also where e is small
      const float ec = clamp_ratio(e), em = expm1f(ec);
      o.kl = em - ec;
      dkl = fabsf(e) > kMaxLogRatio ? 0.0f : -em;
    }
    o.loss = fmaf(p.kl_coef, o.kl, o.loss);
    o.grad = fmaf(p.kl_coef, dkl, o.grad);
  }
  return o;
}

constexpr int kPolicyThreads = 256;
constexpr int kPolicyTokens = 4;  // per thread
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

// A token counts when its target is not ignore_index and, with sequences given,
// it lies in one of them.
__device__ __forceinline__ bool token_valid(const PolicyParams& p, int64_t t, int* seq) {
  *seq = 0;
  if (t >= p.T || p.targets[t] == p.ignore_index) return false;
  if (p.cu) {
    *seq = find_sequence(p.cu, p.S, t);
    if (*seq < 0) return false;
  }
  return true;
}

// Counts: valid tokens of each block, and of each sequence (integers: the order of
// the atomics does not change them).  Also checks cu.
__global__ void __launch_bounds__(kPolicyThreads) policy_count_kernel(const PolicyParams p) {
  __shared__ int sh[kPolicyThreads / 32];
  int n = 0;
  for (int k = 0; k < kPolicyTokens; ++k) {
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kPolicyTokens + k) * kPolicyThreads + threadIdx.x;
    int s;
    if (token_valid(p, t, &s)) {
      ++n;
      if (p.reduction == kSequenceMean) atomicAdd(p.seq_count + s, 1);
    }
  }
  n = block_sum<int, kPolicyThreads>(n, sh);
  if (threadIdx.x == 0) p.block_count[blockIdx.x] = n;
  if (p.cu) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kPolicyThreads;
    bool bad = false;
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * kPolicyThreads + threadIdx.x; s <= p.S; s += stride) {
      const int64_t a = s ? p.cu[s - 1] : 0, b = p.cu[s];
      bad = bad || b < a || b > p.T;
    }
    if (bad) atomicCAS(p.status, 0, kStatusSequences);
  }
}

__global__ void __launch_bounds__(kPolicyThreads) policy_main_kernel(const PolicyParams p) {
  __shared__ double sh[kPolicyThreads / 32];
  __shared__ int sh_i[kPolicyThreads / 32];
  __shared__ float scale;
  // the weight that all tokens share: 1, 1 / n_valid or 1 / (sequences with a valid token)
  int c = 0;
  if (p.reduction == kMean)
    for (int i = threadIdx.x; i < p.blocks; i += kPolicyThreads) c += p.block_count[i];
  if (p.reduction == kSequenceMean)
    for (int i = threadIdx.x; i < p.S; i += kPolicyThreads) c += p.seq_count[i] > 0;
  c = block_sum<int, kPolicyThreads>(c, sh_i);
  if (threadIdx.x == 0) scale = p.reduction == kMean || p.reduction == kSequenceMean ? 1.0f / fmaxf(c, 1.0f) : 1.0f;
  __syncthreads();
  const float up = p.dloss && p.reduction != kNone ? p.dloss[0] : 1.0f;
  float sum[kSums] = {};
  for (int k = 0; k < kPolicyTokens; ++k) {
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kPolicyTokens + k) * kPolicyThreads + threadIdx.x;
    if (t >= p.T) break;
    int s;
    float l = 0.0f, g = 0.0f;
    if (token_valid(p, t, &s)) {
      const PolicyTerm o =
          policy_token(p, p.logp[t], p.old_logp[t], p.ref ? p.ref[t] : 0.0f, p.adv[p.adv_per_seq ? s : t]);
      const float w = p.reduction == kSequenceMean ? scale / p.seq_count[s] : scale;
      l = o.loss;
      g = o.grad * w * (p.reduction == kNone && p.dloss ? p.dloss[t] : up);
      sum[0] += p.reduction == kSequenceMean ? o.loss * w : o.loss;
      sum[1] += o.kl, sum[2] += o.cut, sum[3] += o.d, sum[4] += o.rho;
    }
    if (p.dlogp) p.dlogp[t] = g;
    if (p.loss && p.reduction == kNone) p.loss[t] = l;
  }
  for (int i = 0; i < kSums; ++i) {
    const double s = block_sum<double, kPolicyThreads>(static_cast<double>(sum[i]), sh);
    if (threadIdx.x == 0) p.block_sum[blockIdx.x * kSums + i] = s;
  }
}

__global__ void __launch_bounds__(kPolicyThreads) policy_reduce_kernel(const PolicyParams p) {
  __shared__ double sh[kPolicyThreads / 32];
  __shared__ long long sh_n[kPolicyThreads / 32];
  long long n = 0;
  double sum[kSums] = {};
  for (int b = threadIdx.x; b < p.blocks; b += kPolicyThreads) {
    n += p.block_count[b];
    for (int i = 0; i < kSums; ++i) sum[i] += p.block_sum[b * kSums + i];
  }
  n = block_sum<long long, kPolicyThreads>(n, sh_n);
  for (int i = 0; i < kSums; ++i) sum[i] = block_sum<double, kPolicyThreads>(sum[i], sh);
  if (threadIdx.x != 0) return;
  const double inv = n > 0 ? 1.0 / static_cast<double>(n) : 0.0;
  if (p.loss && p.reduction != kNone) p.loss[0] = static_cast<float>(p.reduction == kMean ? sum[0] * inv : sum[0]);
  if (p.stats)
    for (int i = 1; i < kSums; ++i) p.stats[i - 1] = static_cast<float>(sum[i] * inv);
  if (p.n_valid) *p.n_valid = n;
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

constexpr int kPairThreads = 256;

// One block per pair: the sums of both sequences, the pair's loss, then the
// gradient, which is one number per sequence.
__global__ void __launch_bounds__(kPairThreads) preference_kernel(const PreferenceParams p) {
  __shared__ double sh[kPairThreads / 32];
  __shared__ int sh_n[kPairThreads / 32];
  __shared__ float slope_of[2];
  const int pair = blockIdx.x;
  int64_t at[3];
  bool bad = false;
  for (int i = 0; i < 3; ++i) {
    const int64_t v = p.cu[2 * static_cast<int64_t>(pair) + i];
    at[i] = min(max(v, int64_t(0)), p.T);  // no access outside [0, T) whatever cu holds
    bad = bad || v != at[i];
  }
  bad = bad || at[1] < at[0] || at[2] < at[1];
  double S[2];
  int n[2];
  for (int side = 0; side < 2; ++side) {
    float s = 0.0f;
    int c = 0;
    for (int64_t t = at[side] + threadIdx.x; t < at[side + 1]; t += kPairThreads)
      if (p.targets[t] != p.ignore_index) {
        s += p.ref ? p.logp[t] - p.ref[t] : p.logp[t];
        ++c;
      }
    S[side] = block_sum<double, kPairThreads>(static_cast<double>(s), sh);
    n[side] = block_sum<int, kPairThreads>(c, sh_n);
  }
  if (threadIdx.x == 0) {
    for (int side = 0; side < 2; ++side)
      if (p.normalize) S[side] /= max(n[side], 1);
    float value, slope;
    pair_loss(p, static_cast<float>(S[0] - S[1]), &value, &slope);
    const float up = p.dloss ? p.dloss[p.reduction == kNone ? pair : 0] : 1.0f;
    slope *= p.reduction == kMean ? up / static_cast<float>(p.P) : up;
    slope_of[0] = p.normalize ? slope / max(n[0], 1) : slope;
    slope_of[1] = p.normalize ? -slope / max(n[1], 1) : -slope;
    if (p.chosen) p.chosen[pair] = static_cast<float>(p.beta * S[0]);
    if (p.rejected) p.rejected[pair] = static_cast<float>(p.beta * S[1]);
    if (p.loss && p.reduction == kNone) p.loss[pair] = value;
    p.pair_loss[pair] = value;
    p.pair_bad[pair] = bad;
  }
  __syncthreads();
  if (!p.dlogp) return;
  for (int side = 0; side < 2; ++side)
    for (int64_t t = at[side] + threadIdx.x; t < at[side + 1]; t += kPairThreads)
      p.dlogp[t] = p.targets[t] != p.ignore_index ? slope_of[side] : 0.0f;
  // tokens of no sequence: before the first and after the last
  if (pair == 0)
    for (int64_t t = threadIdx.x; t < at[0]; t += kPairThreads) p.dlogp[t] = 0.0f;
  if (pair == p.P - 1)
    for (int64_t t = at[2] + threadIdx.x; t < p.T; t += kPairThreads) p.dlogp[t] = 0.0f;
}

__global__ void __launch_bounds__(kPairThreads) preference_reduce_kernel(const PreferenceParams p) {
  __shared__ double sh[kPairThreads / 32];
  __shared__ int sh_n[kPairThreads / 32];
  double s = 0.0;
  int bad = 0;
  for (int i = threadIdx.x; i < p.P; i += kPairThreads) s += p.pair_loss[i], bad += p.pair_bad[i];
  s = block_sum<double, kPairThreads>(s, sh);
  bad = block_sum<int, kPairThreads>(bad, sh_n);
  if (threadIdx.x != 0) return;
  if (p.loss && p.reduction != kNone) p.loss[0] = static_cast<float>(p.reduction == kMean ? s / p.P : s);
  *p.status = bad ? kStatusSequences : 0;
}

}  // namespace loss
}  // namespace flce
