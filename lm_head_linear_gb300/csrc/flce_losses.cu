// Host side of the policy and preference losses of include/flce.h.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "flce_host.cuh"
#include "loss_kernels.cuh"

using namespace flce;
using namespace flce::host;

namespace {

constexpr int64_t kClusterTokens = loss::kClusterThreads * loss::kGroup;  // of one CTA

// Header (status, ticket, nonempty) | block_sum | block_count | block_bad | words | seq_count.
// Both forms of the call fit: the larger one is laid out.
constexpr size_t kTicketOff = 16, kNonemptyOff = 32;
struct PolicyLayout {
  int64_t chunk, blocks;  // the counting launch: tokens of a block, blocks (at most kMaxBlocks)
  int64_t ctas;           // the second launch
  size_t sum_off, count_off, bad_off, words_off, seq_off, total;
};
PolicyLayout policy_layout(int64_t T, int64_t S) {
  PolicyLayout L;
  const int64_t steps = std::max<int64_t>(cdiv(T, loss::kStep), 1);
  L.chunk = cdiv(steps, loss::kMaxBlocks) * loss::kStep;
  L.blocks = std::max<int64_t>(cdiv(T, L.chunk), 1);
  L.ctas = std::min<int64_t>(steps, 2 * loss::kMaxBlocks);
  size_t off = kHeaderBytes;
  L.sum_off = off;
  off = align_up(off + sizeof(double) * loss::kSums * L.ctas, 256);
  L.count_off = off;
  off = align_up(off + sizeof(int32_t) * L.blocks, 256);
  L.bad_off = off;
  off = align_up(off + sizeof(int32_t) * L.blocks, 256);
  L.words_off = off;
  off = align_up(off + sizeof(uint2) * static_cast<size_t>(cdiv(std::max<int64_t>(T, 1), 32)), 256);
  L.seq_off = off;
  off = align_up(off + sizeof(int32_t) * std::max<int64_t>(S, 1), 256);
  L.total = off;
  return L;
}

struct PairLayout {
  size_t loss_off, bad_off, total;
};
PairLayout pair_layout(int64_t P) {
  PairLayout L;
  size_t off = kHeaderBytes;
  L.loss_off = off;
  off = align_up(off + sizeof(double) * std::max<int64_t>(P, 1), 256);
  L.bad_off = off;
  off = align_up(off + sizeof(int32_t) * std::max<int64_t>(P, 1), 256);
  L.total = off;
  return L;
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// CTAs of the largest cluster these kernels may use on a device: 16 where the
// device schedules it (queried once), else the portable 8.
flce_status largest_cluster(int dev, int* ctas) {
  static std::mutex mu;
  static int known[64] = {};
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev] == 0) {
    const void* kernels[] = {reinterpret_cast<const void*>(loss::policy_cluster_kernel),
                             reinterpret_cast<const void*>(loss::preference_kernel<true>)};
    int most = loss::kClusterCtas;
    for (const void* k : kernels) {
      CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
      cudaLaunchAttribute at{};
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = loss::kClusterCtas, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(loss::kClusterCtas);
      cfg.blockDim = dim3(loss::kClusterThreads);
      cfg.attrs = &at, cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        most = 8;
      }
    }
    known[dev] = most;
  }
  *ctas = known[dev];
  return FLCE_OK;
}

template <typename P>
flce_status launch_cluster(void (*kernel)(P), const P& p, int64_t grid, int ctas, int threads, cudaStream_t s) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(ctas), at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cfg.attrs = &at, cfg.numAttrs = 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
  return FLCE_OK;
}

int pow2_up(int64_t v, int most) {
  int r = 1;
  while (r < v && r < most) r *= 2;
  return r;
}

flce_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws) return fail(FLCE_ERR_WORKSPACE, "workspace is NULL");
  if (bytes < need) return fail(FLCE_ERR_WORKSPACE, "workspace of %zu bytes < %zu required", bytes, need);
  if (reinterpret_cast<uintptr_t>(ws) & 255) return fail(FLCE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  return FLCE_OK;
}

}  // namespace

extern "C" {

size_t flce_policy_loss_workspace_size(int64_t T, int64_t n_seqs) {
  if (T < 0 || T >= kMaxRows || n_seqs < 0 || n_seqs >= kMaxRows) return 0;
  return policy_layout(T, n_seqs).total;
}

flce_status flce_policy_loss(const float* dloss, const float* logp, const float* old_logp, const float* ref_logp,
                             const float* advantages, int32_t advantages_per_sequence, const int64_t* targets,
                             const int64_t* cu_seqlens, int64_t n_seqs, int64_t T, int64_t ignore_index,
                             int32_t reduction, float clip_low, float clip_high, float dual_clip, float kl_coef,
                             int32_t kl_kind, float* loss, float* dlogp, float* stats, int64_t* n_valid,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || T >= kMaxRows) return fail(FLCE_ERR_INVALID_ARG, "T = %lld out of range", (long long)T);
  if (n_seqs < 0 || n_seqs >= kMaxRows)
    return fail(FLCE_ERR_INVALID_ARG, "n_seqs = %lld out of range", (long long)n_seqs);
  if (reduction < FLCE_REDUCTION_NONE || reduction > FLCE_REDUCTION_SEQUENCE_MEAN)
    return fail(FLCE_ERR_INVALID_ARG, "unknown reduction %d", reduction);
  if (kl_kind < FLCE_KL_K1 || kl_kind > FLCE_KL_K3) return fail(FLCE_ERR_INVALID_ARG, "unknown KL kind %d", kl_kind);
  if (!(clip_low >= 0.0f && clip_low < 1.0f) || !(clip_high >= 0.0f))
    return fail(FLCE_ERR_INVALID_ARG, "clip_low must lie in [0, 1) and clip_high must not be negative");
  if (dual_clip != 0.0f && !(dual_clip > 1.0f)) return fail(FLCE_ERR_INVALID_ARG, "dual_clip is 0 or above 1");
  if (!std::isfinite(kl_coef)) return fail(FLCE_ERR_INVALID_ARG, "kl_coef must be finite");
  if (!ref_logp && kl_coef != 0.0f) return fail(FLCE_ERR_INVALID_ARG, "kl_coef without ref_logp");
  if ((reduction == FLCE_REDUCTION_SEQUENCE_MEAN || advantages_per_sequence) && !cu_seqlens)
    return fail(FLCE_ERR_INVALID_ARG, "sequences are needed, and cu_seqlens is NULL");
  if (!loss && !dlogp && T > 0) return fail(FLCE_ERR_INVALID_ARG, "neither loss nor dlogp is given");
  if (T > 0 && (!logp || !old_logp || !targets || (!advantages && (!advantages_per_sequence || n_seqs > 0))))
    return fail(FLCE_ERR_INVALID_ARG, "logp, old_logp, advantages or targets is NULL");
  if (misaligned(dloss) || misaligned(logp) || misaligned(old_logp) || misaligned(ref_logp) || misaligned(advantages) ||
      misaligned(targets) || misaligned(cu_seqlens) || misaligned(loss) || misaligned(dlogp) || misaligned(stats) ||
      misaligned(n_valid))
    return fail(FLCE_ERR_ALIGNMENT, "a float array is not 4-byte or an int64 array not 8-byte aligned");
  flce_status st;
  const PolicyLayout L = policy_layout(T, n_seqs);
  if ((st = check_workspace(workspace, workspace_bytes, L.total)) != FLCE_OK) return st;
  int dev = 0, sms = 0;
  if ((st = current_device(&dev, &sms)) != FLCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  loss::PolicyParams p{};
  p.dloss = dloss, p.logp = logp, p.old_logp = old_logp, p.ref = ref_logp, p.adv = advantages;
  p.targets = targets, p.cu = cu_seqlens, p.loss = loss, p.dlogp = dlogp, p.stats = stats, p.n_valid = n_valid;
  p.ignore_index = ignore_index, p.T = static_cast<int32_t>(T), p.S = cu_seqlens ? static_cast<int32_t>(n_seqs) : 0;
  p.adv_per_seq = advantages_per_sequence != 0, p.reduction = reduction, p.kl_kind = kl_kind;
  p.log_hi = static_cast<float>(std::log1p(static_cast<double>(clip_high)));
  p.log_lo = static_cast<float>(std::log1p(-static_cast<double>(clip_low)));
  p.ratio_hi = 1.0f + clip_high, p.ratio_lo = 1.0f - clip_low;
  p.log_dual = dual_clip != 0.0f ? static_cast<float>(std::log(static_cast<double>(dual_clip))) : INFINITY;
  p.dual = dual_clip, p.kl_coef = kl_coef;
  p.status = reinterpret_cast<int32_t*>(ws);
  p.block_sum = reinterpret_cast<double*>(ws + L.sum_off);
  p.block_count = reinterpret_cast<int32_t*>(ws + L.count_off);
  p.block_bad = reinterpret_cast<int32_t*>(ws + L.bad_off);
  p.words = reinterpret_cast<uint2*>(ws + L.words_off);
  p.seq_count = reinterpret_cast<int32_t*>(ws + L.seq_off);
  p.ticket = reinterpret_cast<int32_t*>(ws + kTicketOff);
  p.nonempty = reinterpret_cast<int32_t*>(ws + kNonemptyOff);
  p.vec = !(off16(logp) || off16(old_logp) || off16(ref_logp) || (!advantages_per_sequence && off16(advantages)) ||
            off16(targets) || off16(dlogp) ||
            (reduction == FLCE_REDUCTION_NONE && (off16(loss) || off16(dloss))));
  int most = 0;
  if ((st = largest_cluster(dev, &most)) != FLCE_OK) return st;
  KernelScope ks(FLCE_KERNEL_POLICY_LOSS, s, 20.0 * T, T * (12.0 + (ref_logp ? 4.0 : 0.0) + 8.0 + (dlogp ? 4.0 : 0.0)));
  if (T <= most * kClusterTokens) {
    p.blocks = pow2_up(cdiv(T, kClusterTokens), most);
    st = launch_cluster(loss::policy_cluster_kernel, p, p.blocks, p.blocks, loss::kClusterThreads, s);
  } else {
    p.blocks = static_cast<int32_t>(L.blocks), p.chunk = static_cast<int32_t>(L.chunk);
    // an ordinary launch: policy_main_kernel reads its inputs before its wait
    loss::policy_count_kernel<<<p.blocks, loss::kManyThreads, 0, s>>>(p);
    if (reduction == FLCE_REDUCTION_SEQUENCE_MEAN && n_seqs >= loss::kCuShared)
      loss::policy_nonempty_kernel<<<static_cast<unsigned>(std::min<int64_t>(cdiv(n_seqs, loss::kManyThreads), sms)),
                                     loss::kManyThreads, 0, s>>>(p);
    st = launch_overlapped(loss::policy_main_kernel, dim3(static_cast<unsigned>(L.ctas)), loss::kManyThreads, 0, s, p);
  }
  if (st != FLCE_OK) return st;
  ks.done();
  return check_launch("policy_loss");
}

size_t flce_preference_loss_workspace_size(int64_t n_pairs) {
  if (n_pairs < 0 || n_pairs >= kMaxRows / 2) return 0;
  return pair_layout(n_pairs).total;
}

flce_status flce_preference_loss(const float* dloss, const float* logp, const float* ref_logp, const int64_t* targets,
                                 const int64_t* cu_seqlens, int64_t n_pairs, int64_t T, int64_t ignore_index,
                                 int32_t reduction, int32_t kind, float beta, float label_smoothing, float margin,
                                 int32_t length_normalize, float* loss, float* dlogp, float* chosen_rewards,
                                 float* rejected_rewards, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || T >= kMaxRows) return fail(FLCE_ERR_INVALID_ARG, "T = %lld out of range", (long long)T);
  if (n_pairs < 0 || n_pairs >= kMaxRows / 2)
    return fail(FLCE_ERR_INVALID_ARG, "n_pairs = %lld out of range", (long long)n_pairs);
  if (reduction < FLCE_REDUCTION_NONE || reduction > FLCE_REDUCTION_SUM)
    return fail(FLCE_ERR_INVALID_ARG, "unknown reduction %d", reduction);
  if (kind < FLCE_PREFERENCE_SIGMOID || kind > FLCE_PREFERENCE_IPO)
    return fail(FLCE_ERR_INVALID_ARG, "unknown preference loss %d", kind);
  if (!(beta > 0.0f) || !std::isfinite(beta)) return fail(FLCE_ERR_INVALID_ARG, "beta must be positive and finite");
  if (!(label_smoothing >= 0.0f && label_smoothing < 0.5f))
    return fail(FLCE_ERR_INVALID_ARG, "label_smoothing must lie in [0, 0.5)");
  if (!std::isfinite(margin)) return fail(FLCE_ERR_INVALID_ARG, "margin must be finite");
  if ((label_smoothing != 0.0f && kind != FLCE_PREFERENCE_SIGMOID) || (margin != 0.0f && kind == FLCE_PREFERENCE_IPO))
    return fail(FLCE_ERR_INVALID_ARG, "label_smoothing is the sigmoid loss's, margin the sigmoid and hinge losses'");
  if (!loss && !dlogp && (T > 0 || n_pairs > 0))
    return fail(FLCE_ERR_INVALID_ARG, "neither loss nor dlogp is given");
  if (n_pairs > 0 && !cu_seqlens) return fail(FLCE_ERR_INVALID_ARG, "cu_seqlens is NULL");
  if (T > 0 && (!logp || !targets)) return fail(FLCE_ERR_INVALID_ARG, "logp or targets is NULL");
  if (misaligned(dloss) || misaligned(logp) || misaligned(ref_logp) || misaligned(targets) || misaligned(cu_seqlens) ||
      misaligned(loss) || misaligned(dlogp) || misaligned(chosen_rewards) || misaligned(rejected_rewards))
    return fail(FLCE_ERR_ALIGNMENT, "a float array is not 4-byte or an int64 array not 8-byte aligned");
  flce_status st;
  const PairLayout L = pair_layout(n_pairs);
  if ((st = check_workspace(workspace, workspace_bytes, L.total)) != FLCE_OK) return st;
  int dev = 0, sms = 0;
  if ((st = current_device(&dev, &sms)) != FLCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (n_pairs == 0) {
    CUDA_TRY(cudaMemsetAsync(ws, 0, kHeaderBytes, s));
    if (loss && reduction != FLCE_REDUCTION_NONE) CUDA_TRY(cudaMemsetAsync(loss, 0, sizeof(float), s));
    if (dlogp && T > 0) CUDA_TRY(cudaMemsetAsync(dlogp, 0, sizeof(float) * T, s));
    return FLCE_OK;
  }
  loss::PreferenceParams p{};
  p.dloss = dloss, p.logp = logp, p.ref = ref_logp, p.targets = targets, p.cu = cu_seqlens;
  p.loss = loss, p.dlogp = dlogp, p.chosen = chosen_rewards, p.rejected = rejected_rewards;
  p.ignore_index = ignore_index, p.T = T, p.P = static_cast<int32_t>(n_pairs);
  p.reduction = reduction, p.kind = kind, p.normalize = length_normalize != 0;
  p.beta = beta, p.smoothing = label_smoothing, p.margin = margin;
  p.inv_2beta = static_cast<float>(0.5 / static_cast<double>(beta));
  p.status = reinterpret_cast<int32_t*>(ws);
  p.pair_loss = reinterpret_cast<double*>(ws + L.loss_off);
  p.pair_bad = reinterpret_cast<int32_t*>(ws + L.bad_off);
  KernelScope ks(FLCE_KERNEL_PREFERENCE_LOSS, s, 4.0 * T, T * (12.0 + (ref_logp ? 4.0 : 0.0) + (dlogp ? 4.0 : 0.0)));
  p.vec = !(off16(logp) || off16(ref_logp) || off16(targets) || off16(dlogp));
  int most = 0;
  if ((st = largest_cluster(dev, &most)) != FLCE_OK) return st;
  const int64_t mean = cdiv(T, n_pairs);
  // One cluster while every CTA has at most one pair (a second one costs another 2 us:
  // 17 pairs of 2 x 329 tokens 8.3 us, in two launches 5.7); else a cluster per pair, with
  // enough CTAs to fill the device, of at least 2048 tokens each.
  if (n_pairs <= most && mean <= 8192) {
    p.ctas = pow2_up(n_pairs, most);
    st = launch_cluster(loss::preference_kernel<true>, p, p.ctas, p.ctas, loss::kPairThreads, s);
  } else {
    p.ctas = pow2_up(std::min<int64_t>(mean / 2048, 2 * sms / n_pairs), 8);
    st = launch_cluster(loss::preference_kernel<false>, p, n_pairs * p.ctas, p.ctas, loss::kPairThreads, s);
    if (st == FLCE_OK) st = launch_overlapped(loss::preference_reduce_kernel, dim3(1), loss::kReduceThreads, 0, s, p);
  }
  if (st != FLCE_OK) return st;
  ks.done();
  return check_launch("preference_loss");
}

}  // extern "C"
