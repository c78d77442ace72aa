// Host side of flce_sample of include/flce.h.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "flce_host.cuh"
#include "sample_kernels.cuh"

using namespace flce;
using namespace flce::host;

namespace {

constexpr int64_t kMaxVocab = 393216;      // an index has 19 bits, a sum of weights 63
constexpr int64_t kChunkBytes = 65024;     // of a row on a CTA, where a cluster can be larger: two CTAs on an SM
constexpr int kMaxSmem = 232448 - 4096;    // less the static part

// The largest cluster of this kernel: 16 CTAs where the device schedules it (queried once), else 8.
template <typename E, bool SEARCH>
flce_status set_up(int dev, int* most) {
  static std::mutex mu;
  static int known[64] = {};
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev] == 0) {
    const void* k = reinterpret_cast<const void*>(sample::sample_kernel<E, SEARCH>);
    CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem));
    CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = sample::kMaxCtas, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sample::kMaxCtas);
    cfg.blockDim = dim3(sample::kMaxThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cfg.attrs = &at, cfg.numAttrs = 1;
    int n = 0;
    const bool fits = cudaOccupancyMaxActiveClusters(&n, k, &cfg) == cudaSuccess && n >= 1;
    if (!fits) (void)cudaGetLastError();
    known[dev] = fits ? sample::kMaxCtas : 8;
  }
  *most = known[dev];
  return FLCE_OK;
}

// CTAs of a row, pieces of 16 bytes on each, and threads.
template <typename E, bool SEARCH>
flce_status launch(sample::Params& p, int64_t T, int dev, int sms, cudaStream_t s) {
  int most = 8;
  flce_status st = set_up<E, SEARCH>(dev, &most);
  if (st != FLCE_OK) return st;
  constexpr int64_t kPer = 16 / sizeof(E);
  const int64_t pieces = cdiv(p.V + kPer - 1, kPer);  // a row that starts on the last element of a piece
  int ctas = 1;
  while (ctas < 8 && cdiv(pieces, ctas) * 16 > kChunkBytes) ctas *= 2;
  while (ctas < most && T * ctas * 2 <= sms && cdiv(pieces, ctas) > 256) ctas *= 2;
  while (ctas < most && sample::shared_bytes(static_cast<int>(cdiv(pieces, ctas)), SEARCH) > kMaxSmem) ctas *= 2;
  if (sample::shared_bytes(static_cast<int>(cdiv(pieces, ctas)), SEARCH) > kMaxSmem)
    return fail(FLCE_ERR_UNSUPPORTED, "V = %d does not fit into a cluster of %d CTAs on this device", p.V, ctas);
  p.ctas = ctas;
  p.unit = sample::kMostUnit;
  while ((static_cast<int64_t>(p.V) >> (63 - p.unit)) != 0) --p.unit;
  p.chunk = static_cast<int32_t>(cdiv(pieces, ctas));
  const int threads = static_cast<int>(std::min<int64_t>(sample::kMaxThreads, std::max<int64_t>(128, cdiv(p.chunk, 256) * 128)));
  const size_t smem = sample::shared_bytes(p.chunk, SEARCH);
  if (T * ctas >= (int64_t(1) << 31)) return fail(FLCE_ERR_INVALID_ARG, "T = %lld is too large", (long long)T);
  int pow2 = 128;
  while (pow2 < threads) pow2 *= 2;  // a whole share of the bins for each thread
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(ctas), at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T * ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(pow2));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at, cfg.numAttrs = 2;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, sample::sample_kernel<E, SEARCH>, p));
  return FLCE_OK;
}

bool within(double v, double lo, double hi) { return v >= lo && v <= hi; }

}  // namespace

extern "C" {

flce_status flce_sample(const void* logits, int32_t dtype, int64_t ldl, const float* u, int64_t T, int64_t V,
                        const float* temperature, double temperature_all, const int32_t* top_k, int64_t top_k_all,
                        const float* top_p, double top_p_all, const float* min_p, double min_p_all, int64_t ignore_index,
                        int64_t* tokens, float* logp, void* stream) {
  if (T < 0 || T >= kMaxRows) return fail(FLCE_ERR_INVALID_ARG, "T = %lld out of range", (long long)T);
  if (V < 1) return fail(FLCE_ERR_INVALID_ARG, "V = %lld out of range", (long long)V);
  if (V > kMaxVocab) return fail(FLCE_ERR_UNSUPPORTED, "V = %lld is above %lld", (long long)V, (long long)kMaxVocab);
  if (dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) return fail(FLCE_ERR_INVALID_ARG, "unknown element type");
  if (ldl < V) return fail(FLCE_ERR_INVALID_ARG, "ldl is smaller than V");
  if (ignore_index >= 0 && ignore_index < V) return fail(FLCE_ERR_INVALID_ARG, "ignore_index must lie outside [0, V)");
  if (!temperature && !within(temperature_all, 0.0, 1e300))
    return fail(FLCE_ERR_INVALID_ARG, "temperature must not be negative");
  if (!top_p && !within(top_p_all, 0.0, 1.0)) return fail(FLCE_ERR_INVALID_ARG, "top_p must lie in [0, 1]");
  if (!min_p && !within(min_p_all, 0.0, 1.0)) return fail(FLCE_ERR_INVALID_ARG, "min_p must lie in [0, 1]");
  if (T > 0 && (!logits || !u || !tokens)) return fail(FLCE_ERR_INVALID_ARG, "logits, u or tokens is NULL");
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == FLCE_DTYPE_F32 ? 4 : 2) || misaligned(u) || misaligned(temperature) ||
      misaligned(top_k) || misaligned(top_p) || misaligned(min_p) || misaligned(tokens) || misaligned(logp))
    return fail(FLCE_ERR_ALIGNMENT, "an array is not aligned to its element type");
  int dev = 0, sms = 0;
  flce_status st = current_device(&dev, &sms);
  if (st != FLCE_OK) return st;
  if (T == 0) return FLCE_OK;
  sample::Params p{};
  p.logits = logits, p.u = u, p.temperature = temperature, p.top_k = top_k, p.top_p = top_p, p.min_p = min_p;
  p.temperature_all = temperature_all, p.top_k_all = top_k_all, p.top_p_all = top_p_all;
  p.log_min_p_all = min_p_all > 0.0 ? std::log(min_p_all) : 0.0;
  const double c = temperature_all > 0.0 ? std::min(1.4426950408889634 / temperature_all, 1e37) : 1.0;
  p.c_hi_all = static_cast<float>(c);
  p.c_lo_all = static_cast<float>(c - static_cast<double>(p.c_hi_all));
  p.temperature_like = temperature_all > 0.0 ? 1.0f : 0.0f;
  p.top_p_like = top_p_all <= 0.0 ? 0.0f : top_p_all < 1.0 ? 0.5f : 1.0f;
  p.min_p_like = min_p_all > 0.0 ? 0.5f : 0.0f;
  p.ldl = ldl, p.ignore_index = ignore_index, p.tokens = tokens, p.logp = logp, p.V = static_cast<int32_t>(V);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KernelScope ks(FLCE_KERNEL_SAMPLE, s, 4.0 * T * V, T * (V * (dtype == FLCE_DTYPE_F32 ? 4.0 : 2.0) + 16.0));
  if (top_k || top_k_all > 0 || top_p || top_p_all < 1.0)
    st = dtype == FLCE_DTYPE_F32 ? launch<float, true>(p, T, dev, sms, s) : launch<uint16_t, true>(p, T, dev, sms, s);
  else
    st = dtype == FLCE_DTYPE_F32 ? launch<float, false>(p, T, dev, sms, s) : launch<uint16_t, false>(p, T, dev, sms, s);
  if (st != FLCE_OK) return st;
  ks.done();
  return check_launch("sample");
}

}  // extern "C"
