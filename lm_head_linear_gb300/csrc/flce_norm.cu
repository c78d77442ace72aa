// Host side of the residual add + RMS norm entry points of include/flce.h.
#include <algorithm>
#include <mutex>

#include "flce_host.cuh"
#include "norm_kernels.cuh"

using namespace flce;
using namespace flce::host;

namespace {

constexpr int64_t kMaxNormHd = 16384;   // a row stays in the registers of one CTA
constexpr int64_t kMaxNormBlocks = 512; // CTAs of the backward: rows of its workspace

bool known_dtype(int32_t d) { return d == FLCE_DTYPE_BF16 || d == FLCE_DTYPE_F32; }
int64_t size_of(int32_t d) { return d == FLCE_DTYPE_F32 ? 4 : 2; }
bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
bool bad_ld(int64_t ld, int64_t Hd, int32_t dtype) { return ld < Hd || (ld * size_of(dtype)) % 16 != 0; }

// Vectors of 8 channels per thread and threads per row.  Up to a row per SM: one vector
// per thread, the shortest chain from load to store.  More rows: two (1531 x 4112 from
// fp32: 14.6 us, 18.4 us as one run of two), and from 16 rows per SM on four in runs of
// two, which needs fewer warps for a row, has more loads of a warp in flight and half the
// scales to work out (65,536 x 2048 to 8 bits: 141 us against 146 us with four runs of
// one, both with a slower rounding; 138 us now).
struct Shape {
  int vecs, group, threads;
};
Shape pick_shape(int64_t T, int64_t Hd, int sms) {
  const int nvec = static_cast<int>(Hd / kVec);
  int vecs = T <= sms ? 1 : T <= 16 * sms ? 2 : 4;
  while (cdiv(cdiv(nvec, vecs), 32) * 32 > norm::max_threads(vecs)) vecs *= 2;
  while (vecs > 1 && (vecs / 2) * 32 >= nvec) vecs /= 2;  // a warp would leave whole steps idle
  Shape s;
  s.vecs = vecs;
  s.group = static_cast<int>(cdiv(cdiv(nvec, vecs), 32) * 32);
  s.threads = T > sms ? std::max(s.group, 128 / s.group * s.group) : s.group;
  return s;
}
template <typename TX, typename TR, bool EXACT>
flce_status launch_fwd(const norm::FwdParams& p, const Shape& s, cudaStream_t st) {
  const int rows = s.threads / s.group;
  const dim3 grid(static_cast<unsigned>(cdiv(p.T, rows))), block(s.group, rows);
  if (s.vecs == 1) return launch_overlapped(norm::add_rms_norm_kernel<TX, TR, 1, 1, EXACT>, grid, block, 0, st, p);
  if (s.vecs == 2) return launch_overlapped(norm::add_rms_norm_kernel<TX, TR, 2, 1, EXACT>, grid, block, 0, st, p);
  return launch_overlapped(norm::add_rms_norm_kernel<TX, TR, 2, 2, EXACT>, grid, block, 0, st, p);
}

// The backward: four vectors per thread (two or one where they cover a row), and as many
// groups as fit 512 threads and an SM's shared memory with a stage each beside the weights,
// but no more than spread the rows over the SMs; and the stages that then fit.  bf16
// weights always leave room for a stage: 14 bytes a channel, 16384 channels, 224 KB.  fp32
// weights next to fp32 rows of dy, h and dh of more than 14336 channels do not.
constexpr int64_t kBwdSmem = 224 * 1024;
struct BwdShape {
  int nv, group, threads, stages;
  bool w_shared;
  size_t smem;
};
BwdShape pick_bwd_shape(int64_t T, int64_t Hd, int64_t row_bytes, bool w_f32, int sms) {
  const int64_t nvec = Hd / kVec;
  BwdShape s;
  s.nv = 4;
  while (s.nv > 1 && (s.nv / 2) * 32 >= nvec) s.nv /= 2;
  s.group = static_cast<int>(cdiv(cdiv(nvec, s.nv), 32) * 32);
  int64_t w_bytes = Hd * (w_f32 ? 4 : 2);
  s.w_shared = row_bytes + w_bytes <= kBwdSmem;
  if (!s.w_shared) w_bytes = 0;
  const int64_t room = kBwdSmem - w_bytes;
  int64_t groups = std::min<int64_t>(norm::kBwdThreads / s.group, room / row_bytes);
  groups = std::max<int64_t>(std::min<int64_t>(groups, cdiv(T, sms)), 1);
  s.threads = static_cast<int>(groups) * s.group;
  const int64_t per_stage = groups * row_bytes;
  s.stages = static_cast<int>(std::min<int64_t>(room / per_stage, norm::kBwdMaxStages));
  s.smem = std::max<size_t>(s.stages * per_stage + w_bytes, groups > 1 ? sizeof(float) * groups * Hd : 0);
  return s;
}

template <typename TY, typename TH, int NV, bool W32>
flce_status launch_bwd(const norm::BwdParams& p, const BwdShape& s, int64_t blocks, cudaStream_t st) {
  static std::mutex mu;
  static bool set[64] = {};
  int dev = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  {
    std::lock_guard<std::mutex> lk(mu);
    if (dev >= 0 && dev < 64 && !set[dev]) {
      CUDA_TRY(cudaFuncSetAttribute(norm::norm_backward_kernel<TY, TH, NV, W32>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdSmem));
      set[dev] = true;
    }
  }
  return launch_overlapped(norm::norm_backward_kernel<TY, TH, NV, W32>, dim3(static_cast<unsigned>(blocks)),
                           s.threads, s.smem, st, p);
}

template <typename TY, typename TH, bool W32>
flce_status launch_bwd_nv(const norm::BwdParams& p, const BwdShape& s, int64_t blocks, cudaStream_t st) {
  if (s.nv == 1) return launch_bwd<TY, TH, 1, W32>(p, s, blocks, st);
  if (s.nv == 2) return launch_bwd<TY, TH, 2, W32>(p, s, blocks, st);
  return launch_bwd<TY, TH, 4, W32>(p, s, blocks, st);
}

template <typename TY, typename TH>
flce_status launch_bwd_types(const norm::BwdParams& p, const BwdShape& s, int64_t blocks, bool w_f32, cudaStream_t st) {
  return w_f32 ? launch_bwd_nv<TY, TH, true>(p, s, blocks, st) : launch_bwd_nv<TY, TH, false>(p, s, blocks, st);
}

flce_status check_sizes(int64_t T, int64_t Hd) {
  if (T < 0 || T >= kMaxRows) return fail(FLCE_ERR_INVALID_ARG, "T = %lld out of range", (long long)T);
  if (Hd < 1) return fail(FLCE_ERR_INVALID_ARG, "Hd = %lld out of range", (long long)Hd);
  if (Hd % 16 != 0 || Hd > kMaxNormHd)
    return fail(FLCE_ERR_UNSUPPORTED, "Hd = %lld is not a multiple of 16 up to %lld", (long long)Hd,
                (long long)kMaxNormHd);
  return FLCE_OK;
}

}  // namespace

extern "C" {

flce_status flce_add_rms_norm(const void* x, int32_t x_dtype, int64_t ldx, const void* residual,
                              int32_t residual_dtype, int64_t ldr, const void* weight, int32_t weight_dtype,
                              int64_t T, int64_t Hd, float eps, void* h, int64_t ldh, void* y, float* rstd, void* q,
                              uint8_t* q_scale, void* stream) {
  flce_status st = check_sizes(T, Hd);
  if (st != FLCE_OK) return st;
  if (!known_dtype(x_dtype) || !known_dtype(weight_dtype) || (residual && !known_dtype(residual_dtype)))
    return fail(FLCE_ERR_INVALID_ARG, "unknown element type");
  if (!(eps >= 0.0f)) return fail(FLCE_ERR_INVALID_ARG, "eps must not be negative");
  if (!weight || (T > 0 && !x)) return fail(FLCE_ERR_INVALID_ARG, "x or weight is NULL");
  if ((residual != nullptr) != (h != nullptr) && T > 0)
    return fail(FLCE_ERR_INVALID_ARG, "residual and h are given together or not at all");
  if ((q != nullptr) != (q_scale != nullptr)) return fail(FLCE_ERR_INVALID_ARG, "q and q_scale are given together");
  if (T > 0 && !y && !q) return fail(FLCE_ERR_INVALID_ARG, "neither y nor q is given");
  if (bad_ld(ldx, Hd, x_dtype) || (residual && (bad_ld(ldr, Hd, residual_dtype) || bad_ld(ldh, Hd, residual_dtype))))
    return fail(FLCE_ERR_ALIGNMENT, "row strides must be at least Hd and whole multiples of 16 bytes");
  if (off16(x) || off16(residual) || off16(weight) || off16(h) || off16(y) || off16(q))
    return fail(FLCE_ERR_ALIGNMENT, "x, residual, weight, h, y and q must be 16-byte aligned");
  if (misaligned(rstd)) return fail(FLCE_ERR_ALIGNMENT, "rstd must be 4-byte aligned");
  int dev = 0, sms = 0;
  if ((st = current_device(&dev, &sms)) != FLCE_OK) return st;
  if (T == 0) return FLCE_OK;
  norm::FwdParams p{};
  p.x = x, p.r = residual, p.w = weight, p.h = h;
  p.y = static_cast<uint16_t*>(y), p.rstd = rstd, p.q = static_cast<uint8_t*>(q), p.qs = q_scale;
  p.ldx = ldx, p.ldr = ldr, p.ldh = ldh, p.T = T, p.Hd = static_cast<int32_t>(Hd);
  p.w_f32 = weight_dtype == FLCE_DTYPE_F32, p.eps = eps;
  p.inv_hd = static_cast<float>(1.0 / static_cast<double>(Hd));
  p.inv_hd_lo = static_cast<float>(1.0 / static_cast<double>(Hd) - static_cast<double>(p.inv_hd));
  const Shape s = pick_shape(T, Hd, sms);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const double n = static_cast<double>(T) * Hd;
  KernelScope ks(FLCE_KERNEL_ADD_RMS_NORM, cs, 8.0 * n,
                 n * (size_of(x_dtype) + (residual ? 2.0 * size_of(residual_dtype) : 0.0) + (y ? 2.0 : 0.0) +
                      (q ? 1.0 + 1.0 / 128 : 0.0)));
  const bool xf = x_dtype == FLCE_DTYPE_F32, rf = residual ? residual_dtype == FLCE_DTYPE_F32 : xf;
  if (rf)  // h in fp32
    st = xf ? launch_fwd<float, float, false>(p, s, cs) : launch_fwd<uint16_t, float, false>(p, s, cs);
  else if (p.w_f32)
    st = xf ? launch_fwd<float, uint16_t, false>(p, s, cs) : launch_fwd<uint16_t, uint16_t, false>(p, s, cs);
  else
    st = xf ? launch_fwd<float, uint16_t, true>(p, s, cs) : launch_fwd<uint16_t, uint16_t, true>(p, s, cs);
  if (st != FLCE_OK) return st;
  ks.done();
  return check_launch("add_rms_norm");
}

size_t flce_add_rms_norm_backward_workspace_size(int64_t T, int64_t Hd) {
  if (T < 0 || Hd < 1) return 0;
  return kHeaderBytes + sizeof(float) * static_cast<size_t>(std::min<int64_t>(std::max<int64_t>(T, 1), kMaxNormBlocks)) *
                            static_cast<size_t>(Hd);
}

flce_status flce_add_rms_norm_backward(const void* dy, int32_t dy_dtype, int64_t lddy, const void* h, int32_t h_dtype,
                                       int64_t ldh, const void* weight, int32_t weight_dtype, const float* rstd,
                                       const void* dh, int64_t lddh, int64_t T, int64_t Hd, void* dx, float* dweight,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  flce_status st = check_sizes(T, Hd);
  if (st != FLCE_OK) return st;
  if (!known_dtype(dy_dtype) || !known_dtype(h_dtype) || !known_dtype(weight_dtype))
    return fail(FLCE_ERR_INVALID_ARG, "unknown element type");
  if (!weight || !dweight || (T > 0 && (!dy || !h || !rstd || !dx)))
    return fail(FLCE_ERR_INVALID_ARG, "dy, h, weight, rstd, dx or dweight is NULL");
  if (bad_ld(lddy, Hd, dy_dtype) || bad_ld(ldh, Hd, h_dtype) || (dh && bad_ld(lddh, Hd, h_dtype)))
    return fail(FLCE_ERR_ALIGNMENT, "row strides must be at least Hd and whole multiples of 16 bytes");
  if (off16(dy) || off16(h) || off16(weight) || off16(dh) || off16(dx))
    return fail(FLCE_ERR_ALIGNMENT, "dy, h, weight, dh and dx must be 16-byte aligned");
  if (misaligned(rstd) || misaligned(dweight)) return fail(FLCE_ERR_ALIGNMENT, "rstd and dweight must be 4-byte aligned");
  if (!workspace) return fail(FLCE_ERR_WORKSPACE, "workspace is NULL");
  if (workspace_bytes < flce_add_rms_norm_backward_workspace_size(T, Hd))
    return fail(FLCE_ERR_WORKSPACE, "workspace of %zu bytes < %zu required", workspace_bytes,
                flce_add_rms_norm_backward_workspace_size(T, Hd));
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(FLCE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  int dev = 0, sms = 0;
  if ((st = current_device(&dev, &sms)) != FLCE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    CUDA_TRY(cudaMemsetAsync(workspace, 0, kHeaderBytes, cs));
    CUDA_TRY(cudaMemsetAsync(dweight, 0, sizeof(float) * Hd, cs));
    return FLCE_OK;
  }
  norm::BwdParams p{};
  p.dy = dy, p.h = h, p.w = weight, p.rstd = rstd, p.dh = dh, p.dx = dx;
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
  p.lddy = lddy, p.ldh = ldh, p.lddh = lddh, p.T = T, p.Hd = static_cast<int32_t>(Hd);
  p.inv_hd = 1.0f / static_cast<float>(Hd);
  p.status = static_cast<int32_t*>(workspace);
  p.timeout_ns = wait_limit_ns(0);
  const BwdShape s = pick_bwd_shape(T, Hd, Hd * (size_of(dy_dtype) + (dh ? 2 : 1) * size_of(h_dtype)),
                                    weight_dtype == FLCE_DTYPE_F32, sms);
  p.group = s.group, p.stages = s.stages, p.w_shared = s.w_shared;
  const int64_t blocks = std::min<int64_t>(std::min<int64_t>(cdiv(T, s.threads / s.group), sms), kMaxNormBlocks);
  const double n = static_cast<double>(T) * Hd;
  {
    KernelScope ks(FLCE_KERNEL_NORM_BWD, cs, 10.0 * n,
                   n * (size_of(dy_dtype) + (dh ? 3.0 : 2.0) * size_of(h_dtype)) + 4.0 * Hd);
    const bool yf = dy_dtype == FLCE_DTYPE_F32, hf = h_dtype == FLCE_DTYPE_F32, wf = weight_dtype == FLCE_DTYPE_F32;
    st = yf && hf ? launch_bwd_types<float, float>(p, s, blocks, wf, cs)
         : yf     ? launch_bwd_types<float, uint16_t>(p, s, blocks, wf, cs)
         : hf     ? launch_bwd_types<uint16_t, float>(p, s, blocks, wf, cs)
                  : launch_bwd_types<uint16_t, uint16_t>(p, s, blocks, wf, cs);
    if (st != FLCE_OK) return st;
    ks.done();
    if ((st = check_launch("norm_bwd")) != FLCE_OK) return st;
  }
  KernelScope ks(FLCE_KERNEL_NORM_DW, cs, 0.0, 4.0 * blocks * Hd + 4.0 * Hd);
  st = launch_overlapped(norm::norm_dw_kernel, dim3(static_cast<unsigned>(cdiv(Hd, 32))), 32 * norm::kDwSlices, 0, cs,
                         static_cast<const float*>(p.partial), static_cast<int>(blocks), p.Hd, dweight);
  if (st != FLCE_OK) return st;
  ks.done();
  return check_launch("norm_dw");
}

}  // extern "C"
