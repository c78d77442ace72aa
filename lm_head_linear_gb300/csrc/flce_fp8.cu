// Host side of the 8-bit entry points of include/flce.h.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "flce_host.cuh"
#include "fp8_kernels.cuh"

using namespace flce;
using namespace flce::host;

namespace {

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// A row-major matrix of `rows` x `inner` elements, rows `pitch` bytes apart; out of
// range reads as zero, stores are clipped.
flce_status matrix_map(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* ptr,
                       int64_t inner, int64_t rows, int64_t pitch, int box_inner, int box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t step[2] = {1, 1};
  CUresult r = g_encode(m, type, 2, const_cast<void*>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(FLCE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for {%lld, %lld} pitch %lld box {%d, %d}",
                static_cast<int>(r), (long long)inner, (long long)rows, (long long)pitch, box_inner, box_rows);
  return FLCE_OK;
}

// Co-resident CTA pairs per device, queried once.
template <bool TOKENS_M>
flce_status resident_pairs(int dev, int sms, int* pairs) {
  static std::mutex mu;
  static int known[64] = {};
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev] == 0) {
    CUDA_TRY(cudaFuncSetAttribute(fp8::linear_fp8_kernel<TOKENS_M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  fp8::kSmemLimit));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * std::max(sms / 2, 1));
    cfg.blockDim = dim3(fp8::kThreads);
    cfg.dynamicSmemBytes = fp8::kSmemLimit;
    int n = 0;
    CUDA_TRY(cudaOccupancyMaxActiveClusters(&n, fp8::linear_fp8_kernel<TOKENS_M>, &cfg));
    known[dev] = std::max(1, std::min(n, sms / 2));
  }
  *pairs = known[dev];
  return FLCE_OK;
}

}  // namespace

extern "C" {

flce_status flce_quantize_fp8(const void* a, int32_t a_dtype, int64_t lda, int64_t rows, int64_t K, int32_t block_rows,
                              void* q, uint8_t* q_scale, void* stream) {
  if (rows < 0 || rows >= kMaxRows) return fail(FLCE_ERR_INVALID_ARG, "rows = %lld out of range", (long long)rows);
  if (K < 1 || K >= (int64_t(1) << 24)) return fail(FLCE_ERR_INVALID_ARG, "K = %lld out of range", (long long)K);
  if (K % 16 != 0) return fail(FLCE_ERR_UNSUPPORTED, "K = %lld is not a multiple of 16", (long long)K);
  if (a_dtype != FLCE_DTYPE_BF16 && a_dtype != FLCE_DTYPE_F32) return fail(FLCE_ERR_INVALID_ARG, "unknown element type");
  if (block_rows != 1 && block_rows != 128) return fail(FLCE_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  if (rows > 0 && (!a || !q || !q_scale)) return fail(FLCE_ERR_INVALID_ARG, "a, q or q_scale is NULL");
  if (lda < K || (lda * (a_dtype == FLCE_DTYPE_F32 ? 4 : 2)) % 16 != 0)
    return fail(FLCE_ERR_ALIGNMENT, "the row stride must be at least K and a whole multiple of 16 bytes");
  if (off16(a) || off16(q)) return fail(FLCE_ERR_ALIGNMENT, "a and q must be 16-byte aligned");
  const int64_t blocks = cdiv(rows, 128) * cdiv(K, 128);
  if (blocks >= (int64_t(1) << 31)) return fail(FLCE_ERR_INVALID_ARG, "too many blocks");
  int dev = 0, sms = 0;
  flce_status st = current_device(&dev, &sms);
  if (st != FLCE_OK) return st;
  if (rows == 0) return FLCE_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(blocks);
  uint8_t* qb = static_cast<uint8_t*>(q);
  const int k = static_cast<int>(K);
  KernelScope ks(FLCE_KERNEL_QUANTIZE_FP8, s, 2.0 * rows * K, rows * K * (a_dtype == FLCE_DTYPE_F32 ? 5.0 : 3.0));
  if (a_dtype == FLCE_DTYPE_F32) {
    const float* f = static_cast<const float*>(a);
    if (block_rows == 128) fp8::quantize_kernel<float, true><<<grid, fp8::kQuantThreads, 0, s>>>(f, lda, rows, k, qb, q_scale);
    else fp8::quantize_kernel<float, false><<<grid, fp8::kQuantThreads, 0, s>>>(f, lda, rows, k, qb, q_scale);
  } else {
    const uint16_t* f = static_cast<const uint16_t*>(a);
    if (block_rows == 128) fp8::quantize_kernel<uint16_t, true><<<grid, fp8::kQuantThreads, 0, s>>>(f, lda, rows, k, qb, q_scale);
    else fp8::quantize_kernel<uint16_t, false><<<grid, fp8::kQuantThreads, 0, s>>>(f, lda, rows, k, qb, q_scale);
  }
  ks.done();
  return check_launch("quantize_fp8");
}

size_t flce_linear_fp8_workspace_size(int64_t T, int64_t K, int64_t V) {
  if (T < 0 || K < 1 || V < 1) return 0;
  return kHeaderBytes;
}

flce_status flce_linear_fp8(const void* x, const uint8_t* x_scale, const void* W, const uint8_t* W_scale, int64_t T,
                            int64_t K, int64_t V, void* y, int32_t y_dtype, int64_t ldy, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (T < 0 || T >= kMaxRows) return fail(FLCE_ERR_INVALID_ARG, "T = %lld out of range", (long long)T);
  if (V < 1 || V >= kMaxRows) return fail(FLCE_ERR_INVALID_ARG, "V = %lld out of range", (long long)V);
  if (K < 1 || K >= (int64_t(1) << 24)) return fail(FLCE_ERR_INVALID_ARG, "K = %lld out of range", (long long)K);
  if (K % 16 != 0) return fail(FLCE_ERR_UNSUPPORTED, "K = %lld is not a multiple of 16", (long long)K);
  if (y_dtype != FLCE_DTYPE_BF16 && y_dtype != FLCE_DTYPE_F32) return fail(FLCE_ERR_INVALID_ARG, "unknown element type");
  if (!W || !W_scale) return fail(FLCE_ERR_INVALID_ARG, "W or W_scale is NULL");
  if (T > 0 && (!x || !x_scale || !y)) return fail(FLCE_ERR_INVALID_ARG, "x, x_scale or y is NULL");
  if (ldy < V) return fail(FLCE_ERR_INVALID_ARG, "ldy is smaller than V");
  if (off16(x) || off16(W)) return fail(FLCE_ERR_ALIGNMENT, "x and W must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(y) % (y_dtype == FLCE_DTYPE_F32 ? 4 : 2))
    return fail(FLCE_ERR_ALIGNMENT, "y must be aligned to its element type");
  if (!workspace) return fail(FLCE_ERR_WORKSPACE, "workspace is NULL");
  if (workspace_bytes < kHeaderBytes)
    return fail(FLCE_ERR_WORKSPACE, "workspace of %zu bytes < %zu required", workspace_bytes, kHeaderBytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(FLCE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  int dev = 0, sms = 0, pairs = 0;
  flce_status st = current_device(&dev, &sms);
  if (st != FLCE_OK) return st;
  if ((st = get_encoder()) != FLCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    CUDA_TRY(cudaMemsetAsync(workspace, 0, kHeaderBytes, s));
    return FLCE_OK;
  }
  fp8::Params p;
  std::memset(&p, 0, sizeof(p));
  const int64_t es = y_dtype == FLCE_DTYPE_F32 ? 4 : 2;
  p.v_tma = static_cast<int32_t>(V & ~(16 / es - 1));
  p.y_tma = !off16(y) && (ldy * es) % 16 == 0 && p.v_tma > 0;
  if ((st = resident_pairs<true>(dev, sms, &pairs)) != FLCE_OK || (st = resident_pairs<false>(dev, sms, &pairs)) != FLCE_OK)
    return st;
  // One token tile: the vocabulary on M.  More: the side and the width of the tiles that
  // take the fewest rounds times what a round costs, which is about its operands' rows (128 and
  // N of each CTA), and a tenth more with the vocabulary on M for its epilogue.  Large
  // problems get N = 224; small ones narrower tiles on more of the SM pairs (301 x 1040 x
  // 4097: 96 tokens, 68 pairs, 9.0 us; 160 tokens, 34 pairs, 9.8 us.  400 x 4096 x 32,000:
  // tokens on M 44.7 us, vocabulary on M 47.9 us).
  bool tokens_m = false;
  int64_t n = cdiv(T, 32) * 32, n_tiles = 1, m_tiles = cdiv(V, 2 * fp8::kRowsCta);
  double least = 0.0;
  for (int side = 0; side < 2 && T > fp8::kMaxN; ++side) {
    const int64_t mt = cdiv(side ? T : V, 2 * fp8::kRowsCta);
    for (int64_t w = fp8::kMaxN; w >= 32; w -= 32) {
      const int64_t nt = cdiv(side ? V : T, w);
      const double cost = static_cast<double>(cdiv(mt * nt, pairs)) * static_cast<double>(128 + w) * (side ? 1.0 : 1.1);
      if (least == 0.0 || cost < least) least = cost, tokens_m = side, n = w, n_tiles = nt, m_tiles = mt;
    }
  }
  const int64_t units = m_tiles * n_tiles;
  if (units >= (int64_t(1) << 31) - 1024) return fail(FLCE_ERR_INVALID_ARG, "T x V is too large");
  p.n = static_cast<int32_t>(n), p.n_tiles = static_cast<int32_t>(n_tiles), p.m_tiles = static_cast<int32_t>(m_tiles);
  p.units = static_cast<int32_t>(units);
  p.stage_bytes = fp8::kABytes + p.n / 2 * fp8::kBlockK;
  p.staging_bytes = tokens_m && es == 2 && !p.y_tma ? fp8::kImageBytes : fp8::kStagingBytes;
  p.stages = std::min((fp8::kSmemLimit - 1024 - p.staging_bytes - fp8::kSmemTail) / p.stage_bytes, fp8::kMaxStages);
  const bool granules = !tokens_m && n_tiles == 1;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if ((st = matrix_map(tokens_m ? &p.tmB : &p.tmA, u8, CU_TENSOR_MAP_SWIZZLE_128B, W, K, V, K, fp8::kBlockK,
                       tokens_m ? p.n / 2 : (granules ? 32 : fp8::kRowsCta))) != FLCE_OK)
    return st;
  if ((st = matrix_map(tokens_m ? &p.tmA : &p.tmB, u8, CU_TENSOR_MAP_SWIZZLE_128B, x, K, T, K, fp8::kBlockK,
                       tokens_m ? fp8::kRowsCta : p.n / 2)) != FLCE_OK)
    return st;
  const CUtensorMapSwizzle y_swizzle = es == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (p.y_tma && (st = matrix_map(&p.tmY, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                  y_swizzle, y, p.v_tma, T, ldy * es, 32, 32)) != FLCE_OK)
    return st;
  p.sx = x_scale, p.sw = W_scale, p.y = y, p.ldy = ldy;
  p.status = static_cast<int32_t*>(workspace);
  p.timeout_ns = wait_limit_ns(K);
  p.T = static_cast<int32_t>(T), p.K = static_cast<int32_t>(K), p.V = static_cast<int32_t>(V);
  p.kb = static_cast<int32_t>(cdiv(K, fp8::kBlockK));
  p.y_f32 = y_dtype == FLCE_DTYPE_F32;
  const int64_t shares = granules ? cdiv(V, fp8::kGranule) : units;  // a pair takes at least one
  const int grid = 2 * static_cast<int>(std::min<int64_t>(pairs, shares));
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * p.stage_bytes + p.staging_bytes + fp8::kSmemTail;
  KernelScope ks(FLCE_KERNEL_LINEAR_FP8, s, 2.0 * T * K * V,
                 1.0 * T * K + 1.0 * V * K + (p.y_f32 ? 4.0 : 2.0) * T * V);
  st = launch_overlapped(tokens_m ? fp8::linear_fp8_kernel<true> : fp8::linear_fp8_kernel<false>, dim3(grid),
                         fp8::kThreads, smem, s, p);
  if (st != FLCE_OK) return st;
  ks.done();
  return check_launch("linear_fp8");
}

}  // extern "C"
