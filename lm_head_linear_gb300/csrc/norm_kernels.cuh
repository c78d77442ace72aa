// Residual add + RMS norm, its 8-bit output with block scales, and its backward.
//
//   h = round(x + r)            (rounded to the residual's type: what the next layer reads)
//   rstd = (mean_c h_c^2 + eps)^(-1/2),   y_c = h_c rstd w_c
//
// and, in 8 bits, per row and block of 128 channels with a = max |y| over the block:
//   s = the smallest power of two with a / s <= 448 (at least 2^-126),  q = e4m3(y / s).
// A power of two makes y / s exact (one rounding in all, to e4m3), and one E8M0
// byte per block is what the tensor cores' scaled products take.
//
// Bound: HBM.  A row stays in registers from the load to the last store, so
// every input is read once and every output written once.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "vec8.cuh"

namespace flce {
namespace norm {

// Threads per CTA for a thread that holds NV vectors (its row values live in
// registers: 8 NV floats, plus the raw loads).
__host__ __device__ constexpr int max_threads(int nv) { return nv <= 2 ? 1024 : (nv <= 4 ? 512 : 256); }

// Eight weights, bf16 or fp32 (read by every row: they stay in L1).
__device__ __forceinline__ void load_weight8(const void* w, bool w_f32, int c, float (&v)[kVec]) {
  Raw8 r;
  if (w_f32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(w) + c);
    r.a = __ldg(p);
    r.b = __ldg(p + 1);
    unpack8<float>(r, v);
  } else {
    r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c));
    unpack8<uint16_t>(r, v);
  }
}

// ------------------------------------------------------------------ reductions
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Sum over the `warps` warps of this thread's row group, in warp order (the same
// result on every thread).  `slot` holds `warps` floats per group; the caller
// alternates between two slots, so one barrier per sum is enough.
__device__ __forceinline__ float group_sum(float v, float* slot, int warps, int warp_in_group) {
  v = warp_sum(v);
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) slot[warp_in_group] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < warps; ++i) s += slot[i];
  return s;
}

// ------------------------------------------------------------------ forward
struct FwdParams {
  const void* x;
  const void* r;   // residual, or nullptr
  const void* w;
  void* h;         // residual output, or nullptr
  uint16_t* y;     // bf16 [T, Hd], or nullptr
  float* rstd;     // [T], or nullptr
  uint8_t* q;      // e4m3 [T, Hd], or nullptr
  uint8_t* qs;     // E8M0 [T, ceil(Hd / 128)]
  int64_t ldx, ldr, ldh;
  int64_t T;
  int32_t Hd;
  int32_t group;   // threads per row (a multiple of 32)
  int32_t w_f32;
  float eps, inv_hd;
};

// One row per group of `group` threads; thread i of the group holds channels
// 8 (i + group k) .., k < NV.
template <typename TX, typename TR, int NV>
__global__ void __launch_bounds__(max_threads(NV)) add_rms_norm_kernel(const FwdParams p) {
  __shared__ float red[32];
  const int g = threadIdx.x / p.group;
  const int i = threadIdx.x - g * p.group;
  const int warps = p.group >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / p.group) + g;
  const bool live = row < p.T;
  const int nvec = p.Hd / kVec;
  const TX* x = static_cast<const TX*>(p.x) + (live ? row : 0) * p.ldx;
  const TR* r = p.r ? static_cast<const TR*>(p.r) + (live ? row : 0) * p.ldr : nullptr;

  Raw8 rx[NV], rr[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = i + k * p.group;
    if (live && c < nvec) {
      rx[k] = load8(x + c * kVec);
      if (r) rr[k] = load8(r + c * kVec);
    }
  }
  float v[NV][kVec];
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = i + k * p.group;
    if (live && c < nvec) {
      unpack8<TX>(rx[k], v[k]);
      if (r) {
        float o[kVec];
        unpack8<TR>(rr[k], o);
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[j] += v[k][j];
        const Raw8 packed = pack8<TR>(o);
        store8(static_cast<TR*>(p.h) + row * p.ldh + c * kVec, packed);
        unpack8<TR>(packed, v[k]);
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) ss = fmaf(v[k][j], v[k][j], ss);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[k][j] = 0.0f;
    }
  }
  ss = group_sum(ss, red + g * warps, warps, i >> 5);
  const float rstd = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
  if (live && i == 0 && p.rstd) p.rstd[row] = rstd;
  const int nblk = (p.Hd + 127) / 128;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = i + k * p.group;
    const bool mine = live && c < nvec;
    if (mine) {
      float w[kVec];
      load_weight8(p.w, p.w_f32 != 0, c * kVec, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[k][j] = v[k][j] * rstd * w[j];
      if (p.y) store8(p.y + row * p.Hd + c * kVec, pack8<uint16_t>(v[k]));
    }
    if (p.q) {  // the same for every thread of the launch
      // fmaxf drops NaN: the scale comes from the block's numbers, a NaN stays NaN in q
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) a = fmaxf(a, fabsf(v[k][j]));
#pragma unroll
      for (int d = kBlockVecs / 2; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
      if (mine) {
        const uint32_t e = e8m0_of(a);
        *reinterpret_cast<uint2*>(p.q + row * p.Hd + c * kVec) = to_e4m3x8(v[k], inv_scale(e));
        if ((threadIdx.x & (kBlockVecs - 1)) == 0) p.qs[row * nblk + c / kBlockVecs] = static_cast<uint8_t>(e);
      }
    }
  }
}

// ------------------------------------------------------------------ backward
//   u = dy w,   c = mean(u h),   dx = rstd (u - h rstd^2 c) + dh,   dw = sum_t dy h rstd
// (the same dx for x and for the residual).  Persistent CTAs walk the rows with a
// fixed stride and keep their share of dw in registers (a thread's channels are
// the same in every row); the shares go to the workspace and
// norm_dw_kernel adds them in CTA order, so dw is the same on every run.
struct BwdParams {
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dh;     // gradient that reaches h directly, or nullptr
  void* dx;
  float* partial;     // [gridDim.x, Hd]
  int64_t lddy, ldh, lddh;
  int64_t T;
  int32_t Hd;
  int32_t group;
  int32_t w_f32;
  float inv_hd;
};

template <typename TY, typename TH, int NV>
__global__ void __launch_bounds__(max_threads(NV)) norm_backward_kernel(const BwdParams p) {
  extern __shared__ float sh[];  // groups x Hd for the CTA's sum of dw (when it has several groups)
  __shared__ float red[2][32];
  const int groups = blockDim.x / p.group;
  const int g = threadIdx.x / p.group;
  const int i = threadIdx.x - g * p.group;
  const int warps = p.group >> 5;
  const int nvec = p.Hd / kVec;
  float acc[NV][kVec];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int j = 0; j < kVec; ++j) acc[k][j] = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int flip = 0;
  // every group of the CTA makes the same number of rounds (group_sum's barrier)
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < p.T; base += step) {
    const int64_t row = base + g;
    const bool live = row < p.T;
    const TY* dy = static_cast<const TY*>(p.dy) + (live ? row : 0) * p.lddy;
    const TH* h = static_cast<const TH*>(p.h) + (live ? row : 0) * p.ldh;
    Raw8 ry[NV], rh[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = i + k * p.group;
      if (live && c < nvec) {
        ry[k] = load8(dy + c * kVec);
        rh[k] = load8(h + c * kVec);
      }
    }
    const float rstd = live ? p.rstd[row] : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = i + k * p.group;
      if (live && c < nvec) {
        float y[kVec], hv[kVec], w[kVec];
        unpack8<TY>(ry[k], y);
        unpack8<TH>(rh[k], hv);
        load_weight8(p.w, p.w_f32 != 0, c * kVec, w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          s = fmaf(y[j] * w[j], hv[j], s);
          acc[k][j] = fmaf(y[j], hv[j] * rstd, acc[k][j]);
        }
      }
    }
    s = group_sum(s, red[flip] + g * warps, warps, i >> 5);
    flip ^= 1;
    const float m = s * p.inv_hd * rstd * rstd;
    if (live) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = i + k * p.group;
        if (c < nvec) {
          float y[kVec], hv[kVec], w[kVec];
          unpack8<TY>(ry[k], y);
          unpack8<TH>(rh[k], hv);
          load_weight8(p.w, p.w_f32 != 0, c * kVec, w);
#pragma unroll
          for (int j = 0; j < kVec; ++j) y[j] = rstd * (y[j] * w[j] - hv[j] * m);
          if (p.dh) {
            float d[kVec];
            unpack8<TH>(load8(static_cast<const TH*>(p.dh) + row * p.lddh + c * kVec), d);
#pragma unroll
            for (int j = 0; j < kVec; ++j) y[j] += d[j];
          }
          store8(static_cast<TH*>(p.dx) + row * p.Hd + c * kVec, pack8<TH>(y));
        }
      }
    }
  }
  // the CTA's sum over its groups, in group order
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.Hd;
  if (groups == 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = i + k * p.group;
      if (c < nvec) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) out[c * kVec + j] = acc[k][j];
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = i + k * p.group;
    if (c < nvec) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) sh[g * p.Hd + c * kVec + j] = acc[k][j];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.Hd; c += blockDim.x) {
    float s = 0.0f;
    for (int gg = 0; gg < groups; ++gg) s += sh[gg * p.Hd + c];
    out[c] = s;
  }
}

// dw[c] = sum over CTAs of partial[b][c]: 32 columns per CTA, the CTAs' shares cut
// into kDwSlices fixed slices that are then added in order.
constexpr int kDwSlices = 32;

__global__ void __launch_bounds__(32 * kDwSlices) norm_dw_kernel(const float* partial, int blocks, int Hd, float* dw,
                                                               int32_t* status) {
  __shared__ float sh[kDwSlices][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;  // no error depends on the data here
  float s = 0.0f;
  if (c < Hd)
    for (int b = slice; b < blocks; b += kDwSlices) s += partial[static_cast<int64_t>(b) * Hd + c];
  sh[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < Hd) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < kDwSlices; ++k) t += sh[k][lane];
    dw[c] = t;
  }
}

}  // namespace norm
}  // namespace flce
