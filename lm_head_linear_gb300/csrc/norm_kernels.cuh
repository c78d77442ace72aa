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

__device__ __forceinline__ void load_weight_pairs(const void* w, bool w_f32, int c, F2 (&v)[kPairs]) {
  Raw8 r;
  if (w_f32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(w) + c);
    r.a = __ldg(p);
    r.b = __ldg(p + 1);
    unpack_pairs<float>(r, v);
  } else {
    r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c));
    unpack_pairs<uint16_t>(r, v);
  }
}

// ------------------------------------------------------------------ reductions
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Sum over the `warps` warps of this thread's row group, in warp order (the same
// result on every thread).  `slot` holds `warps` floats per group; a barrier lies
// between one sum's last read and the next one's first write.
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
  ptx::launch_dependents();
  ptx::wait_prerequisites();
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
// (the same dx for x and for the residual).  Persistent CTAs, whose groups of threads
// each walk the rows with a fixed stride and keep their share of dw in registers (a
// thread's channels are the same in every row); the shares go to the workspace and
// norm_dw_kernel adds them in CTA order, so dw is the same on every run.
//
// A row is needed twice, before and after its mean, and nothing of the next row
// depends on it: every group has a ring of shared-memory stages of its own, into
// which one of its threads copies the rows of dy, h and dh ahead (bulk copies), so
// loads stay in flight across the reductions.  A group is one warp up to 2048
// channels, and no group waits for another: with 12 warps an SM's loads and arithmetic
// overlap even where shared memory has one stage for each.  32,768 x 2048 with dh, 537
// MB, both launches: 100 us; 8 warps with two stages each 111 us, one ring for the CTA
// with its barriers 102 us, loads into registers 112 us.
constexpr int kBwdThreads = 384;
constexpr int kBwdMaxStages = 8;
constexpr int kBwdMaxGroups = kBwdThreads / 32;
constexpr int kStatusTimeout = 7;  // FLCE_ERR_TIMEOUT

struct BwdParams {
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dh;     // gradient that reaches h directly, or nullptr
  void* dx;
  float* partial;     // [gridDim.x, Hd]
  int32_t* status;
  uint64_t timeout_ns;
  int64_t lddy, ldh, lddh;
  int64_t T;
  int32_t Hd;
  int32_t group;
  int32_t stages;
  int32_t w_f32;
  float inv_hd;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Barrier of one group (named barrier 1 + g; a warp needs none of them), and whether
// any of its threads passed true.
__device__ __forceinline__ void group_sync(int g, int threads) {
  if (threads == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(threads) : "memory");
}
__device__ __forceinline__ bool group_any(int g, int threads, bool v) {
  if (threads == 32) return __any_sync(0xffffffffu, v);
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %3, 0;\n\t"
      "bar.red.or.pred b, %1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(1 + g), "r"(threads), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

template <typename TY, typename TH, int NV>
__global__ void __launch_bounds__(kBwdThreads) norm_backward_kernel(const BwdParams p) {
  // groups x stages x (dy, h, dh rows); afterwards the CTA's dw
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[kBwdThreads / 32];
  __shared__ __align__(8) uint64_t full[kBwdMaxGroups * kBwdMaxStages];
  const int groups = blockDim.x / p.group;
  const int g = threadIdx.x / p.group;
  const int i = threadIdx.x - g * p.group;
  const int warps = p.group >> 5;
  const int nvec = p.Hd / kVec;
  const uint32_t y_bytes = p.Hd * static_cast<uint32_t>(sizeof(TY)), h_bytes = p.Hd * static_cast<uint32_t>(sizeof(TH));
  const uint32_t row_bytes = y_bytes + h_bytes + (p.dh ? h_bytes : 0u);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups + g;
  uint8_t* mine = ring + static_cast<size_t>(g) * p.stages * row_bytes;
  uint64_t* bars = full + g * kBwdMaxStages;
  // the group's first thread: the copies of row `row` into stage `slot`
  const auto fill = [&](int64_t row, int slot) {
    if (row >= p.T) return;
    const uint32_t bar = ptx::smem_u32(bars + slot);
    const uint32_t to = ptx::smem_u32(mine + static_cast<size_t>(slot) * row_bytes);
    ptx::mbar_arrive_expect_tx(bar, row_bytes);
    bulk_load(to, static_cast<const TY*>(p.dy) + row * p.lddy, y_bytes, bar);
    bulk_load(to + y_bytes, static_cast<const TH*>(p.h) + row * p.ldh, h_bytes, bar);
    if (p.dh) bulk_load(to + y_bytes + h_bytes, static_cast<const TH*>(p.dh) + row * p.lddh, h_bytes, bar);
  };
  if (threadIdx.x == 0) {
    for (int k = 0; k < groups; ++k)
      for (int q = 0; q < p.stages; ++q) ptx::mbar_init(ptx::smem_u32(full + k * kBwdMaxStages + q), 1);
    ptx::fence_barrier_init();
    ptx::fence_proxy_async_smem();
  }
  ptx::launch_dependents();
  __syncthreads();
  ptx::wait_prerequisites();
  // The status of this call: cleared by the first CTA, dispatched first; a wait that
  // runs out sets it a millisecond later at the earliest.
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  if (i == 0)
    for (int k = 0; k < p.stages; ++k) fill(row0 + k * step, k);

  F2 acc[NV][kPairs];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int j = 0; j < kPairs; ++j) acc[k][j] = 0;
  float rstd_next = row0 < p.T ? p.rstd[row0] : 0.0f;
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int64_t row = row0; row < p.T; row += step) {
    const float rstd = rstd_next;
    rstd_next = row + step < p.T ? p.rstd[row + step] : 0.0f;
    ok = ptx::wait_bounded(ptx::smem_u32(bars + slot), phase, p.timeout_ns, nullptr);
    if (group_any(g, p.group, !ok)) {
      ok = false;
      break;
    }
    const uint8_t* stage = mine + static_cast<size_t>(slot) * row_bytes;
    const TY* dy = reinterpret_cast<const TY*>(stage);
    const TH* h = reinterpret_cast<const TH*>(stage + y_bytes);
    const TH* dh = reinterpret_cast<const TH*>(stage + y_bytes + h_bytes);
    // with q = dy h:  c = sum q w,  dw += q rstd
    const F2 rstd2 = both(rstd);
    F2 s2[2] = {0, 0};  // two chains
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = i + k * p.group;
      if (c < nvec) {
        F2 y[kPairs], hv[kPairs], w[kPairs];
        unpack_pairs<TY>(load8(dy + c * kVec), y);
        unpack_pairs<TH>(load8(h + c * kVec), hv);
        load_weight_pairs(p.w, p.w_f32 != 0, c * kVec, w);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const F2 q = mul2(y[j], hv[j]);
          s2[j & 1] = fma2(q, w[j], s2[j & 1]);
          acc[k][j] = fma2(q, rstd2, acc[k][j]);
        }
      }
    }
    float s, sx, sy, sz;
    split(s2[0], s, sx);
    split(s2[1], sy, sz);
    s = (s + sx) + (sy + sz);
    s = warp_sum(s);
    if (warps > 1) {
      float* slots = red + g * warps;
      if ((i & 31) == 0) slots[i >> 5] = s;
      group_sync(g, p.group);
      s = 0.0f;
      for (int k = 0; k < warps; ++k) s += slots[k];
    }
    // dx = dy (rstd w) - h (rstd^3 c / Hd) + dh
    const F2 back = both(-(s * p.inv_hd * rstd * rstd * rstd));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = i + k * p.group;
      if (c < nvec) {
        F2 y[kPairs], hv[kPairs], w[kPairs], d[kPairs];
        unpack_pairs<TY>(load8(dy + c * kVec), y);
        unpack_pairs<TH>(load8(h + c * kVec), hv);
        load_weight_pairs(p.w, p.w_f32 != 0, c * kVec, w);
        if (p.dh) {
          unpack_pairs<TH>(load8(dh + c * kVec), d);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) d[j] = fma2(hv[j], back, d[j]);
        } else {
#pragma unroll
          for (int j = 0; j < kPairs; ++j) d[j] = mul2(hv[j], back);
        }
#pragma unroll
        for (int j = 0; j < kPairs; ++j) d[j] = fma2(y[j], mul2(w[j], rstd2), d[j]);
        store8(static_cast<TH*>(p.dx) + row * p.Hd + c * kVec, pack_pairs<TH>(d));
      }
    }
    group_sync(g, p.group);  // the group has read the stage, and red
    if (i == 0) fill(row + p.stages * step, slot);
    if (++slot == p.stages) slot = 0, phase ^= 1u;
  }
  if (!ok && i == 0) {
    // a copy did not arrive: report it, and give the others time before leaving
    atomicCAS(p.status, 0, kStatusTimeout);
    for (int k = 0; k < p.stages; ++k) {
      const int at = (slot + k) % p.stages;
      ptx::wait_bounded(ptx::smem_u32(bars + at), slot + k < p.stages ? phase : phase ^ 1u, 1000000000ull, nullptr);
    }
  }
  __syncthreads();  // no copy is in flight any more
  // the CTA's sum over its groups, in group order
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.Hd;
  float* sh = reinterpret_cast<float*>(ring);
  if (groups == 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = i + k * p.group;
      if (c < nvec) store8(out + c * kVec, pack_pairs<float>(acc[k]));
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = i + k * p.group;
    if (c < nvec) store8(sh + g * p.Hd + c * kVec, pack_pairs<float>(acc[k]));
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

// Dispatched while the backward still runs.
__global__ void __launch_bounds__(32 * kDwSlices) norm_dw_kernel(const float* partial, int blocks, int Hd, float* dw) {
  __shared__ float sh[kDwSlices][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  ptx::wait_prerequisites();
  if (c < Hd)
    for (int b = slice; b < blocks; b += kDwSlices) s += __ldcg(partial + static_cast<int64_t>(b) * Hd + c);
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
