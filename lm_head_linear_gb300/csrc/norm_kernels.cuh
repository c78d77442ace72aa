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

// Threads per row at most for a thread that holds `vecs` vectors of 8 channels (their
// values live in registers, next to the raw loads).
__host__ __device__ constexpr int max_threads(int vecs) { return vecs == 1 ? 1024 : 512; }

// Eight weights, bf16 or fp32 (read by every row: they stay in L1).
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
// result on every thread).  `slot` holds `warps` of them per group.
__device__ __forceinline__ Twofold group_sum(Twofold v, Twofold* slot, int warps, int warp_in_group) {
  Twofold s = warp_sum_twofold(v);
  if (warps == 1) return s;
  if ((threadIdx.x & 31) == 0) slot[warp_in_group] = s;
  __syncthreads();
  s = slot[0];
  for (int i = 1; i < warps; ++i) s = s + slot[i];
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
  int32_t w_f32;
  float eps, inv_hd, inv_hd_lo;  // inv_hd + inv_hd_lo = 1 / Hd
};

// One row per group of `group` threads; thread i of the group holds channels
// 8 B (i + group k) .., k < NV: NV runs of B vectors.
//
// An e4m3 number is the 64-bit definition's but for one in 10^8: an error of rstd moves
// a whole row against the rounding boundaries (3e-8, half a unit of fp32, changes one
// element in a million), so the sums of squares and rstd carry what fp32 rounds off, the
// products are rounded once, and that once to odd, so that the rounding to four bits
// sees the value itself and not a rounded one.  Of the 134 M numbers of 65,536 x 2048
// one or none differs from the definition's; 61 to 102 did with each step rounded to
// nearest, 7 to 20 with plain sums of 32 squares.  EXACT: h and w are bf16, so that h w
// is exact in fp32.
//
// Bound by memory: 65,536 x 2048 with residual to 8 bits (941 MB) takes 138 us, 6.8 TB/s,
// with 64 % of the issue slots taken (135 us with plain sums of 32 squares); pairs of
// channels go through one instruction.  Rounding to odd by both directed roundings and a
// choice took 10 us more, and exact squares from the first on another 25: the issue
// slots ran out.
template <typename TX, typename TR, int NV, int B, bool EXACT>
__global__ void __launch_bounds__(max_threads(NV * B)) add_rms_norm_kernel(const FwdParams p) {
  constexpr int kRun = B * kVec, kRunPairs = B * kPairs, kBlockRuns = 128 / kRun;
  __shared__ Twofold red[32];
  ptx::launch_dependents();
  ptx::wait_prerequisites();
  const int group = blockDim.x, g = threadIdx.y, i = threadIdx.x;  // threads per row: a multiple of 32
  const int warps = group >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + g;
  const bool live = row < p.T;
  const TX* x = static_cast<const TX*>(p.x) + (live ? row : 0) * p.ldx;
  const TR* r = p.r ? static_cast<const TR*>(p.r) + (live ? row : 0) * p.ldr : nullptr;

  Raw8 rx[NV][B], rr[NV][B];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (i + k * group) * kRun;
    if (live && c < p.Hd) {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        rx[k][b] = load8(x + c + b * kVec);
        if (r) rr[k][b] = load8(r + c + b * kVec);
      }
    }
  }
  F2 v[NV][kRunPairs];
  F2 sq[kRunPairs] = {};  // 8 B chains of NV squares
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (i + k * group) * kRun;
    if (live && c < p.Hd) {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        F2 o[kPairs];
        unpack_pairs<TX>(rx[k][b], o);
        if (r) {
          F2 a[kPairs];
          unpack_pairs<TR>(rr[k][b], a);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) o[j] = add2(a[j], o[j]);
          const Raw8 packed = pack_pairs<TR>(o);
          store8(static_cast<TR*>(p.h) + row * p.ldh + c + b * kVec, packed);
          unpack_pairs<TR>(packed, o);
        }
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          v[k][b * kPairs + j] = o[j];
          sq[b * kPairs + j] = fma2(o[j], o[j], sq[b * kPairs + j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kRunPairs; ++j) v[k][j] = 0;
    }
  }
  F2 off = 0;  // what the sums below round off
#pragma unroll
  for (int d = kRunPairs / 2; d > 0; d >>= 1) {
#pragma unroll
    for (int j = 0; j < d; ++j) sq[j] = add2(sq[j], sq[j + d], off);
  }
  float even, odd, even_lo, odd_lo;
  split(sq[0], even, odd);
  split(off, even_lo, odd_lo);
  const Twofold ss = group_sum(Twofold{even, even_lo} + Twofold{odd, odd_lo}, red + g * warps, warps, i >> 5);
  // mean = ss / Hd + eps, then rstd as hi + lo by one Newton step on rsqrtf()'s value
  Twofold mean{ss.hi * p.inv_hd, 0.0f};
  mean.lo = fmaf(ss.hi, p.inv_hd, -mean.hi) + fmaf(ss.hi, p.inv_hd_lo, ss.lo * p.inv_hd);
  mean = mean + Twofold{p.eps, 0.0f};
  float hi = rsqrtf(mean.hi), lo = 0.0f;
  if (mean.hi > 0.0f && mean.hi < INFINITY) {
    const float t = mean.hi * hi, te = fmaf(mean.hi, hi, -t) + mean.lo * hi;
    const float step = 0.5f * hi * (fmaf(-t, hi, 1.0f) - te * hi);
    const float better = hi + step;
    lo = step - (better - hi);
    hi = better;
  }
  if (live && i == 0 && p.rstd) p.rstd[row] = hi;
  const F2 hi2 = both(hi), lo2 = both(lo), minus = both(-1.0f);
  // Rounding to odd: towards zero, and the last bit set where that cut something off.
  // With lo != 0 every product but 0 is cut (the odd part of hi + lo alone has more than
  // 24 bits).  With lo == 0, hi is a power of two (or 0 or infinite): what is cut is what
  // h w rounds off, nothing where that is exact, so what is exact stays exact.
  const uint32_t odd_bit = lo != 0.0f ? 1u : 0u;
  const int nblk = (p.Hd + 127) / 128;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int run = i + k * group, c = run * kRun;
    const bool mine = live && c < p.Hd;
    float y[kRun];
    float amax = 0.0f;
    if (mine) {
      F2 rest[kRunPairs];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        F2 w[kPairs];
        load_weight_pairs(p.w, !EXACT && p.w_f32 != 0, c + b * kVec, w);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {  // h w (hi + lo) = a hi + rest, a = round(h w)
          F2& h = v[k][b * kPairs + j];
          F2& t = rest[b * kPairs + j];
          const F2 a = mul2(h, w[j]);
          t = mul2(a, lo2);
          if constexpr (!EXACT) t = fma2(fma2(h, w[j], mul2(a, minus)), hi2, t);
          h = a;
        }
        if (p.y) {
          F2 s[kPairs];
#pragma unroll
          for (int j = 0; j < kPairs; ++j) s[j] = mul2(v[k][b * kPairs + j], hi2);
          store8(p.y + row * p.Hd + c + b * kVec, pack_pairs<uint16_t>(s));
        }
      }
      if (p.q) {  // rounded to odd; fmaxf drops NaN: the scale comes from the block's numbers, a NaN stays NaN in q
#pragma unroll
        for (int j = 0; j < kRunPairs; ++j) split(fma2_zero(v[k][j], hi2, rest[j]), y[2 * j], y[2 * j + 1]);
        if constexpr (!EXACT) {
          if (odd_bit == 0) {  // rare, and the same for the whole row
#pragma unroll
            for (int j = 0; j < kRunPairs; ++j) {
              float cut[2];
              split(rest[j], cut[0], cut[1]);
#pragma unroll
              for (int b = 0; b < 2; ++b)
                if (cut[b] != 0.0f) y[2 * j + b] = __uint_as_float(__float_as_uint(y[2 * j + b]) | 1u);
            }
          }
        }
#pragma unroll
        for (int b = 0; b < kRun; ++b) {
          y[b] = __uint_as_float(__float_as_uint(y[b]) | odd_bit);
          amax = fmaxf(amax, fabsf(y[b]));
        }
      }
    }
    if (p.q) {  // the same for every thread of the launch
#pragma unroll
      for (int d = kBlockRuns / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      if (mine) {
        const uint32_t e = e8m0_of(amax);  // the odd bit of a zero is below the least scale
        uint8_t* q = p.q + row * p.Hd + c;
        const uint2 a = to_e4m3x8(y, inv_scale(e));
        if constexpr (B == 2) {
          const uint2 b = to_e4m3x8(y + kVec, inv_scale(e));
          *reinterpret_cast<uint4*>(q) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
          *reinterpret_cast<uint2*>(q) = a;
        }
        if ((i & (kBlockRuns - 1)) == 0) p.qs[row * nblk + run / kBlockRuns] = static_cast<uint8_t>(e);
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
// loads stay in flight across the reductions.  The weights, which every row needs
// twice, are in shared memory too: what the stages leave of L1 does not hold them
// against the stores.  32,768 x 2048 with dh (537 MB): 87 us, both launches.  After the
// forward that wrote its inputs, the two together:
//     16 warps, two to a row, two stages, weights in shared memory   166 us
//     the same, weights through L1                                   181 us (169 with one stage)
//     12 warps, one to a row, one stage, weights through L1          172 us
constexpr int kBwdThreads = 512;
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
  int32_t w_shared;   // the weights are kept in shared memory
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

// W32: fp32 weights (bf16 ones always fit beside the stages).
template <typename TY, typename TH, int NV, bool W32>
__global__ void __launch_bounds__(kBwdThreads) norm_backward_kernel(const BwdParams p) {
  // groups x stages x (dy, h, dh rows), weights; afterwards the CTA's dw
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
  const uint32_t w_at = static_cast<uint32_t>(groups * p.stages) * row_bytes;
  if (p.w_shared) {
    for (int k = threadIdx.x; k < (W32 ? 2 : 1) * nvec; k += blockDim.x)
      reinterpret_cast<uint4*>(ring + w_at)[k] = __ldg(static_cast<const uint4*>(p.w) + k);
    __syncthreads();
  }
  const auto weight_pairs = [&](int c, F2 (&v)[kPairs]) {
    if constexpr (!W32)
      unpack_pairs<uint16_t>(load8(reinterpret_cast<const uint16_t*>(ring + w_at) + c * kVec), v);
    else if (p.w_shared)
      unpack_pairs<float>(load8(reinterpret_cast<const float*>(ring + w_at) + c * kVec), v);
    else
      load_weight_pairs(p.w, true, c * kVec, v);
  };
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
        weight_pairs(c, w);
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
        weight_pairs(c, w);
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
