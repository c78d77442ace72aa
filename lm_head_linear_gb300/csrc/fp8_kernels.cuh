// 8-bit head product: Y = (X sx)(W sw)^T with e4m3 operands and one power-of-two
// scale per 128 channels of a row of X and per 128 x 128 block of W.
//
//   Y[t, v] = sum_b sx[t, b] sw[v / 128, b] sum_{k in block b} X[t, k] W[v, k]
//
// And the same with 4-bit weights (W4): W of e2m1 numbers with one scale per row and 32 channels,
//
//   Y[t, v] = sum_g sx[t, g / 4] sw[g / 4, v, g % 4] sum_{k in group g} X[t, k] W[v, k]
//
// The scales are E8M0 bytes, which the tensor cores apply themselves
// (kind::mxf8f6f4 with block scaling): the products of a block are scaled on
// their way into the fp32 accumulator, and no partial sum leaves TMEM before the
// whole K loop is done.
//
// Two orientations of the 256 x N tile of an SM pair (128 rows of the M side per CTA):
//   vocabulary on M, tokens on N (N = 32 .. 224): a decoding step of a few tokens
//     runs narrow tiles over wide W tiles and is bound by reading W;
//   tokens on M, vocabulary on N: a prompt.  A lane of the accumulator is then
//     a token and its columns are consecutive logits, which go to the staging buffer
//     16 bytes at a time (with the vocabulary on M they take a 2-byte store each:
//     8192 x 2048 x 124,160 takes 1358 us this way and 1443 us that way).  Stored from
//     the registers straight to the rows, without the staging buffer and TMA, it takes
//     1540 us with 32 bytes a store and 1720 us with 16, against 1450 us on that box.
//     N falls below 224 where the tiles would not fill the device (flce_fp8.cu).
//
// A CTA has 14 warps: the TMA producer, the MMA issuer (even CTA of the pair),
// eight epilogue warps and four scale warps.  The scale bytes come from their plain
// row-major arrays: a scale warp loads, for the 32 TMEM lanes it may write, the
// words of four consecutive K blocks and stores them to TMEM, four blocks a stage.
// 224, not 256, tokens per tile: two accumulators (448 columns) and four stages
// of scales (64 columns) fill the 512 columns of TMEM.
//
// 4-bit weights: TMA unpacks them, 16 numbers (8 bytes) to 16 bytes of shared memory, which is
// how the tensor cores read them beside e4m3; nothing is converted.  Every row has a word of scales
// for each K block: 32 to 40 columns a stage of four K blocks instead of 16, so tiles end at N = 192.
//
// Bound: few tokens by reading W (1 x 2048 x 124,160: 43 us for 254 MB, of which a
// kernel that only reads takes 37.1; 93 x 4096 x 248,320: 157 to 160 us, 6.7 TB/s); a prompt by
// shared memory and the clock.  A K block of a 256 x 224 tile keeps the tensor pipe busy
// for 448 cycles, shared memory for about 480 (operands in by TMA, out to the MMA) and
// for 56 more of the epilogue's transposes; it measures 535 cycles at K = 2048 and 503 at
// K = 4096.  8192 x 2048 x 124,160: 1360 to 1470 us, 2.8 to 3.1 PFLOP/s, at the 1.4 to
// 1.6 GHz that the power cap leaves.
//   4-bit weights, few tokens: 1 x 2048 x 124,160 30.4 us for 135 MB, 93 x 4096 x 248,320 109 to 110 us
// for 587 MB (5.4 TB/s).  The former with the tokens' copies, the scales' copies and stores
// and three of four MMAs left out takes 24.9 us; the rest is scales and the chain of barriers between
// their warps, the MMA issuer and the producer, which has half as long for a K block as
// with 8-bit weights.  W fetched into L2 ahead by TMA took 47 us: the copy engine needs 1.4 ns
// for a row of 64 bytes, wherever it goes.  A prompt runs at the 8-bit rate (2048 x 2048 x 124,160 under
// the power cap: 367 us at 1740 MHz, 372 at 1470 with 8-bit weights; in a burst 337 and 328).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "vec8.cuh"

namespace flce {
namespace fp8 {

constexpr int kBlockK = 128;                  // bytes of a K block: one swizzled 128-byte row, one scale
constexpr int kRowsCta = 128;                 // vocabulary rows of one CTA: one row block of W's scales
constexpr int kABytes = kRowsCta * kBlockK;   // 16 KB
constexpr int kMaxN = 224;
constexpr int kMaxN4 = 192;                   // with 4-bit weights
constexpr int kMaxStages = 12;
constexpr int kScaleStages = 4;
constexpr int kEpiWarps = 8;   // two for each quarter of the TMEM lanes, on alternate columns
constexpr int kScaleWarps = 4;
constexpr int kThreads = 32 * (2 + kEpiWarps + kScaleWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kStagingWarp = 32 * 32 * 4;  // of an epilogue warp: two 32 x 32 boxes of bf16 or one of fp32
constexpr int kStagingBytes = kEpiWarps * kStagingWarp;
// Whole rows of a bf16 tile (see store_images): a row's bytes and what it lies off 16, an
// odd number of 16-byte pieces, and a skew of one piece every eight rows.
constexpr int kImagePitch = kMaxN * 2 + 16;
constexpr int kImageWarp = 32 * kImagePitch + 64;  // 32 rows
constexpr int kImageBytes = 4 * kImageWarp;
static_assert(kImagePitch % 32 == 16, "image pitch");
constexpr int kSmemTail = 512;
constexpr int kSmemLimit = 232448;
constexpr int kStatusTimeout = 7;
constexpr uint64_t kDrainNs = 200000000ull;   // for copies and MMAs in flight when a kernel gives up
constexpr uint64_t kSettleNs = 200000ull;

// What the kinds of weights and the two orientations differ in.
//
// The columns of TMEM: two accumulators, then kStages stages of scale words, each of four K
// blocks.  A word holds four bytes of a row: the scales of four K blocks (a token's, and
// 8-bit weights', one per 128 channels), or the four of one K block (4-bit weights', one per
// 32): A's words of K block 4 g + j at a(j), B's at b(j).
template <bool TOKENS_M, bool W4>
struct Form {
  static constexpr int kAcc = W4 ? kMaxN4 : kMaxN;  // columns of an accumulator
  static constexpr int kBase = 2 * kAcc;
  static constexpr int kCols = !W4 ? 16 : TOKENS_M ? 40 : 32;
  static constexpr int kStages = W4 && TOKENS_M ? 3 : kScaleStages;
  __host__ __device__ static constexpr uint32_t a(uint32_t j) { return W4 && !TOKENS_M ? 4 * j : 0; }
  __host__ __device__ static constexpr uint32_t b(uint32_t j) { return !W4 ? 8 : TOKENS_M ? 8 + 8 * j : 16; }
  static_assert(kBase + kStages * kCols <= static_cast<int>(kTmemCols), "TMEM columns");
};

// Scale words of 4-bit weights on their way to TMEM: a ring in shared memory, kDepth stages of
// four K blocks ahead: kWRows words of W for each K block, then kTRows of the tokens.
template <bool TOKENS_M>
struct Ring4 {
  static constexpr int kWRows = TOKENS_M ? kMaxN4 : kRowsCta;
  static constexpr int kTRows = TOKENS_M ? kRowsCta : kMaxN4;
  static constexpr int kBytes = 4 * (4 * kWRows + kTRows);
  static constexpr int kDepth = TOKENS_M ? 3 : 4;
};
constexpr int kRing4Bytes = 11264;
static_assert(Ring4<true>::kBytes * Ring4<true>::kDepth <= kRing4Bytes && Ring4<false>::kBytes * Ring4<false>::kDepth <= kRing4Bytes,
              "scale ring");

struct Params {
  CUtensorMap tmA;   // the M side, [rows, K] bytes, box 128 x 128 rows (one token tile: x 32 rows)
  CUtensorMap tmB;   // the N side, box 128 x N / 2 rows
  CUtensorMap tmY;   // [T, v_tma] logits, box 32 logits x 32 tokens (y_tma)
  const uint8_t* sx; // [T, kb]
  const uint8_t* sw; // [ceil(V / 128), kb]; 4-bit weights: words [kb, V]
  void* y;
  int64_t ldy;
  int32_t* status;
  uint64_t timeout_ns;
  int32_t T, K, V;
  int32_t kb;        // K blocks
  int32_t n;         // N (a multiple of 32 up to kMaxN)
  int32_t n_tiles, m_tiles, units;
  int32_t stages, stage_bytes, staging_bytes;
  int32_t y_f32;
  int32_t y_tma;     // y's rows start on 16-byte boundaries: boxes leave by TMA, else row by row
  int32_t v_tma;     // V rounded down to whole 16 bytes: TMA writes 16-byte pieces, also past its bounds
};

// full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], scale_full[4], scale_empty[4], drain
struct Smem {
  uint8_t* stages;
  uint8_t* staging;
  uint8_t* ring;  // 4-bit weights' scales
  uint64_t* bars;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  __device__ __forceinline__ uint32_t bar(int i) const { return ptx::smem_u32(bars + i); }
  __device__ __forceinline__ uint32_t full(int i) const { return bar(i); }
  __device__ __forceinline__ uint32_t empty(int i) const { return bar(kMaxStages + i); }
  __device__ __forceinline__ uint32_t acc_full(int i) const { return bar(2 * kMaxStages + i); }
  __device__ __forceinline__ uint32_t acc_empty(int i) const { return bar(2 * kMaxStages + 2 + i); }
  __device__ __forceinline__ uint32_t scale_full(int i) const { return bar(2 * kMaxStages + 4 + i); }
  __device__ __forceinline__ uint32_t scale_empty(int i) const { return bar(2 * kMaxStages + 4 + kScaleStages + i); }
  __device__ __forceinline__ uint32_t drain() const { return bar(2 * kMaxStages + 4 + 2 * kScaleStages); }
};
constexpr int kBars = 2 * kMaxStages + 4 + 2 * kScaleStages + 1;
static_assert(kBars * 8 + 8 <= kSmemTail, "smem tail");

__device__ __forceinline__ void give_up(const Params& p, const Smem& s) {
  *s.abort_flag = 1;
  atomicCAS(p.status, 0, kStatusTimeout);
}

// A ring position: slot and the phase bit its barriers are at.
struct Slot {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) i = 0, phase ^= 1u;
  }
};

// The tiles of one pair.  Several token tiles: tiles of 256 M rows, tokens fastest
// (the pairs in flight share W's rows and the tokens stay in L2), strided over the
// pairs.  One token tile (decoding, bound by reading W): every pair takes an equal
// share of W in granules of 64 rows, in tiles of up to four; 485 tiles of 256 rows over
// 76 pairs would leave 9 % of them idle in the last round.
struct Unit {
  int row;    // this CTA's first row of the M side
  int boxes;  // 32-row boxes this CTA holds (4: a full tile)
  int n0;     // the tile's first row of the N side
};
struct Work {
  int first, count, step;  // tile indexes
  int g0, g1;              // granules (one token tile)
};
constexpr int kGranule = 64;

template <bool TOKENS_M>
__device__ __forceinline__ Work work_of(const Params& p) {
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  Work w{pair, p.units, pairs, 0, 0};
  if (!TOKENS_M && p.n_tiles == 1) {
    const int64_t total = (static_cast<int64_t>(p.V) + kGranule - 1) / kGranule;
    w.g0 = static_cast<int>(total * pair / pairs);
    w.g1 = static_cast<int>(total * (pair + 1) / pairs);
    w.first = 0, w.step = 1, w.count = (w.g1 - w.g0 + 3) / 4;
  }
  return w;
}

template <bool TOKENS_M>
__device__ __forceinline__ Unit unit_of(const Params& p, const Work& w, int u, uint32_t rank) {
  Unit r;
  if constexpr (TOKENS_M) {
    const int nb = u / p.m_tiles;
    r.boxes = 4;
    r.row = (2 * (u - nb * p.m_tiles) + static_cast<int>(rank)) * kRowsCta;
    r.n0 = nb * p.n;
  } else if (p.n_tiles == 1) {
    const int g = w.g0 + 4 * u;
    r.boxes = min(4, w.g1 - g);
    r.row = g * kGranule + static_cast<int>(rank) * 32 * r.boxes;
    r.n0 = 0;
  } else {
    const int m = u / p.n_tiles;
    r.boxes = 4;
    r.row = (2 * m + static_cast<int>(rank)) * kRowsCta;
    r.n0 = (u - m * p.n_tiles) * p.n;
  }
  return r;
}

// An arrival on a barrier of the even CTA that passes no generic memory on (what it
// orders is TMEM, through tcgen05.wait and the tcgen05 fences): relaxed, since a
// release would first wait for the thread's own loads and stores in flight
// (1 x 2048 x 124,160: 67.8 us with release, 50.2 us relaxed).
__device__ __forceinline__ void arrive_even(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(ptx::mapa(bar, 0)) : "memory");
}

// Both CTAs: this CTA's 128 rows of the M side and its half of the N side.
// STEP: K blocks of a stage of operands.
template <bool TOKENS_M, bool W4, int STEP>
__device__ __forceinline__ void producer(const Params& p, const Smem& s, const Work& w, uint32_t rank) {
  Slot at;
  uint32_t used = 0;
  bool ok = true;
  const bool small = !TOKENS_M && p.n_tiles == 1;
  const int step_bytes = STEP == 1 ? p.stage_bytes : kABytes + p.n / 2 * kBlockK;  // of a K block
  // The barriers count bytes as they lie in memory: a row of 128 4-bit numbers is 64.
  constexpr int kARow = W4 && !TOKENS_M ? kBlockK / 2 : kBlockK, kBRow = W4 && TOKENS_M ? kBlockK / 2 : kBlockK;
  for (int u = w.first; u < w.count && ok; u += w.step) {
    const Unit un = unit_of<TOKENS_M>(p, w, u, rank);
    const int n_row = un.n0 + static_cast<int>(rank) * (p.n / 2);
    const uint32_t tx = 2u * static_cast<uint32_t>(un.boxes * 32 * kARow + (step_bytes - kABytes) / (kBlockK / kBRow));
    for (int kb = 0; kb < p.kb; kb += STEP) {
      if (!ptx::wait_bounded_cluster(s.empty(at.i), at.phase ^ 1u, p.timeout_ns, s.abort_flag)) {
        give_up(p, s);
        ok = false;
        break;
      }
      const int blocks = STEP == 1 ? 1 : min(STEP, p.kb - kb);
      if (rank == 0) ptx::mbar_arrive_expect_tx(s.full(at.i), tx * blocks);
      const uint32_t full = ptx::mapa(s.full(at.i), 0);
#pragma unroll
      for (int j = 0; j < STEP; ++j) {
        if (j >= blocks) break;
        const uint32_t a = ptx::smem_u32(s.stages + at.i * p.stage_bytes) + j * step_bytes;
        const int c = (kb + j) * kBlockK;
        if (small) {
          for (int b = 0; b < un.boxes; ++b)
            ptx::tma_load_2d_pair(a + b * 32 * kBlockK, &p.tmA, c, un.row + 32 * b, full);
        } else {
          ptx::tma_load_2d_pair(a, &p.tmA, c, un.row, full);
        }
        ptx::tma_load_2d_pair(a + kABytes, &p.tmB, c, n_row, full);
      }
      used |= 1u << at.i;
      at.next(p.stages);
    }
  }
  // the even CTA's barriers count both CTAs' loads: none is in flight once their
  // last armed phase has completed
  if (rank == 0)
    for (int i = 0; i < p.stages; ++i)
      if ((used & (1u << i)) && !ptx::wait_bounded(s.full(i), i < at.i ? at.phase : at.phase ^ 1u, kDrainNs, nullptr))
        break;  // the odd CTA gave up before its half: what it did issue has landed by now
}

// Even CTA only.  One thread issues everything, and what it works out between two MMAs counts: the
// test for the end of K in stages of one K block, where the loop has made it, took the 8-bit
// 8192 x 2048 x 124,160 from 1374 to 1484 us.
template <bool TOKENS_M, bool W4, int STEP>
__device__ __forceinline__ void mma_issuer(const Params& p, const Smem& s, const Work& w, uint32_t tmem) {
  using F = Form<TOKENS_M, W4>;
  Slot at, sc, acc;
  bool ok = true;
  static_assert(4 % STEP == 0, "a stage of scales is whole stages of operands");
  const int step_bytes = kABytes + p.n / 2 * kBlockK;
  const uint32_t idesc0 = ptx::idesc_mxf8(2 * kRowsCta, static_cast<uint32_t>(p.n), 0) |
                          (!W4 ? 0u : TOKENS_M ? ptx::kIdescB2M1 : ptx::kIdescA2M1);
  for (int u = w.first; u < w.count && ok; u += w.step) {
    ok = ptx::wait_bounded_cluster(s.acc_empty(acc.i), acc.phase ^ 1u, p.timeout_ns, s.abort_flag);
    if (!ok) break;
    ptx::tc_fence_after();
    const uint32_t d = tmem + acc.i * F::kAcc;
    for (int kb = 0; kb < p.kb; kb += STEP) {
      if ((kb & 3) == 0) {
        ok = ptx::wait_bounded_cluster(s.scale_full(sc.i), sc.phase, p.timeout_ns, s.abort_flag);
        if (!ok) break;
      }
      ok = ptx::wait_bounded(s.full(at.i), at.phase, p.timeout_ns, s.abort_flag);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t scales = tmem + F::kBase + sc.i * F::kCols;
#pragma unroll
      for (int j = 0; j < STEP; ++j) {
        if (STEP > 1 && kb + j >= p.kb) break;
        const uint32_t a = ptx::smem_u32(s.stages + at.i * p.stage_bytes) + j * step_bytes;
        const uint32_t sf = static_cast<uint32_t>((kb + j) & 3);
#pragma unroll
        for (uint32_t k = 0; k < kBlockK / 32; ++k) {
          // the byte of A's and of B's words
          const uint32_t idesc = idesc0 | ((W4 && TOKENS_M ? k : sf) << 4) | ((W4 && !TOKENS_M ? k : sf) << 29);
          ptx::mma_mxf8_pair(d, ptx::smem_desc_sw128(a + k * 32, 16, 1024),
                             ptx::smem_desc_sw128(a + kABytes + k * 32, 16, 1024), idesc, scales + F::a(sf),
                             scales + F::b(sf), (static_cast<uint32_t>(kb + j) | k) != 0 ? 1u : 0u);
        }
      }
      ptx::mma_commit_pair(s.empty(at.i), 0x3);
      at.next(p.stages);
      if (STEP == 1 ? (kb & 3) == 3 || kb == p.kb - 1 : ((kb + STEP) & 3) == 0 || kb + STEP >= p.kb) {
        ptx::mma_commit_pair(s.scale_empty(sc.i), 0x3);
        sc.next(F::kStages);
      }
    }
    if (!ok) break;
    ptx::mma_commit_pair(s.acc_full(acc.i), 0x3);
    acc.next(2);
  }
  if (!ok) give_up(p, s);
  // every MMA issued so far is done before TMEM is freed
  ptx::mma_commit_pair(s.drain(), 0x1);
  ptx::wait_bounded(s.drain(), 0, kDrainNs, nullptr);
}

// Four scale bytes from any byte address: the two aligned words they lie in, loaded
// here, and combined by bytes_of() when they are used, so that nothing waits for the
// loads before.  Bytes of the pair outside the array are never touched.  Plain loads: a kernel
// dispatched early lives while the one before it writes the tokens' scales.
struct TwoWords {
  uint32_t lo, hi;
};
__device__ __forceinline__ TwoWords load_words(const uint8_t* base, int64_t bytes, int64_t at) {
  const uint8_t* a = base + at;
  const uint8_t* p = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(a) & ~uintptr_t(3));
  TwoWords w;
  if (p >= base && p + 8 <= base + bytes) {
    w.lo = *reinterpret_cast<const uint32_t*>(p);
    w.hi = *(reinterpret_cast<const uint32_t*>(p) + 1);
  } else {  // the array's first or last bytes
    w.lo = w.hi = 0;
    for (int j = 0; j < 8; ++j)
      if (p + j >= base && p + j < base + bytes) {
        const uint32_t v = static_cast<uint32_t>(p[j]) << (8 * (j & 3));
        if (j < 4) w.lo |= v;
        else w.hi |= v;
      }
  }
  return w;
}
__device__ __forceinline__ uint32_t bytes_of(const TwoWords& w, const uint8_t* base, int64_t at) {
  return __funnelshift_r(w.lo, w.hi, 8 * (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(base + at)) & 3u));
}

// What one scale stage is made of, K blocks 4 g .. 4 g + 3: a word for each token row
// of a column (32 j + lane), and one for each 128-row block of W that the columns
// touch.  Bytes of a word past the last K block belong to the next row and are not
// selected by any product.
template <bool TOKENS_M>
struct ScaleWords {
  static constexpr int kTokens = TOKENS_M ? 4 : 8;  // columns of the tokens' side
  static constexpr int kBlocks = TOKENS_M ? 3 : 2;  // 224 (128) rows from a multiple of 32 on
  TwoWords t[kTokens], w[kBlocks];
  int t0, r0, g;                                    // first token, first row of W
};

// Each of the four warps writes the same words to its own quarter of the lanes:
// row r of A (or B) is lane r % 32, column r / 32, in every quarter.  The words of
// the next two stages are on their way while one is written: nothing but the store
// uses them, so a load's latency does not stand between two stages.
template <bool TOKENS_M>
__device__ __forceinline__ void scale_writer(const Params& p, const Smem& s, const Work& w, uint32_t tmem,
                                             uint32_t rank, int warp, int lane) {
  using Words = ScaleWords<TOKENS_M>;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const int groups = (p.kb + 3) / 4;
  const int last_block = (p.V + kRowsCta - 1) / kRowsCta - 1;
  const int64_t x_bytes = static_cast<int64_t>(p.T) * p.kb, w_bytes = static_cast<int64_t>(last_block + 1) * p.kb;
  const auto token_at = [&](const Words& r, int j) { return static_cast<int64_t>(r.t0 + 32 * j + lane) * p.kb + 4 * r.g; };
  const auto block_at = [&](const Words& r, int b) {
    return static_cast<int64_t>(min(r.r0 / kRowsCta + b, last_block)) * p.kb + 4 * r.g;
  };
  Slot at;
  int u = w.first, g = 0;  // of the next load
  const auto next = [&](Words& r) {
    if (u >= w.count) return false;
    const Unit un = unit_of<TOKENS_M>(p, w, u, rank);
    r.t0 = TOKENS_M ? un.row : un.n0;
    r.r0 = TOKENS_M ? un.n0 : un.row;
    r.g = g;
#pragma unroll
    for (int j = 0; j < Words::kTokens; ++j)
      if (r.t0 + 32 * j + lane < p.T && (TOKENS_M || 32 * j < p.n)) r.t[j] = load_words(p.sx, x_bytes, token_at(r, j));
#pragma unroll
    for (int b = 0; b < Words::kBlocks; ++b) r.w[b] = load_words(p.sw, w_bytes, block_at(r, b));
    if (++g == groups) g = 0, u += w.step;
    return true;
  };
  const auto put = [&](const Words& r) {
    if (!ptx::wait_bounded_cluster(s.scale_empty(at.i), at.phase ^ 1u, p.timeout_ns, s.abort_flag)) {
      give_up(p, s);
      return false;
    }
    uint32_t tw[Words::kTokens], ww[Words::kBlocks];
#pragma unroll
    for (int j = 0; j < Words::kTokens; ++j)  // rows past T meet zeros: any scale but NaN will do
      tw[j] = r.t0 + 32 * j + lane < p.T ? bytes_of(r.t[j], p.sx, token_at(r, j)) : 0x7f7f7f7fu;
#pragma unroll
    for (int b = 0; b < Words::kBlocks; ++b) ww[b] = bytes_of(r.w[b], p.sw, block_at(r, b));
    const int off = (r.r0 / 32) & 3;
    const auto block_word = [&](int j) {
      const int b = (off + j) >> 2;
      return b == 0 ? ww[0] : b == 1 ? ww[1] : ww[Words::kBlocks - 1];
    };
    ptx::tc_fence_after();
    __syncwarp();
    const uint32_t col = tmem + lanes + Form<TOKENS_M, false>::kBase + at.i * Form<TOKENS_M, false>::kCols;
    if constexpr (TOKENS_M) {
      ptx::tmem_st4(col, tw[0], tw[1], tw[2], tw[3]);
      const uint32_t b[8] = {block_word(0), block_word(1), block_word(2), block_word(3),
                             block_word(4), block_word(5), block_word(6), block_word(6)};
      ptx::tmem_st8(col + 8, b);
    } else {
      ptx::tmem_st4(col, block_word(0), block_word(1), block_word(2), block_word(3));
      ptx::tmem_st8(col + 8, tw);
    }
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_even(s.scale_full(at.i));
    at.next(kScaleStages);
    return true;
  };
  // Two sets of registers in turn: copying one to the other would wait for its loads.
  Words x, y;
  bool more_x = next(x), more_y = next(y);
  while (more_x) {
    if (!put(x)) return;
    more_x = next(x);
    if (!more_y || !put(y)) return;
    more_y = next(y);
  }
}

// All scale warps of the CTA: a barrier, and whether any thread passed true.
__device__ __forceinline__ bool scale_any(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %2, 0;\n\t"
      "bar.red.or.pred b, 5, %1, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "n"(32 * kScaleWarps), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

// The scale words of 4-bit weights, 16 bytes a row and stage.  They come from memory, where
// the operands ahead of them keep every load waiting for microseconds, so they are copied
// Ring4::kDepth - 1 stages ahead into shared memory, a quarter by each warp (W's words of K
// block j by warp j, the tokens' by columns), and every warp then writes all of them to its
// lanes; four stages before that they are fetched into L2 (1 x 2048 x 124,160: 50 us with the words
// loaded into registers two stages ahead; 93 x 4096 x 248,320: 121 us without the fetch, 109 with).
template <bool TOKENS_M>
__device__ __forceinline__ void scale_writer4(const Params& p, const Smem& s, const Work& w, uint32_t tmem,
                                              uint32_t rank, int warp, int lane) {
  using F = Form<TOKENS_M, true>;
  using R = Ring4<TOKENS_M>;
  constexpr int kMyTokens = (R::kTRows / 32 + kScaleWarps - 1) / kScaleWarps;
  const int part = warp & 3;
  const uint32_t lanes = static_cast<uint32_t>(part * 32) << 16;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(p.sw);
  const int groups = (p.kb + 3) / 4;
  const int64_t x_bytes = static_cast<int64_t>(p.T) * p.kb;
  const int w_cols = TOKENS_M ? p.n / 32 : kRowsCta / 32, t_cols = TOKENS_M ? kRowsCta / 32 : p.n / 32;
  uint32_t* ring = reinterpret_cast<uint32_t*>(s.ring);
  constexpr int kSlotWords = R::kBytes / 4;

  struct Next {
    TwoWords t[kMyTokens];
    int t0, g, slot;
    bool live = false;
  } held;
  int u = w.first, g = 0, slot = 0;  // of the next stage to copy, and the slot it goes to
  int ahead_u = w.first, ahead_g = 0;  // of the next stage to fetch into L2, four stages ahead of the copies
  for (int i = 0; i < 4 && ahead_u < w.count; ++i)
    if (++ahead_g == groups) ahead_g = 0, ahead_u += w.step;
  // W's words into the next slot; the tokens' into registers
  const auto copy = [&]() {
    if (ahead_u < w.count) {  // into L2, further ahead
      const Unit un = unit_of<TOKENS_M>(p, w, ahead_u, rank);
      const int row = (TOKENS_M ? un.n0 : un.row) + 32 * lane, b = 4 * ahead_g + part;
      if (lane < w_cols && row < p.V && b < p.kb)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(words + static_cast<int64_t>(b) * p.V + row));
      if (++ahead_g == groups) ahead_g = 0, ahead_u += w.step;
    }
    held.live = u < w.count;
    if (held.live) {
      const Unit un = unit_of<TOKENS_M>(p, w, u, rank);
      held.t0 = TOKENS_M ? un.row : un.n0;
      held.g = g;
      held.slot = slot;
      const int r0 = TOKENS_M ? un.n0 : un.row, b = 4 * g + part;
      const uint32_t to = ptx::smem_u32(ring + slot * kSlotWords + part * R::kWRows + lane);
#pragma unroll
      for (int c = 0; c < R::kWRows / 32; ++c) {
        const int row = r0 + 32 * c + lane;
        const bool in = row < p.V && b < p.kb && c < w_cols;
        const uint32_t* from = words + (in ? static_cast<int64_t>(b) * p.V + row : 0);
        // past V and K: zero bytes, a scale like any other
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 128 * c), "l"(from), "r"(in ? 4 : 0) : "memory");
      }
#pragma unroll
      for (int i = 0; i < kMyTokens; ++i) {
        const int c = part + kScaleWarps * i, t = held.t0 + 32 * c + lane;
        if (c < t_cols && t < p.T) held.t[i] = load_words(p.sx, x_bytes, static_cast<int64_t>(t) * p.kb + 4 * g);
      }
      if (++g == groups) g = 0, u += w.step;
      if (++slot == R::kDepth) slot = 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const auto put_tokens = [&]() {  // what copy() loaded, into its slot
    if (held.live) {
#pragma unroll
      for (int i = 0; i < kMyTokens; ++i) {
        const int c = part + kScaleWarps * i, t = held.t0 + 32 * c + lane;
        if (c < t_cols)  // rows past T meet zeros: any scale but NaN will do
          ring[held.slot * kSlotWords + 4 * R::kWRows + 32 * c + lane] =
              t < p.T ? bytes_of(held.t[i], p.sx, static_cast<int64_t>(t) * p.kb + 4 * held.g) : 0x7f7f7f7fu;
      }
      held.live = false;
    }
  };
  for (int i = 0; i < R::kDepth - 1; ++i) {
    copy();
    put_tokens();
  }

  // One stage a turn.  At its barrier every warp's part of the stage is in its slot, and the
  // slot of the turn before has been read by all: the stage kDepth - 1 turns on goes there.
  // Its tokens' words follow a turn later, when they have come (kDepth >= 3).
  static_assert(R::kDepth >= 3, "ring depth");
  Slot at;
  int from = 0, left = 0;
  for (int v = w.first; v < w.count; v += w.step) left += groups;
  for (; left > 0; --left) {
    const bool ok = ptx::wait_bounded_cluster(s.scale_empty(at.i), at.phase ^ 1u, p.timeout_ns, s.abort_flag);
    asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 2) : "memory");
    if (scale_any(!ok)) {
      give_up(p, s);
      break;
    }
    put_tokens();
    copy();
    const uint32_t* have = ring + from * kSlotWords + lane;
    uint32_t ww[4][R::kWRows / 32], tw[8] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < R::kWRows / 32; ++c) ww[j][c] = have[j * R::kWRows + 32 * c];
#pragma unroll
    for (int c = 0; c < R::kTRows / 32; ++c)
      if (c < t_cols) tw[c] = have[4 * R::kWRows + 32 * c];
    ptx::tc_fence_after();
    __syncwarp();
    const uint32_t col = tmem + lanes + F::kBase + at.i * F::kCols;
    if constexpr (TOKENS_M) {
      ptx::tmem_st4(col + F::a(0), tw[0], tw[1], tw[2], tw[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t b[8] = {ww[j][0], ww[j][1], ww[j][2], ww[j][3], ww[j][4], ww[j][5], ww[j][5], ww[j][5]};
        ptx::tmem_st8(col + F::b(j), b);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) ptx::tmem_st4(col + F::a(j), ww[j][0], ww[j][1], ww[j][2], ww[j][3]);
      ptx::tmem_st8(col + F::b(0), tw);
    }
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_even(s.scale_full(at.i));
    at.next(F::kStages);
    if (++from == R::kDepth) from = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Staging of 32 logits of 32 tokens: token rows of 64 (fp32: 128) bytes in the TMA's
// 64-byte (128-byte) swizzle, 16-byte piece k of row r at k ^ (r / 2 % 4) (k ^ r % 8).
template <typename E>
__device__ __forceinline__ uint32_t staged(uint32_t buf, int row, int piece) {
  if constexpr (sizeof(E) == 4)
    return buf + row * 128 + ((piece ^ (row & 7)) << 4);
  else
    return buf + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}

// Tokens on M: lane = token, column = logit.  Each lane writes its row in 16-byte
// pieces; the swizzle keeps the eight lanes of a phase on different banks.
template <typename E>
__device__ __forceinline__ void stage_tokens_m(uint32_t buf, const uint32_t (&r)[32], int lane) {
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      ptx::st_shared_v4(staged<E>(buf, lane, k), r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = ptx::pack_bf16x2(__uint_as_float(r[8 * k + 2 * i]), __uint_as_float(r[8 * k + 2 * i + 1]));
      ptx::st_shared_v4(staged<E>(buf, lane, k), h[0], h[1], h[2], h[3]);
    }
  }
}

// Vocabulary on M: lane = vocabulary row, column = token: one token's 32 logits at a
// time, 32 lanes on consecutive addresses.
template <typename E>
__device__ __forceinline__ void stage_vocab_m(uint32_t buf, const uint32_t (&r)[32], int lane) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if constexpr (sizeof(E) == 4)
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(staged<E>(buf, j, lane >> 2) + (lane & 3) * 4), "r"(r[j]) : "memory");
    else
      asm volatile("st.shared.b16 [%0], %1;" ::"r"(staged<E>(buf, j, lane >> 3) + (lane & 7) * 2),
                   "h"(__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(r[j]))))
                   : "memory");
  }
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// The staged box into rows of y that do not start on 16 bytes: tokens t0 .., logits
// v0 .. v0 + 31, clipped at T and V.  fp32: a token a step.  bf16: two tokens a step, a
// half warp each, in 32-bit words.  A half warp's rows are an even number of rows
// apart, so all of them start on an even element or all on an odd one; in the odd
// case the words are made of two staged ones.  The first or last logit that is left
// over goes alone, for all 32 tokens at once.
template <typename E>
__device__ __forceinline__ void store_rows(const Params& p, uint32_t buf, int t0, int v0, int lane) {
  const int tokens = p.T - t0, logits = min(32, p.V - v0);
  if constexpr (sizeof(E) == 4) {
    float* y = static_cast<float*>(p.y) + static_cast<int64_t>(t0) * p.ldy + v0 + lane;
    uint32_t v[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) v[r] = ld_shared_u32(staged<E>(buf, r, lane >> 2) + (lane & 3) * 4);
    if (lane < logits) {
#pragma unroll
      for (int r = 0; r < 32; ++r, y += p.ldy)
        if (r < tokens) *y = __uint_as_float(v[r]);
    }
  } else {
    const int w = lane & 15, half = lane >> 4, next = min(w + 1, 15);
    uint16_t* y = static_cast<uint16_t*>(p.y) + static_cast<int64_t>(t0 + half) * p.ldy + v0;
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(y) >> 1) & 1;
    const int e = 2 * w + odd;  // this lane's first logit
    uint32_t lo[16], hi[16];    // row 2 i + half
#pragma unroll
    for (int i = 0; i < 16; ++i)
      lo[i] = ld_shared_u32(buf + (2 * i + half) * 64 + (((w >> 2) ^ (i & 3)) << 4) + (w & 3) * 4);
    if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        hi[i] = ld_shared_u32(buf + (2 * i + half) * 64 + (((next >> 2) ^ (i & 3)) << 4) + (next & 3) * 4);
        hi[i] = odd ? __funnelshift_r(lo[i], hi[i], 16) : lo[i];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) lo[i] = hi[i];
    }
    y += e;
    if (e + 1 < logits) {
#pragma unroll
      for (int i = 0; i < 16; ++i, y += 2 * p.ldy)
        if (2 * i + half < tokens) *reinterpret_cast<uint32_t*>(y) = lo[i];
    }
    // the logits without a partner, a row per lane: the first where it starts odd, the last
    if (lane < tokens) {
      uint16_t* row = static_cast<uint16_t*>(p.y) + static_cast<int64_t>(t0 + lane) * p.ldy + v0;
      const int alone = static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1) & 1;
      const auto element = [&](int k) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(staged<E>(buf, lane, k >> 3) + (k & 7) * 2) : "memory");
        return v;
      };
      if (alone) row[0] = element(0);
      if (((logits - alone) & 1) && logits > alone) row[logits - 1] = element(logits - 1);
    }
  }
}

// The up to 14 bytes of each row that TMA leaves of a box: logits v_tma .. V - 1, a row
// per lane.  TMA stores whole 16-byte pieces, so a box clipped inside one would write
// zeros over what follows the row's last logit.
template <typename E>
__device__ __forceinline__ void store_tail(const Params& p, uint32_t buf, int t0, int v0, int lane) {
  if (t0 + lane >= p.T) return;
  E* y = static_cast<E*>(p.y) + static_cast<int64_t>(t0 + lane) * p.ldy;
  constexpr int kPiece = 16 / static_cast<int>(sizeof(E));
  for (int v = p.v_tma; v < p.V; ++v) {
    const int k = v - v0;
    const uint32_t a = staged<E>(buf, lane, k / kPiece) + (k % kPiece) * static_cast<int>(sizeof(E));
    if constexpr (sizeof(E) == 4) {
      y[v] = __uint_as_float(ld_shared_u32(a));
    } else {
      uint16_t h;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(a) : "memory");
      y[v] = __ushort_as_bfloat16(h);
    }
  }
}

// bf16, tokens on M, rows of y off 16 bytes (an odd vocabulary).  The two warps of a
// quarter put its 32 rows into shared memory whole, each as it lies in memory (its first
// byte d bytes into a 16-byte piece); then one warp has the copy engine store every row's
// whole pieces, and the other stores the up to 14 bytes before and behind them.  4189 x
// 224 x 226,081 takes 574 us, 2048 x 1024 x 50,257 90 us; with store_rows(), whose 64
// bytes of a row are three sectors, two of them partial, and 18 stores a box, 1177 and 119.
__device__ __forceinline__ uint32_t image_row(uint32_t image, int lane) { return image + lane * kImagePitch + (lane >> 3) * 16; }
__device__ __forceinline__ uint32_t image_offset(const Params& p, int token, int logit) {
  return (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.y)) +
          2u * (static_cast<uint32_t>(token) * static_cast<uint32_t>(p.ldy) + static_cast<uint32_t>(logit))) & 15u;
}
__device__ __forceinline__ void st_shared_u32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(v)) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}

// Columns c .. c + 31 of this lane's row, into its image that starts d bytes after `row`.
__device__ __forceinline__ void stage_image(uint32_t row, uint32_t d, int c, const uint32_t (&r)[32]) {
  uint32_t h[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) h[k] = ptx::pack_bf16x2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
  const bool odd = (d & 2u) != 0;  // words of columns 1 and 2, 3 and 4, ..
  const uint32_t at = row + d + 2 * c;
  const uint32_t words = at + (d & 2u);
#pragma unroll
  for (int k = 0; k < 15; ++k) st_shared_u32(words + 4 * k, odd ? __funnelshift_r(h[k], h[k + 1], 16) : h[k]);
  if (odd) {
    st_shared_u16(at, h[0]);
    st_shared_u16(at + 62, h[15] >> 16);
  } else {
    st_shared_u32(words + 60, h[15]);
  }
}

// The whole pieces of this lane's row (`bytes` long), `to` its first byte in memory less d.
__device__ __forceinline__ void store_pieces(uint32_t row, uint32_t d, uint32_t bytes, uint8_t* to) {
  const uint32_t begin = d ? 16u : 0u, end = (d + bytes) & ~15u;
  if (end > begin)
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to + begin), "r"(row + begin),
                 "r"(end - begin)
                 : "memory");
}
// And what lies around them, in words and one element at each end.
__device__ __forceinline__ void store_ends(uint32_t row, uint32_t d, uint32_t bytes, uint8_t* to) {
  const uint32_t te = d + bytes, tail = max(te & ~15u, d ? 16u : 0u);
  if (d & 2u) *reinterpret_cast<uint16_t*>(to + d) = static_cast<uint16_t>(ld_shared_u16(row + d));
  if (te & 2u) *reinterpret_cast<uint16_t*>(to + te - 2) = static_cast<uint16_t>(ld_shared_u16(row + te - 2));
#pragma unroll
  for (uint32_t k = 4; k < 16; k += 4)
    if (d && k >= d && k + 4 <= te) *reinterpret_cast<uint32_t*>(to + k) = ld_shared_u32(row + k);
#pragma unroll
  for (uint32_t k = 0; k < 12; k += 4)
    if (tail + k + 4 <= te) *reinterpret_cast<uint32_t*>(to + tail + k) = ld_shared_u32(row + tail + k);
}

// Both warps of a quarter of the lanes: a barrier, and whether any thread passed true.
__device__ __forceinline__ bool quarter_any(int q, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %2, 0;\n\t"
      "bar.red.or.pred b, %1, 64, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(1 + q), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

// A tile's rows through images, for store_images' two warps.
__device__ __forceinline__ void store_images(const Params& p, uint32_t image, const Unit& un, uint32_t col, int q, int part,
                                             int lane) {
  const int m0 = un.row + q * 32, token = m0 + lane;
  const uint32_t d = image_offset(p, token, un.n0), row = image_row(image, lane);
  const int logits = min(p.n, p.V - un.n0);
  if (part == 0) ptx::bulk_wait_read<0>();  // this lane's copy of the tile before
  quarter_any(q, false);                    // every row's, and its ends
#pragma unroll 1
  for (int c = 32 * part; c < logits; c += 64) {
    uint32_t r[32];
    ptx::tmem_ld32(col + c, r);
    ptx::tmem_wait_ld32(r);
    stage_image(row, d, c, r);
  }
  ptx::fence_proxy_async_smem();
  quarter_any(q, false);
  if (token < p.T) {
    uint8_t* to = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.y) + static_cast<int64_t>(token) * p.ldy + un.n0) - d;
    if (part == 0) store_pieces(row, d, 2u * static_cast<uint32_t>(logits), to);
    else store_ends(row, d, 2u * static_cast<uint32_t>(logits), to);
  }
  if (part == 0) ptx::bulk_commit();
  __syncwarp();
}

// A warp's 32 lanes x 32 columns at a time.
template <typename E, bool TOKENS_M, bool W4>
__device__ __forceinline__ void epilogue(const Params& p, const Smem& s, const Work& w, uint32_t tmem, uint32_t rank,
                                         int warp, int lane) {
  const int q = warp & 3, part = (warp - 2) >> 2;
  const uint32_t staging = ptx::smem_u32(s.staging) + (warp - 2) * kStagingWarp;
  constexpr bool kMayImage = TOKENS_M && sizeof(E) == 2;
  const bool images = kMayImage && !p.y_tma;
  Slot acc;
  uint32_t box = 0;
  for (int u = w.first; u < w.count; u += w.step) {
    const Unit un = unit_of<TOKENS_M>(p, w, u, rank);
    bool ok = ptx::wait_bounded_cluster(s.acc_full(acc.i), acc.phase, p.timeout_ns, s.abort_flag);
    if (images) ok = !quarter_any(q, !ok);  // its two warps meet at barriers: both go on, or neither
    if (!ok) {
      give_up(p, s);
      break;
    }
    __syncwarp();
    ptx::tc_fence_after();
    const uint32_t col = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc.i * Form<TOKENS_M, W4>::kAcc;
    const int m0 = un.row + q * 32;
    const int m_end = TOKENS_M ? p.T : p.V, n_end = TOKENS_M ? p.V : p.T;
    if (images) {
      if (m0 < m_end) store_images(p, ptx::smem_u32(s.staging) + q * kImageWarp, un, col, q, part, lane);
    } else if (q < un.boxes && m0 < m_end) {
#pragma unroll 1
      for (int c = 32 * part; c < p.n && un.n0 + c < n_end; c += 64) {
        uint32_t r[32];
        ptx::tmem_ld32(col + c, r);
        const int n0 = un.n0 + c;
        constexpr int kBoxes = kStagingWarp / (32 * 32 * static_cast<int>(sizeof(E)));
        const uint32_t buf = staging + (box % kBoxes) * (kStagingWarp / kBoxes);
        if (lane == 0) ptx::bulk_wait_read<kBoxes - 1>();  // the store that used this buffer has read it
        __syncwarp();
        ptx::tmem_wait_ld32(r);
        if constexpr (TOKENS_M)
          stage_tokens_m<E>(buf, r, lane);
        else
          stage_vocab_m<E>(buf, r, lane);
        if (p.y_tma) {
          const int v0 = TOKENS_M ? n0 : m0, t0 = TOKENS_M ? m0 : n0;
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (v0 + 32 <= p.v_tma) {
            if (lane == 0) {
              ptx::tma_store_2d(&p.tmY, buf, v0, t0);
              ptx::bulk_commit();
            }
          } else {
            if (lane == 0) {
              if (v0 < p.v_tma) ptx::tma_store_2d(&p.tmY, buf, v0, t0);
              ptx::bulk_commit();
            }
            store_tail<E>(p, buf, t0, v0, lane);
          }
        } else if constexpr (!kMayImage) {
          __syncwarp();
          store_rows<E>(p, buf, TOKENS_M ? m0 : n0, TOKENS_M ? n0 : m0, lane);
        }
        ++box;
      }
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_even(s.acc_empty(acc.i));
    acc.next(2);
  }
  if (lane == 0 || images) ptx::bulk_wait<0>();  // shared memory stays until the stores have read it
  __syncwarp();
}

// W4: the weights are 4-bit numbers.
template <bool TOKENS_M, bool W4, int STEP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem s;
  s.stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  s.staging = s.stages + p.stages * p.stage_bytes;
  s.ring = s.staging + p.staging_bytes;
  uint8_t* tail = s.ring + (W4 ? kRing4Bytes : 0);
  s.bars = reinterpret_cast<uint64_t*>(tail);
  s.tmem_slot = reinterpret_cast<uint32_t*>(tail + kBars * 8);
  s.abort_flag = reinterpret_cast<volatile int*>(tail + kBars * 8 + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const Work w = work_of<TOKENS_M>(p);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      ptx::mbar_init(s.full(i), 1);
      ptx::mbar_init(s.empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(s.acc_full(i), 1);
      ptx::mbar_init(s.acc_empty(i), 2 * kEpiWarps);
    }
    for (int i = 0; i < kScaleStages; ++i) {
      ptx::mbar_init(s.scale_full(i), 2 * kScaleWarps);
      ptx::mbar_init(s.scale_empty(i), 1);
    }
    ptx::mbar_init(s.drain(), 1);
    *s.abort_flag = 0;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&p.tmA);
    ptx::prefetch_tmap(&p.tmB);
    if (p.y_tma) ptx::prefetch_tmap(&p.tmY);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(s.tmem_slot), kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::launch_dependents();
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *s.tmem_slot;
  // Up to here nothing has touched global memory.
  ptx::wait_prerequisites();
  // The status of this call.  The first CTA is dispatched first and clears the word
  // before anything else; a wait that runs out does so a millisecond later at the
  // earliest.
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;

  if (warp == 0) {
    if (ptx::elect_one()) producer<TOKENS_M, W4, STEP>(p, s, w, rank);
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && ptx::elect_one()) mma_issuer<TOKENS_M, W4, STEP>(p, s, w, tmem);
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
    if (p.y_f32)
      epilogue<float, TOKENS_M, W4>(p, s, w, tmem, rank, warp, lane);
    else
      epilogue<__nv_bfloat16, TOKENS_M, W4>(p, s, w, tmem, rank, warp, lane);
    __syncwarp();
  } else {
    if constexpr (W4)
      scale_writer4<TOKENS_M>(p, s, w, tmem, rank, warp, lane);
    else
      scale_writer<TOKENS_M>(p, s, w, tmem, rank, warp, lane);
    __syncwarp();
  }

  // After an abort the odd CTA's loads may not have been consumed: give a TMA write
  // still in flight time to land before shared memory is released.
  if (warp == 0 && *s.abort_flag) {
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < kSettleNs) {
    }
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ quantising a matrix
// a [R, K] -> e4m3 values and one E8M0 byte per block of `rows` x 128, rows = 1 or 128
// (the scale rule of the norm's 8-bit output).  One CTA per 128 x 128 block: 16
// threads across a row, 16 rows at a time.
constexpr int kQuantThreads = 256;

template <typename E, bool SQUARE>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const E* a, int64_t lda, int64_t R, int K, uint8_t* q,
                                                                 uint8_t* qs) {
  constexpr int kSteps = 128 / (kQuantThreads / 16);
  __shared__ float red[kQuantThreads / 32];
  const int nb = (K + 127) / 128;
  const int64_t rb = blockIdx.x / nb;
  const int kb = static_cast<int>(blockIdx.x - rb * nb);
  const int c = kb * 128 + (threadIdx.x & 15) * kVec;
  const int64_t r0 = rb * 128 + (threadIdx.x >> 4);
  Raw8 raw[kSteps];  // as loaded: the unpacked floats of eight rows would halve the loads in flight
  float m[kSteps];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = r0 + i * (kQuantThreads / 16);
    if (r < R && c < K) raw[i] = load8(a + r * lda + c);
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    m[i] = 0.0f;
    if (r0 + i * (kQuantThreads / 16) < R && c < K) {
      float v[kVec];
      unpack8<E>(raw[i], v);
#pragma unroll
      for (int j = 0; j < kVec; ++j) m[i] = fmaxf(m[i], fabsf(v[j]));
    }
    amax = fmaxf(amax, m[i]);
  }
  if constexpr (SQUARE) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int i = 1; i < kQuantThreads / 32; ++i) amax = fmaxf(amax, red[i]);
    if (threadIdx.x == 0) qs[rb * nb + kb] = static_cast<uint8_t>(e8m0_of(amax));
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = r0 + i * (kQuantThreads / 16);
    float top = amax;
    if constexpr (!SQUARE) {
      top = m[i];
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    if (r < R && c < K) {
      const uint32_t e = e8m0_of(top);
      float v[kVec];
      unpack8<E>(raw[i], v);
      *reinterpret_cast<uint2*>(q + r * K + c) = to_e4m3x8(v, inv_scale(e));
      if (!SQUARE && (threadIdx.x & 15) == 0) qs[r * nb + kb] = static_cast<uint8_t>(e);
    }
  }
}

// a [R, K] -> packed e2m1 numbers [R, 64 kb], kb = ceil(K / 128), and one E8M0 byte per row
// and group of 32: the smallest 2^e with amax / 2^e <= 6 = 1.5 * 2^2, -126 <= e <= 125 (above,
// 6 * 2^e is no fp32 number: it saturates).  A group with a NaN in it gets the scale NaN,
// since e2m1 has none.  Rows are filled up to whole K blocks with zeros.
//
// Four threads to a group, 16 to a row's K block: the scales (q_scale [kb, R, 4]) of a
// warp's two rows are 8 consecutive bytes.  124,160 x 2048 bf16: 131 us for 643 MB, 72 % of the issue
// slots taken (weights are laid out once).
__device__ __forceinline__ uint32_t e8m0_of_e2m1(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0);
  return static_cast<uint32_t>(min(max(e, 1), 252));
}

// Eight floats to e2m1, round to nearest even, the first in the low bits.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&v)[kVec], float inv) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t b;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(b)
        : "f"(v[2 * i + 1] * inv), "f"(v[2 * i] * inv));
    r |= b << (8 * i);
  }
  return r;
}

constexpr int kQuant4Rows = kQuantThreads / 16;  // rows of a step
constexpr int kQuant4Steps = 8;

template <typename E>
__global__ void __launch_bounds__(kQuantThreads) quantize_fp4_kernel(const E* a, int64_t lda, int64_t R, int K, uint32_t* q,
                                                                     uint8_t* qs) {
  const int kb = (K + 127) / 128;
  const int64_t rb = blockIdx.x / kb;
  const int b = static_cast<int>(blockIdx.x - rb * kb);
  const int piece = threadIdx.x & 15, c = b * 128 + piece * kVec;
  const int64_t r0 = rb * (kQuant4Rows * kQuant4Steps) + (threadIdx.x >> 4);
  Raw8 raw[kQuant4Steps];
#pragma unroll
  for (int i = 0; i < kQuant4Steps; ++i) {
    const int64_t r = r0 + i * kQuant4Rows;
    if (r < R && c < K) raw[i] = load8(a + r * lda + c);
  }
#pragma unroll
  for (int i = 0; i < kQuant4Steps; ++i) {
    const int64_t r = r0 + i * kQuant4Rows;
    float v[kVec] = {};
    if (r < R && c < K) unpack8<E>(raw[i], v);
    float amax = 0.0f;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      amax = fmaxf(amax, fabsf(v[j]));
      nan = nan || v[j] != v[j];
    }
    uint32_t bits = nan ? 0x7fffffffu : __float_as_uint(amax);  // the largest bits of all
    bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
    bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 2));
    nan = bits > 0x7f800000u;
    const uint32_t e = e8m0_of_e2m1(__uint_as_float(nan ? 0u : bits));
    const uint32_t codes = nan ? 0u : to_e2m1x8(v, inv_scale(e));
    if (r < R) {
      q[(r * kb + b) * 16 + piece] = codes;
      if ((piece & 3) == 0) qs[(static_cast<int64_t>(b) * R + r) * 4 + (piece >> 2)] = static_cast<uint8_t>(nan ? 255u : e);
    }
  }
}

}  // namespace fp8
}  // namespace flce
