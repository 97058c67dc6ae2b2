// Products of rows and weights in e4m3 with a scale for every block of 128, on the tensor cores (tcgen05).
//
//   D[m, n] = sum over blocks b of 128 of  sa[b, m] * sb[b, n] * sum_{k in b} A[m, k] B[n, k]
//
// The tensor cores sum one block of 128 in fp32 (products of two e4m3 are exact there); since its scales differ
// from the next block's, every block's sum leaves TMEM, is multiplied by its scales and added to fp32
// accumulators in registers.  That costs a fused multiply-add and a TMEM read for every 128 multiply-adds of the
// tensor cores, on other units and by other warps, so it runs beside them: TMEM holds several blocks' sums.
//
// One persistent CTA per SM on tiles of 128 x 256, or of 128 x 128 where those are few.  384 threads:
//   warp 0      TMA producer (a ring of S stages, 128 rows x 128 bytes of A, 128 or 256 of B)
//   warp 1      issues the MMAs, four to a block, into the next of NB sums in TMEM
//   warps 2, 3  bring the scales into shared memory (alternate blocks), multiplied where they go together
//   warps 4-11  take the sums: a thread a row (TMEM lane) of half of the columns; then the epilogue
// Operands whose contraction runs down the rows of memory (the weights in the rows' gradient, both operands in the
// weights' gradient) are MN-major: the same 128 x 128 boxes under another descriptor, so nothing is transposed in
// memory and the weights are kept once.
// Items are (tile, part of the contraction) in a fixed order; a product of few tiles is split, the parts' sums kept
// in `partial` and added in order by whichever CTA finishes the tile: the same bits every time.
// Every wait is bounded by the call's limit: when one gives up, all roles stop, copies and MMAs in flight are
// waited for (at most kDrain each), TMEM is freed and the device's status word gets a bit.
//
// Measured on one GB300 (this kernel alone): 8192 tokens, two of eight experts of 14336 x 4096, 0.71 ms (2.7 PFLOP/s, 1.4
// of cuBLAS bf16; tensor pipe busy 0.61); its gradients, 0.82 ms for the rows and 1.41 ms for the weights; one token, two
// experts of 4096 x 14336 x 2, 44 us (5.3 TB/s).  What bounds wide tiles is the way of a block's sum: the takers need about
// 500 cycles for it beside the tensor cores (their multiply-adds 320, reads of TMEM 240, on one port), waits on barriers
// 200 more, as shared memory is busy with operands: 48 KB written and 48 read a block, 750 cycles at 128 bytes a cycle.
// The weights' gradient multiplies twice for every value (1000 cycles a block) and writes 4 or 2 bytes a weight.  Narrow
// tiles are bound by HBM and the same waits.
#pragma once

#include <mutex>

#include "fp8_internal.cuh"
#include "tcgen05_ptx.cuh"

namespace colibri {
namespace fp8 {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168, kOtherRegs = 88, kTakerRegs = 208;  // of a thread
static_assert(128 * kOtherRegs + 256 * kTakerRegs <= kThreads * kLaunchRegs, "a warpgroup's share comes out of the launch's");
constexpr int kTakers = 8, kTaker0 = 4;       // warps that take the sums
constexpr int kTileBytes = 128 * 128;         // an operand's 128 rows (or columns) of a block
constexpr int kBoxBytes = 32 * 128;           // the smallest box of rows
constexpr int kStageLd = 12;                  // epilogue staging: 32 rows of 8 words a warp, and 4 between
constexpr Fp8Limit kDrain = {50000000, 63};   // 50 ms, far above the time of a copy or of a stage's MMAs

constexpr int MT = 128;                       // tile rows

template <int FORM>
struct Form {
  static constexpr int NT = FORM == kFp8Narrow ? 128 : 256;  // tile columns
  static constexpr int kB = NT * 128;                        // bytes of a block of theirs
  static constexpr int C = NT / 2;             // columns of a taker thread
  static constexpr int NB = 512 / NT;          // sums in TMEM
  static constexpr int S = FORM == kFp8Wide ? 4 : 6;
  // Blocks whose scales are in shared memory.  Those of block j are written once the MMAs of block j - S are done, which
  // began when the sum of block j - S - NB had been taken: S + NB slots are never written while they are read.
  static constexpr int SF = S + NB;
  static constexpr int kScales = 128 + NT;  // of a slot: a row's (with the weights'), and a second one or the columns'
  static constexpr int kBars = 2 * S + 2 * NB + 3;
  static constexpr int kSmem = 1024 + S * (kTileBytes + kB) + SF * kScales * 4 + kTakers * 32 * kStageLd * 4 + kBars * 8 + 32 +
                               4 * (3 * kFp8MaxExperts + 1);
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

// Waits for the phase of `bar` with parity `parity`, at most limit.ns or until *abort.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, Fp8Limit limit) {
  uint64_t t0 = 0;
  for (uint32_t tries = 1;; ++tries) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((tries & limit.clock_mask) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort || now - t0 > limit.ns) return false;
    }
  }
}

// Box of an expert's matrix (z, y, x).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// MN-major operand of 128 rows of the contraction x 128 columns, as a box with the 128-byte swizzle leaves it: atoms of
// 8 rows x 128 bytes, the next eight rows 1024 bytes on (a second 128 columns would be kTileBytes on).
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kTileBytes >> 4) << 16;  // next columns
  d |= static_cast<uint64_t>(1024 >> 4) << 32;        // next 8 rows
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// e4m3 x e4m3 -> fp32, m x n.
constexpr uint32_t idesc(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0) | (b_mn ? 1u << 16 : 0) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t more) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(more)
      : "memory");
}

// Two fp32 in one register pair.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t two(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm volatile("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void one_each(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t x, uint64_t f) {
  asm volatile("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(x), "l"(f));
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t f) {
  uint64_t r;
  asm volatile("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(f));
  return r;
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// 32 TMEM lanes x 16 columns; to be read after tmem_wait().
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr)
               : "memory");
}
// 16 TMEM lanes x 32 columns, a thread two neighbouring columns of every eight, of two lanes: r[4 i] and r[4 i + 1] are
// lane l / 4 of columns 8 i + 2 (l % 4) and the next, r[4 i + 2] and r[4 i + 3] those of lane l / 4 + 8.
__device__ __forceinline__ void tmem_ld_spread(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// silu(v) u as it is stored: fast exp and quotient for bf16; for fp32 expf of what cannot overflow and the
// approximate reciprocal, good to an ulp, of a sum between 1 and 2.
template <typename O>
__device__ __forceinline__ float gated_value(float v, float u) {
  if constexpr (sizeof(O) == 2) return silu_fast(v) * u;
  const float t = expf(-fabsf(v));
  float s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + t));
  return v * (v < 0.f ? t * s : s) * u;
}

struct Item {
  int i;               // item number
  int tile, part;
  int e, row, n;       // expert, first row, rows of the tile
  int col;             // first column of the tile (of y)
  int kb0, kb1;        // blocks of the contraction
  int first;           // kFp8Weights: the expert's first block of rows
};

template <int MODE, int FORM, bool GATED, typename O>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_mma_kernel(const __grid_constant__ Fp8Maps tm, const __grid_constant__ Fp8Args a) {
  using F = Form<FORM>;
  constexpr int S = F::S, NB = F::NB, NT = F::NT, C = F::C;
  constexpr bool kWeights = MODE == kFp8Weights, kFromWeights = !kWeights;  // whether B is the weights
  static_assert(!GATED || MODE == kFp8Forward);
  constexpr int kCh = GATED ? NT / 2 : NT;  // columns of y in a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_a = smem;
  uint8_t* s_b = s_a + S * kTileBytes;
  float* s_scale = reinterpret_cast<float*>(s_b + S * F::kB);
  float* s_stage = s_scale + F::SF * F::kScales;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_stage + kTakers * 32 * kStageLd);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + F::kBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_last = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* s_row0 = reinterpret_cast<int*>(tmem_slot + 8);  // first row of each expert
  int* s_rows = s_row0 + kFp8MaxExperts;                // its rows
  int* s_tiles = s_rows + kFp8MaxExperts;               // row tiles (kFp8Weights: blocks of rows) before it [E + 1]

  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S;
  const uint32_t tfull0 = empty0 + 8 * S, tempty0 = tfull0 + 8 * NB;
  const uint32_t drain = tempty0 + 8 * NB, joined = drain + 8, decided = joined + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full0 + 8 * i, 2);  // A and B landed, the scales are there
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(tfull0 + 8 * i, 1);
      mbar_init(tempty0 + 8 * i, kTakers);
    }
    mbar_init(drain, 1);
    mbar_init(joined, kTakers);
    mbar_init(decided, 1);
    *s_abort = 0;
    fence_mbar_init();
    for (int i = 0; i < kFp8TokMaps; ++i) prefetch_tmap(&tm.a[i]);
    prefetch_tmap(&tm.b);
    if constexpr (GATED) prefetch_tmap(&tm.b3);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // The quantiser lets this kernel start once everything before it is done: offsets and weights may be read at once;
  // the warps that read its rows and scales wait for it.
  if (warp == 2)
    fp8_segments(a.offsets, a.E, a.R, lane, s_row0, s_rows, s_tiles,
                 [](int n) { return kWeights ? (n + kFp8Block - 1) / kFp8Block : (n + MT - 1) / MT; });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int out_cols = MODE == kFp8Forward ? a.N : a.K;  // of y
  const int col_tiles = (out_cols + kCh - 1) / kCh;
  const int m_tiles = (a.N + MT - 1) / MT;               // kFp8Weights
  const int kblocks = ((MODE == kFp8Forward ? a.K : a.N) + kFp8Block - 1) / kFp8Block;  // not kFp8Weights
  const int64_t tiles = kWeights ? (int64_t)a.E * m_tiles * col_tiles : (int64_t)s_tiles[a.E] * col_tiles;
  const int units = gridDim.x, unit = blockIdx.x;
  // Parts of the contraction: the number that leaves the SMs least idle in the last wave, a little against more parts.
  int parts = 1;
  if (tiles < 2 * (int64_t)units) {
    const int most = kWeights ? max(1, (a.R + kFp8Block - 1) / kFp8Block) : kblocks;
    float least = 1e30f;
    for (int p = 1; p <= kFp8MaxSplits && p <= most && tiles * p <= a.max_items; ++p) {
      const int waves = (int)((tiles * p + units - 1) / units);
      const float cost = (float)waves / p + (p > 1 ? 0.04f : 0.f) + 0.01f * p;
      if (cost < least) least = cost, parts = p;
    }
  }
  const int items = (int)(tiles * parts);  // y itself has more bytes

  // item -> its tile: row tiles of an expert fastest, so that CTAs at work share the other operand in L2
  auto item_at = [&](int i) {
    Item it;
    it.i = i;
    it.tile = i / parts;
    it.part = i - it.tile * parts;
    int blocks = kblocks;
    if constexpr (kWeights) {
      const int each = m_tiles * col_tiles;
      it.e = it.tile / each;
      const int local = it.tile - it.e * each;
      it.col = local / m_tiles * kCh;
      it.row = local % m_tiles * MT;  // of d_w's N rows
      it.n = min(a.N - it.row, MT);
      it.first = s_tiles[it.e];
      blocks = s_tiles[it.e + 1] - it.first;
    } else {
      int lo = 0, hi = a.E;  // the last expert whose tiles begin at or before it (those without rows begin with it)
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if ((int64_t)s_tiles[mid] * col_tiles <= it.tile)
          lo = mid;
        else
          hi = mid;
      }
      it.e = lo;
      const int tt = s_tiles[lo + 1] - s_tiles[lo], local = it.tile - s_tiles[lo] * col_tiles;
      it.col = local / tt * kCh;
      const int t = local % tt, n = s_rows[lo];
      const int each = ((n + tt - 1) / tt + 31) / 32 * 32;  // even tiles, whole boxes
      it.row = s_row0[lo] + t * each;
      it.n = min(each, n - t * each);
      it.first = 0;
    }
    it.kb0 = (int)((int64_t)blocks * it.part / parts);
    it.kb1 = (int)((int64_t)blocks * (it.part + 1) / parts);
    return it;
  };

  bool ok = true;
  if (warp < kTaker0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      const bool elected = elect_one();
      const uint32_t a0 = smem_u32(s_a), b0 = smem_u32(s_b);
      auto boxes_of = [](const Item& t) { return kWeights ? 4 : (t.n + 31) / 32; };
      auto arm = [&](uint32_t st, int boxes) {
        mbar_arrive_expect_tx(full0 + 8 * st, F::kB + boxes * kBoxBytes);
      };
      auto load_b = [&](const Item& t, int kb, uint32_t st) {
        const uint32_t full = full0 + 8 * st, dst = b0 + st * F::kB;
        const int k = kb * kFp8Block;
        if constexpr (kWeights) {
#pragma unroll
          for (int r = 0; r < F::kB / kTileBytes; ++r)
            tma_load_2d(dst + r * kTileBytes, &tm.b, full, t.col + r * 128, (t.first + kb) * kFp8Block);
        } else if constexpr (MODE == kFp8Rows) {
#pragma unroll
          for (int r = 0; r < F::kB / kTileBytes; ++r)
            tma_load_3d(dst + r * kTileBytes, &tm.b, full, t.col + r * 128, k, t.e);
        } else if constexpr (GATED) {
          // every taker thread's columns: C / 2 channels of w, then the same of w3
          constexpr int kBytes = C / 2 * 128;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int ch = t.col + r * (C / 2);
            tma_load_3d(dst + 2 * r * kBytes, &tm.b, full, k, ch, t.e);
            tma_load_3d(dst + (2 * r + 1) * kBytes, &tm.b3, full, k, ch, t.e);
          }
        } else {
#pragma unroll
          for (int r = 0; r < F::kB / kTileBytes; ++r)
            tma_load_3d(dst + r * kTileBytes, &tm.b, full, k, t.col + r * 128, t.e);
        }
      };
      auto load_a = [&](const Item& t, int kb, uint32_t st, int boxes) {
        const uint32_t full = full0 + 8 * st;
        uint32_t dst = a0 + st * kTileBytes;
        if constexpr (kWeights) {
          tma_load_2d(dst, &tm.a[2], full, t.row, (t.first + kb) * kFp8Block);
        } else {
          int row = t.row;
#pragma unroll
          for (int b = kFp8TokMaps - 1; b >= 0; --b)  // at most one copy of each box height
            if (boxes >> b & 1) {
              tma_load_2d(dst, &tm.a[b], full, kb * kFp8Block, row);
              dst += kBoxBytes << b, row += 32 << b;
            }
        }
      };
      // Weights do not hang on the quantiser: those of the first stages are on their way while it runs.
      uint32_t early = 0;
      if (kFromWeights && unit < items) {
        const Item t = item_at(unit);
        early = min(S, t.kb1 - t.kb0);
        for (uint32_t st = 0; st < early; ++st) {
          if (elected) {
            arm(st, boxes_of(t));
            load_b(t, t.kb0 + st, st);
          }
          __syncwarp();
        }
      }
      pdl_wait();
      uint32_t it = 0, st = 0, ph = 0;
      for (int i = unit; ok && i < items; i += units) {
        const Item t = item_at(i);
        const int boxes = boxes_of(t);
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          if (!__all_sync(~0u, wait_for(empty0 + 8 * st, ph ^ 1, s_abort, a.limit))) {
            ok = false;
            break;
          }
          if (elected) {
            if (it >= early) {
              arm(st, boxes);
              load_b(t, kb, st);
            }
            load_a(t, kb, st, boxes);
          }
          __syncwarp();
          if (++st == S) st = 0, ph ^= 1;
        }
      }
      if (!ok && lane == 0) *s_abort = 1;
      // Every copy has landed before the CTA can leave.  After a wait that gave up a stage may lack its other operand or its
      // scales: the wait for it ends by kDrain.
      volatile int never = 0;
      it = max(it, early);
      for (uint32_t j = it > S ? it - S : 0; j < it; ++j) wait_for(full0 + 8 * (j % S), j / S & 1, &never, kDrain);
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------------- MMA issuer
      constexpr uint32_t id = idesc(MT, NT, kWeights, MODE != kFp8Forward);
      constexpr int kStepA = kWeights ? 4096 >> 4 : 2, kStepB = MODE != kFp8Forward ? 4096 >> 4 : 2;  // 32 of the block
      const bool elected = elect_one();
      const uint64_t da0 = kWeights ? mn_desc(smem_u32(s_a)) : sw128_desc(smem_u32(s_a));
      const uint64_t db0 = MODE != kFp8Forward ? mn_desc(smem_u32(s_b)) : sw128_desc(smem_u32(s_b));
      uint32_t st = 0, ph = 0, buf = 0, bph = 0;
      for (int i = unit; ok && i < items; i += units) {
        const Item t = item_at(i);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          bool got = wait_for(tempty0 + 8 * buf, bph ^ 1, s_abort, a.limit);
          got = got && wait_for(full0 + 8 * st, ph, s_abort, a.limit);
          if (!__all_sync(~0u, got)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = da0 + st * (kTileBytes >> 4), db = db0 + st * (F::kB >> 4);
          if (elected) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma(tmem_base + buf * NT, da + k * kStepA, db + k * kStepB, id, k != 0);
            umma_commit(empty0 + 8 * st);
            umma_commit(tfull0 + 8 * buf);
          }
          __syncwarp();
          if (++st == S) st = 0, ph ^= 1;
          if (++buf == NB) buf = 0, bph ^= 1;
        }
      }
      if (!ok && lane == 0) *s_abort = 1;
      if (elected) {
        umma_commit(drain);  // completes when every MMA of this thread has
        volatile int never = 0;
        wait_for(drain, 0, &never, kDrain);
      }
      __syncwarp();
    } else {
      // -------------------------------------------------------------- scales
      pdl_wait();
      const int kb_w = (a.K + kFp8Block - 1) / kFp8Block, nb_w = (a.N + kFp8Block - 1) / kFp8Block;  // the weights' blocks
      uint32_t it = 0;  // block number over all items; this warp has those of its parity
      for (int i = unit; ok && i < items; i += units) {
        const Item t = item_at(i);
        const int n = t.kb1 - t.kb0, last = max(t.n - 1, 0);
        // four rows a lane; a tile past the last row or column takes the last one's
        const float* sa = a.a_scale + (int64_t)(t.first + t.kb0) * a.lda + t.row;
        int m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = min(lane + 32 * j, last);
        if (t.n == 0) sa = a.a_scale;  // nothing of it is used
        const float *w0 = nullptr, *w1 = nullptr;  // of the tile's two halves, or of the two projections
        int64_t w_step = 0;
        if constexpr (kFromWeights) {
          const int c0 = t.col / kFp8Block, c1 = GATED || NT == 128 ? c0 : c0 + 1;
          const int most = (MODE == kFp8Forward ? nb_w : kb_w) - 1;
          auto at = [&](int c) {
            return MODE == kFp8Forward ? ((int64_t)t.e * nb_w + min(c, most)) * kb_w + t.kb0
                                       : ((int64_t)t.e * nb_w + t.kb0) * kb_w + min(c, most);
          };
          w0 = a.w_scale + at(c0), w1 = (GATED ? a.w3_scale : a.w_scale) + at(c1);
          w_step = MODE == kFp8Forward ? 1 : kb_w;
        }
        constexpr int kAhead = 4;  // of this warp's blocks whose loads are on their way
        float fa[kAhead][4], f0[kAhead], f1[kAhead], fx[kAhead][kWeights ? NT / 32 : 1];
        auto fetch = [&](int k, int kb) {
          if (kb >= n) return;
#pragma unroll
          for (int j = 0; j < 4; ++j) fa[k][j] = sa[kb * a.lda + m[j]];
          if constexpr (kFromWeights) f0[k] = w0[kb * w_step], f1[k] = w1[kb * w_step];
          if constexpr (kWeights) {
#pragma unroll
            for (int j = 0; j < NT / 32; ++j)
              fx[k][j] = a.x_scale[(int64_t)(t.first + t.kb0 + kb) * a.ldx + t.col + lane + 32 * j];
          }
        };
        const int odd = (it ^ warp) & 1;  // the first of this warp's blocks in the item
#pragma unroll
        for (int k = 0; k < kAhead; ++k) fetch(k, odd + 2 * k);
        for (int kb0 = odd; ok && kb0 < n; kb0 += 2 * kAhead) {
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int kb = kb0 + 2 * k;
            if (kb >= n) break;
            const uint32_t j = it + kb, st = j % S;
            if (!__all_sync(~0u, wait_for(empty0 + 8 * st, (j / S & 1) ^ 1, s_abort, a.limit))) {
              ok = false;
              break;
            }
            float* slot = s_scale + j % F::SF * F::kScales;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              slot[lane + 32 * r] = kFromWeights ? fa[k][r] * f0[k] : fa[k][r];
              if constexpr (kFromWeights && (GATED || NT == 256)) slot[128 + lane + 32 * r] = fa[k][r] * f1[k];
            }
            if constexpr (kWeights) {
#pragma unroll
              for (int r = 0; r < NT / 32; ++r) {  // in the order that the takers' threads read them
                const int c = (lane + 32 * r) % C;
                slot[128 + (lane + 32 * r - c) + (c % 8 / 2) * (C / 4) + c / 8 * 2 + c % 2] = fx[k][r];
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(full0 + 8 * st);
            fetch(k, kb + 2 * kAhead);
          }
        }
        it += n;
      }
      if (!ok && lane == 0) *s_abort = 1;
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------------- takers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTakerRegs));
    pdl_wait();
    const int q = warp & 3, half = (warp - kTaker0) >> 2;  // TMEM lanes 32 q .. of columns half * C ..
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    uint32_t* stage = reinterpret_cast<uint32_t*>(s_stage) + (warp - kTaker0) * (32 * kStageLd);
    uint32_t buf = 0, bph = 0, sf = 0, joins = 0;
    for (int i = unit; ok && i < items; i += units) {
      bool mine;  // whether any of this warp's rows exist
      int left;   // blocks to go
      {
        const Item t = item_at(i);
        mine = q * 32 < t.n, left = t.kb1 - t.kb0;
      }
      uint64_t acc[C / 2];
#pragma unroll
      for (int c = 0; c < C / 2; ++c) acc[c] = 0;
      bool ready = false;  // the next sum was seen to be there
#pragma unroll 1
      for (; left > 0; --left) {
        if (!ready && !__all_sync(~0u, wait_for(tfull0 + 8 * buf, bph, s_abort, a.limit))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t from = tmem_base + lanes + buf * NT + half * C, freed = tempty0 + 8 * buf;
        const float* scale = s_scale + sf * F::kScales;
        if (++buf == NB) buf = 0, bph ^= 1;
        if (++sf == F::SF) sf = 0;
        if (mine) {
          if constexpr (kWeights) {
            // A scale for every column as well.  With a row a thread each would have to read all of them, and reads of shared
            // memory wait for the tensor cores' (2150 cycles a block against 500 without); with columns spread over four
            // threads an eighth of the reads do.
            uint64_t fr[4];  // of rows lane / 4 + 8 g
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float f = scale[q * 32 + lane / 4 + 8 * g];
              fr[g] = two(f, f);
            }
            const float4* x4 = reinterpret_cast<const float4*>(scale + 128 + half * C + (lane & 3) * (C / 4));
#pragma unroll
            for (int c0 = 0; c0 < C; c0 += 32) {
              const float4 x[2] = {x4[c0 / 16], x4[c0 / 16 + 1]};
#pragma unroll
              for (int h = 0; h < 2; ++h) {  // 16 rows
                uint32_t u[16];
                tmem_ld_spread(from + (static_cast<uint32_t>(16 * h) << 16) + c0, u);
                tmem_wait();
                if (c0 + 32 == C && h == 1) {
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(freed);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float4 xi = x[i / 2];
                  const uint64_t fx = i & 1 ? two(xi.z, xi.w) : two(xi.x, xi.y);
#pragma unroll
                  for (int g = 0; g < 2; ++g)
                    fma2(acc[((2 * h + g) * C + c0 + 8 * i) / 8], mul2(two(u[4 * i + 2 * g], u[4 * i + 2 * g + 1]), fx),
                         fr[2 * h + g]);
                }
              }
            }
          } else {
            // the weights' block is the half's, or that of one of the projections
            const float f0 = scale[(kFromWeights && NT == 256 && !GATED ? half * 128 : 0) + q * 32 + lane];
            const float f1 = GATED ? scale[128 + q * 32 + lane] : 0.f;
            // 16 columns at a time: larger pieces, or one behind another on its way, cost more in moves between registers than
            // they hid (8192 tokens, 14336 x 4096: 0.87 to 1.5 ms against 0.80).  Everything from the load to the products is
            // volatile, so that none of it moves above the wait.
#pragma unroll
            for (int c0 = 0; c0 < C; c0 += 16) {
              uint32_t u[16];
              tmem_ld(from + c0, u);
              tmem_wait();
              if (c0 + 16 == C) {  // this warp has its values: the sum may be overwritten
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(freed);
              }
              const float f = GATED && c0 >= C / 2 ? f1 : f0;
              const uint64_t ff = two(f, f);
#pragma unroll
              for (int c = 0; c < 16; c += 2) fma2(acc[(c0 + c) / 2], two(u[c], u[c + 1]), ff);
            }
          }
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(freed);
        }
        ready = left > 1 && __all_sync(~0u, mbar_test(tfull0 + 8 * buf, bph));
      }
      if (!ok) {
        if (lane == 0) *s_abort = 1;
        break;
      }
      int again = i;
      asm volatile("" : "+r"(again));  // its coordinates are computed again rather than held in registers above
      const Item t = item_at(again);
      float v[C];
#pragma unroll
      for (int c = 0; c < C / 2; ++c) one_each(acc[c], v[2 * c], v[2 * c + 1]);
      if (parts > 1) {
        const int64_t at = (int64_t)(half * C) * 128 + q * 32 + lane;
        if (mine) {
          float* part = a.partial + (int64_t)t.i * (NT * 128) + at;
#pragma unroll
          for (int c = 0; c < C; ++c) part[c * 128] = v[c];
        }
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(joined);
        bool got = true;
        if (warp == kTaker0 && lane == 0) {
          got = wait_for(joined, joins & 1, s_abort, a.limit);
          if (got) {
            __threadfence();
            *s_last = atomicAdd(&a.ticket[t.tile], 1u) == (uint32_t)(parts - 1);
            mbar_arrive(decided);
          }
        }
        __syncwarp();
        got = got && wait_for(decided, joins & 1, s_abort, a.limit);
        ++joins;
        if (!__all_sync(~0u, got)) {
          if (lane == 0) *s_abort = 1;
          ok = false;
          break;
        }
        if (!*s_last) continue;
        __threadfence();
        if (mine) {
          const float* all = a.partial + (int64_t)t.tile * parts * (NT * 128) + at;
#pragma unroll
          for (int c = 0; c < C; ++c) v[c] = 0.f;
          for (int p = 0; p < parts; ++p)
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] += __ldcg(all + (int64_t)p * (NT * 128) + c * 128);
        }
      }
      if (!mine) continue;
      if constexpr (kWeights) {
        // Four threads hold eight columns of a row, two each.  They trade, so that each has 16 bytes of one row: in fp32
        // half of one of two runs of eight columns, in bf16 all of one of four (stores of 4 bytes: 16384 rows, 8 x 4096
        // x 14336 in bf16, 1.57 ms against 1.42).
        const int64_t row = (int64_t)t.e * a.N + t.row + q * 32 + lane / 4;
        const int rows = t.n - q * 32 - lane / 4;  // from this thread's first one on
        O* y = static_cast<O*>(a.y) + row * out_cols;
        constexpr int kRuns = 16 / (2 * sizeof(O));  // runs of eight columns traded at once
        const bool odd = lane & 1, high = lane & 2;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
          for (int j = 0; j < C / 8; j += kRuns) {
            const float* from = v + 2 * (g * C / 8 + j);
            uint4 out;
            int col = t.col + half * C + 8 * j;
            if constexpr (sizeof(O) == 4) {
              const float a0 = __shfl_xor_sync(~0u, odd ? from[0] : from[2], 1);
              const float a1 = __shfl_xor_sync(~0u, odd ? from[1] : from[3], 1);
              const float k0 = odd ? from[2] : from[0], k1 = odd ? from[3] : from[1];
              out = make_uint4(__float_as_uint(odd ? a0 : k0), __float_as_uint(odd ? a1 : k1), __float_as_uint(odd ? k0 : a0),
                               __float_as_uint(odd ? k1 : a1));
              col += (odd ? 8 : 0) + (high ? 4 : 0);
            } else {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = pack_bf16(from[2 * i], from[2 * i + 1]);
              const uint32_t r0 = __shfl_xor_sync(~0u, odd ? w[0] : w[1], 1), r2 = __shfl_xor_sync(~0u, odd ? w[2] : w[3], 1);
              const uint32_t a0 = odd ? r0 : w[0], a1 = odd ? w[1] : r0, a2 = odd ? r2 : w[2], a3 = odd ? w[3] : r2;
              const uint32_t s0 = __shfl_xor_sync(~0u, high ? a0 : a2, 2), s1 = __shfl_xor_sync(~0u, high ? a1 : a3, 2);
              out = high ? make_uint4(s0, s1, a2, a3) : make_uint4(a0, a1, s0, s1);
              col += 8 * (lane & 3);
            }
            if (8 * g < rows && col < out_cols)  // K is a multiple of 16: a thread's columns are inside together
              *reinterpret_cast<uint4*>(y + (int64_t)(8 * g) * out_cols + col) = out;
          }
        }
        continue;
      }
      // 32 bytes of every row at a time through shared memory, so that stores cover whole sectors of a row
      constexpr int kOut = GATED ? C / 2 : C, kCols = 32 / sizeof(O);
      const int rows = min(t.n - q * 32, 32);
      O* y = static_cast<O*>(a.y) + (int64_t)(t.row + q * 32) * out_cols;
      const bool wide = out_cols % (kCols / 2) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
#pragma unroll
      for (int c0 = 0; c0 < kOut; c0 += kCols) {
        const int col = t.col + half * kOut + c0;
        uint32_t word[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          auto value = [&](int c) {
            if constexpr (GATED) return gated_value<O>(v[c], v[kOut + c]);
            return v[c];
          };
          if constexpr (sizeof(O) == 2)
            word[j] = pack_bf16(value(c0 + 2 * j), value(c0 + 2 * j + 1));
          else
            word[j] = __float_as_uint(value(c0 + j));
        }
        __syncwarp();  // the last columns have been read
        uint4* mine4 = reinterpret_cast<uint4*>(stage + lane * kStageLd);
        mine4[0] = make_uint4(word[0], word[1], word[2], word[3]);
        mine4[1] = make_uint4(word[4], word[5], word[6], word[7]);
        __syncwarp();
        if (wide) {
          const int c = (lane & 1) * (kCols / 2);
#pragma unroll
          for (int r = lane >> 1; r < 32; r += 16)
            if (r < rows && col + c < out_cols)
              *reinterpret_cast<uint4*>(y + (int64_t)r * out_cols + col + c) =
                  *reinterpret_cast<const uint4*>(stage + r * kStageLd + (lane & 1) * 4);
        } else {
          const int c = lane % kCols;
          if (col + c < out_cols)
            for (int r = lane / kCols; r < rows; r += 32 / kCols)
              y[(int64_t)r * out_cols + col + c] = reinterpret_cast<const O*>(stage + r * kStageLd)[c];
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  if (threadIdx.x == 0 && *s_abort) atomicOr(a.status, COLIBRI_FP8_WAIT_EXPIRED);
}

template <int MODE, int FORM, bool GATED, typename O>
cudaError_t launch(const Fp8Maps& maps, const Fp8Args& a, int device, int sms, cudaStream_t s) {
  static std::mutex mu;
  static bool ready[kOpsMaxDevices] = {};
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[device]) {
      const cudaError_t e = cudaFuncSetAttribute(fp8_mma_kernel<MODE, FORM, GATED, O>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, Form<FORM>::kSmem);
      if (e != cudaSuccess) return e;
      // the register split above waits for ever for more than the block was launched with
      cudaFuncAttributes at;
      const cudaError_t f = cudaFuncGetAttributes(&at, fp8_mma_kernel<MODE, FORM, GATED, O>);
      if (f != cudaSuccess) return f;
      if (at.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
      ready[device] = true;
    }
  }
  return pdl_launch(fp8_mma_kernel<MODE, FORM, GATED, O>, dim3(sms), dim3(kThreads), Form<FORM>::kSmem, s, maps, a);
}

}  // namespace fp8
}  // namespace colibri
