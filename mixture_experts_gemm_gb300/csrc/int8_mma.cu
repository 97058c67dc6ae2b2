// Products of quantised rows with 8-bit expert weights on the tensor cores (tcgen05), weights streamed
// as bytes.
//
//   acc[n, r] = sum_k w[e, n, k] q[r, k],   y[r, n] = acc * w_scale[e, n] * scale[r]   (or silu(.) * .)
//
// The integer tensor rate of this chip is a small fraction of its 16-bit rate, and every 8-bit integer is
// exact in fp16, so the products run as kind::f16 with fp32 accumulation: products are exact, and so are
// sums while their magnitudes stay below 2^24 (beyond, fp32 rounding).  Weights cross HBM and L2 as bytes
// and become fp16 on their way through shared memory; activation rows are fp16 from the quantiser.
//
// Weight rows on the MMA's M side (128 lanes), an expert's token rows on N (32..NT columns, sized to the
// rows): each weight tile is converted once per token tile, and few rows cost few columns.  With a gate
// and an up projection a tile holds 64 channels of each, 16 + 16 in every quarter of 32 TMEM lanes, so
// the epilogue finds both values of a channel 16 lanes apart in one warp.
//
// One persistent CTA per SM, 512 threads:
//   warp 0       TMA producer of the raw weights (RS stages);
//   warp 6       TMA producer of the token rows (SB stages);
//   warps 8..15  converters to the fp16 weights (SA stages), two groups of four that take alternate
//                stages: 16 bytes a thread become two 16-byte stores of fp16 in the 128-byte swizzled
//                layout (byte ^ 0x80 under an exponent of 2^10 is 1024 + (v + 128); one subtraction
//                leaves v);
//   warp 1       issues the MMAs, two accumulators in TMEM;
//   warps 2..5   epilogue.
// The converters' work is about 1.5 instructions per weight, so it hides behind the MMAs of wide tiles (512
// cycles a block of 64 columns of K) and behind HBM for narrow ones.  Items are (tile, part of K) in a
// fixed order; a product of few tiles is split along K, the parts' sums kept in `partial` and added in order by
// whichever CTA finishes the tile (no floating-point atomics: the same bits every time).
//
// Bytes become fp16 by the exponent: the byte is placed under that of 2^10, and one subtraction leaves the integer (a
// known method: Kim et al., "Who Says Elephants Can't Run: Bringing Large Scale MoE Models into Cloud Scale
// Production", 2022).
//
// Measured on one GB300 (whole calls, quantiser included): one token, two experts of 4096 x 14336 x 2, 47 us
// (235 MB of weights, 5.0 TB/s, 0.73 of the measured copy rate); 512 tokens, eight experts of 2048 x 5632 x 2,
// 79 to 84 us; 1021 tokens, top-6 of 64 experts of 2048 x 1409, 85 to 88 us; 8192 tokens, eight experts of
// 14336 x 4096, 1.29 ms in a burst, 1.48 ms kept up (power), of which this kernel 1.10 ms (1.74 PFLOP/s, 0.91 of
// cuBLAS bf16; tensor pipe active 0.76).  The widest tiles are bound by the tensor cores, the narrowest by HBM and
// about 10 us of launches, first copies and epilogue, those between (tensor pipe 0.24 to 0.29, DRAM 0.33 to
// 0.39, issue 0.43) by the MMA warp's loop and the epilogue (without it 512 tokens take about 10 us less).
//
// Every wait is bounded by the call's limit: when one gives up, all roles stop, copies and MMAs in flight are waited
// for (at most kDrain each, whatever the limit), TMEM is freed and the device's status word gets a bit.
#include <mutex>

#include "int8_internal.cuh"
#include "tcgen05_ptx.cuh"

namespace colibri {
namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kConvWarp0 = 8, kConvGroups = 2, kConvGroupWarps = 4;
constexpr int BM = 128, BK = 64;
constexpr int kRawBytes = BM * BK;       // 8 KB
constexpr int kABytes = BM * BK * 2;     // 16 KB
constexpr int kTokBox = 32;              // token rows of the smallest TMA box
constexpr int kTokBoxBytes = kTokBox * BK * 2;
constexpr int kMaxExperts = 512;
constexpr Int8Limit kDrain = {50000000, 63};  // 50 ms, far above the time of a copy or of a stage's MMAs

// What the waits of all products on this device have come to since it was last taken: 1 once one gave up.
__device__ int g_status;
__device__ int g_taken;
__global__ void take_status_kernel() { g_taken = atomicExch(&g_status, 0); }

// Rings, in stages of KS blocks of 64 columns of K: raw weights (RS), converted weights (SA), token rows
// (SB).  One full and one done barrier serve stage `it` for both operands, at it % kSync.  The MMA warp's
// loop (a wait, four MMAs a block, a commit) takes about 500 cycles a stage of one block, 700 of two.  Two
// blocks a stage pay where HBM could go faster (32 rows: one token 56 -> 49 us); wider tiles lose in
// rings what they gain (128 rows: 512 tokens 81 -> 85 us).  All of them fill the 227 KB.
constexpr int kSync = 8;
template <int NT>
struct Form {
  static constexpr int KS = NT == 32 ? 2 : 1;
  static constexpr int SA = NT == 256 ? 3 : NT == 128 ? 5 : NT == 64 ? 6 : 3;
  static constexpr int SB = NT == 256 ? 4 : NT == 128 ? 5 : NT == 64 ? 6 : 4;
  static constexpr int RS = NT == 256 ? 5 : NT == 128 ? 6 : NT == 64 ? 8 : 5;
  static constexpr int kRaw = KS * kRawBytes, kA = KS * kABytes;
  static constexpr int kB1 = NT * BK * 2, kB = KS * kB1;
  static constexpr int kBars = 2 * kSync + 2 * RS + 7;
  static constexpr uint32_t kTmemCols = 2 * NT;
  static constexpr int kSmem = 1024 + SA * kA + SB * kB + RS * kRaw + kBars * 8 + 32 + 4 * (3 * kMaxExperts + 1);
  static_assert(SA < kSync && SB < kSync, "a barrier is not reused before both rings are");
  // A raw slot alternates between the converter groups unless RS is a multiple of their number.  A group
  // waits for its phase by parity, so the phase before (the other group's, stage it - RS) must be over by
  // then: the group's own last stage, it - kConvGroups, needed the MMAs of stage it - kConvGroups - SA.
  static_assert(RS % kConvGroups == 0 || RS >= SA + kConvGroups, "raw phases by parity");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

// Waits for the phase of `bar` with parity `parity`, at most limit.ns or until *abort.  A try that fails lasts
// about 8 us.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, Int8Limit limit) {
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

// Two bytes of signed integers (selected by `sel` out of w ^ 0x80808080) as two exact fp16.
__device__ __forceinline__ uint32_t bytes_to_half2(uint32_t biased, uint32_t sel) {
  const uint32_t u = __byte_perm(biased, 0x64646464u, sel);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));  // - 1152
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 bytes_to_half8(uint32_t lo, uint32_t hi) {
  lo ^= 0x80808080u, hi ^= 0x80808080u;
  return make_uint4(bytes_to_half2(lo, 0x4140), bytes_to_half2(lo, 0x4342), bytes_to_half2(hi, 0x4140),
                    bytes_to_half2(hi, 0x4342));
}

// fp16 x fp16 -> fp32, both operands K-major.
__device__ __forceinline__ uint32_t idesc_f16(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(BM >> 4) << 24);
}

// silu(v) u as it is stored.  The fast exp and quotient are off by about 2 + 1.2 |v| ulp of fp32 and give 0 below v
// near -87: far below a rounding to bf16, but not for an fp32 result.  That takes expf of what cannot overflow
// and the approximate reciprocal, good to an ulp, of a sum between 1 and 2 (512 tokens: 82 us, 80 with the fast
// forms, 92 with a true quotient and its range checks).
template <typename O>
__device__ __forceinline__ O gated(float v, float u) {
  if constexpr (sizeof(O) == 2) return from_float<O>(silu_fast(v) * u);
  const float t = expf(-fabsf(v));
  float s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + t));
  return from_float<O>(v * (v < 0.f ? t * s : s) * u);
}

struct Item {
  int e, row, n;       // expert, first row, rows of the tile
  int ch;              // weight tile
  int part, tile;      // part of K, tile number
  int kb0, kb1;        // stages of K
};

template <int NT, bool SWIGLU, typename O>
__global__ void __launch_bounds__(kThreads, 1)
    int8_mma_kernel(const __grid_constant__ Int8Maps tm, const Int8Args a) {
  using F = Form<NT>;
  constexpr int SA = F::SA, SB = F::SB, RS = F::RS, KS = F::KS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_a = smem;
  uint8_t* s_b = s_a + SA * F::kA;
  uint8_t* s_raw = s_b + SB * F::kB;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_raw + RS * F::kRaw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + F::kBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_last = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* s_row0 = reinterpret_cast<int*>(tmem_slot + 8);  // first row of each expert
  int* s_rows = s_row0 + kMaxExperts;                   // its rows
  int* s_tiles = s_rows + kMaxExperts;                  // token tiles before it [E + 1]

  const uint32_t full0 = smem_u32(bars), done0 = full0 + 8 * kSync;
  const uint32_t rfull0 = done0 + 8 * kSync, rempty0 = rfull0 + 8 * RS;
  const uint32_t tfull0 = rempty0 + 8 * RS, tempty0 = tfull0 + 16, drain = tempty0 + 16;
  const uint32_t joined = drain + 8, decided = joined + 8;  // a split tile's partial sums are out; who adds them
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < kSync; ++i) {
      mbar_init(full0 + 8 * i, 1 + kConvGroupWarps);  // token rows landed, weights converted
      mbar_init(done0 + 8 * i, 1);
    }
    for (int i = 0; i < RS; ++i) {
      mbar_init(rfull0 + 8 * i, 1);
      mbar_init(rempty0 + 8 * i, kConvGroupWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull0 + 8 * i, 1);
      mbar_init(tempty0 + 8 * i, 4);
    }
    mbar_init(drain, 1);
    mbar_init(joined, 4);
    mbar_init(decided, 1);
    *s_abort = 0;
    fence_mbar_init();
    for (int i = 0; i < kTokMaps; ++i) prefetch_tmap(&tm.q[i]);
    prefetch_tmap(&tm.w);
    if constexpr (SWIGLU) prefetch_tmap(&tm.w3);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), F::kTmemCols);
    tmem_relinquish();
  }
  // The quantiser lets this kernel start once everything before it is done: offsets and weights may be read
  // at once; the warps that read its rows and scales (6, 2..5) wait for it.
  if (warp == 7) {
    // Segments inside 0..R, none reaching back into an earlier one; tiles of each expert.
    const int per = (a.E + 31) / 32;
    int top = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < a.E) top = max(top, min(max(a.offsets[e + 1], 0), a.R));
    }
    int reach = top;  // the furthest end of any expert before this lane's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, reach, o);
      if (lane >= o) reach = max(reach, v);
    }
    reach = __shfl_up_sync(~0u, reach, 1);
    if (lane == 0) reach = 0;
    int tiles = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e >= a.E) break;
      const int hi = min(max(a.offsets[e + 1], 0), a.R);
      const int lo = max(min(max(a.offsets[e], 0), a.R), reach);
      reach = max(reach, hi);
      const int n = max(hi - lo, 0);
      s_row0[e] = lo, s_rows[e] = n;
      s_tiles[e] = tiles;
      tiles += (n + NT - 1) / NT;
    }
    int before_me = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, before_me, o);
      if (lane >= o) before_me += v;
    }
    if (lane == 31) s_tiles[a.E] = before_me;
    before_me -= tiles;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < a.E) s_tiles[e] += before_me;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  constexpr int kCh = SWIGLU ? 64 : 128;  // output channels of a tile
  const int ch_tiles = (a.N + kCh - 1) / kCh;
  const int kblocks = (a.K + BK * KS - 1) / (BK * KS);
  const int64_t tiles = (int64_t)s_tiles[a.E] * ch_tiles;
  // Parts of K: the number that leaves the SMs least idle in the last wave, a little against more parts.
  int parts = 1;
  if (tiles < 2 * (int64_t)gridDim.x) {
    float least = 1e30f;
    for (int p = 1; p <= kInt8MaxSplits && p <= kblocks && tiles * p <= a.max_items; ++p) {
      const int waves = (int)((tiles * p + gridDim.x - 1) / gridDim.x);
      const float cost = (float)waves / p + (p > 1 ? 0.04f : 0.f) + 0.01f * p;
      if (cost < least) least = cost, parts = p;
    }
  }
  const int64_t items = tiles * parts;

  // item -> its tile: an expert's token tiles fastest, so that CTAs at work share a weight tile in L2
  auto item_at = [&](int64_t i) {
    Item it;
    it.tile = (int)(i / parts);
    it.part = (int)(i - (int64_t)it.tile * parts);
    int lo = 0, hi = a.E;  // the last expert whose tiles begin at or before it (those without rows begin with it)
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if ((int64_t)s_tiles[mid] * ch_tiles <= it.tile)
        lo = mid;
      else
        hi = mid;
    }
    it.e = lo;
    const int tt = s_tiles[lo + 1] - s_tiles[lo], local = it.tile - s_tiles[lo] * ch_tiles;
    it.ch = local / tt;
    const int t = local - it.ch * tt, n = s_rows[lo];
    const int each = ((n + tt - 1) / tt + 31) / 32 * 32;  // even tiles, whole boxes
    it.row = s_row0[lo] + t * each;
    it.n = max(min(each, n - t * each), 0);
    it.kb0 = (int)((int64_t)kblocks * it.part / parts);
    it.kb1 = (int)((int64_t)kblocks * (it.part + 1) / parts);
    return it;
  };

  // Waits until the MMAs of block it - behind are done: the slot that block `it` takes is free.  A done
  // barrier cannot run two phases ahead of a waiter, because the blocks between need the waiter's work.
  auto slot_free = [&](uint32_t it, uint32_t behind) {
    const uint32_t j = it - behind;
    return it < behind || wait_for(done0 + 8 * (j % kSync), j / kSync & 1, s_abort, a.limit);
  };

  // The producers' and the MMA warp run their loops with all lanes and let one elected lane issue: addresses
  // and descriptors then stay in uniform registers (inside `if (lane == 0)` four MMAs and their loop took 600
  // cycles, and a copy about 90).
  bool ok = true;
  if (warp == 0) {
    // -------------------------------------------------------------- raw weights
    const bool elected = elect_one();
    const uint32_t raw0 = smem_u32(s_raw);
    uint32_t issued = 0, r = 0, ph = 0;
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item t = item_at(i);
      const int w_row = t.e * a.N + t.ch * kCh;
      for (int kb = t.kb0; kb < t.kb1; ++kb, ++issued) {
        if (!__all_sync(~0u, wait_for(rempty0 + 8 * r, ph ^ 1, s_abort, a.limit))) {
          ok = false;
          break;
        }
        const uint32_t full = rfull0 + 8 * r, dst = raw0 + r * F::kRaw;
        const int x = kb * (BK * KS);
        if (elected) {
          mbar_arrive_expect_tx(full, F::kRaw);
          tma_load_2d(dst, &tm.w, full, x, w_row);  // columns past K read as zeros
          if constexpr (SWIGLU) tma_load_2d(dst + F::kRaw / 2, &tm.w3, full, x, w_row);
        }
        __syncwarp();
        if (++r == RS) r = 0, ph ^= 1;
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
    // every copy has landed before the CTA can leave
    volatile int never = 0;
    for (uint32_t j = issued > RS ? issued - RS : 0; j < issued; ++j)
      wait_for(rfull0 + 8 * (j % RS), j / RS & 1, &never, kDrain);
    __syncwarp();
  } else if (warp == 6) {
    // -------------------------------------------------------------- token rows
    pdl_wait();
    const bool elected = elect_one();
    const uint32_t b0 = smem_u32(s_b);
    const int copy = blockIdx.x % a.copies * a.R;
    uint32_t it = 0, sb = 0;
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item t = item_at(i);
      const int boxes = (t.n + kTokBox - 1) / kTokBox;
      for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
        if (!__all_sync(~0u, slot_free(it, SB))) {
          ok = false;
          break;
        }
        const uint32_t full = full0 + 8 * (it % kSync);
        uint32_t dst = b0 + sb * F::kB;
        const int x = kb * (BK * KS);
        if (elected) {
          mbar_arrive_expect_tx(full, KS * boxes * kTokBoxBytes);
          int row = t.row + copy;
#pragma unroll
          for (int b = kTokMaps - 1; b >= 0; --b)  // at most one copy of each box height
            if (boxes >> b & 1) {
#pragma unroll
              for (int k = 0; k < KS; ++k) tma_load_2d(dst + k * F::kB1, &tm.q[b], full, x + k * BK, row);
              dst += kTokBoxBytes << b, row += kTokBox << b;
            }
        }
        __syncwarp();
        if (++sb == SB) sb = 0;
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
    // Whichever role stopped early: the copies of the last SB stages (those before had their MMAs) land before the
    // CTA can leave.  A stage may then lack its converters' arrivals, and its barrier never completes: the
    // wait for it ends by kDrain.
    volatile int never = 0;
    for (uint32_t j = it > SB ? it - SB : 0; j < it; ++j)
      wait_for(full0 + 8 * (j % kSync), j / kSync & 1, &never, kDrain);
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    const bool elected = elect_one();
    const uint64_t da0 = sw128_desc(smem_u32(s_a)), db0 = sw128_desc(smem_u32(s_b));
    uint32_t it = 0, acc_it = 0, sa = 0, sb = 0;
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x, ++acc_it) {
      const Item t = item_at(i);
      const uint32_t acc = acc_it & 1;
      if (!__all_sync(~0u, wait_for(tempty0 + 8 * acc, (acc_it >> 1 & 1) ^ 1, s_abort, a.limit))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem_base + acc * NT, idesc = idesc_f16((t.n + kTokBox - 1) / kTokBox * kTokBox);
      uint32_t more = 0;  // the first MMA of a tile overwrites the accumulator
      for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
        if (!__all_sync(~0u, wait_for(full0 + 8 * (it % kSync), it / kSync & 1, s_abort, a.limit))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t da = da0 + sa * (F::kA >> 4), db = db0 + sb * (F::kB >> 4);
        if (elected) {
#pragma unroll
          for (int k = 0; k < 4 * KS; ++k)
            umma_bf16(d, da + (k >> 2) * (kABytes >> 4) + 2 * (k & 3), db + (k >> 2) * (F::kB1 >> 4) + 2 * (k & 3), idesc,
                      k ? 1 : more);
          umma_commit(done0 + 8 * (it % kSync));
        }
        __syncwarp();
        more = 1;
        if (++sa == SA) sa = 0;
        if (++sb == SB) sb = 0;
      }
      if (!ok) break;
      if (elected) umma_commit(tfull0 + 8 * acc);
      __syncwarp();
    }
    if (!ok && lane == 0) *s_abort = 1;
    if (elected) {
      umma_commit(drain);  // completes when every MMA of this thread has
      volatile int never = 0;
      wait_for(drain, 0, &never, kDrain);
    }
    __syncwarp();
  } else if (warp >= kConvWarp0) {
    // -------------------------------------------------------------- converters
    const uint32_t group = (warp - kConvWarp0) / kConvGroupWarps;
    // A warp takes 32 rows, eight at a time: a lane one row's 16 bytes (16 columns of one block of 64), two
    // neighbouring swizzled chunks of fp16.  Which row makes both sides free of bank conflicts among eight
    // neighbouring lanes (two rows, 4 c's): they write to rows of opposite parity (even against odd chunks);
    // they read 64-byte raw rows in a row, or 128-byte raw rows, swizzled by the copy, whose numbers differ
    // in bit 2.  Everything but the stage is known before the loop.
    const int w4 = (warp - kConvWarp0) % kConvGroupWarps, c = lane & 3, pair = lane >> 3;
    const int r8 = KS == 1 ? lane >> 2 : (lane & 4 ? 4 + ((pair + 1) & 3) : pair);
    const uint32_t src0 = KS == 1 ? (w4 * 32 + r8) * 64 + c * 16 : (w4 * 32 + r8) * 128 + ((c ^ r8) << 4);
    // gate rows 0..63 and up rows 64..127 alternate in runs of 16 lanes
    const int m0 = SWIGLU ? (w4 & 1) * 64 + (w4 >> 1) * 16 : w4 * 32;
    const uint32_t dst0 = (m0 + r8) * 128 + (((2 * c) ^ r8) << 4);
    uint32_t it0 = 0, r = group % RS, ph = group / RS & 1, sa = group % SA;  // this group's next block
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item t = item_at(i);
      const uint32_t n = t.kb1 - t.kb0;
      for (uint32_t j = (group - it0) % kConvGroups; j < n; j += kConvGroups) {
        const uint32_t it = it0 + j;
        bool got = wait_for(rfull0 + 8 * r, ph, s_abort, a.limit);
        uint4 v[4 * KS];
        const uint8_t* src = s_raw + r * F::kRaw;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int o = 0; o < 4; ++o)  // chunk 4 + c of a swizzled row is 64 bytes away from chunk c
            v[4 * k + o] = *reinterpret_cast<const uint4*>(src + (src0 ^ (k * 64)) + o * 8 * (KS * 64));
        got = got && slot_free(it, SA);
        if (!__all_sync(~0u, got)) {
          ok = false;
          break;
        }
        __syncwarp();  // every lane has its bytes
        if (lane == 0) mbar_arrive(rempty0 + 8 * r);
        uint8_t* dst = s_a + sa * F::kA;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int o = 0; o < 4; ++o) {
            const int row = SWIGLU ? (o >> 1) * 32 + (o & 1) * 8 : o * 8;
            const uint4 q = v[4 * k + o];
            *reinterpret_cast<uint4*>(dst + k * kABytes + row * 128 + dst0) = bytes_to_half8(q.x, q.y);
            *reinterpret_cast<uint4*>(dst + k * kABytes + row * 128 + (dst0 ^ 16)) = bytes_to_half8(q.z, q.w);
          }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full0 + 8 * (it % kSync));
        r += kConvGroups;
        if (r >= RS) r -= RS, ph ^= 1;
        sa += kConvGroups;
        if (sa >= SA) sa -= SA;
      }
      it0 += n;
    }
    if (!ok && lane == 0) *s_abort = 1;
  } else if (warp >= 2 && warp < 6) {
    // -------------------------------------------------------------- epilogue
    pdl_wait();
    const int q = warp & 3;  // the TMEM lanes this warp may read
    uint32_t acc_it = 0;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x, ++acc_it) {
      const Item t = item_at(i);
      const uint32_t acc = acc_it & 1;
      if (!__all_sync(~0u, wait_for(tfull0 + 8 * acc, acc_it >> 1 & 1, s_abort, a.limit))) {
        if (lane == 0) *s_abort = 1;
        break;
      }
      tc_fence_after();
      const uint32_t base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * NT;
      // this lane's channel: of the tile, or with two projections gate (lanes 0..15) and up of 16 channels
      const int n = SWIGLU ? t.ch * kCh + q * 16 + (lane & 15) : t.ch * kCh + q * 32 + lane;
      const bool in = n < a.N;
      float ws = 0.f;
      if (in) ws = (SWIGLU && lane >= 16 ? a.w3_scale : a.w_scale)[(int64_t)t.e * a.N + n];
      // columns c0 .. c0 + 31 of the tile, summed over K, to y; eight at a time, none past the tile's rows
      auto finish = [&](const float (&v)[32], int c0) {
        const float sx = c0 + lane < t.n ? a.scale[t.row + c0 + lane] : 0.f;
        O* out = static_cast<O*>(a.y) + (int64_t)(t.row + c0 + (SWIGLU ? lane >> 4 : 0)) * a.N + n;
        const int left = in ? t.n - c0 - (SWIGLU ? lane >> 4 : 0) : 0;  // rows from this lane's first one on
#pragma unroll
        for (int c8 = 0; c8 < 32; c8 += 8) {
          if (c0 + c8 >= t.n) break;
          float h[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) h[c] = v[c8 + c] * ws * __shfl_sync(~0u, sx, c8 + c);
          if constexpr (SWIGLU) {
            // lanes 0..15 take the even columns, the others the odd ones: one exchange gives both their
            // second value
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
              const float other = __shfl_xor_sync(~0u, lane < 16 ? h[c + 1] : h[c], 16);
              const float g = lane < 16 ? h[c] : other, u = lane < 16 ? other : h[c + 1];
              if (c8 + c < left) out[(int64_t)(c8 + c) * a.N] = gated<O>(g, u);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (c8 + c < left) out[(int64_t)(c8 + c) * a.N] = from_float<O>(h[c]);
          }
        }
      };
      float* part = a.partial + i * (NT * 128) + q * 32 + lane;
#pragma unroll 1
      for (int c0 = 0; c0 < t.n; c0 += 32) {
        uint32_t raw[32];
        tmem_ld32_sync(base + c0, raw);
        float v[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(raw[c]);
        if (parts == 1) {
          finish(v, c0);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c < t.n) part[(c0 + c) * 128] = v[c];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
      if (parts > 1) {
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(joined);
        bool got = true;
        if (warp == 2 && lane == 0) {
          got = wait_for(joined, acc_it & 1, s_abort, a.limit);
          if (got) {
            __threadfence();
            *s_last = atomicAdd(&a.ticket[t.tile], 1u) == (uint32_t)(parts - 1);
            mbar_arrive(decided);
          }
        }
        got = got && wait_for(decided, acc_it & 1, s_abort, a.limit);
        if (!__all_sync(~0u, got)) {
          if (lane == 0) *s_abort = 1;
          break;
        }
        if (*s_last) {
          __threadfence();
          const float* all = a.partial + (int64_t)t.tile * parts * (NT * 128) + q * 32 + lane;
#pragma unroll 1
          for (int c0 = 0; c0 < t.n; c0 += 32) {
            float v[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = 0.f;
            for (int p = 0; p < parts; ++p)
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c0 + c < t.n) v[c] += __ldcg(all + (int64_t)p * (NT * 128) + (c0 + c) * 128);
            finish(v, c0);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem_base, F::kTmemCols);
  if (threadIdx.x == 0 && *s_abort) atomicOr(&g_status, COLIBRI_INT8_WAIT_EXPIRED);
}

bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t rows, int elem,
              uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promo) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {inner, rows}, strides[1] = {inner * elem};
  const cuuint32_t box[2] = {box_cols, box_rows}, estr[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promo,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool SWIGLU, typename O>
cudaError_t launch(const Int8Maps& maps, const Int8Args& a, int device, int grid, cudaStream_t s) {
  static std::mutex mu;
  static bool ready[kOpsMaxDevices] = {};
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[device]) {
      const cudaError_t e = cudaFuncSetAttribute(int8_mma_kernel<NT, SWIGLU, O>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, Form<NT>::kSmem);
      if (e != cudaSuccess) return e;
      ready[device] = true;
    }
  }
  return pdl_launch(int8_mma_kernel<NT, SWIGLU, O>, dim3(grid), dim3(kThreads), Form<NT>::kSmem, s, maps, a);
}

}  // namespace

bool int8_tensor_maps(int tile_rows, const void* q, int64_t rows, const int8_t* w, const int8_t* w3, int E, int N, int K,
                      Int8Maps* maps) {
  for (int i = 0; i < kTokMaps; ++i)
    if (!make_map(&maps->q[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, q, K, (uint64_t)rows, 2, BK, kTokBox << i,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
      return false;
  const int blocks = tile_rows == 256   ? Form<256>::KS
                     : tile_rows == 128 ? Form<128>::KS
                     : tile_rows == 64  ? Form<64>::KS
                                        : Form<32>::KS;
  for (int i = 0; i < 2; ++i)
    if (!make_map(i ? &maps->w3 : &maps->w, CU_TENSOR_MAP_DATA_TYPE_UINT8, i && w3 ? w3 : w, K, (uint64_t)E * N, 1,
                  BK * blocks, w3 ? 64 : 128, blocks == 2 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
      return false;
  return true;
}

cudaError_t int8_take_status(int* status) {
  static std::mutex mu;  // g_taken holds one caller's answer at a time
  std::lock_guard<std::mutex> lock(mu);
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return e;
  take_status_kernel<<<1, 1>>>();
  e = cudaGetLastError();
  return e != cudaSuccess ? e : cudaMemcpyFromSymbol(status, g_taken, sizeof(int));
}

cudaError_t launch_int8_mma(const Int8Maps& maps, int tile_rows, bool swiglu, bool bf16_out, const Int8Args& a, int device,
                            int sms, cudaStream_t s) {
  auto with = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    using B = __nv_bfloat16;
    if (swiglu)
      return bf16_out ? launch<NT, true, B>(maps, a, device, sms, s) : launch<NT, true, float>(maps, a, device, sms, s);
    return bf16_out ? launch<NT, false, B>(maps, a, device, sms, s) : launch<NT, false, float>(maps, a, device, sms, s);
  };
  if (tile_rows == 256) return with(std::integral_constant<int, 256>{});
  if (tile_rows == 128) return with(std::integral_constant<int, 128>{});
  if (tile_rows == 64) return with(std::integral_constant<int, 64>{});
  return with(std::integral_constant<int, 32>{});
}

}  // namespace colibri
