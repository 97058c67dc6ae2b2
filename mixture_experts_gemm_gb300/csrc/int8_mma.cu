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
//   warp 0       TMA producer of the raw weight ring (RS stages of 128 rows x 64 bytes);
//   warp 6       TMA producer of the token rows of the operand ring (ST stages, 64 columns of K);
//   warps 8..15  converters, two groups of four that take alternate stages: 16 bytes a thread become two
//                16-byte stores of fp16 in the 128-byte swizzled layout (byte ^ 0x80 under an exponent of
//                2^10 is 1024 + (v + 128); one subtraction leaves v);
//   warp 1       one lane issues the MMAs, two accumulators in TMEM;
//   warps 2..5   epilogue.
// The converters' work is 2 instructions per weight (about 120 issue slots of the 512 cycles that the
// MMAs of a 256-column stage take), so it hides behind the MMAs of wide tiles and behind HBM for narrow
// ones.  Items are (tile, part of K) in a fixed order; a narrow product of few tiles is split along K, the
// parts' sums kept in `partial` and added in order by whichever CTA finishes the tile (no floating-point
// atomics: the same bits every time).
//
// Every wait is bounded by timeout_ns: when one gives up, all roles stop, copies in flight are waited for
// (bounded) and TMEM is freed.
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
constexpr int kTokBox = 32;              // token rows of one TMA box
constexpr int kTokBoxBytes = kTokBox * BK * 2;
constexpr int kMaxExperts = 512;

template <int NT>
struct Form {
  static constexpr int ST = NT == kInt8WideRows ? 3 : 5;   // operand stages
  static constexpr int RS = NT == kInt8WideRows ? 8 : 10;  // raw weight stages
  static constexpr int kBBytes = NT * BK * 2;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kBars = 2 * ST + 2 * RS + 7;
  static constexpr uint32_t kTmemCols = 2 * NT;
  static constexpr int kSmem = 1024 + ST * kStage + RS * kRawBytes + kBars * 8 + 32 + 4 * (3 * kMaxExperts + 1);
};
static_assert(Form<kInt8WideRows>::kSmem <= 227 * 1024 && Form<kInt8NarrowRows>::kSmem <= 227 * 1024, "shared memory");

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

struct Item {
  int e, row, n;       // expert, first row, rows of the tile
  int ch;              // weight tile
  int part, tile;      // part of K, tile number
  int kb0, kb1;        // K blocks
};

template <int NT, bool SWIGLU, typename O>
__global__ void __launch_bounds__(kThreads, 1)
    int8_mma_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_w3, const Int8Args a) {
  using F = Form<NT>;
  constexpr int ST = F::ST, RS = F::RS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_a = smem;
  uint8_t* s_b = s_a + ST * kABytes;
  uint8_t* s_raw = s_b + ST * F::kBBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_raw + RS * kRawBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + F::kBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_last = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* s_row0 = reinterpret_cast<int*>(tmem_slot + 8);  // first row of each expert
  int* s_rows = s_row0 + kMaxExperts;                   // its rows
  int* s_tiles = s_rows + kMaxExperts;                  // token tiles before it [E + 1]

  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * ST;
  const uint32_t rfull0 = empty0 + 8 * ST, rempty0 = rfull0 + 8 * RS;
  const uint32_t tfull0 = rempty0 + 8 * RS, tempty0 = tfull0 + 16, drain = tempty0 + 16;
  const uint32_t joined = drain + 8, decided = joined + 8;  // a split tile's partial sums are out; who adds them
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full0 + 8 * i, 1 + kConvGroupWarps);  // token rows landed, weights converted
      mbar_init(empty0 + 8 * i, 1);
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
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_w);
    if constexpr (SWIGLU) prefetch_tmap(&tm_w3);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), F::kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();  // the quantised rows, and the offsets of the routing before
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
  const int kblocks = (a.K + BK - 1) / BK;
  const int64_t tiles = (int64_t)s_tiles[a.E] * ch_tiles;
  // Parts of K: the number that leaves the SMs least idle in the last wave, a little against more parts.
  int parts = 1;
  if (a.partial && tiles < 2 * (int64_t)gridDim.x) {
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

  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ raw weights
      uint32_t it = 0, issued = 0;
      for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
        const Item t = item_at(i);
        const int w_row = t.e * a.N + t.ch * kCh;
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const uint32_t r = it % RS;
          if (!mbar_wait(rempty0 + 8 * r, (it / RS & 1) ^ 1, s_abort, a.timeout_ns)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(rfull0 + 8 * r, kRawBytes);
          const uint32_t dst = smem_u32(s_raw + r * kRawBytes);
          tma_load_2d(dst, &tm_w, rfull0 + 8 * r, kb * BK, w_row);
          if constexpr (SWIGLU) tma_load_2d(dst + kRawBytes / 2, &tm_w3, rfull0 + 8 * r, kb * BK, w_row);
          issued = it + 1;
        }
      }
      if (!ok) *s_abort = 1;
      // every copy of this thread has landed before the CTA can leave
      volatile int never = 0;
      for (uint32_t j = issued > RS ? issued - RS : 0; j < issued; ++j)
        mbar_wait(rfull0 + 8 * (j % RS), j / RS & 1, &never, a.timeout_ns);
    }
  } else if (warp == 6) {
    if (lane == 0) {
      // ------------------------------------------------------------ token rows
      uint32_t it = 0, issued = 0;
      for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
        const Item t = item_at(i);
        const int boxes = (t.n + kTokBox - 1) / kTokBox;
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const uint32_t s = it % ST;
          if (!mbar_wait(empty0 + 8 * s, (it / ST & 1) ^ 1, s_abort, a.timeout_ns)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full0 + 8 * s, boxes * kTokBoxBytes);
          const uint32_t dst = smem_u32(s_b + s * F::kBBytes);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(dst + b * kTokBoxBytes, &tm_q, full0 + 8 * s, kb * BK, t.row + b * kTokBox);
          issued = it + 1;
        }
      }
      if (!ok) {
        *s_abort = 1;
        // stopped early: no MMA reads the stages any more, but the copies must land.  A full barrier may
        // lack its converters' arrivals, so give the copies the bound of one wait instead.
        volatile int never = 0;
        const uint32_t j = issued ? issued - 1 : 0;
        if (issued) mbar_wait(full0 + 8 * (j % ST), j / ST & 1, &never, a.timeout_ns / 8);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      uint32_t it = 0, acc_it = 0;
      for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x, ++acc_it) {
        const Item t = item_at(i);
        const uint32_t acc = acc_it & 1;
        if (!mbar_wait(tempty0 + 8 * acc, (acc_it >> 1 & 1) ^ 1, s_abort, a.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * NT, idesc = idesc_f16((t.n + kTokBox - 1) / kTokBox * kTokBox);
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const uint32_t s = it % ST;
          if (!mbar_wait(full0 + 8 * s, it / ST & 1, s_abort, a.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t pa = smem_u32(s_a + s * kABytes), pb = smem_u32(s_b + s * F::kBBytes);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_bf16(d, sw128_desc(pa + 32 * k), sw128_desc(pb + 32 * k), idesc, kb != t.kb0 || k != 0);
          umma_commit(empty0 + 8 * s);
        }
        if (!ok) break;
        umma_commit(tfull0 + 8 * acc);
      }
      if (!ok) *s_abort = 1;
      umma_commit(drain);  // completes when every MMA of this thread has
      volatile int never = 0;
      mbar_wait(drain, 0, &never, a.timeout_ns);
    }
  } else if (warp >= kConvWarp0) {
    // -------------------------------------------------------------- converters
    const int group = (warp - kConvWarp0) / kConvGroupWarps;
    const int tid = threadIdx.x - 32 * (kConvWarp0 + group * kConvGroupWarps);  // 0..127
    uint32_t it = 0;
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item t = item_at(i);
      for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
        if (it % kConvGroups != (uint32_t)group) continue;
        const uint32_t r = it % RS, s = it % ST;
        bool got = mbar_wait(rfull0 + 8 * r, it / RS & 1, s_abort, a.timeout_ns);
        got = got && mbar_wait(empty0 + 8 * s, (it / ST & 1) ^ 1, s_abort, a.timeout_ns);
        if (!__all_sync(~0u, got)) {
          ok = false;
          break;
        }
        const uint4* src = reinterpret_cast<const uint4*>(s_raw + r * kRawBytes);
        uint8_t* dst = s_a + s * kABytes;
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = src[tid + 128 * j];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // 16 bytes of raw row `row`: columns 16 c .. 16 c + 15, swizzled chunks 2 c and 2 c + 1
          const int row = (tid >> 2) + 32 * j, c = tid & 3;
          // gate rows 0..63 and up rows 64..127 alternate in runs of 16 lanes
          const int m = SWIGLU ? (row & 48) * 2 + (row & 15) + (row >> 6) * 16 : row;
          uint8_t* line = dst + m * 128;
          *reinterpret_cast<uint4*>(line + (((2 * c) ^ (m & 7)) << 4)) = bytes_to_half8(v[j].x, v[j].y);
          *reinterpret_cast<uint4*>(line + (((2 * c + 1) ^ (m & 7)) << 4)) = bytes_to_half8(v[j].z, v[j].w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full0 + 8 * s);
          mbar_arrive(rempty0 + 8 * r);
        }
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
  } else if (warp >= 2 && warp < 6) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;  // the TMEM lanes this warp may read
    uint32_t acc_it = 0;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x, ++acc_it) {
      const Item t = item_at(i);
      const uint32_t acc = acc_it & 1;
      if (!__all_sync(~0u, mbar_wait(tfull0 + 8 * acc, acc_it >> 1 & 1, s_abort, a.timeout_ns))) {
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
      // columns c0 .. c0 + 31 of the tile, summed over K, to y
      auto finish = [&](const float (&v)[32], int c0) {
        const float sx = c0 + lane < t.n ? a.scale[t.row + c0 + lane] : 0.f;
        if constexpr (SWIGLU) {
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            // lanes 0..15 take column c, the others c + 1: one exchange gives both their second value
            const float s0 = __shfl_sync(~0u, sx, c), s1 = __shfl_sync(~0u, sx, c + 1);
            const float v0 = v[c] * ws * s0, v1 = v[c + 1] * ws * s1;
            const float other = __shfl_xor_sync(~0u, lane < 16 ? v1 : v0, 16);
            const float g = lane < 16 ? v0 : other, u = lane < 16 ? other : v1;
            const int col = c0 + c + (lane >> 4);
            const float h = g / (1.f + expf(-g)) * u;
            if (in && col < t.n) static_cast<O*>(a.y)[(int64_t)(t.row + col) * a.N + n] = from_float<O>(h);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float h = v[c] * ws * __shfl_sync(~0u, sx, c);
            if (in && c0 + c < t.n) static_cast<O*>(a.y)[(int64_t)(t.row + c0 + c) * a.N + n] = from_float<O>(h);
          }
        }
      };
      float* part = a.partial + i * (kInt8NarrowRows * 128) + q * 32 + lane;
#pragma unroll 1
      for (int c0 = 0; c0 < t.n; c0 += 32) {
        uint32_t raw[32];
        tmem_ld32_sync(base + c0, raw);
        float v[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(raw[c]);
        if (NT == kInt8WideRows || parts == 1) {
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
      if (NT != kInt8WideRows && parts > 1) {
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(joined);
        bool got = true;
        if (warp == 2 && lane == 0) {
          got = mbar_wait(joined, acc_it & 1, s_abort, a.timeout_ns);
          if (got) {
            __threadfence();
            *s_last = atomicAdd(&a.ticket[t.tile], 1u) == (uint32_t)(parts - 1);
            mbar_arrive(decided);
          }
        }
        got = got && mbar_wait(decided, acc_it & 1, s_abort, a.timeout_ns);
        if (!__all_sync(~0u, got)) {
          if (lane == 0) *s_abort = 1;
          break;
        }
        if (*s_last) {
          __threadfence();
          const float* all = a.partial + (int64_t)t.tile * parts * (kInt8NarrowRows * 128) + q * 32 + lane;
#pragma unroll 1
          for (int c0 = 0; c0 < t.n; c0 += 32) {
            float v[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = 0.f;
            for (int p = 0; p < parts; ++p)
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c0 + c < t.n) v[c] += __ldcg(all + (int64_t)p * (kInt8NarrowRows * 128) + (c0 + c) * 128);
            finish(v, c0);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem_base, F::kTmemCols);
}

bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t rows, int elem,
              uint32_t box_rows, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promo) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {inner, rows}, strides[1] = {inner * elem};
  const cuuint32_t box[2] = {BK, box_rows}, estr[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promo,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool SWIGLU, typename O>
cudaError_t launch(const CUtensorMap* maps, const Int8Args& a, int device, int grid, cudaStream_t s) {
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
  return pdl_launch(int8_mma_kernel<NT, SWIGLU, O>, dim3(grid), dim3(kThreads), Form<NT>::kSmem, s, maps[0], maps[1],
                    maps[2], a);
}

}  // namespace

bool int8_tensor_maps(const void* q, int R, const int8_t* w, const int8_t* w3, int E, int N, int K, CUtensorMap* maps) {
  const uint32_t box = w3 ? 64 : 128;
  if (!make_map(&maps[0], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, q, K, R, 2, kTokBox, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return false;
  if (!make_map(&maps[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, w, K, (uint64_t)E * N, 1, box, CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return false;
  return make_map(&maps[2], CU_TENSOR_MAP_DATA_TYPE_UINT8, w3 ? w3 : w, K, (uint64_t)E * N, 1, box,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

cudaError_t launch_int8_mma(const CUtensorMap* maps, bool wide, bool swiglu, bool bf16_out, const Int8Args& a, int device,
                            int sms, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (wide) {
    if (swiglu)
      return bf16_out ? launch<kInt8WideRows, true, B>(maps, a, device, sms, s)
                      : launch<kInt8WideRows, true, float>(maps, a, device, sms, s);
    return bf16_out ? launch<kInt8WideRows, false, B>(maps, a, device, sms, s)
                    : launch<kInt8WideRows, false, float>(maps, a, device, sms, s);
  }
  if (swiglu)
    return bf16_out ? launch<kInt8NarrowRows, true, B>(maps, a, device, sms, s)
                    : launch<kInt8NarrowRows, true, float>(maps, a, device, sms, s);
  return bf16_out ? launch<kInt8NarrowRows, false, B>(maps, a, device, sms, s)
                  : launch<kInt8NarrowRows, false, float>(maps, a, device, sms, s);
}

}  // namespace colibri
