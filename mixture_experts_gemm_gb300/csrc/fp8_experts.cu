// Experts in 8-bit floating point: the quantisers and the entry points (the products are in fp8_mma.cuh).
//
//   scale = max |x| / 448 over a block of 128,  q = e4m3(x / scale)   (IEEE fp32 quotients, ties to even)
//
// Blocks lie along a row (activations and gradients, for products that sum over a row's columns), down 128 rows of
// an expert (for the weights' gradient, which sums over rows), or cover 128 x 128 (weights).
#include <algorithm>
#include <mutex>

#include <cuda_fp8.h>

#include "fp8_internal.cuh"

namespace colibri {
namespace {

__device__ int g_status;  // what the waits of all products on this device have come to since it was last taken
__device__ int g_taken;
__global__ void take_status_kernel() { g_taken = atomicExch(&g_status, 0); }

constexpr float kTop = 448.f;

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if one of them is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A block's scale from its largest |x| (NaN or infinite where a value is), and 1 / scale: 0 for a scale of 0 (whose
// values are), negative where every quotient is to be a division: 1 / scale may overflow, or the scale is NaN.
struct Scale {
  float scale, inv;
  __device__ __forceinline__ explicit Scale(float top) {
    scale = top < INFINITY ? __fdiv_rn(top, kTop) : NAN;
    inv = scale == 0.f ? 0.f : scale >= 1e-30f ? __frcp_rn(scale) : -1.f;
  }
};

// e4m3 of the IEEE quotients x0 / s0 and x1 / s1, two bytes.  x * inv is within 3 ulp of a quotient, so the quotient
// lies between x * inv * (1 - 2^-21) and x * inv * (1 + 2^-21), and where both ends round to the same e4m3 so does
// it.  Where they do not (of fp32 values one pair in 2^15; of bf16 values a few in a hundred, as quotients of few bits
// often are the middle of two), a bit of `doubt` is set and the division decides, one pair after another.
struct Ends {
  float lo, hi;
  __device__ __forceinline__ explicit Ends(float inv) : lo(inv * (1.f - 0x1p-21f)), hi(inv * (1.f + 0x1p-21f)) {}
};
__device__ __forceinline__ uint32_t quotients(float x0, float x1, const Ends& e0, const Ends& e1, uint32_t& doubt, int bit) {
  const uint32_t lo = e4m3_pair(x0 * e0.lo, x1 * e1.lo), hi = e4m3_pair(x0 * e0.hi, x1 * e1.hi);
  if (lo != hi) doubt |= 1u << bit;
  return lo;
}
__device__ __forceinline__ float quotient(float x, float scale) { return scale > 0.f ? __fdiv_rn(x, scale) : 0.f; }
// Columns col and col + 1 of a row (zeros without one), by division.
template <typename T>
__device__ __forceinline__ uint16_t divided(const T* row, int col, int cols, float s0, float s1) {
  const float x0 = row && col < cols ? to_float(row[col]) : 0.f, x1 = row && col + 1 < cols ? to_float(row[col + 1]) : 0.f;
  return (uint16_t)e4m3_pair(quotient(x0, s0), quotient(x1, s1));
}

// Eight values of a row as loaded; zeros past its end.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ void set(int i, float x) { v[i] = x; }
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
  __device__ __forceinline__ void set(int i, float x) {  // of zeros
    w[i >> 1] |= i & 1 ? __float_as_uint(x) : __float_as_uint(x) >> 16;
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
};
template <bool VEC, typename T>
__device__ __forceinline__ Raw8<T> read8(const T* row, int col, int cols) {
  Raw8<T> r = {};
  if constexpr (VEC) {
    if (col < cols) r.load(row + col);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < cols) r.set(j, to_float(row[col + j]));
  }
  return r;
}

// Largest |v| of eight columns, column by column or of all.
template <typename T>
struct Top8;
template <>
struct Top8<float> {
  float v[8] = {};
  __device__ __forceinline__ void take(const Raw8<float>& r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = max_nan(v[i], fabsf(r.v[i]));
  }
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ float all() const {
    return max_nan(max_nan(max_nan(v[0], v[1]), max_nan(v[2], v[3])), max_nan(max_nan(v[4], v[5]), max_nan(v[6], v[7])));
  }
  __device__ __forceinline__ void across(int lanes) {  // with the thread whose lane differs in this bit
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = max_nan(v[i], __shfl_xor_sync(~0u, v[i], lanes));
  }
};
template <>
struct Top8<__nv_bfloat16> {
  uint32_t w[4] = {};
  static __device__ __forceinline__ uint32_t two(uint32_t a, uint32_t b) {
    const __nv_bfloat162 *pa = reinterpret_cast<const __nv_bfloat162*>(&a), *pb = reinterpret_cast<const __nv_bfloat162*>(&b);
    const __nv_bfloat162 m = __hmax2_nan(*pa, *pb);
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  __device__ __forceinline__ void take(const Raw8<__nv_bfloat16>& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = two(w[i], r.w[i] & 0x7fff7fffu);
  }
  __device__ __forceinline__ float get(int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
  __device__ __forceinline__ float all() const {
    const uint32_t m = two(two(w[0], w[1]), two(w[2], w[3]));
    return max_nan(bf16_lo(m), bf16_hi(m));
  }
  __device__ __forceinline__ void across(int lanes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = two(w[i], __shfl_xor_sync(~0u, w[i], lanes));
  }
};

// Eight values by one scale; doubtful pairs as bits from `bit` on.
template <typename T>
__device__ __forceinline__ uint2 quantised8(const Raw8<T>& r, float inv, uint32_t& doubt, int bit) {
  const Ends e(inv);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = quotients(r.get(2 * i), r.get(2 * i + 1), e, e, doubt, bit + i);
  if (inv < 0.f) doubt |= 15u << bit;
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// ------------------------------------------------------------------------------------- along rows
struct RowQuant {
  const void* x;
  int64_t ldx;
  int n_tokens;
  const int32_t* rows;  // token of each row, or nullptr: the row itself
  int n, cols;          // rows to write (CHAINS: tokens); columns of x
  uint8_t* q;           // [n][ldq], zeros from cols on
  int ldq;
  float* scale;         // of row r, block b at b * block_step + r * row_step
  int64_t row_step, block_step;
  uint32_t* ticket;     // cleared for the product, or nullptr
  int n_ticket;
  // CHAINS: rows of each token, head[t], then next[r] until it is negative, by the first `chained` blocks of threads; the
  // *n_direct + 1 rows of `direct` by the others, each for itself
  const int32_t *head, *next, *direct, *n_direct;
  int chained;
};

constexpr int kRowThreads = 256, kRowsAt = 32, kColsAt = 256;  // rows and columns of a thread block

// Half a warp a block of 128, a warp four rows' 256 columns; all four are on their way before the first is used.  The
// warp's eight scales are computed at once, a lane one of them, and handed back.  16384 rows of 14336 from 8192 tokens:
// 0.16 ms row by row, bound by issue slots (0.82 busy, 21 instructions a value, half of them the two products and
// conversions), 0.12 ms token by token (0.07 ms of bytes).  Six blocks of
// threads an SM: with four the whole call takes 862 us in place of 833.
template <typename T, bool VEC, bool CHAINS>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 2 ? 6 : 4) quantise_rows_kernel(RowQuant a) {
  __shared__ float s_scale[kRowsAt][2];
  pdl_wait();
  pdl_trigger();  // after the wait: what starts early may read what was there before this kernel
  if (blockIdx.y == 0)
    for (int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; i < a.n_ticket; i += (int64_t)gridDim.x * kRowThreads)
      a.ticket[i] = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.y * kColsAt + lane * 8;
  const bool direct = CHAINS && (int)blockIdx.x >= a.chained;
  const int n = direct ? *a.n_direct + 1 : a.n;
  // f(row) for every row that i stands for
  auto rows_of = [&](int i, auto f) {
    if constexpr (CHAINS) {
      if (direct)
        f(a.direct[i]);
      else
        for (int r = a.head[i]; r >= 0; r = a.next[r]) f(r);
    } else {
      f(i);
    }
  };
  auto source = [&](int i) -> const T* {  // nullptr: zeros
    const int t = direct ? a.rows[a.direct[i]] : CHAINS || !a.rows ? i : a.rows[i];
    return t >= 0 && t < a.n_tokens ? static_cast<const T*>(a.x) + t * a.ldx : nullptr;
  };
  const int64_t step = (int64_t)(direct ? gridDim.x - a.chained : gridDim.x) * kRowsAt;
  for (int64_t at = (int64_t)(direct ? blockIdx.x - a.chained : blockIdx.x) * kRowsAt; at < n; at += step) {
    const int r0 = (int)at;
    Raw8<T> v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = r0 + j * 8 + warp;
      const T* x = i < n ? source(i) : nullptr;
      v[j] = read8<VEC>(x, col, x ? a.cols : 0);
    }
    float mine = 0.f;  // the largest |x| of row lane & 3
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Top8<T> top;
      top.take(v[j]);
      float m = top.all();
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
      if ((lane & 3) == j) mine = m;
    }
    const Scale own(mine);
    if ((lane & 15) < 4) s_scale[(lane & 3) * 8 + warp][lane >> 4] = own.scale;
    uint32_t doubt = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = r0 + j * 8 + warp;
      const uint2 q = quantised8(v[j], __shfl_sync(~0u, own.inv, (lane & 16) + j), doubt, 4 * j);
      if (i < n && col < a.ldq)
        rows_of(i, [&](int r) { *reinterpret_cast<uint2*>(a.q + (int64_t)r * a.ldq + col) = q; });
    }
    __syncthreads();
    if (col >= a.ldq) doubt = 0;
    for (; doubt; doubt &= doubt - 1) {
      const int bit = __ffs(doubt) - 1, j = bit >> 2, k = 2 * (bit & 3), i = r0 + j * 8 + warp;
      if (i >= n) break;
      const float scale = s_scale[j * 8 + warp][lane >> 4];
      const uint16_t q = divided(source(i), col + k, a.cols, scale, scale);
      rows_of(i, [&](int r) { *reinterpret_cast<uint16_t*>(a.q + (int64_t)r * a.ldq + col + k) = q; });
    }
    if (threadIdx.x < 2 * kRowsAt) {
      const int b = threadIdx.x / kRowsAt, i = threadIdx.x % kRowsAt, blk = blockIdx.y * 2 + b;
      if (r0 + i < n && blk * kFp8Block < a.cols)
        rows_of(r0 + i, [&](int r) { a.scale[blk * a.block_step + r * a.row_step] = s_scale[i][b]; });
    }
    if (CHAINS) __syncthreads();  // the scales, before the next rows'
  }
}

// The rows of each token as chains, so that a token is quantised once; a chain's order is of no account.  Rows without a
// token, and those behind a token's first kChainMost (a chain is walked row after row), are listed for themselves.
// Everything that is counted begins at -1, as one fill leaves it.
constexpr int kChainMost = 16;
__global__ void __launch_bounds__(256) chain_rows_kernel(const int32_t* rows, int R, int n_tokens, int32_t* head, int32_t* count,
                                                         int32_t* n_direct, int32_t* next, int32_t* direct) {
  pdl_wait();
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < R; r += (int64_t)gridDim.x * 256) {
    const int t = rows[r];
    if (t >= 0 && t < n_tokens && atomicAdd(count + t, 1) + 1 < kChainMost)
      next[r] = atomicExch(head + t, (int)r);
    else
      direct[atomicAdd(n_direct, 1) + 1] = (int)r;
  }
}

// ------------------------------------------------------------------------------ tiles of 128 x 128
enum TileScale { kColumns, kSquare };

struct TileQuant {
  const void* x;
  int64_t ldx;
  int n_tokens;
  const int32_t* rows;     // token of each row, or nullptr: the row itself
  const int32_t* offsets;  // kColumns: [E + 1], the experts' rows; a tile's rows are 128 of one expert
  int E, R;
  int matrix_rows;         // kSquare: rows of each matrix; a tile's rows are 128 of one matrix
  int cols;
  uint8_t* q;              // kColumns: [tiles * 128][ldq], zeros past an expert's rows; kSquare: [rows][ldq]
  int ldq;
  float* scale;            // kColumns: [tiles][lds]; kSquare: [tiles][ceil(cols / 128)]
  int64_t lds;
  uint8_t* row_q;          // or nullptr: the same rows with scales along them, [R][ldq] and
  float* row_scale;        // [ceil(cols / 128)][R]
  uint32_t* ticket;
  int n_ticket;
};

constexpr int kTileThreads = 256;

// A block of threads takes tiles of the same 128 rows: a thread eight columns of eight rows, 16 apart.  The scales of
// the columns (or of the square) are computed by a thread each and shared.  16384 rows of 14336 in columns 0.21 ms, of
// 4096 both ways 0.10 ms: issue slots 0.5 busy, the rest barriers and loads that three blocks of threads an SM hide
// in part.
template <typename T, bool VEC, int KIND>
__global__ void __launch_bounds__(kTileThreads, sizeof(T) == 2 ? 3 : 2) quantise_tiles_kernel(TileQuant a) {
  __shared__ int s_row0[kFp8MaxExperts], s_rows[kFp8MaxExperts], s_tiles[kFp8MaxExperts + 1];
  __shared__ __align__(16) float s_top[8][kFp8Block], s_scale[kFp8Block], s_inv[kFp8Block];
  __shared__ float s_row_scale[kFp8Block];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.y == 0)
    for (int64_t i = (int64_t)blockIdx.x * kTileThreads + threadIdx.x; i < a.n_ticket; i += (int64_t)gridDim.x * kTileThreads)
      a.ticket[i] = 0;
  int64_t first;  // row of x (or of `rows`)
  int n;
  if constexpr (KIND == kColumns) {
    if (warp == 0)
      fp8_segments(a.offsets, a.E, a.R, lane, s_row0, s_rows, s_tiles, [](int m) { return (m + kFp8Block - 1) / kFp8Block; });
    __syncthreads();
    if ((int)blockIdx.x >= s_tiles[a.E]) return;
    int lo = 0, hi = a.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_tiles[mid] <= (int)blockIdx.x)
        lo = mid;
      else
        hi = mid;
    }
    const int at = ((int)blockIdx.x - s_tiles[lo]) * kFp8Block;
    first = s_row0[lo] + at;
    n = min(s_rows[lo] - at, kFp8Block);
  } else {
    const int per = (a.matrix_rows + kFp8Block - 1) / kFp8Block, m = blockIdx.x / per, at = (blockIdx.x - m * per) * kFp8Block;
    first = (int64_t)m * a.matrix_rows + at;
    n = min(a.matrix_rows - at, kFp8Block);
  }
  const int ty = threadIdx.x >> 4, c = (threadIdx.x & 15) * 8;
  const int64_t out0 = KIND == kColumns ? (int64_t)blockIdx.x * kFp8Block : first;
  auto source = [&](int i) -> const T* {  // row i of the tile in x, or nullptr
    int64_t t = -1;
    if (i < n) t = a.rows ? a.rows[first + i] : first + i;
    return t >= 0 && t < a.n_tokens ? static_cast<const T*>(a.x) + t * a.ldx : nullptr;
  };
  const T* src[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) src[j] = source(ty + 16 * j);
  for (int ct = blockIdx.y; ct * kFp8Block < a.ldq; ct += gridDim.y) {
    const int col = ct * kFp8Block + c;
    Raw8<T> v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = read8<VEC>(src[j], col, src[j] ? a.cols : 0);
    Top8<T> top;
#pragma unroll
    for (int j = 0; j < 8; ++j) top.take(v[j]);
    if constexpr (KIND == kSquare) {
      const float m = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top.all())));  // ordered as its bits, NaN above
      if (lane == 0) s_top[warp][0] = m;
    } else {
      top.across(16);
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s_top[warp][c + i] = top.get(i);
      }
    }
    uint32_t doubt_rows = 0;
    if (KIND == kColumns && a.row_q) {
      // along the rows, too: the half-warp's eight scales at once, a lane one of them
      float mine = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        Top8<T> row;
        row.take(v[j]);
        float m = row.all();
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
        if ((lane & 7) == j) mine = m;
      }
      const Scale own(mine);
      if ((lane & 15) < 8) s_row_scale[ty + 16 * (lane & 7)] = own.scale;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = ty + 16 * j;
        const uint2 q = quantised8(v[j], __shfl_sync(~0u, own.inv, (lane & 16) + j), doubt_rows, 4 * j);
        if (i < n && col < a.ldq) *reinterpret_cast<uint2*>(a.row_q + (first + i) * a.ldq + col) = q;
      }
    }
    __syncthreads();
    if (col >= a.ldq) doubt_rows = 0;
    for (; doubt_rows; doubt_rows &= doubt_rows - 1) {
      const int bit = __ffs(doubt_rows) - 1, i = ty + 16 * (bit >> 2), k = 2 * (bit & 3);
      if (i >= n) break;
      *reinterpret_cast<uint16_t*>(a.row_q + (first + i) * a.ldq + col + k) =
          divided(source(i), col + k, a.cols, s_row_scale[i], s_row_scale[i]);
    }
    uint32_t doubt = 0;
    if constexpr (KIND == kSquare) {
      float m = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = max_nan(m, s_top[w][0]);
      const Scale s(m);
      if (threadIdx.x == 0) a.scale[(int64_t)blockIdx.x * a.lds + ct] = s.scale;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint2 q = quantised8(v[j], s.inv, doubt, 4 * j);
        if (ty + 16 * j < n && col < a.ldq) *reinterpret_cast<uint2*>(a.q + (out0 + ty + 16 * j) * a.ldq + col) = q;
      }
      if (col >= a.ldq) doubt = 0;
      for (; doubt; doubt &= doubt - 1) {
        const int bit = __ffs(doubt) - 1, i = ty + 16 * (bit >> 2), k = 2 * (bit & 3);
        if (i >= n) break;
        *reinterpret_cast<uint16_t*>(a.q + (out0 + i) * a.ldq + col + k) =
            divided(source(i), col + k, a.cols, s.scale, s.scale);
      }
    } else {
      if (threadIdx.x < kFp8Block) {
        float m = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max_nan(m, s_top[w][threadIdx.x]);
        const Scale s(m);
        s_scale[threadIdx.x] = s.scale, s_inv[threadIdx.x] = s.inv;
        a.scale[(int64_t)blockIdx.x * a.lds + ct * kFp8Block + threadIdx.x] = s.scale;
        if (a.row_q && (int)threadIdx.x < n) a.row_scale[(int64_t)ct * a.R + first + threadIdx.x] = s_row_scale[threadIdx.x];
      }
      __syncthreads();
      uint32_t out[8][2] = {};
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 inv = *reinterpret_cast<const float2*>(s_inv + c + i);
        const Ends e0(inv.x), e1(inv.y);
        if (inv.x < 0.f || inv.y < 0.f) doubt |= 0xffu << 4 * i;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          out[j][i >> 2] |= quotients(v[j].get(i), v[j].get(i + 1), e0, e1, doubt, 4 * i + j) << (i & 2 ? 16 : 0);
      }
      if (col < a.ldq) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint2*>(a.q + (out0 + ty + 16 * j) * a.ldq + col) = make_uint2(out[j][0], out[j][1]);
        for (; doubt; doubt &= doubt - 1) {
          const int bit = __ffs(doubt) - 1, i = ty + 16 * (bit & 7), k = 2 * (bit >> 3);
          *reinterpret_cast<uint16_t*>(a.q + (out0 + i) * a.ldq + col + k) =
              divided(source(i), col + k, a.cols, s_scale[c + k], s_scale[c + k + 1]);
        }
      }
    }
    __syncthreads();  // the next tile's maxima
  }
}

// --------------------------------------------------------------------------------------- host side
constexpr int kMaxK = 65536, kMaxN = 131072;
constexpr int kWaitUs = 2000000, kMaxWaitUs = 10000000;

int check_config(const colibri_moe_fp8_config_t* c) {
  if (!c || c->in_features <= 0 || c->out_features <= 0 || c->num_experts <= 0 || !ops_dtype(c->dtype) ||
      !ops_dtype(c->out_dtype) || (c->trusted_pointers & ~1) || c->wait_limit_us < 0 || c->wait_limit_us > kMaxWaitUs)
    return COLIBRI_ERR_INVALID_ARG;
  if (c->in_features % 16 || c->in_features > kMaxK || c->out_features > kMaxN || c->num_experts > kFp8MaxExperts)
    return COLIBRI_ERR_UNSUPPORTED;
  return COLIBRI_OK;
}
// The clock is read once in 64 tries of about 8 us, at every one under a millisecond's limit.
Fp8Limit limit_of(const colibri_moe_fp8_config_t* c) {
  const int us = c->wait_limit_us ? c->wait_limit_us : kWaitUs;
  return {us * 1000ull, us < 1000 ? 0u : 63u};
}

int up(int n, int to) { return (n + to - 1) / to * to; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int blocks_of(int n) { return (n + kFp8Block - 1) / kFp8Block; }

// The status word's address on the current device, looked up once.
int* status_word(int device) {
  static std::mutex mu;
  static int* at[kOpsMaxDevices] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (!at[device] && cudaGetSymbolAddress(reinterpret_cast<void**>(&at[device]), g_status) != cudaSuccess) {
    cudaGetLastError();
    at[device] = nullptr;
  }
  return at[device];
}

template <typename F>
cudaError_t with_type(int32_t t, F f) {
  return t == COLIBRI_DTYPE_F32 ? f(float()) : f(__nv_bfloat16());
}
bool vectors(const void* x, int64_t ldx, int cols) { return ops_aligned16(x) && ldx % 8 == 0 && cols % 8 == 0; }

template <bool CHAINS>
cudaError_t quantise_rows(int dtype, const RowQuant& a, int direct_blocks, cudaStream_t s) {
  const unsigned blocks = (unsigned)(((int64_t)a.n + kRowsAt - 1) / kRowsAt);
  const dim3 grid(blocks + direct_blocks, (a.ldq + kColsAt - 1) / kColsAt), block(kRowThreads);
  return with_type(dtype, [&](auto t) {
    return vectors(a.x, a.ldx, a.cols) ? pdl_launch(quantise_rows_kernel<decltype(t), true, CHAINS>, grid, block, 0, s, a)
                                       : pdl_launch(quantise_rows_kernel<decltype(t), false, CHAINS>, grid, block, 0, s, a);
  });
}
// Whether tokens are quantised once and written to each of their rows: where that saves more than the chains' two launches
// cost.  Whole calls, us, without / with, by the values that are saved: 8 million 78 / 78, 476 / 475; 10 million 78 / 80; 42
// million 211 / 197; 117 million (8192 tokens of 14336, two rows each) 889 / 833.
bool chained(const int32_t* rows, int n_tokens, int R, int K) {
  return rows && n_tokens > 0 && n_tokens < R && (int64_t)(R - n_tokens) * K >= (1 << 24);
}
template <int KIND>
cudaError_t quantise_tiles(int dtype, const TileQuant& a, unsigned tiles, int sms, cudaStream_t s) {
  // column tiles of the same rows to one block of threads, as many blocks as fill the card
  const int across = (a.ldq + kFp8Block - 1) / kFp8Block;
  const unsigned share = (unsigned)std::min<int64_t>(across, std::max<int64_t>(1, ((int64_t)sms * 12 + tiles - 1) / tiles));
  const dim3 grid(tiles, share), block(kTileThreads);
  return with_type(dtype, [&](auto t) {
    return vectors(a.x, a.ldx, a.cols) ? pdl_launch(quantise_tiles_kernel<decltype(t), true, KIND>, grid, block, 0, s, a)
                                       : pdl_launch(quantise_tiles_kernel<decltype(t), false, KIND>, grid, block, 0, s, a);
  });
}

// ---- tensor maps: bytes in boxes of 128 columns under the 128-byte swizzle
bool map_of(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_rows(CUtensorMap* m, const void* q, int64_t rows, int ldq, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)ldq, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ldq};
  return map_of(m, q, 2, dims, strides, box_rows);
}
bool map_weights(CUtensorMap* m, const void* w, const colibri_moe_fp8_config_t* c, int box_rows) {
  const cuuint64_t K = c->in_features, N = c->out_features;
  const cuuint64_t dims[3] = {K, N, (cuuint64_t)c->num_experts}, strides[2] = {K, N * K};
  return map_of(m, w, 3, dims, strides, box_rows);
}

// Wide tiles where there are two or more an SM: a block's sum costs its takers much the same waits however wide it is, but
// few tiles fill the SMs unevenly.  us on a GB300, narrow / wide:
//   one token, two experts of 4096 x 14336 x 2 (224 wide tiles)  47 / 50     four tokens (672)  106 / 99
//   rows of an expert   64 / 128 / 256, eight experts of 2048 x 5632 x 2     47 / 62 / 101   46 / 52 / 77
//                                       eight of 4096 x 4096                 38 / 47 /  69   36 / 46 / 61
//                                       64 of 2048 x 1408, unevenly loaded   46 / 54 /  74   44 / 48 / 64
// (CTA pairs on tiles of 256 x 256 took 62, 48, 70 at 128 rows and 92, 67, 79 at 256; 8192 tokens, 14336 x 4096: 0.95 ms
// in all against 0.87: what a block's sum waits for then comes from two SMs.)
Fp8Form wide_from(int64_t tiles, int sms) { return tiles >= 2 * (int64_t)sms ? kFp8Wide : kFp8Narrow; }
Fp8Form rows_form(int R, int E, int cols, int sms) {
  const int used = std::min(E, R), mean = R / used;  // the exact numbers are on the device
  return wide_from((int64_t)used * ((mean + 127) / 128) * ((cols + 255) / 256), sms);
}
// The weights' gradient sums over an expert's rows: of up to two blocks a wide tile is mostly its epilogue (256 rows, eight
// experts of 1024 x 1408: 53 / 57; 512, 16 of 2048 x 1408: 181 / 168 with the rows' gradient).
Fp8Form weights_form(int R, int E, int N, int K, int sms) {
  if (R / std::min(E, R) <= 2 * kFp8Block) return kFp8Narrow;
  return wide_from((int64_t)E * ((N + 127) / 128) * ((K + 255) / 256), sms);
}

struct Workspace {
  size_t q, scale, ticket, partial, chain;   // rows' values and scales; forward: chains of tokens' rows
  size_t dq, dscale, xq, xscale;             // by columns, for the weights' gradient
  size_t bytes;
  int items, blocks;                         // of split tiles; blocks of 128 rows of one expert, at most
};
Workspace workspace_of(const colibri_moe_fp8_config_t* c, int R, int sms, bool backward) {
  Workspace w = {};
  const int cols = backward ? up(c->out_features, 16) : c->in_features;
  w.items = 2 * sms;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += round256(bytes);
    return was;
  };
  w.q = take((size_t)R * cols);
  w.scale = take((size_t)R * blocks_of(cols) * sizeof(float));
  w.ticket = take(2 * w.items * sizeof(uint32_t));
  w.partial = take((size_t)w.items * 128 * 256 * sizeof(float));
  if (!backward) w.chain = take((4 * (size_t)R + 1) * sizeof(int32_t));  // more than two of each token and two of each row
  if (backward) {
    w.blocks = (int)((R + 127 * (int64_t)std::min(c->num_experts, R)) / 128);
    w.dq = take((size_t)w.blocks * 128 * cols);
    w.dscale = take((size_t)w.blocks * up(c->out_features, 256) * sizeof(float));
    w.xq = take((size_t)w.blocks * 128 * c->in_features);
    w.xscale = take((size_t)w.blocks * up(c->in_features, 256) * sizeof(float));
  }
  w.bytes = at;
  return w;
}

int check_pointers(const colibri_moe_fp8_config_t* c, std::initializer_list<const void*> ps, int device) {
  for (const void* p : ps)
    if (p && !c->trusted_pointers && !ops_on_device(p, device)) return COLIBRI_ERR_INVALID_ARG;
  return COLIBRI_OK;
}
int workspace_bytes_of(const colibri_moe_fp8_config_t* c, int32_t n_tokens, int32_t R, size_t* bytes, bool backward) {
  const int rc = check_config(c);
  if (rc) return rc;
  if (!bytes || n_tokens < 0 || R < 0) return COLIBRI_ERR_INVALID_ARG;
  if (R > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  *bytes = R ? workspace_of(c, R, sms, backward).bytes : 0;
  return COLIBRI_OK;
}

}  // namespace
}  // namespace colibri

using namespace colibri;

extern "C" int colibri_moe_fp8_quantize(const colibri_moe_fp8_config_t* cfg, const void* x, int64_t ldx, int32_t n,
                                        int32_t square, uint8_t* q, float* scale, void* stream) {
  const int rc = check_config(cfg);
  if (rc) return rc;
  if (n < 0 || (square & ~1) || (square && n % cfg->num_experts)) return COLIBRI_ERR_INVALID_ARG;
  if (n > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  if (n == 0) return COLIBRI_OK;
  if (!x || !q || !scale || ldx < cfg->in_features || !ops_aligned16(q)) return COLIBRI_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  if (const int bad = check_pointers(cfg, {x, q, scale}, device)) return bad;
  const int K = cfg->in_features;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (square) {
    TileQuant a = {};
    a.x = x, a.ldx = ldx, a.n_tokens = n, a.matrix_rows = n / cfg->num_experts, a.cols = a.ldq = K, a.q = q;
    a.scale = scale, a.lds = blocks_of(K);
    e = quantise_tiles<kSquare>(cfg->dtype, a, (unsigned)cfg->num_experts * blocks_of(a.matrix_rows), sms, s);
  } else {
    e = quantise_rows<false>(cfg->dtype, {x, ldx, n, nullptr, n, K, q, K, scale, blocks_of(K), 1, nullptr, 0}, 0, s);
  }
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}

extern "C" int colibri_moe_fp8_experts_workspace(const colibri_moe_fp8_config_t* cfg, int32_t n_tokens, int32_t R,
                                                 size_t* bytes) {
  return workspace_bytes_of(cfg, n_tokens, R, bytes, false);
}

extern "C" int colibri_moe_fp8_experts(const colibri_moe_fp8_config_t* cfg, const void* x, int64_t ldx,
                                       int32_t n_tokens, const int32_t* rows, int32_t R, const int32_t* offsets,
                                       const uint8_t* w, const float* w_scale, const uint8_t* w3,
                                       const float* w3_scale, void* y, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  const int rc = check_config(cfg);
  if (rc) return rc;
  if (n_tokens < 0 || R < 0 || (!rows && R > n_tokens)) return COLIBRI_ERR_INVALID_ARG;
  if (R > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  if (R == 0) return COLIBRI_OK;
  const int K = cfg->in_features, N = cfg->out_features, E = cfg->num_experts;
  if ((n_tokens > 0 && (!x || ldx < K)) || !offsets || !w || !w_scale || !y || (w3 != nullptr) != (w3_scale != nullptr))
    return COLIBRI_ERR_INVALID_ARG;
  if (!ops_aligned16(w) || !ops_aligned16(w3)) return COLIBRI_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return COLIBRI_ERR_INVALID_ARG;
  if (workspace_bytes < workspace_of(cfg, R, 0, false).bytes) return COLIBRI_ERR_INVALID_ARG;  // what any device needs
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  const Workspace lay = workspace_of(cfg, R, sms, false);
  if (workspace_bytes < lay.bytes) return COLIBRI_ERR_INVALID_ARG;
  if (const int bad = check_pointers(cfg, {n_tokens ? x : nullptr, rows, offsets, w, w_scale, w3, w3_scale, y, workspace},
                                     device))
    return bad;
  int* word = status_word(device);
  if (!word) return COLIBRI_ERR_CUDA;
  const bool gated = w3 != nullptr;
  const Fp8Form form = rows_form(R, E, gated ? 2 * N : N, sms);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  Fp8Maps maps;
  bool ok = true;
  for (int i = 0; i < kFp8TokMaps; ++i) ok = ok && map_rows(&maps.a[i], ws + lay.q, R, K, 32 << i);
  const int box = !gated ? 128 : form == kFp8Narrow ? 32 : 64;
  ok = ok && map_weights(&maps.b, w, cfg, box) && map_weights(&maps.b3, gated ? w3 : w, cfg, box);
  if (!ok) return COLIBRI_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* scale = reinterpret_cast<float*>(ws + lay.scale);
  uint32_t* ticket = reinterpret_cast<uint32_t*>(ws + lay.ticket);
  RowQuant quant = {x, ldx, n_tokens, rows, R, K, ws + lay.q, K, scale, 1, R, ticket, lay.items};
  if (chained(rows, n_tokens, R, K)) {  // n_tokens < R
    int32_t* head = reinterpret_cast<int32_t*>(ws + lay.chain);
    int32_t *count = head + n_tokens, *n_direct = count + n_tokens, *next = n_direct + 1, *direct = next + R;
    if (cudaMemsetAsync(head, 0xff, (2 * (size_t)n_tokens + 1) * sizeof(int32_t), s) != cudaSuccess) return COLIBRI_ERR_CUDA;
    const dim3 grid((unsigned)std::min<int64_t>(((int64_t)R + 255) / 256, (int64_t)sms * 8));
    if (pdl_launch(chain_rows_kernel, grid, dim3(256), 0, s, rows, R, n_tokens, head, count, n_direct, next, direct) !=
        cudaSuccess)
      return COLIBRI_ERR_CUDA;
    quant.head = head, quant.next = next, quant.direct = direct, quant.n_direct = n_direct, quant.n = n_tokens;
    quant.chained = (n_tokens + kRowsAt - 1) / kRowsAt;
    if (quantise_rows<true>(cfg->dtype, quant, 2 * sms, s) != cudaSuccess) return COLIBRI_ERR_CUDA;
  } else if (quantise_rows<false>(cfg->dtype, quant, 0, s) != cudaSuccess) {
    return COLIBRI_ERR_CUDA;
  }
  const Fp8Args a = {offsets, scale, R, w_scale, w3_scale, nullptr, 0, y, reinterpret_cast<float*>(ws + lay.partial),
                     ticket, lay.items, R, E, N, K, limit_of(cfg), word};
  const cudaError_t e =
      launch_fp8_forward(maps, a, form, gated, cfg->out_dtype == COLIBRI_DTYPE_BF16, device, sms, s);
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}

extern "C" int colibri_moe_fp8_experts_backward_workspace(const colibri_moe_fp8_config_t* cfg, int32_t n_tokens,
                                                          int32_t R, size_t* bytes) {
  return workspace_bytes_of(cfg, n_tokens, R, bytes, true);
}

extern "C" int colibri_moe_fp8_experts_backward(const colibri_moe_fp8_config_t* cfg, const void* d_y, int64_t ld_dy,
                                                const void* x, int64_t ldx, int32_t n_tokens, const int32_t* rows,
                                                int32_t R, const int32_t* offsets, const uint8_t* w,
                                                const float* w_scale, void* d_rows, void* d_w, void* workspace,
                                                size_t workspace_bytes, void* stream) {
  const int rc = check_config(cfg);
  if (rc) return rc;
  if (n_tokens < 0 || R < 0 || (d_w && !rows && R > n_tokens)) return COLIBRI_ERR_INVALID_ARG;
  if (R > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  const int K = cfg->in_features, N = cfg->out_features, E = cfg->num_experts;
  if (!d_rows && !d_w) return COLIBRI_ERR_INVALID_ARG;
  if ((d_rows != nullptr) != (w != nullptr) || (w != nullptr) != (w_scale != nullptr) || !ops_aligned16(w))
    return COLIBRI_ERR_INVALID_ARG;
  if (R > 0 && (!d_y || ld_dy < N || !offsets)) return COLIBRI_ERR_INVALID_ARG;
  if (!ops_aligned16(d_w) || (d_w && R > 0 && n_tokens > 0 && (!x || ldx < K))) return COLIBRI_ERR_INVALID_ARG;
  if (R > 0) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return COLIBRI_ERR_INVALID_ARG;
    if (workspace_bytes < workspace_of(cfg, R, 0, true).bytes) return COLIBRI_ERR_INVALID_ARG;
  }
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const int bad = check_pointers(cfg, {d_w}, device)) return bad;
  if (R == 0) {
    if (!d_w) return COLIBRI_OK;
    const size_t bytes = (size_t)E * N * K * ops_elem(cfg->out_dtype);
    return cudaMemsetAsync(d_w, 0, bytes, s) == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
  }
  const Workspace lay = workspace_of(cfg, R, sms, true);
  if (workspace_bytes < lay.bytes) return COLIBRI_ERR_INVALID_ARG;
  if (const int bad = check_pointers(cfg, {d_y, d_w && n_tokens ? x : nullptr, d_w ? rows : nullptr, offsets, w, w_scale,
                                           d_rows, workspace},
                                     device))
    return bad;
  int* word = status_word(device);
  if (!word) return COLIBRI_ERR_CUDA;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const int ldn = up(N, 16);
  float* scale = reinterpret_cast<float*>(ws + lay.scale);
  float* partial = reinterpret_cast<float*>(ws + lay.partial);
  uint32_t* ticket = reinterpret_cast<uint32_t*>(ws + lay.ticket);  // the products' tickets, one after the other
  float *dscale = reinterpret_cast<float*>(ws + lay.dscale), *xscale = reinterpret_cast<float*>(ws + lay.xscale);
  Fp8Maps maps, wmaps;
  if (d_rows) {
    bool ok = true;
    for (int i = 0; i < kFp8TokMaps; ++i) ok = ok && map_rows(&maps.a[i], ws + lay.q, R, ldn, 32 << i);
    if (!ok || !map_weights(&maps.b, w, cfg, 128)) return COLIBRI_ERR_CUDA;
    maps.b3 = maps.b;
  }
  if (d_w) {
    bool ok = map_rows(&wmaps.a[0], ws + lay.dq, (int64_t)lay.blocks * 128, ldn, 128);
    ok = ok && map_rows(&wmaps.b, ws + lay.xq, (int64_t)lay.blocks * 128, K, 128);
    if (!ok) return COLIBRI_ERR_CUDA;
    wmaps.a[1] = wmaps.a[2] = wmaps.a[0];
    wmaps.b3 = wmaps.b;
  }
  cudaError_t e = cudaSuccess;
  if (d_w) {
    TileQuant t = {};
    t.x = d_y, t.ldx = ld_dy, t.n_tokens = R, t.offsets = offsets, t.E = E, t.R = R, t.cols = N, t.ldq = ldn;
    t.q = ws + lay.dq, t.scale = dscale, t.lds = up(N, 256);
    t.row_q = d_rows ? ws + lay.q : nullptr, t.row_scale = scale;
    t.ticket = ticket, t.n_ticket = 2 * lay.items;
    e = quantise_tiles<kColumns>(cfg->dtype, t, lay.blocks, sms, s);
    if (e != cudaSuccess) return COLIBRI_ERR_CUDA;
    t.x = x, t.ldx = ldx, t.n_tokens = n_tokens, t.rows = rows, t.cols = t.ldq = K;
    t.q = ws + lay.xq, t.scale = xscale, t.lds = up(K, 256), t.row_q = nullptr, t.n_ticket = 0;
    e = quantise_tiles<kColumns>(cfg->dtype, t, lay.blocks, sms, s);
  } else {
    e = quantise_rows<false>(
        cfg->dtype, {d_y, ld_dy, R, nullptr, R, N, ws + lay.q, ldn, scale, 1, R, ticket, 2 * lay.items}, 0, s);
  }
  if (e != cudaSuccess) return COLIBRI_ERR_CUDA;
  if (d_rows) {
    const Fp8Args a = {offsets, scale, R, w_scale, nullptr, nullptr, 0, d_rows, partial, ticket, lay.items, R, E, N, K,
                       limit_of(cfg), word};
    e = launch_fp8_rows(maps, a, rows_form(R, E, K, sms), cfg->dtype == COLIBRI_DTYPE_BF16, device, sms, s);
    if (e != cudaSuccess) return COLIBRI_ERR_CUDA;
  }
  if (d_w) {
    const Fp8Args a = {offsets, dscale, up(N, 256), nullptr, nullptr, xscale, up(K, 256), d_w, partial,
                       ticket + lay.items, lay.items, R, E, N, K, limit_of(cfg), word};
    e = launch_fp8_weights(wmaps, a, weights_form(R, E, N, K, sms), cfg->out_dtype == COLIBRI_DTYPE_BF16, device, sms, s);
  }
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}

extern "C" int colibri_moe_fp8_status(int32_t* status) {
  if (!status) return COLIBRI_ERR_INVALID_ARG;
  int device = 0, sms = 0, v = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  static std::mutex mu;  // g_taken holds one caller's answer at a time
  std::lock_guard<std::mutex> lock(mu);
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) {
    take_status_kernel<<<1, 1>>>();
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_taken, sizeof(int));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return COLIBRI_ERR_CUDA;
  }
  *status = v;
  return COLIBRI_OK;
}
