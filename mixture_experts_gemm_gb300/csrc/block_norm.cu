// Norms before and after a block, fused with the block's gate and the residual scale.
//
//   z  = norm_after(y) * w_a + b_a            (y: the block's output; norm none, RMS or layer)
//   x1 = residual_scale * x + block_scale * gate * z
//   p  = norm_before(x1) * w_b + b_b          (the next block's input; from x1 as stored)
//   RMS:   norm(v) = v / sqrt(mean(v^2) + eps)
//   layer: norm(v) = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps)
//
// The backward pass, with D the gradient of x1 from both of its uses, n = norm(v), r = 1 / deviation:
//   d_v = r (d_n - n mean(d_n n) [- mean(d_n), layer])     d_n = d_out * w
//   D   = d_x1 + (d_v of norm_before at x1),  d_x = residual_scale * D,  d_z = block_scale * gate * D
//   d_y = d_v of norm_after at y,  and column sums over the rows for w_a, b_a, w_b, b_b and the gate.
//
// HBM-bound: each of x, y read once, x1, p written once; a row stays in registers between the loads
// and the stores, so both norms cost no second pass.  All statistics and sums are fp32, the variance is
// taken about the mean in a second sum over the registers (no E[v^2] - mean^2 cancellation).
//
// Measured on one GB300 (bf16 stream, RMS norms, 8192 x 4096): forward with an fp32 block output 67 us
// (336 MB, 5.0 TB/s, 0.74 of the measured copy rate), backward 115 us (403 MB, 3.5 TB/s, 0.51).  Neither DRAM
// (0.54 and 0.41 busy) nor instruction issue (0.52 and 0.65 of the slots; the forward pass executes about 320
// instructions a warp and row, for 8 columns a lane) is full: between them stand the row sums' barriers, which
// 30 and 16 resident warps an SM do not hide.  Without the rows ahead the forward pass took 92 us, with more
// instructions 78.  Odd widths take single-column accesses: 3001 x 1409 fp32, layer norms, 29 us, floor 10.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "ops_common.cuh"
#include "tcgen05_ptx.cuh"

namespace colibri {
namespace {

struct NormArgs {
  const void *x, *y, *wa, *ba, *wb, *bb, *gate;
  void *x1, *p;                    // forward outputs
  const void *dx1, *dp;            // backward inputs
  void *dx, *dy;                   // backward outputs
  float* part;                     // backward: [blocks][kSlots][d] column sums of each block
  float* dgate;                    // backward: [gates][d]; groups inside one block's rows go straight here
  int64_t ldx, ldy, lddx1, lddp;   // row strides, elements
  int64_t rpg;                     // rows per gate row
  int rows_per_gate;               // the same, at most T
  int T, d, after, before, param_bf16;
  int rows_per_block;              // backward
  float alpha, beta, eps;
};

// Column-sum slots of a block: the four parameter vectors, the gate row that began in an earlier block
// and the one that goes on in the next.
enum { kSumWb, kSumBb, kSumWa, kSumBa, kSumGateFirst, kSumGateLast, kSlots };

// How a thread's 8 * C values lie in a row: VEC, chunks of 8 consecutive columns (16-byte accesses; d,
// row strides and addresses are multiples of 16 bytes); else single columns a block width apart.
template <bool VEC, typename T>
__device__ __forceinline__ void load_cols(const T* row, int c, int d, float (&v)[8]) {
  if constexpr (VEC) {
    const int col = (c * blockDim.x + threadIdx.x) * 8;
    if (col < d) {
      load8(row + col, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = (c * 8 + j) * blockDim.x + threadIdx.x;
      v[j] = col < d ? to_float(row[col]) : 0.f;
    }
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_cols(T* row, int c, int d, const float (&v)[8]) {
  if constexpr (VEC) {
    const int col = (c * blockDim.x + threadIdx.x) * 8;
    if (col < d) store8(row + col, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = (c * 8 + j) * blockDim.x + threadIdx.x;
      if (col < d) row[col] = from_float<T>(v[j]);
    }
  }
}
// What a thread holds of the rows ahead of the one it works on.  kRing: kDepth - 1 rows on their way by
// asynchronous copies into 16-byte slots of shared memory that this thread alone writes and reads (no
// barrier; registers hold one row only).  Else the next row's values in registers.
constexpr int kDepth = 3;
enum { kScalar, kVector, kRing };
template <int MODE, typename T>
struct Ahead {  // kScalar
  T v[8];
  static constexpr int kVecs = 0;
  __device__ __forceinline__ void load(uint4*, const T* row, int c, int d) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = (c * 8 + j) * blockDim.x + threadIdx.x;
      v[j] = col < d ? row[col] : T(0.f);
    }
  }
  __device__ __forceinline__ void get(const uint4*, int, int, float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = to_float(v[j]);
  }
};
template <typename T>
struct Ahead<kVector, T> {
  uint4 v[sizeof(T) / 2];
  static constexpr int kVecs = 0;
  __device__ __forceinline__ void load(uint4*, const T* row, int c, int d) {
    const int col = (c * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      v[i] = col < d ? reinterpret_cast<const uint4*>(row + col)[i] : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(const uint4*, int, int, float (&o)[8]) const {
    load8(reinterpret_cast<const T*>(v), o);
  }
};
template <typename T>
struct Ahead<kRing, T> {
  static constexpr int kVecs = sizeof(T) / 2;  // slots of eight values, a block width apart
  __device__ __forceinline__ void load(uint4* slot, const T* row, int c, int d) {
    const int col = (c * blockDim.x + threadIdx.x) * 8;
    if (col >= d) return;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      ptx::cp_async_16(ptx::smem_u32(slot + i * blockDim.x), reinterpret_cast<const uint4*>(row + col) + i);
  }
  __device__ __forceinline__ void get(const uint4* slot, int, int, float (&o)[8]) const {
    uint4 v[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = slot[i * blockDim.x];
    load8(reinterpret_cast<const T*>(v), o);
  }
};
// The slots of columns past d are never copied into: zeros, once, keep them out of the row sums.
template <int MODE>
__device__ __forceinline__ void clear_slots(uint4* slots, int n) {
  if (MODE == kRing)
    for (int i = 0; i < n; ++i) slots[i * blockDim.x + threadIdx.x] = make_uint4(0, 0, 0, 0);
}

template <bool VEC>
__device__ __forceinline__ bool col_in(int c, int j, int d) {
  return (VEC ? (c * (int)blockDim.x + (int)threadIdx.x) * 8 + j : (c * 8 + j) * (int)blockDim.x + (int)threadIdx.x) < d;
}
template <bool VEC>
__device__ __forceinline__ void load_param(const void* p, int bf16, int64_t row, int c, int d, float (&v)[8]) {
  if (bf16)
    load_cols<VEC>(static_cast<const __nv_bfloat16*>(p) + row * d, c, d, v);
  else
    load_cols<VEC>(static_cast<const float*>(p) + row * d, c, d, v);
}

// f(c, j) for every value of a thread.
template <int C, typename F>
__device__ __forceinline__ void each(F f) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) f(c, j);
}

// Subtracts the row's mean (layer); the values past d stay zero.
template <bool VEC, int C>
__device__ __forceinline__ void center(float (&v)[C][8], float mean, int d) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[c][j] = col_in<VEC>(c, j, d) ? v[c][j] - mean : 0.f;
}
template <int C>
__device__ __forceinline__ float sum_of(const float (&v)[C][8]) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[c][j];
  return s;
}
template <int C>
__device__ __forceinline__ float dot_of(const float (&v)[C][8], const float (&w)[C][8]) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(v[c][j], w[c][j], s);
  return s;
}

// v <- (v [- mean]) and returns 1 / deviation.
template <bool VEC, int C, bool LAYER>
__device__ __forceinline__ float norm_stats(float (&v)[C][8], int kind, int d, float inv_d, float eps, float* buf,
                                            int& turn) {
  if (LAYER && kind == COLIBRI_NORM_LAYER) {
    float s[1] = {sum_of(v)};
    block_sum(s, buf, turn);
    center<VEC>(v, s[0] * inv_d, d);
  }
  float s[1] = {dot_of(v, v)};
  block_sum(s, buf, turn);
  return rsqrtf(fmaf(s[0], inv_d, eps));
}

// The vectors of a call: in registers where a thread has one chunk of columns, else loaded for every row.
template <bool VEC, int C, bool BIAS>
struct Vectors {
  static constexpr bool kKeep = C == 1;
  float wa[C][8], wb[C][8], g[C][8], ba[BIAS ? C : 1][8], bb[BIAS ? C : 1][8];
  int group = -1;
  __device__ __forceinline__ void load(const NormArgs& a) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (a.after) load_param<VEC>(a.wa, a.param_bf16, 0, c, a.d, wa[c]);
      if (a.before) load_param<VEC>(a.wb, a.param_bf16, 0, c, a.d, wb[c]);
      if constexpr (BIAS) {
        if (a.ba) load_param<VEC>(a.ba, a.param_bf16, 0, c, a.d, ba[c]);
        if (a.bb) load_param<VEC>(a.bb, a.param_bf16, 0, c, a.d, bb[c]);
      }
    }
  }
  __device__ __forceinline__ void load_gate(const NormArgs& a, int now) {
    if (kKeep && now == group) return;
    group = now;
#pragma unroll
    for (int c = 0; c < C; ++c) load_param<VEC>(a.gate, a.param_bf16, now, c, a.d, g[c]);
  }
};

// A block walks over rows; while it works on one, the loads of the next are in flight, so that the loads
// do not wait for the row sums.  BIAS: either norm is a layer norm (with or without bias vectors).
template <typename S, typename Y, int MODE, int C, bool BIAS, int MAXT, int BLOCKS>
__global__ void __launch_bounds__(MAXT, BLOCKS) block_norm_kernel(NormArgs a) {
  __shared__ float buf[kSumBuf];
  extern __shared__ uint4 slots[];
  constexpr bool VEC = MODE != kScalar, RING = MODE == kRing;
  int turn = 0;
  using AX = Ahead<MODE, S>;
  using AY = Ahead<MODE, Y>;
  Vectors<VEC, C, BIAS> v;
  AX rx[C];
  AY ry[C];
  const int row_slots = (AX::kVecs + (a.y ? AY::kVecs : 0)) * C * blockDim.x;
  pdl_wait();
  clear_slots<MODE>(slots, kDepth * (AX::kVecs + (a.y ? AY::kVecs : 0)) * C);
  auto fetch = [&](int row, int stage) {
    if (row < a.T) {
      uint4* slot = slots + stage * row_slots + threadIdx.x;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        rx[c].load(slot, static_cast<const S*>(a.x) + row * a.ldx, c, a.d);
        slot += AX::kVecs * blockDim.x;
        if (a.y) {
          ry[c].load(slot, static_cast<const Y*>(a.y) + row * a.ldy, c, a.d);
          slot += AY::kVecs * blockDim.x;
        }
      }
    }
    if (RING) ptx::cp_async_commit();
  };
  const int step = gridDim.x;
  const float inv_d = 1.f / a.d;
  const bool one_gate = a.rows_per_gate >= a.T;
  for (int i = 0; i < (RING ? kDepth - 1 : 1); ++i) fetch(blockIdx.x + i * step, i);
  if (v.kKeep) v.load(a);
  int stage = 0;
  for (int row = blockIdx.x; row < a.T; row += step) {
    float x[C][8], z[C][8];
    if constexpr (RING) {
      fetch(row + (kDepth - 1) * step, stage ? stage - 1 : kDepth - 1);
      ptx::cp_async_wait<kDepth - 1>();
    }
    const uint4* slot = slots + stage * row_slots + threadIdx.x;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      rx[c].get(slot, c, a.d, x[c]);
      slot += AX::kVecs * blockDim.x;
      if (a.y) {
        ry[c].get(slot, c, a.d, z[c]);
        slot += AY::kVecs * blockDim.x;
      }
    }
    if (++stage == kDepth) stage = 0;
    if (!RING) fetch(row + step, 0);
    if (a.gate) v.load_gate(a, one_gate ? 0 : row / a.rows_per_gate);
    if (!v.kKeep) v.load(a);
    if (a.y) {
      if (a.after) {
        const float r = norm_stats<VEC, C, BIAS>(z, a.after, a.d, inv_d, a.eps, buf, turn);
        each<C>([&](int c, int j) { z[c][j] *= r * v.wa[c][j]; });
        if (BIAS && a.ba) each<C>([&](int c, int j) { z[c][j] += v.ba[BIAS ? c : 0][j]; });
      }
      if (a.gate) each<C>([&](int c, int j) { z[c][j] *= v.g[c][j]; });
      // the next norm reads x1 as it is stored, rounded to the stream's type
      each<C>([&](int c, int j) {
        x[c][j] = to_float(from_float<S>(fmaf(a.beta, z[c][j], a.alpha * x[c][j])));
      });
#pragma unroll
      for (int c = 0; c < C; ++c) {
        store_cols<VEC>(static_cast<S*>(a.x1) + (int64_t)row * a.d, c, a.d, x[c]);
      }
    }
    if (a.before) {
      const float r = norm_stats<VEC, C, BIAS>(x, a.before, a.d, inv_d, a.eps, buf, turn);
      each<C>([&](int c, int j) { x[c][j] *= r * v.wb[c][j]; });
      if (BIAS && a.bb) each<C>([&](int c, int j) { x[c][j] += v.bb[BIAS ? c : 0][j]; });
#pragma unroll
      for (int c = 0; c < C; ++c) {
        store_cols<VEC>(static_cast<S*>(a.p) + (int64_t)row * a.d, c, a.d, x[c]);
      }
    }
  }
}

// The gate row of group g lies in [g * rpg, (g + 1) * rpg); block b owns rows [b * R, (b + 1) * R).
// A group inside one block is written by it; one that crosses blocks leaves a partial sum in slot
// kSumGateLast of the block where it begins and kSumGateFirst of every later one.
template <bool VEC, int C>
__device__ __forceinline__ void flush_gate(const NormArgs& a, int64_t g, int r0, int r1, float (&acc)[C][8]) {
  const int64_t first = g * a.rpg, last = min((g + 1) * a.rpg, (int64_t)a.T) - 1;
  float* out = first >= r0 && last < r1
                   ? a.dgate + g * a.d
                   : a.part + ((int64_t)blockIdx.x * kSlots + (first < r0 ? kSumGateFirst : kSumGateLast)) * a.d;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    store_cols<VEC>(out, c, a.d, acc[c]);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[c][j] = 0.f;
  }
}

// A block takes consecutive rows and keeps the column sums of its own columns in registers; the sums
// of all blocks are added by norm_sums_kernel in block order (no atomics: the same bits every time).
// BIAS: either norm is a layer norm (two more column sums).
template <typename S, typename Y, int MODE, int C, bool BIAS, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_backward_kernel(NormArgs a) {
  __shared__ float buf[kSumBuf];
  extern __shared__ uint4 slots[];
  constexpr bool VEC = MODE != kScalar, RING = MODE == kRing;
  int turn = 0;
  float swb[C][8] = {}, swa[C][8] = {}, sg[C][8] = {};
  float sbb[BIAS ? C : 1][8] = {}, sba[BIAS ? C : 1][8] = {};
  const int r0 = blockIdx.x * a.rows_per_block, r1 = min(r0 + a.rows_per_block, a.T);
  const float inv_d = 1.f / a.d;
  using AS = Ahead<MODE, S>;
  using AY = Ahead<MODE, Y>;
  Vectors<VEC, C, BIAS> v;
  AS rd[C], rq[C], rx[C];  // d_x1, d_p, x1
  AY ry[C];
  const int slot_d = 0, slot_q = slot_d + (a.dx1 ? AS::kVecs : 0), slot_x = slot_q + (a.before ? AS::kVecs : 0);
  const int slot_y = slot_x + (a.before ? AS::kVecs : 0), slot_n = slot_y + (a.y ? AY::kVecs : 0);
  pdl_wait();
  clear_slots<MODE>(slots, kDepth * slot_n * C);
  auto fetch = [&](int row, int stage) {
    if (row < r1) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        uint4* slot = slots + (stage * C + c) * slot_n * blockDim.x + threadIdx.x;
        if (a.dx1) rd[c].load(slot + slot_d * blockDim.x, static_cast<const S*>(a.dx1) + row * a.lddx1, c, a.d);
        if (a.before) {
          rq[c].load(slot + slot_q * blockDim.x, static_cast<const S*>(a.dp) + row * a.lddp, c, a.d);
          rx[c].load(slot + slot_x * blockDim.x, static_cast<const S*>(a.x) + row * a.ldx, c, a.d);
        }
        if (a.y) ry[c].load(slot + slot_y * blockDim.x, static_cast<const Y*>(a.y) + row * a.ldy, c, a.d);
      }
    }
    if (RING) ptx::cp_async_commit();
  };
  for (int i = 0; i < (RING ? kDepth - 1 : 1); ++i) fetch(r0 + i, i);
  if (v.kKeep) v.load(a);
  int stage = 0;
  int group = a.gate ? r0 / a.rows_per_gate : 0;
  const bool one_gate = a.rows_per_gate >= a.T;
  for (int row = r0; row < r1; ++row) {
    if (a.gate) {
      const int now = one_gate ? 0 : row / a.rows_per_gate;
      if (now != group) {
        flush_gate<VEC, C>(a, group, r0, r1, sg);
        group = now;
      }
      v.load_gate(a, group);
    }
    if (!v.kKeep) v.load(a);
    if constexpr (RING) {
      fetch(row + kDepth - 1, stage ? stage - 1 : kDepth - 1);
      ptx::cp_async_wait<kDepth - 1>();
    }
    float D[C][8], x[C][8], q[C][8], y[C][8];
    const float zero[8] = {};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint4* slot = slots + (stage * C + c) * slot_n * blockDim.x + threadIdx.x;
      if (a.dx1) {
        rd[c].get(slot + slot_d * blockDim.x, c, a.d, D[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) D[c][j] = zero[j];
      }
      if (a.before) {
        rq[c].get(slot + slot_q * blockDim.x, c, a.d, q[c]);
        rx[c].get(slot + slot_x * blockDim.x, c, a.d, x[c]);
      }
      if (a.y) ry[c].get(slot + slot_y * blockDim.x, c, a.d, y[c]);
    }
    if (++stage == kDepth) stage = 0;
    if (!RING) fetch(row + 1, 0);
    // Row sums: about the mean first (layer), then both norms' squares with the terms of the next norm's
    // gradient, which need no deviation yet: sum(d_n n) = r sum(d_n x).
    const bool lb = BIAS && a.before == COLIBRI_NORM_LAYER, la = BIAS && a.after == COLIBRI_NORM_LAYER;
    if (BIAS && (lb || la)) {
      float s[2] = {lb ? sum_of(x) : 0.f, la ? sum_of(y) : 0.f};
      block_sum(s, buf, turn);
      if (lb) center<VEC>(x, s[0] * inv_d, a.d);
      if (la) center<VEC>(y, s[1] * inv_d, a.d);
    }
    float ra = 1.f;
    if (a.before || a.after) {
      float t[4] = {0.f, 0.f, 0.f, a.after ? dot_of(y, y) : 0.f};
      if (a.before) {
        t[0] = dot_of(x, x);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float dn = q[c][j] * v.wb[c][j];
            t[1] = fmaf(dn, x[c][j], t[1]);
            if constexpr (BIAS) t[2] += dn;
          }
      }
      block_sum(t, buf, turn);
      ra = rsqrtf(t[3] * inv_d + a.eps);
      if (a.before) {
        const float r = rsqrtf(t[0] * inv_d + a.eps), m1 = t[1] * inv_d * r, m0 = lb ? t[2] * inv_d : 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float n = x[c][j] * r, dn = q[c][j] * v.wb[c][j];
            swb[c][j] = fmaf(q[c][j], n, swb[c][j]);
            if constexpr (BIAS) sbb[c][j] += q[c][j];
            D[c][j] = fmaf(r, dn - n * m1 - m0, D[c][j]);
          }
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = a.alpha * D[c][j];
      store_cols<VEC>(static_cast<S*>(a.dx) + (int64_t)row * a.d, c, a.d, o);
    }
    if (a.y) {
      float t[2] = {0.f, 0.f};
      each<C>([&](int c, int j) { D[c][j] *= a.beta; });
      if (a.after) each<C>([&](int c, int j) { y[c][j] *= ra; });  // now n
      if (a.gate) {
        if (BIAS && a.ba) {
          each<C>([&](int c, int j) {
            sg[c][j] = fmaf(D[c][j], fmaf(y[c][j], v.wa[c][j], v.ba[BIAS ? c : 0][j]), sg[c][j]);
          });
        } else if (a.after) {
          each<C>([&](int c, int j) { sg[c][j] = fmaf(D[c][j], y[c][j] * v.wa[c][j], sg[c][j]); });
        } else {
          each<C>([&](int c, int j) { sg[c][j] = fmaf(D[c][j], y[c][j], sg[c][j]); });
        }
        each<C>([&](int c, int j) { D[c][j] *= v.g[c][j]; });
      }
      if (a.after)
        each<C>([&](int c, int j) {
          swa[c][j] = fmaf(D[c][j], y[c][j], swa[c][j]);
          if constexpr (BIAS) sba[c][j] += D[c][j];
          D[c][j] *= v.wa[c][j];  // now d_n
          t[0] = fmaf(D[c][j], y[c][j], t[0]);
          if constexpr (BIAS) t[1] += D[c][j];
        });
      if (a.after) {
        block_sum(t, buf, turn);
        const float m1 = t[0] * inv_d, m0 = la ? t[1] * inv_d : 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) D[c][j] = ra * (D[c][j] - y[c][j] * m1 - m0);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) store_cols<VEC>(static_cast<Y*>(a.dy) + (int64_t)row * a.d, c, a.d, D[c]);
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * kSlots * a.d;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (a.before) store_cols<VEC>(part + (int64_t)kSumWb * a.d, c, a.d, swb[c]);
    if (a.after) store_cols<VEC>(part + (int64_t)kSumWa * a.d, c, a.d, swa[c]);
    if constexpr (BIAS) {
      if (a.before) store_cols<VEC>(part + (int64_t)kSumBb * a.d, c, a.d, sbb[c]);
      if (a.after) store_cols<VEC>(part + (int64_t)kSumBa * a.d, c, a.d, sba[c]);
    }
  }
  if (a.gate) flush_gate<VEC, C>(a, group, r0, r1, sg);
}

struct NormSumsArgs {
  const float* part;
  float* out[4];       // d_wb, d_bb, d_wa, d_ba (kSumWb..kSumBa), nullptr where not wanted
  float* dgate;        // [gates][d] or nullptr
  int64_t rpg;
  int T, d, blocks, rows_per_block;
};

constexpr int kSumCols = 32, kSumLanes = 8;

// Adds the blocks' column sums: 32 columns x 8 lanes a block, each lane every eighth partial in order,
// then the lanes in order.
__global__ void __launch_bounds__(kSumCols * kSumLanes) norm_sums_kernel(NormSumsArgs a) {
  __shared__ float red[kSumLanes][kSumCols];
  const int tx = threadIdx.x % kSumCols, ty = threadIdx.x / kSumCols;
  const int col = blockIdx.x * kSumCols + tx;
  pdl_wait();
  const int64_t stride = (int64_t)kSlots * a.d;
  auto total = [&](float mine) {
    red[ty][tx] = mine;
    __syncthreads();
    float s = 0.f;
    if (ty == 0)
      for (int i = 0; i < kSumLanes; ++i) s += red[i][tx];
    __syncthreads();
    return s;
  };
  if (blockIdx.y < 4) {
    float* out = a.out[blockIdx.y];
    if (!out) return;
    float s = 0.f;
    if (col < a.d) {
      const float* p = a.part + (int64_t)blockIdx.y * a.d + col;
#pragma unroll 8
      for (int b = ty; b < a.blocks; b += kSumLanes) s += p[b * stride];
    }
    s = total(s);
    if (ty == 0 && col < a.d) out[col] = s;
    return;
  }
  if (!a.dgate) return;
  // the groups that begin in block b and go on past it: of each block the one of its last row
  for (int b = 0; b + 1 < a.blocks;) {
    const int64_t r0 = (int64_t)b * a.rows_per_block, r1 = r0 + a.rows_per_block;
    const int64_t g = (r1 - 1) / a.rpg, first = g * a.rpg, last = min((g + 1) * a.rpg, (int64_t)a.T) - 1;
    const int end = (int)(last / a.rows_per_block);
    if (first < r0 || last < r1) {  // began earlier, or ends with the block
      ++b;
      continue;
    }
    float s = 0.f;
    if (col < a.d) {
      const float* p = a.part + col;
      if (ty == 0) s = p[b * stride + (int64_t)kSumGateLast * a.d];
#pragma unroll 8
      for (int i = b + 1 + ty; i <= end; i += kSumLanes) s += p[i * stride + (int64_t)kSumGateFirst * a.d];
    }
    s = total(s);
    if (ty == 0 && col < a.d) a.dgate[g * a.d + col] = s;
    b = end;  // the next group to cross blocks begins in this group's last one at the earliest
  }
}

constexpr int kNormMaxD = 16384;

// Threads of a block with `chunks` runs of 8 columns each.
int norm_threads(int d, int chunks) { return ((d + 8 * chunks - 1) / (8 * chunks) + 31) / 32 * 32; }

// What the widest form's rows ahead take: 512 threads of 2 chunks, x and y in fp32.
constexpr int kRingBytes = kDepth * 4 * 2 * 512 * (int)sizeof(uint4);

// Launches a kernel with the shared memory of its rows ahead.  The limit that a kernel has on a device is raised
// once, to what any call needs, and never lowered: it belongs to the kernel, not to the call, and other
// threads launch the same kernel at other widths.
template <void (*kernel)(NormArgs)>
cudaError_t launch_rows(int slots, int chunks, int blocks, int threads, int device, cudaStream_t s, const NormArgs& a) {
  const size_t smem = (size_t)kDepth * slots * chunks * threads * sizeof(uint4);
  if (smem > kRingBytes) return cudaErrorInvalidConfiguration;
  if (smem > 32 * 1024) {
    static std::mutex mu;
    static bool ready[kOpsMaxDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[device]) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
      if (e != cudaSuccess) return e;
      ready[device] = true;
    }
  }
  return pdl_launch(kernel, dim3(blocks), dim3(threads), smem, s, a);
}
template <void (*kernel)(NormArgs)>
using Kernel = std::integral_constant<void (*)(NormArgs), kernel>;

// Forms by width: threads of a block, chunks of 8 columns a thread, blocks an SM.  The row sums' barriers
// want several blocks an SM, the vectors registers; a layer norm's two more vectors, or values in
// registers instead of the ring, cost the second block of 512.  The ring takes at most 196 KB.
template <typename S, typename Y, bool VEC, bool BIAS>
cudaError_t launch_forward_t(const NormArgs& a, int device, int sms, cudaStream_t s) {
  constexpr int R = VEC ? kRing : kScalar, V = VEC ? kVector : kScalar;
  constexpr int kBlocks = VEC && !BIAS ? 2 : 1;
  const int slots = Ahead<R, S>::kVecs + (a.y ? Ahead<R, Y>::kVecs : 0);
  auto go = [&](auto kernel, int slots, int chunks, int per_sm) {
    const int blocks = (int)std::min<int64_t>(a.T, (int64_t)sms * per_sm);
    return launch_rows<kernel>(slots, chunks, blocks, norm_threads(a.d, chunks), device, s, a);
  };
  if (a.d > 8 * 1024) return go(Kernel<block_norm_kernel<S, Y, V, 2, BIAS, 1024, 1>>{}, 0, 2, 1);
  if (a.d > 4 * 1024) return go(Kernel<block_norm_kernel<S, Y, R, 2, BIAS, 512, 1>>{}, slots, 2, 1);
  if (a.d > 2 * 1024) return go(Kernel<block_norm_kernel<S, Y, R, 1, BIAS, 512, kBlocks>>{}, slots, 1, kBlocks);
  return go(Kernel<block_norm_kernel<S, Y, R, 1, BIAS, 256, 2 * kBlocks>>{}, slots, 1,
            2 * kBlocks * std::max(1, 256 / norm_threads(a.d, 1)));
}
template <typename S, typename Y, bool VEC>
cudaError_t launch_forward(const NormArgs& a, int device, int sms, cudaStream_t s) {
  if (a.after == COLIBRI_NORM_LAYER || a.before == COLIBRI_NORM_LAYER)
    return launch_forward_t<S, Y, VEC, true>(a, device, sms, s);
  return launch_forward_t<S, Y, VEC, false>(a, device, sms, s);
}

// Blocks of the backward pass: enough to fill the SMs at about 512 threads each, and at least 8 rows a
// block where the batch allows, so that the partial column sums stay small beside the rows.
int backward_blocks(int T, int d, int sms, int* rows_per_block) {
  const int want = std::min(sms * std::max(1, 512 / norm_threads(d, d > 8 * 1024 ? 2 : 1)), std::max(sms, T / 8));
  *rows_per_block = (T + want - 1) / want;
  return (T + *rows_per_block - 1) / *rows_per_block;
}

template <typename S, typename Y, bool VEC, bool BIAS>
cudaError_t launch_backward_t(const NormArgs& a, int blocks, int device, cudaStream_t s) {
  constexpr int R = VEC ? kRing : kScalar, V = VEC ? kVector : kScalar, one = Ahead<R, S>::kVecs;
  const int slots = (a.dx1 ? one : 0) + (a.before ? 2 * one : 0) + (a.y ? Ahead<R, Y>::kVecs : 0);
  auto go = [&](auto kernel, int slots, int chunks) {
    return launch_rows<kernel>(slots, chunks, blocks, norm_threads(a.d, chunks), device, s, a);
  };
  if (a.d > 8 * 1024) return go(Kernel<block_norm_backward_kernel<S, Y, V, 2, BIAS, 1024>>{}, 0, 2);
  if (a.d > 4 * 1024) return go(Kernel<block_norm_backward_kernel<S, Y, V, 1, BIAS, 1024>>{}, 0, 1);
  if (a.d > 2 * 1024) return go(Kernel<block_norm_backward_kernel<S, Y, R, 1, BIAS, 512>>{}, slots, 1);
  return go(Kernel<block_norm_backward_kernel<S, Y, R, 1, BIAS, 256>>{}, slots, 1);
}

template <typename S, typename Y, bool VEC>
cudaError_t launch_backward(const NormArgs& a, int blocks, int device, cudaStream_t s) {
  if (a.after == COLIBRI_NORM_LAYER || a.before == COLIBRI_NORM_LAYER)
    return launch_backward_t<S, Y, VEC, true>(a, blocks, device, s);
  return launch_backward_t<S, Y, VEC, false>(a, blocks, device, s);
}

template <typename F>
cudaError_t by_type(int dtype, int block_dtype, bool vec, F f) {
  using B = __nv_bfloat16;
  if (dtype == COLIBRI_DTYPE_F32)
    return block_dtype == COLIBRI_DTYPE_F32 ? f(float{}, float{}, vec) : f(float{}, B{}, vec);
  return block_dtype == COLIBRI_DTYPE_F32 ? f(B{}, float{}, vec) : f(B{}, B{}, vec);
}

bool norm_kind(int32_t k) { return k == COLIBRI_NORM_NONE || k == COLIBRI_NORM_RMS || k == COLIBRI_NORM_LAYER; }

// The checks that need no device.
int check_norm_config(const colibri_moe_norm_config_t* c, const colibri_moe_norm_params_t* w, bool block, int32_t T) {
  if (!c || !w || T < 0) return COLIBRI_ERR_INVALID_ARG;
  if (c->d_model <= 0 || !ops_dtype(c->dtype) || !ops_dtype(c->block_dtype) || !ops_dtype(c->param_dtype) ||
      !norm_kind(c->after) || !norm_kind(c->before) || !(c->eps >= 0.f) || (c->trusted_pointers & ~1))
    return COLIBRI_ERR_INVALID_ARG;
  if (c->d_model > kNormMaxD || T > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  // without a block output there is nothing to norm after, to gate or to add
  if (!block && (c->after != COLIBRI_NORM_NONE || w->gate || c->before == COLIBRI_NORM_NONE))
    return COLIBRI_ERR_INVALID_ARG;
  if ((c->after != COLIBRI_NORM_NONE) != (w->after_weight != nullptr) ||
      (c->before != COLIBRI_NORM_NONE) != (w->before_weight != nullptr))
    return COLIBRI_ERR_INVALID_ARG;
  if ((w->after_bias && c->after != COLIBRI_NORM_LAYER) || (w->before_bias && c->before != COLIBRI_NORM_LAYER))
    return COLIBRI_ERR_INVALID_ARG;
  if (w->gate && c->rows_per_gate <= 0) return COLIBRI_ERR_INVALID_ARG;
  return COLIBRI_OK;
}

bool stride_ok(int64_t ld, int32_t d) { return ld >= d; }

// [p, p + bytes) as compared for overlap.
struct Span {
  const void* p;
  int64_t bytes;
};
bool spans_overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
int64_t span_of(int32_t T, int64_t ld, int32_t d, int elem) { return T ? ((int64_t)(T - 1) * ld + d) * elem : 0; }

}  // namespace
}  // namespace colibri

using namespace colibri;

extern "C" int colibri_moe_block_norm(const colibri_moe_norm_config_t* cfg, const colibri_moe_norm_params_t* w,
                                      const void* x, int64_t ldx, const void* y, int64_t ldy, int32_t T, void* x1,
                                      void* p, void* stream) {
  int rc = check_norm_config(cfg, w, y != nullptr || T == 0, T);  // no rows: y may be NULL either way
  if (rc) return rc;
  const int d = cfg->d_model;
  const bool next = cfg->before != COLIBRI_NORM_NONE;
  if (T == 0) return COLIBRI_OK;
  if (!x || !stride_ok(ldx, d) || (y && !stride_ok(ldy, d)) || (y != nullptr) != (x1 != nullptr) || next != (p != nullptr))
    return COLIBRI_ERR_INVALID_ARG;
  const int es = ops_elem(cfg->dtype), ey = ops_elem(cfg->block_dtype);
  const Span sx{x, span_of(T, ldx, d, es)}, sy{y, span_of(T, ldy, d, ey)};
  const Span o1{x1, (int64_t)T * d * es}, op{p, (int64_t)T * d * es};
  // x1 may be x itself (the stream updated in place): a row is read before it is written
  if ((spans_overlap(sx, o1) && !(x1 == x && ldx == d)) || spans_overlap(sy, o1) || spans_overlap(sx, op) ||
      spans_overlap(sy, op) || spans_overlap(o1, op))
    return COLIBRI_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  for (const void* q : {x, y, w->after_weight, w->after_bias, w->before_weight, w->before_bias, w->gate,
                        (const void*)x1, (const void*)p})
    if (q && !cfg->trusted_pointers && !ops_on_device(q, device)) return COLIBRI_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = x, a.y = y, a.wa = w->after_weight, a.ba = w->after_bias, a.wb = w->before_weight, a.bb = w->before_bias;
  a.gate = w->gate, a.x1 = x1, a.p = p, a.ldx = ldx, a.ldy = ldy, a.rpg = cfg->rows_per_gate, a.T = T, a.d = d;
  a.after = cfg->after, a.before = cfg->before, a.param_bf16 = cfg->param_dtype == COLIBRI_DTYPE_BF16;
  a.rows_per_gate = (int)std::min<int64_t>(std::max<int64_t>(cfg->rows_per_gate, 1), T);
  a.alpha = cfg->residual_scale, a.beta = cfg->block_scale, a.eps = cfg->eps;
  bool vec = d % 8 == 0 && ldx % 8 == 0 && (!y || ldy % 8 == 0);
  for (const void* q : {x, y, a.wa, a.ba, a.wb, a.bb, a.gate, (const void*)x1, (const void*)p}) vec = vec && ops_aligned16(q);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = by_type(cfg->dtype, cfg->block_dtype, vec, [&](auto st, auto yt, bool v) {
    using S = decltype(st);
    using Y = decltype(yt);
    return v ? launch_forward<S, Y, true>(a, device, sms, s) : launch_forward<S, Y, false>(a, device, sms, s);
  });
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}

extern "C" int colibri_moe_block_norm_backward_workspace(const colibri_moe_norm_config_t* cfg, int32_t T,
                                                         size_t* bytes) {
  if (!cfg || !bytes || T < 0 || cfg->d_model <= 0) return COLIBRI_ERR_INVALID_ARG;
  if (cfg->d_model > kNormMaxD || T > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  int device = 0, sms = 0, rows = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  *bytes = T ? (size_t)backward_blocks(T, cfg->d_model, sms, &rows) * kSlots * cfg->d_model * sizeof(float) : 0;
  return COLIBRI_OK;
}

extern "C" int colibri_moe_block_norm_backward(const colibri_moe_norm_config_t* cfg,
                                               const colibri_moe_norm_params_t* w, const void* d_x1, int64_t ld_dx1,
                                               const void* d_p, int64_t ld_dp, const void* x1, int64_t ldx1,
                                               const void* y, int64_t ldy, int32_t T, void* d_x, void* d_y,
                                               const colibri_moe_norm_grads_t* grads, void* workspace,
                                               size_t workspace_bytes, void* stream) {
  int rc = check_norm_config(cfg, w, y != nullptr || T == 0, T);  // no rows: y may be NULL either way
  if (rc) return rc;
  if (!grads) return COLIBRI_ERR_INVALID_ARG;
  const int d = cfg->d_model;
  const bool next = cfg->before != COLIBRI_NORM_NONE;
  // a gradient can be asked for only where the parameter is
  if ((grads->after_weight && !w->after_weight) || (grads->after_bias && cfg->after != COLIBRI_NORM_LAYER) ||
      (grads->before_weight && !w->before_weight) || (grads->before_bias && cfg->before != COLIBRI_NORM_LAYER) ||
      (grads->gate != nullptr) != (w->gate != nullptr))
    return COLIBRI_ERR_INVALID_ARG;
  if (T > 0) {
    if (next != (d_p != nullptr) || (next && !x1) || (!next && !d_x1) || !d_x || (y != nullptr) != (d_y != nullptr))
      return COLIBRI_ERR_INVALID_ARG;
    if ((d_x1 && !stride_ok(ld_dx1, d)) || (d_p && !stride_ok(ld_dp, d)) || (next && !stride_ok(ldx1, d)) ||
        (y && !stride_ok(ldy, d)))
      return COLIBRI_ERR_INVALID_ARG;
    const int es = ops_elem(cfg->dtype), ey = ops_elem(cfg->block_dtype);
    const Span in[] = {{d_x1, span_of(T, ld_dx1, d, es)},
                       {d_p, span_of(T, ld_dp, d, es)},
                       {next ? x1 : nullptr, span_of(T, ldx1, d, es)},
                       {y, span_of(T, ldy, d, ey)}};
    const Span ox{d_x, (int64_t)T * d * es}, oy{d_y, (int64_t)T * d * ey};
    for (const Span& q : in)
      if (spans_overlap(q, ox) || spans_overlap(q, oy)) return COLIBRI_ERR_INVALID_ARG;
    if (spans_overlap(ox, oy)) return COLIBRI_ERR_INVALID_ARG;
  }
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  for (const void* q : {d_x1, d_p, next ? x1 : nullptr, y, w->after_weight, w->after_bias, w->before_weight,
                        w->before_bias, w->gate, (const void*)d_x, (const void*)d_y, (const void*)grads->after_weight,
                        (const void*)grads->after_bias, (const void*)grads->before_weight,
                        (const void*)grads->before_bias, (const void*)grads->gate, (const void*)workspace})
    if (q && !cfg->trusted_pointers && !ops_on_device(q, device)) return COLIBRI_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // no rows: the column sums are zero (there is no gate row to sum into)
    for (float* g : {grads->after_weight, grads->after_bias, grads->before_weight, grads->before_bias})
      if (g && cudaMemsetAsync(g, 0, d * sizeof(float), s) != cudaSuccess) {
        cudaGetLastError();
        return COLIBRI_ERR_CUDA;
      }
    return COLIBRI_OK;
  }
  int rows = 0;
  const int blocks = backward_blocks(T, d, sms, &rows);
  if (!workspace || workspace_bytes < (size_t)blocks * kSlots * d * sizeof(float) || !ops_aligned16(workspace))
    return COLIBRI_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = x1, a.y = y, a.wa = w->after_weight, a.ba = w->after_bias, a.wb = w->before_weight, a.bb = w->before_bias;
  a.gate = w->gate, a.dx1 = d_x1, a.dp = d_p, a.dx = d_x, a.dy = d_y, a.part = static_cast<float*>(workspace);
  a.dgate = grads->gate, a.ldx = ldx1, a.ldy = ldy, a.lddx1 = ld_dx1, a.lddp = ld_dp, a.rpg = cfg->rows_per_gate;
  a.T = T, a.d = d, a.after = cfg->after, a.before = cfg->before, a.rows_per_block = rows;
  a.rows_per_gate = (int)std::min<int64_t>(std::max<int64_t>(cfg->rows_per_gate, 1), T);
  a.param_bf16 = cfg->param_dtype == COLIBRI_DTYPE_BF16;
  a.alpha = y ? cfg->residual_scale : 1.f, a.beta = cfg->block_scale, a.eps = cfg->eps;
  bool vec = d % 8 == 0 && (!d_x1 || ld_dx1 % 8 == 0) && (!next || (ldx1 % 8 == 0 && ld_dp % 8 == 0)) && (!y || ldy % 8 == 0);
  for (const void* q : {d_x1, d_p, next ? x1 : nullptr, y, a.wa, a.ba, a.wb, a.bb, a.gate, (const void*)d_x,
                        (const void*)d_y, (const void*)grads->gate})
    vec = vec && ops_aligned16(q);
  cudaError_t e = by_type(cfg->dtype, cfg->block_dtype, vec, [&](auto st, auto yt, bool v) {
    using S = decltype(st);
    using Y = decltype(yt);
    return v ? launch_backward<S, Y, true>(a, blocks, device, s) : launch_backward<S, Y, false>(a, blocks, device, s);
  });
  if (e != cudaSuccess) return COLIBRI_ERR_CUDA;
  NormSumsArgs q = {a.part,
                    {grads->before_weight, grads->before_bias, grads->after_weight, grads->after_bias},
                    grads->gate, cfg->rows_per_gate, T, d, blocks, rows};
  e = pdl_launch(norm_sums_kernel, dim3((d + kSumCols - 1) / kSumCols, 5), dim3(kSumCols * kSumLanes), 0, s, q);
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}
