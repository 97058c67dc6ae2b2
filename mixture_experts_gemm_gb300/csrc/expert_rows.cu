// Tokens to their experts' rows and back, and the gated activation between the projections, with gradients.
//
//   order:     the slots (t, s) of an expert e = idx[t, s], tokens ascending, experts one after another
//   rows       rows[r] = x[token_of_row[r]]                      (zeros where there is no token)
//   back       d_x[t] = sum_s d_rows[row_of[t, s]]               (slot order, fp32)
//   combine's  d_y[row_of[t, s]] = gate[t, s] d_out[t],  d_gate[t, s] = <d_out[t], y[row_of[t, s]]>
//   gated      h = silu(u) v,  d_u = d_h v silu'(u),  d_v = d_h silu(u),   silu(u) = u p, p = 1 / (1 + exp(-u)),
//              silu'(u) = p (1 + u (1 - p))
//
// All of them move bytes: a value is loaded once, in fp32 while it is worked on, and rounded once.
#include <algorithm>
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace colibri {
namespace {

namespace cg = cooperative_groups;

constexpr int kOrderMaxE = 512, kOrderMaxK = 32, kRowsMaxWidth = 65536;

// ------------------------------------------------------------------------------------------- order
// A stable counting sort in one launch: one cluster, every warp a run of consecutive slots.  A warp counts its
// run into its own histogram, 32 slots at a time (lanes of one expert rank themselves by their mask); the
// histograms are scanned over warps in shared memory and over CTAs through the cluster, the experts' totals
// give the offsets, and a second pass over the run adds up.  No atomics: the order is the definition's.  Latency of
// its four steps: 8 us for 8 slots of 256 experts as for 16384 of 8.
constexpr int kOrderThreads = 1024, kOrderWarps = kOrderThreads / 32;

struct OrderArgs {
  const int32_t* idx;
  int slots, k, E;
  int32_t *counts, *offsets, *row_of, *token_of_row;
};

__global__ void __launch_bounds__(kOrderThreads, 1) order_kernel(OrderArgs a) {
  extern __shared__ int32_t hist[];  // [warps][E]
  __shared__ int total[kOrderMaxE], base[kOrderMaxE + 1], warp_sum_of[kOrderWarps];
  auto cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.E;
  // 64-bit runs: the last warps' may begin past the end
  const int64_t per = ((int64_t)a.slots + ranks * kOrderThreads - 1) / (ranks * kOrderThreads) * 32;
  const int64_t here = min((int64_t)a.slots - per * kOrderWarps * rank, per * kOrderWarps);  // slots of this CTA
  const int used = here > 0 ? (int)((here + per - 1) / per) : 0;                             // warps that have some
  for (int i = threadIdx.x; i < used * E; i += kOrderThreads) hist[i] = 0;
  pdl_wait();
  __syncthreads();
  const int64_t lo = per * (rank * kOrderWarps + warp), hi = min(lo + per, (int64_t)a.slots);
  int32_t* mine = hist + warp * E;
  for (int64_t i0 = lo; i0 < hi; i0 += 128) {
    int e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + 32 * j + lane;
      e[j] = i < hi ? a.idx[i] : -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + 32 * j + lane;
      const bool in = e[j] >= 0 && e[j] < E;
      const uint32_t same = __match_any_sync(~0u, in ? e[j] : -1);
      const int before = __popc(same & ((1u << lane) - 1));
      const int rank_of = in ? mine[e[j]] + before : -1;
      __syncwarp();
      if (in && before == 0) mine[e[j]] += __popc(same);
      __syncwarp();
      if (i < hi) a.row_of[i] = rank_of;  // inside the warp's run, for now
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kOrderThreads) {
    int sum = 0;
    for (int w = 0; w < used; ++w) {
      const int v = hist[w * E + e];
      hist[w * E + e] = sum;
      sum += v;
    }
    total[e] = sum;
  }
  cluster.sync();
  // thread e: slots of e in CTAs before this one, and in all; then the experts' offsets
  int all = 0, before = 0;
  if (threadIdx.x < E) {
    for (int r = 0; r < ranks; ++r) {
      const int v = *cluster.map_shared_rank(total + threadIdx.x, r);
      if (r < rank) before += v;
      all += v;
    }
  }
  int run = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31) warp_sum_of[warp] = run;
  __syncthreads();
  for (int w = 0; w < warp; ++w) run += warp_sum_of[w];  // at most 16 warps hold experts
  if (threadIdx.x < E) {
    base[threadIdx.x] = run - all + before;
    if (rank == 0) {
      a.counts[threadIdx.x] = all;
      a.offsets[threadIdx.x + 1] = run;
    }
  }
  if (threadIdx.x == E - 1) base[kOrderMaxE] = run;  // rows in all
  if (rank == 0 && threadIdx.x == 0) a.offsets[0] = 0;
  __syncthreads();
  for (int64_t i = lo + lane; i < hi; i += 32) {
    const int e = a.idx[i];
    int row = -1;
    if (e >= 0 && e < E) {
      row = base[e] + mine[e] + a.row_of[i];
      a.token_of_row[row] = (int)((uint32_t)i / (uint32_t)a.k);
    }
    a.row_of[i] = row;
  }
  for (int64_t r = base[kOrderMaxE] + (int64_t)rank * kOrderThreads + threadIdx.x; r < a.slots;
       r += (int64_t)ranks * kOrderThreads)
    a.token_of_row[r] = -1;
  cluster.sync();  // no CTA leaves while another may read its totals
}

// -------------------------------------------------------------------------------------- rows there
// A warp takes stretches of one row, kStep accesses of a lane in flight.  8192 tokens of 4096 bf16 to two experts: 35 us
// (30 us of bytes), DRAM busy 0.59: half of the reads come from L2.
constexpr int kRowThreads = 256, kStep = 4;

struct RowsArgs {
  const void* x;
  int64_t row_bytes, ldx_bytes;  // of an output row, and between x's rows
  int T, R;
  const int32_t* token_of_row;
  void* rows;
  int parts;  // warps that share a row
};

template <typename V>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(RowsArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int n = (int)(a.row_bytes / sizeof(V));
  const int64_t items = (int64_t)a.R * a.parts, step = (int64_t)gridDim.x * (kRowThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); i < items; i += step) {
    const int64_t r = i / a.parts;
    const int part = (int)(i - r * a.parts);
    const int t = a.token_of_row[r];
    const bool real = t >= 0 && t < a.T;
    const V* src = reinterpret_cast<const V*>(static_cast<const char*>(a.x) + (real ? t : 0) * a.ldx_bytes);
    V* dst = reinterpret_cast<V*>(static_cast<char*>(a.rows) + r * a.row_bytes);
    for (int c = part * 32 * kStep + lane; c < n; c += a.parts * 32 * kStep) {
      V v[kStep] = {};
      if (real) {
#pragma unroll
        for (int j = 0; j < kStep; ++j)
          if (c + 32 * j < n) v[j] = __ldg(src + c + 32 * j);
      }
#pragma unroll
      for (int j = 0; j < kStep; ++j)
        if (c + 32 * j < n) __stcs(dst + c + 32 * j, v[j]);
    }
  }
}

// --------------------------------------------------------------------------------------- rows back
// W consecutive values of a row as fp32, loaded and stored in one access where W is 8.
template <typename T, int W>
__device__ __forceinline__ void load_w(const T* p, float (&v)[W]) {
  if constexpr (W == 8)
    load8(p, v);
  else
    v[0] = to_float(*p);
}
template <typename T, int W>
__device__ __forceinline__ void store_w(T* p, const float (&v)[W]) {
  if constexpr (W == 8)
    store8(p, v);
  else
    *p = from_float<T>(v[0]);
}

struct BackArgs {
  const void* d_rows;
  const int32_t* row_of;
  void* d_x;
  int T, R, k, d;
  int parts;  // warps that share a token
};

// Accesses of W columns that a lane has in flight.
__host__ __device__ constexpr int back_units(int W) { return W == 8 ? 2 : 8; }

// A warp takes stretches of one token: W columns a lane, the token's rows one after another.  4099 tokens of 4 slots x 1409
// fp32 (rows off 16 bytes): 30 us whole, 16 us of bytes; with two accesses in flight 58.
template <typename T, typename O, int W>
__global__ void __launch_bounds__(kRowThreads) rows_back_kernel(BackArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int n = a.d / W;
  const int64_t items = (int64_t)a.T * a.parts, step = (int64_t)gridDim.x * (kRowThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); i < items; i += step) {
    const int64_t t = i / a.parts;
    const int part = (int)(i - t * a.parts);
    const int row = lane < a.k ? a.row_of[t * a.k + lane] : -1;
    const int own = row >= 0 && row < a.R ? row : -1;
    constexpr int U = back_units(W);
    for (int c0 = part * 32 * U; c0 < n; c0 += a.parts * 32 * U) {
      float sum[U][W] = {};
      for (int s = 0; s < a.k; ++s) {
        const int r = __shfl_sync(~0u, own, s);
        if (r < 0) continue;
        const T* src = static_cast<const T*>(a.d_rows) + (int64_t)r * a.d;
        float v[U][W] = {};
#pragma unroll
        for (int j = 0; j < U; ++j)
          if (c0 + 32 * j + lane < n) load_w(src + (int64_t)(c0 + 32 * j + lane) * W, v[j]);
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int w = 0; w < W; ++w) sum[j][w] = __fadd_rn(sum[j][w], v[j][w]);
      }
      O* dst = static_cast<O*>(a.d_x) + t * a.d;
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (c0 + 32 * j + lane < n) store_w(dst + (int64_t)(c0 + 32 * j + lane) * W, sum[j]);
    }
  }
}

// ------------------------------------------------------------------------------- combine's gradients
struct CombineBackArgs {
  const void* d_out;
  int64_t ld_out;
  const void* y;
  const int32_t* row_of;
  const float* gate;
  const int32_t* token_of_row;
  void* d_y;
  float* d_gate;
  int T, R, k, d;
};

constexpr int kCombineBackThreads = 128;

// One block a token: d_out once, the rows of its slots in order.  A slot's dot product is summed by columns in each
// thread, then over the block in a fixed order.  Every block then clears its share of the rows that no token has.  8192
// tokens of 4096 bf16, two slots: 66 us (49 us of bytes), bound by loads that wait on one another's barriers.
template <typename T, typename Y, int W, int KS>
__global__ void __launch_bounds__(kCombineBackThreads) combine_back_kernel(CombineBackArgs a) {
  constexpr int kWarps = kCombineBackThreads / 32;
  __shared__ int s_row[kOrderMaxK];
  __shared__ float s_gate[kOrderMaxK], s_dot[2][kWarps][KS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = a.d / W;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    __syncthreads();  // the last token's rows and gates have been read
    if (warp == 0) {
      const int row = lane < a.k ? a.row_of[t * a.k + lane] : -1;
      const bool in = row >= 0 && row < a.R;
      float g = in ? a.gate[t * a.k + lane] : 0.f;
      // a row that several slots of the token name takes all their gates, in slot order
      const uint32_t same = __match_any_sync(~0u, in ? row : -1 - lane);
      if (__any_sync(~0u, in && (same & (same - 1)))) {
        float all = 0.f;
        for (int s = 0; s < 32; ++s) {
          const float v = __shfl_sync(~0u, g, s);
          if (same >> s & 1) all += v;
        }
        g = all;
      }
      if (lane < a.k) s_row[lane] = in ? row : -1, s_gate[lane] = g;
    }
    __syncthreads();
    for (int s0 = 0; s0 < a.k; s0 += KS, turn ^= 1) {  // KS slots a pass over d_out
      float dot[KS] = {};
      for (int c = threadIdx.x; c < n; c += kCombineBackThreads) {
        float g[W];
        load_w(static_cast<const T*>(a.d_out) + t * a.ld_out + (int64_t)c * W, g);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          if (s0 + s >= a.k) break;
          const int64_t r = s_row[s0 + s];
          if (r < 0) continue;
          const float gate = s_gate[s0 + s];
          float y[W], o[W];
          load_w(static_cast<const Y*>(a.y) + r * a.d + (int64_t)c * W, y);
#pragma unroll
          for (int w = 0; w < W; ++w) dot[s] = fmaf(g[w], y[w], dot[s]), o[w] = gate * g[w];
          store_w(static_cast<Y*>(a.d_y) + r * a.d + (int64_t)c * W, o);
        }
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const float v = warp_sum(dot[s]);
        if (lane == 0) s_dot[turn][warp][s] = v;
      }
      __syncthreads();
      if (threadIdx.x < KS && s0 + threadIdx.x < a.k) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += s_dot[turn][w][threadIdx.x];
        a.d_gate[t * a.k + s0 + threadIdx.x] = s_row[s0 + threadIdx.x] < 0 ? 0.f : v;
      }
    }
  }
  // rows of no token
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  for (int64_t r0 = ((int64_t)blockIdx.x * kWarps + warp) * 32; r0 < a.R; r0 += warps * 32) {
    const int t = r0 + lane < a.R ? a.token_of_row[r0 + lane] : 0;
    uint32_t empty = __ballot_sync(~0u, t < 0 || t >= a.T);
    while (empty) {
      const int64_t r = r0 + __ffs(empty) - 1;
      empty &= empty - 1;
      const float none[W] = {};
      for (int c = lane; c < n; c += 32) store_w(static_cast<Y*>(a.d_y) + r * a.d + (int64_t)c * W, none);
    }
  }
}

// ---------------------------------------------------------------------------------- gated activation
struct GatedArgs {
  const void *d_h, *u, *v;
  int64_t ld_h, ldu, ldv;  // ld_h: of d_h
  void *h, *d_u, *d_v;     // contiguous
  int R, f;
};

// p = 1 / (1 + exp(-u)) and 1 - p.  fp32 results take expf of what cannot overflow and the approximate reciprocal,
// good to an ulp, of a sum between 1 and 2; results in bf16 the fast exp, whose error is far below their rounding.
template <bool FAST>
__device__ __forceinline__ void sigmoid_of(float u, float& p, float& q) {
  const float t = FAST ? __expf(-fabsf(u)) : expf(-fabsf(u));
  float s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + t));
  const float small = t * s;
  p = u < 0.f ? small : s, q = u < 0.f ? s : small;
}

constexpr int kGatedThreads = 256;
// Accesses of W columns that a thread has in flight.
__host__ __device__ constexpr int gated_units(int W, bool backward) { return W == 8 ? (backward ? 1 : 2) : 4; }

// A block takes a stretch of one row, or several short rows.  16384 x 14336 bf16 backward: 0.32 ms, the copy rate; 6126 x
// 1409 fp32 at rows off 16 bytes: 22 us (15 us of bytes), issue slots 0.67 busy.
template <typename T, typename O, int W, bool BACKWARD>
__global__ void __launch_bounds__(kGatedThreads) gated_kernel(GatedArgs a) {
  constexpr bool kFast = BACKWARD ? sizeof(T) == 2 : sizeof(O) == 2;
  constexpr int kUnits = gated_units(W, BACKWARD);
  pdl_wait();
  pdl_trigger();
  const int n = a.f / W, across = blockDim.x;  // threads along a row
  for (int64_t r = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; r < a.R; r += (int64_t)gridDim.y * blockDim.y) {
    const T *u = static_cast<const T*>(a.u) + r * a.ldu, *v = static_cast<const T*>(a.v) + r * a.ldv;
    for (int c0 = blockIdx.x * across * kUnits + threadIdx.x; c0 < n; c0 += gridDim.x * across * kUnits) {
      float x[kUnits][W], y[kUnits][W], g[kUnits][W];
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int c = c0 + i * across;
        if (c >= n) break;
        load_w(u + (int64_t)c * W, x[i]), load_w(v + (int64_t)c * W, y[i]);
        if constexpr (BACKWARD) load_w(static_cast<const O*>(a.d_h) + r * a.ld_h + (int64_t)c * W, g[i]);
      }
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int c = c0 + i * across;
        if (c >= n) break;
        float p, q;
        if constexpr (BACKWARD) {
          float du[W], dv[W];
#pragma unroll
          for (int w = 0; w < W; ++w) {
            sigmoid_of<kFast>(x[i][w], p, q);
            dv[w] = g[i][w] * (x[i][w] * p);
            du[w] = g[i][w] * y[i][w] * (p * fmaf(x[i][w], q, 1.f));
          }
          store_w(static_cast<T*>(a.d_u) + r * a.f + (int64_t)c * W, du);
          store_w(static_cast<T*>(a.d_v) + r * a.f + (int64_t)c * W, dv);
        } else {
          float h[W];
#pragma unroll
          for (int w = 0; w < W; ++w) {
            sigmoid_of<kFast>(x[i][w], p, q);
            h[w] = x[i][w] * p * y[i][w];
          }
          store_w(static_cast<O*>(a.h) + r * a.f + (int64_t)c * W, h);
        }
      }
    }
  }
}

// --------------------------------------------------------------------------------------- host side
int check_pointers(int32_t trusted, std::initializer_list<const void*> ps, int* sms) {
  int device = 0;
  if (!ops_device(&device, sms)) return COLIBRI_ERR_CUDA;
  for (const void* p : ps)
    if (p && !trusted && !ops_on_device(p, device)) return COLIBRI_ERR_INVALID_ARG;
  return COLIBRI_OK;
}
int status(cudaError_t e) { return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA; }

// Calls f(a value of the type that t stands for).
template <typename F>
cudaError_t with_type(int32_t t, F f) {
  return t == COLIBRI_DTYPE_F32 ? f(float()) : f(__nv_bfloat16());
}
// 8-column accesses: whole units, and 16-byte rows of the narrower type.
bool vectors_of_8(int d, std::initializer_list<const void*> ps, std::initializer_list<int64_t> strides) {
  if (d % 8) return false;
  for (const void* p : ps)
    if (!ops_aligned16(p)) return false;
  for (int64_t l : strides)
    if (l % 8) return false;
  return true;
}

// Warps that share a row or token so that `rows` of them fill the card, at most one for each `unit` columns.
int shares(int64_t rows, int64_t n, int unit, int sms) {
  const int64_t want = (int64_t)sms * 32 / std::max<int64_t>(rows, 1), most = (n + unit - 1) / unit;
  return (int)std::max<int64_t>(1, std::min(want, most));
}
unsigned warp_grid(int64_t items, int sms) {
  constexpr int per = kRowThreads / 32;
  return (unsigned)std::min<int64_t>((items + per - 1) / per, (int64_t)sms * 8);
}

}  // namespace
}  // namespace colibri

using namespace colibri;

extern "C" int colibri_moe_dispatch_order(const int32_t* idx, int32_t T, int32_t k, int32_t E, int32_t* counts,
                                          int32_t* offsets, int32_t* row_of, int32_t* token_of_row,
                                          int32_t trusted_pointers, void* stream) {
  if (T < 0 || k < 1 || E < 1 || (trusted_pointers & ~1)) return COLIBRI_ERR_INVALID_ARG;
  if (k > kOrderMaxK || E > kOrderMaxE || (int64_t)T * k > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  if (!counts || !offsets || (T > 0 && (!idx || !row_of || !token_of_row))) return COLIBRI_ERR_INVALID_ARG;
  int sms = 0;
  if (const int rc = check_pointers(trusted_pointers, {idx, counts, offsets, row_of, token_of_row}, &sms)) return rc;
  int device = 0;
  cudaGetDevice(&device);
  static bool ready[kOpsMaxDevices];  // the same call whichever thread makes it first
  if (!__atomic_load_n(&ready[device], __ATOMIC_ACQUIRE)) {
    if (cudaFuncSetAttribute(order_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kOrderWarps * kOrderMaxE * (int)sizeof(int32_t)) != cudaSuccess)
      return COLIBRI_ERR_CUDA;
    __atomic_store_n(&ready[device], true, __ATOMIC_RELEASE);
  }
  const OrderArgs a = {idx, T * k, k, E, counts, offsets, row_of, token_of_row};
  const int ranks = a.slots <= kOrderThreads ? 1 : a.slots <= 2 * kOrderThreads ? 2 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kOrderThreads);
  cfg.dynamicSmemBytes = kOrderWarps * E * sizeof(int32_t);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return status(cudaLaunchKernelEx(&cfg, order_kernel, a));
}

extern "C" int colibri_moe_dispatch_rows(const void* x, int32_t dtype, int64_t ldx, int32_t T, const int32_t* token_of_row,
                                         int32_t R, int32_t d, void* rows, int32_t trusted_pointers, void* stream) {
  if (T < 0 || R < 0 || d < 1 || !ops_dtype(dtype) || (trusted_pointers & ~1)) return COLIBRI_ERR_INVALID_ARG;
  if (d > kRowsMaxWidth || R > kOpsMaxRows || T > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  if (R == 0) return COLIBRI_OK;
  if ((T > 0 && (!x || ldx < d)) || !token_of_row || !rows) return COLIBRI_ERR_INVALID_ARG;
  int sms = 0;
  if (const int rc = check_pointers(trusted_pointers, {x, token_of_row, rows}, &sms)) return rc;
  const int es = ops_elem(dtype);
  RowsArgs a = {x, (int64_t)d * es, ldx * es, T, R, token_of_row, rows, 1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto v) {
    using V = decltype(v);
    a.parts = shares(R, a.row_bytes / (int)sizeof(V), 32 * kStep, sms);
    return pdl_launch(rows_kernel<V>, dim3(warp_grid((int64_t)R * a.parts, sms)), dim3(kRowThreads), 0, s, a);
  };
  const bool vec = a.row_bytes % 16 == 0 && a.ldx_bytes % 16 == 0 && ops_aligned16(x) && ops_aligned16(rows);
  return status(vec ? go(uint4()) : es == 4 ? go(uint32_t()) : go((unsigned short)0));
}

extern "C" int colibri_moe_dispatch_backward(const void* d_rows, int32_t dtype, int32_t R, const int32_t* row_of,
                                             int32_t T, int32_t k, int32_t d, void* d_x, int32_t out_dtype,
                                             int32_t trusted_pointers, void* stream) {
  if (T < 0 || R < 0 || k < 1 || d < 1 || !ops_dtype(dtype) || !ops_dtype(out_dtype) || (trusted_pointers & ~1))
    return COLIBRI_ERR_INVALID_ARG;
  if (k > kOrderMaxK || d > kRowsMaxWidth || T > kOpsMaxRows || R > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  if (T == 0) return COLIBRI_OK;
  if ((R > 0 && !d_rows) || !row_of || !d_x) return COLIBRI_ERR_INVALID_ARG;
  int sms = 0;
  if (const int rc = check_pointers(trusted_pointers, {d_rows, row_of, d_x}, &sms)) return rc;
  BackArgs a = {d_rows, row_of, d_x, T, R, k, d, 1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = vectors_of_8(d, {d_rows, d_x}, {});
  a.parts = shares(T, d / (vec ? 8 : 1), 32 * back_units(vec ? 8 : 1), sms);
  const dim3 grid(warp_grid((int64_t)T * a.parts, sms)), block(kRowThreads);
  return status(with_type(dtype, [&](auto t) {
    return with_type(out_dtype, [&](auto o) {
      return vec ? pdl_launch(rows_back_kernel<decltype(t), decltype(o), 8>, grid, block, 0, s, a)
                 : pdl_launch(rows_back_kernel<decltype(t), decltype(o), 1>, grid, block, 0, s, a);
    });
  }));
}

extern "C" int colibri_moe_combine_backward(const void* d_out, int32_t dtype, int64_t ld_out, const void* y,
                                            int32_t y_dtype, int32_t R, const int32_t* row_of, const float* gate,
                                            const int32_t* token_of_row, int32_t T, int32_t k, int32_t d, void* d_y,
                                            float* d_gate, int32_t trusted_pointers, void* stream) {
  if (T < 0 || R < 0 || k < 1 || d < 1 || !ops_dtype(dtype) || !ops_dtype(y_dtype) || (trusted_pointers & ~1))
    return COLIBRI_ERR_INVALID_ARG;
  if (k > kOrderMaxK || d > kRowsMaxWidth || T > kOpsMaxRows || R > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  if (T == 0 && R == 0) return COLIBRI_OK;
  if ((T > 0 && (!d_out || ld_out < d || !row_of || !gate || !d_gate)) || (R > 0 && (!y || !token_of_row || !d_y)))
    return COLIBRI_ERR_INVALID_ARG;
  int sms = 0;
  if (const int rc = check_pointers(trusted_pointers, {d_out, y, row_of, gate, token_of_row, d_y, d_gate}, &sms))
    return rc;
  const CombineBackArgs a = {d_out, ld_out, y, row_of, gate, token_of_row, d_y, d_gate, T, R, k, d};
  const bool vec = vectors_of_8(d, {d_out, y, d_y}, {ld_out});
  const int64_t blocks = std::max<int64_t>(T, ((int64_t)R + kCombineBackThreads - 1) / kCombineBackThreads);
  const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)sms * 16)), block(kCombineBackThreads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status(with_type(dtype, [&](auto t) {
    return with_type(y_dtype, [&](auto o) {
      using A = decltype(t);
      using Y = decltype(o);
      if (vec)
        return k <= 2 ? pdl_launch(combine_back_kernel<A, Y, 8, 2>, grid, block, 0, s, a)
                      : pdl_launch(combine_back_kernel<A, Y, 8, 8>, grid, block, 0, s, a);
      return k <= 2 ? pdl_launch(combine_back_kernel<A, Y, 1, 2>, grid, block, 0, s, a)
                    : pdl_launch(combine_back_kernel<A, Y, 1, 8>, grid, block, 0, s, a);
    });
  }));
}

namespace {

int gated(bool backward, const void* d_h, int64_t ld_h, const void* u, int64_t ldu, const void* v, int64_t ldv,
          int32_t dtype, int32_t R, int32_t f, void* h, void* d_u, void* d_v, int32_t h_dtype, int32_t trusted,
          void* stream) {
  if (R < 0 || f < 1 || !ops_dtype(dtype) || !ops_dtype(h_dtype) || (trusted & ~1)) return COLIBRI_ERR_INVALID_ARG;
  if (R > kOpsMaxRows || f > kRowsMaxWidth) return COLIBRI_ERR_UNSUPPORTED;
  if (R == 0) return COLIBRI_OK;
  if (!u || !v || ldu < f || ldv < f || (backward ? !d_h || ld_h < f || !d_u || !d_v : !h)) return COLIBRI_ERR_INVALID_ARG;
  int sms = 0;
  if (const int rc = check_pointers(trusted, {d_h, u, v, h, d_u, d_v}, &sms)) return rc;
  const GatedArgs a = {d_h, u, v, ld_h, ldu, ldv, h, d_u, d_v, R, f};
  const bool vec = vectors_of_8(f, {d_h, u, v, h, d_u, d_v}, {ld_h, ldu, ldv});
  const int n = vec ? f / 8 : f, units = gated_units(vec ? 8 : 1, backward);
  int across = 32;  // threads along a row
  while (across < kGatedThreads && across * units < n) across *= 2;
  const int down = kGatedThreads / across;
  const dim3 grid((n + across * units - 1) / (across * units), std::min((R + down - 1) / down, 65535)), block(across, down);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status(with_type(dtype, [&](auto t) {
    return with_type(h_dtype, [&](auto o) {
      using A = decltype(t);
      using O = decltype(o);
      if (backward)
        return vec ? pdl_launch(gated_kernel<A, O, 8, true>, grid, block, 0, s, a)
                   : pdl_launch(gated_kernel<A, O, 1, true>, grid, block, 0, s, a);
      return vec ? pdl_launch(gated_kernel<A, O, 8, false>, grid, block, 0, s, a)
                 : pdl_launch(gated_kernel<A, O, 1, false>, grid, block, 0, s, a);
    });
  }));
}

}  // namespace

extern "C" int colibri_moe_gated(const void* u, int64_t ldu, const void* v, int64_t ldv, int32_t dtype, int32_t R,
                                 int32_t f, void* h, int32_t out_dtype, int32_t trusted_pointers, void* stream) {
  return gated(false, nullptr, 0, u, ldu, v, ldv, dtype, R, f, h, nullptr, nullptr, out_dtype, trusted_pointers, stream);
}

extern "C" int colibri_moe_gated_backward(const void* d_h, int32_t h_dtype, int64_t ld_h, const void* u, int64_t ldu,
                                          const void* v, int64_t ldv, int32_t dtype, int32_t R, int32_t f, void* d_u,
                                          void* d_v, int32_t trusted_pointers, void* stream) {
  return gated(true, d_h, ld_h, u, ldu, v, ldv, dtype, R, f, nullptr, d_u, d_v, h_dtype, trusted_pointers, stream);
}
