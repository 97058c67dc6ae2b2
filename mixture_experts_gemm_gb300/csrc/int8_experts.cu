// Experts in 8-bit integers: activations quantised per row, weights per output channel; the combine.
//
//   scale_t = max |x_t| / 127,  q = round(x / scale_t)  (IEEE fp32 quotients, ties to even)
//   v[r, n] = scale_{rows[r]} w_scale[e, n] sum_k q[rows[r], k] w[e, n, k]
//   y = v, or silu(v) * v3 with a second set of weights
//
// This file: the quantiser (rows in dispatch order, as fp16 whole numbers that the tensor cores take), the
// entry points, and the gate-weighted combine.  The products are in int8_mma.cu.
#include <algorithm>

#include "int8_internal.cuh"

namespace colibri {
namespace {

__device__ __forceinline__ void store_q8(__half* p, const float (&v)[8]) {
  __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}
__device__ __forceinline__ void store_q8(int8_t* p, const float (&v)[8]) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= (uint32_t)((int)v[i] & 0xff) << (8 * (i & 3));
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <typename Q>
__device__ __forceinline__ Q q_value(float v);
template <>
__device__ __forceinline__ __half q_value<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ int8_t q_value<int8_t>(float v) {
  return (int8_t)(int)v;
}

__device__ __forceinline__ float quotient(float x, float scale) {
  return fminf(fmaxf(rintf(__fdiv_rn(x, scale)), -127.f), 127.f);
}
// round(x / scale) as the IEEE quotient gives it.  The product with 1 / scale is within 127 * 2^-22 of the
// quotient; only where that could cross a half is the division done (about one value in five thousand).
// Adding and taking away 1.5 * 2^23 rounds to an integer, ties to even.
__device__ __forceinline__ void quotients(float (&v)[8], float scale, float inv, bool exact) {
  float t[8], worst = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float p = v[j] * inv;
    t[j] = __fadd_rn(__fadd_rn(p, 12582912.f), -12582912.f);
    worst = fmaxf(worst, fabsf(p - t[j]));
  }
  if (exact || worst > 0.4999f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = quotient(v[j], scale);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = t[j];
}

constexpr int kQuantThreads = 256;

// Eight values as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p), b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
  }
};

// One block a row, held in registers between the maximum and the quotients: C chunks of 8 columns a
// thread (16-byte loads), or read twice (C == 0).  The row once in, its fp16 once out: 16384 rows of 14336 from
// 8192 tokens in 0.17 ms by itself (705 MB of floor, 0.10 ms; issue slots 0.64, DRAM 0.68 busy).
template <typename T, typename Q, int C, bool COPIES>
__global__ void __launch_bounds__(kQuantThreads, C <= 2 ? 6 : 4) quantize_rows_kernel(QuantArgs a) {
  __shared__ float s_max[kQuantThreads / 32];
  pdl_wait();
  pdl_trigger();  // after the wait: what starts early may read what was there before this kernel
  for (int64_t i = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x; i < a.n_ticket; i += (int64_t)gridDim.x * kQuantThreads)
    a.ticket[i] = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.x;
  int t = r;
  if (a.rows) t = a.rows[r];
  const bool real = t >= 0 && t < a.n_tokens;
  const T* x = static_cast<const T*>(a.x) + (real ? t : 0) * a.ldx;
  Q* q = static_cast<Q*>(a.q) + (int64_t)r * a.K;
  Raw8<T> raw[C ? C : 1] = {};
  float top = 0.f, zero = 0.f;  // of |x|; 0, or NaN once a NaN or an infinity was there
  auto take = [&](float v) {
    top = fmaxf(top, fabsf(v));
    zero = fmaf(v, 0.f, zero);
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * kQuantThreads + threadIdx.x) * 8;
      if (real && col < a.K) raw[c].load(x + col);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[8];
      raw[c].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) take(v[j]);
    }
  } else if (real) {
    for (int i = threadIdx.x; i < a.K; i += kQuantThreads) take(to_float(x[i]));
  }
  if (!(zero == 0.f)) top = INFINITY;
  top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));  // not negative: ordered as its bits
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQuantThreads / 32; ++i) top = fmaxf(top, s_max[i]);
  const float scale = top < INFINITY ? __fdiv_rn(top, 127.f) : NAN;
  if (threadIdx.x == 0) a.scale[r] = scale;
  const bool live = scale > 0.f, exact = scale < 1e-30f;  // 1 / scale may overflow there
  const float inv = live ? __frcp_rn(scale) : 0.f;
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * kQuantThreads + threadIdx.x) * 8;
      if (col >= a.K) break;
      float v[8] = {};
      if (live) {
        raw[c].get(v);
        quotients(v, scale, inv, exact);
      }
      store_q8(q + col, v);
      if (COPIES)
        for (int i = 1; i < a.copies; ++i) store_q8(q + (int64_t)i * a.n * a.K + col, v);
    }
  } else {
    for (int i = threadIdx.x; i < a.K; i += kQuantThreads) {
      const Q v = q_value<Q>(live ? quotient(to_float(x[i]), scale) : 0.f);
      for (int j = 0; j < a.copies; ++j) q[(int64_t)j * a.n * a.K + i] = v;
    }
  }
}

constexpr int kInt8MaxE = 512, kInt8MaxK = 65536, kInt8MaxN = 131072;
constexpr int kInt8WaitUs = 2000000, kInt8MaxWaitUs = 10000000;
// The clock is read once in 64 tries of about 8 us, at every one under a millisecond's limit.
Int8Limit int8_limit(int us) { return {us * 1000ull, us < 1000 ? 0u : 63u}; }

int check_int8_config(const colibri_moe_int8_config_t* c) {
  if (!c || c->in_features <= 0 || c->out_features <= 0 || c->num_experts <= 0 || !ops_dtype(c->dtype) ||
      !ops_dtype(c->out_dtype) || (c->trusted_pointers & ~1) || c->wait_limit_us < 0 ||
      c->wait_limit_us > kInt8MaxWaitUs)
    return COLIBRI_ERR_INVALID_ARG;
  if (c->in_features % 16 || c->in_features > kInt8MaxK || c->out_features > kInt8MaxN || c->num_experts > kInt8MaxE)
    return COLIBRI_ERR_UNSUPPORTED;
  return COLIBRI_OK;
}

template <typename T, typename Q, bool COPIES>
cudaError_t quantize_t(const QuantArgs& q, cudaStream_t s) {
  const dim3 grid(q.n), block(kQuantThreads);
  const bool vec = q.ldx % 8 == 0 && ops_aligned16(q.x) && ops_aligned16(q.q);  // K is a multiple of 16
  const int chunks = (q.K + 8 * kQuantThreads - 1) / (8 * kQuantThreads);
  if (!vec || chunks > 8) return pdl_launch(quantize_rows_kernel<T, Q, 0, COPIES>, grid, block, 0, s, q);
  if (chunks == 1) return pdl_launch(quantize_rows_kernel<T, Q, 1, COPIES>, grid, block, 0, s, q);
  if (chunks == 2) return pdl_launch(quantize_rows_kernel<T, Q, 2, COPIES>, grid, block, 0, s, q);
  if (chunks <= 4) return pdl_launch(quantize_rows_kernel<T, Q, 4, COPIES>, grid, block, 0, s, q);
  return pdl_launch(quantize_rows_kernel<T, Q, 8, COPIES>, grid, block, 0, s, q);
}

template <typename Q, bool COPIES>
cudaError_t quantize(int dtype, const QuantArgs& q, cudaStream_t s) {
  return dtype == COLIBRI_DTYPE_F32 ? quantize_t<float, Q, COPIES>(q, s) : quantize_t<__nv_bfloat16, Q, COPIES>(q, s);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Token rows of a tile, by the rows that an expert gets on average (the exact numbers are on the device): narrow
// tiles leave more room for weights in flight, and rows that do not fit one tile have the expert's weights
// converted again.  us on a GB300 with random routing, for eight experts of 2048 x 5632 x 2 / 64 of 2048 x 1409,
// top-6, unevenly loaded / eight of 4096 x 4096, by the mean:
//   mean  16: 32 rows  46 /  57 / 64,  64 rows  55 /  65 / 45
//   mean  24: 32 rows  47 /  63 / 60,  64 rows  56 /  66 / 47
//   mean  40: 64 rows  58 /  76 / 47, 128 rows  59 /  70 / 48
//   mean  56: 64 rows  62 /  88 / 58, 128 rows  61 /  74 / 49
//   mean  80: 128 rows 64 /  86 / 51, 256 rows  64 /  83 / 51
//   mean 112: 128 rows 68 / 100 / 63, 256 rows  67 /  92 / 54
//   mean 160: 128 rows 109 / 117 / 82, 256 rows 82 / 113 / 60
// The steps at 16 and 48 lie between the shapes' own; the one at 128 lies above all of theirs (about 80).
int int8_tile_rows(int R, int E) {
  const int64_t mean = R / std::min(E, R);
  return mean <= 16 ? 32 : mean <= 48 ? 64 : mean <= 128 ? 128 : 256;
}

// Of few rows, all SMs read the same few kilobytes at the same time; copies spread them over L2.  One copy / eight,
// us: 8 rows 40 / 37, 30 rows 48 / 45, 64 rows 44 / 44, 96 rows 45 / 45, 128 rows 45 / 46 (the writes).
constexpr int kInt8CopiedRows = 64, kInt8Copies = 8;

// The workspace of a product: the rows' scales and fp16 values, tickets and partial sums of split tiles.
struct Int8Workspace {
  size_t scale, q, ticket, partial, bytes;
  int items, tile_rows, copies;
};
Int8Workspace int8_workspace(const colibri_moe_int8_config_t* c, int R, int sms) {
  Int8Workspace w = {};
  w.tile_rows = int8_tile_rows(R, c->num_experts);
  w.items = sms * (kInt8PartialRows / w.tile_rows);
  w.copies = R <= kInt8CopiedRows ? kInt8Copies : 1;
  w.q = round256((size_t)R * sizeof(float));
  w.ticket = w.q + round256((size_t)w.copies * R * c->in_features * 2);
  w.partial = w.ticket + round256(w.items * sizeof(uint32_t));
  w.bytes = w.partial + (size_t)w.items * w.tile_rows * 128 * sizeof(float);
  return w;
}

struct CombineManyArgs {
  const void* y;
  const int32_t* row_of;
  const float* gate;
  void* out;
  int R, T, k, d;
};

// One block a token and stretch of columns; slots in order, each product and each sum rounded once.
template <typename Y, typename O>
__global__ void __launch_bounds__(256) combine_rows_kernel(CombineManyArgs a) {
  pdl_wait();
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c >= a.d) return;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    float s = 0.f;
    for (int i = 0; i < a.k; ++i) {
      const int r = a.row_of[(int64_t)t * a.k + i];
      if (r < 0 || r >= a.R) continue;
      s = __fadd_rn(s, __fmul_rn(a.gate[(int64_t)t * a.k + i], to_float(static_cast<const Y*>(a.y)[(int64_t)r * a.d + c])));
    }
    static_cast<O*>(a.out)[(int64_t)t * a.d + c] = from_float<O>(s);
  }
}

}  // namespace
}  // namespace colibri

using namespace colibri;

extern "C" int colibri_moe_int8_quantize(const colibri_moe_int8_config_t* cfg, const void* x, int64_t ldx, int32_t n,
                                         int8_t* q, float* scale, void* stream) {
  const int rc = check_int8_config(cfg);
  if (rc) return rc;
  if (n < 0) return COLIBRI_ERR_INVALID_ARG;
  if (n == 0) return COLIBRI_OK;
  if (!x || !q || !scale || ldx < cfg->in_features) return COLIBRI_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  for (const void* p : {x, (const void*)q, (const void*)scale})
    if (!cfg->trusted_pointers && !ops_on_device(p, device)) return COLIBRI_ERR_INVALID_ARG;
  const QuantArgs a = {x, ldx, n, nullptr, n, cfg->in_features, q, 1, scale, nullptr, 0};
  const cudaError_t e = quantize<int8_t, false>(cfg->dtype, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}

extern "C" int colibri_moe_int8_experts_workspace(const colibri_moe_int8_config_t* cfg, int32_t n_tokens, int32_t R,
                                                  size_t* bytes) {
  const int rc = check_int8_config(cfg);
  if (rc) return rc;
  if (!bytes || n_tokens < 0 || R < 0) return COLIBRI_ERR_INVALID_ARG;
  if (R > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  *bytes = R ? int8_workspace(cfg, R, sms).bytes : 0;
  return COLIBRI_OK;
}

extern "C" int colibri_moe_int8_experts(const colibri_moe_int8_config_t* cfg, const void* x, int64_t ldx,
                                        int32_t n_tokens, const int32_t* rows, int32_t R, const int32_t* offsets,
                                        const int8_t* w, const float* w_scale, const int8_t* w3,
                                        const float* w3_scale, void* y, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  const int rc = check_int8_config(cfg);
  if (rc) return rc;
  if (n_tokens < 0 || R < 0 || (!rows && R > n_tokens)) return COLIBRI_ERR_INVALID_ARG;
  if (R > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  if (R == 0) return COLIBRI_OK;
  if ((n_tokens > 0 && (!x || ldx < cfg->in_features)) || !offsets || !w || !w_scale || !y ||
      (w3 != nullptr) != (w3_scale != nullptr))
    return COLIBRI_ERR_INVALID_ARG;
  if (!ops_aligned16(w) || !ops_aligned16(w3)) return COLIBRI_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return COLIBRI_ERR_INVALID_ARG;
  if (workspace_bytes < int8_workspace(cfg, R, 0).bytes) return COLIBRI_ERR_INVALID_ARG;  // what any device needs
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  const Int8Workspace lay = int8_workspace(cfg, R, sms);
  if (workspace_bytes < lay.bytes) return COLIBRI_ERR_INVALID_ARG;
  for (const void* p : {n_tokens ? x : nullptr, (const void*)rows, (const void*)offsets, (const void*)w,
                        (const void*)w_scale, (const void*)w3, (const void*)w3_scale, (const void*)y,
                        (const void*)workspace})
    if (p && !cfg->trusted_pointers && !ops_on_device(p, device)) return COLIBRI_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const QuantArgs qa = {x, ldx, n_tokens, rows, R, cfg->in_features, ws + lay.q, lay.copies,
                        reinterpret_cast<float*>(ws + lay.scale),
                        reinterpret_cast<uint32_t*>(ws + lay.ticket), lay.items};
  Int8Maps maps;
  if (!int8_tensor_maps(lay.tile_rows, qa.q, (int64_t)lay.copies * R, w, w3, cfg->num_experts, cfg->out_features,
                        cfg->in_features, &maps))
    return COLIBRI_ERR_CUDA;
  const cudaError_t quantized =
      qa.copies > 1 ? quantize<__half, true>(cfg->dtype, qa, s) : quantize<__half, false>(cfg->dtype, qa, s);
  if (quantized != cudaSuccess) return COLIBRI_ERR_CUDA;
  const Int8Args a = {qa.scale, offsets, w_scale, w3_scale, y, reinterpret_cast<float*>(ws + lay.partial),
                      qa.ticket, lay.items, R, cfg->num_experts, cfg->in_features, cfg->out_features, lay.copies,
                      int8_limit(cfg->wait_limit_us ? cfg->wait_limit_us : kInt8WaitUs)};
  const bool bf16_out = cfg->out_dtype == COLIBRI_DTYPE_BF16;
  const cudaError_t e = launch_int8_mma(maps, lay.tile_rows, w3 != nullptr, bf16_out, a, device, sms, s);
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}

extern "C" int colibri_moe_int8_status(int32_t* status) {
  if (!status) return COLIBRI_ERR_INVALID_ARG;
  int device = 0, sms = 0, v = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  if (int8_take_status(&v) != cudaSuccess) {
    cudaGetLastError();
    return COLIBRI_ERR_CUDA;
  }
  *status = v;
  return COLIBRI_OK;
}

extern "C" int colibri_moe_combine_rows(const void* y, int32_t y_dtype, int32_t R, const int32_t* row_of,
                                        const float* gate, int32_t T, int32_t k, int32_t d, void* out,
                                        int32_t out_dtype, void* stream) {
  if (T < 0 || R < 0 || k < 1 || d < 1 || !ops_dtype(y_dtype) || !ops_dtype(out_dtype)) return COLIBRI_ERR_INVALID_ARG;
  if (k > 32 || d > 65535 * 256 || T > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  if (T == 0) return COLIBRI_OK;
  if ((R > 0 && !y) || !row_of || !gate || !out) return COLIBRI_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  for (const void* p : {R ? y : nullptr, (const void*)row_of, (const void*)gate, (const void*)out})
    if (p && !ops_on_device(p, device)) return COLIBRI_ERR_INVALID_ARG;
  const CombineManyArgs a = {y, row_of, gate, out, R, T, k, d};
  const dim3 grid(std::min(T, 32768), (d + 255) / 256);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (y_dtype == COLIBRI_DTYPE_F32)
    e = out_dtype == COLIBRI_DTYPE_F32 ? pdl_launch(combine_rows_kernel<float, float>, grid, dim3(256), 0, s, a)
                                       : pdl_launch(combine_rows_kernel<float, __nv_bfloat16>, grid, dim3(256), 0, s, a);
  else
    e = out_dtype == COLIBRI_DTYPE_F32
            ? pdl_launch(combine_rows_kernel<__nv_bfloat16, float>, grid, dim3(256), 0, s, a)
            : pdl_launch(combine_rows_kernel<__nv_bfloat16, __nv_bfloat16>, grid, dim3(256), 0, s, a);
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}
