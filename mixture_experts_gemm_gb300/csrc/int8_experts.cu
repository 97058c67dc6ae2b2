// Experts in 8-bit integers: activations quantised per row, weights per output channel.
//
//   scale_t = max |x_t| / 127,  q = round(x / scale_t)  (IEEE fp32 quotients, ties to even)
//   v[r, n] = scale_{rows[r]} w_scale[e, n] sum_k q[rows[r], k] w[e, n, k]
//   y = v, or silu(v) * v3 with a second set of weights
//
// Sums are exact: 8-bit products added in 32-bit integers (K <= 65536: below 2^30).
#include <algorithm>

#include "int8_internal.cuh"

namespace colibri {
namespace {

// One block a row: the largest magnitude, then the quotients.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantArgs a) {
  __shared__ float s_max[8];
  __shared__ int s_bad[8];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = blockIdx.x; r < a.n; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    float top = 0.f;
    bool bad = false;
    for (int i = threadIdx.x; i < a.K; i += 256) {
      const float v = fabsf(to_float(x[i]));
      bad |= !(v < INFINITY);
      top = fmaxf(top, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    bad = __any_sync(~0u, bad);
    if (lane == 0) s_max[warp] = top, s_bad[warp] = bad;
    __syncthreads();
    for (int i = 0; i < 8; ++i) top = fmaxf(top, s_max[i]), bad |= s_bad[i] != 0;
    const float scale = bad ? NAN : __fdiv_rn(top, 127.f);
    if (threadIdx.x == 0) a.scale[r] = scale;
    for (int i = threadIdx.x; i < a.K; i += 256) {
      const float q = scale > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(to_float(x[i]), scale)), -127.f), 127.f) : 0.f;
      a.q[(int64_t)r * a.K + i] = (int8_t)q;
    }
    __syncthreads();
  }
}

constexpr int kTile = 64;

// A block computes 64 rows of one expert x 64 channels; K in steps of 64 bytes through shared memory.
template <typename O, bool SWIGLU>
__global__ void __launch_bounds__(256) int8_tile_kernel(Int8Args a) {
  __shared__ int sa[kTile][17], sb[kTile][17], sc[SWIGLU ? kTile : 1][17];
  __shared__ int s_e, s_r0, s_n;
  pdl_wait();
  if (threadIdx.x == 0) {
    int tile = blockIdx.y;
    s_e = -1;
    for (int e = 0; e < a.E; ++e) {
      const int lo = min(max(a.offsets[e], 0), a.R), hi = min(max(a.offsets[e + 1], lo), a.R);
      const int tiles = (hi - lo + kTile - 1) / kTile;
      if (tile < tiles) {
        s_e = e, s_r0 = lo + tile * kTile, s_n = min(kTile, hi - s_r0);
        break;
      }
      tile -= tiles;
    }
  }
  __syncthreads();
  const int e = s_e, r0 = s_r0, n = s_n, c0 = blockIdx.x * kTile;
  if (e < 0) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int lr = threadIdx.x >> 2, lc = (threadIdx.x & 3) * 4;  // this thread's 16 bytes of a tile
  int64_t tok = -1;
  if (lr < n) {
    tok = a.rows ? a.rows[r0 + lr] : r0 + lr;
    if (tok < 0 || tok >= a.n_tokens) tok = -1;
  }
  const bool wc = c0 + lr < a.N;
  int acc[4][4] = {}, acc3[SWIGLU ? 4 : 1][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 64) {
    const bool in = k0 + lc * 4 < a.K;
    int4 va = make_int4(0, 0, 0, 0), vb = va, vc = va;
    if (tok >= 0 && in) va = *reinterpret_cast<const int4*>(a.q + tok * a.K + k0 + lc * 4);
    const int64_t wo = ((int64_t)e * a.N + c0 + lr) * a.K + k0 + lc * 4;
    if (wc && in) {
      vb = *reinterpret_cast<const int4*>(a.w + wo);
      if (SWIGLU) vc = *reinterpret_cast<const int4*>(a.w3 + wo);
    }
    __syncthreads();
    sa[lr][lc] = va.x, sa[lr][lc + 1] = va.y, sa[lr][lc + 2] = va.z, sa[lr][lc + 3] = va.w;
    sb[lr][lc] = vb.x, sb[lr][lc + 1] = vb.y, sb[lr][lc + 2] = vb.z, sb[lr][lc + 3] = vb.w;
    if constexpr (SWIGLU) sc[lr][lc] = vc.x, sc[lr][lc + 1] = vc.y, sc[lr][lc + 2] = vc.z, sc[lr][lc + 3] = vc.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = __dp4a(sa[ty + 16 * i][k], sb[tx + 16 * j][k], acc[i][j]);
          if constexpr (SWIGLU) acc3[i][j] = __dp4a(sa[ty + 16 * i][k], sc[tx + 16 * j][k], acc3[i][j]);
        }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    if (r >= n) continue;
    int64_t t = a.rows ? a.rows[r0 + r] : r0 + r;
    const bool real = t >= 0 && t < a.n_tokens;
    const float sx = real ? a.scale[t] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + tx + 16 * j;
      if (c >= a.N) continue;
      float v = __int2float_rn(acc[i][j]) * a.w_scale[(int64_t)e * a.N + c] * sx;
      if constexpr (SWIGLU) {
        const float u = __int2float_rn(acc3[i][j]) * a.w3_scale[(int64_t)e * a.N + c] * sx;
        v = v / (1.f + expf(-v)) * u;
      }
      static_cast<O*>(a.y)[(int64_t)(r0 + r) * a.N + c] = from_float<O>(v);
    }
  }
}

constexpr int kInt8MaxE = 512, kInt8MaxK = 65536, kInt8MaxN = 131072;

int check_int8_config(const colibri_moe_int8_config_t* c) {
  if (!c || c->in_features <= 0 || c->out_features <= 0 || c->num_experts <= 0 || !ops_dtype(c->dtype) ||
      !ops_dtype(c->out_dtype))
    return COLIBRI_ERR_INVALID_ARG;
  if (c->in_features % 16 || c->in_features > kInt8MaxK || c->out_features > kInt8MaxN || c->num_experts > kInt8MaxE)
    return COLIBRI_ERR_UNSUPPORTED;
  return COLIBRI_OK;
}

cudaError_t quantize(int dtype, const QuantArgs& q, int sms, cudaStream_t s) {
  const dim3 grid(std::min(q.n, sms * 8));
  return dtype == COLIBRI_DTYPE_F32 ? pdl_launch(quantize_rows_kernel<float>, grid, dim3(256), 0, s, q)
                                    : pdl_launch(quantize_rows_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, q);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

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
    if (!ops_on_device(p, device)) return COLIBRI_ERR_INVALID_ARG;
  const QuantArgs a = {x, ldx, n, cfg->in_features, q, scale};
  return quantize(cfg->dtype, a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}

extern "C" int colibri_moe_int8_experts_workspace(const colibri_moe_int8_config_t* cfg, int32_t n_tokens, int32_t R,
                                                  size_t* bytes) {
  const int rc = check_int8_config(cfg);
  if (rc) return rc;
  if (!bytes || n_tokens < 0 || R < 0) return COLIBRI_ERR_INVALID_ARG;
  *bytes = round256((size_t)n_tokens * sizeof(float)) + round256((size_t)n_tokens * cfg->in_features);
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
  if (R == 0) return COLIBRI_OK;
  if ((n_tokens > 0 && (!x || ldx < cfg->in_features)) || !offsets || !w || !w_scale || !y || (w3 != nullptr) != (w3_scale != nullptr))
    return COLIBRI_ERR_INVALID_ARG;
  if (!ops_aligned16(w) || !ops_aligned16(w3)) return COLIBRI_ERR_INVALID_ARG;
  size_t need = 0;
  colibri_moe_int8_experts_workspace(cfg, n_tokens, R, &need);
  if (need && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)))
    return COLIBRI_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  for (const void* p : {n_tokens ? x : nullptr, (const void*)rows, (const void*)offsets, (const void*)w,
                        (const void*)w_scale, (const void*)w3, (const void*)w3_scale, (const void*)y,
                        (const void*)workspace})
    if (p && !ops_on_device(p, device)) return COLIBRI_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  float* scale = reinterpret_cast<float*>(ws);
  int8_t* q = reinterpret_cast<int8_t*>(ws + round256((size_t)n_tokens * sizeof(float)));
  if (n_tokens > 0) {
    const QuantArgs qa = {x, ldx, n_tokens, cfg->in_features, q, scale};
    if (quantize(cfg->dtype, qa, sms, s) != cudaSuccess) return COLIBRI_ERR_CUDA;
  }
  const Int8Args a = {q, scale, rows, offsets, w, w3, w_scale, w3_scale, y, n_tokens, R, cfg->num_experts,
                      cfg->in_features, cfg->out_features};
  const dim3 grid((cfg->out_features + kTile - 1) / kTile, R / kTile + std::min(cfg->num_experts, R));
  cudaError_t e;
  if (cfg->out_dtype == COLIBRI_DTYPE_F32)
    e = w3 ? pdl_launch(int8_tile_kernel<float, true>, grid, dim3(256), 0, s, a)
           : pdl_launch(int8_tile_kernel<float, false>, grid, dim3(256), 0, s, a);
  else
    e = w3 ? pdl_launch(int8_tile_kernel<__nv_bfloat16, true>, grid, dim3(256), 0, s, a)
           : pdl_launch(int8_tile_kernel<__nv_bfloat16, false>, grid, dim3(256), 0, s, a);
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}

extern "C" int colibri_moe_combine_rows(const void* y, int32_t y_dtype, int32_t R, const int32_t* row_of,
                                        const float* gate, int32_t T, int32_t k, int32_t d, void* out,
                                        int32_t out_dtype, void* stream) {
  if (T < 0 || R < 0 || k < 1 || d < 1 || !ops_dtype(y_dtype) || !ops_dtype(out_dtype)) return COLIBRI_ERR_INVALID_ARG;
  if (k > 32 || d > 65535 * 256) return COLIBRI_ERR_UNSUPPORTED;
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
