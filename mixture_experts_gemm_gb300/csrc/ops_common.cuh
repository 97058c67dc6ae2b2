// Shared by the layer-block operators (block norms, routing to many experts, 8-bit experts): element
// loads and stores, block reductions and the checks of the C entry points.
#pragma once

#include "colibri_moe.h"
#include "moe_internal.cuh"

namespace colibri {

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Eight consecutive elements from a 16-byte aligned address.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
  v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over all threads of the block, the same bits in every thread (each warp adds the warps' sums in
// the same order).  `buf` holds kSumBuf floats of shared memory, two halves used in turn: one barrier a call
// is enough, because no warp can write the half that a slower one still reads without passing the
// barrier of the call between.
constexpr int kSumBuf = 2 * 32 * 4;
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* buf, int& turn) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (warps == 1) return;
  static_assert(N <= 4, "kSumBuf");
  float* b = buf + turn * (kSumBuf / 2);
  turn ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[warp * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? b[lane * N + i] : 0.f);
}

// ---- host side of the entry points
constexpr int kOpsMaxDevices = 64;
// Row numbers are 32-bit.  Loops over rows, and rows fetched ahead, pass the last one by a few grid widths or one
// block's rows (at most 2^31 / 128): with this limit none of them wraps.
constexpr int32_t kOpsMaxRows = INT32_MAX - (1 << 24);

inline bool ops_on_device(const void* p, int device) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == device);
}
// The current device's index and SM count; false without a usable device.
inline bool ops_device(int* device, int* sms) {
  static int cached[kOpsMaxDevices];  // SM counts: the same value whichever thread stores it
  if (cudaGetDevice(device) != cudaSuccess || *device < 0 || *device >= kOpsMaxDevices) {
    cudaGetLastError();
    return false;
  }
  int n = __atomic_load_n(&cached[*device], __ATOMIC_RELAXED);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *device) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return false;
    }
    __atomic_store_n(&cached[*device], n, __ATOMIC_RELAXED);
  }
  *sms = n;
  return true;
}
inline bool ops_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool ops_dtype(int32_t t) { return t == COLIBRI_DTYPE_F32 || t == COLIBRI_DTYPE_BF16; }
inline int ops_elem(int32_t t) { return t == COLIBRI_DTYPE_F32 ? 4 : 2; }

}  // namespace colibri
