// Arguments and launchers of the kernels for experts in 8-bit floating point (quantisers and entry points in
// fp8_experts.cu, products in fp8_mma.cuh).
#pragma once

#include <cudaTypedefs.h>

#include "ops_common.cuh"

namespace colibri {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // colibri_moe.cu; nullptr if the driver has none

constexpr int kFp8Block = 128;       // values of a scale's block
constexpr int kFp8MaxExperts = 512;
constexpr int kFp8MaxSplits = 8;     // parts of the contraction that a tile may be split into
constexpr int kFp8TokMaps = 3;       // boxes of 32, 64 and 128 rows

// How long a wait may last, and how often it reads the clock: at the tries whose number has none of these bits.
struct Fp8Limit {
  uint64_t ns;
  uint32_t clock_mask;
};

// The three products of a layer  y = x w^T:
//   kFp8Forward   y [R, N]:    rows of x times rows of w        (contraction K, blocks along K)
//   kFp8Rows      d_x [R, K]:  rows of d_y times columns of w   (contraction N, blocks along N)
//   kFp8Weights   d_w [N, K]:  columns of d_y times columns of x (contraction the expert's rows, blocks of 128 of them)
enum Fp8Mode { kFp8Forward, kFp8Rows, kFp8Weights };

struct Fp8Maps {
  CUtensorMap a[kFp8TokMaps];  // rows in boxes of 32, 64 and 128 (kFp8Weights: the last one)
  CUtensorMap b, b3;
};

struct Fp8Args {
  const int32_t* offsets;             // [E + 1]
  const float* a_scale;               // [blocks][lda]: of the M side's rows
  int64_t lda;
  const float *w_scale, *w3_scale;    // [E, nblocks, kblocks] of the weights
  const float* x_scale;               // kFp8Weights: [blocks][ldx], of the N side's columns
  int64_t ldx;
  void* y;                            // [R, out] or [E, N, out], out the product's columns
  float* partial;                     // [items][tile columns][128] sums of parts of the contraction
  uint32_t* ticket;                   // [items], zero at launch: parts of a tile done
  int max_items;                      // capacity of the two
  int R, E, N, K;
  Fp8Limit limit;
  int* status;                        // the device's status word
};

// The segments of the experts' rows inside 0..R, none reaching back into an earlier one, by one warp: first row and
// rows of each expert, and tiles[e] = sum of per_rows(rows) over the experts before e, for e = 0..E.
template <typename F>
__device__ __forceinline__ void fp8_segments(const int32_t* offsets, int E, int R, int lane, int* row0, int* rows,
                                             int* tiles, F per_rows) {
  const int per = (E + 31) / 32;
  int reach = 0;  // the furthest end of any expert before this lane's
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < E) reach = max(reach, min(max(offsets[e + 1], 0), R));
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, reach, o);
    if (lane >= o) reach = max(reach, v);
  }
  reach = __shfl_up_sync(~0u, reach, 1);
  if (lane == 0) reach = 0;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e >= E) break;
    const int hi = min(max(offsets[e + 1], 0), R);
    const int lo = max(min(max(offsets[e], 0), R), reach);
    reach = max(reach, hi);
    const int n = max(hi - lo, 0);
    row0[e] = lo, rows[e] = n, tiles[e] = sum;
    sum += per_rows(n);
  }
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) tiles[E] = before;
  before -= sum;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < E) tiles[e] += before;
  }
}

// Forms of the products: tiles of 128 rows x 128 or 256 columns.
enum Fp8Form { kFp8Narrow, kFp8Wide };
cudaError_t launch_fp8_forward(const Fp8Maps& m, const Fp8Args& a, Fp8Form form, bool gated, bool bf16_out, int device, int sms,
                               cudaStream_t s);
cudaError_t launch_fp8_rows(const Fp8Maps& m, const Fp8Args& a, Fp8Form form, bool bf16_out, int device, int sms,
                            cudaStream_t s);
cudaError_t launch_fp8_weights(const Fp8Maps& m, const Fp8Args& a, Fp8Form form, bool bf16_out, int device, int sms,
                               cudaStream_t s);

}  // namespace colibri
