// Arguments and launchers of the 8-bit experts' kernels (quantiser in int8_experts.cu, products in
// int8_mma.cu).
#pragma once

#include <cudaTypedefs.h>

#include "ops_common.cuh"

namespace colibri {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // colibri_moe.cu; nullptr if the driver has none

constexpr int kInt8MaxSplits = 8;     // parts of K a tile may be split into
constexpr int kInt8PartialRows = 256;  // tile rows x items (tiles x parts) per SM that a split product may hold

// How long a wait may last, and how often it reads the clock: at the tries whose number has none of these bits.
struct Int8Limit {
  uint64_t ns;
  uint32_t clock_mask;
};

struct Int8Args {
  const float* scale;               // [R] of the quantised rows
  const int32_t* offsets;           // [E + 1]
  const float *w_scale, *w3_scale;  // [E, N]
  void* y;                          // [R, N]
  float* partial;                   // [items][tile rows][128] sums of parts of K
  uint32_t* ticket;                 // [items], zero at launch: parts of a tile done
  int max_items;                    // capacity of the two
  int R, E, K, N;
  int copies;                       // of the quantised rows, R apart
  Int8Limit limit;
};

struct QuantArgs {
  const void* x;        // [n_tokens, K] rows of stride ldx
  int64_t ldx;
  int n_tokens;
  const int32_t* rows;  // token of each row, or nullptr: the row itself
  int n, K;             // rows to write
  void* q;              // [copies][n, K] int8 or fp16
  int copies;
  float* scale;         // [n]
  uint32_t* ticket;     // cleared for the product kernel, or nullptr
  int n_ticket;
};

// Tensor maps: the quantised rows in boxes of 32, 64, 128 and 256 rows x 64 columns, the weights in boxes of
// 128 rows (64 of each projection) x a stage's bytes (64 or 128).
constexpr int kTokMaps = 4;
struct Int8Maps {
  CUtensorMap q[kTokMaps], w, w3;
};

// q [rows, K] fp16 whole numbers; w, w3: [E * N, K] int8.
bool int8_tensor_maps(int tile_rows, const void* q, int64_t rows, const int8_t* w, const int8_t* w3, int E, int N, int K,
                      Int8Maps* maps);
// tile_rows: 32, 64, 128 or 256 token rows a tile.
cudaError_t launch_int8_mma(const Int8Maps& maps, int tile_rows, bool swiglu, bool bf16_out, const Int8Args& a, int device,
                            int sms, cudaStream_t s);
// Waits for the current device, then reads and clears its status word.
cudaError_t int8_take_status(int* status);

}  // namespace colibri
