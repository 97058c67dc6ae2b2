// Arguments and launchers of the 8-bit experts' kernels (quantiser in int8_experts.cu, products in
// int8_mma.cu).
#pragma once

#include <cudaTypedefs.h>

#include "ops_common.cuh"

namespace colibri {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // colibri_moe.cu; nullptr if the driver has none

// The product kernel's forms: most token rows of a tile.
constexpr int kInt8WideRows = 256, kInt8NarrowRows = 64;
constexpr int kInt8MaxSplits = 8;     // parts of K a tile may be split into
constexpr int kInt8SplitWaves = 4;    // items (tiles x parts) of a split product, at most this many per SM

struct Int8Args {
  const float* scale;               // [R] of the quantised rows
  const int32_t* offsets;           // [E + 1]
  const float *w_scale, *w3_scale;  // [E, N]
  void* y;                          // [R, N]
  float* partial;                   // narrow form: [items][kInt8NarrowRows][128], or nullptr: never split
  uint32_t* ticket;                 // [items], zero at launch: parts of a tile done
  int max_items;                    // capacity of the two
  int R, E, K, N;
  uint64_t timeout_ns;
};

struct QuantArgs {
  const void* x;        // [n_tokens, K] rows of stride ldx
  int64_t ldx;
  int n_tokens;
  const int32_t* rows;  // token of each row, or nullptr: the row itself
  int n, K;             // rows to write
  void* q;              // [n, K] int8 or fp16
  float* scale;         // [n]
  uint32_t* ticket;     // cleared for the product kernel, or nullptr
  int n_ticket;
};

// rows: q [R, K] fp16 whole numbers; w, w3: [E * N, K] int8.
bool int8_tensor_maps(const void* q, int R, const int8_t* w, const int8_t* w3, int E, int N, int K, CUtensorMap* maps);
cudaError_t launch_int8_mma(const CUtensorMap* maps, bool wide, bool swiglu, bool bf16_out, const Int8Args& a, int device,
                            int sms, cudaStream_t s);

}  // namespace colibri
