// Arguments of the 8-bit experts' kernels.
#pragma once

#include "ops_common.cuh"

namespace colibri {

struct QuantArgs {
  const void* x;   // [n, K] rows of stride ldx
  int64_t ldx;
  int n, K;
  int8_t* q;       // [n, K]
  float* scale;    // [n]
};

struct Int8Args {
  const int8_t* q;         // [n_tokens, K] quantised activations
  const float* scale;      // [n_tokens]
  const int32_t* rows;     // [R] token of each row, or nullptr: the row itself
  const int32_t* offsets;  // [E + 1]
  const int8_t *w, *w3;    // [E, N, K]
  const float *w_scale, *w3_scale;  // [E, N]
  void* y;                 // [R, N]
  int n_tokens, R, E, K, N;
};

}  // namespace colibri
