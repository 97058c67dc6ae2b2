// Experts in e4m3, the gradients:  d_x [R, K] = rows of d_y times columns of the weights (read as they lie, MN-major), and
// d_w [E, N, K] = columns of d_y times columns of x over an expert's rows.
#include "fp8_mma.cuh"

namespace colibri {

template <int MODE>
static cudaError_t with_form(const Fp8Maps& m, const Fp8Args& a, bool pair, bool bf16_out, int device, int sms,
                             cudaStream_t s) {
  using B = __nv_bfloat16;
  if (pair)
    return bf16_out ? fp8::launch<MODE, true, false, B>(m, a, device, sms, s)
                    : fp8::launch<MODE, true, false, float>(m, a, device, sms, s);
  return bf16_out ? fp8::launch<MODE, false, false, B>(m, a, device, sms, s)
                  : fp8::launch<MODE, false, false, float>(m, a, device, sms, s);
}

cudaError_t launch_fp8_rows(const Fp8Maps& m, const Fp8Args& a, bool pair, bool bf16_out, int device, int sms, cudaStream_t s) {
  return with_form<kFp8Rows>(m, a, pair, bf16_out, device, sms, s);
}
cudaError_t launch_fp8_weights(const Fp8Maps& m, const Fp8Args& a, bool pair, bool bf16_out, int device, int sms,
                               cudaStream_t s) {
  return with_form<kFp8Weights>(m, a, pair, bf16_out, device, sms, s);
}

}  // namespace colibri
