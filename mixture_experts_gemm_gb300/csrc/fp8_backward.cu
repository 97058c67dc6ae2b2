// Experts in e4m3, the gradients:  d_x [R, K] = rows of d_y times columns of the weights (read as they lie, MN-major), and
// d_w [E, N, K] = columns of d_y times columns of x over an expert's rows.
#include "fp8_mma.cuh"

namespace colibri {

template <int MODE, typename O>
static cudaError_t with_form(const Fp8Maps& m, const Fp8Args& a, Fp8Form form, int device, int sms, cudaStream_t s) {
  if (form == kFp8Wide) return fp8::launch<MODE, kFp8Wide, false, O>(m, a, device, sms, s);
  return fp8::launch<MODE, kFp8Narrow, false, O>(m, a, device, sms, s);
}

cudaError_t launch_fp8_rows(const Fp8Maps& m, const Fp8Args& a, Fp8Form form, bool bf16_out, int device, int sms,
                            cudaStream_t s) {
  return bf16_out ? with_form<kFp8Rows, __nv_bfloat16>(m, a, form, device, sms, s)
                  : with_form<kFp8Rows, float>(m, a, form, device, sms, s);
}
cudaError_t launch_fp8_weights(const Fp8Maps& m, const Fp8Args& a, Fp8Form form, bool bf16_out, int device, int sms,
                               cudaStream_t s) {
  return bf16_out ? with_form<kFp8Weights, __nv_bfloat16>(m, a, form, device, sms, s)
                  : with_form<kFp8Weights, float>(m, a, form, device, sms, s);
}

}  // namespace colibri
