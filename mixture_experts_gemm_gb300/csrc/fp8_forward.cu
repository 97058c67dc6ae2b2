// Experts in e4m3, forward:  y [R, N] = rows of x times rows of the experts' weights, with or without the gated pair.
#include "fp8_mma.cuh"

namespace colibri {

template <bool GATED, typename O>
static cudaError_t with_form(const Fp8Maps& m, const Fp8Args& a, Fp8Form form, int device, int sms, cudaStream_t s) {
  if (form == kFp8Wide) return fp8::launch<kFp8Forward, kFp8Wide, GATED, O>(m, a, device, sms, s);
  return fp8::launch<kFp8Forward, kFp8Narrow, GATED, O>(m, a, device, sms, s);
}

cudaError_t launch_fp8_forward(const Fp8Maps& m, const Fp8Args& a, Fp8Form form, bool gated, bool bf16_out, int device, int sms,
                               cudaStream_t s) {
  using B = __nv_bfloat16;
  if (gated)
    return bf16_out ? with_form<true, B>(m, a, form, device, sms, s) : with_form<true, float>(m, a, form, device, sms, s);
  return bf16_out ? with_form<false, B>(m, a, form, device, sms, s) : with_form<false, float>(m, a, form, device, sms, s);
}

}  // namespace colibri
