// Experts in e4m3, forward:  y [R, N] = rows of x times rows of the experts' weights, with or without the gated pair.
#include "fp8_mma.cuh"

namespace colibri {

cudaError_t launch_fp8_forward(const Fp8Maps& m, const Fp8Args& a, bool pair, bool gated, bool bf16_out, int device, int sms,
                               cudaStream_t s) {
  using B = __nv_bfloat16;
  auto with = [&](auto p) {
    constexpr bool P = decltype(p)::value;
    if (gated)
      return bf16_out ? fp8::launch<kFp8Forward, P, true, B>(m, a, device, sms, s)
                      : fp8::launch<kFp8Forward, P, true, float>(m, a, device, sms, s);
    return bf16_out ? fp8::launch<kFp8Forward, P, false, B>(m, a, device, sms, s)
                    : fp8::launch<kFp8Forward, P, false, float>(m, a, device, sms, s);
  };
  return pair ? with(std::true_type()) : with(std::false_type());
}

}  // namespace colibri
