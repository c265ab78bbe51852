// Rules of the block-128 FP8 format shared by its quantizers, the norms and
// the product.
#pragma once

#include "mxq_common.cuh"

namespace mxq {

constexpr int F_BLOCK = 128;                     // elements per scale
constexpr float F_TINY = 1.17549435e-38f;        // 2^-126, the smallest scale

template <int FMT>
struct Fp8 {
  static_assert(FMT == MXQ_E4M3 || FMT == MXQ_E5M2, "8-bit formats");
  static constexpr float fmax = FMT == MXQ_E4M3 ? 448.0f : 57344.0f;
};

// Scale and multiplier of a block from its amax: the multiplier is 0 for a
// block with a NaN or an infinity, whose scale is NaN and whose codes are 0.
template <int FMT>
MXQ_DEV void fp8_scale(float amax, float& scale, float& mul) {
  if (!(amax <= 3.402823466e38f)) {
    scale = __uint_as_float(0x7FFFFFFFu);
    mul = 0.0f;
    return;
  }
  scale = fmaxf(__fdiv_rn(amax, Fp8<FMT>::fmax), F_TINY);
  mul = __fdiv_rn(1.0f, scale);
}

// Four codes of values already multiplied, a0 in the lowest byte.
template <int FMT>
MXQ_DEV uint32_t fp8_cvt4(float a0, float a1, float a2, float a3) {
  if constexpr (FMT == MXQ_E4M3) return cvt_e4m3x4(a0, a1, a2, a3);
  else return cvt_e5m2x4(a0, a1, a2, a3);
}

// Eight codes of eight values times mul (0: a block without a finite amax).
template <int FMT>
MXQ_DEV uint2 fp8_encode8(const float (&v)[8], float mul) {
  uint2 w;
  w.x = fp8_cvt4<FMT>(__fmul_rn(v[0], mul), __fmul_rn(v[1], mul), __fmul_rn(v[2], mul),
                      __fmul_rn(v[3], mul));
  w.y = fp8_cvt4<FMT>(__fmul_rn(v[4], mul), __fmul_rn(v[5], mul), __fmul_rn(v[6], mul),
                      __fmul_rn(v[7], mul));
  if (mul == 0.0f) w = make_uint2(0u, 0u);
  return w;
}

}  // namespace mxq
