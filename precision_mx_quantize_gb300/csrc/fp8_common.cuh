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

// Elements `at` to `at` + 7 of a 16-byte aligned buffer, cut out of the aligned
// 16-byte words around them: two loads and fifteen selects and shifts (fp32:
// three and eighteen) in place of eight loads.  The words end REACH elements
// after `at`, at most, which has to be inside the buffer.
template <typename T>
struct Across;

template <>
struct Across<__nv_bfloat16> {
  static constexpr int REACH = 16;
  uint4 a, b;
  MXQ_DEV void clear() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  MXQ_DEV void load(const __nv_bfloat16* buf, int64_t at) {
    const uint4* q = reinterpret_cast<const uint4*>(buf + (at & ~int64_t(7)));
    a = q[0];
    b = q[1];
  }
  MXQ_DEV void cut(int64_t at, uint32_t (&w)[4]) const {
    const bool two = at & 4, one = at & 2;
    const uint32_t u[6] = {two ? a.z : a.x, two ? a.w : a.y, two ? b.x : a.z,
                           two ? b.y : a.w, two ? b.z : b.x, two ? b.w : b.y};
    const uint32_t odd = 16 * (static_cast<uint32_t>(at) & 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __funnelshift_r(one ? u[i + 1] : u[i], one ? u[i + 2] : u[i + 1], odd);
  }
};

template <>
struct Across<float> {
  static constexpr int REACH = 12;
  float4 a, b, c;
  MXQ_DEV void clear() { a = b = c = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  MXQ_DEV void load(const float* buf, int64_t at) {
    const float4* q = reinterpret_cast<const float4*>(buf + (at & ~int64_t(3)));
    a = q[0];
    b = q[1];
    c = q[2];
  }
  MXQ_DEV void cut(int64_t at, float (&f)[8]) const {
    const bool two = at & 2, one = at & 1;
    const float u[9] = {two ? a.z : a.x, two ? a.w : a.y, two ? b.x : a.z,
                        two ? b.y : a.w, two ? b.z : b.x, two ? b.w : b.y,
                        two ? c.x : b.z, two ? c.y : b.w, two ? c.z : c.x};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = one ? u[i + 1] : u[i];
  }
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
