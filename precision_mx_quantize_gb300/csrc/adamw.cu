// AdamW over many tensors in one launch.  With g the gradient times its scale, t the step:
//   m <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2,
//   p <- p - lr decay p - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32, and a bf16 copy of p for the quantizers.  The moments are held in fp32, or in
// 8 bits: m and r = sqrt(v) as E4M3 codes with one fp32 scale per block of 128 elements
// (the block-128 format's rule).  r and not v, because v's range is twice r's in powers
// of two and E4M3 spans 17 of them; and an r above zero keeps at least the smallest code,
// because p's step divides by it.  p's step uses m and v before their rounding.
//
// An element's work is a few dozen instructions for 18 to 30 bytes, so memory bounds it:
// each CTA takes a chunk of one tensor and every thread has several 16-byte loads in flight.
#include <math.h>

#include "fp8_common.cuh"
#include "mxq_host.h"

namespace mxq {

__device__ uint32_t g_err_adamw;

namespace {

constexpr int A_THREADS = 256;
constexpr int A_CHUNK = 8192;      // elements of a CTA, a multiple of A_THREADS * 4 and F_BLOCK
constexpr int A_MAX = 384;         // tensors of a launch (their table is a kernel argument)

struct AdamTensor {
  float* p;
  void *m, *v;                     // fp32 moments, or codes of m and r
  float *m_scale, *r_scale;
  __nv_bfloat16* copy;             // or NULL
  int64_t n;
  int32_t chunk0;                  // first chunk in the launch
  float decay;
};

struct AdamScalars {
  float b1, c1, b2, c2;            // c = 1 - b
  float log_b1, log_b2;
  float eps, lr, k1, inv_r;        // k1 = 1 / (1 - b1^t), inv_r = 1 / sqrt(1 - b2^t)
  const float *lr_at, *scale_at;   // or NULL
  const int64_t* step_at;          // or NULL
};

template <int MAX>
struct AdamLaunch {
  AdamTensor t[MAX];
  const void* g[MAX];
  AdamScalars s;
  int32_t count;
};

// What a step multiplies by, the same in every thread.
struct AdamStep {
  float b1, c1, b2, c2, eps, lr, step_size, inv_r, scale;
  bool skip;
  MXQ_DEV explicit AdamStep(const AdamScalars& s)
      : b1(s.b1), c1(s.c1), b2(s.b2), c2(s.c2), eps(s.eps), lr(s.lr_at ? *s.lr_at : s.lr),
        inv_r(s.inv_r), scale(1.0f), skip(false) {
    float k1 = s.k1;
    if (s.step_at) {   // 1 - b^t without the cancellation at small t
      const float t = static_cast<float>(max(*s.step_at, int64_t(1)));
      k1 = 1.0f / -expm1f(t * s.log_b1);
      inv_r = rsqrtf(-expm1f(t * s.log_b2));
    }
    step_size = lr * k1;
    if (s.scale_at) {
      scale = *s.scale_at;
      skip = !(fabsf(scale) <= 3.402823466e38f);   // NaN or infinity: leave all as it is
    }
  }
  // One element: m and v become the new moments, r = sqrt(v); returns the new p.
  MXQ_DEV float update(float p, float g, float decay, float& m, float& v, float& r) const {
    g *= scale;
    m = fmaf(b1, m, c1 * g);
    v = fmaf(b2, v, c2 * g * g);
    r = sqrtf(v);
    const float kept = fmaf(-lr * decay, p, p);
    return fmaf(-step_size, m / fmaf(r, inv_r, eps), kept);
  }
};

// N consecutive elements; vec: at an address for one load or two.
template <int N>
MXQ_DEV void load_n(const float* p, bool vec, int n, float (&f)[N]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = i < n ? p[i] : 0.0f;
  }
}

MXQ_DEV void load_n(const __nv_bfloat16* p, bool vec, int n, float (&f)[4]) {
  if (vec) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    f[0] = bf16lo(v.x); f[1] = bf16hi(v.x); f[2] = bf16lo(v.y); f[3] = bf16hi(v.y);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
  }
}

MXQ_DEV void store_n(float* p, bool vec, int n, const float (&f)[4]) {
  if (vec) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = f[i];
  }
}

MXQ_DEV void store_n(__nv_bfloat16* p, bool vec, int n, const float (&f)[4]) {
  if (vec) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = __float2bfloat16_rn(f[i]);
  }
}

MXQ_DEV uint32_t load_codes(const uint8_t* p, bool vec, int n) {
  if (vec) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) w |= static_cast<uint32_t>(p[i]) << (8 * i);
  return w;
}

MXQ_DEV void store_codes(uint8_t* p, bool vec, int n, uint32_t w) {
  if (vec) {
    *reinterpret_cast<uint32_t*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(w >> (8 * i));
  }
}

// Values of four E4M3 codes.
MXQ_DEV void decode4(uint32_t w, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// Codes of a block of 128, four values per lane; `least` is the smallest code's value
// that a value above zero keeps (0: none).
MXQ_DEV uint32_t encode_block(const float (&x)[4], float least, float& scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  top = __reduce_max_sync(~0u, top);   // magnitudes order as their bits, NaN above infinity
  float mul;
  fp8_scale<MXQ_E4M3>(__uint_as_float(top), scale, mul);
  if (mul == 0.0f) return 0u;
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = __fmul_rn(x[i], mul);
    if (x[i] > 0.0f) q[i] = fmaxf(q[i], least);
  }
  return cvt_e4m3x4(q[0], q[1], q[2], q[3]);
}

template <int MAX, typename G, bool CODES>
__global__ void __launch_bounds__(A_THREADS) adamw_kernel(const __grid_constant__ AdamLaunch<MAX> a) {
  griddep_wait();
  griddep_launch_dependents();
  int lo = 0, hi = a.count;   // the chunk's tensor
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.t[mid].chunk0 <= static_cast<int>(blockIdx.x)) lo = mid;
    else hi = mid;
  }
  const AdamTensor& t = a.t[lo];
  const G* g = static_cast<const G*>(a.g[lo]);
  const AdamStep step(a.s);
  if (step.skip) return;
  const int64_t first = int64_t(static_cast<int>(blockIdx.x) - t.chunk0) * A_CHUNK;
  const int64_t end = min(first + A_CHUNK, t.n);
  if (!MXQ_IN_BOUNDS(first >= 0 && first < t.n, &g_err_adamw, SITE_B_ADAMW)) return;
  // every pointer of the tensor at a 16-byte boundary: four elements are one access
  const uintptr_t bits = reinterpret_cast<uintptr_t>(t.p) | reinterpret_cast<uintptr_t>(g) |
                         reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v) |
                         reinterpret_cast<uintptr_t>(t.copy);
  const bool aligned = (bits & 15u) == 0;
  const int lane = threadIdx.x & 31;
#pragma unroll 2
  for (int64_t i = first + threadIdx.x * 4; i - lane * 4 < end; i += A_THREADS * 4) {
    const int n = static_cast<int>(max(min(end - i, int64_t(4)), int64_t(0)));
    const bool vec = aligned && n == 4;
    float p[4], d[4], m[4], v[4], r[4];
    load_n(t.p + i, vec, n, p);
    load_n(g + i, vec, n, d);
    if constexpr (CODES) {
      const float ms = t.m_scale[i / F_BLOCK], rs = t.r_scale[i / F_BLOCK];   // the warp's block
      decode4(load_codes(static_cast<const uint8_t*>(t.m) + i, vec, n), m);
      decode4(load_codes(static_cast<const uint8_t*>(t.v) + i, vec, n), v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] *= ms;
        v[j] *= rs;
        v[j] *= v[j];
      }
    } else {
      load_n(static_cast<const float*>(t.m) + i, vec, n, m);
      load_n(static_cast<const float*>(t.v) + i, vec, n, v);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p[j] = step.update(p[j], d[j], t.decay, m[j], v[j], r[j]);
      if (j >= n) m[j] = r[j] = 0.0f;
    }
    store_n(t.p + i, vec, n, p);
    if (t.copy) store_n(t.copy + i, vec, n, p);
    if constexpr (CODES) {
      float ms, rs;
      const uint32_t mc = encode_block(m, 0.0f, ms);
      const uint32_t rc = encode_block(r, 0.001953125f, rs);
      store_codes(static_cast<uint8_t*>(t.m) + i, vec, n, mc);
      store_codes(static_cast<uint8_t*>(t.v) + i, vec, n, rc);
      if (lane == 0) {
        t.m_scale[i / F_BLOCK] = ms;
        t.r_scale[i / F_BLOCK] = rs;
      }
    } else {
      store_n(static_cast<float*>(t.m) + i, vec, n, m);
      store_n(static_cast<float*>(t.v) + i, vec, n, v);
    }
  }
}

template <int MAX>
mxq_status adamw_launch(const mxq_adamw_tensor* t, const void* const* g, int count, bool bf16,
                        bool codes, const AdamScalars& s, cudaStream_t st) {
  AdamLaunch<MAX> a;
  a.s = s;
  int i = 0;
  while (i < count) {
    int64_t chunks = 0;
    a.count = 0;
    for (; i < count && a.count < MAX; ++i) {
      if (t[i].n == 0) continue;
      const int64_t c = (t[i].n + A_CHUNK - 1) / A_CHUNK;
      if (chunks + c >= (int64_t(1) << 31)) break;
      AdamTensor& d = a.t[a.count];
      d.p = t[i].param;
      d.m = t[i].m;
      d.v = t[i].v;
      d.m_scale = t[i].m_scale;
      d.r_scale = t[i].r_scale;
      d.copy = static_cast<__nv_bfloat16*>(t[i].copy);
      d.n = t[i].n;
      d.chunk0 = static_cast<int32_t>(chunks);
      d.decay = t[i].weight_decay;
      a.g[a.count++] = g[i];
      chunks += c;
    }
    if (a.count == 0) continue;
    const unsigned grid = static_cast<unsigned>(chunks);
    const auto run = [&](auto kernel) { return launch_early(kernel, grid, A_THREADS, 0, st, a); };
    using B = __nv_bfloat16;
    const bool ok = codes ? (bf16 ? run(adamw_kernel<MAX, B, true>) : run(adamw_kernel<MAX, float, true>))
                          : (bf16 ? run(adamw_kernel<MAX, B, false>) : run(adamw_kernel<MAX, float, false>));
    if (!ok) return MXQ_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace

uint32_t take_adamw_error() {
  uint32_t h = 0;
  if (cudaMemcpyFromSymbol(&h, g_err_adamw, sizeof(h)) != cudaSuccess) return MXQ_ERR_CUDA;
  if (h) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_err_adamw, &z, sizeof(z));
  }
  return h;
}

}  // namespace mxq

using namespace mxq;

extern "C" mxq_status mxq_adamw(const mxq_adamw_tensor* tensors, const void* const* grads,
                                int count, const mxq_adamw_args* args, void* stream) {
  if (!args || count < 0 || (count > 0 && (!tensors || !grads))) return MXQ_ERR_ARG;
  const mxq_adamw_args& q = *args;
  if ((q.grad_dtype != MXQ_OUT_F32 && q.grad_dtype != MXQ_OUT_BF16) ||
      (q.state_bits != 8 && q.state_bits != 32))
    return MXQ_ERR_ARG;
  if (!(q.beta1 >= 0.0 && q.beta1 < 1.0 && q.beta2 >= 0.0 && q.beta2 < 1.0 && q.eps >= 0.0) ||
      (!q.step_at && q.step < 1))
    return MXQ_ERR_ARG;
  if (!aligned4(q.lr_at) || !aligned4(q.grad_scale_at) ||
      (reinterpret_cast<uintptr_t>(q.step_at) & 7u) != 0)
    return MXQ_ERR_ALIGN;
  const bool codes = q.state_bits == 8, bf16 = q.grad_dtype == MXQ_OUT_BF16;
  for (int i = 0; i < count; ++i) {
    const mxq_adamw_tensor& t = tensors[i];
    if (t.n < 0) return MXQ_ERR_ARG;
    if (t.n == 0) continue;
    if (!t.param || !t.m || !t.v || !grads[i] || (codes && (!t.m_scale || !t.r_scale)))
      return MXQ_ERR_ARG;
    const uintptr_t words = reinterpret_cast<uintptr_t>(t.param) |
                            reinterpret_cast<uintptr_t>(t.m_scale) |
                            reinterpret_cast<uintptr_t>(t.r_scale) |
                            (codes ? 0 : reinterpret_cast<uintptr_t>(t.m) |
                                             reinterpret_cast<uintptr_t>(t.v)) |
                            (bf16 ? 0 : reinterpret_cast<uintptr_t>(grads[i]));
    const uintptr_t halves = reinterpret_cast<uintptr_t>(t.copy) |
                             reinterpret_cast<uintptr_t>(grads[i]);
    if ((words & 3u) != 0 || (halves & 1u) != 0) return MXQ_ERR_ALIGN;
  }
  AdamScalars s = {};
  s.b1 = static_cast<float>(q.beta1);
  s.c1 = static_cast<float>(1.0 - q.beta1);
  s.b2 = static_cast<float>(q.beta2);
  s.c2 = static_cast<float>(1.0 - q.beta2);
  s.log_b1 = static_cast<float>(std::log(q.beta1));
  s.log_b2 = static_cast<float>(std::log(q.beta2));
  s.eps = static_cast<float>(q.eps);
  s.lr = static_cast<float>(q.lr);
  const double t = static_cast<double>(q.step_at ? 1 : q.step);
  s.k1 = static_cast<float>(1.0 / (1.0 - std::pow(q.beta1, t)));
  s.inv_r = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(q.beta2, t)));
  s.lr_at = q.lr_at;
  s.step_at = q.step_at;
  s.scale_at = q.grad_scale_at;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // The table is copied with the launch: a small one for few tensors.
  if (count <= 32) return adamw_launch<32>(tensors, grads, count, bf16, codes, s, st);
  return adamw_launch<A_MAX>(tensors, grads, count, bf16, codes, s, st);
}
