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
// Measured, with a bf16 copy and fp32 gradients: 218 M elements in fp32 967 us (6.76 TB/s,
// the rate of a copy), 67.6 M in 8 bits 193 us (6.36 TB/s).
#include <math.h>

#include "fp8_common.cuh"
#include "mxq_host.h"

namespace mxq {

__device__ uint32_t g_err_adamw;

namespace {

constexpr int A_THREADS = 256;
constexpr int A_CHUNK = 8192;      // elements of a CTA, a multiple of A_THREADS * 4 and F_BLOCK
constexpr float A_LEAST = 0.001953125f;   // 2^-9, the smallest code above zero
constexpr int64_t A_CHUNKS = int64_t(1) << 31;   // of a launch, fewer than
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
  // The moments take one rounding per operation, the root's included: an 8-bit state
  // amplifies a last bit into a whole code where a value lies next to a border, and so
  // the same state comes from any fp32 program that follows the formula step by step.
  // The quotient is rounded once too.  The hardware's, within 2^-22, took 956 instead of
  // 967 us in 32 bits and 189 instead of 193 in 8 (the cases above): not worth two bits.
  MXQ_DEV float update(float p, float g, float decay, float& m, float& v, float& r) const {
    g = __fmul_rn(g, scale);
    m = __fadd_rn(__fmul_rn(m, b1), __fmul_rn(g, c1));
    v = __fadd_rn(__fmul_rn(v, b2), __fmul_rn(__fmul_rn(g, g), c2));
    r = __fsqrt_rn(v);
    const float kept = fmaf(-lr * decay, p, p);
    return fmaf(-step_size, __fdiv_rn(m, fmaf(r, inv_r, eps)), kept);
  }
};

// Scale and multiplier of a block of a moment from its amax: the block-128 format's rule
// with a product by 1 / 448 in place of the division.
MXQ_DEV void moment_scale(float amax, float& scale, float& mul) {
  const bool finite = amax <= 3.402823466e38f;
  scale = finite ? fmaxf(__fmul_rn(amax, 1.0f / 448.0f), F_TINY) : __uint_as_float(0x7FFFFFFFu);
  mul = finite ? __fdiv_rn(1.0f, scale) : 0.0f;
}

// Four consecutive elements, the first n where they are fewer; vec: one access.
MXQ_DEV void load_n(const float* p, bool vec, int n, float (&f)[4]) {
  if (vec) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? p[i] : 0.0f;
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

// A chunk [first, end) of a tensor with moments in 8 bits: a warp has four blocks of 128
// at a time, each lane four elements of every block: eight 16-byte and eight 4-byte loads
// in flight per lane (67.6 M elements: one block at a time 320 us, two 216 us, four 199 us).
// Three CTAs share an SM: 80 registers, of which a few are spilled, hide more of the
// memory's latency than two CTAs with 95 (with the hardware's quotient 189 against 211 us).
constexpr int A_BLOCKS = 4;

// FULL: all of them are there, every pointer is on a 16-byte boundary.
template <bool FULL, typename G>
MXQ_DEV void update_blocks(const AdamTensor& t, const G* g, const AdamStep& step, int64_t base,
                           int64_t end, bool aligned) {
  const int lane = threadIdx.x & 31;
  const int64_t at = base + lane * 4;
  float* const tp = t.p + at;
  const G* const tg = g + at;
  uint8_t *const mc = static_cast<uint8_t*>(t.m) + at, *const rc = static_cast<uint8_t*>(t.v) + at;
  float p[A_BLOCKS][4], d[A_BLOCKS][4];
  uint32_t mw[A_BLOCKS], rw[A_BLOCKS];
  int n[A_BLOCKS];
  bool vec[A_BLOCKS];
  // scales: the first A_BLOCKS lanes hold m's of the blocks, the next ones r's
  const int64_t block = base / F_BLOCK + lane % A_BLOCKS;
  const bool scaled = lane < 2 * A_BLOCKS && (FULL || block * F_BLOCK < end);
  float* const scale_at = (lane < A_BLOCKS ? t.m_scale : t.r_scale) + block;
  float scale = scaled ? *scale_at : 0.0f;
#pragma unroll
  for (int q = 0; q < A_BLOCKS; ++q) {
    const int i = q * F_BLOCK;
    n[q] = FULL ? 4 : static_cast<int>(max(min(end - at - i, int64_t(4)), int64_t(0)));
    vec[q] = FULL || (aligned && n[q] == 4);
    load_n(tp + i, vec[q], n[q], p[q]);
    load_n(tg + i, vec[q], n[q], d[q]);
    mw[q] = load_codes(mc + i, vec[q], n[q]);
    rw[q] = load_codes(rc + i, vec[q], n[q]);
  }
  float m[A_BLOCKS][4], r[A_BLOCKS][4], top = 0.0f;
#pragma unroll
  for (int q = 0; q < A_BLOCKS; ++q) {
    const int i = q * F_BLOCK;
    const float ms = __shfl_sync(~0u, scale, q), rs = __shfl_sync(~0u, scale, A_BLOCKS + q);
    float v[4];
    decode4(mw[q], m[q]);
    decode4(rw[q], v);
    uint32_t m_top = 0, r_top = 0;   // magnitudes order as their bits, NaN above infinity
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[q][j] *= ms;
      v[j] *= rs;
      v[j] *= v[j];
      p[q][j] = step.update(p[q][j], d[q][j], t.decay, m[q][j], v[j], r[q][j]);
      if (!FULL && j >= n[q]) m[q][j] = r[q][j] = 0.0f;
      m_top = max(m_top, __float_as_uint(m[q][j]) & 0x7FFFFFFFu);
      r_top = max(r_top, __float_as_uint(r[q][j]) & 0x7FFFFFFFu);
    }
    store_n(tp + i, vec[q], n[q], p[q]);
    if (t.copy) store_n(t.copy + at + i, vec[q], n[q], p[q]);
    m_top = __reduce_max_sync(~0u, m_top);
    r_top = __reduce_max_sync(~0u, r_top);
    if (lane == q) top = __uint_as_float(m_top);
    if (lane == A_BLOCKS + q) top = __uint_as_float(r_top);
  }
  // all scales and their reciprocals at once, one per lane
  float mul;
  moment_scale(top, scale, mul);
  if (scaled) *scale_at = scale;
#pragma unroll
  for (int q = 0; q < A_BLOCKS; ++q) {
    const int i = q * F_BLOCK;
    const float km = __shfl_sync(~0u, mul, q), kr = __shfl_sync(~0u, mul, A_BLOCKS + q);
    float a[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __fmul_rn(m[q][j], km);
      b[j] = __fmul_rn(r[q][j], kr);
      if (r[q][j] > 0.0f) b[j] = fmaxf(b[j], A_LEAST);
    }
    const uint32_t ca = km == 0.0f ? 0u : cvt_e4m3x4(a[0], a[1], a[2], a[3]);
    const uint32_t cb = kr == 0.0f ? 0u : cvt_e4m3x4(b[0], b[1], b[2], b[3]);
    store_codes(mc + i, vec[q], n[q], ca);
    store_codes(rc + i, vec[q], n[q], cb);
  }
}

template <typename G>
MXQ_DEV void update_codes(const AdamTensor& t, const G* g, const AdamStep& step, int64_t first,
                          int64_t end, bool aligned) {
  constexpr int SPAN = A_BLOCKS * F_BLOCK;
  for (int64_t base = first + (threadIdx.x >> 5) * SPAN; base < end;
       base += A_THREADS / 32 * SPAN) {
    if (aligned && base + SPAN <= end) update_blocks<true>(t, g, step, base, end, true);
    else update_blocks<false>(t, g, step, base, end, aligned);
  }
}

template <typename G>
MXQ_DEV void update_floats(const AdamTensor& t, const G* g, const AdamStep& step, int64_t first,
                           int64_t end, bool aligned) {
  float *tm = static_cast<float*>(t.m), *tv = static_cast<float*>(t.v);
#pragma unroll 2
  for (int64_t i = first + threadIdx.x * 4; i < end; i += A_THREADS * 4) {
    const int n = static_cast<int>(min(end - i, int64_t(4)));
    const bool vec = aligned && n == 4;
    float p[4], d[4], m[4], v[4], r;
    load_n(t.p + i, vec, n, p);
    load_n(g + i, vec, n, d);
    load_n(tm + i, vec, n, m);
    load_n(tv + i, vec, n, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = step.update(p[j], d[j], t.decay, m[j], v[j], r);
    store_n(t.p + i, vec, n, p);
    if (t.copy) store_n(t.copy + i, vec, n, p);
    store_n(tm + i, vec, n, m);
    store_n(tv + i, vec, n, v);
  }
}

template <int MAX, typename G, bool CODES>
__global__ void __launch_bounds__(A_THREADS, CODES ? 3 : 1) adamw_kernel(const __grid_constant__ AdamLaunch<MAX> a) {
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
  if constexpr (CODES) update_codes(t, g, step, first, end, aligned);
  else update_floats(t, g, step, first, end, aligned);
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
      if (c >= A_CHUNKS) return MXQ_ERR_ARG;
      if (chunks + c >= A_CHUNKS) break;   // the next launch takes it
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
