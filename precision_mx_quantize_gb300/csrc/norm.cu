// Layer norm and RMS norm: forward (to x's type, to FP8 codes with one scale
// per block of 128, or both) and backward with the gradients of weight and
// bias.
//
//   layer  h = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   RMS    h = x rstd,           rstd = 1 / sqrt(mean(x^2) + eps)
//   y = h w + b
//   dx = rstd (g - mean(g) - h mean(g h)),  g = dy w   (RMS: no mean(g))
//   dw = sum_r dy h,  db = sum_r dy
//
// Everything between the loads and the one rounding of an output is fp32.
// The variance is taken about the mean (two passes over the row), not as a
// difference of moments, so that a large common offset costs no digits.  Sums
// over rows run in a fixed order: no atomics.
#include "fp8_common.cuh"
#include "mxq_host.h"

namespace mxq {

__device__ uint32_t g_err_norm;

namespace {

constexpr int N_MAX_WARPS = 32;

// Eight consecutive elements of a row from `col` on, zero past its end.  vec:
// the row's start is 16-byte aligned and cols % 8 == 0.
MXQ_DEV void load8(const __nv_bfloat16* row, int64_t col, int64_t cols, bool vec, float (&f)[8]) {
  if (vec) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + col);
    f[0] = bf16lo(w.x); f[1] = bf16hi(w.x); f[2] = bf16lo(w.y); f[3] = bf16hi(w.y);
    f[4] = bf16lo(w.z); f[5] = bf16hi(w.z); f[6] = bf16lo(w.w); f[7] = bf16hi(w.w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = col + j < cols ? __bfloat162float(row[col + j]) : 0.0f;
  }
}

MXQ_DEV void load8(const float* row, int64_t col, int64_t cols, bool vec, float (&f)[8]) {
  if (vec) {
    const float4 a = *reinterpret_cast<const float4*>(row + col);
    const float4 b = *reinterpret_cast<const float4*>(row + col + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = col + j < cols ? row[col + j] : 0.0f;
  }
}

MXQ_DEV uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}

MXQ_DEV void store8(__nv_bfloat16* row, int64_t col, int64_t cols, bool vec, const float (&f)[8]) {
  if (vec) {
    *reinterpret_cast<uint4*>(row + col) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                   pack_bf16(f[6], f[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < cols) row[col + j] = __float2bfloat16_rn(f[j]);
  }
}

MXQ_DEV void store8(float* row, int64_t col, int64_t cols, bool vec, const float (&f)[8]) {
  if (vec) {
    *reinterpret_cast<float4*>(row + col) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(row + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < cols) row[col + j] = f[j];
  }
}

MXQ_DEV float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// Sum over the CTA, the same in every thread.
MXQ_DEV float cta_sum(float v, float* buf) {
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_sum(v);
  __syncthreads();   // the buffer's last readers are done
  if ((threadIdx.x & 31) == 0) buf[warp] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < nw; ++w) s += buf[w];
  return s;
}

// Codes of the eight values a lane holds of a 128-element block that 16
// neighbouring lanes share, and the block's scale.
template <int FMT>
MXQ_DEV uint2 encode_block(const float (&f)[8], float& scale) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int j = 1; j < 7; j += 2) m = max3_abs_nan(m, f[j], f[j + 1]);
  m = max3_abs_nan(m, f[7], f[7]);
#pragma unroll
  for (int d = 8; d; d >>= 1) {
    const float o = __shfl_xor_sync(~0u, m, d);
    m = max3_abs_nan(m, o, o);
  }
  float mul;
  fp8_scale<FMT>(m, scale, mul);
  return fp8_encode8<FMT>(f, mul);
}

struct NArgs {
  const void* x;
  const void* weight;
  const void* bias;
  void* y;
  float* mean;
  float* rstd;
  uint8_t* codes;
  float* scales;
  int64_t rows, cols, pitch, lines;
  float eps;
  int32_t vec;
};

// One CTA per row, reading the row again for each pass (rows of any length).
template <typename XT, typename WT, bool LAYER, int FMT>
__global__ void __launch_bounds__(256) norm_rows(const NArgs a) {
  __shared__ float buf[N_MAX_WARPS];
  const int64_t r = blockIdx.x, cols = a.cols;
  const int64_t n_chunks = (cols + 7) / 8, n_pad = (n_chunks + 15) / 16 * 16;
  const XT* x = static_cast<const XT*>(a.x) + r * cols;
  const WT* w = static_cast<const WT*>(a.weight);
  const WT* b = static_cast<const WT*>(a.bias);
  const bool vec = a.vec != 0;
  const float inv_n = 1.0f / static_cast<float>(cols);
  float f[8], mean = 0.0f;
  if (LAYER) {
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < n_chunks; c += blockDim.x) {
      load8(x, 8 * c, cols, vec, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += f[j];
    }
    mean = cta_sum(s, buf) * inv_n;
  }
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < n_chunks; c += blockDim.x) {
    load8(x, 8 * c, cols, vec, f);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (8 * c + j < cols) s += (f[j] - mean) * (f[j] - mean);
  }
  const float rstd = 1.0f / sqrtf(cta_sum(s, buf) * inv_n + a.eps);
  if (threadIdx.x == 0) {
    if (LAYER && a.mean) a.mean[r] = mean;
    if (a.rstd) a.rstd[r] = rstd;
  }
  for (int64_t c = threadIdx.x; c < n_pad; c += blockDim.x) {
    float wf[8], bf[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = wf[j] = bf[j] = 0.0f;
    if (c < n_chunks) {
      load8(x, 8 * c, cols, vec, f);
      load8(w, 8 * c, cols, vec, wf);
      if (b) load8(b, 8 * c, cols, vec, bf);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = (f[j] - mean) * rstd * wf[j] + bf[j];
      if (!vec)
        for (int j = 0; j < 8; ++j)
          if (8 * c + j >= cols) f[j] = 0.0f;
      if (a.y) store8(static_cast<XT*>(a.y) + r * cols, 8 * c, cols, vec, f);
    }
    if constexpr (FMT >= 0) {
      float scale;
      const uint2 q = encode_block<FMT>(f, scale);
      if (8 * c < a.pitch)
        *reinterpret_cast<uint2*>(a.codes + r * a.pitch + 8 * c) = q;
      if ((c & 15) == 0) a.scales[(c >> 4) * a.lines + r] = scale;
    }
  }
}

// Scales of the padding lines: those of an all-zero block.
__global__ void norm_pad_scales(float* scales, int64_t rows, int64_t lines, int64_t kb) {
  const int64_t n = lines - rows;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n * kb;
       i += int64_t(gridDim.x) * blockDim.x)
    scales[(i / n) * lines + rows + i % n] = F_TINY;
}

struct NGrad {
  const void* dy;
  const void* x;
  const void* weight;
  const float* mean;
  const float* rstd;
  void* dx;
  float* dweight;
  float* dbias;
  float* part;        // [splits][2][cols] partial sums of dw and db
  int64_t rows, cols;
  int32_t splits;
  int32_t vec;
};

// dx of one row per CTA (rows of any length).
template <typename XT, typename WT, bool LAYER>
__global__ void __launch_bounds__(256) norm_grad_rows(const NGrad a) {
  __shared__ float buf[N_MAX_WARPS];
  const int64_t r = blockIdx.x, cols = a.cols, n_chunks = (cols + 7) / 8;
  const XT* x = static_cast<const XT*>(a.x) + r * cols;
  const XT* dy = static_cast<const XT*>(a.dy) + r * cols;
  const WT* w = static_cast<const WT*>(a.weight);
  const bool vec = a.vec != 0;
  const float mean = LAYER ? a.mean[r] : 0.0f, rstd = a.rstd[r];
  const float inv_n = 1.0f / static_cast<float>(cols);
  float f[8], g[8], wf[8], s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = threadIdx.x; c < n_chunks; c += blockDim.x) {
    load8(x, 8 * c, cols, vec, f);
    load8(dy, 8 * c, cols, vec, g);
    load8(w, 8 * c, cols, vec, wf);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = g[j] * wf[j];   // zero past the row's end
      s1 += t;
      s2 += t * ((f[j] - mean) * rstd);
    }
  }
  const float c1 = LAYER ? cta_sum(s1, buf) * inv_n : 0.0f;
  const float c2 = cta_sum(s2, buf) * inv_n;
  for (int64_t c = threadIdx.x; c < n_chunks; c += blockDim.x) {
    load8(x, 8 * c, cols, vec, f);
    load8(dy, 8 * c, cols, vec, g);
    load8(w, 8 * c, cols, vec, wf);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      f[j] = rstd * (g[j] * wf[j] - c1 - (f[j] - mean) * rstd * c2);
    store8(static_cast<XT*>(a.dx) + r * cols, 8 * c, cols, vec, f);
  }
}

// Partial sums of dw and db: a CTA takes 256 columns and every splits-th
// group of rows, one column per thread.
template <typename XT, bool LAYER>
__global__ void __launch_bounds__(256) norm_grad_cols(const NGrad a) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.cols) return;
  const XT* x = static_cast<const XT*>(a.x) + c;
  const XT* dy = static_cast<const XT*>(a.dy) + c;
  float dw = 0.0f, db = 0.0f;
  for (int64_t r = blockIdx.y; r < a.rows; r += a.splits) {
    const float g = static_cast<float>(dy[r * a.cols]);
    const float h = (static_cast<float>(x[r * a.cols]) - (LAYER ? a.mean[r] : 0.0f)) * a.rstd[r];
    dw += g * h;
    db += g;
  }
  float* p = a.part + int64_t(blockIdx.y) * 2 * a.cols;
  p[c] = dw;
  p[a.cols + c] = db;
}

// The partial sums of each column, in the order of the splits.
__global__ void __launch_bounds__(256) norm_grad_join(const float* part, int64_t cols, int splits,
                                                      float* dweight, float* dbias) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= cols) return;
  float dw = 0.0f, db = 0.0f;
  for (int s = 0; s < splits; ++s) {
    dw += part[int64_t(s) * 2 * cols + c];
    db += part[int64_t(s) * 2 * cols + cols + c];
  }
  dweight[c] = dw;
  if (dbias) dbias[c] = db;
}

int grad_splits(int64_t rows, int64_t cols) {
  const int64_t groups = (cols + 255) / 256;
  const int64_t want = std::max<int64_t>(1, 8 * 152 / groups);
  return static_cast<int>(std::min<int64_t>(std::min<int64_t>(rows, want), 512));
}

template <typename XT, typename WT, bool LAYER>
mxq_status run_forward(const NArgs& a, int fmt, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(a.rows);
  if (!a.codes) norm_rows<XT, WT, LAYER, -1><<<grid, 256, 0, st>>>(a);
  else if (fmt == MXQ_E4M3) norm_rows<XT, WT, LAYER, MXQ_E4M3><<<grid, 256, 0, st>>>(a);
  else norm_rows<XT, WT, LAYER, MXQ_E5M2><<<grid, 256, 0, st>>>(a);
  if (a.codes && a.lines > a.rows)
    norm_pad_scales<<<1, 256, 0, st>>>(a.scales, a.rows, a.lines, (a.cols + 127) / 128);
  return launch_status();
}

template <typename XT, typename WT, bool LAYER>
mxq_status run_backward(const NGrad& a, cudaStream_t st) {
  norm_grad_rows<XT, WT, LAYER><<<static_cast<unsigned>(a.rows), 256, 0, st>>>(a);
  const unsigned groups = static_cast<unsigned>((a.cols + 255) / 256);
  norm_grad_cols<XT, LAYER><<<dim3(groups, static_cast<unsigned>(a.splits)), 256, 0, st>>>(a);
  norm_grad_join<<<groups, 256, 0, st>>>(a.part, a.cols, a.splits, a.dweight, a.dbias);
  return launch_status();
}

// Calls f<XT, WT, LAYER>() for the run-time types.
template <typename F>
mxq_status dispatch(int x_dtype, int w_dtype, int kind, F f) {
  using B = __nv_bfloat16;
  const bool layer = kind == MXQ_NORM_LAYER;
  if (x_dtype == MXQ_OUT_BF16) {
    if (w_dtype == MXQ_OUT_BF16)
      return layer ? f.template operator()<B, B, true>() : f.template operator()<B, B, false>();
    return layer ? f.template operator()<B, float, true>()
                 : f.template operator()<B, float, false>();
  }
  if (w_dtype == MXQ_OUT_BF16)
    return layer ? f.template operator()<float, B, true>() : f.template operator()<float, B, false>();
  return layer ? f.template operator()<float, float, true>()
               : f.template operator()<float, float, false>();
}

struct Forward {
  const NArgs& a;
  int fmt;
  cudaStream_t st;
  template <typename XT, typename WT, bool LAYER>
  mxq_status operator()() const { return run_forward<XT, WT, LAYER>(a, fmt, st); }
};

struct Backward {
  const NGrad& a;
  cudaStream_t st;
  template <typename XT, typename WT, bool LAYER>
  mxq_status operator()() const { return run_backward<XT, WT, LAYER>(a, st); }
};

mxq_status check_common(int64_t rows, int64_t cols, int kind, int x_dtype, int w_dtype) {
  const int64_t lim = int64_t(1) << 31;
  if (rows < 0 || cols < 0 || rows >= lim || cols >= lim) return MXQ_ERR_ARG;
  if (kind != MXQ_NORM_LAYER && kind != MXQ_NORM_RMS) return MXQ_ERR_ARG;
  if ((x_dtype != MXQ_OUT_F32 && x_dtype != MXQ_OUT_BF16) ||
      (w_dtype != MXQ_OUT_F32 && w_dtype != MXQ_OUT_BF16))
    return MXQ_ERR_ARG;
  return MXQ_OK;
}

}  // namespace

uint32_t take_norm_error() {
  uint32_t h = 0;
  if (cudaMemcpyFromSymbol(&h, g_err_norm, sizeof(h)) != cudaSuccess) return MXQ_ERR_CUDA;
  if (h) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_err_norm, &z, sizeof(z));
  }
  return h;
}

}  // namespace mxq

using namespace mxq;

extern "C" mxq_status mxq_norm_forward(const mxq_norm_args* p, void* stream) {
  if (!p) return MXQ_ERR_ARG;
  const mxq_status st = check_common(p->rows, p->cols, p->kind, p->x_dtype, p->w_dtype);
  if (st != MXQ_OK) return st;
  if (!(p->eps >= 0.0f)) return MXQ_ERR_ARG;
  if (!p->codes != !p->scales || (p->codes && !is_fp8(p->fmt))) return MXQ_ERR_ARG;
  if (p->mean && p->kind != MXQ_NORM_LAYER) return MXQ_ERR_ARG;
  if (p->rows == 0 || p->cols == 0) return MXQ_OK;
  if (!p->x || !p->weight || (!p->y && !p->codes)) return MXQ_ERR_ARG;
  if (!aligned16(p->x) || !aligned16(p->weight) || !aligned16(p->bias) || !aligned16(p->y) ||
      !aligned16(p->codes) || !aligned16(p->scales))
    return MXQ_ERR_ALIGN;
  NArgs a = {};
  a.x = p->x;
  a.weight = p->weight;
  a.bias = p->bias;
  a.y = p->y;
  a.mean = p->mean;
  a.rstd = p->rstd;
  a.codes = static_cast<uint8_t*>(p->codes);
  a.scales = p->scales;
  a.rows = p->rows;
  a.cols = p->cols;
  a.pitch = fp8_pitch(p->cols);
  a.lines = fp8_lines(p->rows);
  a.eps = p->eps;
  a.vec = p->cols % 8 == 0;
  return dispatch(p->x_dtype, p->w_dtype, p->kind,
                  Forward{a, p->fmt, static_cast<cudaStream_t>(stream)});
}

extern "C" size_t mxq_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (check_common(rows, cols, MXQ_NORM_LAYER, MXQ_OUT_F32, MXQ_OUT_F32) != MXQ_OK) return 0;
  if (rows == 0 || cols == 0) return 0;
  return static_cast<size_t>(grad_splits(rows, cols)) * 2 * cols * sizeof(float);
}

extern "C" mxq_status mxq_norm_backward(const mxq_norm_grad_args* p, void* stream) {
  if (!p) return MXQ_ERR_ARG;
  mxq_status st = check_common(p->rows, p->cols, p->kind, p->x_dtype, p->w_dtype);
  if (st != MXQ_OK) return st;
  if (p->cols == 0) return MXQ_OK;
  if (!p->dweight) return MXQ_ERR_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->rows == 0) {
    const size_t bytes = static_cast<size_t>(p->cols) * sizeof(float);
    if (cudaMemsetAsync(p->dweight, 0, bytes, s) != cudaSuccess) return MXQ_ERR_CUDA;
    if (p->dbias && cudaMemsetAsync(p->dbias, 0, bytes, s) != cudaSuccess) return MXQ_ERR_CUDA;
    return MXQ_OK;
  }
  if (!p->dy || !p->x || !p->weight || !p->rstd || !p->dx || !p->workspace) return MXQ_ERR_ARG;
  if (p->kind == MXQ_NORM_LAYER && !p->mean) return MXQ_ERR_ARG;
  if (!aligned16(p->dy) || !aligned16(p->x) || !aligned16(p->weight) || !aligned16(p->dx))
    return MXQ_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(p->workspace) & 255u) != 0) return MXQ_ERR_ALIGN;
  if (p->workspace_bytes < mxq_norm_backward_workspace_size(p->rows, p->cols))
    return MXQ_ERR_WORKSPACE;
  NGrad a = {};
  a.dy = p->dy;
  a.x = p->x;
  a.weight = p->weight;
  a.mean = p->mean;
  a.rstd = p->rstd;
  a.dx = p->dx;
  a.dweight = p->dweight;
  a.dbias = p->dbias;
  a.part = static_cast<float*>(p->workspace);
  a.rows = p->rows;
  a.cols = p->cols;
  a.splits = grad_splits(p->rows, p->cols);
  a.vec = p->cols % 8 == 0;
  return dispatch(p->x_dtype, p->w_dtype, p->kind, Backward{a, s});
}
