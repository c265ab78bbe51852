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
//
// Bound by HBM; a row's reductions must not keep the loads waiting, hence the
// rings below.  Measured, 8192x4096 bf16: RMS forward 22 us (0.90 of the copy
// rate), layer norm forward 24.7 us (0.80), RMS to codes 24.2 us, layer norm
// backward 38.9 us with the join of the column sums (0.76).  Rows that start
// between 16-byte boundaries come through the same rings in the aligned words
// around them: 8001x4097 bf16, fp32 weight, layer norm forward 51.6 us (element by
// element 146), to codes 56.8 (111), backward 95 (222).
#include "norm_common.cuh"

namespace mxq {

__device__ uint32_t g_err_norm;

namespace {

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
  int32_t center;     // LAYER kernels: 0 for an RMS norm with a bias, whose mean is taken as 0
  int32_t vec;
  int32_t slots;      // norm_ring: rows in flight
  uint64_t timeout_ns;
};

// The scale of block kb of row r; the last row also writes those of the
// padding lines (an all-zero block's).
MXQ_DEV void store_scale(const NArgs& a, int64_t kb, int64_t r, float scale) {
  if (!MXQ_IN_BOUNDS(kb * F_BLOCK < a.cols && r < a.rows, &g_err_norm, SITE_B_NORM)) return;
  float* s = a.scales + kb * a.lines;
  s[r] = scale;
  if (r == a.rows - 1)
    for (int64_t l = a.rows; l < a.lines; ++l) s[l] = F_TINY;
}

// Codes and scales of the I chunks of eight values that a lane holds of row r,
// chunk i at column c0 + i * step (a multiple of 128): 16 neighbouring lanes
// share a block.  The two divisions of a block's scale cost as much as the rest
// of its codes, so of the I blocks each lane works out one.
template <int FMT, int I>
MXQ_DEV void encode_chunks(const NArgs& a, int64_t r, int64_t c0, int64_t step,
                           const float (&f)[I][8]) {
  const int lane = threadIdx.x & 31, which = lane & (I - 1);
  float own = 0.0f;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    float m = fabsf(f[i][0]);
#pragma unroll
    for (int j = 1; j < 7; j += 2) m = max3_abs_nan(m, f[i][j], f[i][j + 1]);
    m = max3_abs_nan(m, f[i][7], f[i][7]);
#pragma unroll
    for (int d = 8; d; d >>= 1) {
      const float o = __shfl_xor_sync(~0u, m, d);
      m = max3_abs_nan(m, o, o);
    }
    if (i == which) own = m;
  }
  float scale, mul;
  fp8_scale<FMT>(own, scale, mul);
  const int64_t block = (c0 + which * step) >> 7;
  if ((lane & 15) < I && block * 128 < a.cols) store_scale(a, block, r, scale);
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const float k = __shfl_sync(~0u, mul, (lane & 16) + i);
    const int64_t c = c0 + i * step;
    const uint2 q = fp8_encode8<FMT>(f[i], k);
    if (c < a.pitch && MXQ_IN_BOUNDS(c + 8 <= a.pitch, &g_err_norm, SITE_B_NORM))
      *reinterpret_cast<uint2*>(a.codes + r * a.pitch + c) = q;
  }
}

// One CTA per row, reading the row again for each pass (rows of any length).
template <typename XT, typename WT, bool LAYER, int FMT>
__global__ void __launch_bounds__(256) norm_rows(const NArgs a) {
  __shared__ float buf[N_MAX_WARPS];
  const int64_t r = blockIdx.x, cols = a.cols;
  const int64_t n_chunks = (cols + 7) / 8;
  griddep_wait();
  griddep_launch_dependents();
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
    mean = a.center ? cta_sum(s, buf) * inv_n : 0.0f;
  }
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < n_chunks; c += blockDim.x) {
    load8(x, 8 * c, cols, vec, f);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (8 * c + j < cols) s += (f[j] - mean) * (f[j] - mean);
  }
  const float rstd = 1.0f / sqrtf(cta_sum(s, buf) * inv_n + a.eps);
  if (threadIdx.x == 0 && MXQ_IN_BOUNDS(r < a.rows, &g_err_norm, SITE_B_NORM)) {
    if (LAYER && a.mean) a.mean[r] = mean;
    if (a.rstd) a.rstd[r] = rstd;
  }
  const int64_t n_all = (n_chunks + 31) / 32 * 32;   // whole warps
  for (int64_t c = threadIdx.x; c < n_all; c += blockDim.x) {
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
      if (a.y && MXQ_IN_BOUNDS(r < a.rows && 8 * c < cols, &g_err_norm, SITE_B_NORM))
        store8(static_cast<XT*>(a.y) + r * cols, 8 * c, cols, vec, f);
    }
    if constexpr (FMT >= 0) {
      float chunk[1][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) chunk[0][j] = f[j];
      encode_chunks<FMT, 1>(a, r, 8 * c, 0, chunk);
    }
  }
}

// Rows of at most 8 I elements per thread, read once and kept in registers:
// a warp per row (WARP, eight rows a CTA) or a CTA per row.
//
// Bound by HBM.  A row's reductions are two round trips through shared memory
// (RMS one), hidden by the other rows resident on the SM; weight and bias are
// loaded before them.
template <typename XT, typename WT, bool LAYER, int FMT, bool WARP, int I, bool VEC>
__global__ void __launch_bounds__(WARP ? 256 : 512) norm_regs(const NArgs a) {
  __shared__ float buf[WARP ? 1 : 2 * N_MAX_WARPS];
  const int cols = static_cast<int>(a.cols);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = WARP ? int64_t(blockIdx.x) * 8 + warp : blockIdx.x;
  const int t = WARP ? lane : threadIdx.x, nt = WARP ? 32 : blockDim.x;
  griddep_wait();
  griddep_launch_dependents();
  if (r >= a.rows) return;   // whole warps, and only where a warp has its own row
  Raw8<XT> raw[I];
  Raw8<WT> w[I], b[I];
  {
    const XT* x = static_cast<const XT*>(a.x);
    const int64_t start = r * a.cols, n = a.rows * a.cols;
    Chunk<XT, VEC> in[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (t + i * nt);
      in[i].load(x, start + c, n, c, cols);
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      load_param<VEC>(w[i], a.weight, 8 * (t + i * nt), cols);
      if (LAYER && a.bias) load_param<VEC>(b[i], a.bias, 8 * (t + i * nt), cols);
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (t + i * nt);
      raw[i] = in[i].get(x, start + c, n, c, cols);
    }
  }
  // Sum over the row; `part` numbers the reduction, each with its own buffer.
  auto row_sum = [&](float v, int part) {
    v = warp_sum(v);
    if constexpr (WARP) return v;
    const int nw = nt >> 5;
    float* mine = buf + (WARP ? 0 : part * N_MAX_WARPS);
    if (lane == 0) mine[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? mine[lane] : 0.0f);
  };
  const float inv_n = 1.0f / static_cast<float>(cols);
  float mean = 0.0f, s = 0.0f;
  if constexpr (LAYER) {
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += raw[i][j];   // zero past the row's end
    mean = row_sum(s, 0) * inv_n;
    if (!a.center) mean = 0.0f;
    s = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int n = cols - 8 * (t + i * nt);   // elements of this chunk inside the row
    if (n >= 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s += (raw[i][j] - mean) * (raw[i][j] - mean);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) s += (raw[i][j] - mean) * (raw[i][j] - mean);
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum(s, 1) * inv_n + a.eps);
  if (t == 0 && MXQ_IN_BOUNDS(r < a.rows, &g_err_norm, SITE_B_NORM)) {
    if (LAYER && a.mean) a.mean[r] = mean;
    if (a.rstd) a.rstd[r] = rstd;
  }
  float f[I][8];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = 8 * (t + i * nt);
    // weight and bias are zero past the row's end, and so is f
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[i][j] = (raw[i][j] - mean) * rstd * w[i][j];
      if (LAYER && a.bias) f[i][j] += b[i][j];
    }
    if (a.y && c < cols && MXQ_IN_BOUNDS(r < a.rows, &g_err_norm, SITE_B_NORM))
      store8(static_cast<XT*>(a.y) + r * a.cols, c, cols, VEC, f[i]);
  }
  if constexpr (FMT >= 0) encode_chunks<FMT, I>(a, r, 8 * t, 8 * nt, f);
}

// The same for many rows: persistent CTAs keep
// their columns' weight and bias in registers, and the rows come through a
// ring in shared memory, filled by bulk copies a.slots rows ahead.  With a CTA
// for every row, loads fill a third of its life and the memory waits for the
// rest (8192x4096 bf16, layer norm: 34.6 us against 24.7).
template <typename XT, typename WT, bool LAYER, int FMT, int I, bool VEC>
__global__ void __launch_bounds__(512) norm_ring(const NArgs a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[N_MAX_SLOTS];
  __shared__ float buf[2][2][16];
  const int cols = static_cast<int>(a.cols), nt = blockDim.x, t = threadIdx.x;
  const int lane = t & 31, warp = t >> 5;
  const float inv_n = 1.0f / static_cast<float>(cols);
  const uint32_t row_bytes = static_cast<uint32_t>(ring_row_bytes(cols, sizeof(XT)));
  const XT* const all = static_cast<const XT*>(a.x);
  const int64_t n = a.rows * a.cols;
  const int slots = a.slots;
  if (t == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(smem_u32(&full[i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  auto fetch = [&](int64_t r, int slot) {   // one thread
    if (r >= a.rows) return;
    const uint32_t bar = smem_u32(&full[slot]);
    const RowCopy<XT, VEC> c(all, r, a.rows, a.cols);
    if (!MXQ_IN_BOUNDS(slot < slots && c.inside(all, n) && c.bytes <= row_bytes, &g_err_norm,
                       SITE_B_NORM))
      return;
    mbar_arrive_expect_tx(bar, c.bytes);
    bulk_load(smem_u32(ring) + slot * row_bytes, c.src, c.bytes, bar);
  };
  if (t == 0)
    for (int i = 0; i < slots; ++i) fetch(blockIdx.x + int64_t(i) * gridDim.x, i);
  Raw8<WT> w[I], b[I];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    load_param<VEC>(w[i], a.weight, 8 * (t + i * nt), cols);
    if (LAYER && a.bias) load_param<VEC>(b[i], a.bias, 8 * (t + i * nt), cols);
  }
  int slot = 0, phase = 0, parity = 0;
  bool ok = true;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, parity ^= 1) {
    if (ok && !mbar_wait(smem_u32(&full[slot]), phase, a.timeout_ns)) {
      record_error(&g_err_norm, MXQ_ERR_TIMEOUT, SITE_NORM_FULL);
      ok = false;   // the results are void; no further wait
    }
    const XT* x = reinterpret_cast<const XT*>(ring + slot * row_bytes);
    Raw8<XT> raw[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (t + i * nt);
      Chunk<XT, VEC> in;
      in.load_ring(x, r * a.cols + c, n, c, cols);
      raw[i] = in.get(all, r * a.cols + c, n, c, cols);
    }
    // Sum over the row.  Each of a row's sums has its own buffer, and rows take
    // them in turn: a warp writes row k + 2's after a barrier of row k + 1,
    // which every warp reached after reading row k's.
    auto row_sum = [&](float v, int part) {
      v = warp_sum(v);
      if (lane == 0) buf[parity][part][warp] = v;
      __syncthreads();
      v = (lane & 15) < (nt >> 5) ? buf[parity][part][lane & 15] : 0.0f;
#pragma unroll
      for (int d = 8; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
      return v;
    };
    float mean = 0.0f, s = 0.0f;
    if constexpr (LAYER) {
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += raw[i][j];   // zero past the row's end
      mean = row_sum(s, 0) * inv_n;
      if (!a.center) mean = 0.0f;
      s = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int inside = cols - 8 * (t + i * nt);
      if (inside <= 0) break;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (VEC || j < inside) s += (raw[i][j] - mean) * (raw[i][j] - mean);
    }
    const float rstd = 1.0f / sqrtf(row_sum(s, 1) * inv_n + a.eps);
    // past a barrier: every thread has read the slot
    if (t == 0) {
      fetch(r + int64_t(slots) * gridDim.x, slot);
      if (LAYER && a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    if (++slot == slots) { slot = 0; phase ^= 1; }
    float f[I][8];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (t + i * nt);
      // weight and bias are zero past the row's end, and so is f
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[i][j] = (raw[i][j] - mean) * rstd * w[i][j];
        if (LAYER && a.bias) f[i][j] += b[i][j];
      }
      if (a.y && c < cols && MXQ_IN_BOUNDS(r < a.rows, &g_err_norm, SITE_B_NORM))
        store8(static_cast<XT*>(a.y) + r * a.cols, c, cols, VEC, f[i]);
    }
    if constexpr (FMT >= 0) encode_chunks<FMT, I>(a, r, 8 * t, 8 * nt, f);
  }
  if (!ok && t == 0) drain_ring(full, slots, a.rows, a.timeout_ns);
}

// Forward.  Up to 1024 columns a warp holds a row (no barrier).  Longer rows
// take a CTA: with few rows, one chunk a thread (latency: a row spread over
// more threads); with many, two, which halves the warps of each reduction.
RowPlan forward_plan(int64_t rows, int64_t cols) {
  const int64_t chunks = (cols + 7) / 8;
  if (chunks <= 128) return {true, 256, chunks <= 32 ? 1 : chunks <= 64 ? 2 : 4};
  const int least = rows >= 4 * sm_count() ? 2 : 1;
  for (int i = least; i <= 4; i *= 2)
    if (chunks <= 512 * i)
      return {false, static_cast<int>(((chunks + i - 1) / i + 31) / 32 * 32), i};
  return {false, 256, 0};
}

// Persistent CTAs for norm_ring: four chunks a thread, 512 threads an SM.  Two
// chunks and 1024 threads leave twice the reductions per element (8192x4096
// bf16, layer norm 30.6 us against 24.7, RMS to codes 31.1 against 24.2).  Rows
// of up to 1024 columns, a warp each either way, gain from the ring but for RMS
// norm to codes (32768x1024: layer norm 33.6 us without, 26.5 with it, to codes
// 36.8 and 32.6; RMS to codes 21.8 and 25.6).
constexpr int N_RING_I = 4;
struct RingPlan {
  int nt, ctas, slots;   // slots == 0: not for these rows
};

RingPlan forward_ring(int64_t rows, int64_t cols, int64_t size, bool rms_codes) {
  const int64_t chunks = (cols + 7) / 8;
  RingPlan p = {0, 0, 0};
  if (chunks <= (rms_codes ? 128 : 64) || chunks > 512 * N_RING_I) return p;
  p.nt = static_cast<int>(((chunks + N_RING_I - 1) / N_RING_I + 31) / 32 * 32);
  const int per_sm = std::max(1, 512 / p.nt);
  p.ctas = per_sm * sm_count();
  const int64_t fit = (200 * 1024 / per_sm) / ring_row_bytes(cols, size);
  if (rows >= 2 * p.ctas && fit >= 2)
    p.slots = static_cast<int>(std::min<int64_t>(fit, N_MAX_SLOTS));
  return p;
}

template <typename XT, typename WT, bool LAYER, int FMT, bool VEC>
mxq_status launch_forward(NArgs a, cudaStream_t st) {
  const RingPlan ring = forward_ring(a.rows, a.cols, sizeof(XT), !LAYER && FMT >= 0);
  bool ok;
  if (ring.slots) {
    a.slots = ring.slots;
    a.timeout_ns = wait_timeout_ns();
    const auto kernel = norm_ring<XT, WT, LAYER, FMT, N_RING_I, VEC>;
    const size_t smem = size_t(ring.slots) * ring_row_bytes(a.cols, sizeof(XT));
    ok = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem)) &&
         launch_early(kernel, static_cast<unsigned>(ring.ctas), ring.nt, smem, st, a);
    return ok ? launch_status() : MXQ_ERR_CUDA;
  }
  const RowPlan p = forward_plan(a.rows, a.cols);
  const unsigned rows = static_cast<unsigned>(a.rows), groups = (rows + 7) / 8;
  if (p.warp) {
    ok = p.i == 1 ? launch_early(norm_regs<XT, WT, LAYER, FMT, true, 1, VEC>, groups, 256, 0, st, a)
       : p.i == 2 ? launch_early(norm_regs<XT, WT, LAYER, FMT, true, 2, VEC>, groups, 256, 0, st, a)
                  : launch_early(norm_regs<XT, WT, LAYER, FMT, true, 4, VEC>, groups, 256, 0, st, a);
  } else {
    ok = p.i == 1 ? launch_early(norm_regs<XT, WT, LAYER, FMT, false, 1, VEC>, rows, p.nt, 0, st, a)
       : p.i == 2 ? launch_early(norm_regs<XT, WT, LAYER, FMT, false, 2, VEC>, rows, p.nt, 0, st, a)
       : p.i == 4 ? launch_early(norm_regs<XT, WT, LAYER, FMT, false, 4, VEC>, rows, p.nt, 0, st, a)
                  : launch_early(norm_rows<XT, WT, LAYER, FMT>, rows, 256, 0, st, a);
  }
  return ok ? launch_status() : MXQ_ERR_CUDA;
}

template <typename XT, typename WT, bool LAYER>
mxq_status run_forward(const NArgs& a, int fmt, cudaStream_t st) {
  if (!a.codes)
    return a.vec ? launch_forward<XT, WT, LAYER, -1, true>(a, st)
                 : launch_forward<XT, WT, LAYER, -1, false>(a, st);
  if (fmt == MXQ_E4M3)
    return a.vec ? launch_forward<XT, WT, LAYER, MXQ_E4M3, true>(a, st)
                 : launch_forward<XT, WT, LAYER, MXQ_E4M3, false>(a, st);
  return a.vec ? launch_forward<XT, WT, LAYER, MXQ_E5M2, true>(a, st)
               : launch_forward<XT, WT, LAYER, MXQ_E5M2, false>(a, st);
}

struct Forward {
  const NArgs& a;
  int fmt;
  cudaStream_t st;
  template <typename XT, typename WT, bool LAYER>
  mxq_status operator()() const { return run_forward<XT, WT, LAYER>(a, fmt, st); }
};

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
  const mxq_status st = norm_check(p->rows, p->cols, p->kind, p->x_dtype, p->w_dtype);
  if (st != MXQ_OK) return st;
  if (!(p->eps >= 0.0f)) return MXQ_ERR_ARG;
  if (!p->codes != !p->scales || (p->codes && !is_fp8(p->fmt))) return MXQ_ERR_ARG;
  if (p->mean && p->kind != MXQ_NORM_LAYER) return MXQ_ERR_ARG;
  if (p->rows == 0 || p->cols == 0) return MXQ_OK;
  if (!p->x || !p->weight || (!p->y && !p->codes)) return MXQ_ERR_ARG;
  if (!aligned16(p->x) || !aligned16(p->weight) || !aligned16(p->bias) || !aligned16(p->y) ||
      !aligned16(p->codes) || !aligned16(p->scales) || !aligned4(p->mean) || !aligned4(p->rstd))
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
  // The kernels without a mean hold no bias in registers: an RMS norm with one
  // runs those of the layer norm.
  a.center = p->kind == MXQ_NORM_LAYER;
  const int kind = p->bias ? MXQ_NORM_LAYER : p->kind;
  return dispatch(p->x_dtype, p->w_dtype, kind,
                  Forward{a, p->fmt, static_cast<cudaStream_t>(stream)});
}
