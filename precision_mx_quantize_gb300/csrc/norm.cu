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
// backward 38.9 us with the join of the column sums (0.76).
#include <type_traits>

#include "fp8_common.cuh"
#include "mxq_host.h"

namespace mxq {

__device__ uint32_t g_err_norm;

namespace {

constexpr int N_MAX_WARPS = 32;
constexpr int N_MAX_SLOTS = 8;

// Eight consecutive elements of a row from `col` on, zero past its end.  vec:
// the row's start is 16-byte aligned and cols % 8 == 0.
template <typename Ix>
MXQ_DEV void load8(const __nv_bfloat16* row, Ix col, Ix cols, bool vec, float (&f)[8]) {
  if (vec) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + col);
    f[0] = bf16lo(w.x); f[1] = bf16hi(w.x); f[2] = bf16lo(w.y); f[3] = bf16hi(w.y);
    f[4] = bf16lo(w.z); f[5] = bf16hi(w.z); f[6] = bf16lo(w.w); f[7] = bf16hi(w.w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = col + j < cols ? __bfloat162float(row[col + j]) : 0.0f;
  }
}

template <typename Ix>
MXQ_DEV void load8(const float* row, Ix col, Ix cols, bool vec, float (&f)[8]) {
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

template <typename Ix>
MXQ_DEV void store8(__nv_bfloat16* row, Ix col, Ix cols, bool vec, const float (&f)[8]) {
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

template <typename Ix>
MXQ_DEV void store8(float* row, Ix col, Ix cols, bool vec, const float (&f)[8]) {
  if (vec) {
    *reinterpret_cast<float4*>(row + col) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(row + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < cols) row[col + j] = f[j];
  }
}

// Eight elements of a row as they lie in memory.
template <typename XT>
struct Raw8;

template <>
struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  MXQ_DEV void load(const __nv_bfloat16* row, int col, int cols, bool vec) {
    w[0] = w[1] = w[2] = w[3] = 0u;
    if (col >= cols) return;
    if (vec) {
      const uint4 t = *reinterpret_cast<const uint4*>(row + col);
      w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(row + col);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < cols) w[j >> 1] |= static_cast<uint32_t>(q[j]) << (16 * (j & 1));
    }
  }
  MXQ_DEV float operator[](int j) const { return j & 1 ? bf16hi(w[j >> 1]) : bf16lo(w[j >> 1]); }
};

template <>
struct Raw8<float> {
  float f[8];
  MXQ_DEV void load(const float* row, int col, int cols, bool vec) {
    if (col < cols) {
      load8(row, col, cols, vec, f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    }
  }
  MXQ_DEV float operator[](int j) const { return f[j]; }
};

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

// After a wait ran out: waits (bounded) until the copies of a ring that serves
// every grid-th row have landed, so that shared memory can be released.
MXQ_DEV void drain_ring(uint64_t* full, int slots, int64_t rows, uint64_t limit_ns) {
  const int64_t fetched = (rows - blockIdx.x + gridDim.x - 1) / gridDim.x;
  const uint64_t t0 = global_ns();
  for (int i = 0; i < slots && i < fetched; ++i) {
    const int64_t last = (fetched - 1 - i) / slots;   // the slot's last phase
    while (!mbar_try_wait(smem_u32(&full[i]), last & 1) && global_ns() - t0 < limit_ns) {
    }
  }
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
  int32_t slots;      // norm_ring: rows in flight
  uint64_t timeout_ns;
};

// The scale of block kb of row r; the last row also writes those of the
// padding lines (an all-zero block's).
MXQ_DEV void store_scale(const NArgs& a, int64_t kb, int64_t r, float scale) {
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
      if (a.y) store8(static_cast<XT*>(a.y) + r * cols, 8 * c, cols, vec, f);
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
template <typename XT, typename WT, bool LAYER, int FMT, bool WARP, int I>
__global__ void __launch_bounds__(WARP ? 256 : 512) norm_regs(const NArgs a) {
  __shared__ float buf[WARP ? 1 : 2 * N_MAX_WARPS];
  const int cols = static_cast<int>(a.cols);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = WARP ? int64_t(blockIdx.x) * 8 + warp : blockIdx.x;
  const int t = WARP ? lane : threadIdx.x, nt = WARP ? 32 : blockDim.x;
  const bool vec = a.vec != 0;
  griddep_wait();
  griddep_launch_dependents();
  if (r >= a.rows) return;   // whole warps, and only where a warp has its own row
  const XT* x = static_cast<const XT*>(a.x) + r * a.cols;
  Raw8<XT> raw[I];
  Raw8<WT> w[I], b[I];
#pragma unroll
  for (int i = 0; i < I; ++i) raw[i].load(x, 8 * (t + i * nt), cols, vec);
#pragma unroll
  for (int i = 0; i < I; ++i) {
    w[i].load(static_cast<const WT*>(a.weight), 8 * (t + i * nt), cols, vec);
    if (LAYER && a.bias) b[i].load(static_cast<const WT*>(a.bias), 8 * (t + i * nt), cols, vec);
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
  if (t == 0) {
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
      store8(static_cast<XT*>(a.y) + r * a.cols, c, cols, vec, f[i]);
  }
  if constexpr (FMT >= 0) encode_chunks<FMT, I>(a, r, 8 * t, 8 * nt, f);
}

// The same for many rows whose starts are 16-byte aligned: persistent CTAs keep
// their columns' weight and bias in registers, and the rows come through a
// ring in shared memory, filled by bulk copies a.slots rows ahead.  With a CTA
// for every row, loads fill a third of its life and the memory waits for the
// rest (8192x4096 bf16, layer norm: 34.6 us against 24.7).
template <typename XT, typename WT, bool LAYER, int FMT, int I>
__global__ void __launch_bounds__(512) norm_ring(const NArgs a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[N_MAX_SLOTS];
  __shared__ float buf[2][2][16];
  const int cols = static_cast<int>(a.cols), nt = blockDim.x, t = threadIdx.x;
  const int lane = t & 31, warp = t >> 5;
  const float inv_n = 1.0f / static_cast<float>(cols);
  const uint32_t row_bytes = cols * sizeof(XT);
  const int slots = a.slots;
  if (t == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(smem_u32(&full[i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  auto fetch = [&](int64_t r, int slot) {   // one thread
    if (r >= a.rows || !MXQ_IN_BOUNDS(slot < slots, &g_err_norm, SITE_B_NORM)) return;
    const uint32_t bar = smem_u32(&full[slot]);
    mbar_arrive_expect_tx(bar, row_bytes);
    bulk_load(smem_u32(ring) + slot * row_bytes, static_cast<const XT*>(a.x) + r * a.cols,
              row_bytes, bar);
  };
  if (t == 0)
    for (int i = 0; i < slots; ++i) fetch(blockIdx.x + int64_t(i) * gridDim.x, i);
  Raw8<WT> w[I], b[I];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    w[i].load(static_cast<const WT*>(a.weight), 8 * (t + i * nt), cols, true);
    if (LAYER && a.bias) b[i].load(static_cast<const WT*>(a.bias), 8 * (t + i * nt), cols, true);
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
    for (int i = 0; i < I; ++i) raw[i].load(x, 8 * (t + i * nt), cols, true);
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
      s = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      if (8 * (t + i * nt) >= cols) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += (raw[i][j] - mean) * (raw[i][j] - mean);
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
        store8(static_cast<XT*>(a.y) + r * a.cols, c, cols, true, f[i]);
    }
    if constexpr (FMT >= 0) encode_chunks<FMT, I>(a, r, 8 * t, 8 * nt, f);
  }
  if (!ok && t == 0) drain_ring(full, slots, a.rows, a.timeout_ns);
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
  int32_t slots;      // norm_grad_ring: rows in flight
  uint64_t timeout_ns;
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

// Backward for rows of at most 8 I elements per thread: a warp per row (WARP)
// or a CTA per row, over every grid-th row.  A thread keeps its columns' sums
// of dw and db in registers for all its rows, so x and dy are read once; the
// next row's are loaded under this row's reduction.  The CTA's sums go to
// `part`, which norm_grad_join adds up in order.
template <typename XT, typename WT, bool LAYER, bool WARP, int I>
__global__ void __launch_bounds__(WARP ? 256 : 512) norm_grad_regs(const NGrad a) {
  extern __shared__ float sums[];          // WARP: [8][8 I 32] for the final join
  __shared__ float2 buf[WARP ? 1 : 2 * N_MAX_WARPS];
  const int cols = static_cast<int>(a.cols);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = WARP ? lane : threadIdx.x, nt = WARP ? 32 : blockDim.x;
  const int64_t first = WARP ? int64_t(blockIdx.x) * 8 + warp : blockIdx.x;
  const int64_t step = WARP ? int64_t(gridDim.x) * 8 : gridDim.x;
  const bool vec = a.vec != 0;
  const float inv_n = 1.0f / static_cast<float>(cols);
  griddep_wait();
  griddep_launch_dependents();
  float dw[I][8], db[I][8];
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.0f;
  Raw8<WT> w[I];
#pragma unroll
  for (int i = 0; i < I; ++i) w[i].load(static_cast<const WT*>(a.weight), 8 * (t + i * nt), cols, vec);
  Raw8<XT> x[I], dy[I];
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t r) {
    if (r >= a.rows) return;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      x[i].load(static_cast<const XT*>(a.x) + r * a.cols, 8 * (t + i * nt), cols, vec);
      dy[i].load(static_cast<const XT*>(a.dy) + r * a.cols, 8 * (t + i * nt), cols, vec);
    }
    mean = LAYER ? a.mean[r] : 0.0f;
    rstd = a.rstd[r];
  };
  load(first);
  int phase = 0;
  for (int64_t r = first; r < a.rows; r += step, phase ^= 1) {
    float s1 = 0.0f, s2 = 0.0f;
    float h[I][8], g[I][8];
    const float m = mean, rs = rstd;
#pragma unroll
    for (int i = 0; i < I; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = dy[i][j];               // zero past the row's end
        h[i][j] = (x[i][j] - m) * rs;
        dw[i][j] += d * h[i][j];
        db[i][j] += d;
        g[i][j] = d * w[i][j];
        s1 += g[i][j];
        s2 += g[i][j] * h[i][j];
      }
    }
    load(r + step);
    s2 = warp_sum(s2);
    if (LAYER) s1 = warp_sum(s1);
    if constexpr (!WARP) {
      // two buffers, one barrier a row: a warp writes row k + 2's sums after
      // barrier k + 1, which every warp reached after reading row k's
      float2* mine = buf + phase * N_MAX_WARPS;
      if (lane == 0) mine[warp] = make_float2(s1, s2);
      __syncthreads();
      const float2 v = lane < (nt >> 5) ? mine[lane] : make_float2(0.0f, 0.0f);
      s2 = warp_sum(v.y);
      if (LAYER) s1 = warp_sum(v.x);
    }
    const float c1 = LAYER ? s1 * inv_n : 0.0f, c2 = s2 * inv_n;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (t + i * nt);
      if (c >= cols) break;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = rs * (g[i][j] - c1 - h[i][j] * c2);
      if (MXQ_IN_BOUNDS(r < a.rows, &g_err_norm, SITE_B_NORM_GRAD))
        store8(static_cast<XT*>(a.dx) + r * a.cols, c, cols, vec, f);
    }
  }
  float* part = a.part + int64_t(blockIdx.x) * 2 * a.cols;
  if constexpr (WARP) {
    // the eight warps' sums, in order
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 1 && !LAYER) break;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sums[(warp * 8 * I + 8 * i + j) * 32 + lane] = k ? db[i][j] : dw[i][j];
      __syncthreads();
      for (int e = threadIdx.x; e < 8 * I * 32; e += 256) {
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v += sums[q * 8 * I * 32 + e];
        // element e: lane e % 32, chunk and place e / 32
        const int c = 8 * ((e & 31) + (e >> 8) * 32) + ((e >> 5) & 7);
        if (c < cols) part[k * cols + c] = v;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (t + i * nt);
      if (c >= cols) break;
      store8(part, c, cols, cols % 4 == 0 && vec, dw[i]);
      if (LAYER) store8(part + cols, c, cols, cols % 4 == 0 && vec, db[i]);
    }
  }
}

// The same for rows that a CTA shares and whose starts are 16-byte aligned: the
// rows come through a ring of a.slots pairs (x, dy) in shared memory, filled by
// bulk copies a.slots rows ahead.  One row ahead in registers left each row
// waiting for its loads (8192x4096 bf16, both kernels: 48 us against 39).
template <typename XT, typename WT, bool LAYER, int I>
__global__ void __launch_bounds__(512) norm_grad_ring(const NGrad a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[N_MAX_SLOTS];
  __shared__ float buf[2][2][16];
  const int cols = static_cast<int>(a.cols), nt = blockDim.x, t = threadIdx.x;
  const int lane = t & 31, warp = t >> 5;
  const float inv_n = 1.0f / static_cast<float>(cols);
  const uint32_t row_bytes = cols * sizeof(XT), slot_bytes = 2 * row_bytes;
  const int slots = a.slots;
  if (t == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(smem_u32(&full[i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  auto fetch = [&](int64_t r, int slot) {   // one thread
    if (r >= a.rows || !MXQ_IN_BOUNDS(slot < slots, &g_err_norm, SITE_B_NORM_GRAD)) return;
    const uint32_t bar = smem_u32(&full[slot]), dst = smem_u32(ring) + slot * slot_bytes;
    mbar_arrive_expect_tx(bar, slot_bytes);
    bulk_load(dst, static_cast<const XT*>(a.x) + r * a.cols, row_bytes, bar);
    bulk_load(dst + row_bytes, static_cast<const XT*>(a.dy) + r * a.cols, row_bytes, bar);
  };
  if (t == 0)
    for (int i = 0; i < slots; ++i) fetch(blockIdx.x + int64_t(i) * gridDim.x, i);
  // With four chunks a thread the sums of db do not fit the registers: they
  // stay in shared memory, behind the ring, eight floats a thread and chunk as
  // two planes of float4 (4096x14336 bf16: 146 us spilled, 82 so).
  constexpr bool DB_SHARED = LAYER && I == 4;
  float4* db_at = reinterpret_cast<float4*>(ring + slots * slot_bytes) + t;
  float dw[I][8], db[DB_SHARED ? 1 : I][8];
#pragma unroll
  for (int i = 0; i < I; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    if constexpr (DB_SHARED) {
      db_at[2 * i * nt] = db_at[(2 * i + 1) * nt] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) db[i][j] = 0.0f;
    }
  }
  // The weight stays in registers where there is room, else comes from L1.
  constexpr bool KEEP = I <= 2;
  Raw8<WT> kept[KEEP ? I : 1];
  auto weight = [&](int i) {
    Raw8<WT> w;
    w.load(static_cast<const WT*>(a.weight), 8 * (t + i * nt), cols, true);
    return w;
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < I; ++i) kept[i] = weight(i);
  }
  int slot = 0, phase = 0, parity = 0;
  bool ok = true;
  float next_m = LAYER ? a.mean[blockIdx.x] : 0.0f, next_rs = a.rstd[blockIdx.x];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, parity ^= 1) {
    const float m = next_m, rs = next_rs;
    if (r + gridDim.x < a.rows) {   // a row ahead: the load takes as long as a row
      if (LAYER) next_m = a.mean[r + gridDim.x];
      next_rs = a.rstd[r + gridDim.x];
    }
    if (ok && !mbar_wait(smem_u32(&full[slot]), phase, a.timeout_ns)) {
      record_error(&g_err_norm, MXQ_ERR_TIMEOUT, SITE_NORM_FULL);
      ok = false;   // the results are void; no further wait
    }
    const XT* x = reinterpret_cast<const XT*>(ring + slot * slot_bytes);
    const XT* dy = x + cols;
    float s1 = 0.0f, s2 = 0.0f;
    // x and dy are kept as they lie in memory: two operations more per element
    // below, but bf16 rows then take half the registers
    Raw8<XT> xr[I], dr[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      xr[i].load(x, 8 * (t + i * nt), cols, true);
      dr[i].load(dy, 8 * (t + i * nt), cols, true);
      const Raw8<WT> w = KEEP ? kept[KEEP ? i : 0] : weight(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = dr[i][j], h = (xr[i][j] - m) * rs, g = d * w[j];   // zero past the end
        dw[i][j] += d * h;
        if constexpr (!DB_SHARED) db[i][j] += d;
        s1 += g;
        s2 += g * h;
      }
      if constexpr (DB_SHARED) {
        float4 lo = db_at[2 * i * nt], hi = db_at[(2 * i + 1) * nt];
        lo.x += dr[i][0]; lo.y += dr[i][1]; lo.z += dr[i][2]; lo.w += dr[i][3];
        hi.x += dr[i][4]; hi.y += dr[i][5]; hi.z += dr[i][6]; hi.w += dr[i][7];
        db_at[2 * i * nt] = lo;
        db_at[(2 * i + 1) * nt] = hi;
      }
    }
    // Both sums at once: lanes 0-15 of a warp take s1, lanes 16-31 s2.  Two
    // buffers, one barrier a row: a warp writes row k + 2's sums after barrier
    // k + 1, which every warp reached after reading row k's.
    const bool hi = lane >= 16;
    float v = hi ? s2 : s1;
    v += __shfl_xor_sync(~0u, hi ? s1 : s2, 16);
#pragma unroll
    for (int d = 8; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    if ((lane & 15) == 0) buf[parity][hi][warp] = v;
    __syncthreads();   // and every thread has read the slot
    if (t == 0) fetch(r + int64_t(slots) * gridDim.x, slot);
    if (++slot == slots) { slot = 0; phase ^= 1; }
    v = (lane & 15) < (nt >> 5) ? buf[parity][hi][lane & 15] : 0.0f;
#pragma unroll
    for (int d = 8; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    const float c1 = LAYER ? __shfl_sync(~0u, v, 0) * inv_n : 0.0f;
    const float c2 = __shfl_sync(~0u, v, 16) * inv_n;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (t + i * nt);
      if (c >= cols) break;
      float f[8];
      const Raw8<WT> w = KEEP ? kept[KEEP ? i : 0] : weight(i);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = rs * (dr[i][j] * w[j] - c1 - (xr[i][j] - m) * rs * c2);
      if (MXQ_IN_BOUNDS(r < a.rows, &g_err_norm, SITE_B_NORM_GRAD))
        store8(static_cast<XT*>(a.dx) + r * a.cols, c, cols, true, f);
    }
  }
  if (!ok && t == 0) drain_ring(full, slots, a.rows, a.timeout_ns);
  float* part = a.part + int64_t(blockIdx.x) * 2 * a.cols;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = 8 * (t + i * nt);
    if (c >= cols) break;
    store8(part, c, cols, true, dw[i]);
    if constexpr (DB_SHARED) {
      *reinterpret_cast<float4*>(part + cols + c) = db_at[2 * i * nt];
      *reinterpret_cast<float4*>(part + cols + c + 4) = db_at[(2 * i + 1) * nt];
    } else if (LAYER) {
      store8(part + cols, c, cols, true, db[i]);
    }
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

// The partial sums of each column, in a fixed order: 32 columns a CTA, its 32
// warps take every 32nd split each and are added up in order.
struct JoinArgs {
  const float* part;   // [splits][2][cols]
  int64_t cols;
  int splits;
  float* dweight;
  float* dbias;        // or null
};

__global__ void __launch_bounds__(1024) norm_grad_join(const JoinArgs a) {
  __shared__ float sums[2][32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cols = a.cols, c = int64_t(blockIdx.x) * 32 + lane;
  griddep_wait();
  griddep_launch_dependents();
  float dw = 0.0f, db = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (int s = warp; s < a.splits; s += 32) {
      const float* p = a.part + int64_t(s) * 2 * cols + c;
      dw += p[0];
      if (a.dbias) db += p[cols];
    }
  }
  sums[0][warp][lane] = dw;
  sums[1][warp][lane] = db;
  __syncthreads();
  if (warp < 2 && c < cols) {
    float* out = warp ? a.dbias : a.dweight;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < 32; ++q) v += sums[warp][q][lane];
    if (out && MXQ_IN_BOUNDS(c < cols, &g_err_norm, SITE_B_NORM_GRAD)) out[c] = v;
  }
}

// How a row is split: a warp per row, or a CTA of nt threads, with i chunks of
// eight elements per thread; i == 0: the row does not fit the registers.
struct RowPlan {
  bool warp;
  int nt, i;
};

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

// Backward.  The sums of dw and db take 16 registers a chunk beside x and dy:
// four chunks a thread fit for bf16 rows, two for fp32 and for a warp's row.
RowPlan backward_plan(int64_t cols, int x_dtype) {
  const int64_t chunks = (cols + 7) / 8;
  if (chunks <= 64) return {true, 256, chunks <= 32 ? 1 : 2};
  for (int i = chunks <= 256 ? 1 : 2; i <= (x_dtype == MXQ_OUT_BF16 ? 4 : 2); i *= 2)
    if (chunks <= 512 * i)
      return {false, static_cast<int>(((chunks + i - 1) / i + 31) / 32 * 32), i};
  return {false, 256, 0};
}

int grad_ctas_per_sm(const RowPlan& p) { return std::max(1, (p.i == 1 ? 768 : 512) / p.nt); }

// Shared memory behind the ring for the sums of db.
int grad_db_bytes(const RowPlan& p) { return p.i == 4 ? p.nt * 4 * 32 : 0; }

// Rows in flight of a CTA of norm_grad_ring, 0 where it does not apply: the
// shared memory of an SM (208 KB of it) split among its CTAs.
int grad_slots(const RowPlan& p, int64_t cols, int x_dtype) {
  const int64_t row = cols * (x_dtype == MXQ_OUT_BF16 ? 2 : 4);
  if (p.warp || !p.i || cols % 8 != 0) return 0;
  const int64_t fit = (208 * 1024 / grad_ctas_per_sm(p) - grad_db_bytes(p)) / (2 * row);
  return fit < 2 ? 0 : static_cast<int>(std::min<int64_t>(fit, N_MAX_SLOTS));
}

// Sets of partial sums.  Register kernels: one per CTA, as many CTAs as the
// registers let an SM hold at once (about 768, 512 and 512 threads with one,
// two and four chunks each), but with few rows no more than one an SM or one
// for eight rows, since each costs a set of sums to write and to join
// (517x1001 fp32: 11.2 us against 10.6).  Longer rows: enough that the column sums fill the
// device.
int grad_splits(int64_t rows, int64_t cols, int x_dtype) {
  const RowPlan p = backward_plan(cols, x_dtype);
  if (p.i) {
    const int64_t want = int64_t(grad_ctas_per_sm(p)) * sm_count();
    const int64_t few = std::max<int64_t>(sm_count(), rows / (p.warp ? 64 : 8));
    return static_cast<int>(std::min(std::min<int64_t>(p.warp ? (rows + 7) / 8 : rows, want), few));
  }
  const int64_t want = std::max<int64_t>(1, 8 * sm_count() / ((cols + 255) / 256));
  return static_cast<int>(std::min<int64_t>(std::min<int64_t>(rows, want), 512));
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
  if (cols % 8 != 0 || chunks <= (rms_codes ? 128 : 64) || chunks > 512 * N_RING_I) return p;
  p.nt = static_cast<int>(((chunks + N_RING_I - 1) / N_RING_I + 31) / 32 * 32);
  const int per_sm = std::max(1, 512 / p.nt);
  p.ctas = per_sm * sm_count();
  const int64_t fit = (200 * 1024 / per_sm) / (cols * size);
  if (rows >= 2 * p.ctas && fit >= 2)
    p.slots = static_cast<int>(std::min<int64_t>(fit, N_MAX_SLOTS));
  return p;
}

template <typename XT, typename WT, bool LAYER, int FMT>
bool launch_norm_ring(const NArgs& a, const RingPlan& p, cudaStream_t st) {
  const size_t smem = size_t(p.slots) * a.cols * sizeof(XT);
  return ensure_dynamic_smem(reinterpret_cast<const void*>(norm_ring<XT, WT, LAYER, FMT, N_RING_I>),
                             static_cast<int>(smem)) &&
         launch_early(norm_ring<XT, WT, LAYER, FMT, N_RING_I>, static_cast<unsigned>(p.ctas), p.nt,
                      smem, st, a);
}

template <typename XT, typename WT, bool LAYER, int FMT>
mxq_status launch_forward(NArgs a, cudaStream_t st) {
  const RingPlan ring = forward_ring(a.rows, a.cols, sizeof(XT), !LAYER && FMT >= 0);
  if (ring.slots) {
    a.slots = ring.slots;
    a.timeout_ns = wait_timeout_ns();
    return launch_norm_ring<XT, WT, LAYER, FMT>(a, ring, st) ? launch_status() : MXQ_ERR_CUDA;
  }
  const RowPlan p = forward_plan(a.rows, a.cols);
  const unsigned rows = static_cast<unsigned>(a.rows), groups = (rows + 7) / 8;
  bool ok;
  if (p.warp) {
    ok = p.i == 1   ? launch_early(norm_regs<XT, WT, LAYER, FMT, true, 1>, groups, 256, 0, st, a)
         : p.i == 2 ? launch_early(norm_regs<XT, WT, LAYER, FMT, true, 2>, groups, 256, 0, st, a)
                    : launch_early(norm_regs<XT, WT, LAYER, FMT, true, 4>, groups, 256, 0, st, a);
  } else {
    ok = p.i == 1   ? launch_early(norm_regs<XT, WT, LAYER, FMT, false, 1>, rows, p.nt, 0, st, a)
         : p.i == 2 ? launch_early(norm_regs<XT, WT, LAYER, FMT, false, 2>, rows, p.nt, 0, st, a)
         : p.i == 4 ? launch_early(norm_regs<XT, WT, LAYER, FMT, false, 4>, rows, p.nt, 0, st, a)
                    : launch_early(norm_rows<XT, WT, LAYER, FMT>, rows, 256, 0, st, a);
  }
  return ok ? launch_status() : MXQ_ERR_CUDA;
}

template <typename XT, typename WT, bool LAYER>
mxq_status run_forward(const NArgs& a, int fmt, cudaStream_t st) {
  if (!a.codes) return launch_forward<XT, WT, LAYER, -1>(a, st);
  return fmt == MXQ_E4M3 ? launch_forward<XT, WT, LAYER, MXQ_E4M3>(a, st)
                         : launch_forward<XT, WT, LAYER, MXQ_E5M2>(a, st);
}

template <typename XT, typename WT, bool LAYER, int I>
bool launch_ring(const NGrad& a, int nt, size_t smem, cudaStream_t st) {
  return ensure_dynamic_smem(reinterpret_cast<const void*>(norm_grad_ring<XT, WT, LAYER, I>),
                             static_cast<int>(smem)) &&
         launch_early(norm_grad_ring<XT, WT, LAYER, I>, static_cast<unsigned>(a.splits), nt, smem,
                      st, a);
}

template <typename XT, typename WT, bool LAYER>
mxq_status run_backward(const NGrad& a, cudaStream_t st) {
  const RowPlan p = backward_plan(a.cols, std::is_same<XT, float>::value ? MXQ_OUT_F32
                                                                         : MXQ_OUT_BF16);
  const unsigned grid = static_cast<unsigned>(a.splits);
  bool ok = true;
  if (p.warp) {
    const size_t smem = size_t(8) * 8 * p.i * 32 * sizeof(float);
    ok = p.i == 1 ? launch_early(norm_grad_regs<XT, WT, LAYER, true, 1>, grid, 256, smem, st, a)
                  : launch_early(norm_grad_regs<XT, WT, LAYER, true, 2>, grid, 256, smem, st, a);
  } else if (p.i && a.slots) {
    const size_t smem = size_t(a.slots) * 2 * a.cols * sizeof(XT) + grad_db_bytes(p);
    if (p.i == 1) ok = launch_ring<XT, WT, LAYER, 1>(a, p.nt, smem, st);
    else if (p.i == 2) ok = launch_ring<XT, WT, LAYER, 2>(a, p.nt, smem, st);
    else if constexpr (std::is_same<XT, __nv_bfloat16>::value)
      ok = launch_ring<XT, WT, LAYER, 4>(a, p.nt, smem, st);
  } else if (p.i) {
    if (p.i == 1) ok = launch_early(norm_grad_regs<XT, WT, LAYER, false, 1>, grid, p.nt, 0, st, a);
    else if (p.i == 2)
      ok = launch_early(norm_grad_regs<XT, WT, LAYER, false, 2>, grid, p.nt, 0, st, a);
    else if constexpr (std::is_same<XT, __nv_bfloat16>::value)
      ok = launch_early(norm_grad_regs<XT, WT, LAYER, false, 4>, grid, p.nt, 0, st, a);
  } else {
    // the column sums first: dx may take the place of x or dy
    const unsigned groups = static_cast<unsigned>((a.cols + 255) / 256);
    norm_grad_cols<XT, LAYER><<<dim3(groups, grid), 256, 0, st>>>(a);
    norm_grad_rows<XT, WT, LAYER><<<static_cast<unsigned>(a.rows), 256, 0, st>>>(a);
  }
  if (!ok) return MXQ_ERR_CUDA;
  const JoinArgs j{a.part, a.cols, a.splits, a.dweight, a.dbias};
  ok = launch_early(norm_grad_join, static_cast<unsigned>((a.cols + 31) / 32), 1024, 0, st, j);
  return ok ? launch_status() : MXQ_ERR_CUDA;
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
  const int splits = std::max(grad_splits(rows, cols, MXQ_OUT_BF16),
                              grad_splits(rows, cols, MXQ_OUT_F32));
  return static_cast<size_t>(splits) * 2 * cols * sizeof(float);
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
  if (p->dbias && p->kind != MXQ_NORM_LAYER) return MXQ_ERR_ARG;
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
  a.splits = grad_splits(p->rows, p->cols, p->x_dtype);
  a.vec = p->cols % 8 == 0;
  a.slots = grad_slots(backward_plan(p->cols, p->x_dtype), p->cols, p->x_dtype);
  a.timeout_ns = wait_timeout_ns();
  return dispatch(p->x_dtype, p->w_dtype, p->kind, Backward{a, s});
}
