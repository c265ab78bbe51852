// Quantization to FP8 codes with one fp32 scale per block of 128.
//
// A block of values v gets scale = max(amax / fmax, 2^-126) and codes
// RN_sat(v * (1 / scale)); its amax comes from the raw bf16 bits, so it is
// exact whatever the order of the maxima.  Blocks run along rows, along
// columns (codes stored transposed), both in one read, or span 128x128 tiles
// (with the transposed codes).
//
// A CTA of 256 threads takes one 128x128 tile of x, which holds whole blocks
// of every kind.  A thread keeps an 8x8 piece of it in registers (8 rows of
// one 16-byte load), so a row's amax is a reduction over 16 lanes, a column's
// one over the 16 groups of rows, and the transposed codes of the piece are
// eight 8-byte words that need no byte shuffles: word j is column j of the
// piece.  They go through a swizzled 16 KB tile of shared memory so that the
// transposed lines leave in 16-byte stores, 128 bytes per line.
//
// Bound by HBM: 2 bytes read and one written per element and layout.  A CTA per
// tile, four (128x128 tiles with both codes: three) of them on an SM: 28672x4096
// weight 71 us, 0.97 of the copy rate; 8192x4096 activation, both layouts, 25.8
// us, 0.77 (its 2048 tiles make 3.4 waves).  Persistent CTAs whose next tile
// comes by TMA under the conversion ran 8192x4096 in 24.1 us and the weight in
// 84: not kept.  Rows that start between 16-byte boundaries are cut out of
// aligned loads: 8001x4097 along rows 23.4 us (element by element 33.4), both
// layouts 30.9 (44.0).
#include "fp8_common.cuh"
#include "mxq_host.h"

namespace mxq {

__device__ uint32_t g_err_fp8_quant;

namespace {

enum : int { Q_ROW = 1, Q_COL = 2, Q_DUAL = 3, Q_TILES = 4 };

struct QArgs {
  const __nv_bfloat16* x;
  int64_t rows, cols;
  int64_t n_ct;              // column tiles
  uint8_t* codes_r;          // row-wise codes (tiles: codes), or null
  float* scales_r;
  uint8_t* codes_c;          // transposed codes, or null
  float* scales_c;
  int64_t pitch_r, pitch_c;  // bytes between code lines
  int64_t lines_r, lines_c;  // floats between scale rows
};

// Magnitudes of a bf16 pair without the sign bits.
MXQ_DEV uint32_t mag2(uint32_t w) { return w & 0x7FFF7FFFu; }

// VEC: rows of x start at 16-byte boundaries.
template <int MODE, int FR, int FC, bool VEC>
__global__ void __launch_bounds__(256, MODE == Q_TILES ? 3 : 4) fp8_quant_kernel(const QArgs a) {
  constexpr bool ROW = MODE == Q_ROW || MODE == Q_DUAL;
  constexpr bool COL = MODE == Q_COL || MODE == Q_DUAL;
  constexpr bool TILES = MODE == Q_TILES;
  constexpr bool TRANS = COL || TILES;
  __shared__ __align__(16) uint8_t stage[TRANS ? 128 * 128 : 16];
  __shared__ uint32_t colmax[COL ? 8 * 64 : 1];
  __shared__ __align__(16) float colmul[COL ? 128 : 1];
  __shared__ uint32_t tilemax[TILES ? 8 : 1];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c8 = tid & 15, rg = tid >> 4;   // 8-column chunk, group of 8 rows
  const int64_t ct = blockIdx.x % a.n_ct, rt = blockIdx.x / a.n_ct;
  const int64_t r0 = rt * 128, c0 = ct * 128;
  const int64_t row = r0 + rg * 8, col = c0 + c8 * 8;

  griddep_wait();
  griddep_launch_dependents();
  uint32_t v[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0u;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = row + i;
      // cols % 8 == 0: the whole chunk is inside the row
      if (r < a.rows && col < a.cols &&
          MXQ_IN_BOUNDS(col + 8 <= a.cols, &g_err_fp8_quant, SITE_B_FP8_LOAD)) {
        const uint4 w = *reinterpret_cast<const uint4*>(a.x + r * a.cols + col);
        v[i][0] = w.x; v[i][1] = w.y; v[i][2] = w.z; v[i][3] = w.w;
      }
    }
  } else {
    // rows that start anywhere: four at a time, as the registers allow
    const int64_t n = a.rows * a.cols;
    constexpr int REACH = Across<__nv_bfloat16>::REACH;
#pragma unroll
    for (int i0 = 0; i0 < 8; i0 += 4) {
      Across<__nv_bfloat16> t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t[i].clear();
        const int64_t r = row + i0 + i, at = r * a.cols + col;
        if (r < a.rows && col < a.cols && at + REACH <= n &&
            MXQ_IN_BOUNDS(at >= 0, &g_err_fp8_quant, SITE_B_FP8_LOAD))
          t[i].load(a.x, at);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i].cut((row + i0 + i) * a.cols + col, v[i0 + i]);
    }
    if (col < a.cols && (min(row + 8, a.rows) - 1) * a.cols + col + REACH > n) {
      // the last elements of x
      for (int i = 0; i < 8; ++i) {
        const int64_t r = row + i, at = r * a.cols + col;
        if (r >= a.rows || at + REACH <= n) continue;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at + j < n)
            w[j >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(a.x)[at + j])
                         << (16 * (j & 1));
#pragma unroll
        for (int k = 0; k < 8; ++k)   // v keeps compile-time indices
          if (k == i) {
            v[k][0] = w[0]; v[k][1] = w[1]; v[k][2] = w[2]; v[k][3] = w[3];
          }
      }
    }
    if (col + 8 > a.cols) {   // the next row's elements
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t left = a.cols - col - 2 * j;
        const uint32_t keep = left >= 2 ? ~0u : left == 1 ? 0xFFFFu : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i][j] &= keep;
      }
    }
  }

  auto unpack = [&](int i, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16lo(v[i][j]);
      f[2 * j + 1] = bf16hi(v[i][j]);
    }
  };
  // eight codes of row `i` of the piece
  auto store_row = [&](int i, float mul) {
    float f[8];
    unpack(i, f);
    const uint2 w = fp8_encode8<FR>(f, mul);
    const int64_t r = row + i;
    if (r < a.rows && col < a.pitch_r &&
        MXQ_IN_BOUNDS(col + 8 <= a.pitch_r, &g_err_fp8_quant, SITE_B_FP8_CODES))
      *reinterpret_cast<uint2*>(a.codes_r + r * a.pitch_r + col) = w;
  };
  // eight codes of column `j` of the piece into the staging tile: line
  // c8 * 8 + j, 8-byte chunk rg, the chunks of a line swizzled by c8 so that
  // the 16 lanes of one row group hit distinct banks
  auto stage_col = [&](int j, float mul) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (j & 1) ? bf16hi(v[i][j >> 1]) : bf16lo(v[i][j >> 1]);
    const uint2 w = fp8_encode8<FC>(f, mul);
    *reinterpret_cast<uint2*>(stage + (c8 * 8 + j) * 128 + ((rg ^ c8) & 15) * 8) = w;
  };

  if constexpr (COL) {
    uint32_t m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = mag2(v[0][j]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m[j] = max_abs_bf16x2(m[j], v[i][j]);
      m[j] = max_abs_bf16x2(m[j], __shfl_xor_sync(~0u, m[j], 16));
    }
    if (lane < 16)
      *reinterpret_cast<uint4*>(&colmax[warp * 64 + c8 * 4]) = make_uint4(m[0], m[1], m[2], m[3]);
  }
  if constexpr (ROW) {
    // two rows per packed word: the chunk's pair maxima folded to one value a row
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo = mag2(v[2 * i][0]), hi = mag2(v[2 * i + 1][0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) {
        lo = max_abs_bf16x2(lo, v[2 * i][j]);
        hi = max_abs_bf16x2(hi, v[2 * i + 1][j]);
      }
      m[i] = max_abs_bf16x2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
      for (int d = 8; d; d >>= 1) m[i] = max_abs_bf16x2(m[i], __shfl_xor_sync(~0u, m[i], d));
    }
    // lane c8 works out the scale of row c8 % 8 of the group
    const uint32_t w01 = (c8 & 2) ? m[1] : m[0], w23 = (c8 & 2) ? m[3] : m[2];
    const uint32_t w = mag2((c8 & 4) ? w23 : w01);
    float scale, mul;
    fp8_scale<FR>((c8 & 1) ? bf16hi(w) : bf16lo(w), scale, mul);
    const int64_t r = row + (c8 & 7);
    if (c8 < 8 && r < a.lines_r &&
        MXQ_IN_BOUNDS(ct * 128 < a.cols, &g_err_fp8_quant, SITE_B_FP8_SCALES))
      a.scales_r[ct * a.lines_r + r] = scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) store_row(i, __shfl_sync(~0u, mul, (lane & 16) + i));
  }
  if constexpr (COL) {
    __syncthreads();
    if (tid < 64) {
      uint32_t m = colmax[tid];
#pragma unroll
      for (int w = 1; w < 8; ++w) m = max_abs_bf16x2(m, colmax[w * 64 + tid]);
      m = mag2(m);
      float s0, s1, m0, m1;
      fp8_scale<FC>(bf16lo(m), s0, m0);
      fp8_scale<FC>(bf16hi(m), s1, m1);
      *reinterpret_cast<float2*>(&colmul[2 * tid]) = make_float2(m0, m1);
      const int64_t c = c0 + 2 * tid;   // lines_c is even: both or neither
      if (c < a.lines_c &&
          MXQ_IN_BOUNDS(rt * 128 < a.rows, &g_err_fp8_quant, SITE_B_FP8_SCALES))
        *reinterpret_cast<float2*>(&a.scales_c[rt * a.lines_c + c]) = make_float2(s0, s1);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) stage_col(j, colmul[c8 * 8 + j]);
  }
  if constexpr (TILES) {
    uint32_t m = mag2(v[0][0]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max_abs_bf16x2(m, v[i][j]);
#pragma unroll
    for (int d = 16; d; d >>= 1) m = max_abs_bf16x2(m, __shfl_xor_sync(~0u, m, d));
    if (lane == 0) tilemax[warp] = m;
    __syncthreads();
    m = tilemax[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = max_abs_bf16x2(m, tilemax[w]);
    m = mag2(m);
    m = max_abs_bf16x2(m, __byte_perm(m, m, 0x1032));
    float scale, mul;
    fp8_scale<FR>(bf16lo(mag2(m)), scale, mul);
    const int64_t n_rt = (a.rows + 127) / 128;
    if (tid == 0 &&
        MXQ_IN_BOUNDS(rt < n_rt && ct < a.n_ct, &g_err_fp8_quant, SITE_B_FP8_SCALES)) {
      a.scales_r[rt * a.n_ct + ct] = scale;
      if (a.codes_c) a.scales_c[ct * n_rt + rt] = scale;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) store_row(i, mul);
    if (!a.codes_c) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) stage_col(j, mul);
  }
  if constexpr (TRANS) {
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int p = tid + u * 256;                 // 16-byte piece of the tile
      const int line = p >> 3, k = p & 7;
      const int sw = (line >> 3) & 15;
      const uint4 t = *reinterpret_cast<const uint4*>(stage + line * 128 + (k ^ (sw >> 1)) * 16);
      const uint4 w = (sw & 1) ? make_uint4(t.z, t.w, t.x, t.y) : t;
      const int64_t c = c0 + line, b = r0 + k * 16;
      if (c < a.cols && b < a.pitch_c &&
          MXQ_IN_BOUNDS(b + 16 <= a.pitch_c, &g_err_fp8_quant, SITE_B_FP8_CODES))
        *reinterpret_cast<uint4*>(a.codes_c + c * a.pitch_c + b) = w;
    }
  }
}

template <int MODE, int FR, int FC>
mxq_status launch(const QArgs& a, void* stream) {
  const int64_t n = (a.rows + 127) / 128 * a.n_ct;
  if (n >= (int64_t(1) << 31)) return MXQ_ERR_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned ctas = static_cast<unsigned>(n);
  const bool ok = a.cols % 8 == 0
                      ? launch_early(fp8_quant_kernel<MODE, FR, FC, true>, ctas, 256, 0, st, a)
                      : launch_early(fp8_quant_kernel<MODE, FR, FC, false>, ctas, 256, 0, st, a);
  return ok ? launch_status() : MXQ_ERR_CUDA;
}

mxq_status check_input(const void* x, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31))
    return MXQ_ERR_ARG;
  if (rows && cols && !x) return MXQ_ERR_ARG;
  return aligned16(x) ? MXQ_OK : MXQ_ERR_ALIGN;
}

mxq_status check_out(const void* codes, const void* scales) {
  if (!codes || !scales) return MXQ_ERR_ARG;
  return aligned16(codes) && aligned16(scales) ? MXQ_OK : MXQ_ERR_ALIGN;
}

QArgs args(const void* x, int64_t rows, int64_t cols) {
  QArgs a = {};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.rows = rows;
  a.cols = cols;
  a.n_ct = (cols + 127) / 128;
  a.pitch_r = fp8_pitch(cols);
  a.pitch_c = fp8_pitch(rows);
  a.lines_r = fp8_lines(rows);
  a.lines_c = fp8_lines(cols);
  return a;
}

}  // namespace

uint32_t take_fp8_quant_error() {
  uint32_t h = 0;
  if (cudaMemcpyFromSymbol(&h, g_err_fp8_quant, sizeof(h)) != cudaSuccess) return MXQ_ERR_CUDA;
  if (h) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_err_fp8_quant, &z, sizeof(z));
  }
  return h;
}

}  // namespace mxq

using namespace mxq;

extern "C" size_t mxq_fp8_pitch(int64_t blocked) {
  return blocked > 0 && blocked < (int64_t(1) << 31) ? static_cast<size_t>(fp8_pitch(blocked)) : 0;
}

extern "C" size_t mxq_fp8_scale_count(int64_t lines, int64_t blocked, int scales) {
  if (lines <= 0 || blocked <= 0 || lines >= (int64_t(1) << 31) || blocked >= (int64_t(1) << 31))
    return 0;
  const int64_t kb = (blocked + 127) / 128;
  if (scales == MXQ_FP8_LINES) return static_cast<size_t>(kb * fp8_lines(lines));
  if (scales == MXQ_FP8_TILES) return static_cast<size_t>(kb * ((lines + 127) / 128));
  return 0;
}

extern "C" mxq_status mxq_fp8_quantize(const void* x, int64_t rows, int64_t cols, int layout,
                                       int fmt, void* codes, float* scales, void* stream) {
  if ((layout != MXQ_ROWWISE && layout != MXQ_COLWISE_T) || !is_fp8(fmt)) return MXQ_ERR_ARG;
  mxq_status st = check_input(x, rows, cols);
  if (st != MXQ_OK) return st;
  if (rows == 0 || cols == 0) return MXQ_OK;
  if ((st = check_out(codes, scales)) != MXQ_OK) return st;
  QArgs a = args(x, rows, cols);
  if (layout == MXQ_ROWWISE) {
    a.codes_r = static_cast<uint8_t*>(codes);
    a.scales_r = scales;
    return fmt == MXQ_E4M3 ? launch<Q_ROW, MXQ_E4M3, MXQ_E4M3>(a, stream)
                           : launch<Q_ROW, MXQ_E5M2, MXQ_E5M2>(a, stream);
  }
  a.codes_c = static_cast<uint8_t*>(codes);
  a.scales_c = scales;
  return fmt == MXQ_E4M3 ? launch<Q_COL, MXQ_E4M3, MXQ_E4M3>(a, stream)
                         : launch<Q_COL, MXQ_E5M2, MXQ_E5M2>(a, stream);
}

extern "C" mxq_status mxq_fp8_quantize_dual(const void* x, int64_t rows, int64_t cols, int fmt_r,
                                            void* codes_r, float* scales_r, int fmt_c,
                                            void* codes_c, float* scales_c, void* stream) {
  if (!is_fp8(fmt_r) || !is_fp8(fmt_c)) return MXQ_ERR_ARG;
  mxq_status st = check_input(x, rows, cols);
  if (st != MXQ_OK) return st;
  if (rows == 0 || cols == 0) return MXQ_OK;
  if ((st = check_out(codes_r, scales_r)) != MXQ_OK) return st;
  if ((st = check_out(codes_c, scales_c)) != MXQ_OK) return st;
  QArgs a = args(x, rows, cols);
  a.codes_r = static_cast<uint8_t*>(codes_r);
  a.scales_r = scales_r;
  a.codes_c = static_cast<uint8_t*>(codes_c);
  a.scales_c = scales_c;
  if (fmt_r == MXQ_E4M3)
    return fmt_c == MXQ_E4M3 ? launch<Q_DUAL, MXQ_E4M3, MXQ_E4M3>(a, stream)
                             : launch<Q_DUAL, MXQ_E4M3, MXQ_E5M2>(a, stream);
  return fmt_c == MXQ_E4M3 ? launch<Q_DUAL, MXQ_E5M2, MXQ_E4M3>(a, stream)
                           : launch<Q_DUAL, MXQ_E5M2, MXQ_E5M2>(a, stream);
}

extern "C" mxq_status mxq_fp8_quantize_tiles(const void* x, int64_t rows, int64_t cols, int fmt,
                                             void* codes, float* scales, void* codes_t,
                                             float* scales_t, void* stream) {
  if (!is_fp8(fmt) || !codes_t != !scales_t) return MXQ_ERR_ARG;
  mxq_status st = check_input(x, rows, cols);
  if (st != MXQ_OK) return st;
  if (rows == 0 || cols == 0) return MXQ_OK;
  if (!codes || !scales) return MXQ_ERR_ARG;
  if (!aligned16(codes) || !aligned16(codes_t)) return MXQ_ERR_ALIGN;
  if (((reinterpret_cast<uintptr_t>(scales) | reinterpret_cast<uintptr_t>(scales_t)) & 3u) != 0)
    return MXQ_ERR_ALIGN;
  QArgs a = args(x, rows, cols);
  a.codes_r = static_cast<uint8_t*>(codes);
  a.scales_r = scales;
  a.codes_c = static_cast<uint8_t*>(codes_t);
  a.scales_c = scales_t;
  return fmt == MXQ_E4M3 ? launch<Q_TILES, MXQ_E4M3, MXQ_E4M3>(a, stream)
                         : launch<Q_TILES, MXQ_E5M2, MXQ_E5M2>(a, stream);
}
