// What the norm's forward and backward kernels share: chunks of eight elements
// of a row and their places in shared memory, sums, run-time types.
#pragma once

#include "fp8_common.cuh"
#include "mxq_host.h"

namespace mxq {

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
    __nv_bfloat16* p = row + col;
    if (col + 8 <= cols) {   // pairs between 4-byte boundaries
      uint32_t* q = reinterpret_cast<uint32_t*>(reinterpret_cast<uintptr_t>(p + 1) & ~uintptr_t(3));
      if (reinterpret_cast<uintptr_t>(p) & 2) {
        p[0] = __float2bfloat16_rn(f[0]);
#pragma unroll
        for (int j = 0; j < 3; ++j) q[j] = pack_bf16(f[2 * j + 1], f[2 * j + 2]);
        p[7] = __float2bfloat16_rn(f[7]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < cols) p[j] = __float2bfloat16_rn(f[j]);
  }
}

template <typename Ix>
MXQ_DEV void store8(float* row, Ix col, Ix cols, bool vec, const float (&f)[8]) {
  if (vec) {
    *reinterpret_cast<float4*>(row + col) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(row + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    float* p = row + col;
    if (col + 8 <= cols) {   // pairs between 8-byte boundaries
      float2* q = reinterpret_cast<float2*>(reinterpret_cast<uintptr_t>(p + 1) & ~uintptr_t(7));
      if (reinterpret_cast<uintptr_t>(p) & 4) {
        p[0] = f[0];
#pragma unroll
        for (int j = 0; j < 3; ++j) q[j] = make_float2(f[2 * j + 1], f[2 * j + 2]);
        p[7] = f[7];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = make_float2(f[2 * j], f[2 * j + 1]);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < cols) p[j] = f[j];
  }
}

// Eight elements of a row as they lie in memory.
template <typename XT>
struct Raw8;

template <>
struct Raw8<__nv_bfloat16> {
  using Words = uint32_t[4];
  Words w;
  MXQ_DEV void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
  MXQ_DEV Words& words() { return w; }
  // From a row that starts on a 16-byte boundary; cols % 8 == 0.
  MXQ_DEV void load(const __nv_bfloat16* row, int col, int cols) {
    clear();
    if (col >= cols) return;
    const uint4 t = *reinterpret_cast<const uint4*>(row + col);
    w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
  }
  MXQ_DEV void load_some(const __nv_bfloat16* p, int n) {   // the first n
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) w[j >> 1] |= static_cast<uint32_t>(q[j]) << (16 * (j & 1));
  }
  MXQ_DEV void keep(int n) {   // zeros from element n on
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] &= n >= 2 * j + 2 ? ~0u : n == 2 * j + 1 ? 0xFFFFu : 0u;
  }
  MXQ_DEV float operator[](int j) const { return j & 1 ? bf16hi(w[j >> 1]) : bf16lo(w[j >> 1]); }
};

template <>
struct Raw8<float> {
  using Words = float[8];
  Words f;
  MXQ_DEV void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
  }
  MXQ_DEV Words& words() { return f; }
  MXQ_DEV void load(const float* row, int col, int cols) {
    clear();
    if (col < cols) load8(row, col, cols, true, f);
  }
  MXQ_DEV void load_some(const float* p, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) f[j] = p[j];
  }
  MXQ_DEV void keep(int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= n) f[j] = 0.0f;
  }
  MXQ_DEV float operator[](int j) const { return f[j]; }
};

// Chunk of weight or bias at `col`: VEC as a row of x, else with a part of a
// chunk at its end.
template <bool VEC, typename WT>
MXQ_DEV void load_param(Raw8<WT>& w, const void* p, int col, int cols) {
  const WT* q = static_cast<const WT*>(p);
  if (VEC || col + 8 <= cols) {
    w.load(q, col, cols);
  } else {
    w.clear();
    w.load_some(q + col, cols - col);
  }
}

// A chunk as it is loaded and the row's elements in it, which are cut out where
// rows do not start on 16-byte boundaries (VEC false).  `at` is the chunk's place
// among the n elements of x, `col` its column.
template <typename XT, bool VEC>
struct Chunk;

template <typename XT>
struct Chunk<XT, true> {
  Raw8<XT> raw;
  MXQ_DEV void load(const XT* x, int64_t at, int64_t, int col, int cols) {
    raw.clear();
    if (col < cols) raw.load(x + at, 0, 8);
  }
  // From shared memory, where the row starts at `row`.
  MXQ_DEV void load_ring(const XT* row, int64_t, int64_t, int col, int cols) {
    raw.load(row, col, cols);
  }
  MXQ_DEV Raw8<XT> get(const XT*, int64_t, int64_t, int, int) const { return raw; }
};

template <typename XT>
struct Chunk<XT, false> {
  static constexpr int REACH = Across<XT>::REACH;
  Across<XT> words;
  MXQ_DEV void load(const XT* x, int64_t at, int64_t n, int col, int cols) {
    words.clear();
    if (col < cols && at + REACH <= n) words.load(x, at);
  }
  // `row` holds the aligned 16-byte words that the row begins in.
  MXQ_DEV void load_ring(const XT* row, int64_t at, int64_t n, int col, int cols) {
    words.clear();
    const int skip = static_cast<int>((at - col) & (16 / int(sizeof(XT)) - 1));
    if (col < cols && at + REACH <= n) words.load(row, skip + col);
  }
  MXQ_DEV Raw8<XT> get(const XT* x, int64_t at, int64_t n, int col, int cols) const {
    Raw8<XT> to;
    words.cut(at, to.words());
    if (col + 8 > cols) to.keep(cols - col);
    if (col < cols && at + REACH > n) {   // the last elements of x
      to.clear();
      to.load_some(x + at, cols - col);
    }
    return to;
  }
};

// Bytes of shared memory for a row: VEC false, the 16-byte words it can lie in
// and two more that reading its last chunk may reach.
constexpr int64_t ring_row_bytes(int64_t cols, int64_t size) {
  return cols % 8 == 0 ? cols * size : (cols * size + 29) / 16 * 16 + 32;
}

// Copies row r of x into shared memory; the words that end past x are left out
// (Chunk reads their elements from x).
template <typename XT, bool VEC>
struct RowCopy {
  const XT* src;
  uint32_t bytes;
  MXQ_DEV RowCopy(const XT* x, int64_t r, int64_t rows, int64_t cols) {
    const int64_t start = r * cols, per = 16 / sizeof(XT);
    if (VEC) {
      src = x + start;
      bytes = static_cast<uint32_t>(cols * sizeof(XT));
    } else {
      const int64_t first = start / per * per;
      const int64_t end = min((start + cols + per - 1) / per, rows * cols / per) * per;
      src = x + first;
      bytes = static_cast<uint32_t>((end - first) * sizeof(XT));
    }
  }
  // Whether the copy lies in the n elements from x on.
  MXQ_DEV bool inside(const XT* x, int64_t n) const {
    return src >= x && src + bytes / sizeof(XT) <= x + n;
  }
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

// How a row is split: a warp per row, or a CTA of nt threads, with i chunks of
// eight elements per thread; i == 0: the row does not fit the registers.
struct RowPlan {
  bool warp;
  int nt, i;
};

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

inline mxq_status norm_check(int64_t rows, int64_t cols, int kind, int x_dtype, int w_dtype) {
  const int64_t lim = int64_t(1) << 31;
  if (rows < 0 || cols < 0 || rows >= lim || cols >= lim) return MXQ_ERR_ARG;
  if (kind != MXQ_NORM_LAYER && kind != MXQ_NORM_RMS) return MXQ_ERR_ARG;
  if ((x_dtype != MXQ_OUT_F32 && x_dtype != MXQ_OUT_BF16) ||
      (w_dtype != MXQ_OUT_F32 && w_dtype != MXQ_OUT_BF16))
    return MXQ_ERR_ARG;
  return MXQ_OK;
}

}  // namespace mxq
