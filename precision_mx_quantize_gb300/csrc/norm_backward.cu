// Backward pass of layer norm and RMS norm (the formulas and measurements are
// with the forward pass).
#include <type_traits>

#include "norm_common.cuh"

namespace mxq {

__device__ uint32_t g_err_norm_grad;

namespace {

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

// This CTA's set of partial sums is one of those the workspace holds.
MXQ_DEV bool part_in_bounds(const NGrad& a) {
  return MXQ_IN_BOUNDS(blockIdx.x < a.splits, &g_err_norm_grad, SITE_B_NORM_GRAD);
}

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
    if (MXQ_IN_BOUNDS(r < a.rows && 8 * c < cols, &g_err_norm_grad, SITE_B_NORM_GRAD))
      store8(static_cast<XT*>(a.dx) + r * cols, 8 * c, cols, vec, f);
  }
}

// Backward for rows of at most 256 I elements: a warp per row, over every
// grid-th group of eight.  A lane keeps its columns' sums of dw and db in
// registers for all its rows, so x and dy are read once; the next row's are
// loaded under this row's reduction.  The CTA's sums go to `part`, which
// norm_grad_join adds up in order.
template <typename XT, typename WT, bool LAYER, int I, bool VEC>
__global__ void __launch_bounds__(256) norm_grad_regs(const NGrad a) {
  __shared__ float sums[8 * 8 * I * 32];
  const int cols = static_cast<int>(a.cols);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = int64_t(blockIdx.x) * 8 + warp, step = int64_t(gridDim.x) * 8;
  const int64_t n = a.rows * a.cols;
  const float inv_n = 1.0f / static_cast<float>(cols);
  const XT* const all_x = static_cast<const XT*>(a.x);
  const XT* const all_dy = static_cast<const XT*>(a.dy);
  griddep_wait();
  griddep_launch_dependents();
  float dw[I][8], db[I][8];
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.0f;
  Raw8<WT> w[I];
#pragma unroll
  for (int i = 0; i < I; ++i) load_param<VEC>(w[i], a.weight, 8 * (lane + i * 32), cols);
  Chunk<XT, VEC> x[I], dy[I];
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t r) {
    if (r >= a.rows) return;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (lane + i * 32);
      x[i].load(all_x, r * a.cols + c, n, c, cols);
      dy[i].load(all_dy, r * a.cols + c, n, c, cols);
    }
    mean = LAYER ? a.mean[r] : 0.0f;
    rstd = a.rstd[r];
  };
  load(first);
  for (int64_t r = first; r < a.rows; r += step) {
    float s1 = 0.0f, s2 = 0.0f;
    float h[I][8], g[I][8];
    const float m = mean, rs = rstd;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (lane + i * 32);
      const Raw8<XT> xr = x[i].get(all_x, r * a.cols + c, n, c, cols);
      const Raw8<XT> dr = dy[i].get(all_dy, r * a.cols + c, n, c, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = dr[j];               // zero past the row's end
        h[i][j] = (xr[j] - m) * rs;
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
    const float c1 = LAYER ? s1 * inv_n : 0.0f, c2 = s2 * inv_n;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (lane + i * 32);
      if (c >= cols) break;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = rs * (g[i][j] - c1 - h[i][j] * c2);
      if (MXQ_IN_BOUNDS(r < a.rows, &g_err_norm_grad, SITE_B_NORM_GRAD))
        store8(static_cast<XT*>(a.dx) + r * a.cols, c, cols, VEC, f);
    }
  }
  // the eight warps' sums, in order
  float* part = a.part + int64_t(blockIdx.x) * 2 * a.cols;
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
      if (c < cols && part_in_bounds(a)) part[k * cols + c] = v;
    }
  }
}

// The same for longer rows, a CTA each, over every grid-th row.  The rows come
// through a ring of a.slots pairs (x, dy) in shared memory, filled by
// bulk copies a.slots rows ahead.  One row ahead in registers left each row
// waiting for its loads (8192x4096 bf16, both kernels: 48 us against 39).
template <typename XT, typename WT, bool LAYER, int I, bool VEC>
__global__ void __launch_bounds__(512) norm_grad_ring(const NGrad a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[N_MAX_SLOTS];
  __shared__ float buf[2][2][16];
  const int cols = static_cast<int>(a.cols), nt = blockDim.x, t = threadIdx.x;
  const int lane = t & 31, warp = t >> 5;
  const float inv_n = 1.0f / static_cast<float>(cols);
  const uint32_t row_bytes = static_cast<uint32_t>(ring_row_bytes(cols, sizeof(XT)));
  const uint32_t slot_bytes = 2 * row_bytes;
  const XT* const all_x = static_cast<const XT*>(a.x);
  const XT* const all_dy = static_cast<const XT*>(a.dy);
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
    const uint32_t bar = smem_u32(&full[slot]), dst = smem_u32(ring) + slot * slot_bytes;
    const RowCopy<XT, VEC> cx(all_x, r, a.rows, a.cols), cd(all_dy, r, a.rows, a.cols);
    if (!MXQ_IN_BOUNDS(slot < slots && cx.inside(all_x, n) && cd.inside(all_dy, n) &&
                           cx.bytes <= row_bytes,
                       &g_err_norm_grad, SITE_B_NORM_GRAD))
      return;
    mbar_arrive_expect_tx(bar, cx.bytes + cd.bytes);
    bulk_load(dst, cx.src, cx.bytes, bar);
    bulk_load(dst + row_bytes, cd.src, cd.bytes, bar);
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
    load_param<VEC>(w, a.weight, 8 * (t + i * nt), cols);
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
      record_error(&g_err_norm_grad, MXQ_ERR_TIMEOUT, SITE_NORM_FULL);
      ok = false;   // the results are void; no further wait
    }
    const XT* x = reinterpret_cast<const XT*>(ring + slot * slot_bytes);
    const XT* dy = reinterpret_cast<const XT*>(ring + slot * slot_bytes + row_bytes);
    float s1 = 0.0f, s2 = 0.0f;
    // x and dy are kept as they lie in memory: two operations more per element
    // below, but bf16 rows then take half the registers
    Raw8<XT> xr[I], dr[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 8 * (t + i * nt);
      const int64_t place = r * a.cols + c;
      Chunk<XT, VEC> in;
      in.load_ring(x, place, n, c, cols);
      xr[i] = in.get(all_x, place, n, c, cols);
      in.load_ring(dy, place, n, c, cols);
      dr[i] = in.get(all_dy, place, n, c, cols);
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
      if (MXQ_IN_BOUNDS(r < a.rows, &g_err_norm_grad, SITE_B_NORM_GRAD))
        store8(static_cast<XT*>(a.dx) + r * a.cols, c, cols, VEC, f);
    }
  }
  if (!ok && t == 0) drain_ring(full, slots, a.rows, a.timeout_ns);
  float* part = a.part + int64_t(blockIdx.x) * 2 * a.cols;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = 8 * (t + i * nt);
    if (c >= cols || !part_in_bounds(a)) break;
    store8(part, c, cols, VEC, dw[i]);
    if constexpr (DB_SHARED) {
      const float4 lo = db_at[2 * i * nt], hi = db_at[(2 * i + 1) * nt];
      const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      store8(part + cols, c, cols, VEC, f);
    } else if (LAYER) {
      store8(part + cols, c, cols, VEC, db[i]);
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
  if (!MXQ_IN_BOUNDS(c < a.cols && blockIdx.y < a.splits, &g_err_norm_grad, SITE_B_NORM_GRAD))
    return;
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
    if (out && MXQ_IN_BOUNDS(c < cols, &g_err_norm_grad, SITE_B_NORM_GRAD)) out[c] = v;
  }
}

// Backward.  The sums of dw and db take 16 registers a chunk beside x and dy:
// four chunks a thread fit for bf16 rows, two for fp32 and for a warp's row.
// One chunk only with few rows, where a row's latency counts: with many, two
// halve the warps of each reduction (9661x1040 bf16: 20.0 us against 25.6, but
// 517x1001 fp32 8.3 against 7.9).
RowPlan backward_plan(int64_t rows, int64_t cols, int x_dtype) {
  const int64_t chunks = (cols + 7) / 8;
  if (chunks <= 64) return {true, 256, chunks <= 32 ? 1 : 2};
  const int least = chunks <= 256 && rows < 4 * sm_count() ? 1 : 2;
  for (int i = least; i <= (x_dtype == MXQ_OUT_BF16 ? 4 : 2); i *= 2)
    if (chunks <= 512 * i)
      return {false, static_cast<int>(((chunks + i - 1) / i + 31) / 32 * 32), i};
  return {false, 256, 0};
}

int grad_ctas_per_sm(const RowPlan& p) { return std::max(1, (p.i == 1 ? 768 : 512) / p.nt); }

// Shared memory behind the ring for the sums of db.
int grad_db_bytes(const RowPlan& p) { return p.i == 4 ? p.nt * 4 * 32 : 0; }

// Rows in flight of a CTA of norm_grad_ring: the shared memory of an SM (208 KB
// of it) split among its CTAs; two at least for every plan it serves.
int grad_slots(const RowPlan& p, int64_t cols, int x_dtype) {
  if (p.warp || !p.i) return 0;
  const int64_t row = ring_row_bytes(cols, x_dtype == MXQ_OUT_BF16 ? 2 : 4);
  const int64_t fit = (208 * 1024 / grad_ctas_per_sm(p) - grad_db_bytes(p)) / (2 * row);
  return static_cast<int>(std::min<int64_t>(fit, N_MAX_SLOTS));
}

// Sets of partial sums.  Register kernels: one per CTA, as many CTAs as the
// registers let an SM hold at once (about 768, 512 and 512 threads with one,
// two and four chunks each), but with few rows no more than one an SM or one
// for eight rows, since each costs a set of sums to write and to join
// (517x1001 fp32, element by element: 11.2 us against 10.6).  Longer rows: enough
// that the column sums fill the device.
int grad_splits(int64_t rows, int64_t cols, int x_dtype) {
  const RowPlan p = backward_plan(rows, cols, x_dtype);
  if (p.i) {
    const int64_t want = int64_t(grad_ctas_per_sm(p)) * sm_count();
    const int64_t few = std::max<int64_t>(sm_count(), rows / (p.warp ? 64 : 8));
    return static_cast<int>(std::min(std::min<int64_t>(p.warp ? (rows + 7) / 8 : rows, want), few));
  }
  const int64_t want = std::max<int64_t>(1, 8 * sm_count() / ((cols + 255) / 256));
  return static_cast<int>(std::min<int64_t>(std::min<int64_t>(rows, want), 512));
}

template <typename XT, typename WT, bool LAYER, int I, bool VEC>
bool launch_ring(const NGrad& a, const RowPlan& p, cudaStream_t st) {
  const auto kernel = norm_grad_ring<XT, WT, LAYER, I, VEC>;
  const size_t smem = size_t(a.slots) * 2 * ring_row_bytes(a.cols, sizeof(XT)) + grad_db_bytes(p);
  return ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem)) &&
         launch_early(kernel, static_cast<unsigned>(a.splits), p.nt, smem, st, a);
}

// The kernels whose rows stay on chip.
template <typename XT, typename WT, bool LAYER, bool VEC>
bool launch_backward(const NGrad& a, const RowPlan& p, cudaStream_t st) {
  if (p.warp) {
    const unsigned grid = static_cast<unsigned>(a.splits);
    return p.i == 1 ? launch_early(norm_grad_regs<XT, WT, LAYER, 1, VEC>, grid, 256, 0, st, a)
                    : launch_early(norm_grad_regs<XT, WT, LAYER, 2, VEC>, grid, 256, 0, st, a);
  }
  if (p.i == 1) return launch_ring<XT, WT, LAYER, 1, VEC>(a, p, st);
  if (p.i == 2) return launch_ring<XT, WT, LAYER, 2, VEC>(a, p, st);
  if constexpr (std::is_same<XT, __nv_bfloat16>::value)
    return launch_ring<XT, WT, LAYER, 4, VEC>(a, p, st);
  return false;   // backward_plan gives four chunks to bf16 alone
}

template <typename XT, typename WT, bool LAYER>
mxq_status run_backward(const NGrad& a, cudaStream_t st) {
  const RowPlan p = backward_plan(a.rows, a.cols, std::is_same<XT, float>::value ? MXQ_OUT_F32
                                                                         : MXQ_OUT_BF16);
  bool ok = true;
  if (p.i) {
    ok = a.vec ? launch_backward<XT, WT, LAYER, true>(a, p, st)
               : launch_backward<XT, WT, LAYER, false>(a, p, st);
  } else {
    // the column sums first: dx may take the place of x or dy
    const unsigned groups = static_cast<unsigned>((a.cols + 255) / 256);
    norm_grad_cols<XT, LAYER><<<dim3(groups, static_cast<unsigned>(a.splits)), 256, 0, st>>>(a);
    norm_grad_rows<XT, WT, LAYER><<<static_cast<unsigned>(a.rows), 256, 0, st>>>(a);
  }
  if (!ok) return MXQ_ERR_CUDA;
  const JoinArgs j{a.part, a.cols, a.splits, a.dweight, a.dbias};
  ok = launch_early(norm_grad_join, static_cast<unsigned>((a.cols + 31) / 32), 1024, 0, st, j);
  return ok ? launch_status() : MXQ_ERR_CUDA;
}

struct Backward {
  const NGrad& a;
  cudaStream_t st;
  template <typename XT, typename WT, bool LAYER>
  mxq_status operator()() const { return run_backward<XT, WT, LAYER>(a, st); }
};

}  // namespace

uint32_t take_norm_grad_error() {
  uint32_t h = 0;
  if (cudaMemcpyFromSymbol(&h, g_err_norm_grad, sizeof(h)) != cudaSuccess) return MXQ_ERR_CUDA;
  if (h) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_err_norm_grad, &z, sizeof(z));
  }
  return h;
}

}  // namespace mxq

using namespace mxq;

extern "C" size_t mxq_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (norm_check(rows, cols, MXQ_NORM_LAYER, MXQ_OUT_F32, MXQ_OUT_F32) != MXQ_OK) return 0;
  if (rows == 0 || cols == 0) return 0;
  const int splits = std::max(grad_splits(rows, cols, MXQ_OUT_BF16),
                              grad_splits(rows, cols, MXQ_OUT_F32));
  return static_cast<size_t>(splits) * 2 * cols * sizeof(float);
}

extern "C" mxq_status mxq_norm_backward(const mxq_norm_grad_args* p, void* stream) {
  if (!p) return MXQ_ERR_ARG;
  mxq_status st = norm_check(p->rows, p->cols, p->kind, p->x_dtype, p->w_dtype);
  if (st != MXQ_OK) return st;
  if (p->cols == 0) return MXQ_OK;
  if (!p->dweight) return MXQ_ERR_ARG;
  if (!aligned4(p->dweight) || !aligned4(p->dbias)) return MXQ_ERR_ALIGN;
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
  if (!aligned16(p->dy) || !aligned16(p->x) || !aligned16(p->weight) || !aligned16(p->dx) ||
      !aligned4(p->mean) || !aligned4(p->rstd))
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
  a.slots = grad_slots(backward_plan(p->rows, p->cols, p->x_dtype), p->cols, p->x_dtype);
  a.timeout_ns = wait_timeout_ns();
  return dispatch(p->x_dtype, p->w_dtype, p->kind, Backward{a, s});
}
