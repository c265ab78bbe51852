// The rows form of the products grouped by expert for experts with few rows each (a
// server's tokens).  The weight's bytes bound it, so the operands change places: 128
// lines of the weight are the tensor cores' M and T tokens their N, and a K stage costs
// an MMA of T columns, where a 256x256 tile computes 256 columns for a handful of rows.
//   out[t][n] = sum_k w[n][k] x[t][k]
// Two CTAs per SM walk the tiles (expert, 128 lines, T tokens), the tokens fastest, so
// that CTAs that share a weight's lines run together.  Two, because a tensor-core
// instruction costs the lane that issues it about 100 cycles, however few its columns, and
// 16 KB of weight take five of them (128 tokens of 8 experts of 64, 4096x4096 E2M1, T 16:
// 93.5 us, 115 us with one CTA and a ring as long).
//   warp 0   TMA: 128 bytes of K of the lines and of the tokens, the lines' scale chunks
//   warp 1   tensor memory; one lane issues the MMAs into two accumulators in turn
//   warps 2-5  epilogue: a line per lane, so that a token's 32 outputs are side by side
//   warp 6   one lane copies each stage's scales into tensor memory
//   warp 7   writes the tokens' scales of each stage where the copy reads them, out of
//            the row-major ones: a launch before this one would cost a single token more
//            than its scales do
#pragma once

#include "gemm_kernel.cuh"

namespace mxq {
namespace {

constexpr int W_THREADS = 256;
constexpr int W_LINES = 128;
constexpr int W_OPERAND = W_LINES * G_BKB;   // a stage's lines of the weight

template <int T>
struct Few {
  // scales: up to two chunks of each operand
  static constexpr int STAGE = W_OPERAND + T * G_BKB + 2048;
  static constexpr int STAGES = T == 16 ? 5 : 4;          // two CTAs fit in an SM
  static constexpr uint32_t SF_COL0 = 2 * T;              // two accumulators before them
  static constexpr uint32_t TMEM = T == 16 ? 128 : 256;
  static constexpr int FIXED = STAGES * STAGE + G_BAR_BYTES + 1024;   // and the table
  static_assert(T % 16 == 0 && SF_COL0 + 16 * STAGES <= TMEM, "tensor memory");
  static_assert(STAGE % 1024 == 0, "swizzle atoms");
  static_assert(2 * (FIXED + 3 * 257 * 4 + 1024) <= 228 * 1024, "two CTAs with 256 experts");
};

MXQ_DEV void tc_cp_sf(uint32_t taddr, uint32_t smem_addr) {
  const uint64_t d = smem_desc(smem_addr, 0, 128, 0);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

MXQ_DEV void mma_mxf8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                      uint32_t sfb, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accum), "r"(sfa), "r"(sfb)
      : "memory");
}

MXQ_DEV void mma_mxf4(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                      uint32_t sfb, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], "
      "p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accum), "r"(sfa), "r"(sfb)
      : "memory");
}

// Four scales of a line from p on, the first in the lowest byte; the n that are left of the
// line where they are fewer.  Any alignment.
MXQ_DEV uint32_t scale_word(const uint8_t* p, int n) {
  if (n >= 4 && (reinterpret_cast<uintptr_t>(p) & 3u) == 0)
    return *reinterpret_cast<const uint32_t*>(p);
  uint32_t w = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u < n) w |= static_cast<uint32_t>(p[u]) << (8 * u);
  return w;
}

// Work is the expert table's walker with tiles of 128 lines by T tokens: at(t) gives an
// Item whose mp counts token tiles and nt tiles of lines.
template <typename Work, int T>
__global__ void __launch_bounds__(W_THREADS, 2)
    mx_gemm_few(const __grid_constant__ typename Work::Params g) {
  using F = Few<T>;
  constexpr int S = F::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * F::STAGE);
  uint64_t* empty = full + S;
  uint64_t* sf_ready = empty + S;
  uint64_t* acc_full = sf_ready + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;           // [2]: MMAs, scale copies
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  void* table = smem + S * F::STAGE + G_BAR_BYTES;
  static_assert((3 * S + 6) * 8 + 8 <= G_BAR_BYTES, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const GArgs& a = Work::first(g);
  if (threadIdx.x == 0) {
    Work::prefetch(g);
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 2);   // the copies and the tokens' scales
      mbar_init(smem_u32(&empty[s]), 1);
      mbar_init(smem_u32(&sf_ready[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), 4);
      mbar_init(smem_u32(&drain[b]), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), F::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  Work::load(g, table);
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const int n_tiles = Work(g, table).tiles(), step = static_cast<int>(gridDim.x);
  const uint64_t tmo = a.timeout_ns;
  const bool fp4 = a.fp4 != 0;
  const int n_sf = fp4 ? 2 : 1;
  const int nk = a.nk;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, phase = 0, issued = 0;
      bool ok = true;
      Work work(g, table);
      for (int t = blockIdx.x; t < n_tiles && ok; t += step) {
        const Item it = work.at(t);
        if (!MXQ_IN_BOUNDS(Work::inside(it), &g_err_gemm, SITE_B_GEMM_TILE)) {
          ok = false;   // the MMA lane then waits out its bounded wait
          break;
        }
        for (int ks = 0; ks < nk; ++ks) {
          if (!gwait(smem_u32(&empty[s]), phase ^ 1, tmo, abort_flag)) {
            if (!*abort_flag) gabort(abort_flag, SITE_GEMM_EMPTY);
            ok = false;
            break;
          }
          const uint32_t st = smem_u32(smem + s * F::STAGE), bar = smem_u32(&full[s]);
          mbar_arrive_expect_tx(bar, W_OPERAND + T * G_BKB + 512u * n_sf);
          tma_load_2d(st, it.tb, bar, ks * G_BKB, it.by);
          tma_load_2d(st + W_OPERAND, it.ta, bar, ks * G_BKB, it.ay);
          const uint32_t sf = st + W_OPERAND + T * G_BKB;
          tma_load_2d(sf, it.tsb, bar, 0, it.sb + ks * n_sf);
          ++issued;
          if (++s == S) { s = 0; phase ^= 1; }
        }
      }
      if (!ok)   // the copies in flight land before shared memory is released
        for (uint32_t k = issued > S ? issued - S : 0; k < issued; ++k)
          if (!mbar_wait(smem_u32(&full[k % S]), (k / S) & 1, tmo)) {
            record_error(&g_err_gemm, MXQ_ERR_TIMEOUT, SITE_GEMM_FULL);
            break;
          }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t idesc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t sf_id = fp4 ? ((2 * j) & 3) : j;
        idesc[j] = idesc_block_scaled(static_cast<uint32_t>(a.elem_code), W_LINES, T, sf_id, sf_id);
      }
      const uint64_t w0 = smem_desc(smem_u32(smem), 0, 1024, 2);
      uint32_t s = 0, phase = 0, i = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < n_tiles && ok; t += step, ++i) {
        const uint32_t b = i & 1;
        if (!gwait(smem_u32(&acc_empty[b]), ((i >> 1) & 1) ^ 1, tmo, abort_flag)) {
          if (!*abort_flag) gabort(abort_flag, SITE_GEMM_TMEM_EMPTY);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + b * T;
        for (int ks = 0; ks < nk; ++ks) {
          if (!gwait(smem_u32(&sf_ready[s]), phase, tmo, abort_flag)) {
            if (!*abort_flag) gabort(abort_flag, SITE_GEMM_FULL);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t wd = w0 + s * (F::STAGE >> 4), xd = wd + (W_OPERAND >> 4);
          const uint32_t sw = tmem + F::SF_COL0 + 16 * s, sx = sw + 8;
          const uint32_t more = ks > 0 ? 1u : 0u;
          if (fp4) {
            mma_mxf4(d, wd, xd, idesc[0], sw, sx, more);
            mma_mxf4(d, wd + 2, xd + 2, idesc[1], sw, sx, 1u);
            mma_mxf4(d, wd + 4, xd + 4, idesc[2], sw + 4, sx + 4, 1u);
            mma_mxf4(d, wd + 6, xd + 6, idesc[3], sw + 4, sx + 4, 1u);
          } else {
            mma_mxf8(d, wd, xd, idesc[0], sw, sx, more);
            mma_mxf8(d, wd + 2, xd + 2, idesc[1], sw, sx, 1u);
            mma_mxf8(d, wd + 4, xd + 4, idesc[2], sw, sx, 1u);
            mma_mxf8(d, wd + 6, xd + 6, idesc[3], sw, sx, 1u);
          }
          tc_commit(smem_u32(&empty[s]));
          if (++s == S) { s = 0; phase ^= 1; }
        }
        if (ok) tc_commit(smem_u32(&acc_full[b]));
      }
      tc_commit(smem_u32(&drain[0]));   // every MMA is complete before teardown
      if (!mbar_wait(smem_u32(&drain[0]), 0, tmo))
        record_error(&g_err_gemm, MXQ_ERR_TIMEOUT, SITE_GEMM_DRAIN);
    }
  } else if (warp == 6) {
    if (lane == 0) {
      uint32_t s = 0, phase = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < n_tiles && ok; t += step)
        for (int ks = 0; ks < nk; ++ks) {
          if (!gwait(smem_u32(&full[s]), phase, tmo, abort_flag)) {
            if (!*abort_flag) gabort(abort_flag, SITE_GEMM_FULL);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sf = smem_u32(smem + s * F::STAGE) + W_OPERAND + T * G_BKB;
          const uint32_t col = tmem + F::SF_COL0 + 16 * s;
          tc_cp_sf(col, sf);
          tc_cp_sf(col + 8, sf + 1024);
          if (fp4) {
            tc_cp_sf(col + 4, sf + 512);
            tc_cp_sf(col + 12, sf + 1536);
          }
          tc_commit(smem_u32(&sf_ready[s]));
          if (++s == S) { s = 0; phase ^= 1; }
        }
      tc_commit(smem_u32(&drain[1]));
      if (!mbar_wait(smem_u32(&drain[1]), 0, tmo))
        record_error(&g_err_gemm, MXQ_ERR_TIMEOUT, SITE_GEMM_DRAIN);
    }
  } else if (warp == 7) {
    // A chunk holds row r's four scales at (r % 32) * 16 + (r / 32) * 4; rows from T on
    // are no columns of the MMAs.  The words of AHEAD stages are loaded together, those of
    // the next ones while these are written.
    constexpr int WORDS = T == 16 ? 1 : 4, AHEAD = T == 16 ? 8 : 4;
    const auto& p = g.prep;
    uint32_t s = 0, phase = 0;
    bool ok = true;
    Work work(g, table);
    for (int t = blockIdx.x; t < n_tiles && ok; t += step) {
      const Item it = work.at(t);
      const int rows = min(it.rows - it.mp * T, T);
      uint32_t next[AHEAD][WORDS], now[AHEAD][WORDS];
      auto place = [&](int i, int& row, int& chunk) {
        row = T == 16 ? lane & 15 : lane + 32 * (i & 1);
        chunk = T == 16 ? lane >> 4 : i >> 1;
      };
      auto load = [&](int ks0) {
#pragma unroll
        for (int b = 0; b < AHEAD; ++b)
#pragma unroll
          for (int i = 0; i < WORDS; ++i) {
            int row, chunk;
            place(i, row, chunk);
            const int block = ((ks0 + b) * n_sf + chunk) * 4;
            next[b][i] = 0u;
            if (row < rows && chunk < n_sf && ks0 + b < nk && block < p.kb)
              next[b][i] = scale_word(p.sa + int64_t(it.ay + row) * p.kb + block, p.kb - block);
          }
      };
      load(0);
      for (int ks0 = 0; ks0 < nk && ok; ks0 += AHEAD) {
#pragma unroll
        for (int b = 0; b < AHEAD; ++b)
#pragma unroll
          for (int i = 0; i < WORDS; ++i) now[b][i] = next[b][i];
        load(ks0 + AHEAD);
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) {
          if (ks0 + b >= nk || !ok) break;
          ok = __all_sync(~0u, gwait(smem_u32(&empty[s]), phase ^ 1, tmo, abort_flag));
          if (!ok) {
            if (lane == 0 && !*abort_flag) gabort(abort_flag, SITE_GEMM_EMPTY);
            break;
          }
          uint8_t* const sf = smem + s * F::STAGE + W_OPERAND + T * G_BKB + 1024;
#pragma unroll
          for (int i = 0; i < WORDS; ++i) {
            int row, chunk;
            place(i, row, chunk);
            if (chunk < n_sf)
              *reinterpret_cast<uint32_t*>(sf + chunk * 512 + (row & 31) * 16 + (row >> 5) * 4) =
                  now[b][i];
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&full[s]));
          if (++s == S) { s = 0; phase ^= 1; }
        }
      }
    }
  } else {
    const int quad = warp & 3;   // tensor-memory lane quadrant
    uint32_t i = 0;
    Work work(g, table);
    for (int t = blockIdx.x; t < n_tiles; t += step, ++i) {
      const Item it = work.at(t);
      const uint32_t b = i & 1;
      if (!gwait(smem_u32(&acc_full[b]), (i >> 1) & 1, tmo, abort_flag)) {
        if (lane == 0 && !*abort_flag) gabort(abort_flag, SITE_GEMM_TMEM_FULL);
        break;
      }
      __syncwarp();
      tc_fence_after();
      uint32_t v[T];
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + b * T;
#pragma unroll
      for (int c = 0; c < T; c += 16) MXQ_TMEM_LD16(taddr + c, (v + c));
#pragma unroll
      for (int c = 0; c < T; c += 16) MXQ_TMEM_WAIT16((v + c));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[b]));
      const int64_t n = int64_t(it.nt) * W_LINES + quad * 32 + lane;
      const int rows = min(it.rows - it.mp * T, T);
      if (n < a.N && MXQ_IN_BOUNDS(Work::inside(it), &g_err_gemm, SITE_B_GEMM_STORE)) {
        const int64_t at = (it.c0 + int64_t(it.mp) * T) * a.N + n;
#pragma unroll
        for (int j = 0; j < T; ++j)
          if (j < rows) {
            const float x = __uint_as_float(v[j]);
            if (a.out_bf16)
              static_cast<__nv_bfloat16*>(a.C)[at + int64_t(j) * a.N] = __float2bfloat16_rn(x);
            else static_cast<float*>(a.C)[at + int64_t(j) * a.N] = x;
          }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, F::TMEM);
}

// Launches the kernel on as many CTAs as the device holds, at most `items`.
template <typename Work, int T>
mxq_status gemm_few_run(const typename Work::Params& g, int64_t items, void* stream) {
  // the table takes what this launch's experts need
  const int smem = Few<T>::FIXED + (Work::table_bytes(g) + 15) / 16 * 16;
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(mx_gemm_few<Work, T>), smem))
    return MXQ_ERR_CUDA;
  // Of an SM's 228 KB a CTA takes its own and 1 KB: the table of 640 experts (T 64; T 16:
  // 981) and more leaves room for one.  A second half of the grid that waited for the first
  // to end took 339 us where one takes 281 (1024 experts of 8 rows, 1024x1024 E4M3).
  const int per_sm = 2 * (smem + 1024) <= 228 * 1024 ? 2 : 1;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, per_sm * sm_count()));
  if (!launch_early(mx_gemm_few<Work, T>, grid, W_THREADS, smem, static_cast<cudaStream_t>(stream),
                    g))
    return MXQ_ERR_CUDA;
  return launch_status();
}

}  // namespace
}  // namespace mxq
