// Product of block-128 FP8 codes on the 5th-generation tensor cores (tcgen05).
//
//   C[m][n] = sum_b sA[b][m] sB(n, b) sum_{k in block b} A[m][k] B[n][k]
//
// The scales are arbitrary fp32 values, so the tensor cores cannot apply them
// (their block scales are powers of two): each K block of 128 is one set of
// MMAs into a fresh fp32 accumulator in tensor memory, which the epilogue
// warps read back, scale and add in fp32 registers.
//
// Few tokens (fp8_gemm_lanes): a CTA computes 128 lines of B x T lines of A,
// with the lines of B as the MMA's 128 rows (tensor-memory lanes), so that a
// product of a few tokens still uses whole instructions.
//   warp 0      TMA producer: 128 bytes of K of both operands per stage;
//   warp 1      allocates tensor memory; one lane issues the four MMAs
//               (kind::f8f6f4, K = 32 each) of every stage;
//   warps 2-5   epilogue: lane = line of B, T accumulators per thread.
#include <string.h>

#include "fp8_common.cuh"
#include "mxq_host.h"
#include "mxq_tc.cuh"

namespace mxq {

__device__ uint32_t g_err_fp8_gemm;

namespace {

struct FArgs {
  const float* sA;
  const float* sB;
  void* C;
  int64_t M, N;
  int64_t lines_a, lines_b;    // floats between the K blocks of line scales
  int32_t nk;                  // K blocks
  int32_t tiles;               // 1: sB holds tile scales, 0: line scales
  int32_t out_bf16;
  uint32_t idesc_fmt;          // element types of the instruction descriptor
  uint64_t timeout_ns;
};

MXQ_DEV void fabort(volatile int* abort_flag, uint32_t site) {
  *abort_flag = 1;
  record_error(&g_err_fp8_gemm, MXQ_ERR_TIMEOUT, site);
}

// Instruction descriptor of kind::f8f6f4 with fp32 accumulation, K-major
// operands, m x n; fmt holds the element types (E4M3 0, E5M2 1) at bits 7, 10.
MXQ_DEV uint32_t idesc_f8(uint32_t fmt, uint32_t m, uint32_t n) {
  return (1u << 4) | fmt | ((n >> 3) << 17) | ((m >> 4) << 24);
}

MXQ_DEV void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

MXQ_DEV void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

MXQ_DEV void tmem_alloc(uint32_t dst_smem, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

MXQ_DEV void tmem_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
               : "memory");
}

#define MXQ_TMEM_LD16(taddr, r)                                                                  \
  asm volatile(                                                                                  \
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "    \
      "%11, %12, %13, %14, %15}, [%16];"                                                         \
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),     \
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), \
        "=r"(r[14]), "=r"(r[15])                                                                 \
      : "r"(taddr))

// ---- 128 lines of B x T lines of A per CTA --------------------------------------
constexpr int L_THREADS = 192;
constexpr int L_WBYTES = 128 * 128;   // a stage's lines of B

template <int T>
struct Lanes {
  static constexpr int NB = T == 128 ? 2 : 4;             // accumulators in tensor memory
  static constexpr uint32_t TMEM = NB * T;                // a power of two, at least 32
  static constexpr int STAGE = L_WBYTES + T * 128;
  static constexpr int STAGES = T == 128 ? 3 : T == 64 ? 4 : 5;   // two CTAs fit in an SM
  static constexpr int SMEM = STAGES * STAGE + 2 * T * 4 + 256 + 1024;
  static_assert(TMEM >= 32 && TMEM <= 256, "two CTAs share an SM's tensor memory");
  static_assert(STAGE % 1024 == 0 && 2 * SMEM <= 227 * 1024, "swizzle atoms, two CTAs");
};

template <int T>
__global__ void __launch_bounds__(L_THREADS)
    fp8_gemm_lanes(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                   const FArgs a) {
  using L = Lanes<T>;
  constexpr int S = L::STAGES, NB = L::NB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* sa = reinterpret_cast<float*>(smem + S * L::STAGE);   // [2][T] scales of A
  uint64_t* full = reinterpret_cast<uint64_t*>(sa + 2 * T);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + NB;
  uint64_t* drain = acc_empty + NB;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n0 = int64_t(blockIdx.x) * 128, m0 = int64_t(blockIdx.y) * T;
  const int nk = a.nk;
  const uint64_t tmo = a.timeout_ns;
  if (threadIdx.x == 0) {
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), 4);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), L::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, phase = 0, issued = 0;
      bool ok = true;
      for (int kb = 0; kb < nk; ++kb) {
        if (!gwait(smem_u32(&empty[s]), phase ^ 1, tmo, abort_flag)) {
          if (!*abort_flag) fabort(abort_flag, SITE_FP8_EMPTY);
          ok = false;
          break;
        }
        const uint32_t st = smem_u32(smem + s * L::STAGE), bar = smem_u32(&full[s]);
        mbar_arrive_expect_tx(bar, L::STAGE);
        tma_load_2d(st, &tb, bar, kb * 128, static_cast<int32_t>(n0));
        tma_load_2d(st + L_WBYTES, &ta, bar, kb * 128, static_cast<int32_t>(m0));
        ++issued;
        if (++s == S) { s = 0; phase ^= 1; }
      }
      if (!ok)   // the copies in flight land before shared memory is released
        for (uint32_t k = issued > S ? issued - S : 0; k < issued; ++k)
          if (!mbar_wait(smem_u32(&full[k % S]), (k / S) & 1, tmo)) break;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_f8(a.idesc_fmt, 128, T);
      uint32_t s = 0, phase = 0;
      for (int kb = 0; kb < nk; ++kb) {
        const int b = kb % NB;
        if (!gwait(smem_u32(&acc_empty[b]), ((kb / NB) & 1) ^ 1, tmo, abort_flag)) {
          if (!*abort_flag) fabort(abort_flag, SITE_FP8_TMEM_EMPTY);
          break;
        }
        if (!gwait(smem_u32(&full[s]), phase, tmo, abort_flag)) {
          if (!*abort_flag) fabort(abort_flag, SITE_FP8_FULL);
          break;
        }
        tc_fence_after();
        const uint32_t st = smem_u32(smem + s * L::STAGE);
        const uint64_t wd = smem_desc(st, 0, 1024, 2), xd = smem_desc(st + L_WBYTES, 0, 1024, 2);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f8(tmem + b * T, wd + 2 * j, xd + 2 * j, idesc, j > 0 ? 1u : 0u);
        tc_commit(smem_u32(&empty[s]));
        tc_commit(smem_u32(&acc_full[b]));
        if (++s == S) { s = 0; phase ^= 1; }
      }
      tc_commit(smem_u32(drain));   // every MMA is complete before teardown
      if (!mbar_wait(smem_u32(drain), 0, tmo))
        record_error(&g_err_fp8_gemm, MXQ_ERR_TIMEOUT, SITE_FP8_DRAIN);
    }
  } else {
    const int quad = warp & 3;                // tensor-memory lane quadrant
    const int et = threadIdx.x - 64;          // epilogue thread
    const int64_t n = n0 + quad * 32 + lane;  // this thread's line of B
    const int64_t m = m0 + et;                // the line of A whose scale it stages
    const int64_t n_kb = nk;
    auto scale_a = [&](int kb) {
      return et < T && m < a.M && kb < nk ? a.sA[kb * a.lines_a + m] : 0.0f;
    };
    auto scale_b = [&](int kb) {
      if (n >= a.N || kb >= nk) return 0.0f;
      return a.tiles ? a.sB[(n >> 7) * n_kb + kb] : a.sB[kb * a.lines_b + n];
    };
    float acc[T];
#pragma unroll
    for (int j = 0; j < T; ++j) acc[j] = 0.0f;
    float next_a = scale_a(0), next_b = scale_b(0);
    bool ok = true;
    for (int kb = 0; kb < nk; ++kb) {
      const int b = kb % NB;
      // two scale buffers and one barrier a block: a warp that stages block
      // kb + 2 has passed barrier kb + 1, which every warp reached after its
      // last read of block kb
      if (et < T) sa[(kb & 1) * T + et] = next_a;
      const float sb = next_b;
      next_a = scale_a(kb + 1);
      next_b = scale_b(kb + 1);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok && !gwait(smem_u32(&acc_full[b]), (kb / NB) & 1, tmo, abort_flag)) {
        if (!*abort_flag) fabort(abort_flag, SITE_FP8_TMEM_FULL);
        ok = false;
      }
      if (!__all_sync(~0u, ok)) {
        ok = false;
        continue;   // keeps the barrier count of the other warps
      }
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + b * T;
#pragma unroll
      for (int c = 0; c < T; c += 16) {
        uint32_t v[16];
        MXQ_TMEM_LD16(taddr + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          acc[c + j] = __fmaf_rn(__uint_as_float(v[j]), sb * sa[(kb & 1) * T + c + j], acc[c + j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[b]));
    }
    if (ok && n < a.N) {
#pragma unroll
      for (int j = 0; j < T; ++j) {
        if (m0 + j >= a.M) break;
        if (!MXQ_IN_BOUNDS(n < a.N && m0 + j < a.M, &g_err_fp8_gemm, SITE_B_FP8_GEMM)) continue;
        const int64_t at = (m0 + j) * a.N + n;
        if (a.out_bf16) static_cast<__nv_bfloat16*>(a.C)[at] = __float2bfloat16_rn(acc[j]);
        else static_cast<float*>(a.C)[at] = acc[j];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, L::TMEM);
}

// The 2-D map of `lines` code lines of K elements, in boxes of 128 x `box`.
bool code_map(CUtensorMap* map, const void* codes, int64_t lines, int64_t K, int box) {
  return tensor_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, static_cast<uint64_t>(K),
                       static_cast<uint64_t>(lines), static_cast<uint64_t>(fp8_pitch(K)), 128,
                       static_cast<uint32_t>(box), CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
}

template <int T>
mxq_status launch_lanes(const void* A, const void* B, int64_t K, const FArgs& a, void* stream) {
  CUtensorMap ta, tb;
  if (!code_map(&ta, A, a.M, K, T) || !code_map(&tb, B, a.N, K, 128)) return MXQ_ERR_CUDA;
  const int64_t gx = (a.N + 127) / 128, gy = (a.M + T - 1) / T;
  if (gy > 65535) return MXQ_ERR_ARG;
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(fp8_gemm_lanes<T>), Lanes<T>::SMEM))
    return MXQ_ERR_CUDA;
  fp8_gemm_lanes<T><<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), L_THREADS,
                      Lanes<T>::SMEM, static_cast<cudaStream_t>(stream)>>>(ta, tb, a);
  return launch_status();
}

}  // namespace

uint32_t take_fp8_gemm_error() {
  uint32_t h = 0;
  if (cudaMemcpyFromSymbol(&h, g_err_fp8_gemm, sizeof(h)) != cudaSuccess) return MXQ_ERR_CUDA;
  if (h) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_err_fp8_gemm, &z, sizeof(z));
  }
  return h;
}

}  // namespace mxq

using namespace mxq;

extern "C" mxq_status mxq_fp8_gemm(const void* A, const float* sA, int fmt_a, const void* B,
                                   const float* sB, int fmt_b, int b_scales, int64_t M, int64_t N,
                                   int64_t K, void* C, int out_dtype, void* stream) {
  const int64_t lim = int64_t(1) << 31;
  if (M < 0 || N < 0 || K < 0 || M >= lim || N >= lim || K >= lim) return MXQ_ERR_ARG;
  if (!is_fp8(fmt_a) || !is_fp8(fmt_b)) return MXQ_ERR_ARG;
  if (b_scales != MXQ_FP8_LINES && b_scales != MXQ_FP8_TILES) return MXQ_ERR_ARG;
  if (out_dtype != MXQ_OUT_F32 && out_dtype != MXQ_OUT_BF16) return MXQ_ERR_ARG;
  if (M == 0 || N == 0) return MXQ_OK;
  if (!C) return MXQ_ERR_ARG;
  if (!aligned16(C)) return MXQ_ERR_ALIGN;
  if (K == 0) {
    const size_t bytes = static_cast<size_t>(M) * N * (out_dtype == MXQ_OUT_BF16 ? 2 : 4);
    return cudaMemsetAsync(C, 0, bytes, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MXQ_OK : MXQ_ERR_CUDA;
  }
  if (!A || !sA || !B || !sB) return MXQ_ERR_ARG;
  if (!aligned16(A) || !aligned16(B) || !aligned16(sA)) return MXQ_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(sB) & (b_scales == MXQ_FP8_LINES ? 15u : 3u)) != 0)
    return MXQ_ERR_ALIGN;
  FArgs a = {};
  a.sA = sA;
  a.sB = sB;
  a.C = C;
  a.M = M;
  a.N = N;
  a.lines_a = fp8_lines(M);
  a.lines_b = fp8_lines(N);
  a.nk = static_cast<int32_t>((K + F_BLOCK - 1) / F_BLOCK);
  a.tiles = b_scales == MXQ_FP8_TILES;
  a.out_bf16 = out_dtype == MXQ_OUT_BF16;
  // the lines of B are the MMA's rows (its A operand)
  a.idesc_fmt = (fmt_b == MXQ_E5M2 ? 1u << 7 : 0u) | (fmt_a == MXQ_E5M2 ? 1u << 10 : 0u);
  a.timeout_ns = wait_timeout_ns();
  if (M <= 16) return launch_lanes<16>(A, B, K, a, stream);
  if (M <= 32) return launch_lanes<32>(A, B, K, a, stream);
  if (M <= 64) return launch_lanes<64>(A, B, K, a, stream);
  return launch_lanes<128>(A, B, K, a, stream);
}
