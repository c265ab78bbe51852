// Block-scaled MX GEMM on the 5th-generation tensor cores (tcgen05).
//
// Operation: "AMD顛覆行業認知！終于攻克FP4大模型訓練致命難題", §02-§03 -- the
// forward, activation-gradient and weight-gradient GEMMs run natively on MX
// (FP8 / FP4) codes, each 32-element block scaled by its E8M0 exponent:
//   C[m][n] = sum_k dec(A[m][k]) 2^(sA[m][k/32]-127) dec(B[n][k]) 2^(sB[n][k/32]-127)
// accumulated in fp32.  E4M3 operands use kind::mxf8f6f4 (one scale per 32
// along K per MMA of K=32); E2M1 operands use kind::mxf4 on packed nibbles
// (two scales per MMA of K=64).
//
// Scales: tcgen05.cp reads them in a chunk layout (for every 128-row x
// 4-block chunk, byte (r % 32) * 16 + (r / 32) * 4 + (kb % 4)).  Scales the
// quantizers wrote in that layout are loaded in place; row-major scales are
// first rewritten into it by a small pre-pass kernel in the caller's
// workspace.  The product's kernel is in gemm_kernel.cuh.
#include <string.h>

#include "gemm_kernel.cuh"

namespace mxq {
namespace {

// A launch: up to G_MAX_GROUP problems of one element format and their
// tensor maps, the work items of problem i numbered from p[i].tile0.  One
// problem is the plain GEMM; several are independent GEMMs that run as one
// persistent grid (e.g. the weight gradients of several layers, which no
// layer waits for), so their tiles fill the waves together.
constexpr int G_MAX_GROUP = 8;
struct GGroup {
  CUtensorMap ta[G_MAX_GROUP], tb[G_MAX_GROUP], tsa[G_MAX_GROUP], tsb[G_MAX_GROUP];
  GArgs p[G_MAX_GROUP];
  int32_t count;
  int32_t n_tiles;              // work items of all problems
};

// Work of such a launch.
struct DenseWork {
  using Params = GGroup;
  static constexpr int STAGES = G_STAGES, TABLE = 0;
  static constexpr bool PARTIAL = false, QUANTIZES = true;
  static constexpr StoreBy OUT = STORE_DIRECT;
  const GGroup& g;
  int p = 0;   // problem of the last item asked for

  MXQ_DEV DenseWork(const GGroup& group, const void*) : g(group) {}
  MXQ_DEV static const GArgs& first(const GGroup& g) { return g.p[0]; }
  MXQ_DEV static void prefetch(const GGroup& g) {
    for (int i = 0; i < g.count; ++i) {
      prefetch_tmap(&g.ta[i]);
      prefetch_tmap(&g.tb[i]);
      prefetch_tmap(&g.tsa[i]);
      prefetch_tmap(&g.tsb[i]);
    }
  }
  MXQ_DEV static void load(const GGroup&, void*) {}
  MXQ_DEV int tiles() const { return g.n_tiles; }
  MXQ_DEV Item at(int t) {
    while (p + 1 < g.count && t >= g.p[p + 1].tile0) ++p;
    const GArgs& a = g.p[p];
    Item it;
    it.a = &a;
    it.ta = &g.ta[p];
    it.tb = &g.tb[p];
    it.tsa = &g.tsa[p];
    it.tsb = &g.tsb[p];
    it.nk = a.nk;
    it.last = 4;
    tile_coords(t - a.tile0, a, it.mp, it.nt);
    it.kx = 0;
    it.ay = it.mp * (G_CLUSTER * G_BM);
    it.by = it.nt * G_BN;
    it.sa = G_CLUSTER * it.mp * a.kc_per_row;
    it.sb = 2 * it.nt * a.kc_per_row;
    it.c0 = 0;
    it.rows = a.M;
    it.z = 0;
    it.pace_ns = a.pace_ns;
    return it;
  }
  [[maybe_unused]] MXQ_DEV static bool inside(const Item& it) {
    return it.mp >= 0 && it.mp < it.a->n_mp && it.nt >= 0 && it.nt < it.a->n_nt;
  }
};

// Row-major E8M0 scales [rows][kb] of A and of B -> chunked tensor-core
// layout, zero padded to rows_p rows and kbp blocks, both operands in one
// launch.  One thread writes the four blocks of one row in one chunk.
struct SfSide {
  const uint8_t* s;
  int64_t rows, rows_p;
  uint8_t* out;
};

__global__ void __launch_bounds__(256)
    sf_to_chunks(SfSide sa, SfSide sb, int64_t kb, int64_t kbp) {
  const int64_t kcs = kbp / 4;
  const int64_t total_a = sa.rows_p * kcs, total = total_a + sb.rows_p * kcs;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * blockDim.x) {
    const bool is_a = i < total_a;
    const SfSide& d = is_a ? sa : sb;
    const int64_t j = is_a ? i : i - total_a;
    const int64_t r = j % d.rows_p, kc = j / d.rows_p;
    uint32_t w = 0;
    if (r < d.rows) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t k = kc * 4 + u;
        if (k < kb) w |= static_cast<uint32_t>(d.s[r * kb + k]) << (8 * u);
      }
    }
    const int64_t rt = r / 128, rr = r % 128;
    if (!MXQ_IN_BOUNDS(r < d.rows_p && kc < kcs && kc * 4 + 3 < kbp, &g_err_gemm,
                       SITE_B_SF_CHUNKS))
      continue;
    uint8_t* chunk = d.out + (rt * kcs + kc) * 512;
    *reinterpret_cast<uint32_t*>(chunk + (rr % 32) * 16 + (rr / 32) * 4) = w;
  }
}

struct Plan {
  int64_t kbytes, kb, kbp, mp, np, ws_a, ws_b;
  int skb;
};

bool make_plan(int64_t M, int64_t N, int64_t K, int fmt, Plan& p) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 32 != 0) return false;
  if (fmt != MXQ_E4M3 && fmt != MXQ_E2M1 && fmt != MXQ_E5M2) return false;
  p.kbytes = fmt != MXQ_E2M1 ? K : K / 2;
  p.kb = K / 32;
  p.skb = fmt != MXQ_E2M1 ? 4 : 8;  // k-blocks per 128-byte stage
  p.kbp = (p.kb + p.skb - 1) / p.skb * p.skb;
  p.mp = (M + G_CLUSTER * G_BM - 1) / (G_CLUSTER * G_BM) * (G_CLUSTER * G_BM);
  p.np = (N + G_BN - 1) / G_BN * G_BN;
  p.ws_a = p.mp * p.kbp;
  p.ws_b = p.np * p.kbp;
  return true;
}

}  // namespace

uint32_t take_gemm_error() {
  uint32_t h = 0;
  if (cudaMemcpyFromSymbol(&h, g_err_gemm, sizeof(h)) != cudaSuccess) return MXQ_ERR_CUDA;
  if (h) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_err_gemm, &z, sizeof(z));
  }
  return h;
}

}  // namespace mxq

using namespace mxq;

extern "C" size_t mxq_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int fmt) {
  Plan p;
  if (!make_plan(M, N, K, fmt, p)) return 0;
  return static_cast<size_t>(p.ws_a + p.ws_b);
}

namespace {

// What the epilogue writes: C as fp32 or bf16, or row-wise MX codes of C
// (q_fmt) with their scales.
struct OutSpec {
  void* C;
  int kind;            // 0: fp32, 1: bf16, 2: MX codes
  int q_fmt;
  uint8_t* q_scales;
  int q_scale_layout;  // mxq_scale_layout of q_scales
};

// The argument checks of one problem: sizes, formats, pointers, alignment,
// workspace.  No CUDA call.
mxq_status gemm_validate(const void* A, const uint8_t* sA, const void* B, const uint8_t* sB,
                         int fmt, int64_t M, int64_t N, int64_t K, const void* C,
                         const void* workspace, size_t workspace_bytes, int scale_layout) {
  Plan p;
  if (!make_plan(M, N, K, fmt, p)) return MXQ_ERR_ARG;
  if (scale_layout != MXQ_SCALES_ROWMAJOR && scale_layout != MXQ_SCALES_TC) return MXQ_ERR_ARG;
  const bool tc = scale_layout == MXQ_SCALES_TC;
  if (!A || !sA || !B || !sB || !C || (!tc && !workspace)) return MXQ_ERR_ARG;
  if (tc && K % (fmt == MXQ_E2M1 ? 256 : 128) != 0) return MXQ_ERR_ARG;
  if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31))
    return MXQ_ERR_ARG;
  if (!aligned16(A) || !aligned16(B) || !aligned16(C)) return MXQ_ERR_ALIGN;
  if (tc && (!aligned16(sA) || !aligned16(sB))) return MXQ_ERR_ALIGN;
  if (!tc && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MXQ_ERR_ALIGN;
  if (!tc && workspace_bytes < static_cast<size_t>(p.ws_a + p.ws_b)) return MXQ_ERR_WORKSPACE;
  return MXQ_OK;
}

// Validates one problem, runs its scale re-layout pass (row-major scales),
// and fills its launch arguments and tensor maps (tile0 left at 0).
mxq_status gemm_prepare(const void* A, const uint8_t* sA, const void* B, const uint8_t* sB,
                        int fmt, int64_t M, int64_t N, int64_t K, const OutSpec& out,
                        void* workspace, size_t workspace_bytes, void* stream, int scale_layout,
                        GArgs& a, CUtensorMap& ta, CUtensorMap& tb, CUtensorMap& tsa,
                        CUtensorMap& tsb) {
  void* C = out.C;
  const mxq_status vs = gemm_validate(A, sA, B, sB, fmt, M, N, K, C, workspace, workspace_bytes,
                                      scale_layout);
  if (vs != MXQ_OK) return vs;
  Plan p;
  make_plan(M, N, K, fmt, p);
  // scales already in the tensor-core chunk layout: no re-layout pass and
  // no workspace; the chunks are read in place
  const bool tc = scale_layout == MXQ_SCALES_TC;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (!tc) {
    const int64_t total = (p.mp + p.np) * (p.kbp / 4);
    const int grid = static_cast<int>(std::min<int64_t>((total + 255) / 256, 4 * sm_count()));
    const SfSide sa{sA, M, p.mp, ws}, sb{sB, N, p.np, ws + p.ws_a};
    sf_to_chunks<<<grid, 256, 0, st>>>(sa, sb, p.kb, p.kbp);
  }

  if (tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, A, static_cast<uint64_t>(p.kbytes),
                    static_cast<uint64_t>(M), static_cast<uint64_t>(p.kbytes), G_BKB, G_BM,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) != CUDA_SUCCESS)
    return MXQ_ERR_CUDA;
  if (tensor_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, B, static_cast<uint64_t>(p.kbytes),
                    static_cast<uint64_t>(N), static_cast<uint64_t>(p.kbytes), G_BKB, G_BN_CTA,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) != CUDA_SUCCESS)
    return MXQ_ERR_CUDA;

  // Scale chunks as 2-D tensors of 512-byte rows (128 x uint32), one row per
  // (128-row tile, k-chunk): a stage loads n_sfa consecutive rows.  The
  // workspace holds chunks for the padded 256-row tiles; caller-provided
  // chunks cover only the existing 128-row tiles, and loads of the missing
  // ones read the zero fill.
  {
    const int n_sfa = fmt == MXQ_E2M1 ? 2 : 1;
    const int64_t kcs = p.kbp / 4;
    for (int which = 0; which < 2; ++which) {
      const int64_t lines = which == 0 ? (tc ? M : p.mp) : (tc ? N : p.np);
      const int64_t rows = (lines + G_BM - 1) / G_BM * kcs;
      const void* base = tc ? static_cast<const void*>(which == 0 ? sA : sB)
                            : static_cast<const void*>(ws + (which == 0 ? 0 : p.ws_a));
      if (tensor_map_2d(which == 0 ? &tsa : &tsb, CU_TENSOR_MAP_DATA_TYPE_UINT32, base, 128,
                        static_cast<uint64_t>(rows), 512, 128, static_cast<uint32_t>(n_sfa),
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) !=
          CUDA_SUCCESS)
        return MXQ_ERR_CUDA;
    }
  }

  a = GArgs{};
  a.M = static_cast<int32_t>(M);
  a.N = static_cast<int32_t>(N);
  a.n_mp = static_cast<int32_t>(p.mp / (G_CLUSTER * G_BM));
  a.n_nt = static_cast<int32_t>(p.np / G_BN);
  // one work item = one 256x256 pair tile (one cluster)
  if (int64_t(a.n_mp) * a.n_nt >= (int64_t(1) << 31)) return MXQ_ERR_ARG;
  a.n_tiles = a.n_mp * a.n_nt;
  choose_raster(a.n_mp, a.n_nt, double(p.mp) * p.kbytes, double(p.np) * p.kbytes,
                double(2 * G_BM) * double(p.kbytes), a.group, a.group_n);
  a.nk = static_cast<int32_t>((p.kbytes + G_BKB - 1) / G_BKB);
  a.kc_per_row = static_cast<int32_t>(p.kbp / 4);
  a.sfa = tc ? sA : ws;
  a.sfb = tc ? sB : ws + p.ws_a;
  a.C = C;
  a.out_bf16 = out.kind == 1;
  a.out_q = out.kind == 2;
  a.q_fmt = out.q_fmt;
  a.q_scales = out.q_scales;
  a.q_scale_words = (reinterpret_cast<uintptr_t>(out.q_scales) & 3u) == 0 && (N / 32) % 4 == 0;
  a.q_scale_tc = out.kind == 2 && out.q_scale_layout == MXQ_SCALES_TC;
  a.fp4 = fmt == MXQ_E2M1;
  // kind::mxf8f6f4 element types: E4M3 = 0, E5M2 = 1; kind::mxf4: E2M1 = 1
  a.elem_code = fmt == MXQ_E4M3 ? 0 : 1;
  // 256-bit stores need 32-byte aligned rows: fp32 rows of N % 8 == 0,
  // bf16 rows of N % 16 == 0, one-byte code rows of N % 32 == 0
  const int wide_mult = out.kind == 0 ? 8 : (out.kind == 1 ? 16 : 32);
  a.wide_stores = (reinterpret_cast<uintptr_t>(C) & 31u) == 0 && N % wide_mult == 0;
  a.pace_ns = pace_of(a.nk, a.fp4 != 0, out.kind == 0 ? 16 : (out.kind == 1 ? 8 : 4));
  a.timeout_ns = wait_timeout_ns();
  // every field the kernel dereferences or divides by is set
  if (!a.C || !a.sfa || !a.sfb || a.nk <= 0 || a.kc_per_row <= 0 || a.group <= 0 ||
      a.n_tiles <= 0 || a.n_nt <= 0 || a.n_mp <= 0 || (a.out_q && !a.q_scales))
    return MXQ_ERR_ARG;

  return MXQ_OK;
}

// Launches the prepared problems g.p[0..count) as one persistent grid.
mxq_status gemm_run(GGroup& g, void* stream) {
  int32_t tiles = 0;
  for (int i = 0; i < g.count; ++i) {
    if (int64_t(tiles) + g.p[i].n_tiles >= (int64_t(1) << 31)) return MXQ_ERR_ARG;
    g.p[i].tile0 = tiles;
    tiles += g.p[i].n_tiles;
  }
  g.n_tiles = tiles;
  if (g.count < 1 || g.count > G_MAX_GROUP || tiles <= 0) return MXQ_ERR_ARG;
  return gemm_kernel_run<DenseWork>(g, tiles, stream);
}

mxq_status gemm_launch(const void* A, const uint8_t* sA, const void* B, const uint8_t* sB, int fmt,
                       int64_t M, int64_t N, int64_t K, const OutSpec& out, void* workspace,
                       size_t workspace_bytes, void* stream, int scale_layout) {
  GGroup g;
  memset(&g, 0, sizeof(g));
  const mxq_status st = gemm_prepare(A, sA, B, sB, fmt, M, N, K, out, workspace, workspace_bytes,
                                     stream, scale_layout, g.p[0], g.ta[0], g.tb[0], g.tsa[0],
                                     g.tsb[0]);
  if (st != MXQ_OK) return st;
  g.count = 1;
  return gemm_run(g, stream);
}

}  // namespace

extern "C" mxq_status mxq_gemm(const void* A, const uint8_t* sA, const void* B, const uint8_t* sB,
                               int fmt, int64_t M, int64_t N, int64_t K, void* C, int out_dtype,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (out_dtype != MXQ_OUT_F32 && out_dtype != MXQ_OUT_BF16) return MXQ_ERR_ARG;
  Plan p;
  if (!make_plan(M, N, K, fmt, p)) return MXQ_ERR_ARG;
  if (N % (out_dtype == MXQ_OUT_F32 ? 4 : 8) != 0) return MXQ_ERR_ALIGN;
  const OutSpec out{C, out_dtype == MXQ_OUT_BF16 ? 1 : 0, 0, nullptr, MXQ_SCALES_ROWMAJOR};
  return gemm_launch(A, sA, B, sB, fmt, M, N, K, out, workspace, workspace_bytes, stream,
                     MXQ_SCALES_ROWMAJOR);
}

extern "C" mxq_status mxq_gemm_ex(const void* A, const uint8_t* sA, const void* B,
                                  const uint8_t* sB, int fmt, int64_t M, int64_t N, int64_t K,
                                  void* C, int out_dtype, int scale_layout, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (out_dtype != MXQ_OUT_F32 && out_dtype != MXQ_OUT_BF16) return MXQ_ERR_ARG;
  Plan p;
  if (!make_plan(M, N, K, fmt, p)) return MXQ_ERR_ARG;
  if (N % (out_dtype == MXQ_OUT_F32 ? 4 : 8) != 0) return MXQ_ERR_ALIGN;
  const OutSpec out{C, out_dtype == MXQ_OUT_BF16 ? 1 : 0, 0, nullptr, MXQ_SCALES_ROWMAJOR};
  return gemm_launch(A, sA, B, sB, fmt, M, N, K, out, workspace, workspace_bytes, stream,
                     scale_layout);
}

extern "C" mxq_status mxq_gemm_quantize(const void* A, const uint8_t* sA, const void* B,
                                        const uint8_t* sB, int fmt, int64_t M, int64_t N,
                                        int64_t K, int out_fmt, void* out_codes,
                                        uint8_t* out_scales, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (out_fmt != MXQ_E4M3 && out_fmt != MXQ_E5M2 && out_fmt != MXQ_E2M1) return MXQ_ERR_ARG;
  if (!out_scales) return MXQ_ERR_ARG;
  Plan p;
  if (!make_plan(M, N, K, fmt, p)) return MXQ_ERR_ARG;
  if (N % 32 != 0) return MXQ_ERR_ARG;
  const OutSpec out{out_codes, 2, out_fmt, out_scales, MXQ_SCALES_ROWMAJOR};
  return gemm_launch(A, sA, B, sB, fmt, M, N, K, out, workspace, workspace_bytes, stream,
                     MXQ_SCALES_ROWMAJOR);
}

extern "C" mxq_status mxq_gemm_quantize_ex(const void* A, const uint8_t* sA, const void* B,
                                           const uint8_t* sB, int fmt, int64_t M, int64_t N,
                                           int64_t K, int scale_layout, int out_fmt,
                                           void* out_codes, uint8_t* out_scales,
                                           int out_scale_layout, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  if (out_fmt != MXQ_E4M3 && out_fmt != MXQ_E5M2 && out_fmt != MXQ_E2M1) return MXQ_ERR_ARG;
  if (out_scale_layout != MXQ_SCALES_ROWMAJOR && out_scale_layout != MXQ_SCALES_TC)
    return MXQ_ERR_ARG;
  if (!out_scales) return MXQ_ERR_ARG;
  Plan p;
  if (!make_plan(M, N, K, fmt, p)) return MXQ_ERR_ARG;
  if (N % 32 != 0) return MXQ_ERR_ARG;
  if (out_scale_layout == MXQ_SCALES_TC) {
    if (N % (out_fmt == MXQ_E2M1 ? 256 : 128) != 0) return MXQ_ERR_ARG;
    if (!aligned16(out_scales)) return MXQ_ERR_ALIGN;
  }
  const OutSpec out{out_codes, 2, out_fmt, out_scales, out_scale_layout};
  return gemm_launch(A, sA, B, sB, fmt, M, N, K, out, workspace, workspace_bytes, stream,
                     scale_layout);
}

extern "C" mxq_status mxq_gemm_grouped(const mxq_gemm_problem* problems, int count, int fmt,
                                       void* stream) {
  if (!problems || count < 1 || count > G_MAX_GROUP) return MXQ_ERR_ARG;
  // every problem is checked before any of them is prepared
  for (int i = 0; i < count; ++i) {
    const mxq_gemm_problem& q = problems[i];
    if (q.out_dtype != MXQ_OUT_F32 && q.out_dtype != MXQ_OUT_BF16) return MXQ_ERR_ARG;
    Plan p;
    if (!make_plan(q.M, q.N, q.K, fmt, p)) return MXQ_ERR_ARG;
    if (q.N % (q.out_dtype == MXQ_OUT_F32 ? 4 : 8) != 0) return MXQ_ERR_ALIGN;
    const mxq_status vs = gemm_validate(q.A, q.sA, q.B, q.sB, fmt, q.M, q.N, q.K, q.C, nullptr, 0,
                                        MXQ_SCALES_TC);
    if (vs != MXQ_OK) return vs;
  }
  GGroup g;
  memset(&g, 0, sizeof(g));
  for (int i = 0; i < count; ++i) {
    const mxq_gemm_problem& q = problems[i];
    const OutSpec out{q.C, q.out_dtype == MXQ_OUT_BF16 ? 1 : 0, 0, nullptr, MXQ_SCALES_ROWMAJOR};
    const mxq_status st = gemm_prepare(q.A, q.sA, q.B, q.sB, fmt, q.M, q.N, q.K, out, nullptr, 0,
                                       stream, MXQ_SCALES_TC, g.p[i], g.ta[i], g.tb[i], g.tsa[i],
                                       g.tsb[i]);
    if (st != MXQ_OK) return st;
  }
  g.count = count;
  return gemm_run(g, stream);
}

// ---------------------------------------------------------------------------
// GEMM without caller-provided scratch
// ---------------------------------------------------------------------------
// Some callers cannot allocate device memory at call time: code embedded in a
// host application that owns the whole device memory pool and hands a plug-in
// only its input and output buffers, or code that runs under a fixed memory
// budget where allocating per call is forbidden.  For them the scale
// re-layout scratch lives in one fixed buffer inside this library.
//
// The buffer is a file-scope device array of kNoAllocScratchBytes (16 MiB).
// Every GPU that loads the library holds it until the process exits.  All
// calls share it and it keeps the previous call's contents; each call
// rewrites every byte it reads, so nothing needs clearing, but calls that
// overlap on the GPU (two streams at once, or two host threads) race on it.
namespace {

constexpr size_t kNoAllocScratchBytes = size_t(16) << 20;
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];

// Device address of g_noalloc_scratch for each device, taken once per device
// with that device current (in host code the array's name is only a
// host-side stand-in, not a device address).
void* noalloc_scratch_ptr(mxq_status* st) {
  static std::mutex mu;
  static void* cache[64] = {nullptr};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    *st = MXQ_ERR_CUDA;
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!cache[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) {
      cudaGetLastError();
      *st = MXQ_ERR_CUDA;
      return nullptr;
    }
    cache[dev] = p;
  }
  *st = MXQ_OK;
  return cache[dev];
}

}  // namespace

extern "C" mxq_status mxq_gemm_noalloc(const void* A, const uint8_t* sA, const void* B,
                                       const uint8_t* sB, int fmt, int64_t M, int64_t N,
                                       int64_t K, void* C, int out_dtype, void* stream) {
  const size_t need = mxq_gemm_workspace_size(M, N, K, fmt);
  if (need == 0) return MXQ_ERR_ARG;
  if (need > kNoAllocScratchBytes) return MXQ_ERR_WORKSPACE;
  mxq_status st;
  void* scratch = noalloc_scratch_ptr(&st);
  if (!scratch) return st;
  return mxq_gemm(A, sA, B, sB, fmt, M, N, K, C, out_dtype, scratch, kNoAllocScratchBytes,
                  stream);
}
