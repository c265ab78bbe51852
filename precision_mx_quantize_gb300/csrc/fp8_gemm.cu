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
//   warp 1      allocates tensor memory and issues the four MMAs
//               (kind::f8f6f4, K = 32 each) of every stage;
//   warps 2-5   epilogue: lane = line of B, T accumulators per thread.
// Up to eight CTAs of a cluster share the K blocks of a tile and join their sums
// in order through distributed shared memory.  Bound by the weight's bytes:
// 1x4096x14336 runs in 11.9 us, 0.73 of the HBM copy rate.
//
// Larger products (fp8_gemm_pair): clusters of two CTAs run the pair MMA
// (cta_group::2) on 256x256 tiles, persistent over tiles.  Two accumulators of
// 256 columns fill tensor memory: the MMAs of one K block run while the other
// block's accumulator is read back.
//   warp 0      (both CTAs) TMA producer: own 128 lines of A and of B;
//   warp 1      (both CTAs) tensor memory; the leader's issues the MMAs;
//   warp 2      (both CTAs) scales of the coming K blocks into shared memory;
//   warps 4-11  (both CTAs) accumulation: a thread owns 128 elements of C in
//               registers for the whole K loop, adds each K block with one
//               multiply-add per element (line scales of B: one more multiply),
//               and hands them to a TMA store through shared memory.
// Few tiles with a long K are shared: up to four pairs of a cluster take a part
// of the K blocks each and join their sums in order through distributed shared
// memory (512x4096x14336 31 us, 46 without).
// Bound by the round trip of an accumulator: MMAs (512 cycles), commit, the
// read-back with its additions (360 cycles for a warp's 128 columns), hand-over
// and the next MMAs' start take about 1600 cycles, and tensor memory holds two
// accumulators, so a K block takes 800 (1250 with line scales).  Three of 160
// columns were slower still: the accumulation warps' fixed cost per block
// weighs more (8192x6144x4096 176 us); so were sixteen accumulation warps of 64
// columns (165 us; with line scales no different).  In runs of seconds the
// card's power limit (1400 W) binds as well, for 5 % more.  Measured:
// 8192x6144x4096, tile scales, bf16 out 151 us (2.73 PFLOP/s, 0.70 of twice the
// bf16 rate; the MMAs alone, nothing read back, 118 us); 28672x4096x8192, line
// scales, fp32 out 935-980 us (2.0 PFLOP/s, 0.52).
#include <string.h>

#include <mutex>

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
  uint32_t n_nt, split;        // fp8_gemm_lanes: 128-line tiles of B, CTAs that share one
  int32_t out_bf16;
  uint32_t idesc_fmt;          // element types of the instruction descriptor
  uint64_t timeout_ns;
};

// The warp's index, known to be the same in all of its lanes.
MXQ_DEV int warp_index() { return __shfl_sync(~0u, static_cast<int>(threadIdx.x >> 5), 0); }

// True in one lane of a converged warp.
MXQ_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// A bounded wait that also gives up once another role of this CTA has aborted.
// CTA scope: what the phase guards is tensor memory, or shared memory that
// only the tensor cores and the copy engine touch, so no wait has to order
// other CTAs' ordinary stores.  The timer is read once in 64 polls.  A poll
// that succeeds at once costs 54 cycles in this form and 172 as a nested loop.
MXQ_DEV bool fwait_more(uint32_t bar, uint32_t parity, uint64_t limit,
                        volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
    if ((n & 63u) != 0) continue;
    const uint64_t t = global_ns();
    if (t0 == 0) t0 = t;
    if (*abort_flag || t - t0 > limit) return false;
  }
  return true;
}

MXQ_DEV bool fwait(uint32_t bar, uint32_t parity, uint64_t limit, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || fwait_more(bar, parity, limit, abort_flag);
}

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

// The wait of a role that runs on to its end whatever happens: when the limit
// runs out it records the error, and every later wait of the CTA passes at
// once.  Its warps then need no vote on a result before each warp-wide
// instruction (a vote and its branch cost as much as the wait).
MXQ_DEV void fwait_or_abort(uint32_t bar, uint32_t parity, uint64_t limit,
                            volatile int* abort_flag, uint32_t site) {
  if (mbar_try_wait(bar, parity)) return;
  if (*abort_flag) return;
  if (!fwait_more(bar, parity, limit, abort_flag) && !*abort_flag) fabort(abort_flag, site);
}

// Arrivals of one lane, predicated instead of branched around.
MXQ_DEV void arrive_if(bool p, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(static_cast<uint32_t>(p))
      : "memory");
}

// On a barrier that may live in another CTA; relaxed, as the accumulator's
// loads are complete and nothing else is ordered by it.
MXQ_DEV void arrive_remote_if(bool p, uint32_t cluster_bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_bar),
      "r"(static_cast<uint32_t>(p))
      : "memory");
}

// Waits for this thread's tensor-memory loads; the registers pass through, so
// that no use of them can move above the wait.
#define MXQ_TMEM_WAIT16(r)                                                                       \
  asm volatile("tcgen05.wait::ld.sync.aligned;"                                                  \
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),         \
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),       \
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])                              \
               :                                                                                 \
               : "memory")

// ---- 128 lines of B x T lines of A per CTA --------------------------------------
constexpr int L_THREADS = 192;
constexpr int L_WBYTES = 128 * 128;   // a stage's lines of B
constexpr int L_MAX_SPLIT = 8;        // CTAs of a cluster that share a tile's K blocks

template <int T>
struct Lanes {
  static constexpr int NB = 4;                            // accumulators in tensor memory
  static constexpr uint32_t TMEM = NB * T;                // a power of two, at least 32
  // K blocks whose scales are loaded together
  static constexpr int GROUP = 8;
  static constexpr int STAGE = L_WBYTES + T * 128;
  static constexpr int STAGES = T == 64 ? 4 : 5;          // two CTAs fit in an SM
  static constexpr int SMEM = STAGES * STAGE + 2 * GROUP * T * 4 + 256 + 1024;
  static_assert(TMEM >= 32 && TMEM <= 256, "two CTAs share an SM's tensor memory");
  static_assert(STAGE % 1024 == 0 && 2 * (SMEM + 1024) <= 228 * 1024, "swizzle atoms, two CTAs");
  static_assert(T * 128 * 4 <= STAGES * STAGE, "partial sums fit in the ring");
};

MXQ_DEV float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <int T>
__global__ void __launch_bounds__(L_THREADS, 2)
    fp8_gemm_lanes(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                   const FArgs a) {
  using L = Lanes<T>;
  constexpr int S = L::STAGES, NB = L::NB, G = L::GROUP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* sa = reinterpret_cast<float*>(smem + S * L::STAGE);   // [2][G][T] scales of A
  uint64_t* full = reinterpret_cast<uint64_t*>(sa + 2 * G * T);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + NB;
  uint64_t* drain = acc_empty + NB;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t split = a.split, rank = blockIdx.x % split;
  const uint32_t tile = blockIdx.x / split;
  const int64_t n0 = int64_t(tile % a.n_nt) * 128, m0 = int64_t(tile / a.n_nt) * T;
  // this CTA's K blocks
  const int kb0 = static_cast<int>(int64_t(a.nk) * rank / split);
  const int nk = static_cast<int>(int64_t(a.nk) * (rank + 1) / split) - kb0;
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
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  float acc[T];

  if (warp == 0) {
    const bool one = elect_one();
    uint32_t s = 0, phase = 0, issued = 0;
    bool ok = true;
    for (int kb = 0; kb < nk; ++kb) {
      if (!fwait(smem_u32(&empty[s]), phase ^ 1, tmo, abort_flag)) {
        if (one && !*abort_flag) fabort(abort_flag, SITE_FP8_EMPTY);
        ok = false;
        break;
      }
      const uint32_t st = smem_u32(smem + s * L::STAGE), bar = smem_u32(&full[s]);
      if (one) {
        mbar_arrive_expect_tx(bar, L::STAGE);
        tma_load_2d(st, &tb, bar, (kb0 + kb) * 128, static_cast<int32_t>(n0));
        tma_load_2d(st + L_WBYTES, &ta, bar, (kb0 + kb) * 128, static_cast<int32_t>(m0));
      }
      ++issued;
      if (++s == S) { s = 0; phase ^= 1; }
    }
    if (one && !ok)   // the copies in flight land before shared memory is released
      for (uint32_t k = issued > S ? issued - S : 0; k < issued; ++k)
        if (!mbar_wait(smem_u32(&full[k % S]), (k / S) & 1, tmo)) break;
  } else if (warp == 1) {
    const bool one = elect_one();
    const uint32_t idesc = idesc_f8(a.idesc_fmt, 128, T);
    const uint64_t d0 = smem_desc(smem_u32(smem), 0, 1024, 2);
    uint32_t s = 0, phase = 0;
    for (int kb = 0; kb < nk; ++kb) {
      const int b = kb % NB;
      const uint64_t wd = d0 + s * (L::STAGE >> 4), xd = wd + (L_WBYTES >> 4);
      if (!fwait(smem_u32(&acc_empty[b]), ((kb / NB) & 1) ^ 1, tmo, abort_flag)) {
        if (one && !*abort_flag) fabort(abort_flag, SITE_FP8_TMEM_EMPTY);
        break;
      }
      if (!fwait(smem_u32(&full[s]), phase, tmo, abort_flag)) {
        if (one && !*abort_flag) fabort(abort_flag, SITE_FP8_FULL);
        break;
      }
      tc_fence_after();
      if (one) {
        mma_f8(tmem + b * T, wd, xd, idesc, 0u);
        mma_f8(tmem + b * T, wd + 2, xd + 2, idesc, 1u);
        mma_f8(tmem + b * T, wd + 4, xd + 4, idesc, 1u);
        mma_f8(tmem + b * T, wd + 6, xd + 6, idesc, 1u);
        tc_commit(smem_u32(&acc_full[b]));
        tc_commit(smem_u32(&empty[s]));
      }
      if (++s == S) { s = 0; phase ^= 1; }
    }
    if (one) {   // every MMA is complete before teardown
      tc_commit(smem_u32(drain));
      if (!mbar_wait(smem_u32(drain), 0, tmo))
        record_error(&g_err_fp8_gemm, MXQ_ERR_TIMEOUT, SITE_FP8_DRAIN);
    }
  } else {
    const int quad = warp & 3;                // tensor-memory lane quadrant
    const int et = threadIdx.x - 64;          // epilogue thread
    const int64_t n = n0 + quad * 32 + lane;  // this thread's line of B
    // Scales come in groups of G K blocks, loaded one group ahead (a load
    // takes longer than the copy of a block): those of A through shared
    // memory, those of this thread's line of B in registers.
    constexpr int NA = (G * T + 127) / 128;
    float next_a[NA], next_b[G], sb[G];
    auto load = [&](int kb) {
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        const int e = et + 128 * i, k = kb + e / T;
        const int64_t m = m0 + e % T;
        next_a[i] = e < G * T && k < nk && m < a.M ? a.sA[(kb0 + k) * a.lines_a + m] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int64_t k = kb0 + kb + i;
        next_b[i] = 0.0f;
        if (kb + i < nk && n < a.N)
          next_b[i] = a.tiles ? a.sB[(n >> 7) * a.nk + k] : a.sB[k * a.lines_b + n];
      }
    };
#pragma unroll
    for (int j = 0; j < T; ++j) acc[j] = 0.0f;
    load(0);
    for (int g = 0; g < nk; g += G) {
      // two buffers and one barrier a group: a warp that stages group k + 2
      // has passed barrier k + 1, which every warp reached after its last read
      // of group k
      float* buf = sa + ((g / G) & 1) * G * T;
#pragma unroll
      for (int i = 0; i < NA; ++i)
        if (et + 128 * i < G * T) buf[et + 128 * i] = next_a[i];
#pragma unroll
      for (int i = 0; i < G; ++i) sb[i] = next_b[i];
      load(g + G);
      asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int kb = g + i, b = kb % NB;
        if (kb >= nk) break;
        fwait_or_abort(smem_u32(&acc_full[b]), (kb / NB) & 1, tmo, abort_flag, SITE_FP8_TMEM_FULL);
        __syncwarp();
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + b * T;
#pragma unroll
        for (int c = 0; c < T; c += 16) {
          uint32_t v[16];
          MXQ_TMEM_LD16(taddr + c, v);
          MXQ_TMEM_WAIT16(v);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[c + j] = __fmaf_rn(__fmul_rn(__uint_as_float(v[j]), sb[i]), buf[i * T + c + j],
                                   acc[c + j]);
        }
        tc_fence_before();
        __syncwarp();
        arrive_if(lane == 0, smem_u32(&acc_empty[b]));
      }
    }
  }

  auto store = [&](int64_t row, int64_t col, float v) {
    if (!MXQ_IN_BOUNDS(row < a.M && col < a.N, &g_err_fp8_gemm, SITE_B_FP8_GEMM)) return;
    if (a.out_bf16) static_cast<__nv_bfloat16*>(a.C)[row * a.N + col] = __float2bfloat16_rn(v);
    else static_cast<float*>(a.C)[row * a.N + col] = v;
  };
  // [T][128] partial sums, over the ring: every MMA and copy of this CTA is
  // complete once its last accumulator is
  float* part = reinterpret_cast<float*>(smem);
  const int col = (warp & 3) * 32 + lane;
  if (warp >= 2) {
    if (split == 1) {
      if (n0 + col < a.N && !*abort_flag) {
#pragma unroll
        for (int j = 0; j < T; ++j)
          if (m0 + j < a.M) store(m0 + j, n0 + col, acc[j]);
      }
    } else if (!*abort_flag) {
#pragma unroll
      for (int j = 0; j < T; ++j) part[j * 128 + col] = acc[j];
    }
  }
  tc_fence_before();
  if (split == 1) __syncthreads();
  else cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, L::TMEM);
  if (split == 1) return;
  // Each CTA adds up a share of the tile's lines of A, over the CTAs in order.
  if (warp >= 2 && n0 + col < a.N) {
    const uint32_t mine = smem_u32(part + col);
    for (int j = rank; j < T && m0 + j < a.M; j += split) {
      float v[L_MAX_SPLIT], sum = 0.0f;
#pragma unroll
      for (int r = 0; r < L_MAX_SPLIT; ++r)
        v[r] = r < split ? ld_cluster(map_to_rank(mine + j * 512, r)) : 0.0f;
#pragma unroll
      for (int r = 0; r < L_MAX_SPLIT; ++r) sum += v[r];
      store(m0 + j, n0 + col, sum);
    }
  }
  cluster_sync();   // no CTA leaves while a peer may still read its sums
}

// ---- 256 x 256 tiles on CTA pairs ------------------------------------------------
constexpr int P_THREADS = 384;                   // one control and two accumulation warpgroups
constexpr int P_CTRL_REGS = 104, P_ACC_REGS = 200;
// the split below is drawn from the registers the block is launched with
constexpr int P_MIN_REGS = (128 * P_CTRL_REGS + 256 * P_ACC_REGS + P_THREADS - 1) / P_THREADS;
constexpr int P_OPERAND = 128 * 128;             // a stage's lines of A, or of B, of one CTA
constexpr int P_STAGE = 2 * P_OPERAND;

template <bool LINES>
struct Pair {
  // a K block's scales: [128] rows and [256] columns, or the two products of
  // row and tile scale [2][128]
  static constexpr int SLOT = LINES ? 384 : 256;          // floats
  static constexpr int SLOTS = 16;                        // two groups of eight
  static constexpr int SCALES = SLOTS * SLOT * 4;
  // Four stages run as fast as six (a K block takes longer than a quarter of a
  // stage's turnaround), and leave room for the tiles on their way out.
  static constexpr int STAGES = 4;
  static constexpr int OUT = 2 * 32768;                   // per half tile, 32 KB
  static constexpr int SMEM = STAGES * P_STAGE + OUT + SCALES + 512 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
};

struct PArgs {
  FArgs f;
  int32_t n_mp, n_nt, n_tiles;   // 256-row and 256-column tiles
  int32_t group, group_n;        // tile order (tile_coords)
  int32_t split;                 // pairs of a cluster that share a tile's K blocks
};

// Pairs of a cluster that share a tile leave their sums in shared memory, rows of
// 256 columns this many floats apart: the stores below then meet no bank twice,
// and rows keep to 16 bytes.
constexpr int P_MAX_SPLIT = 4;
template <bool LINES>
constexpr int part_pitch() { return LINES ? 264 : 260; }
static_assert(128 * 264 * 4 <= Pair<true>::STAGES * P_STAGE + Pair<true>::OUT, "over the ring");

MXQ_DEV void mma_f8_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

MXQ_DEV float lds32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Sixteen accumulator words of this thread: tiles, 16 columns of its row;
// lines, the 16 x 256-bit fragments of 32 columns -- rows lane / 4 and 8 more,
// columns 2 (lane % 4) and the next of each group of 8.
template <bool LINES>
MXQ_DEV void load16(uint32_t taddr, uint32_t (&v)[16]) {
  if constexpr (LINES)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
  else
    MXQ_TMEM_LD16(taddr, v);
}

// Tensor-memory address offset of step c of a half tile.
template <bool LINES>
MXQ_DEV uint32_t step16(int c) {
  return LINES ? (c >> 1) * 32 + (static_cast<uint32_t>((c & 1) * 16) << 16) : 16 * c;
}

// acc += s * v for a row of tile scales.  s is the product of the row's scale and
// the tile's, formed once for the row's 128 columns: one operation an element.
// A subnormal s has lost digits, an infinite one makes a NaN of a zero sum; the
// header states that range.  Taking the factors in turn where s is not normal
// cost every call a tenth (8192x6144x4096: 169 us against 152) and those with
// rows of zeros, whose scale is 2^-126, a third (208).
MXQ_DEV void add16(float* acc, const uint32_t (&v)[16], float s) {
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = __fmaf_rn(__uint_as_float(v[j]), s, acc[j]);
}

// Two packed fp32 values.
MXQ_DEV uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}

// acc += row * col * v for a fragment: two rows (each scale twice), the
// columns' scales in col.  Packed pairs: half the instructions of the 256
// multiplies and additions a thread has per K block, whose issue bounds the
// kernel with line scales (28672x4096x8192: 931 us against 1040 unpacked).
MXQ_DEV void add16(float* acc, const uint32_t (&v)[16], uint64_t lo, uint64_t hi,
                   const uint64_t (&col)[4]) {
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    uint64_t x = pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
    uint64_t c = pack2(acc[j], acc[j + 1]);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(x), "l"(col[j >> 2]));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(c) : "l"(x), "l"((j & 2) ? hi : lo), "l"(c));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[j]), "=f"(acc[j + 1]) : "l"(c));
  }
}

// This thread's scales of 32 columns: 2 (lane % 4) and the next of each group
// of 8.
MXQ_DEV void load_cols(uint32_t addr, uint64_t (&col)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(col[q]) : "r"(addr + 32 * q) : "memory");
}

// Place in a half tile of this thread's accumulator j: tiles, one row of 128
// columns; lines, the fragments of load16.
template <bool LINES>
MXQ_DEV int acc_row(int j, int lane) {
  return LINES ? ((j >> 4) & 1) * 16 + ((j >> 1) & 1) * 8 + (lane >> 2) : lane;
}
template <bool LINES>
MXQ_DEV int acc_col(int j, int lane) {
  return LINES ? (j >> 5) * 32 + ((j >> 2) & 3) * 8 + 2 * (lane & 3) + (j & 1) : j;
}

MXQ_DEV void sts(uint32_t addr, uint32_t a) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
}
MXQ_DEV void sts(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
MXQ_DEV void sts(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

MXQ_DEV uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// Writes a half tile, rounded to C's type, as boxes of 128 rows x 128 bytes
// with the 128-byte swizzle of the output's tensor map.  fp32 takes two passes
// of 64 columns.
template <bool LINES>
MXQ_DEV void stage_out(const float (&acc)[128], uint32_t out, int quad, int lane, bool bf16,
                       int pass) {
  auto place = [&](int row, int byte) {   // byte: within the pass's columns
    const int r = quad * 32 + row;
    return out + (byte >> 7) * 16384 + r * 128 + ((byte & 127) ^ ((r & 7) << 4));
  };
  if (bf16) {
#pragma unroll
    for (int j = 0; j < 128; j += LINES ? 2 : 8) {
      const uint32_t at = place(acc_row<LINES>(j, lane), 2 * acc_col<LINES>(j, lane));
      const uint32_t w = bf16x2(acc[j], acc[j + 1]);
      if constexpr (LINES)
        sts(at, w);
      else
        sts(at, w, bf16x2(acc[j + 2], acc[j + 3]), bf16x2(acc[j + 4], acc[j + 5]),
            bf16x2(acc[j + 6], acc[j + 7]));
    }
  } else {
#pragma unroll
    for (int u = 0; u < 64; u += LINES ? 2 : 4) {
      // both passes' registers are named at compile time
      const float a = pass ? acc[64 + u] : acc[u], b = pass ? acc[65 + u] : acc[u + 1];
      const uint32_t at = place(acc_row<LINES>(u, lane), 4 * acc_col<LINES>(u, lane));
      if constexpr (LINES)
        sts(at, __float_as_uint(a), __float_as_uint(b));
      else
        sts(at, __float_as_uint(a), __float_as_uint(b),
            __float_as_uint(pass ? acc[66 + u] : acc[u + 2]),
            __float_as_uint(pass ? acc[67 + u] : acc[u + 3]));
    }
  }
}

MXQ_DEV uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

// An element that copy_out is about to store; its row and column are in C.
MXQ_DEV bool copy_in_bounds(const FArgs& a, int64_t row, int64_t col) {
  return MXQ_IN_BOUNDS(row < a.M && col < a.N, &g_err_fp8_gemm, SITE_B_FP8_GEMM);
}

// Copies a staged pass out to rows of C that no tensor map can describe (not
// 16-byte multiples): each warp its 32 rows, neighbouring lanes neighbouring
// columns, in 4-byte stores (bf16 with an odd N: from the row's first even place
// in C on).  Four rows are read before any is stored: where each store waited
// for its own shared-memory load, 4096x4095x512 with fp32 out took 79 us against
// 44 (sixteen rows 48; 4096x4096x512, by TMA, 21).  col0 < N: the first element of
// an odd row is stored without a test of its column.
template <bool BF16>
MXQ_DEV void copy_out(const FArgs& a, uint32_t out, int quad, int lane, int64_t row0,
                      int64_t col0) {
  constexpr int ROWS = 4;
  const bool odd = BF16 && (a.N & 1);
#pragma unroll 1
  for (int i0 = 0; i0 < 32; i0 += ROWS) {
    uint32_t v[ROWS][2], head[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int r = quad * 32 + i0 + i, skew = (r & 7) << 4;
      const int shift = odd ? static_cast<int>((row0 + r) & 1) : 0;   // col0 * 2 is even
      auto at = [&](int byte) { return out + (byte >> 7) * 16384 + r * 128 + ((byte & 127) ^ skew); };
      head[i] = odd ? lds16(at(0)) : 0u;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int byte = (k * 32 + lane) * 4 + 2 * shift;
        if (odd)
          v[i][k] = lds16(at(byte)) | lds16(at(min(byte + 2, 254))) << 16;
        else
          v[i][k] = __float_as_uint(lds32(at(byte)));
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int64_t row = row0 + quad * 32 + i0 + i;
      const int shift = odd ? static_cast<int>(row & 1) : 0;
      if (row >= a.M) continue;
      if constexpr (BF16) {
        uint16_t* to = static_cast<uint16_t*>(a.C) + row * a.N + col0;
        if (shift && lane == 0 && copy_in_bounds(a, row, col0))
          to[0] = static_cast<uint16_t>(head[i]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = (k * 32 + lane) * 2 + shift;
          if (c < 127 && col0 + c + 1 < a.N) {
            if (copy_in_bounds(a, row, col0 + c + 1))
              *reinterpret_cast<uint32_t*>(to + c) = v[i][k];
          } else if (c < 128 && col0 + c < a.N) {
            if (copy_in_bounds(a, row, col0 + c)) to[c] = static_cast<uint16_t>(v[i][k]);
          }
        }
      } else {
        uint32_t* to = static_cast<uint32_t*>(a.C) + row * a.N + col0;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (col0 + k * 32 + lane < a.N && copy_in_bounds(a, row, col0 + k * 32 + lane))
            to[k * 32 + lane] = v[i][k];
      }
    }
  }
}

// Two neighbouring elements of C from an even column on.
MXQ_DEV void store2(const FArgs& a, int64_t row, int64_t col, float x, float y) {
  if (col >= a.N || !MXQ_IN_BOUNDS(row < a.M, &g_err_fp8_gemm, SITE_B_FP8_GEMM)) return;
  const int64_t at = row * a.N + col;
  const bool two = col + 1 < a.N;
  if (a.out_bf16) {
    __nv_bfloat16* c = static_cast<__nv_bfloat16*>(a.C) + at;
    if (a.N % 2 == 0) {
      *reinterpret_cast<uint32_t*>(c) = bf16x2(x, y);
    } else {
      c[0] = __float2bfloat16_rn(x);
      if (two) c[1] = __float2bfloat16_rn(y);
    }
  } else {
    float* c = static_cast<float*>(a.C) + at;
    if (a.N % 2 == 0) {
      *reinterpret_cast<float2*>(c) = make_float2(x, y);
    } else {
      c[0] = x;
      if (two) c[1] = y;
    }
  }
}

// Four, from a column that is a multiple of four.
MXQ_DEV void store4(const FArgs& a, int64_t row, int64_t col, float4 v) {
  if (col >= a.N || !MXQ_IN_BOUNDS(row < a.M, &g_err_fp8_gemm, SITE_B_FP8_GEMM)) return;
  if (a.N % 4 == 0) {
    const int64_t at = row * a.N + col;
    if (a.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.C) + at) =
          make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(a.C) + at) = v;
  } else {
    store2(a, row, col, v.x, v.y);
    store2(a, row, col + 2, v.z, v.w);
  }
}

MXQ_DEV float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// A barrier of `threads` threads that says, to all of them alike, whether any of
// them saw the CTA abort: on their own readings of the flag some would leave and
// some wait for them.
MXQ_DEV bool sync_any(int id, int threads, bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(v))
      : "memory");
  return any != 0;
}

MXQ_DEV void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}

// How the sums of a tile leave: by TMA where the rows of C are 16-byte multiples,
// else copied; or shared, by p.split pairs of a cluster that take a part of the
// K blocks each and join their sums in order through distributed shared memory.
// A kernel each: with the copies in it, the one for TMA spilled registers
// (8192x6144x4096 153 us against 151).
enum : int { P_TMA = 0, P_COPY = 1, P_SHARED = 2 };

template <bool LINES, int OUT>
__global__ void __launch_bounds__(P_THREADS, 1)
    fp8_gemm_pair(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                  const __grid_constant__ CUtensorMap tc, const PArgs p) {
  using P = Pair<LINES>;
  constexpr int S = P::STAGES, PITCH = part_pitch<LINES>();
  constexpr bool SPLIT = OUT == P_SHARED;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* out = smem + S * P_STAGE;
  float* scales = reinterpret_cast<float*>(out + P::OUT);
  uint64_t* full = reinterpret_cast<uint64_t*>(out + P::OUT + P::SCALES);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* sc_full = acc_full + 4;
  uint64_t* acc_empty = sc_full + 2;    // leader: both CTAs have read the accumulator
  uint64_t* sc_empty = acc_empty + 2;
  uint64_t* drain = sc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // leader: the K blocks the peer's producer issued, once it has stopped
  volatile uint32_t* peer_issued = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);
  constexpr uint32_t kNotYet = 0xFFFFFFFFu;

  const FArgs& a = p.f;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank();
  const uint32_t rank = SPLIT ? crank & 1 : crank;     // in the pair
  const uint32_t first_rank = crank - rank;            // the leader's in the cluster
  const int pair = crank >> 1, split = SPLIT ? p.split : 1;
  const uint16_t both = static_cast<uint16_t>(0x3 << first_rank);
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
    if (OUT == P_TMA) prefetch_tmap(&tc);
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);    // leader: one arrival, bytes of both CTAs
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int g = 0; g < 4; ++g) mbar_init(smem_u32(&acc_full[g]), 1);
    for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&acc_empty[b]), 16);   // 8 warps of each CTA
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sc_full[i]), 1);
      mbar_init(smem_u32(&sc_empty[i]), 8);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    *peer_issued = kNotYet;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
  tc_fence_before();
  cluster_sync();   // barriers of both CTAs exist before anyone signals the peer
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const int cid = blockIdx.x / (2 * split), ncl = gridDim.x / (2 * split);
  const uint32_t tmem = *tmem_slot;
  // this pair's K blocks
  const int k0 = SPLIT ? static_cast<int>(int64_t(a.nk) * pair / split) : 0;
  const int nk = SPLIT ? static_cast<int>(int64_t(a.nk) * (pair + 1) / split) - k0 : a.nk;
  const int n_tiles = p.n_tiles;
  const uint64_t tmo = a.timeout_ns;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P_CTRL_REGS));
    // The control warps run as whole warps and elect a lane for each
    // instruction, which keeps addresses and descriptors in uniform
    // registers: the MMAs and commits of a K block then issue in 139 cycles
    // instead of the 363 they take on one lane of a divergent warp.
    const bool one = elect_one();
    if (warp == 0) {
      // ---------------- TMA producer (both CTAs) ----------------
      const uint32_t full0 = map_to_rank(smem_u32(&full[0]), first_rank);
      uint32_t s = 0, phase = 0, issued = 0;
      bool ok = true;
      for (int t = cid; t < n_tiles && ok; t += ncl) {
        int mp, nt;
        tile_coords(t, p, mp, nt);
        const int ra = (2 * mp + static_cast<int>(rank)) * 128;
        const int rb = nt * 256 + static_cast<int>(rank) * 64;
        for (int kb = 0; kb < nk; ++kb) {
          if (!fwait(smem_u32(&empty[s]), phase ^ 1, tmo, abort_flag)) {
            if (one && !*abort_flag) fabort(abort_flag, SITE_FP8_EMPTY);
            ok = false;
            break;
          }
          const uint32_t st = smem_u32(smem + s * P_STAGE), bar = full0 + s * 8;
          if (one) {
            if (leader) mbar_arrive_expect_tx(smem_u32(&full[s]), 2 * P_STAGE);
            tma_load_2d_pair(st, &ta, bar, (k0 + kb) * 128, ra);
            tma_load_2d_pair(st + P_OPERAND, &tb, bar, (k0 + kb) * 128, rb);
            tma_load_2d_pair(st + P_OPERAND + P_OPERAND / 2, &tb, bar, (k0 + kb) * 128, rb + 128);
          }
          ++issued;
          if (++s == S) { s = 0; phase ^= 1; }
        }
      }
      if (one && !leader) {
        st_cluster_u32(map_to_rank(smem_u32(const_cast<uint32_t*>(peer_issued)), first_rank),
                       issued);
      } else if (one && !ok) {
        // Every copy of both CTAs signals the leader's stage barriers; before
        // the final cluster barrier the leader waits (bounded) for the copies
        // of the last stages either CTA issued, and stages only the peer
        // issued get their expected bytes here.
        const uint64_t t0 = global_ns();
        while (*peer_issued == kNotYet && global_ns() - t0 <= 2 * tmo + 1000000) {
        }
        uint32_t last = issued;
        if (*peer_issued != kNotYet && *peer_issued > last) last = *peer_issued;
        for (uint32_t k = last > S ? last - S : 0; k < last; ++k) {
          if (k >= issued) mbar_arrive_expect_tx(smem_u32(&full[k % S]), P_STAGE);
          if (!mbar_wait(smem_u32(&full[k % S]), (k / S) & 1, tmo)) {
            record_error(&g_err_fp8_gemm, MXQ_ERR_TIMEOUT, SITE_FP8_FULL);
            break;
          }
        }
      }
    } else if (warp == 1) {
      if (leader) {
        // ---------------- pair-MMA issuer (leader CTA) ----------------
        const uint32_t idesc = idesc_f8(a.idesc_fmt, 256, 128);
        const uint64_t ad0 = smem_desc(smem_u32(smem), 0, 1024, 2);
        uint32_t s = 0, phase = 0, it = 0;
        bool ok = true;
        for (int t = cid; t < n_tiles && ok; t += ncl) {
          for (int kb = 0; kb < nk; ++kb, ++it) {
            const uint32_t b = it & 1, d = tmem + b * 256;
            const uint64_t ad = ad0 + s * (P_STAGE >> 4), bd = ad + (P_OPERAND >> 4);
            if (!fwait(smem_u32(&full[s]), phase, tmo, abort_flag) ||
                !fwait(smem_u32(&acc_empty[b]), ((it >> 1) & 1) ^ 1, tmo, abort_flag)) {
              if (one && !*abort_flag) fabort(abort_flag, SITE_FP8_TMEM_EMPTY);
              ok = false;
              break;
            }
            tc_fence_after();
            if (one) {
              mma_f8_pair(d, ad, bd, idesc, 0u);   // columns 0-127 of the tile
              mma_f8_pair(d, ad + 2, bd + 2, idesc, 1u);
              mma_f8_pair(d, ad + 4, bd + 4, idesc, 1u);
              mma_f8_pair(d, ad + 6, bd + 6, idesc, 1u);
              tc_commit_pair_mc(smem_u32(&acc_full[2 * b]), both);
              constexpr uint32_t kHalf = (P_OPERAND / 2) >> 4;   // columns 128-255
              mma_f8_pair(d + 128, ad, bd + kHalf, idesc, 0u);
              mma_f8_pair(d + 128, ad + 2, bd + kHalf + 2, idesc, 1u);
              mma_f8_pair(d + 128, ad + 4, bd + kHalf + 4, idesc, 1u);
              mma_f8_pair(d + 128, ad + 6, bd + kHalf + 6, idesc, 1u);
              tc_commit_pair_mc(smem_u32(&acc_full[2 * b + 1]), both);
              tc_commit_pair_mc(smem_u32(&empty[s]), both);
            }
            if (++s == S) { s = 0; phase ^= 1; }
          }
        }
        if (one) {   // every MMA is complete before teardown
          tc_commit_pair_mc(smem_u32(drain), static_cast<uint16_t>(0x1 << first_rank));
          if (!mbar_wait(smem_u32(drain), 0, tmo))
            record_error(&g_err_fp8_gemm, MXQ_ERR_TIMEOUT, SITE_FP8_DRAIN);
        }
      }
    } else if (warp == 2) {
      // ---------------- scales (both CTAs) ----------------
      // Eight K blocks share a group of slots and its two barriers; BATCH are
      // loaded at a time (what the registers hold), so that a block's share of
      // the load latency is below the time of its MMAs.  Groups start anew
      // with each tile.
      constexpr int BATCH = LINES ? 2 : 4;
      uint32_t grp = 0;
      for (int t = cid; t < n_tiles; t += ncl) {
        int mp, nt;
        tile_coords(t, p, mp, nt);
        const int64_t ra = (int64_t(mp) * 2 + rank) * 128 + 4 * lane, cb = int64_t(nt) * 256;
        // line scales come in rows of a multiple of 4: a float4 is in or out
        const bool a_in = ra < a.lines_a;
        for (int kb8 = 0; kb8 < nk; kb8 += 8, ++grp) {
          const uint32_t i = grp & 1;
          fwait_or_abort(smem_u32(&sc_empty[i]), ((grp >> 1) & 1) ^ 1, tmo, abort_flag,
                         SITE_FP8_SCALES);
#pragma unroll 1
          for (int kb0 = kb8; kb0 < min(kb8 + 8, nk); kb0 += BATCH) {
            float4 va[BATCH], vb[LINES ? BATCH : 1], vc[LINES ? BATCH : 1];
            float s0[BATCH], s1[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
              const int64_t kb = kb0 + u;
              const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              va[u] = zero;
              if (kb < nk && a_in)
                va[u] = *reinterpret_cast<const float4*>(a.sA + (k0 + kb) * a.lines_a + ra);
              if constexpr (LINES) {
                const float* sb = a.sB + (k0 + kb) * a.lines_b + cb + 4 * lane;
                vb[u] = vc[u] = zero;
                if (kb < nk && cb + 4 * lane < a.lines_b)
                  vb[u] = *reinterpret_cast<const float4*>(sb);
                if (kb < nk && cb + 128 + 4 * lane < a.lines_b)
                  vc[u] = *reinterpret_cast<const float4*>(sb + 128);
              } else {
                const float* sb = a.sB + (cb >> 7) * a.nk + k0 + kb;
                s0[u] = s1[u] = 0.0f;
                if (kb < nk && cb < a.N) s0[u] = sb[0];
                if (kb < nk && cb + 128 < a.N) s1[u] = sb[a.nk];
              }
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
              float* slot = scales + (i * 8 + (kb0 & 7) + u) * P::SLOT + 4 * lane;
              const float4 x = va[u];
              if constexpr (LINES) {
                *reinterpret_cast<float4*>(slot) = x;
                *reinterpret_cast<float4*>(slot + 128) = vb[u];
                *reinterpret_cast<float4*>(slot + 256) = vc[u];
              } else {
                const float p0 = s0[u], p1 = s1[u];
                *reinterpret_cast<float4*>(slot) =
                    make_float4(x.x * p0, x.y * p0, x.z * p0, x.w * p0);
                *reinterpret_cast<float4*>(slot + 128) =
                    make_float4(x.x * p1, x.y * p1, x.z * p1, x.w * p1);
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sc_full[i]));
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P_ACC_REGS));
    // ---------------- accumulation (warps 4..11, both CTAs) ----------------
    // Warps 4-7 own the columns of half 0, warps 8-11 those of half 1.  The
    // loop keeps few values beside its 160 accumulators and staged columns:
    // every shared address is an offset from one register.
    const int quad = warp & 3, h = (warp - 4) >> 2;
    const uint32_t bars = smem_u32(acc_full), sc = smem_u32(scales);
    const uint32_t empty_leader = map_to_rank(smem_u32(acc_empty), first_rank);
    const uint32_t taddr0 = tmem + (static_cast<uint32_t>(quad * 32) << 16) + h * 128;
    const uint32_t row_at = 4 * ((LINES ? 0 : h * 128) + quad * 32 + (LINES ? lane >> 2 : lane));
    const uint32_t col_at = 4 * (128 + h * 128 + 2 * (lane & 3));
    uint32_t it = 0, grp = 0;
    for (int t = cid; t < n_tiles; t += ncl) {
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
#pragma unroll 1
      for (int kb8 = 0; kb8 < nk; kb8 += 8, ++grp) {
        uint32_t at = sc + (grp & 1) * (32 * P::SLOT);
        const uint32_t end = at + min(8, nk - kb8) * (4 * P::SLOT);
        fwait_or_abort(bars + 32 + 8 * (grp & 1), (grp >> 1) & 1, a.timeout_ns, abort_flag,
                       SITE_FP8_SCALES);   // sc_full follows acc_full[4]
#pragma unroll 1
        for (; at != end; at += 4 * P::SLOT, ++it) {
          const uint32_t b = it & 1;
          float s1[LINES ? 4 : 1];   // lines: rows lane / 4 + 8 i of the warp's 32
#pragma unroll
          for (int i = 0; i < (LINES ? 4 : 1); ++i) s1[i] = lds32(at + row_at + 32 * i);
          fwait_or_abort(bars + 8 * h + 16 * b, (it >> 1) & 1, a.timeout_ns, abort_flag,
                         SITE_FP8_TMEM_FULL);
          __syncwarp();
          tc_fence_after();
          const uint32_t taddr = taddr0 + b * 256;
          // 16 words in flight while 16 are added
          uint32_t v[2][16];
          uint64_t col[4], rows[LINES ? 4 : 1];
          if constexpr (LINES) {
#pragma unroll
            for (int i = 0; i < 4; ++i) rows[i] = pack2(s1[i], s1[i]);
          }
          load16<LINES>(taddr, v[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            MXQ_TMEM_WAIT16(v[c & 1]);
            if (c < 7) {
              load16<LINES>(taddr + step16<LINES>(c + 1), v[(c + 1) & 1]);
            } else {   // everything is read: hand the accumulator back first
              tc_fence_before();
              __syncwarp();
              arrive_remote_if(lane == 0, empty_leader + b * 8);
            }
            if constexpr (LINES) {
              if ((c & 1) == 0) load_cols(at + col_at + 64 * c, col);
              add16(acc + 16 * c, v[c & 1], rows[2 * (c & 1)], rows[2 * (c & 1) + 1], col);
            } else {
              add16(acc + 16 * c, v[c & 1], s1[0]);
            }
          }
        }
        __syncwarp();
        arrive_if(lane == 0, bars + 64 + 8 * (grp & 1));   // sc_empty
      }
      int mp, nt;
      tile_coords(t, p, mp, nt);
      const int row0 = (mp * 2 + static_cast<int>(rank)) * 128, col0 = nt * 256 + h * 128;
      if (!MXQ_IN_BOUNDS(mp < p.n_mp && nt < p.n_nt, &g_err_fp8_gemm, SITE_B_FP8_GEMM)) continue;
      if constexpr (SPLIT) {
        // over the ring and the staging area: the last accumulators of both
        // halves are complete, so no MMA or copy of this CTA is left
        if (sync_any(3, 256, *abort_flag != 0)) break;
        const uint32_t part = smem_u32(smem) + (quad * 32 * PITCH + h * 128) * 4;
#pragma unroll
        for (int j = 0; j < 128; j += LINES ? 2 : 4) {
          const uint32_t to =
              part + (acc_row<LINES>(j, lane) * PITCH + acc_col<LINES>(j, lane)) * 4;
          if constexpr (LINES)
            sts(to, __float_as_uint(acc[j]), __float_as_uint(acc[j + 1]));
          else
            sts(to, __float_as_uint(acc[j]), __float_as_uint(acc[j + 1]),
                __float_as_uint(acc[j + 2]), __float_as_uint(acc[j + 3]));
        }
        break;   // a cluster has one tile
      }
      // The half tile goes through shared memory and leaves by TMA, under the
      // next tile's K loop: stored from the registers it took as long as three
      // K blocks, and the MMAs only run two ahead.
      const bool bf16 = a.out_bf16 != 0;
      const uint32_t mine = smem_u32(out) + h * 32768;
      const bool first = threadIdx.x % 128 == 0;   // issues and tracks the copies
      bool aborted = false;
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        if (pass && bf16) break;
        if (first) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        // (the half's threads meet here before either pass)
        aborted = sync_any(1 + h, 128, *abort_flag != 0);
        if (aborted) break;
        stage_out<LINES>(acc, mine, quad, lane, bf16, pass);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("bar.sync %0, 128;" ::"r"(1 + h) : "memory");
        const int wide = bf16 ? 64 : 32, x = col0 + 64 * pass;
        if constexpr (OUT == P_COPY) {
          if (x < a.N) {   // the tile's right part may lie past N whole
            if (bf16) copy_out<true>(a, mine, quad, lane, row0, x);
            else copy_out<false>(a, mine, quad, lane, row0, x);
          }
        } else if (first && row0 < a.M) {
          if (x < a.N) tma_store_2d(&tc, mine, x, row0);
          if (x + wide < a.N) tma_store_2d(&tc, mine + 16384, x + wide, row0);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      }
      if (aborted) break;
    }
    if (threadIdx.x % 128 == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  if constexpr (SPLIT) {
    cluster_sync();
    // Each pair adds up a share of the rows, over the pairs in order.
    if (warp >= 4 && !*abort_flag) {
      int mp, nt;
      tile_coords(cid, p, mp, nt);
      const int64_t row0 = (int64_t(mp) * 2 + rank) * 128, col0 = int64_t(nt) * 256 + 4 * lane;
      const int end = 128 * (pair + 1) / split;
      // two rows at a time, eight rows apart
      for (int r = 128 * pair / split + warp - 4; r < end; r += 16) {
        float4 v[2][2][P_MAX_SPLIT];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = r + 8 * (u >> 1);
          const uint32_t mine = smem_u32(smem) + (row * PITCH + 4 * lane + 128 * (u & 1)) * 4;
#pragma unroll
          for (int q = 0; q < P_MAX_SPLIT; ++q)
            v[u >> 1][u & 1][q] = q < split && row < end
                                      ? ld_cluster4(map_to_rank(mine, 2 * q + rank))
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4* t = v[u >> 1][u & 1];
          const int row = r + 8 * (u >> 1);
          float4 x = t[0];
#pragma unroll
          for (int q = 1; q < P_MAX_SPLIT; ++q) {
            x.x += t[q].x;
            x.y += t[q].y;
            x.z += t[q].z;
            x.w += t[q].w;
          }
          if (row < end && row0 + row < a.M) store4(a, row0 + row, col0 + 128 * (u & 1), x);
        }
      }
    }
  }
  tc_fence_before();
  cluster_sync();   // no CTA leaves while another may still signal it or read its sums
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// A launch of the pair kernel, but for its grid; `attr` holds two.
template <bool LINES>
cudaLaunchConfig_t pair_config(cudaLaunchAttribute* attr, int split, void* stream) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // persistent grid: it may start while the previous kernel on the stream
  // drains, and waits for it in the kernel
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(P_THREADS, 1, 1);
  cfg.dynamicSmemBytes = Pair<LINES>::SMEM;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <bool LINES>
auto pair_kernel(int out) {
  return out == P_TMA    ? fp8_gemm_pair<LINES, P_TMA>
         : out == P_COPY ? fp8_gemm_pair<LINES, P_COPY>
                         : fp8_gemm_pair<LINES, P_SHARED>;
}

// Clusters of `split` pairs that fit on the device at once, cached per device;
// 0 if they cannot be had, or if a kernel was built with fewer registers than its
// warpgroups share out among themselves.
template <bool LINES>
int pair_clusters(int split) {
  static std::mutex mu;
  static int cached[64][P_MAX_SPLIT + 1];   // clusters + 1; 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  int& known = cached[dev][split];
  if (known == 0) {
    for (int out = split > 1 ? P_SHARED : P_TMA; out <= (split > 1 ? P_SHARED : P_COPY); ++out) {
      cudaFuncAttributes fa;
      if (!ensure_dynamic_smem(reinterpret_cast<const void*>(pair_kernel<LINES>(out)),
                               Pair<LINES>::SMEM) ||
          cudaFuncGetAttributes(&fa, pair_kernel<LINES>(out)) != cudaSuccess ||
          fa.numRegs < P_MIN_REGS) {
        cudaGetLastError();
        return 0;
      }
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pair_config<LINES>(attr, split, nullptr);
    cfg.numAttrs = 1;   // the cluster dimension
    cfg.gridDim = dim3(static_cast<unsigned>(sm_count() / (2 * split) * 2 * split), 1, 1);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, pair_kernel<LINES>(split > 1 ? P_SHARED : P_TMA), &cfg) != cudaSuccess || n < 0) {
      cudaGetLastError();
      n = split > 1 ? 0 : sm_count() / 2;
    }
    known = n + 1;
  }
  return known - 1;
}

// The 2-D map of `lines` code lines of K elements, in boxes of 128 x `box`.
bool code_map(CUtensorMap* map, const void* codes, int64_t lines, int64_t K, int box) {
  return tensor_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, static_cast<uint64_t>(K),
                       static_cast<uint64_t>(lines), static_cast<uint64_t>(fp8_pitch(K)), 128,
                       static_cast<uint32_t>(box), CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
}

// CTAs that share the K blocks of a tile: as many as leave the grid one wave
// (two CTAs an SM) and each of them six blocks.  A tile alone streams its
// lines of B no faster than one CTA's copies; past one wave or with fewer
// blocks the joins cost more.  Measured at 1, 2, 4 and 8 CTAs: 1x4096x4096 8.6,
// 5.7, 4.1, 4.6 us, 1x4096x14336 26, 15.7, 12.0, 11.6 us, 16x6144x4096 9.1, 7.6,
// 6.3, 8.5 us.
uint32_t lanes_split(int64_t tiles, int nk) {
  uint32_t split = 1;
  while (split < L_MAX_SPLIT && tiles * 2 * split <= 2 * sm_count() &&
         nk >= static_cast<int>(12 * split))
    split *= 2;
  return split;
}

int lanes_tokens(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

// Which kernel, and how many pairs to a tile: modeled times in microseconds,
// fitted to measurements.  Pairs: a K block 0.365 us (line scales 0.56), a tile
// 1, or 6 where no TMA store takes the rows of C, a launch 4.5, a join 5; so
// that few tiles with a long K share each tile among up to four pairs, while
// all of them still run at once.  Lanes: a K block 0.7 or (up to 32 tokens)
// 0.55 with two CTAs an SM, a wave 3, a join 3.  Measured with one, and with as
// many pairs to a tile as this takes: 512x4096x14336 46.3 and 31.0 us (line
// scales 69.7 and 42.8), 484x2592x12534 40.6 and 22.5, 256x4096x4096 16.5 and
// 13.4.  Lanes against pairs: 64x28672x4096 25.7 and 33, 128x4096x4096 12.0 and
// 13.1, 333x1001x1234 8.3 and 11.4.
double pair_time(int64_t tiles, int nk, bool lines, bool tma_out, int clusters, int split) {
  if (clusters <= 0) return 1e30;
  const double block = lines ? 0.56 : 0.365;
  if (split == 1)
    return 4.5 + std::ceil(tiles / double(clusters)) * ((tma_out ? 1.0 : 6.0) + block * nk);
  if (tiles > clusters || nk < 4 * split) return 1e30;
  return 10.5 + block * ((nk + split - 1) / split);
}

// Pairs to a tile, 0: the lanes kernel.
template <bool LINES>
int choose_split(int64_t M, int64_t N, int nk, bool tma_out) {
  const int64_t sms = sm_count(), t = lanes_tokens(M);
  const int64_t pair_tiles = ((M + 255) / 256) * ((N + 255) / 256);
  const int64_t lane_tiles = ((M + t - 1) / t) * ((N + 127) / 128);
  const uint32_t share = lanes_split(lane_tiles, nk);
  const double lane_waves = std::ceil(lane_tiles * share / double(2 * sms));
  double best = (share > 1 ? 3.0 : 0.0) +
                lane_waves * (3.0 + (t == 64 ? 0.7 : 0.55) * nk / share);
  int split = 0;
  for (int s = 1; s <= P_MAX_SPLIT; ++s) {
    if (s > 1 && pair_tiles * s > sms / 2) break;
    const double us = pair_time(pair_tiles, nk, LINES, tma_out, pair_clusters<LINES>(s), s);
    if (us < best) {
      best = us;
      split = s;
    }
  }
  return split;
}

template <int T>
mxq_status launch_lanes(const void* A, const void* B, int64_t K, FArgs a, void* stream) {
  CUtensorMap ta, tb;
  if (!code_map(&ta, A, a.M, K, T) || !code_map(&tb, B, a.N, K, 128)) return MXQ_ERR_CUDA;
  const int64_t n_nt = (a.N + 127) / 128, tiles = n_nt * ((a.M + T - 1) / T);
  a.n_nt = static_cast<uint32_t>(n_nt);
  a.split = lanes_split(tiles, a.nk);
  if (tiles * a.split >= (int64_t(1) << 31)) return MXQ_ERR_ARG;
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(fp8_gemm_lanes<T>), Lanes<T>::SMEM))
    return MXQ_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // a CTA starts the dependents only once it runs itself, so the next kernel
  // never takes the place of CTAs that still have to start
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.split), 1, 1);
  cfg.blockDim = dim3(L_THREADS, 1, 1);
  cfg.dynamicSmemBytes = Lanes<T>::SMEM;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, fp8_gemm_lanes<T>, ta, tb, a) != cudaSuccess) {
    cudaGetLastError();
    return MXQ_ERR_CUDA;
  }
  return launch_status();
}

template <bool LINES>
mxq_status launch_pair(const void* A, const void* B, int64_t K, const FArgs& f, uint32_t idesc_fmt,
                       int split, void* stream) {
  CUtensorMap ta, tb;
  if (!code_map(&ta, A, f.M, K, 128) || !code_map(&tb, B, f.N, K, 64)) return MXQ_ERR_CUDA;
  PArgs p = {};
  p.f = f;
  p.f.idesc_fmt = idesc_fmt;
  const int64_t n_mp = (f.M + 255) / 256, n_nt = (f.N + 255) / 256;
  if (n_mp * n_nt >= (int64_t(1) << 31)) return MXQ_ERR_ARG;
  p.n_mp = static_cast<int32_t>(n_mp);
  p.n_nt = static_cast<int32_t>(n_nt);
  p.n_tiles = p.n_mp * p.n_nt;
  p.split = split;
  choose_raster(p.n_mp, p.n_nt, double(f.M) * K, double(f.N) * K, 256.0 * K, p.group, p.group_n);
  const int e = f.out_bf16 ? 2 : 4;
  CUtensorMap tc = {};
  const int out = split > 1 ? P_SHARED : f.N * e % 16 == 0 ? P_TMA : P_COPY;
  if (out == P_TMA &&
      tensor_map_2d(&tc, f.out_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                    f.C, static_cast<uint64_t>(f.N), static_cast<uint64_t>(f.M),
                    static_cast<uint64_t>(f.N * e), static_cast<uint32_t>(128 / e), 128,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE) != CUDA_SUCCESS)
    return MXQ_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pair_config<LINES>(attr, split, stream);
  const int clusters = pair_clusters<LINES>(split);
  if (clusters <= 0) return MXQ_ERR_CUDA;
  const int tiles = split > 1 ? p.n_tiles : std::min(p.n_tiles, clusters);
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * 2 * split), 1, 1);
  if (cudaLaunchKernelEx(&cfg, pair_kernel<LINES>(out), ta, tb, tc, p) != cudaSuccess) {
    cudaGetLastError();
    return MXQ_ERR_CUDA;
  }
  return launch_status();
}

// The kernel of a product: F_CHOOSE, 0 for lanes, or the pairs to a tile.
constexpr int F_CHOOSE = -1;

mxq_status product(const void* A, const float* sA, int fmt_a, const void* B, const float* sB,
                   int fmt_b, int b_scales, int64_t M, int64_t N, int64_t K, void* C,
                   int out_dtype, int form, void* stream) {
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
  a.timeout_ns = wait_timeout_ns();
  const uint32_t e5a = fmt_a == MXQ_E5M2, e5b = fmt_b == MXQ_E5M2;
  int split = form;
  if (form == F_CHOOSE) {
    const bool tma_out = N * (a.out_bf16 ? 2 : 4) % 16 == 0;
    split = a.tiles ? choose_split<false>(M, N, a.nk, tma_out)
                    : choose_split<true>(M, N, a.nk, tma_out);
  } else if (split > 0) {
    const int clusters = a.tiles ? pair_clusters<false>(split) : pair_clusters<true>(split);
    if (a.nk < split || clusters <= 0) return MXQ_ERR_ARG;
  }
  if (split) {
    const uint32_t types = e5a << 7 | e5b << 10;
    return a.tiles ? launch_pair<false>(A, B, K, a, types, split, stream)
                   : launch_pair<true>(A, B, K, a, types, split, stream);
  }
  // the lines of B are the MMA's rows (its A operand)
  a.idesc_fmt = e5b << 7 | e5a << 10;
  switch (lanes_tokens(M)) {
    case 16: return launch_lanes<16>(A, B, K, a, stream);
    case 32: return launch_lanes<32>(A, B, K, a, stream);
    default: return launch_lanes<64>(A, B, K, a, stream);
  }
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
  return product(A, sA, fmt_a, B, sB, fmt_b, b_scales, M, N, K, C, out_dtype, F_CHOOSE, stream);
}

extern "C" mxq_status mxq_debug_fp8_gemm(const void* A, const float* sA, int fmt_a, const void* B,
                                         const float* sB, int fmt_b, int b_scales, int64_t M,
                                         int64_t N, int64_t K, void* C, int out_dtype, int pairs,
                                         void* stream) {
  if (pairs < 0 || pairs > P_MAX_SPLIT) return MXQ_ERR_ARG;
  return product(A, sA, fmt_a, B, sB, fmt_b, b_scales, M, N, K, C, out_dtype, pairs, stream);
}
