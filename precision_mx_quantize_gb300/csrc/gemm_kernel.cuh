// The kernel of the block-scaled MX products on the 5th-generation tensor cores.
// Which tiles a launch has -- those of a few problems of known sizes, or those of
// experts whose rows only the device knows -- is the template's Work.
//
// Clusters of two CTAs on the two SMs of a TPC run the
// pair MMA (cta_group::2) on 256x256 output tiles, persistent over tiles.
// Each CTA holds 128 rows of A and 128 of the tile's 256 B rows; the pair
// MMA reads both halves, so an SM streams 32 KB of operands per K stage
// instead of the 48 KB a single-SM 128x256 tile needs, which keeps the
// shared-memory traffic (TMA writes + tensor-core reads) within bandwidth.
//   warp 0     (both CTAs) TMA producer: own A rows and own B half, 128 B of
//              K per stage with 128-byte swizzle, plus the stage's scale
//              chunks (own 128 A rows, all 256 B rows) into a ring of five or six;
//   warp 1     (both CTAs) allocates the pair's tensor memory.  In the
//              leader CTA one lane issues the four pair MMAs of each stage
//              into the fp32 accumulators (each CTA: 128 lanes x 256
//              columns), then releases the stage in both CTAs;
//   warps 10-11 (leader) one lane each copies part of each stage's scales
//              into both CTAs' tensor memory (tcgen05.cp) ahead of the MMA
//              lane;
//   warps 2-9  (both CTAs) epilogue: each drains 32 accumulator lanes x 128
//              columns into registers, tells the leader the accumulator is
//              free (a relaxed arrive: it must not wait for earlier stores),
//              and stores its rows -- fp32, bf16, or row-wise MX codes of the
//              product -- paced over the next tile's main loop, with 256-bit
//              stores when aligned.
// The kernel is launched with programmatic stream serialization and waits for the
// previous grid (griddepcontrol) before any global access.
#pragma once

#include <mutex>

#include "mxq_common.cuh"
#include "mxq_host.h"
#include "mxq_tc.cuh"

namespace mxq {
namespace {

__device__ uint32_t g_err_gemm;   // this translation unit's error word

constexpr int G_CLUSTER = 2;                 // CTA pair of one 2-SM MMA
constexpr int G_BM = 128;                    // rows of A per CTA (pair tile: 256)
constexpr int G_BN = 256;                    // columns of the tile (rows of B)
constexpr int G_BN_CTA = G_BN / G_CLUSTER;   // rows of B each CTA holds
constexpr int G_BKB = 128;                   // bytes of K per stage (one 128 B swizzle row)
constexpr int G_STAGES = 6;                  // stages of the operand ring, at most
constexpr int G_THREADS = 384;               // 12 warps
constexpr int G_A_BYTES = G_BM * G_BKB;      // 16 KB
constexpr int G_B_BYTES = G_BN_CTA * G_BKB;  // 16 KB
constexpr int G_SFA_BYTES = 1024;            // own 128 rows: up to 2 chunks of 512 B
constexpr int G_SFB_BYTES = 2048;            // all 256 rows: up to 4 chunks of 512 B
constexpr int G_STAGE_BYTES = G_A_BYTES + G_B_BYTES + G_SFA_BYTES + G_SFB_BYTES;
constexpr int G_BAR_BYTES = 512;
constexpr uint32_t kNotYet = 0xFFFFFFFFu;   // peer's stage count not yet reported
constexpr int G_PITCH = 144;                 // staged epilogue: 128 bytes of a row and its padding

// How a tile leaves: straight from the accumulators, through shared memory and copied out
// by its threads, or through shared memory and by TMA (32 rows of every warp either way).
enum StoreBy { STORE_DIRECT, STORE_STAGED, STORE_TMA };
constexpr int out_bytes(StoreBy by) {   // of shared memory, one piece per warp
  return by == STORE_STAGED ? 8 * 32 * G_PITCH : by == STORE_TMA ? 8 * 32 * 128 : 0;
}
constexpr uint32_t G_TMEM_COLS = 512;
constexpr uint32_t G_SFA_COL0 = 256;                 // 8 columns per stage
constexpr uint32_t G_SFB_COL0 = 256 + 8 * G_STAGES;  // 16 columns per stage
static_assert(G_SFB_COL0 + 16 * G_STAGES <= G_TMEM_COLS, "tensor memory budget");
static_assert(G_STAGE_BYTES % 1024 == 0, "stages keep 1024-byte alignment");

// One GEMM problem of a launch.  Fields up to q_scale_tc may differ between
// the problems of a grouped launch; the element format, the epilogue kind and
// the wait limit are those of problem 0 for all.
struct GArgs {
  int32_t M, N;
  int32_t tile0;                // first work item of this problem in the launch
  int32_t n_mp, n_nt, n_tiles;  // 256-row pair tiles along M, 256-col tiles along N
  int32_t group;                // tiles per raster group along the grouped dimension
  int32_t group_n;              // 1: groups run along N, 0: along M
  int32_t nk;                   // K stages
  int32_t kc_per_row;           // 512-byte scale chunks per 128-row tile (KBp / 4)
  const uint8_t* sfa;           // chunked scales of A in the workspace
  const uint8_t* sfb;           // chunked scales of B
  void* C;
  int32_t out_bf16;
  int32_t fp4;
  int32_t elem_code;            // A/B element type field of the instruction descriptor
  int32_t wide_stores;          // rows of C are 32-byte aligned: 256-bit stores
  int32_t out_q;                // 1: C receives row-wise MX codes of the product
  int32_t q_fmt;                // their element format
  uint8_t* q_scales;            // their E8M0 scales [M][N/32]
  int32_t q_scale_words;        // scale rows are 4-byte aligned: one word per 4 blocks
  int32_t q_scale_tc;           // output scales in the tensor cores' chunk layout
  uint32_t pace_ns;             // epilogue: pause after each 16/32-byte store (see below)
  uint64_t timeout_ns;
};

// Copy one 512-byte scale chunk (32 rows x 16 B) of each CTA's shared memory
// into 4 columns of the same CTA's tensor memory, replicated to all four
// 32-lane quadrants.
MXQ_DEV void tc_cp_sf_pair(uint32_t taddr, uint32_t smem_addr) {
  const uint64_t d = smem_desc(smem_addr, 0, 128, 0);
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

MXQ_DEV void mma_mxf8_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                           uint32_t sfb, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accum), "r"(sfa), "r"(sfb)
      : "memory");
}

MXQ_DEV void mma_mxf4_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                           uint32_t sfb, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accum), "r"(sfa), "r"(sfb)
      : "memory");
}

// Instruction descriptor of a block-scaled m x n MMA: K-major A and B, E8M0 scales,
// scale-factor byte ids.
MXQ_DEV uint32_t idesc_block_scaled(uint32_t fmt_code, uint32_t m, uint32_t n, uint32_t a_sf,
                                    uint32_t b_sf) {
  uint32_t d = 0;
  d |= (b_sf & 3u) << 4;
  d |= (fmt_code & 7u) << 7;    // A format
  d |= (fmt_code & 7u) << 10;   // B format
  d |= (n >> 3) << 17;
  d |= 1u << 23;                // scale type: UE8M0
  d |= (m >> 4) << 24;
  d |= (a_sf & 3u) << 29;
  return d;
}

MXQ_DEV void gabort(volatile int* abort_flag, uint32_t site) {
  *abort_flag = 1;
  record_error(&g_err_gemm, MXQ_ERR_TIMEOUT, site);
}

// Store pacing.  A tile's epilogue stores leave the SM in one burst
// (64-256 KB per CTA) right when the next tile's main loop needs the same
// SM-to-L2 path for its TMA loads; the burst lengthens the loads' latency,
// and the latency-bound operand ring stalls the tensor pipe.  Spreading each
// thread's stores over part of the next tile's main loop avoids that (+3-12%
// measured, most on MXFP4 with fp32 output).  The last tile of a CTA is
// stored at full speed, since nothing runs behind it.
MXQ_DEV void pace(uint32_t ns) {
  if (ns) __nanosleep(ns);
}

// Row-wise MX quantization of the 128 fp32 accumulators a thread holds for
// one output row (four 32-column blocks, nblk of them inside N): per block
// the amax of the fp32 values, its E8M0 exponent, the exact power-of-two
// scaling and the round-to-nearest-even saturating conversion -- the rules
// of the quantizer, applied to the fp32 product without a bf16 rounding.
template <int QF>
MXQ_DEV void store_row_codes(const uint32_t (&v)[128], const GArgs& a, int64_t row, int64_t col0,
                             int nblk, uint32_t pace_ns) {
  constexpr uint32_t emax = QF == MXQ_E4M3 ? 8u : (QF == MXQ_E5M2 ? 15u : 2u);
  constexpr int cb = QF == MXQ_E2M1 ? 16 : 32;   // code bytes per block
  const int64_t row_bytes = QF == MXQ_E2M1 ? int64_t(a.N) / 2 : int64_t(a.N);
  uint8_t* crow = static_cast<uint8_t*>(a.C) + row * row_bytes + (col0 / 32) * cb;
  uint32_t sw = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (b < nblk) {
      const uint32_t* x = v + 32 * b;
      float m = fabsf(__uint_as_float(x[0]));
#pragma unroll
      for (int j = 1; j < 31; j += 2)
        m = max3_abs_nan(m, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
      m = max3_abs_nan(m, __uint_as_float(x[31]), __uint_as_float(x[31]));
      const uint32_t sc = scale_of(__float_as_uint(m) & 0x7FFFFFFFu, emax);
      const float k = inv_scale(sc);
      auto f = [&](int j) { return __fmul_rn(__uint_as_float(x[j]), k); };
      uint32_t w[8];
      if constexpr (QF == MXQ_E2M1) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[q] = cvt_e2m1x8(f(8 * q), f(8 * q + 1), f(8 * q + 2), f(8 * q + 3), f(8 * q + 4),
                            f(8 * q + 5), f(8 * q + 6), f(8 * q + 7));
      } else if constexpr (QF == MXQ_E5M2) {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = cvt_e5m2x4(f(4 * q), f(4 * q + 1), f(4 * q + 2), f(4 * q + 3));
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = cvt_e4m3x4(f(4 * q), f(4 * q + 1), f(4 * q + 2), f(4 * q + 3));
      }
      if (sc == 255u) {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = 0u;
      }
      uint8_t* dst = crow + b * cb;
      if constexpr (QF == MXQ_E2M1) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (a.wide_stores) {
        st_global_v8(dst, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
      }
      pace(pace_ns);
      sw |= sc << (8 * b);
    }
  }
  if (!MXQ_IN_BOUNDS(row < a.M && col0 + 32 * nblk <= a.N && (!a.q_scale_tc || nblk == 4),
                     &g_err_gemm, SITE_B_GEMM_QSCALE))
    return;
  if (a.q_scale_tc) {
    // one word of chunk (row / 128, col0 / 128): N % 128 == 0, so nblk == 4
    uint8_t* chunk = a.q_scales + ((row >> 7) * (int64_t(a.N) >> 7) + (col0 >> 7)) * 512;
    *reinterpret_cast<uint32_t*>(chunk + (row & 31) * 16 + ((row & 127) >> 5) * 4) = sw;
    return;
  }
  uint8_t* srow = a.q_scales + row * (int64_t(a.N) / 32) + col0 / 32;
  if (a.q_scale_words && nblk == 4) {
    *reinterpret_cast<uint32_t*>(srow) = sw;
  } else {
    for (int b = 0; b < nblk; ++b) srow[b] = static_cast<uint8_t>(sw >> (8 * b));
  }
}

// Staged epilogue: a warp's 32 rows of up to 128 columns of C through its piece of shared
// memory, 128 bytes of every row at a time, so that a store writes whole 128-byte lines
// (four rows at a time).  A store straight from the accumulators has a row per lane and
// touches 32 lines for 1 KB, one line a cycle: with few K stages to a tile that alone
// takes longer than the products.  The pitch of 144 bytes keeps eight lanes' 16-byte
// accesses on different banks both ways.
MXQ_DEV void store_staged(const uint32_t (&v)[128], const GArgs& a, uint8_t* buf, int64_t row0,
                          int rows, int64_t col0, int ncols) {
  const int lane = threadIdx.x & 31, sub = lane >> 3, at = lane & 7;
  const int per = a.out_bf16 ? 64 : 32;   // columns of 128 bytes
  const int size = a.out_bf16 ? 2 : 4;
  uint8_t* const mine = buf + lane * G_PITCH;
  uint8_t* const c = static_cast<uint8_t*>(a.C) + ((row0 + sub) * a.N + col0) * size + at * 16;
  const int64_t step = int64_t(4) * a.N * size;
  auto out = [&](int first) {
    __syncwarp();
    const bool in = first + (at + 1) * (16 / size) <= ncols;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int r = 4 * q + sub;
      if (in && r < rows)
        *reinterpret_cast<uint4*>(c + q * step + first * size) =
            *reinterpret_cast<const uint4*>(buf + r * G_PITCH + at * 16);
    }
    __syncwarp();
  };
  if (a.out_bf16) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s * per >= ncols) break;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const __nv_bfloat162 b =
              __floats2bfloat162_rn(__uint_as_float(v[64 * s + 8 * q + 2 * u]),
                                    __uint_as_float(v[64 * s + 8 * q + 2 * u + 1]));
          w[u] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(mine + q * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      out(s * per);
    }
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s * per >= ncols) break;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4*>(mine + q * 16) =
            make_uint4(v[32 * s + 4 * q], v[32 * s + 4 * q + 1], v[32 * s + 4 * q + 2],
                       v[32 * s + 4 * q + 3]);
      out(s * per);
    }
  }
}

// The same by TMA: the copy engine reads the lines from shared memory itself, which
// spares the pass that a thread's loads make, and leaves out what lies past the map's
// ends.  128-byte swizzle: the 16-byte piece q of row r lies at q ^ (r & 7), so that eight
// lanes' stores meet different banks.  `z`, `y` and `x`: matrix, row and column of C.
template <typename Work>
MXQ_DEV void store_tma(const uint32_t (&v)[128], const typename Work::Params& g, bool bf16,
                       uint8_t* buf, int z, int y, int x, int ncols) {
  const int lane = threadIdx.x & 31;
  const int per = bf16 ? 64 : 32;   // columns of 128 bytes
  uint8_t* const mine = buf + lane * 128;
  auto ready = [&] {   // the copy of the lines before has been read
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
  };
  auto put = [&](int q, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    *reinterpret_cast<uint4*>(mine + (q ^ (lane & 7)) * 16) = make_uint4(a, b, c, d);
  };
  auto out = [&](int first) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(Work::store_map(g), smem_u32(buf), x + first, y, z);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  };
  if (bf16) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s * per >= ncols) break;
      ready();
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const __nv_bfloat162 b =
              __floats2bfloat162_rn(__uint_as_float(v[64 * s + 8 * q + 2 * u]),
                                    __uint_as_float(v[64 * s + 8 * q + 2 * u + 1]));
          w[u] = *reinterpret_cast<const uint32_t*>(&b);
        }
        put(q, w[0], w[1], w[2], w[3]);
      }
      out(s * per);
    }
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s * per >= ncols) break;
      ready();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        put(q, v[32 * s + 4 * q], v[32 * s + 4 * q + 1], v[32 * s + 4 * q + 2],
            v[32 * s + 4 * q + 3]);
      out(s * per);
    }
  }
}

// One work item (a 256x256 tile) as the roles of the kernel see it.
struct Item {
  const GArgs* a;                            // what its problem's items have in common
  const CUtensorMap *ta, *tb, *tsa, *tsb;
  int nk;                                    // K stages
  int last;                                  // MMAs of the last one (1 to 4)
  int mp, nt;                                // pair tile along M, tile along N
  int kx;                                    // first byte of K in the lines of A and B
  int ay, by;                                // first lines of A and B
  int sa, sb;                                // first scale chunks of A's pair tile and B's tile
  int64_t c0;                                // row of C that row 0 of the problem goes to
  int rows;                                  // rows of the problem
  int z;                                     // its number among the matrices of C
  uint32_t pace_ns;
};

// Work says which items a launch has and where they lie:
//   Params, the launch's __grid_constant__ argument; STAGES of the operand ring;
//   TABLE, bytes of shared memory; OUT, how tiles leave (by TMA: store_map(g));
//   first(g), the arguments that all items share; prefetch(g), of its tensor maps;
//   load(g, table), by all threads, once the previous grid is complete;
//   an object per role, whose tiles() counts the items and at(t) describes item t
//   (asked in increasing order); PARTIAL, whether `last` can be below four.
template <typename Work>
__global__ void __launch_bounds__(G_THREADS, 1)
    mx_gemm_kernel(const __grid_constant__ typename Work::Params g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* out = smem + Work::STAGES * G_STAGE_BYTES;   // staged tiles
  uint64_t* full = reinterpret_cast<uint64_t*>(out + out_bytes(Work::OUT));
  uint64_t* empty = full + Work::STAGES;
  uint64_t* sf_ready = empty + Work::STAGES;
  uint64_t* tmem_full = sf_ready + Work::STAGES;
  uint64_t* tmem_empty = tmem_full + 1;      // leader: both CTAs drained the accumulator
  uint64_t* drain = tmem_empty + 1;
  uint32_t* tmem_base_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_slot + 1);
  // leader: the number of K stages the peer CTA's producer issued, written
  // by the peer when its producer stops (kNotYet until then)
  volatile uint32_t* peer_issued = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const GArgs& a0 = Work::first(g);   // format, epilogue kind and wait limit of the launch
  void* table = out + out_bytes(Work::OUT) + G_BAR_BYTES;
  if (threadIdx.x == 0) {
    Work::prefetch(g);
    for (int s = 0; s < Work::STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);    // leader: one arrival, bytes of both CTAs
      mbar_init(smem_u32(&empty[s]), 1);
      mbar_init(smem_u32(&sf_ready[s]), 2);  // two scale-copy warps
    }
    mbar_init(smem_u32(tmem_full), 1);
    mbar_init(smem_u32(tmem_empty), 8 * G_CLUSTER);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    *peer_issued = kNotYet;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_base_slot), G_TMEM_COLS);
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs exist before anyone signals the peer
  tc_fence_after();
  griddep_wait();  // the previous kernel's writes (codes, scales) are visible
  griddep_launch_dependents();
  const int cid = blockIdx.x / G_CLUSTER, ncl = gridDim.x / G_CLUSTER;
  const uint32_t tmem = *tmem_base_slot;
  if (Work::TABLE) {
    Work::load(g, table);
    __syncthreads();
  }
  const int n_tiles = Work(g, table).tiles();
  const uint64_t tmo = a0.timeout_ns;

  const int n_sfa = a0.fp4 ? 2 : 1;           // 512-byte chunks of own-A scales per stage
  const uint32_t sf_bytes_a = 512u * n_sfa;   // per 128 rows
  // bytes one CTA brings into a stage; the leader's barrier counts both CTAs
  const uint32_t cta_tx = G_A_BYTES + G_B_BYTES + 3 * sf_bytes_a;

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    if (lane == 0) {
      // every load of both CTAs completes on the leader's stage barrier
      const uint32_t full0 = map_to_rank(smem_u32(&full[0]), 0);
      uint32_t s = 0, phase = 0, issued = 0;
      bool ok = true;
      Work work(g, table);
      for (int t = cid; t < n_tiles && ok; t += ncl) {
        const Item it = work.at(t);
        const int nk = it.nk;
        if (!MXQ_IN_BOUNDS(Work::inside(it), &g_err_gemm, SITE_B_GEMM_TILE)) {
          ok = false;   // the MMA lane then waits out its bounded wait
          break;
        }
        // this CTA's 128-row tile of A, and the first scale chunk rows
        const int ay = it.ay + static_cast<int>(rank) * G_BM;
        const int by = it.by + static_cast<int>(rank) * G_BN_CTA;
        const int srow_a = it.sa + static_cast<int>(rank) * it.a->kc_per_row;
        const int srow_b0 = it.sb, srow_b1 = it.sb + it.a->kc_per_row;
        for (int ks = 0; ks < nk; ++ks) {
          if (!mbar_try_wait_cluster(smem_u32(&empty[s]), phase ^ 1) &&
              !gwait(smem_u32(&empty[s]), phase ^ 1, tmo, abort_flag)) {
            if (!*abort_flag) gabort(abort_flag, SITE_GEMM_EMPTY);
            ok = false;
            break;
          }
          const uint32_t st = smem_u32(smem + s * G_STAGE_BYTES);
          const uint32_t bar = full0 + s * 8;
          if (leader) mbar_arrive_expect_tx(smem_u32(&full[s]), G_CLUSTER * cta_tx);
          tma_load_2d_pair(st, it.ta, bar, it.kx + ks * G_BKB, ay);
          tma_load_2d_pair(st + G_A_BYTES, it.tb, bar, it.kx + ks * G_BKB, by);
          const int kc = ks * n_sfa;
          tma_load_2d_pair(st + G_A_BYTES + G_B_BYTES, it.tsa, bar, 0, srow_a + kc);
          tma_load_2d_pair(st + G_A_BYTES + G_B_BYTES + G_SFA_BYTES, it.tsb, bar, 0,
                           srow_b0 + kc);
          tma_load_2d_pair(st + G_A_BYTES + G_B_BYTES + G_SFA_BYTES + sf_bytes_a, it.tsb, bar,
                           0, srow_b1 + kc);
          ++issued;
          if (++s == Work::STAGES) { s = 0; phase ^= 1; }
        }
      }
      if (!leader) {
        // tell the leader how many stages this CTA's copies were issued for
        st_cluster_u32(map_to_rank(smem_u32(const_cast<uint32_t*>(peer_issued)), 0), issued);
      } else if (!ok) {
        // Every copy of both CTAs signals the leader's stage barriers, and
        // the peer's land in the peer's shared memory, which stays in use
        // until the final cluster barrier.  So before that barrier the leader
        // waits (bounded) for the copies of the last stages either CTA
        // issued; stages only the peer issued get their expected bytes here.
        const uint64_t t0 = global_ns();
        while (*peer_issued == kNotYet && global_ns() - t0 <= 2 * tmo + 1000000) {
        }
        uint32_t last = issued;
        if (*peer_issued != kNotYet && *peer_issued > last) last = *peer_issued;
        for (uint32_t k = last > Work::STAGES ? last - Work::STAGES : 0; k < last; ++k) {
          if (k >= issued) mbar_arrive_expect_tx(smem_u32(&full[k % Work::STAGES]), cta_tx);
          if (!mbar_wait(smem_u32(&full[k % Work::STAGES]), (k / Work::STAGES) & 1, tmo)) {
            // a stage one CTA never issued: later stages were not issued either
            record_error(&g_err_gemm, MXQ_ERR_TIMEOUT, SITE_GEMM_FULL);
            break;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------- pair-MMA issuer (leader CTA) ----------------
      // Everything that does not change per stage is computed once: each
      // tcgen05 instruction costs the issuing thread ~100 cycles, so the
      // loop keeps nothing else on its path.
      const uint32_t fmt_code = static_cast<uint32_t>(a0.elem_code);
      uint32_t idesc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t sf_id = a0.fp4 ? ((2 * j) & 3) : j;
        idesc[j] = idesc_block_scaled(fmt_code, G_CLUSTER * G_BM, G_BN, sf_id, sf_id);
      }
      const uint32_t st0 = smem_u32(smem);
      const uint64_t adesc_s0 = smem_desc(st0, 0, 1024, 2);
      const uint64_t bdesc_s0 = smem_desc(st0 + G_A_BYTES, 0, 1024, 2);
      constexpr uint32_t kStageDesc = G_STAGE_BYTES >> 4;   // stage stride in descriptor units
      const bool fp4 = a0.fp4 != 0;
      uint32_t s = 0, phase = 0, tile_i = 0;
      bool ok = true;
      Work work(g, table);
      for (int t = cid; t < n_tiles && ok; t += ncl, ++tile_i) {
        const Item it = work.at(t);
        const int nk = it.nk;
        if (!mbar_try_wait_cluster(smem_u32(tmem_empty), (tile_i & 1) ^ 1) &&
            !gwait(smem_u32(tmem_empty), (tile_i & 1) ^ 1, tmo, abort_flag)) {
          if (!*abort_flag) gabort(abort_flag, SITE_GEMM_TMEM_EMPTY);
          ok = false;
          break;
        }
        tc_fence_after();
        for (int ks = 0; ks < nk; ++ks) {
          if (!mbar_try_wait_cluster(smem_u32(&sf_ready[s]), phase) &&
              !gwait(smem_u32(&sf_ready[s]), phase, tmo, abort_flag)) {
            if (!*abort_flag) gabort(abort_flag, SITE_GEMM_FULL);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sfa_t = tmem + G_SFA_COL0 + 8 * s;
          const uint32_t sfb_t = tmem + G_SFB_COL0 + 16 * s;
          const uint64_t ad = adesc_s0 + s * kStageDesc;
          const uint64_t bd = bdesc_s0 + s * kStageDesc;
          // scales of this stage are already in tensor memory (sf_ready)
          const int n = Work::PARTIAL && ks == nk - 1 ? it.last : 4;
          if (fp4) {
            // each MMA consumes 32 bytes of K (K=64 packed E2M1), k-blocks 2j, 2j+1
            mma_mxf4_pair(tmem, ad, bd, idesc[0], sfa_t, sfb_t, ks > 0 ? 1u : 0u);
            if (n > 1) mma_mxf4_pair(tmem, ad + 2, bd + 2, idesc[1], sfa_t, sfb_t, 1u);
            if (n > 2) mma_mxf4_pair(tmem, ad + 4, bd + 4, idesc[2], sfa_t + 4, sfb_t + 8, 1u);
            if (n > 3) mma_mxf4_pair(tmem, ad + 6, bd + 6, idesc[3], sfa_t + 4, sfb_t + 8, 1u);
          } else {
            // each MMA consumes 32 bytes of K (K=32 E4M3), k-block j
            mma_mxf8_pair(tmem, ad, bd, idesc[0], sfa_t, sfb_t, ks > 0 ? 1u : 0u);
            if (n > 1) mma_mxf8_pair(tmem, ad + 2, bd + 2, idesc[1], sfa_t, sfb_t, 1u);
            if (n > 2) mma_mxf8_pair(tmem, ad + 4, bd + 4, idesc[2], sfa_t, sfb_t, 1u);
            if (n > 3) mma_mxf8_pair(tmem, ad + 6, bd + 6, idesc[3], sfa_t, sfb_t, 1u);
          }
          tc_commit_pair_mc(smem_u32(&empty[s]), 0x3);   // stage free in both CTAs
          if (++s == Work::STAGES) { s = 0; phase ^= 1; }
        }
        if (!ok) break;
        tc_commit_pair_mc(smem_u32(tmem_full), 0x3);     // accumulators ready in both CTAs
      }
      // all pair MMAs issued by this thread are complete before teardown
      tc_commit_pair_mc(smem_u32(drain), 0x1);
      if (!mbar_wait(smem_u32(drain), 0, tmo))
        record_error(&g_err_gemm, MXQ_ERR_TIMEOUT, SITE_GEMM_DRAIN);
    }
  } else if (warp >= 10) {
    if (lane == 0 && leader) {
      // ---------------- scale copiers (leader CTA, warps 10 and 11) -------
      // Copy each stage's scales into both CTAs' tensor memory ahead of the
      // MMA lane and signal it through sf_ready (two arrivals per stage).
      // Separate threads get the scales into tensor memory as soon as a
      // stage lands, while the MMA lane is still busy with earlier stages;
      // copies issued by the MMA lane itself, just before each stage's MMAs,
      // measured 10-30% slower.  E4M3: warp 10 copies the A scales and those
      // of B rows 0-127, warp 11 those of B rows 128-255.  E2M1 (twice the
      // chunks): warp 10 the two A chunks and the first B chunk, warp 11 the
      // other three.
      const bool first = warp == 10;
      const uint32_t st0 = smem_u32(smem);
      const bool fp4 = a0.fp4 != 0;
      uint32_t s = 0, phase = 0;
      uint32_t total = 0;   // K stages of this cluster's work items
      {
        Work work(g, table);
        for (int t = cid; t < n_tiles; t += ncl) total += static_cast<uint32_t>(work.at(t).nk);
      }
      for (uint32_t it = 0; it < total; ++it) {
        if (!mbar_try_wait_cluster(smem_u32(&full[s]), phase) &&
            !gwait(smem_u32(&full[s]), phase, tmo, abort_flag)) {
          if (!*abort_flag) gabort(abort_flag, SITE_GEMM_FULL);
          break;
        }
        tc_fence_after();
        const uint32_t sfa_smem = st0 + s * G_STAGE_BYTES + G_A_BYTES + G_B_BYTES;
        const uint32_t sfb_smem = sfa_smem + G_SFA_BYTES;
        const uint32_t sfa_t = tmem + G_SFA_COL0 + 8 * s;
        const uint32_t sfb_t = tmem + G_SFB_COL0 + 16 * s;
        // A: chunk c -> columns +4c.  B: k-chunk c of rows 0-127 -> +8c,
        // rows 128-255 -> +8c+4 (rows 128-255 start sf_bytes_a into the slot).
        // E4M3: 3 chunks per stage (2 + 1); E2M1: 6 chunks (3 + 3).
        if (fp4) {
          if (first) {
            tc_cp_sf_pair(sfa_t, sfa_smem);
            tc_cp_sf_pair(sfa_t + 4, sfa_smem + 512);
            tc_cp_sf_pair(sfb_t, sfb_smem);
          } else {
            tc_cp_sf_pair(sfb_t + 8, sfb_smem + 512);
            tc_cp_sf_pair(sfb_t + 4, sfb_smem + sf_bytes_a);
            tc_cp_sf_pair(sfb_t + 12, sfb_smem + sf_bytes_a + 512);
          }
        } else if (first) {
          tc_cp_sf_pair(sfa_t, sfa_smem);
          tc_cp_sf_pair(sfb_t, sfb_smem);
        } else {
          tc_cp_sf_pair(sfb_t + 4, sfb_smem + sf_bytes_a);
        }
        tc_commit_pair_mc(smem_u32(&sf_ready[s]), 0x1);
        if (++s == Work::STAGES) { s = 0; phase ^= 1; }
      }
    }
  } else {
    // ---------------- epilogue (warps 2..9, both CTAs) ----------------
    const int quad = warp & 3;                   // tensor-memory lane quadrant
    const int colh = (warp - 2) >> 2;            // 0: columns 0-127, 1: 128-255
    const uint32_t empty_leader = map_to_rank(smem_u32(tmem_empty), 0);
    uint32_t tile_i = 0;
    Work work(g, table);
    for (int t = cid; t < n_tiles; t += ncl, ++tile_i) {
      const Item it = work.at(t);
      const GArgs& a = *it.a;
      if (!gwait(smem_u32(tmem_full), tile_i & 1, tmo, abort_flag)) {
        if (lane == 0 && !*abort_flag) gabort(abort_flag, SITE_GEMM_TMEM_FULL);
        break;
      }
      tc_fence_after();
      uint32_t v[128];
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + colh * 128;
      MXQ_TMEM_LD32(taddr + 0, (v + 0));
      MXQ_TMEM_LD32(taddr + 32, (v + 32));
      MXQ_TMEM_LD32(taddr + 64, (v + 64));
      MXQ_TMEM_LD32(taddr + 96, (v + 96));
#pragma unroll
      for (int i = 0; i < 128; i += 16) MXQ_TMEM_WAIT16((v + i));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(empty_leader);

      if (Work::PARTIAL && it.nk == 0) {   // no MMA wrote the accumulators
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i] = 0u;
      }
      [[maybe_unused]] const uint32_t pn =
          t + ncl < n_tiles ? it.pace_ns : 0u;   // last tile: no pacing
      const int64_t row = (int64_t(it.mp) * G_CLUSTER + rank) * G_BM + quad * 32 + lane;
      const int64_t col0 = int64_t(it.nt) * G_BN + colh * 128;
      if (Work::QUANTIZES && a.q_scale_tc && row >= a.M &&
          row < ((int64_t(a.M) + 127) & ~int64_t(127)) && col0 < a.N) {
        // lines past M inside the last 128-line tile: zero scales, as in
        // every chunk-layout buffer
        uint8_t* chunk = a.q_scales + ((row >> 7) * (int64_t(a.N) >> 7) + (col0 >> 7)) * 512;
        *reinterpret_cast<uint32_t*>(chunk + (row & 31) * 16 + ((row & 127) >> 5) * 4) = 0u;
      }
      if constexpr (Work::OUT != STORE_DIRECT) {
        uint8_t* const buf = out + (warp - 2) * (out_bytes(Work::OUT) / 8);
        const int rows = static_cast<int>(min(int64_t(it.rows) - (row - lane), int64_t(32)));
        if (rows > 0 && col0 < a.N &&
            MXQ_IN_BOUNDS(Work::inside(it) && row - lane + rows <= it.rows, &g_err_gemm,
                          SITE_B_GEMM_STORE)) {
          const int ncols = static_cast<int>(min(a.N - col0, int64_t(128)));
          if constexpr (Work::OUT == STORE_TMA)
            store_tma<Work>(v, g, a.out_bf16 != 0, buf, it.z, static_cast<int>(row - lane),
                            static_cast<int>(col0), ncols);
          else store_staged(v, a, buf, it.c0 + row - lane, rows, col0, ncols);
        }
      } else if (row < it.rows && col0 < a.N &&
          MXQ_IN_BOUNDS(Work::inside(it) && row >= 0 && col0 >= 0 && (col0 & 31) == 0,
                        &g_err_gemm, SITE_B_GEMM_STORE)) {
        const int64_t ncols = (a.N - col0) < 128 ? (a.N - col0) : 128;
        if (Work::QUANTIZES && a.out_q) {
          const int nblk = static_cast<int>(ncols >> 5);   // N % 32 == 0
          if (a.q_fmt == MXQ_E2M1) store_row_codes<MXQ_E2M1>(v, a, row, col0, nblk, pn);
          else if (a.q_fmt == MXQ_E5M2) store_row_codes<MXQ_E5M2>(v, a, row, col0, nblk, pn);
          else store_row_codes<MXQ_E4M3>(v, a, row, col0, nblk, pn);
        } else if (a.out_bf16) {
          __nv_bfloat16* crow = static_cast<__nv_bfloat16*>(a.C) + (it.c0 + row) * a.N + col0;
          uint32_t p[64];
#pragma unroll
          for (int u = 0; u < 64; ++u) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[2 * u]),
                                                           __uint_as_float(v[2 * u + 1]));
            p[u] = *reinterpret_cast<const uint32_t*>(&b);
          }
          if (a.wide_stores) {
#pragma unroll
            for (int c = 0; c < 128; c += 16)
              if (c < ncols) {
                st_global_v8(crow + c, p[c / 2], p[c / 2 + 1], p[c / 2 + 2], p[c / 2 + 3],
                             p[c / 2 + 4], p[c / 2 + 5], p[c / 2 + 6], p[c / 2 + 7]);
                pace(pn);
              }
          } else {
#pragma unroll
            for (int c = 0; c < 128; c += 8)
              if (c < ncols) {
                *reinterpret_cast<uint4*>(crow + c) =
                    make_uint4(p[c / 2], p[c / 2 + 1], p[c / 2 + 2], p[c / 2 + 3]);
                pace(pn >> 1);
              }
          }
        } else {
          float* crow = static_cast<float*>(a.C) + (it.c0 + row) * a.N + col0;
          if (a.wide_stores) {
#pragma unroll
            for (int c = 0; c < 128; c += 8)
              if (c < ncols) {
                st_global_v8(crow + c, v[c], v[c + 1], v[c + 2], v[c + 3], v[c + 4], v[c + 5],
                             v[c + 6], v[c + 7]);
                pace(pn);
              }
          } else {
#pragma unroll
            for (int c = 0; c < 128; c += 4)
              if (c < ncols) {
                *reinterpret_cast<uint4*>(crow + c) = make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                pace(pn >> 1);
              }
          }
        }
      }
    }
  }

  // the copies out of shared memory are complete (only epilogue lanes have any)
  if (Work::OUT == STORE_TMA && lane == 0)
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  tc_fence_before();
  cluster_sync();  // no CTA leaves while its peer may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, G_TMEM_COLS);
}

// Clusters of G_CLUSTER CTAs of a kernel that fit on the device at once (cached per
// device; one cache per instantiation).
template <typename Work>
int max_gemm_clusters(cudaLaunchConfig_t cfg) {
  static std::mutex mu;
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cached[dev] == 0) {
    cfg.gridDim = dim3(static_cast<unsigned>(G_CLUSTER * sm_count()), 1, 1);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, mx_gemm_kernel<Work>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = sm_count() / G_CLUSTER;
    }
    cached[dev] = n;
  }
  return cached[dev];
}

// Launches the kernel on as many clusters as the device holds, at most `items`.
template <typename Work>
mxq_status gemm_kernel_run(const typename Work::Params& g, int64_t items, void* stream) {
  constexpr int smem = Work::STAGES * G_STAGE_BYTES + G_BAR_BYTES + Work::TABLE +
                       out_bytes(Work::OUT) + 1024;
  static_assert(Work::STAGES <= G_STAGES && Work::TABLE % 16 == 0, "shared memory layout");
  static_assert(smem <= 232448, "shared memory of a CTA");
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(mx_gemm_kernel<Work>), smem))
    return MXQ_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = G_CLUSTER;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(G_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int max_clusters = max_gemm_clusters<Work>(cfg);
  // persistent grid (every cluster resident): it may start while the
  // previous kernel on the stream drains, and waits for it in the kernel
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  if (max_clusters <= 0) return MXQ_ERR_CUDA;
  cfg.gridDim = dim3(static_cast<unsigned>(
                         G_CLUSTER * std::min<int64_t>(items, max_clusters)), 1, 1);
  if (cudaLaunchKernelEx(&cfg, mx_gemm_kernel<Work>, g) != cudaSuccess) return MXQ_ERR_CUDA;
  return launch_status();
}

// Store pause of a tile with nk stages (see pace): a thread's stores of one tile are
// spread over roughly a third to a half of the next tile's main loop, modeled as nk
// stages of 64 ns (E4M3/E5M2) or 128 ns (E2M1; its stages are longer and its ring
// more sensitive to load latency), capped at 1 us per store.  Calibrated by timing
// 64-512 ns pauses on the block-pass shapes.  stores: 32-byte stores per row.
inline __host__ __device__ uint32_t pace_of(int nk, bool fp4, int stores) {
  const int64_t ns = int64_t(nk) * (fp4 ? 128 : 64) / stores;
  return static_cast<uint32_t>(ns < 1000 ? ns : 1000);
}

}  // namespace
}  // namespace mxq
