// tcgen05, tensor-memory and cluster helpers shared by the tensor-core GEMMs.
#pragma once

#include <cmath>

#include "mxq_common.cuh"

namespace mxq {

// ---- tcgen05 / cluster wrappers --------------------------------------------
MXQ_DEV void tmem_alloc_pair(uint32_t dst_smem, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

MXQ_DEV void tmem_dealloc_pair(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
               : "memory");
}

MXQ_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
MXQ_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrive (once the pair's earlier tcgen05 operations complete) on the
// barrier at `bar`'s offset in every CTA of cta_mask.
MXQ_DEV void tc_commit_pair_mc(uint32_t bar, uint16_t cta_mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"(cta_mask)
      : "memory");
}

// Shared-memory matrix descriptor: start, leading / stride byte offsets,
// descriptor version 1, layout (0 = no swizzle, 2 = 128-byte swizzle).
MXQ_DEV uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(layout & 7u) << 61;
  return d;
}

#define MXQ_TMEM_LD32(taddr, r)                                                                  \
  asm volatile(                                                                                  \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "    \
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "    \
      "%28, %29, %30, %31}, [%32];"                                                              \
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),     \
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), \
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),           \
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),           \
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])            \
      : "r"(taddr))

// 256-bit global store of eight 32-bit words (32-byte aligned address).
MXQ_DEV void st_global_v8(void* p, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t a4,
                          uint32_t a5, uint32_t a6, uint32_t a7) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a0),
               "r"(a1), "r"(a2), "r"(a3), "r"(a4), "r"(a5), "r"(a6), "r"(a7)
               : "memory");
}

MXQ_DEV void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

MXQ_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

MXQ_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Address of the same shared-memory location in CTA `rank` of the cluster.
MXQ_DEV uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Arrive, without release semantics, on a barrier that may live in another
// CTA of the cluster.  The epilogue uses it to hand the accumulator back: its tensor-memory loads have already completed
// (tcgen05.wait::ld), which is all the next tile's MMAs need, while a
// release arrive would also wait for the thread's earlier global stores
// (the previous tile's output) to complete -- about 1700 cycles per tile
// in which the tensor pipe sat idle.
MXQ_DEV void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// Store a word into shared memory of a CTA of the cluster (`addr` from mapa).
MXQ_DEV void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.release.cluster.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

MXQ_DEV bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// A bounded wait (cluster-scope acquire) that also gives up once another
// role of this CTA has aborted.
MXQ_DEV bool gwait(uint32_t bar, uint32_t parity, uint64_t limit, volatile int* abort_flag) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (*abort_flag) return false;
    if (global_ns() - t0 > limit) return false;
  }
  return true;
}

// TMA load whose completion is signalled on a barrier that may live in the
// peer CTA of the pair (`bar` is a cluster shared-memory address).
MXQ_DEV void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                              int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// ---- tile order ---------------------------------------------------------------
// Work item t -> (mp, nt).  Tiles are visited in groups of `group` rows (or
// columns, when group_n): inside a group the grouped index runs fastest, so
// the clusters working at one time cover `group` panels of one operand and a
// few of the other, and the grouped operand's panels stay in L2 while the
// group sweeps the other dimension.
template <typename Args>
MXQ_DEV void tile_coords(int t, const Args& a, int& mp, int& nt) {
  const int n_g = a.group_n ? a.n_nt : a.n_mp;   // grouped dimension
  const int n_o = a.group_n ? a.n_mp : a.n_nt;   // swept dimension
  const int per_group = a.group * n_o;
  const int g = t / per_group;
  const int first = g * a.group;
  const int size = min(a.group, n_g - first);
  const int local = t - g * per_group;
  const int gi = first + local % size, oi = local / size;
  mp = a.group_n ? oi : gi;
  nt = a.group_n ? gi : oi;
}

// Group size and orientation of tile_coords.  The grouped panels (`panel`
// bytes each) are touched by every wave of the group and stay in L2 (budget
// 64 MB); the swept operand streams from DRAM once per group.  Modeled DRAM
// bytes: grouped_total + swept_total * n_groups; the orientation and group
// size with the fewest bytes win.
inline void choose_raster(int n_mp, int n_nt, double a_bytes, double b_bytes, double panel,
                          int32_t& group, int32_t& group_n) {
  const double l2_budget = 64.0 * (1 << 20);
  const int g_fit = static_cast<int>(std::max(1.0, std::floor(l2_budget / panel)));
  double best = -1.0;
  for (int orient = 0; orient < 2; ++orient) {
    const int n_g = orient ? n_nt : n_mp;
    const double grouped = orient ? b_bytes : a_bytes, swept = orient ? a_bytes : b_bytes;
    for (int g = 1; g <= std::min(g_fit, n_g); ++g) {
      const double bytes = grouped + swept * std::ceil(double(n_g) / g);
      if (best < 0.0 || bytes < best - 1.0) {
        best = bytes;
        group_n = orient;
        group = g;
      }
    }
  }
}

}  // namespace mxq
