// Block-scaled MX products grouped by expert, for rows that lie sorted by expert:
//   rows   C[r] = dec(A[r]) dec(B[e])^T       for the rows r of expert e (forward: the
//          tokens against the expert's weight; input gradient: against its transpose)
//   wgrad  C[e] = dec(A[:, r]) dec(B[:, r])^T over the rows r of expert e
// Expert e holds rows offsets[e] to offsets[e + 1]; only the device knows them, so no
// call waits for the host and a captured launch follows the routing.  They cut M in
// the first form and K in the second.
//
// A first kernel turns the offsets into a table (first row, first tile and first scale
// chunk of every expert) and rewrites row-major scales into the tensor cores' chunks,
// for every expert from a chunk of its own.  The product's kernel (gemm_kernel.cuh) then
// walks the tiles of all experts as one persistent grid.  With few rows to an expert
// there is no first kernel: the product's makes the table and A's chunks itself.
//
// rows: rows of a tile past the expert's end are the next expert's; they are computed
// and not stored.  Experts with few rows have tiles of their own (gemm_few.cuh).
// wgrad: offsets are multiples of an MMA's K (32 elements, E2M1 64), so the last stage of
// an expert issues one to four MMAs and none reads the next expert's codes; an expert
// without rows gets zeros.
#include <string.h>

#include "gemm_few.cuh"
#include "gemm_kernel.cuh"

namespace mxq {
namespace {

constexpr int X_MAX = 1024;                 // experts
constexpr int X_TABLE = 3 * (X_MAX + 1);    // words of the table

// What the table and the scale chunks are made from.
struct PrepareArgs {
  const int32_t* offsets;
  int32_t rows, experts;
  int32_t unit;            // offsets are multiples of it
  int32_t n_nt;            // rows: tiles along N
  int32_t tile_rows, chunk_rows;   // rows: of a tile, of a scale chunk of A
  int32_t tiles;           // wgrad: tiles of an expert
  int32_t stage_rows;      // wgrad: elements of K per stage
  int32_t stage_chunks;    // wgrad: chunks per stage
  int32_t* table;
  const uint8_t *sa, *sb;  // row-major scales; sb NULL: B's are in chunks already
  uint8_t *ca, *cb;
  int32_t lines_a, lines_b;   // wgrad: lines of A and of B; rows: lines of one expert's B
  int32_t kb, kcs;            // blocks in a line of scales, chunks per 128-line tile
};

// The table: off[experts + 1], tile0[experts + 1], sf0[experts + 1].  sf0 counts, in
// the form rows, 128-row tiles of A's scale chunks; in wgrad, chunks along K.
struct ExpertParams {
  CUtensorMap ta, tb, tsa, tsb;
  CUtensorMap tc;        // wgrad: C
  GArgs a;
  const int32_t* table;
  int32_t experts;
  int32_t b_tiles;       // rows: 128-line scale tiles of one expert's B
  int32_t stores;        // 32-byte stores per row of a tile
  PrepareArgs prep;      // few rows: the kernel makes its table itself
};

// The table from the offsets, by one warp.  Offsets that fall, lie outside the rows or
// split an MMA's K are moved to the nearest that do not, so that no tile leaves the
// buffers, and reported.
template <bool ALONG_K>
MXQ_DEV void make_table(const PrepareArgs& p, int32_t* table, bool report) {
  int32_t *off = table, *tile0 = off + p.experts + 1, *sf0 = tile0 + p.experts + 1;
  const int lane = threadIdx.x & 31;
  bool bad = false;
  auto placed = [&](int i) {
    const int raw = p.offsets[i];
    const int v = min(max(raw, 0), p.rows) / p.unit * p.unit;
    bad |= v != raw;
    return v;
  };
  int end = placed(0), tiles = 0, sfs = 0;
  if (lane == 0) {
    off[0] = end;
    tile0[0] = sf0[0] = 0;
  }
  for (int i = lane; i - lane < p.experts; i += 32) {
    const bool live = i < p.experts;
    int v = live ? placed(i + 1) : 0;
    const int own = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(~0u, v, d);
      if (lane >= d) v = max(v, o);
    }
    v = max(v, end);
    bad |= live && v != own;
    int before = __shfl_up_sync(~0u, v, 1);
    if (lane == 0) before = end;
    const int len = v - before;
    int nt, ns;
    if (ALONG_K) {
      nt = live ? p.tiles : 0;
      ns = (len + p.stage_rows - 1) / p.stage_rows * p.stage_chunks;
    } else {
      nt = (len + p.tile_rows - 1) / p.tile_rows * p.n_nt;
      ns = (len + p.chunk_rows - 1) / p.chunk_rows;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(~0u, nt, d), b = __shfl_up_sync(~0u, ns, d);
      if (lane >= d) {
        nt += a;
        ns += b;
      }
    }
    if (live) {
      off[i + 1] = v;
      tile0[i + 1] = tiles + nt;
      sf0[i + 1] = sfs + ns;
    }
    end = __shfl_sync(~0u, v, 31);
    tiles += __shfl_sync(~0u, nt, 31);
    sfs += __shfl_sync(~0u, ns, 31);
  }
  if (bad && report) record_error(&g_err_gemm, MXQ_ERR_ARG, SITE_EXPERT_OFFSETS);
}

// How a launch's tiles lie: 256 rows of an expert by 256 of its columns, stored straight
// from the accumulators or through shared memory; a weight gradient's 256x256; or T
// rows by 128 columns (gemm_few.cuh).
enum Form { ROWS, ROWS_STAGED, WGRAD, FEW16, FEW64 };

constexpr bool is_few(Form f) { return f == FEW16 || f == FEW64; }
constexpr int tile_rows(Form f) { return f == FEW16 ? 16 : f == FEW64 ? 64 : G_CLUSTER * G_BM; }
constexpr int tile_cols(Form f) { return is_few(f) ? W_LINES : G_BN; }
constexpr int chunk_rows(Form f) { return is_few(f) ? tile_rows(f) : G_BM; }   // of a scale chunk

template <Form FORM>
struct ExpertWork {
  using Params = ExpertParams;
  [[maybe_unused]] static constexpr bool PARTIAL = FORM == WGRAD, QUANTIZES = false;
  [[maybe_unused]] static constexpr StoreBy OUT =
      FORM == WGRAD ? STORE_TMA : FORM == ROWS_STAGED ? STORE_STAGED : STORE_DIRECT;
  // a stage less makes room for staged tiles
  [[maybe_unused]] static constexpr int STAGES = OUT == STORE_DIRECT ? 6 : 5;
  static constexpr int TABLE = (X_TABLE * 4 + 15) / 16 * 16;
  static constexpr int TR = tile_rows(FORM), TC = tile_cols(FORM);
  const ExpertParams& g;
  const int32_t *off, *tile0, *sf0;
  int e = 0;   // expert of the last item asked for

  MXQ_DEV ExpertWork(const ExpertParams& p, const void* table) : g(p) {
    off = static_cast<const int32_t*>(table);
    tile0 = off + g.experts + 1;
    sf0 = tile0 + g.experts + 1;
  }
  MXQ_DEV static const GArgs& first(const ExpertParams& g) { return g.a; }
  MXQ_DEV static void prefetch(const ExpertParams& g) {
    prefetch_tmap(&g.ta);
    prefetch_tmap(&g.tb);
    if (!is_few(FORM)) prefetch_tmap(&g.tsa);
    prefetch_tmap(&g.tsb);
    if (FORM == WGRAD) prefetch_tmap(&g.tc);
  }
  MXQ_DEV static void load(const ExpertParams& g, void* table) {
    if constexpr (is_few(FORM)) {
      if (threadIdx.x < 32) make_table<false>(g.prep, static_cast<int32_t*>(table), blockIdx.x == 0);
    } else {
      for (int i = threadIdx.x; i < 3 * (g.experts + 1); i += blockDim.x)
        static_cast<int32_t*>(table)[i] = g.table[i];
    }
  }
  static int table_bytes(const ExpertParams& g) { return 3 * (g.experts + 1) * 4; }
  MXQ_DEV static const CUtensorMap* store_map(const ExpertParams& g) { return &g.tc; }
  MXQ_DEV int tiles() const { return tile0[g.experts]; }
  MXQ_DEV Item at(int t) {
    while (e + 1 < g.experts && t >= tile0[e + 1]) ++e;
    const int lo = off[e], len = off[e + 1] - lo;
    Item it;
    it.a = &g.a;
    it.ta = &g.ta;
    it.tb = &g.tb;
    it.tsa = &g.tsa;
    it.tsb = &g.tsb;
    it.z = e;
    if constexpr (FORM == WGRAD) {
      const int bytes = g.a.fp4 ? len >> 1 : len;
      it.nk = (bytes + G_BKB - 1) / G_BKB;
      it.last = ((bytes - 1) % G_BKB) / 32 + 1;
      tile_coords(t - tile0[e], g.a, it.mp, it.nt);
      it.kx = g.a.fp4 ? lo >> 1 : lo;
      it.ay = it.mp * TR;
      it.by = it.nt * TC;
      it.sa = G_CLUSTER * it.mp * g.a.kc_per_row + sf0[e];
      it.sb = 2 * it.nt * g.a.kc_per_row + sf0[e];
      it.c0 = int64_t(e) * g.a.M;
      it.rows = g.a.M;
      it.pace_ns = pace_of(it.nk, g.a.fp4 != 0, g.stores);
    } else {
      it.nk = g.a.nk;
      it.last = 4;
      const int n_mp = (len + TR - 1) / TR;
      const Grid grid{n_mp, g.a.n_nt, is_few(FORM) ? n_mp : g.a.group, 0};
      tile_coords(t - tile0[e], grid, it.mp, it.nt);
      it.kx = 0;
      it.ay = lo + it.mp * TR;
      it.by = e * g.a.N + it.nt * TC;
      it.sa = (sf0[e] + it.mp * (TR / chunk_rows(FORM))) * g.a.kc_per_row;
      it.sb = (e * g.b_tiles + it.nt * (TC / G_BM)) * g.a.kc_per_row;
      it.c0 = lo;
      it.rows = len;
      it.pace_ns = g.a.pace_ns;
    }
    return it;
  }
  [[maybe_unused]] MXQ_DEV static bool inside(const Item& it) {
    return it.mp >= 0 && it.mp * TR < it.rows && it.nt >= 0 && it.nt < it.a->n_nt;
  }

 private:
  struct Grid {
    int n_mp, n_nt, group, group_n;
  };
};

// ---- the table and the scale chunks -------------------------------------------

// Largest i with first[i] <= at (first[0] == 0, first[n] > at).
MXQ_DEV int holder(const int32_t* first, int n, int at) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= at) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One 512-byte chunk by a warp: 128 lines from `line` on, the `n` blocks from `block`
// on; zeros for what is missing.  Lane l holds lines l, l + 32, l + 64, l + 96, whose
// words lie side by side.
MXQ_DEV void write_chunk(uint8_t* chunk, const uint8_t* s, int64_t line, int64_t lines, int64_t kb,
                         int64_t block, int n) {
  const int lane = threadIdx.x & 31;
  uint32_t w[4];
  // Lines lie at any byte: a word is cut out of the two aligned ones around it, eight loads
  // in flight per lane, unless those reach past the scales' ends or the line's.
  const uintptr_t begin = reinterpret_cast<uintptr_t>(s), end = begin + lines * kb;
  uint32_t lo[4], hi[4], shift[4];
  bool fast[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t r = line + lane + 32 * q;
    const uintptr_t at = begin + r * kb + block, word = at & ~uintptr_t(3);
    shift[q] = static_cast<uint32_t>(at & 3) * 8;
    fast[q] = r < lines && n >= 4 && word >= begin && word + 8 <= end;
    lo[q] = hi[q] = 0u;
    if (fast[q]) {
      lo[q] = reinterpret_cast<const uint32_t*>(word)[0];
      hi[q] = reinterpret_cast<const uint32_t*>(word)[1];
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t r = line + lane + 32 * q;
    w[q] = __funnelshift_r(lo[q], hi[q], shift[q]);
    if (!fast[q] && r < lines) w[q] = scale_word(s + r * kb + block, n);
  }
  *reinterpret_cast<uint4*>(chunk + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool ALONG_K>
__global__ void __launch_bounds__(256) experts_prepare(const PrepareArgs p) {
  __shared__ int32_t table[X_TABLE];
  const int32_t *off = table, *sf0 = off + 2 * (p.experts + 1);
  griddep_wait();
  griddep_launch_dependents();
  if (threadIdx.x < 32) make_table<ALONG_K>(p, table, blockIdx.x == 0);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < 3 * (p.experts + 1); i += blockDim.x) p.table[i] = table[i];

  const int64_t warp = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t warps = (int64_t(gridDim.x) * blockDim.x) >> 5;
  const int sf = sf0[p.experts];
  if (ALONG_K) {
    const int64_t tiles_a = (p.lines_a + 127) / 128, tiles_b = (p.lines_b + 127) / 128;
    for (int64_t u = warp; u < (tiles_a + tiles_b) * sf; u += warps) {
      const int64_t tile = u / sf;
      const int kc = static_cast<int>(u % sf), e = holder(sf0, p.experts, kc);
      const int block = off[e] / 32 + (kc - sf0[e]) * 4, n = off[e + 1] / 32 - block;
      const bool is_a = tile < tiles_a;
      const int64_t t = is_a ? tile : tile - tiles_a;
      if (!MXQ_IN_BOUNDS(kc < p.kcs && block >= 0 && block + min(n, 4) <= p.kb, &g_err_gemm,
                         SITE_B_EXPERT_CHUNKS))
        continue;
      write_chunk((is_a ? p.ca : p.cb) + (t * p.kcs + kc) * 512, is_a ? p.sa : p.sb, t * 128,
                  is_a ? p.lines_a : p.lines_b, p.kb, block, n);
    }
  } else {
    const int64_t tiles_b = (p.lines_b + 127) / 128;
    const int64_t units_a = p.sa ? int64_t(sf) * p.kcs : 0;   // few rows: B's chunks alone
    const int64_t units = units_a + (p.sb ? p.experts * tiles_b * p.kcs : 0);
    for (int64_t u = warp; u < units; u += warps) {
      const bool is_a = u < units_a;
      const int64_t v = is_a ? u : u - units_a, tile = v / p.kcs;
      const int kc = static_cast<int>(v % p.kcs);
      int64_t line, lines;
      if (is_a) {
        const int e = holder(sf0, p.experts, static_cast<int>(tile));
        line = off[e] + (tile - sf0[e]) * p.chunk_rows;
        lines = min(int64_t(off[e + 1]), line + p.chunk_rows);
      } else {
        const int64_t e = tile / tiles_b;
        line = e * p.lines_b + (tile % tiles_b) * 128;
        lines = (e + 1) * p.lines_b;
      }
      if (!MXQ_IN_BOUNDS(line >= 0 && (!is_a || lines <= p.rows), &g_err_gemm,
                         SITE_B_EXPERT_CHUNKS))
        continue;
      write_chunk((is_a ? p.ca : p.cb) + v * 512, is_a ? p.sa : p.sb, line, lines, p.kb,
                  int64_t(kc) * 4, p.kb - kc * 4);
    }
  }
}

// ---- sizes ----------------------------------------------------------------------

struct ExpertPlan {
  Form form;
  int64_t kbytes;              // bytes of a line of codes
  int64_t stage_rows;          // elements of a K stage
  int64_t stage_chunks;
  int64_t kcs;                 // chunks per 128-line tile
  int64_t tiles_a, tiles_b;    // 128-line tiles of scale chunks (rows: of all experts)
  int64_t n_mp, n_nt, items;   // n_mp: wgrad only; items: an upper bound for rows
  int64_t table, ws_a, ws_b;   // bytes
};

constexpr int64_t X_LIM = int64_t(1) << 31;

// The form of a rows product from its sizes; the device alone knows the experts' rows, so
// it goes by their average over the experts that can have any.  Measured, 64 experts of
// 4096x4096 E2M1 (2048x2048 E4M3), us at an average of 1 (of 8 experts), 8, 16, 32, 64
// (*: with the scales from a launch of their own, 3 us):
//   FEW16  17.1 (12.2)   85.8 (45.2)   89.4 (47.4)   118* (63.7*)  184* (96.5*)
//   FEW64  24.0* (16.6*) 90.7* (51.5*) 93.5* (52.5*) 101 (52.4)    108* (60.5*)
//   ROWS   27.2 (16.4)   97.3 (56.4)   102 (56.9)    105 (58.3)    108 (60.3)
// With one expert that has half or nine tenths of the rows instead (512 to 8192 rows of 64
// experts, 2048x2048 E4M3), the chosen form takes up to 1.2 times as long, and a buffer four
// times as long as its rows, which the average counts, changes that by 8 % at most.
// Through shared memory, the stores of a tile take less of the SM's memory path, and a
// stage of the ring less.  16 experts of 512 rows, N 2048, E4M3, us staged (direct):
//   stages of a tile      4           9            12           16           32
//   bf16                  21.8 (24.3) 31.2 (32.3)  36.4 (36.8)  44.7 (43.7)  75.9 (71.4)
//   fp32                  27.9 (32.1) 35.7 (40.0)  41.0 (44.2)  49.3 (51.6)  80.8 (78.4)
// E2M1 turns between 6 and 9 stages in bf16 (3 % at 12) and at 16 in fp32.  1233 rows of 7
// experts, N 1004, with less than a tile for every cluster, E4M3 fp32: 12 stages 13.3
// (15.6), 16 stages 14.9 (17.2).
Form rows_form(const mxq_experts_args& q, int64_t kbytes) {
  const int64_t average = q.rows / std::max<int64_t>(1, std::min<int64_t>(q.experts, q.rows));
  if (average <= 16) return FEW16;
  if (average <= 48) return FEW64;
  return kbytes <= 12 * G_BKB ? ROWS_STAGED : ROWS;
}

bool expert_plan(const mxq_experts_args& q, bool wgrad, ExpertPlan& p) {
  if (q.rows < 0 || q.N < 1 || q.experts < 1 || q.experts > X_MAX || q.rows >= X_LIM ||
      q.N >= X_LIM)
    return false;
  if (q.fmt != MXQ_E4M3 && q.fmt != MXQ_E2M1 && q.fmt != MXQ_E5M2) return false;
  const bool fp4 = q.fmt == MXQ_E2M1;
  p.stage_rows = fp4 ? 256 : 128;
  p.stage_chunks = fp4 ? 2 : 1;
  p.table = (3 * (int64_t(q.experts) + 1) * 4 + 255) / 256 * 256;
  if (wgrad) {
    if (q.M < 1 || q.M >= X_LIM || q.rows % 32 != 0) return false;
    p.form = WGRAD;
    p.n_nt = (q.N + G_BN - 1) / G_BN;
    const int64_t unit = fp4 ? 64 : 32;
    const int64_t stages =
        q.rows / p.stage_rows + std::min<int64_t>(q.experts, q.rows / unit) + 1;
    p.kbytes = fp4 ? q.rows / 2 : q.rows;
    p.kcs = stages * p.stage_chunks;
    p.tiles_a = (q.M + 127) / 128;
    p.tiles_b = (q.N + 127) / 128;
    p.n_mp = (q.M + G_CLUSTER * G_BM - 1) / (G_CLUSTER * G_BM);
    p.items = q.experts * p.n_mp * p.n_nt;
    p.ws_b = p.tiles_b * p.kcs * 512;
  } else {
    if (q.K < 32 || q.K >= X_LIM || q.K % 32 != 0 || q.experts * q.N >= X_LIM) return false;
    if (q.b_scale_layout != MXQ_SCALES_ROWMAJOR && q.b_scale_layout != MXQ_SCALES_TC) return false;
    p.kbytes = fp4 ? q.K / 2 : q.K;
    p.form = rows_form(q, p.kbytes);
    p.n_nt = (q.N + tile_cols(p.form) - 1) / tile_cols(p.form);
    p.kcs = (q.K + p.stage_rows - 1) / p.stage_rows * p.stage_chunks;
    p.tiles_a = q.rows / chunk_rows(p.form) + std::min<int64_t>(q.experts, q.rows);
    p.tiles_b = q.experts * ((q.N + 127) / 128);
    p.n_mp = 0;
    p.items = (q.rows / tile_rows(p.form) + std::min<int64_t>(q.experts, q.rows)) * p.n_nt;
    p.ws_b = q.b_scale_layout == MXQ_SCALES_TC ? 0 : p.tiles_b * p.kcs * 512;
  }
  p.ws_a = is_few(p.form) ? 0 : p.tiles_a * p.kcs * 512;   // few rows: chunks are made in place
  // tile numbers and chunk numbers are 32-bit (up to two tiles past the last are named)
  return p.items < X_LIM && (p.tiles_a + 2) * p.kcs < X_LIM && (p.tiles_b + 2) * p.kcs < X_LIM;
}

template <bool ALONG_K>
mxq_status experts_launch(const mxq_experts_args& q, void* stream) {
  ExpertPlan p;
  if (q.out_dtype != MXQ_OUT_F32 && q.out_dtype != MXQ_OUT_BF16) return MXQ_ERR_ARG;
  if (!expert_plan(q, ALONG_K, p)) return MXQ_ERR_ARG;
  const bool fp4 = q.fmt == MXQ_E2M1, bf16 = q.out_dtype == MXQ_OUT_BF16;
  const bool tc = !ALONG_K && q.b_scale_layout == MXQ_SCALES_TC;
  const bool few = is_few(p.form);
  if (tc && q.K % p.stage_rows != 0) return MXQ_ERR_ARG;
  if (q.N % (bf16 ? 8 : 4) != 0) return MXQ_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (q.rows == 0) {
    if (!ALONG_K) return MXQ_OK;
    if (!q.C) return MXQ_ERR_ARG;
    const size_t bytes = size_t(q.experts) * q.M * q.N * (bf16 ? 2 : 4);
    return cudaMemsetAsync(q.C, 0, bytes, st) == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
  }
  if (!q.A || !q.sA || !q.B || !q.sB || !q.offsets || !q.C || !q.workspace) return MXQ_ERR_ARG;
  if (!aligned16(q.A) || !aligned16(q.B) || !aligned16(q.C) || !aligned4(q.offsets) ||
      (tc && !aligned16(q.sB)) || (reinterpret_cast<uintptr_t>(q.workspace) & 255u) != 0)
    return MXQ_ERR_ALIGN;
  if (q.workspace_bytes < static_cast<size_t>(p.table + p.ws_a + p.ws_b)) return MXQ_ERR_WORKSPACE;

  uint8_t* ws = static_cast<uint8_t*>(q.workspace);
  PrepareArgs r = {};
  r.offsets = q.offsets;
  r.rows = static_cast<int32_t>(q.rows);
  r.experts = q.experts;
  r.unit = ALONG_K ? (fp4 ? 64 : 32) : 1;
  r.n_nt = static_cast<int32_t>(p.n_nt);
  r.tile_rows = tile_rows(p.form);
  r.chunk_rows = chunk_rows(p.form);
  r.tiles = static_cast<int32_t>(p.n_mp * p.n_nt);
  r.stage_rows = static_cast<int32_t>(p.stage_rows);
  r.stage_chunks = static_cast<int32_t>(p.stage_chunks);
  r.table = reinterpret_cast<int32_t*>(ws);
  r.sa = q.sA;
  r.sb = tc ? nullptr : q.sB;
  r.ca = ws + p.table;
  r.cb = r.ca + p.ws_a;
  r.lines_a = ALONG_K ? static_cast<int32_t>(q.M) : 0;
  r.lines_b = static_cast<int32_t>(q.N);
  r.kb = static_cast<int32_t>((ALONG_K ? q.rows : q.K) / 32);
  r.kcs = static_cast<int32_t>(p.kcs);

  ExpertParams g;
  memset(&g, 0, sizeof(g));
  const uint64_t kbytes = static_cast<uint64_t>(p.kbytes);
  const uint64_t lines_a = static_cast<uint64_t>(ALONG_K ? q.M : q.rows);
  const uint64_t lines_b = static_cast<uint64_t>(ALONG_K ? q.N : q.experts * q.N);
  const auto codes = [&](CUtensorMap* m, const void* base, uint64_t lines, int box) {
    return tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, kbytes, lines, kbytes, G_BKB,
                         static_cast<uint32_t>(box), CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
  };
  const auto chunks = [&](CUtensorMap* m, const void* base, int64_t tiles) {
    return tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, base, 128,
                         static_cast<uint64_t>(tiles * p.kcs), 512, 128,
                         static_cast<uint32_t>(p.stage_chunks), CU_TENSOR_MAP_SWIZZLE_NONE,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
  };
  if (!codes(&g.ta, q.A, lines_a, chunk_rows(p.form)) || !codes(&g.tb, q.B, lines_b, G_BM) ||
      (!few && !chunks(&g.tsa, r.ca, p.tiles_a)) ||
      !chunks(&g.tsb, tc ? static_cast<const void*>(q.sB) : r.cb, p.tiles_b))
    return MXQ_ERR_CUDA;
  if (ALONG_K) {
    const uint64_t size = bf16 ? 2 : 4;
    if (tensor_map_3d(&g.tc, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                      q.C, static_cast<uint64_t>(q.N), static_cast<uint64_t>(q.M),
                      static_cast<uint64_t>(q.experts), q.N * size, q.M * q.N * size,
                      static_cast<uint32_t>(128 / size), 32, 1, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_NONE) != CUDA_SUCCESS)
      return MXQ_ERR_CUDA;
  }
  GArgs& a = g.a;
  a.M = static_cast<int32_t>(ALONG_K ? q.M : 0);
  a.N = static_cast<int32_t>(q.N);
  a.n_mp = static_cast<int32_t>(p.n_mp);
  a.n_nt = static_cast<int32_t>(p.n_nt);
  a.nk = static_cast<int32_t>((p.kbytes + G_BKB - 1) / G_BKB);
  a.kc_per_row = static_cast<int32_t>(p.kcs);
  if (ALONG_K) {   // an expert of average length
    const double k = std::max(1.0, double(p.kbytes) / q.experts);
    choose_raster(a.n_mp, a.n_nt, q.M * k, q.N * k, 2 * G_BM * k, a.group, a.group_n);
  } else {
    // eight row tiles of an expert by the columns that the other clusters reach: about
    // as many lines of A as of B in flight, and B stays in L2 for the next eight
    a.group = 8;
  }
  a.C = q.C;
  a.out_bf16 = bf16;
  a.fp4 = fp4;
  a.elem_code = q.fmt == MXQ_E4M3 ? 0 : 1;
  a.wide_stores = (reinterpret_cast<uintptr_t>(q.C) & 31u) == 0 && q.N % (bf16 ? 16 : 8) == 0;
  g.stores = bf16 ? 8 : 16;
  a.pace_ns = pace_of(a.nk, fp4, g.stores);
  a.timeout_ns = wait_timeout_ns();
  g.table = r.table;
  g.experts = q.experts;
  g.b_tiles = static_cast<int32_t>((q.N + 127) / 128);

  g.prep = r;
  if (few) r.sa = nullptr;
  if (!few || !tc) {
    const int64_t units = ((few ? 0 : p.tiles_a) + (tc ? 0 : p.tiles_b)) * p.kcs;
    const unsigned grid =
        static_cast<unsigned>(std::min<int64_t>((units + 7) / 8, 8 * sm_count()));
    if (!launch_early(experts_prepare<ALONG_K>, grid, 256, 0, st, r)) return MXQ_ERR_CUDA;
  }
  if constexpr (ALONG_K) {
    return gemm_kernel_run<ExpertWork<WGRAD>>(g, p.items, stream);
  } else {
    switch (p.form) {
      case FEW16: return gemm_few_run<ExpertWork<FEW16>, 16>(g, p.items, stream);
      case FEW64: return gemm_few_run<ExpertWork<FEW64>, 64>(g, p.items, stream);
      case ROWS_STAGED: return gemm_kernel_run<ExpertWork<ROWS_STAGED>>(g, p.items, stream);
      default: return gemm_kernel_run<ExpertWork<ROWS>>(g, p.items, stream);
    }
  }
}

}  // namespace

uint32_t take_experts_error() {
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

extern "C" mxq_status mxq_gemm_experts(const mxq_experts_args* args, void* stream) {
  if (!args) return MXQ_ERR_ARG;
  return experts_launch<false>(*args, stream);
}

extern "C" mxq_status mxq_gemm_experts_wgrad(const mxq_experts_args* args, void* stream) {
  if (!args) return MXQ_ERR_ARG;
  return experts_launch<true>(*args, stream);
}

extern "C" size_t mxq_gemm_experts_workspace_size(int64_t rows, int64_t N, int64_t K, int experts,
                                                  int fmt, int b_scale_layout) {
  mxq_experts_args q = {};
  q.rows = rows;
  q.N = N;
  q.K = K;
  q.experts = experts;
  q.fmt = fmt;
  q.b_scale_layout = b_scale_layout;
  ExpertPlan p;
  if (!expert_plan(q, false, p)) return 0;
  return static_cast<size_t>(p.table + p.ws_a + p.ws_b);
}

extern "C" size_t mxq_gemm_experts_wgrad_workspace_size(int64_t rows, int64_t M, int64_t N,
                                                        int experts, int fmt) {
  mxq_experts_args q = {};
  q.rows = rows;
  q.M = M;
  q.N = N;
  q.experts = experts;
  q.fmt = fmt;
  ExpertPlan p;
  if (!expert_plan(q, true, p)) return 0;
  return static_cast<size_t>(p.table + p.ws_a + p.ws_b);
}
