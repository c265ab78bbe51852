// Rows of a buffer sorted by expert: which row each choice of the router gets, tokens
// gathered into the rows, rows summed back into the tokens, and that sum's gradients.
//
// Order: a stable counting sort of the choices by expert.  With h(b, e) the choices of
// expert e in block b of the choices,
//   counts[e] = sum_b h(b, e),  offsets[e] = sum_{e' < e} ceil(counts[e'] / align) align,
//   row of a choice = offsets[e] + sum_{b' < b} h(b', e) + its rank in its block.
// Ranks come from votes between the lanes and sums over warps in a fixed order, never
// from the order of atomics, so a routing always gives the same rows.  Latency bounds it:
// 65536 choices of 64 experts take 8.6 us in two launches (11.8 us with the vote on whole
// numbers, taken twice), 4096 take 5.9 us in one.
//
// Gather, combine and their gradients move rows: a team of 32 to 256 threads holds a
// token and all rows of its choices, so that a token's row is read (or written) once.
// 8192x8 tokens of 64 experts x 4096 bf16: gather 96.5 us (6.3 TB/s), combine 88 us (6.8
// TB/s), its gradients 188 us (6.1 TB/s); a plain copy reaches 6.7 TB/s.
#include <mutex>

#include "fp8_common.cuh"
#include "mxq_host.h"

namespace mxq {

__device__ uint32_t g_err_rows;

namespace {

constexpr int O_THREADS = 1024;
constexpr int O_WARPS = O_THREADS / 32;
constexpr int O_MAX_EXPERTS = 1024;
constexpr int O_MIN_BLOCK = 4096;    // choices of a block, at least
constexpr int O_MAX_BLOCKS = 152;
constexpr int O_KEPT = O_MIN_BLOCK / O_THREADS;   // steps of a warp in such a block

struct OrderArgs {
  const void* ids;
  int64_t n;              // choices
  int64_t block;          // choices of a block, a multiple of O_THREADS
  int32_t wide;           // ids are 64-bit
  int32_t experts, align;
  int32_t *row_of, *offsets, *counts;
  int32_t* hist;          // [blocks][experts]
};

// Expert of choice i, or -1 for one that goes to no expert.
MXQ_DEV int expert_of(const OrderArgs& a, int64_t i) {
  int64_t e = a.wide ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
  return e >= 0 && e < a.experts ? static_cast<int>(e) : -1;
}

// Lanes whose choice is of the same expert (none is -1, which stands for itself).  One vote
// per bit of an expert's number; the vote on whole numbers takes a turn per distinct one.
MXQ_DEV uint32_t same_expert(int e, int bits) {
  const uint32_t live = __ballot_sync(~0u, e >= 0);
  uint32_t same = e >= 0 ? live : ~live;
  for (int b = 0; b < bits; ++b) {
    const bool one = (e >> b) & 1;
    const uint32_t ones = __ballot_sync(~0u, one);
    same &= one ? ones : ~ones;
  }
  return same;
}

__global__ void __launch_bounds__(O_THREADS) order_count(const OrderArgs a) {
  extern __shared__ int32_t hist[];
  griddep_wait();
  griddep_launch_dependents();
  for (int e = threadIdx.x; e < a.experts; e += O_THREADS) hist[e] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * a.block, end = min(first + a.block, a.n);
  for (int64_t i = first + threadIdx.x; i < end; i += O_THREADS) {
    const int e = expert_of(a, i);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += O_THREADS)
    a.hist[int64_t(blockIdx.x) * a.experts + e] = hist[e];
}

// hist of all blocks -> offsets and counts (block 0) and the rows of this block's choices.
__global__ void __launch_bounds__(O_THREADS) order_rows(const OrderArgs a) {
  extern __shared__ int32_t next[];   // [warps][experts]: the warp's next row of an expert
  __shared__ int32_t sums[O_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t part = a.block / O_WARPS;   // a warp's choices, a multiple of 32
  const int64_t first = blockIdx.x * a.block + warp * part;
  const int64_t end = min(first + part, a.n);
  int32_t* mine = next + warp * a.experts;
  griddep_wait();
  griddep_launch_dependents();
  for (int i = threadIdx.x; i < O_WARPS * a.experts; i += O_THREADS) next[i] = 0;
  __syncthreads();
  const int bits = 32 - __clz(a.experts - 1);
  auto look = [&](int64_t i, int& x, uint32_t& same) {
    x = i + lane < end ? expert_of(a, i + lane) : -1;
    same = same_expert(x, bits);
  };
  auto count = [&](int x, uint32_t same) {
    if (x >= 0 && lane == __ffs(same) - 1) mine[x] += __popc(same);
    __syncwarp();
  };
  int kept_x[O_KEPT];   // the first choices of the warp, looked at once
  uint32_t kept[O_KEPT];
#pragma unroll
  for (int q = 0; q < O_KEPT; ++q)
    if (first + 32 * q < end) look(first + 32 * q, kept_x[q], kept[q]);
#pragma unroll
  for (int q = 0; q < O_KEPT; ++q)
    if (first + 32 * q < end) count(kept_x[q], kept[q]);
  for (int64_t i = first + 32 * O_KEPT; i < end; i += 32) {
    int x;
    uint32_t same;
    look(i, x, same);
    count(x, same);
  }
  __syncthreads();
  const int e = threadIdx.x;
  int before = 0, total = 0;
  if (e < a.experts) {
    if (gridDim.x == 1) {
      for (int w = 0; w < O_WARPS; ++w) total += next[w * a.experts + e];
    } else {
      const int nb = static_cast<int>(gridDim.x);
#pragma unroll 8
      for (int b = 0; b < nb; ++b) {
        const int h = a.hist[int64_t(b) * a.experts + e];
        total += h;
        if (b < static_cast<int>(blockIdx.x)) before += h;
      }
    }
  }
  const int rows = (total + a.align - 1) / a.align * a.align;
  int upto = rows;   // inclusive sum over the experts
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += sums[w];
  if (e < a.experts) {
    if (blockIdx.x == 0) {
      if (e == 0) a.offsets[0] = 0;
      a.offsets[e + 1] = upto;
      a.counts[e] = total;
    }
    int at = upto - rows + before;
    for (int w = 0; w < O_WARPS; ++w) {
      const int h = next[w * a.experts + e];
      next[w * a.experts + e] = at;
      at += h;
    }
  }
  __syncthreads();
  auto place = [&](int64_t i, int x, uint32_t same) {
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int row = x >= 0 ? mine[x] + rank : -1;
    __syncwarp();
    if (x >= 0 && rank == 0) mine[x] += __popc(same);
    __syncwarp();
    if (i + lane < end && MXQ_IN_BOUNDS(i + lane < a.n, &g_err_rows, SITE_B_EXPERT_ROWS))
      a.row_of[i + lane] = row;
  };
#pragma unroll
  for (int q = 0; q < O_KEPT; ++q)
    if (first + 32 * q < end) place(first + 32 * q, kept_x[q], kept[q]);
  for (int64_t i = first + 32 * O_KEPT; i < end; i += 32) {
    int x;
    uint32_t same;
    look(i, x, same);
    place(i, x, same);
  }
}

// ---- rows -------------------------------------------------------------------------

struct RowsArgs {
  const void* x;             // [tokens][cols]: the tokens, or the gradient of their sums
  const void* y;             // [rows][cols]
  void* out;                 // gather, combine_backward: [rows][cols]; combine: [tokens][cols]
  const int32_t* row_of;     // [tokens][topk]
  const int32_t *offsets, *counts;
  const float* weights;      // [tokens][topk], or NULL: ones
  float* dweights;           // [tokens][topk]
  int64_t tokens, rows, cols;
  int32_t topk, experts, team;
  int32_t parts;             // teams that clear an expert's padding
  int64_t units;             // tokens and experts' parts
};

constexpr int R_THREADS = 256;
constexpr int R_MOST = 8;   // choices handled together, at most

// Rows of up to G choices of a token from j0 on and their weights.  ready() puts -1 and
// weight 0 where a choice has no row, so that what follows needs no branches; a row
// outside the buffer is reported and left out.
template <int G>
struct Choices {
  int32_t row[G];
  float w[G];
  MXQ_DEV void load(const RowsArgs& a, int64_t t, int j0) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const bool is = t < a.tokens && j0 + j < a.topk;
      row[j] = is ? a.row_of[t * a.topk + j0 + j] : -1;
      w[j] = is && a.weights ? a.weights[t * a.topk + j0 + j] : 1.0f;
    }
  }
  MXQ_DEV void ready(const RowsArgs& a) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (row[j] >= a.rows) {
        bad = true;
        row[j] = -1;
      }
      if (row[j] < 0) w[j] = 0.0f;
    }
    if (bad) record_error(&g_err_rows, MXQ_ERR_ARG, SITE_EXPERT_ROW);
  }
};

// Eight bf16 or four fp32 elements of a row, as they lie in memory.  VEC: 16 consecutive
// bytes (rows on 16-byte boundaries).  Else one element in every `stride`, so that the
// accesses of neighbouring threads still touch neighbouring elements; `left` elements of
// the row remain from p on.
template <typename T, bool VEC>
struct Piece;

template <typename T>
struct Piece<T, true> {
  static constexpr int N = 16 / sizeof(T);
  static constexpr int REACH = N;   // elements from a thread's piece to its neighbour's
  uint4 v;
  MXQ_DEV void load(const T* p, int, int64_t) { v = *reinterpret_cast<const uint4*>(p); }
  MXQ_DEV void clear() { v = make_uint4(0u, 0u, 0u, 0u); }
  MXQ_DEV void store(T* p, int, int64_t) const { *reinterpret_cast<uint4*>(p) = v; }
  MXQ_DEV void get(float (&f)[N]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(w[i]);
      else f[i] = i & 1 ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]);
    }
  }
  MXQ_DEV void set(const float (&f)[N]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(f[i]);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename T>
struct Piece<T, false> {
  static constexpr int N = 4;
  static constexpr int REACH = 1;
  T v[N];
  MXQ_DEV void load(const T* p, int stride, int64_t left) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i * stride < left ? p[i * stride] : T(0.0f);
  }
  MXQ_DEV void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = T(0.0f);
  }
  MXQ_DEV void store(T* p, int stride, int64_t left) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * stride < left) p[i * stride] = v[i];
  }
  MXQ_DEV void get(float (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = static_cast<float>(v[i]);
  }
  MXQ_DEV void set(const float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = f[i];
      else v[i] = __float2bfloat16_rn(f[i]);
    }
  }
};

// Zeros in the rows between an expert's choices and the next expert's rows, by the
// teams behind the tokens': team `u` of them takes every parts-th row of an expert's.
template <typename T, bool VEC>
MXQ_DEV void clear_padding(const RowsArgs& a, int64_t u, int at) {
  using P = Piece<T, VEC>;
  if (u >= a.units - a.tokens) return;
  P zero;
  zero.clear();
  const int e = static_cast<int>(u) % a.experts, part = static_cast<int>(u) / a.experts;
  const int64_t lo = max(int64_t(a.offsets[e]) + a.counts[e], int64_t(0));
  const int64_t hi = min(int64_t(a.offsets[e + 1]), a.rows);
  for (int64_t r = lo + part; r < hi; r += a.parts)
    for (int64_t c = int64_t(at) * P::REACH; c < a.cols; c += int64_t(a.team) * P::N)
      zero.store(static_cast<T*>(a.out) + r * a.cols + c, a.team, a.cols - c);
}

// Teams walk the tokens (and, past them, the padding that they clear) a grid apart, and
// load a token's choices while the one before is on its way.
struct Team {
  int at, threads;   // place in the team, its size
  int64_t t, step;   // first token, tokens from one to the next
  MXQ_DEV explicit Team(const RowsArgs& a) : threads(a.team) {
    const int per = R_THREADS / a.team;
    at = threadIdx.x & (a.team - 1);
    t = int64_t(blockIdx.x) * per + threadIdx.x / a.team;
    step = int64_t(gridDim.x) * per;
  }
};

// The pieces of all choices' rows at column c.  VEC: a choice without a row reads the
// first one, which is there and not used, because a branch around a load makes the next
// one wait (combine, 8192x8 tokens x 4096 bf16: 141 us with branches, 117 us without).
// Unaligned rows have a load per element and more of them in flight; leaving out those
// of no use is worth more there (backward, 4099x3 x 1001 fp32: 25.5 us, else 33.2 us).
template <typename T, bool VEC, int G>
MXQ_DEV void load_rows(Piece<T, VEC> (&v)[G], const Choices<G>& k, const T* y, const RowsArgs& a,
                       const Team& team, int64_t c) {
#pragma unroll
  for (int j = 0; j < G; ++j) {
    if constexpr (VEC) {
      v[j].load(y + max(k.row[j], 0) * a.cols, team.threads, a.cols - c);
    } else {
      v[j].clear();
      if (k.row[j] >= 0) v[j].load(y + k.row[j] * a.cols, team.threads, a.cols - c);
    }
  }
}

template <typename T, bool VEC, int G>
__global__ void __launch_bounds__(R_THREADS) expert_gather(const RowsArgs a) {
  using P = Piece<T, VEC>;
  griddep_wait();
  griddep_launch_dependents();
  const Team team(a);
  T* out = static_cast<T*>(a.out);
  Choices<G> next;
  next.load(a, team.t, 0);
  int64_t t = team.t;
  for (; t < a.tokens; t += team.step) {
    Choices<G> k = next;
    next.load(a, t + team.step, 0);
    const T* x = static_cast<const T*>(a.x) + t * a.cols;
    for (int j0 = 0; j0 < a.topk; j0 += G) {
      if (j0) k.load(a, t, j0);
      k.ready(a);
      for (int64_t c = int64_t(team.at) * P::REACH; c < a.cols; c += int64_t(team.threads) * P::N) {
        P v;
        v.load(x + c, team.threads, a.cols - c);
        float f[P::N];
        v.get(f);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          if (k.row[j] < 0) continue;
          P s = v;
          if (a.weights) {
            float g[P::N];
#pragma unroll
            for (int i = 0; i < P::N; ++i) g[i] = f[i] * k.w[j];
            s.set(g);
          }
          s.store(out + k.row[j] * a.cols + c, team.threads, a.cols - c);
        }
      }
    }
  }
  for (; t < a.units; t += team.step) clear_padding<T, VEC>(a, t - a.tokens, team.at);
}

// out[t] = sum_j w[t][j] y[row of (t, j)], in the order of j, in fp32.  The loads of all
// choices are in flight together.
template <typename T, bool VEC, int G>
__global__ void __launch_bounds__(R_THREADS) expert_combine(const RowsArgs a) {
  using P = Piece<T, VEC>;
  griddep_wait();
  griddep_launch_dependents();
  const Team team(a);
  const T* y = static_cast<const T*>(a.y);
  Choices<G> next;
  next.load(a, team.t, 0);
  for (int64_t t = team.t; t < a.tokens; t += team.step) {
    Choices<G> k = next;
    next.load(a, t + team.step, 0);
    k.ready(a);
    for (int64_t c = int64_t(team.at) * P::REACH; c < a.cols; c += int64_t(team.threads) * P::N) {
      float sum[P::N];
#pragma unroll
      for (int i = 0; i < P::N; ++i) sum[i] = 0.0f;
      for (int j0 = 0; j0 < a.topk; j0 += G) {
        if (a.topk > G) {
          k.load(a, t, j0);
          k.ready(a);
        }
        P v[G];
        load_rows(v, k, y + c, a, team, c);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          float f[P::N];
          v[j].get(f);
#pragma unroll
          for (int i = 0; i < P::N; ++i)
            sum[i] = k.row[j] < 0 ? sum[i] : fmaf(k.w[j], f[i], sum[i]);
        }
      }
      P s;
      s.set(sum);
      s.store(static_cast<T*>(a.out) + t * a.cols + c, team.threads, a.cols - c);
    }
  }
}

// The same for aligned rows, with the rows' pieces on their way into shared memory while
// those of the two units before are summed (a unit: a thread's piece of all rows of a
// token).  Every thread copies and reads its own 16 bytes of a row, so no barrier is
// needed, and no registers hold what is in flight.
constexpr int C_AHEAD = 2;

template <typename T, int G>
__global__ void __launch_bounds__(R_THREADS) expert_combine_ring(const RowsArgs a) {
  using P = Piece<T, true>;
  extern __shared__ uint4 ring[];   // [C_AHEAD + 1][G][R_THREADS]
  griddep_wait();
  griddep_launch_dependents();
  const Team team(a);
  const T* const y = static_cast<const T*>(a.y);
  T* const out = static_cast<T*>(a.out);
  const int64_t c0 = int64_t(team.at) * P::REACH, step = int64_t(team.threads) * P::N;
  if (team.t >= a.tokens || c0 >= a.cols) return;
  uint4* const mine = ring + threadIdx.x;
  // the unit that is fetched next; its token's choices, loaded when the last one's were used
  int64_t ft = team.t, fc = c0;
  Choices<G> k;
  k.load(a, ft, 0);
  int put = 0;
  auto fetch = [&] {
    if (ft < a.tokens) {
      if (fc == c0) k.ready(a);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int bytes = k.row[j] < 0 ? 0 : 16;   // none: zeros are written
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         smem_u32(mine + (put * G + j) * R_THREADS)),
                     "l"(y + max(k.row[j], 0) * a.cols + fc), "r"(bytes)
                     : "memory");
      }
      fc += step;
      if (fc >= a.cols) {
        fc = c0;
        ft += team.step;
        k.load(a, ft, 0);
      }
      put = put == C_AHEAD ? 0 : put + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < C_AHEAD; ++i) fetch();
  int get = 0;
  for (int64_t t = team.t; t < a.tokens; t += team.step) {
    Choices<G> now;   // read anew: they are in the first-level cache
    now.load(a, t, 0);
    for (int64_t c = c0; c < a.cols; c += step) {
      fetch();
      asm volatile("cp.async.wait_group %0;" ::"n"(C_AHEAD) : "memory");
      if (c == c0) now.ready(a);
      float sum[P::N];
#pragma unroll
      for (int i = 0; i < P::N; ++i) sum[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        P v;
        v.v = mine[(get * G + j) * R_THREADS];
        float f[P::N];
        v.get(f);
#pragma unroll
        for (int i = 0; i < P::N; ++i) sum[i] = now.row[j] < 0 ? sum[i] : fmaf(now.w[j], f[i], sum[i]);
      }
      get = get == C_AHEAD ? 0 : get + 1;
      P r;
      r.set(sum);
      r.store(out + t * a.cols + c, team.threads, a.cols - c);
    }
  }
}

// out[row of (t, j)] = w[t][j] x[t],  dweights[t][j] = <x[t], y[row of (t, j)]>.  out may
// be y: a thread reads a piece of all its rows before it writes any.
template <typename T, bool VEC, int G>
__global__ void __launch_bounds__(R_THREADS) expert_combine_backward(const RowsArgs a) {
  using P = Piece<T, VEC>;
  __shared__ float part[2][R_THREADS / 32][G];
  griddep_wait();
  griddep_launch_dependents();
  const Team team(a);
  const T* y = static_cast<const T*>(a.y);
  T* out = static_cast<T*>(a.out);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Choices<G> next;
  next.load(a, team.t, 0);
  int64_t t = team.t;
  int turn = 0;
  // a CTA's teams make the same number of turns: the sums between its warps need all
  const int64_t first = int64_t(blockIdx.x) * (R_THREADS / a.team);
  for (int64_t block = first; block < a.tokens; block += team.step, t += team.step) {
    Choices<G> k = next;
    next.load(a, t + team.step, 0);
    const bool live = t < a.tokens;
    if (!live) clear_padding<T, VEC>(a, t - a.tokens, team.at);
    const T* x = static_cast<const T*>(a.x) + t * a.cols;
    for (int j0 = 0; j0 < a.topk; j0 += G, turn ^= 1) {
      if (j0) k.load(a, t, j0);
      k.ready(a);
      float dot[G];
#pragma unroll
      for (int j = 0; j < G; ++j) dot[j] = 0.0f;
      for (int64_t c = int64_t(team.at) * P::REACH; live && c < a.cols;
           c += int64_t(team.threads) * P::N) {
        P d, v[G];
        d.load(x + c, team.threads, a.cols - c);
        load_rows(v, k, y + c, a, team, c);
        float f[P::N];
        d.get(f);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          float g[P::N];
          v[j].get(g);
#pragma unroll
          for (int i = 0; i < P::N; ++i) {
            dot[j] = fmaf(f[i], g[i], dot[j]);
            g[i] = f[i] * k.w[j];
          }
          v[j].set(g);
        }
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (k.row[j] >= 0) v[j].store(out + k.row[j] * a.cols + c, team.threads, a.cols - c);
      }
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float s = k.row[j] >= 0 ? dot[j] : 0.0f;
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        if (lane == 0) part[turn][warp][j] = s;
      }
      // two buffers in turn: whoever writes one again has passed the barrier of the
      // other, behind this one's readers
      __syncthreads();
      if (live && team.at < G && j0 + team.at < a.topk) {
        float s = 0.0f;
        for (int v = 0; v < team.threads / 32; ++v) s += part[turn][warp + v][team.at];
        a.dweights[t * a.topk + j0 + team.at] = s;
      }
    }
  }
  for (; t < a.units; t += team.step) clear_padding<T, VEC>(a, t - a.tokens, team.at);
}

// The same for aligned rows and more than four choices, with the pieces two units ahead as
// in expert_combine_ring (8192x8 x 4096 bf16: 210 us in registers, 188 us).  With fewer
// choices the registers hold as much (4096x4 x 2048 fp32: 51.6 us, 53.8 us), and unaligned
// rows copied element by element lose (4099x3 x 1001 fp32: 25.5 us, 27.8 us).
template <typename T, int G>
__global__ void __launch_bounds__(R_THREADS) expert_combine_backward_ring(const RowsArgs a) {
  using P = Piece<T, true>;
  static_assert(sizeof(P) == 16, "a slot of the ring");
  extern __shared__ uint4 ring[];   // [C_AHEAD + 1][G + 1][R_THREADS], x's piece first
  __shared__ float part[2][R_THREADS / 32][G];
  griddep_wait();
  griddep_launch_dependents();
  const Team team(a);
  const T* const x = static_cast<const T*>(a.x);
  const T* const y = static_cast<const T*>(a.y);
  T* const out = static_cast<T*>(a.out);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c0 = int64_t(team.at) * P::REACH, step = int64_t(team.threads) * P::N;
  uint4* const mine = ring + threadIdx.x;
  int64_t ft = c0 < a.cols ? team.t : a.tokens, fc = c0;
  Choices<G> k;
  k.load(a, ft, 0);
  int put = 0;
  auto copy = [&](int slot, const T* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     smem_u32(mine + (put * (G + 1) + slot) * R_THREADS)),
                 "l"(from), "r"(bytes)
                 : "memory");
  };
  auto fetch = [&] {
    if (ft < a.tokens) {
      if (fc == c0) k.ready(a);
      copy(0, x + ft * a.cols + fc, 16);
#pragma unroll
      for (int j = 0; j < G; ++j)
        copy(1 + j, y + max(k.row[j], 0) * a.cols + fc, k.row[j] < 0 ? 0 : 16);
      fc += step;
      if (fc >= a.cols) {
        fc = c0;
        ft += team.step;
        k.load(a, ft, 0);
      }
      put = put == C_AHEAD ? 0 : put + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < C_AHEAD; ++i) fetch();
  int get = 0, turn = 0;
  int64_t t = team.t;
  // a CTA's teams make the same number of turns: the sums between its warps need all
  const int64_t first = int64_t(blockIdx.x) * (R_THREADS / a.team);
  for (int64_t block = first; block < a.tokens; block += team.step, t += team.step, turn ^= 1) {
    const bool live = t < a.tokens;
    if (!live) clear_padding<T, true>(a, t - a.tokens, team.at);
    Choices<G> now;   // read anew: they are in the first-level cache
    now.load(a, t, 0);
    now.ready(a);
    float dot[G];
#pragma unroll
    for (int j = 0; j < G; ++j) dot[j] = 0.0f;
    for (int64_t c = c0; live && c < a.cols; c += step) {
      fetch();
      asm volatile("cp.async.wait_group %0;" ::"n"(C_AHEAD) : "memory");
      const uint4* const unit = mine + get * (G + 1) * R_THREADS;
      float f[P::N];
      reinterpret_cast<const P*>(unit)->get(f);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if (now.row[j] < 0) continue;
        float g[P::N];
        reinterpret_cast<const P*>(unit + (1 + j) * R_THREADS)->get(g);
#pragma unroll
        for (int i = 0; i < P::N; ++i) {
          dot[j] = fmaf(f[i], g[i], dot[j]);
          g[i] = f[i] * now.w[j];
        }
        P s;
        s.set(g);
        s.store(out + now.row[j] * a.cols + c, team.threads, a.cols - c);
      }
      get = get == C_AHEAD ? 0 : get + 1;
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      float s = dot[j];
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      if (lane == 0) part[turn][warp][j] = s;
    }
    __syncthreads();   // two buffers in turn, as above
    if (live && team.at < a.topk) {
      float s = 0.0f;
      for (int v = 0; v < team.threads / 32; ++v) s += part[turn][warp + v][team.at];
      a.dweights[t * a.topk + team.at] = s;
    }
  }
  for (; t < a.units; t += team.step) clear_padding<T, true>(a, t - a.tokens, team.at);
}

enum RowsOp { GATHER, COMBINE, BACKWARD };

// Teams that the device holds at once, or as many as there are.
template <void (*KERNEL)(RowsArgs), int SMEM = 0>
bool rows_launch_resident(int64_t ctas, cudaStream_t st, const RowsArgs& a) {
  if (SMEM && !ensure_dynamic_smem(reinterpret_cast<const void*>(KERNEL), SMEM)) return false;
  static std::mutex mu;
  static int resident[64] = {0};   // CTAs of an SM, per device
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  {
    std::lock_guard<std::mutex> lock(mu);
    n = resident[dev];
  }
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, R_THREADS, SMEM) != cudaSuccess ||
        n <= 0) {
      cudaGetLastError();
      n = 1;
    }
    std::lock_guard<std::mutex> lock(mu);
    resident[dev] = n;
  }
  const int64_t grid = std::min<int64_t>(ctas, int64_t(n) * sm_count());
  return launch_early(KERNEL, static_cast<unsigned>(grid), R_THREADS, SMEM, st, a);
}

template <typename T, bool VEC, int G>
bool rows_launch_group(RowsOp op, int64_t ctas, cudaStream_t st, const RowsArgs& a) {
  switch (op) {
    // one token a team: its stores wait for nothing (8192x8 x 4096 bf16 with the order:
    // 107 us; 118 us where teams walk the tokens)
    case GATHER:
      return launch_early(expert_gather<T, VEC, G>, static_cast<unsigned>(ctas), R_THREADS, 0, st,
                          a);
    case COMBINE: {
      constexpr int SMEM = (C_AHEAD + 1) * G * R_THREADS * 16;
      if constexpr (VEC && G < R_MOST) {   // no more choices than G
        return rows_launch_resident<expert_combine_ring<T, G>, SMEM>(ctas, st, a);
      } else {
        if constexpr (VEC)
          if (a.topk <= G)
            return rows_launch_resident<expert_combine_ring<T, G>, SMEM>(ctas, st, a);
        return rows_launch_resident<expert_combine<T, VEC, G>>(ctas, st, a);
      }
    }
    default: {
      constexpr int SMEM = (C_AHEAD + 1) * (G + 1) * R_THREADS * 16;
      if constexpr (VEC && G > 4 && G < R_MOST) {
        return rows_launch_resident<expert_combine_backward_ring<T, G>, SMEM>(ctas, st, a);
      } else {
        if constexpr (VEC && G > 4)
          if (a.topk <= G)
            return rows_launch_resident<expert_combine_backward_ring<T, G>, SMEM>(ctas, st, a);
        return rows_launch_resident<expert_combine_backward<T, VEC, G>>(ctas, st, a);
      }
    }
  }
}

// As many choices at a time as there are, rounded up to two, at most eight: the others'
// loads, registers and instructions (combine, 20000x6 x 512 fp32: 59 us with eight, 48 us
// with six).
template <typename T, bool VEC>
bool rows_launch(RowsOp op, int64_t ctas, cudaStream_t st, const RowsArgs& a) {
  if (a.topk <= 2) return rows_launch_group<T, VEC, 2>(op, ctas, st, a);
  if (a.topk <= 4) return rows_launch_group<T, VEC, 4>(op, ctas, st, a);
  if (a.topk <= 6) return rows_launch_group<T, VEC, 6>(op, ctas, st, a);
  return rows_launch_group<T, VEC, R_MOST>(op, ctas, st, a);
}

mxq_status rows_run(RowsOp op, const mxq_expert_rows_args* q, void* stream) {
  const int64_t lim = int64_t(1) << 31;
  if (!q || q->tokens < 0 || q->rows < 0 || q->cols < 0 || q->topk < 1 || q->tokens >= lim ||
      q->rows >= lim || q->cols >= lim || q->topk > 1024 || q->tokens * q->topk >= lim)
    return MXQ_ERR_ARG;
  if (q->dtype != MXQ_OUT_F32 && q->dtype != MXQ_OUT_BF16) return MXQ_ERR_ARG;
  const bool pads = op != COMBINE;
  if (pads && (q->experts < 1 || q->experts > O_MAX_EXPERTS)) return MXQ_ERR_ARG;
  if (q->tokens == 0 || (q->cols == 0 && op != BACKWARD)) return MXQ_OK;
  // an empty buffer has no address
  const bool x = op != COMBINE && q->cols, y = op != GATHER && q->rows && q->cols;
  const bool out = op == COMBINE || (q->rows && q->cols);
  if (!q->row_of || (x && !q->x) || (y && !q->y) || (out && !q->out) ||
      (pads && (!q->offsets || !q->counts)) || (op == BACKWARD && !q->dweights))
    return MXQ_ERR_ARG;
  const void* words[] = {q->row_of, q->offsets, q->counts, q->weights, q->dweights};
  for (const void* p : words)
    if (!aligned4(p)) return MXQ_ERR_ALIGN;
  const void* data[] = {q->x, q->y, q->out};
  for (const void* p : data)
    if (!aligned16(p)) return MXQ_ERR_ALIGN;
  if (op != GATHER && (q->rows == 0 || q->cols == 0)) {   // no choice has a row: sums of nothing
    const size_t size = q->dtype == MXQ_OUT_BF16 ? 2 : 4;
    const size_t bytes = op == COMBINE ? size_t(q->tokens) * q->cols * size
                                       : size_t(q->tokens) * q->topk * 4;
    void* const sums = op == COMBINE ? q->out : q->dweights;
    return cudaMemsetAsync(sums, 0, bytes, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MXQ_OK : MXQ_ERR_CUDA;
  }
  RowsArgs a = {};
  a.x = q->x;
  a.y = q->y;
  a.out = q->out;
  a.row_of = q->row_of;
  a.offsets = q->offsets;
  a.counts = q->counts;
  a.weights = q->weights;
  a.dweights = q->dweights;
  a.tokens = q->tokens;
  a.rows = q->rows;
  a.cols = q->cols;
  a.topk = q->topk;
  a.experts = pads ? q->experts : 0;
  const bool bf16 = q->dtype == MXQ_OUT_BF16;
  const bool vec = q->cols % (bf16 ? 8 : 4) == 0;
  // as many threads as a row has pieces, at most a CTA
  const int64_t pieces = vec ? q->cols / (bf16 ? 8 : 4) : (q->cols + 3) / 4;
  a.team = 32;
  while (a.team < R_THREADS && a.team * 2 <= pieces) a.team *= 2;
  const int per = R_THREADS / a.team;
  // The buffer says how long an expert's padding may be; only the device knows how long it
  // is.  A team has about 32 rows (gather, 8192x8 of 64 x 4096 bf16: at an align of 4096
  // 307 us, 898 us with one team an expert; at 256 106 and 147 us; at 32 it is one team).
  const int64_t choices = a.tokens * a.topk;
  const int64_t padding = a.experts ? (a.rows - choices) / std::min<int64_t>(a.experts, choices) : 0;
  a.parts = static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>((padding + 31) / 32, 1), 128));
  a.units = a.tokens + int64_t(a.experts) * a.parts;
  const int64_t grid = (a.units + per - 1) / per;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  const bool ok = bf16 ? (vec ? rows_launch<B, true>(op, grid, st, a)
                              : rows_launch<B, false>(op, grid, st, a))
                       : (vec ? rows_launch<float, true>(op, grid, st, a)
                              : rows_launch<float, false>(op, grid, st, a));
  return ok ? launch_status() : MXQ_ERR_CUDA;
}

// Choices of a block and the number of blocks.
void order_blocks(int64_t n, int64_t& block, int64_t& blocks) {
  const int64_t even = (n + O_MAX_BLOCKS - 1) / O_MAX_BLOCKS;
  block = std::max<int64_t>(O_MIN_BLOCK, (even + O_THREADS - 1) / O_THREADS * O_THREADS);
  blocks = (n + block - 1) / block;
}

bool order_sizes_ok(int64_t n, int experts, int align) {
  return n >= 0 && experts >= 1 && experts <= O_MAX_EXPERTS && align >= 1 && align <= 4096 &&
         n + int64_t(experts) * align < (int64_t(1) << 31);
}

}  // namespace

uint32_t take_rows_error() {
  uint32_t h = 0;
  if (cudaMemcpyFromSymbol(&h, g_err_rows, sizeof(h)) != cudaSuccess) return MXQ_ERR_CUDA;
  if (h) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_err_rows, &z, sizeof(z));
  }
  return h;
}

}  // namespace mxq

using namespace mxq;

extern "C" size_t mxq_expert_order_workspace_size(int64_t n, int experts) {
  if (!order_sizes_ok(n, experts, 1)) return 0;
  int64_t block, blocks;
  order_blocks(n, block, blocks);
  return blocks > 1 ? static_cast<size_t>(blocks * experts * 4) : 0;
}

extern "C" mxq_status mxq_expert_order(const void* ids, int id_bytes, int64_t n, int experts,
                                       int align, int32_t* row_of, int32_t* offsets,
                                       int32_t* counts, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  if (!order_sizes_ok(n, experts, align) || (id_bytes != 4 && id_bytes != 8)) return MXQ_ERR_ARG;
  if (!offsets || !counts || (n > 0 && (!ids || !row_of))) return MXQ_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(ids) & (id_bytes - 1)) != 0 || !aligned4(row_of) ||
      !aligned4(offsets) || !aligned4(counts) || !aligned4(workspace))
    return MXQ_ERR_ALIGN;
  OrderArgs a = {};
  int64_t blocks;
  order_blocks(n, a.block, blocks);
  if (blocks > 1) {
    if (!workspace || workspace_bytes < static_cast<size_t>(blocks * experts * 4))
      return MXQ_ERR_WORKSPACE;
  }
  a.ids = ids;
  a.n = n;
  a.wide = id_bytes == 8;
  a.experts = experts;
  a.align = align;
  a.row_of = row_of;
  a.offsets = offsets;
  a.counts = counts;
  a.hist = static_cast<int32_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int smem = O_WARPS * experts * 4;
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(order_rows), smem)) return MXQ_ERR_CUDA;
  if (blocks > 1 && !launch_early(order_count, static_cast<unsigned>(blocks), O_THREADS,
                                  size_t(experts) * 4, st, a))
    return MXQ_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(blocks, 1));
  if (!launch_early(order_rows, grid, O_THREADS, smem, st, a)) return MXQ_ERR_CUDA;
  return launch_status();
}

extern "C" mxq_status mxq_expert_gather(const mxq_expert_rows_args* args, void* stream) {
  return rows_run(GATHER, args, stream);
}

extern "C" mxq_status mxq_expert_combine(const mxq_expert_rows_args* args, void* stream) {
  return rows_run(COMBINE, args, stream);
}

extern "C" mxq_status mxq_expert_combine_backward(const mxq_expert_rows_args* args, void* stream) {
  return rows_run(BACKWARD, args, stream);
}
