// The routed experts with 16-bit weights: entry points, and products grouped by
// expert.
//
// Forward: x w1[e]^T with the gate in its epilogue, h w2[e]^T.  Backward: dh =
// dout w2[e] with the gate's derivative in its epilogue, dx rows = d_gate_up
// w1[e], dw1[e] = d_gate_up^T x and dw2[e] = dout^T h over expert e's rows.
//
// The rows of an expert are known on the device only, so a one-block kernel
// first lists the row tiles: whole ones (of 256, 128 or 64 rows, by the sizes of the
// call) and one for an expert's remainder, filed by what it needs (more than 128
// rows, 65 to 128, up to 64).  Every product of the call then takes its tiles from
// that list, the large ones first; the grid is what the rows could need at most,
// and blocks past the list's end return.  Few rows need no list.  A weight gradient
// has the same tiles for every expert and the expert's rows as its K.
//
// What bounds it: with a few rows an expert the reading of its weights (192 rows
// over 137 of 256 experts of 4096 x 2048: 1.07 to 1.14 ms, 6.0 to 6.4 TB/s); with
// many the dense tiles' K loop (dense_tile.h) and their ends, which one block a CU
// does not hide (49152 rows over 32 experts, forward and backward: 7.8 to 8.0 ms,
// 0.93 PFLOP/s).
#include <algorithm>

#include "dense_few.h"
#include "dense_small.h"
#include "dense_tile.h"

namespace mxmoe {
namespace {

constexpr int kMaxExperts = 8192;
constexpr int kClasses = 3;
// Tiles of an expert that go through all its columns together, so that they
// share its weights' tiles in the L2.  (Groups of four that did not mind where an
// expert ends: 32 experts of 1536 rows took 1737 us for 4096 x 4096 with the gate,
// one expert of all those rows 1586.)
constexpr int kTileGroup = 6;

// The list of row tiles: how many of each class, then their entries.
struct RowTile {
  int32_t expert, row, rows;   // rows [row, row + rows) of `expert`
  int32_t group;               // its group's first tile << 4 | tiles, for an expert's whole tiles
};
struct RowPlan {
  int32_t count[8];
  __host__ __device__ RowTile* list(int cls, int cap) {
    return reinterpret_cast<RowTile*>(this + 1) + (size_t)cls * cap;
  }
};
// Row tiles that the rows can make at most, in any class.
int tile_cap(int rows, int E) { return rows / 64 + std::min(E, rows) + 1; }
size_t plan_bytes(int rows, int E) {
  return align_up(sizeof(RowPlan) + (size_t)kClasses * tile_cap(rows, E) * sizeof(RowTile), 256);
}

// Expert e's rows, cut to [0, rows).
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int rows, int* first, int* count) {
  const int a = min(max(offsets[e], 0), rows), b = min(max(offsets[e + 1], a), rows);
  *first = a, *count = b - a;
}
__device__ __forceinline__ int tile_class(int rows) { return rows > 128 ? 0 : rows > 64 ? 1 : 2; }

// One block; thread t lists experts [t per, (t + 1) per) behind those of the
// threads before it.  Ascending offsets make cap tiles of a class at most.  Others can
// claim up to 2^22 tiles for each of 8192 experts, past 2^31 together: every sum stops
// at cap (64 lanes of up to cap < 2^23 each stay below 2^29, 16 waves below 2^27), and
// nothing is listed from there on.
__global__ __launch_bounds__(1024) void plan_rows_kernel(const int32_t* offsets, int E, int rows, int whole, int cap,
                                                         RowPlan* plan) {
  __shared__ int sums[16][kClasses];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = (E + blockDim.x - 1) / blockDim.x;
  const int e0 = min((int)threadIdx.x * per, E), wc = tile_class(whole);
  int n[kClasses] = {0, 0, 0}, at[kClasses], first = 0, count = 0;
  for (int i = 0; i < per; ++i) {
    count = 0;
    if (e0 + i < E) expert_rows(offsets, e0 + i, rows, &first, &count);
    n[wc] += count / whole;
    if (count % whole) n[tile_class(count % whole)]++;
  }
#pragma unroll
  for (int c = 0; c < kClasses; ++c) {
    n[c] = min(n[c], cap);
    int v = n[c];   // inclusive sum over the wave's lanes
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(v, off);
      if (lane >= off) v += u;
    }
    if (lane == 63) sums[wave][c] = min(v, cap);
    at[c] = v - n[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kClasses; ++c) {
    int total = 0;
    for (int w = 0; w < (int)blockDim.x >> 6; ++w) {
      if (w == wave) at[c] += total;
      total += sums[w][c];
    }
    if (threadIdx.x == 0) plan->count[c] = min(total, cap);
    at[c] = min(at[c], cap);
  }
  auto put = [&](int c, int i, const RowTile& t) {
    if (i < cap) plan->list(c, cap)[i] = t;
  };
  for (int i = 0; i < per; ++i) {
    const int e = e0 + i;
    if (per > 1) {   // (one expert a thread: still in registers)
      count = 0;
      if (e < E) expert_rows(offsets, e, rows, &first, &count);
    }
    const int rest = count % whole, rc = tile_class(rest), full = count / whole;
    const int tiles = full + (rest && rc == wc);   // of the whole tiles' class
    // in groups of equal size, the larger ones first
    auto put_tile = [&](int k, int e, int first, int count, int tiles, int at) {
      const int groups = (tiles + kTileGroup - 1) / kTileGroup, small = tiles / groups, more = tiles - groups * small;
      const bool big = k < more * (small + 1);
      const int size = big ? small + 1 : small;
      const int begin = big ? k / size * size : more * (small + 1) + (k - more * (small + 1)) / size * size;
      put(wc, at + k, RowTile{e, first + k * whole, min(count - k * whole, whole), (at + begin) << 4 | size});
    };
    // an expert of many goes out by the wave's lanes together
    constexpr int kMany = 16;
    for (uint64_t many = __ballot(tiles > kMany); many; many &= many - 1) {
      const int l = __ffsll((unsigned long long)many) - 1;
      const int le = __builtin_amdgcn_readlane(e, l), lf = __builtin_amdgcn_readlane(first, l);
      const int lc = __builtin_amdgcn_readlane(count, l), lt = __builtin_amdgcn_readlane(tiles, l);
      const int la = __builtin_amdgcn_readlane(at[wc], l);
      for (int k = lane; k < min(lt, cap - la); k += 64) put_tile(k, le, lf, lc, lt, la);
    }
    if (tiles <= kMany)
      for (int k = 0; k < tiles; ++k) put_tile(k, e, first, count, tiles, at[wc]);
    at[wc] = min(at[wc] + tiles, cap);
    if (rest && rc != wc) {
      put(rc, at[rc], RowTile{e, first + full * whole, rest, at[rc] << 4 | 1});
      at[rc] = min(at[rc] + 1, cap);
    }
  }
}

// A product for every expert: the job of rows 0 and expert 0, and how far the
// next expert's weights are.
struct GroupJob {
  DenseJob job;
  RowPlan* plan;
  int cap;
  int64_t b_step;   // elements
};

// The job of one row tile.  (What memory gives is the same for the whole block
// but not to the compiler, which would keep the buffer resources' bases in vector
// registers and read them back for every DMA: 1472 against 1363 us for 49152 x 4096
// x 4096.)
__device__ __forceinline__ DenseJob tile_job(const GroupJob& g, const RowTile& at) {
  const RowTile t{__builtin_amdgcn_readfirstlane(at.expert), __builtin_amdgcn_readfirstlane(at.row),
                  __builtin_amdgcn_readfirstlane(at.rows), 0};
  DenseJob p = g.job;
  const int64_t row = t.row;
  p.M = t.rows;
  if (p.gather) p.gather += row;
  else p.a = static_cast<const char*>(p.a) + row * p.lda * 2;
  p.b = static_cast<const char*>(p.b) + t.expert * g.b_step * 2;
  p.c = static_cast<char*>(p.c) + row * p.ldc * (p.c_dtype == MOE_FLOAT_FP32 ? 4 : 2);
  if (p.gu) {
    const int64_t width = p.epi == kEpiGate ? p.N : 2 * (int64_t)p.N;
    p.gu = static_cast<char*>(p.gu) + row * width * (p.gu_dtype == MOE_FLOAT_FP32 ? 4 : 2);
  }
  if (p.h) p.h = static_cast<char*>(p.h) + row * p.N * 2;
  return p;
}

// Unit t of a class of row tiles, nts column tiles each: a group's tiles side by
// side, column by column.
__device__ __forceinline__ RowTile unit_at(const GroupJob& g, int cls, int t, int nts, int* nt) {
  const RowTile* const list = g.plan->list(cls, g.cap);
  const int group = __builtin_amdgcn_readfirstlane(list[t / nts].group), first = group >> 4;
  const int tiles = min(group & 15, g.cap - first);   // (a group that the list cuts off)
  const int in = t - first * nts;
  *nt = in / tiles;
  return list[first + in % tiles];
}

__device__ __forceinline__ int up8(int v) { return (v + 7) & ~7; }

// One block's unit among a product's, number b from the class of the largest row
// tiles on; returns what b is behind them all, -1 once it had one (or a gap: each
// class begins at a multiple of 8, so that its run on every XCD is contiguous).
// Wide: tiles of 256 columns (128 gate and 128 up ones).  Tiles of 256 rows go in
// groups that share an expert's weights in the L2; the other classes have one tile
// an expert, whose rows stay in the L2 while all its columns pass.
// Narrow: tiles of up to 128 rows and 128 columns, two blocks per CU.  Split: 64 x 64
// tiles whose waves split K, two blocks per CU.
constexpr int kNarrowLds = 72 << 10;
enum Shape { kWide, kNarrow, kSplit };
template <typename E, int SHAPE, bool TB, int EPI, bool GATHER>
__device__ __forceinline__ int product_unit(const GroupJob& g, int b, char* lds) {
  constexpr bool WIDE = SHAPE == kWide;
  const int cols = (WIDE ? 256 : SHAPE == kNarrow ? 128 : 64) >> (EPI == kEpiGate ? 1 : 0);
  const int width = EPI == kEpiGate ? g.job.N >> 1 : g.job.N, nts = (width + cols - 1) / cols;
  const int n0 = WIDE ? g.plan->count[0] : 0, n1 = SHAPE != kSplit ? g.plan->count[1] : 0, n2 = g.plan->count[2];
  int nt;
  if constexpr (WIDE) {
    if (b < up8(n0 * nts)) {
      if (b >= n0 * nts) return -1;
      const DenseJob p = tile_job(g, unit_at(g, 0, xcd_run(b, n0 * nts), nts, &nt));
      dense_tile<E, false, TB, EPI, false, 4, 4, 4, 32, GATHER>(p, 0, nt, lds);
      return -1;
    }
    b -= up8(n0 * nts);
  }
  if constexpr (SHAPE == kSplit) {
    if (b < up8(n2 * nts)) {
      if (b >= n2 * nts) return -1;
      const DenseJob p = tile_job(g, unit_at(g, 2, xcd_run(b, n2 * nts), nts, &nt));
      split_k_tile<E, false, TB, EPI, false, 32, GATHER>(p, 0, nt, lds);
      return -1;
    }
    return b - up8(n2 * nts);
  } else {
    if (b < up8(n1 * nts)) {
      if (b >= n1 * nts) return -1;
      const int t = xcd_run(b, n1 * nts);
      if constexpr (WIDE) {
        const DenseJob p = tile_job(g, g.plan->list(1, g.cap)[t / nts]);
        dense_tile<E, false, TB, EPI, false, 2, 4, 3, 64, GATHER>(p, 0, t % nts, lds);
      } else {
        const DenseJob p = tile_job(g, unit_at(g, 1, t, nts, &nt));
        dense_tile<E, false, TB, EPI, false, 2, 2, 4, 32, GATHER>(p, 0, nt, lds);
      }
      return -1;
    }
    b -= up8(n1 * nts);
    if (b < up8(n2 * nts)) {
      if (b >= n2 * nts) return -1;
      const int t = xcd_run(b, n2 * nts);
      const DenseJob p = tile_job(g, g.plan->list(2, g.cap)[t / nts]);
      dense_tile<E, false, TB, EPI, false, 1, WIDE ? 4 : 2, 3, 64, GATHER>(p, 0, t % nts, lds);
      return -1;
    }
    return b - up8(n2 * nts);
  }
}

template <typename E, int SHAPE, bool TB, int EPI, bool GATHER>
__global__ __launch_bounds__(256, SHAPE == kWide ? 1 : 2) void group_tile_kernel(GroupJob g) {
  __shared__ __attribute__((aligned(1024))) char lds[SHAPE == kWide ? kTileLds : kNarrowLds];
  product_unit<E, SHAPE, TB, EPI, GATHER>(g, blockIdx.x, lds);
}

// Row tile y of all experts' in order, found from the offsets by every wave for
// itself; none: rows 0.
__device__ __forceinline__ RowTile nth_tile(const int32_t* offsets, int E, int rows, int whole, int y) {
  const int lane = threadIdx.x & 63;
  constexpr int C = 16;
  for (int e0 = 0; e0 < E; e0 += 64 * C) {
    int f[C], n[C];   // C times 64 experts, their loads in flight together
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int e = e0 + i * 64 + lane;
      f[i] = n[i] = 0;
      if (e < E) expert_rows(offsets, e, rows, &f[i], &n[i]);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int mine = (n[i] + whole - 1) / whole;
      uint64_t past = __ballot(mine > 0);   // the lanes up to whose expert there are more than y tiles
      int upto = mine;                      // tiles of this lane's expert and those before it
      if (__ballot(mine > 1)) {
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const int u = __shfl_up(upto, off);
          if (lane >= off) upto += u;
        }
        past = __ballot(upto > y);
        if (!past) {
          y -= __builtin_amdgcn_readlane(upto, 63);
          continue;
        }
      } else {
        const int c = __popcll(past);
        if (y >= c) {
          y -= c;
          continue;
        }
        for (; y > 0; --y) past &= past - 1;
        upto = 1;
      }
      const int l = __ffsll((unsigned long long)past) - 1;
      const int r = (y - __builtin_amdgcn_readlane(upto - mine, l)) * whole;
      return RowTile{e0 + i * 64 + l, __builtin_amdgcn_readlane(f[i], l) + r,
                     min(__builtin_amdgcn_readlane(n[i], l) - r, whole), 0};
    }
  }
  return RowTile{0, 0, 0, 0};
}

// Few rows (decode): a block takes 16 NB weight rows of one expert for up to 16 MB
// of its rows, as the dense kernel of few rows does; bound by reading the weights
// of the experts that have rows.  Four waves split K, not eight: they have 16 turns
// of 64 k each at K = 4096, not 8, beside a block's ends, and with 48 or 32 KB of LDS
// three to five blocks a CU cover each other's.  Us with four / eight waves, forward:
// 256 experts of 4096 x 2048, 6 rows 58 / 68, 24 rows 208 / 213; 64 of 2048 x 1024, 64
// rows 149 / 168; 8 of 4096 x 3584, 16 rows 123 / 142, and the other way 128 rows 131 /
// 128.  Every block finds its rows by itself from the offsets: no launch ahead of the
// product.
constexpr int kGroupFewWaves = 4;
template <typename E, int MB, int NB, int EPI, int D, bool GATHER>
__global__ __launch_bounds__(64 * kGroupFewWaves) void group_few_kernel(GroupJob g, const int32_t* offsets, int experts,
                                                                        int rows) {
  __shared__ __attribute__((aligned(1024))) char lds[FewLds<MB, NB, true, D, kGroupFewWaves>::BYTES];
  const RowTile t = nth_tile(offsets, experts, rows, 16 * MB, blockIdx.y);
  if (t.rows == 0) return;
  few_block<E, MB, NB, EPI, true, D, GATHER, kGroupFewWaves>(tile_job(g, t), blockIdx.x, lds);
}

// A weight gradient's tile, number t of the experts' in turn, 64 F rows and
// columns each: C[e] = A^T B over expert e's rows, both stored [rows][..].
template <typename E, bool WIDE, int F>
__device__ __forceinline__ void grad_unit(const GroupJob& g, const int32_t* offsets, int rows, int t, char* lds) {
  constexpr int TILE = 64 * F;
  const int mts = (g.job.M + TILE - 1) / TILE, nts = (g.job.N + TILE - 1) / TILE, e = t / (mts * nts);
  int first, mt, nt;
  DenseJob p = g.job;
  expert_rows(offsets, e, rows, &first, &p.K);
  first = __builtin_amdgcn_readfirstlane(first), p.K = __builtin_amdgcn_readfirstlane(p.K);   // (as in tile_job)
  if (p.K == 0 && p.add) return;
  tile_at(t % (mts * nts), mts, nts, &mt, &nt);
  mt = __builtin_amdgcn_readfirstlane(mt), nt = __builtin_amdgcn_readfirstlane(nt);
  p.a = uniform_ptr(static_cast<const char*>(p.a) + (int64_t)first * p.lda * 2);
  p.b = uniform_ptr(static_cast<const char*>(p.b) + (int64_t)first * p.ldb * 2);
  const int64_t step = (int64_t)e * p.M * p.ldc * (p.c_dtype == MOE_FLOAT_FP32 ? 4 : 2);
  p.c = static_cast<char*>(p.c) + step;
  if (p.add) p.add = static_cast<const char*>(p.add) + step;
  if constexpr (F == 4) dense_tile<E, true, true, kEpiPlain, false, 4, 4, 4, 32>(p, mt * TILE, nt, lds);
  else if constexpr (WIDE) dense_tile<E, true, true, kEpiPlain, false, 2, 2, 4, 64>(p, mt * TILE, nt, lds);
  else dense_tile<E, true, true, kEpiPlain, false, 2, 2, 4, 32>(p, mt * TILE, nt, lds);
}

// dx's rows, dw1 and dw2, which need nothing of each other: those of one launch (or
// one of them alone), the weight gradients' tiles behind dx's.
struct BackJobs {
  GroupJob dx, dw[2];
  int has_dx, units[2];   // tiles of dw1 and dw2
};
template <typename E, int SHAPE, int F>
__global__ __launch_bounds__(256, SHAPE == kWide ? 1 : 2) void group_back_kernel(BackJobs j, const int32_t* offsets, int rows) {
  __shared__ __attribute__((aligned(1024))) char lds[SHAPE == kWide ? kTileLds : kNarrowLds];
  int b = blockIdx.x;
  if (j.has_dx) b = product_unit<E, SHAPE, true, kEpiPlain, false>(j.dx, b, lds);
  if (b < 0) return;
  const int second = b >= up8(j.units[0]);
  if (second) b -= up8(j.units[0]);
  if (b >= j.units[second]) return;
  grad_unit<E, SHAPE == kWide, F>(j.dw[second], offsets, rows, xcd_run(b, j.units[second]), lds);
}

// x's rows in expert order (the weight gradient's products take no gather).
template <typename E>
__global__ __launch_bounds__(256) void gather_rows_kernel(DenseJob p, const int32_t* offsets, int experts, int rows,
                                                          void* out) {
  const int lo = max(offsets[0], 0), hi = min(offsets[experts], rows);
  for (int64_t r = lo + (int64_t)blockIdx.x; r < hi; r += gridDim.x) {
    const int g = p.gather[r], row = g / p.gather_div;
    const bool in = g >= 0 && row < p.gather_rows;
    for (int v = threadIdx.x; v < p.K >> 3; v += 256) {
      uint4 q{};
      if (in) q = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.a) + row * p.lda + 8 * v);
      *reinterpret_cast<uint4*>(static_cast<E*>(out) + r * p.K + 8 * v) = q;
    }
  }
}

// dx[t] = the sum of the token's rows, in slot order.
template <typename E>
__global__ __launch_bounds__(512) void sum_rows_kernel(const float* __restrict__ dxr, const int32_t* __restrict__ dest,
                                                       const int32_t* __restrict__ offsets, int experts, int rows,
                                                       int tokens, int div, int H, void* __restrict__ dx, int dx_dtype,
                                                       int64_t dx_stride) {
  const int lo = max(offsets[0], 0), hi = min(offsets[experts], rows);
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int v = threadIdx.x; v < H >> 3; v += blockDim.x) {
      F8 s{};
      for (uint32_t j0 = 0; j0 < (uint32_t)div; j0 += 8) {
        F8 r[8];
        bool in[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int d = j0 + j < (uint32_t)div ? dest[t * div + j0 + j] : -1;
          in[j] = d >= lo && d < hi;
          if (in[j]) r[j] = load8<E>(dxr, MOE_FLOAT_FP32, (size_t)d * H + 8 * v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (in[j])
#pragma unroll
            for (int e = 0; e < 8; ++e) s.v[e] += r[j].v[e];
      }
      store8<E>(dx, dx_dtype, t * dx_stride + 8 * v, s);
    }
  }
}

// ---- launches ------------------------------------------------------------
struct Group {
  int rows, E;
  const int32_t* offsets;
  RowPlan* plan;
  int shape;  // Shape of the tiles
  int whole() const { return shape == kWide ? 256 : shape == kNarrow ? 128 : 64; }   // its rows and columns
  int most;   // rows that an expert has at most where a token goes to it once
};

// A few rows an expert, and too few experts with rows for narrow tiles to fill the
// chip: the weights stream in tiles of 32 rows of them.  Us with these kernels / in
// narrow tiles, whole forward passes, rows spread evenly: 256 experts of 4096 x 2048, 6
// rows 58 / 60, 24 rows 208 / 207, 48 rows (past the bound) 415 / 404; 64 of 2048 x
// 1024, 64 rows 149 / 166, 256 rows 151 / 167; 8 of 4096 x 3584, 2 rows 33 / 49, 16 rows
// 123 / 138, 128 rows 131 / 138; 6 of 1096 x 1032, 96 rows 14 / 23.  Short rows of the
// weights gain nothing: both products of 64 of 1024 x 768, 512 rows, 61 / 55 (its FC1,
// with rows of just 1024, still comes here: 60), of 16 of 1096 x 776, 256 rows, 23.9 /
// 23.9.  Past 32 rows an expert a second tile would read its weights again; from 16 to
// 32 the two are within 3 % (8 of 4096 x 3584, 192 rows 135 / 139; 16 of 1096 x 776, 320
// rows 24.4 / 24.7).
// A block's rows (of a split gate also their up rows) lie within 31 bits of the first.
bool takes_few(const Group& g, const DenseJob& j) {
  const int64_t reach = j.epi == kEpiGate && !j.interleaved ? (int64_t)(j.N / 2 + 16) * j.ldb * 2 : 0;
  const int64_t n = std::min(g.E, g.rows);
  return !j.tb && j.K >= 1024 && g.rows <= 16 * n && n * ((j.N + 127) / 128) <= 1024 && reach < (1ll << 30);
}

template <typename E, int MB, int NB, int D>
moe_status launch_few(const Group& g, const DenseJob& j, int64_t b_step, hipStream_t s) {
  const GroupJob q{j, nullptr, 0, b_step};
  const dim3 grid((j.N + 16 * NB - 1) / (16 * NB), g.rows / (16 * MB) + std::min(g.E, g.rows)), block(64 * kGroupFewWaves);
  if (j.epi == kEpiGate && j.gather)
    hipLaunchKernelGGL((group_few_kernel<E, MB, NB, kEpiGate, D, true>), grid, block, 0, s, q, g.offsets, g.E, g.rows);
  else if (j.epi == kEpiGate)
    hipLaunchKernelGGL((group_few_kernel<E, MB, NB, kEpiGate, D, false>), grid, block, 0, s, q, g.offsets, g.E, g.rows);
  else
    hipLaunchKernelGGL((group_few_kernel<E, MB, NB, kEpiPlain, D, false>), grid, block, 0, s, q, g.offsets, g.E, g.rows);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

// Tiles of 256 columns read the least for their products, but need many of them and
// long sums: narrow ones where, with the rows spread evenly, they would leave a
// third of the CUs idle, where the weights' stream is what counts, and where short
// sums leave the tiles' ends much of the time, which two blocks a CU hide.  Us,
// wide / narrow, whole forward passes, rows spread evenly (an asterisk: what the rule
// takes):
//   8 experts of 4096 x 2048    1024 rows 126 / 112*, 2048 rows 192 / 168*, 2560 rows 198* / 234
//   11 of 4096 x 2048           1408 rows 156 / 175*, 2816 rows 210 / 227* (176 tiles: just at the bound)
//   24 of 1096 x 776            384 rows 33 / 33*, 3000 rows 49 / 52*
//   8 of 7168 x 3584            512 rows (224 tiles) 223* / 237
//   256 of 4096 x 2048          384 rows 2184 / 2123*, 6144 rows 2260 / 2220*, 24576 rows 2378* / 2796
//   32 of 2048 x 1024           2048 rows 105 / 96*, 4096 rows 117 / 113*, 5120 rows 146* / 168
//   64 of 2048 x 1024           6144 rows 212 / 205*, 12288 rows 282* / 364
// (128 x 256 tiles of 32-deep stages, two blocks a CU, lie between the two.)
// Where even narrow tiles are fewer than the CUs' room for them, a block's time is
// its K loop's latency: 64 x 64 tiles whose four waves split K (narrow / split: 9
// experts of 1096 x 776, 512 rows 24.8 / 21.4*, 1034 rows 36.8 / 29.4*, 1400 rows 35.1* /
// 33.8, 2048 rows 37.0* / 43.4; 24 of them, 1000 rows, 504 tiles, 35.2* / 40.0; 16 of
// them, 64 to 320 rows, 336 tiles, 24 / 28*: with one row tile an expert two blocks
// a CU of narrow tiles would do).
int tile_shape(int rows, int E, int H, int I) {
  const int n = std::max(std::min(E, rows), 1), each = (rows + n - 1) / n;
  // columns: of the two products, on average
  if (n * ((each + 63) / 64) * (((H + 63) / 64 + (I + 31) / 32) / 2) <= 400) return kSplit;
  const int64_t columns = ((H + 255) / 256 + (I + 127) / 128) / 2;
  const bool idle = n * ((each + 255) / 256) * columns <= 176, brief = H + I < 4096 && each <= 128;
  return each <= 32 || idle || brief ? kNarrow : kWide;
}

moe_status launch_plan(const Group& g, hipStream_t s) {
  const dim3 block(std::min(1024, (g.E + 63) / 64 * 64));
  hipLaunchKernelGGL(plan_rows_kernel, dim3(1), block, 0, s, g.offsets, g.E, g.rows, g.whole(),
                     tile_cap(g.rows, g.E), g.plan);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

// Blocks that a product's units can need.
int64_t unit_bound(const Group& g, const DenseJob& j) {
  const int cols = j.epi == kEpiGate ? g.whole() / 2 : g.whole(), width = j.epi == kEpiGate ? j.N / 2 : j.N;
  return (int64_t)(g.rows / g.whole() + std::min(g.E, g.rows)) * ((width + cols - 1) / cols) + 24;
}

template <typename E>
moe_status launch_group_typed(const Group& g, const DenseJob& j, int64_t b_step, hipStream_t s) {
  if (takes_few(g, j))
    return g.most <= 16 ? launch_few<E, 1, 2, 2>(g, j, b_step, s) : launch_few<E, 2, 2, 1>(g, j, b_step, s);
  const GroupJob q{j, g.plan, tile_cap(g.rows, g.E), b_step};
  const dim3 grid((unsigned)unit_bound(g, j)), block(256);
#define MXMOE_LAUNCH(TB, EPI, GATHER)                                                                      \
  if (g.shape == kWide) hipLaunchKernelGGL((group_tile_kernel<E, kWide, TB, EPI, GATHER>), grid, block, 0, s, q);         \
  else if (g.shape == kNarrow) hipLaunchKernelGGL((group_tile_kernel<E, kNarrow, TB, EPI, GATHER>), grid, block, 0, s, q); \
  else hipLaunchKernelGGL((group_tile_kernel<E, kSplit, TB, EPI, GATHER>), grid, block, 0, s, q)
  if (j.epi == kEpiGate && j.gather) { MXMOE_LAUNCH(false, kEpiGate, true); }
  else if (j.epi == kEpiGate) { MXMOE_LAUNCH(false, kEpiGate, false); }
  else if (j.epi == kEpiGateGrad) { MXMOE_LAUNCH(true, kEpiGateGrad, false); }
  else { MXMOE_LAUNCH(false, kEpiPlain, false); }
#undef MXMOE_LAUNCH
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}
moe_status launch_group(const Group& g, const DenseJob& j, int64_t b_step, hipStream_t s) {
  return j.dtype == MOE_FLOAT_BF16 ? launch_group_typed<__bf16>(g, j, b_step, s)
                                   : launch_group_typed<_Float16>(g, j, b_step, s);
}

// dx, dw1 and dw2; null pointers of c where one is not asked for.  In one launch
// where they are small: 1034 rows over 9 experts of 1096 x 776, the whole training step
// 142 -> 122 us.  Wide tiles one after the other: side by side they lose more of what
// they share in the L2 than their ends leave idle (49152 rows, 32 experts of 4096 x
// 2048: 4071 us together, 3905 in turn, the best of 24).
template <typename E>
moe_status launch_back_typed(const Group& g, const DenseJob& dx, int64_t dx_step, const DenseJob& dw1, const DenseJob& dw2,
                             hipStream_t s) {
  auto tiles = [&](const DenseJob& j, int n) {
    return j.c ? (int64_t)g.E * ((j.M + n - 1) / n) * ((j.N + n - 1) / n) : 0;
  };
  // (315 and 189 tiles of 256 x 256 and short K: 150 us the whole training step, in tiles of 128 x 128 134)
  const bool wide = g.shape == kWide, big = wide && tiles(dw1, 256) + tiles(dw2, 256) >= 512;
  auto units = [&](const DenseJob& j) { return (tiles(j, big ? 256 : 128) + 7) / 8 * 8; };
  // Each of them has fewer than 2^24 blocks (check_experts), a launch may have no more:
  // its threads are counted in 32 bits, and what passes them is not run, without an error.
  const bool apart = wide || (dx.c ? unit_bound(g, dx) : 0) + units(dw1) + units(dw2) >= 1 << 24;
  for (int part = 0; part < (apart ? 3 : 1); ++part) {
    BackJobs q{{dx, g.plan, tile_cap(g.rows, g.E), dx_step}, {{dw1, nullptr, 0, 0}, {dw2, nullptr, 0, 0}}, 0, {}};
    q.has_dx = dx.c != nullptr && part == 0;
    int64_t blocks = q.has_dx ? unit_bound(g, dx) : 0;
    for (int i = 0; i < 2; ++i) {
      const bool now = !apart || part == i + 1;
      q.units[i] = now ? (int)tiles(q.dw[i].job, big ? 256 : 128) : 0;
      if (now) blocks += units(q.dw[i].job);
    }
    if (blocks == 0) continue;
    const dim3 grid((unsigned)blocks), block(256);
    if (big) hipLaunchKernelGGL((group_back_kernel<E, kWide, 4>), grid, block, 0, s, q, g.offsets, g.rows);
    else if (wide) hipLaunchKernelGGL((group_back_kernel<E, kWide, 2>), grid, block, 0, s, q, g.offsets, g.rows);
    else if (g.shape == kNarrow)
      hipLaunchKernelGGL((group_back_kernel<E, kNarrow, 2>), grid, block, 0, s, q, g.offsets, g.rows);
    else hipLaunchKernelGGL((group_back_kernel<E, kSplit, 2>), grid, block, 0, s, q, g.offsets, g.rows);
    MXMOE_HIP(hipGetLastError());
  }
  return MOE_OK;
}

// ---- checks and workspaces -------------------------------------------------
moe_status check_experts(const char* what, int rows, int H, int I, int E, int layout, int act, int dtype) {
  MXMOE_TRY(check_width(what, "H", H));
  MXMOE_TRY(check_width(what, "I", I));
  if (E < 1 || E > kMaxExperts) return fail(MOE_ERR_SHAPE, "%s: E = %d outside [1, %d]", what, E, kMaxExperts);
  if (rows < 0 || rows > kMaxTokens) return fail(MOE_ERR_SHAPE, "%s: rows = %d outside [0, %d]", what, rows, kMaxTokens);
  const int64_t wide = std::max(H, 2 * I);
  if (((int64_t)rows / 64 + std::min(E, rows) + 1) * ((wide + 63) / 64) >= 1 << 24)
    return fail(MOE_ERR_SHAPE, "%s: %d rows of %lld are too many for one launch", what, rows, (long long)wide);
  if ((int64_t)E * ((H + 63) / 64) * ((2 * I + 63) / 64) >= 1 << 24)
    return fail(MOE_ERR_SHAPE, "%s: %d experts of %d x %d are too many for one launch", what, E, 2 * I, H);
  if (layout != MOE_EPI_SWIGLU_SPLIT && layout != MOE_EPI_SWIGLU_INTERLEAVED)
    return fail(MOE_ERR_INVALID_ARG, "%s: layout %d must be a SWIGLU epilogue", what, layout);
  if (act != MOE_GATE_SILU && act != MOE_GATE_GELU)
    return fail(MOE_ERR_INVALID_ARG, "%s: bad gate_act %d", what, act);
  return check_dtype16(what, dtype);
}
bool within_limits(int rows, int H, int I, int E) {
  return rows >= 0 && rows <= kMaxTokens && H > 0 && H <= kMaxWidth && I > 0 && I <= kMaxWidth && E > 0 &&
         E <= kMaxExperts;
}
moe_status check_gather(const char* what, const int32_t* gather, int rows, int tokens, int div, int64_t stride) {
  if (div < 0 || (div == 0 && gather))
    return fail(MOE_ERR_SHAPE, "%s: gather_div = %d must be at least 1 with gather, 0 without", what, div);
  if (div == 0) return MOE_OK;
  if (!gather && rows > 0) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer (gather)", what);
  if (tokens < 0) return fail(MOE_ERR_SHAPE, "%s: tokens = %d < 0", what, tokens);
  if (tokens * stride >= 1ll << 30)
    return fail(MOE_ERR_SHAPE, "%s: gathered rows reach over %lld elements, past 2^30", what, (long long)(tokens * stride));
  return MOE_OK;
}
// Index arrays: 4-byte aligned, apart from every output.
moe_status check_words(const char* what, const Span* out, int n_out, const Span* words, int n) {
  for (int i = 0; i < n; ++i) {
    if (reinterpret_cast<uintptr_t>(words[i].p) & 3)
      return fail(MOE_ERR_INVALID_ARG, "%s: %s is not 4-byte aligned", what, words[i].name);
    for (int j = 0; j < n_out; ++j)
      if (overlap(out[j], words[i]))
        return fail(MOE_ERR_INVALID_ARG, "%s: %s overlaps %s", what, out[j].name, words[i].name);
  }
  return MOE_OK;
}

struct ForwardWs {
  size_t h, total;
};
ForwardWs forward_ws(int rows, int H, int I, int E) {
  ForwardWs w{};
  w.h = plan_bytes(rows, E);
  w.total = w.h + align_up((size_t)rows * I * 2, 256) + 256;
  return w;
}
struct GradWs {
  size_t dgu, h, x, dx, total;   // x in expert order and dx by row: gathered calls
};
GradWs grad_ws(int rows, int H, int I, int E, bool gathered) {
  GradWs w{};
  w.dgu = plan_bytes(rows, E);
  w.h = w.dgu + align_up((size_t)rows * 2 * I * 2, 256);
  w.x = w.h + align_up((size_t)rows * I * 2, 256);
  w.dx = w.x + (gathered ? align_up((size_t)rows * H * 2, 256) : 0);
  w.total = w.dx + (gathered ? align_up((size_t)rows * H * 4, 256) : 0) + 256;
  return w;
}

}  // namespace
}  // namespace mxmoe

using namespace mxmoe;

extern "C" {

size_t moe_expert_ffn_workspace_size(int32_t rows, int32_t H, int32_t I, int32_t E) {
  return within_limits(rows, H, I, E) ? forward_ws(rows, H, I, E).total : 0;
}

moe_status moe_expert_ffn_forward(const moe_expert_ffn_args* a, void* stream) {
  const char* what = "expert FFN";
  clear_error();
  if (!a) return fail(MOE_ERR_INVALID_ARG, "%s: null args", what);
  MXMOE_TRY(check_experts(what, a->rows, a->H, a->I, a->E, a->layout, a->gate_act, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "out_dtype", a->out_dtype, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "save_dtype", a->save_dtype, a->dtype));
  MXMOE_TRY(check_stride(what, "x_stride", a->x_stride, a->H));
  MXMOE_TRY(check_stride(what, "out_stride", a->out_stride, a->H));
  MXMOE_TRY(check_gather(what, a->gather, a->rows, a->tokens, a->gather_div, a->x_stride));
  const int64_t rows = a->rows, H = a->H, I = a->I, E = a->E;
  const bool gathered = a->gather_div > 0;
  const ForwardWs w = forward_ws(a->rows, a->H, a->I, a->E);
  if (rows > 0) {
    if ((!a->x && !(gathered && a->tokens == 0)) || !a->expert_offsets || !a->w1 || !a->w2 || !a->out)
      return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!a->workspace || a->workspace_bytes < w.total)
      return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", what, a->workspace_bytes, w.total);
    const Span out[] = {span("out", a->out, rows, H, a->out_stride, a->out_dtype),
                        span("gate_up", a->gate_up, rows, 2 * I, 2 * I, a->save_dtype),
                        {"workspace", a->workspace, w.total}};
    const Span in[] = {span("x", a->x, gathered ? a->tokens : rows, H, a->x_stride, a->dtype),
                       span("w1", a->w1, E * 2 * I, H, H, a->dtype), span("w2", a->w2, E * H, I, I, a->dtype)};
    MXMOE_TRY(check_spans(what, out, 3, in, 3));
    const Span words[] = {{"expert_offsets", a->expert_offsets, (size_t)(E + 1) * 4},
                          {"gather", a->gather, a->gather ? (size_t)rows * 4 : 0}};
    MXMOE_TRY(check_words(what, out, 3, words, 2));
  }
  MXMOE_TRY(check_device());
  if (rows == 0) return MOE_OK;
  const hipStream_t s = (hipStream_t)stream;
  uint8_t* const ws = static_cast<uint8_t*>(a->workspace);
  const Group g{a->rows, a->E, a->expert_offsets, reinterpret_cast<RowPlan*>(ws),
                tile_shape(a->rows, a->E, a->H, a->I), gathered ? std::min(a->rows, a->tokens) : a->rows};

  DenseJob j{};
  j.dtype = a->dtype;
  j.act = a->gate_act;
  j.interleaved = a->layout == MOE_EPI_SWIGLU_INTERLEAVED;
  j.a = a->x, j.lda = a->x_stride;
  j.gather = a->gather, j.gather_div = a->gather_div, j.gather_rows = a->tokens;
  j.b = a->w1, j.ldb = H;
  j.N = 2 * a->I, j.K = a->H;
  j.epi = kEpiGate;
  j.c = ws + w.h, j.ldc = I, j.c_dtype = a->dtype;
  j.gu = a->gate_up, j.gu_dtype = a->save_dtype;

  DenseJob k = j;
  k.a = ws + w.h, k.lda = I;
  k.gather = nullptr;
  k.b = a->w2, k.ldb = I;
  k.N = a->H, k.K = a->I;
  k.epi = kEpiPlain;
  k.gu = nullptr;
  k.c = a->out, k.ldc = a->out_stride, k.c_dtype = a->out_dtype;

  if (!takes_few(g, j) || !takes_few(g, k)) MXMOE_TRY(launch_plan(g, s));
  MXMOE_TRY(launch_group(g, j, 2 * I * H, s));
  return launch_group(g, k, H * I, s);
}

size_t moe_expert_ffn_grad_workspace_size(int32_t rows, int32_t H, int32_t I, int32_t E, int32_t gathered) {
  return within_limits(rows, H, I, E) ? grad_ws(rows, H, I, E, gathered != 0).total : 0;
}

moe_status moe_expert_ffn_backward(const moe_expert_ffn_grad_args* a, void* stream) {
  const char* what = "expert FFN backward";
  clear_error();
  if (!a) return fail(MOE_ERR_INVALID_ARG, "%s: null args", what);
  MXMOE_TRY(check_experts(what, a->rows, a->H, a->I, a->E, a->layout, a->gate_act, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "save_dtype", a->save_dtype, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "dx_dtype", a->dx_dtype, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "dw_dtype", a->dw_dtype, a->dtype));
  if (a->accumulate != 0 && a->accumulate != 1)
    return fail(MOE_ERR_INVALID_ARG, "%s: accumulate %d must be 0 or 1", what, a->accumulate);
  MXMOE_TRY(check_stride(what, "dout_stride", a->dout_stride, a->H));
  if (a->dw1) MXMOE_TRY(check_stride(what, "x_stride", a->x_stride, a->H));
  if (a->dx) MXMOE_TRY(check_stride(what, "dx_stride", a->dx_stride, a->H));
  MXMOE_TRY(check_gather(what, a->gather, a->rows, a->tokens, a->gather_div, a->dw1 ? a->x_stride : 0));
  const bool gathered = a->gather_div > 0;
  if (gathered && a->dx && (int64_t)a->tokens * a->gather_div >= 1ll << 31)
    return fail(MOE_ERR_SHAPE, "%s: tokens * gather_div overflows int32", what);
  const int64_t rows = a->rows, H = a->H, I = a->I, E = a->E;
  const int64_t x_rows = gathered ? a->tokens : rows, slots = gathered ? x_rows * a->gather_div : 0;
  const GradWs w = grad_ws(a->rows, a->H, a->I, a->E, gathered);
  if (gathered && a->dx && x_rows > 0 && !a->dest_row) return fail(MOE_ERR_INVALID_ARG, "%s: dx with gather needs dest_row", what);
  if (rows > 0) {
    if (!a->dout || !a->expert_offsets || !a->w2 || !a->gate_up || (a->dw1 && !a->x && x_rows > 0) || (a->dx && !a->w1))
      return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!a->workspace || a->workspace_bytes < w.total)
      return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", what, a->workspace_bytes, w.total);
  } else if (((gathered && a->dx && x_rows > 0) || a->dw1 || a->dw2) && !a->expert_offsets) {
    return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
  }
  const Span out[] = {span("dx", a->dx, x_rows, H, a->dx_stride, a->dx_dtype),
                      span("dw1", a->dw1, E * 2 * I, H, H, a->dw_dtype), span("dw2", a->dw2, E * H, I, I, a->dw_dtype),
                      {"workspace", a->workspace, rows > 0 ? w.total : 0}};
  const Span in[] = {span("dout", a->dout, rows, H, a->dout_stride, a->dtype),
                     span("x", a->dw1 ? a->x : nullptr, x_rows, H, a->x_stride, a->dtype),
                     span("w1", a->dx ? a->w1 : nullptr, E * 2 * I, H, H, a->dtype),
                     span("w2", a->w2, E * H, I, I, a->dtype),
                     span("gate_up", a->gate_up, rows, 2 * I, 2 * I, a->save_dtype)};
  MXMOE_TRY(check_spans(what, out, 4, in, 5));
  const Span words[] = {{"expert_offsets", a->expert_offsets, (size_t)(E + 1) * 4},
                        {"gather", a->gather, a->gather ? (size_t)rows * 4 : 0},
                        {"dest_row", a->dx ? a->dest_row : nullptr, a->dx ? (size_t)slots * 4 : 0}};
  MXMOE_TRY(check_words(what, out, 4, words, 3));
  MXMOE_TRY(check_device());
  if (!a->dx && !a->dw1 && !a->dw2) return MOE_OK;
  const hipStream_t s = (hipStream_t)stream;
  uint8_t* const ws = static_cast<uint8_t*>(a->workspace);
  const Group g{a->rows, a->E, a->expert_offsets, reinterpret_cast<RowPlan*>(ws),
                tile_shape(a->rows, a->E, a->H, a->I), a->rows};

  DenseJob j{};
  j.dtype = a->dtype;
  j.act = a->gate_act;
  j.interleaved = a->layout == MOE_EPI_SWIGLU_INTERLEAVED;
  const bool any = rows > 0;
  if (any) {
    MXMOE_TRY(launch_plan(g, s));
    // the gradients of gate and up, and h
    j.a = a->dout, j.lda = a->dout_stride;
    j.b = a->w2, j.ldb = I, j.tb = 1;
    j.N = a->I, j.K = a->H;
    j.epi = kEpiGateGrad;
    j.gu = const_cast<void*>(a->gate_up), j.gu_dtype = a->save_dtype;
    j.c = ws + w.dgu, j.ldc = 2 * I, j.c_dtype = a->dtype;
    j.h = ws + w.h;
    MXMOE_TRY(launch_group(g, j, H * I, s));
  }
  j.epi = kEpiPlain;
  j.gu = j.h = nullptr;
  DenseJob dx{}, dw1{}, dw2{};
  if (a->dx && any) {
    dx = j;
    dx.a = ws + w.dgu, dx.lda = 2 * I;
    dx.b = a->w1, dx.ldb = H, dx.tb = 1;
    dx.N = a->H, dx.K = 2 * a->I;
    if (gathered) dx.c = ws + w.dx, dx.ldc = H, dx.c_dtype = MOE_FLOAT_FP32;
    else dx.c = a->dx, dx.ldc = a->dx_stride, dx.c_dtype = a->dx_dtype;
  }
  // the weights' gradients sum over the expert's rows
  j.ta = j.tb = 1;
  j.c_dtype = a->dw_dtype;
  const bool sums = any || !a->accumulate;
  if (a->dw1 && sums) {
    dw1 = j;
    dw1.a = ws + w.dgu, dw1.lda = 2 * I;
    dw1.b = a->x, dw1.ldb = a->x_stride;
    if (gathered && any) {
      DenseJob q{};
      q.a = a->x, q.lda = a->x_stride, q.K = a->H;
      q.gather = a->gather, q.gather_div = a->gather_div, q.gather_rows = a->tokens;
      hipLaunchKernelGGL((gather_rows_kernel<_Float16>), dim3((unsigned)std::min<int64_t>(rows, 1 << 20)), dim3(256), 0, s,
                         q, a->expert_offsets, a->E, a->rows, ws + w.x);   // (any 16 bits)
      MXMOE_HIP(hipGetLastError());
      dw1.b = ws + w.x, dw1.ldb = H;
    }
    dw1.M = 2 * a->I, dw1.N = a->H;
    dw1.c = a->dw1, dw1.ldc = H;
    dw1.add = a->accumulate ? a->dw1 : nullptr, dw1.ldadd = H;
  }
  if (a->dw2 && sums) {
    dw2 = j;
    dw2.a = a->dout, dw2.lda = a->dout_stride;
    dw2.b = ws + w.h, dw2.ldb = I;
    dw2.M = a->H, dw2.N = a->I;
    dw2.c = a->dw2, dw2.ldc = I;
    dw2.add = a->accumulate ? a->dw2 : nullptr, dw2.ldadd = I;
  }
  const int64_t dx_step = 2 * I * H;
  MXMOE_TRY(a->dtype == MOE_FLOAT_BF16 ? launch_back_typed<__bf16>(g, dx, dx_step, dw1, dw2, s)
                                       : launch_back_typed<_Float16>(g, dx, dx_step, dw1, dw2, s));
  if (a->dx && gathered && x_rows > 0) {
    // (up to 512 threads a block: the launch stays below 2^32)
    const dim3 grid((unsigned)std::min<int64_t>(x_rows, 1 << 22)), block(std::min(512, (a->H / 8 + 63) / 64 * 64));
    const float* const dxr = reinterpret_cast<const float*>(ws + w.dx);
    if (a->dtype == MOE_FLOAT_BF16)
      hipLaunchKernelGGL((sum_rows_kernel<__bf16>), grid, block, 0, s, dxr, a->dest_row, a->expert_offsets, a->E, a->rows,
                         a->tokens, a->gather_div, a->H, a->dx, a->dx_dtype, a->dx_stride);
    else
      hipLaunchKernelGGL((sum_rows_kernel<_Float16>), grid, block, 0, s, dxr, a->dest_row, a->expert_offsets, a->E,
                         a->rows, a->tokens, a->gather_div, a->H, a->dx, a->dx_dtype, a->dx_stride);
    MXMOE_HIP(hipGetLastError());
  }
  return MOE_OK;
}

}  // extern "C"
