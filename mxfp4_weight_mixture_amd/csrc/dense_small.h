// The dense kernel for small products: 64 x 64 tiles, four waves that split K.
//
// Where few tiles exist a block's time is the latency of its K loop, and
// barriers between short stages are most of it.  Here no wave waits for
// another before the end: wave w takes the BK-deep stages w, w + 4, ..., with a
// DMA ring of its own, and holds the whole 64 x 64 tile (2 x 2 fragments of
// 32x32x16); the four sums meet in the LDS.  Bound by the L2 -> LDS path: 8 KB
// per 32 k against 64 clocks of matrix work, at 25 to 30 bytes a clock and CU
// (50 where every line hits and nothing else runs).
// A ring of two 32-deep stages a wave leaves room for two blocks per CU, which
// measured faster than rings of four and one block (512 x 4096 x 4096 32
// against 34 us, 1552 x 1096 x 517 9.0 against 11.9).  Long rows do better in
// stages of 64 k, a whole line per row and load (192 x 4096 x 4096 15.0 against
// 17.4 us, 100 x 7168 x 7168 22.4 against 27.0), short ones do not (517 x 1096
// x 1552 8.7 against 8.2).  The sides meet lower than the choice at K = 4096:
// 100 x 4096 outputs take 7.1 us in 32-deep stages and 7.9 in 64-deep ones at
// K = 1552, 8.3 and 8.9 at 2560, 14.4 and 12.5 at 3584; 512 x 4096 take 17.6 and
// 18.7, 24.1 and 22.0, 31.4 and 26.8.
//
// Adapters: each thread adds its row's low-rank product to its eight columns,
// so mixed adapters cost no more than equal ones.
#pragma once

#include "dense_tile.h"

namespace mxmoe {
namespace {

// sum over r of s[r] B[row][r] for `cols` rows of B, `step` elements apart
template <typename E>
__device__ __forceinline__ void add_low_rank(F8& v, const float* s, const E* lb, int64_t step, int rank, int cols = 8) {
  typedef typename Vec<E>::v8 v8;
  for (int r = 0; r < rank; r += 8) {
    F8 sv = load8<E>(s, MOE_FLOAT_FP32, r);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c >= cols) break;
      const v8 b = *reinterpret_cast<const v8*>(lb + c * step + r);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (r + e < rank) v.v[c] += sv.v[e] * (float)b[e];
    }
  }
}

// This wave's share of a K loop: stages wave, wave + 4, ... of 32 k, through a
// ring of NST stages of its own.  acc[fm][fn] += A fragments x B fragments.
template <typename E, int FM, int FN, int NST, int BK, typename A, typename B>
__device__ __forceinline__ void split_k_product(const A& a, const B& b, int K, int wave, int lane, char* ring,
                                                v16f (&acc)[FM][FN]) {
  typedef typename Vec<E>::v8 v8;
  constexpr int STAGE = A::BYTES + B::BYTES, LOADS = A::LOADS + B::LOADS;
  static_assert(NST % 2 == 0, "fragment registers alternate by turn");
  constexpr int KS = BK / 16;
  const int turns = ((K + BK - 1) / BK - wave + 3) >> 2;
  auto issue = [&](int j, int t, int buf) {
    if (j < A::LOADS) a.issue(j, wave + 4 * t, K, 0, ring + buf * STAGE);
    else b.issue(j - A::LOADS, wave + 4 * t, K, 0, ring + buf * STAGE + A::BYTES);
  };
  v8 fa[2][KS][FM], fb[2][KS][FN];   // [turn parity][k step][fragment]
  constexpr int NR = KS * (FM + FN), MF = KS / 2 * FM * FN, EARLY = LOADS / 2;
  auto read = [&](int r, int buf, int d) {
    const int ks = r / (FM + FN), f = r % (FM + FN);
    if (f < FN) fb[d][ks][f] = B::frag(ring + buf * STAGE + A::BYTES, f * 32, ks, lane);
    else fa[d][ks][f - FN] = A::frag(ring + buf * STAGE, (f - FN) * 32, ks, lane);
  };
#pragma unroll
  for (int t = 0; t < NST; ++t)
#pragma unroll
    for (int j = 0; j < LOADS; ++j) issue(j, t, t);
  wait_vm<(NST - 1) * LOADS>();
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int r = 0; r < NR; ++r) read(r, 0, 0);
  auto product = [&](int d, int i) {
    const int ks = i / (FM * FN), fm = i % FM, fn = i % (FM * FN) / FM;
    acc[fm][fn] = mfma32(fb[d][ks][fn], fa[d][ks][fm], acc[fm][fn]);
  };
  // NST turns per step without a way out: turns past the end read zeros
  for (int t0 = 0; t0 < turns; t0 += NST) {
#pragma unroll
    for (int u = 0; u < NST; ++u) {
      // This turn is in registers, so its buffer takes turn t + NST: half the
      // DMA beside the first half's products, half beside the second's, and
      // there the next turn, which has landed by then, is read as well.
      wait_lgkm0();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        product(u & 1, i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = EARLY * i / MF; j < EARLY * (i + 1) / MF; ++j) issue(j, t0 + u + NST, u);
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_vm<(NST - 2) * LOADS + EARLY>();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        product(u & 1, MF + i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = NR * i / MF; r < NR * (i + 1) / MF; ++r) read(r, (u + 1) % NST, (u + 1) & 1);
#pragma unroll
        for (int j = EARLY + (LOADS - EARLY) * i / MF; j < EARLY + (LOADS - EARLY) * (i + 1) / MF; ++j)
          issue(j, t0 + u + NST, u);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  wait_vm<0>();
  wait_lgkm0();
  __builtin_amdgcn_sched_barrier(0);
}

// A wave's sums to its LDS area: lane = row, rows of 32 FN values, 16-byte
// chunks permuted by row.
template <int FM, int FN>
__device__ __forceinline__ void put_sums(char* area, int lane, const v16f (&acc)[FM][FN]) {
  constexpr int CH = FN * 8;
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = fm * 32 + (lane & 31), c = fn * 8 + 2 * q + (lane >> 5);
        *reinterpret_cast<v4f*>(area + row * (CH * 16) + ((c ^ (row & (CH - 1))) << 4)) =
            v4f{acc[fm][fn][4 * q], acc[fm][fn][4 * q + 1], acc[fm][fn][4 * q + 2], acc[fm][fn][4 * q + 3]};
      }
}
// The four waves' sums of eight columns, from chunk c on, in wave order.
template <int FN>
__device__ __forceinline__ F8 get_sum8(const char* areas, int area_bytes, int row, int c) {
  constexpr int CH = FN * 8;
  F8 r;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const char* base = areas + w * area_bytes + row * (CH * 16);
    const v4f x = *reinterpret_cast<const v4f*>(base + ((c ^ (row & (CH - 1))) << 4));
    const v4f y = *reinterpret_cast<const v4f*>(base + (((c + 1) ^ (row & (CH - 1))) << 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r.v[e] = w ? r.v[e] + x[e] : x[e];
      r.v[4 + e] = w ? r.v[4 + e] + y[e] : y[e];
    }
  }
  return r;
}

constexpr int split_k_lds(int BK) { return BK == 32 ? 64 << 10 : 128 << 10; }

// The C tile of 64 rows from m0 and the nt-th 64 columns of B.
template <typename E, bool TA, bool TB, int EPI, bool LORA, int BK>
__device__ __forceinline__ void split_k_tile(const DenseJob& p, int m0, int nt, char* lds) {
  constexpr int NST = 2;
  using A = Operand<E, 64, TA, 1, BK>;
  using B = Operand<E, 64, TB, 1, BK>;
  constexpr int STAGE = A::BYTES + B::BYTES;
  constexpr int AREA = 64 * 64 * 4, RING = NST * STAGE > AREA ? NST * STAGE : AREA;
  static_assert(4 * RING <= split_k_lds(BK), "LDS of a tile");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = EPI == kEpiGate ? 32 : 64, width = EPI == kEpiGate ? p.N >> 1 : p.N;
  const int n0 = nt * cols;

  A a;
  B b;
  a.init(p.a, p.lda, p.M, m0, 0, lane);
  if constexpr (EPI == kEpiGate) b.init_gate(p, nt, 0, lane);
  else b.init(p.b, p.ldb, p.N, n0, 0, lane);
  v16f acc[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[i >> 1][i & 1][q] = 0.0f;
  char* const ring = lds + wave * RING;
  split_k_product<E, 2, 2, NST, BK>(a, b, p.K, wave, lane, ring, acc);
  // an adapter's rank, 0 for none
  auto rank_of = [&](int id) {
    if (id < 0 || id >= p.num_adapters) return 0;
    return p.ranks ? min(max(p.ranks[id], 0), p.R) : p.R;
  };
  put_sums<2, 2>(ring, lane, acc);
  __syncthreads();
  // units of eight columns (eight gate and eight up columns) of a row
  constexpr int PER = EPI == kEpiGate ? 4 : 8;
#pragma unroll
  for (int it = 0; it < 64 * PER / 256; ++it) {
    const int unit = it * 256 + threadIdx.x, row = unit / PER, x = unit % PER, m = m0 + row;
    if constexpr (EPI == kEpiGate) {
      const int blk = x >> 2, c = blk * 16 + (x & 3) * 2, i = n0 + x * 8;
      if (m >= p.M || i >= width) continue;
      F8 gt = get_sum8<2>(lds, RING, row, c), up = get_sum8<2>(lds, RING, row, c + 8);
      if constexpr (LORA) {
        const int id = p.ids[m], rank = rank_of(id);
        if (rank > 0) {
          const float* s = p.s + (size_t)m * p.R;
          const E* lb = static_cast<const E*>(p.lb) + ((size_t)id * p.N + (p.interleaved ? 2 * i : i)) * p.R;
          const int64_t step = p.interleaved ? 2 * p.R : p.R;
          add_low_rank<E>(gt, s, lb, step, rank, width - i);
          add_low_rank<E>(up, s, lb + (p.interleaved ? p.R : (int64_t)width * p.R), step, rank, width - i);
        }
      }
      finish_gate<E>(p, m, i, gt, up);
    } else {
      const int n = n0 + x * 8;
      if (m >= p.M || n >= width) continue;
      F8 v = get_sum8<2>(lds, RING, row, 2 * x);
      if constexpr (EPI == kEpiGateGrad) {
        finish_gate_grad<E>(p, m, n, v);
      } else {
        if constexpr (LORA) {
          const int id = p.ids[m], rank = rank_of(id);
          if (rank > 0)
            add_low_rank<E>(v, p.s + (size_t)m * p.R, static_cast<const E*>(p.lb) + ((size_t)id * p.N + n) * p.R,
                            p.R, rank);
        }
        finish_plain<E>(p, m, n, v);
      }
    }
  }
}

// The C tile of block `block` of `blocks`.
template <typename E, bool TA, bool TB, int EPI, bool LORA, int BK>
__device__ __forceinline__ void split_k_block(const DenseJob& p, int block, int blocks, char* lds) {
  const int cols = EPI == kEpiGate ? 32 : 64, width = EPI == kEpiGate ? p.N >> 1 : p.N;
  const int mts = (p.M + 63) >> 6, nts = (width + cols - 1) / cols, t = xcd_run(block, blocks);
  if (t >= mts * nts) return;
  int mt, nt;
  tile_at(t, mts, nts, &mt, &nt);
  split_k_tile<E, TA, TB, EPI, LORA, BK>(p, mt * 64, nt, lds);
}

template <typename E, bool TA, bool TB, int EPI, bool LORA, int BK>
__global__ __launch_bounds__(256, BK == 32 ? 2 : 1) void small_kernel(DenseJob p, float* partial, int splits) {
  __shared__ __attribute__((aligned(1024))) char lds[split_k_lds(BK)];
  int block = blockIdx.x, blocks = gridDim.x;
  if (splits > 1) {   // (a multiple of 8 blocks per part: each keeps its XCD)
    blocks /= splits;
    take_part(p, partial, block / blocks, splits);
    block %= blocks;
  }
  split_k_block<E, TA, TB, EPI, LORA, BK>(p, block, blocks, lds);
}

// Independent products in one launch: their few blocks share the chip, and
// only one launch's ends are paid for.  Blocks [start[i], start[i + 1]) are
// job i's (the starts multiples of 8, which keeps every job's blocks on the
// XCDs they are dealt to; blocks past a job's tiles do nothing).
struct SmallGroup {
  DenseJob job[3];
  int start[4], tiles[3];
};
template <typename E>
__global__ __launch_bounds__(256, 2) void small_group_kernel(SmallGroup g) {
  __shared__ __attribute__((aligned(1024))) char lds[split_k_lds(32)];
  const int b = blockIdx.x, i = b >= g.start[2] ? 2 : b >= g.start[1] ? 1 : 0, block = b - g.start[i];
  if (block >= g.tiles[i]) return;
  if (g.job[i].ta) split_k_block<E, true, true, kEpiPlain, false, 32>(g.job[i], block, g.tiles[i], lds);
  else split_k_block<E, false, true, kEpiPlain, false, 32>(g.job[i], block, g.tiles[i], lds);
}

}  // namespace
}  // namespace mxmoe
