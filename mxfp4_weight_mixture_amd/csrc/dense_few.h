// The dense kernel for few rows (decode): bound by reading the weights once.
//
// A block owns 16 NB weight rows (groups of 8 gate + 8 up rows for a gated
// epilogue) and all rows of A, up to 16 MB of them; its waves split K in turns of 64 (one
// 128-byte line of every weight row) and add their sums up through the LDS.
//
// Operand layout of the 16x16x32 MFMA: lane l holds row l % 16, k 8 (l / 16) ..
// + 8.  Loads straight into it touch 16 lines with 16 neighbouring lanes, which
// costs the vector L1 64 clocks per KB (16 bytes a clock and CU, measured), as
// much as the weights alone may take.  So both operands go to the LDS by DMA, in
// whole 128-byte lines (20 clocks per KB), each wave its own turns D ahead, and
// from there to the products; chunks are permuted by row (chunk ^ row / 2) so
// that 16 rows cover all banks.  32 rows of 7168 x 7168: 26.2 us, against 33.4
// with the weights loaded directly and 41 with both.  With up to four rows
// A's lanes coincide and everything goes directly (DMA = false; one row of
// 4096 x 4096: 9.1 against 9.3 us).
// NB = 2 halves what A costs, and is taken once 16 rows a block would give
// more blocks than CUs.  A turn past the end, or k past the end, reads zeros
// without a request.
// Rows past the end repeat the last one; their sums are not used.
#pragma once

#include "dense_dma.h"
#include "dense_rows.h"

namespace mxmoe {
namespace {

constexpr int kFewWaves = 8;

// LDS of a block: the waves' turns (then their parts of the sums), and the sums.
// (One array: with several, the compiler gives each alias scopes by which it
// drains all LDS DMA before an LDS read.)
template <int MB, int NB, bool DMA, int D, int W = kFewWaves>
struct FewLds {
  static constexpr int PITCH = 16 * NB + 4;
  static constexpr int TURN = DMA ? (MB + NB) * 2048 : 0;         // bytes of a wave's turn: A, then weights
  static constexpr int PART = W * MB * NB * 1024, XBUF = W * D * TURN;
  static constexpr int BUF = XBUF > PART ? XBUF : PART;
  static constexpr int BYTES = BUF + MB * 16 * PITCH * 4;
};

// Weight columns [block * COLS, + COLS) for all rows of A (up to 16 MB).
template <typename E, int MB, int NB, int EPI, bool DMA, int D, bool GATHER = false, int WAVES = kFewWaves>
__device__ __forceinline__ void few_block(const DenseJob& p, int block, char* lds) {
  typedef typename Vec<E>::v8 v8;
  using L = FewLds<MB, NB, DMA, D, WAVES>;
  constexpr int COLS = NB * (EPI == kEpiGate ? 8 : 16), PITCH = L::PITCH, TURN = L::TURN, BUF = L::BUF;
  float (*const sums)[PITCH] = reinterpret_cast<float (*)[PITCH]>(lds + BUF);   // padded: reads spread over the banks
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int width = EPI == kEpiGate ? p.N >> 1 : p.N, n0 = block * COLS;
  // weight row behind column c of the block's 16 NB
  auto b_row = [&](int c) {
    if (EPI != kEpiGate) return min(n0 + c, width - 1);
    const int i = min(n0 + (c >> 4) * 8 + (c & 7), width - 1), up = (c >> 3) & 1;
    return p.interleaved ? 2 * i + up : up * width + i;
  };
  const int l16 = lane & 15, kl = 8 * (lane >> 4);
  const int K = p.K;
  const int turns = (((K + 63) >> 6) - wave + WAVES - 1) / WAVES;  // lines wave, wave + WAVES, ...
  const int row0 = __builtin_amdgcn_readfirstlane(b_row(0));       // the lowest of the block's rows
  const char* const wbase = static_cast<const char*>(p.b) + (int64_t)row0 * p.ldb * 2;
  const char* const xbase = static_cast<const char*>(p.a);
  // this lane's offsets: by DMA row 8 j + lane / 8 of 2 * 8 rows per block of
  // 16 (row / 2 % 8 is 4 (j % 2) + lane / 16), directly row 16 i + lane % 16
  const int c8 = (lane & 7) ^ ((lane >> 4) & 3);
  constexpr int PER = DMA ? 2 : 1;
  uint32_t xoff[PER * MB], woff[PER * NB];
#pragma unroll
  for (int j = 0; j < PER * MB; ++j) {
    int row = min(DMA ? 8 * j + (lane >> 3) : 16 * j + l16, p.M - 1);
    const int g = GATHER ? p.gather[row] : 0;
    if constexpr (GATHER) row = g / p.gather_div;
    xoff[j] = (uint32_t)(row * (p.lda * 2)) + (DMA ? (c8 ^ ((j & 1) << 2)) * 16 : kl * 2);
    if (GATHER && (g < 0 || row >= p.gather_rows)) xoff[j] = kOut;
  }
#pragma unroll
  for (int j = 0; j < PER * NB; ++j)
    woff[j] = (uint32_t)((b_row(DMA ? 8 * j + (lane >> 3) : 16 * j + l16) - row0) * (p.ldb * 2)) +
              (DMA ? (c8 ^ ((j & 1) << 2)) * 16 : kl * 2);
  char* const ring = lds + wave * D * TURN;
  v8 xr[DMA ? 1 : D][2][MB], wr[DMA ? 1 : D][2][NB];
  auto load = [&](int t, int u) {
    const int k = (wave + t * WAVES) * 64;
    const auto rx = rsrc_at(xbase + (int64_t)k * 2), rw = rsrc_at(wbase + (int64_t)k * 2);
    if constexpr (DMA) {
#pragma unroll
      for (int j = 0; j < 2 * (MB + NB); ++j) {
        const uint32_t o = j < 2 * MB ? xoff[j < 2 * MB ? j : 0] : woff[j < 2 * MB ? 0 : j - 2 * MB];
        dma16(j < 2 * MB ? rx : rw, k + (c8 ^ ((j & 1) << 2)) * 8 < K ? o : kOut, ring + u * TURN + j * 1024);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = k + 32 * h + kl < K;
#pragma unroll
        for (int i = 0; i < MB; ++i) xr[u][h][i] = load16<E>(rx, in ? xoff[i] + 64 * h : kOut);   // (kOut + 64: behind, too)
#pragma unroll
        for (int n = 0; n < NB; ++n) wr[u][h][n] = load16<E>(rw, in ? woff[n] + 64 * h : kOut);
      }
    }
  };
  // operand h of block i of the turn in buffer u (A's blocks, then the weights')
  auto operand = [&](int u, int h, int i) {
    const int row = i * 16 + l16;
    return read_lds((const __attribute__((address_space(3))) v8*)(
        ring + u * TURN + row * 128 + (((h * 4 + (lane >> 4)) ^ ((row >> 1) & 7)) << 4)));
  };

  v4f acc[NB][MB];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[n][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < D; ++u) {
    load(u, u);
    __builtin_amdgcn_sched_barrier(0);   // the waits below count on this order
  }
  // D turns per step without a way out between them, so that every load has a
  // register of its own for good (a copy would wait for it); turns past the end
  // add zeros
  for (int t0 = 0; t0 < turns; t0 += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      v8 a[2][MB], b[2][NB];
      if constexpr (DMA) {
        // this turn's loads have landed; those of the D - 1 younger turns may fly
        wait_vm<(D - 1) * 2 * (MB + NB)>();
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          if constexpr (DMA) a[h][i] = operand(u, h, i);
          else a[h][i] = xr[u][h][i];
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if constexpr (DMA) b[h][n] = operand(u, h, MB + n);
          else b[h][n] = wr[u][h][n];
        }
      }
      if constexpr (DMA) {
        wait_lgkm0();                      // the buffer has been read
        __builtin_amdgcn_sched_barrier(0);
        load(t0 + u + D, u);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < MB; ++i) acc[n][i] = mfma16(b[h][n], a[h][i], acc[n][i]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (!DMA) {
        load(t0 + u + D, u);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if constexpr (DMA) {   // the sums take the place of A's turns
    wait_vm<0>();
    __syncthreads();
  }
  v4f (*const part)[NB * MB][64] = reinterpret_cast<v4f (*)[NB * MB][64]>(lds);
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < MB; ++i) part[wave][n * MB + i][lane] = acc[n][i];
  __syncthreads();
  // accumulator q of lane l: row l % 16, column 4 (l / 16) + q
  for (int t = threadIdx.x; t < NB * MB * 64; t += 64 * WAVES) {
    const int f = t >> 6, l = t & 63;
    v4f v = part[0][f][l];
#pragma unroll
    for (int j = 1; j < WAVES; ++j) v += part[j][f][l];
    *reinterpret_cast<v4f*>(&sums[f % MB * 16 + (l & 15)][f / MB * 16 + 4 * (l >> 4)]) = v;
  }
  __syncthreads();
  // each row's adapter: one thread per (row, column)
  if (p.ids) {
    for (int t = threadIdx.x; t < MB * NB * 256; t += 64 * WAVES) {
      const int m = t / (16 * NB), c = t % (16 * NB);
      if (m >= p.M) break;
      const int id = p.ids[m];
      if (id < 0 || id >= p.num_adapters) continue;
      int rank = p.R;
      if (p.ranks) rank = min(max(p.ranks[id], 0), p.R);
      const float* const s = p.s + (size_t)m * p.R;
      const E* const lb = static_cast<const E*>(p.lb) + ((size_t)id * p.N + b_row(c)) * p.R;
      float v = 0.0f;
      for (int r = 0; r < rank; r += 8) {
        const v8 bv = *reinterpret_cast<const v8*>(lb + r);
        const F8 sv = load8<E>(s, MOE_FLOAT_FP32, r);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (r + e < rank) v += sv.v[e] * (float)bv[e];
      }
      sums[m][c] += v;
    }
    __syncthreads();
  }
  auto sums8 = [&](int m, int c) {
    const v4f a = *reinterpret_cast<const v4f*>(&sums[m][c]), b = *reinterpret_cast<const v4f*>(&sums[m][c + 4]);
    return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  };
  const int t = threadIdx.x;
  if constexpr (EPI == kEpiGate) {
    const int m = t / NB, n = t % NB;
    if (m < p.M && n0 + 8 * n < width) finish_gate<E>(p, m, n0 + 8 * n, sums8(m, 16 * n), sums8(m, 16 * n + 8));
  } else {
    const int m = t / (2 * NB), c = t % (2 * NB) * 8;
    if (m < p.M && n0 + c < width) finish_plain<E>(p, m, n0 + c, sums8(m, c));
  }
}

template <typename E, int MB, int NB, int EPI, bool DMA, int D>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(DenseJob p) {
  __shared__ __attribute__((aligned(1024))) char lds[FewLds<MB, NB, DMA, D>::BYTES];
  few_block<E, MB, NB, EPI, DMA, D>(p, blockIdx.x, lds);
}

}  // namespace
}  // namespace mxmoe
