// The dense kernel for few rows (decode): bound by reading the weights once.
//
// A block owns 16 NB weight rows (groups of 8 gate + 8 up rows for a gated
// epilogue) and all rows of A, up to 16 MB of them; its waves split K in turns of 64 (one
// 128-byte line of every weight row) and add their sums up through the LDS.
//
// Weights go straight to registers in the 16x16x32 MFMA's operand layout (lane
// l: row l % 16, k 8 (l / 16) .. + 8): each is used once.  In that layout 16
// neighbouring lanes touch 16 lines, which costs the vector L1 64 clocks per
// KB (16 bytes a clock and CU, measured); the weights alone stay under that,
// but A, which every block reads whole, would not.  So A takes the other way:
// DMA to the LDS in whole 128-byte lines (50 bytes a clock), each wave its own
// turns, and fragments from there; chunks are permuted by row (chunk ^ row / 2)
// so that 16 rows cover all banks.  With up to four rows the lanes' addresses
// coincide and direct loads are as cheap (XLDS = false).
// Loads return in order, so both run the same D turns ahead: 2 KB of weights
// per wave and turn, of which a CU needs some 24 KB in flight.
// NB = 2 halves what A costs, and is taken once 16 rows a block would give
// more blocks than CUs.
// A turn past the end, or k past the end, reads zeros without a request.
// Rows past the end repeat the last one; their sums are not used.
#pragma once

#include "dense_dma.h"
#include "dense_rows.h"

namespace mxmoe {
namespace {

constexpr int kFewWaves = 8;

template <typename E, int MB, int NB, int EPI, bool XLDS, int D>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(DenseJob p) {
  typedef typename Vec<E>::v8 v8;
  constexpr int WAVES = kFewWaves;
  constexpr int COLS = NB * (EPI == kEpiGate ? 8 : 16), PITCH = 16 * NB + 4;
  constexpr int TURN_X = XLDS ? MB * 2048 : 0;                     // LDS bytes of a wave's turn of A
  constexpr int PART = WAVES * MB * NB * 1024, XBUF = WAVES * D * TURN_X;
  constexpr int BUF = XBUF > PART ? XBUF : PART;
  // one array: with several, the compiler gives each alias scopes by which it
  // drains all LDS DMA before an LDS read
  __shared__ __attribute__((aligned(1024))) char lds[BUF + MB * 16 * PITCH * 4];
  float (*const sums)[PITCH] = reinterpret_cast<float (*)[PITCH]>(lds + BUF);   // padded: reads spread over the banks
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int width = EPI == kEpiGate ? p.N >> 1 : p.N, n0 = blockIdx.x * COLS;
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
  uint32_t woff[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) woff[n] = (uint32_t)((b_row(16 * n + l16) - row0) * (p.ldb * 2)) + kl * 2;
  const char* const wbase = static_cast<const char*>(p.b) + (int64_t)row0 * p.ldb * 2;
  const char* const xbase = static_cast<const char*>(p.a);
  // W of a turn: two operands (k 0..31 and 32..63 of the line)
  v8 b[D][2][NB];
  auto load_w = [&](int t, int u) {
    const int k = (wave + t * WAVES) * 64;
    const auto rs = rsrc_at(wbase + (int64_t)k * 2);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NB; ++n) b[u][h][n] = load16<E>(rs, k + 32 * h + kl < K ? woff[n] + 64 * h : kOut);
  };
  // A of a turn: into LDS buffer u, or registers
  uint32_t xoff[XLDS ? 2 * MB : MB];
  const int xc = (lane & 7) ^ ((lane >> 4) & 3);                   // row r = 8 j + lane / 8: r / 2 % 8 is
  if constexpr (XLDS) {                                            // 4 (j % 2) + lane / 16
#pragma unroll
    for (int j = 0; j < 2 * MB; ++j)
      xoff[j] = (uint32_t)(min(8 * j + (lane >> 3), p.M - 1) * (p.lda * 2)) + (xc ^ ((j & 1) << 2)) * 16;
  } else {
#pragma unroll
    for (int i = 0; i < MB; ++i) xoff[i] = (uint32_t)(min(i * 16 + l16, p.M - 1) * (p.lda * 2)) + kl * 2;
  }
  char* const xbuf = lds + wave * D * TURN_X;
  v8 xr[XLDS ? 1 : D][2][MB];
  auto load_x = [&](int t, int u) {
    const int k = (wave + t * WAVES) * 64;
    const auto rs = rsrc_at(xbase + (int64_t)k * 2);
    if constexpr (XLDS) {
#pragma unroll
      for (int j = 0; j < 2 * MB; ++j)
        dma16(rs, k + (xc ^ ((j & 1) << 2)) * 8 < K ? xoff[j] : kOut, xbuf + u * TURN_X + j * 1024);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MB; ++i) xr[u][h][i] = load16<E>(rs, k + 32 * h + kl < K ? xoff[i] + 64 * h : kOut);
    }
  };

  v4f acc[NB][MB];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[n][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < D; ++u) {
    load_x(u, u);
    load_w(u, u);
    __builtin_amdgcn_sched_barrier(0);   // the waits below count on this order
  }
  // D turns per step without a way out between them, so that every load has a
  // register of its own for good (a copy would wait for it); turns past the end
  // add zeros
  for (int t0 = 0; t0 < turns; t0 += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      const int t = t0 + u;
      v8 a[2][MB];
      if constexpr (XLDS) {
        // this turn's loads have landed; those of the D - 1 younger turns may fly
        wait_vm<(D - 1) * (2 * MB + 2 * NB)>();
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const int row = i * 16 + l16;
          if constexpr (XLDS)
            a[h][i] = read_lds((const __attribute__((address_space(3))) v8*)(
                xbuf + u * TURN_X + row * 128 + (((h * 4 + (lane >> 4)) ^ ((row >> 1) & 7)) << 4)));
          else a[h][i] = xr[u][h][i];
        }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < MB; ++i) acc[n][i] = mfma16(b[u][h][n], a[h][i], acc[n][i]);
      if constexpr (XLDS) wait_lgkm0();    // the buffer has been read
      __builtin_amdgcn_sched_barrier(0);
      load_x(t + D, u);
      load_w(t + D, u);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (XLDS) {   // the sums take the place of A's turns
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

}  // namespace
}  // namespace mxmoe
