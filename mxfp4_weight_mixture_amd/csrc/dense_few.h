// The dense kernel for few rows (decode): bound by reading the weights once.
//
// A block of eight waves owns 16 weight rows (8 gate + 8 up rows for a gated
// epilogue) and all rows of A, up to 16 MB of them; the waves split K in turns
// of 64 (one 128-byte line of every weight row) and add their sums up through
// the LDS.  Weights go straight to registers in the 16x16x32 MFMA's operand
// layout (lane l: row l % 16, k 8 (l / 16) .. + 8): each is used once, so the
// LDS would only add a hop.  A is small and comes from the L2.  Rows past the
// end repeat the last one; their sums are not used.
#pragma once

#include "dense_rows.h"

namespace mxmoe {
namespace {

constexpr int kFewWaves = 8;

template <typename E>
__device__ __forceinline__ typename Vec<E>::v8 load_stream(const E* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const typename Vec<E>::v8*>(p));
}

template <typename E, int MB, int EPI>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(DenseJob p) {
  typedef typename Vec<E>::v8 v8;
  constexpr int UNROLL = MB >= 4 ? 2 : 4;
  constexpr int COLS = EPI == kEpiGate ? 8 : 16;
  __shared__ __attribute__((aligned(16))) v4f part[kFewWaves][MB][64];
  __shared__ __attribute__((aligned(16))) float sums[MB * 16][20];   // 80-byte rows: 16-byte reads spread over the banks
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int width = EPI == kEpiGate ? p.N >> 1 : p.N, n0 = blockIdx.x * COLS;
  // weight row behind column c of the block's 16
  auto b_row = [&](int c) {
    if (EPI != kEpiGate) return min(n0 + c, width - 1);
    const int i = min(n0 + (c & 7), width - 1), up = c >> 3;
    return p.interleaved ? 2 * i + up : up * width + i;
  };
  const int kl = 8 * (lane >> 4);
  const E* const w = static_cast<const E*>(p.b) + (size_t)b_row(lane & 15) * p.ldb + kl;
  const E* x[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
    x[i] = static_cast<const E*>(p.a) + (size_t)min(i * 16 + (lane & 15), p.M - 1) * p.lda + kl;

  v4f acc[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int TURN = 64 * kFewWaves;
  int k = wave * 64;
  for (; k + (UNROLL - 1) * TURN + 64 <= p.K; k += UNROLL * TURN) {
    v8 b[UNROLL][2], a[UNROLL][2][MB];
#pragma unroll
    for (int q = 0; q < UNROLL; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        b[q][h] = load_stream<E>(w + k + q * TURN + h * 32);
#pragma unroll
        for (int i = 0; i < MB; ++i) a[q][h][i] = *reinterpret_cast<const v8*>(x[i] + k + q * TURN + h * 32);
      }
#pragma unroll
    for (int q = 0; q < UNROLL; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[i] = mfma16(b[q][h], a[q][h][i], acc[i]);
  }
  for (; k < p.K; k += TURN) {
    v8 b[2] = {}, a[2][MB] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (k + h * 32 + kl < p.K) {
        b[h] = load_stream<E>(w + k + h * 32);
#pragma unroll
        for (int i = 0; i < MB; ++i) a[h][i] = *reinterpret_cast<const v8*>(x[i] + k + h * 32);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MB; ++i) acc[i] = mfma16(b[h], a[h][i], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  // accumulator q of lane l: row l % 16, column 4 (l / 16) + q
  for (int t = threadIdx.x; t < MB * 64; t += 64 * kFewWaves) {
    const int i = t >> 6, l = t & 63;
    v4f v = part[0][i][l];
#pragma unroll
    for (int j = 1; j < kFewWaves; ++j) v += part[j][i][l];
    *reinterpret_cast<v4f*>(&sums[i * 16 + (l & 15)][4 * (l >> 4)]) = v;
  }
  __syncthreads();
  // each row's adapter: one thread per (row, column)
  if (p.ids) {
    for (int t = threadIdx.x; t < MB * 256; t += 64 * kFewWaves) {
      const int m = t >> 4, c = t & 15;
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
    if (t < p.M && n0 < width) finish_gate<E>(p, t, n0, sums8(t, 0), sums8(t, 8));
  } else {
    const int m = t >> 1, c = (t & 1) * 8;
    if (m < p.M && n0 + c < width) finish_plain<E>(p, m, n0 + c, sums8(m, c));
  }
}

}  // namespace
}  // namespace mxmoe
