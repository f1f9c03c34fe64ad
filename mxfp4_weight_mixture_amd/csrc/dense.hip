// Dense products with 16-bit operands on the matrix cores, with the epilogues
// of the gated feed-forward block and the adapters' second product.
//
// The weights (B rows) are the MFMA's first operand and the tokens (A rows)
// its second, so a lane's accumulators hold one token row: accumulator q of
// lane l of a 32x32 fragment is C[m = l % 32][n = 8 (q/4) + 4 (l/32) + q%4],
// four runs of four consecutive columns.  For a gated epilogue a tile's
// columns come in groups of 64: 32 gate rows of W, then the 32 matching up
// rows, so that a lane holds both of a pair.
#include "dense.h"

namespace mxmoe {
namespace {

constexpr int BM = 128, BN = 128, BK = 64, kThreads = 256;
constexpr int kPitch = BK + 8;   // LDS elements per row

// Row of B that feeds tile column j of n-tile nt; -1: none.
__device__ __forceinline__ int b_row(const DenseJob& p, int nt, int bn, int j) {
  if (p.epi != kEpiGate) {
    const int r = nt * bn + j;
    return r < p.N ? r : -1;
  }
  const int I = p.N >> 1;
  const int i = nt * (bn >> 1) + (j >> 6) * 32 + (j & 31), up = (j >> 5) & 1;
  if (i >= I) return -1;
  return p.interleaved ? 2 * i + up : up * I + i;
}

// One stage of an operand: rows [r0, ...) x k [k0, k0 + BK) into lds[row][k].
template <typename E>
__device__ __forceinline__ void stage(const E* src, int64_t ld, int t, int rows, int K, int r0, int k0, bool b_map,
                                      const DenseJob& p, int nt, E* lds) {
  typedef typename Vec<E>::v8 v8;
  for (int c = threadIdx.x; c < 128 * BK / 8; c += kThreads) {
    if (!t) {
      const int r = c / (BK / 8), kc = (c % (BK / 8)) * 8;
      const int row = b_map ? b_row(p, nt, BN, r) : (r0 + r < rows ? r0 + r : -1);
      v8 v = {};
      if (row >= 0 && k0 + kc < K) v = *reinterpret_cast<const v8*>(src + (size_t)row * ld + k0 + kc);
      *reinterpret_cast<v8*>(lds + r * kPitch + kc) = v;
    } else {
      const int k = c / 16, r = (c % 16) * 8;
      v8 v = {};
      if (k0 + k < K && r0 + r < rows) v = *reinterpret_cast<const v8*>(src + (size_t)(k0 + k) * ld + r0 + r);
      for (int i = 0; i < 8; ++i) lds[(r + i) * kPitch + k] = v[i];
    }
  }
}

template <typename E>
__global__ __launch_bounds__(kThreads) void tile_kernel(DenseJob p) {
  typedef typename Vec<E>::v8 v8;
  __shared__ __attribute__((aligned(16))) E la[BM * kPitch], lb[BN * kPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const int l32 = lane & 31, g = lane >> 5;
  const int nt = blockIdx.x, m0 = blockIdx.y * BM;

  v16f acc[2][2] = {};   // [fm][fn]
  for (int k0 = 0; k0 < p.K; k0 += BK) {
    __syncthreads();
    stage<E>(static_cast<const E*>(p.a), p.lda, p.ta, p.M, p.K, m0, k0, false, p, 0, la);
    stage<E>(static_cast<const E*>(p.b), p.ldb, p.tb, p.N, p.K, nt * BN, k0, !p.tb, p, nt, lb);
    __syncthreads();
    for (int ks = 0; ks < BK; ks += 16) {
      v8 a[2], b[2];
      for (int f = 0; f < 2; ++f) {
        a[f] = *reinterpret_cast<const v8*>(la + (wm + f * 32 + l32) * kPitch + ks + 8 * g);
        b[f] = *reinterpret_cast<const v8*>(lb + (wn + f * 32 + l32) * kPitch + ks + 8 * g);
      }
      for (int fm = 0; fm < 2; ++fm)
        for (int fn = 0; fn < 2; ++fn) acc[fm][fn] = mfma32(b[fn], a[fm], acc[fm][fn]);
    }
  }

  for (int fm = 0; fm < 2; ++fm) {
    const int m = m0 + wm + fm * 32 + l32;
    // each adapter present in this fragment's rows in turn: its product goes
    // to a sum of its own, which only that adapter's rows take up
    if (p.ids) {
      const int id = m < p.M ? p.ids[m] : -1;
      bool open = id >= 0 && id < p.num_adapters;
      uint64_t left = __ballot(open);
      while (left) {
        const int cur = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
        const bool mine = open && id == cur;
        int rank = p.R;
        if (p.ranks) rank = min(max(p.ranks[cur], 0), p.R);
        for (int fn = 0; fn < 2; ++fn) {
          const int br = b_row(p, nt, BN, wn + fn * 32 + l32);
          v16f t = {};
          for (int r = 0; r < rank; r += 16) {
            v8 sv = {}, bv = {};
            const int k = r + 8 * g;
            if (mine && k < rank) sv = *reinterpret_cast<const v8*>(static_cast<const E*>(p.s) + (size_t)m * p.R + k);
            if (br >= 0 && k < rank)
              bv = *reinterpret_cast<const v8*>(static_cast<const E*>(p.lb) + ((size_t)cur * p.N + br) * p.R + k);
            for (int i = 0; i < 8; ++i)
              if (k + i >= rank) sv[i] = bv[i] = (E)0.0f;
            t = mfma32(bv, sv, t);
          }
          if (mine)
            for (int q = 0; q < 16; ++q) acc[fm][fn][q] += t[q];
        }
        open = open && !mine;
        left = __ballot(open);
      }
    }
    if (m >= p.M) continue;
    if (p.epi == kEpiGate) {
      const int I = p.N >> 1;
      for (int q = 0; q < 4; ++q) {
        const int i = nt * (BN / 2) + wn / 2 + 8 * q + 4 * g;
        if (i >= I) continue;
        v4f gt, up, hv;
        for (int e = 0; e < 4; ++e) {
          gt[e] = acc[fm][0][4 * q + e];
          up[e] = acc[fm][1][4 * q + e];
        }
        const size_t lo = p.interleaved ? 2 * i : i, hi = p.interleaved ? lo + 4 : lo + I;
        if (p.add) {
          const v4f x = load4<E>(p.add, p.c_dtype, (size_t)m * p.ldadd + lo);
          const v4f y = load4<E>(p.add, p.c_dtype, (size_t)m * p.ldadd + hi);
          gt += p.interleaved ? v4f{x[0], x[2], y[0], y[2]} : x;
          up += p.interleaved ? v4f{x[1], x[3], y[1], y[3]} : y;
        }
        if (p.gu) {
          store4<E>(p.gu, p.gu_dtype, (size_t)m * p.N + lo, p.interleaved ? v4f{gt[0], up[0], gt[1], up[1]} : gt);
          store4<E>(p.gu, p.gu_dtype, (size_t)m * p.N + hi, p.interleaved ? v4f{gt[2], up[2], gt[3], up[3]} : up);
        }
        for (int e = 0; e < 4; ++e) hv[e] = gate_act(p.act, gt[e]) * up[e];
        store4<E>(p.c, p.c_dtype, (size_t)m * p.ldc + i, hv);
      }
      continue;
    }
    for (int fn = 0; fn < 2; ++fn)
      for (int q = 0; q < 4; ++q) {
        const int n = nt * BN + wn + fn * 32 + 8 * q + 4 * g;
        if (n >= p.N) continue;
        v4f v;
        for (int e = 0; e < 4; ++e) v[e] = acc[fm][fn][4 * q + e];
        if (p.epi == kEpiPlain) {
          if (p.add) v += load4<E>(p.add, p.c_dtype, (size_t)m * p.ldadd + n);
          store4<E>(p.c, p.c_dtype, (size_t)m * p.ldc + n, v);
          continue;
        }
        // gate gradient: v = dh
        const size_t lo = (size_t)m * 2 * p.N + (p.interleaved ? 2 * n : n), hi = lo + (p.interleaved ? 4 : p.N);
        const v4f x = load4<E>(p.gu, p.gu_dtype, lo), y = load4<E>(p.gu, p.gu_dtype, hi);
        const v4f gt = p.interleaved ? v4f{x[0], x[2], y[0], y[2]} : x;
        const v4f up = p.interleaved ? v4f{x[1], x[3], y[1], y[3]} : y;
        v4f dg, du, hv;
        for (int e = 0; e < 4; ++e) {
          float a, da;
          gate_act_grad(p.act, gt[e], &a, &da);
          hv[e] = a * up[e];
          dg[e] = v[e] * up[e] * da;
          du[e] = v[e] * a;
        }
        store4<E>(p.h, p.dtype, (size_t)m * p.N + n, hv);
        store4<E>(p.c, p.c_dtype, lo, p.interleaved ? v4f{dg[0], du[0], dg[1], du[1]} : dg);
        store4<E>(p.c, p.c_dtype, hi, p.interleaved ? v4f{dg[2], du[2], dg[3], du[3]} : du);
      }
  }
}

}  // namespace

size_t dense_ws_bytes(int M, int N, int K) { return 0; }

moe_status launch_dense(const DenseJob& j, void* ws, hipStream_t s) {
  if (j.M == 0) return MOE_OK;
  const dim3 grid((j.N + BN - 1) / BN, (j.M + BM - 1) / BM);
  if (j.dtype == MOE_FLOAT_BF16)
    hipLaunchKernelGGL((tile_kernel<__bf16>), grid, dim3(kThreads), 0, s, j);
  else
    hipLaunchKernelGGL((tile_kernel<_Float16>), grid, dim3(kThreads), 0, s, j);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

}  // namespace mxmoe
