// What the dense kernels do with their sums, eight consecutive columns of one
// row at a time: 16-byte accesses of the 16-bit tensors (8-byte aligned ones:
// a gated width may be an odd multiple of four, which then ends in half a group).
#pragma once

#include "dense.h"

namespace mxmoe {
namespace {

// Eight consecutive fp32 values.
struct F8 {
  float v[8];
};
template <typename E>
__device__ __forceinline__ F8 load8(const void* base, int dtype, size_t i) {
  F8 r;
  if (dtype == MOE_FLOAT_FP32) {
    const v4f* q = reinterpret_cast<const v4f*>(static_cast<const float*>(base) + i);
    const v4f a = q[0], b = q[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) r.v[e] = a[e], r.v[4 + e] = b[e];
  } else {
    const typename Vec<E>::v8 a = *reinterpret_cast<const typename Vec<E>::v8half*>(static_cast<const E*>(base) + i);
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = (float)a[e];
  }
  return r;
}
template <typename E>
__device__ __forceinline__ void store8(void* base, int dtype, size_t i, const F8& r) {
  if (dtype == MOE_FLOAT_FP32) {
    v4f* q = reinterpret_cast<v4f*>(static_cast<float*>(base) + i);
    q[0] = v4f{r.v[0], r.v[1], r.v[2], r.v[3]};
    q[1] = v4f{r.v[4], r.v[5], r.v[6], r.v[7]};
  } else {
    typename Vec<E>::v8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (E)r.v[e];
    *reinterpret_cast<typename Vec<E>::v8half*>(static_cast<E*>(base) + i) = o;
  }
}
// Eight gate and eight up values of row m, gate index i, from gate_up-shaped memory.
template <typename E>
__device__ __forceinline__ void load_pair(const void* base, int dtype, size_t row, int I, int i, int interleaved,
                                          F8* g, F8* u) {
  if (!interleaved) {
    *g = load8<E>(base, dtype, row + i);
    *u = load8<E>(base, dtype, row + I + i);
  } else {
    const F8 a = load8<E>(base, dtype, row + 2 * i), b = load8<E>(base, dtype, row + 2 * i + 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      g->v[e] = a.v[2 * e], u->v[e] = a.v[2 * e + 1];
      g->v[4 + e] = b.v[2 * e], u->v[4 + e] = b.v[2 * e + 1];
    }
  }
}
template <typename E>
__device__ __forceinline__ void store_pair(void* base, int dtype, size_t row, int I, int i, int interleaved,
                                           const F8& g, const F8& u) {
  if (!interleaved) {
    store8<E>(base, dtype, row + i, g);
    store8<E>(base, dtype, row + I + i, u);
  } else {
    F8 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a.v[2 * e] = g.v[e], a.v[2 * e + 1] = u.v[e];
      b.v[2 * e] = g.v[4 + e], b.v[2 * e + 1] = u.v[4 + e];
    }
    store8<E>(base, dtype, row + 2 * i, a);
    store8<E>(base, dtype, row + 2 * i + 8, b);
  }
}

// The same for the half group that ends a width of 8 n + 4: four gate and four
// up values, one by one.
template <typename E>
__device__ __forceinline__ void load_half_pair(const void* base, int dtype, size_t row, int I, int i, int interleaved,
                                               F8* g, F8* u) {
  for (int e = 0; e < 4; ++e) {
    const size_t a = row + (interleaved ? 2 * (i + e) : i + e), b = interleaved ? a + 1 : a + I;
    g->v[e] = dtype == MOE_FLOAT_FP32 ? static_cast<const float*>(base)[a] : (float)static_cast<const E*>(base)[a];
    u->v[e] = dtype == MOE_FLOAT_FP32 ? static_cast<const float*>(base)[b] : (float)static_cast<const E*>(base)[b];
    g->v[4 + e] = u->v[4 + e] = 0.0f;
  }
}
template <typename E>
__device__ __forceinline__ void store_half(void* base, int dtype, size_t i, const F8& v, int step = 1) {
  for (int e = 0; e < 4; ++e) {
    if (dtype == MOE_FLOAT_FP32) static_cast<float*>(base)[i + e * step] = v.v[e];
    else static_cast<E*>(base)[i + e * step] = (E)v.v[e];
  }
}

// What follows the sums, on eight consecutive columns of one row.
// Plain: v are columns [n, n + 8) of C.
template <typename E>
__device__ __forceinline__ void finish_plain(const DenseJob& p, int m, int n, F8 v) {
  if (p.partial) return store8<E>(p.partial, MOE_FLOAT_FP32, (size_t)m * p.N + n, v);
  if (p.add) {
    const F8 a = load8<E>(p.add, p.c_dtype, (size_t)m * p.ldadd + n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v.v[e] += a.v[e];
  }
  store8<E>(p.c, p.c_dtype, (size_t)m * p.ldc + n, v);
}
// Gate: g, u are the pre-activations of gate indices [i, i + 8).  The gate is
// taken of the fp32 sums; h is rounded once, to the 16 bits that the second
// product's matrix instructions take.  Two parts of it, as the adapters' small
// rows have, would double that product, a third of the block's work, for an
// error of the output 0.7 times as large.
template <typename E>
__device__ __forceinline__ void finish_gate(const DenseJob& p, int m, int i, F8 g, F8 u) {
  const int I = p.N >> 1;
  if (i + 8 > I) {
    if (p.partial) {
      const size_t row = (size_t)m * p.N;
      store_half<E>(p.partial, MOE_FLOAT_FP32, row + (p.interleaved ? 2 * i : i), g, p.interleaved ? 2 : 1);
      store_half<E>(p.partial, MOE_FLOAT_FP32, row + (p.interleaved ? 2 * i + 1 : I + i), u, p.interleaved ? 2 : 1);
      return;
    }
    F8 a{}, b{}, h;
    if (p.add) load_half_pair<E>(p.add, p.c_dtype, (size_t)m * p.ldadd, I, i, p.interleaved, &a, &b);
    for (int e = 0; e < 4; ++e) h.v[e] = gate_act(p.act, g.v[e] + a.v[e]) * (u.v[e] + b.v[e]);
    return store_half<E>(p.c, p.c_dtype, (size_t)m * p.ldc + i, h);   // (gate_up is kept for multiples of 8 only)
  }
  if (p.partial) return store_pair<E>(p.partial, MOE_FLOAT_FP32, (size_t)m * p.N, I, i, p.interleaved, g, u);
  if (p.add) {
    F8 a, b;
    load_pair<E>(p.add, p.c_dtype, (size_t)m * p.ldadd, I, i, p.interleaved, &a, &b);
#pragma unroll
    for (int e = 0; e < 8; ++e) g.v[e] += a.v[e], u.v[e] += b.v[e];
  }
  if (p.gu) store_pair<E>(p.gu, p.gu_dtype, (size_t)m * p.N, I, i, p.interleaved, g, u);
  F8 h;
#pragma unroll
  for (int e = 0; e < 8; ++e) h.v[e] = gate_act(p.act, g.v[e]) * u.v[e];
  store8<E>(p.c, p.c_dtype, (size_t)m * p.ldc + i, h);
}
// Gate gradient: d are dh's columns [i, i + 8), in fp32.  h and the gradients of
// gate and up are rounded once each, to the next products' 16-bit operands, in
// fp16 with its range: the loss is scaled for it, as for dout itself.
template <typename E>
__device__ __forceinline__ void finish_gate_grad(const DenseJob& p, int m, int i, F8 d) {
  if (p.partial) return store8<E>(p.partial, MOE_FLOAT_FP32, (size_t)m * p.N + i, d);
  F8 g, u, h;
  load_pair<E>(p.gu, p.gu_dtype, (size_t)m * 2 * p.N, p.N, i, p.interleaved, &g, &u);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float a, da;
    gate_act_grad(p.act, g.v[e], &a, &da);
    h.v[e] = a * u.v[e];
    g.v[e] = d.v[e] * u.v[e] * da;
    u.v[e] = d.v[e] * a;
  }
  store8<E>(p.h, p.dtype, (size_t)m * p.N + i, h);
  store_pair<E>(p.c, p.c_dtype, (size_t)m * p.ldc, p.N, i, p.interleaved, g, u);
}

// Part z of `splits` of K, in whole 64-deep stages: the job's operands from
// there on.  The adapters go with part 0.
__device__ __forceinline__ void take_part(DenseJob& p, float* partial, int z, int splits) {
  const int stages = (p.K + 63) >> 6, per = (stages + splits - 1) / splits;
  const int k0 = min(z * per * 64, p.K), k1 = min(k0 + per * 64, p.K);
  p.a = static_cast<const char*>(p.a) + (p.ta ? (int64_t)k0 * p.lda : k0) * 2;
  p.b = static_cast<const char*>(p.b) + (p.tb ? (int64_t)k0 * p.ldb : k0) * 2;
  p.K = k1 - k0;
  p.partial = partial + (size_t)z * p.M * p.N;
  if (z > 0) p.num_adapters = 0;
}

// The parts' sums in order, and what follows them: eight columns a thread.
template <typename E, int EPI>
__global__ __launch_bounds__(256) void join_kernel(DenseJob p, const float* partial, int splits) {
  const int width = EPI == kEpiGate ? p.N >> 1 : p.N, per = (width + 7) >> 3;
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int m = (int)(u / per), i = (int)(u % per) * 8;
  if (m >= p.M) return;
  F8 v{}, w{};
  for (int z = 0; z < splits; ++z) {
    const float* const q = partial + (size_t)z * p.M * p.N;
    if constexpr (EPI == kEpiGate) {
      F8 a, b;
      if (i + 8 > width) load_half_pair<E>(q, MOE_FLOAT_FP32, (size_t)m * p.N, width, i, p.interleaved, &a, &b);
      else load_pair<E>(q, MOE_FLOAT_FP32, (size_t)m * p.N, width, i, p.interleaved, &a, &b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v.v[e] += a.v[e], w.v[e] += b.v[e];
    } else {
      const F8 a = load8<E>(q, MOE_FLOAT_FP32, (size_t)m * p.N + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) v.v[e] += a.v[e];
    }
  }
  if constexpr (EPI == kEpiGate) finish_gate<E>(p, m, i, v, w);
  else if constexpr (EPI == kEpiGateGrad) finish_gate_grad<E>(p, m, i, v);
  else finish_plain<E>(p, m, i, v);
}

}  // namespace
}  // namespace mxmoe
