// What the dense kernels do with their sums, eight consecutive columns of one
// row at a time: 16-byte accesses of the 16-bit tensors.
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
    const typename Vec<E>::v8 a = *reinterpret_cast<const typename Vec<E>::v8*>(static_cast<const E*>(base) + i);
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
    *reinterpret_cast<typename Vec<E>::v8*>(static_cast<E*>(base) + i) = o;
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

// What follows the sums, on eight consecutive columns of one row.
// Plain: v are columns [n, n + 8) of C.
template <typename E>
__device__ __forceinline__ void finish_plain(const DenseJob& p, int m, int n, F8 v) {
  if (p.add) {
    const F8 a = load8<E>(p.add, p.c_dtype, (size_t)m * p.ldadd + n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v.v[e] += a.v[e];
  }
  store8<E>(p.c, p.c_dtype, (size_t)m * p.ldc + n, v);
}
// Gate: g, u are the pre-activations of gate indices [i, i + 8).
template <typename E>
__device__ __forceinline__ void finish_gate(const DenseJob& p, int m, int i, F8 g, F8 u) {
  const int I = p.N >> 1;
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
// Gate gradient: d are dh's columns [i, i + 8).
template <typename E>
__device__ __forceinline__ void finish_gate_grad(const DenseJob& p, int m, int i, F8 d) {
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

}  // namespace
}  // namespace mxmoe
