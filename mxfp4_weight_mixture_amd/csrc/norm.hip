// Root-mean-square norm with the residual's addition, 16-bit and MXFP8 outputs;
// its gradients.
//
// Forward: one pass.  A row stays in its block's registers between the sum of
// squares and the scaling, so x and residual are read once and every output is
// written once: bound by memory.  Eight values a thread and vector (16-byte
// loads); an MXFP8 block is four neighbouring threads' values, its amax two
// cross-lane exchanges.
//
// Backward: dx needs two sums over the row, mean(x^2) and mean(g u); both come
// from the same pass, since mean(g u) = inv * mean(g x).  dweight sums over the
// rows: every block holds its rows' part of it in registers, in row order, and
// writes it once; a second kernel adds the blocks' parts in order (no atomics).
#include <math.h>

#include <algorithm>

#include "dense.h"
#include "dense_rows.h"

namespace mxmoe {
namespace {

constexpr int kNormMaxH = 32768;
constexpr int kNormMaxT = (1 << 22) - 1;   // a block of up to 1024 threads a row: fewer than 2^32 threads

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
// Sums of a and b over the block, in every thread.  `area` is used by one call
// at a time: a caller in a loop passes two in turn.
__device__ __forceinline__ void block_sum2(float& a, float& b, float (*area)[2]) {
  a = wave_sum(a), b = wave_sum(b);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) area[threadIdx.x >> 6][0] = a, area[threadIdx.x >> 6][1] = b;
  __syncthreads();
  a = b = 0.0f;
  for (int w = 0; w < waves; ++w) a += area[w][0], b += area[w][1];
}

// E8M0 byte of an MXFP8 block whose largest magnitude has these bits: the
// smallest X with amax 2^-X <= 448 = 1.75 * 2^8, from -127 on; and 2^-X.
__device__ __forceinline__ uint32_t block_scale(uint32_t amax, float* inverse) {
  if (amax >= 0x7f800000u) {          // an infinity or NaN: every code becomes NaN
    *inverse = __uint_as_float(0x7fc00000u);
    return 255u;
  }
  const int e = (int)(amax >> 23) - 127 - ((amax & 0x7fffffu) > 0x600000u ? 7 : 8);
  const int X = max(e, -127);
  // 2^-X for X from -127 to 120
  *inverse = __uint_as_float((uint32_t)(127 - X) << 23);
  return (uint32_t)(X + 127);
}
// Four values of magnitude up to 448 as E4M3, nearest even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  typedef short s2 __attribute__((ext_vector_type(2)));
  const s2 lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(s2{0, 0}, a, b, 1.0f, false);
  const s2 hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(s2{0, 0}, c, d, 1.0f, false);
  return (uint32_t)(uint16_t)lo.x | ((uint32_t)(uint16_t)hi.x << 16);
}

// RES: 0 no residual, 1 in 16 bits, 2 in fp32.  V vectors of eight a thread.
template <typename E, int V, bool X32, int RES>
__global__ __launch_bounds__(1024) void norm_kernel(moe_norm_args p) {
  __shared__ float area[16][2];
  constexpr int XT = X32 ? MOE_FLOAT_FP32 : MOE_FLOAT_BF16, RT = RES == 2 ? MOE_FLOAT_FP32 : MOE_FLOAT_BF16;
  const int nv = p.H >> 3;
  const int64_t row = blockIdx.x;
  F8 r[V], w[V];
  float ss = 0.0f, none = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < nv) r[i] = load8<E>(p.x, XT, row * p.x_stride + 8 * v);
  }
  if constexpr (RES != 0) {
    F8 q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v < nv) q[i] = load8<E>(p.residual, RT, row * p.residual_stride + 8 * v);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v >= nv) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        r[i].v[e] += q[i].v[e];
        if constexpr (RES == 1) r[i].v[e] = (float)(E)r[i].v[e];   // the sum that is kept
      }
      store8<E>(p.residual_out, RT, row * p.residual_out_stride + 8 * v, r[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v >= nv) continue;
    w[i] = load8<E>(p.weight, p.weight_dtype, 8 * v);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(r[i].v[e], r[i].v[e], ss);
  }
  block_sum2(ss, none, area);
  const float inv = 1.0f / sqrtf(ss / (float)p.H + p.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v >= nv) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[i].v[e] = r[i].v[e] * inv * w[i].v[e];
    if (p.out) store8<E>(p.out, p.out_dtype, row * p.out_stride + 8 * v, r[i]);
    if (p.codes) {
      uint32_t amax = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(r[i].v[e]) & 0x7fffffffu);
      amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));   // (H is 32 n: the four threads are in together)
      amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
      float f;
      const uint32_t byte = block_scale(amax, &f);
      uint2 c;
      c.x = e4m3x4(r[i].v[0] * f, r[i].v[1] * f, r[i].v[2] * f, r[i].v[3] * f);
      c.y = e4m3x4(r[i].v[4] * f, r[i].v[5] * f, r[i].v[6] * f, r[i].v[7] * f);
      *reinterpret_cast<uint2*>(p.codes + row * p.H + 8 * v) = c;
      if ((threadIdx.x & 3) == 0) p.scales[(row * p.H >> 5) + (v >> 2)] = (uint8_t)byte;
    }
  }
}

// Eight values as they are stored, in fp32 or 16 bits.
struct Raw8 {
  v4f a, b;
  template <typename E>
  __device__ __forceinline__ void load(const void* p, int dtype, size_t i) {
    if (dtype == MOE_FLOAT_FP32) {
      const v4f* const q = reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i);
      a = q[0], b = q[1];
    } else {
      a = *reinterpret_cast<const v4f*>(static_cast<const E*>(p) + i);
    }
  }
  template <typename E>
  __device__ __forceinline__ F8 values(int dtype) const {
    if (dtype == MOE_FLOAT_FP32) return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    const typename Vec<E>::v8 h = __builtin_bit_cast(typename Vec<E>::v8, a);
    F8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = (float)h[e];
    return r;
  }
};

// Short rows (ALONE): every wave of a block has rows of its own, eight V lanes' worth
// of values, and no barrier but for dweight's parts at the end.  Longer rows: the
// block's threads share one.  The next row's loads go out before this row's sums
// meet, where there are registers for it.  8192 x 4096 in bf16 with a residual's
// gradient 54 us (5.0 TB/s), 64 without the loads ahead; 32768 x 512 36, 119 with a
// block of one wave for each row.
constexpr int kAloneWaves = 8;
template <typename E, int V, bool ALONE>
__global__ __launch_bounds__(ALONE ? 64 * kAloneWaves : 1024) void norm_grad_kernel(moe_norm_grad_args p, float* part) {
  constexpr int AHEAD = ALONE || V == 1 ? 2 : 1;
  __shared__ float area[2][16][2];
  __shared__ v4f sums[ALONE ? kAloneWaves * V * 128 : 1];
  const int nv = p.H >> 3, wave = threadIdx.x >> 6;
  const int lane = ALONE ? threadIdx.x & 63 : threadIdx.x, lanes = ALONE ? 64 : blockDim.x;
  const bool add = p.dx && p.dresidual;
  F8 w[V], dw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * lanes + lane;
    dw[i] = F8{};
    if (v < nv) w[i] = load8<E>(p.weight, p.weight_dtype, 8 * v);
  }
  Raw8 x[AHEAD][V], d[AHEAD][V], q[AHEAD][V];
  auto load = [&](int at, int64_t row) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * lanes + lane;
      if (v >= nv) continue;
      x[at][i].template load<E>(p.x, p.x_dtype, row * p.x_stride + 8 * v);
      d[at][i].template load<E>(p.dout, p.dout_dtype, row * p.dout_stride + 8 * v);
      if (add) q[at][i].template load<E>(p.dresidual, p.dresidual_dtype, row * p.dresidual_stride + 8 * v);
    }
  };
  auto grad = [&](int at, int64_t row, float (*meet)[2]) {
    F8 xv[V], dv[V];
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * lanes + lane;
      if (v >= nv) continue;
      xv[i] = x[at][i].template values<E>(p.x_dtype), dv[i] = d[at][i].template values<E>(p.dout_dtype);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(xv[i].v[e], xv[i].v[e], ss);
        dot = fmaf(dv[i].v[e] * w[i].v[e], xv[i].v[e], dot);
      }
    }
    if constexpr (ALONE) ss = wave_sum(ss), dot = wave_sum(dot);
    else block_sum2(ss, dot, meet);
    const float inv = 1.0f / sqrtf(ss / (float)p.H + p.eps);
    const float c = dot * inv / (float)p.H;   // mean(g u)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * lanes + lane;
      if (v >= nv) continue;
      F8 o{};
      if (add) o = q[at][i].template values<E>(p.dresidual_dtype);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = xv[i].v[e] * inv;
        dw[i].v[e] = fmaf(dv[i].v[e], u, dw[i].v[e]);
        o.v[e] = fmaf(inv, fmaf(-u, c, dv[i].v[e] * w[i].v[e]), o.v[e]);
      }
      if (p.dx) store8<E>(p.dx, p.dx_dtype, row * p.dx_stride + 8 * v, o);
    }
  };
  const int64_t step = ALONE ? (int64_t)gridDim.x * kAloneWaves : gridDim.x;
  const int64_t first = ALONE ? (int64_t)blockIdx.x * kAloneWaves + wave : blockIdx.x;
  if constexpr (AHEAD == 2) {
    // (dx may be written over dout or dresidual: the next row is another one)
    if (first < p.T) load(0, first);
    for (int64_t row = first; row < p.T; row += 2 * step) {
      if (row + step < p.T) load(1, row + step);
      grad(0, row, area[0]);
      if (row + step >= p.T) break;
      if (row + 2 * step < p.T) load(0, row + 2 * step);
      grad(1, row + step, area[1]);
    }
  } else {
    int turn = 0;
    for (int64_t row = first; row < p.T; row += step, turn ^= 1) {
      load(0, row);
      grad(0, row, area[turn]);
    }
  }
  if (!part) return;
  if constexpr (ALONE) {
    // the waves' parts in order
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v4f* const o = sums + (wave * V + i) * 128 + lane * 2;
      o[0] = v4f{dw[i].v[0], dw[i].v[1], dw[i].v[2], dw[i].v[3]};
      o[1] = v4f{dw[i].v[4], dw[i].v[5], dw[i].v[6], dw[i].v[7]};
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.H >> 2; c += 64 * kAloneWaves) {
      v4f t = sums[c];
#pragma unroll
      for (int w = 1; w < kAloneWaves; ++w) t += sums[w * V * 128 + c];
      *reinterpret_cast<v4f*>(part + (int64_t)blockIdx.x * p.H + 4 * c) = t;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * lanes + lane;
    if (v < nv) store8<E>(part, MOE_FLOAT_FP32, (int64_t)blockIdx.x * p.H + 8 * v, dw[i]);
  }
}

// dweight from the blocks' parts: four columns a thread, 32 threads share a
// column's parts (part s, s + 32, ..., eight of them in flight), their sums are
// added in order.
template <typename E>
__global__ __launch_bounds__(256) void norm_weight_kernel(moe_norm_grad_args p, const float* part, int parts) {
  __shared__ v4f sums[32][8];
  const int col = threadIdx.x & 7, s = threadIdx.x >> 3, h = (blockIdx.x * 8 + col) * 4;
  v4f t{0.0f, 0.0f, 0.0f, 0.0f};
  if (h < p.H)
    for (int b0 = s; b0 < parts; b0 += 256) {
      v4f r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        if (b0 + 32 * i < parts) r[i] = *reinterpret_cast<const v4f*>(part + (int64_t)(b0 + 32 * i) * p.H + h);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) t += r[i];
    }
  sums[s][col] = t;
  __syncthreads();
  if (s != 0 || h >= p.H) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) t += sums[i][col];
  for (int e = 0; e < 4; ++e) {
    float v = t[e];
    if (p.dw_dtype == MOE_FLOAT_FP32) {
      float* const o = static_cast<float*>(p.dweight) + h + e;
      *o = p.accumulate ? *o + v : v;
    } else {
      E* const o = static_cast<E*>(p.dweight) + h + e;
      *o = (E)(p.accumulate ? (float)*o + v : v);
    }
  }
}

// Rows of up to this many values: a wave each in the backward pass.
constexpr int kAloneH = 1024;
int norm_vectors(int H) { return H <= 8192 ? 1 : H <= 16384 ? 2 : 4; }
int norm_threads(int H, int V) { return ((H / 8 + V - 1) / V + 63) / 64 * 64; }

template <typename E, int V, bool X32>
moe_status launch_norm(const moe_norm_args& a, hipStream_t s) {
  const dim3 grid((unsigned)a.T), block(norm_threads(a.H, V));
  if (!a.residual) hipLaunchKernelGGL((norm_kernel<E, V, X32, 0>), grid, block, 0, s, a);
  else if (a.residual_dtype == MOE_FLOAT_FP32) hipLaunchKernelGGL((norm_kernel<E, V, X32, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_kernel<E, V, X32, 1>), grid, block, 0, s, a);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}
template <typename E>
moe_status launch_norm(const moe_norm_args& a, hipStream_t s) {
  const bool x32 = a.x_dtype == MOE_FLOAT_FP32;
  switch (norm_vectors(a.H)) {
    case 1: return x32 ? launch_norm<E, 1, true>(a, s) : launch_norm<E, 1, false>(a, s);
    case 2: return x32 ? launch_norm<E, 2, true>(a, s) : launch_norm<E, 2, false>(a, s);
    default: return x32 ? launch_norm<E, 4, true>(a, s) : launch_norm<E, 4, false>(a, s);
  }
}

// Blocks of the backward pass, and parts of dweight: 1024 threads a CU in whole
// rounds.  (8192 x 4096 54 us with 512 blocks, 58 with 1024, 74 with 256; x 2048 32 with
// 1024, 37 with 512; x 7168 110 with 256, 118 with 1024.)
int grad_blocks(int T, int H) {
  const bool alone = H <= kAloneH;
  const int threads = alone ? 64 * kAloneWaves : norm_threads(H, norm_vectors(H));
  return std::min(alone ? (T + kAloneWaves - 1) / kAloneWaves : T, std::max(256, 262144 / threads / 256 * 256));
}

template <typename E>
moe_status launch_norm_grad(const moe_norm_grad_args& a, hipStream_t s) {
  const bool alone = a.H <= kAloneH;
  const int parts = grad_blocks(a.T, a.H);
  float* const part = a.dweight ? static_cast<float*>(a.workspace) : nullptr;
  if (a.T > 0) {
    const int V = norm_vectors(a.H);
    const dim3 grid((unsigned)parts), block(alone ? 64 * kAloneWaves : norm_threads(a.H, V));
    if (a.H <= 512) hipLaunchKernelGGL((norm_grad_kernel<E, 1, true>), grid, block, 0, s, a, part);
    else if (alone) hipLaunchKernelGGL((norm_grad_kernel<E, 2, true>), grid, block, 0, s, a, part);
    else if (V == 1) hipLaunchKernelGGL((norm_grad_kernel<E, 1, false>), grid, block, 0, s, a, part);
    else if (V == 2) hipLaunchKernelGGL((norm_grad_kernel<E, 2, false>), grid, block, 0, s, a, part);
    else hipLaunchKernelGGL((norm_grad_kernel<E, 4, false>), grid, block, 0, s, a, part);
    MXMOE_HIP(hipGetLastError());
  }
  if (a.dweight) {
    hipLaunchKernelGGL((norm_weight_kernel<E>), dim3((a.H + 31) / 32), dim3(256), 0, s, a, part, parts);
    MXMOE_HIP(hipGetLastError());
  }
  return MOE_OK;
}

moe_status check_norm(const char* what, int T, int H, int dtype, float eps) {
  if (H < 8 || H > kNormMaxH || H % 8)
    return fail(MOE_ERR_SHAPE, "%s: H = %d must be a multiple of 8 in [8, %d]", what, H, kNormMaxH);
  if (T < 0 || T > kNormMaxT) return fail(MOE_ERR_SHAPE, "%s: T = %d outside [0, %d]", what, T, kNormMaxT);
  if (!(eps >= 0.0f) || isinf(eps)) return fail(MOE_ERR_INVALID_ARG, "%s: eps %g must be finite and >= 0", what, eps);
  return check_dtype16(what, dtype);
}

// The same rows under two names: allowed to coincide, then dropped from the overlap checks.
bool same_rows(const void* a, int a_dtype, int64_t a_stride, const void* b, int b_dtype, int64_t b_stride) {
  return a == b && a_dtype == b_dtype && a_stride == b_stride;
}

}  // namespace
}  // namespace mxmoe

using namespace mxmoe;

extern "C" {

moe_status moe_rms_norm_forward(const moe_norm_args* a, void* stream) {
  const char* what = "RMS norm";
  clear_error();
  if (!a) return fail(MOE_ERR_INVALID_ARG, "%s: null args", what);
  MXMOE_TRY(check_norm(what, a->T, a->H, a->dtype, a->eps));
  MXMOE_TRY(check_dtype_or_fp32(what, "x_dtype", a->x_dtype, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "weight_dtype", a->weight_dtype, a->dtype));
  MXMOE_TRY(check_stride(what, "x_stride", a->x_stride, a->H));
  if (!a->residual != !a->residual_out)
    return fail(MOE_ERR_INVALID_ARG, "%s: residual and residual_out come together", what);
  if (a->residual) {
    MXMOE_TRY(check_dtype_or_fp32(what, "residual_dtype", a->residual_dtype, a->dtype));
    MXMOE_TRY(check_stride(what, "residual_stride", a->residual_stride, a->H));
    MXMOE_TRY(check_stride(what, "residual_out_stride", a->residual_out_stride, a->H));
  }
  if (a->out) {
    MXMOE_TRY(check_dtype_or_fp32(what, "out_dtype", a->out_dtype, a->dtype));
    MXMOE_TRY(check_stride(what, "out_stride", a->out_stride, a->H));
  }
  if (!a->codes != !a->scales) return fail(MOE_ERR_INVALID_ARG, "%s: codes and scales come together", what);
  if (a->codes && a->H % 32) return fail(MOE_ERR_SHAPE, "%s: MXFP8 needs H %% 32 == 0 (H = %d)", what, a->H);
  const int64_t T = a->T, H = a->H;
  if (T > 0) {
    if (!a->x || !a->weight) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!a->out && !a->codes) return fail(MOE_ERR_INVALID_ARG, "%s: no output (out or codes)", what);
    const bool in_residual = same_rows(a->residual_out, a->residual_dtype, a->residual_out_stride, a->residual,
                                       a->residual_dtype, a->residual_stride);
    const bool in_x = same_rows(a->residual_out, a->residual_dtype, a->residual_out_stride, a->x, a->x_dtype, a->x_stride);
    const bool out_x = same_rows(a->out, a->out_dtype, a->out_stride, a->x, a->x_dtype, a->x_stride);
    const Span out[] = {span("out", a->out, T, H, a->out_stride, a->out_dtype),
                        span("residual_out", a->residual_out, T, H, a->residual_out_stride, a->residual_dtype),
                        {"codes", a->codes, a->codes ? (size_t)(T * H) : 0},
                        {"scales", a->scales, a->scales ? (size_t)(T * H / 32) : 0}};
    const Span in[] = {span("x", a->x, T, H, a->x_stride, a->x_dtype),
                       span("residual", a->residual, T, H, a->residual_stride, a->residual_dtype),
                       span("weight", a->weight, 1, H, H, a->weight_dtype)};
    for (int i = 0; i < 4; ++i) {
      if (i < 3 && !aligned16(out[i].p)) return fail(MOE_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", what, out[i].name);
      for (int j = i + 1; j < 4; ++j)
        if (overlap(out[i], out[j]))
          return fail(MOE_ERR_INVALID_ARG, "%s: %s and %s overlap", what, out[i].name, out[j].name);
      for (int j = 0; j < 3; ++j) {
        const bool same = (i == 0 && j == 0 && out_x) || (i == 1 && j == 0 && in_x) || (i == 1 && j == 1 && in_residual);
        if (!same && overlap(out[i], in[j]))
          return fail(MOE_ERR_INVALID_ARG, "%s: %s overlaps %s", what, out[i].name, in[j].name);
      }
    }
    for (const Span& s : in)
      if (!aligned16(s.p)) return fail(MOE_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", what, s.name);
  }
  MXMOE_TRY(check_device());
  if (T == 0) return MOE_OK;
  const hipStream_t s = (hipStream_t)stream;
  return a->dtype == MOE_FLOAT_BF16 ? launch_norm<__bf16>(*a, s) : launch_norm<_Float16>(*a, s);
}

size_t moe_rms_norm_grad_workspace_size(int32_t T, int32_t H) {
  if (T < 0 || T > kNormMaxT || H < 8 || H > kNormMaxH) return 0;
  return (size_t)grad_blocks(T, H) * H * 4 + 256;
}

moe_status moe_rms_norm_backward(const moe_norm_grad_args* a, void* stream) {
  const char* what = "RMS norm backward";
  clear_error();
  if (!a) return fail(MOE_ERR_INVALID_ARG, "%s: null args", what);
  MXMOE_TRY(check_norm(what, a->T, a->H, a->dtype, a->eps));
  MXMOE_TRY(check_dtype_or_fp32(what, "dout_dtype", a->dout_dtype, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "x_dtype", a->x_dtype, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "weight_dtype", a->weight_dtype, a->dtype));
  if (a->accumulate != 0 && a->accumulate != 1)
    return fail(MOE_ERR_INVALID_ARG, "%s: accumulate %d must be 0 or 1", what, a->accumulate);
  MXMOE_TRY(check_stride(what, "dout_stride", a->dout_stride, a->H));
  MXMOE_TRY(check_stride(what, "x_stride", a->x_stride, a->H));
  if (a->dresidual) {
    MXMOE_TRY(check_dtype_or_fp32(what, "dresidual_dtype", a->dresidual_dtype, a->dtype));
    MXMOE_TRY(check_stride(what, "dresidual_stride", a->dresidual_stride, a->H));
  }
  if (a->dx) {
    MXMOE_TRY(check_dtype_or_fp32(what, "dx_dtype", a->dx_dtype, a->dtype));
    MXMOE_TRY(check_stride(what, "dx_stride", a->dx_stride, a->H));
  }
  if (a->dweight) MXMOE_TRY(check_dtype_or_fp32(what, "dw_dtype", a->dw_dtype, a->dtype));
  const int64_t T = a->T, H = a->H;
  const size_t need = moe_rms_norm_grad_workspace_size(a->T, a->H);
  if (T > 0) {
    if (!a->dout || !a->x || !a->weight) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    if (a->dweight && (!a->workspace || a->workspace_bytes < need))
      return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", what, a->workspace_bytes, need);
  }
  const bool dx_dout = same_rows(a->dx, a->dx_dtype, a->dx_stride, a->dout, a->dout_dtype, a->dout_stride);
  const bool dx_dres = same_rows(a->dx, a->dx_dtype, a->dx_stride, a->dresidual, a->dresidual_dtype, a->dresidual_stride);
  const Span out[] = {span("dx", a->dx, T, H, a->dx_stride, a->dx_dtype),
                      span("dweight", a->dweight, 1, H, H, a->dw_dtype),
                      {"workspace", a->workspace, T > 0 && a->dweight ? need : 0}};
  const Span in[] = {span("dout", dx_dout ? nullptr : a->dout, T, H, a->dout_stride, a->dout_dtype),
                     span("x", a->x, T, H, a->x_stride, a->x_dtype),
                     span("weight", a->weight, 1, H, H, a->weight_dtype),
                     span("dresidual", dx_dres ? nullptr : a->dresidual, T, H, a->dresidual_stride, a->dresidual_dtype)};
  MXMOE_TRY(check_spans(what, out, 3, in, 4));
  MXMOE_TRY(check_device());
  if (!a->dx && !a->dweight) return MOE_OK;
  if (T == 0 && (!a->dweight || a->accumulate)) return MOE_OK;
  const hipStream_t s = (hipStream_t)stream;
  return a->dtype == MOE_FLOAT_BF16 ? launch_norm_grad<__bf16>(*a, s) : launch_norm_grad<_Float16>(*a, s);
}

}  // extern "C"
