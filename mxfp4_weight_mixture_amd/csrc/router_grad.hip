// Gradients of the weighted top-k combine and of the top-k softmax.
//
// Combine: dy[dest] = w dout[t] and dw = <y[dest], dout[t]>, one workgroup a
// token, so that dout is read once: bound by reading y and writing dy.  A
// thread holds its columns of dout and walks the token's rows; the k dot
// products are summed over the block at the end.  y stays in 16 bits until it is
// multiplied (fewer registers, more waves) and dy, which is not read here again,
// is stored past the caches: 8192 tokens, top 6 of 4096 columns, 191 us (4.9 TB/s);
// 214 with y widened as it came, plain stores and blocks of 512 threads, 250 with
// two vectors a thread.
//
// Routing: a row of E zeros but for k values, one wave a token.  Each lane owns
// expert ids and compares them with the token's k, which come from registers of
// the first k lanes: no scatter, so an id listed twice simply adds up.
#include <algorithm>

#include "dense.h"
#include "dense_rows.h"

namespace mxmoe {
namespace {

constexpr int kRows = 8;   // rows of a token handled together

// Sums of eight values over the wave's lanes: lane l gets value l % 8's.  Three
// steps halve the values a lane holds while they double the lanes behind each,
// three more finish: 10 exchanges for 48.
__device__ __forceinline__ float wave_sum8(const float (&v)[kRows], int lane) {
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float keep = lane & 4 ? v[4 + i] : v[i], give = lane & 4 ? v[i] : v[4 + i];
    a[i] = keep + __shfl_xor(give, 4);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = lane & 2 ? a[2 + i] : a[i], give = lane & 2 ? a[i] : a[2 + i];
    b[i] = keep + __shfl_xor(give, 2);
  }
  float c = (lane & 1 ? b[1] : b[0]) + __shfl_xor(lane & 1 ? b[0] : b[1], 1);
#pragma unroll
  for (int off = 8; off < 64; off <<= 1) c += __shfl_xor(c, off);
  return c;
}

// Eight values as they are stored.
template <typename E, bool F32>
struct Raw8 {
  v4f a, b;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    const v4f* const q = reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i);
    a = q[0], b = q[1];
  }
  __device__ __forceinline__ float at(int e) const { return e < 4 ? a[e] : b[e - 4]; }
};
template <typename E>
struct Raw8<E, false> {
  typename Vec<E>::v8 a;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    a = *reinterpret_cast<const typename Vec<E>::v8*>(static_cast<const E*>(p) + i);
  }
  __device__ __forceinline__ float at(int e) const { return (float)a[e]; }
};

// YF, DF: y and dy in fp32 (else types E and D).
template <typename E, typename D, bool YF, bool DF>
__global__ __launch_bounds__(256) void combine_grad_kernel(const float* __restrict__ dout, const void* __restrict__ y,
                                                           const int32_t* __restrict__ dest_row,
                                                           const float* __restrict__ w, int T, int k, int H,
                                                           void* __restrict__ dy, float* __restrict__ dw) {
  __shared__ float sums[4][kRows];
  const int64_t t = blockIdx.x;
  const int64_t rows = (int64_t)T * k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockDim.x, nv = H >> 3;
  for (int j0 = 0; j0 < k; j0 += kRows) {
    float dot[kRows], wj[kRows];
    int64_t dest[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      dot[j] = 0.0f;
      dest[j] = j0 + j < k ? dest_row[t * k + j0 + j] : -1;
      if (dest[j] >= rows) dest[j] = -1;
      wj[j] = dest[j] >= 0 ? w[t * k + j0 + j] : 0.0f;
    }
    for (int v = threadIdx.x; v < nv; v += n) {
      Raw8<E, YF> r[kRows];
      if (dw) {
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (dest[j] >= 0) r[j].load(y, dest[j] * H + 8 * v);
      }
      const F8 d = load8<E>(dout, MOE_FLOAT_FP32, t * H + 8 * v);
      if (dy) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          if (dest[j] < 0) continue;
          if constexpr (DF) {
            F8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o.v[e] = wj[j] * d.v[e];
            store8<D>(dy, MOE_FLOAT_FP32, dest[j] * H + 8 * v, o);
          } else {
            typename Vec<D>::v8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (D)(wj[j] * d.v[e]);
            __builtin_nontemporal_store(o, reinterpret_cast<typename Vec<D>::v8*>(static_cast<D*>(dy) + dest[j] * H + 8 * v));
          }
        }
      }
      if (dw) {
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (dest[j] >= 0)
#pragma unroll
            for (int e = 0; e < 8; ++e) dot[j] = fmaf(r[j].at(e), d.v[e], dot[j]);
      }
    }
    if (!dw) continue;
    const float s8 = wave_sum8(dot, lane);
    if (lane < kRows) sums[wave][lane] = s8;
    __syncthreads();
    if (threadIdx.x < kRows && j0 + (int)threadIdx.x < k) {
      float s = 0.0f;
      for (int i = 0; i < n >> 6; ++i) s += sums[i][threadIdx.x];
      dw[t * k + j0 + threadIdx.x] = s;
    }
    if (j0 + kRows < k) __syncthreads();
  }
}

__global__ __launch_bounds__(256) void route_grad_kernel(const float* __restrict__ dw, const int32_t* __restrict__ ids,
                                                         const float* __restrict__ w, int T, int E, int k,
                                                         float* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const float wj = lane < k ? w[t * k + lane] : 0.0f, dj = lane < k ? dw[t * k + lane] : 0.0f;
  const int id = lane < k ? ids[t * k + lane] : -1;
  float dot = wj * dj;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) dot += __shfl_xor(dot, off);
  const float g = wj * (dj - dot);
  float* const row = dlogits + t * E;
  for (int e0 = 0; e0 < E; e0 += 64) {
    float v = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int i = __builtin_amdgcn_readlane(id, j);
      const float gj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), j));
      v += i == e0 + lane ? gj : 0.0f;
    }
    if (e0 + lane < E) row[e0 + lane] = v;
  }
}

}  // namespace
}  // namespace mxmoe

using namespace mxmoe;

extern "C" {

moe_status moe_combine_backward(const float* dout, const void* y, int32_t y_dtype, const int32_t* dest_row,
                                const float* topk_w, int32_t T, int32_t k, int32_t H, void* dy, int32_t dy_dtype,
                                float* dtopk_w, void* stream) {
  const char* what = "combine backward";
  clear_error();
  if (T < 0 || T >= 1 << 22 || k < 1 || k > 64)   // a block of up to 256 threads a token
    return fail(MOE_ERR_SHAPE, "%s: T = %d, k = %d out of range", what, T, k);
  MXMOE_TRY(check_width(what, "H", H));
  const int64_t rows = (int64_t)T * k;
  auto bad = [](int t) { return t != MOE_FLOAT_BF16 && t != MOE_FLOAT_FP16 && t != MOE_FLOAT_FP32; };
  if (dtopk_w && bad(y_dtype)) return fail(MOE_ERR_INVALID_ARG, "%s: bad y_dtype %d", what, y_dtype);
  if (dy && bad(dy_dtype)) return fail(MOE_ERR_INVALID_ARG, "%s: bad dy_dtype %d", what, dy_dtype);
  if (T > 0) {
    if (!dout || !dest_row || !topk_w || (dtopk_w && !y)) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    const void* words[] = {dest_row, topk_w, dtopk_w};
    for (const void* p : words)
      if (reinterpret_cast<uintptr_t>(p) & 3)
        return fail(MOE_ERR_INVALID_ARG, "%s: dest_row, topk_w and dtopk_w must be 4-byte aligned", what);
    const Span out[] = {span("dy", dy, rows, H, H, dy_dtype)};
    const Span in[] = {span("dout", dout, T, H, H, MOE_FLOAT_FP32), span("y", dtopk_w ? y : nullptr, rows, H, H, y_dtype)};
    MXMOE_TRY(check_spans(what, out, 1, in, 2));
    const Span dw = {"dtopk_w", dtopk_w, dtopk_w ? (size_t)rows * 4 : 0};
    const Span others[] = {{"dest_row", dest_row, (size_t)rows * 4}, {"topk_w", topk_w, (size_t)rows * 4}};
    for (const Span& o : others) {
      if (overlap(out[0], o)) return fail(MOE_ERR_INVALID_ARG, "%s: dy overlaps %s", what, o.name);
      if (overlap(dw, o)) return fail(MOE_ERR_INVALID_ARG, "%s: dtopk_w overlaps %s", what, o.name);
    }
    for (const Span& o : {out[0], in[0], in[1]})
      if (overlap(dw, o)) return fail(MOE_ERR_INVALID_ARG, "%s: dtopk_w and %s overlap", what, o.name);
  }
  MXMOE_TRY(check_device());
  if (T == 0 || (!dy && !dtopk_w)) return MOE_OK;
  const hipStream_t s = (hipStream_t)stream;
  const dim3 grid((unsigned)T), block(std::min(256, (H / 8 + 63) / 64 * 64));
  const int yt = dtopk_w ? y_dtype : MOE_FLOAT_FP32, dt = dy ? dy_dtype : MOE_FLOAT_FP32;
#define MXMOE_LAUNCH(E, D, YF, DF) \
  hipLaunchKernelGGL((combine_grad_kernel<E, D, YF, DF>), grid, block, 0, s, dout, y, dest_row, topk_w, T, k, H, dy, dtopk_w)
#define MXMOE_LAUNCH_Y(E, YF)                                              \
  if (dt == MOE_FLOAT_FP32) MXMOE_LAUNCH(E, __bf16, YF, true);             \
  else if (dt == MOE_FLOAT_BF16) MXMOE_LAUNCH(E, __bf16, YF, false);       \
  else MXMOE_LAUNCH(E, _Float16, YF, false)
  if (yt == MOE_FLOAT_FP32) { MXMOE_LAUNCH_Y(__bf16, true); }
  else if (yt == MOE_FLOAT_BF16) { MXMOE_LAUNCH_Y(__bf16, false); }
  else { MXMOE_LAUNCH_Y(_Float16, false); }
#undef MXMOE_LAUNCH_Y
#undef MXMOE_LAUNCH
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

moe_status moe_route_backward(const float* dtopk_w, const int32_t* topk_ids, const float* topk_w, int32_t T, int32_t E,
                              int32_t k, float* dlogits, void* stream) {
  const char* what = "route backward";
  clear_error();
  // (four tokens a block: fewer than 2^24 blocks, 2^32 threads; a launch of more does not run, without an error)
  if (T < 0 || T > kMaxRouted) return fail(MOE_ERR_SHAPE, "%s: T = %d outside [0, %d]", what, T, kMaxRouted);
  if (E < 1 || E > 1024) return fail(MOE_ERR_SHAPE, "%s: E = %d outside [1, 1024]", what, E);
  if (k < 1 || k > E || k > 64) return fail(MOE_ERR_SHAPE, "%s: k = %d outside [1, min(E=%d, 64)]", what, k, E);
  if (T > 0) {
    if (!dtopk_w || !topk_ids || !topk_w || !dlogits) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    const size_t pairs = (size_t)T * k * 4;
    const Span out = {"dlogits", dlogits, (size_t)T * E * 4};
    const Span in[] = {{"dtopk_w", dtopk_w, pairs}, {"topk_ids", topk_ids, pairs}, {"topk_w", topk_w, pairs}};
    for (const Span& i : in) {
      if (overlap(out, i)) return fail(MOE_ERR_INVALID_ARG, "%s: dlogits overlaps %s", what, i.name);
      if (reinterpret_cast<uintptr_t>(i.p) & 3)
        return fail(MOE_ERR_INVALID_ARG, "%s: %s is not 4-byte aligned", what, i.name);
    }
    if (reinterpret_cast<uintptr_t>(dlogits) & 3)
      return fail(MOE_ERR_INVALID_ARG, "%s: dlogits is not 4-byte aligned", what);
  }
  MXMOE_TRY(check_device());
  if (T == 0) return MOE_OK;
  hipLaunchKernelGGL(route_grad_kernel, dim3((T + 3) / 4), dim3(256), 0, (hipStream_t)stream, dtopk_w, topk_ids, topk_w,
                     T, E, k, dlogits);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

}  // extern "C"
