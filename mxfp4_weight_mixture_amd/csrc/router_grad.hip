// Gradients of the weighted top-k combine and of the top-k softmax.
//
// Combine: dy[dest] = w dout[t] and dw = <y[dest], dout[t]>, one workgroup a
// token, so that dout is read once: bound by reading y and writing dy.  A
// thread holds its columns of dout and walks the token's rows; the k dot
// products are summed over the block at the end.
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

// YF, DF: y and dy in fp32 (else type E).
template <typename E, typename D, bool YF, bool DF>
__global__ __launch_bounds__(512) void combine_grad_kernel(const float* __restrict__ dout, const void* __restrict__ y,
                                                           const int32_t* __restrict__ dest_row,
                                                           const float* __restrict__ w, int T, int k, int H,
                                                           void* __restrict__ dy, float* __restrict__ dw) {
  __shared__ float sums[8][kRows];
  constexpr int YT = YF ? MOE_FLOAT_FP32 : MOE_FLOAT_BF16, DT = DF ? MOE_FLOAT_FP32 : MOE_FLOAT_BF16;
  const int64_t t = blockIdx.x;
  const int64_t rows = (int64_t)T * k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
    for (int v = threadIdx.x; v < H >> 3; v += blockDim.x) {
      const F8 d = load8<E>(dout, MOE_FLOAT_FP32, t * H + 8 * v);
      if (dw) {
        F8 r[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (dest[j] >= 0) r[j] = load8<E>(y, YT, dest[j] * H + 8 * v);
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (dest[j] >= 0)
#pragma unroll
            for (int e = 0; e < 8; ++e) dot[j] = fmaf(r[j].v[e], d.v[e], dot[j]);
      }
      if (dy) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          if (dest[j] < 0) continue;
          F8 o;
#pragma unroll
          for (int e = 0; e < 8; ++e) o.v[e] = wj[j] * d.v[e];
          store8<D>(dy, DT, dest[j] * H + 8 * v, o);
        }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
      if (lane == 0) sums[wave][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kRows && j0 + (int)threadIdx.x < k) {
      float s = 0.0f;
      for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += sums[i][threadIdx.x];
      dw[t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
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
  if (T < 0 || T >= 1 << 22 || k < 1 || k > 64)   // a block of up to 512 threads a token
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
  const dim3 grid((unsigned)T), block(std::min(512, (H / 8 + 63) / 64 * 64));
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
  if (T < 0 || T >= 1 << 26) return fail(MOE_ERR_SHAPE, "%s: T = %d out of range", what, T);
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
