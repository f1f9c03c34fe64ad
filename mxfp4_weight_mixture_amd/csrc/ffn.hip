// The gated feed-forward block with 16-bit weights: entry points.
//
// Forward: one product with the gate in its epilogue (x w1^T -> h, and the
// pre-activations for a training caller), one plain product (h w2^T).
// Backward: dh = dout w2 with the gate's derivative in its epilogue, which
// writes d_gate_up and h; then dx = d_gate_up w1, dw1 = d_gate_up^T x and
// dw2 = dout^T h.  dh itself never reaches memory.
#include <algorithm>

#include "dense.h"

namespace mxmoe {
namespace {

moe_status check_block(const char* what, int T, int H, int I, int layout, int act, int dtype) {
  MXMOE_TRY(check_width(what, "H", H));
  MXMOE_TRY(check_width(what, "I", I));
  MXMOE_TRY(check_tokens(what, T, std::max(H, 2 * I)));
  if (layout != MOE_EPI_SWIGLU_SPLIT && layout != MOE_EPI_SWIGLU_INTERLEAVED)
    return fail(MOE_ERR_INVALID_ARG, "%s: layout %d must be a SWIGLU epilogue", what, layout);
  if (act != MOE_GATE_SILU && act != MOE_GATE_GELU)
    return fail(MOE_ERR_INVALID_ARG, "%s: bad gate_act %d", what, act);
  return check_dtype16(what, dtype);
}

// Sizes that a call may take, as far as the size queries' arithmetic needs it.
bool within_limits(int T, int H, int I) {
  return T >= 0 && T <= kMaxTokens && H > 0 && H <= kMaxWidth && I > 0 && I <= kMaxWidth;
}

// Workspaces: h, for the gradients d_gate_up and h; then the products' scratch
// (they run one after the other).
struct Ws {
  size_t h, gemm, total;
};
Ws ffn_ws(int T, int H, int I) {
  Ws w{};
  w.gemm = align_up((size_t)T * I * 2, 256);
  w.total = w.gemm + 256 +
            std::max(dense_ws_bytes(dense_sizes(T, 2 * I, H, kEpiGate, 0, 0)),
                     dense_ws_bytes(dense_sizes(T, H, I, kEpiPlain, 0, 0)));
  return w;
}
Ws grad_ws(int T, int H, int I) {
  Ws w{};
  w.h = align_up((size_t)T * 2 * I * 2, 256);
  w.gemm = w.h + align_up((size_t)T * I * 2, 256);
  w.total = w.gemm + 256 +
            std::max({dense_ws_bytes(dense_sizes(T, I, H, kEpiGateGrad, 0, 1)),
                      dense_ws_bytes(dense_sizes(T, H, 2 * I, kEpiPlain, 0, 1)),
                      dense_ws_bytes(dense_sizes(2 * I, H, T, kEpiPlain, 1, 1)),
                      dense_ws_bytes(dense_sizes(H, I, T, kEpiPlain, 1, 1))});
  return w;
}

}  // namespace
}  // namespace mxmoe

using namespace mxmoe;

extern "C" {

size_t moe_gated_ffn_workspace_size(int32_t T, int32_t H, int32_t I) {
  if (!within_limits(T, H, I)) return 0;
  return ffn_ws(T, H, I).total;
}

moe_status moe_gated_ffn_check(const moe_ffn_args* a) {
  const char* what = "gated FFN";
  clear_error();
  if (!a) return fail(MOE_ERR_INVALID_ARG, "%s: null args", what);
  MXMOE_TRY(check_block(what, a->T, a->H, a->I, a->layout, a->gate_act, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "out_dtype", a->out_dtype, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "save_dtype", a->save_dtype, a->dtype));
  MXMOE_TRY(check_stride(what, "x_stride", a->x_stride, a->H));
  MXMOE_TRY(check_stride(what, "out_stride", a->out_stride, a->H));
  if (a->add) MXMOE_TRY(check_stride(what, "add_stride", a->add_stride, a->H));
  const size_t need = ffn_ws(a->T, a->H, a->I).total;
  if (a->T > 0) {
    if (!a->x || !a->w1 || !a->w2 || !a->out) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!a->workspace || a->workspace_bytes < need)
      return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", what, a->workspace_bytes, need);
    const int64_t T = a->T, H = a->H, I = a->I;
    const bool in_place = a->add == a->out && a->add_stride == a->out_stride;
    const Span out[] = {span("out", a->out, T, H, a->out_stride, a->out_dtype),
                        span("gate_up", a->gate_up, T, 2 * I, 2 * I, a->save_dtype),
                        {"workspace", a->workspace, need}};
    const Span in[] = {span("x", a->x, T, H, a->x_stride, a->dtype), span("w1", a->w1, 2 * I, H, H, a->dtype),
                       span("w2", a->w2, H, I, I, a->dtype),
                       span("add", in_place ? nullptr : a->add, T, H, a->add_stride, a->out_dtype)};
    MXMOE_TRY(check_spans(what, out, 3, in, 4));
  }
  return check_device();
}

moe_status moe_gated_ffn_forward(const moe_ffn_args* a, void* stream) {
  MXMOE_TRY(moe_gated_ffn_check(a));
  if (a->T == 0) return MOE_OK;
  const Ws w = ffn_ws(a->T, a->H, a->I);
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  const hipStream_t s = (hipStream_t)stream;

  DenseJob j{};
  j.dtype = a->dtype;
  j.M = a->T;
  j.act = a->gate_act;
  j.interleaved = a->layout == MOE_EPI_SWIGLU_INTERLEAVED;
  j.a = a->x, j.lda = a->x_stride;
  j.b = a->w1, j.ldb = a->H;
  j.N = 2 * a->I, j.K = a->H;
  j.epi = kEpiGate;
  j.c = ws, j.ldc = a->I, j.c_dtype = a->dtype;
  j.gu = a->gate_up, j.gu_dtype = a->save_dtype;
  MXMOE_TRY(launch_dense(j, ws + w.gemm, s));

  j.a = ws, j.lda = a->I;
  j.b = a->w2, j.ldb = a->I;
  j.N = a->H, j.K = a->I;
  j.epi = kEpiPlain;
  j.gu = nullptr;
  j.add = a->add, j.ldadd = a->add_stride;
  j.c = a->out, j.ldc = a->out_stride, j.c_dtype = a->out_dtype;
  return launch_dense(j, ws + w.gemm, s);
}

size_t moe_gated_ffn_grad_workspace_size(int32_t T, int32_t H, int32_t I) {
  if (!within_limits(T, H, I)) return 0;
  return grad_ws(T, H, I).total;
}

moe_status moe_gated_ffn_backward(const moe_ffn_grad_args* a, void* stream) {
  const char* what = "gated FFN backward";
  clear_error();
  if (!a) return fail(MOE_ERR_INVALID_ARG, "%s: null args", what);
  MXMOE_TRY(check_block(what, a->T, a->H, a->I, a->layout, a->gate_act, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "save_dtype", a->save_dtype, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "dx_dtype", a->dx_dtype, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "dw_dtype", a->dw_dtype, a->dtype));
  if (a->accumulate != 0 && a->accumulate != 1)
    return fail(MOE_ERR_INVALID_ARG, "%s: accumulate %d must be 0 or 1", what, a->accumulate);
  MXMOE_TRY(check_stride(what, "dout_stride", a->dout_stride, a->H));
  if (a->dw1) MXMOE_TRY(check_stride(what, "x_stride", a->x_stride, a->H));
  if (a->dx) MXMOE_TRY(check_stride(what, "dx_stride", a->dx_stride, a->H));
  const Ws w = grad_ws(a->T, a->H, a->I);
  const size_t need = w.total;
  const int64_t T = a->T, H = a->H, I = a->I;
  if (T > 0) {
    if (!a->dout || !a->w2 || !a->gate_up || (a->dw1 && !a->x) || (a->dx && !a->w1))
      return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!a->workspace || a->workspace_bytes < need)
      return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", what, a->workspace_bytes, need);
  }
  const Span out[] = {span("dx", a->dx, T, H, a->dx_stride, a->dx_dtype),
                      span("dw1", a->dw1, 2 * I, H, H, a->dw_dtype), span("dw2", a->dw2, H, I, I, a->dw_dtype),
                      {"workspace", a->workspace, T > 0 ? need : 0}};
  const Span in[] = {span("dout", a->dout, T, H, a->dout_stride, a->dtype),
                     span("x", a->dw1 ? a->x : nullptr, T, H, a->x_stride, a->dtype),
                     span("w1", a->dx ? a->w1 : nullptr, 2 * I, H, H, a->dtype),
                     span("w2", a->w2, H, I, I, a->dtype),
                     span("gate_up", a->gate_up, T, 2 * I, 2 * I, a->save_dtype)};
  MXMOE_TRY(check_spans(what, out, 4, in, 5));
  MXMOE_TRY(check_device());
  if (!a->dx && !a->dw1 && !a->dw2) return MOE_OK;
  if (T == 0 && a->accumulate) return MOE_OK;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  const hipStream_t s = (hipStream_t)stream;

  uint8_t* const h = ws + w.h;
  DenseJob j{};
  j.dtype = a->dtype;
  j.act = a->gate_act;
  j.interleaved = a->layout == MOE_EPI_SWIGLU_INTERLEAVED;
  // the gradients of gate and up, and h
  j.a = a->dout, j.lda = a->dout_stride;
  j.b = a->w2, j.ldb = I, j.tb = 1;
  j.M = a->T, j.N = a->I, j.K = a->H;
  j.epi = kEpiGateGrad;
  j.gu = const_cast<void*>(a->gate_up), j.gu_dtype = a->save_dtype;
  j.c = ws, j.ldc = 2 * I, j.c_dtype = a->dtype;
  j.h = h;
  MXMOE_TRY(launch_dense(j, ws + w.gemm, s));

  // what is asked for of dx, dw1 and dw2, independent of each other
  DenseJob jobs[3];
  int n = 0;
  j.epi = kEpiPlain;
  j.gu = j.h = nullptr;
  if (a->dx) {
    j.a = ws, j.lda = 2 * I;
    j.b = a->w1, j.ldb = H, j.tb = 1;
    j.M = a->T, j.N = a->H, j.K = 2 * a->I;
    j.c = a->dx, j.ldc = a->dx_stride, j.c_dtype = a->dx_dtype;
    if (a->T > 0) jobs[n++] = j;
  }
  // the weights' gradients sum over the tokens: both operands have the
  // reduction outermost
  j.ta = j.tb = 1;
  j.K = a->T;
  j.c_dtype = a->dw_dtype;
  if (a->dw1) {
    j.a = ws, j.lda = 2 * I;
    j.b = a->x, j.ldb = a->x_stride;
    j.M = 2 * a->I, j.N = a->H;
    j.c = a->dw1, j.ldc = H;
    j.add = a->accumulate ? a->dw1 : nullptr, j.ldadd = H;
    jobs[n++] = j;
  }
  if (a->dw2) {
    j.a = a->dout, j.lda = a->dout_stride;
    j.b = h, j.ldb = I;
    j.M = a->H, j.N = a->I;
    j.c = a->dw2, j.ldc = I;
    j.add = a->accumulate ? a->dw2 : nullptr, j.ldadd = I;
    jobs[n++] = j;
  }
  MXMOE_TRY(launch_dense_group(jobs, n, ws + w.gemm, s));
  return MOE_OK;
}

}  // extern "C"
