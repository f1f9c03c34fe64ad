// Low-rank adapters of many requests beside one shared projection.
//
//   y[t] = (add[t] +) x[t] W^T + s[t] B[a]^T,  s[t] = scales[a] x[t] A[a]^T,
//   a = ids[t] (none outside [0, num_adapters))
// Two launches: the first gives s [T][R] in fp32, the second the shared
// projection with s B^T added to its fp32 sums and the epilogue.
#include "dense.h"

namespace mxmoe {
namespace {

// One wave per (token, row of A): 64 lanes stride over K.
template <typename E>
__global__ __launch_bounds__(256) void shrink_kernel(moe_adapter_args p, float* s) {
  typedef typename Vec<E>::v8 v8;
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t = (int)(w / p.R), r = (int)(w % p.R);
  if (t >= p.T) return;
  const int id = p.ids[t];
  if (id < 0 || id >= p.num_adapters) return;   // its row of s is not read
  if (p.ranks && r >= p.ranks[id]) return;
  const E* x = static_cast<const E*>(p.x) + (size_t)t * p.x_stride;
  const E* a = static_cast<const E*>(p.a) + ((size_t)id * p.R + r) * p.K;
  float sum = 0.0f;
  for (int k = lane * 8; k < p.K; k += 512) {
    const v8 xv = *reinterpret_cast<const v8*>(x + k), av = *reinterpret_cast<const v8*>(a + k);
    for (int i = 0; i < 8; ++i) sum += (float)xv[i] * (float)av[i];
  }
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) s[(size_t)t * p.R + r] = p.scales ? sum * p.scales[id] : sum;
}

moe_status launch_shrink(const moe_adapter_args& a, void* s, hipStream_t st) {
  const dim3 grid((unsigned)(((int64_t)a.T * a.R + 3) / 4));
  if (a.dtype == MOE_FLOAT_BF16)
    hipLaunchKernelGGL((shrink_kernel<__bf16>), grid, dim3(256), 0, st, a, static_cast<float*>(s));
  else
    hipLaunchKernelGGL((shrink_kernel<_Float16>), grid, dim3(256), 0, st, a, static_cast<float*>(s));
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

struct AdapterWs {
  size_t s, gemm, total;
};
AdapterWs adapter_ws(int T, int K, int N, int R) {
  AdapterWs w;
  w.s = 0;
  w.gemm = align_up((size_t)T * R * 4, 256);
  w.total = w.gemm + dense_ws_bytes(T, N, K) + 256;
  return w;
}

}  // namespace
}  // namespace mxmoe

using namespace mxmoe;

extern "C" {

size_t moe_adapter_workspace_size(int32_t T, int32_t K, int32_t N, int32_t num_adapters, int32_t R) {
  if (T < 0 || K < 1 || N < 1 || num_adapters < 0 || R < 1) return 0;
  return adapter_ws(T, K, N, R).total;
}

moe_status moe_adapter_linear(const moe_adapter_args* a, void* stream) {
  const char* what = "adapter projection";
  clear_error();
  if (!a) return fail(MOE_ERR_INVALID_ARG, "%s: null args", what);
  if (a->T < 0) return fail(MOE_ERR_SHAPE, "%s: T = %d < 0", what, a->T);
  MXMOE_TRY(check_width(what, "K", a->K));
  MXMOE_TRY(check_width(what, "N", a->N));
  if (a->num_adapters < 0 || a->num_adapters > 65536)
    return fail(MOE_ERR_SHAPE, "%s: num_adapters = %d outside [0, 65536]", what, a->num_adapters);
  if (a->R < 8 || a->R > 256 || a->R % 8)
    return fail(MOE_ERR_SHAPE, "%s: R = %d must be a multiple of 8 in [8, 256]", what, a->R);
  const bool gate = a->epilogue != MOE_EPI_NONE;
  if (gate && a->epilogue != MOE_EPI_SWIGLU_SPLIT && a->epilogue != MOE_EPI_SWIGLU_INTERLEAVED)
    return fail(MOE_ERR_INVALID_ARG, "%s: bad epilogue %d", what, a->epilogue);
  if (gate && a->N % 16) return fail(MOE_ERR_SHAPE, "%s: N = %d (gate + up) must be a multiple of 16", what, a->N);
  if (gate && a->gate_act != MOE_GATE_SILU && a->gate_act != MOE_GATE_GELU)
    return fail(MOE_ERR_INVALID_ARG, "%s: bad gate_act %d", what, a->gate_act);
  if (gate && !a->w && a->T > 0) return fail(MOE_ERR_INVALID_ARG, "%s: a SWIGLU epilogue needs w", what);
  MXMOE_TRY(check_dtype16(what, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "out_dtype", a->out_dtype, a->dtype));
  const int64_t T = a->T, K = a->K, N = a->N, n = a->num_adapters, R = a->R, n_out = gate ? N / 2 : N;
  MXMOE_TRY(check_stride(what, "x_stride", a->x_stride, K));
  MXMOE_TRY(check_stride(what, "out_stride", a->out_stride, n_out));
  if (a->add) MXMOE_TRY(check_stride(what, "add_stride", a->add_stride, N));
  const AdapterWs w = adapter_ws(a->T, a->K, a->N, a->R);
  if (T > 0) {
    if (!a->x || !a->out || (n > 0 && (!a->ids || !a->a || !a->b)))
      return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!a->workspace || a->workspace_bytes < w.total)
      return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", what, a->workspace_bytes, w.total);
    const void* words[] = {a->ids, a->scales, a->ranks};
    for (const void* p : words)
      if (reinterpret_cast<uintptr_t>(p) & 3)
        return fail(MOE_ERR_INVALID_ARG, "%s: ids, scales and ranks must be 4-byte aligned", what);
    const bool in_place = !gate && a->add == a->out && a->add_stride == a->out_stride;
    const Span out[] = {span("out", a->out, T, n_out, a->out_stride, a->out_dtype),
                        {"workspace", a->workspace, w.total}};
    const Span in[] = {span("x", a->x, T, K, a->x_stride, a->dtype), span("w", a->w, N, K, K, a->dtype),
                       span("a", a->a, n * R, K, K, a->dtype), span("b", a->b, n * N, R, R, a->dtype),
                       span("add", in_place ? nullptr : a->add, T, N, a->add_stride, a->out_dtype)};
    MXMOE_TRY(check_spans(what, out, 2, in, 5));
    const Span words_in[] = {{"ids", a->ids, (size_t)T * 4}, {"scales", a->scales, a->scales ? (size_t)n * 4 : 0},
                             {"ranks", a->ranks, a->ranks ? (size_t)n * 4 : 0}};
    for (const Span& o : out)
      for (const Span& i : words_in)
        if (overlap(o, i)) return fail(MOE_ERR_INVALID_ARG, "%s: %s overlaps %s", what, o.name, i.name);
  }
  MXMOE_TRY(check_device());
  if (T == 0) return MOE_OK;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  const hipStream_t s = (hipStream_t)stream;

  DenseJob j{};
  j.dtype = a->dtype;
  j.M = a->T, j.N = a->N, j.K = a->w ? a->K : 0;
  j.a = a->x, j.lda = a->x_stride;
  j.b = a->w, j.ldb = K;
  j.epi = gate ? kEpiGate : kEpiPlain;
  j.interleaved = a->epilogue == MOE_EPI_SWIGLU_INTERLEAVED;
  j.act = a->gate_act;
  j.add = a->add, j.ldadd = a->add_stride;
  j.c = a->out, j.ldc = a->out_stride, j.c_dtype = a->out_dtype;
  if (n > 0) {
    MXMOE_TRY(launch_shrink(*a, ws + w.s, s));
    j.ids = a->ids, j.ranks = a->ranks;
    j.s = reinterpret_cast<const float*>(ws + w.s), j.lb = a->b;
    j.num_adapters = a->num_adapters, j.R = a->R;
  }
  return launch_dense(j, ws + w.gemm, s);
}

}  // extern "C"
