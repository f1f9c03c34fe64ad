// Low-rank adapters of many requests beside one shared projection.
//
//   y[t] = (add[t] +) x[t] W^T + s[t] B[a]^T,  s[t] = scales[a] x[t] A[a]^T,
//   a = ids[t] (none outside [0, num_adapters))
// Up to kFewTokens tokens are taken for a decode batch (adapters mixed at
// will), more for prompts (adapters in runs); either way any order is right.
// Two launches: the first gives s [T][R] in fp32, the second the shared
// projection with s B^T added to its fp32 sums and the epilogue.
#include <algorithm>

#include "dense_small.h"

namespace mxmoe {
namespace {

constexpr int kMaxAdapters = 65536, kMaxRank = 256;

// s of few tokens.  A block takes one token and four rows of its adapter's A,
// its four waves a quarter of K each: tokens of a decode batch have adapters
// of their own, so there is little to share, and the time is one trip to memory.
template <typename E>
__global__ __launch_bounds__(256) void shrink_token_kernel(moe_adapter_args p, float* s) {
  typedef typename Vec<E>::v8 v8;
  __shared__ float part[4][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int groups = p.R >> 2, t = blockIdx.x / groups, r0 = blockIdx.x % groups * 4;
  const int id = p.ids[t];
  if (id < 0 || id >= p.num_adapters) return;   // its row of s is not read
  if (p.ranks && r0 >= p.ranks[id]) return;
  const E* const x = static_cast<const E*>(p.x) + (size_t)t * p.x_stride;
  const E* const a = static_cast<const E*>(p.a) + ((size_t)id * p.R + r0) * p.K;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
  for (int k = threadIdx.x * 8; k < p.K; k += 2048) {
    const v8 xv = *reinterpret_cast<const v8*>(x + k);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const v8 av = *reinterpret_cast<const v8*>(a + (size_t)r * p.K + k);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[r] += (float)xv[i] * (float)av[i];
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int d = 32; d; d >>= 1) sum[r] += __shfl_xor(sum[r], d);
    if (lane == 0) part[wave][r] = sum[r];
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    const int r = threadIdx.x;
    const float v = part[0][r] + part[1][r] + part[2][r] + part[3][r];
    s[(size_t)t * p.R + r0 + r] = p.scales ? v * p.scales[id] : v;
  }
}

// s of many tokens, whose requests come in runs: a block takes 32 tokens and,
// for each adapter among them (one, mostly), 32 FN rows of A at a time; its
// four waves split K.  Bound by reading x, which a ring of four stages a wave
// keeps in flight.  gridDim.y blocks share a tile's adapters, so that a tile
// where several requests meet takes no longer than the others.
template <typename E, int FN>
__global__ __launch_bounds__(256, 1) void shrink_runs_kernel(moe_adapter_args p, float* s) {
  using A = Operand<E, 32, false, 1>;
  using B = Operand<E, 32 * FN, false, 1>;
  constexpr int NST = 4, RING = NST * (A::BYTES + B::BYTES);
  static_assert(RING >= 32 * 32 * FN * 4, "the sums fit the ring");
  __shared__ __attribute__((aligned(1024))) char lds[4 * RING];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * 32;
  char* const ring = lds + wave * RING;
  A a;
  a.init(p.x, p.x_stride, p.T, t0, 0, lane);
  const int mine = t0 + (lane & 31) < p.T ? p.ids[t0 + (lane & 31)] : -1;
  uint64_t left = __ballot(lane < 32 && mine >= 0 && mine < p.num_adapters);
  for (int turn = 0; left; ++turn) {
    const int cur = __builtin_amdgcn_readlane(mine, __ffsll((unsigned long long)left) - 1);
    left &= ~__ballot(mine == cur);
    if (turn % gridDim.y != blockIdx.y) continue;
    int rank = p.R;
    if (p.ranks) rank = min(max(p.ranks[cur], 0), p.R);
    const float scale = p.scales ? p.scales[cur] : 1.0f;
    for (int r0 = 0; r0 < rank; r0 += 32 * FN) {
      B b;
      b.init(static_cast<const E*>(p.a) + (size_t)cur * p.R * p.K, p.K, rank, r0, 0, lane);
      v16f acc[1][FN];
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[0][f][q] = 0.0f;
      split_k_product<E, 1, FN, NST, 32>(a, b, p.K, wave, lane, ring, acc);
      put_sums<1, FN>(ring, lane, acc);
      __syncthreads();
      const int row = threadIdx.x / (4 * FN), x = threadIdx.x % (4 * FN), t = t0 + row, r = r0 + 8 * x;
      if (row < 32 && t < p.T && r < p.R && p.ids[t] == cur) {
        F8 v = get_sum8<FN>(lds, RING, row, 2 * x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] *= scale;
        store8<E>(s, MOE_FLOAT_FP32, (size_t)t * p.R + r, v);
      }
      __syncthreads();
    }
  }
}

template <typename E>
moe_status launch_shrink(const moe_adapter_args& a, float* s, hipStream_t st) {
  if (a.T <= kFewTokens)
    hipLaunchKernelGGL((shrink_token_kernel<E>), dim3(a.T * (a.R / 4)), dim3(256), 0, st, a, s);
  else if (a.R <= 32)
    hipLaunchKernelGGL((shrink_runs_kernel<E, 1>), dim3((a.T + 31) / 32, 4), dim3(256), 0, st, a, s);
  else
    hipLaunchKernelGGL((shrink_runs_kernel<E, 2>), dim3((a.T + 31) / 32, 4), dim3(256), 0, st, a, s);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

// Workspace: s, then the second product's scratch (the most that any form of
// it takes).
size_t adapter_gemm_offset(int T, int R) { return align_up((size_t)T * R * 4, 256); }
size_t adapter_ws_bytes(int T, int K, int N, int R) {
  size_t most = 0;
  for (int epi : {(int)kEpiPlain, (int)kEpiGate})
    for (bool ids : {false, true}) {
      static const int32_t some = 0;
      DenseJob j = dense_sizes(T, N, K, epi, 0, 0);
      j.ids = ids ? &some : nullptr;
      most = std::max(most, dense_ws_bytes(j));
    }
  return adapter_gemm_offset(T, R) + most + 256;
}

}  // namespace
}  // namespace mxmoe

using namespace mxmoe;

extern "C" {

size_t moe_adapter_workspace_size(int32_t T, int32_t K, int32_t N, int32_t num_adapters, int32_t R) {
  if (T < 0 || T > kMaxTokens || K < 1 || K > kMaxWidth || N < 1 || N > kMaxWidth) return 0;
  if (num_adapters < 0 || num_adapters > kMaxAdapters || R < 1 || R > kMaxRank) return 0;
  return adapter_ws_bytes(T, K, N, R);
}

moe_status moe_adapter_linear(const moe_adapter_args* a, void* stream) {
  const char* what = "adapter projection";
  clear_error();
  if (!a) return fail(MOE_ERR_INVALID_ARG, "%s: null args", what);
  MXMOE_TRY(check_width(what, "K", a->K));
  MXMOE_TRY(check_width(what, "N", a->N));
  MXMOE_TRY(check_tokens(what, a->T, a->N));
  if (a->num_adapters < 0 || a->num_adapters > kMaxAdapters)
    return fail(MOE_ERR_SHAPE, "%s: num_adapters = %d outside [0, %d]", what, a->num_adapters, kMaxAdapters);
  if (a->R < 8 || a->R > kMaxRank || a->R % 8)
    return fail(MOE_ERR_SHAPE, "%s: R = %d must be a multiple of 8 in [8, %d]", what, a->R, kMaxRank);
  const bool gate = a->epilogue != MOE_EPI_NONE;
  if (gate && a->epilogue != MOE_EPI_SWIGLU_SPLIT && a->epilogue != MOE_EPI_SWIGLU_INTERLEAVED)
    return fail(MOE_ERR_INVALID_ARG, "%s: bad epilogue %d", what, a->epilogue);
  if (gate && a->gate_act != MOE_GATE_SILU && a->gate_act != MOE_GATE_GELU)
    return fail(MOE_ERR_INVALID_ARG, "%s: bad gate_act %d", what, a->gate_act);
  if (gate && !a->w && a->T > 0) return fail(MOE_ERR_INVALID_ARG, "%s: a SWIGLU epilogue needs w", what);
  MXMOE_TRY(check_dtype16(what, a->dtype));
  MXMOE_TRY(check_dtype_or_fp32(what, "out_dtype", a->out_dtype, a->dtype));
  const int64_t T = a->T, K = a->K, N = a->N, n = a->num_adapters, R = a->R, n_out = gate ? N / 2 : N;
  MXMOE_TRY(check_stride(what, "x_stride", a->x_stride, K));
  MXMOE_TRY(check_stride(what, "out_stride", a->out_stride, n_out, gate ? 4 : 8));
  if (a->add) MXMOE_TRY(check_stride(what, "add_stride", a->add_stride, N));
  const size_t need = adapter_ws_bytes(a->T, a->K, a->N, a->R);
  if (T > 0) {
    if (!a->x || !a->out || (n > 0 && (!a->ids || !a->a || !a->b)))
      return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!a->workspace || a->workspace_bytes < need)
      return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", what, a->workspace_bytes, need);
    const void* words[] = {a->ids, a->scales, a->ranks};
    for (const void* p : words)
      if (reinterpret_cast<uintptr_t>(p) & 3)
        return fail(MOE_ERR_INVALID_ARG, "%s: ids, scales and ranks must be 4-byte aligned", what);
    const bool in_place = !gate && a->add == a->out && a->add_stride == a->out_stride;
    const Span out[] = {span("out", a->out, T, n_out, a->out_stride, a->out_dtype),
                        {"workspace", a->workspace, need}};
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
    float* const low = static_cast<float*>(a->workspace);
    MXMOE_TRY(a->dtype == MOE_FLOAT_BF16 ? launch_shrink<__bf16>(*a, low, s) : launch_shrink<_Float16>(*a, low, s));
    j.ids = a->ids, j.ranks = a->ranks;
    j.s = low, j.lb = a->b;
    j.num_adapters = a->num_adapters, j.R = a->R;
  }
  return launch_dense(j, static_cast<uint8_t*>(a->workspace) + adapter_gemm_offset(a->T, a->R), s);
}

}  // extern "C"
