// Low-rank adapters of many requests beside one shared projection.
//
//   y[t] = (add[t] +) x[t] W^T + s[t] B[a]^T,  s[t] = scales[a] x[t] A[a]^T,
//   a = ids[t] (none outside [0, num_adapters))
// Up to kFewTokens tokens are taken for a decode batch (adapters mixed at
// will), more for prompts (adapters in runs); either way any order is right.
// Two launches: the first gives s [T][R] in fp32, the second the shared
// projection with s B^T added to its fp32 sums and the epilogue.
#include "dense_dma.h"

namespace mxmoe {
namespace {

// s of few tokens: one wave per (token, row of A), 64 lanes along K.  Tokens of
// a decode batch have adapters of their own, so there is nothing to share.
template <typename E>
__global__ __launch_bounds__(256) void shrink_token_kernel(moe_adapter_args p, float* s) {
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
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += (float)xv[i] * (float)av[i];
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) s[(size_t)t * p.R + r] = p.scales ? sum * p.scales[id] : sum;
}

// s of many tokens, whose requests come in runs: a block takes 16 TB tokens
// and, for each adapter among them (one, mostly), 16 RB rows of A at a time.
// Bound by reading x; eight waves split K in turns of 64 and add their sums up
// through the LDS.  16x16x32 MFMA, A's rows first, so that a lane's sums are
// one token's; loads run two turns ahead, past the end they read zeros.
template <typename E, int TB, int RB>
__global__ __launch_bounds__(512) void shrink_runs_kernel(moe_adapter_args p, float* s) {
  typedef typename Vec<E>::v8 v8;
  constexpr int WAVES = 8, D = 2;
  __shared__ __attribute__((aligned(16))) v4f part[WAVES][RB * TB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, kl = 8 * (lane >> 4), t0 = blockIdx.x * 16 * TB;
  const int K = p.K, turns = (((K + 63) >> 6) - wave + WAVES - 1) / WAVES;
  const char* const xbase = static_cast<const char*>(p.x) + (int64_t)t0 * p.x_stride * 2;
  uint32_t xoff[TB];
#pragma unroll
  for (int i = 0; i < TB; ++i)
    xoff[i] = (uint32_t)((min(t0 + 16 * i + l16, p.T - 1) - t0) * (p.x_stride * 2)) + kl * 2;
  const int mine = t0 + (lane & (16 * TB - 1)) < p.T ? p.ids[t0 + (lane & (16 * TB - 1))] : -1;
  uint64_t left = __ballot(lane < 16 * TB && mine >= 0 && mine < p.num_adapters);
  while (left) {
    const int cur = __builtin_amdgcn_readlane(mine, __ffsll((unsigned long long)left) - 1);
    left &= ~__ballot(mine == cur);
    int rank = p.R;
    if (p.ranks) rank = min(max(p.ranks[cur], 0), p.R);
    const float scale = p.scales ? p.scales[cur] : 1.0f;
    for (int r0 = 0; r0 < rank; r0 += 16 * RB) {
      const char* const abase = static_cast<const char*>(p.a) + ((int64_t)cur * p.R + r0) * K * 2;
      uint32_t aoff[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i)
        aoff[i] = r0 + 16 * i + l16 < rank ? (uint32_t)((16 * i + l16) * (K * 2) + kl * 2) : kOut;
      v8 a[D][2][RB], x[D][2][TB];
      auto load = [&](int t, int u) {
        const int k = (wave + t * WAVES) * 64;
        const auto ra = rsrc_at(abase + (int64_t)k * 2), rx = rsrc_at(xbase + (int64_t)k * 2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = k + 32 * h + kl < K;
#pragma unroll
          for (int i = 0; i < TB; ++i) x[u][h][i] = load16<E>(rx, in ? xoff[i] + 64 * h : kOut);
#pragma unroll
          for (int i = 0; i < RB; ++i) a[u][h][i] = load16<E>(ra, in && aoff[i] != kOut ? aoff[i] + 64 * h : kOut);
        }
      };
      v4f acc[RB][TB];
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < D; ++u) load(u, u);
      for (int tt = 0; tt < turns; tt += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
              for (int j = 0; j < TB; ++j) acc[i][j] = mfma16(a[u][h][i], x[u][h][j], acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
          load(tt + D + u, u);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) part[wave][i * TB + j][lane] = acc[i][j];
      __syncthreads();
      // accumulator q of lane l: token l % 16, row 4 (l / 16) + q
      for (int e = threadIdx.x; e < RB * TB * 64; e += 512) {
        const int f = e >> 6, l = e & 63;
        const int t = t0 + f % TB * 16 + (l & 15), r = r0 + f / TB * 16 + 4 * (l >> 4);
        if (t < p.T && r < p.R && p.ids[t] == cur) {
          v4f v = part[0][f][l];
#pragma unroll
          for (int w = 1; w < WAVES; ++w) v += part[w][f][l];
          *reinterpret_cast<v4f*>(s + (size_t)t * p.R + r) = v * scale;
        }
      }
      __syncthreads();
    }
  }
}

template <typename E, int RB>
void launch_runs(const moe_adapter_args& a, float* s, hipStream_t st) {
  // 32 tokens a block read A half as often, where that leaves enough blocks
  if ((a.T + 31) / 32 >= num_cus() / 2)
    hipLaunchKernelGGL((shrink_runs_kernel<E, 2, RB>), dim3((a.T + 31) / 32), dim3(512), 0, st, a, s);
  else
    hipLaunchKernelGGL((shrink_runs_kernel<E, 1, RB>), dim3((a.T + 15) / 16), dim3(512), 0, st, a, s);
}

template <typename E>
moe_status launch_shrink(const moe_adapter_args& a, float* s, hipStream_t st) {
  if (a.T <= kFewTokens) {
    const dim3 grid((unsigned)((a.T * a.R + 3) / 4));
    hipLaunchKernelGGL((shrink_token_kernel<E>), grid, dim3(256), 0, st, a, s);
  } else if (a.R <= 16) {
    launch_runs<E, 1>(a, s, st);
  } else if (a.R <= 32) {
    launch_runs<E, 2>(a, s, st);
  } else {
    launch_runs<E, 4>(a, s, st);
  }
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
    float* const low = reinterpret_cast<float*>(ws + w.s);
    MXMOE_TRY(a->dtype == MOE_FLOAT_BF16 ? launch_shrink<__bf16>(*a, low, s) : launch_shrink<_Float16>(*a, low, s));
    j.ids = a->ids, j.ranks = a->ranks;
    j.s = low, j.lb = a->b;
    j.num_adapters = a->num_adapters, j.R = a->R;
  }
  return launch_dense(j, ws + w.gemm, s);
}

}  // extern "C"
