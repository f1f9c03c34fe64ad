// Dense products with 16-bit operands: what the gated feed-forward block
// (ffn.hip) and the many-adapter projection (adapter.hip) share.
#pragma once

#include "internal.h"

namespace mxmoe {

// One product C[m][n] = epilogue(sum_k A(m, k) B(n, k)), fp32 accumulation.
// An operand is stored [rows][K] (t == false) or [K][rows] (t == true).
enum DenseEpi { kEpiPlain = 0, kEpiGate = 1, kEpiGateGrad = 2 };

struct DenseJob {
  const void* a;            // M rows
  const void* b;            // N rows (for kEpiGate: the 2I gate and up rows)
  int64_t lda, ldb;         // elements
  int ta, tb;
  int M, N, K;
  int dtype;                // moe_float_dtype of a and b
  int epi;                  // DenseEpi
  int interleaved;          // gate / up order of w1's rows and gate_up's columns
  int act;                  // moe_gate_act
  const void* add;          // [M][N] of c_dtype or null: added to the sum before the epilogue
  int64_t ldadd;
  void* c;                  // plain: [M][N]; gate: h [M][N/2]; gate gradient: d_gate_up [M][2N], stride ldc
  int64_t ldc;
  int c_dtype;
  void* gu;                 // gate: gate_up [M][N] out or null; gate gradient: gate_up [M][2N] in (contiguous)
  int gu_dtype;
  void* h;                  // gate gradient: h [M][N] out, `dtype`, contiguous
  // adapters (null ids: none): += s[m] * lb[ids[m]][n], over R terms
  const int32_t* ids;
  const int32_t* ranks;
  const float* s;           // [M][R]
  const void* lb;           // [num_adapters][N][R]
  int num_adapters, R;
  // K split over blocks: where the block's part of the sums goes, fp32 [M][N]
  // (set by the kernels; null: the sums are whole)
  float* partial;
  // rows of A picked by index (grouped products; null: row m of a): row
  // gather[m] / gather_div of the gather_rows there are, zeros outside them
  const int32_t* gather;
  int gather_div, gather_rows;
};

// Token counts up to this are decode batches: their adapters differ from token
// to token.  (By size, not by what the ids hold: a row's result does not depend
// on its neighbours'.)  Measured on both sides, 4096 x 4096, 48 adapters of rank
// 16, as a decode batch / as a prompt, us: 256 mixed tokens 27 / 61, 256 in runs
// 28 / 34; 512 mixed 49 / 79, 512 in runs 47 / 47; 2048 in runs 173 / 80.  With
// 7 adapters of rank 64, 2216 x 1544: 256 mixed 36 / 52, 256 in runs 35 / 32, 512
// mixed 51 / 53, 512 in runs 49 / 42.  So mixed batches of 257 to 1024 tokens pay
// for the prompts of that size (257 mixed tokens of the first: 170, against 44).
constexpr int kFewTokens = 256;

// Scratch of a product: M, N, K, epi, ta, tb and whether there are ids decide.
size_t dense_ws_bytes(const DenseJob& j);
moe_status launch_dense(const DenseJob& j, void* ws, hipStream_t s);
// Up to three independent plain products of one type with B stored [K][N].
moe_status launch_dense_group(const DenseJob* jobs, int n, void* ws, hipStream_t s);
// The sizes of a product, for dense_ws_bytes.
inline DenseJob dense_sizes(int M, int N, int K, int epi, int ta, int tb) {
  DenseJob j{};
  j.M = M, j.N = N, j.K = K, j.epi = epi, j.ta = ta, j.tb = tb;
  return j;
}

// ---- argument checks shared by the entry points -------------------------
constexpr int kMaxWidth = 1 << 18;
constexpr int64_t kMaxStride = 1 << 21;   // 256 rows of it stay below 2^31 bytes
constexpr int kMaxTokens = 1 << 28;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline size_t float_bytes(int dtype) { return dtype == MOE_FLOAT_FP32 ? 4 : 2; }

// The bytes a [rows][cols] tensor with a row stride covers, from its start.
struct Span {
  const char* name;
  const void* p;
  size_t bytes;
};
inline Span span(const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride, int dtype) {
  return {name, p, p && rows > 0 ? (size_t)((rows - 1) * stride + cols) * float_bytes(dtype) : 0};
}
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// Every span 16-byte aligned; no output overlaps another span.
inline moe_status check_spans(const char* what, const Span* out, int n_out, const Span* in, int n_in) {
  for (int i = 0; i < n_out + n_in; ++i) {
    const Span& s = i < n_out ? out[i] : in[i - n_out];
    if (!aligned16(s.p)) return fail(MOE_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", what, s.name);
  }
  for (int i = 0; i < n_out; ++i) {
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(out[i], out[j]))
        return fail(MOE_ERR_INVALID_ARG, "%s: %s and %s overlap", what, out[i].name, out[j].name);
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j]))
        return fail(MOE_ERR_INVALID_ARG, "%s: %s overlaps %s", what, out[i].name, in[j].name);
  }
  return MOE_OK;
}
inline moe_status check_width(const char* what, const char* name, int v) {
  if (v < 8 || v > kMaxWidth || v % 8)
    return fail(MOE_ERR_SHAPE, "%s: %s = %d must be a multiple of 8 in [8, %d]", what, name, v, kMaxWidth);
  return MOE_OK;
}
// T rows of at most `cols` columns: a grid of 64 x 64 tiles stays below 2^24
// blocks (2^32 threads).
inline moe_status check_tokens(const char* what, int T, int64_t cols) {
  if (T < 0) return fail(MOE_ERR_SHAPE, "%s: T = %d < 0", what, T);
  if (T > kMaxTokens || ((int64_t)T + 63) / 64 * ((cols + 63) / 64) >= 1 << 24)
    return fail(MOE_ERR_SHAPE, "%s: T = %d rows of %lld are too many for one launch", what, T, (long long)cols);
  return MOE_OK;
}
inline moe_status check_stride(const char* what, const char* name, int64_t stride, int64_t cols, int of = 8) {
  if (stride < cols || stride > kMaxStride || stride % of)
    return fail(MOE_ERR_SHAPE, "%s: %s = %lld must be a multiple of %d in [%lld, %lld]", what, name,
                (long long)stride, of, (long long)cols, (long long)kMaxStride);
  return MOE_OK;
}
inline moe_status check_dtype16(const char* what, int dtype) {
  if (dtype != MOE_FLOAT_BF16 && dtype != MOE_FLOAT_FP16)
    return fail(MOE_ERR_INVALID_ARG, "%s: dtype %d must be MOE_FLOAT_BF16 or MOE_FLOAT_FP16", what, dtype);
  return MOE_OK;
}
inline moe_status check_dtype_or_fp32(const char* what, const char* name, int v, int dtype) {
  if (v != dtype && v != MOE_FLOAT_FP32)
    return fail(MOE_ERR_INVALID_ARG, "%s: %s %d must be dtype or MOE_FLOAT_FP32", what, name, v);
  return MOE_OK;
}

#ifdef __HIPCC__
// ---- device helpers -------------------------------------------------------
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));

template <typename E>
struct Vec;
template <>
struct Vec<__bf16> {
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  typedef __bf16 v8half __attribute__((ext_vector_type(8), aligned(8)));
  typedef __bf16 v4 __attribute__((ext_vector_type(4)));
};
template <>
struct Vec<_Float16> {
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  typedef _Float16 v8half __attribute__((ext_vector_type(8), aligned(8)));
  typedef _Float16 v4 __attribute__((ext_vector_type(4)));
};

__device__ __forceinline__ v16f mfma32(Vec<__bf16>::v8 a, Vec<__bf16>::v8 b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v16f mfma32(Vec<_Float16>::v8 a, Vec<_Float16>::v8 b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma16(Vec<__bf16>::v8 a, Vec<__bf16>::v8 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma16(Vec<_Float16>::v8 a, Vec<_Float16>::v8 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// sigmoid, exact at both ends: e^-z overflows to infinity and the reciprocal is 0.
// Hardware exp2 and reciprocal, 1 ulp each: off by (2 + |z|) 2^-23 of the result
// at most, against 2^-8 (bf16) or 2^-11 (fp16) when h is rounded
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// act(g) and act'(g).  The tanh GELU is g * sigmoid(2 p(g)) with
// p(g) = sqrt(2/pi) (g + 0.044715 g^3), since (1 + tanh p) / 2 = sigmoid(2p);
// the polynomial's argument is clamped where the sigmoid is 0 or 1 anyway, so
// that g^3 stays finite.
__device__ __forceinline__ float gate_act(int act, float g) {
  if (act == MOE_GATE_SILU) return g * sigmoid(g);
  const float c = fminf(fmaxf(g, -1e4f), 1e4f);
  return g * sigmoid(1.5957691216057308f * c * (1.0f + 0.044715f * c * c));
}
__device__ __forceinline__ void gate_act_grad(int act, float g, float* a, float* da) {
  if (act == MOE_GATE_SILU) {
    const float s = sigmoid(g);
    *a = g * s;
    *da = s * (1.0f + g * (1.0f - s));
  } else {
    const float c = fminf(fmaxf(g, -1e4f), 1e4f);
    const float s = sigmoid(1.5957691216057308f * c * (1.0f + 0.044715f * c * c));
    *a = g * s;
    *da = s + g * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * c * c);
  }
}

// An fp32 number as a sum of 16-bit ones, the largest first: bf16 three, which
// hold every bit of it, fp16 two, off by 2^-22 of it at most; fp16's range is
// the caller's to keep (row_scale below).  Each takes the leading bits of what
// is left, cut off: so none overflows and all have the number's sign.  A part
// with nothing left is the smallest number of that sign (2^-133, or 2^-24
// beside a row's 2^14) where the whole is not 0: a product with an infinity is
// then that infinity in every part, as it is for the whole.
template <typename E>
struct Parts;
template <>
struct Parts<__bf16> {
  static constexpr int N = 3;
  static __device__ __forceinline__ void split(const float (&x)[8], Vec<__bf16>::v8 (&o)[N]) {
    uint32_t w[N][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t t[N][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = fabsf(x[2 * j + i]), least = fminf(a, 0x1p-133f);
        t[0][i] = __float_as_uint(a) & 0xffff0000u;
        const float d = fmaxf(a - __uint_as_float(t[0][i]), least);   // (`least` behind an infinity)
        t[1][i] = __float_as_uint(d) & 0xffff0000u;
        t[2][i] = __float_as_uint(fmaxf(d - __uint_as_float(t[1][i]), least));
      }
      const uint32_t sign = high_halves(__float_as_uint(x[2 * j]), __float_as_uint(x[2 * j + 1])) & 0x80008000u;
#pragma unroll
      for (int k = 0; k < N; ++k) w[k][j] = high_halves(t[k][0], t[k][1]) | sign;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = __builtin_bit_cast(Vec<__bf16>::v8, w[k]);
  }
  static __device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
  }
};
template <>
struct Parts<_Float16> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void split(const float (&x)[8], Vec<_Float16>::v8 (&o)[N]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const auto top = __builtin_amdgcn_cvt_pkrtz(x[2 * j], x[2 * j + 1]);   // cut off
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = fabsf(x[2 * j + i]);
        const float rest = fmaxf(a - fabsf((float)top[i]), fminf(a, 0x1p-24f));
        o[0][2 * j + i] = (_Float16)top[i];
        o[1][2 * j + i] = (_Float16)copysignf(rest, x[2 * j + i]);
      }
    }
  }
};
// The power of two that brings values of up to `top` below 2^15, the largest
// above 2^14 (values below 2^-100 stay smaller), and its inverse.
__device__ __forceinline__ float row_scale(float top, float* inverse) {
  int e = (int)(__float_as_uint(top) >> 23) - 126;   // top < 2^e; infinity: 129
  e = min(max(e, -100), 128);
  *inverse = __uint_as_float((uint32_t)(112 + e) << 23);
  return __uint_as_float((uint32_t)(142 - e) << 23);
}

#endif

}  // namespace mxmoe
