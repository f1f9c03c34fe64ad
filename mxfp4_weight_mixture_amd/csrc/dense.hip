// Dense products with 16-bit operands: choice of kernel and launch.
#include "dense_few.h"
#include "dense_small.h"
#include "dense_tile.h"

namespace mxmoe {
namespace {

int64_t tiles(const DenseJob& j, int bm, int bn) {
  const int cols = j.epi == kEpiGate ? bn / 2 : bn, width = j.epi == kEpiGate ? j.N / 2 : j.N;
  return (int64_t)((j.M + bm - 1) / bm) * ((width + cols - 1) / cols);
}

// One instance per operand storage and epilogue that a caller uses.
#define MXMOE_DENSE_FORMS(LAUNCH)                             \
  if (j.epi == kEpiGate) LAUNCH(false, false, kEpiGate);       \
  else if (j.epi == kEpiGateGrad) LAUNCH(false, true, kEpiGateGrad); \
  else if (j.ta) LAUNCH(true, true, kEpiPlain);               \
  else if (j.tb) LAUNCH(false, true, kEpiPlain);              \
  else LAUNCH(false, false, kEpiPlain)

template <typename E, int FM, int FN, int NST>
moe_status launch_tile_kernel(const DenseJob& j, hipStream_t s) {
  const dim3 grid((unsigned)tiles(j, 64 * FM, 64 * FN)), block(256);
#define MXMOE_LAUNCH(TA, TB, EPI) hipLaunchKernelGGL((dense_kernel<E, TA, TB, EPI, FM, FN, NST>), grid, block, 0, s, j)
  MXMOE_DENSE_FORMS(MXMOE_LAUNCH);
#undef MXMOE_LAUNCH
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

template <typename E, int NST>
moe_status launch_small(const DenseJob& j, hipStream_t s) {
  const dim3 grid((unsigned)tiles(j, 64, 64)), block(256);
#define MXMOE_LAUNCH(TA, TB, EPI) hipLaunchKernelGGL((small_kernel<E, TA, TB, EPI, NST>), grid, block, 0, s, j)
  MXMOE_DENSE_FORMS(MXMOE_LAUNCH);
#undef MXMOE_LAUNCH
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

template <typename E, int MB, int NB, bool XLDS, int D>
moe_status launch_few(const DenseJob& j, hipStream_t s) {
  const dim3 grid((j.N + 16 * NB - 1) / (16 * NB)), block(64 * kFewWaves);
  if (j.epi == kEpiGate)
    hipLaunchKernelGGL((few_kernel<E, MB, NB, kEpiGate, XLDS, D>), grid, block, 0, s, j);
  else
    hipLaunchKernelGGL((few_kernel<E, MB, NB, kEpiPlain, XLDS, D>), grid, block, 0, s, j);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

int choose_tile(const DenseJob& j) {
#ifdef FORCE_TILE
  return g_force;
#endif
  if (j.ids && j.M <= kFewTokens) return 0;
  if (tiles(j, 256, 256) >= 200) return 2;
  return tiles(j, 128, 128) >= 200 ? 1 : 0;
}

template <typename E>
moe_status launch_typed(const DenseJob& j, void* ws, hipStream_t s) {
  // (the few-row kernel addresses a block's rows with 31 bits from the first;
  // a split gate's up rows lie I rows behind)
  const int64_t reach = j.epi == kEpiGate ? (int64_t)(j.N / 2 + 16) * j.ldb * 2 : 0;
  if (j.M <= 64 && j.epi != kEpiGateGrad && !j.ta && !j.tb && reach < (1ll << 30)) {
    const bool wide = (j.N + 15) / 16 > num_cus();
    if (j.M <= 4) return launch_few<E, 1, 1, false, 4>(j, s);
    if (j.M <= 16) return wide ? launch_few<E, 1, 2, true, 4>(j, s) : launch_few<E, 1, 1, true, 4>(j, s);
    if (j.M <= 32) return wide ? launch_few<E, 2, 2, true, 4>(j, s) : launch_few<E, 2, 1, true, 4>(j, s);
    return wide ? launch_few<E, 4, 2, true, 2>(j, s) : launch_few<E, 4, 1, true, 2>(j, s);
  }
  if (tiles(j, 64, 64) > 0x7fffffff)
    return fail(MOE_ERR_SHAPE, "dense product: %d x %d is too large for one launch", j.M, j.N);
  switch (choose_tile(j)) {
    case 0: return launch_small<E, 4>(j, s);
    case 1: return launch_tile_kernel<E, 2, 2, 8>(j, s);
    default: return launch_tile_kernel<E, 4, 4, 4>(j, s);
  }
}

}  // namespace

size_t dense_ws_bytes(int M, int N, int K) { return 0; }

moe_status launch_dense(const DenseJob& j, void* ws, hipStream_t s) {
  if (j.M == 0) return MOE_OK;
  return j.dtype == MOE_FLOAT_BF16 ? launch_typed<__bf16>(j, ws, s) : launch_typed<_Float16>(j, ws, s);
}

}  // namespace mxmoe
