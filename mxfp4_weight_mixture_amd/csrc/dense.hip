// Dense products with 16-bit operands: choice of kernel and launch.
#include "dense_few.h"
#include "dense_tile.h"

namespace mxmoe {
namespace {

template <typename E, int FM, int FN>
moe_status launch_tile_kernel(const DenseJob& j, hipStream_t s) {
  const int BM = 64 * FM, BN = 64 * FN;
  const int cols = j.epi == kEpiGate ? BN / 2 : BN, width = j.epi == kEpiGate ? j.N / 2 : j.N;
  const int64_t blocks = (int64_t)((j.M + BM - 1) / BM) * ((width + cols - 1) / cols);
  if (blocks > 0x7fffffff) return fail(MOE_ERR_SHAPE, "dense product: %lld tiles", (long long)blocks);
  const dim3 grid((unsigned)blocks), block(256);
  if (j.epi == kEpiGate)
    hipLaunchKernelGGL((dense_kernel<E, false, false, kEpiGate, FM, FN>), grid, block, 0, s, j);
  else if (j.epi == kEpiGateGrad)
    hipLaunchKernelGGL((dense_kernel<E, false, true, kEpiGateGrad, FM, FN>), grid, block, 0, s, j);
  else if (j.ta)
    hipLaunchKernelGGL((dense_kernel<E, true, true, kEpiPlain, FM, FN>), grid, block, 0, s, j);
  else if (j.tb)
    hipLaunchKernelGGL((dense_kernel<E, false, true, kEpiPlain, FM, FN>), grid, block, 0, s, j);
  else
    hipLaunchKernelGGL((dense_kernel<E, false, false, kEpiPlain, FM, FN>), grid, block, 0, s, j);
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
  const int64_t big = (int64_t)((j.M + 255) / 256) * ((j.N + 255) / 256);
  if (big >= 200) return launch_tile_kernel<E, 4, 4>(j, s);
  return launch_tile_kernel<E, 2, 2>(j, s);
}

}  // namespace

size_t dense_ws_bytes(int M, int N, int K) { return 0; }

moe_status launch_dense(const DenseJob& j, void* ws, hipStream_t s) {
  if (j.M == 0) return MOE_OK;
  return j.dtype == MOE_FLOAT_BF16 ? launch_typed<__bf16>(j, ws, s) : launch_typed<_Float16>(j, ws, s);
}

}  // namespace mxmoe
