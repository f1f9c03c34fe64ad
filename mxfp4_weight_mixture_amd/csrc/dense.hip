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

template <typename E, int MB>
moe_status launch_few(const DenseJob& j, hipStream_t s) {
  const dim3 block(64 * kFewWaves);
  if (j.epi == kEpiGate)
    hipLaunchKernelGGL((few_kernel<E, MB, kEpiGate>), dim3(j.N / 16), block, 0, s, j);
  else
    hipLaunchKernelGGL((few_kernel<E, MB, kEpiPlain>), dim3((j.N + 15) / 16), block, 0, s, j);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

template <typename E>
moe_status launch_typed(const DenseJob& j, void* ws, hipStream_t s) {
  if (j.M <= 64 && j.epi != kEpiGateGrad && !j.ta && !j.tb) {
    if (j.M <= 16) return launch_few<E, 1>(j, s);
    return j.M <= 32 ? launch_few<E, 2>(j, s) : launch_few<E, 4>(j, s);
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
