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

// One instance per operand storage, epilogue and adapters that a caller uses.
#define MXMOE_DENSE_FORMS(LAUNCH)                                             \
  if (j.epi == kEpiGateGrad) LAUNCH(false, true, kEpiGateGrad, false);        \
  else if (j.ta) LAUNCH(true, true, kEpiPlain, false);                        \
  else if (j.tb) LAUNCH(false, true, kEpiPlain, false);                       \
  else if (j.epi == kEpiGate && j.ids) LAUNCH(false, false, kEpiGate, true);  \
  else if (j.epi == kEpiGate) LAUNCH(false, false, kEpiGate, false);          \
  else if (j.ids) LAUNCH(false, false, kEpiPlain, true);                      \
  else LAUNCH(false, false, kEpiPlain, false)

// Whole 256 x 256 tiles in full rounds of the CUs, the rest whole or in parts.
struct TilePlan {
  int64_t full, rest, parts;
};
TilePlan plan_tiles(const DenseJob& j, int cus) {
  TilePlan t;
  const int64_t n = tiles(j, 256, 256);
  t.full = n / cus * cus;
  t.rest = n - t.full;
  t.parts = 4 * t.rest <= cus ? 4 : 2 * t.rest <= cus ? 2 : 1;
  return t;
}

template <typename E>
moe_status launch_tiles(const DenseJob& j, hipStream_t s) {
  const TilePlan t = plan_tiles(j, num_cus() / 8 * 8);
  const dim3 grid((unsigned)(t.full + t.rest * t.parts)), block(256);
#define MXMOE_LAUNCH(TA, TB, EPI, LORA) \
  hipLaunchKernelGGL((tile_kernel<E, TA, TB, EPI, LORA>), grid, block, 0, s, j, (int)t.full, (int)t.rest, (int)t.parts)
  MXMOE_DENSE_FORMS(MXMOE_LAUNCH);
#undef MXMOE_LAUNCH
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

template <typename E>
moe_status launch_small(const DenseJob& j, hipStream_t s) {
  const dim3 grid((unsigned)tiles(j, 64, 64)), block(256);
  if (j.K >= 4096 && !j.tb) {   // long rows: stages of 64 k
#define MXMOE_LAUNCH(TA, TB, EPI, LORA) \
  hipLaunchKernelGGL((small_kernel<E, TA, TB, EPI, LORA, 64>), grid, block, 0, s, j)
    if (j.epi == kEpiGate && j.ids) MXMOE_LAUNCH(false, false, kEpiGate, true);
    else if (j.epi == kEpiGate) MXMOE_LAUNCH(false, false, kEpiGate, false);
    else if (j.ids) MXMOE_LAUNCH(false, false, kEpiPlain, true);
    else MXMOE_LAUNCH(false, false, kEpiPlain, false);
#undef MXMOE_LAUNCH
  } else {
#define MXMOE_LAUNCH(TA, TB, EPI, LORA) \
  hipLaunchKernelGGL((small_kernel<E, TA, TB, EPI, LORA, 32>), grid, block, 0, s, j)
    MXMOE_DENSE_FORMS(MXMOE_LAUNCH);
#undef MXMOE_LAUNCH
  }
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

template <typename E, int MB, int NB, bool DMA, int D>
moe_status launch_few(const DenseJob& j, hipStream_t s) {
  const dim3 grid((j.N + 16 * NB - 1) / (16 * NB)), block(64 * kFewWaves);
  if (j.epi == kEpiGate)
    hipLaunchKernelGGL((few_kernel<E, MB, NB, kEpiGate, DMA, D>), grid, block, 0, s, j);
  else
    hipLaunchKernelGGL((few_kernel<E, MB, NB, kEpiPlain, DMA, D>), grid, block, 0, s, j);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

// Whether 64 x 64 tiles are expected to take less time.  In microseconds per
// 32-deep stage, measured on a filled chip: 0.84 a round of whole 256 x 256
// tiles, 0.55 of halves, 0.28 of quarters; 0.22 a round of 64 x 64 tiles, two
// per CU, 0.11 of up to one per CU.  About 4 a round for its ends.
bool small_is_faster(const DenseJob& j) {
  const int cus = num_cus() / 8 * 8;
  const double stages = (j.K + 31) / 32;
  const TilePlan t = plan_tiles(j, cus);
  const double tail = t.rest == 0 ? 0.0 : t.parts == 4 ? stages * 0.28 + 4 : t.parts == 2 ? stages * 0.55 + 4
                                                                                         : stages * 0.84 + 4;
  const double big = (double)(t.full / cus) * (stages * 0.84 + 4) + tail;
  const int64_t n = tiles(j, 64, 64);
  const double small = n <= cus ? stages * 0.11 + 4 : (double)((n + 2 * cus - 1) / (2 * cus)) * (stages * 0.22 + 4);
  return small < big;
}

template <typename E>
moe_status launch_typed(const DenseJob& j, hipStream_t s) {
  // (the few-row kernel addresses a block's rows with 31 bits from the first;
  // a split gate's up rows lie I rows behind)
  const int64_t reach = j.epi == kEpiGate && !j.interleaved ? (int64_t)(j.N / 2 + 16) * j.ldb * 2 : 0;
  if (j.M <= 64 && j.epi != kEpiGateGrad && !j.ta && !j.tb && reach < (1ll << 30)) {
    const bool wide = (j.N + 15) / 16 > num_cus();
    // D: what the LDS holds (128 KB, for 16 rows 64 or 96)
    if (j.M <= 4) return launch_few<E, 1, 1, false, 4>(j, s);
    if (j.M <= 16) return wide ? launch_few<E, 1, 2, true, 2>(j, s) : launch_few<E, 1, 1, true, 2>(j, s);
    if (j.M <= 32) return wide ? launch_few<E, 2, 2, true, 2>(j, s) : launch_few<E, 2, 1, true, 2>(j, s);
    return wide ? launch_few<E, 4, 2, true, 1>(j, s) : launch_few<E, 4, 1, true, 1>(j, s);
  }
  // (a decode batch's mixed adapters are the small kernel's)
  if (j.ids && j.K == 0 && j.M > kFewTokens) {
    hipLaunchKernelGGL((adapters_only_kernel<E>), dim3((unsigned)tiles(j, 64, 128)), dim3(256), 0, s, j);
    MXMOE_HIP(hipGetLastError());
    return MOE_OK;
  }
  if ((j.ids && j.M <= kFewTokens) || small_is_faster(j)) return launch_small<E>(j, s);
  return launch_tiles<E>(j, s);
}

template <typename E>
moe_status launch_group_typed(const DenseJob* jobs, int n, hipStream_t s) {
  SmallGroup g{};
  int64_t at = 0;
  for (int i = 0; i < 3; ++i) {
    g.job[i] = jobs[i < n ? i : 0];
    g.start[i] = (int)at;
    g.tiles[i] = i < n ? (int)tiles(jobs[i], 64, 64) : 0;
    at += (g.tiles[i] + 7) / 8 * 8;
  }
  g.start[3] = (int)at;
  hipLaunchKernelGGL((small_group_kernel<E>), dim3((unsigned)at), dim3(256), 0, s, g);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

}  // namespace

moe_status launch_dense(const DenseJob& j, hipStream_t s) {
  if (j.M == 0) return MOE_OK;
  return j.dtype == MOE_FLOAT_BF16 ? launch_typed<__bf16>(j, s) : launch_typed<_Float16>(j, s);
}

moe_status launch_dense_group(const DenseJob* jobs, int n, hipStream_t s) {
  // one launch where each would run in 64 x 64 tiles that leave CUs idle
  int64_t blocks = 0;
  bool small = n > 1;
  for (int i = 0; i < n; ++i) {
    if (jobs[i].M == 0 || !small_is_faster(jobs[i])) small = false;
    else blocks += tiles(jobs[i], 64, 64);
  }
  if (small && blocks <= 8 * (int64_t)num_cus())
    return jobs[0].dtype == MOE_FLOAT_BF16 ? launch_group_typed<__bf16>(jobs, n, s)
                                           : launch_group_typed<_Float16>(jobs, n, s);
  for (int i = 0; i < n; ++i) MXMOE_TRY(launch_dense(jobs[i], s));
  return MOE_OK;
}

}  // namespace mxmoe
