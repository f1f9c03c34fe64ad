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

// The plan (and with it the scratch) is made for all CUs of an MI355X; a device
// that shows fewer takes more rounds.
constexpr int kCus = 256;

// How a product is cut: 64 x 64 tiles, or 256 x 256 tiles in full rounds of the
// CUs and the rest whole or in parts; K in one or several parts.
struct Plan {
  bool small;
  int splits;
  int64_t full, rest, parts;   // of 256 x 256 tiles
  int64_t blocks() const { return full + rest * parts; }
};

// Expected times in microseconds per 32-deep stage, measured on a filled chip:
// 0.84 a round of whole 256 x 256 tiles, 0.46 of halves, 0.25 of quarters; 0.20
// a round of 64 x 64 tiles, two per CU, 0.10 of up to one per CU.  About 4 a
// round for its ends.  A split of K costs a launch and the sums' way to memory
// and back, at 4 MB a microsecond.
Plan make_plan(const DenseJob& j) {
  const int cus = kCus;
  Plan best{};
  const int64_t n = tiles(j, 256, 256), n64 = tiles(j, 64, 64);
  best.full = n / cus * cus;
  best.rest = n - best.full;
  best.parts = 4 * best.rest <= cus ? 4 : 2 * best.rest <= cus ? 2 : 1;
  best.splits = 1;
  const Plan whole = best;
  double least = 1e30;
  // (a decode batch's mixed adapters are the small kernel's)
  const bool only_small = j.ids && j.M <= kFewTokens;
  for (int splits = 1; splits <= 8; splits *= 2) {
    const double stages = ((j.K + 63) / 64 + splits - 1) / splits * 2;
    if (splits > 1 && stages < 16) break;
    const double join = splits > 1 ? 4 + 2e-6 * splits * j.M * j.N : 0.0;
    if (!only_small && (splits == 1 || whole.full == 0)) {
      const double c = whole.parts == 4 ? 0.25 : whole.parts == 2 ? 0.46 : 0.84;
      const int64_t rest = whole.rest * whole.parts * splits;
      const double t = (double)(whole.full / cus) * (stages * 0.84 + 4) +
                       (double)((rest + cus - 1) / cus) * (stages * c + 4) + join;
      if (t < least) least = t, best = whole, best.splits = splits;
    }
    if (splits == 1 || n64 <= cus) {
      const int64_t b = n64 * splits;
      const double t = (b <= cus ? stages * 0.10 + 4 : (double)((b + 2 * cus - 1) / (2 * cus)) * (stages * 0.20 + 4)) + join;
      if (t < least) least = t, best = whole, best.small = true, best.splits = splits;
    }
  }
  return best;
}

template <typename E>
moe_status launch_tiles(const DenseJob& j, const Plan& t, float* partial, hipStream_t s) {
  const dim3 grid((unsigned)(t.blocks() * t.splits)), block(256);
#define MXMOE_LAUNCH(TA, TB, EPI, LORA)                                                                     \
  hipLaunchKernelGGL((tile_kernel<E, TA, TB, EPI, LORA>), grid, block, 0, s, j, (int)t.full, (int)t.rest,   \
                     (int)t.parts, partial, t.splits)
  MXMOE_DENSE_FORMS(MXMOE_LAUNCH);
#undef MXMOE_LAUNCH
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

template <typename E>
moe_status launch_small(const DenseJob& j, int splits, float* partial, hipStream_t s) {
  const int64_t n = tiles(j, 64, 64);
  const dim3 grid((unsigned)(splits > 1 ? (n + 7) / 8 * 8 * splits : n)), block(256);
  if (j.K >= 4096 && !j.tb) {   // long rows: stages of 64 k
#define MXMOE_LAUNCH(TA, TB, EPI, LORA) \
  hipLaunchKernelGGL((small_kernel<E, TA, TB, EPI, LORA, 64>), grid, block, 0, s, j, partial, splits)
    if (j.epi == kEpiGate && j.ids) MXMOE_LAUNCH(false, false, kEpiGate, true);
    else if (j.epi == kEpiGate) MXMOE_LAUNCH(false, false, kEpiGate, false);
    else if (j.ids) MXMOE_LAUNCH(false, false, kEpiPlain, true);
    else MXMOE_LAUNCH(false, false, kEpiPlain, false);
#undef MXMOE_LAUNCH
  } else {
#define MXMOE_LAUNCH(TA, TB, EPI, LORA) \
  hipLaunchKernelGGL((small_kernel<E, TA, TB, EPI, LORA, 32>), grid, block, 0, s, j, partial, splits)
    MXMOE_DENSE_FORMS(MXMOE_LAUNCH);
#undef MXMOE_LAUNCH
  }
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

template <typename E>
moe_status launch_join(const DenseJob& j, int splits, const float* partial, hipStream_t s) {
  const int64_t units = (int64_t)j.M * (j.epi == kEpiGate ? (j.N / 2 + 7) / 8 : j.N / 8);
  const dim3 grid((unsigned)((units + 255) / 256)), block(256);
  if (j.epi == kEpiGate) hipLaunchKernelGGL((join_kernel<E, kEpiGate>), grid, block, 0, s, j, partial, splits);
  else if (j.epi == kEpiGateGrad)
    hipLaunchKernelGGL((join_kernel<E, kEpiGateGrad>), grid, block, 0, s, j, partial, splits);
  else hipLaunchKernelGGL((join_kernel<E, kEpiPlain>), grid, block, 0, s, j, partial, splits);
  MXMOE_HIP(hipGetLastError());
  return MOE_OK;
}

// Few rows: 64 rows of 7168 x 7168 20.2 us, 23.1 in 64 x 64 tiles, of 4096 x 4096
// 10.2 and 13.7, of 2216 x 1544 5.9 and 8.7 (33 rows 18.2 and 21.4, 8.8 and 11.7,
// 5.8 and 8.1; the same weights each time, from the last-level cache); more rows
// would leave the LDS no room for a turn of 64 k.
// B's rows are contiguous, and a block's rows (16 or 32; of a split gate
// also their up rows, I rows behind) lie within 31 bits of the first.
bool takes_few(const DenseJob& j) {
  const int64_t reach = j.epi == kEpiGate && !j.interleaved ? (int64_t)(j.N / 2 + 16) * j.ldb * 2 : 0;
  return j.M <= 64 && j.epi != kEpiGateGrad && !j.ta && !j.tb && reach < (1ll << 30);
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

template <typename E>
moe_status launch_typed(const DenseJob& j, void* ws, hipStream_t s) {
  if (takes_few(j)) {
    const bool wide = (j.N + 15) / 16 > kCus;
    // turns ahead: what 128 KB of LDS hold
    if (j.M <= 4) return launch_few<E, 1, 1, false, 4>(j, s);
    if (j.M <= 16) return wide ? launch_few<E, 1, 2, true, 2>(j, s) : launch_few<E, 1, 1, true, 2>(j, s);
    if (j.M <= 32) return wide ? launch_few<E, 2, 2, true, 2>(j, s) : launch_few<E, 2, 1, true, 2>(j, s);
    return wide ? launch_few<E, 4, 2, true, 1>(j, s) : launch_few<E, 4, 1, true, 1>(j, s);
  }
  if (j.ids && j.K == 0 && j.M > kFewTokens) {
    hipLaunchKernelGGL((adapters_only_kernel<E>), dim3((unsigned)tiles(j, 64, 128)), dim3(256), 0, s, j);
    MXMOE_HIP(hipGetLastError());
    return MOE_OK;
  }
  const Plan t = make_plan(j);
  float* const partial = static_cast<float*>(ws);
  if (t.small) MXMOE_TRY(launch_small<E>(j, t.splits, partial, s));
  else MXMOE_TRY(launch_tiles<E>(j, t, partial, s));
  return t.splits > 1 ? launch_join<E>(j, t.splits, partial, s) : MOE_OK;
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

size_t dense_ws_bytes(const DenseJob& j) {
  if (j.M == 0 || j.K == 0) return 0;
  const int splits = make_plan(j).splits;
  return splits > 1 ? (size_t)splits * j.M * j.N * 4 : 0;
}

moe_status launch_dense(const DenseJob& j, void* ws, hipStream_t s) {
  if (j.M == 0) return MOE_OK;
  return j.dtype == MOE_FLOAT_BF16 ? launch_typed<__bf16>(j, ws, s) : launch_typed<_Float16>(j, ws, s);
}

moe_status launch_dense_group(const DenseJob* jobs, int n, void* ws, hipStream_t s) {
  // one launch where each would run in whole 64 x 64 tiles that leave CUs idle
  int64_t blocks = 0;
  bool small = n > 1;
  for (int i = 0; i < n; ++i) {
    const Plan t = make_plan(jobs[i]);
    if (jobs[i].M == 0 || !t.small || t.splits > 1) small = false;
    else blocks += tiles(jobs[i], 64, 64);
  }
  if (small && blocks <= 8 * kCus)
    return jobs[0].dtype == MOE_FLOAT_BF16 ? launch_group_typed<__bf16>(jobs, n, s)
                                           : launch_group_typed<_Float16>(jobs, n, s);
  for (int i = 0; i < n; ++i) MXMOE_TRY(launch_dense(jobs[i], ws, s));
  return MOE_OK;
}

}  // namespace mxmoe
