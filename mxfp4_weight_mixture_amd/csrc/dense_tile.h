// The LDS-tiled dense kernel: one block of four waves per C tile.
//
// What bounds it is the matrix cores (32x32x16 MFMA, 32 clocks each on a
// SIMD) next to the LDS: a wave's 32 FM x 32 FN tile reads FM + FN fragments
// (1 KB each) per FM * FN products.  At 256 x 256 with four waves of 128 x 128
// that is 64 bytes a clock of the LDS's 128, beside 32 for the incoming tiles;
// eight waves of 128 x 64 would need 96 + 32 and are LDS-bound.  One wave per
// SIMD then holds 256 accumulators and hides latency by itself: fragments are
// read one 16-deep step ahead of their products.
//
// Tiles move global -> LDS without passing registers (buffer loads to LDS, 16
// bytes a lane) in stages of BK = 32 or 64 k, through a ring of NST buffers.  In
// stage s the block meets once, before its last 16-deep step: by then every
// wave has read all of stage s, so stage s + NST may overwrite it, and
// every wave's part of stage s + 1 has landed.
//
// Measured: 8192 x 7168 x 7168 in 0.64 to 0.66 ms (1.28 to 1.32 PFLOP/s, a library
// product 0.53 to 0.64), 0.72 to 0.75 with the gate; both operands of 4096 x 4096
// x 8192 stored [K][rows] in 0.22 ms (1.27).  The
// loop takes 1242 to 1366 clocks a stage of 1024 clocks' matrix work, 1065
// without its DMA; the clock is at 1.4 to 1.7 GHz then (power limit).
//
// LDS layout of a stage.  An operand stored [rows][K]: 64 or 128 bytes per row,
// its 16-byte chunks permuted by row (chunk ^ (row / 4) % 4, or ^ (row / 2) % 8),
// so that the 16 lanes that share a chunk cover all 64 banks.  An operand
// stored [K][rows] (the weights in the backward products, both operands of a
// weight gradient): BK k-rows of BM or BN values, read through the transposing LDS
// read, which hands lane i of 16 the column i of a 4 x 16 patch; 32-byte
// column groups are permuted by k (^ 2 (k % 4)), so that the 2 x 4 patches'
// rows that 32 lanes read together cover all 64 banks.
//
// Rows, columns and k past the end read as zeros: their lanes' offsets lie
// behind the buffer resource's range, so no memory is touched.
#pragma once

#include <type_traits>

#include "dense_dma.h"
#include "dense_rows.h"

namespace mxmoe {
namespace {

constexpr int kBK = 32;          // k per stage, unless a kernel says otherwise
constexpr int kTileLds = 144 << 10;

// Transposing LDS read: lane i of 16 gets column i of the 4 x 16 patch whose row
// r the lanes 4 r .. 4 r + 3 address, 8 bytes each.  `restrict` gives the read
// alias information; without any, the compiler takes it to depend on every
// LDS DMA in flight and drains them first.
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
__device__ __forceinline__ v4s read_tr(lds_v4s* __restrict__ a) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16(a); }

// Row of B behind tile columns [32 j, 32 j + 32) of n-tile nt: the first one's
// index among the plain (or the gate's, or the up) rows, and whether it is up.
__device__ __forceinline__ void b_block(const DenseJob& p, int nt, int bn, int j, int* first, int* up) {
  const bool gate = p.epi == kEpiGate;
  *first = gate ? nt * (bn >> 1) + (j >> 1) * 32 : nt * bn + 32 * j;
  *up = gate ? j & 1 : 0;
}

// One operand's way from memory to the products: DMA of a stage, fragment reads.
// ROWS: rows of the tile; T: stored [K][rows]; PARTS: waves that share a stage's loads.
// BK: k per stage, 32 or 64.
template <typename E, int ROWS, bool T, int PARTS, int BK = kBK>
struct Operand {
  static constexpr int BYTES = ROWS * BK * 2;             // of a stage
  static constexpr int CPR = T ? ROWS / 8 : BK / 8;       // 16-byte chunks per stored row
  static constexpr int LOADS = BYTES / 1024 / PARTS;      // DMA instructions per wave
  static_assert(LOADS >= 1, "at least 16 rows per wave");
  const char* base;      // of the tile's first row (or column), k = 0
  int64_t stage_step;    // bytes from stage to stage
  uint32_t off[LOADS];
  int64_t up_off;        // bytes from gate to up rows (gate epilogue, split order)
  uint32_t up_mask;      // loads that take up rows
  int kk;                // this lane's k within a stage (of its chunk, or its k-row of load 0)

  static __device__ __forceinline__ int swz(int row) { return BK == 32 ? (row >> 2) & 3 : (row >> 1) & 7; }
  static __device__ __forceinline__ int swz_t(int k) { return ((k & 3) * 2) & (ROWS / 16 - 1); }

  // rows [r0, r0 + ROWS) of an operand with `rows` rows
  __device__ __forceinline__ void init(const void* p, int64_t ld, int rows, int r0, int wave, int lane) {
    up_mask = 0;
    up_off = 0;
    if constexpr (!T) {
      base = static_cast<const char*>(p) + (int64_t)r0 * ld * 2;
      stage_step = BK * 2;
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const int r = (wave * LOADS + j) * (64 / CPR) + lane / CPR;
        const int c = (lane % CPR) ^ swz(r);
        if (j == 0) kk = c * 8;
        off[j] = r0 + r < rows ? (uint32_t)(r * ld * 2 + c * 16) : kOut;
      }
    } else {
      // ROWS * 2 bytes per k-row; a load covers 1024 bytes of them
      base = static_cast<const char*>(p) + (int64_t)r0 * 2;
      stage_step = (int64_t)BK * ld * 2;
      const int slot = lane % CPR;
      kk = (wave * LOADS) * (64 / CPR) + lane / CPR;
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const int k = (wave * LOADS + j) * (64 / CPR) + lane / CPR;
        const int c = slot ^ (swz_t(k) << 1);
        off[j] = r0 + c * 8 < rows ? (uint32_t)(k * ld * 2 + c * 16) : kOut;
      }
    }
  }
  // rows [r0, r0 + ROWS) of p.gather, whose rows of A all lie within 2^31 bytes
  __device__ __forceinline__ void init_gather(const DenseJob& p, int r0, int wave, int lane) {
    static_assert(!T, "rows are gathered where K is contiguous");
    up_mask = 0;
    up_off = 0;
    base = static_cast<const char*>(p.a);
    stage_step = BK * 2;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int r = (wave * LOADS + j) * (64 / CPR) + lane / CPR;
      const int c = (lane % CPR) ^ swz(r);
      if (j == 0) kk = c * 8;
      const int g = r0 + r < p.M ? p.gather[r0 + r] : -1, row = g / p.gather_div;
      off[j] = g >= 0 && row < p.gather_rows ? (uint32_t)(row * p.lda * 2 + c * 16) : kOut;
    }
  }
  // rows of B in gate / up blocks of 32
  __device__ __forceinline__ void init_gate(const DenseJob& p, int nt, int wave, int lane) {
    const int I = p.N >> 1, i0 = nt * (ROWS / 2);
    base = static_cast<const char*>(p.b) + (int64_t)i0 * p.ldb * 2 * (p.interleaved ? 2 : 1);
    stage_step = BK * 2;
    up_off = p.interleaved ? p.ldb * 2 : (int64_t)I * p.ldb * 2;
    up_mask = 0;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int first = (wave * LOADS + j) * (64 / CPR), r = first + lane / CPR;
      const int c = (lane % CPR) ^ swz(r);
      if (j == 0) kk = c * 8;
      const int i = (first >> 6) * 32 + (r & 31);         // 64-row groups: 32 gate rows, 32 up rows
      if (first & 32) up_mask |= 1u << j;
      off[j] = i0 + i < I ? (uint32_t)(i * p.ldb * 2 * (p.interleaved ? 2 : 1) + c * 16) : kOut;
    }
  }
  // load j of stage s into buf (this operand's part of the stage's buffer)
  __device__ __forceinline__ void issue(int j, int s, int K, int wave, char* buf) const {
    const char* b = base + s * stage_step + ((up_mask >> j) & 1 ? up_off : 0);
    int k = kk;
    if constexpr (T) k += j * (64 / CPR);
    else if (BK == 64 && (j & 1)) k ^= 32;                // swz(r) alternates by 8 rows
    const uint32_t o = k < K - s * BK ? off[j] : kOut;
    dma16(rsrc_at(b), o, buf + (wave * LOADS + j) * 1024);
  }
  // fragment of rows [r, r + 32), k [16 ks, 16 ks + 16)
  static __device__ __forceinline__ typename Vec<E>::v8 frag(const char* buf, int r, int ks, int lane) {
    typedef typename Vec<E>::v8 v8;
    if constexpr (!T) {
      const int row = r + (lane & 31), c = 2 * ks + (lane >> 5);
      return *reinterpret_cast<const v8*>(buf + row * (BK * 2) + ((c ^ swz(row)) << 4));
    } else {
      // 16-lane group q: columns 16 (q % 2), k half q / 2; lane i: k-row i / 4, columns 4 (i % 4)
      const int i = lane & 15, q = (lane >> 4) & 1, g = lane >> 5;
      const int k = 16 * ks + 8 * g + (i >> 2);           // second read: k + 4, same swizzle
      const int col32 = ((r >> 4) + q) ^ swz_t(k);
      const char* a = buf + k * (ROWS * 2) + col32 * 32 + (i & 3) * 8;
      const v4s lo = read_tr((lds_v4s*)a), hi = read_tr((lds_v4s*)(a + 4 * ROWS * 2));
      const v8s both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(v8, both);
    }
  }
};

// Consecutive blocks go round the 8 XCDs; each XCD takes one contiguous run of
// the work items.
__device__ __forceinline__ int xcd_run(int b, int blocks) {
  const int xcd = b & 7, per = blocks >> 3, more = blocks & 7;
  return xcd * per + min(xcd, more) + (b >> 3);
}
// C tile number t, of mt x nt: groups of kGroup m-tiles by all n, so that the
// tiles in work on an XCD at one time share operand rows in its L2.
constexpr int kGroup = 4;
__device__ __forceinline__ void tile_at(int t, int mt, int nt, int* m, int* n) {
  const int full = kGroup * nt, grp = t / full, in = t - grp * full;
  const int rows = min(kGroup, mt - grp * kGroup);
  *m = grp * kGroup + in % rows;
  *n = in / rows;
}

// The C tile of 64 FM rows from m0 and the nt-th 64 FN columns of B.
template <typename E, bool TA, bool TB, int EPI, bool LORA, int FM, int FN, int NST, int BK, bool GATHER = false>
__device__ __forceinline__ void dense_tile(const DenseJob& p, int m0, int nt, char* lds) {
  typedef typename Vec<E>::v8 v8;
  constexpr int BM = 64 * FM, BN = 64 * FN;
  using A = Operand<E, BM, TA, 4, BK>;
  using B = Operand<E, BN, TB, 4, BK>;
  constexpr int STAGE = A::BYTES + B::BYTES;
  constexpr int STAGING = 32 * FN * 32 * 4;               // a wave's 32 rows of fp32 sums
  static_assert(NST * STAGE <= kTileLds && 4 * STAGING <= kTileLds, "LDS of a tile");

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, g = lane >> 5;
  const int wm = (wave >> 1) * 32 * FM, wn = (wave & 1) * 32 * FN;
  const int width = EPI == kEpiGate ? p.N >> 1 : p.N;

  // this lane's rows' adapters, -1 for none
  int id[FM];
  if constexpr (LORA) {
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const int m = m0 + wm + fm * 32 + l32;
      id[fm] = m < p.M ? p.ids[m] : -1;
      if (id[fm] < 0 || id[fm] >= p.num_adapters) id[fm] = -1;
    }
  }
  A a;
  B b;
  if constexpr (GATHER) a.init_gather(p, m0, wave, lane);
  else a.init(p.a, p.lda, p.M, m0, wave, lane);
  if constexpr (EPI == kEpiGate) b.init_gate(p, nt, wave, lane);
  else b.init(p.b, p.ldb, p.N, nt * BN, wave, lane);
  const int K = p.K, nst = (K + BK - 1) / BK;
  constexpr int LOADS = A::LOADS + B::LOADS;
  constexpr int EARLY = LOADS * 16 / BK;   // of them, issued half a stage before the rest
  auto issue = [&](int j, int s) {
    char* buf = lds + __builtin_amdgcn_readfirstlane((uint32_t)s % NST * STAGE);
    if (j < A::LOADS) a.issue(j, s, K, wave, buf);
    else b.issue(j - A::LOADS, s, K, wave, buf + A::BYTES);
  };

  v16f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

  if (nst > 0) {
#pragma unroll
    for (int s = 0; s < NST; ++s)
#pragma unroll
      for (int j = 0; j < (s + 1 < NST ? LOADS : EARLY); ++j) issue(j, s);

    v8 fa[2][FM], fb[2][FN];
    // fragment r of step ks of stage s
    auto read = [&](int s, int ks, int r, v8 (&xa)[FM], v8 (&xb)[FN]) {
      const char* buf = lds + __builtin_amdgcn_readfirstlane((uint32_t)s % NST * STAGE);
      if (r < FN) xb[r] = B::frag(buf + A::BYTES, wn + r * 32, ks, lane);
      else xa[r - FN] = A::frag(buf, wm + (r - FN) * 32, ks, lane);
    };
    constexpr int NR = FM + FN, MF = FM * FN;
    constexpr int RP = (NR + MF - 1) / MF;      // reads after each product
    // the DMA of a stage is spread over a whole stage's products: issued in a
    // lump, it takes longer to accept (20 clocks per KB) than the products last
    auto spread = [&](int i, int n, int j0, int j1, int s) {
#pragma unroll
      for (int j = j0; j < j1; ++j)
        if ((j - j0) * n / (j1 - j0) == i) issue(j, s);
    };
    wait_vm<(NST - 2) * LOADS + EARLY>();
    block_barrier();
#pragma unroll
    for (int r = 0; r < NR; ++r) read(0, 0, r, fa[0], fb[0]);
    constexpr int KS = BK / 16;
    for (int s = 0; s < nst; ++s) {
#pragma unroll
      for (int i = 0; i < (KS - 1) * MF; ++i) {
        const int ks = i / MF, f = i % MF;
        acc[f % FM][f / FM] = mfma32(fb[ks & 1][f / FM], fa[ks & 1][f % FM], acc[f % FM][f / FM]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = RP * f; r < RP * f + RP; ++r)
          if (r < NR) read(s, ks + 1, r, fa[(ks + 1) & 1], fb[(ks + 1) & 1]);
        spread(i, (KS - 1) * MF, EARLY, LOADS, s + NST - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      // all of stage s is in this wave's registers; its part of stage s + 1 has landed
      wait_lgkm0();
      wait_vm<(NST - 2) * LOADS>();
      block_barrier();
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        acc[i % FM][i / FM] = mfma32(fb[1][i / FM], fa[1][i % FM], acc[i % FM][i / FM]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = RP * i; r < RP * i + RP; ++r)
          if (r < NR) read(s + 1, 0, r, fa[0], fb[0]);
        spread(i, MF, 0, EARLY, s + NST);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // the epilogue reuses the stages' LDS
    wait_vm<0>();
    block_barrier();
  }

  // each adapter present in the wave's rows in turn: its product goes to sums of
  // its own, which only that adapter's rows take up.  s enters in two or three
  // 16-bit parts (Parts), so that it is not rounded to one, and in fp16 times a
  // power of two of its row's own, which is taken out of the sums: any fp32
  // value of s counts, as it does in the kernels of few tokens.  Two or four
  // 16-deep steps are loaded together, and all rows where there are registers
  // for it (256 accumulators leave none: they would have to leave the matrix
  // cores' registers at once): the time is the loads' latency.
  if constexpr (LORA) {
    constexpr int HS = FM * FN == 4 ? 4 : 2, FB = FM * FN > 8 ? 1 : FM;   // steps, fragment rows together
    auto add_adapters = [&](auto F0) {
    constexpr int f0 = decltype(F0)::value;
    for (;;) {
      int cur = -1;
#pragma unroll
      for (int fm = f0; fm < f0 + FB; ++fm) {
        const uint64_t left = __ballot(id[fm] >= 0);
        if (cur < 0 && left) cur = __builtin_amdgcn_readlane(id[fm], __ffsll((unsigned long long)left) - 1);
      }
      if (cur < 0) break;
      bool mine[FB];
#pragma unroll
      for (int fm = f0; fm < f0 + FB; ++fm) {
        mine[fm - f0] = id[fm] == cur;
        if (mine[fm - f0]) id[fm] = -1;
      }
      int rank = p.R;
      if (p.ranks) rank = min(max(p.ranks[cur], 0), p.R);
      const float* const sp = p.s + (size_t)(m0 + wm + l32) * p.R;
      const E* const lb = static_cast<const E*>(p.lb) + (size_t)cur * p.N * p.R;
      for (int r = 0; r < rank; r += 16 * HS) {
        F8 sv[FB][HS];
        v8 bv[HS][FN];
#pragma unroll
        for (int h = 0; h < HS; ++h) {
          const int k = r + 16 * h + 8 * g;
#pragma unroll
          for (int fn = 0; fn < FN; ++fn) {
            int first, up;
            b_block(p, nt, BN, (wn >> 5) + fn, &first, &up);
            const int i = first + l32;
            const int row = EPI == kEpiGate ? (p.interleaved ? 2 * i + up : up * width + i) : i;
            bv[h][fn] = v8{};
            if (i < width && k < rank) bv[h][fn] = *reinterpret_cast<const v8*>(lb + (size_t)row * p.R + k);
          }
#pragma unroll
          for (int fm = f0; fm < f0 + FB; ++fm) {
            sv[fm - f0][h] = F8{};
            if (mine[fm - f0] && k < rank) sv[fm - f0][h] = load8<E>(sp + (size_t)fm * 32 * p.R, MOE_FLOAT_FP32, k);
          }
        }
        if (rank & 7) {   // what lies behind the rank does not count
#pragma unroll
          for (int h = 0; h < HS; ++h) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (r + 16 * h + 8 * g + e >= rank) {
#pragma unroll
                for (int fn = 0; fn < FN; ++fn) bv[h][fn][e] = (E)0.0f;
#pragma unroll
                for (int fm = f0; fm < f0 + FB; ++fm) sv[fm - f0][h].v[e] = 0.0f;
              }
          }
        }
#pragma unroll
        for (int fm = f0; fm < f0 + FB; ++fm) {
          if (!__ballot(mine[fm - f0])) continue;
          constexpr int NP = Parts<E>::N;
          float scale = 1.0f, unscale = 1.0f;
          if constexpr (std::is_same<E, _Float16>::value) {
            float top = 0.0f;
#pragma unroll
            for (int h = 0; h < HS; ++h)
#pragma unroll
              for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(sv[fm - f0][h].v[e]));
            top = fmaxf(top, __shfl_xor(top, 32));   // the row's other half
            scale = row_scale(top, &unscale);
          }
          v8 part[NP][HS];
#pragma unroll
          for (int h = 0; h < HS; ++h) {
            v8 x[NP];
            if constexpr (std::is_same<E, _Float16>::value) {
#pragma unroll
              for (int e = 0; e < 8; ++e) sv[fm - f0][h].v[e] *= scale;
            }
            Parts<E>::split(sv[fm - f0][h].v, x);
#pragma unroll
            for (int i = 0; i < NP; ++i) part[i][h] = x[i];
          }
#pragma unroll
          for (int fn = 0; fn < FN; ++fn) {
            v16f t;
#pragma unroll
            for (int q = 0; q < 16; ++q) t[q] = 0.0f;
#pragma unroll
            for (int h = 0; h < HS; ++h)
#pragma unroll
              for (int i = NP - 1; i >= 0; --i) t = mfma32(bv[h][fn], part[i][h], t);
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[fm][fn][q] += mine[fm - f0] ? t[q] * unscale : 0.0f;
          }
        }
      }
    }
    };
    add_adapters(std::integral_constant<int, 0>());
    if constexpr (FB < FM) {
      add_adapters(std::integral_constant<int, 1>());
      add_adapters(std::integral_constant<int, 2>());
      add_adapters(std::integral_constant<int, 3>());
    }
  }

  // ---- epilogue: 32 rows of the wave's tile at a time ----
  char* const st = lds + wave * STAGING;
  constexpr int PITCH = FN * 32 * 4;          // bytes of a staged row
  constexpr int CH = PITCH / 16;              // its 16-byte chunks
  auto finish_rows = [&](auto FMI) {
    constexpr int fm = decltype(FMI)::value;
    const int r0 = m0 + wm + fm * 32;
    if (r0 >= p.M) return;
    // the kept pre-activations of these rows, all loads in flight before anything
    // waits for them (group by group of rows they were most of the kernel's end:
    // 49152 x 2048 over K = 4096 1058 us, now 990)
    constexpr int GIT = EPI == kEpiGateGrad ? FN * 2 : 1;
    F8 kg[GIT], ku[GIT];
    if constexpr (EPI == kEpiGateGrad) {
      if (!p.partial) {
        auto load = [&](auto DT) {
#pragma unroll
          for (int it = 0; it < GIT; ++it) {
            const int row = r0 + it * (16 / FN) + lane / (4 * FN), n = nt * BN + wn + lane % (4 * FN) * 8;
            if (row < p.M && n < width)
              load_pair<E>(p.gu, decltype(DT)::value, (size_t)row * 2 * p.N, p.N, n, p.interleaved, &kg[it], &ku[it]);
          }
        };
        if (p.gu_dtype == MOE_FLOAT_FP32) load(std::integral_constant<int, MOE_FLOAT_FP32>());
        else load(std::integral_constant<int, MOE_FLOAT_BF16>());   // (type E)
      }
    }
    // stage: lane = row l32, four columns at a time, chunks permuted by row
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = fn * 8 + 2 * q + g;
        *reinterpret_cast<v4f*>(st + l32 * PITCH + ((c ^ (l32 & (CH - 1))) << 4)) =
            v4f{acc[fm][fn][4 * q], acc[fm][fn][4 * q + 1], acc[fm][fn][4 * q + 2], acc[fm][fn][4 * q + 3]};
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    auto staged8 = [&](int row, int c) {
      const v4f x = *reinterpret_cast<const v4f*>(st + row * PITCH + ((c ^ (row & (CH - 1))) << 4));
      const v4f y = *reinterpret_cast<const v4f*>(st + row * PITCH + (((c + 1) ^ (row & (CH - 1))) << 4));
      return F8{{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}};
    };
    if constexpr (EPI == kEpiGate) {
      constexpr int LPR = FN * 32 / 16;       // lanes per row: eight gate indices each
#pragma unroll
      for (int it = 0; it < 32 * LPR / 64; ++it) {
        const int row = it * (64 / LPR) + lane / LPR, x = lane % LPR;
        const int blk = x >> 2, c = blk * 16 + (x & 3) * 2;       // 64-column block: gate, then up
        const int i = nt * (BN / 2) + (wn >> 1) + blk * 32 + (x & 3) * 8;
        const F8 gt = staged8(row, c), up = staged8(row, c + 8);
        if (r0 + row < p.M && i < width) finish_gate<E>(p, r0 + row, i, gt, up);
      }
    } else {
      constexpr int LPR = FN * 32 / 8;
#pragma unroll
      for (int it = 0; it < 32 * LPR / 64; ++it) {
        const int row = it * (64 / LPR) + lane / LPR, x = lane % LPR;
        const int n = nt * BN + wn + x * 8;
        const F8 v = staged8(row, 2 * x);
        if (r0 + row < p.M && n < width) {
          if constexpr (EPI == kEpiPlain) finish_plain<E>(p, r0 + row, n, v);
          else if (p.partial) finish_gate_grad<E>(p, r0 + row, n, v);
          else finish_gate_grad<E>(p, r0 + row, n, v, kg[it], ku[it]);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  // (a loop this long would not be unrolled, and the sums would leave their registers)
  finish_rows(std::integral_constant<int, 0>());
  if constexpr (FM > 1) finish_rows(std::integral_constant<int, 1>());
  if constexpr (FM > 2) finish_rows(std::integral_constant<int, 2>());
  if constexpr (FM > 3) finish_rows(std::integral_constant<int, 3>());
}

// 256 x 256 tiles, of which the last (fewer than one per CU) may be split into
// 128 x 256 halves or 128 x 128 quarters: a part takes 0.55 or 0.3 of a whole
// tile's time.  Their stages are 64 deep: half the barriers, whole lines.
// `full` whole tiles, then `rest` tiles in `parts` blocks each; with few tiles
// (full == 0) K may be split as well.
template <typename E, bool TA, bool TB, int EPI, bool LORA>
__global__ __launch_bounds__(256, 1) void tile_kernel(DenseJob p, int full, int rest, int parts, float* partial,
                                                      int splits) {
  __shared__ __attribute__((aligned(1024))) char lds[kTileLds];
  const int cols = EPI == kEpiGate ? 128 : 256, width = EPI == kEpiGate ? p.N >> 1 : p.N;
  const int mts = (p.M + 255) >> 8, nts = (width + cols - 1) / cols;
  const int b = blockIdx.x;
  int mt, nt;
  if (b < full) {
    tile_at(xcd_run(b, full), mts, nts, &mt, &nt);
    dense_tile<E, TA, TB, EPI, LORA, 4, 4, 4, 32>(p, mt * 256, nt, lds);
    return;
  }
  int block = b - full;
  if (splits > 1) {
    const int blocks = rest * parts;
    take_part(p, partial, block / blocks, splits);
    block %= blocks;
  }
  const int u = xcd_run(block, rest * parts), part = u % parts;
  tile_at(full + u / parts, mts, nts, &mt, &nt);
  if (parts == 1) {
    dense_tile<E, TA, TB, EPI, LORA, 4, 4, 4, 32>(p, mt * 256, nt, lds);
  } else if (parts == 2) {
    if (mt * 256 + part * 128 < p.M) dense_tile<E, TA, TB, EPI, LORA, 2, 4, 3, 64>(p, mt * 256 + part * 128, nt, lds);
  } else if (mt * 256 + (part & 1) * 128 < p.M && (2 * nt + (part >> 1)) * (cols / 2) < width) {
    dense_tile<E, TA, TB, EPI, LORA, 2, 2, 4, 64>(p, mt * 256 + (part & 1) * 128, 2 * nt + (part >> 1), lds);
  }
}

// The adapters' part alone (no shared projection): bound by reading `add` and
// writing C, so small tiles, several blocks per CU.
template <typename E>
__global__ __launch_bounds__(256, 3) void adapters_only_kernel(DenseJob p) {
  __shared__ __attribute__((aligned(1024))) char lds[32 << 10];
  int mt, nt;
  const int mts = (p.M + 63) >> 6, nts = (p.N + 127) >> 7;
  tile_at(xcd_run(blockIdx.x, gridDim.x), mts, nts, &mt, &nt);
  dense_tile<E, false, false, kEpiPlain, true, 1, 2, 2, 32>(p, mt * 64, nt, lds);
}

}  // namespace
}  // namespace mxmoe
