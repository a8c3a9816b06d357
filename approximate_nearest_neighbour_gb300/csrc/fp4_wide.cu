// The wide product of packed 4-bit rows (fp4_product.cu has the narrow one and
// the entry points): many rows on both sides.
//
// Persistent CTAs, one per SM, of 128 columns of out (rows of b) x T rows of
// out, T = 128 or 256. A cluster of CN x CM CTAs covers CN column tiles and CM
// row tiles: each CTA loads 1/CM of its 128 rows of b and 1/CN of its T rows
// of a and multicasts them to the CTAs that share them, so that L2 is read
// once per cluster and not once per CTA.
//
// 10 warps: warp 0 loads, warp 1 copies scales to TMEM and issues products,
// warps 2..9 store (two per TMEM lane group, half of the columns each). While
// a tile is stored the next one is computed: with T = 256 the two accumulators
// overlap (columns 0..255 and 160..415), so the storing warps first empty the
// 96 shared columns and release them. TMEM columns 416..511 hold two buffers
// of scales, each reused when the products two stages back have finished.
#include <algorithm>

#include "fp4_mma.cuh"

namespace ivfpq {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kSfBase = 416;  // first TMEM column of the scales

template <int FMT, int T>
struct WideCfg {
  static constexpr int kTiles = FMT == IVFPQ_MXFP4 ? 2 : 4;  // scale tiles per stage and 128 rows
  static constexpr int kRt = T / 128;
  static constexpr int kSfTile = kTiles * 512;
  static constexpr int kB = BN * KB;
  static constexpr int kA = T * KB;
  static constexpr int kStage = kB + kA + (1 + kRt) * kSfTile;
  static constexpr int kStages = T == 256 ? 4 : 6;
  static constexpr int kTotal = kStages * kStage + 512 + 1024;
  static constexpr int kSfCols = 4 * kTiles * (1 + kRt);  // TMEM columns of one scale buffer
  static constexpr int kAcc1 = T == 256 ? 160 : T;        // first column of the second accumulator
  static_assert(kSfBase + 2 * kSfCols <= 512 && kAcc1 + T <= kSfBase, "TMEM columns");
  static_assert(kTotal <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void tma_load_2d_mc(uint32_t dst, const CUtensorMap* map, int x, int y,
                                               uint32_t bar, uint16_t mask) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".multicast::cluster [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "h"(mask)
      : "memory");
}
__device__ __forceinline__ void bulk_load_mc(uint32_t dst, const void* src, uint32_t bytes,
                                             uint32_t bar, uint16_t mask) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.multicast::cluster"
      " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "h"(mask)
      : "memory");
}
__device__ __forceinline__ void mma_commit_mc(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 16 accumulator columns (rows r0 .. r0 + 15 of out) of this lane's column.
template <class O>
__device__ __forceinline__ void store16(O* out, int64_t ldo, int64_t r0, int64_t m, bool live,
                                        const uint32_t (&r)[16], float alpha) {
  O* p = out + r0 * ldo;
  if (live) {
    if (r0 + 16 <= m) {
#pragma unroll
      for (int j = 0; j < 16; ++j, p += ldo) *p = from_f32<O>(__uint_as_float(r[j]) * alpha);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j, p += ldo)
        if (r0 + j < m) *p = from_f32<O>(__uint_as_float(r[j]) * alpha);
    }
  }
}

struct Tiling {
  int cl_n, cl_m;   // cluster tiles along n and m
  int m_fast;       // consecutive cluster tiles go along m
};

template <int FMT, int T, int CN, int CM, class O>
__global__ void __launch_bounds__(kThreads, 1)
fp4_wide_kernel(const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_a, const ProdArgs p, const Tiling tl) {
  using C = WideCfg<FMT, T>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t fp4_wide_smem[];
  const uint32_t raw = smem_u32(fp4_wide_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = fp4_wide_smem + (base - raw);
  auto s_b = [&](int s) { return base + s * (C::kB + C::kA); };
  auto s_a = [&](int s) { return base + s * (C::kB + C::kA) + C::kB; };
  const uint32_t sf0 = base + NS * (C::kB + C::kA);
  auto s_sf = [&](int s) { return sf0 + s * (1 + C::kRt) * C::kSfTile; };  // b's, then a's
  const uint32_t bars = base + NS * C::kStage;
  auto bar_full = [&](int s) { return bars + 8 * s; };
  auto bar_empty = [&](int s) { return bars + 8 * (NS + s); };
  auto bar_sf = [&](int b) { return bars + 16 * NS + 8 * b; };
  const uint32_t bar_acc = bars + 16 * NS + 16;
  const uint32_t bar_free = bars + 16 * NS + 24;
  const uint32_t bar_end = bars + 16 * NS + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 16 * NS + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (bars - base) + 16 * NS + 48);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CN * CM > 1 ? int(cluster_rank()) : 0;
  const int rn = rank % CN, rm = rank / CN;
  const int cluster = blockIdx.x / (CN * CM), nclusters = gridDim.x / (CN * CM);
  const int ntiles = tl.cl_n * tl.cl_m;
  const int nk = (p.kp + KE - 1) / KE;
  // first column and row of this CTA's part of cluster tile t
  auto col0 = [&](int t) { return ((tl.m_fast ? t / tl.cl_m : t % tl.cl_n) * CN + rn) * BN; };
  auto row0 = [&](int t) {
    return int64_t((tl.m_fast ? t % tl.cl_m : t / tl.cl_n) * CM + rm) * T;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), CN + CM - 1);
    }
    mbar_init(bar_sf(0), 1);
    mbar_init(bar_sf(1), 1);
    mbar_init(bar_acc, 1);
    mbar_init(bar_free, kEpiWarps);
    mbar_init(bar_end, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CN * CM > 1) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto fail = [&]() {
    atomicExch(p.err, 1);
    *abort_flag = 1;
  };

  if (warp == 0 && lane == 0) {
    // ---- loads. b's rows go to the CTAs of the same column tile (rank rn + CN *
    // any), a's rows to those of the same row tile ----
    uint16_t mask_b = 0, mask_a = 0;
    for (int i = 0; i < CM; ++i) mask_b |= uint16_t(1u << (rn + CN * i));
    for (int i = 0; i < CN; ++i) mask_a |= uint16_t(1u << (i + CN * rm));
    const int last_nt = int((p.n - 1) / BN), last_mt = int((p.m - 1) / 128);
    int it = 0;
    for (int t = cluster; t < ntiles && !*abort_flag; t += nclusters) {
      const int n0 = col0(t);
      const int64_t m0 = row0(t);
      // a scale copy has no bounds of its own: past the end, any tile will do
      const uint8_t* sb = p.b_scales + int64_t(min(n0 / BN, last_nt)) * p.ntile * 512;
      const uint8_t* sa[C::kRt];
      for (int r = 0; r < C::kRt; ++r)
        sa[r] = p.a_scales + int64_t(min(int(m0 / 128) + r, last_mt)) * p.ntile * 512;
      for (int kc = 0; kc < nk; ++kc, ++it) {
        const int s = it % NS;
        if (!mbar_wait(bar_empty(s), ((it / NS) & 1) ^ 1)) {
          fail();
          break;
        }
        const int t0 = kc * C::kTiles;
        const uint32_t sfb = uint32_t(min(C::kTiles, p.ntile - t0)) * 512;
        mbar_expect_tx(bar_full(s), C::kB + C::kA + (1 + C::kRt) * sfb);
        if constexpr (CN * CM == 1) {
          tma_load_2d(s_b(s), &map_b, kc * KB, n0, bar_full(s));
          tma_load_2d(s_a(s), &map_a, kc * KB, int(m0), bar_full(s));
          bulk_load(s_sf(s), sb + int64_t(t0) * 512, sfb, bar_full(s));
          for (int r = 0; r < C::kRt; ++r)
            bulk_load(s_sf(s) + (1 + r) * C::kSfTile, sa[r] + int64_t(t0) * 512, sfb, bar_full(s));
        } else {
          constexpr int RB = BN / CM, RA = T / CN;
          tma_load_2d_mc(s_b(s) + rm * RB * KB, &map_b, kc * KB, n0 + rm * RB, bar_full(s), mask_b);
          tma_load_2d_mc(s_a(s) + rn * RA * KB, &map_a, kc * KB, int(m0) + rn * RA, bar_full(s),
                         mask_a);
          if (rm == 0) bulk_load_mc(s_sf(s), sb + int64_t(t0) * 512, sfb, bar_full(s), mask_b);
          for (int r = 0; r < C::kRt; ++r)
            if (rn == r % CN)
              bulk_load_mc(s_sf(s) + (1 + r) * C::kSfTile, sa[r] + int64_t(t0) * 512, sfb,
                           bar_full(s), mask_a);
        }
      }
    }
    // every stage released by all CTAs it went to: nothing of this CTA's copies
    // or of the others' releases is in flight when it ends
    for (int j = max(0, it - NS); j < it; ++j) mbar_wait(bar_empty(j % NS), (j / NS) & 1);
  } else if (warp == 1 && lane == 0) {
    // ---- scales and products ----
    uint16_t mask = 0;  // the CTAs that load for this one
    for (int i = 0; i < CM; ++i) mask |= uint16_t(1u << (rn + CN * i));
    for (int i = 0; i < CN; ++i) mask |= uint16_t(1u << (i + CN * rm));
    int it = 0, i = 0;
    bool ok = true;
    for (int t = cluster; t < ntiles && ok && !*abort_flag; t += nclusters, ++i) {
      if (i > 0 && !mbar_wait(bar_free, (i - 1) & 1)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + ((i & 1) ? C::kAcc1 : 0);
      for (int kc = 0; kc < nk; ++kc, ++it) {
        const int s = it % NS;
        if (!mbar_wait(bar_full(s), (it / NS) & 1) ||
            (it >= 2 && !mbar_wait(bar_sf(it & 1), ((it >> 1) - 1) & 1))) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const int tiles = min(C::kTiles, p.ntile - kc * C::kTiles);
        const uint32_t tb = tmem + kSfBase + (it & 1) * C::kSfCols;
        const uint32_t ta = tb + 4 * C::kTiles;
        for (int q = 0; q < tiles; ++q) {
          scale_copy(tb + 4 * q, scale_desc(s_sf(s) + 512 * q));
#pragma unroll
          for (int r = 0; r < C::kRt; ++r)
            scale_copy(ta + 4 * (q * C::kRt + r),
                       scale_desc(s_sf(s) + (1 + r) * C::kSfTile + 512 * q));
        }
        const uint64_t db = smem_desc(s_b(s)), da = smem_desc(s_a(s));
        const int steps = min(4, (p.kp - kc * KE + 63) / 64);
        for (int j = 0; j < steps; ++j) {
          const uint64_t adv = uint64_t(j * 32) >> 4;
          const int q = FMT == IVFPQ_MXFP4 ? j >> 1 : j;
          const uint32_t id = FMT == IVFPQ_MXFP4 ? uint32_t(j & 1) * 2 : 0u;
          mma_fp4<FMT>(acc, db + adv, da + adv, fp4_idesc<FMT, T>(id), tb + 4 * q,
                       ta + 4 * C::kRt * q, kc > 0 || j > 0);
        }
        mma_commit(bar_sf(it & 1));
        if constexpr (CN * CM == 1)
          mma_commit(bar_empty(s));
        else
          mma_commit_mc(bar_empty(s), mask);
      }
      if (ok) mma_commit(bar_acc);
    }
    // all products issued have finished before TMEM is freed
    mma_commit(bar_end);
    mbar_wait(bar_end, 0);
  } else if (warp >= 2) {
    // ---- store: warp w reads TMEM lanes 32 * (w % 4) .. +32 ----
    const int lg = warp & 3, half = (warp - 2) >> 2;
    const float alpha = (p.a_ts ? __ldg(p.a_ts) : 1.f) * (p.b_ts ? __ldg(p.b_ts) : 1.f);
    constexpr int kCrit = T == 256 ? 96 : 0;  // columns the next accumulator shares
    constexpr int C1 = kCrit / 2, C2 = (T - kCrit) / 2;
    int i = 0;
    for (int t = cluster; t < ntiles && !*abort_flag; t += nclusters, ++i) {
      if (!mbar_wait(bar_acc, i & 1)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t acc =
          tmem + (uint32_t(32 * lg) << 16) + uint32_t((i & 1) ? C::kAcc1 : 0);
      const int64_t col = col0(t) + 32 * lg + lane, m0 = row0(t);
      const bool live = col < p.n;
      O* out = static_cast<O*>(p.out) + col;
      if constexpr (kCrit > 0) {
        const int c = ((i & 1) ? 0 : T - kCrit) + half * C1;
        uint32_t r[C1 / 16][16];
#pragma unroll
        for (int j = 0; j < C1 / 16; ++j) tmem_ld16(acc + c + 16 * j, r[j]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_free);
#pragma unroll
        for (int j = 0; j < C1 / 16; ++j)
          store16<O>(out, p.ldo, m0 + c + 16 * j, p.m, live, r[j], alpha);
      } else {
        // the other accumulator was emptied before this tile's wait
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_free);
      }
      const int c = ((i & 1) ? kCrit : 0) + half * C2;
      uint32_t r[2][16];
      tmem_ld16(acc + c, r[0]);
#pragma unroll
      for (int j = 0; j < C2 / 16; ++j) {
        tmem_wait_ld();
        if (j + 1 < C2 / 16) tmem_ld16(acc + c + 16 * (j + 1), r[(j + 1) & 1]);
        store16<O>(out, p.ldo, m0 + c + 16 * j, p.m, live, r[j & 1], alpha);
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CN * CM > 1) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

template <int FMT, int T, int CN, int CM, class O>
int launch(const uint8_t* a, const uint8_t* b, const ProdArgs& p, cudaStream_t s) {
  using C = WideCfg<FMT, T>;
  CUtensorMap mb, ma;
  IVFPQ_TRY(fp4_code_map(&mb, b, p.n, p.kp / 2, BN / CM));
  IVFPQ_TRY(fp4_code_map(&ma, a, p.m, p.kp / 2, T / CN));
  auto kern = fp4_wide_kernel<FMT, T, CN, CM, O>;
  IVFPQ_TRY(set_dynamic_smem(kern, C::kTotal));
  Tiling tl;
  tl.cl_n = int(ceil_div(ceil_div(p.n, BN), CN));
  tl.cl_m = int(ceil_div(ceil_div(p.m, T), CM));
  tl.m_fast = p.m <= p.n;  // the smaller operand is the one read again, from L2
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kTotal;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CN * CM;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  static int resident = 0;  // clusters that fit the device at once
  if (resident == 0) {
    cfg.gridDim = dim3(CN * CM);
    int nc = 0;
    IVFPQ_CUDA(cudaOccupancyMaxActiveClusters(&nc, kern, &cfg));
    resident = std::max(1, nc);
  }
  const int64_t tiles = int64_t(tl.cl_n) * tl.cl_m;
  cfg.gridDim = dim3(unsigned(std::min<int64_t>(tiles, resident)) * CN * CM);
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, mb, ma, p, tl));
  IVFPQ_LAUNCHED_K(kern, C::kTotal, kThreads);
  return IVFPQ_OK;
}

template <int FMT, class O>
int choose(const uint8_t* a, const uint8_t* b, const ProdArgs& p, cudaStream_t s) {
  const int64_t tn = ceil_div(p.n, BN);
  if (p.m > 128 && tn * ceil_div(p.m, 256) >= num_sms()) {
    if (p.m > 256 && tn > 1) return launch<FMT, 256, 2, 2, O>(a, b, p, s);
    return launch<FMT, 256, 1, 1, O>(a, b, p, s);
  }
  return launch<FMT, 128, 1, 1, O>(a, b, p, s);
}

}  // namespace

int fp4_product_wide(const uint8_t* a, const uint8_t* b, const ProdArgs& p, int fmt,
                     cudaStream_t s) {
  return by_dtype(p.dtype, [&](auto* t) -> int {
    using O = std::remove_pointer_t<decltype(t)>;
    return fmt == IVFPQ_MXFP4 ? choose<IVFPQ_MXFP4, O>(a, b, p, s)
                              : choose<IVFPQ_NVFP4, O>(a, b, p, s);
  });
}

}  // namespace ivfpq
