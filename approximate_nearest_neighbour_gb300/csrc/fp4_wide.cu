// The wide product of packed 4-bit rows (fp4_product.cu has the narrow one and
// the entry points): many rows on both sides.
//
// Pairs of CTAs (cta_group::2), one CTA per SM, persistent: a pair computes 256
// columns of out (rows of b) x T rows of out, T = 128 or 256. Each CTA holds
// 128 rows of b and T / 2 rows of a and accumulates its 128 columns over all T
// rows, so an SM takes in 38 KB per 256 columns of K where a CTA on its own
// took 54 KB: filling shared memory was the limit (8192 x 16384 x 4096 nvfp4:
// loads alone 157 us, products alone 146 us, together 198 us on single CTAs).
//
// 10 warps: warp 0 loads; warp 1 of the pair's first CTA copies scales to TMEM
// and issues products for both; warps 2..9 store (two per TMEM lane group, half
// of the rows each). While a tile is stored the next one is computed: with T =
// 256 the two accumulators overlap (TMEM columns 0..255 and 160..415), so the
// storing warps first empty the 96 shared columns and release them. Columns
// 416..511 hold two buffers of scales, each reused when the products two
// stages back have finished.
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
  static constexpr int kA = T / 2 * KB;
  static constexpr int kSf = (1 + kRt) * kSfTile;  // b's scales, then all T rows' of a
  static constexpr int kStage = kB + kA + kSf;
  static constexpr int kStages = (226 * 1024 - 1536) / kStage < 8 ? (226 * 1024 - 1536) / kStage : 8;
  static constexpr int kTotal = kStages * kStage + 512 + 1024;
  static constexpr int kSfCols = 4 * kTiles * (1 + kRt);  // TMEM columns of one scale buffer
  static constexpr int kAcc1 = T == 256 ? 160 : T;        // first column of the second accumulator
  static_assert(kSfBase + 2 * kSfCols <= 512 && kAcc1 + T <= kSfBase, "TMEM columns");
  static_assert(kTotal <= 227 * 1024, "shared memory");
};

// A copy into this CTA's shared memory that completes on a barrier of either
// CTA of the pair (bar is a cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y,
                                                 uint32_t bar, uint32_t el) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n"
      " @q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(el)
      : "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
__device__ __forceinline__ void pair_commit(uint32_t bar, uint32_t el) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(
          bar),
      "r"(el)
      : "memory");
}
// Completes on the barrier of both CTAs.
__device__ __forceinline__ void pair_commit_both(uint32_t bar, uint32_t el) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n}" ::"r"(bar),
      "h"(uint16_t(3)), "r"(el)
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
  int tn, tm;   // pair tiles along n and m
  int m_fast;   // consecutive tiles go along m
};

template <int FMT, int T, class O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
fp4_wide_kernel(const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_a,
                const __grid_constant__ CUtensorMap map_sb,
                const __grid_constant__ CUtensorMap map_sa, const ProdArgs p, const Tiling tl) {
  using C = WideCfg<FMT, T>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t fp4_wide_smem[];
  const uint32_t raw = smem_u32(fp4_wide_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = fp4_wide_smem + (base - raw);
  auto s_b = [&](int s) { return base + s * (C::kB + C::kA); };
  auto s_a = [&](int s) { return base + s * (C::kB + C::kA) + C::kB; };
  const uint32_t sf0 = base + NS * (C::kB + C::kA);
  auto s_sf = [&](int s) { return sf0 + s * C::kSf; };
  const uint32_t bars = base + NS * C::kStage;
  auto bar_full = [&](int s) { return bars + 8 * s; };          // first CTA's: both CTAs' copies
  auto bar_empty = [&](int s) { return bars + 8 * (NS + s); };  // each CTA's
  auto bar_sf = [&](int b) { return bars + 16 * NS + 8 * b; };
  const uint32_t bar_acc = bars + 16 * NS + 16;   // each CTA's: a tile is computed
  const uint32_t bar_free = bars + 16 * NS + 24;  // first CTA's: both CTAs' shared columns are read
  const uint32_t bar_end = bars + 16 * NS + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 16 * NS + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (bars - base) + 16 * NS + 48);

  const int warp = __shfl_sync(kFullMask, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = int(cluster_rank());
  const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;
  const int ntiles = tl.tn * tl.tm;
  const int nk = (p.kp + KE - 1) / KE;
  // first column of this CTA and first row of pair tile t
  auto col0 = [&](int t) { return ((tl.m_fast ? t / tl.tm : t % tl.tn) * 2 + rank) * BN; };
  auto row0 = [&](int t) { return (tl.m_fast ? t % tl.tm : t / tl.tn) * T; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_sf(0), 1);
    mbar_init(bar_sf(1), 1);
    mbar_init(bar_acc, 1);
    mbar_init(bar_free, 2 * kEpiWarps);
    mbar_init(bar_end, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto fail = [&]() {
    atomicExch(p.err, 1);
    *abort_flag = 1;
  };

  if (warp == 0) {
    // ---- loads: the whole warp runs, one lane issues ----
    const uint32_t el = elect_one();
    uint32_t s = 0, phase = 1;
    int used = 0;
    bool ok = true;
    for (int t = pair; t < ntiles && ok && !*abort_flag; t += npairs) {
      const int n0 = col0(t), m0 = row0(t);
      const int sb = n0 / BN * p.ntile, sa = m0 / 128 * p.ntile;
      for (int kc = 0; kc < nk; ++kc) {
        if (!mbar_wait(bar_empty(s), phase)) {
          fail();
          ok = false;
          break;
        }
        if (rank == 0 && el) mbar_expect_tx(bar_full(s), 2 * C::kStage);
        const uint32_t bar = map_rank(bar_full(s), 0);
        tma_load_2d_pair(s_b(s), &map_b, kc * KB, n0, bar, el);
        tma_load_2d_pair(s_a(s), &map_a, kc * KB, m0 + rank * (T / 2), bar, el);
        // scale tiles past the row's (or the matrix's) end are read and not used
        tma_load_2d_pair(s_sf(s), &map_sb, 0, sb + kc * C::kTiles, bar, el);
#pragma unroll
        for (int r = 0; r < C::kRt; ++r)
          tma_load_2d_pair(s_sf(s) + (1 + r) * C::kSfTile, &map_sa, 0,
                           sa + r * p.ntile + kc * C::kTiles, bar, el);
        used = min(used + 1, NS);
        if (++s == NS) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // every stage used has been released: no copy, product or release is in
    // flight when the CTA ends
    for (int j = 0; j < used; ++j) {
      s = s == 0 ? NS - 1 : s - 1;
      if (s == NS - 1) phase ^= 1;
      mbar_wait(bar_empty(s), phase ^ 1);
    }
  } else if (warp == 1 && rank == 0) {
    // ---- scales and products of both CTAs: the whole warp runs, one lane issues ----
    const uint32_t el = elect_one();
    const uint64_t d_b = smem_desc(s_b(0)), d_a = smem_desc(s_a(0)), d_sf = scale_desc(s_sf(0));
    const int last_tiles = p.ntile - (nk - 1) * C::kTiles;
    const int last_steps = (p.kp - (nk - 1) * KE + 63) / 64;
    uint32_t s = 0, phase = 0;       // stage, its parity
    uint32_t sb = 0, sphase = 1;     // scale buffer, parity of its last release
    uint32_t fphase = 1;             // parity of the last release of the accumulator
    bool ok = true;
    for (int t = pair, i = 0; t < ntiles && ok && !*abort_flag; t += npairs, ++i) {
      if (i > 0 && !mbar_wait(bar_free, fphase)) {
        fail();
        break;
      }
      fphase ^= 1;
      tc_fence_after();
      const uint32_t acc = tmem + ((i & 1) ? C::kAcc1 : 0);
      for (int kc = 0; kc < nk; ++kc) {
        // a fresh barrier lets a wait for the odd parity through
        if (!mbar_wait(bar_full(s), phase) || !mbar_wait(bar_sf(sb), sphase)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const bool last = kc == nk - 1;
        const uint32_t tb = tmem + kSfBase + sb * C::kSfCols, ta = tb + 4 * C::kTiles;
        const uint64_t sd = d_sf + s * uint32_t(C::kSf >> 4);
        const int tiles = last ? last_tiles : C::kTiles;
#pragma unroll
        for (int q = 0; q < C::kTiles; ++q) {
          if (q < tiles) {
            scale_copy<2>(tb + 4 * q, sd + 32 * q, el);
#pragma unroll
            for (int r = 0; r < C::kRt; ++r)
              scale_copy<2>(ta + 4 * (q * C::kRt + r), sd + ((1 + r) * C::kSfTile + 512 * q) / 16,
                            el);
          }
        }
        const uint64_t db = d_b + s * uint32_t((C::kB + C::kA) >> 4);
        const uint64_t da = d_a + s * uint32_t((C::kB + C::kA) >> 4);
        const int steps = last ? last_steps : 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j < steps) {
            const int q = FMT == IVFPQ_MXFP4 ? j >> 1 : j;
            const uint32_t id = FMT == IVFPQ_MXFP4 ? uint32_t(j & 1) * 2 : 0u;
            mma_fp4<FMT, 2>(acc, db + 2 * j, da + 2 * j, fp4_idesc<FMT, T, 2>(id), tb + 4 * q,
                            ta + 4 * C::kRt * q, kc > 0 || j > 0, el);
          }
        }
        pair_commit(bar_sf(sb), el);
        pair_commit_both(bar_empty(s), el);
        if (++s == NS) {
          s = 0;
          phase ^= 1;
        }
        sb ^= 1;
        sphase ^= sb ^ 1;
      }
      if (ok) pair_commit_both(bar_acc, el);
    }
    // all products issued have finished before TMEM is freed
    pair_commit(bar_end, el);
    mbar_wait(bar_end, 0);
  } else if (warp >= 2) {
    // ---- store: warp w reads TMEM lanes 32 * (w % 4) .. +32 ----
    const int lg = warp & 3, half = (warp - 2) >> 2;
    const float alpha = (p.a_ts ? __ldg(p.a_ts) : 1.f) * (p.b_ts ? __ldg(p.b_ts) : 1.f);
    constexpr int kCrit = T == 256 ? 96 : 0;  // columns the next accumulator shares
    constexpr int C1 = kCrit / 2, C2 = (T - kCrit) / 2;
    const uint32_t free0 = map_rank(bar_free, 0);
    int i = 0;
    for (int t = pair; t < ntiles && !*abort_flag; t += npairs, ++i) {
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
        if (lane == 0) arrive_remote(free0);
#pragma unroll
        for (int j = 0; j < C1 / 16; ++j)
          store16<O>(out, p.ldo, m0 + c + 16 * j, p.m, live, r[j], alpha);
      } else {
        // the other accumulator was emptied before this tile's wait
        __syncwarp();
        if (lane == 0) arrive_remote(free0);
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
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// Scale tiles as rows of 128 words; a box is one stage's tiles of 128 rows.
int scale_map(CUtensorMap* m, const uint8_t* p, int64_t tiles, int box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  IVFPQ_TRY(tensor_map_encoder(&enc));
  cuuint64_t dims[2] = {128, cuuint64_t(tiles)};
  cuuint64_t strides[1] = {512};
  cuuint32_t bx[2] = {128, cuuint32_t(box)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(p), dims, strides,
                   bx, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for %lld scale tiles", int(r), (long long)tiles);
    return IVFPQ_ERR_CUDA;
  }
  return IVFPQ_OK;
}

template <int FMT, int T, class O>
int launch(const uint8_t* a, const uint8_t* b, const ProdArgs& p, cudaStream_t s) {
  using C = WideCfg<FMT, T>;
  CUtensorMap mb, ma, msb, msa;
  IVFPQ_TRY(fp4_code_map(&mb, b, p.n, p.kp / 2, BN));
  IVFPQ_TRY(fp4_code_map(&ma, a, p.m, p.kp / 2, T / 2));
  IVFPQ_TRY(scale_map(&msb, p.b_scales, ceil_div(p.n, 128) * p.ntile, C::kTiles));
  IVFPQ_TRY(scale_map(&msa, p.a_scales, ceil_div(p.m, 128) * p.ntile, C::kTiles));
  auto kern = fp4_wide_kernel<FMT, T, O>;
  IVFPQ_TRY(set_dynamic_smem(kern, C::kTotal));
  Tiling tl;
  tl.tn = int(ceil_div(p.n, 2 * BN));
  tl.tm = int(ceil_div(p.m, T));
  tl.m_fast = p.m <= p.n;  // the smaller operand is the one read again, from L2
  static int resident = 0;  // pairs that fit the device at once
  if (resident == 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kTotal;
    int nc = 0;
    IVFPQ_CUDA(cudaOccupancyMaxActiveClusters(&nc, kern, &cfg));
    resident = std::max(1, nc);
  }
  const int64_t tiles = int64_t(tl.tn) * tl.tm;
  const unsigned grid = unsigned(std::min<int64_t>(tiles, resident)) * 2;
  kern<<<grid, kThreads, C::kTotal, s>>>(mb, ma, msb, msa, p, tl);
  IVFPQ_LAUNCHED_K(kern, C::kTotal, kThreads);
  return IVFPQ_OK;
}

template <int FMT, class O>
int choose(const uint8_t* a, const uint8_t* b, const ProdArgs& p, cudaStream_t s) {
  if (p.m > 128 && ceil_div(p.n, 2 * BN) * ceil_div(p.m, 256) * 2 >= num_sms())
    return launch<FMT, 256, O>(a, b, p, s);
  return launch<FMT, 128, O>(a, b, p, s);
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
