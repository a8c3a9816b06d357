// The wide product of packed 4-bit rows (fp4_product.cu has the narrow one and
// the entry points): many rows on both sides.
//
// Persistent CTAs, one per SM, of 128 columns of out (rows of b) x T rows of
// out, T = 128 or 256, alone (CG = 1) or in pairs (cta_group::2): a pair shares
// the T rows of a, half in each CTA, so an SM takes in 38 KB per 256 columns
// of K instead of 54 KB. Filling shared memory is close to a limit: 8192 x
// 16384 x 4096 NVFP4 takes 157 us for the loads alone, 146 us for the products
// alone (64 columns of K an instruction) and 194 us together on single CTAs, 183 us
// (6.0 PFLOP/s) in pairs; up to 218 us where the device lowers its clock. With
// short K the result's bytes bound it: 10000 x 65536 x 96 to fp32 437 us, 2.6 GB
// at 6.0 TB/s.
//
// 10 warps: warp 0 loads; warp 1 of the pair's first CTA copies scales to TMEM
// and issues products for both; warps 2..9 store (two per TMEM lane group, every
// other 16 rows each). While a tile is stored the next ones are computed: T = 128
// has three accumulators; with T = 256 two overlap (TMEM columns 0..255 and
// 160..415), so the storing warps first empty the 96 shared columns and
// release them. Columns 416..511 hold two buffers of scales, each reused when
// the products two stages back have finished.
#include <algorithm>
#include <atomic>

#include "fp4_mma.cuh"

namespace ivfpq {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kSfBase = 416;  // first TMEM column of the scales
constexpr int64_t kL2Bytes = int64_t(129) << 20;
constexpr int kBounce = 8 * BN * 4;  // 8 rows of a tile on their way out, per half of the warps

template <int FMT, int T, int CG, int KB>
struct WideCfg {
  static constexpr int KE = 2 * KB;  // K columns per stage
  static constexpr int kTiles = KE / (FMT == IVFPQ_MXFP4 ? 128 : 64);  // scale tiles per stage
  static constexpr int kRt = T / 128;
  static constexpr int kSfTile = kTiles * 512;
  static constexpr int kB = BN * KB;
  static constexpr int kA = T / CG * KB;
  static constexpr int kSf = (1 + kRt) * kSfTile;  // b's scales, then all T rows' of a
  static constexpr int kStage = kB + kA + kSf;
  static constexpr int kFit = (227 * 1024 - 1536 - 2 * kBounce) / kStage;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kTotal = kStages * kStage + 512 + 1024 + 2 * kBounce;
  static constexpr int kSfCols = 4 * kTiles * (1 + kRt);  // TMEM columns of one scale buffer
  // accumulators and the columns between their starts
  static constexpr int kAccs = T == 256 ? 2 : 3;
  static constexpr int kAccStep = T == 256 ? 160 : T;
  static_assert(kSfBase + 2 * kSfCols <= 512 && (kAccs - 1) * kAccStep + T <= kSfBase,
                "TMEM columns");
  static_assert(kTotal <= 227 * 1024, "shared memory");
};

// A copy into this CTA's shared memory; in a pair it completes on a barrier of
// either CTA (bar is then a cluster address).
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar, uint32_t el) {
  if (CG == 2)
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n @q cp.async.bulk.tensor.2d.cta_group::2"
        ".shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(el)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n @q cp.async.bulk.tensor.2d"
        ".shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(el)
        : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
// Completes on this CTA's barrier ...
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar, uint32_t el) {
  if (CG == 2)
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(
            bar),
        "r"(el)
        : "memory");
  else
    mma_commit_el(bar, el);
}
// ... or on the barrier of every CTA of the group.
template <int CG>
__device__ __forceinline__ void commit_all(uint32_t bar, uint32_t el) {
  if (CG == 2)
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n @q tcgen05.commit.cta_group::2"
        ".mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::"r"(bar),
        "h"(uint16_t(3)), "r"(el)
        : "memory");
  else
    mma_commit_el(bar, el);
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

// All of the SM's TMEM; in a pair both CTAs take part.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t slot) {
  if (CG == 2)
    asm volatile(
        "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n"
        "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(slot)
        : "memory");
  else
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n"
        "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::"r"(slot)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t tmem) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// 16 accumulator columns (rows r0 .. r0 + 15 of out) of this lane's column. With
// 16-bit outputs and even row lengths two lanes exchange halves, so that each
// stores two neighbouring columns of one of two rows: half the store
// instructions, each of 128 bytes.
template <class O>
__device__ __forceinline__ void store16(O* out, int64_t ldo, int r0, int64_t m, bool live,
                                        bool pairs, const uint32_t (&r)[16], float alpha) {
  if constexpr (sizeof(O) == 2) {
    if (pairs) {
      const int odd = threadIdx.x & 1;
      uint32_t* p = reinterpret_cast<uint32_t*>(out + (r0 + odd) * ldo - odd);
#pragma unroll
      for (int j = 0; j < 16; j += 2, p += ldo) {
        const float v0 = __uint_as_float(r[j]) * alpha, v1 = __uint_as_float(r[j + 1]) * alpha;
        const float got = __shfl_xor_sync(kFullMask, odd ? v0 : v1, 1);
        O w[2] = {from_f32<O>(odd ? got : v0), from_f32<O>(odd ? v1 : got)};
        if (live && r0 + j + odd < m) *p = *reinterpret_cast<const uint32_t*>(w);
      }
      return;
    }
  }
  O* p = out + r0 * ldo;
  if (live) {
#pragma unroll
    for (int j = 0; j < 16; ++j, p += ldo)
      if (r0 + j < m) *p = from_f32<O>(__uint_as_float(r[j]) * alpha);
  }
}

// The same for fp32 rows at odd offsets in a result larger than L2. A warp's 32
// columns leave two sectors of each row half written, and those reach memory
// apart: 10000 x 65535 x 96 took 1070 us, and 457 us with 65528 columns (32-byte
// rows). Here four warps exchange 8 rows of 128 columns through shared memory and
// each writes whole lines of two of them: 760 to 795 us, and 122 us instead of 147 us
// at 1000 x 100003 x 128. Smaller results (77 x 100003: 17.6 us, and 21.8 us
// here), rows on 16 bytes (1000 x 100004: 90 and 122 us) and 16-bit results
// (8192 x 16385 x 4096: 199 and 360 us) are better off without.
__device__ __forceinline__ void half_sync(int half) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + half) : "memory");
}
// Whether all 128 threads of the half say so.
__device__ __forceinline__ bool half_all(int half, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n barrier.cta.red.and.pred p, %2, 128, q;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(r)
      : "r"(uint32_t(ok)), "r"(1 + half)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void store16_lines(float* out, int64_t ldo, int r0, int64_t m, int cols,
                                              float* buf, int lg, int half,
                                              const uint32_t (&r)[16], float alpha) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      buf[j * BN + 32 * lg + lane] = __uint_as_float(r[8 * h + j]) * alpha;
    half_sync(half);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int row = r0 + 8 * h + 2 * lg + q;
      if (row < m) {
        const float* b = buf + (2 * lg + q) * BN;
        float* p = out + row * ldo;
        const int mis = int(reinterpret_cast<uintptr_t>(p) & 127) / 4;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          const int e = i * 32 + lane - mis;
          if (e >= 0 && e < cols) p[e] = b[e];
        }
      }
    }
    half_sync(half);
  }
}

struct Tiling {
  int tn, tm;   // tiles along n and m
  int m_fast;   // consecutive tiles go along m
};

template <int FMT, int T, int CG, int KB, class O>
__global__ void __launch_bounds__(kThreads, 1)
fp4_wide_kernel(const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_a,
                const __grid_constant__ CUtensorMap map_sb,
                const __grid_constant__ CUtensorMap map_sa, const ProdArgs p, const Tiling tl) {
  using C = WideCfg<FMT, T, CG, KB>;
  constexpr int KE = C::KE;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t fp4_wide_smem[];
  const uint32_t raw = smem_u32(fp4_wide_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = fp4_wide_smem + (base - raw);
  auto s_b = [&](int s) { return base + s * (C::kB + C::kA); };
  auto s_a = [&](int s) { return base + s * (C::kB + C::kA) + C::kB; };
  const uint32_t sf0 = base + NS * (C::kB + C::kA);
  auto s_sf = [&](int s) { return sf0 + s * C::kSf; };
  const uint32_t bars = base + NS * C::kStage + 2 * kBounce;
  auto bar_full = [&](int s) { return bars + 8 * s; };          // first CTA's: both CTAs' copies
  auto bar_empty = [&](int s) { return bars + 8 * (NS + s); };  // each CTA's
  auto bar_sf = [&](int b) { return bars + 16 * NS + 8 * b; };
  // per accumulator: each CTA's, a tile is computed; the first CTA's, what the
  // next product overwrites has been read in all CTAs
  auto bar_acc = [&](int b) { return bars + 16 * NS + 16 + 8 * b; };
  auto bar_free = [&](int b) { return bars + 16 * NS + 40 + 8 * b; };
  const uint32_t bar_end = bars + 16 * NS + 64;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 16 * NS + 72);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (bars - base) + 16 * NS + 80);

  const int warp = __shfl_sync(kFullMask, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = CG == 2 ? int(cluster_rank()) : 0;
  const int group = blockIdx.x / CG, ngroups = gridDim.x / CG;
  const int ntiles = tl.tn * tl.tm;
  const int nk = (p.kp + KE - 1) / KE;
  // first column of this CTA and first row of tile t
  auto col0 = [&](int t) { return ((tl.m_fast ? t / tl.tm : t % tl.tn) * CG + rank) * BN; };
  auto row0 = [&](int t) { return (tl.m_fast ? t % tl.tm : t / tl.tn) * T; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_sf(0), 1);
    mbar_init(bar_sf(1), 1);
    for (int b = 0; b < C::kAccs; ++b) {
      mbar_init(bar_acc(b), 1);
      mbar_init(bar_free(b), CG * kEpiWarps);
    }
    mbar_init(bar_end, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(tmem_slot));
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
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
    // one row tile and stages that meet the same K step each time: a's rows stay
    // in the stages after the first turn. Rows are what short K costs (about 6
    // clocks each, however few bytes).
    const bool keep_a = tl.tm == 1 && NS % nk == 0;
    int used = 0;
    bool ok = true;
    grid_wait();
    for (int t = group; t < ntiles && ok && !*abort_flag; t += ngroups) {
      const int n0 = col0(t), m0 = row0(t);
      const int sb = n0 / BN * p.ntile, sa = m0 / 128 * p.ntile;
      for (int kc = 0; kc < nk; ++kc) {
        if (!mbar_wait(bar_empty(s), phase)) {
          fail();
          ok = false;
          break;
        }
        const bool have = keep_a && used == NS;
        const uint32_t bytes = have ? C::kB + C::kSfTile : C::kStage;
        if (rank == 0 && el) mbar_expect_tx(bar_full(s), CG * bytes);
        const uint32_t bar = CG == 2 ? map_rank(bar_full(s), 0) : bar_full(s);
        // scale tiles past the row's (or the matrix's) end are read and not used
        tma_load<CG>(s_b(s), &map_b, kc * KB, n0, bar, el);
        tma_load<CG>(s_sf(s), &map_sb, 0, sb + kc * C::kTiles, bar, el);
        if (!have) {
          tma_load<CG>(s_a(s), &map_a, kc * KB, m0 + rank * (T / CG), bar, el);
#pragma unroll
          for (int r = 0; r < C::kRt; ++r)
            tma_load<CG>(s_sf(s) + (1 + r) * C::kSfTile, &map_sa, 0,
                         sa + r * p.ntile + kc * C::kTiles, bar, el);
        }
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
    const uint64_t d_b = code_desc<KB>(s_b(0)), d_a = code_desc<KB>(s_a(0));
    const uint64_t d_sf = scale_desc(s_sf(0));
    const int last_tiles = p.ntile - (nk - 1) * C::kTiles;
    const int last_steps = (p.kp - (nk - 1) * KE + 63) / 64;
    uint32_t s = 0, phase = 0;       // stage, its parity
    uint32_t sb = 0, sphase = 1;     // scale buffer, parity of its last release
    int b = 0, turn = 0;             // accumulator, how often it has been used
    bool ok = true;
    for (int t = group, i = 0; t < ntiles && ok && !*abort_flag; t += ngroups, ++i) {
      // T = 256: the columns shared with the last tile's accumulator have been
      // read (and all of the one before); else this accumulator's last tile has
      const bool go = T < 256 ? mbar_wait(bar_free(b), (turn & 1) ^ 1)
                              : i == 0 || mbar_wait(bar_free(b ^ 1), ((i - 1) >> 1) & 1);
      if (!go) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + b * C::kAccStep;
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
            scale_copy<CG>(tb + 4 * q, sd + 32 * q, el);
#pragma unroll
            for (int r = 0; r < C::kRt; ++r)
              scale_copy<CG>(ta + 4 * (q * C::kRt + r), sd + ((1 + r) * C::kSfTile + 512 * q) / 16,
                            el);
          }
        }
        const uint64_t db = d_b + s * uint32_t((C::kB + C::kA) >> 4);
        const uint64_t da = d_a + s * uint32_t((C::kB + C::kA) >> 4);
        const int steps = last ? last_steps : KB / 32;
#pragma unroll
        for (int j = 0; j < KB / 32; ++j) {
          if (j < steps) {
            const int q = FMT == IVFPQ_MXFP4 ? j >> 1 : j;
            const uint32_t id = FMT == IVFPQ_MXFP4 ? uint32_t(j & 1) * 2 : 0u;
            mma_fp4<FMT, CG>(acc, db + 2 * j, da + 2 * j, fp4_idesc<FMT, T, CG>(id), tb + 4 * q,
                            ta + 4 * C::kRt * q, kc > 0 || j > 0, el);
          }
        }
        commit<CG>(bar_sf(sb), el);
        commit_all<CG>(bar_empty(s), el);
        if (++s == NS) {
          s = 0;
          phase ^= 1;
        }
        sb ^= 1;
        sphase ^= sb ^ 1;
      }
      if (ok) commit_all<CG>(bar_acc(b), el);
      if (++b == C::kAccs) {
        b = 0;
        ++turn;
      }
    }
    // all products issued have finished before TMEM is freed
    commit<CG>(bar_end, el);
    mbar_wait(bar_end, 0);
  } else if (warp >= 2) {
    // ---- store: warp w reads TMEM lanes 32 * (w % 4) .. +32 ----
    const int lg = warp & 3, half = (warp - 2) >> 2;
    grid_wait();
    const float alpha = (p.a_ts ? __ldg(p.a_ts) : 1.f) * (p.b_ts ? __ldg(p.b_ts) : 1.f);
    constexpr int kCrit = T == 256 ? 96 : 0;  // columns the next accumulator shares
    constexpr int C1 = kCrit / 2, C2 = (T - kCrit) / 2;
    auto release = [&](int b) {
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          arrive_remote(map_rank(bar_free(b), 0));
        else
          mbar_arrive(bar_free(b));
      }
    };
    const bool pairs = p.n % 2 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 3) == 0;
    const bool lines =
        sizeof(O) == 4 &&
        (p.n % 4 != 0 || (reinterpret_cast<uintptr_t>(p.out) & 15) != 0) &&
        p.m * p.n * 4 > kL2Bytes;
    float* bounce = reinterpret_cast<float*>(gbase + NS * C::kStage + half * kBounce);
    int b = 0, turn = 0;
    for (int t = group; t < ntiles; t += ngroups) {
      bool ok = !*abort_flag;
      if (ok && !mbar_wait(bar_acc(b), turn & 1)) {
        fail();
        ok = false;
      }
      // warps that exchange rows go on, or stop, together: none waits at their
      // barrier for one that has given up
      if (lines) ok = half_all(half, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t(32 * lg) << 16) + uint32_t(b * C::kAccStep);
      const int col = col0(t) + 32 * lg + lane, m0 = row0(t);
      const bool live = col < p.n;
      O* out = static_cast<O*>(p.out) + col;
      O* line0 = static_cast<O*>(p.out) + col0(t);
      const int cols = int(min(int64_t(BN), p.n - col0(t)));
      auto put = [&](const uint32_t (&r)[16], int r0) {
        if constexpr (sizeof(O) == 4) {
          if (lines)
            return store16_lines(line0, p.ldo, r0, p.m, cols, bounce, lg, half, r, alpha);
        }
        store16<O>(out, p.ldo, r0, p.m, live, pairs, r, alpha);
      };
      // units of 16 rows, every other one this warp's; those past m are not read
      auto units = [&](int c, int n) {
        const int64_t left = p.m - m0 - c - 16 * half;
        return left <= 0 ? 0 : int(min(int64_t(n), (left + 31) / 32));
      };
      if constexpr (kCrit > 0) {
        const int c = (b ? 0 : T - kCrit) + 16 * half, n = units(c - 16 * half, C1 / 16);
        uint32_t r[C1 / 16][16];
#pragma unroll
        for (int j = 0; j < C1 / 16; ++j)
          if (j < n) tmem_ld16(acc + c + 32 * j, r[j]);
        tmem_wait_ld();
        tc_fence_before();
        release(b);
#pragma unroll
        for (int j = 0; j < C1 / 16; ++j)
          if (j < n) put(r[j], m0 + c + 32 * j);
      }
      const int c = (kCrit && b ? kCrit : 0) + 16 * half, n = units(c - 16 * half, C2 / 16);
      uint32_t r[2][16];
      if (n > 0) tmem_ld16(acc + c, r[0]);
      if (kCrit == 0 && n == 0) release(b);
#pragma unroll
      for (int j = 0; j < C2 / 16; ++j) {
        if (j < n) {
          tmem_wait_ld();
          if (j + 1 < n) {
            tmem_ld16(acc + c + 32 * (j + 1), r[(j + 1) & 1]);
          } else if (kCrit == 0) {
            tc_fence_before();
            release(b);
          }
          put(r[j & 1], m0 + c + 32 * j);
        }
      }
      tc_fence_before();
      if (++b == C::kAccs) {
        b = 0;
        ++turn;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem);
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

template <int FMT, int T, int CG, int KB, class O>
int launch(const uint8_t* a, const uint8_t* b, const ProdArgs& p, cudaStream_t s) {
  using C = WideCfg<FMT, T, CG, KB>;
  CUtensorMap mb, ma, msb, msa;
  IVFPQ_TRY(fp4_code_map(&mb, b, p.n, p.kp / 2, KB, BN));
  IVFPQ_TRY(fp4_code_map(&ma, a, p.m, p.kp / 2, KB, T / CG));
  IVFPQ_TRY(scale_map(&msb, p.b_scales, ceil_div(p.n, 128) * p.ntile, C::kTiles));
  IVFPQ_TRY(scale_map(&msa, p.a_scales, ceil_div(p.m, 128) * p.ntile, C::kTiles));
  auto kern = fp4_wide_kernel<FMT, T, CG, KB, O>;
  IVFPQ_TRY(set_dynamic_smem(kern, C::kTotal));
  Tiling tl;
  tl.tn = int(ceil_div(p.n, CG * BN));
  tl.tm = int(ceil_div(p.m, T));
  tl.m_fast = p.m <= p.n;  // the smaller operand is the one read again, from L2
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(CG);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kTotal;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CG;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  static std::atomic<int> resident{0};  // groups that fit the device at once
  if (resident == 0) {
    int nc = 0;
    IVFPQ_CUDA(cudaOccupancyMaxActiveClusters(&nc, kern, &cfg));
    resident = std::max(1, nc);
  }
  const int64_t tiles = int64_t(tl.tn) * tl.tm;
  cfg.gridDim = dim3(unsigned(std::min<int64_t>(tiles, resident.load())) * CG);
  cfg.numAttrs = p.overlap ? 2 : 1;
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, mb, ma, msb, msa, p, tl));
  IVFPQ_LAUNCHED_K(kern, C::kTotal, kThreads);
  return IVFPQ_OK;
}

template <int FMT, class O>
int choose(const uint8_t* a, const uint8_t* b, const ProdArgs& p, cudaStream_t s) {
  // Rows per tile: 256, unless 128 take fewer or shorter waves (a 128-row tile
  // costs 0.65 of a 256-row one: 8192 x 16384 x 4096 takes 255 us in 128-row
  // tiles and 194 us in 256-row ones; 300 x 100000 x 512, whose second 256 rows
  // are mostly empty, 33 and 39 us).
  const int64_t tn = ceil_div(p.n, BN), sms = num_sms();
  const double w128 = 0.65 * double(ceil_div(tn * ceil_div(p.m, 128), sms));
  const double w256 = double(ceil_div(tn * ceil_div(p.m, 256), sms));
  if (p.kp <= kShortK)
    return w128 < w256 ? launch<FMT, 128, 1, 64, O>(a, b, p, s)
                       : launch<FMT, 256, 1, 64, O>(a, b, p, s);
  if (w128 < w256) return launch<FMT, 128, 1, 128, O>(a, b, p, s);
  // Pairs where K is long and there are many tiles (8192 x 16384 x 4096: 183 us,
  // and 194 us on single CTAs); a pair's hand-over between tiles costs more
  // (1000 x 100000 x 1024: 102 us, and 86 us).
  if (p.kp >= 2048 && w256 >= 8) return launch<FMT, 256, 2, 128, O>(a, b, p, s);
  return launch<FMT, 256, 1, 128, O>(a, b, p, s);
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
