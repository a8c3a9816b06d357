// adapter_linear for many tokens, in tiles of 128 tokens of one adapter.
//
// h = x A^T: a block takes a tile and a part of K, 128 bytes of every row of x and A
// at a time. Eight warps copy them into shared memory in the tensor core's order (tokens
// are gathered, so a row is nobody's neighbour), a ninth issues the products; the
// parts of K are a cluster and joined through its shared memory. Bound by memory: x is
// read once, A once per tile (from L2).
//
// out = base + scale h B^T, in units of a tile by 256 bytes of every row. Bound by
// memory: a unit reads and writes 32 KB, 1.5 us of an SM's share of the
// copy bandwidth, and its product takes a tenth of that. So everything is arranged
// around the two streams of rows:
//  - one persistent block per SM takes an equal run of units, columns first, so that
//    a tile's h is prepared once or twice per block;
//  - warp 0 brings the adapter's rows of B (TMA, zeros past its rank and its last
//    column), warp 1 issues the products: A is h, cut into two or three 16-bit terms,
//    so B is used once per term; the accumulator is one of four in TMEM;
//  - four groups of four warps take units in turn. A warp brings its 32 base rows into
//    a place of its own in shared memory, adds the accumulator to them there, a row
//    per thread, writes them in whole lines, and asks for those of its next unit.
// Measured at 8192 tokens, 4096 x 16384 bf16, rank 64, 6 adapters: h 22 us (67 MB, 3.0 TB/s:
// few blocks, each a chain of copies and products), the output 93 us (537 MB, 5.8 TB/s).
// The output through registers instead of shared memory (a warp's 32 columns of 16 rows,
// fetched four steps ahead) took 176 us; with rows by bulk copies of 256 bytes, which the
// copy engine takes one every 30 clocks or so, 250 us.
#include <limits.h>

#include <algorithm>

#include "adapter.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace ivfpq {
namespace {

constexpr int kRows = kMaxTile;
constexpr int kGroups = 4, kGroupWarps = 4;
constexpr int kEpiThreads = kGroups * kGroupWarps * 32;
constexpr int kThreads = 64 + kEpiThreads;
constexpr int kRowBytes = 256;  // of a row of a unit

template <class T, class O, int KC>
struct Cfg {
  static constexpr int CN = kRowBytes / int(sizeof(O));  // columns of a unit
  static constexpr int TERMS =
      std::is_same<T, __nv_bfloat16>::value && std::is_same<O, float>::value ? 3 : 2;
  // B of so many units; one group's rows fewer where the rest does not leave room
  static constexpr int NB = KC == 1 ? 2 : 1;
  static constexpr int kA = TERMS * KC * kRows * 128;
  static constexpr int kB = KC * CN * 128;
  static constexpr int GROUPS = kA + NB * kB + kGroups * kRows * kRowBytes > 225 * 1024
                                    ? kGroups - 1
                                    : kGroups;
  static constexpr int kBuf = GROUPS * kRows * kRowBytes;
  static constexpr int kBars = 8 * (2 * NB + 2 * kGroups) + 16;
  static constexpr int kTotal = kA + NB * kB + kBuf + kBars + 1024;
  static constexpr int kTmem = kGroups * CN;
  static_assert(kTotal + kRows * 4 <= 227 * 1024, "fits shared memory");
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
template <class T, int N>
__device__ __forceinline__ void mma_16bit(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  constexpr uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
  constexpr uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | (uint32_t(N >> 3) << 17) |
                             (uint32_t(kRows >> 4) << 24);
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---- h = x A^T ------------------------------------------------------------------------
constexpr int kLoadWarps = 8, kShrinkThreads = (kLoadWarps + 1) * 32;
template <int R, bool ALIGNED>
struct ShrinkCfg {
  static constexpr int NR = R < 16 ? 16 : R;  // the instruction's least width is 16
  static constexpr int kStage = (kRows + NR) * 128;
  static constexpr int kFit = ALIGNED ? 200 * 1024 / kStage : 2;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  // not ALIGNED: steps as they lie in memory
  static constexpr int kRawRow = 128 + 16, kRaw = (kRows + NR) * kRawRow;
  static constexpr int kRawFit = ALIGNED ? 0 : (220 * 1024 - kStages * kStage) / kRaw;
  static constexpr int kRaws = kRawFit < 8 ? kRawFit : 8;
  static constexpr int kTotal =
      kStages * kStage + kRaws * kRaw + 8 * (2 * kStages + 1) + 16 + 1024;
  static constexpr int kTmem = NR < 32 ? 32 : NR;
  static_assert(kTotal <= 227 * 1024, "fits shared memory");
};

// ALIGNED: rows of x and A are multiples of 16 bytes and start on one. Others are copied as
// they lie, in whole vectors, and shifted into the operands' place; the sums are the same.
// (8192 rows at rank 128: 27 us with 4096 columns, 50 us with 4097; shifted on their way
// through registers they took 108 us, since the loads of a step's rows waited for each
// other.)
template <class T, int R, bool ALIGNED>
__global__ void __launch_bounds__(kShrinkThreads, 1)
    adapter_shrink_wide_kernel(const AdapterArgs a, int* err) {
  using C = ShrinkCfg<R, ALIGNED>;
  extern __shared__ uint8_t shrink_raw[];
  const uint32_t raw = smem_u32(shrink_raw);
  const uint32_t base_addr = (raw + 1023u) & ~1023u;
  uint8_t* mem = shrink_raw + (base_addr - raw);
  constexpr int kOperands = C::kStages * C::kStage + C::kRaws * C::kRaw;
  const uint32_t bars = base_addr + kOperands;
  auto full = [&](int i) { return bars + 8 * i; };
  auto empty = [&](int i) { return bars + 8 * (C::kStages + i); };
  const uint32_t done = bars + 8 * 2 * C::kStages;
  uint8_t* tail = mem + kOperands + 8 * (2 * C::kStages + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait();
  grid_go();
  const Tile t = tile_at(a, blockIdx.y + int64_t(blockIdx.z) * gridDim.y);
  if (t.count == 0 || t.adapter < 0) return;  // a cluster's blocks alike
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full(i), kLoadWarps);
      mbar_init(empty(i), 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kLoadWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (*abort_flag) return;
    if (!mbar_wait(bar, parity)) {
      atomicExch(err, 1);
      *abort_flag = 1;
    }
  };
  const int64_t k0 = int64_t(blockIdx.x) * a.kpart, k1 = min(a.cols, k0 + a.kpart);
  const int steps = k1 > k0 ? int((k1 - k0 + 63) / 64) : 0;
  if (warp < kLoadWarps) {
    // this thread's pieces: piece ch (16 bytes) of rows r0, r0 + 32, ...; the pieces of
    // row r are swapped around by r mod 8, as the operand's layout wants them
    const int ch = threadIdx.x & 7, r0 = threadIdx.x >> 3;
    constexpr int XR = kRows / 32, WR = (C::NR + 31) / 32;
    const T* x[XR];
#pragma unroll
    for (int i = 0; i < XR; ++i) {
      const int row = r0 + 32 * i;
      x[i] = row < t.count ? static_cast<const T*>(a.x) + token_of(a, t.first + row) * a.ldx
                           : nullptr;
    }
    const T* w = static_cast<const T*>(a.a) + int64_t(t.adapter) * a.rank * a.cols;
    auto w_row = [&](int row) { return row < a.rank ? w + int64_t(row) * a.cols : nullptr; };
    const uint32_t place = uint32_t(r0 * 128 + ((ch ^ (r0 & 7)) * 16));
    auto give = [&](int step) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(full(step % C::kStages));
    };
    if constexpr (ALIGNED) {
      constexpr int L = C::kStages - 1;  // steps on their way
      for (int i = 0; i < steps + L; ++i) {
        if (i < steps) {
          const int s = i % C::kStages;
          wait(empty(s), ((i / C::kStages) & 1) ^ 1);
          const uint32_t at = base_addr + s * C::kStage + place;
          const int64_t k = k0 + int64_t(i) * 64 + ch * 8;
#pragma unroll
          for (int j = 0; j < XR; ++j) {
            const bool live = k < k1 && x[j];
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + 32 * j * 128),
                         "l"(live ? x[j] + k : static_cast<const T*>(a.x)), "r"(live ? 16 : 0)
                         : "memory");
          }
#pragma unroll
          for (int j = 0; j < WR; ++j) {
            if (C::NR % 32 == 0 || r0 + 32 * j < C::NR) {
              const T* p = w_row(r0 + 32 * j);
              const bool live = k < k1 && p;
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                               at + (kRows + 32 * j) * 128),
                           "l"(live ? p + k : static_cast<const T*>(a.a)), "r"(live ? 16 : 0)
                           : "memory");
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (i >= L) {
          asm volatile("cp.async.wait_group %0;" ::"n"(L) : "memory");
          give(i - L);
        }
      }
    } else {
      // the 16-byte vectors that the columns lie in, eight and one more of every row
      constexpr int P = XR + WR, L = C::kRaws - 1;  // steps on their way
      const int bytes = int(k1 - k0) * 2;
      uintptr_t from[P];
      int mis[P];
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int row = r0 + 32 * (j - XR);
        const T* p = j < XR ? x[j < XR ? j : 0] : row < C::NR ? w_row(row) : nullptr;
        const uintptr_t at = reinterpret_cast<uintptr_t>(p + k0);
        mis[j] = int(at & 15);
        from[j] = p ? at - mis[j] + ch * 16 : 0;
      }
      const uintptr_t some = reinterpret_cast<uintptr_t>(a.a) & ~uintptr_t(15);
      auto copy = [&](uint32_t to, uintptr_t row, int at, int left) {  // zeros past the row
        const bool live = row && left > 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                     "l"(reinterpret_cast<const void*>(live ? row + at : some)),
                     "r"(live ? min(left, 16) : 0)
                     : "memory");
      };
      auto here = [&](int j) { return j < XR || C::NR % 32 == 0 || r0 + 32 * (j - XR) < C::NR; };
      const uint32_t raws = uint32_t(C::kStages * C::kStage) + r0 * C::kRawRow + ch * 16;
      for (int i = 0; i < steps + L; ++i) {
        if (i < steps) {
          const uint32_t to = base_addr + raws + i % C::kRaws * C::kRaw;
#pragma unroll
          for (int j = 0; j < P; ++j) {
            if (!here(j)) continue;
            const int left = bytes + mis[j] - i * 128 - ch * 16;
            copy(to + 32 * j * C::kRawRow, from[j], i * 128, left);
            if (ch == 7) copy(to + 32 * j * C::kRawRow + 16, from[j], i * 128 + 16, left - 16);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (i < L) continue;
        const int n = i - L, s = n % C::kStages;
        asm volatile("cp.async.wait_group %0;" ::"n"(L) : "memory");
        __syncwarp();  // a row's nine vectors are one warp's
        wait(empty(s), ((n / C::kStages) & 1) ^ 1);
        const uint8_t* raw = mem + raws + n % C::kRaws * C::kRaw;
        uint8_t* at = mem + s * C::kStage + place;
#pragma unroll
        for (int j = 0; j < P; ++j) {
          if (!here(j)) continue;
          const uint4* v = reinterpret_cast<const uint4*>(raw + 32 * j * C::kRawRow);
          *reinterpret_cast<uint4*>(at + 32 * j * 128) = shift_across(v[0], v[1], mis[j]);
        }
        give(n);
      }
    }
  } else {
    for (int i = 0; i < steps; ++i) {
      const int s = i % C::kStages;
      wait(full(s), (i / C::kStages) & 1);
      tc_fence_after();
      if (lane == 0 && !*abort_flag) {
        const uint32_t at = base_addr + s * C::kStage;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_16bit<T, C::NR>(tmem, smem_desc(at) + 2 * k, smem_desc(at + kRows * 128) + 2 * k,
                              i > 0 || k > 0);
        mma_commit(empty(s));
      }
      __syncwarp();
    }
    if (lane == 0) mma_commit(done);
    __syncwarp();
  }
  // all products have ended; their operands' place takes the sums
  if (!mbar_wait(done, 0)) {
    atomicExch(err, 1);
    *abort_flag = 1;
  }
  tc_fence_after();
  __syncthreads();
  float* part = reinterpret_cast<float*>(mem);
  if (warp < 4) {
    float* row = part + (32 * warp + lane) * R;
#pragma unroll
    for (int c = 0; c < R; c += 32) {
      float v[32];
      tmem_ld32(tmem + (uint32_t(32 * warp) << 16) + uint32_t(c), v);
#pragma unroll
      for (int j = 0; j < 32 && c + j < R; j += 4)
        *reinterpret_cast<float4*>(row + c + j) =
            steps > 0 ? make_float4(v[j], v[j + 1], v[j + 2], v[j + 3])
                      : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kLoadWarps) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::kTmem)
                 : "memory");
  }
  join_parts<R, kShrinkThreads>(a, part, t.count, t.first);
}

template <class T, int R, bool ALIGNED>
int launch_shrink(const AdapterArgs& a, int64_t tiles, cudaStream_t s) {
  using C = ShrinkCfg<R, ALIGNED>;
  int* err = nullptr;
  IVFPQ_TRY(device_status_word(&err));
  auto kern = adapter_shrink_wide_kernel<T, R, ALIGNED>;
  IVFPQ_TRY(set_dynamic_smem(kern, C::kTotal));
  const int64_t y = std::min<int64_t>(tiles, 65535);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(a.splits), unsigned(y), unsigned(ceil_div(tiles, y)));
  cfg.blockDim = dim3(kShrinkThreads);
  cfg.dynamicSmemBytes = C::kTotal;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = unsigned(a.splits);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a, err));
  IVFPQ_LAUNCHED_K(kern, C::kTotal, kShrinkThreads);
  return IVFPQ_OK;
}
template <class T, bool ALIGNED>
int launch_shrink_rank(const AdapterArgs& a, int64_t tiles, cudaStream_t s) {
  switch (a.pitch) {
    case 8: return launch_shrink<T, 8, ALIGNED>(a, tiles, s);
    case 16: return launch_shrink<T, 16, ALIGNED>(a, tiles, s);
    case 32: return launch_shrink<T, 32, ALIGNED>(a, tiles, s);
    case 64: return launch_shrink<T, 64, ALIGNED>(a, tiles, s);
    default: return launch_shrink<T, 128, ALIGNED>(a, tiles, s);
  }
}

// ---- out = base + scale h B^T ----------------------------------------------------------
// A run of units of one tile.
struct Segment {
  Tile tile;
  int64_t chunk;  // first column chunk
  int units;
};

// VEC: rows of base and out are whole vectors on 16-byte boundaries. Others are copied
// in words, from the word that a row's first column lies in: a 16-bit row that starts
// between two words lies half a word further on in shared memory, too, and its thread
// moves the columns while it adds. (7199 x 6040 fp16, rank 24: 38 us; 6038 or 6037: 54 us.)
template <class T, class O, int KC, bool VEC>
__global__ void __launch_bounds__(kThreads, 1)
    adapter_expand_wide_kernel(const __grid_constant__ CUtensorMap map_b, const AdapterArgs a,
                               int* err) {
  using C = Cfg<T, O, KC>;
  constexpr int CN = C::CN;
  extern __shared__ uint8_t wide_raw[];
  __shared__ float up[kRows];
  const uint32_t raw = smem_u32(wide_raw);
  const uint32_t base_addr = (raw + 1023u) & ~1023u;
  uint8_t* mem = wide_raw + (base_addr - raw);
  const uint32_t s_a = base_addr, s_b = s_a + C::kA;
  uint8_t* buf = mem + C::kA + C::NB * C::kB;
  const uint32_t bars = s_b + C::NB * C::kB + C::kBuf;
  auto b_full = [&](int i) { return bars + 8 * i; };
  auto b_empty = [&](int i) { return bars + 8 * (C::NB + i); };
  auto acc_full = [&](int i) { return bars + 8 * (2 * C::NB + i); };
  auto acc_empty = [&](int i) { return bars + 8 * (2 * C::NB + kGroups + i); };
  uint8_t* tail = mem + (bars - base_addr) + 8 * (2 * C::NB + 2 * kGroups);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NB; ++i) {
      mbar_init(b_full(i), 1);
      mbar_init(b_empty(i), 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), kGroupWarps);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Every wait is bounded. One that runs out sets the flag; from then on nothing
  // waits or is issued, but all roles go through their loops to the end, so that
  // the barriers among them stay matched.
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (*abort_flag) return;
    if (!mbar_wait(bar, parity)) {
      atomicExch(err, 1);
      *abort_flag = 1;
    }
  };
  grid_wait();
  const int64_t chunks = (a.n + CN - 1) / CN, units = int64_t(*a.ntiles) * chunks;
  const int64_t u0 = units * blockIdx.x / gridDim.x;
  const int64_t u1 = units * (int64_t(blockIdx.x) + 1) / gridDim.x;
  const bool in_place = a.base == a.out;
  // The next run of units of one tile that has something to do; units 0 at the end.
  auto next = [&](int64_t& u) {
    Segment g;
    g.units = 0;
    while (u < u1 && g.units == 0) {
      const int64_t i = u / chunks;
      g.chunk = u - i * chunks;
      g.units = int(min(chunks - g.chunk, u1 - u));
      u += g.units;
      const int4 t = a.tiles[i];
      g.tile = {t.x, t.y, t.z};
      if (t.x < 0 && in_place) g.units = 0;  // nothing changes
    }
    return g;
  };
  auto row_bytes = [&](int64_t chunk) {
    return int(min(int64_t(CN), a.n - chunk * CN)) * int(sizeof(O));
  };
  const int ksteps = (a.rank + 15) / 16;
  int64_t u = u0;
  int it = 0;  // units so far: accumulator it % kGroups, rows of group it % GROUPS

  if (warp == 0) {
    // ---- B ----
    int jt = 0;
    for (Segment g = next(u); g.units > 0; g = next(u)) {
      if (g.tile.adapter < 0) continue;
      for (int k = 0; k < g.units; ++k, ++jt) {
        const int sb = jt % C::NB;
        wait(b_empty(sb), ((jt / C::NB) & 1) ^ 1);
        if (lane == 0 && !*abort_flag) {
          mbar_expect_tx(b_full(sb), C::kB);
          for (int kc = 0; kc < KC; ++kc)
            tma_load_3d(s_b + sb * C::kB + kc * CN * 128, &map_b, kc * 64,
                        int((g.chunk + k) * CN), g.tile.adapter, b_full(sb));
        }
        __syncwarp();
      }
    }
    // copies still on their way land before the block ends
    for (int j = max(0, jt - C::NB); j < jt; ++j)
      mbar_wait(b_full(j % C::NB), (j / C::NB) & 1, *abort_flag ? 1u << 16 : kSpinLimit);
  } else if (warp == 1) {
    // ---- products ----
    int jt = 0;
    for (Segment g = next(u); g.units > 0; g = next(u)) {
      const bool some = g.tile.adapter >= 0;
      if (some) named_barrier(1, kEpiThreads + 32);  // A is there
      for (int k = 0; k < g.units; ++k, ++it) {
        const int ab = it % kGroups;
        wait(acc_empty(ab), ((it / kGroups) & 1) ^ 1);
        if (some) {
          const int sb = jt % C::NB;
          wait(b_full(sb), (jt / C::NB) & 1);
          ++jt;
          tc_fence_after();
          if (lane == 0 && !*abort_flag) {
            const uint32_t d = tmem + uint32_t(ab * CN);
            uint32_t acc = 0;
#pragma unroll 1
            for (int n = C::TERMS - 1; n >= 0; --n)  // the small terms first
#pragma unroll 1
              for (int ks = 0; ks < ksteps; ++ks) {
                const uint64_t da =
                    smem_desc(s_a + uint32_t((n * KC + ks / 4) * kRows * 128 + (ks % 4) * 32));
                const uint64_t db =
                    smem_desc(s_b + uint32_t(sb * C::kB + (ks / 4) * CN * 128 + (ks % 4) * 32));
                mma_16bit<T, CN>(d, da, db, acc);
                acc = 1;
              }
            mma_commit(b_empty(sb));
            mma_commit(acc_full(ab));
          }
        } else if (lane == 0 && !*abort_flag) {
          mbar_arrive(acc_full(ab));
        }
        __syncwarp();
      }
    }
    // the last products have ended before TMEM and the operands go
    for (int j = max(0, it - kGroups); j < it; ++j)
      mbar_wait(acc_full(j % kGroups), (j / kGroups) & 1, *abort_flag ? 1u << 16 : kSpinLimit);
  } else {
    // ---- h into A, then accumulators and base rows into output rows ----
    const int group = (warp - 2) / kGroupWarps, lg = warp & 3, row = 32 * lg + lane;
    const int e = threadIdx.x - 64;  // 0 .. kEpiThreads - 1
    const bool works = group < C::GROUPS;
    // 32 rows of kRowBytes; the 16-byte pieces of row r are swapped around by r mod 8
    uint8_t* mine = buf + (works ? (group * kGroupWarps + lg) * 32 * kRowBytes : 0);
    auto piece = [&](int r, int c) { return mine + r * kRowBytes + ((c ^ (r & 7)) * 16); };
    const O* base = static_cast<const O*>(a.base);
    // copies: this lane has piece ch of rows sub, sub + 2, ..
    const int sub = lane >> 4, ch = lane & 15;
    uint8_t* copy = mine + sub * kRowBytes;
    int swap[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) swap[j] = (ch ^ (2 * j + sub)) * 16;
    using Pitch = std::conditional_t<VEC, uint32_t, uint64_t>;  // VEC: below 2^32
    const Pitch base_pitch = Pitch(a.ldb * int64_t(sizeof(O)));
    const Pitch out_pitch = Pitch(a.ldo * int64_t(sizeof(O)));
    // not VEC: this lane's words of row i are here and 128 bytes on; `beyond` is the word
    // behind a unit's 64 of the lane's own row, where its columns end in there
    auto word = [&](int i) {
      return mine + i * kRowBytes + (((lane >> 2) ^ (i & 7)) * 16) + (lane & 3) * 4;
    };
    constexpr bool kHalves = !VEC && sizeof(O) == 2;
    uint32_t beyond = 0;
    auto token_here = [&](const Segment& g) {
      return g.units > 0 && row < g.tile.count ? uint32_t(token_of(a, g.tile.first + row)) : 0u;
    };
    // the coming unit of this group: segment, unit in it, and the token of this lane's row
    int64_t fu = u0;
    Segment fg;
    fg.units = 0;
    int fk = works ? group : INT_MAX;
    uint32_t ftok = 0;
    auto settle = [&]() {  // fk may have passed the segment's end
      while (works && fk >= fg.units) {
        fk -= fg.units;
        fg = next(fu);
        if (fg.units == 0) {
          fk = INT_MAX;
          return;
        }
        ftok = token_here(fg);
      }
    };
    auto fetch = [&]() {
      settle();
      if (!VEC && base && works && fk != INT_MAX) {
        const int64_t chunk = fg.chunk + fk;
        const int bytes = row_bytes(chunk), nrows = fg.tile.count - 32 * lg;
        const uintptr_t from = reinterpret_cast<uintptr_t>(base + chunk * CN);
        auto copy_word = [](uint8_t* to, uintptr_t p) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)),
                       "l"(reinterpret_cast<const void*>(p))
                       : "memory");
        };
        if (nrows >= 32 && bytes == kRowBytes) {
#pragma unroll 8
          for (int i = 0; i < 32; ++i) {
            const uintptr_t p = from + __shfl_sync(kFullMask, ftok, i) * base_pitch;
            const uintptr_t w = (p & ~uintptr_t(3)) + 4 * lane;
            copy_word(word(i), w);
            copy_word(word(i) + 128, w + 128);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < min(32, nrows); ++i) {
            const uintptr_t p = from + __shfl_sync(kFullMask, ftok, i) * base_pitch;
            const uintptr_t w = (p & ~uintptr_t(3)) + 4 * lane;
            const int end = bytes + int(p & 3);  // words that begin before are asked for
            if (4 * lane < end) copy_word(word(i), w);
            if (4 * lane + 128 < end) copy_word(word(i) + 128, w + 128);
          }
        }
        if constexpr (kHalves) {
          const uintptr_t p = from + ftok * base_pitch;
          if (lane < nrows && (p & 2) && bytes == kRowBytes)
            beyond = *reinterpret_cast<const uint32_t*>(p - 2 + kRowBytes);
        }
      }
      if (VEC && base && works && fk != INT_MAX) {
        const int64_t chunk = fg.chunk + fk;
        const int bytes = row_bytes(chunk), nrows = fg.tile.count - 32 * lg;
        const char* from = reinterpret_cast<const char*>(base + chunk * CN) + ch * 16;
        const uint32_t to = smem_u32(copy);
        if (nrows >= 32 && bytes == kRowBytes) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t t = __shfl_sync(kFullMask, ftok, 2 * i + sub);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             to + 2 * i * kRowBytes + swap[i & 3]),
                         "l"(from + uint64_t(t) * base_pitch)
                         : "memory");
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < 16; ++i) {
            const int r = 2 * i + sub;
            const uint32_t t = __shfl_sync(kFullMask, ftok, r);
            if (r < nrows && ch * 16 < bytes)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                               smem_u32(piece(r, ch))),
                           "l"(from + uint64_t(t) * base_pitch)
                           : "memory");
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (fk != INT_MAX) fk += C::GROUPS;
    };
    fetch();
    for (Segment g = next(u); g.units > 0; g = next(u)) {
      const bool some = g.tile.adapter >= 0;
      if (some) {
        named_barrier(2, kEpiThreads);  // all groups have seen the last products of the old A
        const float scale = a.scales ? a.scales[g.tile.adapter] : 1.f;
        // threads of a row: chunks of 8 columns p, p + P, ..
        constexpr int P = kEpiThreads / kRows;
        const int r = e / P, p = e % P;
        const float* h = a.h + int64_t(g.tile.first + r) * a.pitch;
        constexpr int J = 8 * KC / P;
        float v[J][8], top = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int k = (p + P * j) * 8;
          float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
          if (r < g.tile.count && k < a.pitch) {
            lo = *reinterpret_cast<const float4*>(h + k);
            hi = *reinterpret_cast<const float4*>(h + k + 4);
          }
          const float w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            v[j][x] = within_rank(a, k + x, w[x]) * scale;
            top = fmaxf(top, magnitude(v[j][x]));
          }
        }
        if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
          for (int d = 1; d < P; d *= 2) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, d));
          const float2 f = fp16_range(top);
#pragma unroll
          for (int j = 0; j < J; ++j)
#pragma unroll
            for (int x = 0; x < 8; ++x) v[j][x] *= f.x;
          if (p == 0) up[r] = f.y;
        }
#pragma unroll
        for (int n = 0; n < C::TERMS; ++n)
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const int cc = p + P * j;  // chunk of 16 bytes of the row
            float f[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) f[x] = term<T>(v[j][x]);
            *reinterpret_cast<uint4*>(mem + (n * KC + cc / 8) * kRows * 128 + r * 128 +
                                      ((cc % 8) ^ (r & 7)) * 16) = pack_vec<T>(f);
          }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        named_barrier(1, kEpiThreads + 32);
      }
      const uint32_t tok = token_here(g);
      const int nrows = min(32, g.tile.count - 32 * lg);
      float f = 1.f;
      if constexpr (std::is_same<T, __half>::value)
        if (some) f = up[row];
      // this group's units of the segment: every GROUPS-th of all units
      const int first = (group + C::GROUPS - it % C::GROUPS) % C::GROUPS;
      for (int k = works ? first : g.units; k < g.units; k += C::GROUPS) {
        const int ab = (it + k) % kGroups;
        const int64_t chunk = g.chunk + k;
        const int bytes = row_bytes(chunk);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        wait(acc_full(ab), ((it + k) / kGroups) & 1);
        __syncwarp();
        tc_fence_after();
        uint8_t* here = mine + lane * kRowBytes;
        const int turn = (lane & 7) * 16;
        // bits by which the row's words are off its columns, read and written
        const uintptr_t out_row = reinterpret_cast<uintptr_t>(static_cast<O*>(a.out) + chunk * CN) +
                                  tok * out_pitch;
        const uint32_t in_off =
            kHalves ? uint32_t((reinterpret_cast<uintptr_t>(base) + tok * base_pitch) & 2) * 8 : 0;
        const uint32_t out_off = kHalves ? uint32_t(out_row & 2) * 8 : 0;
        uint32_t first = 0, before = 0;  // the first two columns, the last two so far
        uint4 ahead;
        if (kHalves && base) ahead = *reinterpret_cast<const uint4*>(here + turn);
#pragma unroll
        for (int c = 0; c < CN; c += 32) {
          uint32_t d[32];
          if (some) {
            tmem_ld32_nowait(tmem + (uint32_t(32 * lg) << 16) + uint32_t(ab * CN + c), d);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) d[x] = 0;
          }
          constexpr int N = Span<O>::N;
#pragma unroll
          for (int q = 0; q < 32 / N; ++q) {
            uint4* at = reinterpret_cast<uint4*>(here + (((c / N + q) * 16) ^ turn));
            float w[N];
#pragma unroll
            for (int x = 0; x < N; ++x) w[x] = __uint_as_float(d[q * N + x]);
            if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
              for (int x = 0; x < N; ++x) w[x] *= f;
            }
            if (base) {
              float v[N];
              if constexpr (kHalves) {
                const int next = c / N + q + 1;
                uint4 h = ahead;
                ahead = next * 16 < kRowBytes
                            ? *reinterpret_cast<const uint4*>(here + ((next * 16) ^ turn))
                            : make_uint4(beyond, 0, 0, 0);
                h.x = __funnelshift_r(h.x, h.y, in_off);
                h.y = __funnelshift_r(h.y, h.z, in_off);
                h.z = __funnelshift_r(h.z, h.w, in_off);
                h.w = __funnelshift_r(h.w, ahead.x, in_off);
                unpack_vec<O>(h, v);
              } else {
                unpack_vec<O>(*at, v);
              }
#pragma unroll
              for (int x = 0; x < N; x += 2)
                unpair(add2(pair(v[x], v[x + 1]), pair(w[x], w[x + 1])), w[x], w[x + 1]);
            }
            uint4 o = pack_vec<O>(w);
            if constexpr (kHalves) {
              if (c + q == 0) first = o.x;
              const uint32_t last = o.w;
              o.w = __funnelshift_l(o.z, o.w, out_off);
              o.z = __funnelshift_l(o.y, o.z, out_off);
              o.y = __funnelshift_l(o.x, o.y, out_off);
              o.x = __funnelshift_l(before, o.x, out_off);
              before = last;
            }
            *at = o;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(ab));
        if (!__any_sync(kFullMask, *abort_flag)) {
          if constexpr (VEC) {
            char* to = reinterpret_cast<char*>(static_cast<O*>(a.out) + chunk * CN) + ch * 16;
            if (nrows == 32 && bytes == kRowBytes) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint32_t t = __shfl_sync(kFullMask, tok, 2 * i + sub);
                *reinterpret_cast<uint4*>(to + uint64_t(t) * out_pitch) =
                    *reinterpret_cast<const uint4*>(copy + 2 * i * kRowBytes + swap[i & 3]);
              }
            } else {
#pragma unroll 1
              for (int i = 0; i < 16; ++i) {
                const int r = 2 * i + sub;
                const uint32_t t = __shfl_sync(kFullMask, tok, r);
                if (r < nrows && ch * 16 < bytes)
                  *reinterpret_cast<uint4*>(to + uint64_t(t) * out_pitch) =
                      *reinterpret_cast<const uint4*>(piece(r, ch));
              }
            }
          } else {
            const uintptr_t to = reinterpret_cast<uintptr_t>(static_cast<O*>(a.out) + chunk * CN);
            if (nrows == 32 && bytes == kRowBytes) {
#pragma unroll 8
              for (int i = 0; i < 32; ++i) {
                const uintptr_t p = to + __shfl_sync(kFullMask, tok, i) * out_pitch;
                uint32_t* w = reinterpret_cast<uint32_t*>((p & ~uintptr_t(3)) + 4 * lane);
                if (!kHalves || lane > 0 || !(p & 2))
                  *w = *reinterpret_cast<const uint32_t*>(word(i));
                w[32] = *reinterpret_cast<const uint32_t*>(word(i) + 128);
              }
            } else {
#pragma unroll 1
              for (int i = 0; i < nrows; ++i) {
                const uintptr_t p = to + __shfl_sync(kFullMask, tok, i) * out_pitch;
                uint32_t* w = reinterpret_cast<uint32_t*>((p & ~uintptr_t(3)) + 4 * lane);
                const int end = bytes + int(p & 3);  // whole words of the row
                if (4 * lane + 4 <= end && (lane > 0 || !(p & 3)))
                  *w = *reinterpret_cast<const uint32_t*>(word(i));
                if (4 * lane + 132 <= end)
                  w[32] = *reinterpret_cast<const uint32_t*>(word(i) + 128);
              }
            }
            if constexpr (kHalves) {  // a row's first and last column in a word with others
              const int end = bytes + int(out_row & 2);
              if (lane < nrows && (out_row & 2))
                *reinterpret_cast<uint16_t*>(out_row) = uint16_t(first);
              if (lane < nrows && (end & 2)) {
                const uint32_t w = end / 4 * 4 == kRowBytes
                                       ? before >> 16
                                       : *reinterpret_cast<const uint32_t*>(
                                             piece(lane, end / 16) + end % 16 / 4 * 4);
                *reinterpret_cast<uint16_t*>(out_row + bytes - 2) = uint16_t(w);
              }
            }
          }
        }
        __syncwarp();
        fetch();
      }
      it += g.units;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::kTmem)
                 : "memory");
  }
}

template <class T, class O, int KC, bool VEC>
int launch(const AdapterArgs& a, cudaStream_t s) {
  using C = Cfg<T, O, KC>;
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  IVFPQ_TRY(tensor_map_encoder(&enc));
  CUtensorMap map;
  const cuuint64_t dims[3] = {cuuint64_t(a.rank), cuuint64_t(a.n),
                              cuuint64_t(std::max(a.adapters, 1))};
  const cuuint64_t strides[2] = {cuuint64_t(a.rank) * 2, cuuint64_t(a.rank) * 2 * cuuint64_t(a.n)};
  const cuuint32_t box[3] = {64, cuuint32_t(C::CN), 1}, estr[3] = {1, 1, 1};
  const CUresult r = enc(
      &map,
      std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
      3, const_cast<void*>(a.b), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for %d adapters of %lld x %d", int(r), a.adapters,
              (long long)a.n, a.rank);
    return IVFPQ_ERR_CUDA;
  }
  int* err = nullptr;
  IVFPQ_TRY(device_status_word(&err));
  auto kern = adapter_expand_wide_kernel<T, O, KC, VEC>;
  IVFPQ_TRY(set_dynamic_smem(kern, C::kTotal));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(num_sms()));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kTotal;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, map, a, err));
  IVFPQ_LAUNCHED_K(kern, C::kTotal, kThreads);
  return IVFPQ_OK;
}
template <class T, class O>
int launch_rank(const AdapterArgs& a, cudaStream_t s) {
  // 32-bit row pitches in bytes for whole rows
  const int64_t limit = (int64_t(1) << 32) / int64_t(sizeof(O));
  if (whole_rows<O>(a) && a.ldb < limit && a.ldo < limit)
    return a.rank <= 64 ? launch<T, O, 1, true>(a, s) : launch<T, O, 2, true>(a, s);
  return a.rank <= 64 ? launch<T, O, 1, false>(a, s) : launch<T, O, 2, false>(a, s);
}

}  // namespace

int adapter_shrink_wide(const AdapterArgs& a, int dtype, int64_t tiles, cudaStream_t s) {
  const bool aligned = a.cols % 8 == 0 && a.ldx % 8 == 0 &&
                       reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.a) % 16 == 0;
  if (dtype == IVFPQ_F16)
    return aligned ? launch_shrink_rank<__half, true>(a, tiles, s)
                   : launch_shrink_rank<__half, false>(a, tiles, s);
  return aligned ? launch_shrink_rank<__nv_bfloat16, true>(a, tiles, s)
                 : launch_shrink_rank<__nv_bfloat16, false>(a, tiles, s);
}
int adapter_expand_wide(const AdapterArgs& a, int dtype, int out_dtype, cudaStream_t s) {
  if (dtype == IVFPQ_F16)
    return out_dtype == IVFPQ_F32 ? launch_rank<__half, float>(a, s)
                                  : launch_rank<__half, __half>(a, s);
  return out_dtype == IVFPQ_F32 ? launch_rank<__nv_bfloat16, float>(a, s)
                                : launch_rank<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace ivfpq
