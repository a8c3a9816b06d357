// fp4_product / fp4_linear: out[i, j] = ga gb sum_t a[i, t] b[j, t] over packed
// 4-bit block-scaled rows (layout: fp4.cuh), on the block-scaled tensor-core
// product of the 5th generation (tcgen05.mma, kind::mxf4nvf4: E2M1 elements
// with an E8M0 scale per 32 or an E4M3 scale per 16, fp32 accumulation).
//
// The table b is the instruction's 128-row operand and the rows of a its
// columns, so an accumulator lane holds one column of out and a warp's store
// covers 32 consecutive columns of one row of out, whatever their alignment;
// and a few rows of a cost a narrow instruction instead of a padded one.
//
// One CTA per (128 columns of out, T rows of out, slice of K), 6 warps:
//  * warp 0, one thread: TMA producer. A stage is 256 columns of K (128 where
//    that is all of K): 128 rows of b and T rows of a and their scale tiles,
//    which are contiguous;
//  * warp 1: TMEM; one thread copies a stage's scale tiles to TMEM and issues
//    one product per 64 columns. Each stage has TMEM columns of its own for
//    its scales: they are rewritten only after the stage's products committed;
//  * warps 2..5: epilogue, a TMEM lane each.
// What bounds it is reading b: 16 KB of codes per stage from memory against 2 KB
// of a, and products of a fraction of that time. Three or four stages of two
// CTAs per SM keep 160 KB per SM in flight. After fp4_linear's quantisation it
// starts while that kernel runs (griddepcontrol) and has its first stages of b
// on their way before a is complete. Measured with the quantisation, on the
// device: one token, 32000 x 4096 MXFP4, 14.8 us (70 MB: 10.4 us at the measured
// copy rate); 37 tokens, 16384 x 4096 NVFP4, 13.7 us (39 MB, 5.9 us). A CTA of
// short K sets up barriers and TMEM for one stage: 16 x 100003 x 128 to fp32 7.2 us
// (2.0 us for the bytes), 16 x 10,000,000 x 128 397 us (197 us).
//
// A cluster splits K between its CTAs when there are few tiles; the partial
// sums are joined in rank order through distributed shared memory. Shared
// memory lets at most two CTAs of a variant that may be split share an SM, and
// two always fit its 512 TMEM columns: no CTA of a cluster waits for TMEM that
// another cluster holds while it waits itself. (Short K is never split.)
#include <algorithm>

#include "fp4_mma.cuh"

namespace ivfpq {

int fp4_quantize_device(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int fmt,
                        const float* tensor_scale, uint8_t* codes, uint8_t* scales,
                        cudaStream_t s);

int fp4_code_map(CUtensorMap* m, const uint8_t* p, int64_t rows, int64_t pitch, int kb,
                 int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  IVFPQ_TRY(tensor_map_encoder(&enc));
  cuuint64_t dims[2] = {cuuint64_t(pitch), cuuint64_t(rows)};
  cuuint64_t strides[1] = {cuuint64_t(pitch)};
  cuuint32_t box[2] = {cuuint32_t(kb), cuuint32_t(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   kb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for %lld rows of %lld code bytes", int(r),
              (long long)rows, (long long)pitch);
    return IVFPQ_ERR_CUDA;
  }
  return IVFPQ_OK;
}

namespace {

constexpr int kThreads = 192;

template <int FMT, int T, int KB>
struct Cfg {
  static constexpr int KE = 2 * KB;  // K columns per stage
  static constexpr int kTilesPerStage = KE / (FMT == IVFPQ_MXFP4 ? 128 : 64);  // scale tiles
  static constexpr int kSf = kTilesPerStage * 512;
  static constexpr int kB = BN * KB;
  static constexpr int kA = T * KB;
  static constexpr int kStage = kB + kA + 2 * kSf;
  static constexpr int kStages = KB < 128 ? 1 : T <= 32 ? 4 : 3;  // short K is one stage
  static constexpr int kBars = 256;
  static constexpr int kTotal = kStages * kStage + kBars + 1024;
  // TMEM: the accumulator, then each stage's scales of b and of a
  static constexpr int kSfCols = 2 * 4 * kTilesPerStage;
  static constexpr int kAccCols = T < 32 ? 32 : T;
  static constexpr int kUsed = kAccCols + kStages * kSfCols;
  static constexpr int kTmem = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : 256;
  static_assert(kUsed <= 256 && (KB < 128 || kTotal > 76 * 1024),
                "two CTAs that may wait for others per SM, and their TMEM fits");
};

// grid (column tiles, row tiles, K slices); the cluster is the K slices.
template <int FMT, int T, int KB>
__global__ void __launch_bounds__(kThreads)
fp4_product_kernel(const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_a, const ProdArgs p) {
  using C = Cfg<FMT, T, KB>;
  constexpr int KE = C::KE;
  extern __shared__ uint8_t fp4_smem_raw[];
  const uint32_t raw = smem_u32(fp4_smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = fp4_smem_raw + (base - raw);
  const uint32_t bars = base + C::kStages * C::kStage;
  auto s_b = [&](int s) { return base + s * (C::kB + C::kA); };
  auto s_a = [&](int s) { return base + s * (C::kB + C::kA) + C::kB; };
  const uint32_t sf0 = base + C::kStages * (C::kB + C::kA);
  auto s_sfb = [&](int s) { return sf0 + s * 2 * C::kSf; };
  auto s_sfa = [&](int s) { return sf0 + s * 2 * C::kSf + C::kSf; };
  auto bar_full = [&](int s) { return bars + 8 * s; };
  auto bar_empty = [&](int s) { return bars + 8 * (C::kStages + s); };
  const uint32_t bar_acc = bars + 16 * C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 16 * C::kStages + 8);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(gbase + (bars - base) + 16 * C::kStages + 16);

  const int warp = __shfl_sync(kFullMask, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int nslice = gridDim.z;
  const int nk = (p.kp + KE - 1) / KE;
  const int k_lo = int(int64_t(nk) * blockIdx.z / nslice);
  const int k_hi = int(int64_t(nk) * (blockIdx.z + 1) / nslice);
  const int n0 = blockIdx.x * BN;
  const int m0 = blockIdx.y * T;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_acc, 1);
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
  auto fail = [&]() {
    atomicExch(p.err, 1);
    *abort_flag = 1;
  };

  if (warp == 0 && lane == 0) {
    // ---- TMA producer. The first stages' rows of b are asked for before the
    // kernel that writes a has ended (overlapping launch) ----
    const uint8_t* sb = p.b_scales + int64_t(blockIdx.x) * p.ntile * 512;
    const uint8_t* sa = p.a_scales + int64_t(m0 >> 7) * p.ntile * 512;
    auto sf_bytes = [&](int kc) {
      return uint32_t(min(C::kTilesPerStage, p.ntile - kc * C::kTilesPerStage)) * 512;
    };
    auto load_b = [&](int kc, int s) {
      mbar_expect_tx(bar_full(s), C::kB + C::kA + 2 * sf_bytes(kc));
      tma_load_2d(s_b(s), &map_b, kc * KB, n0, bar_full(s));
      bulk_load(s_sfb(s), sb + int64_t(kc) * C::kTilesPerStage * 512, sf_bytes(kc), bar_full(s));
    };
    auto load_a = [&](int kc, int s) {
      tma_load_2d(s_a(s), &map_a, kc * KB, m0, bar_full(s));
      bulk_load(s_sfa(s), sa + int64_t(kc) * C::kTilesPerStage * 512, sf_bytes(kc), bar_full(s));
    };
    const int early = min(C::kStages, k_hi - k_lo);
    for (int j = 0; j < early; ++j) load_b(k_lo + j, j);
    grid_wait();
    for (int j = 0; j < early; ++j) load_a(k_lo + j, j);
    int it = early;
    for (int kc = k_lo + early; kc < k_hi && !*abort_flag; ++kc, ++it) {
      const int s = it % C::kStages;
      if (!mbar_wait(bar_empty(s), ((it / C::kStages) & 1) ^ 1)) {
        fail();
        break;
      }
      load_b(kc, s);
      load_a(kc, s);
    }
    // copies still in flight land before the CTA ends
    for (int j = max(0, it - C::kStages); j < it; ++j)
      mbar_wait(bar_full(j % C::kStages), (j / C::kStages) & 1);
  } else if (warp == 1) {
    // ---- scale copies and products: the whole warp runs, one lane issues ----
    const uint32_t el = elect_one();
    const uint64_t d_b = code_desc<KB>(s_b(0)), d_a = code_desc<KB>(s_a(0));
    const uint64_t d_sf = scale_desc(s_sfb(0));
    uint32_t s = 0, phase = 0;
    for (int kc = k_lo; kc < k_hi && !*abort_flag; ++kc) {
      if (!mbar_wait(bar_full(s), phase)) {
        fail();
        break;
      }
      tc_fence_after();
      const int tiles = min(C::kTilesPerStage, p.ntile - kc * C::kTilesPerStage);
      const uint32_t tsb = tmem + C::kAccCols + s * C::kSfCols;
      const uint32_t tsa = tsb + C::kSfCols / 2;
      const uint64_t sd = d_sf + s * uint32_t((2 * C::kSf) >> 4);
#pragma unroll
      for (int t = 0; t < C::kTilesPerStage; ++t) {
        if (t < tiles) {
          scale_copy<1>(tsb + 4 * t, sd + 32 * t, el);
          scale_copy<1>(tsa + 4 * t, sd + 32 * t + C::kSf / 16, el);
        }
      }
      const uint64_t db = d_b + s * uint32_t((C::kB + C::kA) >> 4);
      const uint64_t da = d_a + s * uint32_t((C::kB + C::kA) >> 4);
      const int steps = min(KB / 32, (p.kp - kc * KE + 63) / 64);
#pragma unroll
      for (int j = 0; j < KB / 32; ++j) {
        if (j < steps) {
          const int t = FMT == IVFPQ_MXFP4 ? j >> 1 : j;
          const uint32_t id = FMT == IVFPQ_MXFP4 ? uint32_t(j & 1) * 2 : 0u;
          mma_fp4<FMT, 1>(tmem, db + 2 * j, da + 2 * j, fp4_idesc<FMT, T, 1>(id), tsb + 4 * t,
                       tsa + 4 * t, kc > k_lo || j > 0, el);
        }
      }
      mma_commit_el(bar_empty(s), el);
      if (++s == C::kStages) {
        s = 0;
        phase ^= 1;
      }
    }
    // also the end of every product issued before an early exit
    mma_commit_el(bar_acc, el);
    if (!mbar_wait(bar_acc, 0)) fail();
  } else if (warp >= 2) {
    if (!mbar_wait(bar_acc, 0)) fail();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  grid_wait();
  const float alpha = (p.a_ts ? __ldg(p.a_ts) : 1.f) * (p.b_ts ? __ldg(p.b_ts) : 1.f);
  const bool ok = !*abort_flag;
  // ---- epilogue: warp w of 2..5 reads TMEM lanes 32 * (w % 4) .. +32 ----
  if (nslice == 1) {
    if (warp >= 2 && ok) {
      const int lg = warp & 3;
      const int64_t col = n0 + 32 * lg + lane;
#pragma unroll 1
      for (int c = 0; c < C::kAccCols; c += 32) {
        float v[32];
        tmem_ld32(tmem + (uint32_t(32 * lg) << 16) + uint32_t(c), v);
        if (col < p.n) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < T && m0 + c + j < p.m)
              store_out(p.out, (m0 + c + j) * p.ldo + col, p.dtype, v[j] * alpha);
        }
      }
    }
  } else {
    // partial sums to this CTA's shared memory ([T][128]; every stage has been
    // consumed), then each rank joins its share, four columns of a row at a
    // time, in rank order
    float* part = reinterpret_cast<float*>(gbase);
    if (warp >= 2) {
      const int lg = warp & 3;
#pragma unroll 1
      for (int c = 0; c < C::kAccCols; c += 32) {
        float v[32];
        tmem_ld32(tmem + (uint32_t(32 * lg) << 16) + uint32_t(c), v);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c + j < T) part[(c + j) * BN + 32 * lg + lane] = v[j];
      }
    }
    cluster_sync();
    const int rank = int(cluster_rank());
    const int quads = int(min(int64_t(T), p.m - m0)) * (BN / 4);
    for (int i = rank * kThreads + threadIdx.x; i < quads; i += nslice * kThreads) {
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < nslice) v[r] = ld_cluster4(map_rank(base + 16u * uint32_t(i), uint32_t(r)));
      float4 t = v[0];
#pragma unroll
      for (int r = 1; r < 8; ++r) {
        if (r < nslice) {
          t.x += v[r].x;
          t.y += v[r].y;
          t.z += v[r].z;
          t.w += v[r].w;
        }
      }
      const int64_t col = n0 + 4 * (i % (BN / 4)), at = (m0 + i / (BN / 4)) * p.ldo + col;
      if (ok) {
        if (col < p.n) store_out(p.out, at, p.dtype, t.x * alpha);
        if (col + 1 < p.n) store_out(p.out, at + 1, p.dtype, t.y * alpha);
        if (col + 2 < p.n) store_out(p.out, at + 2, p.dtype, t.z * alpha);
        if (col + 3 < p.n) store_out(p.out, at + 3, p.dtype, t.w * alpha);
      }
    }
    cluster_sync();
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

template <int FMT, int T, int KB>
int launch(const uint8_t* a, const uint8_t* b, const ProdArgs& p, cudaStream_t s) {
  using C = Cfg<FMT, T, KB>;
  constexpr int KE = C::KE;
  CUtensorMap mb, ma;
  IVFPQ_TRY(fp4_code_map(&mb, b, p.n, p.kp / 2, KB, BN));
  IVFPQ_TRY(fp4_code_map(&ma, a, p.m, p.kp / 2, KB, T));
  auto kern = fp4_product_kernel<FMT, T, KB>;
  IVFPQ_TRY(set_dynamic_smem(kern, C::kTotal));
  const int64_t tiles_n = ceil_div(p.n, BN), tiles_m = ceil_div(p.m, T);
  const int64_t nk = ceil_div(p.kp, KE);
  // K slices while the tiles alone leave SMs idle and a slice keeps two stages
  int slices = 1;
  while (slices < 8 && tiles_n * tiles_m * slices * 2 <= 2 * num_sms() && nk >= 4 * slices)
    slices *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(tiles_n), unsigned(tiles_m), unsigned(slices));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kTotal;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = unsigned(slices);
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.overlap ? 2 : 1;
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, mb, ma, p));
  IVFPQ_LAUNCHED_K(kern, C::kTotal, kThreads);
  return IVFPQ_OK;
}

template <int FMT, int KB>
int launch_fmt(const uint8_t* a, const uint8_t* b, const ProdArgs& p, cudaStream_t s) {
  // the narrowest instruction that holds all rows; a narrow one starts at row
  // 0 of its scale tile, so it is only taken where one row tile covers m
  if (p.m <= 16) return launch<FMT, 16, KB>(a, b, p, s);
  if (p.m <= 32) return launch<FMT, 32, KB>(a, b, p, s);
  if (p.m <= 64) return launch<FMT, 64, KB>(a, b, p, s);
  return launch<FMT, 128, KB>(a, b, p, s);
}

int product_device(const uint8_t* a, const uint8_t* a_scales, int64_t m, const uint8_t* b,
                   const uint8_t* b_scales, int64_t n, int64_t cols, int fmt, const float* a_ts,
                   const float* b_ts, void* out, int dtype, bool overlap, cudaStream_t s) {
  ProdArgs p{};
  p.overlap = overlap;
  p.a_scales = a_scales;
  p.b_scales = b_scales;
  p.a_ts = fmt == IVFPQ_NVFP4 ? a_ts : nullptr;
  p.b_ts = fmt == IVFPQ_NVFP4 ? b_ts : nullptr;
  p.out = out;
  p.ldo = n;
  p.m = m;
  p.n = n;
  p.kp = int(fp4_padded_cols(cols));
  p.ntile = int(fp4_scale_tiles(cols, fmt));
  p.dtype = dtype;
  IVFPQ_TRY(device_status_word(&p.err));
  // enough 128 x 128 tiles to keep every SM busy without splitting K
  if (m > 64 && ceil_div(n, BN) * ceil_div(m, 128) >= num_sms())
    return fp4_product_wide(a, b, p, fmt, s);
  if (p.kp <= kShortK)
    return fmt == IVFPQ_MXFP4 ? launch_fmt<IVFPQ_MXFP4, 64>(a, b, p, s)
                              : launch_fmt<IVFPQ_NVFP4, 64>(a, b, p, s);
  return fmt == IVFPQ_MXFP4 ? launch_fmt<IVFPQ_MXFP4, 128>(a, b, p, s)
                            : launch_fmt<IVFPQ_NVFP4, 128>(a, b, p, s);
}

int check_product(const char* fn, int64_t m, int64_t n, int64_t cols, int fmt, int dtype) {
  IVFPQ_REQUIRE(m >= 0 && m <= 65535 * int64_t(128), "%s: m=%lld outside [0, 8388480]", fn,
                (long long)m);
  IVFPQ_REQUIRE(n >= 0 && n < (int64_t(1) << 31) - 1024, "%s: n=%lld outside [0, 2^31 - 1024)", fn,
                (long long)n);
  IVFPQ_REQUIRE(cols >= 1 && cols <= (int64_t(1) << 24), "%s: cols=%lld outside [1, 2^24]", fn,
                (long long)cols);
  IVFPQ_REQUIRE(fmt == IVFPQ_MXFP4 || fmt == IVFPQ_NVFP4, "%s: unknown format %d", fn, fmt);
  IVFPQ_REQUIRE(known_dtype(dtype), "%s: unknown element type %d", fn, dtype);
  return IVFPQ_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace ivfpq

using namespace ivfpq;

extern "C" int fp4_product(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                           const uint8_t* b_codes, const uint8_t* b_scales, int64_t n,
                           int64_t cols, int fmt, const float* a_tensor_scale,
                           const float* b_tensor_scale, void* out, int dtype, void* stream) {
  clear_error();
  IVFPQ_TRY(check_product("fp4_product", m, n, cols, fmt, dtype));
  if (m == 0 || n == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(a_codes && a_scales && b_codes && b_scales && out, "fp4_product: null pointer");
  IVFPQ_REQUIRE(aligned16(a_codes) && aligned16(a_scales) && aligned16(b_codes) &&
                    aligned16(b_scales),
                "fp4_product: codes and scales must be 16-byte aligned");
  return product_device(a_codes, a_scales, m, b_codes, b_scales, n, cols, fmt, a_tensor_scale,
                        b_tensor_scale, out, dtype, false, static_cast<cudaStream_t>(stream));
}

extern "C" int fp4_linear(const void* x, int x_dtype, int64_t m, int64_t ldx,
                          const uint8_t* w_codes, const uint8_t* w_scales, int64_t n, int64_t cols,
                          int fmt, const float* x_tensor_scale, const float* w_tensor_scale,
                          void* out, int dtype, void* stream) {
  clear_error();
  IVFPQ_TRY(check_product("fp4_linear", m, n, cols, fmt, dtype));
  IVFPQ_REQUIRE(known_dtype(x_dtype), "fp4_linear: unknown element type %d", x_dtype);
  IVFPQ_REQUIRE(ldx >= cols || m <= 1 || ldx == 0, "fp4_linear: row stride %lld below cols=%lld",
                (long long)ldx, (long long)cols);
  if (m == 0 || n == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(x && w_codes && w_scales && out, "fp4_linear: null pointer");
  IVFPQ_REQUIRE(aligned16(w_codes) && aligned16(w_scales),
                "fp4_linear: codes and scales must be 16-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Workspace ws(s);
  uint8_t* codes = nullptr;
  const int64_t code_bytes = m * (fp4_padded_cols(cols) / 2);
  const int64_t scale_bytes = ceil_div(m, 128) * fp4_scale_tiles(cols, fmt) * 512;
  IVFPQ_TRY(ws.alloc(&codes, size_t(ceil_div(code_bytes, 512) * 512 + scale_bytes)));
  uint8_t* scales = codes + ceil_div(code_bytes, 512) * 512;
  IVFPQ_TRY(fp4_quantize_device(x, x_dtype, m, cols, ldx, fmt, x_tensor_scale, codes, scales, s));
  return product_device(codes, scales, m, w_codes, w_scales, n, cols, fmt, x_tensor_scale,
                        w_tensor_scale, out, dtype, true, s);
}
