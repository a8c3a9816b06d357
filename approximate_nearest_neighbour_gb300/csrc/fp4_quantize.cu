// fp4_quantize / fp4_dequantize: rows of fp32, binary16 or bfloat16 to 4-bit
// block-scaled form and back (formats and layout: fp4.cuh).
//
// Both are bound by memory: a value costs its own bytes, half a byte of code
// and 1/32 or 1/16 byte of scale. A thread takes 16 neighbouring columns (an
// NVFP4 block; two lanes share an MXFP4 block through one shuffle) of U rows at
// once, and the lanes with the scale bytes of one tile row join them into one
// 32-bit store. Eight columns per thread made more instructions than the loads
// hid (65537 x 4096 bf16 and back: 315 us, and 249 us with 16), thirty-two
// spread a warp's loads too far for fp32 (10000 x 1024: 27.7 us, and 22.5 us).
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace ivfpq {
namespace {

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;
  int64_t kp;      // padded columns
  int64_t ntile;   // scale tiles per row tile
  const float* tensor_scale;
  uint8_t* codes;
  uint8_t* scales;
  bool vec;        // rows start on 16-byte boundaries
};

// 16 values of a row from c0 on, zero past cols.
template <class T>
__device__ __forceinline__ void load16(const T* p, int64_t c0, int64_t cols, bool vec,
                                      float (&v)[16]) {
  if (vec && c0 + 16 <= cols) {
    constexpr int N = Span<T>::N;
    uint4 raw[16 / N];
#pragma unroll
    for (int i = 0; i < 16 / N; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(p + c0) + i);
#pragma unroll
    for (int i = 0; i < 16 / N; ++i) {
      float w[N];
      unpack_vec<T>(raw[i], w);
#pragma unroll
      for (int j = 0; j < N; ++j) v[i * N + j] = w[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = c0 + i < cols ? to_f32(p[c0 + i]) : 0.f;
  }
}

// blockDim = (tx, ty): tx 16-column groups; block (x, y) takes U rows per ty of
// them. The grid covers whole scale tiles, so the padding's bytes are written
// too.
template <class T, int FMT, int U>
__global__ void __launch_bounds__(256) fp4_quantize_kernel(const QuantArgs a) {
  grid_go();
  constexpr int LB = FMT == IVFPQ_MXFP4 ? 2 : 1;  // lanes of a block
  const int64_t grp = int64_t(blockIdx.y) * blockDim.x + threadIdx.x;
  const int64_t c0 = grp * 16;
  const int64_t row0 = int64_t(blockIdx.x) * U * blockDim.y + threadIdx.y;
  const int64_t rows_pad = (a.rows + 127) / 128 * 128;
  const float g = FMT == IVFPQ_NVFP4 && a.tensor_scale ? __ldg(a.tensor_scale) : 1.f;
  float v[U][16];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * blockDim.y;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[u][i] = 0.f;
    if (row < a.rows && c0 < a.cols)
      load16(static_cast<const T*>(a.x) + row * a.ldx, c0, a.cols, a.vec, v[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * blockDim.y;
    const bool live = row < a.rows && c0 < a.kp;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(v[u][i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < LB; o *= 2) amax = max(amax, __shfl_xor_sync(kFullMask, amax, o));
    const BlockScale bs = block_scale<FMT>(amax, g);
    if (live) {
      uint32_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[u][8 * h + i] * bs.factor;
        // factor 0 (no scale, or a block that is not finite): codes 0
        c[h] = bs.factor == 0.f ? 0u : e2m1_pack8(y);
      }
      *reinterpret_cast<uint2*>(a.codes + row * (a.kp / 2) + c0 / 2) = make_uint2(c[0], c[1]);
    }
    // four blocks of the row make one aligned 32-bit word of their scale tile
    uint32_t w = live ? uint32_t(bs.byte) : 0u;
    w |= __shfl_down_sync(kFullMask, w, LB) << 8;
    w |= __shfl_down_sync(kFullMask, w, 2 * LB) << 16;
    if (threadIdx.x % (4 * LB) == 0 && grp < a.ntile * 4 * LB && row < rows_pad)
      *reinterpret_cast<uint32_t*>(a.scales + fp4_scale_at(row, grp / LB, a.ntile)) = w;
  }
}

struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, kp, ntile;
  const float* tensor_scale;
  void* out;
  bool vec;
};

template <class T, int FMT, int U>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(const DequantArgs a) {
  constexpr int LB = FMT == IVFPQ_MXFP4 ? 2 : 1;
  const int64_t grp = int64_t(blockIdx.y) * blockDim.x + threadIdx.x;
  const int64_t c0 = grp * 16;
  const int64_t row0 = int64_t(blockIdx.x) * U * blockDim.y + threadIdx.y;
  if (c0 >= a.cols) return;
  const float g = FMT == IVFPQ_NVFP4 && a.tensor_scale ? __ldg(a.tensor_scale) : 1.f;
  uint2 c[U];
  uint8_t sb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * blockDim.y;
    c[u] = make_uint2(0, 0);
    sb[u] = 0;
    if (row < a.rows) {
      c[u] = __ldg(reinterpret_cast<const uint2*>(a.codes + row * (a.kp / 2) + c0 / 2));
      sb[u] = __ldg(a.scales + fp4_scale_at(row, grp / LB, a.ntile));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * blockDim.y;
    if (row >= a.rows) break;
    const float s = FMT == IVFPQ_MXFP4 ? e8m0_value(sb[u]) : e4m3_value(sb[u]);
    float v[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __half2 q[4];
      e2m1_unpack8(h ? c[u].y : c[u].x, q);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(q[i]);
        // element x block scale is exact in fp32; the tensor's scale rounds once
        v[8 * h + 2 * i] = f.x * s * g;
        v[8 * h + 2 * i + 1] = f.y * s * g;
      }
    }
    T* o = static_cast<T*>(a.out) + row * a.cols + c0;
    if (a.vec && c0 + 16 <= a.cols) {
      store_vec<T>(o, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c0 + i < a.cols) o[i] = from_f32<T>(v[i]);
    }
  }
}

// Block of 256 threads: enough 16-column groups for the row, a power of two (at
// least a scale word's lanes), the rest of the block on rows.
dim3 block_for(int64_t ngrp) {
  unsigned tx = 8;
  while (tx < 256 && int64_t(tx) < ngrp) tx *= 2;
  return dim3(tx, 256 / tx);
}
// Two rows per thread once that leaves eight blocks per SM.
bool two_rows(int64_t rows, int64_t ngrp, const dim3& block) {
  return ceil_div(rows, 2 * block.y) * ceil_div(ngrp, block.x) >= 8 * num_sms();
}

int check_rows(const char* fn, int64_t rows, int64_t cols, int fmt, int dtype) {
  IVFPQ_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), "%s: rows=%lld outside [0, 2^31)", fn,
                (long long)rows);
  IVFPQ_REQUIRE(cols >= 1 && cols <= (int64_t(1) << 24), "%s: cols=%lld outside [1, 2^24]", fn,
                (long long)cols);
  IVFPQ_REQUIRE(fmt == IVFPQ_MXFP4 || fmt == IVFPQ_NVFP4, "%s: unknown format %d", fn, fmt);
  IVFPQ_REQUIRE(known_dtype(dtype), "%s: unknown element type %d", fn, dtype);
  return IVFPQ_OK;
}

bool aligned16(const void* p, int64_t row_bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && row_bytes % 16 == 0;
}

}  // namespace

int fp4_quantize_device(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int fmt,
                        const float* tensor_scale, uint8_t* codes, uint8_t* scales,
                        cudaStream_t s) {
  QuantArgs a;
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.kp = fp4_padded_cols(cols);
  a.ntile = fp4_scale_tiles(cols, fmt);
  a.tensor_scale = tensor_scale;
  a.codes = codes;
  a.scales = scales;
  a.vec = aligned16(x, ldx * dtype_size(dtype));
  const int64_t ngrp = a.ntile * (fmt == IVFPQ_MXFP4 ? 8 : 4);
  const dim3 block = block_for(ngrp);
  const int64_t rows_pad = ceil_div(rows, 128) * 128;
  const int u = two_rows(rows_pad, ngrp, block) ? 2 : 1;
  const dim3 grid(unsigned(ceil_div(rows_pad, u * block.y)), unsigned(ceil_div(ngrp, block.x)));
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    auto kern = fmt == IVFPQ_MXFP4
                    ? (u == 2 ? fp4_quantize_kernel<T, IVFPQ_MXFP4, 2>
                              : fp4_quantize_kernel<T, IVFPQ_MXFP4, 1>)
                    : (u == 2 ? fp4_quantize_kernel<T, IVFPQ_NVFP4, 2>
                              : fp4_quantize_kernel<T, IVFPQ_NVFP4, 1>);
    kern<<<grid, block, 0, s>>>(a);
    IVFPQ_LAUNCHED();
    return IVFPQ_OK;
  });
}

}  // namespace ivfpq

using namespace ivfpq;

extern "C" int fp4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                            int fmt, const float* tensor_scale, uint8_t* codes, uint8_t* scales,
                            void* stream) {
  clear_error();
  IVFPQ_TRY(check_rows("fp4_quantize", rows, cols, fmt, dtype));
  IVFPQ_REQUIRE(ldx >= cols || rows <= 1 || ldx == 0, "fp4_quantize: row stride %lld below cols=%lld",
                (long long)ldx, (long long)cols);
  if (rows == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(x && codes && scales, "fp4_quantize: null pointer");
  IVFPQ_REQUIRE(aligned16(codes, 16) && aligned16(scales, 16),
                "fp4_quantize: codes and scales must be 16-byte aligned");
  return fp4_quantize_device(x, dtype, rows, cols, ldx, fmt, tensor_scale, codes, scales,
                             static_cast<cudaStream_t>(stream));
}

extern "C" int fp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                              int64_t cols, int fmt, const float* tensor_scale, void* out,
                              int dtype, void* stream) {
  clear_error();
  IVFPQ_TRY(check_rows("fp4_dequantize", rows, cols, fmt, dtype));
  if (rows == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(codes && scales && out, "fp4_dequantize: null pointer");
  IVFPQ_REQUIRE(aligned16(codes, 16) && aligned16(scales, 16),
                "fp4_dequantize: codes and scales must be 16-byte aligned");
  DequantArgs a;
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.cols = cols;
  a.kp = fp4_padded_cols(cols);
  a.ntile = fp4_scale_tiles(cols, fmt);
  a.tensor_scale = tensor_scale;
  a.out = out;
  a.vec = aligned16(out, cols * dtype_size(dtype));
  const int64_t ngrp = ceil_div(cols, 16);
  const dim3 block = block_for(ngrp);
  const int u = two_rows(rows, ngrp, block) ? 2 : 1;
  const dim3 grid(unsigned(ceil_div(rows, u * block.y)), unsigned(ceil_div(ngrp, block.x)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    auto kern = fmt == IVFPQ_MXFP4
                    ? (u == 2 ? fp4_dequantize_kernel<T, IVFPQ_MXFP4, 2>
                              : fp4_dequantize_kernel<T, IVFPQ_MXFP4, 1>)
                    : (u == 2 ? fp4_dequantize_kernel<T, IVFPQ_NVFP4, 2>
                              : fp4_dequantize_kernel<T, IVFPQ_NVFP4, 1>);
    kern<<<grid, block, 0, s>>>(a);
    IVFPQ_LAUNCHED();
    return IVFPQ_OK;
  });
}
