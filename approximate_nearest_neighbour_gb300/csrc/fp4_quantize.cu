// fp4_quantize / fp4_dequantize: rows of fp32, binary16 or bfloat16 to 4-bit
// block-scaled form and back (formats and layout: fp4.cuh).
//
// Both are bound by memory: a value costs its own bytes, half a byte of code
// and 1/32 or 1/16 byte of scale.
//
// Quantising, a thread takes 16 neighbouring columns (an NVFP4 block; two lanes
// share an MXFP4 block through one shuffle), and the lanes with the scale bytes
// of one tile row join them into one 32-bit store. Eight columns per thread
// made more instructions than the loads hid (65537 x 4096 bf16 and back: 315
// us, and 249 us with 16), thirty-two spread a warp's loads too far for fp32
// (10000 x 1024: 27.7 us, and 22.5 us), and two rows per thread halved the
// warps (262 us). Magnitudes of 16-bit types are compared two at a time.
//
// Reading back, a lane writes 16 bytes of four rows, so that a warp's store is
// contiguous. Measured: 65537 x 4096 bf16 to MXFP4 and back 210 us, 6.6 TB/s over
// both passes' bytes.
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

// 16 values of a row from c0 on, zero past cols, and the largest magnitude's
// bits as fp32 (the maximum of integers, so that a NaN or an infinity is kept).
template <class T>
__device__ __forceinline__ uint32_t load16(const T* p, int64_t c0, int64_t cols, bool vec,
                                           float (&v)[16]) {
  constexpr int N = Span<T>::N;
  uint32_t amax = 0;
  if (vec && c0 + 16 <= cols) {
    uint4 raw[16 / N];
#pragma unroll
    for (int i = 0; i < 16 / N; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(p + c0) + i);
#pragma unroll
    for (int i = 0; i < 16 / N; ++i) {
      float w[N];
      unpack_vec<T>(raw[i], w);
#pragma unroll
      for (int j = 0; j < N; ++j) v[i * N + j] = w[j];
      if constexpr (sizeof(T) == 2) {
        const uint32_t m = 0x7fff7fffu;
        amax = __vmaxu2(amax, __vmaxu2(__vmaxu2(raw[i].x & m, raw[i].y & m),
                                       __vmaxu2(raw[i].z & m, raw[i].w & m)));
      }
    }
    if constexpr (sizeof(T) == 2) {
      amax = max(amax & 0xffffu, amax >> 16);
      float lo, hi;
      unpack16<T>(amax, lo, hi);
      return __float_as_uint(lo);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = c0 + i < cols ? to_f32(p[c0 + i]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  return amax;
}

// blockDim = (tx, ty): tx 16-column groups of ty rows. The grid covers whole
// scale tiles, so the padding's bytes are written too.
template <class T, int FMT>
__global__ void __launch_bounds__(256) fp4_quantize_kernel(const QuantArgs a) {
  grid_go();
  constexpr int LB = FMT == IVFPQ_MXFP4 ? 2 : 1;  // lanes of a block
  const int64_t grp = int64_t(blockIdx.y) * blockDim.x + threadIdx.x;
  const int64_t c0 = grp * 16;
  const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t rows_pad = (a.rows + 127) / 128 * 128;
  const float g = FMT == IVFPQ_NVFP4 && a.tensor_scale ? __ldg(a.tensor_scale) : 1.f;
  const bool live = row < a.rows && c0 < a.kp;
  float v[16];
  uint32_t amax = 0;
  if (live) amax = load16(static_cast<const T*>(a.x) + row * a.ldx, c0, a.cols, a.vec, v);
#pragma unroll
  for (int o = 1; o < LB; o *= 2) amax = max(amax, __shfl_xor_sync(kFullMask, amax, o));
  const float lift = FMT == IVFPQ_NVFP4 ? nvfp4_lift(g) : 1.f;
  const BlockScale bs = block_scale<FMT>(amax, g, lift);
  if (FMT == IVFPQ_NVFP4 && lift != 1.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= lift;
  }
  if (live) {
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        unpair(mul2(pair(v[8 * h + i], v[8 * h + i + 1]), pair(bs.factor, bs.factor)), y[i],
               y[i + 1]);
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

struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, kp, ntile;
  const float* tensor_scale;
  void* out;
  bool vec;
};

// blockDim = (tx, ty): tx groups of N columns (16 bytes of output); block (x, y)
// takes U rows per ty of them.
template <class T, int FMT, int U>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(const DequantArgs a) {
  constexpr int N = Span<T>::N;
  const int64_t c0 = (int64_t(blockIdx.y) * blockDim.x + threadIdx.x) * N;
  const int64_t row0 = int64_t(blockIdx.x) * U * blockDim.y + threadIdx.y;
  if (c0 >= a.cols) return;
  const int64_t blk = c0 / (FMT == IVFPQ_MXFP4 ? 32 : 16);
  const float g = FMT == IVFPQ_NVFP4 && a.tensor_scale ? __ldg(a.tensor_scale) : 1.f;
  uint32_t c[U];
  uint8_t sb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * blockDim.y;
    c[u] = 0;
    sb[u] = 0;
    if (row < a.rows) {
      const uint8_t* p = a.codes + row * (a.kp / 2) + c0 / 2;
      c[u] = N == 8 ? __ldg(reinterpret_cast<const uint32_t*>(p))
                    : __ldg(reinterpret_cast<const uint16_t*>(p));
      sb[u] = __ldg(a.scales + fp4_scale_at(row, blk, a.ntile));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * blockDim.y;
    if (row >= a.rows) break;
    const float s = FMT == IVFPQ_MXFP4 ? e8m0_value(sb[u]) : e4m3_value(sb[u]);
    float v[N];
    __half2 q[4];
    e2m1_unpack8(c[u], q);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 f = __half22float2(q[i]);
      // element x block scale is exact in fp32; the tensor's scale rounds once
      v[2 * i] = f.x * s * g;
      v[2 * i + 1] = f.y * s * g;
    }
    T* o = static_cast<T*>(a.out) + row * a.cols + c0;
    if (a.vec && c0 + N <= a.cols) {
      store_vec<T>(o, v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c0 + i < a.cols) o[i] = from_f32<T>(v[i]);
    }
  }
}

// Block of 256 threads: enough column groups for the row, a power of two (at
// least a scale word's lanes), the rest of the block on rows.
dim3 block_for(int64_t ngrp) {
  unsigned tx = 8;
  while (tx < 256 && int64_t(tx) < ngrp) tx *= 2;
  return dim3(tx, 256 / tx);
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
  const dim3 grid(unsigned(ceil_div(rows_pad, block.y)), unsigned(ceil_div(ngrp, block.x)));
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    auto kern = fmt == IVFPQ_MXFP4 ? fp4_quantize_kernel<T, IVFPQ_MXFP4>
                                   : fp4_quantize_kernel<T, IVFPQ_NVFP4>;
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
  IVFPQ_REQUIRE(ldx >= cols || rows <= 1 || ldx == 0,
                "fp4_quantize: row stride %lld below cols=%lld", (long long)ldx, (long long)cols);
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
  const int64_t ngrp = ceil_div(cols, 16 / dtype_size(dtype));
  const dim3 block = block_for(ngrp);
  // four rows per thread once that leaves eight blocks per SM
  const int64_t by = ceil_div(ngrp, block.x);
  const int u = ceil_div(rows, 4 * block.y) * by >= 8 * num_sms() ? 4 : 1;
  const dim3 grid(unsigned(ceil_div(rows, u * block.y)), unsigned(by));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    auto kern = fmt == IVFPQ_MXFP4
                    ? (u == 4 ? fp4_dequantize_kernel<T, IVFPQ_MXFP4, 4>
                              : fp4_dequantize_kernel<T, IVFPQ_MXFP4, 1>)
                    : (u == 4 ? fp4_dequantize_kernel<T, IVFPQ_NVFP4, 4>
                              : fp4_dequantize_kernel<T, IVFPQ_NVFP4, 1>);
    kern<<<grid, block, 0, s>>>(a);
    IVFPQ_LAUNCHED();
    return IVFPQ_OK;
  });
}
