// What the kernels of adapter_linear share: arguments, tiles of tokens, and the cut
// of an fp32 value into terms of a 16-bit type.
#pragma once

#include "rowvec.cuh"
#include "tc_ptx.cuh"

namespace ivfpq {

constexpr int kMaxTile = 128;

struct AdapterArgs {
  const void* x;
  int64_t tokens, cols, ldx;
  const void* a;
  const void* b;
  int adapters, rank;
  int64_t n;
  const int32_t* ids;
  const float* scales;
  const void* base;
  int64_t ldb;
  void* out;
  int64_t ldo;
  // tiles of tokens that share an adapter; h and order go by slot, a tile's one after
  // the other
  int32_t* order;   // a slot's token
  int4* tiles;      // (adapter or -1, first slot, tokens, 0)
  int32_t* ntiles;  // null: as many as there are blocks for, some of 0 tokens
  int tile;     // most tokens of a tile
  float* h;     // [slots, pitch]
  int splits;   // parts of K, one per block of a cluster
  int kpart;    // columns of a part, a multiple of 32
  int pitch;    // rank rounded up to whole instructions
  int run;      // output columns of a block
};

struct Tile {
  int adapter, first, count;
};
__device__ __forceinline__ Tile tile_at(const AdapterArgs& a, int64_t i) {
  if (a.ntiles && i >= *a.ntiles) return {-1, 0, 0};
  const int4 t = a.tiles[i];
  return {t.x, t.y, t.z};
}
__device__ __forceinline__ int64_t token_of(const AdapterArgs& a, int slot) {
  return a.order[slot];
}

// The next term of v as an element of T; what is left of it stays in v.
template <class T>
__device__ __forceinline__ float term(float& v) {
  const float t = to_f32(from_f32<T>(v));
  v = fabsf(t) < INFINITY ? v - t : 0.f;
  return t;
}

// Element k of a row of h, 0 past the rank: there h has the products of x with zeros, which
// an infinity or a NaN in x makes a NaN.
__device__ __forceinline__ float within_rank(const AdapterArgs& a, int k, float h) {
  return k < a.rank ? h : 0.f;
}
// |v| where it is finite, else 0.
__device__ __forceinline__ float magnitude(float v) {
  return fabsf(v) < INFINITY ? fabsf(v) : 0.f;
}
// fp16's range: the power of two that takes a row's largest finite magnitude to
// [2^14, 2^15), and its inverse (1 for a row without one that is not 0).
__device__ __forceinline__ float2 fp16_range(float top) {
  const int ex = int(__float_as_uint(top) >> 23);  // 127 + its exponent
  const int by = top > 0.f ? min(141 - ex, 126) : 0;
  return make_float2(__uint_as_float(uint32_t(127 + by) << 23),
                     __uint_as_float(uint32_t(127 - by) << 23));
}

// Elements 8 i .. 8 i + 7 of a row of `len`, zero past its end, whatever its alignment.
template <class T>
__device__ __noinline__ uint4 edge8(const T* p, int64_t len, int64_t at) {
  T t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = at + j < len ? p[at + j] : from_f32<T>(0.f);
  uint4 r;
  memcpy(&r, t, 16);
  return r;
}
template <class T>
__device__ __forceinline__ uint4 row8(const T* p, int64_t len, int64_t at) {
  if (p == nullptr || at >= len) return make_uint4(0, 0, 0, 0);
  const int mis = misalign(p);
  if (mis == 0 && at + 8 <= len) return *reinterpret_cast<const uint4*>(p + at);
  // two neighbouring vectors inside the row
  if (mis != 0 && at >= 8 && at + 16 <= len) return load_inner(p + at, 0, mis);
  return edge8(p, len, at);
}

// The parts of K, each in its block's shared memory ([rows, R]), added in the order
// of the blocks and written to the slots from `first` on; a share per block.
template <int R, int THREADS>
__device__ __forceinline__ void join_parts(const AdapterArgs& a, const float* part, int rows,
                                           int first) {
  static_assert(R % 4 == 0, "whole vectors");
  if (a.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  const uint32_t base = smem_u32(part);
  float* h = a.h + int64_t(first) * R;
  for (int i = blockIdx.x * THREADS + threadIdx.x; i < rows * R / 4; i += a.splits * THREADS) {
    float4 s = ld_cluster4(map_rank(base + 16u * uint32_t(i), 0));
    for (int v = 1; v < a.splits; ++v) {
      const float4 f = ld_cluster4(map_rank(base + 16u * uint32_t(i), uint32_t(v)));
      s.x += f.x;
      s.y += f.y;
      s.z += f.z;
      s.w += f.w;
    }
    reinterpret_cast<float4*>(h)[i] = s;
  }
  if (a.splits > 1) cluster_sync();  // no block leaves while others read its part
}

// Whether rows of base and out are whole vectors on 16-byte boundaries.
template <class O>
bool whole_rows(const AdapterArgs& a) {
  const int64_t per = 16 / int64_t(sizeof(O));
  return a.n % 8 == 0 && a.ldo % per == 0 && a.ldb % per == 0 &&
         reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(a.base) % 16 == 0;
}

// h = x A^T for tiles of kMaxTile tokens, `tiles` of them at most (adapter_wide.cu).
int adapter_shrink_wide(const AdapterArgs& a, int dtype, int64_t tiles, cudaStream_t s);
// out = base + scale h B^T for such tiles: at least one adapter, rank a multiple of 8, b
// on a 16-byte boundary.
int adapter_expand_wide(const AdapterArgs& a, int dtype, int out_dtype, cudaStream_t s);

}  // namespace ivfpq
