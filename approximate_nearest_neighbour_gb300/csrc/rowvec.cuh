// Element types of score rows and 16-byte access to rows of any alignment,
// shared by the kernels that stream them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "common.cuh"

namespace ivfpq {

inline bool known_dtype(int dtype) {
  return dtype == IVFPQ_F32 || dtype == IVFPQ_F16 || dtype == IVFPQ_BF16;
}
inline int dtype_size(int dtype) { return dtype == IVFPQ_F32 ? 4 : 2; }

// ---- element access ---------------------------------------------------------------
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Calls f with a null pointer of the element type that `dtype` names.
template <class F>
int by_dtype(int dtype, F&& f) {
  if (dtype == IVFPQ_F32) return f(static_cast<float*>(nullptr));
  if (dtype == IVFPQ_F16) return f(static_cast<__half*>(nullptr));
  return f(static_cast<__nv_bfloat16*>(nullptr));
}

// ---- 16-byte access to a run of a row -----------------------------------------------
// Elements [0, len) at p by address: a head up to the first 16-byte boundary,
// whole vectors, a tail.
template <class T>
struct Span {
  static constexpr int N = 16 / int(sizeof(T));
  int head, nvec, len;
  __device__ __forceinline__ Span(const T* p, int n) : len(n) {
    head = min(n, int((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / int(sizeof(T)));
    nvec = (n - head) / N;
  }
  // the e-th element outside the vectors (e < rest())
  __device__ __forceinline__ int rest() const { return len - nvec * N; }
  __device__ __forceinline__ int at(int e) const { return e < head ? e : nvec * N + e; }
};
__device__ __forceinline__ void unpack(const uint4& r, float (&v)[4]) {
  v[0] = __uint_as_float(r.x);
  v[1] = __uint_as_float(r.y);
  v[2] = __uint_as_float(r.z);
  v[3] = __uint_as_float(r.w);
}
template <class T>
__device__ __forceinline__ void unpack16(uint32_t w, float& lo, float& hi);
template <>
__device__ __forceinline__ void unpack16<__nv_bfloat16>(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
template <>
__device__ __forceinline__ void unpack16<__half>(uint32_t w, float& lo, float& hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo = f.x;
  hi = f.y;
}
template <class T>
__device__ __forceinline__ void unpack_vec(const uint4& r, float (&v)[Span<T>::N]) {
  if constexpr (sizeof(T) == 4) {
    unpack(r, v);
  } else {
    unpack16<T>(r.x, v[0], v[1]);
    unpack16<T>(r.y, v[2], v[3]);
    unpack16<T>(r.z, v[4], v[5]);
    unpack16<T>(r.w, v[6], v[7]);
  }
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, __nv_bfloat16*) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, __half*) {
  const __half2 t = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
template <class T>
__device__ __forceinline__ uint4 pack_vec(const float (&v)[Span<T>::N]) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  } else {
    T* t = nullptr;
    return make_uint4(pack16(v[0], v[1], t), pack16(v[2], v[3], t), pack16(v[4], v[5], t),
                      pack16(v[6], v[7], t));
  }
}
// M values as whole 16-byte vectors of O at p (16-byte aligned).
template <class O, int M>
__device__ __forceinline__ void store_vec(O* p, const float (&v)[M]) {
  static_assert(M % Span<O>::N == 0, "whole vectors");
#pragma unroll
  for (int q = 0; q < M / Span<O>::N; ++q) {
    float w[Span<O>::N];
#pragma unroll
    for (int i = 0; i < Span<O>::N; ++i) w[i] = v[q * Span<O>::N + i];
    reinterpret_cast<uint4*>(p)[q] = pack_vec<O>(w);
  }
}
template <class T>
__device__ __forceinline__ T lowest_inf();
template <>
__device__ __forceinline__ float lowest_inf<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ __half lowest_inf<__half>() { return __ushort_as_half(0xfc00); }
template <>
__device__ __forceinline__ __nv_bfloat16 lowest_inf<__nv_bfloat16>() {
  return __ushort_as_bfloat16(0xff80);
}
// Elements i N .. i N + N - 1 of the run at p, whatever its alignment (mis =
// address mod 16): two neighbouring 16-byte loads shifted together where both
// lie inside the run (load_inner), element by element in the first and last
// vectors of a misaligned run, so that nothing outside the run is read. Past
// the end: -inf. Which elements go into one vector depends on their index
// alone, and so do the sums over them.
template <class T>
__device__ __forceinline__ uint4 load_inner(const T* p, int i, int mis) {
  if (mis == 0) return reinterpret_cast<const uint4*>(p)[i];
  const uint4* b = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - mis) + i;
  const uint4 x = b[0], y = b[1];
  uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  if (mis & 8) {
#pragma unroll
    for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
  }
  if (mis & 4) {
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
  }
  const int bits = (mis & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}
// The 16 bytes from byte `mis` of x and y on, without a branch.
__device__ __forceinline__ uint4 shift_across(const uint4& x, const uint4& y, int mis) {
  uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
  for (int j = 0; j < 6; ++j) w[j] = mis & 8 ? w[j + 2] : w[j];
#pragma unroll
  for (int j = 0; j < 5; ++j) w[j] = mis & 4 ? w[j + 1] : w[j];
  const int bits = (mis & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}
// The inner vectors of a run are inner_first .. inner_last.
__device__ __forceinline__ int inner_first(int mis) { return mis == 0 ? 0 : 1; }
template <class T>
__device__ __forceinline__ int inner_last(int len, int mis) {
  return len / Span<T>::N - (mis == 0 ? 1 : 2);
}
template <class T>
__device__ __noinline__ uint4 load_edge(const T* p, int len, int i) {
  constexpr int N = Span<T>::N;
  T t[N];
#pragma unroll
  for (int j = 0; j < N; ++j) t[j] = i * N + j < len ? p[i * N + j] : lowest_inf<T>();
  uint4 r;
  memcpy(&r, t, 16);
  return r;
}
template <class T>
__device__ __forceinline__ uint4 load_vec(const T* p, int len, int i, int mis) {
  if (i >= inner_first(mis) && i <= inner_last<T>(len, mis)) return load_inner(p, i, mis);
  return load_edge(p, len, i);
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ int misalign(const void* p) {
  return int(reinterpret_cast<uintptr_t>(p) & 15);
}

// The largest element of a vector; 16-bit types two at a time.
__device__ __forceinline__ float vec_max(const uint4& r, float*) {
  return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
               fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
}
template <class T>
__device__ __forceinline__ float vec_max(const uint4& r, T*) {
  using P = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
  P w[4];
  memcpy(w, &r, 16);
  const P t = __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
  return fmaxf(to_f32(t.x), to_f32(t.y));
}

// Element j of a vector, j not known at compile time.
template <class T>
__device__ __forceinline__ float vec_element(const uint4& r, int j) {
  const int w = sizeof(T) == 4 ? j : j >> 1;
  const uint32_t x = w < 2 ? (w == 0 ? r.x : r.y) : (w == 2 ? r.z : r.w);
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(x);
  } else {
    float lo, hi;
    unpack16<T>(x, lo, hi);
    return j & 1 ? hi : lo;
  }
}

// Starts bringing bytes [from, from + bytes) of the run [p, end) into L2; one
// thread of a block asks for what the block reads a few steps later.
__device__ __forceinline__ void prefetch_run(const void* p, int64_t from, int64_t bytes,
                                             const void* end) {
  const uintptr_t e = reinterpret_cast<uintptr_t>(end) & ~uintptr_t(15);
  const uintptr_t b = (reinterpret_cast<uintptr_t>(p) + from + 15) & ~uintptr_t(15);
  if (b >= e) return;
  const uint32_t n = uint32_t(bytes < int64_t(e - b) ? uintptr_t(bytes) : e - b);
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(b), "r"(n) : "memory");
}

}  // namespace ivfpq
