// topk_distill_*: distillation of a student's score rows from a teacher's top
// list (the values and ids a k-selection or a search returns). With the
// temperature tau and the valid entries i of a row's list
//   p_i = softmax_i(t_i / tau),  q_j = softmax_j(s_j / tau) over all columns,
//   loss = tau^2 sum_i p_i (log p_i - log q_id(i)),
//   d loss / d s_j = tau (P q_j - sum_{i: id(i) = j} p_i),  P = sum_i p_i
// (1, or 0 for a list without valid entries, whose loss and gradient are 0).
//
// Bound by memory: the forward pass reads each score once, the backward pass
// reads and writes each once. Statistics kept per row: the largest score m
// and Z = sum_j exp((s_j - m) / tau), both fp32; q_j comes from the difference
// s_j - m, so scores of any magnitude (a mask of the type's lowest value among
// them) neither overflow nor cancel. A score of -inf has q = 0.
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"

namespace ivfpq {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.44269504088896340736f;

struct DistillArgs {
  const void* scores;
  int64_t rows, cols, lds;
  const float* tv;
  const int64_t* ti;
  int k;
  float tau, inv_tau, sign;
  const float* row_grad;
  float* loss;
  float* stats;  // [rows, 2]
  void* grad;
  int64_t ldg;
};

// exp((s - m) / tau): the difference first, so that the exponent's rounding
// error stays relative to the distance from the maximum; 0 for s = -inf.
__device__ __forceinline__ float shifted_exp(float s, float m, float c) {
  return s == -INFINITY ? 0.f : exp2f((s - m) * c);
}

// Maxima and sums over the block, in a fixed order.
template <int NW>
__device__ __forceinline__ float block_max(float v, float* sh) {
#pragma unroll
  for (int o = 16; o; o /= 2) {
    const float w = __shfl_xor_sync(kFullMask, v, o);
    v = (w > v || w != w) ? w : v;  // keeps a NaN
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = sh[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) r = (sh[i] > r || sh[i] != sh[i]) ? sh[i] : r;
  return r;
}
template <int NW>
__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o; o /= 2) v += __shfl_xor_sync(kFullMask, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i) r += sh[i];
  return r;
}

// The teacher's softmax: entry i is valid if its id is a column and its value
// is not -inf (the padding of a short list).
struct Teacher {
  float m, z;  // largest valid value, sum of exp((t - m) / tau); z = 0: none valid
};
__device__ __forceinline__ bool teacher_entry(const DistillArgs& a, int64_t row, int i, float* t,
                                              int64_t* id) {
  *t = a.tv[row * a.k + i] * a.sign;
  *id = a.ti[row * a.k + i];
  return *id >= 0 && *id < a.cols && *t != -INFINITY;
}
__device__ __forceinline__ Teacher teacher_stats(const DistillArgs& a, int64_t row, float* sh) {
  float m = -INFINITY;
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    float t;
    int64_t id;
    if (teacher_entry(a, row, i, &t, &id)) m = (t > m || t != t) ? t : m;
  }
  Teacher r;
  r.m = block_max<kWarps>(m, sh);
  float z = 0.f;
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    float t;
    int64_t id;
    if (teacher_entry(a, row, i, &t, &id)) z += exp2f((t - r.m) * (a.inv_tau * kLog2e));
  }
  r.z = block_sum<kWarps>(z, sh);
  return r;
}

template <class T>
__global__ void __launch_bounds__(kThreads) distill_forward_kernel(const DistillArgs a) {
  __shared__ float sh[kWarps];
  const int64_t row = blockIdx.x;
  const T* s = static_cast<const T*>(a.scores) + row * a.lds;
  const float c = a.inv_tau * kLog2e;
  float m = -INFINITY;
  for (int64_t j = threadIdx.x; j < a.cols; j += kThreads) {
    const float v = to_f32(s[j]);
    m = (v > m || v != v) ? v : m;
  }
  m = block_max<kWarps>(m, sh);
  float z = 0.f;
  for (int64_t j = threadIdx.x; j < a.cols; j += kThreads) z += shifted_exp(to_f32(s[j]), m, c);
  z = block_sum<kWarps>(z, sh);
  const Teacher te = teacher_stats(a, row, sh);
  // tau^2 sum p (log p + log Z) - tau sum p (s - m): no s - m is divided by
  // tau, so that a listed score of the type's lowest value stays finite
  float l = 0.f, d = 0.f;
  const float logz = z == 0.f ? 0.f : logf(z), logtz = logf(te.z);
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    float t;
    int64_t id;
    if (!teacher_entry(a, row, i, &t, &id)) continue;
    const float lt = (t - te.m) * a.inv_tau;
    const float p = exp2f(lt * kLog2e) / te.z;
    const float sj = to_f32(s[id]);
    if (!(p <= 0.f)) {  // also a NaN
      l += p * (lt - logtz + logz);
      d += p * (sj == -INFINITY ? sj : sj - m);
    }
  }
  l = block_sum<kWarps>(l, sh);
  d = block_sum<kWarps>(d, sh);
  if (threadIdx.x == 0) {
    a.loss[row] = a.tau * (a.tau * l - d);
    a.stats[2 * row] = m;
    a.stats[2 * row + 1] = z;
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) distill_backward_kernel(const DistillArgs a) {
  __shared__ float sh[kWarps];
  __shared__ float fix[IVFPQ_MAX_K];
  const int64_t row = blockIdx.x;
  const T* s = static_cast<const T*>(a.scores) + row * a.lds;
  T* g = static_cast<T*>(a.grad) + row * a.ldg;
  const float c = a.inv_tau * kLog2e;
  const float m = a.stats[2 * row], z = a.stats[2 * row + 1];
  const float w = a.row_grad[row] * a.tau;
  if (w == 0.f) {  // a row that does not count, whatever it holds
    for (int64_t j = threadIdx.x; j < a.cols; j += kThreads) g[j] = from_f32<T>(0.f);
    return;
  }
  const Teacher te = teacher_stats(a, row, sh);
  const float inv_z = z == 0.f ? 0.f : 1.f / z;  // no score above -inf: q = 0
  const float rz = te.z == 0.f ? 0.f : w * inv_z;
  // the listed columns first: the gradient may overwrite the scores
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    float t;
    int64_t id;
    if (!teacher_entry(a, row, i, &t, &id)) continue;
    float p = 0.f;  // of all entries with this id, in list order
    for (int j = 0; j < a.k; ++j) {
      float tj;
      int64_t idj;
      if (teacher_entry(a, row, j, &tj, &idj) && idj == id)
        p += exp2f((tj - te.m) * c) / te.z;
    }
    fix[i] = w * (shifted_exp(to_f32(s[id]), m, c) * inv_z - p);
  }
  __syncthreads();
  for (int64_t j = threadIdx.x; j < a.cols; j += kThreads)
    g[j] = from_f32<T>(shifted_exp(to_f32(s[j]), m, c) * rz);
  __syncthreads();
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    float t;
    int64_t id;
    if (teacher_entry(a, row, i, &t, &id)) g[id] = from_f32<T>(fix[i]);
  }
}

int check_distill(const char* fn, int dtype, int64_t rows, int64_t cols, int64_t lds, int k,
                  float temperature) {
  IVFPQ_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), "%s: rows=%lld outside [0, 2^31)", fn,
                (long long)rows);
  IVFPQ_REQUIRE(cols >= 1 && cols <= (int64_t(1) << 28), "%s: cols=%lld outside [1, 2^28]", fn,
                (long long)cols);
  IVFPQ_REQUIRE(known_dtype(dtype), "%s: unknown element type %d", fn, dtype);
  IVFPQ_REQUIRE(rows <= 1 || lds >= cols || lds == 0, "%s: row stride %lld below cols=%lld", fn,
                (long long)lds, (long long)cols);
  IVFPQ_REQUIRE(k >= 1 && k <= IVFPQ_MAX_K, "%s: k=%d outside [1, %d]", fn, k, IVFPQ_MAX_K);
  IVFPQ_REQUIRE(temperature > 0.f && temperature <= 1e30f && temperature >= 1e-30f,
                "%s: temperature=%g outside [1e-30, 1e30]", fn, double(temperature));
  return IVFPQ_OK;
}

DistillArgs distill_args(const void* scores, int64_t rows, int64_t cols, int64_t lds,
                         const float* tv, const int64_t* ti, int k, float temperature,
                         int negated) {
  DistillArgs a{};
  a.scores = scores;
  a.rows = rows;
  a.cols = cols;
  a.lds = lds;
  a.tv = tv;
  a.ti = ti;
  a.k = k;
  a.tau = temperature;
  a.inv_tau = 1.f / temperature;
  a.sign = negated ? -1.f : 1.f;
  return a;
}

int launch_forward(const DistillArgs& a, int dtype, cudaStream_t s) {
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    distill_forward_kernel<T><<<unsigned(a.rows), kThreads, 0, s>>>(a);
    IVFPQ_LAUNCHED();
    return IVFPQ_OK;
  });
}
int launch_backward(const DistillArgs& a, int dtype, cudaStream_t s) {
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    distill_backward_kernel<T><<<unsigned(a.rows), kThreads, 0, s>>>(a);
    IVFPQ_LAUNCHED();
    return IVFPQ_OK;
  });
}

}  // namespace
}  // namespace ivfpq

using namespace ivfpq;

extern "C" int topk_distill_forward(const void* scores, int dtype, int64_t rows, int64_t cols,
                                    int64_t lds, const float* teacher_vals,
                                    const int64_t* teacher_ids, int k, float temperature,
                                    int negated, float* loss, float* stats, void* stream) {
  clear_error();
  IVFPQ_TRY(check_distill("topk_distill_forward", dtype, rows, cols, lds, k, temperature));
  if (rows == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(scores && teacher_vals && teacher_ids && loss && stats,
                "topk_distill_forward: null pointer");
  DistillArgs a = distill_args(scores, rows, cols, lds, teacher_vals, teacher_ids, k, temperature,
                               negated);
  a.loss = loss;
  a.stats = stats;
  return launch_forward(a, dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int topk_distill_backward(const void* scores, int dtype, int64_t rows, int64_t cols,
                                     int64_t lds, const float* teacher_vals,
                                     const int64_t* teacher_ids, int k, float temperature,
                                     int negated, const float* stats, const float* row_grad,
                                     void* grad, int64_t ldg, void* stream) {
  clear_error();
  IVFPQ_TRY(check_distill("topk_distill_backward", dtype, rows, cols, lds, k, temperature));
  IVFPQ_REQUIRE(rows <= 1 || ldg >= cols, "topk_distill_backward: row stride %lld below cols=%lld",
                (long long)ldg, (long long)cols);
  if (rows == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(scores && teacher_vals && teacher_ids && stats && row_grad && grad,
                "topk_distill_backward: null pointer");
  DistillArgs a = distill_args(scores, rows, cols, lds, teacher_vals, teacher_ids, k, temperature,
                               negated);
  a.stats = const_cast<float*>(stats);
  a.row_grad = row_grad;
  a.grad = grad;
  a.ldg = ldg;
  return launch_backward(a, dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int topk_distill(const void* scores, int dtype, int64_t rows, int64_t cols, int64_t lds,
                            const float* teacher_vals, const int64_t* teacher_ids, int k,
                            float temperature, int negated, const float* row_grad, float* loss,
                            void* grad, int64_t ldg, void* stream) {
  clear_error();
  IVFPQ_TRY(check_distill("topk_distill", dtype, rows, cols, lds, k, temperature));
  IVFPQ_REQUIRE(rows <= 1 || ldg >= cols, "topk_distill: row stride %lld below cols=%lld",
                (long long)ldg, (long long)cols);
  if (rows == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(scores && teacher_vals && teacher_ids && row_grad && loss && grad,
                "topk_distill: null pointer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Workspace ws(s);
  DistillArgs a = distill_args(scores, rows, cols, lds, teacher_vals, teacher_ids, k, temperature,
                               negated);
  IVFPQ_TRY(ws.alloc(&a.stats, size_t(rows) * 2));
  a.loss = loss;
  a.row_grad = row_grad;
  a.grad = grad;
  a.ldg = ldg;
  IVFPQ_TRY(launch_forward(a, dtype, s));
  return launch_backward(a, dtype, s);
}
