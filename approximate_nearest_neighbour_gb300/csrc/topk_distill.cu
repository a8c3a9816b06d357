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

#include "internal.h"
#include "rowvec.cuh"
#include "tc_ptx.cuh"

namespace ivfpq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kPerThread = IVFPQ_MAX_K / kThreads;  // list entries of one thread

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
  int chunk;     // columns of one block
};

// ---- exponentials relative to the row's maximum ------------------------------------
// exp((s - m) / tau) = 2^((s - m) c), c = log2(e) / tau. The difference first:
// its rounding error stays relative to the distance from the maximum, and no
// finite s and m overflow. m = -inf (nothing above it) is taken as 0, so that a
// score of -inf has the value 0 and a NaN stays.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
struct Base {
  float m, c;
  __device__ __forceinline__ Base(float m_, float c_) : m(m_ == -INFINITY ? 0.f : m_), c(c_) {}
  __device__ __forceinline__ float operator()(float s) const { return exp2_fast((s - m) * c); }
  // N values in place
  template <int N>
  __device__ __forceinline__ void all(float (&v)[N]) const {
    const uint64_t nm = pair(-m, -m), cc = pair(c, c);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float x, y;
      unpair(mul2(add2(pair(v[i], v[i + 1]), nm), cc), x, y);
      v[i] = exp2_fast(x);
      v[i + 1] = exp2_fast(y);
    }
  }
};

// A running maximum and sum; the sum is rescaled when the maximum grows.
struct Online {
  float m = -INFINITY, z = 0.f;
  __device__ __forceinline__ void rise(float t, float c) {
    if (t > m) {
      z *= m == -INFINITY ? 0.f : exp2_fast((m - t) * c);
      m = t;
    }
  }
  __device__ __forceinline__ void add(float v, float c) {
    rise(v, c);
    z += Base(m, c)(v);
  }
  // N values, t the largest of them
  template <int N>
  __device__ __forceinline__ void add(float (&v)[N], float t, float c) {
    rise(t, c);
    Base(m, c).all(v);
    uint64_t a = pair(v[0], v[1]);
#pragma unroll
    for (int i = 2; i < N; i += 2) a = add2(a, pair(v[i], v[i + 1]));
    float x, y;
    unpair(a, x, y);
    z += x + y;
  }
  __device__ __forceinline__ void join(float m2, float z2, float c) {
    const float t = fmaxf(m, m2);
    const float f1 = m == t ? 1.f : exp2_fast((m - t) * c);
    const float f2 = m2 == t ? 1.f : exp2_fast((m2 - t) * c);
    z = z * f1 + z2 * f2;
    m = t;
  }
};

// Sums over the block and joins of running maxima and sums, in a fixed order.
__device__ __forceinline__ float2 block_sum2(float2 v, float2* sh) {
#pragma unroll
  for (int o = 16; o; o /= 2) {
    v.x += __shfl_xor_sync(kFullMask, v.x, o);
    v.y += __shfl_xor_sync(kFullMask, v.y, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float2 r = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    r.x += sh[i].x;
    r.y += sh[i].y;
  }
  return r;
}
// The row's and the list's statistics in one step.
__device__ __forceinline__ void block_join(Online& o, Online& l, float c, float2* sh) {
#pragma unroll
  for (int d = 16; d; d /= 2) {
    o.join(__shfl_xor_sync(kFullMask, o.m, d), __shfl_xor_sync(kFullMask, o.z, d), c);
    l.join(__shfl_xor_sync(kFullMask, l.m, d), __shfl_xor_sync(kFullMask, l.z, d), c);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh[threadIdx.x >> 5] = make_float2(o.m, o.z);
    sh[kWarps + (threadIdx.x >> 5)] = make_float2(l.m, l.z);
  }
  __syncthreads();
  o = l = Online{};
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    o.join(sh[i].x, sh[i].y, c);
    l.join(sh[kWarps + i].x, sh[kWarps + i].y, c);
  }
}

// ---- the teacher's list ----------------------------------------------------------------
// A thread's entries i = threadIdx.x + q kThreads: value and column, -1 where
// the entry is not valid (its id is no column, or its value -inf: the padding
// of a short list); and the list's largest value and sum of exp((t - m) / tau),
// over the thread's entries until block_join. A sum of 0 means no valid entry.
struct Teacher {
  float v[kPerThread];
  int id[kPerThread];
  Online all;
  __device__ __forceinline__ bool any() const { return !(all.z == 0.f); }
  // softmax weight of entry q
  __device__ __forceinline__ float p(int q, float c, float inv_z) const {
    return exp2_fast((v[q] - all.m) * c) * inv_z;
  }
};
__device__ __forceinline__ void load_teacher(const DistillArgs& a, int64_t row, Teacher& t) {
  const float* tv = a.tv + row * a.k;
  const int64_t* ti = a.ti + row * a.k;
#pragma unroll
  for (int q = 0; q < kPerThread; ++q) {
    const int i = threadIdx.x + q * kThreads;
    t.id[q] = -1;
    t.v[q] = 0.f;
    if (i < a.k) {
      const float x = __ldg(tv + i) * a.sign;
      const int64_t id = __ldg(ti + i);
      if (id >= 0 && id < a.cols && x != -INFINITY) {
        t.id[q] = int(id);
        t.v[q] = x;
      }
    }
  }
}
__device__ __forceinline__ void teacher_stats(Teacher& t, float c) {
  t.all = Online{};
#pragma unroll
  for (int q = 0; q < kPerThread; ++q) {
    if (t.id[q] >= 0) {
      t.all.add(t.v[q], c);
    }
  }
}

// The gradient's values at the listed columns of [c0, c0 + len), one per entry,
// computed before any of them is written (the gradient may overwrite the
// scores). Entries with one column are found with a bitmap of the columns; only
// if there are any does a thread look through the list, in list order, for the
// sum of the weights of its column.
struct ListSmem {
  int* id;         // [k], relative to c0, -1 outside
  float* p;        // [k]
  uint32_t* seen;  // [chunk / 32]
};
__device__ __forceinline__ void list_to_smem(const DistillArgs& a, const Teacher& t, float c,
                                             int c0, int len, const ListSmem& l, int* repeated) {
  const float inv_tz = 1.f / t.all.z;
  for (int i = threadIdx.x; i < (len + 31) / 32; i += kThreads) l.seen[i] = 0;
  if (threadIdx.x == 0) *repeated = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPerThread; ++q) {
    const int i = threadIdx.x + q * kThreads;
    if (i < a.k) {
      const int id = t.id[q] - c0;
      const bool in = t.id[q] >= c0 && id < len;
      l.id[i] = in ? id : -1;
      l.p[i] = t.p(q, c, inv_tz);
      if (in && (atomicOr(&l.seen[id >> 5], 1u << (id & 31)) >> (id & 31)) & 1u) *repeated = 1;
    }
  }
  __syncthreads();
}
template <class Get>
__device__ __forceinline__ void list_values(const DistillArgs& a, const ListSmem& l, int repeated,
                                            const Base& b, float inv_z, float w, Get&& get,
                                            float (&fix)[kPerThread]) {
#pragma unroll
  for (int q = 0; q < kPerThread; ++q) {
    const int i = threadIdx.x + q * kThreads;
    if (i < a.k && l.id[i] >= 0) {
      float p = l.p[i];
      if (repeated) {
        p = 0.f;
        for (int j = 0; j < a.k; ++j)
          if (l.id[j] == l.id[i]) p += l.p[j];
      }
      fix[q] = w * (b(get(l.id[i])) * inv_z - p);
    }
  }
}
template <class T>
__device__ __forceinline__ void list_write(const DistillArgs& a, const ListSmem& l, T* g,
                                           const float (&fix)[kPerThread]) {
#pragma unroll
  for (int q = 0; q < kPerThread; ++q) {
    const int i = threadIdx.x + q * kThreads;
    if (i < a.k && l.id[i] >= 0) g[l.id[i]] = from_f32<T>(fix[q]);
  }
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

// Maximum and sum over a run of the row. With KEEP the run is also copied to
// shared memory, with the alignment it has in memory (keep is aligned as s).
template <class T, bool KEEP>
__device__ __forceinline__ Online run_stats(const T* s, int len, float c, T* keep) {
  constexpr int N = Span<T>::N, U = 4;
  const int mis = misalign(s);
  const T* from = s;
  if (KEEP && mis != 0) {
    const Span<T> sp(s, len);
    for (int e = threadIdx.x; e < sp.rest(); e += kThreads) keep[sp.at(e)] = s[sp.at(e)];
    const uint4* src = reinterpret_cast<const uint4*>(s + sp.head);
    uint4* dst = reinterpret_cast<uint4*>(keep + sp.head);
    for (int i = threadIdx.x; i < sp.nvec; i += U * kThreads) {
      uint4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kThreads < sp.nvec) r[u] = src[i + u * kThreads];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kThreads < sp.nvec) dst[i + u * kThreads] = r[u];
    }
    __syncthreads();
    from = keep;
  }
  Online o;
  auto sum = [&](const uint4& r, int i) {
    if (KEEP && mis == 0) reinterpret_cast<uint4*>(keep)[i] = r;
    float v[N];
    unpack_vec<T>(r, v);
    o.add(v, vec_max(r, static_cast<T*>(nullptr)), c);
  };
  // a thread's vectors in ascending order: U inner ones at a time, the others
  // one by one
  const int nvec = (len + N - 1) / N, last = inner_last<T>(len, mis);
  int i = threadIdx.x;
  if (mis != 0 && i < nvec) {
    sum(load_vec(from, len, i, mis), i);
    i += kThreads;
  }
  for (; i + (U - 1) * kThreads <= last; i += U * kThreads) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = load_inner(from, i + u * kThreads, mis);
#pragma unroll
    for (int u = 0; u < U; ++u) sum(r[u], i + u * kThreads);
  }
#pragma unroll 1
  for (; i < nvec; i += kThreads) sum(load_vec(from, len, i, mis), i);
  return o;
}

// g = r exp(...) over a run, from global or shared scores, by the 16-byte
// vectors of g.
template <class T>
__device__ __forceinline__ void run_grad(const T* s, int len, const Base& b, float r, T* g) {
  constexpr int N = Span<T>::N;
  const Span<T> sp(g, len);
  for (int e = threadIdx.x; e < sp.rest(); e += kThreads)
    g[sp.at(e)] = from_f32<T>(b(to_f32(s[sp.at(e)])) * r);
  const T* src = s + sp.head;
  const int mis = misalign(src);
  uint4* dst = reinterpret_cast<uint4*>(g + sp.head);
  constexpr int U = 4;
  const int n = len - sp.head, last = min(sp.nvec - 1, inner_last<T>(n, mis));
  auto put = [&](const uint4& x, int i) {
    float v[N];
    unpack_vec<T>(x, v);
    b.all(v);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] *= r;
    dst[i] = pack_vec<T>(v);
  };
  int i = threadIdx.x;
  if (mis != 0 && i < sp.nvec) {
    put(load_vec(src, n, i, mis), i);
    i += kThreads;
  }
  for (; i + (U - 1) * kThreads <= last; i += U * kThreads) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = load_inner(src, i + u * kThreads, mis);
#pragma unroll
    for (int u = 0; u < U; ++u) put(x[u], i + u * kThreads);
  }
#pragma unroll 1
  for (; i < sp.nvec; i += kThreads) put(load_vec(src, n, i, mis), i);
}
template <class T>
__device__ __forceinline__ void run_zero(T* g, int len) {
  const Span<T> sp(g, len);
  for (int e = threadIdx.x; e < sp.rest(); e += kThreads) g[sp.at(e)] = from_f32<T>(0.f);
  for (int i = threadIdx.x; i < sp.nvec; i += kThreads)
    reinterpret_cast<uint4*>(g + sp.head)[i] = make_uint4(0, 0, 0, 0);
}

// The cluster's blocks each hold (x, y) in *mine; returns all of them joined
// with f in rank order. A second barrier later keeps *mine alive for readers.
template <class F>
__device__ __forceinline__ void cluster_each(float2 v, float2* mine, int nranks, F&& f) {
  if (threadIdx.x == 0) *mine = v;
  if (nranks == 1) {
    f(v);
    return;
  }
  cluster_sync();
  const uint32_t at = smem_u32(mine);
  for (int r = 0; r < nranks; ++r) f(make_float2(ld_cluster(at, r), ld_cluster(at + 4, r)));
}

// Loss over the entries in [c0, c0 + len): tau^2 sum p (log p + log Z) - tau
// sum p (s - m). No s - m is divided by tau, so that a listed score of the
// type's lowest value stays finite.
template <class Get>
__device__ __forceinline__ float2 list_loss(const DistillArgs& a, const Teacher& t, float c, int c0,
                                            int len, float m, float logz, Get&& get) {
  float2 l = make_float2(0.f, 0.f);
  const float inv_tz = 1.f / t.all.z, logtz = logf(t.all.z);
#pragma unroll
  for (int q = 0; q < kPerThread; ++q) {
    const int id = t.id[q] - c0;
    if (t.id[q] >= c0 && id < len) {
      const float p = t.p(q, c, inv_tz), s = get(id);
      if (!(p <= 0.f)) {  // also a NaN
        l.x += p * ((t.v[q] - t.all.m) * a.inv_tau - logtz + logz);
        l.y += p * (s == -INFINITY ? s : s - m);
      }
    }
  }
  return l;
}

// Loss and statistics: a cluster of blocks per row, a run of columns each.
template <class T>
__global__ void __launch_bounds__(kThreads, 4) distill_forward_kernel(const DistillArgs a) {
  __shared__ float2 sh[2 * kWarps];
  __shared__ float2 part[2];
  const int nranks = int(gridDim.x), rank = int(blockIdx.x);  // the cluster is a row of the grid
  const int64_t row = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  if (row >= a.rows) return;  // whole clusters
  const int c0 = int(min(int64_t(rank) * a.chunk, a.cols));
  const int len = int(min(int64_t(a.chunk), a.cols - c0));
  const T* s = static_cast<const T*>(a.scores) + row * a.lds + c0;
  const float c = a.inv_tau * kLog2e;
  Teacher t;
  load_teacher(a, row, t);
  Online o = run_stats<T, false>(s, len, c, nullptr);
  teacher_stats(t, c);
  block_join(o, t.all, c, sh);
  Online all;
  cluster_each(make_float2(o.m, o.z), &part[0], nranks,
               [&](float2 v) { all.join(v.x, v.y, c); });
  const float logz = all.z == 0.f ? 0.f : logf(all.z);
  float2 l = list_loss(a, t, c, c0, len, all.m, logz, [&](int i) { return to_f32(s[i]); });
  l = block_sum2(l, sh);
  float2 sum = make_float2(0.f, 0.f);
  cluster_each(l, &part[1], nranks, [&](float2 v) {
    sum.x += v.x;
    sum.y += v.y;
  });
  if (rank == 0 && threadIdx.x == 0) {
    a.loss[row] = t.any() ? a.tau * (a.tau * sum.x - sum.y) : 0.f;
    a.stats[2 * row] = all.m;
    a.stats[2 * row + 1] = all.z;
  }
  if (nranks > 1) cluster_sync();
}

// Gradient from the forward's statistics: a block per run of columns.
template <class T>
__global__ void __launch_bounds__(kThreads, 4) distill_backward_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) uint8_t distill_smem[];
  __shared__ float2 sh[2 * kWarps];
  __shared__ int repeated;
  const int64_t row = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  if (row >= a.rows) return;
  const int c0 = int(blockIdx.x) * a.chunk;
  const int len = int(min(int64_t(a.chunk), a.cols - c0));
  const T* s = static_cast<const T*>(a.scores) + row * a.lds + c0;
  T* g = static_cast<T*>(a.grad) + row * a.ldg + c0;
  const float w = a.row_grad[row] * a.tau;
  if (w == 0.f) return run_zero(g, len);  // a row that does not count, whatever it holds
  const float c = a.inv_tau * kLog2e;
  Teacher t;
  load_teacher(a, row, t);
  teacher_stats(t, c);
  Online none;
  block_join(none, t.all, c, sh);
  ListSmem l;
  l.id = reinterpret_cast<int*>(distill_smem);
  l.p = reinterpret_cast<float*>(l.id + a.k);
  l.seen = reinterpret_cast<uint32_t*>(l.p + a.k);
  list_to_smem(a, t, c, c0, len, l, &repeated);
  const float m = a.stats[2 * row], z = a.stats[2 * row + 1];
  const Base b(m, c);
  const float inv_z = z == 0.f ? 0.f : 1.f / z;  // no score above -inf: q = 0
  float fix[kPerThread];
  list_values(a, l, repeated, b, inv_z, w, [&](int i) { return to_f32(s[i]); }, fix);
  __syncthreads();
  if (t.any())
    run_grad<T>(s, len, b, w * inv_z, g);
  else
    run_zero(g, len);
  __syncthreads();
  list_write(a, l, g, fix);
}

// Loss and gradient with the row held in the shared memory of a cluster: each
// score is read from memory once.
template <class T>
__global__ void __launch_bounds__(kThreads, 4) distill_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) uint8_t distill_smem[];
  __shared__ float2 sh[2 * kWarps];
  __shared__ float2 part[2];
  __shared__ int repeated;
  const int nranks = int(gridDim.x), rank = int(blockIdx.x);
  const int64_t row = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  if (row >= a.rows) return;
  const int c0 = int(min(int64_t(rank) * a.chunk, a.cols));
  const int len = int(min(int64_t(a.chunk), a.cols - c0));
  const T* s = static_cast<const T*>(a.scores) + row * a.lds + c0;
  T* g = static_cast<T*>(a.grad) + row * a.ldg + c0;
  const float c = a.inv_tau * kLog2e;
  T* keep = reinterpret_cast<T*>(distill_smem) + misalign(s) / int(sizeof(T));
  ListSmem l;
  l.id = reinterpret_cast<int*>(distill_smem + (size_t(a.chunk) + Span<T>::N) * sizeof(T));
  l.p = reinterpret_cast<float*>(l.id + a.k);
  l.seen = reinterpret_cast<uint32_t*>(l.p + a.k);

  Teacher t;
  load_teacher(a, row, t);
  Online o = run_stats<T, true>(s, len, c, keep);
  teacher_stats(t, c);
  block_join(o, t.all, c, sh);  // its barriers also publish the copy
  Online all;
  cluster_each(make_float2(o.m, o.z), &part[0], nranks,
               [&](float2 v) { all.join(v.x, v.y, c); });
  auto score = [&](int i) { return to_f32(keep[i]); };
  const float logz = all.z == 0.f ? 0.f : logf(all.z);
  const float2 mine = block_sum2(list_loss(a, t, c, c0, len, all.m, logz, score), sh);
  float2 sum = make_float2(0.f, 0.f);
  cluster_each(mine, &part[1], nranks, [&](float2 v) {
    sum.x += v.x;
    sum.y += v.y;
  });
  if (rank == 0 && threadIdx.x == 0)
    a.loss[row] = t.any() ? a.tau * (a.tau * sum.x - sum.y) : 0.f;

  const float w = a.row_grad[row] * a.tau;
  if (w == 0.f || !t.any()) {
    run_zero(g, len);
  } else {
    const Base b(all.m, c);
    const float inv_z = all.z == 0.f ? 0.f : 1.f / all.z;
    list_to_smem(a, t, c, c0, len, l, &repeated);
    float fix[kPerThread];
    list_values(a, l, repeated, b, inv_z, w, score, fix);
    run_grad<T>(keep, len, b, w * inv_z, g);
    __syncthreads();
    list_write(a, l, g, fix);
  }
  if (nranks > 1) cluster_sync();
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

dim3 grid_of(int64_t per_row, int64_t rows) {
  const int64_t y = std::min<int64_t>(rows, 65535);
  return dim3(unsigned(per_row), unsigned(y), unsigned(ceil_div(rows, y)));
}

template <class K>
int launch_cluster(K kern, const DistillArgs& a, int ranks, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid_of(ranks, a.rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(ranks);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
  IVFPQ_LAUNCHED_K(kern, smem, kThreads);
  return IVFPQ_OK;
}

// Columns of one block when a row is split over `ranks` blocks.
int chunk_of(int64_t cols, int ranks) { return int(ceil_div(ceil_div(cols, ranks), 8) * 8); }

// More blocks per row while the rows alone do not fill the device twice, down
// to runs of 4,096 columns.
int ranks_for(int64_t rows, int64_t cols, int ranks) {
  while (ranks < kMaxCluster && rows * ranks < 2 * num_sms() && cols > 4096 * int64_t(ranks))
    ranks *= 2;
  return ranks;
}

int launch_forward(DistillArgs a, int dtype, cudaStream_t s) {
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    const int ranks = ranks_for(a.rows, a.cols, 1);
    a.chunk = chunk_of(a.cols, ranks);
    return launch_cluster(distill_forward_kernel<T>, a, ranks, 0, s);
  });
}
int launch_backward(DistillArgs a, int dtype, cudaStream_t s) {
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    // runs long enough to carry the list's work, short enough to fill the
    // device; at most 65,536 columns, whose bitmap takes 8 KB
    int64_t per_row = ceil_div(a.cols, 65536);
    while (a.rows * per_row < 4 * num_sms() && a.cols > 4096 * per_row) per_row *= 2;
    a.chunk = chunk_of(a.cols, int(per_row));
    per_row = ceil_div(a.cols, a.chunk);
    const size_t smem = size_t(a.k) * 8 + size_t(ceil_div(a.chunk, 32)) * 4;
    distill_backward_kernel<T><<<grid_of(per_row, a.rows), kThreads, smem, s>>>(a);
    IVFPQ_LAUNCHED();
    return IVFPQ_OK;
  });
}
// Loss and gradient in one kernel where eight blocks can hold a row.
bool fits_cluster(const DistillArgs& a, int dtype, int* ranks, size_t* smem) {
  const int size = dtype_size(dtype);
  auto bytes = [&](int r) {
    const int64_t ch = chunk_of(a.cols, r);
    return size_t(ch + 16 / size) * size + size_t(a.k) * 8 + size_t(ceil_div(ch, 32)) * 4;
  };
  // three blocks share an SM's shared memory, so that one loads while another
  // computes or stores; two or one where a row is too long for that
  int r = 1;
  while (r < kMaxCluster && bytes(r) > 75 * 1024) r *= 2;
  r = ranks_for(a.rows, a.cols, r);
  *ranks = r;
  *smem = bytes(r);
  return *smem <= 224 * 1024;
}
int launch_both(DistillArgs a, int dtype, int ranks, size_t smem, cudaStream_t s) {
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    a.chunk = chunk_of(a.cols, ranks);
    IVFPQ_TRY(set_dynamic_smem(distill_kernel<T>, smem));
    return launch_cluster(distill_kernel<T>, a, ranks, smem, s);
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
  DistillArgs a = distill_args(scores, rows, cols, lds, teacher_vals, teacher_ids, k, temperature,
                               negated);
  a.loss = loss;
  a.row_grad = row_grad;
  a.grad = grad;
  a.ldg = ldg;
  int ranks = 0;
  size_t smem = 0;
  if (fits_cluster(a, dtype, &ranks, &smem)) return launch_both(a, dtype, ranks, smem, s);
  Workspace ws(s);
  IVFPQ_TRY(ws.alloc(&a.stats, size_t(rows) * 2));
  IVFPQ_TRY(launch_forward(a, dtype, s));
  return launch_backward(a, dtype, s);
}
