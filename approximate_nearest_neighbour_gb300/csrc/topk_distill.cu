// topk_distill_*: distillation of a student's score rows from a teacher's top
// list (the values and ids a k-selection or a search returns). With the
// temperature tau and the valid entries i of a row's list
//   p_i = softmax_i(t_i / tau),  q_j = softmax_j(s_j / tau) over all columns,
//   loss = tau^2 sum_i p_i (log p_i - log q_id(i)),
//   d loss / d s_j = tau (P q_j - sum_{i: id(i) = j} p_i),  P = sum_i p_i
// (1, or 0 for a list without valid entries, whose loss and gradient are 0).
//
// Bound by memory: the forward pass reads each score once, the backward pass
// reads and writes each once, and so does topk_distill, which holds a row in the
// shared memory of a cluster of up to eight blocks between its two uses (rows
// too long for that take the two passes). Measured on the device at 2048 x 65536
// bf16, k = 100: forward 51 us (40 us at the measured copy rate), backward 92 us
// (81 us; 82 us at 65537 columns, which two blocks share), both in one 119 us (81
// us), where the exponentials of both uses and the exchange between them are not
// hidden behind three blocks per SM. Rows of odd length cost the forward pass its
// shifted loads (2048 x 65537: 72 us), and short rows are bound by the joins and
// list work of a whole block per row (4000 x 5001 binary16, k = 300: both in one 52
// us, 14 us for the bytes).
//
// Statistics kept per row: the largest score m and Z = sum_j exp((s_j - m) /
// tau), both fp32; q_j comes from the difference s_j - m, so scores of any
// magnitude (a mask of the type's lowest value among them) neither overflow nor
// cancel. A score of -inf has q = 0.
#include <algorithm>

#include "internal.h"
#include "rowvec.cuh"
#include "tc_ptx.cuh"

namespace ivfpq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;  // a power of two
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.44269504088896340736f;

struct DistillArgs {
  const void* scores;
  int64_t rows, cols, lds;
  const float* tv;
  const int64_t* ti;
  int k;
  float tau, inv_tau, sign;
  float tau_small, tau_large;  // tau kSmall, tau / kSmall
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
};

// Joins of running maxima and sums over the block, in a fixed order.
// What a sum relative to the maximum m is, relative to the larger t.
__device__ __forceinline__ float rescaled(float m, float z, float t, float c) {
  return m == t ? z : z * exp2_fast((m - t) * c);
}
// The row's and the list's statistics in one step: maxima first, so that each
// sum is rescaled once and the exponentials do not wait for each other.
__device__ __forceinline__ void block_join(Online& o, Online& l, float c, float4* sh) {
  float mo = o.m, ml = l.m;
#pragma unroll
  for (int d = 16; d; d /= 2) {
    mo = fmaxf(mo, __shfl_xor_sync(kFullMask, mo, d));
    ml = fmaxf(ml, __shfl_xor_sync(kFullMask, ml, d));
  }
  float zo = rescaled(o.m, o.z, mo, c), zl = rescaled(l.m, l.z, ml, c);
#pragma unroll
  for (int d = 16; d; d /= 2) {
    zo += __shfl_xor_sync(kFullMask, zo, d);
    zl += __shfl_xor_sync(kFullMask, zl, d);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float4(mo, zo, ml, zl);
  __syncthreads();
  // lane i takes warp i's
  const int lane = threadIdx.x & 31;
  const float4 v = lane < kWarps ? sh[lane] : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
  mo = v.x;
  ml = v.z;
#pragma unroll
  for (int d = kWarps / 2; d; d /= 2) {
    mo = fmaxf(mo, __shfl_xor_sync(kFullMask, mo, d));
    ml = fmaxf(ml, __shfl_xor_sync(kFullMask, ml, d));
  }
  zo = rescaled(v.x, v.y, mo, c);
  zl = rescaled(v.z, v.w, ml, c);
#pragma unroll
  for (int d = kWarps / 2; d; d /= 2) {
    zo += __shfl_xor_sync(kFullMask, zo, d);
    zl += __shfl_xor_sync(kFullMask, zl, d);
  }
  o.m = __shfl_sync(kFullMask, mo, 0);
  o.z = __shfl_sync(kFullMask, zo, 0);
  l.m = __shfl_sync(kFullMask, ml, 0);
  l.z = __shfl_sync(kFullMask, zl, 0);
}

// ---- the teacher's list ----------------------------------------------------------------
// In shared memory; thread t handles the entries t, t + kThreads, ... in every
// step, so that they need no barrier between steps. An entry is valid if its
// id is a column and its value not -inf (the padding of a short list).
struct List {
  int* id;         // [k] column, -1 where not valid; then relative to the block's run, -1 outside
  float* p;        // [k] value; then softmax weight; then the gradient at the column
  float* fix;      // [k]
  uint32_t* seen;  // [chunk / 32] columns of the run that are listed
  __device__ __forceinline__ List(uint8_t* smem, int k) {
    id = reinterpret_cast<int*>(smem);
    p = reinterpret_cast<float*>(id + k);
    fix = p + k;
    seen = reinterpret_cast<uint32_t*>(fix + k);
  }
};
inline size_t list_bytes(int k, int64_t chunk) {
  return size_t(k) * 12 + size_t(ceil_div(chunk, 32)) * 4;
}

// Loads the row's entries; returns the largest value and the sum of
// exp((t - m) / tau) over the thread's. A sum of 0 means no valid entry.
__device__ __forceinline__ Online list_load(const DistillArgs& a, int64_t row, const List& l,
                                            float c) {
  Online o;
#pragma unroll 4
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    const float x = __ldg(a.tv + row * a.k + i) * a.sign;
    const int64_t id = __ldg(a.ti + row * a.k + i);
    const bool ok = id >= 0 && id < a.cols && x != -INFINITY;
    l.id[i] = ok ? int(id) : -1;
    l.p[i] = x;
    if (ok) o.add(x, c);
  }
  return o;
}

// What the loss needs of a run of columns, with p and t over the entries in it:
// sum p log p, sum p, sum p (s - m) kSmall, m the run's own maximum. kSmall, a
// power of two, leaves room above: a list masked throughout by fp32's lowest value
// has differences of that size, and its weights may sum to a little more than 1.
constexpr float kSmall = 0x1p-8f;
struct LossPart {
  float a = 0.f, p = 0.f, y = 0.f;
};
// Entries to run-relative columns and softmax weights; with LOSS their part of
// the loss; with MARK a bitmap of the listed columns (cleared before), and
// *repeated if one comes twice.
template <bool LOSS, bool MARK, class Get>
__device__ __forceinline__ LossPart list_weights(const DistillArgs& a, const List& l,
                                                 const Online& t, float c, int c0, int len, float m,
                                                 int* repeated, Get&& get) {
  LossPart r;
  const float inv_tz = 1.f / t.z, logtz = logf(t.z);
#pragma unroll 1
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    const int id = l.id[i] - c0;
    const bool in = l.id[i] >= c0 && id < len;
    l.id[i] = in ? id : -1;
    if (in) {
      const float v = l.p[i], p = exp2_fast((v - t.m) * c) * inv_tz;
      l.p[i] = p;
      if (LOSS && !(p <= 0.f)) {  // also a NaN
        const float s = get(id);
        r.a += p * ((v - t.m) * a.inv_tau - logtz);
        r.p += p;
        r.y += p * kSmall * (s == -INFINITY ? s : s - m);
      }
      if (MARK && (atomicOr(&l.seen[id >> 5], 1u << (id & 31)) >> (id & 31)) & 1u) *repeated = 1;
    }
  }
  return r;
}
// The gradient at the listed columns, one value per entry, computed before any
// is written (the gradient may overwrite the scores). Only if a column comes
// twice does a thread look through the list, in list order, for the sum of its
// weights.
template <class Get>
__device__ __forceinline__ void list_values(const DistillArgs& a, const List& l, bool repeated,
                                            const Base& b, float inv_z, float w, Get&& get) {
#pragma unroll 4
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    const int id = l.id[i];
    if (id >= 0) {
      float p = l.p[i];
      if (repeated) {
        p = 0.f;
#pragma unroll 1
        for (int j = 0; j < a.k; ++j)
          if (l.id[j] == id) p += l.p[j];
      }
      l.fix[i] = w * (b(get(id)) * inv_z - p);
    }
  }
}
template <class T>
__device__ __forceinline__ void list_write(const DistillArgs& a, const List& l, T* g) {
#pragma unroll 1
  for (int i = threadIdx.x; i < a.k; i += kThreads)
    if (l.id[i] >= 0) g[l.id[i]] = from_f32<T>(l.fix[i]);
}

// The sums of a thread's vectors go on in ascending order of their index.
template <class T>
__device__ __forceinline__ void sum_vec(Online& o, const uint4& r, float c) {
  float v[Span<T>::N];
  unpack_vec<T>(r, v);
  o.add(v, vec_max(r, static_cast<T*>(nullptr)), c);
}

// Maximum and sum over a run of the row. AHEAD: the run is in global memory, and
// is brought into L2 kAhead steps before it is read.
constexpr int kAhead = 3;
template <class T, bool AHEAD>
__device__ __forceinline__ Online run_stats(const T* s, int len, float c) {
  constexpr int N = Span<T>::N, U = 4;
  const int mis = misalign(s);
  Online o;
  if (AHEAD && threadIdx.x == 0) prefetch_run(s, 0, kAhead * U * kThreads * 16, s + len);
  // U inner vectors at a time, the others one by one
  const int nvec = (len + N - 1) / N, last = inner_last<T>(len, mis);
  int i = threadIdx.x;
  if (mis != 0 && i < nvec) {
    sum_vec<T>(o, load_vec(s, len, i, mis), c);
    i += kThreads;
  }
  for (; i + (U - 1) * kThreads <= last; i += U * kThreads) {
    uint4 r[U];
    if (AHEAD && threadIdx.x == 0)
      prefetch_run(s, (i + kAhead * U * kThreads) * 16, U * kThreads * 16, s + len);
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = load_inner(s, i + u * kThreads, mis);
#pragma unroll
    for (int u = 0; u < U; ++u) sum_vec<T>(o, r[u], c);
  }
#pragma unroll 1
  for (; i < nvec; i += kThreads) sum_vec<T>(o, load_vec(s, len, i, mis), c);
  return o;
}

// The same, with the run copied to shared memory, where it keeps the alignment
// it has in memory (keep is aligned as s). All copies are started at once, in
// four groups, so that a block's whole run is on its way from memory while the
// blocks beside it compute.
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}
template <class T, class F>
__device__ __forceinline__ Online run_stats_keep(const T* s, int len, float c, T* keep,
                                                 F&& meanwhile) {
  constexpr int N = Span<T>::N, G = 4;
  const int mis = misalign(s);
  const Span<T> sp(s, len);
  const uint4* src = reinterpret_cast<const uint4*>(s + sp.head);
  uint4* dst = reinterpret_cast<uint4*>(keep + sp.head);
  const int per = (sp.nvec + G * kThreads - 1) / (G * kThreads);  // vectors of a thread and group
  const uint32_t to = smem_u32(dst);
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    for (int v = 0; v < per; ++v) {
      const int i = threadIdx.x + (g * per + v) * kThreads;
      if (i < sp.nvec)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16u * uint32_t(i)),
                     "l"(src + i)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (int e = threadIdx.x; e < sp.rest(); e += kThreads) keep[sp.at(e)] = s[sp.at(e)];
  meanwhile();
  Online o;
  if (mis == 0) {
    // a thread's own copies, group by group
    auto group = [&](int g) {
      constexpr int U = 4;
      for (int v0 = 0; v0 < per; v0 += U) {
        uint4 r[U];
        const int i0 = threadIdx.x + (g * per + v0) * kThreads;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u < per && i0 + u * kThreads < sp.nvec) r[u] = dst[i0 + u * kThreads];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u < per && i0 + u * kThreads < sp.nvec) sum_vec<T>(o, r[u], c);
      }
    };
    copies_wait<3>();
    group(0);
    copies_wait<2>();
    group(1);
    copies_wait<1>();
    group(2);
    copies_wait<0>();
    group(3);
    if (len > sp.nvec * N && sp.nvec % kThreads == int(threadIdx.x))
      sum_vec<T>(o, load_edge(s, len, sp.nvec), c);
  } else {
    copies_wait<0>();
    __syncthreads();
    o = run_stats<T, false>(keep, len, c);
  }
  return o;
}

// g = r exp(...) over a run, from global or shared scores, by the 16-byte
// vectors of g.
template <class T, bool AHEAD>
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
    for (int j = 0; j < N; j += 2) unpair(mul2(pair(v[j], v[j + 1]), pair(r, r)), v[j], v[j + 1]);
    dst[i] = pack_vec<T>(v);
  };
  int i = threadIdx.x;
  if (mis != 0 && i < sp.nvec) {
    put(load_vec(src, n, i, mis), i);
    i += kThreads;
  }
  for (; i + (U - 1) * kThreads <= last; i += U * kThreads) {
    uint4 x[U];
    if (AHEAD && threadIdx.x == 0)
      prefetch_run(src, (i + kAhead * U * kThreads) * 16, U * kThreads * 16, s + len);
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

// A block's part of a row's statistics and loss, and their join over the
// cluster in a fixed order. The parts' owners stay until all have read them
// (cluster_leave); what is in between overlaps with the others' reading.
struct __align__(16) RowPart {
  float m, z;
  LossPart l;
  float pad[3];
};
struct RowSum {
  Online all;
  float x = 0.f, y = 0.f;  // sum p (log p + log Z), sum p (s - m) kSmall
};
__device__ __forceinline__ RowSum row_join(const Online& o, const LossPart& part, RowPart* mine,
                                           int nranks, float c) {
  RowSum s;
  if (nranks == 1) {
    s.all = o;
    s.x = part.a + (o.z == 0.f ? 0.f : logf(o.z)) * part.p;
    s.y = part.y;
    return s;
  }
  if (threadIdx.x == 0) {
    mine->m = o.m;
    mine->z = o.z;
    mine->l = part;
  }
  cluster_sync();
  // lane r reads rank r's part
  const int lane = threadIdx.x & 31;
  float4 v = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  float y = 0.f;
  if (lane < nranks) {
    const uint32_t at = map_rank(smem_u32(mine), uint32_t(lane));
    v = ld_cluster4(at);
    y = ld_cluster4(at + 16).x;
  }
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  float m = v.x;
#pragma unroll
  for (int d = kMaxCluster / 2; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, d));
  m = __shfl_sync(kFullMask, m, 0);
  float z = rescaled(v.x, v.y, m, c), x = v.z, p = v.w;
  // the part's differences are from its own maximum
  if (!(p == 0.f) && v.x != m) y += (v.x - m) * (p * kSmall);
#pragma unroll
  for (int d = kMaxCluster / 2; d; d /= 2) {
    z += __shfl_xor_sync(kFullMask, z, d);
    x += __shfl_xor_sync(kFullMask, x, d);
    p += __shfl_xor_sync(kFullMask, p, d);
    y += __shfl_xor_sync(kFullMask, y, d);
  }
  s.all.m = m;
  s.all.z = __shfl_sync(kFullMask, z, 0);
  s.x = x;  // these two count in thread 0 only
  s.y = y;
  s.x += (s.all.z == 0.f ? 0.f : logf(s.all.z)) * p;
  return s;
}
__device__ __forceinline__ float row_loss(const DistillArgs& a, const Online& t, const RowSum& r) {
  return t.z == 0.f ? 0.f : a.tau_large * (a.tau_small * r.x - r.y);
}
__device__ __forceinline__ void cluster_leave(int nranks) {
  if (nranks > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Sums over the block, in a fixed order, for thread 0.
__device__ __forceinline__ LossPart block_loss(LossPart l, float4* sh) {
#pragma unroll
  for (int o = 16; o; o /= 2) {
    l.a += __shfl_xor_sync(kFullMask, l.a, o);
    l.p += __shfl_xor_sync(kFullMask, l.p, o);
    l.y += __shfl_xor_sync(kFullMask, l.y, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float4(l.a, l.p, l.y, 0.f);
  __syncthreads();
  // of use to thread 0 only
  const int lane = threadIdx.x & 31;
  const float4 v = lane < kWarps ? sh[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
  l.a = v.x;
  l.p = v.y;
  l.y = v.z;
#pragma unroll
  for (int d = kWarps / 2; d; d /= 2) {
    l.a += __shfl_xor_sync(kFullMask, l.a, d);
    l.p += __shfl_xor_sync(kFullMask, l.p, d);
    l.y += __shfl_xor_sync(kFullMask, l.y, d);
  }
  return l;
}

// Loss and statistics: a cluster of blocks per row, a run of columns each.
template <class T>
__global__ void __launch_bounds__(kThreads, 4) distill_forward_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) uint8_t distill_smem[];
  __shared__ float4 sh[kWarps];
  __shared__ RowPart part;
  const int nranks = int(gridDim.x), rank = int(blockIdx.x);  // the cluster is a row of the grid
  const int64_t row = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  if (row >= a.rows) return;  // whole clusters
  const int c0 = int(min(int64_t(rank) * a.chunk, a.cols));
  const int len = int(min(int64_t(a.chunk), a.cols - c0));
  const T* s = static_cast<const T*>(a.scores) + row * a.lds + c0;
  const float c = a.inv_tau * kLog2e;
  const List l(distill_smem, a.k);
  Online t = list_load(a, row, l, c);
  Online o = run_stats<T, true>(s, len, c);
  block_join(o, t, c, sh);
  auto score = [&](int i) { return to_f32(s[i]); };
  const LossPart mine =
      block_loss(list_weights<true, false>(a, l, t, c, c0, len, o.m, nullptr, score), sh);
  const RowSum r = row_join(o, mine, &part, nranks, c);
  if (rank == 0 && threadIdx.x == 0) {
    a.loss[row] = row_loss(a, t, r);
    a.stats[2 * row] = r.all.m;
    a.stats[2 * row + 1] = r.all.z;
  }
  cluster_leave(nranks);
}

// Gradient from the forward's statistics: a block per run of columns.
template <class T>
__global__ void __launch_bounds__(kThreads, 4) distill_backward_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) uint8_t distill_smem[];
  __shared__ float4 sh[kWarps];
  __shared__ int repeated;
  const int64_t row = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  if (row >= a.rows) return;
  const int c0 = int(blockIdx.x) * a.chunk;
  const int len = int(min(int64_t(a.chunk), a.cols - c0));
  const T* s = static_cast<const T*>(a.scores) + row * a.lds + c0;
  T* g = static_cast<T*>(a.grad) + row * a.ldg + c0;
  const float w = a.row_grad[row] * a.tau;
  if (w == 0.f) return run_zero(g, len);  // a row that does not count, whatever it holds
  if (threadIdx.x == 0) prefetch_run(s, 0, kAhead * 4 * kThreads * 16, s + len);
  const float c = a.inv_tau * kLog2e;
  const List l(distill_smem, a.k);
  Online t = list_load(a, row, l, c), none;
  for (int i = threadIdx.x; i < (len + 31) / 32; i += kThreads) l.seen[i] = 0;
  if (threadIdx.x == 0) repeated = 0;
  block_join(none, t, c, sh);
  const float m = a.stats[2 * row], z = a.stats[2 * row + 1];
  auto score = [&](int i) { return to_f32(s[i]); };
  list_weights<false, true>(a, l, t, c, c0, len, m, &repeated, score);
  __syncthreads();
  const Base b(m, c);
  const float inv_z = z == 0.f ? 0.f : 1.f / z;  // no score above -inf: q = 0
  list_values(a, l, repeated != 0, b, inv_z, w, score);
  __syncthreads();
  if (t.z == 0.f)
    run_zero(g, len);
  else
    run_grad<T, true>(s, len, b, w * inv_z, g);
  __syncthreads();
  list_write(a, l, g);
}

// Loss and gradient with the row held in the shared memory of a cluster: each
// score is read from memory once.
template <class T>
__global__ void __launch_bounds__(kThreads, 4) distill_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) uint8_t distill_smem[];
  __shared__ float4 sh[kWarps];
  __shared__ RowPart part;
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
  const List l(distill_smem + (size_t(a.chunk) + Span<T>::N) * sizeof(T), a.k);
  const float w = a.row_grad[row] * a.tau;

  Online t;
  Online o = run_stats_keep<T>(s, len, c, keep, [&] {
    t = list_load(a, row, l, c);
    for (int i = threadIdx.x; i < (len + 31) / 32; i += kThreads) l.seen[i] = 0;
    if (threadIdx.x == 0) repeated = 0;
  });
  block_join(o, t, c, sh);  // its barriers also publish the copy
  auto score = [&](int i) { return to_f32(keep[i]); };
  const LossPart mine =
      block_loss(list_weights<true, true>(a, l, t, c, c0, len, o.m, &repeated, score), sh);
  const RowSum r = row_join(o, mine, &part, nranks, c);
  if (rank == 0 && threadIdx.x == 0)
    a.loss[row] = row_loss(a, t, r);
  if (w == 0.f || t.z == 0.f) {
    run_zero(g, len);
  } else {
    const Base b(r.all.m, c);
    const float inv_z = r.all.z == 0.f ? 0.f : 1.f / r.all.z;
    list_values(a, l, repeated != 0, b, inv_z, w, score);
    run_grad<T, false>(keep, len, b, w * inv_z, g);
    __syncthreads();
    list_write(a, l, g);
  }
  cluster_leave(nranks);
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
  a.tau_small = temperature * kSmall;
  a.tau_large = temperature / kSmall;
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
    return launch_cluster(distill_forward_kernel<T>, a, ranks, list_bytes(a.k, 0), s);
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
    const size_t smem = list_bytes(a.k, a.chunk);
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
    return size_t(ch + 16 / size) * size + list_bytes(a.k, ch);
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
