// beam_select: the k best continuations of every request's beams. For beam b of
// a group, with t its running total and s its score row,
//   total(b, c) = t + s_c - log sum_j exp(s_j)
// and the k largest over (b, c) are taken, equal ones by (b, c). A finished beam
// has one continuation, (b, end_id), whose total is t.
//
// Bound by memory: each score is read once. Within a row totals are ordered as
// scores, so a row's own k best are enough and need no normalisation:
//  1. One pass keeps per thread the largest score and the sum of exponentials
//     relative to it (rescaled when it grows), and of every four vectors that a
//     thread takes (a batch) the largest score, in shared memory.
//  2. The k-th largest of the threads' maxima is a lower bound of the k-th largest
//     score; every warp finds it, or something a little lower, by halving the range
//     between them. Only batches that reach the bound are read again, a vector per
//     thread, from L2, and their scores at or above it kept.
//  3. The kept ones are ranked among themselves. Where a cluster of blocks shares a
//     row, its first block gets the lists of the others and ranks all of them.
//  4. Totals are compared in fp64: they differ by the rounding of their sums of
//     exponentials, not of the comparison. Where few beams have few continuations, a
//     cluster takes a whole group and its first block ranks the beams' lists too (one
//     kernel, no workspace); else a second kernel, already waiting, merges the
//     beams' lists of a group, two at a time.
// Keys hold (score, inverted column), so that no step depends on the order in
// which threads append and the lowest column of equal scores comes first.
//
// Measured on the device: 64 x 8 rows of 131072 bf16, k = 16 (134 MB) 28.9 us, 4.6 TB/s
// (at the copy rate 20.1 us): the rest is the second look and the ranking with
// their barriers, which the SM's other blocks hide only in part. 4 rows of 32000 fp32,
// k = 8: 9.3 us, nearly all of it one block's chain of barriers and exchanges.
#include <algorithm>

#include "internal.h"
#include "rowvec.cuh"
#include "tc_ptx.cuh"

namespace ivfpq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxGroup = 16;     // blocks of a cluster that takes a group
constexpr int kUnroll = 4;         // vectors of a batch
constexpr int kMaxSteps = 16;      // batches per thread whose maxima are kept apart
constexpr int kSlack = 8;          // how many threads more than k the bound may let pass
constexpr int kCap = 4096;         // kept scores before the worse ones are dropped
constexpr int kRound = kThreads * 8;  // most scores that one round can keep
constexpr float kLog2e = 1.4426950408889634f;

// What the row kernel leaves for the merge. Z is relative to m, so that totals
// of rows near fp32's limits lose nothing: total = (s - m) + base.
struct RowLists {
  float* val;    // [rows, k], descending
  int32_t* id;   // [rows, k]
  int32_t* len;  // [rows]
  float* m;      // [rows]
  double* base;  // [rows], t - log Z
};

struct SelectArgs {
  const void* scores;
  int64_t rows, cols, lds;
  const float* totals;      // [rows]
  const uint8_t* finished;  // [rows] or null
  int32_t end_id;
  int k, chunk, shift;
  RowLists o;
  // a cluster per group
  int beams, rank_shift;  // 2^rank_shift blocks per beam
  float* out_totals;      // [groups, k]
  int32_t* out_beams;
  int32_t* out_ids;
};

struct MergeArgs {
  RowLists o;
  int64_t groups;
  int beams, k;
  float* totals;
  int32_t* beam_ids;
  int32_t* ids;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// -0 and +0 are equal scores.
__device__ __forceinline__ uint32_t score_key(float v) { return float_to_key(v + 0.f); }
__device__ __forceinline__ uint64_t entry(uint32_t key, uint32_t col) {
  return (uint64_t(key) << 32) | uint32_t(~col);
}

// Largest score and sum of exp(s - m). m = -inf: nothing yet, z = 0.
struct Online {
  float m = -INFINITY, z = 0.f;
  __device__ __forceinline__ void raise(float v) {
    if (v > m) {
      z *= m == -INFINITY ? 0.f : exp2_fast((m - v) * kLog2e);  // a NaN stays
      m = v;
    }
  }
  __device__ __forceinline__ void join(float m2, float z2) {
    if (m2 == -INFINITY) {
      z += z2;  // 0, or NaN from a NaN among scores of -inf
      return;
    }
    raise(m2);
    z += z2 * exp2_fast((m2 - m) * kLog2e);
  }
};

template <class T>
__device__ __forceinline__ uint4 empty_vec() {
  const uint32_t w = sizeof(T) == 4 ? 0xff800000u
                     : std::is_same<T, __half>::value ? 0xfc00fc00u
                                                      : 0xff80ff80u;
  return make_uint4(w, w, w, w);
}

// A run's vectors; past its end -inf. VEC: rows are whole vectors on 16-byte boundaries.
template <class T, bool VEC>
struct Run {
  const T* p;
  int len, nvec, mis, first, last;
  __device__ __forceinline__ Run(const T* q, int n) : p(q), len(n) {
    nvec = (n + Span<T>::N - 1) / Span<T>::N;
    mis = VEC ? 0 : misalign(q);
    first = inner_first(mis);
    last = VEC ? nvec - 1 : inner_last<T>(n, mis);
  }
  __device__ __forceinline__ uint4 inner(int i) const {
    if constexpr (VEC) return __ldg(reinterpret_cast<const uint4*>(p) + i);
    return load_inner(p, i, mis);
  }
  __device__ __forceinline__ uint4 at(int i) const {
    if (i >= first && i <= last) return inner(i);
    if constexpr (!VEC) {
      if (i < nvec) return load_edge(p, len, i);
    }
    return empty_vec<T>();
  }
};

// The batch of step i: vectors (i * kUnroll + u) * kThreads + thread.
template <class T, bool VEC>
__device__ __forceinline__ void load_batch(const Run<T, VEC>& run, int step, uint4 (&r)[kUnroll]) {
  const int i0 = step * kUnroll * kThreads + threadIdx.x;
  if (i0 >= run.first && i0 + (kUnroll - 1) * kThreads <= run.last) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u] = run.inner(i0 + u * kThreads);
  } else {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u] = run.at(i0 + u * kThreads);
  }
}

// The sum of a vector's exponentials relative to m where there is nothing yet (m = 0), or
// where m is too large for add_batch's rounded product.
template <class T>
__device__ __noinline__ float far_vec(uint4 r, float m) {
  constexpr int N = Span<T>::N;
  float v[N], z = 0.f;
  unpack_vec<T>(r, v);
#pragma unroll
  for (int j = 0; j < N; ++j) z += exp2_fast((v[j] - m) * kLog2e);
  return z;
}

// Adds a batch's exponentials to o, whose m is at least its largest score.
template <class T>
__device__ __forceinline__ void add_batch(const uint4 (&r)[kUnroll], Online& o) {
  constexpr int N = Span<T>::N;
  const uint64_t scale = pair(kLog2e, kLog2e);
  uint64_t z = pair(0.f, 0.f);
  float z0, z1;
  if (fabsf(o.m) < 0x1p30f) {
    // exp2(s c - b) with b = m c rounded, one operation per score; what the
    // rounding of b does to all of them alike is taken back below: a factor of 2^64 at
    // most, as b is below 2^31 and a step there 2^7. (Further on one of the two factors
    // would be infinite and the other 0: scores are subtracted first, as for masks of
    // -1e10 and beyond.)
    const float b = o.m * kLog2e;
    const uint64_t minus = pair(-b, -b);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float v[N];
      unpack_vec<T>(r[u], v);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        float x, y;
        unpair(fma2(pair(v[j], v[j + 1]), scale, minus), x, y);
        z = add2(z, pair(exp2_fast(x), exp2_fast(y)));
      }
    }
    unpair(z, z0, z1);
    o.z += (z0 + z1) * exp2_fast(-fmaf(o.m, kLog2e, -b));
  } else {
    const float m = o.m == -INFINITY ? 0.f : o.m;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) o.z += far_vec<T>(r[u], m);
  }
}

// One pass over the run. peak[g * kThreads + thread]: the largest score of the
// thread's steps g << shift and following, as a key; r: its first batch.
template <class T, bool VEC>
__device__ __forceinline__ void run_stats(const Run<T, VEC>& run, int steps, int shift,
                                          uint4 (&r)[kUnroll], uint32_t* peak, Online& o) {
  float top = -INFINITY;
  auto take = [&](int i, const uint4 (&v)[kUnroll]) {
    float m = vec_max(v[0], static_cast<T*>(nullptr));
#pragma unroll
    for (int u = 1; u < kUnroll; ++u) m = fmaxf(m, vec_max(v[u], static_cast<T*>(nullptr)));
    top = fmaxf(top, m);
    if (((i + 1) & ((1 << shift) - 1)) == 0 || i + 1 == steps) {
      peak[(i >> shift) * kThreads + threadIdx.x] = score_key(top);
      top = -INFINITY;
    }
    o.raise(m);
    add_batch<T>(v, o);
  };
  // one batch on its way while the other is taken
  uint4 q[kUnroll];
  for (int i = 0; i < steps; i += 2) {
    if (i + 1 < steps) load_batch(run, i + 1, q);
    take(i, r);
    if (i + 1 < steps) {
      if (i + 2 < steps) load_batch(run, i + 2, r);
      take(i + 1, q);
    }
  }
}

// Sorts n entries (descending) in place; the space up to the next power of two
// is filled with zeros. kCap bounds n.
__device__ void sort_entries(uint64_t* e, int n) {
  int p = 32;
  while (p < n) p *= 2;
  for (int i = n + threadIdx.x; i < p; i += kThreads) e[i] = 0;
  for (int size = 2; size <= p; size *= 2) {
    for (int step = size / 2; step > 0; step /= 2) {
      __syncthreads();
      for (int t = threadIdx.x; t < p / 2; t += kThreads) {
        const int i = 2 * t - (t & (step - 1)), j = i + step;
        const uint64_t a = e[i], b = e[j];
        if ((a < b) == ((i & size) == 0)) {
          e[i] = b;
          e[j] = a;
        }
      }
    }
  }
  __syncthreads();
}

// A key that at least k of the block's keys (one per thread) reach, and no more than
// k + kSlack of them unless keys are equal; 0 if fewer than k are above that of -inf.
__device__ __forceinline__ uint32_t kth_bound(const uint32_t* keys, int k) {
  constexpr uint32_t kNothing = 0x007fffffu;  // -inf
  const int lane = threadIdx.x & 31;
  uint32_t v[kThreads / 32], lo = 0xffffffffu, hi = 0;
  unsigned n = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    v[i] = keys[i * 32 + lane];
    if (v[i] > kNothing) {
      lo = min(lo, v[i]);
      ++n;
    }
    hi = max(hi, v[i]);
  }
  hi = __reduce_max_sync(kFullMask, hi);
  lo = __reduce_min_sync(kFullMask, lo);
  if (int(__reduce_add_sync(kFullMask, n)) < k) return 0;
  while (lo < hi) {  // at least k keys reach lo, fewer than k pass hi
    const uint32_t mid = hi - (hi - lo) / 2;
    unsigned c = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) c += v[i] >= mid;
    const int all = int(__reduce_add_sync(kFullMask, c));
    if (all < k) {
      hi = mid - 1;
    } else {
      lo = mid;
      if (all <= k + kSlack) break;
    }
  }
  return lo;
}

__device__ __forceinline__ void st_cluster64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// fp64 totals as unsigned integers of the same order.
__device__ __forceinline__ uint64_t total_key(double v) {
  const uint64_t u = uint64_t(__double_as_longlong(v + 0.0));
  return u ^ (uint64_t(int64_t(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_total(uint64_t k) {
  return __longlong_as_double(int64_t(k ^ (uint64_t(int64_t(~k) >> 63) | 0x8000000000000000ull)));
}

// A block's statistics and the length of its list.
struct alignas(16) Part {
  float m, z;
  int len;
  float t;  // the beam's running total
};
// The statistics of `parts` parts (at most 8), in every lane of a warp.
__device__ __forceinline__ Online join_stats(float m, float z) {
  Online o;
  o.m = m;
  o.z = z;
#pragma unroll
  for (int d = 4; d > 0; d /= 2) {
    const float m2 = __shfl_xor_sync(kFullMask, o.m, d), z2 = __shfl_xor_sync(kFullMask, o.z, d);
    const bool upper = (threadIdx.x & d) != 0;  // the same operations in both lanes
    Online j;
    j.join(upper ? m2 : o.m, upper ? z2 : o.z);
    j.join(upper ? o.m : m2, upper ? o.z : z2);
    o = j;
  }
  return o;
}

// log Z from its exponent, exactly, and its mantissa in [3/4, 3/2), whose logarithm in
// fp32 is off by 2^-25 at most.
__device__ __forceinline__ double log_sum(float z) {
  const uint32_t u = __float_as_uint(z) - 0x3f400000u;
  const int ex = int(u) >> 23;
  const float f = __uint_as_float((u & 0x007fffffu) + 0x3f400000u);
  return double(ex) * 0.69314718055994530942 + double(logf(f));
}
// No softmax: only -inf, or a NaN or +inf among the scores.
__device__ __forceinline__ bool has_softmax(const Online& o) {
  return o.z > 0.f && o.z < INFINITY;
}

// Entries of a list where a cluster ranks several: whole 16-byte vectors, zeros at the end.
__host__ __device__ inline int list_stride(int k) { return (k + 1) & ~1; }

// The lists of a group's blocks ([size, stride], 2^rank_shift of them per beam), ranked.
__device__ void rank_group(const SelectArgs& a, int64_t group, int size, const uint64_t* lists,
                           uint64_t* totals, const Part* all) {
  __shared__ double base[kMaxGroup];  // t - log Z
  __shared__ float top[kMaxGroup];
  __shared__ int len[kMaxGroup];  // of each beam's list, 0 where it has no softmax
  const int k = a.k, stride = list_stride(k), shift = a.rank_shift;
  if (threadIdx.x < a.beams) {
    Online o;
    int n = 0;
    const int p0 = int(threadIdx.x) << shift;
    for (int p = p0; p < p0 + (1 << shift); ++p) {
      o.join(all[p].m, all[p].z);
      n += all[p].len;
    }
    const bool ok = has_softmax(o);
    top[threadIdx.x] = o.m;
    base[threadIdx.x] = ok ? double(all[p0].t) - log_sum(o.z) : 0.0;
    len[threadIdx.x] = ok ? n : 0;
  }
  __syncthreads();
  // size * stride entries, one per thread at most
  const int i = threadIdx.x, p = i / stride, beam = p >> shift;
  uint64_t mine = 0, e = 0;
  if (p < size) {
    e = lists[i];
    if (len[beam] > 0 && i - p * stride < all[p].len)
      mine = total_key(double(key_to_float(uint32_t(e >> 32))) - double(top[beam]) + base[beam]);
    totals[i] = mine;  // 0 is below every total
  }
  __syncthreads();
  int n = 0;
  for (int b = 0; b < a.beams; ++b) n += len[b];
  if (mine != 0) {
    int place = 0;
    for (int q = 0; q < size; ++q) {
      const int b = q >> shift;
      // a beam's own entries by score; of equal totals the lower beam's come first
      const ulonglong2* of =
          reinterpret_cast<const ulonglong2*>((b == beam ? lists : totals) + q * stride);
      const uint64_t than = b == beam ? e : mine - (b < beam);
#pragma unroll 4
      for (int j = 0; j < stride / 2; ++j) {
        const ulonglong2 v = of[j];
        place += (v.x > than) + (v.y > than);
      }
    }
    if (place < k) {
      a.out_totals[group * k + place] = float(key_total(mine));
      a.out_beams[group * k + place] = beam;
      a.out_ids[group * k + place] = int32_t(~uint32_t(e));
    }
  }
  for (int j = n + threadIdx.x; j < k; j += kThreads) {
    a.out_totals[group * k + j] = -INFINITY;
    a.out_beams[group * k + j] = -1;
    a.out_ids[group * k + j] = -1;
  }
}

// GROUP: a cluster takes a group, else a row.
template <class T, bool VEC, bool GROUP>
__global__ void __launch_bounds__(kThreads, 4) beam_rows_kernel(const SelectArgs a) {
  constexpr int N = Span<T>::N;
  extern __shared__ __align__(16) uint64_t select_smem[];
  const int stride = list_stride(a.k);
  uint64_t* kept = select_smem;  // [kCap]
  uint64_t* top = kept + kCap;   // [k]
  uint64_t* others = top + stride;  // [blocks, stride] where a cluster has several
  // the peaks (one array with `kept`, which is filled when they have been read)
  uint32_t* peak = reinterpret_cast<uint32_t*>(select_smem);
  __shared__ uint16_t chosen[kMaxSteps * kThreads];
  __shared__ float2 sh[kWarps];
  __shared__ Part all[kMaxGroup];  // in the first block of a cluster: of all its blocks
  __shared__ int nkept, nchosen;
  __shared__ uint32_t keys[kThreads];
  const int size = int(gridDim.x), block = int(blockIdx.x);  // of the cluster
  const int ranks = GROUP ? 1 << a.rank_shift : size, rank = GROUP ? block & (ranks - 1) : block;
  const int64_t item = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  const int64_t row = GROUP ? item * a.beams + (block >> a.rank_shift) : item;
  if (item >= (GROUP ? a.rows / a.beams : a.rows)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float t = a.totals[row];
  const bool done = a.finished && a.finished[row];
  const int64_t c0 = min(int64_t(rank) * a.chunk, a.cols);
  const Run<T, VEC> run(static_cast<const T*>(a.scores) + row * a.lds + c0,
                   int(min(int64_t(a.chunk), a.cols - c0)));
  uint4 r[kUnroll];
  load_batch(run, 0, r);  // on its way while the total is
  if (threadIdx.x == 0) nkept = nchosen = 0;
  // the blocks of a cluster must have started before one writes to another
  if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const bool alive = fabsf(t) < INFINITY;  // neither infinite nor NaN
  int n = 0;
  Online o_block;  // in the last warp
  if (!alive || done) {
    // nothing, or the one continuation of a finished beam: its own total
    if (alive && rank == 0) {
      n = 1;
      o_block.m = 0.f;
      o_block.z = 1.f;
      if (threadIdx.x == 0) top[0] = entry(score_key(0.f), uint32_t(a.end_id));
    }
  } else {
    const int steps = (run.nvec + kUnroll * kThreads - 1) / (kUnroll * kThreads);
    const int groups = (steps + (1 << a.shift) - 1) >> a.shift;
    Online o;
    run_stats(run, steps, a.shift, r, peak, o);
    if (!GROUP) grid_go();
    keys[threadIdx.x] = score_key(o.m);
    // the block's statistics
    {
      const float m = key_to_float(__reduce_max_sync(kFullMask, score_key(o.m)));
      float z = o.z * exp2_fast(m == -INFINITY ? 0.f : (o.m - m) * kLog2e);
#pragma unroll
      for (int d = 16; d > 0; d /= 2) z += __shfl_xor_sync(kFullMask, z, d);
      if (lane == 0) sh[warp] = make_float2(m, z);
    }
    __syncthreads();
    const uint32_t bound = kth_bound(keys, a.k);
    // the batches that reach the bound
    if (score_key(o.m) >= bound) {
      for (int g = 0; g < groups; ++g)
        if (peak[g * kThreads + threadIdx.x] >= bound)
          chosen[atomicAdd(&nchosen, 1)] = uint16_t(g * kThreads + threadIdx.x);
    }
    __syncthreads();  // also: the peaks are read
    const int per = kUnroll << a.shift, nread = nchosen * per;  // vectors
    uint64_t bar = uint64_t(bound) << 32;
    // the same as a score; -inf (and what lies past the end) is no continuation
    const float least = fmaxf(key_to_float(bound), -3.402823466e38f);
    for (int v0 = 0; v0 < nread; v0 += kThreads) {
      const int q = v0 + threadIdx.x;
      if (q < nread) {
        const int b = chosen[q / per], e = q % per;
        const int i = ((b / kThreads) * per + e) * kThreads + b % kThreads;
        const uint4 w = run.at(i);
        float v[N];
        unpack_vec<T>(w, v);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (v[j] >= least) {
            const uint64_t x = entry(score_key(v[j]), uint32_t(c0) + uint32_t(i * N + j));
            if (x >= bar) kept[atomicAdd(&nkept, 1)] = x;
          }
        }
      }
      __syncthreads();
      const int n = nkept;
      if (n > kCap - kRound) {
        sort_entries(kept, n);
        bar = kept[a.k - 1];
        if (threadIdx.x == 0) nkept = a.k;
        __syncthreads();
      } else if (v0 + kThreads < nread) {
        __syncthreads();  // n is read before the next round adds to it
      }
    }
    n = nkept;
    if (n <= kThreads) {
      if (threadIdx.x < n) {
        const uint64_t e = kept[threadIdx.x];
        int above = 0;
#pragma unroll 4
        for (int i = 0; i < n; ++i) above += kept[i] > e;
        if (above < a.k) top[above] = e;
      }
    } else {
      sort_entries(kept, n);
      for (int i = threadIdx.x; i < min(n, a.k); i += kThreads) top[i] = kept[i];
    }
    n = min(n, a.k);
    if (warp == kWarps - 1) o_block = join_stats(sh[lane % kWarps].x, sh[lane % kWarps].y);
  }
  __syncthreads();
  int count = n;
  uint64_t* lists = top;
  if (size > 1 || GROUP) {
    // to the first block: its `others` and `all`
    if (size > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    for (int i = threadIdx.x; i < stride; i += kThreads)
      st_cluster64(map_rank(smem_u32(others + block * stride + i), 0), i < n ? top[i] : 0);
    if (threadIdx.x == kThreads - 1) {
      const uint32_t at = map_rank(smem_u32(&all[block]), 0);
      st_cluster64(at, pair(o_block.m, o_block.z));
      st_cluster64(at + 8, uint64_t(n) | uint64_t(__float_as_uint(t)) << 32);
    }
    if (size > 1) {
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      if (block > 0) return;
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      __syncthreads();
    }
    if constexpr (GROUP) {
      // the totals take the place of the scores that were kept
      rank_group(a, item, size, others, kept, all);
      return;
    }
    lists = others;
    count = 0;
    for (int p = 0; p < ranks; ++p) count += all[p].len;
    if (warp == kWarps - 1) {
      const Part& p = all[lane % ranks];
      o_block = join_stats(lane % kMaxCluster < ranks ? p.m : -INFINITY,
                           lane % kMaxCluster < ranks ? p.z : 0.f);
    }
  }
  for (int i = threadIdx.x; i < ranks * stride; i += kThreads) {
    const int mine = i / stride, at = i - mine * stride;
    if (at >= (ranks > 1 ? all[mine].len : n)) continue;
    const uint64_t e = lists[i];
    int place = at;
    if (ranks > 1 && ranks * stride <= kThreads) {
      // few: those above this one, counted (nothing is below every entry)
      place = 0;
#pragma unroll 4
      for (int j = 0; j < ranks * stride; ++j) place += lists[j] > e;
    }
    for (int p = 0; p < ranks && ranks * stride > kThreads; ++p) {
      if (p == mine) continue;
      int lo = 0, hi = all[p].len;  // entries of that list above mine
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (lists[p * stride + mid] > e)
          lo = mid + 1;
        else
          hi = mid;
      }
      place += lo;
    }
    if (place < a.k) {
      a.o.val[row * a.k + place] = key_to_float(uint32_t(e >> 32));
      a.o.id[row * a.k + place] = int32_t(~uint32_t(e));
    }
  }
  if (threadIdx.x == kThreads - 1) {
    const bool ok = has_softmax(o_block);
    a.o.len[row] = ok ? min(count, a.k) : 0;
    a.o.m[row] = o_block.m;
    a.o.base[row] = ok ? double(t) - log_sum(o_block.z) : 0.0;
  }
}

// One block per group: the beams' lists merged two neighbours at a time; of equal
// totals the left list's (the lower beam's) come first.
__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const MergeArgs a) {
  extern __shared__ __align__(16) uint64_t merge_smem[];
  const int k = a.k, half = (a.beams + 1) / 2;
  uint64_t* key[2] = {merge_smem, merge_smem + a.beams * k};
  uint64_t* ref[2] = {key[1] + half * k, key[1] + half * k + a.beams * k};  // beam, id
  __shared__ int len[2][64];
  grid_wait();
  for (int64_t g = blockIdx.x; g < a.groups; g += gridDim.x) {
    const int64_t row0 = g * a.beams;
    __syncthreads();
    if (threadIdx.x < a.beams) len[0][threadIdx.x] = a.o.len[row0 + threadIdx.x];
    for (int i = threadIdx.x; i < a.beams * k; i += kThreads) {
      const int b = i / k;
      if (i - b * k < a.o.len[row0 + b]) {
        const double d = double(a.o.val[row0 * k + i]) - double(a.o.m[row0 + b]);
        key[0][i] = total_key(d + a.o.base[row0 + b]);
        ref[0][i] = (uint64_t(b) << 32) | uint32_t(a.o.id[row0 * k + i]);
      }
    }
    int lists = a.beams, at = 0;
    for (; lists > 1; lists = (lists + 1) / 2, at ^= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < lists * k; i += kThreads) {
        const int l = i / k, e = i - l * k;
        if (e >= len[at][l]) continue;
        const uint64_t mine = key[at][i];
        int lo = 0, hi = (l ^ 1) < lists ? len[at][l ^ 1] : 0;
        const uint64_t* other = key[at] + (l ^ 1) * k;
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (other[mid] > mine || (l & 1 && other[mid] == mine))
            lo = mid + 1;
          else
            hi = mid;
        }
        if (e + lo < k) {
          key[at ^ 1][l / 2 * k + e + lo] = mine;
          ref[at ^ 1][l / 2 * k + e + lo] = ref[at][i];
        }
      }
      for (int l = 2 * threadIdx.x; l < lists; l += 2 * kThreads)
        len[at ^ 1][l / 2] = min(k, len[at][l] + (l + 1 < lists ? len[at][l + 1] : 0));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < k; i += kThreads) {
      const bool ok = i < len[at][0];
      const uint64_t r = ok ? ref[at][i] : ~uint64_t(0);
      a.totals[g * k + i] = ok ? float(key_total(key[at][i])) : -INFINITY;
      a.beam_ids[g * k + i] = int32_t(r >> 32);
      a.ids[g * k + i] = int32_t(uint32_t(r));
    }
  }
}

dim3 grid_of(int64_t per_row, int64_t rows) {
  const int64_t y = std::min<int64_t>(rows, 65535);
  return dim3(unsigned(per_row), unsigned(y), unsigned(ceil_div(rows, y)));
}

// More blocks per row while the rows alone do not fill the device twice, down to runs
// of 4,096 columns; at most `most`. (512 rows of 131072 bf16: 33 us so, where one block
// takes a row, and 38, 41 and 56 us with 2, 4 and 8 blocks per row; Few
// rows are bound by how many SMs read them.)
int ranks_for(int64_t rows, int64_t cols, int most) {
  int ranks = 1;
  while (2 * ranks <= most && rows * ranks < 2 * num_sms() && cols > 4096 * int64_t(ranks))
    ranks *= 2;
  return ranks;
}
// Whether a cluster per group does: few entries to rank against each other, and runs
// that are as long as they would be otherwise or of 16,384 columns at most. (One group
// of 4 x 32000 fp32 as a program calls it: 16.2 us in one kernel, 21.5 us in two.)
bool group_fits(const SelectArgs& a, int* ranks) {
  if (a.beams > kMaxGroup) return false;
  *ranks = ranks_for(a.rows, a.cols, kMaxGroup / a.beams);
  return a.beams * *ranks * list_stride(a.k) <= kThreads &&
         (*ranks == ranks_for(a.rows, a.cols, kMaxCluster) || a.cols <= 16384 * int64_t(*ranks));
}

template <class T, bool GROUP>
int launch_rows(SelectArgs a, int ranks, cudaStream_t s) {
  a.rank_shift = 0;
  while (1 << a.rank_shift < ranks) ++a.rank_shift;  // ranks are powers of two
  a.chunk = int(ceil_div(ceil_div(a.cols, ranks), 8) * 8);
  const int64_t steps = ceil_div(a.chunk, int64_t(kThreads) * kUnroll * Span<T>::N);
  a.shift = 0;
  while (ceil_div(steps, int64_t(1) << a.shift) > kMaxSteps) ++a.shift;
  const int size = GROUP ? a.beams * ranks : ranks;
  const size_t smem =
      (size_t(kCap) + size_t(list_stride(a.k)) * (size == 1 && !GROUP ? 1 : 1 + size)) * 8;
  constexpr int N = Span<T>::N;
  const bool vec = a.cols % N == 0 && a.lds % N == 0 &&
                   reinterpret_cast<uintptr_t>(a.scores) % 16 == 0;
  auto kern = vec ? beam_rows_kernel<T, true, GROUP> : beam_rows_kernel<T, false, GROUP>;
  // 48 KB with the static part need no leave
  if (smem > 36 * 1024) IVFPQ_TRY(set_dynamic_smem(kern, smem));
  if (size > kMaxCluster)
    IVFPQ_CUDA(cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                    cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid_of(size, GROUP ? a.rows / a.beams : a.rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(size);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
  IVFPQ_LAUNCHED_K(kern, smem, kThreads);
  return IVFPQ_OK;
}

int launch_merge(const MergeArgs& a, cudaStream_t s) {
  const size_t smem = size_t(a.beams + (a.beams + 1) / 2) * a.k * 16;
  if (smem > 40 * 1024) IVFPQ_TRY(set_dynamic_smem(beam_merge_kernel, smem));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(std::min<int64_t>(a.groups, int64_t(1) << 20)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, beam_merge_kernel, a));
  IVFPQ_LAUNCHED_K(beam_merge_kernel, smem, kThreads);
  return IVFPQ_OK;
}

}  // namespace
}  // namespace ivfpq

using namespace ivfpq;

extern "C" int beam_select(const void* scores, int dtype, int64_t groups, int beams, int64_t cols,
                           int64_t lds, const float* totals, const uint8_t* finished,
                           int32_t end_id, int k, float* out_totals, int32_t* out_beams,
                           int32_t* out_ids, void* stream) {
  clear_error();
  IVFPQ_REQUIRE(known_dtype(dtype), "beam_select: unknown element type %d", dtype);
  IVFPQ_REQUIRE(beams >= 1 && beams <= IVFPQ_MAX_BEAMS, "beam_select: beams=%d outside [1, %d]",
                beams, IVFPQ_MAX_BEAMS);
  IVFPQ_REQUIRE(groups >= 0 && groups < (int64_t(1) << 31) && groups * beams < (int64_t(1) << 31),
                "beam_select: groups=%lld of %d beams outside [0, 2^31)", (long long)groups, beams);
  IVFPQ_REQUIRE(cols >= 1 && cols <= (int64_t(1) << 28), "beam_select: cols=%lld outside [1, 2^28]",
                (long long)cols);
  IVFPQ_REQUIRE(k >= 1 && k <= IVFPQ_MAX_BEAM_K, "beam_select: k=%d outside [1, %d]", k,
                IVFPQ_MAX_BEAM_K);
  IVFPQ_REQUIRE(groups * beams <= 1 || lds >= cols || lds == 0,
                "beam_select: row stride %lld below cols=%lld", (long long)lds, (long long)cols);
  if (groups == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(scores && totals && out_totals && out_beams && out_ids,
                "beam_select: null pointer");
  IVFPQ_REQUIRE(!finished || (end_id >= 0 && end_id < cols),
                "beam_select: end_id=%d outside [0, %lld)", end_id, (long long)cols);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = groups * beams;
  SelectArgs a{scores, rows, cols, lds, totals, finished, end_id, k, 0, 0, {}, beams, 0, out_totals,
               out_beams, out_ids};
  int ranks = 0;
  if (group_fits(a, &ranks))
    return by_dtype(dtype, [&](auto* t) -> int {
      return launch_rows<std::remove_pointer_t<decltype(t)>, true>(a, ranks, s);
    });
  Workspace ws(s);
  RowLists& o = a.o;
  // one buffer: base, val, id, len, m
  double* w = nullptr;
  const size_t words = size_t(rows) * (size_t(k) * 2 + 2);
  IVFPQ_TRY(ws.alloc(&w, size_t(rows) + (words + 1) / 2));
  o.base = w;
  o.val = reinterpret_cast<float*>(w + rows);
  o.id = reinterpret_cast<int32_t*>(o.val + rows * k);
  o.len = o.id + rows * k;
  o.m = reinterpret_cast<float*>(o.len + rows);
  ranks = ranks_for(rows, cols, kMaxCluster);
  IVFPQ_TRY(by_dtype(dtype, [&](auto* t) -> int {
    return launch_rows<std::remove_pointer_t<decltype(t)>, false>(a, ranks, s);
  }));
  return launch_merge({o, groups, beams, k, out_totals, out_beams, out_ids}, s);
}
