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
//  2. The k-th largest of the batches' maxima is a lower bound of the k-th
//     largest score; bisection over its bits finds it, or something a little
//     lower. Only batches that reach the bound are read again (about k of them, a
//     thread each, from L2), and their scores at or above it kept.
//  3. The kept ones are ranked among themselves; a cluster of blocks that shares
//     a row ranks its lists against each other by binary search.
//  4. A second kernel, already waiting, merges the beams' lists of a group, two
//     at a time. Totals are compared in fp64: they differ by the rounding of
//     their sums of exponentials, not of the comparison.
// Keys hold (score, inverted column), so that no step depends on the order in
// which threads append and the lowest column of equal scores comes first.
#include <algorithm>

#include "internal.h"
#include "rowvec.cuh"
#include "tc_ptx.cuh"

namespace ivfpq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 4;         // vectors of a batch
constexpr int kMaxSteps = 4;       // batches per thread whose maxima are kept apart
constexpr int kSlack = 32;         // how many batches more than k the bound may let pass
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

// A run's vectors; past its end -inf.
template <class T>
struct Run {
  const T* p;
  int len, nvec, mis, first, last;
  __device__ __forceinline__ Run(const T* q, int n) : p(q), len(n) {
    nvec = (n + Span<T>::N - 1) / Span<T>::N;
    mis = misalign(q);
    first = inner_first(mis);
    last = inner_last<T>(n, mis);
  }
  __device__ __forceinline__ uint4 at(int i) const {
    if (i >= first && i <= last) return load_inner(p, i, mis);
    return i < nvec ? load_edge(p, len, i) : empty_vec<T>();
  }
};

// The batch of step i: vectors (i * kUnroll + u) * kThreads + thread.
template <class T>
__device__ __forceinline__ void load_batch(const Run<T>& run, int step, uint4 (&r)[kUnroll]) {
  const int i0 = step * kUnroll * kThreads + threadIdx.x;
  if (i0 >= run.first && i0 + (kUnroll - 1) * kThreads <= run.last) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u] = load_inner(run.p, i0 + u * kThreads, run.mis);
  } else {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u] = run.at(i0 + u * kThreads);
  }
}

// Adds a batch's exponentials to o, whose m is at least its largest score.
template <class T>
__device__ __forceinline__ void add_batch(const uint4 (&r)[kUnroll], Online& o) {
  constexpr int N = Span<T>::N;
  const uint64_t scale = pair(kLog2e, kLog2e);
  uint64_t z = pair(0.f, 0.f);
  float z0, z1;
  if (fabsf(o.m) < 1e38f) {
    // exp2(s c - b) with b = m c rounded, one operation per score; what the
    // rounding of b does to all of them alike is taken back below
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
    // nothing yet, or scores whose products pass fp32
    const float ref = o.m == -INFINITY ? 0.f : o.m;
    const uint64_t minus = pair(-ref, -ref);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float v[N];
      unpack_vec<T>(r[u], v);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        float x, y;
        unpair(mul2(add2(pair(v[j], v[j + 1]), minus), scale), x, y);
        z = add2(z, pair(exp2_fast(x), exp2_fast(y)));
      }
    }
    unpair(z, z0, z1);
    o.z += z0 + z1;
  }
}

// One pass over the run. peak[g * kThreads + thread]: the largest score of the
// thread's steps g << shift and following, as a key; r: its first batch.
template <class T>
__device__ __forceinline__ void run_stats(const Run<T>& run, int steps, int shift,
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

// A key that at least k of the block's peaks reach (`groups` per thread), and no more
// than k + kSlack of them unless peaks are equal in their upper 16 bits; 0 if there
// are fewer than k. A bit per step, from the highest one in which peaks differ.
// votes: [34] zeros.
__device__ __forceinline__ uint32_t kth_bound(const uint32_t* peak, int groups, int k,
                                              unsigned* votes) {
  const int lane = threadIdx.x & 31;
  uint32_t v[kMaxSteps], lo = 0xffffffffu, hi = 0;
#pragma unroll
  for (int i = 0; i < kMaxSteps; ++i) {
    v[i] = i < groups ? peak[i * kThreads + threadIdx.x] : 0u;
    if (i < groups) lo = min(lo, v[i]);
    hi = max(hi, v[i]);
  }
  // votes[32], votes[33]: the largest key, and of the inverted ones
  hi = __reduce_max_sync(kFullMask, hi);
  lo = __reduce_min_sync(kFullMask, lo);
  if (lane == 0) {
    atomicMax(&votes[32], hi);
    atomicMax(&votes[33], ~lo);
  }
  __syncthreads();
  if (groups * kThreads < k) return 0;
  hi = votes[32];
  lo = ~votes[33];
  if ((lo ^ hi) >> 16 == 0) return lo & 0xffff0000u;
  const int top = 31 - __clz(lo ^ hi);
  uint32_t bound = hi & ~((2u << top) - 1u);
  for (int bit = top; bit >= 16; --bit) {
    const uint32_t t = bound | (1u << bit);
    int c = 0;
#pragma unroll
    for (int i = 0; i < kMaxSteps; ++i) c += v[i] >= t;
    const unsigned w = __reduce_add_sync(kFullMask, unsigned(c));
    if (lane == 0 && w) atomicAdd(&votes[bit], w);
    __syncthreads();
    const int all = int(votes[bit]);
    if (all >= k) {
      bound = t;
      if (all <= k + kSlack) break;
    }
  }
  return bound;
}

__device__ __forceinline__ uint64_t ld_cluster64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// What a block tells the others of its row.
struct alignas(16) Part {
  float m, z;
  int len, pad;
};

template <class T>
__global__ void __launch_bounds__(kThreads, 4) beam_rows_kernel(const SelectArgs a) {
  constexpr int N = Span<T>::N;
  extern __shared__ __align__(16) uint64_t select_smem[];
  uint64_t* kept = select_smem;  // [kCap]
  uint64_t* top = kept + kCap;   // [k]
  uint64_t* others = top + a.k;  // [ranks, k] where a row has several blocks
  // the peaks (one array with `kept`, which is filled when they have been read)
  uint32_t* peak = reinterpret_cast<uint32_t*>(select_smem);
  __shared__ uint16_t chosen[kMaxSteps * kThreads];
  __shared__ float2 sh[kWarps];
  __shared__ Part part;
  __shared__ Part all[kMaxCluster];
  __shared__ int nkept, nchosen;
  __shared__ unsigned votes[34];
  const int ranks = int(gridDim.x), rank = int(blockIdx.x);
  const int64_t row = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  if (row >= a.rows) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float t = a.totals[row];
  const bool done = a.finished && a.finished[row];
  const int64_t c0 = min(int64_t(rank) * a.chunk, a.cols);
  const Run<T> run(static_cast<const T*>(a.scores) + row * a.lds + c0,
                   int(min(int64_t(a.chunk), a.cols - c0)));
  uint4 r[kUnroll];
  load_batch(run, 0, r);  // on its way while the total is
  if (threadIdx.x < 34) votes[threadIdx.x] = 0;
  if (threadIdx.x == 0) nkept = nchosen = 0;
  const bool alive = fabsf(t) < INFINITY;  // neither infinite nor NaN
  if (!alive || done) {
    if (rank == 0 && threadIdx.x == 0) {
      a.o.len[row] = alive ? 1 : 0;
      a.o.val[row * a.k] = 0.f;
      a.o.id[row * a.k] = a.end_id;
      a.o.m[row] = 0.f;
      a.o.base[row] = double(t);
    }
    return;
  }
  const int steps = (run.nvec + kUnroll * kThreads - 1) / (kUnroll * kThreads);
  const int groups = (steps + (1 << a.shift) - 1) >> a.shift;
  Online o;
  run_stats<T>(run, steps, a.shift, r, peak, o);
  grid_go();
  // the block's statistics
  {
    const float m = key_to_float(__reduce_max_sync(kFullMask, score_key(o.m)));
    float z = o.z * exp2_fast(m == -INFINITY ? 0.f : (o.m - m) * kLog2e);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) z += __shfl_xor_sync(kFullMask, z, d);
    if (lane == 0) sh[warp] = make_float2(m, z);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    Online j;
    for (int w = 0; w < kWarps; ++w) j.join(sh[w].x, sh[w].y);
    part.m = j.m;
    part.z = j.z;
  }
  const uint32_t bound = kth_bound(peak, groups, a.k, votes);
  // the batches that reach the bound
  for (int g = 0; g < groups; ++g)
    if (peak[g * kThreads + threadIdx.x] >= bound)
      chosen[atomicAdd(&nchosen, 1)] = uint16_t(g * kThreads + threadIdx.x);
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
  int n = nkept;
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
  if (threadIdx.x == 0) part.len = n;
  __syncthreads();
  Online j;
  int total = n, place = threadIdx.x;
  const uint64_t mine = threadIdx.x < n ? top[threadIdx.x] : 0;
  if (ranks == 1) {
    j.join(part.m, part.z);
  } else {
    cluster_sync();
    for (int i = threadIdx.x; i < ranks * a.k; i += kThreads)
      others[i] = ld_cluster64(map_rank(smem_u32(top + i % a.k), uint32_t(i / a.k)));
    if (threadIdx.x < ranks) {
      const float4 p = ld_cluster4(map_rank(smem_u32(&part), threadIdx.x));
      all[threadIdx.x] = {p.x, p.y, __float_as_int(p.z), 0};
    }
    cluster_sync();
    total = 0;
    for (int p = 0; p < ranks; ++p) {
      j.join(all[p].m, all[p].z);
      const int len = all[p].len;
      total += len;
      if (p == rank || threadIdx.x >= n) continue;
      int lo = 0, hi = len;  // entries of that list above mine
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (others[p * a.k + mid] > mine)
          lo = mid + 1;
        else
          hi = mid;
      }
      place += lo;
    }
  }
  if (threadIdx.x < n && place < a.k) {
    a.o.val[row * a.k + place] = key_to_float(uint32_t(mine >> 32));
    a.o.id[row * a.k + place] = int32_t(~uint32_t(mine));
  }
  if (rank == 0 && threadIdx.x == 0) {
    // no softmax: only -inf, or a NaN or +inf among the scores
    const bool ok = j.z > 0.f && j.z < INFINITY;
    a.o.len[row] = ok ? min(total, a.k) : 0;
    a.o.m[row] = j.m;
    // log Z from its exponent, exactly, and its mantissa in [3/4, 3/2), whose
    // logarithm in fp32 is off by 2^-25 at most
    const uint32_t u = __float_as_uint(j.z) - 0x3f400000u;
    const int ex = int(u) >> 23;
    const float f = __uint_as_float((u & 0x007fffffu) + 0x3f400000u);
    a.o.base[row] = double(t) - (double(ex) * 0.69314718055994530942 + double(logf(f)));
  }
}

// fp64 totals as unsigned integers of the same order.
__device__ __forceinline__ uint64_t total_key(double v) {
  const uint64_t u = uint64_t(__double_as_longlong(v + 0.0));
  return u ^ (uint64_t(int64_t(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_total(uint64_t k) {
  return __longlong_as_double(int64_t(k ^ (uint64_t(int64_t(~k) >> 63) | 0x8000000000000000ull)));
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

template <class T>
int launch_rows(SelectArgs a, cudaStream_t s) {
  // more blocks per row while the rows alone do not fill the device twice, down
  // to runs of 4,096 columns
  int ranks = 1;
  while (ranks < kMaxCluster && a.rows * ranks < 2 * num_sms() && a.cols > 4096 * int64_t(ranks))
    ranks *= 2;
  a.chunk = int(ceil_div(ceil_div(a.cols, ranks), 8) * 8);
  const int64_t steps = ceil_div(a.chunk, int64_t(kThreads) * kUnroll * Span<T>::N);
  a.shift = 0;
  while (ceil_div(steps, int64_t(1) << a.shift) > kMaxSteps) ++a.shift;
  const size_t smem = (size_t(kCap) + size_t(a.k) * (ranks == 1 ? 1 : 1 + ranks)) * 8;
  auto kern = beam_rows_kernel<T>;
  if (smem > 40 * 1024) IVFPQ_TRY(set_dynamic_smem(kern, smem));
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
  IVFPQ_REQUIRE(groups >= 0 && groups * beams < (int64_t(1) << 31) && groups < (int64_t(1) << 31),
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
  Workspace ws(s);
  RowLists o{};
  // one buffer: base, val, id, len, m
  double* w = nullptr;
  const size_t words = size_t(rows) * (size_t(k) * 2 + 2);
  IVFPQ_TRY(ws.alloc(&w, size_t(rows) + (words + 1) / 2));
  o.base = w;
  o.val = reinterpret_cast<float*>(w + rows);
  o.id = reinterpret_cast<int32_t*>(o.val + rows * k);
  o.len = o.id + rows * k;
  o.m = reinterpret_cast<float*>(o.len + rows);
  SelectArgs a{scores, rows, cols, lds, totals, finished, end_id, k, 0, 0, o};
  IVFPQ_TRY(by_dtype(dtype, [&](auto* t) -> int {
    return launch_rows<std::remove_pointer_t<decltype(t)>>(a, s);
  }));
  return launch_merge({o, groups, beams, k, out_totals, out_beams, out_ids}, s);
}
