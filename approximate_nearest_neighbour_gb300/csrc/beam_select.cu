// beam_select: the k best continuations of every request's beams. For beam b of
// a group, with t its running total and s its score row,
//   total(b, c) = t + s_c - log sum_j exp(s_j)
// and the k largest over (b, c) are taken, equal ones by (b, c). A finished beam
// has one continuation, (b, end_id), whose total is t.
//
// Bound by memory: each score is read once. Within a row totals are ordered as
// scores, so a row's own k best are enough and need no normalisation:
//  1. A warp's load of 32 vectors is a batch. One pass keeps per thread the
//     largest score and the sum of exponentials relative to it (rescaled when it
//     grows), and per batch the largest score, in shared memory.
//  2. The k-th largest of the batches' maxima is a lower bound of the k-th
//     largest score, found by bisection over its bits by one warp. Only batches
//     that reach it are read again (about k of them, from L2), and their scores
//     at or above it kept: about k, more only where scores are equal.
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
constexpr int kMaxBatches = 1024;  // a block's maxima: 32 per lane of the bisecting warp
constexpr int kCap = 4096;         // kept scores before the worse ones are dropped
constexpr int kRound = kWarps * 32 * 8;  // most scores that one round can keep
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

template <class T>
__device__ __forceinline__ void run_stats(const Run<T>& run, int shift, uint32_t* bmax,
                                          Online& o) {
  constexpr int N = Span<T>::N, U = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nload = (run.nvec + 31) / 32;
  for (int l0 = warp * U; l0 < nload; l0 += kWarps * U) {
    uint4 r[U];
    const int i0 = l0 * 32 + lane;
    if (i0 >= run.first && i0 + (U - 1) * 32 <= run.last) {
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = load_inner(run.p, i0 + u * 32, run.mis);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = run.at(i0 + u * 32);
    }
    float vm[U], m = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      vm[u] = vec_max(r[u], static_cast<T*>(nullptr));
      m = fmaxf(m, vm[u]);
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t k = __reduce_max_sync(kFullMask, score_key(vm[u]));
      if (lane == u && l0 + u < nload) {
        if (shift == 0)
          bmax[l0 + u] = k;
        else
          atomicMax(&bmax[(l0 + u) >> shift], k);
      }
    }
    o.raise(m);
    const float ref = o.m == -INFINITY ? 0.f : o.m;
    const uint64_t minus = pair(-ref, -ref), scale = pair(kLog2e, kLog2e);
    float z[2] = {0.f, 0.f};
    uint64_t zz = pair(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[N];
      unpack_vec<T>(r[u], v);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        float a, b;
        unpair(mul2(add2(pair(v[j], v[j + 1]), minus), scale), a, b);
        zz = add2(zz, pair(exp2_fast(a), exp2_fast(b)));
      }
    }
    unpair(zz, z[0], z[1]);
    o.z += z[0] + z[1];
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

// The largest 2^16-aligned key that at least k of the n keys reach (0 if there
// are fewer): one warp, its keys in registers, a bit per step from the highest
// one in which they differ.
__device__ __forceinline__ uint32_t kth_bound(const uint32_t* keys, int n, int k) {
  const int lane = threadIdx.x & 31;
  if (n < k) return 0;
  uint32_t v[kMaxBatches / 32], lo = 0xffffffffu, hi = 0;
#pragma unroll
  for (int i = 0; i < kMaxBatches / 32; ++i) {
    v[i] = i * 32 + lane < n ? keys[i * 32 + lane] : 0u;
    if (i * 32 + lane < n) lo = min(lo, v[i]);
    hi = max(hi, v[i]);
  }
  lo = __reduce_min_sync(kFullMask, lo);
  hi = __reduce_max_sync(kFullMask, hi);
  if ((lo ^ hi) >> 16 == 0) return lo & 0xffff0000u;
  const int top = 31 - __clz(lo ^ hi);
  uint32_t bound = hi & ~((2u << top) - 1u);
  for (int bit = top; bit >= 16; --bit) {
    const uint32_t t = bound | (1u << bit);
    int c = 0;
    if (n <= kMaxBatches / 4) {
#pragma unroll
      for (int i = 0; i < kMaxBatches / 128; ++i) c += v[i] >= t;
    } else {
#pragma unroll
      for (int i = 0; i < kMaxBatches / 32; ++i) c += v[i] >= t;
    }
    if (int(__reduce_add_sync(kFullMask, unsigned(c))) >= k) bound = t;
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
__global__ void __launch_bounds__(kThreads, 5) beam_rows_kernel(const SelectArgs a) {
  constexpr int N = Span<T>::N;
  extern __shared__ __align__(16) uint64_t select_smem[];
  uint64_t* kept = select_smem;                 // [kCap]
  uint64_t* top = kept + kCap;                  // [k]
  uint64_t* others = top + a.k;                 // [ranks, k] where a row has several blocks
  __shared__ uint32_t bmax[kMaxBatches];
  __shared__ uint16_t chosen[kMaxBatches];
  __shared__ float2 sh[kWarps];
  __shared__ Part part;
  __shared__ Part all[kMaxCluster];
  __shared__ int nkept, nchosen;
  __shared__ uint32_t bound;
  const int ranks = int(gridDim.x), rank = int(blockIdx.x);
  const int64_t row = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  if (row >= a.rows) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float t = a.totals[row];
  const bool alive = fabsf(t) < INFINITY;  // neither infinite nor NaN
  if (!alive || (a.finished && a.finished[row])) {
    if (rank == 0 && threadIdx.x == 0) {
      a.o.len[row] = alive ? 1 : 0;
      a.o.val[row * a.k] = 0.f;
      a.o.id[row * a.k] = a.end_id;
      a.o.m[row] = 0.f;
      a.o.base[row] = double(t);
    }
    return;
  }
  const int64_t c0 = min(int64_t(rank) * a.chunk, a.cols);
  const Run<T> run(static_cast<const T*>(a.scores) + row * a.lds + c0,
                   int(min(int64_t(a.chunk), a.cols - c0)));
  const int nload = (run.nvec + 31) / 32;
  const int nbatch = (nload + (1 << a.shift) - 1) >> a.shift;
  if (threadIdx.x == 0) nkept = nchosen = 0;
  if (a.shift > 0) {
    for (int i = threadIdx.x; i < nbatch; i += kThreads) bmax[i] = 0;
    __syncthreads();
  }
  Online o;
  run_stats<T>(run, a.shift, bmax, o);
  grid_go();
  // the block's statistics
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    const float m2 = __shfl_xor_sync(kFullMask, o.m, d), z2 = __shfl_xor_sync(kFullMask, o.z, d);
    const float m1 = o.m, z1 = o.z;
    // the same operations in both lanes of a pair
    Online j;
    j.join(lane & d ? m2 : m1, lane & d ? z2 : z1);
    j.join(lane & d ? m1 : m2, lane & d ? z1 : z2);
    o = j;
  }
  if (lane == 0) sh[warp] = make_float2(o.m, o.z);
  __syncthreads();
  if (warp == 0) {
    const uint32_t b = kth_bound(bmax, nbatch, a.k);
    if (lane == 0) bound = b;
  } else if (warp == 1 && lane == 0) {
    Online j;
    for (int w = 0; w < kWarps; ++w) j.join(sh[w].x, sh[w].y);
    part.m = j.m;
    part.z = j.z;
  }
  __syncthreads();
  // the batches that reach the bound
  for (int i = threadIdx.x; i < nbatch; i += kThreads)
    if (bmax[i] >= bound) chosen[atomicAdd(&nchosen, 1)] = uint16_t(i);
  __syncthreads();
  const int nread = nchosen << a.shift;
  uint64_t bar = uint64_t(bound) << 32;
  for (int r0 = 0; r0 < nread; r0 += kWarps) {
    const int r = r0 + warp;
    if (r < nread) {
      const int i = ((int(chosen[r >> a.shift]) << a.shift) + (r & ((1 << a.shift) - 1))) * 32 + lane;
      const uint4 q = run.at(i);
      float v[N];
      unpack_vec<T>(q, v);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint64_t e = entry(score_key(v[j]), uint32_t(c0) + uint32_t(i * N + j));
        // a score of -inf (and what lies past the end) is no continuation
        if (v[j] > -INFINITY && e >= bar) kept[atomicAdd(&nkept, 1)] = e;
      }
    }
    __syncthreads();
    const int n = nkept;
    if (n > kCap - kRound) {
      sort_entries(kept, n);
      bar = kept[a.k - 1];
      if (threadIdx.x == 0) nkept = a.k;
      __syncthreads();
    } else if (r0 + kWarps < nread) {
      __syncthreads();  // n is read before the next round adds to it
    }
  }
  int n = nkept;
  if (n <= kThreads) {
    const uint64_t e = threadIdx.x < n ? kept[threadIdx.x] : 0;
    int above = 0;
    for (int i = 0; i < n; ++i) above += kept[i] > e;
    if (threadIdx.x < n && above < a.k) top[above] = e;
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
    for (int r = 0; r < ranks; ++r) {
      j.join(all[r].m, all[r].z);
      const int len = all[r].len;
      total += len;
      if (r == rank || threadIdx.x >= n) continue;
      int lo = 0, hi = len;  // entries of that list above mine
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (others[r * a.k + mid] > mine)
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
  const int64_t loads = ceil_div(a.chunk, 32 * Span<T>::N);
  a.shift = 0;
  while ((loads >> a.shift) + 1 > kMaxBatches) ++a.shift;
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
