// embedding_lookup: rows of a table by token, scaled; and embedding_gradient, the
// table's gradient, row v = scale times the sum of the gradient rows of token v.
//
// Both are bound by memory. The lookup reads and writes each row once, in vectors
// that start on a 16-byte boundary of the output.
//
// The gradient's sums are taken in the order of the positions, so that they repeat
// bit for bit:
//  1. The positions are sorted by token (stably). Block c owns the tokens that are
//     c modulo the number of blocks, so that neighbouring frequent tokens fall to
//     different blocks; it reads all ids, which are few bytes beside the gradient's
//     rows, counts its own and those of the lower classes, and so knows where its
//     tokens go without hearing from the other blocks. One warp places them, 32 in
//     order at a time.
//  2. The sorted positions are cut into slabs of equal length. A block adds a slab's
//     rows over a run of columns in registers (fp32) and writes a row where the
//     token changes. A token that goes on beyond its slab is finished by the block in
//     whose slab it starts; one with more positions than a slab has (a frequent token
//     is many slabs' work, not one block's) leaves a partial sum in every slab.
//     Further blocks zero the rows without a token.
//  3. The partial sums of a frequent token are added in slab order.
#include <algorithm>

#include "internal.h"
#include "rowvec.cuh"
#include "tc_ptx.cuh"

namespace ivfpq {
namespace {

dim3 grid_of(int64_t per_row, int64_t rows) {
  const int64_t y = std::min<int64_t>(rows, 65535);
  return dim3(unsigned(per_row), unsigned(y), unsigned(ceil_div(rows, y)));
}
__device__ __forceinline__ int64_t grid_row() {
  return blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
}

// ---- lookup ---------------------------------------------------------------------------
constexpr int kLookupThreads = 256;

struct LookupArgs {
  const void* table;
  int64_t rows, cols, ldt;
  const void* ids;
  int wide;  // ids are int64
  int64_t tokens;
  float scale;
  void* out;
  int64_t ldo;
  int tx;  // threads along a row, a power of two
};

__device__ __forceinline__ int64_t id_at(const void* ids, int wide, int64_t t) {
  return wide ? static_cast<const int64_t*>(ids)[t] : int64_t(static_cast<const int32_t*>(ids)[t]);
}

// Rows whose vectors all lie on 16-byte boundaries, in the table and the output.
template <class T, class O, int U>
__global__ void __launch_bounds__(kLookupThreads) lookup_aligned_kernel(const LookupArgs a) {
  constexpr int N = Span<T>::N;
  const int ty = kLookupThreads / a.tx, x = threadIdx.x & (a.tx - 1), y = threadIdx.x / a.tx;
  const int64_t t0 = grid_row() * (ty * U) + y;
  const int nvec = int(a.cols) / N, step = int(gridDim.x) * a.tx;
  int64_t id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * ty;
    id[u] = t < a.tokens ? id_at(a.ids, a.wide, t) : -1;
  }
  for (int i = int(blockIdx.x) * a.tx + x; i < nvec; i += step) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r[u] = make_uint4(0, 0, 0, 0);
      if (id[u] >= 0 && id[u] < a.rows)
        r[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.table) +
                                                    id[u] * a.ldt) + i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * ty;
      if (t >= a.tokens) continue;
      float v[N];
      unpack_vec<T>(r[u], v);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] *= a.scale;
      store_vec<O>(static_cast<O*>(a.out) + t * a.ldo + int64_t(i) * N, v);
    }
  }
}

// Rows at any offset: vectors that start on a 16-byte boundary of the output, each
// from two of the table's, and single elements before and after them.
template <class T, class O>
__global__ void __launch_bounds__(kLookupThreads) lookup_any_kernel(const LookupArgs a) {
  constexpr int N = Span<T>::N, U = 2;
  const int ty = kLookupThreads / a.tx, x = threadIdx.x & (a.tx - 1), y = threadIdx.x / a.tx;
  const int64_t t = grid_row() * ty + y;
  if (t >= a.tokens) return;
  const int cols = int(a.cols), step = int(gridDim.x) * a.tx;
  int64_t id = id_at(a.ids, a.wide, t);
  if (id < 0 || id >= a.rows) id = -1;
  O* dst = static_cast<O*>(a.out) + t * a.ldo;
  const T* src = static_cast<const T*>(a.table) + (id < 0 ? 0 : id * a.ldt);
  const int head = min(cols, int((16 - misalign(dst)) & 15) / int(sizeof(O)));
  const int nvec = (cols - head) / N, rest = cols - nvec * N;
  const int mis = misalign(src + head);
  const int first = inner_first(mis), last = inner_last<T>(cols - head, mis);
  const int x0 = int(blockIdx.x) * a.tx + x;
  for (int e = x0; e < rest; e += step) {
    const int c = e < head ? e : nvec * N + e;
    dst[c] = from_f32<O>((id >= 0 ? to_f32(src[c]) : 0.f) * a.scale);
  }
  for (int i0 = x0; i0 < nvec; i0 += U * step) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * step;
      r[u] = make_uint4(0, 0, 0, 0);
      if (id >= 0 && i < nvec)
        r[u] = i >= first && i <= last ? load_inner(src + head, i, mis)
                                       : load_edge(src + head, cols - head, i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * step;
      if (i >= nvec) continue;
      float v[N];
      unpack_vec<T>(r[u], v);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] *= a.scale;
      store_vec<O>(dst + head + i * N, v);
    }
  }
}

template <class T, class O>
int launch_lookup(LookupArgs a, cudaStream_t s) {
  constexpr int N = Span<T>::N;
  const int64_t nvec = std::max<int64_t>(1, a.cols / N);
  a.tx = 8;
  while (a.tx < kLookupThreads && a.tx < nvec) a.tx *= 2;
  const int ty = kLookupThreads / a.tx;
  const bool aligned = a.cols % N == 0 && a.ldt % N == 0 && a.ldo % N == 0 &&
                       reinterpret_cast<uintptr_t>(a.table) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  int64_t runs = std::min<int64_t>(ceil_div(nvec, a.tx), 64);
  if (!aligned) {
    lookup_any_kernel<T, O><<<grid_of(runs, ceil_div(a.tokens, ty)), kLookupThreads, 0, s>>>(a);
  } else if (a.tokens * runs >= int64_t(16) * num_sms() * ty) {
    // four tokens per thread hide their latency behind each other; one while there
    // are few, for more blocks
    lookup_aligned_kernel<T, O, 4>
        <<<grid_of(runs, ceil_div(a.tokens, 4 * ty)), kLookupThreads, 0, s>>>(a);
  } else {
    lookup_aligned_kernel<T, O, 1>
        <<<grid_of(runs, ceil_div(a.tokens, ty)), kLookupThreads, 0, s>>>(a);
  }
  IVFPQ_LAUNCHED();
  return IVFPQ_OK;
}

// ---- gradient: positions by token ----------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kMaxLocal = 16384;  // a block's tokens: 64 KB of counters
constexpr int kPerThread = 16;    // ids per thread and step
constexpr int kListed = 4096;     // a class's positions kept in shared memory

struct SortArgs {
  const void* ids;
  int wide;
  int64_t tokens, rows, padding;
  int shift;  // 2^shift classes, one per block
  int local;  // tokens of a class
  int32_t* list;   // [tokens] scratch: the class's positions in order
  int32_t* pos;    // [tokens] positions sorted by (class, token, position)
  int32_t* token;  // [tokens] their tokens
  int32_t* count;  // [rows] positions of each token
  int32_t* valid;  // [1] positions that hold a token
  int slab;
  int4* frequent;  // (token, first sorted position, positions, 0), by class
  int2* classes;   // [classes] each class's first entry there and how many it has
};

__device__ __forceinline__ int block_sum(int v, uint64_t* sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = int(__reduce_add_sync(kFullMask, unsigned(v)));
  __syncthreads();
  if (lane == 0) sh[warp] = uint64_t(v);
  __syncthreads();
  return int(__reduce_add_sync(kFullMask, lane < kSortThreads / 32 ? unsigned(sh[lane]) : 0u));
}
// The sum of v over the threads before this one; all: over the block. v may hold
// several counters side by side.
__device__ __forceinline__ uint64_t block_before(uint64_t v, uint64_t* sh, uint64_t* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int W = kSortThreads / 32;
  uint64_t in = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint64_t t = __shfl_up_sync(kFullMask, in, d);
    if (lane >= d) in += t;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = in;
  __syncthreads();
  uint64_t below = 0;
  *all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const uint64_t t = sh[w];
    if (w < warp) below += t;
    *all += t;
  }
  return below + in - v;
}

// The positions of a step that thread x takes: four groups of four, (j kSortThreads + x)
// 4 + e, so that a warp's loads are whole lines.
__device__ __forceinline__ int64_t position(int64_t t0, int j) {
  return t0 + (int64_t(j) * kSortThreads + threadIdx.x) * 4;
}
// Their tokens, -1 where there is none to count.
__device__ __forceinline__ void read_tokens(const SortArgs& a, int64_t t0, int (&v)[kPerThread]) {
  auto token = [&](int64_t id) {
    return id >= 0 && id < a.rows && id != a.padding ? int(id) : -1;
  };
  if (t0 + kSortThreads * kPerThread <= a.tokens && misalign(a.ids) == 0) {
    if (a.wide) {
      longlong2 w[kPerThread / 2];
#pragma unroll
      for (int j = 0; j < kPerThread / 2; ++j)
        w[j] = reinterpret_cast<const longlong2*>(static_cast<const int64_t*>(a.ids) +
                                                  position(t0, j / 2))[j % 2];
#pragma unroll
      for (int j = 0; j < kPerThread / 2; ++j) {
        v[2 * j] = token(w[j].x);
        v[2 * j + 1] = token(w[j].y);
      }
    } else {
      int4 w[kPerThread / 4];
#pragma unroll
      for (int j = 0; j < kPerThread / 4; ++j)
        w[j] = *reinterpret_cast<const int4*>(static_cast<const int32_t*>(a.ids) + position(t0, j));
#pragma unroll
      for (int j = 0; j < kPerThread / 4; ++j) {
        v[4 * j] = token(w[j].x);
        v[4 * j + 1] = token(w[j].y);
        v[4 * j + 2] = token(w[j].z);
        v[4 * j + 3] = token(w[j].w);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int64_t t = position(t0, j / 4) + j % 4;
    v[j] = t < a.tokens ? token(id_at(a.ids, a.wide, t)) : -1;
  }
}

__global__ void __launch_bounds__(kSortThreads, 1) embedding_sort_kernel(const SortArgs a) {
  extern __shared__ int sort_smem[];
  int* next = sort_smem;  // [local]: counts, then where a token's next position goes
  __shared__ int2 listed[kListed];  // (position, token) in order
  __shared__ uint64_t sh[kSortThreads / 32];
  __shared__ int nfrequent;
  const int c = blockIdx.x, mask = (1 << a.shift) - 1;
  const int lane = threadIdx.x & 31;
  constexpr int64_t step = int64_t(kSortThreads) * kPerThread;
  constexpr int G = kPerThread / 4;
  grid_go();
  int before = 0, v[kPerThread];
  read_tokens(a, 0, v);
  if (threadIdx.x == 0) nfrequent = 0;
  for (int i = threadIdx.x; i < a.local; i += kSortThreads) next[i] = 0;
  __syncthreads();
  for (int64_t t0 = 0; t0 < a.tokens; t0 += step) {
    if (t0 > 0) read_tokens(a, t0, v);
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int cls = v[j] & mask;
      before += v[j] >= 0 && cls < c;
      if (v[j] >= 0 && cls == c) atomicAdd(&next[v[j] >> a.shift], 1);
    }
  }
  const int base = block_sum(before, sh);
  // counts out; their running sums stay
  int n = 0;
  for (int i0 = 0; i0 < a.local; i0 += kSortThreads) {
    const int i = i0 + threadIdx.x;
    const int64_t token = (int64_t(i) << a.shift) + c;
    const int k = i < a.local ? next[i] : 0;
    if (i < a.local && token < a.rows) a.count[token] = k;
    uint64_t all;
    const int at = int(block_before(uint64_t(k), sh, &all));
    if (i < a.local) next[i] = n + at;
    // a class of n positions has at most n / (slab + 1) frequent tokens, so that no
    // two classes' entries meet
    if (k > a.slab)
      a.frequent[base / (a.slab + 1) + atomicAdd(&nfrequent, 1)] =
          make_int4(int(token), base + n + at, k, 0);
    n += int(all);
  }
  if (c == mask && threadIdx.x == 0) *a.valid = base + n;
  __syncthreads();
  if (threadIdx.x == 0) a.classes[c] = make_int2(base / (a.slab + 1), nfrequent);
  if (n == 0) return;
  // the class's positions in order, in shared memory while they fit
  int found = 0;
  const bool fits = n <= kListed;
  for (int64_t t0 = 0; found < n && t0 < a.tokens; t0 += step) {
    if (a.tokens > step) read_tokens(a, t0, v);
    // a 16-bit counter per group of four: a group has 4 kSortThreads at most
    uint64_t mine = 0;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      mine += uint64_t(v[j] >= 0 && (v[j] & mask) == c) << (16 * (j / 4));
    uint64_t all;
    const uint64_t at = block_before(mine, sh, &all);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      int place = found + int(at >> (16 * g) & 0xffff);
      if (mine >> (16 * g) & 0xffff) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int id = v[4 * g + e];
          if (id >= 0 && (id & mask) == c) {
            const int p = int(position(t0, g)) + e;
            if (fits)
              listed[place] = make_int2(p, id);
            else
              a.list[base + place] = p;
            ++place;
          }
        }
      }
      found += int(all >> (16 * g) & 0xffff);
    }
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  auto entry = [&](int i) {
    if (i >= n) return make_int2(-1, -1);
    if (fits) return listed[i];
    const int p = a.list[base + i];
    return make_int2(p, int(id_at(a.ids, a.wide, p)));
  };
  // what does not depend on the rows before is there ahead, four rows at a time
  constexpr int U = 4;
  for (int i0 = 0; i0 < n; i0 += 32 * U) {
    int2 e[U];
    unsigned same[U];
#pragma unroll
    for (int u = 0; u < U; ++u) e[u] = entry(i0 + 32 * u + lane);
#pragma unroll
    for (int u = 0; u < U; ++u) same[u] = __match_any_sync(kFullMask, e[u].y);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned below = same[u] & ((1u << lane) - 1u);
      int at = 0;
      if (e[u].y >= 0) at = next[e[u].y >> a.shift] + __popc(below);
      __syncwarp();
      if (e[u].y >= 0) {
        if (below == 0) next[e[u].y >> a.shift] = at + __popc(same[u]);
        a.pos[base + at] = e[u].x;
        a.token[base + at] = e[u].y;
      }
      __syncwarp();
    }
  }
}

// ---- gradient: sums ---------------------------------------------------------------------
constexpr int kMaxSlab = 256;
constexpr int kZeroRows = 8;  // rows that one block looks at to zero them

struct SumArgs {
  const void* grad;
  int64_t cols, ldg, rows, tokens;
  const int32_t* pos;
  const int32_t* token;
  const int32_t* count;
  const int32_t* valid;
  const int4* frequent;
  const int2* classes;
  int slab;
  int64_t slabs;
  float scale;
  int accumulate;
  float* part;  // [slabs, 2, pitch]: of the frequent token that goes on from the slab
                // before, and of the one that starts here and goes on into the next
  int64_t pitch;
  void* out;
  int64_t ldo;
};

// Row values of columns N cv .. N cv + N - 1 of token v.
template <class T, class O>
__device__ __forceinline__ void write_row(const SumArgs& a, int64_t v, int cv,
                                          const float (&s)[Span<T>::N]) {
  constexpr int N = Span<T>::N;
  O* dst = static_cast<O*>(a.out) + v * a.ldo + int64_t(cv) * N;
  const int have = int(min(int64_t(N), a.cols - int64_t(cv) * N));
  if (have == N && misalign(dst) == 0) {
    float w[N];
#pragma unroll
    for (int j = 0; j < N; ++j) w[j] = s[j] * a.scale;
    if (a.accumulate) {
      constexpr int M = Span<O>::N;
#pragma unroll
      for (int q = 0; q < N / M; ++q) {
        float old[M];
        unpack_vec<O>(reinterpret_cast<const uint4*>(dst)[q], old);
#pragma unroll
        for (int j = 0; j < M; ++j) w[q * M + j] += old[j];
      }
    }
    store_vec<O>(dst, w);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j < have) {
        float w = s[j] * a.scale;
        if (a.accumulate) w += to_f32(dst[j]);
        dst[j] = from_f32<O>(w);
      }
    }
  }
}
template <int N>
__device__ __forceinline__ float* part_at(const SumArgs& a, int64_t slab, int which, int cv) {
  return a.part + (slab * 2 + which) * a.pitch + int64_t(cv) * N;
}

template <class T, class O>
__device__ void zero_row(O* p, int len, int x, int step) {
  const Span<O> sp(p, len);
  for (int e = x; e < sp.rest(); e += step) p[sp.at(e)] = from_f32<O>(0.f);
  for (int i = x; i < sp.nvec; i += step)
    reinterpret_cast<uint4*>(p + sp.head)[i] = make_uint4(0, 0, 0, 0);
}

template <class T, class O>
__global__ void __launch_bounds__(256) embedding_sum_kernel(const SumArgs a) {
  constexpr int N = Span<T>::N, U = 8;
  __shared__ int32_t pos[2 * kMaxSlab], token[2 * kMaxSlab + 1];
  const int64_t slab = grid_row();
  grid_wait();
  grid_go();
  if (slab >= a.slabs) {
    // rows without a token
    const int step = int(gridDim.x * blockDim.x), x = int(blockIdx.x * blockDim.x + threadIdx.x);
    const int64_t v0 = (slab - a.slabs) * kZeroRows;
    for (int64_t v = v0; v < min(v0 + kZeroRows, a.rows); ++v)
      if (a.count[v] == 0)
        zero_row<T, O>(static_cast<O*>(a.out) + v * a.ldo, int(a.cols), x, step);
    return;
  }
  const int valid = *a.valid;
  const int64_t i0 = slab * a.slab;
  if (i0 >= valid) return;
  const int n = int(min(int64_t(a.slab), valid - i0));
  // this slab's and the next one's; token[0]: the last of the one before
  for (int i = threadIdx.x; i <= 2 * a.slab; i += blockDim.x) {
    const int64_t j = i0 + i - 1;
    token[i] = j >= 0 && j < valid ? a.token[j] : -1;
    if (i >= 1) pos[i - 1] = j < valid ? a.pos[j] : 0;
  }
  __syncthreads();
  // where a run of equal tokens that starts at i ends
  auto run_end = [&](int i, int hi) {
    const int32_t id = token[i];
    int lo = i;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (token[mid] == id)
        lo = mid;
      else
        hi = mid;
    }
    return hi;
  };
  // entries begin .. end - 1 (token[1 + i], pos[i]) are this block's
  int begin = 0, end = n;
  bool first = false, last = false;  // the first and the last token's sums are partial
  if (token[0] >= 0 && token[0] == token[1]) {
    if (a.count[token[1]] > a.slab)
      first = true;
    else
      begin = run_end(1, n + 1) - 1;
  }
  if (n == a.slab && token[n + 1] >= 0 && token[n] == token[n + 1]) {
    if (a.count[token[n]] > a.slab)
      last = true;
    else if (begin < n)
      end = run_end(n, 2 * a.slab + 1) - 1;
  }
  const int cv = int(blockIdx.x * blockDim.x + threadIdx.x);
  if (int64_t(cv) * N >= a.cols) return;
  const T* grad = static_cast<const T*>(a.grad);
  const int cols = int(a.cols);
  float s[N];
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = 0.f;
  for (int b = begin; b < end; b += U) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u < end) {
        const T* p = grad + pos[b + u] * a.ldg;
        r[u] = load_vec(p, cols, cv, misalign(p));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + u;
      if (i >= end) break;
      float v[N];
      unpack_vec<T>(r[u], v);
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] += v[j];
      if (i == end - 1 || token[i + 2] != token[i + 1]) {
        if (first || (last && i == end - 1)) {
          float* q = part_at<N>(a, slab, first ? 0 : 1, cv);
#pragma unroll
          for (int j = 0; j < N; j += 4)
            *reinterpret_cast<float4*>(q + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        } else {
          write_row<T, O>(a, token[i + 1], cv, s);
        }
        first = false;
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] = 0.f;
      }
    }
  }
}

// The frequent tokens, a class per row of blocks.
constexpr int kJoinThreads = 64, kJoinParts = 4;
template <class O>
__global__ void __launch_bounds__(kJoinThreads* kJoinParts) embedding_join_kernel(const SumArgs a) {
  __shared__ float4 sums[kJoinParts][kJoinThreads];
  grid_wait();
  const int2 mine = a.classes[blockIdx.y];
  const int c = int(blockIdx.x * kJoinThreads + threadIdx.x) * 4;
  for (int i = 0; i < mine.y; ++i) {
    const int4 token = a.frequent[mine.x + i];
    const int64_t slab = token.y / a.slab;
    const int more = int((int64_t(token.y) + token.z - 1) / a.slab - slab);
    // the first partial sum and those of the slabs it goes on for, in kJoinParts runs
    // of equal length, each summed in order, and the runs' sums in order
    const int run = (more + kJoinParts) / kJoinParts;
    const int k0 = threadIdx.y * run, k1 = min(k0 + run, more + 1);
    const float* from = a.part + slab * 2 * a.pitch + c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;
    for (int k = k0; k < k1 && c < a.cols; k += U) {
      float4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k + u < k1)
          w[u] = *reinterpret_cast<const float4*>(from + ((k + u) * 2 + (k + u == 0)) * a.pitch);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k + u < k1) {
          s.x += w[u].x;
          s.y += w[u].y;
          s.z += w[u].z;
          s.w += w[u].w;
        }
    }
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < a.cols) {
#pragma unroll
      for (int y = 1; y < kJoinParts; ++y) {
        const float4 t = sums[y][threadIdx.x];
        s.x += t.x;
        s.y += t.y;
        s.z += t.z;
        s.w += t.w;
      }
      const float v[4] = {s.x, s.y, s.z, s.w};
      O* dst = static_cast<O*>(a.out) + token.x * a.ldo + c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (c + j < a.cols) {
          float w = v[j] * a.scale;
          if (a.accumulate) w += to_f32(dst[j]);
          dst[j] = from_f32<O>(w);
        }
      }
    }
    __syncthreads();
  }
}

template <class K, class A>
int launch_after(K kern, dim3 grid, dim3 threads, const A& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
  IVFPQ_LAUNCHED_K(kern, 0, int(threads.x * threads.y));
  return IVFPQ_OK;
}

template <class T, class O>
int launch_sums(const SumArgs& a, int classes, cudaStream_t s) {
  const int64_t nvec = ceil_div(a.cols, Span<T>::N);
  int threads = 32;
  while (threads < 128 && threads < nvec) threads *= 2;
  const int64_t runs = ceil_div(nvec, threads);
  const int64_t zero = a.accumulate ? 0 : ceil_div(a.rows, kZeroRows);
  IVFPQ_TRY(launch_after(embedding_sum_kernel<T, O>, grid_of(runs, a.slabs + zero),
                         dim3(unsigned(threads)), a, s));
  if (a.slabs <= 1) return IVFPQ_OK;
  return launch_after(embedding_join_kernel<O>,
                      dim3(unsigned(ceil_div(a.cols, 4 * kJoinThreads)), unsigned(classes)),
                      dim3(kJoinThreads, kJoinParts), a, s);
}

int check_common(const char* fn, int dtype, int out_dtype, int64_t rows, int64_t cols,
                 int64_t tokens, int ids_bytes) {
  IVFPQ_REQUIRE(known_dtype(dtype) && known_dtype(out_dtype), "%s: unknown element type", fn);
  IVFPQ_REQUIRE(out_dtype == dtype || out_dtype == IVFPQ_F32,
                "%s: the output is of the input's type or fp32", fn);
  IVFPQ_REQUIRE(rows >= 0 && rows <= (int64_t(1) << 24), "%s: rows=%lld outside [0, 2^24]", fn,
                (long long)rows);
  IVFPQ_REQUIRE(cols >= 0 && cols <= (int64_t(1) << 20), "%s: cols=%lld outside [0, 2^20]", fn,
                (long long)cols);
  IVFPQ_REQUIRE(tokens >= 0 && tokens < (int64_t(1) << 30), "%s: tokens=%lld outside [0, 2^30)",
                fn, (long long)tokens);
  IVFPQ_REQUIRE(ids_bytes == 4 || ids_bytes == 8, "%s: ids of %d bytes", fn, ids_bytes);
  return IVFPQ_OK;
}

}  // namespace
}  // namespace ivfpq

using namespace ivfpq;

extern "C" int embedding_lookup(const void* table, int dtype, int64_t rows, int64_t cols,
                                int64_t ldt, const void* ids, int ids_bytes, int64_t tokens,
                                float scale, void* out, int out_dtype, int64_t ldo, void* stream) {
  clear_error();
  IVFPQ_TRY(check_common("embedding_lookup", dtype, out_dtype, rows, cols, tokens, ids_bytes));
  IVFPQ_REQUIRE(rows <= 1 || ldt >= cols || ldt == 0,
                "embedding_lookup: row stride %lld below cols=%lld", (long long)ldt,
                (long long)cols);
  IVFPQ_REQUIRE(tokens <= 1 || ldo >= cols, "embedding_lookup: row stride %lld below cols=%lld",
                (long long)ldo, (long long)cols);
  if (tokens == 0 || cols == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(ids && out && (table || rows == 0), "embedding_lookup: null pointer");
  const LookupArgs a{table, rows, cols, ldt, ids, ids_bytes == 8, tokens, scale, out, ldo, 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    return out_dtype == dtype ? launch_lookup<T, T>(a, s) : launch_lookup<T, float>(a, s);
  });
}

extern "C" int embedding_gradient(const void* grad, int dtype, int64_t tokens, int64_t cols,
                                  int64_t ldg, const void* ids, int ids_bytes, int64_t rows,
                                  float scale, int64_t padding, int accumulate, void* out,
                                  int out_dtype, int64_t ldo, void* stream) {
  clear_error();
  IVFPQ_TRY(check_common("embedding_gradient", dtype, out_dtype, rows, cols, tokens, ids_bytes));
  IVFPQ_REQUIRE(tokens <= 1 || ldg >= cols || ldg == 0,
                "embedding_gradient: row stride %lld below cols=%lld", (long long)ldg,
                (long long)cols);
  IVFPQ_REQUIRE(rows <= 1 || ldo >= cols, "embedding_gradient: row stride %lld below cols=%lld",
                (long long)ldo, (long long)cols);
  if (rows == 0 || cols == 0 || (tokens == 0 && accumulate)) return IVFPQ_OK;
  IVFPQ_REQUIRE(out && ((ids && grad) || tokens == 0), "embedding_gradient: null pointer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  SortArgs o{};
  o.ids = ids;
  o.wide = ids_bytes == 8;
  o.tokens = tokens;
  o.rows = rows;
  o.padding = padding;
  // a block per SM or nearly, and more where a class would have too many tokens
  o.shift = 7;
  while (ceil_div(rows, int64_t(1) << o.shift) > kMaxLocal) ++o.shift;
  o.local = int(ceil_div(rows, int64_t(1) << o.shift));
  SumArgs a{};
  a.grad = grad;
  a.cols = cols;
  a.ldg = ldg;
  a.rows = rows;
  a.tokens = tokens;
  a.scale = scale;
  a.accumulate = accumulate != 0;
  a.out = out;
  a.ldo = ldo;
  a.slab = 32;
  while (a.slab < kMaxSlab && tokens > int64_t(a.slab) * 1024) a.slab *= 2;
  a.slabs = ceil_div(tokens, a.slab);
  a.pitch = ceil_div(cols, 8) * 8;
  Workspace ws(s);
  // the slabs' partial sums, the frequent tokens and the sorted positions
  const size_t parts = a.slabs > 1 ? size_t(a.slabs) * 2 * size_t(a.pitch) : 0;
  const size_t frequent = size_t(tokens / (a.slab + 1) + 1), classes = size_t(1) << o.shift;
  int4* w = nullptr;
  IVFPQ_TRY(ws.alloc(&w, parts / 4 + frequent + (classes + 1) / 2 +
                             (size_t(tokens) * 3 + size_t(rows) + 4) / 4));
  a.part = reinterpret_cast<float*>(w);
  o.frequent = w + parts / 4;
  o.classes = reinterpret_cast<int2*>(o.frequent + frequent);
  o.list = reinterpret_cast<int32_t*>(o.frequent + frequent + (classes + 1) / 2);
  o.pos = o.list + tokens;
  o.token = o.pos + tokens;
  o.count = o.token + tokens;
  o.valid = o.count + rows;
  o.slab = a.slab;
  a.frequent = o.frequent;
  a.classes = o.classes;
  a.pos = o.pos;
  a.token = o.token;
  a.count = o.count;
  a.valid = o.valid;
  const size_t smem = size_t(o.local) * 4;
  // 48 KB with the static part need no leave
  if (smem > 12 * 1024) IVFPQ_TRY(set_dynamic_smem(embedding_sort_kernel, smem));
  embedding_sort_kernel<<<1u << o.shift, kSortThreads, smem, s>>>(o);
  IVFPQ_LAUNCHED_K(embedding_sort_kernel, smem, kSortThreads);
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    return out_dtype == dtype ? launch_sums<T, T>(a, 1 << o.shift, s)
                              : launch_sums<T, float>(a, 1 << o.shift, s);
  });
}
