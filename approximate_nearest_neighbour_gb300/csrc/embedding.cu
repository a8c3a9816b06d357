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
//     tokens go without hearing from the other blocks. They are put into their
//     tokens' places in any order, and then ordered by rank, or by a bitmap of the
//     positions where a token has many: a range of positions at a time, only those that
//     hold one. A class that does not fit shared memory is put in place a range after the
//     other, so that each looks at its own part of the list alone.
//  2. The sorted positions are cut into slabs of equal length. A block adds a slab's
//     rows over a run of columns in registers (fp32) and writes a row where the
//     token changes. A token that goes on beyond its slab is finished by the block in
//     whose slab it starts; one with more positions than a slab has (a frequent token
//     is many slabs' work, not one block's) leaves a partial sum in every slab.
//     Further blocks zero the rows without a token.
//  3. The partial sums of a frequent token are added in slab order.
// Up to 256 positions one kernel does all of it, without workspace: a block finds the
// positions of its class, sorts them by rank, and a warp adds each token's rows.
//
// Measured: lookup of 8192 x 4096 bf16 17.5 us on the device, 6.7 TB/s, the copy rate;
// with 4095 columns 28.8 us as a program calls it (20.7 us with 4096), two bytes per lane
// and access. Gradient of 16384 x 4096 bf16 into 32000 rows (396 MB) 55.3 us for the sums,
// 6.0 TB/s, behind 10.7 us of sorting, which reads all ids once per class, and before
// 8.9 us of joining the frequent tokens (all with cold caches). Bulk copies for the rows
// and a prefetch of them into L2 were slower than plain loads of eight rows at a time.
// Positions of one token throughout, one block's work, take time as they are many: 65536 x 8
// fp32 0.28 ms, 2^20 3.1 ms, 2^23 28 ms.
#include <limits.h>

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
// Tokens of a thread, whose latencies hide behind each other. (One token per thread: 29
// instead of 21 us for 8192 tokens of 4096 bf16, 31 instead of 29 us for 4095; 37
// tokens take 3.3 us on the device with one and 3.5 us with four.)
constexpr int kAlignedTokens = 4, kAnyTokens = 2;

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
template <class T, class O>
__global__ void __launch_bounds__(kLookupThreads) lookup_aligned_kernel(const LookupArgs a) {
  constexpr int N = Span<T>::N, U = kAlignedTokens;
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
      // an id outside the table: zeros, whatever the scale
      const float scale = id[u] >= 0 && id[u] < a.rows ? a.scale : 0.f;
      float v[N];
      unpack_vec<T>(r[u], v);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] *= scale;
      store_vec<O>(static_cast<O*>(a.out) + t * a.ldo + int64_t(i) * N, v);
    }
  }
}

// Rows at any offset: a thread has one of every 32 of its warp's 32 N columns, so that
// loads and stores are whole lines but for their ends.
template <class T, class O>
__global__ void __launch_bounds__(kLookupThreads) lookup_any_kernel(const LookupArgs a) {
  constexpr int N = Span<T>::N, U = kAnyTokens;
  const int ty = kLookupThreads / a.tx, x = threadIdx.x & (a.tx - 1), y = threadIdx.x / a.tx;
  const int64_t t0 = grid_row() * (ty * U) + y;
  const int cols = int(a.cols), step = int(gridDim.x) * a.tx * N;
  const T* src[U];
  O* dst[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * ty;
    const int64_t id = t < a.tokens ? id_at(a.ids, a.wide, t) : -1;
    src[u] = id >= 0 && id < a.rows ? static_cast<const T*>(a.table) + id * a.ldt : nullptr;
    dst[u] = t < a.tokens ? static_cast<O*>(a.out) + t * a.ldo : nullptr;
  }
  const int lane = x & 31;
  for (int c0 = (int(blockIdx.x) * a.tx + x - lane) * N + lane; c0 < cols; c0 += step) {
    T r[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < N; ++j)
        r[u][j] = src[u] && c0 + 32 * j < cols ? src[u][c0 + 32 * j] : from_f32<T>(0.f);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (dst[u] && c0 + 32 * j < cols)
          dst[u][c0 + 32 * j] = from_f32<O>(to_f32(r[u][j]) * (src[u] ? a.scale : 0.f));
  }
}

template <class T, class O>
int launch_lookup(LookupArgs a, cudaStream_t s) {
  constexpr int N = Span<T>::N;
  const int64_t nvec = ceil_div(a.cols, N);
  const bool aligned = a.cols % N == 0 && a.ldt % N == 0 && a.ldo % N == 0 &&
                       reinterpret_cast<uintptr_t>(a.table) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  a.tx = aligned ? 8 : 32;
  while (a.tx < kLookupThreads && a.tx < nvec) a.tx *= 2;
  const int ty = kLookupThreads / a.tx;
  const int64_t runs = std::min<int64_t>(ceil_div(nvec, a.tx), 64);
  const dim3 grid = grid_of(runs, ceil_div(a.tokens, ty * (aligned ? kAlignedTokens : kAnyTokens)));
  auto kern = aligned ? lookup_aligned_kernel<T, O> : lookup_any_kernel<T, O>;
  kern<<<grid, kLookupThreads, 0, s>>>(a);
  IVFPQ_LAUNCHED();
  return IVFPQ_OK;
}

// ---- gradient: positions by token ----------------------------------------------------
constexpr int kMaxLocal = 16384;  // a block's tokens: 128 KB of counters
constexpr int kPerThread = 16;    // ids per thread and step
constexpr int kMostListed = 8192;  // a class's positions kept in shared memory
constexpr int kRanked = 128;      // a token's positions that are ordered by rank
constexpr int kBitmap = 1024;     // words of the bitmap of positions
constexpr int kRange = kBitmap * 32;  // positions of a bitmap

struct SortArgs {
  const void* ids;
  int64_t tokens;
  uint32_t rows, padding;  // padding: no row where there is none
  int shift;  // 2^shift classes, one per block
  int local;  // tokens of a class
  int2* list;      // [tokens] scratch: a class's (position, token) by token
  int32_t* pos;    // [tokens] positions sorted by (class, token, position)
  int32_t* token;  // [tokens] their tokens; kFrequent marks those with more than `slab`
  int32_t* count;  // [rows] positions of each token
  int32_t* valid;  // [1] positions that hold a token
  int slab;
  int listed;      // a class's positions that fit shared memory
  int4* frequent;  // (token, first sorted position, positions, 0), by class
  int2* classes;   // [classes] each class's first entry there and how many it has
};

template <int THREADS>
__device__ __forceinline__ int block_sum(int v, int* sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = int(__reduce_add_sync(kFullMask, unsigned(v)));
  __syncthreads();
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  return int(__reduce_add_sync(kFullMask, lane < THREADS / 32 ? unsigned(sh[lane]) : 0u));
}
// The sum of v over the threads before this one; all: over the block.
template <int THREADS>
__device__ __forceinline__ int block_before(int v, int* sh, int* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int in = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int t = __shfl_up_sync(kFullMask, in, d);
    if (lane >= d) in += t;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = in;
  __syncthreads();
  const int w = lane < THREADS / 32 ? sh[lane] : 0;
  *all = int(__reduce_add_sync(kFullMask, unsigned(w)));
  return int(__reduce_add_sync(kFullMask, unsigned(lane < warp ? w : 0))) + in - v;
}

// The positions of a step that thread x takes: four groups of four, (j THREADS + x)
// 4 + e, so that a warp's loads are whole lines.
template <int THREADS>
__device__ __forceinline__ int64_t position(int64_t t0, int j) {
  return t0 + (int64_t(j) * THREADS + threadIdx.x) * 4;
}
// Their tokens, kNone where there is none to count.
constexpr uint32_t kNone = 0xffffffffu;
constexpr int32_t kFrequent = 1 << 30;  // above any token
template <bool WIDE, int THREADS>
__device__ __forceinline__ void read_tokens(const SortArgs& a, int64_t t0,
                                            uint32_t (&v)[kPerThread]) {
  using Id = std::conditional_t<WIDE, int64_t, int32_t>;
  const Id* ids = static_cast<const Id*>(a.ids);
  auto token = [&](Id id) {
    const uint32_t u = uint32_t(id);
    const bool ok = u < a.rows && u != a.padding && (!WIDE || Id(u) == id);
    return ok ? u : kNone;
  };
  if (t0 + THREADS * kPerThread <= a.tokens && misalign(a.ids) == 0) {
    Id w[kPerThread];
    constexpr int V = 16 / int(sizeof(Id));  // ids of a load
#pragma unroll
    for (int j = 0; j < kPerThread / V; ++j)
      *reinterpret_cast<uint4*>(w + j * V) =
          reinterpret_cast<const uint4*>(ids + position<THREADS>(t0, j * V / 4))[j % (4 / V)];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) v[j] = token(w[j]);
    return;
  }
#pragma unroll 4
  for (int j = 0; j < kPerThread; ++j) {
    const int64_t t = position<THREADS>(t0, j / 4) + j % 4;
    v[j] = t < a.tokens ? token(ids[t]) : kNone;
  }
}

// counter[i] of every lane with i >= 0 grows by one; returns what it was before the lane.
// One addition per counter and warp: a frequent token is most of its class.
__device__ __forceinline__ int take_place(int* counter, int i) {
  const int lane = threadIdx.x & 31;
  const unsigned same = __match_any_sync(kFullMask, i);
  const int first = __ffs(same) - 1;
  int at = 0;
  if (i >= 0 && lane == first) at = atomicAdd(&counter[i], __popc(same));
  at = __shfl_sync(kFullMask, at, first);
  return at + __popc(same & ((1u << lane) - 1u));
}

template <bool WIDE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) embedding_sort_kernel(const SortArgs a) {
  extern __shared__ int sort_smem[];
  int* start = sort_smem;  // [local + 1]: counts, then where a token's positions start
  int* fill = start + a.local + 1;  // [local]: how many of them have a place
  int2* list_smem = reinterpret_cast<int2*>(start + (2 * a.local + 2) / 2 * 2);  // [listed]
  int2* met = list_smem + a.listed;  // [listed] the class's positions as they were met
  __shared__ uint32_t bitmap[kBitmap];
  __shared__ int sh[THREADS / 32];
  __shared__ int nfrequent, nmet;
  const uint32_t c = blockIdx.x, mask = (1u << a.shift) - 1;
  constexpr int64_t step = int64_t(THREADS) * kPerThread;
  grid_go();
  int before = 0;
  uint32_t v[kPerThread];
  read_tokens<WIDE, THREADS>(a, 0, v);
  if (threadIdx.x == 0) nfrequent = nmet = 0;
  for (int i = threadIdx.x; i < 2 * a.local + 1; i += THREADS) start[i] = 0;
  __syncthreads();
  // (kNone's class is the last: it counts as before none)
  const int lane = threadIdx.x & 31;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += step) {
    if (t0 > 0) read_tokens<WIDE, THREADS>(a, t0, v);
    uint32_t hits = 0;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const uint32_t cls = v[j] & mask;
      before += cls < c;
      hits |= uint32_t(cls == c && v[j] != kNone) << j;
    }
    if (!__any_sync(kFullMask, hits != 0)) continue;
    int in = __popc(hits);
    const int own = in;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int t = __shfl_up_sync(kFullMask, in, d);
      if (lane >= d) in += t;
    }
    int i = 0;
    if (lane == 31) i = atomicAdd(&nmet, in);
    i = __shfl_sync(kFullMask, i, 31) + in - own;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (hits >> j & 1) {
        if (i < a.listed)
          met[i] = make_int2(int(position<THREADS>(t0, j / 4)) + j % 4, int(v[j]));
        ++i;
      }
    }
  }
  const int base = block_sum<THREADS>(before, sh);
  const int found = nmet;
  const bool fits = found <= a.listed;
  // Calls f(j, token, place) for this thread's ids of the class among v: their places among
  // the token's that `counter` counts. An addition per id, unless many are of the class
  // and so perhaps of one token.
  auto count_step = [&](int* counter, auto&& f) {
    unsigned hits = 0;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      hits |= unsigned((v[j] & mask) == c && v[j] != kNone) << j;
    if (__reduce_add_sync(kFullMask, unsigned(__popc(hits))) > 4 * kPerThread) {
      // (four copies of the code: all sixteen slow the other branch, too)
#pragma unroll 1
      for (int q = 0; q < kPerThread; q += 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t t = v[e];
#pragma unroll
          for (int j = 4; j < kPerThread; j += 4) t = q == j ? v[j + e] : t;
          const bool hit = hits >> (q + e) & 1;
          const int at = take_place(counter, hit ? int(t >> a.shift) : -1);
          if (hit) f(q + e, t, at);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPerThread; ++j)
        if (hits >> j & 1) f(j, v[j], atomicAdd(&counter[v[j] >> a.shift], 1));
    }
  };
  if (fits) {
    for (int i0 = 0; i0 < found; i0 += THREADS) {
      const int i = i0 + threadIdx.x;
      take_place(start, i < found ? met[i].y >> a.shift : -1);
    }
  } else {
    for (int64_t t0 = 0; t0 < a.tokens; t0 += step) {
      read_tokens<WIDE, THREADS>(a, t0, v);
      count_step(start, [](int, uint32_t, int) {});
    }
  }
  __syncthreads();
  // counts out; their running sums stay
  int n = 0;
  for (int i0 = 0; i0 < a.local; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    const int64_t token = (int64_t(i) << a.shift) + c;
    const int k = i < a.local ? start[i] : 0;
    if (i < a.local && token < a.rows) a.count[token] = k;
    int all;
    const int at = n + block_before<THREADS>(k, sh, &all);
    if (i < a.local) start[i] = at;
    if (k > a.slab) {
      // a class of n positions has at most n / (slab + 1) frequent tokens, so that no
      // two classes' entries meet
      const int j = atomicAdd(&nfrequent, 1);
      a.frequent[base / (a.slab + 1) + j] = make_int4(int(token), base + at, k, 0);
    }
    n += all;
  }
  if (threadIdx.x == 0) start[a.local] = n;
  if (c == mask && threadIdx.x == 0) *a.valid = base + n;
  __syncthreads();
  if (threadIdx.x == 0) a.classes[c] = make_int2(base / (a.slab + 1), nfrequent);
  if (n == 0) return;
  // positions to their tokens' places, in any order
  int2* list = fits ? list_smem : a.list + base;
  if (fits) {
    for (int i0 = 0; i0 < n; i0 += THREADS) {
      const int i = i0 + threadIdx.x;
      const int2 e = i < n ? met[i] : make_int2(0, 0);
      const int l = i < n ? e.y >> a.shift : -1, at = take_place(fill, l);
      if (i < n) list[start[l] + at] = e;
    }
  } else {
    read_tokens<WIDE, THREADS>(a, 0, v);
    for (int64_t t0 = 0; t0 < a.tokens; t0 += step) {
      uint32_t next[kPerThread];
      if (t0 + step < a.tokens) read_tokens<WIDE, THREADS>(a, t0 + step, next);
      count_step(fill, [&](int j, uint32_t t, int at) {
        list[start[t >> a.shift] + at] =
            make_int2(int(position<THREADS>(t0, j / 4)) + j % 4, int(t));
      });
      if ((t0 + step) % kRange == 0) __syncthreads();  // these lie before the next range's
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) v[j] = next[j];
    }
  }
  __syncthreads();
  // few of a token: each by its rank among them
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const int2 e = list[i];
    const int l = e.y >> a.shift, from = start[l], k = start[l + 1] - from;
    if (k > kRanked) continue;
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < k; ++j) rank += list[from + j].x < e.x;
    a.pos[base + from + rank] = e.x;
    a.token[base + from + rank] = e.y | (k > a.slab ? kFrequent : 0);
  }
  // many: a bitmap of the positions, a range of them at a time. `later`: a position
  // in the next range that holds one.
  static_assert(kRange % step == 0, "whole steps");
  __shared__ int later;
  unsigned more = 0;  // of 32 tokens from l0 on, the same in every warp
  for (int l0 = -32;;) {
    while (more == 0 && (l0 += 32) < a.local)
      more = __ballot_sync(kFullMask, l0 + lane < a.local &&
                                          start[min(l0 + lane + 1, a.local)] -
                                                  start[min(l0 + lane, a.local)] > kRanked);
    if (more == 0) break;
    const int l = l0 + __ffs(more) - 1, from = start[l], k = start[l + 1] - from;
    more &= more - 1;
    const int id = int((uint32_t(l) << a.shift) + c) | (k > a.slab ? kFrequent : 0);
    int done = 0;  // positions of the token that have their place
    for (int64_t t0 = 0; t0 < a.tokens;) {
      __syncthreads();
      for (int i = threadIdx.x; i < kBitmap; i += THREADS) bitmap[i] = 0;
      if (threadIdx.x == 0) later = INT_MAX;
      __syncthreads();
      int behind = INT_MAX;
      for (int i = (fits ? 0 : done) + threadIdx.x; i < k; i += THREADS) {
        const int x = list[from + i].x;
        const int64_t p = x - t0;
        if (p >= kRange) {
          behind = min(behind, x);
          if (!fits) break;  // so are all that follow
        } else if (p >= 0) {
          atomicOr(&bitmap[p >> 5], 1u << (p & 31));
        }
      }
      behind = __reduce_min_sync(kFullMask, behind);
      if (lane == 0 && behind != INT_MAX) atomicMin(&later, behind);
      __syncthreads();
      const int next = later;
      constexpr int W = kBitmap / THREADS;  // words of a thread
      uint32_t bits[W];
      int mine = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        bits[i] = bitmap[threadIdx.x * W + i];
        mine += __popc(bits[i]);
      }
      int all, to = base + from + done + block_before<THREADS>(mine, sh, &all);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        for (; bits[i]; bits[i] &= bits[i] - 1) {
          a.pos[to] = int(t0) + (int(threadIdx.x) * W + i) * 32 + __ffs(bits[i]) - 1;
          a.token[to++] = id;
        }
      }
      done += all;
      if (next == INT_MAX) break;
      t0 = int64_t(next / kRange) * kRange;
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

// A thread has N columns of a row. VEC (rows of grad and out are whole vectors on
// 16-byte boundaries): a vector, N cv and following. Else one of every 32 in its warp's
// 32 N columns: whole lines whatever the offset, and nothing at the ends.
template <int N, bool VEC>
__device__ __forceinline__ int column(int cv, int j) {
  const int lane = threadIdx.x & 31;
  return VEC ? cv * N + j : (cv - lane) * N + j * 32 + lane;
}
// The row of token v.
template <class T, class O, bool VEC>
__device__ __forceinline__ void write_row(const SumArgs& a, int64_t v, int cv,
                                          const float (&s)[Span<T>::N]) {
  constexpr int N = Span<T>::N, M = Span<O>::N;
  if constexpr (VEC) {
    O* dst = static_cast<O*>(a.out) + v * a.ldo + int64_t(cv) * N;
#pragma unroll
    for (int q = 0; q < N / M; ++q) {
      float w[M];
#pragma unroll
      for (int j = 0; j < M; ++j) w[j] = s[q * M + j] * a.scale;
      if (a.accumulate) {
        float old[M];
        unpack_vec<O>(reinterpret_cast<const uint4*>(dst)[q], old);
#pragma unroll
        for (int j = 0; j < M; ++j) w[j] += old[j];
      }
      reinterpret_cast<uint4*>(dst)[q] = pack_vec<O>(w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = column<N, VEC>(cv, j);
      if (c < a.cols) {
        O* dst = static_cast<O*>(a.out) + v * a.ldo + c;
        float w = s[j] * a.scale;
        if (a.accumulate) w += to_f32(*dst);
        *dst = from_f32<O>(w);
      }
    }
  }
}
// Adds the rows pos[b], pos[b + 1], .. before `end`, U of them at most: add(u, values).
template <class T, bool VEC, int U, class F>
__device__ __forceinline__ void take_rows(const SumArgs& a, const int32_t* pos, int b, int end,
                                          int cv, F&& add) {
  constexpr int N = Span<T>::N;
  const T* grad = static_cast<const T*>(a.grad);
  if constexpr (VEC) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (b + u < end) r[u] = reinterpret_cast<const uint4*>(grad + pos[b + u] * a.ldg)[cv];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u < end) {
        float v[N];
        unpack_vec<T>(r[u], v);
        add(b + u, v);
      }
    }
  } else {
    T r[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u < end) {
        const T* p = grad + pos[b + u] * a.ldg;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int c = column<N, VEC>(cv, j);
          r[u][j] = c < a.cols ? p[c] : from_f32<T>(0.f);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u < end) {
        float v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = to_f32(r[u][j]);
        add(b + u, v);
      }
    }
  }
}
// The partial sums of a slab's token.
template <int N, bool VEC>
__device__ __forceinline__ void write_part(const SumArgs& a, int64_t slab, int which, int cv,
                                           const float (&s)[N]) {
  float* q = a.part + (slab * 2 + which) * a.pitch;
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < N; j += 4)
      *reinterpret_cast<float4*>(q + cv * N + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = column<N, VEC>(cv, j);
      if (c < a.cols) q[c] = s[j];
    }
  }
}

template <class O>
__device__ __forceinline__ void zero_row(O* p, int len, int x, int step) {
  const Span<O> sp(p, len);
  for (int e = x; e < sp.rest(); e += step) p[sp.at(e)] = from_f32<O>(0.f);
  for (int i = x; i < sp.nvec; i += step)
    reinterpret_cast<uint4*>(p + sp.head)[i] = make_uint4(0, 0, 0, 0);
}

template <class T, class O, bool VEC>
__global__ void __launch_bounds__(128) embedding_sum_kernel(const SumArgs a) {
  constexpr int N = Span<T>::N, U = VEC ? 8 : 4;
  __shared__ int32_t pos[2 * kMaxSlab], token[2 * kMaxSlab + 1];
  const int64_t slab = grid_row();
  grid_wait();
  grid_go();
  if (slab >= a.slabs) {
    // rows without a token
    const int step = int(gridDim.x * blockDim.x), x = int(blockIdx.x * blockDim.x + threadIdx.x);
    const int64_t v0 = (slab - a.slabs) * kZeroRows;
    int32_t count[kZeroRows];
#pragma unroll
    for (int i = 0; i < kZeroRows; ++i) count[i] = v0 + i < a.rows ? a.count[v0 + i] : 1;
#pragma unroll 1
    for (int i = 0; i < kZeroRows; ++i) {
      if (count[0] == 0)
        zero_row(static_cast<O*>(a.out) + (v0 + i) * a.ldo, int(a.cols), x, step);
#pragma unroll
      for (int j = 0; j + 1 < kZeroRows; ++j) count[j] = count[j + 1];
    }
    return;
  }
  const int64_t i0 = slab * a.slab;
  const int valid = *a.valid;
  // this slab's and the next one's; token[0]: the last of the one before. (What lies
  // past the valid positions is read along with them and not looked at.)
  for (int i = threadIdx.x; i <= 2 * a.slab; i += blockDim.x) {
    const int64_t j = i0 + i - 1;
    const bool there = j >= 0 && j < a.tokens;
    const int32_t id = there ? a.token[j] : -1, p = there ? a.pos[j] : 0;
    token[i] = j < valid ? id : -1;
    if (i >= 1) pos[i - 1] = p;
  }
  if (i0 >= valid) return;
  const int n = int(min(int64_t(a.slab), valid - i0));
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
    if (token[1] & kFrequent)
      first = true;
    else
      begin = run_end(1, n + 1) - 1;
  }
  if (n == a.slab && token[n + 1] >= 0 && token[n] == token[n + 1]) {
    if (token[n] & kFrequent)
      last = true;
    else if (begin < n)
      end = run_end(n, 2 * a.slab + 1) - 1;
  }
  const int cv = int(blockIdx.x * blockDim.x + threadIdx.x);
  if (column<N, VEC>(cv, 0) >= a.cols) return;
  float s[N];
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = 0.f;
  for (int b = begin; b < end; b += U)
    take_rows<T, VEC, U>(a, pos, b, end, cv, [&](int i, const float (&v)[N]) {
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] += v[j];
      if (i == end - 1 || token[i + 2] != token[i + 1]) {
        if (first || (last && i == end - 1))
          write_part<N, VEC>(a, slab, first ? 0 : 1, cv, s);
        else
          write_row<T, O, VEC>(a, token[i + 1] & ~kFrequent, cv, s);
        first = false;
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] = 0.f;
      }
    });
}

// The frequent tokens, a class per row of blocks.
constexpr int kJoinThreads = 64, kJoinParts = 4;
template <class O>
__global__ void __launch_bounds__(kJoinThreads* kJoinParts) embedding_join_kernel(const SumArgs a) {
  __shared__ float4 sums[kJoinParts][kJoinThreads];
  grid_wait();
  const int2 mine = a.classes[blockIdx.y];
  const int c = int(blockIdx.x * kJoinThreads + threadIdx.x) * 4;
  for (int i = blockIdx.z; i < mine.y; i += gridDim.z) {
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

// Whether rows of grad and out are whole vectors on 16-byte boundaries.
template <class T, class O>
bool whole_vectors(const SumArgs& a) {
  return a.cols % Span<T>::N == 0 && a.ldg % Span<T>::N == 0 && a.ldo % Span<O>::N == 0 &&
         reinterpret_cast<uintptr_t>(a.grad) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
}

// ---- gradient of few positions -------------------------------------------------------
constexpr int kFew = 256;
constexpr int kFewThreads = 512;
constexpr int kFewShift = 8;  // 256 classes, one per block
constexpr int kFewLocal = (1 << 24) >> kFewShift;

struct FewArgs {
  SumArgs sum;
  const void* ids;
  int wide;
  int64_t padding;
};

template <class T, class O, bool VEC>
__global__ void __launch_bounds__(kFewThreads) embedding_few_kernel(const FewArgs f) {
  constexpr int N = Span<T>::N, U = VEC ? 8 : 4;
  const SumArgs& a = f.sum;
  __shared__ int32_t token[kFew], pos[kFew];    // the class's, by position
  __shared__ int32_t stoken[kFew], spos[kFew];  // sorted by token
  __shared__ int starts[kFew + 1];              // where tokens begin there
  __shared__ uint32_t there[kFewLocal / 32];    // tokens of the class that occur
  __shared__ int found[kFew / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t c = blockIdx.x, mask = (1u << kFewShift) - 1;
  const int local = int((a.rows - c + mask) >> kFewShift);  // rows of the class
  // the number of flagged threads before this one among the first kFew; n: of all
  auto compact = [&](bool flag, int& n) {
    const unsigned b = __ballot_sync(kFullMask, flag);
    __syncthreads();
    if (lane == 0 && warp < kFew / 32) found[warp] = __popc(b);
    __syncthreads();
    int at = __popc(b & ((1u << lane) - 1u));
    n = 0;
#pragma unroll
    for (int w = 0; w < kFew / 32; ++w) {
      if (w < warp) at += found[w];
      n += found[w];
    }
    return at;
  };
  const int t = threadIdx.x;
  int64_t id = -1;
  if (t < a.tokens) id = id_at(f.ids, f.wide, t);
  for (int i = t; i < (local + 31) / 32; i += kFewThreads) there[i] = 0;
  const bool mine = t < a.tokens && id >= 0 && id < a.rows && id != f.padding &&
                    (uint32_t(id) & mask) == c;
  int n;
  const int at = compact(mine, n);
  if (mine) {
    token[at] = int32_t(id);
    pos[at] = t;
    const uint32_t l = uint32_t(id) >> kFewShift;
    atomicOr(&there[l >> 5], 1u << (l & 31));
  }
  __syncthreads();
  if (t < n) {
    const int32_t v = token[t];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += token[j] < v || (token[j] == v && j < t);
    stoken[rank] = v;
    spos[rank] = pos[t];
  }
  __syncthreads();
  int segments;
  const bool begins = t < n && (t == 0 || stoken[t - 1] != stoken[t]);
  const int s_at = compact(begins, segments);
  if (begins) starts[s_at] = t;
  if (t == 0) starts[segments] = n;
  __syncthreads();
  const int nvec = int((a.cols + N - 1) / N), runs = (nvec + 31) / 32;
  for (int i = warp; i < segments * runs; i += kFewThreads / 32) {
    const int g = i / runs, cv = (i - g * runs) * 32 + lane, end = starts[g + 1];
    if (column<N, VEC>(cv, 0) >= a.cols) continue;
    float s[N];
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = 0.f;
    for (int b = starts[g]; b < end; b += U)
      take_rows<T, VEC, U>(a, spos, b, end, cv, [&](int, const float (&v)[N]) {
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] += v[j];
      });
    write_row<T, O, VEC>(a, stoken[starts[g]], cv, s);
  }
  if (a.accumulate) return;
  for (int l = warp; l < local; l += kFewThreads / 32)
    if (!(there[l >> 5] >> (l & 31) & 1))
      zero_row(static_cast<O*>(a.out) + ((int64_t(l) << kFewShift) + c) * a.ldo, int(a.cols), lane,
               32);
}

template <class T, class O>
int launch_few(const FewArgs& f, cudaStream_t s) {
  const unsigned blocks = unsigned(std::min<int64_t>(f.sum.rows, int64_t(1) << kFewShift));
  if (whole_vectors<T, O>(f.sum))
    embedding_few_kernel<T, O, true><<<blocks, kFewThreads, 0, s>>>(f);
  else
    embedding_few_kernel<T, O, false><<<blocks, kFewThreads, 0, s>>>(f);
  IVFPQ_LAUNCHED();
  return IVFPQ_OK;
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
  const bool vec = whole_vectors<T, O>(a);
  IVFPQ_TRY(launch_after(vec ? embedding_sum_kernel<T, O, true> : embedding_sum_kernel<T, O, false>,
                         grid_of(runs, a.slabs + zero), dim3(unsigned(threads)), a, s));
  return launch_after(embedding_join_kernel<O>,
                      dim3(unsigned(ceil_div(a.cols, 4 * kJoinThreads)), unsigned(classes), 4),
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
  const bool wide = ids_bytes == 8;
  if (tokens <= kFew) {
    const FewArgs f{a, ids, wide, padding};
    return by_dtype(dtype, [&](auto* t) -> int {
      using T = std::remove_pointer_t<decltype(t)>;
      return out_dtype == dtype ? launch_few<T, T>(f, s) : launch_few<T, float>(f, s);
    });
  }
  SortArgs o{};
  o.ids = ids;
  o.tokens = tokens;
  o.rows = uint32_t(rows);
  o.padding = padding >= 0 && padding < rows ? uint32_t(padding) : kNone;
  // a block per SM or nearly, and more where a class would have too many tokens
  // (65536 x 904 bf16 into 100000 rows, with 32, 64, 128 and 256 classes: 106, 96, 92 and
  // 91 us; 16384 x 4096 into 32000: 82, 80, 82 and 88 us)
  o.shift = 7;
  while (ceil_div(rows, int64_t(1) << o.shift) > kMaxLocal) ++o.shift;
  o.local = int(ceil_div(rows, int64_t(1) << o.shift));
  // short slabs while they are few: a block takes its positions one after the other,
  // and long ones leave fewer partial sums. (16384 x 4096 bf16 into 32000 rows: 80, 82 and
  // 88 us with slabs four times as long, these, and a quarter; 65536 x 512: 65, 56, 66.)
  const int64_t runs = ceil_div(cols, 128 * (16 / dtype_size(dtype)));
  a.slab = 8;
  while (a.slab < kMaxSlab && tokens * runs > int64_t(a.slab) * 4096) a.slab *= 2;
  a.slabs = ceil_div(tokens, a.slab);
  a.pitch = ceil_div(cols, 8) * 8;
  Workspace ws(s);
  // the slabs' partial sums, the frequent tokens and the sorted positions
  const size_t parts = size_t(a.slabs) * 2 * size_t(a.pitch);
  const size_t frequent = size_t(tokens / (a.slab + 1) + 1), classes = size_t(1) << o.shift;
  const size_t words = size_t(tokens) * 4 + size_t(rows) + 1;
  int4* w = nullptr;
  IVFPQ_TRY(ws.alloc(&w, parts / 4 + frequent + (classes + 1) / 2 + (words + 3) / 4));
  a.part = reinterpret_cast<float*>(w);
  o.frequent = w + parts / 4;
  o.classes = reinterpret_cast<int2*>(o.frequent + frequent);
  o.list = o.classes + 2 * ((classes + 1) / 2);
  o.pos = reinterpret_cast<int32_t*>(o.list + tokens);
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
  // counters, and what else fits of positions, as they are met and by token
  const int64_t counters = (int64_t(o.local) * 2 + 2) / 2 * 8;
  o.listed = int(std::min<int64_t>({tokens, kMostListed, (216 * 1024 - counters) / 16}));
  const size_t smem = size_t(counters) + size_t(o.listed) * 16;
  // more threads where each has several steps of ids (1000 tokens: 6.3 us with 512
  // threads, 9.9 us with 1024)
  const bool many = tokens > 16384;
  auto sort = many ? (wide ? embedding_sort_kernel<true, 1024> : embedding_sort_kernel<false, 1024>)
                   : (wide ? embedding_sort_kernel<true, 512> : embedding_sort_kernel<false, 512>);
  IVFPQ_TRY(set_dynamic_smem(sort, smem));
  sort<<<1u << o.shift, many ? 1024 : 512, smem, s>>>(o);
  IVFPQ_LAUNCHED_K(sort, smem, many ? 1024 : 512);
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    return out_dtype == dtype ? launch_sums<T, T>(a, 1 << o.shift, s)
                              : launch_sums<T, float>(a, 1 << o.shift, s);
  });
}
