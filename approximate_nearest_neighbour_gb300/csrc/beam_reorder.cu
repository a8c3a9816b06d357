// beam_reorder: the states of a group's beams (caches, histories) into the order
// of the selected continuations,
//   dst[g * n + j, outer, p] = src[g * width + beams[g, j], outer, p],  p < lengths[g]
// where rows whose beam is outside [0, width) and positions past the length stay
// as they were.
//
// Bound by memory: each row is written once, and each source row that is taken is
// read once, whatever the number of its continuations, but in place, where it is
// read for each of them and rows that stay where they are are not touched. Up to 32
// states of a call go through one launch (a decoder has two per layer). A block takes
// a run of one segment for all rows of a group. Elsewhere than in place, the rows are
// visited in the order of their sources, and a thread loads its part when the source
// changes. In place, a thread first keeps its part of the source of every row that
// moves in shared memory, and then writes: its bytes are its own, so no barrier is
// needed.
//
// Measured: 16 x 4 rows of two states of 8 x 4096 x 128 bf16 and their histories, lengths
// from a quarter to all, not in place: 153 to 163 us; as many bytes at the copy rate take
// 163 us. 4 rows of four states of 8 x 200 x 128: 5.8 us on the device, the launch and one
// dependent chain (ids, lengths, rows). In place the large batch takes 272 us and its bytes
// 123: blocks of one vector per thread and row, each of which finds the order of the rows.
#include <algorithm>
#include <utility>

#include "common.cuh"

namespace ivfpq {
namespace {

constexpr int kThreads = 256;
constexpr int kInPlaceThreads = 128;
constexpr int kUnroll = 4;
constexpr int kMaxStates = 32;  // per launch: the kernel's parameters hold them

struct StateArg {
  const char* src;
  char* dst;
  int64_t src_row, dst_row, outer, src_outer, dst_outer, inner, unit;
  int64_t blocks;  // of this and the earlier states
  int granule;     // bytes that every address and length of this state is a multiple of
};
struct ReorderArgs {
  const int32_t* beams;
  const int32_t* lengths;
  int64_t groups, blocks;
  int width, n, count;
  int run;  // granules of a block's run, a multiple of its threads
  StateArg state[kMaxStates];
};

// The rows of a group in the order of their sources; returns how many have one.
__device__ int sources(const int32_t* beams, int width, int n, bool in_place, uint8_t* to,
                       uint8_t* from) {
  __shared__ int32_t b[IVFPQ_MAX_BEAMS];
  __shared__ int valid;
  __syncthreads();
  if (threadIdx.x == 0) valid = 0;
  auto takes = [&](int j) { return b[j] >= 0 && b[j] < width && !(in_place && b[j] == j); };
  if (threadIdx.x < n) b[threadIdx.x] = beams[threadIdx.x];
  __syncthreads();
  const int j = threadIdx.x;
  if (j < n && takes(j)) {
    int place = 0;
    for (int i = 0; i < n; ++i) place += takes(i) && (b[i] < b[j] || (b[i] == b[j] && i < j));
    to[place] = uint8_t(j);
    from[place] = uint8_t(b[j]);
    atomicAdd(&valid, 1);
  }
  __syncthreads();
  return valid;
}

template <class V, bool IN_PLACE>
__device__ __forceinline__ void move(const char* src, char* dst, int64_t src_row, int64_t dst_row,
                                     int64_t left, int valid, const uint8_t* to,
                                     const uint8_t* from, char* keep) {
  const int at = threadIdx.x, threads = blockDim.x;
  if constexpr (IN_PLACE) {
    // left: bytes of this block's run; one vector per thread
    if (int64_t(at + 1) * int(sizeof(V)) > left) return;
    V* k = reinterpret_cast<V*>(keep);
#pragma unroll 8
    for (int i = 0; i < valid; ++i)
      k[i * threads + at] = reinterpret_cast<const V*>(src + from[i] * src_row)[at];
#pragma unroll 8
    for (int i = 0; i < valid; ++i)
      reinterpret_cast<V*>(dst + to[i] * dst_row)[at] = k[i * threads + at];
  } else {
    V v[kUnroll];
    int cur = -1;
    const int have = int(min(left / int(sizeof(V)), int64_t(kUnroll) * threads));
    for (int i = 0; i < valid; ++i) {
      if (from[i] != cur) {
        cur = from[i];
        const V* p = reinterpret_cast<const V*>(src + cur * src_row);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (at + u * threads < have) v[u] = p[at + u * threads];
      }
      V* q = reinterpret_cast<V*>(dst + to[i] * dst_row);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (at + u * threads < have) q[at + u * threads] = v[u];
    }
  }
}

template <bool IN_PLACE>
__global__ void __launch_bounds__(IN_PLACE ? kInPlaceThreads : kThreads, 4)
    beam_reorder_kernel(const __grid_constant__ ReorderArgs a) {
  extern __shared__ __align__(16) char reorder_smem[];
  __shared__ uint8_t to[IVFPQ_MAX_BEAMS], from[IVFPQ_MAX_BEAMS];
  for (int64_t block = blockIdx.x; block < a.blocks; block += gridDim.x) {
    int i = 0;
    while (block >= a.state[i].blocks) ++i;
    const StateArg& s = a.state[i];
    const int64_t within = block - (i > 0 ? a.state[i - 1].blocks : 0);
    const int64_t run = int64_t(s.granule) * a.run;
    const int64_t runs = (s.inner + run - 1) / run;
    const int64_t g = within / (s.outer * runs), rest = within - g * (s.outer * runs);
    const int64_t o = rest / runs, at = (rest - o * runs) * run;
    int64_t bytes = s.inner;
    if (a.lengths && s.unit > 0) {
      // (the product may pass 63 bits: a length is any number, a position any size)
      const uint64_t n = uint64_t(max(a.lengths[g], 0)), unit = uint64_t(s.unit);
      if (__umul64hi(n, unit) == 0) bytes = int64_t(min(uint64_t(bytes), n * unit));
    }
    if (at >= bytes) continue;
    const int valid = sources(a.beams + g * a.n, a.width, a.n, IN_PLACE, to, from);
    const char* src = s.src + g * a.width * s.src_row + o * s.src_outer + at;
    char* dst = s.dst + g * a.n * s.dst_row + o * s.dst_outer + at;
    const int64_t left = min(bytes - at, run);
    switch (s.granule) {
      case 16:
        move<uint4, IN_PLACE>(src, dst, s.src_row, s.dst_row, left, valid, to, from, reorder_smem);
        break;
      case 4:
        move<uint32_t, IN_PLACE>(src, dst, s.src_row, s.dst_row, left, valid, to, from,
                                 reorder_smem);
        break;
      case 2:
        move<uint16_t, IN_PLACE>(src, dst, s.src_row, s.dst_row, left, valid, to, from,
                                 reorder_smem);
        break;
      default:
        move<uint8_t, IN_PLACE>(src, dst, s.src_row, s.dst_row, left, valid, to, from,
                                reorder_smem);
    }
  }
}

template <bool IN_PLACE>
int launch(ReorderArgs& a, cudaStream_t s) {
  if (a.count == 0) return IVFPQ_OK;
  const int threads = IN_PLACE ? kInPlaceThreads : kThreads;
  // (one vector per thread and source: 295 instead of 168 us for 16 x 4 rows of two states
  // of 8 x 4096 x 128 bf16, 6.2 instead of 6.4 us for 4 rows of four of 8 x 200 x 128)
  a.run = threads * (IN_PLACE ? 1 : kUnroll);
  a.blocks = 0;
  for (int i = 0; i < a.count; ++i) {
    StateArg& t = a.state[i];
    a.blocks += a.groups * t.outer * ceil_div(t.inner, int64_t(t.granule) * a.run);
    t.blocks = a.blocks;
  }
  const size_t smem = IN_PLACE ? size_t(a.n) * threads * 16 : 0;
  if (smem > 40 * 1024) IVFPQ_TRY(set_dynamic_smem(beam_reorder_kernel<IN_PLACE>, smem));
  const unsigned grid = unsigned(std::min<int64_t>(a.blocks, int64_t(1) << 30));
  beam_reorder_kernel<IN_PLACE><<<grid, threads, smem, s>>>(a);
  IVFPQ_LAUNCHED_K(beam_reorder_kernel<IN_PLACE>, smem, threads);
  a.count = 0;
  return IVFPQ_OK;
}

int granule_of(const ivfpq_state& t) {
  const uint64_t all = uint64_t(reinterpret_cast<uintptr_t>(t.src)) |
                       uint64_t(reinterpret_cast<uintptr_t>(t.dst)) | uint64_t(t.src_row) |
                       uint64_t(t.dst_row) | uint64_t(t.src_outer) | uint64_t(t.dst_outer) |
                       uint64_t(t.inner) | uint64_t(t.unit);
  return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
}

// Whether no two of rows * outer runs of `inner` bytes meet, `row` and `step` bytes from
// one to the next.
bool apart(int64_t rows, int64_t row, int64_t outer, int64_t step, int64_t inner) {
  if (outer > rows) {
    std::swap(rows, outer);
    std::swap(row, step);
  }
  if ((rows > 1 && row < inner) || (outer > 1 && step < inner)) return false;
  if (outer == 1) return true;
  // one within the other's gaps, as in every view of a dense tensor
  if ((row - inner) / step >= outer - 1 || (step - inner) / row >= rows - 1) return true;
  // run o of the first row lies `rest` behind the start of row q
  int64_t q = 0, rest = 0;
  for (int64_t o = 1; o < outer; ++o) {
    q += step / row;
    rest += step % row;
    if (rest >= row) {
      rest -= row;
      ++q;
    }
    if (q >= rows) break;
    if (rest < inner || (q + 1 < rows && row - rest < inner)) return false;
  }
  return true;
}

}  // namespace
}  // namespace ivfpq

using namespace ivfpq;

extern "C" int beam_reorder(const ivfpq_state* states, int count, const int32_t* beams,
                            int64_t groups, int width, int n, const int32_t* lengths,
                            void* stream) {
  clear_error();
  IVFPQ_REQUIRE(width >= 1 && width <= IVFPQ_MAX_BEAMS && n >= 1 && n <= IVFPQ_MAX_BEAMS,
                "beam_reorder: width=%d or n=%d outside [1, %d]", width, n, IVFPQ_MAX_BEAMS);
  IVFPQ_REQUIRE(groups >= 0 && groups < (int64_t(1) << 31) / IVFPQ_MAX_BEAMS,
                "beam_reorder: groups=%lld outside [0, 2^31 / %d)", (long long)groups,
                IVFPQ_MAX_BEAMS);
  IVFPQ_REQUIRE(count >= 0, "beam_reorder: count=%d", count);
  if (groups == 0 || count == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(states && beams, "beam_reorder: null pointer");
  for (int i = 0; i < count; ++i) {
    const ivfpq_state& t = states[i];
    IVFPQ_REQUIRE(t.outer >= 0 && t.inner >= 0 && t.unit >= 0 && t.src_row >= 0 &&
                      t.dst_row >= 0 && t.src_outer >= 0 && t.dst_outer >= 0,
                  "beam_reorder: a negative size or stride of state %d", i);
    IVFPQ_REQUIRE(t.outer < (int64_t(1) << 31) && t.inner < (int64_t(1) << 40),
                  "beam_reorder: state %d is too large", i);
    if (t.outer == 0 || t.inner == 0) continue;
    IVFPQ_REQUIRE(t.src && t.dst, "beam_reorder: null pointer in state %d", i);
    IVFPQ_REQUIRE(t.dst_row < (int64_t(1) << 56) && t.dst_outer < (int64_t(1) << 56),
                  "beam_reorder: state %d is too large", i);
    IVFPQ_REQUIRE(apart(groups * n, t.dst_row, t.outer, t.dst_outer, t.inner),
                  "beam_reorder: state %d's written rows or segments overlap", i);
    IVFPQ_REQUIRE(t.src != t.dst || (width == n && t.src_row == t.dst_row &&
                                     (t.outer == 1 || t.src_outer == t.dst_outer)),
                  "beam_reorder: state %d in place takes as many rows as there are, of one layout",
                  i);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ReorderArgs a[2];
  for (ReorderArgs& x : a) {
    x.beams = beams;
    x.lengths = lengths;
    x.groups = groups;
    x.width = width;
    x.n = n;
    x.count = 0;
  }
  for (int i = 0; i < count; ++i) {
    const ivfpq_state& t = states[i];
    if (t.outer == 0 || t.inner == 0) continue;
    const bool in_place = t.src == t.dst;
    ReorderArgs& x = a[in_place];
    StateArg& y = x.state[x.count];
    y = {static_cast<const char*>(t.src), static_cast<char*>(t.dst), t.src_row, t.dst_row, t.outer,
         t.src_outer, t.dst_outer, t.inner, t.unit, 0, granule_of(t)};
    if (++x.count == kMaxStates)
      IVFPQ_TRY(in_place ? launch<true>(x, s) : launch<false>(x, s));
  }
  IVFPQ_TRY(launch<false>(a[0], s));
  return launch<true>(a[1], s);
}
