// score_adjust: the changes a score row gets between the product that made it
// and the k-selection that reads it. For row r and column c
//   x = score[r, c]
//   c in the row's history:            x = x > 0 ? x / repetition : x * repetition
//   n = occurrences past the prompt:   x -= n * frequency + (n > 0) * presence
//   c in the row's bias list:          x += bias
//   x /= temperature;  not allowed by the mask: x = -inf;  negated if asked
//
// Bound by memory: each score is read and written once. (To skip what the mask
// rules out, the scores would have to wait for the mask: a microsecond more
// with a quarter of the columns allowed.) A block takes a run of columns of one
// row:
//  1. its first mask words, tokens and scores are loaded, and wait in registers;
//  2. the history's occurrences in the run are counted in shared memory and the
//     bias entries noted (integer atomics: the result does not depend on their
//     order), and a bitmap marks their columns;
//  3. the run is streamed in 16-byte vectors; only marked columns look at the
//     tables.
// Every block of a row reads the whole history, so runs are as long as leaves
// enough blocks (run_for). Measured at 256 x 131072 bf16: 22 us with the
// temperature alone (its bytes take 20 us), 29 us with a mask, 33 us with 64
// biases too, 45 us with histories of up to 4,096 tokens besides; what is above
// the bytes is instructions (2.4 per clock and SM) and the steps before the
// stream, not memory. Runs of 4,096 and 16,384 columns and blocks of 128 and
// 512 threads measured 46 to 59 us.
#include <algorithm>

#include "internal.h"
#include "rowvec.cuh"

namespace ivfpq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRun = 8192;  // columns per block
constexpr int kMinRun = 1024;

// A run's table: per column the occurrences past the prompt, whether the prompt
// has it, and 1 + the last bias entry for it. SHORT packs them into one word
// (bits 0..14, bit 15, bits 16..31), so that five blocks share an SM instead of
// three; it holds histories of up to 32,767 tokens and 65,535 bias entries.
// The long form has the counter with bit 31 for the prompt, and a second word.
constexpr int kShortHistory = 32767, kShortBias = 65535;

struct AdjustArgs {
  const void* scores;
  int64_t rows, cols, lds;
  const int32_t* history;
  int64_t hist_cols, ldh;
  const int32_t* history_len;
  const int32_t* prompt_len;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_ids;
  const float* bias_vals;
  int64_t nb;
  const float* temperature;
  const int32_t* mask;
  int64_t ldm;  // 0: one mask for all rows
  float sign;
  void* out;
  int64_t ldo;
  int run;
};

// Bits b .. b + N - 1 of a bit string of words, as far as word `last`, in the
// low bits. The second word is read only where they reach into it.
template <int N, class W>
__device__ __forceinline__ uint32_t bits_at(const W* words, int b, int last) {
  const int w = b >> 5, sh = b & 31;
  uint32_t r = uint32_t(words[w]) >> sh;
  if (sh > 32 - N && w < last) r |= uint32_t(words[w + 1]) << (32 - sh);
  return r & ((1u << N) - 1);
}

template <class T, class O, bool HIST, bool BIAS, bool MASK, bool SHORT>
__global__ void __launch_bounds__(kThreads, 5) score_adjust_kernel(const AdjustArgs a) {
  extern __shared__ __align__(16) uint32_t adjust_smem[];
  constexpr bool MARK = HIST || BIAS;
  uint32_t* mark = adjust_smem;  // a bit per column of the run
  uint32_t* count = mark + a.run / 32;
  uint32_t* slot = count + (SHORT ? 0 : a.run);
  constexpr uint32_t kPrompt = SHORT ? 0x8000u : 0x80000000u;
  const int64_t row = blockIdx.x;
  const int64_t c0 = int64_t(blockIdx.y) * a.run;
  const int len = int(min(int64_t(a.run), a.cols - c0));
  const int words = (len + 31) / 32;
  const T* src = static_cast<const T*>(a.scores) + row * a.lds + c0;
  O* dst = static_cast<O*>(a.out) + row * a.ldo + c0;
  const int32_t* mask = MASK ? a.mask + row * a.ldm + (c0 >> 5) : nullptr;
  // vectors of N scores that start on a 16-byte boundary of the output
  constexpr int N = Span<T>::N, U = 4;
  const int head = min(len, int((16 - misalign(dst)) & 15) / int(sizeof(O)));
  const int nvec = (len - head) / N;
  const int mis = misalign(src + head);
  uint4 r[U];
  uint32_t ok[U];
  const int first = inner_first(mis), last = inner_last<T>(len - head, mis);
  auto load_mask = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      ok[u] = (1u << N) - 1;
      if (MASK && i < nvec) ok[u] = bits_at<N>(mask, head + i * N, words - 1);
    }
  };
  auto load_scores = [&](int i0) {
    if (i0 >= first && i0 + (U - 1) * kThreads <= last) {
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = load_inner(src + head, i0 + u * kThreads, mis);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * kThreads < nvec)
          r[u] = load_vec(src + head, len - head, i0 + u * kThreads, mis);
    }
  };
  load_mask(threadIdx.x);
  load_scores(threadIdx.x);
  if constexpr (MARK) {
    const int32_t* h = HIST && a.history ? a.history + row * a.ldh : nullptr;
    const int32_t* bi = BIAS && a.bias_ids ? a.bias_ids + row * a.nb : nullptr;
    // counters are unsigned: one step past a list of up to 2^31 - 1 does not wrap
    const uint32_t hcols = h ? uint32_t(a.hist_cols) : 0;
    // the first tokens are on their way before their number is known
    constexpr int V = 8;
    int32_t t[V];
    auto load_tokens = [&](uint32_t i0, uint32_t end) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        t[v] = i0 + v * kThreads < end ? __ldg(h + i0 + v * kThreads) : -1;
    };
    if (HIST) load_tokens(threadIdx.x, hcols);
    uint32_t n = hcols, np = 0;
    if (HIST && h) {
      if (a.history_len) n = min(n, uint32_t(max(0, a.history_len[row])));
      if (a.prompt_len) np = uint32_t(max(0, a.prompt_len[row]));
    }
    const int clear = a.run / 32 + a.run * (SHORT ? 1 : 2);  // a multiple of 4 words
    for (int i = threadIdx.x; i < clear / 4; i += kThreads)
      reinterpret_cast<uint4*>(mark)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (HIST) {
      for (uint32_t i0 = threadIdx.x; i0 < n; i0 += V * kThreads) {
        if (i0 != threadIdx.x) load_tokens(i0, n);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          // out of the run (or of the row, or negative): past len
          const uint32_t c = uint32_t(t[v]) - uint32_t(c0);
          const uint32_t i = i0 + v * kThreads;
          if (c < uint32_t(len) && i < n) {
            atomicOr(&mark[c >> 5], 1u << (c & 31));
            if (i < np)
              atomicOr(&count[c], kPrompt);
            else
              atomicAdd(&count[c], 1u);
          }
        }
      }
    }
    if (BIAS) {
      if (HIST && SHORT) __syncthreads();  // the counters are complete
      for (uint32_t i = threadIdx.x; i < uint32_t(a.nb); i += kThreads) {
        const int64_t c = int64_t(__ldg(bi + i)) - c0;
        if (c >= 0 && c < len) {
          atomicOr(&mark[c >> 5], 1u << (c & 31));
          if (SHORT) {
            uint32_t old = slot[c];
            while ((old >> 16) < i + 1u) {
              const uint32_t seen =
                  atomicCAS(&slot[c], old, (old & 0xffffu) | ((i + 1u) << 16));
              if (seen == old) break;
              old = seen;
            }
          } else {
            atomicMax(&slot[c], i + 1u);
          }
        }
      }
    }
    __syncthreads();
  }
  const float rep = HIST && a.repetition ? a.repetition[row] : 1.f;
  const float pres = HIST && a.presence ? a.presence[row] : 0.f;
  const float freq = HIST && a.frequency ? a.frequency[row] : 0.f;
  // the division by the temperature and the sign, as one factor per row
  const float t = a.temperature ? a.temperature[row] : 1.f;
  const float f = __fdiv_rn(a.sign, t);
  const float masked = -INFINITY * a.sign;
  auto marked = [&](int c, float x) {
    const uint32_t e = count[c];
    const uint32_t seen = SHORT ? e & 0xffffu : e;
    if (HIST && seen != 0) {
      const uint32_t n = seen & (kPrompt - 1u);
      x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
      if (n) x -= float(n) * freq + pres;
    }
    if (BIAS) {
      const uint32_t b = SHORT ? e >> 16 : slot[c];
      if (b != 0) x += a.bias_vals[row * a.nb + b - 1];
    }
    return x;
  };
  auto one = [&](int c, bool divide) {
    float x = to_f32(src[c]);
    if (MARK && (mark[c >> 5] >> (c & 31)) & 1u) x = marked(c, x);
    x = divide ? __fdiv_rn(x, t) * a.sign : x * f;
    if (MASK && !((uint32_t(mask[c >> 5]) >> (c & 31)) & 1u)) x = masked;
    dst[c] = from_f32<O>(x);
  };
  if (t != 0.f && fabsf(t) < 0x1p-126f) {
    // a subnormal temperature, whose reciprocal may pass fp32: score by score
    for (int c = threadIdx.x; c < len; c += kThreads) one(c, true);
    return;
  }
  for (int e = threadIdx.x; e < len - nvec * N; e += kThreads)
    one(e < head ? e : nvec * N + e, false);
  for (int i0 = threadIdx.x; i0 < nvec; i0 += U * kThreads) {
    if (i0 != int(threadIdx.x)) {
      load_mask(i0);
      load_scores(i0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= nvec) continue;
      float v[N];
      unpack_vec<T>(r[u], v);
#pragma unroll
      for (int j = 0; j < N; j += 2) unpair(mul2(pair(v[j], v[j + 1]), pair(f, f)), v[j], v[j + 1]);
      if constexpr (MASK) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = (ok[u] >> j) & 1u ? v[j] : masked;
      }
      store_vec<O>(dst + head + i * N, v);
      if constexpr (MARK) {
        // the few marked columns again, one by one, from the loaded scores
        uint32_t m = bits_at<N>(mark, head + i * N, words - 1) & ok[u];
        while (m) {
          const int j = __ffs(m) - 1, c = head + i * N + j;
          m &= m - 1;
          dst[c] = from_f32<O>(marked(c, vec_element<T>(r[u], j)) * f);
        }
      }
    }
  }
}

// Runs of kMaxRun columns, halved while the blocks do not fill the device
// three times.
int run_for(int64_t rows, int64_t cols) {
  int run = kMaxRun;
  while (run > kMinRun && rows * ceil_div(cols, run) < 3 * num_sms()) run /= 2;
  return run;
}

template <class T, class O, bool HIST, bool BIAS, bool MASK, bool SHORT>
int launch(AdjustArgs a, cudaStream_t s) {
  a.run = run_for(a.rows, a.cols);
  const size_t smem =
      HIST || BIAS ? size_t(a.run) / 8 + size_t(a.run) * 4 * (SHORT ? 1 : 2) : 0;
  auto kern = score_adjust_kernel<T, O, HIST, BIAS, MASK, SHORT>;
  IVFPQ_TRY(set_dynamic_smem(kern, smem));
  const dim3 grid(unsigned(a.rows), unsigned(ceil_div(a.cols, a.run)));
  kern<<<grid, kThreads, smem, s>>>(a);
  IVFPQ_LAUNCHED_K(kern, smem, kThreads);
  return IVFPQ_OK;
}
template <class T, class O>
int launch_types(const AdjustArgs& a, cudaStream_t s) {
  const int which = (a.history ? 4 : 0) | (a.bias_ids ? 2 : 0) | (a.mask ? 1 : 0);
  if ((a.history && a.hist_cols > kShortHistory) || (a.bias_ids && a.nb > kShortBias))
    return a.mask ? launch<T, O, true, true, true, false>(a, s)
                  : launch<T, O, true, true, false, false>(a, s);
  switch (which) {
    case 0: return launch<T, O, false, false, false, true>(a, s);
    case 1: return launch<T, O, false, false, true, true>(a, s);
    case 2: return launch<T, O, false, true, false, true>(a, s);
    case 3: return launch<T, O, false, true, true, true>(a, s);
    case 4: return launch<T, O, true, false, false, true>(a, s);
    case 5: return launch<T, O, true, false, true, true>(a, s);
    case 6: return launch<T, O, true, true, false, true>(a, s);
    default: return launch<T, O, true, true, true, true>(a, s);
  }
}

}  // namespace
}  // namespace ivfpq

using namespace ivfpq;

extern "C" int score_adjust(const void* scores, int dtype, int64_t rows, int64_t cols, int64_t lds,
                            const int32_t* history, int64_t hist_cols, int64_t ldh,
                            const int32_t* history_len, const int32_t* prompt_len,
                            const float* repetition, const float* presence, const float* frequency,
                            const int32_t* bias_ids, const float* bias_vals, int64_t nb,
                            const float* temperature, const int32_t* mask, int64_t ldm, int negate,
                            void* out, int out_dtype, int64_t ldo, void* stream) {
  clear_error();
  IVFPQ_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), "score_adjust: rows=%lld outside [0, 2^31)",
                (long long)rows);
  IVFPQ_REQUIRE(cols >= 0 && cols <= (int64_t(1) << 28),
                "score_adjust: cols=%lld outside [0, 2^28]", (long long)cols);
  IVFPQ_REQUIRE(known_dtype(dtype) && known_dtype(out_dtype), "score_adjust: unknown element type");
  IVFPQ_REQUIRE(out_dtype == dtype || out_dtype == IVFPQ_F32,
                "score_adjust: the output is of the scores' type or fp32");
  IVFPQ_REQUIRE(rows <= 1 || ((lds >= cols || lds == 0) && ldo >= cols),
                "score_adjust: row strides %lld, %lld below cols=%lld", (long long)lds,
                (long long)ldo, (long long)cols);
  IVFPQ_REQUIRE(hist_cols >= 0 && hist_cols < (int64_t(1) << 31) && nb >= 0 &&
                    nb < (int64_t(1) << 31),
                "score_adjust: bad history or bias length");
  if (rows == 0 || cols == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(scores && out, "score_adjust: null pointer");
  IVFPQ_REQUIRE(history || !(history_len || prompt_len),
                "score_adjust: history lengths without a history");
  IVFPQ_REQUIRE((bias_ids == nullptr) == (bias_vals == nullptr),
                "score_adjust: bias ids and values go together");
  AdjustArgs a{scores, rows, cols, lds, hist_cols ? history : nullptr, hist_cols, ldh, history_len,
               prompt_len, repetition, presence, frequency, nb ? bias_ids : nullptr, bias_vals,
               bias_ids ? nb : 0, temperature, mask, ldm, negate ? -1.f : 1.f, out, ldo, 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    return out_dtype == dtype ? launch_types<T, T>(a, s) : launch_types<T, float>(a, s);
  });
}
