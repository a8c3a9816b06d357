// score_adjust: the changes a score row gets between the product that made it
// and the k-selection that reads it. For row r and column c
//   x = score[r, c]
//   c in the row's history:            x = x > 0 ? x / repetition : x * repetition
//   n = occurrences past the prompt:   x -= n * frequency + (n > 0) * presence
//   c in the row's bias list:          x += bias
//   x /= temperature;  not allowed by the mask: x = -inf;  negated if asked
//
// Bound by memory: each score is read and written once. A block takes a run
// of columns of one row, counts the history's tokens that fall into it in
// shared memory (integer atomics: the result does not depend on their order)
// and then streams the run once. Bit 31 of a counter marks a token of the
// prompt, the bits below count occurrences past it.
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"

namespace ivfpq {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 4096;  // columns per block

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
};

template <class T, class O>
__global__ void __launch_bounds__(kThreads) score_adjust_kernel(const AdjustArgs a) {
  __shared__ uint32_t count[kRun];
  __shared__ uint32_t slot[kRun];  // 1 + the last bias entry for the column
  const int64_t row = blockIdx.x;
  const int64_t c0 = int64_t(blockIdx.y) * kRun;
  const int len = int(min(int64_t(kRun), a.cols - c0));
  const bool has_hist = a.history != nullptr, has_bias = a.bias_ids != nullptr;
  if (has_hist || has_bias) {
    for (int i = threadIdx.x; i < len; i += kThreads) {
      count[i] = 0;
      slot[i] = 0;
    }
    __syncthreads();
    if (has_hist) {
      const int64_t n = max(int64_t(0), min(a.history_len ? int64_t(a.history_len[row]) : a.hist_cols,
                                            a.hist_cols));
      const int64_t np = a.prompt_len ? int64_t(a.prompt_len[row]) : 0;
      const int32_t* h = a.history + row * a.ldh;
      for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const int64_t c = int64_t(h[i]) - c0;
        if (c >= 0 && c < len) {
          if (i < np)
            atomicOr(&count[c], 0x80000000u);
          else
            atomicAdd(&count[c], 1u);
        }
      }
    }
    if (has_bias) {
      const int32_t* b = a.bias_ids + row * a.nb;
      for (int64_t i = threadIdx.x; i < a.nb; i += kThreads) {
        const int64_t c = int64_t(b[i]) - c0;
        if (c >= 0 && c < len) atomicMax(&slot[c], uint32_t(i) + 1u);
      }
    }
    __syncthreads();
  }
  const float rep = a.repetition ? a.repetition[row] : 1.f;
  const float pres = a.presence ? a.presence[row] : 0.f;
  const float freq = a.frequency ? a.frequency[row] : 0.f;
  const float temp = a.temperature ? a.temperature[row] : 1.f;
  const T* src = static_cast<const T*>(a.scores) + row * a.lds + c0;
  O* dst = static_cast<O*>(a.out) + row * a.ldo + c0;
  const int32_t* mask = a.mask ? a.mask + row * a.ldm : nullptr;
  for (int i = threadIdx.x; i < len; i += kThreads) {
    float x = to_f32(src[i]);
    if (has_hist && count[i] != 0) {
      const uint32_t n = count[i] & 0x7fffffffu;
      x = x > 0.f ? x / rep : x * rep;
      if (n) x -= float(n) * freq + pres;
    }
    if (has_bias && slot[i] != 0) x += a.bias_vals[row * a.nb + slot[i] - 1];
    x /= temp;
    if (mask && !((uint32_t(mask[(c0 + i) >> 5]) >> ((c0 + i) & 31)) & 1u)) x = -INFINITY;
    dst[i] = from_f32<O>(x * a.sign);
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
  IVFPQ_REQUIRE(cols >= 0 && cols <= (int64_t(1) << 28), "score_adjust: cols=%lld outside [0, 2^28]",
                (long long)cols);
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
               prompt_len, repetition, presence, frequency, nb ? bias_ids : nullptr, bias_vals, nb,
               temperature, mask, ldm, negate ? -1.f : 1.f, out, ldo};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_dtype(dtype, [&](auto* t) -> int {
    using T = std::remove_pointer_t<decltype(t)>;
    const dim3 grid(unsigned(rows), unsigned(ceil_div(cols, kRun)));
    if (out_dtype == dtype)
      score_adjust_kernel<T, T><<<grid, kThreads, 0, s>>>(a);
    else
      score_adjust_kernel<T, float><<<grid, kThreads, 0, s>>>(a);
    IVFPQ_LAUNCHED();
    return IVFPQ_OK;
  });
}
