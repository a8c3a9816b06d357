// adapter_linear: low-rank adapters of many requests, added to the result of a
// projection that they share,
//   out[t] = base[t] + scale_i (x[t] A_i^T) B_i^T,   i = ids[t]
// with A_i [rank, cols] and B_i [n, rank]; a token without an adapter (an id
// outside the list) gets its base row.
//
// Bound by memory: of 2 tokens rank (cols + n) operations per tokens (cols + 2 n)
// elements moved, even rank 64 is 40 operations per byte, a fifth of what the
// tensor cores need to be the limit. So both products run on warp-level matrix
// instructions whose operands come straight from memory into registers: the sum
// over K may run in any order if both operands take the same one, so that each
// lane loads 16 consecutive bytes of a row and uses them as its part of two
// instructions, and the columns of a result tile may be any 8, so that a lane's
// results of four tiles are 8 neighbouring columns.
//  1. Tokens are grouped by adapter into tiles: by every block for itself up to 256
//     tokens (tiles of 16), by a kernel of one block above (tiles of 128). Order
//     within a tile does not matter: a token's sums do not depend on its neighbours.
//  2. h = x A^T: a block takes a tile and a part of K, its warps parts of that; the
//     warps' parts are added in shared memory, then the blocks', which are a
//     cluster, in fixed order.
//  3. out = base + scale h B^T: a block keeps the tile's h in shared memory and runs
//     over columns. h is fp32: it is cut into two terms of the operands' type
//     (three, if bf16 operands make an fp32 output), each exact to the next, so
//     that nothing of it is rounded away beyond 2^-17 (2^-22 for fp16, 2^-25 for three).
// Many tokens go through kernels of their own (adapter_wide.cu), but for the second
// product where an adapter's rows of B are not multiples of 16 bytes.
//
// Measured: 77 tokens of 64 adapters, rank 16, 4096 x 16384 bf16 (35 MB): 7.9 us for h and
// 13.4 us for the output with cold caches, which overlap to 21.4 to 23.1 us as a program
// calls it; 5.3 us are the bytes. Each block of the second product waits for the kernel that
// makes h, then for its tile and B, h and its base rows, and a wave is all there is. (B and the
// base rows could be on their way before h is there; the tile that names them is not.) One token,
// 4096 x 16384: 5.9 and 4.3 us, two starts of a kernel.
#include <algorithm>

#include "adapter.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace ivfpq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kPlanThreads = 1024;

// ---- tokens by adapter ------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) adapter_plan_kernel(const AdapterArgs a) {
  extern __shared__ int plan_smem[];
  int* slot = plan_smem;            // [adapters + 1]: counts, then the next slot
  __shared__ int sh[2][32];
  const int bins = a.adapters + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_go();
  for (int i = threadIdx.x; i < bins; i += kPlanThreads) slot[i] = 0;
  __syncthreads();
  // one addition per adapter and warp: prompts bring thousands of tokens of one
  auto take = [&](int id) {
    const unsigned same = __match_any_sync(kFullMask, id);
    int at = 0;
    if (id >= 0 && lane == __ffs(same) - 1) at = atomicAdd(&slot[id], __popc(same));
    at = __shfl_sync(kFullMask, at, __ffs(same) - 1);
    return at + __popc(same & ((1u << lane) - 1u));
  };
  constexpr int kIds = 8;  // per thread and step
  constexpr int64_t step = int64_t(kPlanThreads) * kIds;
  int v[kIds];
  auto read = [&](int64_t t0) {
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      const int64_t t = t0 + j * kPlanThreads + threadIdx.x;
      v[j] = t < a.tokens ? a.ids[t] : -1;
      if (t < a.tokens && (v[j] < 0 || v[j] >= a.adapters)) v[j] = a.adapters;
    }
  };
  for (int64_t t0 = 0; t0 < a.tokens; t0 += step) {
    read(t0);
#pragma unroll
    for (int j = 0; j < kIds; ++j)
      if (t0 + j * kPlanThreads < a.tokens) take(v[j]);
  }
  __syncthreads();
  // running sums of the counts and of the tiles
  int slots = 0, tiles = 0;
  for (int i0 = 0; i0 < bins; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int c = i < bins ? slot[i] : 0, t = (c + a.tile - 1) / a.tile;
    int ic = c, it = t;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int u = __shfl_up_sync(kFullMask, ic, d), v = __shfl_up_sync(kFullMask, it, d);
      if (lane >= d) {
        ic += u;
        it += v;
      }
    }
    __syncthreads();
    if (lane == 31) {
      sh[0][warp] = ic;
      sh[1][warp] = it;
    }
    __syncthreads();
    const int wc = sh[0][lane], wt = sh[1][lane];
    const int bc = int(__reduce_add_sync(kFullMask, unsigned(lane < warp ? wc : 0)));
    const int bt = int(__reduce_add_sync(kFullMask, unsigned(lane < warp ? wt : 0)));
    const int first = slots + bc + ic - c, ftile = tiles + bt + it - t;
    if (i < bins) {
      slot[i] = first;
      for (int k = 0; k < t; ++k)
        a.tiles[ftile + k] = make_int4(i < a.adapters ? i : -1, first + k * a.tile,
                                       min(a.tile, c - k * a.tile), 0);
    }
    slots += int(__reduce_add_sync(kFullMask, unsigned(wc)));
    tiles += int(__reduce_add_sync(kFullMask, unsigned(wt)));
  }
  if (threadIdx.x == 0) *a.ntiles = tiles;
  __syncthreads();
  for (int64_t t0 = 0; t0 < a.tokens; t0 += step) {
    if (a.tokens > step) read(t0);
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      if (t0 + j * kPlanThreads >= a.tokens) break;
      const int at = take(v[j]);
      if (v[j] >= 0) a.order[at] = int32_t(t0 + j * kPlanThreads + threadIdx.x);
    }
  }
}

// ---- matrix instructions ----------------------------------------------------------------
// D += A B for 16 x 16 and 16 x 8 operands of 16-bit type.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1, __nv_bfloat16*) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1, __half*) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---- h = x A^T ----------------------------------------------------------------------------
constexpr int kFew = 256;  // tokens up to which every block finds its tile itself
constexpr int kFewTile = 16;
struct FewPlan {
  int4 bin[kFew / 4];         // tokens' adapters, `adapters` for none
  unsigned heads[kFew / 32];  // tokens that begin a tile
  int token[kFewTile];
  int first, rank, count;
};
// Tile `index` of the tokens: tiles are numbered by their first tokens, a token begins
// one if the number of earlier tokens of its adapter is a multiple of kFewTile.
__device__ __forceinline__ Tile few_tile(const AdapterArgs& a, int index, FewPlan& p) {
  const int tokens = int(a.tokens), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* bin = reinterpret_cast<int*>(p.bin);
  constexpr int J = kFew / kThreads;
  int mine[J], before[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int t = j * kThreads + threadIdx.x;
    mine[j] = t < tokens ? a.ids[t] : -2;
    if (t < tokens && (mine[j] < 0 || mine[j] >= a.adapters)) mine[j] = a.adapters;
    if (t >= tokens) mine[j] = -2;
    bin[t] = mine[j];
    before[j] = 0;
  }
  if (threadIdx.x == 0) {
    p.first = -1;
    p.count = 0;
  }
  __syncthreads();
  for (int i = 0; i < (tokens + 3) / 4; ++i) {
    const int4 v = p.bin[i];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int t = j * kThreads + threadIdx.x - 4 * i;
      before[j] += (v.x == mine[j] && t > 0) + (v.y == mine[j] && t > 1) +
                   (v.z == mine[j] && t > 2) + (v.w == mine[j] && t > 3);
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const unsigned h =
        __ballot_sync(kFullMask, mine[j] != -2 && before[j] % kFewTile == 0);
    if (lane == 0) p.heads[j * kWarps + warp] = h;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int w = j * kWarps + warp;
    if (p.heads[w] >> lane & 1) {
      int at = __popc(p.heads[w] & ((1u << lane) - 1u));
      for (int i = 0; i < w; ++i) at += __popc(p.heads[i]);
      if (at == index) {
        p.first = mine[j];
        p.rank = before[j];
      }
    }
  }
  __syncthreads();
  const int of = p.first;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int at = before[j] - p.rank;
    if (of >= 0 && mine[j] == of && at >= 0 && at < kFewTile) {
      p.token[at] = j * kThreads + threadIdx.x;
      atomicAdd(&p.count, 1);
    }
  }
  __syncthreads();
  return {of >= 0 && of < a.adapters ? of : -1, index * kFewTile, p.count};
}

template <class T, int NT>
__global__ void __launch_bounds__(kThreads) adapter_shrink_kernel(const AdapterArgs a) {
  constexpr int R = NT * 8;
  __shared__ __align__(16) float part[kWarps][16 * R];
  __shared__ FewPlan plan;
  T* const type = nullptr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3, r = lane >> 2;
  grid_go();
  const int index = int(blockIdx.y + int64_t(blockIdx.z) * gridDim.y);
  const Tile t = few_tile(a, index, plan);
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.tiles[index] = make_int4(t.adapter, t.first, t.count, 0);
    if (threadIdx.x < t.count) a.order[t.first + threadIdx.x] = plan.token[threadIdx.x];
  }
  if (t.count == 0 || t.adapter < 0) return;  // a cluster's blocks alike
  const T* x[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    x[e] = e * 8 + r < t.count
               ? static_cast<const T*>(a.x) + int64_t(plan.token[e * 8 + r]) * a.ldx
               : nullptr;
  const T* w = static_cast<const T*>(a.a) + (int64_t(t.adapter) * a.rank + r) * a.cols;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  const int64_t k0 = int64_t(blockIdx.x) * a.kpart, k1 = min(a.cols, k0 + a.kpart);
  constexpr int U = NT <= 4 ? 4 : NT <= 8 ? 2 : 1;
  for (int64_t k = k0 + warp * 32; k < k1; k += kWarps * 32 * U) {
    uint4 xv[U][2], wv[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = k + u * kWarps * 32 + 8 * q;
      const int64_t len = k + u * kWarps * 32 < k1 ? a.cols : 0;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        wv[u][j] = row8(j * 8 + r < a.rank ? w + int64_t(j * 8) * a.cols : nullptr, len, at);
#pragma unroll
      for (int e = 0; e < 2; ++e) xv[u][e] = row8(x[e], len, at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4 &p = xv[u][0], &s = xv[u][1], &v = wv[u][j];
        mma16(acc[j], p.x, s.x, p.y, s.y, v.x, v.y, type);
        mma16(acc[j], p.z, s.z, p.w, s.w, v.z, v.w, type);
      }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      *reinterpret_cast<float2*>(&part[warp][(e * 8 + r) * R + j * 8 + 2 * q]) =
          make_float2(acc[j][2 * e], acc[j][2 * e + 1]);
  __syncthreads();
  // the warps' parts into the first warp's place
  for (int i = threadIdx.x; i < t.count * R; i += kThreads) {
    float s = part[0][i];
#pragma unroll
    for (int v = 1; v < kWarps; ++v) s += part[v][i];
    part[0][i] = s;
  }
  join_parts<R, kThreads>(a, part[0], t.count, t.first);
}

// ---- out = base + scale h B^T ----------------------------------------------------------------
// A lane's part of a row of B: 4 KS consecutive elements from 4 KS q on, as two
// registers per instruction.
template <class T, int KS>
__device__ __forceinline__ void load_b(const T* p, int rank, int q, bool whole,
                                       uint32_t (&b)[KS][2]) {
#pragma unroll
  for (int s = 0; s < KS; ++s) b[s][0] = b[s][1] = 0;
  if (p == nullptr) return;
  const int k = 4 * KS * q;
  if (whole) {
    if constexpr (KS == 1) {
      if (k < rank) {
        const uint2 v = *reinterpret_cast<const uint2*>(p + k);
        b[0][0] = v.x;
        b[0][1] = v.y;
      }
    } else {
#pragma unroll
      for (int s = 0; s < KS; s += 2) {
        if (k + 4 * s < rank) {
          const uint4 v = *reinterpret_cast<const uint4*>(p + k + 4 * s);
          b[s][0] = v.x;
          b[s][1] = v.y;
          b[s + 1][0] = v.z;
          b[s + 1][1] = v.w;
        }
      }
    }
  } else {
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        T t[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int i = k + 4 * s + 2 * e + f;
          t[f] = i < rank ? p[i] : from_f32<T>(0.f);
        }
        memcpy(&b[s][e], t, 4);
      }
  }
}

// VEC: base and output rows lie on 16-byte boundaries and are whole vectors.
// ONE: tiles have at most 16 tokens.
template <class T, class O, int KS, int TERMS, bool VEC, bool ONE>
__global__ void __launch_bounds__(kThreads) adapter_expand_kernel(const AdapterArgs a) {
  extern __shared__ __align__(16) uint4 expand_smem[];  // [m tiles, KS, TERMS, 32]
  __shared__ float up[kMaxTile];                        // a row's power of two
  __shared__ int64_t token[kMaxTile];
  __shared__ float turned[VEC ? 1 : kWarps][VEC ? 1 : 16 * 33];
  T* const type = nullptr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3, r = lane >> 2;
  grid_wait();
  const Tile t = tile_at(a, blockIdx.y + int64_t(blockIdx.z) * gridDim.y);
  if (t.count == 0) return;
  const bool some = t.adapter >= 0;
  const O* base = static_cast<const O*>(a.base);
  O* out = static_cast<O*>(a.out);
  if (!some && base == out) return;  // in place: nothing changes
  // B's first columns are asked for before h is, both after the wait for the kernel that
  // makes h and the tiles
  const bool whole = a.rank % (KS == 1 ? 4 : 8) == 0 && misalign(a.b) == 0;
  const T* b0 = some ? static_cast<const T*>(a.b) + int64_t(t.adapter) * a.n * a.rank : nullptr;
  const int64_t cend = min(a.n, (int64_t(blockIdx.x) + 1) * a.run);
  const int64_t c0 = int64_t(blockIdx.x) * a.run + warp * 32;
  auto fetch_b = [&](int64_t at, uint32_t (&b)[4][KS][2]) {
    if (!some) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = at + 8 * (r / 2) + 2 * j + (r & 1);
      load_b<T, KS>(c < cend ? b0 + c * a.rank : nullptr, a.rank, q, whole, b[j]);
    }
  };
  uint32_t bq[4][KS][2];
  constexpr bool AHEAD = KS <= 2;  // the next columns' B as well, where it takes few registers
  uint32_t bn[4][AHEAD ? KS : 1][2];
  if constexpr (AHEAD) fetch_b(c0, bq);
  for (int i = threadIdx.x; i < t.count; i += kThreads) token[i] = token_of(a, t.first + i);
  const int mtiles = ONE ? 1 : (t.count + 15) / 16;
  if (some) {
    const float scale = a.scales ? a.scales[t.adapter] : 1.f;
    for (int m = warp; m < mtiles; m += kWarps) {
      float v[2][4 * KS];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = m * 16 + e * 8 + r;
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 4 * KS; ++k) v[e][k] = 0.f;
        if (i < t.count) {
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const int k = 4 * KS * q + 4 * s;
            if (k >= a.pitch) continue;
            const float4 f =
                *reinterpret_cast<const float4*>(a.h + int64_t(t.first + i) * a.pitch + k);
            v[e][4 * s] = within_rank(a, k, f.x);
            v[e][4 * s + 1] = within_rank(a, k + 1, f.y);
            v[e][4 * s + 2] = within_rank(a, k + 2, f.z);
            v[e][4 * s + 3] = within_rank(a, k + 3, f.w);
          }
        }
#pragma unroll
        for (int k = 0; k < 4 * KS; ++k) {
          v[e][k] *= scale;
          top = fmaxf(top, magnitude(v[e][k]));
        }
        if constexpr (std::is_same<T, __half>::value) {
          // fp16's range: the row's largest value to [2^14, 2^15)
          top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
          top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
          const float2 f = fp16_range(top);
#pragma unroll
          for (int k = 0; k < 4 * KS; ++k) v[e][k] *= f.x;
          if (q == 0 && i < t.count) up[i] = f.y;
        }
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int n = 0; n < TERMS; ++n) {
          float f[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < 4; ++k) f[e][k] = term<T>(v[e][4 * s + k]);
          expand_smem[((m * KS + s) * TERMS + n) * 32 + lane] =
              make_uint4(pack16(f[0][0], f[0][1], type), pack16(f[1][0], f[1][1], type),
                         pack16(f[0][2], f[0][3], type), pack16(f[1][2], f[1][3], type));
        }
    }
  }
  __syncthreads();
  if (c0 >= cend) return;
  const int items = int((cend - c0 + kWarps * 32 - 1) / (kWarps * 32)) * mtiles;
  // the base rows of the coming items, on their way
  constexpr int W = int(sizeof(O)) / 2;
  constexpr int D = VEC ? 2 : 1;
  uint4 raw[D][2][W];
  int fm = 0;
  int64_t fc = c0;  // the next item to fetch
  auto fetch = [&](uint4 (&v)[2][W]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = fm * 16 + e * 8 + r;
#pragma unroll
      for (int g = 0; g < W; ++g) {
        v[e][g] = make_uint4(0, 0, 0, 0);
        if (VEC && base && i < t.count && fc + 8 * q < cend)
          v[e][g] = reinterpret_cast<const uint4*>(base + token[i] * a.ldb + fc + 8 * q)[g];
      }
    }
    if (++fm == mtiles) {
      fm = 0;
      fc += kWarps * 32;
    }
  };
  if constexpr (!AHEAD) fetch_b(c0, bq);
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(raw[d]);
  int m = 0;
  int64_t c = c0;
  for (int it0 = 0; it0 < items; it0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (it0 + d >= items) break;
      if constexpr (AHEAD) {
        if (m == 0 && c + kWarps * 32 < cend) fetch_b(c + kWarps * 32, bn);
      }
      float acc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
      if (some) {
#pragma unroll
        for (int n = TERMS - 1; n >= 0; --n)  // the small terms first
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const uint4 f = expand_smem[((m * KS + s) * TERMS + n) * 32 + lane];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma16(acc[j], f.x, f.y, f.z, f.w, bq[j][s][0], bq[j][s][1], type);
          }
        if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = m * 16 + e * 8 + r;
            const float f = i < t.count ? up[i] : 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[j][2 * e] *= f;
              acc[j][2 * e + 1] *= f;
            }
          }
        }
      }
      if constexpr (VEC) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = m * 16 + e * 8 + r;
          float y[8];
          constexpr int M = Span<O>::N;
#pragma unroll
          for (int g = 0; g < W; ++g) {
            float w[M];
            unpack_vec<O>(raw[d][e][g], w);
#pragma unroll
            for (int j = 0; j < M; ++j) y[g * M + j] = w[j];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[2 * j] += acc[j][2 * e];
            y[2 * j + 1] += acc[j][2 * e + 1];
          }
          if (i < t.count && c + 8 * q < cend) store_vec<O>(out + token[i] * a.ldo + c + 8 * q, y);
        }
        fetch(raw[d]);
      } else {
        // rows at any offset: through shared memory, a column per lane
        float* mine = turned[warp];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mine[(e * 8 + r) * 33 + 8 * q + 2 * j] = acc[j][2 * e];
            mine[(e * 8 + r) * 33 + 8 * q + 2 * j + 1] = acc[j][2 * e + 1];
          }
        __syncwarp();
        const bool in = c + lane < cend;
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          y[i] = base && in && m * 16 + i < t.count
                     ? to_f32(base[token[m * 16 + i] * a.ldb + c + lane])
                     : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (in && m * 16 + i < t.count)
            out[token[m * 16 + i] * a.ldo + c + lane] = from_f32<O>(y[i] + mine[i * 33 + lane]);
      }
      if (++m == mtiles) {
        m = 0;
        c += kWarps * 32;
        if constexpr (AHEAD) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              bq[j][s][0] = bn[j][s][0];
              bq[j][s][1] = bn[j][s][1];
            }
        } else if (c < cend) {
          fetch_b(c, bq);
        }
      }
    }
  }
}

// ---- host side ---------------------------------------------------------------------------------
dim3 grid_of(int64_t per_row, int64_t rows) {
  const int64_t y = std::min<int64_t>(rows, 65535);
  return dim3(unsigned(per_row), unsigned(y), unsigned(ceil_div(rows, y)));
}
template <class K>
int launch(K kern, dim3 grid, int threads, size_t smem, const AdapterArgs& a, bool overlap,
           int cluster, cudaStream_t s) {
  // 48 KB with the static part need no leave
  if (smem > 32 * 1024) IVFPQ_TRY(set_dynamic_smem(kern, smem));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = unsigned(cluster);
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  if (overlap) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = unsigned(n);
  IVFPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
  IVFPQ_LAUNCHED_K(kern, smem, threads);
  return IVFPQ_OK;
}

template <class T, int NT>
int launch_shrink(const AdapterArgs& a, int64_t tiles, cudaStream_t s) {
  return launch(adapter_shrink_kernel<T, NT>, grid_of(a.splits, tiles), kThreads, 0, a, false,
                a.splits, s);
}
template <class T>
int launch_shrink_rank(const AdapterArgs& a, int64_t tiles, cudaStream_t s) {
  switch (a.pitch / 8) {
    case 1: return launch_shrink<T, 1>(a, tiles, s);
    case 2: return launch_shrink<T, 2>(a, tiles, s);
    case 4: return launch_shrink<T, 4>(a, tiles, s);
    case 8: return launch_shrink<T, 8>(a, tiles, s);
    default: return launch_shrink<T, 16>(a, tiles, s);
  }
}
template <class T, class O, int KS>
int launch_expand(const AdapterArgs& a, int64_t tiles, cudaStream_t s) {
  constexpr int TERMS =
      std::is_same<T, __nv_bfloat16>::value && std::is_same<O, float>::value ? 3 : 2;
  const size_t smem = size_t((a.tile + 15) / 16) * KS * TERMS * 512;
  const dim3 grid = grid_of(ceil_div(a.n, a.run), tiles);
  const bool vec = whole_rows<O>(a);
  auto kern = a.tile > 16 ? (vec ? adapter_expand_kernel<T, O, KS, TERMS, true, false>
                                 : adapter_expand_kernel<T, O, KS, TERMS, false, false>)
                          : (vec ? adapter_expand_kernel<T, O, KS, TERMS, true, true>
                                 : adapter_expand_kernel<T, O, KS, TERMS, false, true>);
  return launch(kern, grid, kThreads, smem, a, true, 1, s);
}
template <class T, class O>
int launch_expand_rank(const AdapterArgs& a, int64_t tiles, cudaStream_t s) {
  switch (a.pitch / 8) {
    case 1:
    case 2: return launch_expand<T, O, 1>(a, tiles, s);
    case 4: return launch_expand<T, O, 2>(a, tiles, s);
    case 8: return launch_expand<T, O, 4>(a, tiles, s);
    default: return launch_expand<T, O, 8>(a, tiles, s);
  }
}
template <class T>
int launch_types(const AdapterArgs& a, int out_dtype, int64_t tiles, cudaStream_t s) {
  const int dtype = std::is_same<T, __half>::value ? IVFPQ_F16 : IVFPQ_BF16;
  if (a.tile == kMaxTile)
    IVFPQ_TRY(adapter_shrink_wide(a, dtype, tiles, s));
  else
    IVFPQ_TRY(launch_shrink_rank<T>(a, tiles, s));
  if (a.tile == kMaxTile && a.adapters > 0 && a.rank % 8 == 0 &&
      reinterpret_cast<uintptr_t>(a.b) % 16 == 0)
    return adapter_expand_wide(a, dtype, out_dtype, s);
  return out_dtype == IVFPQ_F32 ? launch_expand_rank<T, float>(a, tiles, s)
                                : launch_expand_rank<T, T>(a, tiles, s);
}

}  // namespace
}  // namespace ivfpq

using namespace ivfpq;

extern "C" int adapter_linear(const void* x, int dtype, int64_t tokens, int64_t cols, int64_t ldx,
                              const void* a, const void* b, int adapters, int rank, int64_t n,
                              const int32_t* ids, const float* scales, const void* base,
                              int64_t ldb, void* out, int out_dtype, int64_t ldo, void* stream) {
  clear_error();
  IVFPQ_REQUIRE(dtype == IVFPQ_F16 || dtype == IVFPQ_BF16,
                "adapter_linear: x and the adapters are fp16 or bf16");
  IVFPQ_REQUIRE(out_dtype == dtype || out_dtype == IVFPQ_F32,
                "adapter_linear: the output is of x's type or fp32");
  IVFPQ_REQUIRE(tokens >= 0 && tokens < (int64_t(1) << 24),
                "adapter_linear: tokens=%lld outside [0, 2^24)", (long long)tokens);
  IVFPQ_REQUIRE(cols >= 1 && cols <= (int64_t(1) << 20) && n >= 0 && n <= (int64_t(1) << 24),
                "adapter_linear: cols=%lld outside [1, 2^20] or n=%lld outside [0, 2^24]",
                (long long)cols, (long long)n);
  IVFPQ_REQUIRE(rank >= 1 && rank <= IVFPQ_MAX_RANK, "adapter_linear: rank=%d outside [1, %d]",
                rank, IVFPQ_MAX_RANK);
  IVFPQ_REQUIRE(adapters >= 0 && adapters <= IVFPQ_MAX_ADAPTERS,
                "adapter_linear: adapters=%d outside [0, %d]", adapters, IVFPQ_MAX_ADAPTERS);
  IVFPQ_REQUIRE(tokens <= 1 || ((ldx >= cols || ldx == 0) && ldo >= n &&
                                (!base || ldb >= n || ldb == 0)),
                "adapter_linear: a row stride below its row");
  if (tokens == 0 || n == 0) return IVFPQ_OK;
  IVFPQ_REQUIRE(x && ids && out && ((a && b) || adapters == 0), "adapter_linear: null pointer");
  IVFPQ_REQUIRE(base != out || tokens <= 1 || ldb == ldo,
                "adapter_linear: in place, base and out have one row stride");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AdapterArgs p{};
  p.x = x;
  p.tokens = tokens;
  p.cols = cols;
  p.ldx = ldx;
  p.a = a;
  p.b = b;
  p.adapters = adapters;
  p.rank = rank;
  p.n = n;
  p.ids = ids;
  p.scales = scales;
  p.base = base;
  p.ldb = ldb;
  p.out = out;
  p.ldo = ldo;
  p.pitch = 8;
  while (p.pitch < rank) p.pitch *= 2;
  // tiles of 128 tokens also where few adapters of a high rank have many each: a tile of
  // 16 reads its adapter's B again (256 tokens of one adapter, 4096 x 16384: rank 128 44 us
  // in tiles of 16 and 29 us in tiles of 128, rank 16 21.5 us, and 26 us for 257 tokens)
  const bool wide =
      tokens > kFew || (rank > 32 && tokens >= 64 && tokens >= 32 * int64_t(adapters));
  p.tile = wide ? kMaxTile : kFewTile;
  const int64_t tiles =
      tokens / p.tile + std::min<int64_t>(tokens, int64_t(adapters) + 1);  // at most
  // parts of K until there are blocks for every SM, of some steps each
  const int64_t items = wide ? 2 * ceil_div(tokens, kMaxTile) : ceil_div(tiles, 2);
  const int64_t least = wide ? 256 : 128;
  p.splits = 1;
  while (p.splits < 8 && items * p.splits < num_sms() && cols > least * p.splits) p.splits *= 2;
  p.kpart = int(ceil_div(ceil_div(cols, p.splits), 64) * 64);
  // runs of columns, long where there are many tiles (77 tokens of 64 adapters, rank 16,
  // 4096 x 16384: 21 us at this length, 23 to 25 us at twice and half of it)
  p.run = 128;
  while (p.run < 2048 && ceil_div(n, p.run) * tiles > 16 * num_sms()) p.run *= 2;
  // the sums, and behind them the tiles
  const int64_t slots = wide ? tokens : tiles * kFewTile;
  const size_t h = size_t(slots) * size_t(p.pitch) / 4;
  Workspace ws(s);
  float4* w = nullptr;
  IVFPQ_TRY(ws.alloc(&w, h + size_t(tiles) + size_t(ceil_div(slots + 1, 4))));
  p.h = reinterpret_cast<float*>(w);
  p.tiles = reinterpret_cast<int4*>(w + h);
  p.order = reinterpret_cast<int32_t*>(p.tiles + tiles);
  if (wide) {
    p.ntiles = p.order + slots;
    IVFPQ_TRY(launch(adapter_plan_kernel, dim3(1), kPlanThreads, size_t(adapters + 1) * 4, p, false,
                     1, s));
  }
  return dtype == IVFPQ_F16 ? launch_types<__half>(p, out_dtype, tiles, s)
                            : launch_types<__nv_bfloat16>(p, out_dtype, tiles, s);
}
