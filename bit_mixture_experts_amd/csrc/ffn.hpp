// Pieces shared by the forward and backward kernels of the dense gated feed-forward block.
#pragma once

#include "dense_gemm.hpp"
#include "internal.hpp"
#include "mx.hpp"

namespace moe4 {

// Row of the [2I, H] gate/up stack that row r of a tile of gate/up pairs takes: the tile's
// 32-row MFMA tiles alternate between 32 gate rows and the up rows of the same pairs, so that
// a lane holds both halves of a pair at the same place of neighbouring accumulators.
__device__ __forceinline__ int pair_row(int layout, int I, int j0, int r) {
  const int j = j0 + (r >> 6) * 32 + (r & 31);
  if (j >= I) return -1;
  const bool up = (r >> 5) & 1;
  return layout == MOE4_GU_HALVES ? (up ? I + j : j) : 2 * j + (up ? 1 : 0);
}

// The activation and its gradients. Comparisons, not fmin/fmax, so that a NaN stays one.
struct FfnAct {
  int act;
  float alpha, limit;
  __device__ __forceinline__ float apply(float g, float u) const {
    if (act == MOE4_ACT_SWIGLU) return g * sigmoidf_(g) * u;
    const float gc = g > limit ? limit : g;
    const float uc = u > limit ? limit : u < -limit ? -limit : u;
    return (uc + 1.0f) * gc * sigmoidf_(alpha * gc);
  }
  // h, and dg, du for an upstream gradient dh; beyond a clamp's border the gradient is zero,
  // on the border it passes
  __device__ __forceinline__ void backward(float g, float u, float dh, float& h, float& dg,
                                           float& du) const {
    if (act == MOE4_ACT_SWIGLU) {
      const float s = sigmoidf_(g), gs = g * s;
      h = gs * u;
      du = dh * gs;
      dg = dh * u * (s + gs * (1.0f - s));
    } else {
      const float gc = g > limit ? limit : g;
      const float uc = u > limit ? limit : u < -limit ? -limit : u;
      const float s = sigmoidf_(alpha * gc), gs = gc * s, lin = uc + 1.0f;
      h = lin * gs;
      dg = g > limit ? 0.0f : dh * lin * (s + alpha * gs * (1.0f - s));
      du = u > limit || u < -limit ? 0.0f : dh * gs;
    }
  }
};

__device__ __forceinline__ void load8_bf16(const uint16_t* p, float* v) {
  const u32x4 x = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo(x[i]);
    v[2 * i + 1] = bf16hi(x[i]);
  }
}
__device__ __forceinline__ void load8_f32(const float* p, float* v) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ u32x4 pack8_bf16(const float* v) {
  u32x4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  return x;
}
__device__ __forceinline__ void store8_f32(float* p, const float* v) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
// 8 values of a tensor that is bf16 or fp32 (a uniform branch)
__device__ __forceinline__ void load8_dt(const void* p, int dtype, int64_t i, float* v) {
  if (dtype == MOE4_DTYPE_F32) load8_f32(static_cast<const float*>(p) + i, v);
  else load8_bf16(static_cast<const uint16_t*>(p) + i, v);
}
__device__ __forceinline__ void store8_dt(void* p, int dtype, int64_t i, const float* v) {
  if (dtype == MOE4_DTYPE_F32) store8_f32(static_cast<float*>(p) + i, v);
  else *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = pack8_bf16(v);
}

// 8 values as they lie in memory (bf16: the first half)
struct Raw16 {
  u32x4 v[2];
};

// One product of the block and what its epilogue does: out[b][a] = sum_k A B (+ bias[a]) (+
// add[b][a]), a < na, b < nb.
struct FfnProduct {
  Operand A, B;
  int64_t na_s, nb_s;   // bytes of the operands' scales (MXFP8)
  int K, na, nb;
  const uint16_t* bias;
  const void* add;
  int add_dtype;
  void* out;
  int out_dtype;
  int splits;           // parts of k; 1: the tile's epilogue finishes the output
  float* part;          // [splits][nb][na] sums to be joined
};

// The tile's end: its sums go to the part's place, or are finished and stored.
template <typename S>
__device__ __forceinline__ void ffn_product_end(const FfnProduct& p, const f32x16 (&acc)[S::TA][S::TB],
                                                int a0, int b0, int split, uint8_t* lds) {
  if constexpr (S::kSplits) {
    if (p.splits > 1) {
      float* part = p.part + (int64_t)split * p.nb * p.na;
      for_each8<S, false, 1>(acc, lds, [](int, int) { return NoPre{}; },
                             [&](int row, int a, float* v, const NoPre&) {
        const int b = b0 + row, c = a0 + a;
        if (b < p.nb && c < p.na) store8_f32(part + (int64_t)b * p.na + c, v);
      });
      return;
    }
  }
  const bool add32 = p.add_dtype == MOE4_DTYPE_F32;
  float bias[8] = {};   // the same columns in every turn
  if (const int c = a0 + lane_a<S, false>(); p.bias && c < p.na) load8_bf16(p.bias + c, bias);
  for_each8<S, false, 8>(
      acc, lds,
      [&](int row, int a) {
        Raw16 r;
        const int b = b0 + row, c = a0 + a;
        if (p.add && b < p.nb && c < p.na) {
          const int64_t at = (int64_t)b * p.na + c;
          if (add32) {
            const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const float*>(p.add) + at);
            r.v[0] = q[0];
            r.v[1] = q[1];
          } else {
            r.v[0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.add) + at);
          }
        }
        return r;
      },
      [&](int row, int a, float* v, const Raw16& r) {
        const int b = b0 + row, c = a0 + a;
        if (b >= p.nb || c >= p.na) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += bias[i];
        if (p.add) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] += add32 ? __uint_as_float(r.v[i / 4][i % 4])
                          : (i & 1 ? bf16hi(r.v[0][i / 2]) : bf16lo(r.v[0][i / 2]));
        }
        store8_dt(p.out, p.out_dtype, (int64_t)b * p.na + c, v);
      });
}

template <typename S, int MA, int MB, bool FP8>
__device__ __forceinline__ void ffn_product_tile(const FfnProduct& p, int ia, int ib, int split,
                                                 uint8_t* lds) {
  const int a0 = ia * S::BA, b0 = ib * S::BB;
  OpLoader<S, MA, S::BA, FP8> la;
  OpLoader<S, MB, S::BB, FP8> lb;
  constexpr int es = FP8 ? 1 : 2;
  const KPart k(p.K, es, split, S::kSplits ? p.splits : 1);
  if constexpr (MA == kOpRow) {
    const int n = min(S::BA, p.na - a0);
    la.init_row(p.A.from_row(k.kt0), es, k.K, a0, n, [=](int r) { return r < n ? r : -1; });
  } else {
    la.init_col(p.A.from_col(k.kt0), k.K, a0);
  }
  if constexpr (MB == kOpRow) {
    const int n = min(S::BB, p.nb - b0);
    lb.init_row(p.B.from_row(k.kt0), es, k.K, b0, n, [=](int r) { return r < n ? r : -1; });
  } else {
    lb.init_col(p.B.from_col(k.kt0), k.K, b0);
  }
  const MxScales mx = {p.A.s, p.B.s, p.na_s, p.nb_s, p.K / 32, k.kt0 * 4};
  f32x16 acc[S::TA][S::TB];
  gemm_loop<S, MA, MB, FP8>(
      acc, lds, la, lb, k.K, mx, [&](int r) { return a0 + r < p.na ? a0 + r : -1; },
      [&](int r) { return b0 + r < p.nb ? b0 + r : -1; });
  ffn_product_end<S>(p, acc, a0, b0, split, lds);
}

template <typename S, int MA, int MB, bool FP8>
__global__ __launch_bounds__(S::kThreads, 2) void k_ffn_product(const FfnProduct p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t stage_mem[];
  const int na = (p.na + S::BA - 1) / S::BA, nb = (p.nb + S::BB - 1) / S::BB;
  int ia, ib;
  const int id = xcd_remap(blockIdx.x, gridDim.x), tile = id % (na * nb);
  tile_of(tile, na, nb, ia, ib);
  ffn_product_tile<S, MA, MB, FP8>(p, ia, ib, id / (na * nb), stage_mem);
}

// f(layout, activation) as compile-time constants
template <typename F>
inline hipError_t with_kind(int layout, int act, F f) {
  using H = std::integral_constant<int, MOE4_GU_HALVES>;
  using N = std::integral_constant<int, MOE4_GU_INTERLEAVED>;
  using S = std::integral_constant<int, MOE4_ACT_SWIGLU>;
  using C = std::integral_constant<int, MOE4_ACT_SWIGLU_CLAMPED>;
  if (layout == MOE4_GU_HALVES) return act == MOE4_ACT_SWIGLU ? f(H{}, S{}) : f(H{}, C{});
  return act == MOE4_ACT_SWIGLU ? f(N{}, S{}) : f(N{}, C{});
}

// Which tiles, by rounds of the chip: a round is 256 tiles of 256 x 256 or 512 of 128 x 128,
// and one of the small tiles takes two thirds of one of the large (half the work, at three
// quarters of the rate: each LDS operand feeds half as many MFMAs). Few tokens or a ragged last
// round go to the small ones. Us of a forward, large and small tiles throughout (few tokens cut
// along k): bf16 1024 tokens at 2880, 2880 92 and 74, 2048 121 and 118 (each product by the rule
// 109), 8192 363 and 402; 4096 at 2048, 768 67 and 53, 8192 81 and 96; 1024 at 4096, 8192 194 and
// 221, 4096 640 and 808. MXFP8 1024 at 2880, 2880 72 and 65, 2048 87 and 91 (by the rule 80),
// 4096 135 and 165; 4096 at 2048, 768 44 and 39, 8192 56 and 65; 1024 at 4096, 8192 134 and 166,
// 2048 230 and 303 (by the rule 248: the one size tried where it loses).
template <typename S>
inline int64_t tiles_of(int64_t na, int64_t nb) {
  return ((na + S::BA - 1) / S::BA) * ((nb + S::BB - 1) / S::BB);
}
inline bool large_tiles(int64_t n256, int64_t n128) {
  return 3 * ((n256 + 255) / 256) <= 2 * ((n128 + 511) / 512);
}
inline bool large_tiles_for(int64_t na, int64_t nb) {
  return large_tiles(tiles_of<Tile256>(na, nb), tiles_of<Tile128>(na, nb));
}

// Parts of k for n tiles of 128 x 128 that leave most of a round (512) empty: as many as fill it,
// each with at least eight k-tiles of 128 bytes (in bf16 a part's own first loads, the launch that
// joins and its reads cost about as much as eight). Us of a forward, whole and in parts, bf16: 64
// tokens at H 4096, I 8192 126 and 55, at 2880, 2880 60 and 32; 128 at 2880, 2880 65 and 36, at 2048,
// 768 29 and 25; 512 147 and 115, 66 and 58, 37 and 33; 1024 at 2048, 768 38 and 36, 2048 39 and 42.
// MXFP8, whose k-tiles multiply in half the time while the join costs the same: 64 61 and 40, 35 and
// 29; 128 at 2880, 2880 41 and 34; but 512 95 and 92, 44 and 50, 21 and 24, and 2048 at 2048, 768
// 25 and 34: parts are too short there.
constexpr int kMostSplits = 16;
inline int k_splits(int64_t n128, int K, int es) {
  const int nk = (int)(((int64_t)K * es + 127) / 128);
  const int64_t most = 512 / n128, long_enough = nk / 8;
  const int64_t s = most < long_enough ? most : long_enough;
  return s < 2 ? 1 : (int)(s < kMostSplits ? s : kMostSplits);
}

// Bytes that the parts of a product [nb, na] cut into at most `splits` take, for this nb or any
// smaller one: parts x tiles are at most 512, and a tile holds 64 KiB. Workspaces are sized by
// this, not by the call's own parts, which become fewer as nb grows: a buffer made for the most
// tokens serves any fewer.
constexpr int64_t kMostPartBytes = 512 * 128 * 128 * 4;
inline int64_t part_bytes(int64_t na, int64_t nb, int64_t splits) {
  const int64_t b = splits < 2 ? 0 : splits * na * nb * 4;
  return b < kMostPartBytes ? b : kMostPartBytes;
}
// the most parts that k_splits makes of a product with na columns and a reduction of K
inline int64_t most_k_splits(int64_t na, int K, int es) {
  if ((na + 127) / 128 > 256) return 1;
  const int64_t s = ((int64_t)K * es + 127) / 128 / 8;
  return s < kMostSplits ? s : kMostSplits;
}

// The sums of split products (those of up to three, one after another), with what their tiles'
// epilogue would have added: 8 values of a row to a thread.
struct JoinArgs {
  FfnProduct p[3];
  int first[4];   // first workgroup of each, and the end
};
hipError_t launch_join(JoinArgs a, int n, hipStream_t s);

template <typename S, int MA, int MB, bool FP8>
inline hipError_t launch_product(const FfnProduct& p, hipStream_t s) {
  const int64_t n = tiles_of<S>(p.na, p.nb) * p.splits;
  auto* k = &k_ffn_product<S, MA, MB, FP8>;
  constexpr int kBytes = FP8 ? S::kLdsMx : S::kLds;
  hipError_t e = allow_lds<kBytes>(k);
  if (e != hipSuccess) return e;
  k<<<(uint32_t)n, S::kThreads, kBytes, s>>>(p);
  return hipGetLastError();
}

}  // namespace moe4
