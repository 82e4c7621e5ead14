// Rows of activations in registers, shared by the kernels that norm them: 8 columns of a row to a
// chunk, sums over the waves of a row.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "internal.hpp"

namespace moe4 {

// 8 elements of a row in registers as they lie in memory: bf16 (16 bytes) or fp32 (32 bytes)
template <int DT>
struct Raw8 {
  u32x4 r[DT == MOE4_DTYPE_F32 ? 2 : 1];
  // column c of a row whose resource is rs; zeros past its end
  __device__ __forceinline__ void load(rsrc_t rs, int c) {
    if constexpr (DT == MOE4_DTYPE_F32) {
      r[0] = buf_load_b128(rs, 4 * c);
      r[1] = buf_load_b128(rs, 4 * c + 16);
    } else {
      r[0] = buf_load_b128(rs, 2 * c);
    }
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE4_DTYPE_F32) {
        v[i] = __uint_as_float(r[0][i]);
        v[4 + i] = __uint_as_float(r[1][i]);
      } else {
        v[2 * i] = bf16lo(r[0][i]);
        v[2 * i + 1] = bf16hi(r[0][i]);
      }
    }
  }
  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE4_DTYPE_F32) {
        r[0][i] = __float_as_uint(v[i]);
        r[1][i] = __float_as_uint(v[4 + i]);
      } else {
        r[0][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      }
    }
  }
  // stores past the row's end are dropped
  __device__ __forceinline__ void store(rsrc_t rs, int c) const {
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    if constexpr (DT == MOE4_DTYPE_F32) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, r[0]), rs, 4 * c, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, r[1]), rs, 4 * c + 16, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, r[0]), rs, 2 * c, 0, 0);
    }
  }
};

template <int DT>
__device__ __forceinline__ rsrc_t row_rsrc(const void* p, int64_t row, int H) {
  constexpr int es = DT == MOE4_DTYPE_F32 ? 4 : 2;
  return make_rsrc_uniform(static_cast<const uint8_t*>(p) + row * H * es, (uint32_t)H * es);
}

// fp32 sum over the wave, in every lane: DPP and permlane steps, no LDS round trip
__device__ __forceinline__ float wave_sum_f32(float x) {
  auto dpp = [](float v, auto ctl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctl)::value,
                                                      0xF, 0xF, false));
  };
  x += dpp(x, std::integral_constant<int, 0xB1>{});    // quad_perm [1,0,3,2]
  x += dpp(x, std::integral_constant<int, 0x4E>{});    // quad_perm [2,3,0,1]
  x += dpp(x, std::integral_constant<int, 0x141>{});   // row_half_mirror
  x += dpp(x, std::integral_constant<int, 0x140>{});   // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// sum over the W waves of a row, in every lane; slot alternates between calls so that one
// barrier a call is enough
template <int W>
__device__ __forceinline__ float row_sum(float x, float (&red)[2][W], int slot) {
  x = wave_sum_f32(x);
  if constexpr (W == 1) return x;
  if (lane_id() == 0) red[slot][wave_id()] = x;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) s += red[slot][i];
  return s;
}

// W waves of a row; W == 1 puts four rows into a workgroup
template <int W>
constexpr int kNormThreads = W == 1 ? 256 : 64 * W;


// Waves of a row: each lane holds at most 32 columns (the registers of the operands of one
// row, at four waves a SIMD), and a row of few goes over four waves. Us in bf16, forward /
// backward with dweight, at 1, 2, 4 and 16 waves:
//   1 x 2048      2.9 / 6.2   2.8 / 5.1   2.4 / 4.5   3.2 / 5.6
//   512 x 2048    3.8 / 8.2   3.9 / 8.2   3.2 / 7.6   5.5 / 8.9
//   512 x 512     2.6 / 5.8   3.5 / 6.3   2.9 / 5.7   5.2 / 7.9
//   2047 x 1024   4.1 / 7.9   5.2 / 11.1  4.9 / 9.9   13 / 18    (one wave would do from here on)
//   8192 x 1024   11.5 / 17   13.8 / 22   12.4 / 18   43 / 60
//   8192 x 2880               29.6 / 34   29.6 / 35   46 / 62
//   1 x 8192                              3.3 / 6.0   3.4 / 5.8
//   8192 x 8192                           97 / 112    96 / 109
constexpr int64_t kManyRows = 2048;
inline int norm_waves(int64_t T, int H) {
  if (H > 8192) return 16;
  if (H > 4096 || (T < kManyRows && H > 512)) return 4;
  return H > 2048 ? 2 : 1;
}

// f(waves, chunks) for the smallest instance that holds H columns
template <typename F>
inline hipError_t pick_shape(int64_t T, int H, F f) {
  const int W = norm_waves(T, H), nv = (H + 512 * W - 1) / (512 * W);
#define MOE4_NORM(w, n) return f(std::integral_constant<int, w>{}, std::integral_constant<int, n>{})
  if (W == 1) {
    if (nv <= 1) MOE4_NORM(1, 1);
    if (nv <= 2) MOE4_NORM(1, 2);
    MOE4_NORM(1, 4);
  }
  if (W == 2) {
    if (nv <= 3) MOE4_NORM(2, 3);
    MOE4_NORM(2, 4);
  }
  if (W == 4) {
    if (nv <= 1) MOE4_NORM(4, 1);
    if (nv <= 2) MOE4_NORM(4, 2);
    MOE4_NORM(4, 4);
  }
  MOE4_NORM(16, 2);
#undef MOE4_NORM
}

}  // namespace moe4
