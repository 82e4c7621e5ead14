// Top-k selection of one token by one wave, shared by the kernels that route.
#pragma once

#include "common.hpp"

namespace moe4 {

// Selection order: larger logit first, then lower expert index; +0 == -0.
// order_key maps a logit's bits to an unsigned order (negative values have all
// bits flipped, the others get the sign bit set; -0 is taken as +0). NaN maps to
// the lowest value (0; the next one up is -infinity's 0x7FFFFF), so the k
// chosen experts are always distinct and in range.
__device__ __forceinline__ uint32_t order_key(float v) {
  uint32_t u = __float_as_uint(v);
  if (u == 0x80000000u) u = 0u;
  uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  if (v != v) o = 0u;
  return o;
}
// The logit a key was made from (-0 comes back as +0, and below -infinity's key are NaNs).
__device__ __forceinline__ float key_logit(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
// Each candidate becomes one 64-bit key that is unique and ordered the same
// way: its logit's, then the inverted expert index. Key 0 marks a lane slot
// with no candidate (past E, or already chosen).
__device__ __forceinline__ uint64_t select_key(float v, int e) {
  return ((uint64_t)order_key(v) << 32) | (uint32_t)~(uint32_t)e;
}

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// DPP move of a 64-bit value inside each row of 16 lanes (CTRL as in
// v_mov_b32_dpp: quad_perm, row_half_mirror, row_mirror).
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t x) {
  const int lo = __builtin_amdgcn_update_dpp((int)(uint32_t)x, (int)(uint32_t)x, CTRL, 0xF, 0xF,
                                             false);
  const int hi = __builtin_amdgcn_update_dpp((int)(uint32_t)(x >> 32), (int)(uint32_t)(x >> 32),
                                             CTRL, 0xF, 0xF, false);
  return ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo;
}

// Maximum over the wave, returned in every lane (the whole wave active):
// lanes xor 1 and 2 by quad permutes, xor 4 and 8 by the half-row and row
// mirrors, then rows pairwise by v_permlane16_swap and halves by
// v_permlane32_swap; no LDS round trip.
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t x) {
  x = max_u64(x, dpp_u64<0xB1>(x));   // quad_perm [1,0,3,2]
  x = max_u64(x, dpp_u64<0x4E>(x));   // quad_perm [2,3,0,1]
  x = max_u64(x, dpp_u64<0x141>(x));  // row_half_mirror
  x = max_u64(x, dpp_u64<0x140>(x));  // row_mirror
  {
    const uint32_t lo = (uint32_t)x, hi = (uint32_t)(x >> 32);
    const auto a = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    x = max_u64(((uint64_t)b[0] << 32) | a[0], ((uint64_t)b[1] << 32) | a[1]);
  }
  {
    const uint32_t lo = (uint32_t)x, hi = (uint32_t)(x >> 32);
    const auto a = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    x = max_u64(((uint64_t)b[0] << 32) | a[0], ((uint64_t)b[1] << 32) | a[1]);
  }
  return x;
}

// Sum over the wave, in every lane, by the exchange pattern of wave_max_u64
// (every lane adds the same pairs in the same tree, so all lanes agree bit
// for bit).
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float x) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(__float_as_int(x), __float_as_int(x), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_sum_dpp(float x) {
  x += dpp_f32<0xB1>(x);
  x += dpp_f32<0x4E>(x);
  x += dpp_f32<0x141>(x);
  x += dpp_f32<0x140>(x);
  {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  return x;
}

// Routing of one token by one wave (all 64 lanes active); lane l holds
// experts l, l+64, ... (NPL per lane). The k chosen experts and their weights
// go to idx[0..k) and w[0..k) (device or LDS memory). Each of the k picks is
// one wave-wide maximum of the remaining keys; the owner lane then clears the
// chosen key.
template <int NPL>
__device__ __forceinline__ void route_token(const float* __restrict__ row, int E, int k,
                                            int renorm, int32_t* idx, float* wout) {
  const int l = lane_id();
  float v[NPL];
  float selv[NPL];
  uint64_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = l + kWave * i;
    v[i] = 0.0f;
    selv[i] = 0.0f;
    key[i] = 0;
    if (e < E) {
      v[i] = row[e];
      key[i] = select_key(v[i], e);
    }
  }
  float top = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) best = max_u64(best, key[i]);
    best = wave_max_u64(best);
    // the same in every lane: take it into scalar registers
    const uint32_t be = ~(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)best);
    const float bv = key_logit((uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(best >> 32)));
    if (j == 0) top = bv;
    if ((int)(be & (kWave - 1)) == l) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i == (int)(be / kWave)) key[i] = 0;
    }
    if ((j & (kWave - 1)) == l) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i == j / kWave) selv[i] = bv;
      idx[j] = (int32_t)be;
    }
  }
  // weights: exp(v - top) normalised over the selection or over all experts
  float part = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if (renorm) {
      const int j = l + kWave * i;
      if (j < k) part += expf(selv[i] - top);
    } else if (l + kWave * i < E) {
      part += expf(v[i] - top);
    }
  }
  const float denom = wave_sum_dpp(part);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int j = l + kWave * i;
    if (j < k) wout[j] = expf(selv[i] - top) / denom;
  }
}

}  // namespace moe4
