// A whole routed layer for the few tokens of a decode step, in two launches:
//   1. k_layer_up: every workgroup routes all tokens itself, from which it knows the experts that
//      were chosen and their rows, and takes an even share of their gate/up pairs. h goes to the
//      workspace, with the list of experts and rows.
//   2. k_layer_down: a panel, 8 or 16 output columns of 8 tokens, is a sum over all experts that those
//      chose. Few units of work: a workgroup to a panel; many: the units of all panels are dealt to
//      the workgroups in equal runs, and the one that comes last to a panel that was cut adds its
//      parts, in their order.
// Sums are in a fixed order: which workgroup comes last decides who adds, not what.
//
// Both stream 4-bit weights for a handful of rows. One tile of either is 8 weight rows, and a step
// 256 k of them: its two halves of 128 k as the 16 columns (c, q) of a 16x16x32 MFMA, against 8
// tokens' activations in the same halves as its 16 rows (t, q'): the products with q = q' are
// wanted, the others are not read. So a wave's 16-byte loads take whole lines of 128 bytes of 8
// rows, a layer's rows give twice the tiles that 16-row tiles would, and no operand is padded to 16
// tokens.

#include <type_traits>

#include "common.hpp"
#include "formats.hpp"
#include "gemm_common.hpp"
#include "internal.hpp"
#include "mx.hpp"
#include "route.hpp"

namespace moe4 {
namespace {

constexpr int kRowsPass = 8;   // tokens that one pass over an expert's weights serves
static_assert(MOE4_LAYER_MOST_TOKENS <= 32, "an expert's tokens are the bits of a word");

// ---------------------------------------------------------------- weights

// NF4 without rounding: a level is the sum of two bf16 (to 8.1e-6 of it, 2^-16.9, and all but one to
// 2^-17), both multiply the activations exactly, and the block's absmax is applied to the fp32 sums of
// its 64 products. Both parts of a level but 0 have its sign and are not zero, +-1's too, so that an infinite
// activation gives the infinity that the level would, not the NaN of opposite ones or of infinity * 0.
// byte -> (high parts of its two levels, low parts): 8 bytes. LDS holds 32 copies of an entry, a row
// of 256 bytes, and lane l reads copy l mod 32: no two lanes of a half wave meet in a bank, and a
// lookup's address is its byte beside the lane's own (one v_perm).
struct alignas(16) Nf4Split {
  uint32_t v[512];
};
constexpr uint32_t bits_of(float f) { return __builtin_bit_cast(uint32_t, f); }
constexpr uint32_t bf16_rne(float f) {
  const uint32_t u = bits_of(f);
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}
constexpr Nf4Split make_nf4_split() {
  Nf4Split s{};
  for (int i = 0; i < 256; ++i)
    for (int h = 0; h < 2; ++h) {
      const float f = kNf4Levels[h ? i >> 4 : i & 15];
      // the bf16 next to it towards zero
      const uint32_t hi = f == 0.0f ? 0u : (bits_of(f) - 1) >> 16;
      const uint32_t lo = bf16_rne(f - __builtin_bit_cast(float, hi << 16));
      s.v[2 * i] |= hi << (16 * h);
      s.v[2 * i + 1] |= lo << (16 * h);
    }
  return s;
}
__device__ constexpr Nf4Split kNf4Split = make_nf4_split();
constexpr int kLutCopies = 32;
// (double-quantised: the codebook of the absmax behind it)
constexpr int lut_bytes(int fmt) {
  return fmt == MOE4_FMT_MXFP4 ? 0 : 2048 * kLutCopies + (fmt == MOE4_FMT_NF4_DQ ? 1024 : 0);
}

template <int FMT>
__device__ __forceinline__ void fill_lut(uint8_t* lut, const float* book) {
  if constexpr (FMT == MOE4_FMT_NF4_DQ) {
    if (threadIdx.x < 256) reinterpret_cast<float*>(lut + 2048 * kLutCopies)[threadIdx.x] = book[threadIdx.x];
  }
  if constexpr (FMT != MOE4_FMT_MXFP4) {
    // 16 bytes (two copies) at a time, four reads in flight
    constexpr int kAll = 256 * kLutCopies / 2;
    for (int i0 = threadIdx.x; i0 < kAll; i0 += 4 * blockDim.x) {
      u32x2 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = min(i0 + u * (int)blockDim.x, kAll - 1) / (kLutCopies / 2);
        v[u] = reinterpret_cast<const u32x2*>(kNf4Split.v)[e];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * (int)blockDim.x;
        if (i < kAll) reinterpret_cast<u32x4*>(lut)[i] = __builtin_shufflevector(v[u], v[u], 0, 1, 0, 1);
      }
    }
  }
}
// (the table begins LDS, so that the byte and the lane's place are the address: the kernels have no
// static LDS, and their dynamic LDS begins with it; tests/test_layer_resources.py holds them to that)
__device__ __forceinline__ u32x2 lookup(uint32_t w, int byte, uint32_t lane8) {
  typedef const u32x2 __attribute__((address_space(3))) entry_t;
  return *reinterpret_cast<entry_t*>(__builtin_amdgcn_perm(w, lane8, 0x0C0C0000u | (4 + byte) << 8));
}

// 4x4 transpose of dwords across the four 16-lane rows of a wave: row g holds D[g][0..3] before and
// D[0..3][g] after
__device__ __forceinline__ u32x4 transpose4(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{(uint32_t)c[0], (uint32_t)c[1], (uint32_t)d[0], (uint32_t)d[1]};
}

// A stack's matrices [rows][K] as its kernels read them.
struct Stack {
  const uint8_t* q;
  const void* s;
  const float *s2, *soff, *book;
  int K, rows;
};

constexpr int kStep = 256;   // k of a step: two halves of 128
__host__ __device__ constexpr int steps_of(int K) { return (K + kStep - 1) / kStep; }

// One expert's matrix from a row on, and a lane's place in it: its row (counted from there) and its
// half of a step. Loads past the matrix or past K give zeros. (A load that is to give zeros everywhere
// has no scalar offset: the range check subtracts that from the size.)
//
// Scales come for a run of four steps at once, those of step g to the lanes of row g of the
// wave (16 lanes), and are handed to all rows where their step is multiplied: a load of scales costs
// the memory pipeline as much as one of weights.
template <int FMT>
struct Stream {
  static constexpr bool kMx = FMT == MOE4_FMT_MXFP4, kDq = FMT == MOE4_FMT_NF4_DQ;
  static constexpr int kBlock = Format<FMT>::kBlock, kSb = FMT == MOE4_FMT_NF4 ? 4 : 1;
  // as loaded: NF4 two absmax; MXFP4 the dwords around the step's four bytes; double-quantised the
  // two codes, and the blocks' second absmax
  struct Raw {
    uint32_t v[2];
    uint32_t at;   // MXFP4: where the first byte is among them
    float a2[2];
  };
  const uint8_t *q, *s;
  const float* s2;
  uint32_t q_bytes, s_bytes;   // from there to the matrix' end
  int first;                   // double-quantised: flat index of its first absmax, mod 256
  int k0;                      // the lane's first k of a step
  uint32_t vq, vs;

  __device__ __forceinline__ void open(const Stack& st, int e, int row0, bool on) {
    const int nb = st.K / kBlock;
    const int64_t r0 = (int64_t)e * st.rows + row0;
    const int left = on ? st.rows - row0 : 0;
    q = st.q + r0 * (st.K / 2);
    s = static_cast<const uint8_t*>(st.s) + r0 * nb * kSb;
    q_bytes = (uint32_t)left * (uint32_t)(st.K / 2);
    s_bytes = (uint32_t)left * (uint32_t)(nb * kSb);
    if constexpr (kDq) {
      s2 = st.s2 + ((r0 * nb) >> 8);
      first = (int)((r0 * nb) & 255);
    }
  }
  __device__ __forceinline__ void place(int K, int row, int q_) {
    k0 = 128 * q_;
    vq = (uint32_t)(row * (K / 2) + k0 / 2 + 16 * (lane_id() >> 4));
    vs = (uint32_t)((row * (K / kBlock) + k0 / kBlock) * kSb);
  }
  // 16 bytes, the lane's 32 k of step st, `rows` (uniform) rows further on
  __device__ __forceinline__ u32x4 codes(int K, int st, int rows, bool on) const {
    const rsrc_t r = make_rsrc_uniform(q, on ? q_bytes : 0u);
    const int at = k0 + kStep * st + 32 * (lane_id() >> 4) < K ? (int)(vq + kStep / 2 * st) : kOob;
    // (the rows as the load's scalar offset: no vector register for each)
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, on ? rows * (K / 2) : 0, 0));
  }
  // the scales of the four steps from st on
  __device__ __forceinline__ void scales(Raw& p, int K, int st, int rows, bool on) const {
    const int nb = K / kBlock, k = k0 + kStep * (st + (lane_id() >> 4));
    const bool in = k < K;
    if constexpr (kMx) {
      // They start at any byte: the aligned dwords around them (the last may reach up to 3 bytes past
      // the scales' end, never past the aligned dword that holds their last byte).
      const uint64_t from = reinterpret_cast<uint64_t>(s) + (uint32_t)(rows * nb);
      const int lead = (int)(from & 3);
      const uint32_t size = on ? (uint32_t)((int)s_bytes - rows * nb + lead + 3) & ~3u : 0u;
      const rsrc_t r = make_rsrc_uniform(reinterpret_cast<const void*>(from & ~(uint64_t)3), size);
      const uint32_t at = vs + lead + (st + (lane_id() >> 4)) * 8;
      const u32x2 v = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, in ? (int)(at & ~3u) : kOob, 0, 0));
      p.v[0] = v[0];
      p.v[1] = v[1];
      p.at = at & 3;
    } else if constexpr (!kDq) {
      const rsrc_t r = make_rsrc_uniform(s, on ? s_bytes : 0u);
      const u32x2 v = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                     r, in ? (int)(vs + (st + (lane_id() >> 4)) * 16) : kOob, on ? rows * nb * 4 : 0, 0));
      p.v[0] = v[0];
      p.v[1] = v[1];
    } else {
      const rsrc_t r = make_rsrc_uniform(s, on ? s_bytes : 0u);
      const int at = (int)(vs + (st + (lane_id() >> 4)) * 4 + rows * nb);
      const bool here = on && in && (uint32_t)at < s_bytes, both = here && k + 64 < K;
      p.v[0] = buf_load_u8(r, here ? at : kOob);
      p.v[1] = buf_load_u8(r, both ? at + 1 : kOob);
      p.a2[0] = s2[here ? (first + at) >> 8 : 0];
      p.a2[1] = s2[both ? (first + at + 1) >> 8 : 0];
    }
  }
  // them as they multiply: NF4 two fp32, MXFP4 four bytes; 0 past K (what was loaded there belongs to
  // the next row)
  __device__ __forceinline__ void finish(Raw& p, int K, int st, const float* book, float off) const {
    const int k = k0 + kStep * (st + (lane_id() >> 4));
    if constexpr (kMx) {
      const int left = (K - k) / 32;
      const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1;
      p.v[0] = __builtin_amdgcn_alignbyte(p.v[1], p.v[0], p.at) & keep;
    } else {
      if constexpr (kDq) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          p.v[i] = __float_as_uint(mul_then_add(book[p.v[i]], p.a2[i], off));
        if (k >= K) p.v[0] = 0u;
      }
      if (k + 64 >= K) p.v[1] = 0u;
    }
  }
};
// the value that the lanes of row S of the wave hold, in all of them
template <int S>
__device__ __forceinline__ uint32_t from_row(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(a[S / 2], a[S / 2], false, false);
  return b[S % 2];
}

// The activations of one lane for a 128-k step as MFMA operands. MXFP4: four, of the lane's own 32
// k. NF4: each operand serves two bytes of codes, {high, low parts} of each, so it holds their two
// pairs of activations twice.
template <int FMT>
struct Acts {
  u32x4 v[FMT == MOE4_FMT_MXFP4 ? 4 : 8];
  __device__ __forceinline__ void set(int i, u32x4 x) {
    if constexpr (FMT == MOE4_FMT_MXFP4) {
      v[i] = x;
    } else {
      v[2 * i] = u32x4{x[0], x[0], x[1], x[1]};
      v[2 * i + 1] = u32x4{x[2], x[2], x[3], x[3]};
    }
  }
};
// the first k, within the step, of the lane's i-th 8
template <int FMT>
__device__ __forceinline__ int act_k(int i) {
  const int g = lane_id() >> 4;
  return FMT == MOE4_FMT_MXFP4 ? 32 * g + 8 * i : 32 * i + 8 * g;
}
// off: byte offset of the lane's row in the resource (kOob: no row); its half of the step starts at k.
// The lane's 32 k are all in K, or NF4's two blocks of 64 each are, or not.
template <int FMT>
__device__ __forceinline__ void load_acts(u32x4 (&x)[4], rsrc_t r, int off, int k, int K) {
  constexpr int kEach = FMT == MOE4_FMT_MXFP4 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < 4; i += kEach) {
    const int kk = k + act_k<FMT>(i), at = off != kOob && kk < K ? off + 2 * kk : kOob;
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      x[i + j] = buf_load_b128(r, offset_past(at, 2 * (act_k<FMT>(i + j) - act_k<FMT>(i))));
  }
}

// the same from a row in LDS; past K zeros
template <int FMT>
__device__ __forceinline__ void read_acts(u32x4 (&x)[4], const uint8_t* row, int k, int K) {
  constexpr int kEach = FMT == MOE4_FMT_MXFP4 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < 4; i += kEach) {
    const int kk = k + act_k<FMT>(i);
    const bool on = kk < K;
    const uint8_t* p = row + (on ? 2 * kk : 0);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(p + (on ? 2 * (act_k<FMT>(i + j) - act_k<FMT>(i)) : 0));
      x[i + j] = on ? v : u32x4{0u, 0u, 0u, 0u};
    }
  }
}

// acc += one step's products of TT tiles (which share their activations, or with NX = TT are so many
// steps of one tile, whose acc are to be added); s0, s1: their scales (NF4 two fp32, MXFP4 the four bytes in
// s0). MXFP4: the lane's 32 k are one block, each weight exact in bf16. NF4: the codes are put in
// MFMA order, so that two dwords of a lane make a block; lookups run ahead of the MFMAs that take
// them, by as much as covers LDS' latency, and the two blocks and the tiles take turns, so that no
// MFMA waits for the one before it. (Left to the compiler, which looked four bytes up, waited and
// multiplied, the first launch took 59 us for 16 tokens through
// 81 of 128 experts of 2048 x 768, and 53 so.)
template <int FMT, int TT, int NX>
__device__ __forceinline__ void step(const u32x4 (&codes)[TT], const uint32_t (&s0)[TT], const uint32_t (&s1)[TT],
                                     const Acts<FMT> (&x)[NX], uint32_t lane8, f32x4 (&acc)[TT]) {
  if constexpr (FMT == MOE4_FMT_MXFP4) {
    uint32_t byte[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) byte[j] = s0[j] >> (8 * (lane_id() >> 4)) & 255u;
    // (conversions a product ahead of it: a matrix instruction waits for operands just written)
    u32x4 b = mx4_bf16x8(codes[0][0], byte[0]);
#pragma unroll
    for (int i = 0; i < 4 * TT; ++i) {
      const int j = i % TT, jn = (i + 1) % TT, in = (i + 1) / TT;
      const u32x4 now = b;
      if (i + 1 < 4 * TT) b = mx4_bf16x8(codes[jn][in], byte[jn]);
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[NX == 1 ? 0 : j].v[i / TT]),
                                                       __builtin_bit_cast(bf16x8, now), acc[j], 0, 0, 0);
    }
  } else {
    constexpr int kAhead = TT >= 4 ? 1 : 4 / TT;
    u32x4 w[TT];
    u32x2 v[kAhead + 1][TT][2];
    f32x4 d[TT][2];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      w[j] = transpose4(codes[j]);
      d[j][0] = d[j][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto look = [&](int m) {   // block m % 2, its (m / 2)-th pair of bytes
      const int i = 4 * (m & 1) + m / 2;
#pragma unroll
      for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[m % (kAhead + 1)][j][h] = lookup(w[j][i / 2], 2 * (i & 1) + h, lane8);
    };
#pragma unroll
    for (int m = 0; m < kAhead; ++m) look(m);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      if (m + kAhead < 8) look(m + kAhead);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const u32x2* e = v[m % (kAhead + 1)][j];
        d[j][m & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, x[NX == 1 ? 0 : j].v[4 * (m & 1) + m / 2]),
            __builtin_bit_cast(bf16x8, __builtin_shufflevector(e[0], e[1], 0, 1, 2, 3)), d[j][m & 1], 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[j][i] = fmaf(__uint_as_float(s1[j]), d[j][1][i], fmaf(__uint_as_float(s0[j]), d[j][0][i], acc[j][i]));
  }
}

// ------------------------------------------------------------------ launch 1

// Up to 8 rows of one expert: the expert (10 bits), how many rows (4), the first one's place among
// all rows, which are ordered by expert and token (9)
__device__ __forceinline__ uint32_t make_entry(int e, int n, int row) { return (uint32_t)(e | n << 10 | row << 14); }
__device__ __forceinline__ int entry_expert(uint32_t v) { return v & 1023; }
__device__ __forceinline__ int entry_rows(uint32_t v) { return (v >> 10) & 15; }
__device__ __forceinline__ int entry_first(uint32_t v) { return (v >> 14) & 511; }
static_assert(MOE4_LAYER_MOST_SLOTS <= 512, "an entry holds a row in 9 bits");

// What the second launch knows of an expert that some of a group of 8 tokens chose: the expert (12
// bits), its first row; and all tokens of the expert as bits
struct Use {
  uint32_t what, tokens;
};

struct LayerArgs {
  Stack gu, dn;
  int E, H, I, layout, act;
  float alpha, limit;
  const uint16_t *gu_bias, *dn_bias;
  const uint16_t* x;
  const float* logits;
  int T, k, renorm;
  const void* residual;
  int res_dtype;
  void* out;
  int out_dtype;
  int32_t* user_idx;
  float* user_w;
  int runs, run_steps;   // runs of steps of the second launch: how many, of how many
  // workspace
  uint16_t* h;       // [rows = T * k][I], weighted
  int32_t* idx;      // [T * k] experts of the slots
  float* w;          // [T * k] and their weights
  Use* uses;         // [T * k], by groups of 8 tokens
  int32_t* count;    // [4] how many of each group
  float* part;       // [2 workgroups][8][64] parts of panels
  int32_t* arrived;  // [panels] how many of a panel's parts are there
  int panels;
};

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
  x = max_dpp<0xB1>(x);    // quad_perm [1,0,3,2]
  x = max_dpp<0x4E>(x);    // quad_perm [2,3,0,1]
  x = max_dpp<0x141>(x);   // row_half_mirror
  x = max_dpp<0x140>(x);   // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}

// A token's keys (route.hpp's order) in a wave: lane l holds experts l, l + 64, ... 0 is no candidate, a
// NaN 1. Of equal logits the lower expert is taken first, by where the key is found.
template <int NPL>
struct Keys {
  uint32_t key[NPL];
  float v[NPL];   // as loaded
  __device__ __forceinline__ void load(const float* row, int E) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = row[min(lane_id() + kWave * i, E - 1)];
  }
  __device__ __forceinline__ void order(int E) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = lane_id() + kWave * i < E ? max(order_key(v[i]), 1u) : 0u;
  }
  // takes the first expert of the order out; its key in *k
  __device__ __forceinline__ int pick(uint32_t* k) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) best = max(best, key[i]);
    best = __builtin_amdgcn_readfirstlane(wave_max_u32(best));
    int e = -1;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const uint64_t b = __ballot(key[i] == best);
      if (e < 0 && b) {
        e = (__ffsll((long long)b) - 1) + kWave * i;
        if ((e & (kWave - 1)) == lane_id()) key[i] = 0u;
      }
    }
    *k = best;
    return e;
  }
};

// A tile is 4 gate/up pairs (gates are its rows 0..3, ups 4..7). The tiles of all entries are dealt to
// all waves in equal runs, and a wave takes its run by itself, up to four tiles of an entry at a
// time over all of k: the activations' operands serve all four, and no wave waits for another
// after the routing. (The waves of a workgroup splitting k of the same tiles, with a barrier
// and a sum through LDS for each 16 pairs, took as
// long for many tokens and 2 us more for one.) Us: 16 tokens through 81 of 128 NF4 experts of 2048 x
// 768 51 (143 MB; 9 of them routing and table), 8 through 20 of 32 MXFP4 experts of 2880 x 2880 46 (180
// MB), one token 13. Without the arithmetic and the activations the loads alone take 41, 42 and 9.

// LDS of the first launch, after the table: tokens of an expert [E] as bits, its first
// row [E], entries [S], tokens and weights of the rows [S], experts and weights of the slots [S], how many entries
__host__ __device__ constexpr int route_lds(int E, int S) { return 8 * E + 20 * S + 4; }

//
// XL (MXFP4): the tokens' activations stand in LDS (x_lds bytes), where they fit, instead of being loaded
// by every wave in the matrix instruction's layout, which takes four loads beside a step's weights (8
// tokens through 20 experts of 2880 x 2880 50 us, 46 so; NF4 51 either
// way).
constexpr int kXPad = 32;   // bytes between rows: the rows of a read in different banks
__host__ __device__ constexpr int x_lds(int T, int H) { return T * (2 * H + kXPad); }

template <int FMT, int NPL, bool XL>
__global__ __launch_bounds__(512) void k_layer_up(const LayerArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int nw = 8;
  const int wv = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id();
  const int S = a.T * a.k;
  uint8_t* lut = smem;
  uint32_t* chose = reinterpret_cast<uint32_t*>(smem + lut_bytes(FMT));
  int* base = reinterpret_cast<int*>(chose + a.E);
  uint32_t* entries = reinterpret_cast<uint32_t*>(base + a.E);
  int* row_t = reinterpret_cast<int*>(entries + S);
  float* row_w = reinterpret_cast<float*>(row_t + S);
  int* slot_e = reinterpret_cast<int*>(row_w + S);
  float* slot_w = reinterpret_cast<float*>(slot_e + S);
  int& s_count = *reinterpret_cast<int*>(slot_w + S);
  uint8_t* const xs = smem + (lut_bytes(FMT) + route_lds(a.E, S) + 15) / 16 * 16;
  const int steps = steps_of(a.H);
  const int c = l & 7, q = (l >> 3) & 1, g = l >> 4;   // a weight column (c, q), an activation row (t, q)
  const bool writer = blockIdx.x == 0;                 // hands the routing on

  // ---- routing: a token by one wave
  // (its logits are on their way while the table is filled, or the token before is routed)
  Keys<NPL> keys;
  auto fetch = [&](int t) { keys.load(a.logits + (int64_t)min(t, a.T - 1) * a.E, a.E); };
  auto route = [&](int t) {
    keys.order(a.E);
    fetch(t + nw);
    float all = 0.0f, some = 0.0f, top = 0.0f;
    if (!a.renorm) {   // softmax over all experts, not over the chosen alone
      uint32_t m = keys.key[0];
#pragma unroll
      for (int i = 1; i < NPL; ++i) m = max(m, keys.key[i]);
      top = key_logit(wave_max_u32(m));
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (keys.key[i]) all += expf(key_logit(keys.key[i]) - top);
    }
    for (int j0 = 0; j0 < a.k; j0 += kWave) {
      int mine = 0;
      uint32_t mykey = 0;
      const int n = min(kWave, a.k - j0);
      for (int j = 0; j < n; ++j) {
        uint32_t key;
        const int e = keys.pick(&key);
        if (j0 + j == 0 && a.renorm) top = key_logit(key);
        if (l == j) {
          mine = e;
          mykey = key;
        }
      }
      if (l < n) {
        const int s = t * a.k + j0 + l;
        slot_e[s] = mine;
        if (a.T > 1) atomicOr(&chose[mine], 1u << t);
        const float v = expf(key_logit(mykey) - top);
        slot_w[s] = v;
        some += v;
      }
    }
    const float denom = wave_sum_dpp(a.renorm ? some : all);
    for (int j = l; j < a.k; j += kWave) {
      const int s = t * a.k + j;
      const float w = slot_w[s] / denom;
      slot_w[s] = w;
      if (writer) {
        a.idx[s] = slot_e[s];
        a.w[s] = w;
        if (a.user_idx) a.user_idx[s] = slot_e[s];
        if (a.user_w) a.user_w[s] = w;
      }
    }
  };
  fetch(wv);
  if constexpr (XL) {
    const int per = a.H / 8;   // 16-byte pieces of a row
    for (int i0 = threadIdx.x; i0 < a.T * per; i0 += 4 * 512) {
      u32x4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = reinterpret_cast<const u32x4*>(a.x)[min(i0 + u * 512, a.T * per - 1)];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * 512, t = i / per;
        if (i < a.T * per) *reinterpret_cast<u32x4*>(xs + t * (2 * a.H + kXPad) + (i - t * per) * 16) = v[u];
      }
    }
  }
  for (int i = blockIdx.x * 512 + threadIdx.x; i < a.panels; i += gridDim.x * 512) a.arrived[i] = 0;
  if (a.T == 1) {
    // an expert's rows are one row each, in the order of the choice
    if (wv == 0) {
      route(0);
      for (int j = l; j < a.k; j += kWave) {
        entries[j] = make_entry(slot_e[j], 1, j);
        row_t[j] = 0;
        row_w[j] = slot_w[j];
        if (writer) a.uses[j] = {(uint32_t)(slot_e[j] | j << 12), 1u};
      }
      if (l == 0) {
        s_count = a.k;
        if (writer) a.count[0] = a.k, a.count[1] = a.count[2] = a.count[3] = 0;
      }
    }
    fill_lut<FMT>(lut, a.gu.book);
    __syncthreads();
  } else {
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) chose[i] = 0;
    fill_lut<FMT>(lut, a.gu.book);
    __syncthreads();
    for (int t = wv; t < a.T; t += nw) route(t);
    __syncthreads();
    if (wv == 0) {
      int rows = 0, count = 0;
      for (int e0 = 0; e0 < a.E; e0 += kWave) {
        const int e = e0 + l;
        const uint32_t bits = e < a.E ? chose[e] : 0u;
        const int n = __popc(bits), m = (n + kRowsPass - 1) / kRowsPass;
        const int r = wave_scan_dpp(n), p = wave_scan_dpp(m);
        if (e < a.E) base[e] = rows + r - n;
        for (int i = 0; i < m; ++i)
          entries[count + p - m + i] =
              make_entry(e, min(n - i * kRowsPass, kRowsPass), rows + r - n + i * kRowsPass);
        rows += __builtin_amdgcn_readlane(r, 63);
        count += __builtin_amdgcn_readlane(p, 63);
      }
      if (l == 0) s_count = count;
    }
    __syncthreads();
    if (writer && wv == 0) {
      int uses = 0;
      for (int i = 0; i < 4; ++i) {
        const int from = uses;
        for (int e0 = 0; e0 < a.E; e0 += kWave) {
          const int e = e0 + l;
          const uint32_t bits = e < a.E ? chose[e] : 0u;
          const int here = (bits >> (8 * i) & 255u) != 0, u = wave_scan_dpp(here);
          if (here) a.uses[uses + u - 1] = {(uint32_t)(e | base[e] << 12), bits};
          uses += __builtin_amdgcn_readlane(u, 63);
        }
        if (l == 0) a.count[i] = uses - from;
      }
    }
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
      const int t = s / a.k, e = slot_e[s];
      const int r = base[e] + __popc(chose[e] & ((1u << t) - 1));
      row_t[r] = t;
      row_w[r] = slot_w[s];
    }
    __syncthreads();
  }
  const int count = __builtin_amdgcn_readfirstlane(s_count);

  // ---- this wave's run of tiles
  const int per = a.I / 4, all = count * per, wid = blockIdx.x * nw + wv, waves = gridDim.x * nw;
  const int first = (int)((int64_t)all * wid / waves), end = (int)((int64_t)all * (wid + 1) / waves);
  const int mult = a.layout == MOE4_GU_HALVES ? 1 : 2;
  const rsrc_t rx = make_rsrc_uniform(a.x, (uint32_t)(a.T * a.H * 2));
  const float* book = FMT == MOE4_FMT_NF4_DQ ? reinterpret_cast<const float*>(lut + 2048 * kLutCopies) : nullptr;
  const float off = FMT == MOE4_FMT_NF4_DQ ? a.gu.soff[0] : 0.0f;
  const uint32_t lane8 = 8 * (l & (kLutCopies - 1));
  Stream<FMT> in;
  in.place(a.H, c < 4 ? gate_row(a.layout, a.I, c & 3) : up_row(a.layout, a.I, c & 3), q);
  // TT tiles (n of them there) from tile j0 of an entry on
  auto run = [&](auto tc, uint32_t entry, int j0, int n) {
    constexpr int TT = decltype(tc)::value;
    constexpr int kDepth = TT > 2 ? 2 : 4;               // steps in flight
    constexpr int kX = !XL ? kDepth : TT == 1 ? 2 : 1;   // of activations (in LDS: those of the next product)
    const int rows = entry_rows(entry);
    in.open(a.gu, entry_expert(entry), 4 * j0 * mult, true);
    // the lane's row of activations (XL: of those that are there, which the product has no more rows than)
    const int tok = row_t[entry_first(entry) + (c < rows ? c : 0)];
    const int xoff = XL ? tok * (2 * a.H + kXPad) : c < rows ? tok * a.H * 2 : kOob;
    // the lane's tile, pair and tokens at the end: tile 2 (g / 2) + q, pair c & 3 (gates in lanes c < 4),
    // tokens 4 (g % 2) ...
    const int mj = 2 * (g >> 1) + q, pair = 4 * (j0 + mj) + (c & 3);
    uint32_t bias = 0;
    if (a.gu_bias) {
      const rsrc_t rb = make_rsrc_uniform(a.gu_bias + (int64_t)entry_expert(entry) * 2 * a.I, 4 * a.I);
      const int at = c < 4 ? gate_row(a.layout, a.I, pair) : up_row(a.layout, a.I, pair);
      bias = __builtin_amdgcn_raw_buffer_load_b16(rb, mj < n ? 2 * at : kOob, 0, 0);
    }
    u32x4 w[kDepth][TT], xr[kX][4];
    typename Stream<FMT>::Raw sc[TT], next[TT];
    auto load_w = [&](int d, int st) {
#pragma unroll
      for (int j = 0; j < TT; ++j) w[d][j] = in.codes(a.H, st, 4 * j * mult, j < n);
    };
    auto load_x = [&](int d, int st) {
      if constexpr (XL) read_acts<FMT>(xr[d], xs + xoff, in.k0 + kStep * st, a.H);
      else load_acts<FMT>(xr[d], rx, xoff, in.k0 + kStep * st, a.H);
    };
    f32x4 acc[TT], pair_acc[2];
    pair_acc[0] = pair_acc[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      in.scales(next[j], a.H, 0, 4 * j * mult, j < n);
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      load_w(d, d);
      if (d < kX) load_x(d, d);
    }
    for (int s0 = 0; s0 < steps; s0 += 4) {
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        sc[j] = next[j];
        in.finish(sc[j], a.H, s0, book, off);
        in.scales(next[j], a.H, s0 + 4, 4 * j * mult, j < n);
      }
      // (steps past the last: zeros)
      if constexpr (TT == 1) {   // two steps at a time, for something to do while one waits
        auto two = [&](auto ic) {
          constexpr int i = decltype(ic)::value;
          Acts<FMT> x[2];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            x[0].set(v, xr[i % kX][v]);
            x[1].set(v, xr[(i + 1) % kX][v]);
          }
          if constexpr (XL) {
            load_x(0, s0 + i + 2);
            load_x(1, s0 + i + 3);
          }
          const u32x4 both[2] = {w[i][0], w[i + 1][0]};
          const uint32_t lo[2] = {from_row<i>(sc[0].v[0]), from_row<i + 1>(sc[0].v[0])};
          const uint32_t hi[2] = {FMT == MOE4_FMT_MXFP4 ? 0u : from_row<i>(sc[0].v[1]),
                                  FMT == MOE4_FMT_MXFP4 ? 0u : from_row<i + 1>(sc[0].v[1])};
          step<FMT, 2, 2>(both, lo, hi, x, lane8, pair_acc);
          __builtin_amdgcn_sched_barrier(0);
          load_w(i, s0 + i + 4);
          load_w(i + 1, s0 + i + 5);
          if constexpr (!XL) {
            load_x(i, s0 + i + 4);
            load_x(i + 1, s0 + i + 5);
          }
          __builtin_amdgcn_sched_barrier(0);
        };
        two(std::integral_constant<int, 0>{});
        two(std::integral_constant<int, 2>{});
      } else {
        auto one = [&](auto ic) {
          constexpr int i = decltype(ic)::value, d = i % kDepth;
          Acts<FMT> x[1];
#pragma unroll
          for (int v = 0; v < 4; ++v) x[0].set(v, xr[d % kX][v]);
          if constexpr (XL) load_x(0, s0 + i + 1);
          uint32_t lo[TT], hi[TT];
#pragma unroll
          for (int j = 0; j < TT; ++j) {
            lo[j] = from_row<i>(sc[j].v[0]);
            hi[j] = FMT == MOE4_FMT_MXFP4 ? 0u : from_row<i>(sc[j].v[1]);
          }
          step<FMT, TT, 1>(w[d], lo, hi, x, lane8, acc);
          __builtin_amdgcn_sched_barrier(0);
          load_w(d, s0 + i + kDepth);
          if constexpr (!XL) load_x(d, s0 + i + kDepth);
          __builtin_amdgcn_sched_barrier(0);
        };
        one(std::integral_constant<int, 0>{});
        one(std::integral_constant<int, 1>{});
        one(std::integral_constant<int, 2>{});
        one(std::integral_constant<int, 3>{});
      }
    }
    if constexpr (TT == 1) acc[0] = pair_acc[0] + pair_acc[1];
    // D[m][n]: lane n = (c, q) holds rows m = 4 g .. 4 g + 3, those of half q' = g / 2. The halves' sum of
    // tile mj to the lanes of mj.
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const uint32_t b = __float_as_uint(acc[j][r]);
        const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);   // tokens' first, second half
        const float own = __uint_as_float(q ? h[1] : h[0]);
        const float sum = own + dpp_f32<0x128>(own);   // row_ror:8
        v[r] = j == 0 || mj == j ? sum : v[r];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r >= rows) break;
      const int t = 4 * (g & 1) + r;
      const float u = v[r] + bf16_to_f32(bias);
      const float gt = u, up = dpp_f32<0x104>(u);   // row_shl:4: lane c takes c + 4's
      float h;
      if (a.act == MOE4_ACT_SWIGLU) {
        h = gt * sigmoidf_(gt) * up;
      } else {   // comparisons, so that a NaN stays one
        const float gc = gt > a.limit ? a.limit : gt;
        const float uc = up > a.limit ? a.limit : up < -a.limit ? -a.limit : up;
        h = (uc + 1.0f) * gc * sigmoidf_(a.alpha * gc);
      }
      // weighted, and rounded once to bf16, the operand type of the second product
      if (c < 4 && t < rows && mj < n) {
        const int at = entry_first(entry) + t;
        a.h[(int64_t)at * a.I + pair] = f32_to_bf16(h * row_w[at]);
      }
    }
  };
  // (double-quantised scales take more registers: two tiles at a time)
  constexpr int kMost = FMT == MOE4_FMT_NF4_DQ ? 2 : 4;
  for (int at = first; at < end;) {
    const int e = at / per, j0 = at - e * per, n = min(min(end - at, per - j0), kMost);
    const uint32_t entry = __builtin_amdgcn_readfirstlane(entries[e]);
    if constexpr (kMost == 4) {
      if (n > 2) {
        run(std::integral_constant<int, 4>{}, entry, j0, n);
        at += n;
        continue;
      }
    }
    if (n == 2) run(std::integral_constant<int, 2>{}, entry, j0, n);
    else run(std::integral_constant<int, 1>{}, entry, j0, n);
    at += n;
  }
}

// ------------------------------------------------------------------ launch 2

// A panel is 8 TT kSide output columns of a group of 8 tokens; its units are the experts that some of them
// chose, each cut into runs of RS steps. kSide waves of a workgroup take 8 TT columns each of the same
// unit, the others the units between; a unit's loads are asked for while the unit before is multiplied. A token's row
// of activations stands at the token's place in the MFMA's first operand (zeros where it did not
// choose the expert), and h is weighted, so a wave's sums over its units stay in its accumulators.
// The waves' sums are added in their order.
//
// CUT: the units of all panels, in a row, are dealt evenly to the workgroups, which leaves none idle
// where the panels are few or no multiple of the chip's 256 (8 tokens through 20 of 32 MXFP4 experts of
// 2880 x 2880, 360 panels of 8 columns with a workgroup each, took 40 us, and 32 so; 16 tokens through
// 81 NF4 experts of 2048 x 768, 256 panels, 34 either way). A panel that was cut is written in parts; who comes last (a counter for each panel, zeroed
// by the first launch) adds them.
//
// A workgroup to a CU is two waves to a SIMD (NF4's 208 registers allow no more), which in NF4 wait for 45% of
// their time while vector instructions take 42% of the cycles, the matrix cores 15%, LDS 16%, and HBM gives 2.1
// TB/s. The separate calls' down kernel, with 106 registers, reads the same 72 MB in 26 us.
template <int FMT, int TT, int RS, bool CUT>
__global__ __launch_bounds__(512) void k_layer_down(const LayerArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  // waves side by side in a panel, and those that share its units
  constexpr int kSide = CUT ? 4 : 1, nw = 8 / kSide, kCols = 8 * TT * kSide;
  const int S = a.T * a.k;
  const int wid = __builtin_amdgcn_readfirstlane(wave_id()), wv = wid / kSide, side = wid % kSide, l = lane_id();
  // LDS: table | sums [nw][8][kCols] | uses [S] | experts and weights of the slots [S] (biases)
  uint8_t* lut = smem;
  float* sums = reinterpret_cast<float*>(smem + lut_bytes(FMT));
  Use* uses = reinterpret_cast<Use*>(sums + nw * 8 * kCols);
  int* slot_e = reinterpret_cast<int*>(uses + S);
  float* slot_w = reinterpret_cast<float*>(slot_e + S);
  int& s_last = *reinterpret_cast<int*>(slot_w + S);
  const int c = l & 7, q = (l >> 3) & 1, g = l >> 4;
  int cnt[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) cnt[i] = __builtin_amdgcn_readfirstlane(a.count[i]);
  const int used = cnt[0] + cnt[1] + cnt[2] + cnt[3];
  for (int i = threadIdx.x; i < S; i += 512) {
    uses[i] = a.uses[i];   // (those past the last are never looked at; not to wait for how many there are)
    if (a.dn_bias) {
      slot_e[i] = a.idx[i];
      slot_w[i] = a.w[i];
    }
  }
  fill_lut<FMT>(lut, a.dn.book);
  __syncthreads();
  const int G = (a.H + kCols - 1) / kCols, steps = steps_of(a.I);
  // this workgroup's units
  const int64_t N = (int64_t)used * a.runs * G, W = min((int64_t)gridDim.x, N);
  int64_t first, end;
  if constexpr (CUT) {
    if (blockIdx.x >= W) return;   // every workgroup that stays has a unit
    first = N * blockIdx.x / W;
    end = N * (blockIdx.x + 1) / W;
  } else {
    int tg = 0, skip = 0;
    while ((int)blockIdx.x >= (tg + 1) * G) skip += cnt[tg++];
    first = ((int64_t)skip * G + (int64_t)(blockIdx.x - tg * G) * cnt[tg]) * a.runs;
    end = first + cnt[tg] * a.runs;
  }
  const rsrc_t rh = make_rsrc_uniform(a.h, (uint32_t)(S * a.I * 2));
  const float off = FMT == MOE4_FMT_NF4_DQ ? a.dn.soff[0] : 0.0f;
  const float* book = FMT == MOE4_FMT_NF4_DQ ? reinterpret_cast<const float*>(lut + 2048 * kLutCopies) : nullptr;
  const uint32_t lane8 = 8 * (l & (kLutCopies - 1));
  Stream<FMT> in;
  in.place(a.I, c, q);

  for (int64_t at = first; at < end;) {
    // the panel that unit `at` belongs to: token group, column group, units, and where they begin
    int tg = 0, skip = 0;
    int64_t base = 0;
    while (at >= base + (int64_t)cnt[tg] * a.runs * G) {
      base += (int64_t)cnt[tg] * a.runs * G;
      skip += cnt[tg++];
    }
    const int U = cnt[tg] * a.runs, cg = (int)((at - base) / U), u0 = (int)(at - base - (int64_t)cg * U);
    const int n = (int)min(end - at, (int64_t)(U - u0)), c0 = cg * kCols, mine0 = c0 + 8 * TT * side;
    // ---- the wave's units
    u32x4 w[RS][TT], xr[RS][4];
    typename Stream<FMT>::Raw raw[TT], sc[TT];
    int u = u0 + wv, s0 = 0, xoff = kOob;
    uint32_t tokens = 0;
    auto open = [&] {
      const bool on = u < u0 + n && mine0 < a.H;
      const int i = on ? u / a.runs : 0;
      const Use use = uses[skip + i];
      const uint32_t what = __builtin_amdgcn_readfirstlane(use.what);
      const uint32_t all = on ? __builtin_amdgcn_readfirstlane(use.tokens) : 0u;
      s0 = on ? (u - i * a.runs) * a.run_steps : 0;
      in.open(a.dn, what & 4095, on ? mine0 : 0, on);
      tokens = all >> (8 * tg) & 255u;
      const int r = (int)(what >> 12) + __popc(all & ((1u << (8 * tg + c)) - 1));
      xoff = tokens >> c & 1 ? r * a.I * 2 : kOob;
#pragma unroll
      for (int j = 0; j < TT; ++j) in.scales(raw[j], a.I, s0, 8 * j, on);
    };
    auto load = [&](int i) {   // (a run may have fewer steps than RS)
      const int st = i < a.run_steps ? s0 + i : steps + 1;
#pragma unroll
      for (int j = 0; j < TT; ++j) w[i][j] = in.codes(a.I, st, 8 * j, in.q_bytes != 0);
      load_acts<FMT>(xr[i], rh, xoff, in.k0 + kStep * st, a.I);
    };
    f32x4 acc[TT], d[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    open();
#pragma unroll
    for (int i = 0; i < RS; ++i) load(i);
    while (u < u0 + n) {
      const uint32_t mine = tokens;
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        sc[j] = raw[j];
        in.finish(sc[j], a.I, s0, book, off);
        d[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      u += nw;
      open();
      auto one = [&](auto ic) {
        constexpr int i = decltype(ic)::value;
        if constexpr (i < RS) {
          Acts<FMT> x[1];
#pragma unroll
          for (int v = 0; v < 4; ++v) x[0].set(v, xr[i][v]);
          uint32_t lo[TT], hi[TT];
#pragma unroll
          for (int j = 0; j < TT; ++j) {
            lo[j] = from_row<i>(sc[j].v[0]);
            hi[j] = FMT == MOE4_FMT_MXFP4 ? 0u : from_row<i>(sc[j].v[1]);
          }
          step<FMT, TT, 1>(w[i], lo, hi, x, lane8, d);
          __builtin_amdgcn_sched_barrier(0);
          load(i);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      one(std::integral_constant<int, 0>{});
      one(std::integral_constant<int, 1>{});
      one(std::integral_constant<int, 2>{});
      one(std::integral_constant<int, 3>{});
      // (a token that did not choose the expert takes nothing of it: its zeros times an infinite or
      // NaN weight are no zeros)
#pragma unroll
      for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] += mine >> (4 * (g & 1) + r) & 1 ? d[j][r] : 0.0f;
    }
    // ---- what the thread's output takes besides: residual, and the biases' sum
    const int ot = 8 * tg + (int)threadIdx.x / kCols, oc = c0 + threadIdx.x % kCols;
    const bool out = (int)threadIdx.x < 8 * kCols && ot < a.T && oc < a.H;
    const int64_t oat = (int64_t)ot * a.H + oc;
    float more = 0.0f;
    if (out && a.dn_bias) {
      for (int j0 = 0; j0 < a.k; j0 += 4) {
        float b[4], v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int sl = ot * a.k + min(j0 + j, a.k - 1);
          v[j] = j0 + j < a.k ? slot_w[sl] : 0.0f;
          b[j] = bf16_to_f32(a.dn_bias[(int64_t)slot_e[sl] * a.H + oc]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) more = j0 + j < a.k ? fmaf(v[j], b[j], more) : more;
      }
    }
    if (out && a.residual)
      more += a.res_dtype == MOE4_DTYPE_F32 ? static_cast<const float*>(a.residual)[oat]
                                            : bf16_to_f32(static_cast<const uint16_t*>(a.residual)[oat]);
    // ---- D[m][n]: lane n = (c, q) holds rows m = 4 g .. 4 g + 3, those of half q' = g / 2. The halves'
    // sum of tile mj to the lanes of mj.
    const int mj = 2 * (g >> 1) + q;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float v = 0.0f;
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const uint32_t b = __float_as_uint(acc[j][r]);
        const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);   // tokens' first, second half
        const float own = __uint_as_float(q ? h[1] : h[0]);
        const float sum = own + dpp_f32<0x128>(own);   // row_ror:8
        v = j == 0 || mj == j ? sum : v;
      }
      if (mj < TT) sums[(wv * 8 + 4 * (g & 1) + r) * kCols + 8 * (TT * side + mj) + c] = v;
    }
    __syncthreads();
    float v = 0.0f;
    if ((int)threadIdx.x < 8 * kCols) {
#pragma unroll
      for (int p = 0; p < nw; ++p) v += sums[p * 8 * kCols + threadIdx.x];
    }
    bool done = true;
    if constexpr (CUT) {
      if (n < U) {
        // workgroups i0 .. i1 have a part of the panel each, at place 2 i where it is the first thing
        // they do, else (it is their last) at 2 i + 1
        const int64_t p0 = base + (int64_t)cg * U;
        const int64_t i0 = ((p0 + 1) * W - 1) / N, i1 = ((p0 + U) * W - 1) / N;
        // Parts and counters are only touched by atomics of device scope, which go through to where
        // all dies meet, in both directions; a part is there (its wave waits for that) before the
        // barrier behind which the counter says so. (Fences of device scope, which write a die's whole
        // cache back, took 140 us.)
        if ((int)threadIdx.x < 8 * kCols) {
          float* to = a.part + (2 * (int64_t)blockIdx.x + (at != first)) * 8 * kCols + threadIdx.x;
          __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        wait_vmcnt<0>();
        __syncthreads();
        if (threadIdx.x == 0)
          s_last = __hip_atomic_fetch_add(&a.arrived[tg * G + cg], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == i1 - i0;
        __syncthreads();
        done = s_last;
        if (done && (int)threadIdx.x < 8 * kCols) {
          v = 0.0f;
          for (int64_t i = i0; i <= i1; ++i) {
            const float* from = a.part + (2 * i + (i == i0 && N * i / W < p0)) * 8 * kCols + threadIdx.x;
            v += __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          }
        }
      }
    }
    if (done && out) {
      if (a.out_dtype == MOE4_DTYPE_F32) static_cast<float*>(a.out)[oat] = v + more;
      else static_cast<uint16_t*>(a.out)[oat] = f32_to_bf16(v + more);
    }
    at += n;
    __syncthreads();   // the sums, and s_last, are used again
  }
}

constexpr int kDownRoom = 256;   // workgroups of the second launch where panels are cut
struct LayerWs {
  size_t idx, w, uses, count, arrived, part, end;
  LayerWs(int H, int I, int T, int k) {
    const size_t S = (size_t)T * k;
    idx = align_up(S * I * 2, 256);
    w = idx + align_up(S * 4, 256);
    uses = w + align_up(S * 4, 256);
    count = uses + align_up(S * sizeof(Use), 256);
    arrived = count + 256;
    part = arrived + align_up((size_t)((H + 63) / 64) * 4 * 4, 256);
    end = part + (size_t)2 * kDownRoom * 8 * 64 * 4;
  }
};

constexpr int kLdsAll = 160 * 1024;   // of a CU

template <int FMT>
hipError_t launch_layer(LayerArgs a, hipStream_t s) {
  const int S = a.T * a.k;
  constexpr bool kMx = FMT == MOE4_FMT_MXFP4;
  const int dsteps = steps_of(a.I);
  constexpr int kRun = kMx ? 4 : 3;   // (registers)
  a.runs = (dsteps + kRun - 1) / kRun;
  a.run_steps = (dsteps + a.runs - 1) / a.runs;
  a.runs = (dsteps + a.run_steps - 1) / a.run_steps;
  // Panels are cut (and two tiles share their activations) from so many units on. Us cut and not: NF4
  // experts of 2048 x 768, 8 each, 4 tokens 17.4 14.1, 8 (8192 by this count) 21.8 19.5, 16 34 39; MXFP4
  // 2880 x 2880, 4 each, 2 tokens 18.9 16.6, 4 (8640) 25.2 25.0, 8 32 37.
  const int groups = (a.T + 7) / 8;
  const bool cut = (int64_t)(a.H / 16) * S * a.runs >= 12288;
  a.panels = cut ? (a.H + 63) / 64 * groups : 0;
  // as many workgroups as the chip holds at once (some of their waves idle where tiles are few), or one
  // for every tile
  const int64_t tiles = (int64_t)S * (a.I / 4), room = 256;
  const int lds = (lut_bytes(FMT) + route_lds(a.E, S) + 15) / 16 * 16;
  static_assert(lut_bytes(FMT) + route_lds(1024, MOE4_LAYER_MOST_SLOTS) + 16 <= kLdsAll, "any call's first launch fits");
  const bool xl = kMx && lds + x_lds(a.T, a.H) <= kLdsAll;
  auto up = [&](auto* k) {
    const int bytes = lds + (xl ? x_lds(a.T, a.H) : 0);
    hipError_t e = allow_lds<kLdsAll>(k);
    if (e != hipSuccess) return e;
    k<<<(uint32_t)(tiles < room ? tiles : room), 512, bytes, s>>>(a);
    return hipGetLastError();
  };
  hipError_t e;
  if (xl) e = a.E <= 128 ? up(&k_layer_up<FMT, 2, kMx>) : up(&k_layer_up<FMT, 16, kMx>);
  else e = a.E <= 128 ? up(&k_layer_up<FMT, 2, false>) : up(&k_layer_up<FMT, 16, false>);
  if (e != hipSuccess) return e;
  auto down = [&](auto* k, int grid, int tt) {
    const int bytes = lut_bytes(FMT) + 8 * 8 * 8 * tt * 4 + S * ((int)sizeof(Use) + 8) + 4;
    hipError_t r = allow_lds<kLdsAll>(k);
    if (r != hipSuccess) return r;
    k<<<grid, 512, bytes, s>>>(a);
    return hipGetLastError();
  };
  auto by_steps = [&](auto rc) {
    constexpr int RS = decltype(rc)::value;
    if (cut) return down(&k_layer_down<FMT, 2, RS, true>, kDownRoom, 2);
    return down(&k_layer_down<FMT, 1, RS, false>, a.H / 8 * groups, 1);
  };
  if (a.run_steps <= 2) return by_steps(std::integral_constant<int, 2>{});
  if constexpr (kRun == 4)
    if (a.run_steps == 4) return by_steps(std::integral_constant<int, 4>{});
  return by_steps(std::integral_constant<int, 3>{});
}

}  // namespace

size_t layer_decode_ws_bytes(const moe4_experts& ex, int T, int k) { return LayerWs(ex.H, ex.I, T, k).end; }

hipError_t launch_layer_decode(const moe4_experts& ex, const uint16_t* x, const float* logits,
                               int T, int k, int renorm, const void* residual, int res_dtype,
                               void* out, int out_dtype, int32_t* topk_idx, float* topk_w,
                               void* ws, hipStream_t s) {
  uint8_t* const w8 = static_cast<uint8_t*>(ws);
  const LayerWs at(ex.H, ex.I, T, k);
  LayerArgs a = {};
  a.gu = {static_cast<const uint8_t*>(ex.gu_q), ex.gu_s, ex.gu_s2, ex.gu_soff, ex.dq_book, ex.H, 2 * ex.I};
  a.dn = {static_cast<const uint8_t*>(ex.dn_q), ex.dn_s, ex.dn_s2, ex.dn_soff, ex.dq_book, ex.I, ex.H};
  a.E = ex.E;
  a.H = ex.H;
  a.I = ex.I;
  a.layout = ex.gu_layout;
  a.act = ex.act;
  a.alpha = ex.act_alpha;
  a.limit = ex.act_limit;
  a.gu_bias = ex.gu_bias;
  a.dn_bias = ex.dn_bias;
  a.x = x;
  a.logits = logits;
  a.T = T;
  a.k = k;
  a.renorm = renorm;
  a.residual = residual;
  a.res_dtype = res_dtype;
  a.out = out;
  a.out_dtype = out_dtype;
  a.user_idx = topk_idx;
  a.user_w = topk_w;
  a.h = reinterpret_cast<uint16_t*>(w8);
  a.idx = reinterpret_cast<int32_t*>(w8 + at.idx);
  a.w = reinterpret_cast<float*>(w8 + at.w);
  a.uses = reinterpret_cast<Use*>(w8 + at.uses);
  a.count = reinterpret_cast<int32_t*>(w8 + at.count);
  a.arrived = reinterpret_cast<int32_t*>(w8 + at.arrived);
  a.part = reinterpret_cast<float*>(w8 + at.part);
  if (ex.format == MOE4_FMT_NF4) return launch_layer<MOE4_FMT_NF4>(a, s);
  if (ex.format == MOE4_FMT_MXFP4) return launch_layer<MOE4_FMT_MXFP4>(a, s);
  return launch_layer<MOE4_FMT_NF4_DQ>(a, s);
}

}  // namespace moe4
