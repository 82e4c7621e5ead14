// A whole routed layer for the few tokens of a decode step, in two launches:
//   1. k_layer_up: every workgroup takes one routed slot and some gate/up pairs. It finds the slot's
//      expert from the logits itself and, among all tokens, those that chose the same expert; the
//      first slot of an expert works for all of them, the others end. h goes to the workspace.
//   2. k_layer_down: every workgroup takes 8 output columns and runs over all experts that were
//      chosen, so the weighted sum over a token's slots stays inside it.
// No counter, flag or order of arrival decides anything: sums are in a fixed order.
//
// Both stream 4-bit weights for a handful of rows. One tile of either is 8 weight rows, each cut
// into two halves of k, as the 16 columns (c, q) of a 16x16x32 MFMA, against 8 tokens' activations
// in the same two halves as its 16 rows (t, q'): the products with q = q' are wanted, the others
// are not read. So a wave's 16-byte loads cover 256 k of 8 rows, a layer's rows give twice the
// tiles that 16-row tiles would, and no operand is padded to 16 tokens.
#include <type_traits>

#include "common.hpp"
#include "formats.hpp"
#include "gemm_common.hpp"
#include "internal.hpp"
#include "mx.hpp"
#include "route.hpp"

namespace moe4 {
namespace {

constexpr int kMostT = MOE4_LAYER_MOST_TOKENS;
constexpr int kRowsPass = 8;   // tokens that one pass over an expert's weights serves
static_assert(kMostT <= 32, "a row list's entries hold a token in 5 bits");

// ---------------------------------------------------------------- weights

// NF4 without rounding: a level is the sum of two bf16 (to 2^-17 of it), both multiply the
// activations exactly, and the block's absmax is applied to the fp32 sums of its 64 products.
// byte -> (high parts of its two levels, low parts); LDS holds kLutCopies copies, lane l reads
// copy l % kLutCopies, which spreads the lookups of a wave over the banks.
struct Nf4Split {
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
      const uint32_t hi = bf16_rne(f);
      const uint32_t lo = bf16_rne(f - __builtin_bit_cast(float, hi << 16));
      s.v[2 * i] |= hi << (16 * h);
      s.v[2 * i + 1] |= lo << (16 * h);
    }
  return s;
}
__device__ constexpr Nf4Split kNf4Split = make_nf4_split();
constexpr int kLutCopies = 4;
constexpr int kLutBytes = 2048 * kLutCopies;

__device__ __forceinline__ void fill_lut(u32x2* lut) {
  for (int i = threadIdx.x; i < 256; i += blockDim.x) {
    const u32x2 v = {kNf4Split.v[2 * i], kNf4Split.v[2 * i + 1]};
#pragma unroll
    for (int c = 0; c < kLutCopies; ++c) lut[i * kLutCopies + c] = v;
  }
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

// One expert's matrix [rows][K] as its kernels read it.
struct Stack {
  const uint8_t* q;
  const void* s;
  const float *s2, *soff, *book;
  int K, rows;
};

// The scales of one lane's 128 k of a weight row: NF4 two blocks, MXFP4 the lane's own 32
template <int FMT>
struct LaneScale {
  uint32_t v[FMT == MOE4_FMT_MXFP4 ? 1 : 2];
  float a2[FMT == MOE4_FMT_NF4_DQ ? 2 : 1];
};

// A weight row's piece in a lane: 16 bytes (32 k) and what scales them. row < st.rows, k the first
// of the lane's 128-k step (its own 32 k at k + 32 g); pieces past K read as zeros.
template <int FMT>
struct Piece {
  u32x4 w;
  LaneScale<FMT> s;
  __device__ __forceinline__ void load(const Stack& st, int e, int row, int k) {
    const int g = lane_id() >> 4;
    const rsrc_t rq = make_rsrc_uniform(st.q + (int64_t)e * st.rows * (st.K / 2),
                                        (uint32_t)((int64_t)st.rows * (st.K / 2)));
    const int kk = k + 32 * g;
    w = buf_load_b128(rq, kk < st.K ? (int)((uint32_t)row * (st.K / 2) + kk / 2) : kOob);
    if constexpr (FMT == MOE4_FMT_MXFP4) {
      const int nb = st.K / 32;
      const rsrc_t rs = make_rsrc_uniform(static_cast<const uint8_t*>(st.s) + (int64_t)e * st.rows * nb,
                                          (uint32_t)(st.rows * nb));
      s.v[0] = buf_load_u8(rs, kk < st.K ? row * nb + kk / 32 : kOob);
    } else if constexpr (FMT == MOE4_FMT_NF4) {
      const int nb = st.K / 64;
      const rsrc_t rs = make_rsrc_uniform(static_cast<const float*>(st.s) + (int64_t)e * st.rows * nb,
                                          (uint32_t)(st.rows * nb) * 4);
      // (a second block past the row's end belongs to the next row: its weights are zeros' codes
      // against zero activations)
      const u32x2 r = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                     rs, k < st.K ? (int)((uint32_t)(row * nb + k / 64) * 4) : kOob, 0, 0));
      s.v[0] = r[0];
      s.v[1] = k + 64 < st.K ? r[1] : 0u;
    } else {
      const int nb = st.K / 64;
      const int64_t first = (int64_t)e * st.rows * nb;
      const uint8_t* codes = static_cast<const uint8_t*>(st.s) + first;
      const int at = row * nb + min(k, st.K - 64) / 64;
      const int at1 = k + 64 < st.K ? at + 1 : at;
      s.v[0] = codes[at];
      s.v[1] = codes[at1];
      s.a2[0] = st.s2[(first + at) >> 8];
      s.a2[1] = st.s2[(first + at1) >> 8];
    }
  }
};

// The activations of one lane for a 128-k step: four MFMA operands
struct Acts {
  u32x4 v[4];
};
// off: byte offset of the lane's row in the resource (kOob: no row); its step starts at k
template <int FMT>
__device__ __forceinline__ void load_acts(Acts& x, rsrc_t r, int off, int k, int K) {
  const int g = lane_id() >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int kk = k + (FMT == MOE4_FMT_MXFP4 ? 32 * g + 8 * i : 32 * i + 8 * g);
    x.v[i] = buf_load_b128(r, off != kOob && kk < K ? off + 2 * kk : kOob);
  }
}

// acc += one step's products. MXFP4: the lane's 32 k are one block, each weight exact in bf16. NF4:
// the codes are put in MFMA order, so that two operands make a block.
template <int FMT>
__device__ __forceinline__ void step(const Piece<FMT>& p, const Acts& x, const u32x2* lut, float off,
                                     const float* book, f32x4& acc) {
  if constexpr (FMT == MOE4_FMT_MXFP4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x.v[i]),
                                                    __builtin_bit_cast(bf16x8, mx4_bf16x8(p.w[i], p.s.v[0])),
                                                    acc, 0, 0, 0);
  } else {
    const u32x4 w = transpose4(p.w);
    const u32x2* mine = lut + (lane_id() & (kLutCopies - 1));
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 2 * b; i < 2 * b + 2; ++i) {
        u32x4 hi, lo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x2 v = mine[((w[i] >> (8 * j)) & 255u) * kLutCopies];
          hi[j] = v[0];
          lo[j] = v[1];
        }
        const bf16x8 a = __builtin_bit_cast(bf16x8, x.v[i]);
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, hi), d, 0, 0, 0);
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, lo), d, 0, 0, 0);
      }
      float s;
      if constexpr (FMT == MOE4_FMT_NF4) s = __uint_as_float(p.s.v[b]);
      else s = mul_then_add(book[p.s.v[b]], p.s.a2[b], off);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, d[i], acc[i]);
    }
  }
}

// first k of the second half of a row: a multiple of 128, so that steps and blocks stay whole
__host__ __device__ constexpr int half_k(int K) { return (K + 255) / 256 * 128; }

// ------------------------------------------------------------------ launch 1

// A row list's entry: the slot, and its token
__device__ __forceinline__ uint32_t list_entry(int slot, int t) { return (uint32_t)(slot | t << 16); }

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
  // workspace
  uint16_t* h;       // [T * k][I], by slot
  int32_t* idx;      // [T * k]
  float* w;          // [T * k]
  int32_t* cnt;      // [T * k] rows of the expert whose first slot this is, else 0
  uint32_t* list;    // [T * k][kMostT] those rows' entries, tokens ascending
};

// A token's experts in the order of moe4_route, by one wave: each pick is the largest key below the
// one before
template <int NPL>
struct Picks {
  uint64_t key[NPL], last = ~0ull;
  __device__ __forceinline__ void init(const float* row, int E) {
    const int l = lane_id();
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      key[i] = l + kWave * i < E ? select_key(row[l + kWave * i], l + kWave * i) : 0;
  }
  // the next expert (the same in every lane)
  __device__ __forceinline__ int next() {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) best = max_u64(best, key[i] < last ? key[i] : 0);
    last = wave_max_u64(best);
    return (int)~(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)last);
  }
};
// How many experts a token puts before expert e, by one wave
template <int NPL>
__device__ __forceinline__ int rank_of_expert(const float* row, int E, int e) {
  const int l = lane_id();
  const uint64_t mine = select_key(row[e], e);
  int n = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int o = l + kWave * i;
    n += __popcll(__ballot(o < E && select_key(row[min(o, E - 1)], o) > mine));
  }
  return n;
}

// TG tiles of 4 gate/up pairs to a workgroup; wave v takes the 128-k steps v, v + waves, ... of both
// halves of k for all of them, so its activations stay in registers and its loads are weights.
template <int FMT, int TG, int NPL>
__global__ __launch_bounds__(512) void k_layer_up(const LayerArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  u32x2* lut = reinterpret_cast<u32x2*>(smem);
  float* red = reinterpret_cast<float*>(smem + (FMT == MOE4_FMT_MXFP4 ? 0 : kLutBytes));
  constexpr int kRed = 68;   // floats of a tile's half: [c][t], padded
  __shared__ int s_rank[kMostT], s_idx[MOE4_LAYER_MOST_SLOTS];
  __shared__ float s_w[MOE4_LAYER_MOST_SLOTS];
  const int nw = blockDim.x >> 6, wv = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id();
  const int ntg = a.I / (4 * TG);
  const int slot = blockIdx.x / ntg, tg = blockIdx.x - slot * ntg;
  const int t0 = slot / a.k, j0 = slot - t0 * a.k;
  if constexpr (FMT != MOE4_FMT_MXFP4) fill_lut(lut);
  Picks<NPL> picks;
  picks.init(a.logits + (int64_t)t0 * a.E, a.E);
  int e = picks.next();
  for (int j = 0; j < j0; ++j) e = picks.next();
  for (int t = wv; t < a.T; t += nw) {
    const int r = t == t0 ? j0 : rank_of_expert<NPL>(a.logits + (int64_t)t * a.E, a.E, e);
    if (l == 0) s_rank[t] = r;
  }
  __syncthreads();
  // tokens that chose e, as bits: the same in every wave
  const uint32_t chose = (uint32_t)__ballot(l < a.T && s_rank[min(l, kMostT - 1)] < a.k);
  const bool first = (chose & ((1u << t0) - 1)) == 0;
  const int n = __popc(chose);
  if (tg == 0 && wv == 0) {
    // what the second launch reads: the slot's rows, and a token's routing by its first slot
    if (l == 0) a.cnt[slot] = first ? n : 0;
    if (first && (chose >> l & 1) && l < kMostT) {
      const int at = __popc(chose & ((1u << l) - 1));
      a.list[slot * kMostT + at] = list_entry(l * a.k + s_rank[l], l);
    }
  }
  if (first) {
    const int Kh = half_k(a.H), steps = Kh / 128;
    const int m = l & 15, c = m & 7, q = m >> 3;   // a weight column (c, q), an activation row (t, q)
    // the row of the gate/up stack of column c: gates 0..3, ups 4..7 of the tile's pairs
    const rsrc_t rx = make_rsrc_uniform(a.x, (uint32_t)(a.T * a.H * 2));
    for (int pass = 0; pass * kRowsPass < n; ++pass) {
      // the token of activation row c of this pass
      uint32_t left = chose;
      for (int i = 0; i < pass * kRowsPass + c; ++i) left &= left - 1;
      const int xoff = left ? (__ffs(left) - 1) * a.H * 2 : kOob;
      f32x4 acc[TG];
#pragma unroll
      for (int j = 0; j < TG; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int st = wv; st < steps; st += nw) {
        const int k = q * Kh + 128 * st;
        Acts x;
        load_acts<FMT>(x, rx, xoff, k, a.H);
        Piece<FMT> p[TG];
#pragma unroll
        for (int j = 0; j < TG; ++j) {
          const int pair = (tg * TG + j) * 4 + (c & 3);
          const int row = c < 4 ? gate_row(a.layout, a.I, pair) : up_row(a.layout, a.I, pair);
          p[j].load(a.gu, e, row, k);
        }
        const float off = FMT == MOE4_FMT_NF4_DQ ? a.gu.soff[0] : 0.0f;
#pragma unroll
        for (int j = 0; j < TG; ++j) step<FMT>(p[j], x, lut, off, a.gu.book, acc[j]);
      }
      // D[m][n]: lane n = (c, q) holds rows m = 4 g .. 4 g + 3, those of half q' = g / 2
      const int g = l >> 4;
      if (pass) __syncthreads();   // the sums of the pass before have been read
      if ((g >> 1) == q) {
#pragma unroll
        for (int j = 0; j < TG; ++j)
          *reinterpret_cast<f32x4*>(red + ((wv * 2 + q) * TG + j) * kRed + c * 8 + 4 * (g & 1)) = acc[j];
      }
      __syncthreads();
      for (int i = threadIdx.x; i < TG * 4 * kRowsPass; i += blockDim.x) {
        const int p = i % (TG * 4), t = i / (TG * 4), j = p / 4, cp = p & 3;
        const int r = pass * kRowsPass + t;
        if (r >= n) continue;
        uint32_t rest = chose;
        for (int u = 0; u < r; ++u) rest &= rest - 1;
        const int tok = __ffs(rest) - 1, pair = (tg * TG + j) * 4 + cp;
        float gt = 0.0f, up = 0.0f;
        for (int v = 0; v < 2 * nw; ++v) {
          const float* s = red + (v * TG + j) * kRed + cp * 8 + t;
          gt += s[0];
          up += s[32];
        }
        if (a.gu_bias) {
          const uint16_t* b = a.gu_bias + (int64_t)e * 2 * a.I;
          gt += bf16_to_f32(b[gate_row(a.layout, a.I, pair)]);
          up += bf16_to_f32(b[up_row(a.layout, a.I, pair)]);
        }
        float h;
        if (a.act == MOE4_ACT_SWIGLU) {
          h = gt * sigmoidf_(gt) * up;
        } else {   // comparisons, so that a NaN stays one
          const float gc = gt > a.limit ? a.limit : gt;
          const float uc = up > a.limit ? a.limit : up < -a.limit ? -a.limit : up;
          h = (uc + 1.0f) * gc * sigmoidf_(a.alpha * gc);
        }
        // rounded once to bf16, the operand type of the second product
        a.h[(int64_t)(tok * a.k + s_rank[tok]) * a.I + pair] = f32_to_bf16(h);
      }
    }
  }
  if (tg == 0 && j0 == 0 && wv == nw - 1) {
    // the token's whole choice and its weights
    picks.init(a.logits + (int64_t)t0 * a.E, a.E);
    picks.last = ~0ull;
    for (int j = 0; j < a.k; ++j) {
      const int i = picks.next();
      if (l == 0) {
        s_idx[j] = i;
        s_w[j] = key_value(picks.last);
      }
    }
    // softmax over the chosen or over all experts
    const float top = s_w[0];
    float part = 0.0f;
    if (a.renorm) {
      for (int j = l; j < a.k; j += kWave) part += expf(s_w[j] - top);
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (l + kWave * i < a.E) part += expf(key_value(picks.key[i]) - top);
    }
    const float denom = wave_sum_dpp(part);
    for (int j = l; j < a.k; j += kWave) {
      const int i = s_idx[j], at = t0 * a.k + j;
      const float w = expf(s_w[j] - top) / denom;
      a.idx[at] = i;
      a.w[at] = w;
      if (a.user_idx) a.user_idx[at] = i;
      if (a.user_w) a.user_w[at] = w;
    }
  }
}

// ------------------------------------------------------------------ launch 2

// 8 output columns to a workgroup; a unit is one expert (8 of its rows) and one 128-k step of both
// halves of its k, and wave v takes the units v, v + waves, ... Each wave sums into its own part of
// LDS, weighted, in its units' order; the parts are added in the waves' order.
template <int FMT>
__global__ __launch_bounds__(1024) void k_layer_down(const LayerArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int S = a.T * a.k;
  const int nw = blockDim.x >> 6, wv = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id();
  // LDS: table | sums [nw][2][T][8] | weights [S] | experts [S] | units [2 S] | their count
  u32x2* lut = reinterpret_cast<u32x2*>(smem);
  float* sums = reinterpret_cast<float*>(smem + (FMT == MOE4_FMT_MXFP4 ? 0 : kLutBytes));
  float* sw = sums + nw * 2 * a.T * 8;
  int* se = reinterpret_cast<int*>(sw + S);
  uint32_t* units = reinterpret_cast<uint32_t*>(se + S);
  __shared__ int s_units;
  if constexpr (FMT != MOE4_FMT_MXFP4) fill_lut(lut);
  for (int i = threadIdx.x; i < nw * 2 * a.T * 8; i += blockDim.x) sums[i] = 0.0f;
  for (int i = threadIdx.x; i < S; i += blockDim.x) {
    sw[i] = a.w[i];
    se[i] = a.idx[i];
  }
  if (wv == 0) {
    // experts in the order of their first slots, every 8 rows of one an entry of its own: the
    // slot, which 8, and how many
    int base = 0;
    for (int s0 = 0; s0 < S; s0 += kWave) {
      const int s = s0 + l, n = s < S ? a.cnt[s] : 0, passes = (n + kRowsPass - 1) / kRowsPass;
      const int incl = wave_scan_dpp(passes), at = base + incl - passes;
      for (int p = 0; p < passes; ++p)
        units[at + p] = (uint32_t)s | (uint32_t)p << 16 | (uint32_t)min(n - p * kRowsPass, kRowsPass) << 24;
      base += __builtin_amdgcn_readlane(incl, 63);
    }
    if (l == 0) s_units = base;
  }
  __syncthreads();
  const int Kh = half_k(a.I), steps = Kh / 128;
  const int c0 = blockIdx.x * 8;
  const int m = l & 15, c = m & 7, q = m >> 3, g = l >> 4;
  const rsrc_t rh = make_rsrc_uniform(a.h, (uint32_t)(S * a.I * 2));
  const int total = __builtin_amdgcn_readfirstlane(s_units) * steps;
  const float off = FMT == MOE4_FMT_NF4_DQ ? a.dn.soff[0] : 0.0f;
  struct Unit {
    Piece<FMT> p;
    Acts x;
    uint32_t row[4];   // list entries of the lane's four output rows
    int rows;          // rows of the unit
  };
  auto load = [&](Unit& u, int i) {
    const bool on = i < total;
    const uint32_t w = __builtin_amdgcn_readfirstlane(units[on ? i / steps : 0]);
    const int st = on ? i % steps : 0;
    const int s = w & 0xFFFF, pass = (w >> 16) & 255, n = on ? w >> 24 : 0;
    const int e = __builtin_amdgcn_readfirstlane(se[s]);
    const uint32_t* list = a.list + s * kMostT + pass * kRowsPass;
    const int k = q * Kh + 128 * st;
    u.rows = n;
    u.p.load(a.dn, e, c0 + c, on ? k : a.I);
    const uint32_t mine = c < n ? list[c] : 0;
    load_acts<FMT>(u.x, rh, c < n ? (int)(mine & 0xFFFF) * a.I * 2 : kOob, k, a.I);
#pragma unroll
    for (int r = 0; r < 4; ++r) u.row[r] = 4 * (g & 1) + r < n ? list[4 * (g & 1) + r] : 0;
  };
  auto finish = [&](const Unit& u) {
    f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
    step<FMT>(u.p, u.x, lut, off, a.dn.book, d);
    if ((g >> 1) == q) {
      float* mine = sums + (wv * 2 + q) * a.T * 8 + c;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * (g & 1) + r < u.rows)
          mine[(u.row[r] >> 16) * 8] += sw[u.row[r] & 0xFFFF] * d[r];
    }
  };
  Unit u0, u1;
  int i = wv;
  load(u0, i);
  while (i < total) {
    load(u1, i + nw);
    finish(u0);
    i += nw;
    if (i >= total) break;
    load(u0, i + nw);
    finish(u1);
    i += nw;
  }
  __syncthreads();
  for (int o = threadIdx.x; o < a.T * 8; o += blockDim.x) {
    const int t = o >> 3, col = c0 + (o & 7);
    float v = 0.0f;
    for (int p = 0; p < 2 * nw; ++p) v += sums[p * a.T * 8 + o];
    if (a.dn_bias) {
      for (int j = 0; j < a.k; ++j)
        v = fmaf(sw[t * a.k + j], bf16_to_f32(a.dn_bias[(int64_t)se[t * a.k + j] * a.H + col]), v);
    }
    const int64_t at = (int64_t)t * a.H + col;
    if (a.residual)
      v += a.res_dtype == MOE4_DTYPE_F32 ? static_cast<const float*>(a.residual)[at]
                                         : bf16_to_f32(static_cast<const uint16_t*>(a.residual)[at]);
    if (a.out_dtype == MOE4_DTYPE_F32) static_cast<float*>(a.out)[at] = v;
    else static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(v);
  }
}

// Waves that share a workgroup's 128-k steps: as many rounds of them as eight, six or four waves
// need, whichever leaves fewest idle
int up_waves(int H) {
  const int steps = half_k(H) / 128;
  int best = 8;
  for (int n : {6, 4})
    if ((steps + n - 1) / n * n < (steps + best - 1) / best * best) best = n;
  return best;
}

struct LayerWs {
  size_t idx, w, cnt, list, end;
  LayerWs(int I, int T, int k) {
    const size_t S = (size_t)T * k;
    idx = align_up(S * I * 2, 256);
    w = idx + align_up(S * 4, 256);
    cnt = w + align_up(S * 4, 256);
    list = cnt + align_up(S * 4, 256);
    end = list + S * kMostT * 4;
  }
};

template <int FMT>
hipError_t launch_layer(const LayerArgs& a, hipStream_t s) {
  const int S = a.T * a.k;
  const int nw = up_waves(a.H);
  auto up = [&](auto tc, auto pc) {
    constexpr int TG = decltype(tc)::value;
    const int lds = (FMT == MOE4_FMT_MXFP4 ? 0 : kLutBytes) + nw * 2 * TG * 68 * 4;
    k_layer_up<FMT, TG, decltype(pc)::value><<<S * (a.I / (4 * TG)), nw * 64, lds, s>>>(a);
    return hipGetLastError();
  };
  using I2 = std::integral_constant<int, 2>;
  using I16 = std::integral_constant<int, 16>;
  using I4 = std::integral_constant<int, 4>;
  using I8 = std::integral_constant<int, 8>;
  const bool wide = (int64_t)S * (a.I / 32) >= 512;
  hipError_t e = a.E <= 128 ? (wide ? up(I8{}, I2{}) : up(I4{}, I2{}))
                            : (wide ? up(I8{}, I16{}) : up(I4{}, I16{}));
  if (e != hipSuccess) return e;
  const int dw = 8;
  const int lds = (FMT == MOE4_FMT_MXFP4 ? 0 : kLutBytes) + dw * 2 * a.T * 8 * 4 + S * 8 + S * 8;
  k_layer_down<FMT><<<a.H / 8, dw * 64, lds, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t layer_decode_ws_bytes(const moe4_experts& ex, int T, int k) { return LayerWs(ex.I, T, k).end; }

hipError_t launch_layer_decode(const moe4_experts& ex, const uint16_t* x, const float* logits,
                               int T, int k, int renorm, const void* residual, int res_dtype,
                               void* out, int out_dtype, int32_t* topk_idx, float* topk_w,
                               void* ws, hipStream_t s) {
  uint8_t* const w8 = static_cast<uint8_t*>(ws);
  const LayerWs at(ex.I, T, k);
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
  a.cnt = reinterpret_cast<int32_t*>(w8 + at.cnt);
  a.list = reinterpret_cast<uint32_t*>(w8 + at.list);
  if (ex.format == MOE4_FMT_NF4) return launch_layer<MOE4_FMT_NF4>(a, s);
  if (ex.format == MOE4_FMT_MXFP4) return launch_layer<MOE4_FMT_MXFP4>(a, s);
  return launch_layer<MOE4_FMT_NF4_DQ>(a, s);
}

}  // namespace moe4
