// Forward of the dense gated feed-forward block (the shared expert beside the routed ones):
//   gu = x W_gu^T + b_gu;  h = act(gate, up);  out = h W_dn^T + b_dn + residual
// on bf16 weights and activations, or on MXFP8 ones (h is then quantised to MXFP8 between the
// two products). Two launches: both projections with the activation, then the second product
// with its bias and residual.
//
// Many tokens are bound by the matrix cores: 4096 tokens at H 4096, I 8192 in bf16 take 640-650 us,
// 1.29 PFLOP/s (a large library product reaches 1.24 to 1.55 on this card; of the k loop's
// cycles 85% multiply, at a clock that the load pulls to 1.9 GHz); 2048 in MXFP8 at H = I = 2880
// 82 us, 1.24 PFLOP/s (the second product's 96 large or 368 small tiles do not fill the chip).
// Few tokens are bound by launches and by load instructions: one token at H 2048, I 768 5.5 + 3.8
// us, 16 in MXFP8 at 2880, 2880 12.5 + 5.1 us; one token at H 4096, I 8192 43 us, 4.7 TB/s.
#include "ffn.hpp"

namespace moe4 {
namespace {

struct GateUpArgs {
  Operand W, X;
  int64_t w_s, x_s;       // bytes of the scales (MXFP8)
  int T, H, I, layout;
  FfnAct act;
  const uint16_t* bias;
  float* save_gu;
  uint16_t* h;            // bf16 [T, I]
  uint8_t *hq, *hs;       // MXFP8 [T, I], [T, I / 32]
  int splits;             // parts of k
  float* part;            // [splits][T][2][I] sums of gates and ups to be joined
};

// element of row t of save_gu that pair j's gate (or, with `up`, up) value has
__device__ __forceinline__ int gu_col(int layout, int I, int j, bool up) {
  return layout == MOE4_GU_HALVES ? (up ? I + j : j) : 2 * j + (up ? 1 : 0);
}

// the biases of 8 pairs j .. j+7 as they lie in memory (bf16); zeros without
struct RawBias {
  u32x4 v[2];
};
__device__ __forceinline__ RawBias load_bias8(const GateUpArgs& a, int j) {
  RawBias r = {};
  if (!a.bias || j >= a.I) return r;
  const bool halves = a.layout == MOE4_GU_HALVES;
  r.v[0] = *reinterpret_cast<const u32x4*>(a.bias + (halves ? j : 2 * j));
  r.v[1] = *reinterpret_cast<const u32x4*>(a.bias + (halves ? a.I + j : 2 * j + 8));
  return r;
}
// gates, then ups
__device__ __forceinline__ void unpack_bias8(const GateUpArgs& a, const RawBias& r, float* b) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t h = r.v[0][i / 2], f = r.v[i / 4][i % 4];
    const uint32_t u = r.v[1][i / 2];
    if (a.layout == MOE4_GU_HALVES) {
      b[i] = i & 1 ? bf16hi(h) : bf16lo(h);
      b[8 + i] = i & 1 ? bf16hi(u) : bf16lo(u);
    } else {
      b[i] = bf16lo(f);
      b[8 + i] = bf16hi(f);
    }
  }
}

// bias, saved pre-activations and activation of 8 pairs j .. j+7 of token t, in place of g
__device__ __forceinline__ void finish8(const GateUpArgs& a, int t, int j, const float* bias,
                                        float* g, float* u) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g[i] += bias[i];
    u[i] += bias[8 + i];
  }
  if (a.save_gu) {
    float* s = a.save_gu + (int64_t)t * 2 * a.I;
    if (a.layout == MOE4_GU_HALVES) {
      store8_f32(s + j, g);
      store8_f32(s + a.I + j, u);
    } else {
      float x[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[2 * i] = g[i];
        x[2 * i + 1] = u[i];
      }
      store8_f32(s + 2 * j, x);
      store8_f32(s + 2 * j + 8, x + 8);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = a.act.apply(g[i], u[i]);
}

template <bool FP8>
__device__ __forceinline__ void store_h8(const GateUpArgs& a, int t, int j, bool on,
                                         const float* h) {
  if constexpr (FP8) {
    // the four lanes of a block come together (I is a multiple of 32: all on, or none)
    uint32_t byte;
    const u32x2 q = mx_quantize8(h, byte);
    if (on) {
      *reinterpret_cast<u32x2*>(a.hq + (int64_t)t * a.I + j) = q;
      if ((j & 31) == 0) a.hs[(int64_t)t * (a.I / 32) + j / 32] = (uint8_t)byte;
    }
  } else if (on) {
    // rounded once to bf16, the operand type of the second product
    *reinterpret_cast<u32x4*>(a.h + (int64_t)t * a.I + j) = pack8_bf16(h);
  }
}

template <typename S, bool FP8, int LAYOUT, int ACT>
__global__ __launch_bounds__(S::kThreads, 2) void k_ffn_gate_up(GateUpArgs a) {
  a.layout = LAYOUT;
  a.act.act = ACT;
  extern __shared__ __attribute__((aligned(16))) uint8_t stage_mem[];
  constexpr int kPairs = S::BA / 2, es = FP8 ? 1 : 2;
  const int na = (a.I + kPairs - 1) / kPairs, nb = (a.T + S::BB - 1) / S::BB;
  int ia, ib;
  const int id = xcd_remap(blockIdx.x, gridDim.x), split = id / (na * nb);
  tile_of(id % (na * nb), na, nb, ia, ib);
  const int j0 = ia * kPairs, t0 = ib * S::BB;
  const int nt = min(S::BB, a.T - t0);
  OpLoader<S, kOpRow, S::BA, FP8> la;
  OpLoader<S, kOpRow, S::BB, FP8> lb;
  const KPart k(a.H, es, split, S::kSplits ? a.splits : 1);
  la.init_row(a.W.from_row(k.kt0), es, k.K, 0, 2 * a.I,
              [&](int r) { return pair_row(a.layout, a.I, j0, r); });
  lb.init_row(a.X.from_row(k.kt0), es, k.K, t0, nt, [=](int r) { return r < nt ? r : -1; });
  const MxScales mx = {a.W.s, a.X.s, a.w_s, a.x_s, a.H / 32, k.kt0 * 4};
  f32x16 acc[S::TA][S::TB];
  gemm_loop<S, kOpRow, kOpRow, FP8>(
      acc, stage_mem, la, lb, k.K, mx, [&](int r) { return pair_row(a.layout, a.I, j0, r); },
      [&](int r) { return r < nt ? t0 + r : -1; });
  if constexpr (S::kSplits) {
    if (a.splits > 1) {
      float* part = a.part + (int64_t)split * a.T * 2 * a.I;
      for_each8<S, true, 1>(acc, stage_mem, [](int, int) { return NoPre{}; },
                            [&](int row, int jj, float* g, float* u) {
        const int j = j0 + jj;
        if (row >= nt || j >= a.I) return;
        float* o = part + (int64_t)(t0 + row) * 2 * a.I + j;
        store8_f32(o, g);
        store8_f32(o + a.I, u);
      });
      return;
    }
  }
  float bias[16];   // the same pairs in every turn
  unpack_bias8(a, load_bias8(a, j0 + lane_a<S, true>()), bias);
  for_each8<S, true, 1>(acc, stage_mem, [](int, int) { return NoPre{}; },
                        [&](int row, int jj, float* g, float* u) {
    const int t = t0 + row, j = j0 + jj;
    const bool on = row < nt && j < a.I;
    if (on) finish8(a, t, j, bias, g, u);
    store_h8<FP8>(a, t, j, on, g);
  });
}

// The parts of a split gate/up product, joined: 8 pairs of a token to a thread (four
// neighbours share a block of MXFP8).
template <bool FP8>
__global__ __launch_bounds__(256) void k_ffn_gate_up_join(const GateUpArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = a.I / 8;
  const int64_t t = i / per;
  const int j = (int)(i - t * per) * 8;
  const bool on = t < a.T;
  float g[8] = {}, u[8] = {};
  if (on) {
    float bias[16];
    unpack_bias8(a, load_bias8(a, j), bias);
    for (int s = 0; s < a.splits; ++s) {
      const float* p = a.part + ((int64_t)s * a.T + t) * 2 * a.I + j;
      float x[8], y[8];
      load8_f32(p, x);
      load8_f32(p + a.I, y);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        g[q] += x[q];
        u[q] += y[q];
      }
    }
    finish8(a, (int)t, j, bias, g, u);
  }
  store_h8<FP8>(a, (int)t, j, on, g);
}

__global__ __launch_bounds__(256) void k_ffn_join(const JoinArgs a) {
  const int q = (int)blockIdx.x < a.first[1] ? 0 : (int)blockIdx.x < a.first[2] ? 1 : 2;
  const FfnProduct& p = a.p[q];
  const int64_t at = ((int64_t)(blockIdx.x - a.first[q]) * 256 + threadIdx.x) * 8;
  if (at >= (int64_t)p.nb * p.na) return;
  const int c = (int)(at % p.na);
  float v[8] = {};
  for (int s = 0; s < p.splits; ++s) {
    float x[8];
    load8_f32(p.part + (int64_t)s * p.nb * p.na + at, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += x[i];
  }
  if (p.bias) {
    float x[8];
    load8_bf16(p.bias + c, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += x[i];
  }
  if (p.add) {
    float x[8];
    load8_dt(p.add, p.add_dtype, at, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += x[i];
  }
  store8_dt(p.out, p.out_dtype, at, v);
}

// ------------------------------------------------------------- few tokens

// A decode step reads every weight for a handful of tokens, so the kernel is a stream of the
// weights: one workgroup takes 16 RT weight rows and its KS waves split K; each multiplies
// the RT tiles of 16 rows with NT tiles of 16 tokens on 16x16 MFMAs (weights as the first
// operand: a lane ends with 4 weight rows of one token). Loads of the next batch of steps
// (128 bytes of a row each) are in flight while one is multiplied; the partial sums meet in
// LDS, in the order of the K splits. What bounds it at these sizes is the number of load
// instructions of a CU (each touches 16 rows), so a wave keeps its tokens' operands for all
// its row tiles and asks for nothing past its range.
//
// MXFP8 operands are taken to bf16 on the way (exact) and multiplied as such: the e4m3 matrix
// instruction keeps a product only to 2^-16 of its block's largest, which sends a few more values
// of h to a neighbouring code. The loads hide most of it: 16 tokens at 2880, 2880 17.0 us with that
// instruction and 17.6 so, 2.6e-3 and 1.7e-3 off in relative 2-norm, 1.7e-3 being bf16's rounding.
template <int RT, int KS, int NT, bool FP8>
struct Skinny {
  static constexpr int kThreads = KS * 64;
  static constexpr int kLds = KS * RT * NT * 256 * 4;
  // steps of a batch: about the same registers for any shape
  static constexpr int kU = RT + NT >= 5 ? 1 : 8 / (RT + NT);

  struct Batch {
    u32x4 w[kU][RT][2], x[kU][NT][2];
    uint32_t ws[FP8 ? kU : 1][RT], xs[FP8 ? kU : 1][NT];
  };

  // row_of(rt): the weight row of this lane in row tile rt, or -1; sums in red[ks][rt][nt][256]
  template <typename RowOf>
  static __device__ __forceinline__ void run(const Operand& W, int64_t wrows, RowOf row_of,
                                             const Operand& X, int t0, int nt, int K,
                                             float* red) {
    const int ks = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id();
    const int n = l & 15, g = l >> 4;
    const int kb = FP8 ? K : 2 * K;    // bytes of a row
    const int nb = K / 32;
    const rsrc_t rw = make_rsrc_uniform(W.p, (uint32_t)(wrows * kb));
    const rsrc_t rx = make_rsrc_uniform(static_cast<const uint8_t*>(X.p) + (int64_t)t0 * kb,
                                        (uint32_t)(nt * kb));
    const rsrc_t rws = make_rsrc_uniform(W.s, FP8 ? (uint32_t)(wrows * nb) : 0u);
    const rsrc_t rxs = make_rsrc_uniform(FP8 ? X.s + (int64_t)t0 * nb : X.s,
                                         FP8 ? (uint32_t)(nt * nb) : 0u);
    uint32_t wo[RT], wso[RT], xo[NT], xso[NT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = row_of(i);
      wo[i] = r >= 0 ? (uint32_t)r * kb : (uint32_t)kOob;
      wso[i] = r >= 0 ? (uint32_t)r * nb : (uint32_t)kOob;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = 16 * i + n;
      xo[i] = t < nt ? (uint32_t)t * kb : (uint32_t)kOob;
      xso[i] = t < nt ? (uint32_t)t * nb : (uint32_t)kOob;
    }
    // a lane's two 16-byte pieces of a 128-byte step are neighbours (any split of k that both
    // operands share will do): for e4m3 they are a block with one scale
    const int p0 = 32 * g, p1 = p0 + 16;
    const int steps = (kb + 127) / 128;
    const int s0 = steps * ks / KS, s1 = steps * (ks + 1) / KS;
    auto load = [&](Batch& b, int s) {
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int k = 128 * (s + i);
        const bool in0 = s + i < s1 && k + p0 < kb, in1 = s + i < s1 && k + p1 < kb;
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          b.w[i][j][0] = buf_load_b128(rw, in0 ? (int)(wo[j] + k + p0) : kOob);
          b.w[i][j][1] = buf_load_b128(rw, in1 ? (int)(wo[j] + k + p1) : kOob);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          b.x[i][j][0] = buf_load_b128(rx, in0 ? (int)(xo[j] + k + p0) : kOob);
          b.x[i][j][1] = buf_load_b128(rx, in1 ? (int)(xo[j] + k + p1) : kOob);
        }
        if constexpr (FP8) {
          const int blk = 4 * (s + i) + g;
          const bool on = s + i < s1 && blk < nb;
#pragma unroll
          for (int j = 0; j < RT; ++j) b.ws[i][j] = buf_load_u8(rws, on ? (int)(wso[j] + blk) : kOob);
#pragma unroll
          for (int j = 0; j < NT; ++j) b.xs[i][j] = buf_load_u8(rxs, on ? (int)(xso[j] + blk) : kOob);
        }
      }
    };
    f32x4 acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // chunk c of 8 k of a step in a lane, as bf16
    constexpr int kC = FP8 ? 4 : 2;
    auto operand = [](const u32x4* v, int c, uint32_t scale) {
      if constexpr (FP8) return mx_bf16x8(v[c / 2][2 * (c % 2)], v[c / 2][2 * (c % 2) + 1], scale);
      else return __builtin_bit_cast(bf16x8, v[c]);
    };
    auto mul = [&](const Batch& b) {
#pragma unroll
      for (int i = 0; i < kU; ++i)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          bf16x8 x[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) x[j] = operand(b.x[i][j], c, b.xs[FP8 ? i : 0][j]);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const bf16x8 w = operand(b.w[i][r], c, b.ws[FP8 ? i : 0][r]);
#pragma unroll
            for (int j = 0; j < NT; ++j)
              acc[r][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[j], acc[r][j], 0, 0, 0);
          }
        }
    };
    // (a batch that follows is asked for in straight line with the one before it: behind a
    // branch of its own the compiler would wait for all loads in flight)
    Batch b0, b1;
    int s = s0;
    load(b0, s);
    for (;;) {
      if (s + kU >= s1) {
        mul(b0);
        break;
      }
      load(b1, s + kU);
      mul(b0);
      s += kU;
      if (s + kU >= s1) {
        mul(b1);
        break;
      }
      load(b0, s + kU);
      mul(b1);
      s += kU;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        *reinterpret_cast<f32x4*>(red + ((ks * RT + i) * NT + j) * 256 + l * 4) = acc[i][j];
    __syncthreads();
  }

  // sum of the K splits at weight row r (0 .. 16 RT - 1) and token m
  static __device__ __forceinline__ float sum(const float* red, int r, int m) {
    const int at = ((r >> 4) * NT + (m >> 4)) * 256 + (((r & 15) >> 2) * 16 + (m & 15)) * 4 + (r & 3);
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) v += red[k * RT * NT * 256 + at];
    return v;
  }
};

template <int RT, int KS, int NT, bool FP8>
__global__ __launch_bounds__(KS * 64) void k_ffn_gate_up_skinny(const GateUpArgs a) {
  using S = Skinny<RT, KS, NT, FP8>;
  extern __shared__ __attribute__((aligned(16))) float red[];
  constexpr int NJ = 8 * RT;   // pairs of the workgroup: gate rows first, then up rows
  const int j0 = blockIdx.x * NJ, t0 = blockIdx.y * 16 * NT, nt = min(16 * NT, a.T - t0);
  // 8 pairs of a token to a thread; NJ = 32 gives a block of MXFP8 to four neighbours
  static_assert(16 * NT * RT <= S::kThreads, "a thread for every 8 pairs");
  const int m = threadIdx.x / RT, jj = 8 * (threadIdx.x % RT);
  // what the end needs from memory is asked for first
  const RawBias raw = load_bias8(a, j0 + jj);
  S::run(
      a.W, 2 * (int64_t)a.I,
      [&](int rt) {
        const int r = 16 * rt + (lane_id() & 15), j = j0 + (r < NJ ? r : r - NJ);
        return j < a.I ? gu_col(a.layout, a.I, j, r >= NJ) : -1;
      },
      a.X, t0, nt, a.H, red);
  if (m >= 16 * NT) return;
  const bool on = m < nt && j0 + jj < a.I;
  float g[8], u[8], bias[16];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    g[q] = S::sum(red, jj + q, m);
    u[q] = S::sum(red, NJ + jj + q, m);
  }
  unpack_bias8(a, raw, bias);
  if (on) finish8(a, t0 + m, j0 + jj, bias, g, u);
  store_h8<FP8>(a, t0 + m, j0 + jj, on, g);
}

template <int RT, int KS, int NT, bool FP8>
__global__ __launch_bounds__(KS * 64) void k_ffn_down_skinny(const FfnProduct p) {
  using S = Skinny<RT, KS, NT, FP8>;
  extern __shared__ __attribute__((aligned(16))) float red[];
  const int a0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * 16 * NT, nt = min(16 * NT, p.nb - t0);
  // what the end needs from memory is asked for first: bias and addend of the thread's values
  constexpr int kAll = 16 * NT * 16 * RT, kTurns = (kAll + S::kThreads - 1) / S::kThreads;
  uint32_t bias[kTurns], add[kTurns];
  const bool add32 = p.add_dtype == MOE4_DTYPE_F32;
  auto each = [&](auto f) {
#pragma unroll
    for (int n = 0; n < kTurns; ++n) {
      const int i = n * S::kThreads + threadIdx.x, m = i / (16 * RT), c = i % (16 * RT);
      if (m < nt && a0 + c < p.na) f(n, m, c, (int64_t)(t0 + m) * p.na + a0 + c);
    }
  };
#pragma unroll
  for (int n = 0; n < kTurns; ++n) bias[n] = add[n] = 0;
  each([&](int n, int, int c, int64_t at) {
    if (p.bias) bias[n] = p.bias[a0 + c];
    if (p.add)
      add[n] = add32 ? static_cast<const uint32_t*>(p.add)[at] : static_cast<const uint16_t*>(p.add)[at];
  });
  S::run(
      p.A, p.na,
      [&](int rt) {
        const int r = a0 + 16 * rt + (lane_id() & 15);
        return r < p.na ? r : -1;
      },
      p.B, t0, nt, p.K, red);
  each([&](int n, int m, int c, int64_t at) {
    float v = S::sum(red, c, m);
    v += __uint_as_float(bias[n] << 16);
    v += __uint_as_float(add32 ? add[n] : add[n] << 16);
    if (p.out_dtype == MOE4_DTYPE_F32) static_cast<float*>(p.out)[at] = v;
    else static_cast<uint16_t*>(p.out)[at] = f32_to_bf16(v);
  });
}

// Eight waves split K. (In MXFP8, one and 16 tokens at 2880, 2880 to 4096, 8192, twelve took 1%
// longer, sixteen, with 128 registers a lane, 25 to 45%.)
//
// Row tiles of a workgroup of the bf16 kernels and of the second product: a wave's loads are 2 RT
// for weights and 2 NT for tokens a step, so more row tiles save token loads, as long as
// there is a workgroup for most CUs. Us at 16, 64 tokens, H 4096, I 8192: one row tile 60,
// 119; by this rule 51, 90.
// (Four with 64 tokens would not fit the registers.)
template <int NT, typename F>
hipError_t with_row_tiles(int64_t rows, F f) {
  if constexpr (NT < 4)
    if (rows >= 64 * 192) return f(std::integral_constant<int, 4>{});
  if (rows >= 32 * 192) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1>{});
}

template <int NT, bool FP8>
hipError_t launch_skinny(const GateUpArgs& g, const FfnProduct& d, hipStream_t s) {
  const uint32_t nt = (g.T + 16 * NT - 1) / (16 * NT);
  auto gate_up = [&](auto rc) {
    // MXFP8: h is quantised in blocks of 32, so a workgroup takes 32 pairs
    constexpr int kRt = FP8 ? 4 : decltype(rc)::value;
    using G = Skinny<kRt, 8, NT, FP8>;
    auto* k = &k_ffn_gate_up_skinny<kRt, 8, NT, FP8>;
    hipError_t e = allow_lds(k, G::kLds);
    if (e != hipSuccess) return e;
    k<<<dim3((g.I + 8 * kRt - 1) / (8 * kRt), nt), G::kThreads, G::kLds, s>>>(g);
    return hipGetLastError();
  };
  hipError_t e;
  if constexpr (FP8) e = gate_up(std::integral_constant<int, 4>{});
  else e = with_row_tiles<NT>(2 * (int64_t)g.I, gate_up);
  if (e != hipSuccess) return e;
  return with_row_tiles<NT>(d.na, [&](auto rc) {
    constexpr int kRt = decltype(rc)::value;
    using D = Skinny<kRt, 8, NT, FP8>;
    auto* k = &k_ffn_down_skinny<kRt, 8, NT, FP8>;
    hipError_t r = allow_lds(k, D::kLds);
    if (r != hipSuccess) return r;
    k<<<dim3((d.na + 16 * kRt - 1) / (16 * kRt), nt), D::kThreads, D::kLds, s>>>(d);
    return hipGetLastError();
  });
}

template <typename S, bool FP8>
hipError_t launch_gate_up(const GateUpArgs& g, hipStream_t s) {
  return with_kind(g.layout, g.act.act, [&](auto l, auto c) {
    auto* k = &k_ffn_gate_up<S, FP8, decltype(l)::value, decltype(c)::value>;
    constexpr int kBytes = FP8 ? S::kLdsMx : S::kLds;
    hipError_t e = allow_lds(k, kBytes);
    if (e != hipSuccess) return e;
    k<<<(uint32_t)(tiles_of<S>(2 * (int64_t)g.I, g.T) * g.splits), S::kThreads, kBytes, s>>>(g);
    return hipGetLastError();
  });
}

template <bool FP8>
hipError_t launch_forward(const GateUpArgs& g, const FfnProduct& d, int variant, hipStream_t s) {
  if (variant == MOE4_VARIANT_SKINNY) {
    if (g.T <= 16) return launch_skinny<1, FP8>(g, d, s);
    if constexpr (FP8) return launch_skinny<2, FP8>(g, d, s);
    else return g.T <= 32 ? launch_skinny<2, FP8>(g, d, s) : launch_skinny<4, FP8>(g, d, s);
  }
  hipError_t e;
  if (g.splits > 1) {
    e = launch_gate_up<Tile128, FP8>(g, s);
    if (e != hipSuccess) return e;
    k_ffn_gate_up_join<FP8><<<(uint32_t)(((int64_t)g.T * (g.I / 8) + 255) / 256), 256, 0, s>>>(g);
    e = hipGetLastError();
  } else {
    e = large_tiles_for(2 * (int64_t)g.I, g.T) ? launch_gate_up<Tile256, FP8>(g, s)
                                               : launch_gate_up<Tile128, FP8>(g, s);
  }
  if (e != hipSuccess) return e;
  if (d.splits > 1) {
    e = launch_product<Tile128, kOpRow, kOpRow, FP8>(d, s);
    if (e != hipSuccess) return e;
    JoinArgs j = {};
    j.p[0] = d;
    return launch_join(j, 1, s);
  }
  return large_tiles_for(d.na, d.nb) ? launch_product<Tile256, kOpRow, kOpRow, FP8>(d, s)
                                     : launch_product<Tile128, kOpRow, kOpRow, FP8>(d, s);
}

}  // namespace

hipError_t launch_join(JoinArgs a, int n, hipStream_t s) {
  a.first[0] = 0;
  for (int i = 0; i < 3; ++i)
    a.first[i + 1] =
        a.first[i] + (i < n ? (int)(((int64_t)a.p[i].nb * a.p[i].na / 8 + 255) / 256) : 0);
  k_ffn_join<<<a.first[3], 256, 0, s>>>(a);
  return hipGetLastError();
}

namespace {

// workspace: h (and its scales), the partial sums of a product that is split along k (the two
// products' follow each other in time and share the place). It does not fall as T grows.
struct FwdWs {
  int gate_splits, down_splits;
  size_t scales, part, end;
  FwdWs(const moe4_ffn& f, int64_t T) {
    const bool mx = f.format == MOE4_FFN_MXFP8;
    const int es = mx ? 1 : 2;
    // (for either variant: the size does not change with the one that is pinned)
    gate_splits = T > 0 ? k_splits(tiles_of<Tile128>(2 * (int64_t)f.I, T), f.H, es) : 1;
    down_splits = T > 0 ? k_splits(tiles_of<Tile128>(f.H, T), f.I, es) : 1;
    scales = align_up((size_t)T * f.I * es, 256);
    part = scales + (mx ? align_up((size_t)T * (f.I / 32), 256) : 0);
    const int64_t g = part_bytes(2 * (int64_t)f.I, T, most_k_splits(2 * (int64_t)f.I, f.H, es));
    const int64_t d = part_bytes(f.H, T, most_k_splits(f.H, f.I, es));
    end = part + align_up((size_t)(g > d ? g : d), 256);
  }
};

}  // namespace

size_t ffn_forward_ws_bytes(const moe4_ffn& f, int64_t T) { return FwdWs(f, T).end; }

int ffn_variant(const moe4_ffn& f, int64_t T) {
  if (f.variant != MOE4_VARIANT_AUTO) return f.variant;
  // The skinny kernels read the weights once for every 64 tokens (MXFP8: 32), mostly from the
  // caches, the tiled ones pay two or three launches of long tiles. Us, skinny and tiled, in
  // bf16: 128 tokens at H 2048, I 768 (18.9 MB read) 18 and 24, 256 32 and 26; 256 at 512, 512 (6.3
  // MB) 10 and 17, 1024 (25 MB) 24 and 18; 128 at 2880, 2880 (100 MB) 70 and 36. MXFP8: 32 at 2880,
  // 2880 18 and 25, 64 (50 MB) 27 and 28, 128 44 and 34; 128 at 1024, 1024 (12.6 MB) 13 and 18,
  // 512 (50 MB) 31 and 19; 32 at H 4096, I 8192 40 and 36. Small weights and many tokens are
  // bound by the workgroups' number instead: at 64, 64 4096 tokens 9.0 and 10.2 (MXFP8 11.3 and
  // 11.5), 16384 25 and 11 (37 and 12).
  const bool mx = f.format == MOE4_FFN_MXFP8;
  const int64_t weights = 3 * (int64_t)f.H * f.I * (mx ? 1 : 2), at_once = mx ? 32 : 64;
  return T <= 32 || (T <= 4096 && (T + at_once - 1) / at_once * weights <= 20 << 20)
             ? MOE4_VARIANT_SKINNY
             : MOE4_VARIANT_TILED;
}

hipError_t launch_ffn_forward(const moe4_ffn& f, const void* x, const uint8_t* x_s, int T,
                              const void* residual, int residual_dtype, void* out,
                              int out_dtype, float* save_gu, void* ws, int* variant,
                              hipStream_t s) {
  const bool mx = f.format == MOE4_FFN_MXFP8;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  const FwdWs at(f, T);
  float* part = reinterpret_cast<float*>(w8 + at.part);
  GateUpArgs g = {};
  g.splits = at.gate_splits;
  g.part = part;
  g.W = {f.w_gu, f.gu_s, f.H, 2 * f.I};
  g.X = {x, x_s, f.H, T};
  g.w_s = (int64_t)2 * f.I * (f.H / 32);
  g.x_s = (int64_t)T * (f.H / 32);
  g.T = T;
  g.H = f.H;
  g.I = f.I;
  g.layout = f.gu_layout;
  g.act = {f.act, f.act_alpha, f.act_limit};
  g.bias = f.gu_bias;
  g.save_gu = save_gu;
  if (mx) {
    g.hq = w8;
    g.hs = w8 + at.scales;
  } else {
    g.h = reinterpret_cast<uint16_t*>(w8);
  }
  FfnProduct d = {};
  d.A = {f.w_dn, f.dn_s, f.I, f.H};
  d.B = {ws, g.hs, f.I, T};
  d.na_s = (int64_t)f.H * (f.I / 32);
  d.nb_s = (int64_t)T * (f.I / 32);
  d.K = f.I;
  d.na = f.H;
  d.nb = T;
  d.bias = f.dn_bias;
  d.add = residual;
  d.add_dtype = residual_dtype;
  d.out = out;
  d.out_dtype = out_dtype;
  d.splits = at.down_splits;
  d.part = part;
  *variant = ffn_variant(f, T);
  return mx ? launch_forward<true>(g, d, *variant, s) : launch_forward<false>(g, d, *variant, s);
}

}  // namespace moe4
