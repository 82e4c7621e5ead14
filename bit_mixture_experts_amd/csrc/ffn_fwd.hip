// Forward of the dense gated feed-forward block (the shared expert beside the routed ones):
//   gu = x W_gu^T + b_gu;  h = act(gate, up);  out = h W_dn^T + b_dn + residual
// on bf16 weights and activations, or on MXFP8 ones (h is then quantised to MXFP8 between the
// two products). Two launches: both projections with the activation, then the second product
// with its bias and residual.
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
};

// element of row t of save_gu that pair j's gate (or, with `up`, up) value has
__device__ __forceinline__ int gu_col(int layout, int I, int j, bool up) {
  return layout == MOE4_GU_HALVES ? (up ? I + j : j) : 2 * j + (up ? 1 : 0);
}

// the biases of 8 pairs j .. j+7: gates, then ups; zeros without
__device__ __forceinline__ void load_bias8(const GateUpArgs& a, int j, float* b) {
#pragma unroll
  for (int i = 0; i < 16; ++i) b[i] = 0.0f;
  if (!a.bias || j >= a.I) return;
  if (a.layout == MOE4_GU_HALVES) {
    load8_bf16(a.bias + j, b);
    load8_bf16(a.bias + a.I + j, b + 8);
  } else {
    float x[16];
    load8_bf16(a.bias + 2 * j, x);
    load8_bf16(a.bias + 2 * j + 8, x + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      b[i] = x[2 * i];
      b[8 + i] = x[2 * i + 1];
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
  tile_of(xcd_remap(blockIdx.x, gridDim.x), na, nb, ia, ib);
  const int j0 = ia * kPairs, t0 = ib * S::BB;
  const int nt = min(S::BB, a.T - t0);
  OpLoader<S, kOpRow, S::BA, FP8> la;
  OpLoader<S, kOpRow, S::BB, FP8> lb;
  la.init_row(a.W, es, a.H, 0, 2 * a.I, [&](int r) { return pair_row(a.layout, a.I, j0, r); });
  lb.init_row(a.X, es, a.H, t0, nt, [=](int r) { return r < nt ? r : -1; });
  MxState<FP8> mx;
  if constexpr (FP8) mx = {a.W.s, a.X.s, a.w_s, a.x_s};
  f32x16 acc[S::TA][S::TB];
  gemm_loop<S, kOpRow, kOpRow, FP8>(
      acc, stage_mem, la, lb, a.H, mx, [&](int r) { return pair_row(a.layout, a.I, j0, r); },
      [&](int r) { return r < nt ? t0 + r : -1; });
  float bias[16];   // the same pairs in every turn
  load_bias8(a, j0 + lane_a<S, true>(), bias);
  for_each8<S, true, 1>(acc, stage_mem, [](int, int) { return NoPre{}; },
                        [&](int row, int jj, float* g, float* u) {
    const int t = t0 + row, j = j0 + jj;
    const bool on = row < nt && j < a.I;
    if (on) finish8(a, t, j, bias, g, u);
    store_h8<FP8>(a, t, j, on, g);
  });
}

// ------------------------------------------------------------- few tokens

// A decode step reads every weight for a handful of tokens, so the kernel is a stream of the
// weights: one workgroup takes 16 RT weight rows, its KS groups of RT waves split K, and each
// wave multiplies its 16 rows with NT tiles of 16 tokens on 16x16 MFMAs (weights as the first
// operand: a lane ends with 4 weight rows of one token). Loads of the next batch of steps
// (128 bytes of a row each) are in flight while one is multiplied; the partial sums meet in
// LDS, in the order of the K splits.
template <int RT, int KS, int NT, bool FP8>
struct Skinny {
  static constexpr int kThreads = RT * KS * 64;
  static constexpr int kLds = KS * RT * NT * 256 * 4;
  static constexpr int kU = 4 / NT;   // steps of a batch: the same registers for any NT

  struct Batch {
    u32x4 w[kU][2], x[kU][NT][2];
    uint32_t ws[FP8 ? kU : 1], xs[FP8 ? kU : 1][NT];
  };

  // row: the lane's weight row or -1; sums in red[ks][rt][nt][256]
  static __device__ __forceinline__ void run(const Operand& W, int64_t wrows, int row,
                                             const Operand& X, int t0, int nt, int K,
                                             float* red) {
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id();
    const int rt = w % RT, ks = w / RT, n = l & 15, g = l >> 4;
    const int kb = FP8 ? K : 2 * K;    // bytes of a row
    const int nb = K / 32;
    const rsrc_t rw = make_rsrc_uniform(W.p, (uint32_t)(wrows * kb));
    const rsrc_t rx = make_rsrc_uniform(static_cast<const uint8_t*>(X.p) + (int64_t)t0 * kb,
                                        (uint32_t)(nt * kb));
    const rsrc_t rws = make_rsrc_uniform(W.s, FP8 ? (uint32_t)(wrows * nb) : 0u);
    const rsrc_t rxs = make_rsrc_uniform(FP8 ? X.s + (int64_t)t0 * nb : X.s,
                                         FP8 ? (uint32_t)(nt * nb) : 0u);
    const uint32_t wo = row >= 0 ? (uint32_t)row * kb : (uint32_t)kOob;
    const uint32_t wso = row >= 0 ? (uint32_t)row * nb : (uint32_t)kOob;
    uint32_t xo[NT], xso[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = 16 * i + n;
      xo[i] = t < nt ? (uint32_t)t * kb : (uint32_t)kOob;
      xso[i] = t < nt ? (uint32_t)t * nb : (uint32_t)kOob;
    }
    // the lane's two 16-byte pieces of a 128-byte step: neighbours for bf16 (any split of k
    // that both operands share will do), k = 64 c + 16 g for e4m3, where the scales fix it
    const int p0 = FP8 ? 16 * g : 32 * g, p1 = p0 + (FP8 ? 64 : 16);
    const int steps = (kb + 127) / 128;
    const int s0 = steps * ks / KS, s1 = steps * (ks + 1) / KS;
    auto load = [&](Batch& b, int s) {
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int k = 128 * (s + i);
        const bool in0 = s + i < s1 && k + p0 < kb, in1 = s + i < s1 && k + p1 < kb;
        b.w[i][0] = buf_load_b128(rw, in0 ? (int)(wo + k + p0) : kOob);
        b.w[i][1] = buf_load_b128(rw, in1 ? (int)(wo + k + p1) : kOob);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          b.x[i][j][0] = buf_load_b128(rx, in0 ? (int)(xo[j] + k + p0) : kOob);
          b.x[i][j][1] = buf_load_b128(rx, in1 ? (int)(xo[j] + k + p1) : kOob);
        }
        if constexpr (FP8) {
          const int blk = 4 * (s + i) + g;
          const bool on = s + i < s1 && blk < nb;
          b.ws[i] = buf_load_u8(rws, on ? (int)(wso + blk) : kOob);
#pragma unroll
          for (int j = 0; j < NT; ++j) b.xs[i][j] = buf_load_u8(rxs, on ? (int)(xso[j] + blk) : kOob);
        }
      }
    };
    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto join = [](u32x4 lo, u32x4 hi) {
      const auto v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(i32x8, v);
    };
    auto mul = [&](const Batch& b) {
#pragma unroll
      for (int i = 0; i < kU; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (FP8) {
            acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                join(b.w[i][0], b.w[i][1]), join(b.x[i][j][0], b.x[i][j][1]), acc[j], 0, 0, 0,
                (int)b.ws[i], 0, (int)b.xs[i][j]);
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, b.w[i][c]), __builtin_bit_cast(bf16x8, b.x[i][j][c]),
                  acc[j], 0, 0, 0);
          }
        }
    };
    // steps past s1 load zeros
    Batch b0, b1;
    load(b0, s0);
    for (int s = s0; s < s1; s += 2 * kU) {
      load(b1, s + kU);
      mul(b0);
      load(b0, s + 2 * kU);
      mul(b1);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<f32x4*>(red + ((ks * RT + rt) * NT + j) * 256 + l * 4) = acc[j];
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
__global__ __launch_bounds__(RT * KS * 64) void k_ffn_gate_up_skinny(const GateUpArgs a) {
  using S = Skinny<RT, KS, NT, FP8>;
  extern __shared__ __attribute__((aligned(16))) float red[];
  constexpr int NJ = 8 * RT;   // pairs of the workgroup: gate rows first, then up rows
  const int j0 = blockIdx.x * NJ, t0 = blockIdx.y * 16 * NT, nt = min(16 * NT, a.T - t0);
  const int r = 16 * (wave_id() % RT) + (lane_id() & 15);
  const int jr = j0 + (r < NJ ? r : r - NJ);
  S::run(a.W, 2 * (int64_t)a.I, jr < a.I ? gu_col(a.layout, a.I, jr, r >= NJ) : -1, a.X, t0, nt,
         a.H, red);
  // 8 pairs of a token to a thread; NJ = 32 gives a block of MXFP8 to four neighbours
  for (int i = threadIdx.x; i < 16 * NT * RT; i += S::kThreads) {
    const int m = i / RT, jj = 8 * (i % RT);
    const bool on = m < nt && j0 + jj < a.I;
    float g[8], u[8], bias[16];
    load_bias8(a, j0 + jj, bias);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      g[q] = S::sum(red, jj + q, m);
      u[q] = S::sum(red, NJ + jj + q, m);
    }
    if (on) finish8(a, t0 + m, j0 + jj, bias, g, u);
    store_h8<FP8>(a, t0 + m, j0 + jj, on, g);
  }
}

template <int RT, int KS, int NT, bool FP8>
__global__ __launch_bounds__(RT * KS * 64) void k_ffn_down_skinny(const FfnProduct p) {
  using S = Skinny<RT, KS, NT, FP8>;
  extern __shared__ __attribute__((aligned(16))) float red[];
  const int a0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * 16 * NT, nt = min(16 * NT, p.nb - t0);
  const int r = a0 + 16 * (wave_id() % RT) + (lane_id() & 15);
  S::run(p.A, p.na, r < p.na ? r : -1, p.B, t0, nt, p.K, red);
  for (int i = threadIdx.x; i < 16 * NT * 16 * RT; i += S::kThreads) {
    const int m = i / (16 * RT), c = i % (16 * RT);
    if (m >= nt || a0 + c >= p.na) continue;
    const int64_t at = (int64_t)(t0 + m) * p.na + a0 + c;
    float v = S::sum(red, c, m);
    if (p.bias) v += bf16_to_f32(p.bias[a0 + c]);
    if (p.add)
      v += p.add_dtype == MOE4_DTYPE_F32 ? static_cast<const float*>(p.add)[at]
                                         : bf16_to_f32(static_cast<const uint16_t*>(p.add)[at]);
    if (p.out_dtype == MOE4_DTYPE_F32) static_cast<float*>(p.out)[at] = v;
    else static_cast<uint16_t*>(p.out)[at] = f32_to_bf16(v);
  }
}

template <int NT, bool FP8>
hipError_t launch_skinny(const GateUpArgs& g, const FfnProduct& d, hipStream_t s) {
  constexpr int kRt = FP8 ? 4 : 1, kKs = !FP8 ? 8 : NT == 1 ? 4 : 2;
  using G = Skinny<kRt, kKs, NT, FP8>;
  using D = Skinny<1, 8, NT, FP8>;
  const uint32_t nt = (g.T + 16 * NT - 1) / (16 * NT);
  k_ffn_gate_up_skinny<kRt, kKs, NT, FP8>
      <<<dim3((g.I + 8 * kRt - 1) / (8 * kRt), nt), G::kThreads, G::kLds, s>>>(g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_ffn_down_skinny<1, 8, NT, FP8><<<dim3((d.na + 15) / 16, nt), D::kThreads, D::kLds, s>>>(d);
  return hipGetLastError();
}

template <typename S, bool FP8>
hipError_t launch_tiled(const GateUpArgs& g, const FfnProduct& d, hipStream_t s) {
  const int64_t n = (int64_t)((g.I + S::BA / 2 - 1) / (S::BA / 2)) * ((g.T + S::BB - 1) / S::BB);
  hipError_t e = with_kind(g.layout, g.act.act, [&](auto l, auto c) {
    auto* k = &k_ffn_gate_up<S, FP8, decltype(l)::value, decltype(c)::value>;
    constexpr int kBytes = FP8 ? S::kLdsMx : S::kLds;
    hipError_t r = allow_lds(k, kBytes);
    if (r != hipSuccess) return r;
    k<<<(uint32_t)n, S::kThreads, kBytes, s>>>(g);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  return launch_product<S, kOpRow, kOpRow, FP8>(d, s);
}

template <bool FP8>
hipError_t launch_forward(const GateUpArgs& g, const FfnProduct& d, int variant, hipStream_t s) {
  if (variant == MOE4_VARIANT_SKINNY) {
    if (g.T <= 16) return launch_skinny<1, FP8>(g, d, s);
    if (g.T <= 32) return launch_skinny<2, FP8>(g, d, s);
    return launch_skinny<4, FP8>(g, d, s);
  }
  const int64_t big = (int64_t)((g.I + 127) / 128) * ((g.T + 255) / 256);
  if (big >= 192) return launch_tiled<Tile256, FP8>(g, d, s);
  return launch_tiled<Tile128, FP8>(g, d, s);
}

}  // namespace

size_t ffn_forward_ws_bytes(const moe4_ffn& f, int64_t T) {
  if (f.format == MOE4_FFN_MXFP8)
    return align_up((size_t)T * f.I, 256) + align_up((size_t)T * (f.I / 32), 256);
  return align_up((size_t)T * f.I * 2, 256);
}

int ffn_variant(const moe4_ffn& f, int64_t T) {
  if (f.variant != MOE4_VARIANT_AUTO) return f.variant;
  return T <= 64 ? MOE4_VARIANT_SKINNY : MOE4_VARIANT_TILED;
}

hipError_t launch_ffn_forward(const moe4_ffn& f, const void* x, const uint8_t* x_s, int T,
                              const void* residual, int residual_dtype, void* out,
                              int out_dtype, float* save_gu, void* ws, int* variant,
                              hipStream_t s) {
  const bool mx = f.format == MOE4_FFN_MXFP8;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  GateUpArgs g = {};
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
    g.hs = w8 + align_up((size_t)T * f.I, 256);
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
  *variant = ffn_variant(f, T);
  return mx ? launch_forward<true>(g, d, *variant, s) : launch_forward<false>(g, d, *variant, s);
}

}  // namespace moe4
