// The dense product with an MXFP4 weight, y = x W^T + bias + residual, on bf16, MXFP8 or MXFP4
// activations, and its input gradient dx = dY W.
//
// Many tokens: tiles as in dense_gemm.hpp (256 x 256, 256 x 128 or 128 x 64), the weight
// as the matrix instruction's first operand.
//   * MXFP8 and MXFP4 activations: the scaled e2m1 instructions on the codes as they are, 64 k a
//     step.
//   * bf16 activations: a lane reads 16 bytes of codes, one block, as the operands of the four
//     16-k steps of a k-tile (which k a step takes is free as long as both operands agree), and
//     converts them in registers while the matrix cores are busy: four conversions for two MFMAs
//     of 32 cycles each.
//   * dx: the reduction runs over the weight's rows, so the codes are converted once, by the thread
//     that loads them, and written to LDS as bf16 in the layout of the transposing reads.
// Few tokens: the weight is streamed once, K split over the waves of a workgroup.
#include <algorithm>

#include "ffn.hpp"

namespace moe4 {
namespace {

constexpr int kXB = MOE4_X_BF16, kX8 = MOE4_X_MXFP8, kX4 = MOE4_X_MXFP4;

// k runs in turns of 256: 128 bytes, a whole line, and eight scales of every row of the weight, which
// travel together; a k-tile is 128 bytes of a row of activations. (With the weight's 32 bytes of a
// k-tile loaded for each, 2048 tokens bf16 at 4096 took 68 us: lines were asked for four times.)
template <int XF>
struct LinK {
  static constexpr int kTile = XF == kXB ? 64 : XF == kX8 ? 128 : 256;   // k of a k-tile
  static constexpr int kSub = 256 / kTile;                               // k-tiles of a turn
  static constexpr int kSteps = XF == kX8 ? 2 : 4;
  // bytes of k values of a row of activations
  static __host__ __device__ constexpr int64_t bytes(int64_t k) { return k * 128 / kTile; }
};

// The scales of a turn, eight bytes for each row of the tile, through LDS: thread t of the workgroup
// reads those of tile row t (A's rows, then B's), of two turns at a time (rows are far apart, so that
// a load of few bytes moves as much as one of 16; 8192 MXFP4 tokens at N 8192, K 4096 took 187 us with
// a load for every turn, 170 so). Rows start at any byte, so the aligned dwords around them are
// loaded and shifted. Blocks past K take scale 0: the bytes there belong to the next row and may be
// e8m0 NaNs.
template <typename S>
struct TurnScales {
  static constexpr int kRows = (S::BA + S::BB + S::kThreads - 1) / S::kThreads;   // of a thread, kThreads apart
  static constexpr int kBytes = kRows * S::kThreads * 8;
  rsrc_t r[kRows];
  int nb;
  uint32_t off[kRows];
  u32x4 raw[kRows];
  uint32_t more[kRows];
  bool shifted;   // some row does not begin at a dword
  template <typename RowA, typename RowB>
  __device__ __forceinline__ void init(const MxScales& m, int blocks, RowA row_a, RowB row_b) {
    nb = blocks;
    shifted = m.pitch & 3;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      more[i] = 0;
      const int t = threadIdx.x + i * S::kThreads;
      // whole waves belong to one operand
      const bool is_a = __builtin_amdgcn_readfirstlane(wave_id()) * 64 + i * S::kThreads < S::BA;
      r[i] = make_rsrc_uniform(is_a ? m.sa : m.sb, (uint32_t)(((is_a ? m.na : m.nb) + 3) & ~(int64_t)3));
      const int row = is_a ? row_a(t) : t - S::BA < S::BB ? row_b(t - S::BA) : -1;
      off[i] = row >= 0 ? (uint32_t)row * m.pitch + m.first : (uint32_t)kOob;
    }
  }
  // of turns 2 pair and 2 pair + 1
  __device__ __forceinline__ void load(int pair) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int at = (int)((off[i] & ~3u) + 16 * pair);
      raw[i] = buf_load_b128(r[i], at);
      if (shifted) more[i] = buf_load_b32(r[i], offset_past(at, 16));
    }
  }
  __device__ __forceinline__ void store(int turn, uint8_t* lds) const {
    const int left = nb - 8 * turn;   // blocks of this turn
    const bool odd = turn & 1;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t sh = off[i] & 3;
      const uint32_t d0 = odd ? raw[i][2] : raw[i][0], d1 = odd ? raw[i][3] : raw[i][1], d2 = odd ? more[i] : raw[i][2];
      u32x2 v = {__builtin_amdgcn_alignbyte(d1, d0, sh), __builtin_amdgcn_alignbyte(d2, d1, sh)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = left - 4 * h;
        v[h] &= n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1;
      }
      reinterpret_cast<u32x2*>(lds)[threadIdx.x + i * S::kThreads] = v;
    }
  }
  // of a tile row: the bytes of the lane's half in the turn's four 64-k units
  static __device__ __forceinline__ uint32_t get(const uint8_t* lds, int row) {
    const u32x2 v = reinterpret_cast<const u32x2*>(lds)[row];
    return __builtin_amdgcn_perm(v[1], v[0], lane_id() & 32 ? 0x07050301u : 0x06040200u);
  }
};

__device__ __forceinline__ i32x8 widen(i32x4 v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }

// one 64-k MFMA of a weight operand (e2m1) with activations in e4m3 or e2m1; the scales are byte
// `unit` (a constant once the loops are unrolled) of sa and sb
template <int XF, typename FB>
__device__ __forceinline__ f32x16 mfma_scaled(i32x4 a, FB b, f32x16 c, int unit, uint32_t sa, uint32_t sb) {
  constexpr int kB = XF == kX8 ? 0 : 4;
  i32x8 bw;
  if constexpr (XF == kX8) bw = b;
  else bw = widen(b);
  switch (unit) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), bw, c, 4, kB, 0, (int)sa, 0, (int)sb);
    case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), bw, c, 4, kB, 1, (int)sa, 1, (int)sb);
    case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), bw, c, 4, kB, 2, (int)sa, 2, (int)sb);
    default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), bw, c, 4, kB, 3, (int)sa, 3, (int)sb);
  }
}

template <typename S>
using WLoader = Loader<kOpRow, S::BA, S::kThreads, 128>;
template <typename S>
using XLoader = Loader<kOpRow, S::BB, S::kThreads, 128>;

// LDS: two turns of the weight, two or four k-tiles of activations (the epilogue stages its tile there
// too), two turns of scales
template <typename S, int XF>
struct LinLds {
  static constexpr int kA = S::BA * 128, kB = S::BB * 128;
  static constexpr int kStages = S::BB == 256 || XF == kX4 ? 2 : 4;   // of activations
  static constexpr int kScales = 2 * kA + kStages * kB;
  static_assert(kScales >= S::kLds, "the epilogue's staging fits");
  static constexpr int kBytes = kScales + 2 * TurnScales<S>::kBytes;
};

// The k loop: acc += W x^T. Loads go out between the MFMAs, all of a stage's behind the barrier that
// frees it (8192 MXFP8 tokens at 4096 139 us, and 151 with half of them at the beginning of the next
// k-tile; bf16 in four stages the other way round, 61 and 60, and so); the operands of a step are read
// from LDS while the step before multiplies.
template <typename S, int XF, typename RowA, typename RowB>
__device__ __forceinline__ void lin_loop(f32x16 (&acc)[S::TA][S::TB], uint8_t* lds, const WLoader<S>& la,
                                         const XLoader<S>& lb, int K, const MxScales& mx, RowA row_a,
                                         RowB row_b) {
  using P = LinK<XF>;
  using M = LinLds<S, XF>;
  constexpr int kSub = P::kSub, kSteps = P::kSteps, kN = M::kStages;
  constexpr int kEarly = XF == kXB && kN > 2 ? 4 : 8;   // 8ths of a stage's loads behind the barrier
  uint8_t* const ldb = lds + 2 * M::kA;
  const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id();
  const int wa = w % S::WA, wb = w / S::WA, r = l & 31, half = l >> 5;
  const int turns = (K + 255) / 256;
  // first byte of the lane's rows, and what their chunks' places are swizzled by
  const int arow = (wa * S::TA * 32 + r) * 128, brow = (wb * S::TB * 32 + r) * 128, key = (r >> 1) & 7;
  // weights: 16 bytes of step s of the turn's k-tile h (bf16: of the whole k-tile)
  auto read_a = [&](const uint8_t* st, int t, int h, int s) {
    const int chunk = XF == kXB ? 2 * h + half : 2 * (kSteps * h + s) + half;
    return *reinterpret_cast<const i32x4*>(st + arow + t * 32 * 128 + ((chunk ^ key) * 16));
  };
  using FB = std::conditional_t<XF == kX8, i32x8, i32x4>;
  auto read_b = [&](const uint8_t* st, int t, int s) {
    const uint8_t* p = st + brow + t * 32 * 128;
    auto chunk = [&](int c) { return *reinterpret_cast<const i32x4*>(p + ((c ^ key) * 16)); };
    if constexpr (XF == kXB) return chunk(4 * half + s);      // 8 k of the half's block
    else if constexpr (XF == kX4) return chunk(2 * s + half);  // 32 k
    else   // k = 32 c + 16 half .. + 15 in the c-th 16 bytes
      return __builtin_shufflevector(chunk(4 * s + half), chunk(4 * s + 2 + half), 0, 1, 2, 3, 4, 5, 6, 7);
  };
  i32x4 fa[S::TA];
  FB fb[2][S::TB];
  TurnScales<S> sc;
  uint8_t* const sclds = lds + M::kScales;
  uint32_t xa[S::TA], xb[S::TB], na[S::TA], nb[S::TB];
  auto next_scales = [&](int turn) {
    const uint8_t* p = sclds + (turn & 1) * TurnScales<S>::kBytes;
#pragma unroll
    for (int t = 0; t < S::TA; ++t) na[t] = sc.get(p, (wa * S::TA + t) * 32 + r);
    if constexpr (XF != kXB) {
#pragma unroll
      for (int u = 0; u < S::TB; ++u) nb[u] = sc.get(p, S::BA + (wb * S::TB + u) * 32 + r);
    }
  };
  // loads [n0, n1) of 8ths of a turn of weights, of a k-tile of activations
  constexpr int kLa = WLoader<S>::kLoads, kLb = XLoader<S>::kLoads;
  auto issue_a = [&](int turn, int n0, int n1) {
#pragma unroll
    for (int i = kLa * n0 / 8; i < kLa * n1 / 8; ++i) la.template issue<false>(turn, i, lds + (turn & 1) * M::kA);
  };
  auto issue_b = [&](int kt, int n0, int n1, uint8_t* st) {
#pragma unroll
    for (int i = kLb * n0 / 8; i < kLb * n1 / 8; ++i) lb.template issue<false>(kt, i, st);
  };
#pragma unroll
  for (int i = 0; i < S::TA; ++i)
#pragma unroll
    for (int j = 0; j < S::TB; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

  sc.init(mx, K / 32, row_a, row_b);
  sc.load(0);
  issue_a(0, 0, 8);
  issue_b(0, 0, 8, ldb);
  issue_a(1, 0, kEarly);
#pragma unroll
  for (int i = 1; i < kN; ++i) issue_b(i, 0, i < kN - 1 ? 8 : kEarly, ldb + i * M::kB);
  wait_vmcnt<kLa * kEarly / 8 + (kN - 2) * kLb + kLb * kEarly / 8>();
  sc.store(0, sclds);
  wait_lgkm0();
  lds_barrier();
  next_scales(0);
#pragma unroll
  for (int t = 0; t < S::TA; ++t) fa[t] = read_a(lds, t, 0, 0);
#pragma unroll
  for (int t = 0; t < S::TB; ++t) fb[0][t] = read_b(ldb, t, 0);
  int at_cur = 0, at_prev = (kN - 1) * M::kB;   // this k-tile's stage, and the one before
  for (int kp = 0; kp < turns; ++kp) {
#pragma unroll
    for (int t = 0; t < S::TA; ++t) xa[t] = na[t];
    if constexpr (XF != kXB) {
#pragma unroll
      for (int u = 0; u < S::TB; ++u) xb[u] = nb[u];
    }
    sc.store(kp + 1, sclds + ((kp + 1) & 1) * TurnScales<S>::kBytes);
    if (!(kp & 1)) sc.load(kp / 2 + 1);
    const uint8_t* const cur_a = lds + (kp & 1) * M::kA;
    const uint8_t* const nxt_a = lds + ((kp + 1) & 1) * M::kA;
#pragma unroll
    for (int h = 0; h < kSub; ++h) {
      const int kt = kp * kSub + h, at_nxt = at_cur == (kN - 1) * M::kB ? 0 : at_cur + M::kB;
      uint8_t *const cur = ldb + at_cur, *const nxt = ldb + at_nxt, *const prev = ldb + at_prev;
      at_prev = at_cur;
      at_cur = at_nxt;
      const bool end = h == kSub - 1;   // of the turn
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const bool last = s == kSteps - 1;
        const int sn = (s + 1) % kSteps, hn = last ? (h + 1) % kSub : h;
        const uint8_t* from = last ? nxt : cur;
        const uint8_t* from_a = last && end ? nxt_a : cur_a;
        if (last) {
          // the tile's barrier: the wave's loads of the next tile have landed, its reads of this one
          // are done, and so are the others'
          // (activations of kN - 2 tiles more may be in flight, at a turn's end those asked for after the
          // next turn's weights)
          if (end) wait_vmcnt<(kN - 2 < kSub - 1 ? kN - 2 : kSub - 1) * kLb>();
          else wait_vmcnt<(kN - 2) * kLb>();
          wait_lgkm0();
          lds_barrier();
          if (end) next_scales(kp + 1);
        }
        // (past the last tile: stale values, read and never used)
#pragma unroll
        for (int u = 0; u < S::TB; ++u) fb[(s + 1) & 1][u] = read_b(from, u, sn);
        const int unit = XF == kXB ? h : h * kSteps + s;   // of the turn's four 64-k units
        bf16x8 ahead;
        auto convert = [&](int t) {
          return __builtin_bit_cast(bf16x8, mx4_bf16x8((uint32_t)fa[t][s], xa[t] >> (8 * unit) & 255u));
        };
        if constexpr (XF == kXB) ahead = convert(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < S::TA; ++t) {
          if constexpr (XF == kXB) {
            const bf16x8 a = ahead;
            if (t + 1 < S::TA) ahead = convert(t + 1);
#pragma unroll
            for (int u = 0; u < S::TB; ++u)
              acc[t][u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, __builtin_bit_cast(bf16x8, fb[s & 1][u]),
                                                                  acc[t][u], 0, 0, 0);
            if (last) fa[t] = read_a(from_a, t, hn, 0);
          } else {
#pragma unroll
            for (int u = 0; u < S::TB; ++u)
              acc[t][u] = mfma_scaled<XF>(fa[t], fb[s & 1][u], acc[t][u], unit, xa[t], xb[u]);
            fa[t] = read_a(from_a, t, hn, sn);
          }
          const int n0 = kEarly * t / S::TA, n1 = kEarly * (t + 1) / S::TA;
          const int m0 = kEarly + (8 - kEarly) * t / S::TA, m1 = kEarly + (8 - kEarly) * (t + 1) / S::TA;
          if (last) {
            issue_b(kt + kN, n0, n1, cur);
            if (end) issue_a(kp + 2, n0, n1);
          }
          if (s == 0) {
            issue_b(kt + kN - 1, m0, m1, prev);
            if (h == 0) issue_a(kp + 1, m0, m1);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  wait_vmcnt<0>();   // the zeros of the tiles past the last, before the stages are used again
}

// FfnProduct: A the weight (p codes, s scales), B the activations; K in values. Bf16, 2048 tokens at N = K =
// 4096: 60 us, 1.15 PFLOP/s (a library bf16 product of the same shape 59, and 47 here without the loads).
// MXFP4, 8192 tokens, N 8192, K 4096: 170 us, 3.2 PFLOP/s. By the counters the matrix cores are busy for 41% of the
// cycles (MXFP8, 8192 tokens at 4096, 55%; bf16 above 63%), LDS for 24% and without conflicts, 82% of L2's
// requests hit, and a wave waits for 39% of its time: neither the operands' 6.3 TB/s from L2 nor any unit is at
// its limit, but one workgroup to a CU has nothing else to run while a k-tile's barrier waits for loads, or
// a tile ends and the next begins. How much each of the two costs has not been taken apart.
template <typename S, int XF>
__global__ __launch_bounds__(S::kThreads, 2) void k_linear(const FfnProduct p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t stage_mem[];
  const int na = (p.na + S::BA - 1) / S::BA, nb = (p.nb + S::BB - 1) / S::BB;
  int ia, ib;
  const int id = xcd_remap(blockIdx.x, gridDim.x), split = id / (na * nb);
  tile_of(id % (na * nb), na, nb, ia, ib);
  const int a0 = ia * S::BA, b0 = ib * S::BB;
  const int n_a = min(S::BA, p.na - a0), n_b = min(S::BB, p.nb - b0);
  // this part's turns of k
  const int turns = (p.K + 255) / 256, parts = S::kSplits ? p.splits : 1;
  const int t0 = (int)((int64_t)turns * split / parts), t1 = (int)((int64_t)turns * (split + 1) / parts);
  const int K = min(t1 * 256, p.K) - t0 * 256;
  WLoader<S> la;
  XLoader<S> lb;
  const Operand A = {static_cast<const uint8_t*>(p.A.p) + (int64_t)t0 * 128, nullptr, p.K / 2, p.na};
  const Operand B = {static_cast<const uint8_t*>(p.B.p) + LinK<XF>::bytes(256) * t0, nullptr,
                     LinK<XF>::bytes(p.K), p.nb};
  la.init_row(A, 1, K / 2, a0, n_a, [=](int r) { return r < n_a ? r : -1; });
  lb.init_row(B, 1, (int)LinK<XF>::bytes(K), b0, n_b, [=](int r) { return r < n_b ? r : -1; });
  const MxScales mx = {p.A.s, p.B.s, p.na_s, p.nb_s, p.K / 32, t0 * 8};
  f32x16 acc[S::TA][S::TB];
  lin_loop<S, XF>(
      acc, stage_mem, la, lb, K, mx, [&](int r) { return r < n_a ? a0 + r : -1; },
      [&](int r) { return XF != kXB && r < n_b ? b0 + r : -1; });
  ffn_product_end<S>(p, acc, a0, b0, split, stage_mem);
}

// --------------------------------------------------------------- gradient

// Weight codes of one k-tile (64 weight rows x BA columns) in registers: 16 bytes, one block, and its
// scale to a thread.
template <typename S>
struct GradCodes {
  static constexpr int kPer = S::BA / 32;   // threads of a weight row
  static_assert(64 * kPer == S::kThreads, "a block to a thread");
  const uint8_t *q, *sc;
  int K, N;
  uint32_t off, soff;
  int lds[4];       // where the thread's four 16-byte pieces of bf16 go
  bool odd, two;    // and how its dwords are turned so that they follow those places
  u32x4 w;
  uint32_t s;
  __device__ __forceinline__ void init(const void* codes, const uint8_t* scales, int K_, int N_, int col0) {
    const int n = threadIdx.x / kPer, b = threadIdx.x % kPer;
    q = static_cast<const uint8_t*>(codes);
    sc = scales;
    K = K_;
    N = N_;
    const bool on = col0 + 32 * b < K;
    off = on ? (uint32_t)(n * (K / 2) + col0 / 2 + 16 * b) : (uint32_t)kOob;
    soff = on ? (uint32_t)(n * (K / 32) + col0 / 32 + b) : (uint32_t)kOob;
    // Row n of the tile at n * 2 BA, its 64-byte runs b at b ^ (n & 3) (two of the 32-byte units that
    // the transposing reads swizzle). The pieces of a run are written in an order that differs
    // between the four lanes of 16 whose runs share the banks.
    const int turn = kPer == 8 ? ((b >> 2) + 2 * (n & 1)) & 3 : n & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) lds[i] = n * 2 * S::BA + ((b ^ (n & 3)) * 64) + ((i + turn) & 3) * 16;
    odd = turn & 1;
    two = turn & 2;
  }
  __device__ __forceinline__ void load(int kt) {
    const int left = max(min(N - kt * 64, 64), 0);
    w = buf_load_b128(make_rsrc_uniform(q + (int64_t)kt * 64 * (K / 2), (uint32_t)(left * (K / 2))), (int)off);
    s = buf_load_u8(make_rsrc_uniform(sc + (int64_t)kt * 64 * (K / 32), (uint32_t)(left * (K / 32))), (int)soff);
  }
  // the dwords in the order of their places
  __device__ __forceinline__ void turn_dwords() {
    const u32x4 a = {odd ? w[1] : w[0], odd ? w[2] : w[1], odd ? w[3] : w[2], odd ? w[0] : w[3]};
    w = u32x4{two ? a[2] : a[0], two ? a[3] : a[1], two ? a[0] : a[2], two ? a[1] : a[3]};
  }
  __device__ __forceinline__ void store(int i, uint8_t* st) const {
    *reinterpret_cast<u32x4*>(st + lds[i]) = mx4_bf16x8(w[i], s);
  }
};

// The k loop as of the bf16 product above, in two stages of 64 weight rows each: tile kt + 2 is
// written to LDS (the weights) and asked for (the activations) as tile kt leaves it. 4095 tokens at 4096:
// 112 us, 1.23 PFLOP/s, 60% of the cycles of the matrix cores at the clock the load allows.
template <typename S>
__global__ __launch_bounds__(S::kThreads, 2) void k_linear_dx(const FfnProduct p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t stage_mem[];
  uint8_t* const lds = stage_mem;
  const int na = (p.na + S::BA - 1) / S::BA, nb = (p.nb + S::BB - 1) / S::BB;
  int ia, ib;
  const int id = xcd_remap(blockIdx.x, gridDim.x), split = id / (na * nb);
  tile_of(id % (na * nb), na, nb, ia, ib);
  const int a0 = ia * S::BA, b0 = ib * S::BB, n_b = min(S::BB, p.nb - b0);
  const KPart k(p.K, 2, split, S::kSplits ? p.splits : 1);   // weight rows, 64 to a k-tile
  const int N = k.K, nk = (N + 63) / 64;
  constexpr int kA = S::BA * 128, kStage = kA + S::BB * 128;
  GradCodes<S> ga;
  ga.init(static_cast<const uint8_t*>(p.A.p) + (int64_t)k.kt0 * 64 * (p.na / 2),
          p.A.s + (int64_t)k.kt0 * 64 * (p.na / 32), p.na, N, a0);
  XLoader<S> lb;
  lb.init_row(p.B.from_row(k.kt0), 2, N, b0, n_b, [=](int r) { return r < n_b ? r : -1; });
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  Reader<kOpCol, S::BA, S::TA, 128> ra;
  Reader<kOpRow, S::BB, S::TB, 128> rb;
  ra.init((w % S::WA) * S::TA * 32);
  rb.init((w / S::WA) * S::TB * 32);
  f32x16 acc[S::TA][S::TB];
#pragma unroll
  for (int i = 0; i < S::TA; ++i)
#pragma unroll
    for (int j = 0; j < S::TB; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  constexpr int kLoads = XLoader<S>::kLoads, kEarly = kLoads / 2;
  auto issue = [&](int kt, int i0, int i1, uint8_t* st) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (i >= i0 && i < i1) lb.template issue<true>(kt, i, st + kA);
  };
  // codes of the first two k-tiles into LDS, those of the third into registers
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    ga.load(t);
    ga.turn_dwords();
#pragma unroll
    for (int i = 0; i < 4; ++i) ga.store(i, lds + t * kStage);
  }
  ga.load(2);
  issue(0, 0, kLoads, lds);
  issue(1, 0, kEarly, lds + kStage);
  wait_vmcnt<kEarly>();
  wait_lgkm0();
  lds_barrier();
  bf16x8 fa[S::TA], fb[2][S::TB];
#pragma unroll
  for (int t = 0; t < S::TA; ++t) fa[t] = ra.bf16(lds, t, 0);
#pragma unroll
  for (int t = 0; t < S::TB; ++t) fb[0][t] = rb.bf16(lds + kA, t, 0);
  for (int kt = 0; kt < nk; ++kt) {
    uint8_t* const cur = lds + (kt & 1) * kStage;
    uint8_t* const nxt = lds + ((kt + 1) & 1) * kStage;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const bool last = s == 3;
      const int sn = (s + 1) & 3;
      const uint8_t* from = last ? nxt : cur;
      if (last) {
        // the tile's barrier: the next tile has landed whole, this one has been read by all
        wait_vmcnt<0>();
        wait_lgkm0();
        lds_barrier();
        ga.turn_dwords();
      }
#pragma unroll
      for (int u = 0; u < S::TB; ++u) fb[(s + 1) & 1][u] = rb.bf16(from + kA, u, sn);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < S::TA; ++t) {
#pragma unroll
        for (int u = 0; u < S::TB; ++u)
          acc[t][u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[t], fb[s & 1][u], acc[t][u], 0, 0, 0);
        fa[t] = ra.bf16(from, t, sn);
        if (last) {
          // the tile after next: its codes (converted here) and part of its activations take the
          // stage that the barrier freed
#pragma unroll
          for (int i = 4 * t / S::TA; i < 4 * (t + 1) / S::TA; ++i) ga.store(i, cur);
          if (t == S::TA - 1) ga.load(kt + 3);
          issue(kt + 2, kEarly * t / S::TA, kEarly * (t + 1) / S::TA, cur);
        }
        if (s == 0)
          issue(kt + 1, kEarly + (kLoads - kEarly) * t / S::TA, kEarly + (kLoads - kEarly) * (t + 1) / S::TA, nxt);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  wait_vmcnt<0>();
  ffn_product_end<S>(p, acc, a0, b0, split, lds);
}

// Column sums of a bf16 matrix [T, N] of few rows, in one launch: 64 columns, a line, to a workgroup, whose
// 32 groups of eight threads take every 32nd row and meet in LDS in their order.
__global__ __launch_bounds__(256) void k_bias_grad(const uint16_t* m, int T, int N, void* out, int dtype) {
  __shared__ __attribute__((aligned(16))) float red[32][68];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3, at = blockIdx.x * 64 + c * 8;
  float s[8] = {};
  if (at < N) {
#pragma unroll 8
    for (int r = g; r < T; r += 32) {
      float v[8];
      load8_bf16(m + (int64_t)r * N + at, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += v[i];
    }
  }
  *reinterpret_cast<f32x4*>(&red[g][c * 8]) = f32x4{s[0], s[1], s[2], s[3]};
  *reinterpret_cast<f32x4*>(&red[g][c * 8 + 4]) = f32x4{s[4], s[5], s[6], s[7]};
  __syncthreads();
  const int col = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x >= 64 || col >= N) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += red[i][threadIdx.x];
  if (dtype == MOE4_DTYPE_F32) static_cast<float*>(out)[col] = v;
  else static_cast<uint16_t*>(out)[col] = f32_to_bf16(v);
}

// ------------------------------------------------------------- few tokens

// One workgroup takes 16 RT weight rows and NT tiles of 16 tokens; its eight waves split K, 128 k
// (four blocks) a step, and meet in LDS in their order. A lane holds a block of its weight row a
// step, as the operands of four MFMAs, and its tokens' same 32 k; all are multiplied as bf16
// (MXFP8 and MXFP4 are exact there). The next batch of steps is in flight while one is multiplied. One
// token, N 5760, K 2880 (8.8 MB): 5.3 us, of which a launch takes 2.1 and the bytes 1.7 at a copy's rate;
// the rest is one round trip to HBM and the waves' meeting.
template <int RT, int NT, int XF>
struct LinSkinny {
  static constexpr int KS = 8, kThreads = KS * 64;
  static constexpr int kX = XF == kXB ? 4 : XF == kX8 ? 2 : 1;   // 16-byte loads of a token's step
  static constexpr int kU = RT + NT * kX > 8 ? 1 : 2;            // steps of a batch
  static constexpr int kLds = KS * RT * NT * 256 * 4;
  struct Batch {
    u32x4 w[kU][RT], x[kU][NT][kX];
    uint32_t ws[kU][RT], xs[kU][NT];
  };
};

template <int RT, int NT, int XF>
__global__ __launch_bounds__(512) void k_linear_skinny(const FfnProduct p) {
  using C = LinSkinny<RT, NT, XF>;
  extern __shared__ __attribute__((aligned(16))) float red[];
  const int a0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * 16 * NT, nt = min(16 * NT, p.nb - t0);
  const int ks = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), n = l & 15, g = l >> 4;
  const int K = p.K, nb = K / 32;
  const int64_t xb = LinK<XF>::bytes(K);
  // what the end needs from memory is asked for first: bias and addend of the thread's values
  constexpr int kAll = 16 * NT * 16 * RT, kTurns = (kAll + 511) / 512;
  uint32_t bias[kTurns], add[kTurns];
  const bool add32 = p.add_dtype == MOE4_DTYPE_F32;
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int o = i * 512 + threadIdx.x, m = o / (16 * RT), c = o % (16 * RT);
      if (m < nt && a0 + c < p.na) f(i, m, c, (int64_t)(t0 + m) * p.na + a0 + c);
    }
  };
#pragma unroll
  for (int i = 0; i < kTurns; ++i) bias[i] = add[i] = 0;
  each([&](int i, int, int c, int64_t at) {
    if (p.bias) bias[i] = p.bias[a0 + c];
    if (p.add)
      add[i] = add32 ? static_cast<const uint32_t*>(p.add)[at] : static_cast<const uint16_t*>(p.add)[at];
  });
  const rsrc_t rw = make_rsrc_uniform(p.A.p, (uint32_t)((int64_t)p.na * (K / 2)));
  const rsrc_t rws = make_rsrc_uniform(p.A.s, (uint32_t)(p.na * nb));
  const rsrc_t rx = make_rsrc_uniform(static_cast<const uint8_t*>(p.B.p) + t0 * xb, (uint32_t)(nt * xb));
  const rsrc_t rxs = make_rsrc_uniform(XF == kXB ? p.A.s : p.B.s + (int64_t)t0 * nb, XF == kXB ? 0u : (uint32_t)(nt * nb));
  uint32_t wo[RT], wso[RT], xo[NT], xso[NT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = a0 + 16 * i + n;
    wo[i] = r < p.na ? (uint32_t)r * (K / 2) + 16 * g : (uint32_t)kOob;
    wso[i] = r < p.na ? (uint32_t)r * nb + g : (uint32_t)kOob;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = 16 * i + n;
    xo[i] = t < nt ? (uint32_t)(t * xb) + C::kX * 16 * g : (uint32_t)kOob;
    xso[i] = t < nt ? (uint32_t)(t * nb + g) : (uint32_t)kOob;
  }
  const int steps = (K + 127) / 128, s0 = steps * ks / C::KS, s1 = steps * (ks + 1) / C::KS;
  auto load = [&](typename C::Batch& b, int s) {
#pragma unroll
    for (int i = 0; i < C::kU; ++i) {
      const int st = s + i;
      const bool on = st < s1 && 128 * st + 32 * g < K;
#pragma unroll
      for (int j = 0; j < RT; ++j) b.w[i][j] = buf_load_b128(rw, on ? (int)(wo[j] + 64 * st) : kOob);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < C::kX; ++c)
          b.x[i][j][c] = buf_load_b128(rx, on ? (int)(xo[j] + C::kX * 64 * st + 16 * c) : kOob);
#pragma unroll
      for (int j = 0; j < RT; ++j) b.ws[i][j] = buf_load_u8(rws, on ? (int)(wso[j] + 4 * st) : kOob);
      if constexpr (XF != kXB) {
#pragma unroll
        for (int j = 0; j < NT; ++j) b.xs[i][j] = buf_load_u8(rxs, on ? (int)(xso[j] + 4 * st) : kOob);
      }
    }
  };
  f32x4 acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto mul = [&](const typename C::Batch& b) {
#pragma unroll
    for (int i = 0; i < C::kU; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        bf16x8 x[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const u32x4* v = b.x[i][j];
          if constexpr (XF == kXB) x[j] = __builtin_bit_cast(bf16x8, v[c]);
          else if constexpr (XF == kX8) x[j] = mx_bf16x8(v[c / 2][2 * (c % 2)], v[c / 2][2 * (c % 2) + 1], b.xs[i][j]);
          else x[j] = __builtin_bit_cast(bf16x8, mx4_bf16x8(v[0][c], b.xs[i][j]));
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const bf16x8 w = __builtin_bit_cast(bf16x8, mx4_bf16x8(b.w[i][r][c], b.ws[i][r]));
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[r][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[j], acc[r][j], 0, 0, 0);
        }
      }
  };
  // (a batch that follows is asked for in straight line with the one before it: behind a branch of
  // its own the compiler would wait for all loads in flight)
  typename C::Batch b0, b1;
  int s = s0;
  load(b0, s);
  for (;;) {
    if (s + C::kU >= s1) {
      mul(b0);
      break;
    }
    load(b1, s + C::kU);
    mul(b0);
    s += C::kU;
    if (s + C::kU >= s1) {
      mul(b1);
      break;
    }
    load(b0, s + C::kU);
    mul(b1);
    s += C::kU;
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<f32x4*>(red + ((ks * RT + i) * NT + j) * 256 + l * 4) = acc[i][j];
  __syncthreads();
  each([&](int i, int m, int c, int64_t at) {
    const int from = ((c >> 4) * NT + (m >> 4)) * 256 + (((c & 15) >> 2) * 16 + (m & 15)) * 4 + (c & 3);
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < C::KS; ++k) v += red[k * RT * NT * 256 + from];
    v += __uint_as_float(bias[i] << 16);
    v += __uint_as_float(add32 ? add[i] : add[i] << 16);
    if (p.out_dtype == MOE4_DTYPE_F32) static_cast<float*>(p.out)[at] = v;
    else static_cast<uint16_t*>(p.out)[at] = f32_to_bf16(v);
  });
}

template <int XF, int NT>
hipError_t launch_skinny(const FfnProduct& p, hipStream_t s) {
  auto run = [&](auto rc) {
    constexpr int RT = decltype(rc)::value;
    using C = LinSkinny<RT, NT, XF>;
    auto* k = &k_linear_skinny<RT, NT, XF>;
    hipError_t e = allow_lds<C::kLds>(k);
    if (e != hipSuccess) return e;
    k<<<dim3((p.na + 16 * RT - 1) / (16 * RT), (p.nb + 16 * NT - 1) / (16 * NT)), 512, C::kLds, s>>>(p);
    return hipGetLastError();
  };
  // More row tiles save token loads, as long as there is a workgroup for most CUs. Us with 1, 2 and 4, bf16:
  // N 4096, K 4096 T 1 5.5 7.3 11.1; N 5760, K 2880 T 1 5.9 5.6 7.9, 16 9.1 7.5 10.2; N 16384, K 4096 T 1
  // 13.9 14.2 13.5, 16 24 20 16.6; MXFP8 there T 1 12.9 12.0 13.4, 16 21 16 16.
  if constexpr (XF != kX8 || NT == 1)   // (the other's operands do not fit the registers)
    if (p.na >= 64 * 192 && p.nb > 8) return run(std::integral_constant<int, 4>{});
  if (p.na >= 32 * 160) return run(std::integral_constant<int, 2>{});
  return run(std::integral_constant<int, 1>{});
}

// 256 x 128 of eight waves, 128 x 64 of four (two workgroups per CU)
using TileMid = TileShape<4, 2, 2, 2>;
using TileSmall = TileShape<2, 2, 2, 1>;

// Which tiles, by rounds of the chip (256 tiles of 256 x 256 or 256 x 128, 512 of 128 x 64), a round of
// them taking about 15, 8 and 5 units. Us, bf16: N = K = 4096, 2048 tokens 89 (half a round) and 60, 1024 37 with the
// smallest; MXFP8 509 tokens at 2880 (one round of each, mostly empty) 27 with 256 x 128, 15 with 128 x 64.
enum { kLarge, kMid, kSmall };
int lin_tiles(int64_t na, int64_t nb) {
  auto rounds = [](int64_t n, int64_t at_once) { return (n + at_once - 1) / at_once; };
  const int64_t large = 15 * rounds(tiles_of<Tile256>(na, nb), 256), mid = 8 * rounds(tiles_of<TileMid>(na, nb), 256),
                small = 5 * rounds(tiles_of<TileSmall>(na, nb), 512);
  return large <= mid && large <= small ? kLarge : mid <= small ? kMid : kSmall;
}

// Parts of k where the smallest tiles leave half of the CUs without one: as many as give each one,
// each of at least 512 k, 1024 or 2048 (the same time on the matrix cores, which pays for the launch
// that joins them: with every CU busy, 509 tokens at 2880, two parts take 14 us instead of 15, and the
// join 5).
int64_t most_lin_splits(int K, int x_format) {
  return std::min<int64_t>((K + 255) / 256 / (x_format == kXB ? 2 : x_format == kX8 ? 4 : 8), kMostSplits);
}
int lin_splits(int64_t na, int64_t nb, int K, int x_format) {
  if (lin_tiles(na, nb) != kSmall) return 1;
  const int64_t s = std::min<int64_t>(256 / tiles_of<TileSmall>(na, nb), most_lin_splits(K, x_format));
  return s < 2 ? 1 : (int)s;
}

template <int XF>
hipError_t launch_tiled(const FfnProduct& p, hipStream_t s) {
  auto run = [&](auto sc) {
    using S = decltype(sc);
    auto* k = &k_linear<S, XF>;
    hipError_t e = allow_lds<LinLds<S, XF>::kBytes>(k);
    if (e != hipSuccess) return e;
    k<<<(uint32_t)(tiles_of<S>(p.na, p.nb) * p.splits), S::kThreads, LinLds<S, XF>::kBytes, s>>>(p);
    return hipGetLastError();
  };
  const int tiles = lin_tiles(p.na, p.nb);
  if (tiles == kLarge) return run(Tile256{});
  if (tiles == kMid) return run(TileMid{});
  hipError_t e = run(TileSmall{});
  if (e != hipSuccess || p.splits == 1) return e;
  JoinArgs j = {};
  j.p[0] = p;
  return launch_join(j, 1, s);
}

// Tiles or few tokens: a tile costs the same for one token as for its 64, the skinny kernels read the
// tokens for every 16 to 64 weight rows. Us, skinny and tiled, bf16: N 5760, K 2880, T 16 7.5 12.3, 32 10.1
// 12.8; N 4096, K 4096, T 32 11.8 13.4, 48 17.8 14.7; N 16384, K 4096, T 16 16.6 18.7, 32 21.1 19.2; N 1024,
// K 1024, T 64 4.7 8.4 (MXFP8 4.8 7.0, MXFP4 4.3 6.2).
int linear_variant(const moe4_linear& l, int64_t T) {
  if (l.variant != MOE4_VARIANT_AUTO) return l.variant;
  const bool few = T <= 32 && T * l.N <= 384 << 10, small = T <= 64 && (T + 31) / 32 * ((l.N + 15) / 16) <= 256;
  return few || small ? MOE4_VARIANT_SKINNY : MOE4_VARIANT_TILED;
}

}  // namespace

// where the bias gradient's one launch takes less than two (us at N 4096: 128 rows 4.0 and 6.8, 512 7.5 and 9.1)
constexpr int kFewRows = 512;

size_t linear_ws_bytes(const moe4_linear& l, int64_t T, bool backward) {
  // (forward: at most 256 workgroups, each of 128 columns or fewer)
  if (!backward) return (size_t)part_bytes(l.N, T, (l.N + 127) / 128 > 128 ? 1 : most_lin_splits(l.K, kXB));
  return align_up((size_t)part_bytes(l.K, T, most_k_splits(l.K, l.N, 2)), 256) + (size_t)kColParts * l.N * 4;
}

hipError_t launch_linear_forward(const moe4_linear& l, const void* x, int x_format,
                                 const uint8_t* x_s, int T, const void* residual, int res_dtype,
                                 void* out, int out_dtype, void* ws, int* variant, hipStream_t s) {
  FfnProduct p = {};
  p.A = {l.w_q, l.w_s, l.K, l.N};
  p.B = {x, x_s, l.K, T};
  p.na_s = (int64_t)l.N * (l.K / 32);
  p.nb_s = x_format == kXB ? 0 : (int64_t)T * (l.K / 32);
  p.K = l.K;
  p.na = l.N;
  p.nb = T;
  p.bias = l.bias;
  p.add = residual;
  p.add_dtype = residual ? res_dtype : MOE4_DTYPE_BF16;
  p.out = out;
  p.out_dtype = out_dtype;
  p.splits = lin_splits(l.N, T, l.K, x_format);
  p.part = static_cast<float*>(ws);
  *variant = linear_variant(l, T);
  auto go = [&](auto fc) {
    constexpr int XF = decltype(fc)::value;
    if (*variant == MOE4_VARIANT_TILED) return launch_tiled<XF>(p, s);
    return T <= 16 ? launch_skinny<XF, 1>(p, s) : launch_skinny<XF, 2>(p, s);
  };
  if (x_format == kXB) return go(std::integral_constant<int, kXB>{});
  if (x_format == kX8) return go(std::integral_constant<int, kX8>{});
  return go(std::integral_constant<int, kX4>{});
}

hipError_t launch_linear_backward(const moe4_linear& l, const uint16_t* dy, int T,
                                  const void* dx_add, int add_dtype, void* dx, int dx_dtype,
                                  void* db, int db_dtype, void* ws, hipStream_t s) {
  float* const part = static_cast<float*>(ws);
  const size_t parts = align_up((size_t)part_bytes(l.K, T, most_k_splits(l.K, l.N, 2)), 256);
  if (dx) {
    FfnProduct p = {};
    p.A = {l.w_q, l.w_s, l.K, l.N};
    p.B = {dy, nullptr, l.N, T};
    p.K = l.N;
    p.na = l.K;
    p.nb = T;
    p.add = dx_add;
    p.add_dtype = dx_add ? add_dtype : MOE4_DTYPE_BF16;
    p.out = dx;
    p.out_dtype = dx_dtype;
    // (128 x 128 tiles and their rule: the smaller ones' conversions serve half the tokens, and 512
    // tokens at 4096 took 50 us with them, 38 so; 256 x 128 80, 2048 tokens, and 77 so)
    p.splits = k_splits(tiles_of<Tile128>(l.K, T), l.N, 2);
    p.part = part;
    auto run = [&](auto sc) {
      using S = decltype(sc);
      auto* k = &k_linear_dx<S>;
      hipError_t e = allow_lds<S::kLds>(k);
      if (e != hipSuccess) return e;
      k<<<(uint32_t)(tiles_of<S>(l.K, T) * p.splits), S::kThreads, S::kLds, s>>>(p);
      return hipGetLastError();
    };
    hipError_t e = p.splits == 1 && large_tiles_for(l.K, T) ? run(Tile256{}) : run(Tile128{});
    if (e == hipSuccess && p.splits > 1) {
      JoinArgs j = {};
      j.p[0] = p;
      e = launch_join(j, 1, s);
    }
    if (e != hipSuccess) return e;
  }
  if (!db) return hipSuccess;
  if (T <= kFewRows) {
    k_bias_grad<<<(l.N + 63) / 64, 256, 0, s>>>(dy, T, l.N, db, db_dtype);
    return hipGetLastError();
  }
  return launch_col_sums(dy, T, l.N, reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + parts), db, db_dtype, s);
}

}  // namespace moe4
