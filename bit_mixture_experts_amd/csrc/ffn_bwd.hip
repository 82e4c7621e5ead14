// Backward of the dense gated feed-forward block on bf16 weights:
//   dH = dY W_dn;  dGU = act'(gu) * dH;  dX = dGU W_gu (+ add)
//   dW_dn = dY^T h;  dW_gu = dGU^T x;  db_dn = sum_t dY;  db_gu = sum_t dGU
// The first product's epilogue applies the activation's derivative to its fp32 accumulators
// and writes dGU and the recomputed h in bf16, the operand type of the products that follow.
//
// 8192 tokens at H = I = 2880 with biases: 820-855 us, 0.97 PFLOP/s. dH 214 us: its epilogue reads
// 189 MB of pre-activations and writes 141 MB while the matrix cores stand (37% of a tile's
// time; small tiles, two workgroups to a CU, overlap it but multiply more slowly: 202 to 218
// us), and 384 tiles are one and a half rounds. The other products 607 us, 1.12 PFLOP/s. The
// biases' column sums 12 + 10 us.
#include "ffn.hpp"

namespace moe4 {
namespace {

struct DhArgs {
  Operand W, dY;
  int T, H, I;
  FfnAct act;
  const float* gu;      // [T, 2I]
  uint16_t* dgu;        // [T, 2I]
  uint16_t* h;          // [T, I] or null (no gradient of W_dn wanted)
  float* part;          // [row tiles, or the join's rows of workgroups][2I] column sums of dGU, or null
  int splits;           // parts of k (few tokens and a wide stream)
  float* dh;            // [splits][T][I] sums to be joined
};

// the saved pre-activations of 8 pairs: gate and up (halves), or pairs in turn (interleaved)
struct RawGu {
  u32x4 v[4];
};

// dGU (and h) of 8 pairs j .. j+7 of token t from dH and their pre-activations; d: dGU in the
// order of memory, the runs that start at col0 and col1
template <int LAYOUT, int ACT>
struct Pairs8 {
  static constexpr bool kHalves = LAYOUT == MOE4_GU_HALVES;
  static __device__ __forceinline__ int col0(int j) { return kHalves ? j : 2 * j; }
  static __device__ __forceinline__ int col1(const DhArgs& a, int j) {
    return kHalves ? a.I + j : 2 * j + 8;
  }
  static __device__ __forceinline__ RawGu load(const DhArgs& a, int64_t t, int j) {
    RawGu r;
    const float* p = a.gu + t * 2 * a.I;
    const u32x4* q = reinterpret_cast<const u32x4*>(p + col0(j));
    const u32x4* s = reinterpret_cast<const u32x4*>(p + col1(a, j));
    r.v[0] = q[0];
    r.v[1] = q[1];
    r.v[2] = s[0];
    r.v[3] = s[1];
    return r;
  }
  static __device__ __forceinline__ void finish(const DhArgs& a, int64_t t, int j, const float* dh,
                                                const RawGu& r, float* d) {
    const FfnAct act = {ACT, a.act.alpha, a.act.limit};
    float x[16], h[8];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r.v[i / 4][i % 4]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (kHalves) act.backward(x[i], x[8 + i], dh[i], h[i], d[i], d[8 + i]);
      else act.backward(x[2 * i], x[2 * i + 1], dh[i], h[i], d[2 * i], d[2 * i + 1]);
    }
    uint16_t* o = a.dgu + t * 2 * a.I;
    *reinterpret_cast<u32x4*>(o + col0(j)) = pack8_bf16(d);
    *reinterpret_cast<u32x4*>(o + col1(a, j)) = pack8_bf16(d + 8);
    if (a.h) *reinterpret_cast<u32x4*>(a.h + t * a.I + j) = pack8_bf16(h);
  }
};

// LAYOUT, ACT: the block's (their branches would double the epilogue's code four times over)
template <typename S, int LAYOUT, int ACT>
__global__ __launch_bounds__(S::kThreads, 2) void k_ffn_dh(const DhArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t stage_mem[];
  const int na = (a.I + S::BA - 1) / S::BA, nb = (a.T + S::BB - 1) / S::BB;
  int ia, ib;
  const int id = xcd_remap(blockIdx.x, gridDim.x), split = id / (na * nb);
  tile_of(id % (na * nb), na, nb, ia, ib);
  const int j0 = ia * S::BA, t0 = ib * S::BB, nt = min(S::BB, a.T - t0);
  OpLoader<S, kOpCol, S::BA, false> la;
  OpLoader<S, kOpRow, S::BB, false> lb;
  const KPart k(a.H, 2, split, S::kSplits ? a.splits : 1);
  la.init_col(a.W.from_col(k.kt0), k.K, j0);
  lb.init_row(a.dY.from_row(k.kt0), 2, k.K, t0, nt, [=](int r) { return r < nt ? r : -1; });
  f32x16 acc[S::TA][S::TB];
  gemm_loop<S, kOpCol, kOpRow, false>(
      acc, stage_mem, la, lb, k.K, MxScales{}, [](int) { return -1; }, [](int) { return -1; });
  if constexpr (S::kSplits) {
    if (a.splits > 1) {
      float* part = a.dh + (int64_t)split * a.T * a.I;
      for_each8<S, false, 1>(acc, stage_mem, [](int, int) { return NoPre{}; },
                                    [&](int row, int jj, float* v, const NoPre&) {
        const int j = j0 + jj;
        if (row < nt && j < a.I) store8_f32(part + (int64_t)(t0 + row) * a.I + j, v);
      });
      return;
    }
  }
  using P = Pairs8<LAYOUT, ACT>;
  float sums[16] = {};   // of dGU over the lane's rows, in fp32 before the rounding
  for_each8<S, false, 4>(
      acc, stage_mem,
      [&](int row, int jj) {
        RawGu r;
        if (row < nt && j0 + jj < a.I) r = P::load(a, t0 + row, j0 + jj);
        return r;
      },
      [&](int row, int jj, float* dh, const RawGu& r) {
        if (row >= nt || j0 + jj >= a.I) return;
        float d[16];
        P::finish(a, t0 + row, j0 + jj, dh, r, d);
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[i] += d[i];
      });
  if (!a.part) return;
  // the lane's sums, over the wave's rows (lanes of the same columns), then over its WB waves in
  // order through LDS
  constexpr int W = S::TA * 32, kPer = W / 8;
  const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id();
  const int wa = w % S::WA, wb = w / S::WA;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int m = kPer; m < 64; m <<= 1) sums[i] += __shfl_xor(sums[i], m, kWave);
  f32x4* red = reinterpret_cast<f32x4*>(stage_mem);   // [wb][wa][kPer][4]
  __syncthreads();
  if (l < kPer) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      red[((wb * S::WA + wa) * kPer + l) * 4 + i] =
          f32x4{sums[4 * i], sums[4 * i + 1], sums[4 * i + 2], sums[4 * i + 3]};
  }
  __syncthreads();
  if (wb != 0 || l >= kPer) return;
  const int j = j0 + wa * W + 8 * l;
  if (j >= a.I) return;
  float* o = a.part + (int64_t)ib * 2 * a.I;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f32x4 s = red[(wa * kPer + l) * 4 + i];
#pragma unroll
    for (int v = 1; v < S::WB; ++v) s += red[((v * S::WA + wa) * kPer + l) * 4 + i];
    *reinterpret_cast<f32x4*>(o + (i < 2 ? P::col0(j) + 4 * i : P::col1(a, j) + 4 * (i - 2))) = s;
  }
}

// The products that follow dGU, in one launch: their tiles are dealt product by product,
// longest reduction first, so that the chip is full until the last of them (one launch each
// left most CUs idle in its last round). Each product's run of workgroups starts at a
// multiple of 8 (an XCD each): ids past a product's tiles have nothing to do.
struct GradArgs {
  FfnProduct p[3];
  int first[4];     // first workgroup of each, and the end
  int col_b[3];     // whether B is a col operand (a weight's gradient) or a row one (dX)
};

template <typename S>
__global__ __launch_bounds__(S::kThreads, 2) void k_ffn_grads(const GradArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t stage_mem[];
  const int q = (int)blockIdx.x < a.first[1] ? 0 : (int)blockIdx.x < a.first[2] ? 1 : 2;
  const FfnProduct& p = a.p[q];
  const int na = (p.na + S::BA - 1) / S::BA, nb = (p.nb + S::BB - 1) / S::BB;
  int id = blockIdx.x - a.first[q];
  if (id >= na * nb * p.splits) return;
  id = xcd_remap(id, na * nb * p.splits);
  int ia, ib;
  tile_of(id % (na * nb), na, nb, ia, ib);
  const int split = id / (na * nb);
  if (a.col_b[q]) ffn_product_tile<S, kOpCol, kOpCol, false>(p, ia, ib, split, stage_mem);
  else ffn_product_tile<S, kOpCol, kOpRow, false>(p, ia, ib, split, stage_mem);
}

template <typename S>
hipError_t launch_grads(GradArgs a, int n, hipStream_t s) {
  auto* k = &k_ffn_grads<S>;
  hipError_t e = allow_lds<S::kLds>(k);
  if (e != hipSuccess) return e;
  a.first[0] = 0;
  for (int i = 0; i < 3; ++i)
    a.first[i + 1] = a.first[i] + (i < n ? (int)((tiles_of<S>(a.p[i].na, a.p[i].nb) * a.p[i].splits + 7) / 8 * 8) : 0);
  k<<<a.first[3], S::kThreads, S::kLds, s>>>(a);
  return hipGetLastError();
}

// The parts of a split dH, joined: 8 pairs of a token to a thread, 128 pairs of kJoinRows tokens
// to a workgroup, which leaves its column sums of dGU in part, in fp32 before the rounding as
// the whole dH's epilogue does. (Summed from dGU in memory they cost a pass of their own and
// hold each term's rounding to bf16. Us of the whole backward with biases: 100 tokens at 2880,
// 2880 62.5 that way and 59.3 this, 1024 175 and 171.5, 128 at H 4096, I 8192 166.3 and 160.7.)
constexpr int kJoinRows = 16;
template <int LAYOUT, int ACT>
__global__ __launch_bounds__(256) void k_ffn_dh_join(const DhArgs a) {
  __shared__ __attribute__((aligned(16))) f32x4 red[4][16][4];   // [wave][8 pairs][16 values]
  using P = Pairs8<LAYOUT, ACT>;
  const int x = threadIdx.x & 15, w = wave_id();
  const int t = blockIdx.y * kJoinRows + (threadIdx.x >> 4), j = (blockIdx.x * 16 + x) * 8;
  float d[16] = {};
  if (t < a.T && j < a.I) {
    const RawGu r = P::load(a, t, j);
    float dh[8] = {};
    for (int s = 0; s < a.splits; ++s) {
      float v[8];
      load8_f32(a.dh + ((int64_t)s * a.T + t) * a.I + j, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) dh[q] += v[q];
    }
    P::finish(a, t, j, dh, r, d);
  }
  if (!a.part) return;
  // the wave's four tokens, then the four waves in order
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    d[i] += __shfl_xor(d[i], 16, kWave);
    d[i] += __shfl_xor(d[i], 32, kWave);
  }
  if (lane_id() < 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      red[w][x][i] = f32x4{d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]};
  }
  __syncthreads();
  // four values of 8 pairs to a thread of the first wave
  const int c = threadIdx.x >> 2, i = threadIdx.x & 3, jc = (blockIdx.x * 16 + c) * 8;
  if (w != 0 || jc >= a.I) return;
  const f32x4 s = red[0][c][i] + red[1][c][i] + red[2][c][i] + red[3][c][i];
  float* o = a.part + (int64_t)blockIdx.y * 2 * a.I;
  *reinterpret_cast<f32x4*>(o + (i < 2 ? P::col0(jc) + 4 * i : P::col1(a, jc) + 4 * (i - 2))) = s;
}

// Column sums of a bf16 matrix [T, N]: workgroup (x, p) sums part p's rows of 512 columns in
// fp32 into part[p][N]; its four waves take every fourth row and meet in LDS.
__global__ __launch_bounds__(256) void k_col_sums(const uint16_t* m, int T, int N, float* part) {
  __shared__ __attribute__((aligned(16))) f32x4 red[4][2][64];
  const int l = lane_id(), w = wave_id(), c = (blockIdx.x * 64 + l) * 8;
  const int r0 = (int)((int64_t)T * blockIdx.y / gridDim.y);
  const int r1 = (int)((int64_t)T * (blockIdx.y + 1) / gridDim.y);
  float s[8] = {};
  if (c < N) {
#pragma unroll 16
    for (int r = r0 + w; r < r1; r += 4) {
      float v[8];
      load8_bf16(m + (int64_t)r * N + c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += v[i];
    }
  }
  red[w][0][l] = f32x4{s[0], s[1], s[2], s[3]};
  red[w][1][l] = f32x4{s[4], s[5], s[6], s[7]};
  __syncthreads();
  if (w < 2 && c < N) {
    const f32x4 v = red[0][w][l] + red[1][w][l] + red[2][w][l] + red[3][w][l];
    *reinterpret_cast<f32x4*>(part + (int64_t)blockIdx.y * N + c + 4 * w) = v;
  }
}

constexpr int kMostGradSplits = 32;

template <typename S, int LAYOUT, int ACT>
hipError_t launch_dh(const DhArgs& a, hipStream_t s) {
  auto* k = &k_ffn_dh<S, LAYOUT, ACT>;
  hipError_t e = allow_lds<S::kLds>(k);
  if (e != hipSuccess) return e;
  k<<<(uint32_t)(tiles_of<S>(a.I, a.T) * a.splits), S::kThreads, S::kLds, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  k_ffn_dh_join<LAYOUT, ACT><<<dim3((a.I + 127) / 128, (a.T + kJoinRows - 1) / kJoinRows), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

static int col_parts(int T) { return T < kColParts ? (T > 0 ? T : 1) : kColParts; }

hipError_t launch_col_sums(const uint16_t* m, int T, int N, float* part, void* out, int dtype,
                    hipStream_t s) {
  const int P = col_parts(T);
  k_col_sums<<<dim3((N + 511) / 512, P), 256, 0, s>>>(m, T, N, part);
  hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_sum_rows(part, P, N, out, dtype, s);
}

// workspace: dGU, h, the partial sums of the two biases' gradients, of dH where it is split along
// k, and of the products after it: one whose reduction is several times a workgroup's share of
// all their k-tiles (few tokens: dX; a small block and many tokens: the weights' gradients)
// would still run when the others have ended. Every region's size is one that does not fall as T
// grows (part_bytes), whatever this T is split into.
struct BwdWs {
  size_t h, part_gu, part_dn, dh, part[3], end;
  int dh_splits, splits[3];   // dX, dW_gu, dW_dn
  BwdWs(const moe4_ffn& f, int64_t T) {
    h = align_up((size_t)T * 2 * f.I * 2, 256);
    part_gu = h + align_up((size_t)T * f.I * 2, 256);
    dh_splits = T > 0 ? k_splits(tiles_of<Tile128>(f.I, T), f.H, 2) : 1;
    // dH whole leaves a row of bias sums per row tile, the join one per kJoinRows tokens of the
    // at most 256 tiles that are split
    const int64_t most_dh = most_k_splits(f.I, f.H, 2), whole = (T + Tile128::BB - 1) / Tile128::BB;
    int64_t joined = most_dh > 1 ? 256 / ((f.I + 127) / 128) * (Tile128::BB / kJoinRows) : 0;
    if (joined > (T + kJoinRows - 1) / kJoinRows) joined = (T + kJoinRows - 1) / kJoinRows;
    part_dn = part_gu + align_up((size_t)(joined > whole ? joined : whole) * 2 * f.I * 4, 256);
    dh = part_dn + align_up((size_t)kColParts * f.H * 4, 256);
    end = dh + align_up((size_t)part_bytes(f.I, T, most_dh), 256);
    const int64_t size[3][3] = {{f.H, T, 2 * (int64_t)f.I}, {f.H, 2 * (int64_t)f.I, T}, {f.I, f.H, T}};
    int64_t work = 0;   // k-tiles of 64
    for (const auto& z : size) work += tiles_of<Tile128>(z[0], z[1]) * ((z[2] + 63) / 64);
    const int64_t share = (work + 511) / 512 > 8 ? (work + 511) / 512 : 8;
    // parts x tiles of the three together: at most work / share, so at most 512
    size_t at = end, most = 0;
    for (int i = 0; i < 3; ++i) {
      const int64_t nk = (size[i][2] + 63) / 64, s = nk / share, ms = nk / 8;
      splits[i] = s < 2 ? 1 : (int)(s < kMostGradSplits ? s : kMostGradSplits);
      part[i] = at;
      if (splits[i] > 1) at += align_up((size_t)splits[i] * size[i][0] * size[i][1] * 4, 256);
      most += align_up((size_t)part_bytes(size[i][0], size[i][1], ms < kMostGradSplits ? ms : kMostGradSplits), 256);
    }
    const size_t all = (size_t)kMostPartBytes + 3 * 256;
    end += most < all ? most : all;
  }
};

size_t ffn_backward_ws_bytes(const moe4_ffn& f, int64_t T) { return BwdWs(f, T).end; }

hipError_t launch_ffn_backward(const moe4_ffn& f, const uint16_t* x, int T, const float* gu,
                               const uint16_t* dy, const void* add, int add_dtype, void* dx,
                               int dx_dtype, void* dw_gu, void* dw_dn, void* db_gu, void* db_dn,
                               int dw_dtype, void* ws, hipStream_t s) {
  const int H = f.H, I = f.I;
  const BwdWs at(f, T);
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  uint16_t* dgu = reinterpret_cast<uint16_t*>(w8);
  uint16_t* h = reinterpret_cast<uint16_t*>(w8 + at.h);
  float* part_gu = reinterpret_cast<float*>(w8 + at.part_gu);
  float* part_dn = reinterpret_cast<float*>(w8 + at.part_dn);
  hipError_t e = hipSuccess;
  if (dx || dw_gu || dw_dn || db_gu) {
    DhArgs a = {{f.w_dn, nullptr, I, I}, {dy, nullptr, H, T}, T, H, I,
                {f.act, f.act_alpha, f.act_limit}, gu, dgu, dw_dn ? h : nullptr,
                db_gu ? part_gu : nullptr, at.dh_splits, reinterpret_cast<float*>(w8 + at.dh)};
    const bool big = at.dh_splits == 1 && large_tiles_for(I, T);
    e = with_kind(f.gu_layout, f.act, [&](auto l, auto c) {
      constexpr int L = decltype(l)::value, A = decltype(c)::value;
      return big ? launch_dh<Tile256, L, A>(a, s) : launch_dh<Tile128, L, A>(a, s);
    });
    if (e != hipSuccess) return e;
    if (db_gu) {
      const int rows = at.dh_splits > 1 ? kJoinRows : big ? Tile256::BB : Tile128::BB;
      e = launch_sum_rows(part_gu, (T + rows - 1) / rows, 2 * I, db_gu, dw_dtype, s);
      if (e != hipSuccess) return e;
    }
  }
  GradArgs g = {};
  int n = 0;
  JoinArgs join = {};
  int joins = 0;
  auto put = [&](FfnProduct p, int which, bool col_b) {
    p.splits = at.splits[which];
    p.part = reinterpret_cast<float*>(w8 + at.part[which]);
    if (p.splits > 1) join.p[joins++] = p;
    // longest reduction first
    int i = n++;
    for (; i > 0 && g.p[i - 1].K < p.K; --i) {
      g.p[i] = g.p[i - 1];
      g.col_b[i] = g.col_b[i - 1];
    }
    g.p[i] = p;
    g.col_b[i] = col_b;
  };
  if (dx)
    put({{f.w_gu, nullptr, H, H}, {dgu, nullptr, 2 * I, T}, 0, 0, 2 * I, H, T, nullptr, add,
         add_dtype, dx, dx_dtype}, 0, false);
  if (dw_gu)
    put({{x, nullptr, H, H}, {dgu, nullptr, 2 * I, 2 * I}, 0, 0, T, H, 2 * I, nullptr, nullptr, 0,
         dw_gu, dw_dtype}, 1, true);
  if (dw_dn)
    put({{h, nullptr, I, I}, {dy, nullptr, H, H}, 0, 0, T, I, H, nullptr, nullptr, 0, dw_dn,
         dw_dtype}, 2, true);
  if (n) {
    int64_t n256 = 0, n128 = 0;
    for (int i = 0; i < n; ++i) {
      n256 += tiles_of<Tile256>(g.p[i].na, g.p[i].nb);
      n128 += tiles_of<Tile128>(g.p[i].na, g.p[i].nb);
    }
    e = joins == 0 && large_tiles(n256, n128) ? launch_grads<Tile256>(g, n, s)
                                              : launch_grads<Tile128>(g, n, s);
    if (e == hipSuccess && joins) e = launch_join(join, joins, s);
    if (e != hipSuccess) return e;
  }
  return db_dn ? launch_col_sums(dy, T, H, part_dn, db_dn, dw_dtype, s) : hipSuccess;
}

}  // namespace moe4
