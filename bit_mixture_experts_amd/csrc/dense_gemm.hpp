// The tiled matrix product of the dense gated feed-forward block (bf16 or MXFP8 operands,
// fp32 accumulators), shared by its forward and backward kernels.
//
//   C[b][a] = sum_k A(a, k) B(b, k)
//
// a is the contiguous axis of the output, b its rows. Each operand comes in one of two
// layouts: "row" (k contiguous: a weight against activations, y = x W^T) or "col" (k
// strided, the a or b axis contiguous: the gradient products, whose reduction runs over the
// rows of what is in memory).
//
// One workgroup makes a BA x BB tile of C with WA x WB waves of TA x TB 32x32 MFMA tiles.
// k runs in tiles of 128 bytes per row (64 bf16 values) through two LDS stages, or of 64 bytes
// (64 e4m3 values) through four, filled by direct loads (no register round trip). An e4m3
// tile is multiplied in half the time of a bf16 one of the same bytes, so its loads need to
// be further ahead; for bf16 the shorter rows cost more (twice the requests) than the depth
// gave.
//
//  * Row operand: LDS [rows][128 B]; the 16-byte chunk c of row r sits at c ^ ((r >> 1) & 7),
//    so that the 16 rows of an operand read hit 16 different 16-byte bank groups (two rows
//    share a 256-byte bank line). 64-byte rows: c ^ ((r >> 2) & 3) (four rows a line).
//  * Col operand: LDS [64 k][rows * 2 B] as in memory; the MFMA wants 8 consecutive k of one
//    row in a lane, which ds_read_b64_tr_b16 delivers: 16 lanes read a 4 (k) x 16 (row)
//    block of 8 bytes each and get its transpose. The 32-byte unit u of row k sits at
//    u ^ 2 (k & 3): the four k rows and two units of half a wave's read cover all 64 banks.
//
// Pipeline: the operands of MFMA step s + 1 are read from LDS while step s multiplies, and
// in the last step of a k-tile those of the next tile's first step, behind the tile's one
// barrier. The barrier says two things at once: every wave's loads of tile kt + 1 have
// landed (each waits for its own first), and every wave has read all of tile kt, whose stage
// then takes the loads of the tile as many on as there are stages.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace moe4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

enum { kOpRow = 0, kOpCol = 1 };

// One operand as it lies in memory. Row: element (r, k) at p + (r * ld + k) * es, r < rows.
// Col: element (k, r) at p + (k * ld + r) * 2. s: the e8m0 scales of an MXFP8 operand
// [rows][ld / 32].
struct Operand {
  const void* p;
  const uint8_t* s;
  int64_t ld;
  int rows;
  // the same operand from k-tile kt on
  __device__ __forceinline__ Operand from_row(int kt) const {
    return {static_cast<const uint8_t*>(p) + (int64_t)kt * 128, s, ld, rows};
  }
  __device__ __forceinline__ Operand from_col(int kt) const {
    return {static_cast<const uint8_t*>(p) + (int64_t)kt * 128 * ld, s, ld, rows};
  }
};

template <int WA_, int WB_, int TA_, int TB_>
struct TileShape {
  static constexpr int WA = WA_, WB = WB_, TA = TA_, TB = TB_;
  static constexpr bool kSplits = TA * TB < 8;   // whether k may be cut (few tiles: small ones)
  static constexpr int BA = WA * TA * 32, BB = WB * TB * 32;
  static constexpr int kWaves = WA * WB, kThreads = kWaves * 64;
  static constexpr int kLds = 2 * (BA + BB) * 128;   // the stages, of either kind
  static constexpr int kLdsMx = kLds + 2 * (BA + BB) * 4;   // with two pairs of k-tiles' scales
};
// 256 x 256, eight waves, one workgroup per CU. (Four waves of 128 x 128, which read a third less
// from LDS, ran 10% slower: one wave a SIMD does not cover its own waits.)
using Tile256 = TileShape<2, 4, 4, 2>;
// 128 x 128, four waves, two workgroups per CU
using Tile128 = TileShape<2, 2, 2, 2>;

// Part s of S of a product's k axis, in whole k-tiles of 128 bytes: the first one, and how many
// elements of k the part has. A product with too few tiles for the chip is cut along k; the
// parts' fp32 sums are joined, in their order, by a launch of their own.
struct KPart {
  int kt0, K;
  __device__ __forceinline__ KPart(int K_, int es, int s, int S) {
    const int per = 128 / es, nk = (K_ + per - 1) / per;
    kt0 = (int)((int64_t)nk * s / S);
    K = min((int)((int64_t)nk * (s + 1) / S) * per, K_) - kt0 * per;
  }
};

// Tile (ia, ib) of workgroup id among na x nb: ids that run together on one XCD (a
// contiguous run of the remapped id) form blocks of kGroup b-tiles, b fastest, so that the 32
// workgroups of an XCD share kGroup B panels and a few A panels in its L2.
constexpr int kGroup = 8;
__device__ __forceinline__ void tile_of(int id, int na, int nb, int& ia, int& ib) {
  const int per = kGroup * na;
  const int g = id / per, r = id - g * per;
  const int gb = min(kGroup, nb - g * kGroup);
  ia = r / gb;
  ib = g * kGroup + (r - ia * gb);
}

// ds_read_b64_tr_b16 of the 8 bytes at p per lane
__device__ __forceinline__ s16x4 lds_tr16(const uint8_t* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_v;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v*)MOE4_LDS(p));
}

// A direct load of 16 bytes per lane into LDS (lane l at dst + 16 l), byte offset off of the
// resource with base p and size `bytes` (zeros past it). ASM: as an instruction that the
// compiler does not know for a load. It makes each ds_read_b64_tr_b16 wait for every direct
// load in flight, since it cannot tell their LDS addresses apart, and so for the k-tile that
// was asked for a moment before; the loops here wait for their loads themselves, before the
// barrier. The load has no destination register that the compiler could reuse meanwhile, and
// its own loads' wait counts stay sufficient: a load it does not count only makes them stricter.
// The five wait states are those between a vector instruction that writes a scalar register
// and the memory instruction that reads it, which the compiler would see to.
template <bool ASM>
__device__ __forceinline__ void load_lds16(const void* p, uint32_t bytes, uint8_t* dst,
                                           uint32_t off) {
  if constexpr (!ASM) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc_uniform(p, bytes), MOE4_LDS(dst), 16,
                                             (int)off, 0, 0, 0);
  } else {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const i32x4 r = {__builtin_amdgcn_readfirstlane((int)a),
                     __builtin_amdgcn_readfirstlane((int)(a >> 32) & 0xFFFF),
                     __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
    const int m = __builtin_amdgcn_readfirstlane((int)(uintptr_t)MOE4_LDS(dst));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(m), "v"(off), "s"(r)
                 : "memory", "m0");
  }
}

// Loader of one operand: N rows (a or b axis) and RB bytes of k (col: RB / 2 rows of k) per
// k-tile.
template <int MODE, int N, int THREADS, int RB>
struct Loader {
  static constexpr int kLoads = N * RB / (16 * THREADS);
  static_assert(kLoads * 16 * THREADS == N * RB, "whole loads per thread");
  const uint8_t* base;    // first element of the tile (row) or of column 0 of k row 0 (col)
  uint32_t size;          // row: bytes from base the tile may read
  int64_t ldb;            // bytes from row to row
  uint32_t off[kLoads];
  int chunk;              // row: byte of k that the thread's pieces start at in a k-tile
  int kb;                 // bytes (row) or rows (col) of k in all

  // row_of(r): the operand's row of tile row r, or -1; rows_from: the row that base is at
  template <typename RowOf>
  __device__ __forceinline__ void init_row(const Operand& o, int es, int K, int64_t row0,
                                           int64_t nrows, RowOf row_of) {
    const int t = threadIdx.x;
    ldb = o.ld * es;
    base = static_cast<const uint8_t*>(o.p) + row0 * ldb;
    size = (uint32_t)(nrows * ldb);
    kb = K * es;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int piece = i * THREADS + t, r = piece / (RB / 16);
      const int c = RB == 128 ? (piece & 7) ^ ((r >> 1) & 7) : (piece & 3) ^ ((r >> 2) & 3);
      chunk = c * 16;   // the same for every i: loads are a multiple of 16 rows apart
      const int rr = row_of(r);
      off[i] = rr >= 0 ? (uint32_t)(rr * ldb) + c * 16 : (uint32_t)kOob;
    }
  }
  __device__ __forceinline__ void init_col(const Operand& o, int K, int col0) {
    const int t = threadIdx.x;
    ldb = o.ld * 2;
    base = static_cast<const uint8_t*>(o.p);
    size = 0;
    kb = K;
    constexpr int kCpr = N / 8;   // 16-byte chunks of a k row
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int piece = i * THREADS + t, k = piece / kCpr;
      const int c = (piece % kCpr) ^ (4 * (k & 3));
      const int col = col0 + 8 * c;
      off[i] = col < o.rows ? (uint32_t)(k * ldb) + 2 * col : (uint32_t)kOob;
    }
  }
  // load i of k-tile kt into the operand's part of a stage
  template <bool ASM>
  __device__ __forceinline__ void issue(int kt, int i, uint8_t* lds) const {
    uint8_t* dst = lds + __builtin_amdgcn_readfirstlane(wave_id()) * 1024 + i * THREADS * 16;
    if constexpr (MODE == kOpRow) {
      const int k0 = kt * RB;
      load_lds16<ASM>(base, size, dst, k0 + chunk < kb ? off[i] + k0 : (uint32_t)kOob);
    } else {
      constexpr int kRows = RB / 2;
      const int left = max(min(kb - kt * kRows, kRows), 0);
      load_lds16<ASM>(base + (int64_t)kt * kRows * ldb, (uint32_t)(left * ldb), dst, off[i]);
    }
  }
};

// LDS reader of one operand: T 32-row MFMA tiles of a wave, rows w0 ...
template <int MODE, int N, int T, int RB>
struct Reader {
  int a[MODE == kOpRow ? 1 : T];
  __device__ __forceinline__ void init(int w0) {
    const int l = lane_id();
    if constexpr (MODE == kOpRow) {
      const int r = l & 31;
      a[0] = (w0 + r) * RB + (((l >> 5) ^ (RB == 128 ? (r >> 1) & 7 : (r >> 2) & 3)) * 16);
    } else {
      const int k = (l >> 5) * 8 + ((l >> 2) & 3);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int u = (w0 + 32 * t) / 16 + ((l >> 4) & 1);
        a[t] = k * 2 * N + ((u ^ (2 * (k & 3))) * 32) + (l & 3) * 8;
      }
    }
  }
  // the lane's 8 bf16 of MFMA tile t, step s (16 k)
  __device__ __forceinline__ bf16x8 bf16(const uint8_t* lds, int t, int s) const {
    if constexpr (MODE == kOpRow) {
      return *reinterpret_cast<const bf16x8*>(lds + (a[0] ^ (s * 32)) + t * 32 * RB);
    } else {
      const s16x4 lo = lds_tr16(lds + a[t] + s * 16 * 2 * N);
      const s16x4 hi = lds_tr16(lds + a[t] + s * 16 * 2 * N + 4 * 2 * N);
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  // the lane's 32 e4m3 of MFMA tile t (64 k): the matrix instruction takes k = 32 c + 16 (lane /
  // 32) .. + 15 in its c-th 16 bytes
  __device__ __forceinline__ i32x8 fp8(const uint8_t* lds, int t) const {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + a[0] + t * 32 * RB);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(lds + (a[0] ^ 32) + t * 32 * RB);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// The scales of both MXFP8 operands: bytes in all, blocks of a whole row, and the block that the
// loop's k begins with.
struct MxScales {
  const uint8_t *sa, *sb;
  int64_t na, nb;
  int pitch, first;
};

// e8m0 scales of both MXFP8 operands: thread t of the workgroup reads those of tile row t (A's
// rows, then B's), two k-tiles' (4 bytes) at a time, and the waves take them from LDS, where
// each row's lie as one dword. Read by every wave for its own rows they were fetched three
// times over, a gather of 32 rows to an instruction, and took the memory pipeline longer than
// the operands did (gate/up of 2048 tokens at H = I = 2880: 57 us, and 50 through LDS).
// The 4 bytes start at any byte, so the two dwords around them are loaded and shifted into
// one. The last dword may reach up to 3 bytes past the scales' end (never past the aligned
// dword that holds their last byte). Blocks past the row's end (their codes are zeros) take
// scale 0: the bytes there belong to the next row and may be e8m0 NaNs.
template <typename S>
struct ScaleStage {
  static_assert(S::kThreads == S::BA + S::BB, "a thread for every row");
  static constexpr int kBytes = S::kThreads * 4;   // of a pair of k-tiles
  rsrc_t r;
  int nb;            // blocks of a row that the loop runs over
  uint32_t off;      // byte of the first of them
  u32x2 raw;
  template <typename RowA, typename RowB>
  __device__ __forceinline__ void init(const MxScales& m, int blocks, RowA row_a, RowB row_b) {
    // whole waves belong to one operand
    const int t = threadIdx.x;
    const bool is_a = __builtin_amdgcn_readfirstlane(wave_id()) * 64 < S::BA;
    r = make_rsrc_uniform(is_a ? m.sa : m.sb, (uint32_t)(((is_a ? m.na : m.nb) + 3) & ~(int64_t)3));
    nb = blocks;
    const int row = is_a ? row_a(t) : row_b(t - S::BA);
    off = row >= 0 ? (uint32_t)row * m.pitch + m.first : (uint32_t)kOob;
  }
  __device__ __forceinline__ void load(int pair) {
    raw = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)((off & ~3u) + 4 * pair), 0, 0));
  }
  // the loaded scales of a pair of k-tiles into LDS
  __device__ __forceinline__ void store(u32x2 raw, int pair, uint8_t* lds) const {
    const int left = nb - 4 * pair;
    const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1;
    const uint32_t v = (uint32_t)((((uint64_t)raw[1] << 32) | raw[0]) >> (8 * (off & 3))) & keep;
    typedef uint32_t u32x1 __attribute__((ext_vector_type(1)));
    reinterpret_cast<u32x1*>(lds)[threadIdx.x] = u32x1{v};
  }
  // the dword of tile row `row` (byte 2 h + lane / 32 is the pair's h-th tile's)
  static __device__ __forceinline__ uint32_t get(const uint8_t* lds, int row) {
    typedef uint32_t u32x1 __attribute__((ext_vector_type(1)));
    return reinterpret_cast<const u32x1*>(lds)[row][0];
  }
};

constexpr int row_bytes(bool fp8) { return fp8 ? 64 : 128; }
template <typename S, int MODE, int N, bool FP8>
using OpLoader = Loader<MODE, N, S::kThreads, row_bytes(FP8)>;

// The k loop. acc[ta][tb] += A B^T over all of K. When it returns this wave has no load in
// flight, but other waves may still be reading: a barrier stands before the stages are used
// for anything else.
template <typename S, int MA, int MB, bool FP8, typename RowA, typename RowB>
__device__ __forceinline__ void gemm_loop(f32x16 (&acc)[S::TA][S::TB], uint8_t* lds,
                                          OpLoader<S, MA, S::BA, FP8>& la,
                                          OpLoader<S, MB, S::BB, FP8>& lb, int K,
                                          const MxScales& mx, RowA row_a, RowB row_b) {
  constexpr int kRb = row_bytes(FP8), kSub = 128 / kRb;   // k-tiles of 128 bytes of k
  constexpr int kSteps = FP8 ? 1 : 4, kStages = 2 * kSub;
  constexpr int kStage = (S::BA + S::BB) * kRb;
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const int wa = w % S::WA, wb = w / S::WA;
  Reader<MA, S::BA, S::TA, kRb> ra;
  Reader<MB, S::BB, S::TB, kRb> rb;
  ra.init(wa * S::TA * 32);
  rb.init(wb * S::TB * 32);
  constexpr int kA = S::BA * kRb;   // offset of the B part of a stage
  constexpr bool kAsm = MA == kOpCol || MB == kOpCol;
  const int nk = (K * (FP8 ? 1 : 2) + 127) / 128;   // turns of the loop, 128 bytes of k each

  using Frag = std::conditional_t<FP8, i32x8, bf16x8>;
  // bf16: all A operands of a step and the B operands of two. e4m3, with twice the registers
  // an operand: a ring of two A operands and the B operands of one step, reloaded as the
  // step's last MFMAs take them (twice the MFMA time covers the read).
  constexpr int kRing = FP8 ? 2 : S::TA, kB = FP8 ? 1 : 2;
  Frag fa[kRing], fb[kB][S::TB];
  auto read_a = [&](const uint8_t* st, int t, int s) {
    if constexpr (FP8) return ra.fp8(st, t);
    else return ra.bf16(st, t, s);
  };
  auto read_b = [&](const uint8_t* st, int t, int s) {
    if constexpr (FP8) return rb.fp8(st + kA, t);
    else return rb.bf16(st + kA, t, s);
  };
  // e4m3: this pair's scales, shifted for the lane's half, and the next one's as they come
  ScaleStage<S> sc;
  uint8_t* const sclds = lds + S::kLds;
  uint32_t xa[FP8 ? S::TA : 1], xb[FP8 ? S::TB : 1], na[FP8 ? S::TA : 1], nb[FP8 ? S::TB : 1];
  auto next_scales = [&](int pair) {
    const uint8_t* p = sclds + (pair & 1) * ScaleStage<S>::kBytes;
    const int r = lane_id() & 31;
#pragma unroll
    for (int t = 0; t < S::TA; ++t) na[t] = sc.get(p, (wa * S::TA + t) * 32 + r);
#pragma unroll
    for (int u = 0; u < S::TB; ++u) nb[u] = sc.get(p, S::BA + (wb * S::TB + u) * 32 + r);
  };
  u32x2 first;
  if constexpr (FP8) {
    // both before the operands' loads: the loop then finds as many loads behind the scales'
    // as it issues itself, and does not wait for more of them
    sc.init(mx, K / 32, row_a, row_b);
    sc.load(0);
    first = sc.raw;
    sc.load(1);
  }

#pragma unroll
  for (int i = 0; i < S::TA; ++i)
#pragma unroll
    for (int j = 0; j < S::TB; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

  // A k-tile's loads go out a few at a time between the MFMAs, behind the barrier that frees
  // their stage up to the next one. Sent in one go they filled the memory pipeline's queue, and
  // the waves stood at their next load instead of multiplying (forward of 4096 tokens at H
  // 4096, I 8192: 675 us, and 641 spread). Tiles past the last load zeros: no branch in the
  // loop, which the compiler would sink the MFMAs before it past.
  constexpr int kLa = OpLoader<S, MA, S::BA, FP8>::kLoads;
  constexpr int kLoads = kLa + OpLoader<S, MB, S::BB, FP8>::kLoads;
  // groups of MFMAs between the barrier and the tile's end, and in the next tile's first step
  // before its barrier; the loads that go out in the first ones
  constexpr int kAfter = kRing, kBefore = FP8 ? S::TA - kRing : S::TA;
  constexpr int kEarly = kBefore ? kLoads / 2 : kLoads;
  auto issue = [&](int kt, int i0, int i1, uint8_t* st) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < i0 || i >= i1) continue;
      if (i < kLa) la.template issue<kAsm>(kt, i, st);
      else lb.template issue<kAsm>(kt, i - kLa, st + kA);
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i, 0, kLoads, lds + i * kStage);
  issue(kStages - 1, 0, kEarly, lds + (kStages - 1) * kStage);
  wait_vmcnt<(kStages - 2) * kLoads + kEarly>();
  if constexpr (FP8) {
    sc.store(first, 0, sclds);
    wait_lgkm0();
  }
  lds_barrier();
  if constexpr (FP8) next_scales(0);
#pragma unroll
  for (int t = 0; t < kRing; ++t) fa[t] = read_a(lds, t, 0);
#pragma unroll
  for (int t = 0; t < S::TB; ++t) fb[0][t] = read_b(lds, t, 0);
  for (int kp = 0; kp < nk; ++kp) {
    if constexpr (FP8) {
      const int half = 8 * (lane_id() >> 5);
#pragma unroll
      for (int t = 0; t < S::TA; ++t) xa[t] = na[t] >> half;
#pragma unroll
      for (int u = 0; u < S::TB; ++u) xb[u] = nb[u] >> half;
      sc.store(sc.raw, kp + 1, sclds + ((kp + 1) & 1) * ScaleStage<S>::kBytes);
      sc.load(kp + 2);
    }
    uint8_t* const base = lds + (kp & 1) * kSub * kStage;
    uint8_t* const other = lds + ((kp + 1) & 1) * kSub * kStage;
#pragma unroll
    for (int h = 0; h < kSub; ++h) {
      const int kt = kp * kSub + h;
      uint8_t* const cur = base + h * kStage;
      uint8_t* const nxt = h + 1 < kSub ? cur + kStage : other;
      uint8_t* const prv = h > 0 ? cur - kStage : other + (kSub - 1) * kStage;
      // the tile's barrier: the wave's loads of the next tile have landed (those of the tiles
      // after it may be in flight), its reads of this one are done, and so are the others'
      auto turn = [&]() {
        wait_vmcnt<(kStages - 2) * kLoads>();
        wait_lgkm0();
        lds_barrier();
        if (FP8 && h == kSub - 1) next_scales(kp + 1);
      };
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const bool last = s == kSteps - 1;
        const int sn = (s + 1) % kSteps;
        // operands of the next step (past the last tile: stale values, read and never used)
        const uint8_t* from = last ? nxt : cur;
        if constexpr (!FP8) {
          if (last) turn();
#pragma unroll
          for (int u = 0; u < S::TB; ++u) fb[(s + 1) % kB][u] = read_b(from, u, sn);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < S::TA; ++t) {
          Frag& a = fa[t % kRing];
#pragma unroll
          for (int u = 0; u < S::TB; ++u) {
            Frag& b = fb[s % kB][u];
            if constexpr (FP8)
              acc[t][u] = h == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                       a, b, acc[t][u], 0, 0, 0, (int)xa[t], 0, (int)xb[u])
                                 : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                       a, b, acc[t][u], 0, 0, 2, (int)xa[t], 2, (int)xb[u]);
            else
              acc[t][u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[t][u], 0, 0, 0);
            if (FP8 && t == S::TA - kRing && u == S::TB - 1) turn();
            if (FP8 && t == S::TA - 1) b = read_b(from, u, sn);
          }
          // the operand kRing tiles on: of this step, or of the next
          a = t + kRing < S::TA ? read_a(cur, t + kRing, s) : read_a(from, t + kRing - S::TA, sn);
          const int slot = t - (S::TA - kAfter);
          if (last && slot >= 0)
            issue(kt + kStages, kEarly * slot / kAfter, kEarly * (slot + 1) / kAfter, cur);
          if (s == 0 && t < kBefore)
            issue(kt + kStages - 1, kEarly + (kLoads - kEarly) * t / kBefore,
                  kEarly + (kLoads - kEarly) * (t + 1) / kBefore, prv);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  wait_vmcnt<0>();   // the zeros of the tiles past the last, before the stages are used again
}

// the first a (PAIR: pair) of the tile that for_each8 hands this lane
template <typename S, bool PAIR>
__device__ __forceinline__ int lane_a() {
  constexpr int W = S::TA * 32, kPer = PAIR ? W / 16 : W / 8;
  const int wa = __builtin_amdgcn_readfirstlane(wave_id()) % S::WA, c = lane_id() % kPer;
  return PAIR ? wa * (W / 2) + 32 * (c / 4) + 8 * (c % 4) : wa * W + 8 * c;
}

// Epilogue: hands every value of the tile to f(b, a, v, pre) as 8 consecutive a of one row b in
// one lane (PAIR: 8 gate and 8 up values whose MFMA tiles are neighbours, f(b, j, g, u) with j
// the pair's place in the tile), in an order that makes a wave's stores whole row segments.
// Through LDS, 32 rows b of the wave at a time as fp32 [32][TA * 32]: the 16-byte chunk c of
// row b sits at c ^ (b & 15), which spreads the 16 rows of a write over the banks.
// load(b, a) gives pre, what f reads from memory for the same values: it is asked for DEPTH
// turns ahead of f, since one turn is far shorter than a load. a is the same in every turn of
// a lane.
template <typename S, bool PAIR, int DEPTH, typename L, typename F>
__device__ __forceinline__ void for_each8(const f32x16 (&acc)[S::TA][S::TB], uint8_t* lds, L load,
                                          F f) {
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const int wb = w / S::WA, l = lane_id();
  constexpr int W = S::TA * 32;              // fp32 values of a row
  constexpr int kKey = W / 4 >= 16 ? 15 : W / 4 - 1;
  static_assert(S::kWaves * 32 * W * 4 <= S::kLds, "staging fits the stages");
  constexpr int kPer = PAIR ? W / 16 : W / 8;   // lanes of a row
  constexpr int kRows = 64 / kPer, kTurns = 32 / kRows, kAll = kTurns * S::TB;
  uint8_t* st = lds + w * 32 * W * 4;
  const int c = l % kPer;
  // turn n = (u, i): the tile's row of the lane, and its first a (PAIR: its first pair)
  auto row_at = [&](int n) { return wb * S::TB * 32 + n * kRows + l / kPer; };
  const int a_at = lane_a<S, PAIR>();
  using Pre = decltype(load(0, 0));
  Pre pre[DEPTH];
#pragma unroll
  for (int n = 0; n < DEPTH; ++n)
    if (n < kAll) pre[n] = load(row_at(n), a_at);
  lds_barrier();   // every wave is done with the k loop's stages
#pragma unroll
  for (int u = 0; u < S::TB; ++u) {
    const int b = l & 31;
#pragma unroll
    for (int t = 0; t < S::TA; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 v = {acc[t][u][4 * q], acc[t][u][4 * q + 1], acc[t][u][4 * q + 2],
                         acc[t][u][4 * q + 3]};
        const int ch = 8 * t + 2 * q + (l >> 5);
        *reinterpret_cast<f32x4*>(st + b * W * 4 + ((ch ^ (b & kKey)) * 16)) = v;
      }
    wait_lgkm0();
    asm volatile("" ::: "memory");
    auto get = [&](int bb, int a, float* v) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(
            st + bb * W * 4 + (((a / 4 + h) ^ (bb & kKey)) * 16));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = x[i];
      }
    };
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int n = u * kTurns + i, bb = i * kRows + l / kPer;
      const Pre mine = pre[n % DEPTH];
      if (n + DEPTH < kAll) pre[n % DEPTH] = load(row_at(n + DEPTH), a_at);
      if constexpr (PAIR) {
        const int p = c / 4, j = 8 * (c % 4);   // pair group (two MFMA tiles), place in it
        float g[8], uu[8];
        get(bb, 64 * p + j, g);
        get(bb, 64 * p + 32 + j, uu);
        f(row_at(n), a_at, g, uu);
      } else {
        float v[8];
        get(bb, 8 * c, v);
        f(row_at(n), a_at, v, mine);
      }
    }
    wait_lgkm0();
    asm volatile("" ::: "memory");
  }
}

struct NoPre {};

}  // namespace moe4
