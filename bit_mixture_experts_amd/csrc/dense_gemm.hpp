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
// k runs in tiles of 128 bytes per row (64 bf16 or 128 e4m3 values) through two LDS stages,
// filled by direct loads (no register round trip).
//
//  * Row operand: LDS [rows][128 B]; the 16-byte chunk c of row r sits at c ^ ((r >> 1) & 7),
//    so that the 16 rows of an operand read hit 16 different 16-byte bank groups (two rows
//    share a 256-byte bank line).
//  * Col operand: LDS [64 k][rows * 2 B] as in memory; the MFMA wants 8 consecutive k of one
//    row in a lane, which ds_read_b64_tr_b16 delivers: 16 lanes read a 4 (k) x 16 (row)
//    block of 8 bytes each and get its transpose. The 32-byte unit u of row k sits at
//    u ^ 2 (k & 3): the four k rows and two units of half a wave's read cover all 64 banks.
//
// Pipeline: the operands of MFMA step s + 1 are read from LDS while step s multiplies, and
// in the last step of a k-tile those of the next tile's first step, behind the tile's one
// barrier. The barrier says two things at once: every wave's loads of tile kt + 1 have
// landed (each waits for its own first), and every wave has read all of tile kt, whose stage
// then takes the loads of tile kt + 2.
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
};

template <int WA_, int WB_, int TA_, int TB_>
struct TileShape {
  static constexpr int WA = WA_, WB = WB_, TA = TA_, TB = TB_;
  static constexpr int BA = WA * TA * 32, BB = WB * TB * 32;
  static constexpr int kWaves = WA * WB, kThreads = kWaves * 64;
  static constexpr int kStage = (BA + BB) * 128;
  static constexpr int kLds = 2 * kStage;
};
using Tile256 = TileShape<2, 4, 4, 2>;   // 256 x 256, eight waves, one workgroup per CU
using Tile128 = TileShape<2, 2, 2, 2>;   // 128 x 128, four waves, two workgroups per CU

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

// Loader of one operand: N rows (a or b axis) per k-tile.
template <int MODE, int N, int THREADS>
struct Loader {
  static constexpr int kLoads = N * 128 / (16 * THREADS);
  static_assert(kLoads * 16 * THREADS == N * 128, "whole loads per thread");
  static constexpr int kRowB = MODE == kOpRow ? 128 : 2 * N;   // LDS bytes of a row
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
      const int piece = i * THREADS + t, r = piece >> 3;
      const int c = (piece & 7) ^ ((r >> 1) & 7);
      chunk = c * 16;   // the same for every i: loads are THREADS / 8 rows apart, a multiple of 16
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
      const int k0 = kt * 128;
      load_lds16<ASM>(base, size, dst, k0 + chunk < kb ? off[i] + k0 : (uint32_t)kOob);
    } else {
      const int left = max(min(kb - kt * 64, 64), 0);
      load_lds16<ASM>(base + (int64_t)kt * 64 * ldb, (uint32_t)(left * ldb), dst, off[i]);
    }
  }
};

// LDS reader of one operand: T 32-row MFMA tiles of a wave, rows w0 ...
template <int MODE, int N, int T>
struct Reader {
  int a[MODE == kOpRow ? 1 : T];
  __device__ __forceinline__ void init(int w0) {
    const int l = lane_id();
    if constexpr (MODE == kOpRow) {
      const int r = l & 31;
      a[0] = (w0 + r) * 128 + (((l >> 5) ^ ((r >> 1) & 7)) * 16);
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
      return *reinterpret_cast<const bf16x8*>(lds + (a[0] ^ (s * 32)) + t * 4096);
    } else {
      const s16x4 lo = lds_tr16(lds + a[t] + s * 16 * 2 * N);
      const s16x4 hi = lds_tr16(lds + a[t] + s * 16 * 2 * N + 4 * 2 * N);
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  // the lane's 32 e4m3 of MFMA tile t, step s (64 k): the matrix instruction takes k = 32 c +
  // 16 (lane / 32) .. + 15 in its c-th 16 bytes
  __device__ __forceinline__ i32x8 fp8(const uint8_t* lds, int t, int s) const {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + (a[0] ^ (s * 64)) + t * 4096);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(lds + (a[0] ^ (s * 64) ^ 32) + t * 4096);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// e8m0 scales of an MXFP8 operand, read per lane: the 4 bytes of a row and k-tile start at
// any byte, so the two dwords around them are loaded and shifted into one. The last dword
// may reach up to 3 bytes past the scales' end (never past the aligned dword that holds their
// last byte). Of the lane's dword, byte 2 s + lane / 32 is step s's: one shift by the lane's
// half puts it at byte 2 s.
template <int T>
struct ScaleReader {
  rsrc_t r;
  int nb;              // blocks of a row
  uint32_t off[T];     // byte of the row's first scale
  u32x2 raw[T];
  uint32_t v[T];
  template <typename RowOf>
  __device__ __forceinline__ void init(const uint8_t* s, int64_t bytes, int blocks, int w0,
                                       RowOf row_of) {
    const int l = lane_id();
    r = make_rsrc_uniform(s, (uint32_t)((bytes + 3) & ~(int64_t)3));
    nb = blocks;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int row = row_of(w0 + 32 * t + (l & 31));
      off[t] = row >= 0 ? (uint32_t)row * nb : (uint32_t)kOob;
    }
  }
  __device__ __forceinline__ void prefetch(int kt) {
#pragma unroll
    for (int t = 0; t < T; ++t)
      raw[t] = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)((off[t] & ~3u) + 4 * kt), 0, 0));
  }
  // Blocks past the row's end (their codes are zeros) take scale 0: the bytes there belong to
  // the next row and may be e8m0 NaNs.
  __device__ __forceinline__ void take(int kt) {
    const int left = nb - 4 * kt, h = lane_id() >> 5;
    const uint32_t keep = (h < left ? 0xFFu : 0u) | (2 + h < left ? 0xFF0000u : 0u);
#pragma unroll
    for (int t = 0; t < T; ++t)
      v[t] = (uint32_t)((((uint64_t)raw[t][1] << 32) | raw[t][0]) >> (8 * ((off[t] & 3) + h))) & keep;
  }
};

template <bool FP8>
struct MxState {};
template <>
struct MxState<true> {
  const uint8_t *sa, *sb;   // scales
  int64_t na, nb;           // their bytes
};

// The k loop. acc[ta][tb] += A B^T over all of K. When it returns this wave has no load in
// flight, but other waves may still be reading: a barrier stands before the stages are used
// for anything else.
template <typename S, int MA, int MB, bool FP8, typename RowA, typename RowB>
__device__ __forceinline__ void gemm_loop(f32x16 (&acc)[S::TA][S::TB], uint8_t* lds,
                                          Loader<MA, S::BA, S::kThreads>& la,
                                          Loader<MB, S::BB, S::kThreads>& lb, int K,
                                          const MxState<FP8>& mx, RowA row_a, RowB row_b) {
  constexpr int kSteps = FP8 ? 2 : 4, KT = FP8 ? 128 : 64;
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const int wa = w % S::WA, wb = w / S::WA;
  Reader<MA, S::BA, S::TA> ra;
  Reader<MB, S::BB, S::TB> rb;
  ra.init(wa * S::TA * 32);
  rb.init(wb * S::TB * 32);
  constexpr int kA = S::BA * 128;   // offset of the B part of a stage
  constexpr bool kAsm = MA == kOpCol || MB == kOpCol;
  const int nk = (K + KT - 1) / KT;

  using Frag = std::conditional_t<FP8, i32x8, bf16x8>;
  // bf16: all A operands of a step and the B operands of two. e4m3, with twice the registers
  // an operand: a ring of two A operands and the B operands of one step, reloaded as the
  // step's last MFMAs take them (twice the MFMA time covers the read).
  constexpr int kRing = FP8 ? 2 : S::TA, kB = FP8 ? 1 : 2;
  Frag fa[kRing], fb[kB][S::TB];
  auto read_a = [&](const uint8_t* st, int t, int s) {
    if constexpr (FP8) return ra.fp8(st, t, s);
    else return ra.bf16(st, t, s);
  };
  auto read_b = [&](const uint8_t* st, int t, int s) {
    if constexpr (FP8) return rb.fp8(st + kA, t, s);
    else return rb.bf16(st + kA, t, s);
  };
  ScaleReader<FP8 ? S::TA : 1> xa;
  ScaleReader<FP8 ? S::TB : 1> xb;
  if constexpr (FP8) {
    xa.init(mx.sa, mx.na, K / 32, wa * S::TA * 32, row_a);
    xb.init(mx.sb, mx.nb, K / 32, wb * S::TB * 32, row_b);
    xa.prefetch(0);
    xb.prefetch(0);
  }

#pragma unroll
  for (int i = 0; i < S::TA; ++i)
#pragma unroll
    for (int j = 0; j < S::TB; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

  // A k-tile's loads go out a few at a time between the MFMAs: half of them in the last step of
  // the tile whose stage they take, half in the next tile's first step. Sent in one go they
  // filled the memory pipeline's queue, and the waves stood at their next load instead of
  // multiplying (forward of 4096 tokens at H 4096, I 8192: 675 us, and 641 spread). Tiles past the last load
  // zeros: no branch in the loop, which the compiler would sink the MFMAs before it past.
  constexpr int kLa = Loader<MA, S::BA, S::kThreads>::kLoads;
  constexpr int kLoads = kLa + Loader<MB, S::BB, S::kThreads>::kLoads, kHalf = kLoads / 2;
  auto issue = [&](int kt, int i0, int i1, uint8_t* st) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < i0 || i >= i1) continue;
      if (i < kLa) la.template issue<kAsm>(kt, i, st);
      else lb.template issue<kAsm>(kt, i - kLa, st + kA);
    }
  };
  issue(0, 0, kLoads, lds);
  wait_vmcnt<0>();
  lds_barrier();
  issue(1, 0, kHalf, lds + S::kStage);
#pragma unroll
  for (int t = 0; t < kRing; ++t) fa[t] = read_a(lds, t, 0);
#pragma unroll
  for (int t = 0; t < S::TB; ++t) fb[0][t] = read_b(lds, t, 0);
  for (int kt = 0; kt < nk; ++kt) {
    uint8_t* cur = lds + (kt & 1) * S::kStage;
    uint8_t* nxt = lds + ((kt + 1) & 1) * S::kStage;
    if constexpr (FP8) {
      xa.take(kt);
      xb.take(kt);
      xa.prefetch(kt + 1);
      xb.prefetch(kt + 1);
    }
    // the tile's barrier: the wave's loads of the next k-tile have landed, its reads of this
    // one are done, and so are the others'
    auto turn = [&]() {
      wait_vmcnt<0>();
      wait_lgkm0();
      lds_barrier();
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
            acc[t][u] = s == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                     a, b, acc[t][u], 0, 0, 0, (int)xa.v[t], 0, (int)xb.v[u])
                               : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                     a, b, acc[t][u], 0, 0, 2, (int)xa.v[t], 2, (int)xb.v[u]);
          else
            acc[t][u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[t][u], 0, 0, 0);
          if (FP8 && last && t == S::TA - kRing && u == S::TB - 1) turn();
          if (FP8 && t == S::TA - 1) b = read_b(from, u, sn);
        }
        // the operand kRing tiles on: of this step, or of the next
        a = t + kRing < S::TA ? read_a(cur, t + kRing, s) : read_a(from, t + kRing - S::TA, sn);
        // loads of the tile after next once its stage is free, the rest in the next tile
        constexpr int kSlots = FP8 ? kRing : S::TA;   // groups of MFMAs behind the barrier
        const int slot = t - (S::TA - kSlots);
        if (last && slot >= 0)
          issue(kt + 2, kHalf * slot / kSlots, kHalf * (slot + 1) / kSlots, cur);
        if (s == 0)
          issue(kt + 1, kHalf + kHalf * t / S::TA, kHalf + kHalf * (t + 1) / S::TA, nxt);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  wait_vmcnt<0>();   // the zeros of the tiles past the last, before the stages are used again
}

// Epilogue: hands every value of the tile to f(b, a, v, pre) as 8 consecutive a of one row b in
// one lane (PAIR: 8 gate and 8 up values whose MFMA tiles are neighbours, f(b, j, g, u) with j
// the pair's place in the tile), in an order that makes a wave's stores whole row segments.
// Through LDS, 32 rows b of the wave at a time as fp32 [32][TA * 32]: the 16-byte chunk c of
// row b sits at c ^ (b & 15), which spreads the 16 rows of a write over the banks.
// load(b, a) gives pre, what f reads from memory for the same values: it is asked for two
// turns ahead of f, so that its latency hides behind the turns between.
template <typename S, bool PAIR, typename L, typename F>
__device__ __forceinline__ void for_each8(const f32x16 (&acc)[S::TA][S::TB], uint8_t* lds, L load,
                                          F f) {
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const int wa = w % S::WA, wb = w / S::WA, l = lane_id();
  constexpr int W = S::TA * 32;              // fp32 values of a row
  constexpr int kKey = W / 4 >= 16 ? 15 : W / 4 - 1;
  static_assert(S::kWaves * 32 * W * 4 <= S::kLds, "staging fits the stages");
  constexpr int kPer = PAIR ? W / 16 : W / 8;   // lanes of a row
  constexpr int kRows = 64 / kPer, kTurns = 32 / kRows, kAll = kTurns * S::TB;
  uint8_t* st = lds + w * 32 * W * 4;
  const int c = l % kPer;
  // turn n = (u, i): the tile's row of the lane, and its first a (PAIR: its first pair)
  auto row_at = [&](int n) { return wb * S::TB * 32 + n * kRows + l / kPer; };
  const int a_at = PAIR ? wa * (W / 2) + 32 * (c / 4) + 8 * (c % 4) : wa * W + 8 * c;
  using Pre = decltype(load(0, 0));
  Pre pre[2];
  pre[0] = load(row_at(0), a_at);
  pre[1] = load(row_at(1), a_at);
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
      const Pre mine = pre[n & 1];
      if (n + 2 < kAll) pre[n & 1] = load(row_at(n + 2), a_at);
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
