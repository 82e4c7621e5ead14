// Backward of the dense gated feed-forward block on bf16 weights:
//   dH = dY W_dn;  dGU = act'(gu) * dH;  dX = dGU W_gu (+ add)
//   dW_dn = dY^T h;  dW_gu = dGU^T x;  db_dn = sum_t dY;  db_gu = sum_t dGU
// The first product's epilogue applies the activation's derivative to its fp32 accumulators
// and writes dGU and the recomputed h in bf16, the operand type of the products that follow.
#include "ffn.hpp"

namespace moe4 {
namespace {

struct DhArgs {
  Operand W, dY;
  int T, H, I, layout;
  FfnAct act;
  const float* gu;      // [T, 2I]
  uint16_t* dgu;        // [T, 2I]
  uint16_t* h;          // [T, I] or null (no gradient of W_dn wanted)
};

template <typename S>
__global__ __launch_bounds__(S::kThreads, 2) void k_ffn_dh(const DhArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t stage_mem[];
  const int na = (a.I + S::BA - 1) / S::BA, nb = (a.T + S::BB - 1) / S::BB;
  int ia, ib;
  tile_of(xcd_remap(blockIdx.x, gridDim.x), na, nb, ia, ib);
  const int j0 = ia * S::BA, t0 = ib * S::BB, nt = min(S::BB, a.T - t0);
  Loader<kOpCol, S::BA, S::kThreads> la;
  Loader<kOpRow, S::BB, S::kThreads> lb;
  la.init_col(a.W, a.H, j0);
  lb.init_row(a.dY, 2, a.H, t0, nt, [=](int r) { return r < nt ? r : -1; });
  f32x16 acc[S::TA][S::TB];
  gemm_loop<S, kOpCol, kOpRow, false>(
      acc, stage_mem, la, lb, a.H, MxState<false>{}, [](int) { return -1; }, [](int) { return -1; });
  for_each8<S, false>(acc, stage_mem, [&](int row, int jj, float* dh) {
    const int t = t0 + row, j = j0 + jj;
    if (row >= nt || j >= a.I) return;
    const int64_t base = (int64_t)t * 2 * a.I;
    float g[8], u[8], h[8], d[16];
    if (a.layout == MOE4_GU_HALVES) {
      load8_f32(a.gu + base + j, g);
      load8_f32(a.gu + base + a.I + j, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) a.act.backward(g[i], u[i], dh[i], h[i], d[i], d[8 + i]);
      *reinterpret_cast<u32x4*>(a.dgu + base + j) = pack8_bf16(d);
      *reinterpret_cast<u32x4*>(a.dgu + base + a.I + j) = pack8_bf16(d + 8);
    } else {
      float x[16];
      load8_f32(a.gu + base + 2 * j, x);
      load8_f32(a.gu + base + 2 * j + 8, x + 8);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        a.act.backward(x[2 * i], x[2 * i + 1], dh[i], h[i], d[2 * i], d[2 * i + 1]);
      *reinterpret_cast<u32x4*>(a.dgu + base + 2 * j) = pack8_bf16(d);
      *reinterpret_cast<u32x4*>(a.dgu + base + 2 * j + 8) = pack8_bf16(d + 8);
    }
    if (a.h) *reinterpret_cast<u32x4*>(a.h + (int64_t)t * a.I + j) = pack8_bf16(h);
  });
}

// Column sums of a bf16 matrix [T, N]: part p of P sums its rows in fp32 into part[p][N].
__global__ __launch_bounds__(256) void k_col_sums(const uint16_t* m, int T, int N, float* part) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= N) return;
  const int r0 = (int)((int64_t)T * blockIdx.y / gridDim.y);
  const int r1 = (int)((int64_t)T * (blockIdx.y + 1) / gridDim.y);
  float s[8] = {};
  for (int r = r0; r < r1; ++r) {
    float v[8];
    load8_bf16(m + (int64_t)r * N + c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += v[i];
  }
  store8_f32(part + (int64_t)blockIdx.y * N + c, s);
}

constexpr int kColParts = 256;
int col_parts(int T) { return T < kColParts ? (T > 0 ? T : 1) : kColParts; }

hipError_t col_sums(const uint16_t* m, int T, int N, float* part, void* out, int dtype,
                    hipStream_t s) {
  const int P = col_parts(T);
  k_col_sums<<<dim3((N + 2047) / 2048, P), 256, 0, s>>>(m, T, N, part);
  hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_sum_rows(part, P, N, out, dtype, s);
}

template <int MA, int MB>
hipError_t product(const FfnProduct& p, hipStream_t s) {
  const int64_t big = (int64_t)((p.na + 255) / 256) * ((p.nb + 255) / 256);
  return big >= 192 ? launch_product<Tile256, MA, MB, false>(p, s)
                    : launch_product<Tile128, MA, MB, false>(p, s);
}

template <typename S>
hipError_t launch_dh(const DhArgs& a, hipStream_t s) {
  auto* k = &k_ffn_dh<S>;
  hipError_t e = allow_lds(k, S::kLds);
  if (e != hipSuccess) return e;
  const int64_t n = (int64_t)((a.I + S::BA - 1) / S::BA) * ((a.T + S::BB - 1) / S::BB);
  k<<<(uint32_t)n, S::kThreads, S::kLds, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t ffn_backward_ws_bytes(const moe4_ffn& f, int64_t T) {
  const int n = 2 * f.I > f.H ? 2 * f.I : f.H;
  return align_up((size_t)T * 2 * f.I * 2, 256) + align_up((size_t)T * f.I * 2, 256) +
         align_up((size_t)kColParts * n * 4, 256);
}

hipError_t launch_ffn_backward(const moe4_ffn& f, const uint16_t* x, int T, const float* gu,
                               const uint16_t* dy, const void* add, int add_dtype, void* dx,
                               int dx_dtype, void* dw_gu, void* dw_dn, void* db_gu, void* db_dn,
                               int dw_dtype, void* ws, hipStream_t s) {
  const int H = f.H, I = f.I;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  uint16_t* dgu = reinterpret_cast<uint16_t*>(w8);
  uint16_t* h = reinterpret_cast<uint16_t*>(w8 + align_up((size_t)T * 2 * I * 2, 256));
  float* part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(h) +
                                         align_up((size_t)T * I * 2, 256));
  hipError_t e = hipSuccess;
  if (dx || dw_gu || dw_dn || db_gu) {
    DhArgs a = {{f.w_dn, nullptr, I, I}, {dy, nullptr, H, T}, T,  H, I, f.gu_layout,
                {f.act, f.act_alpha, f.act_limit}, gu, dgu, dw_dn ? h : nullptr};
    const int64_t big = (int64_t)((I + 255) / 256) * ((T + 255) / 256);
    e = big >= 192 ? launch_dh<Tile256>(a, s) : launch_dh<Tile128>(a, s);
    if (e != hipSuccess) return e;
  }
  if (dx) {
    FfnProduct p = {{f.w_gu, nullptr, H, H}, {dgu, nullptr, 2 * I, T}, 0, 0, 2 * I, H, T,
                    nullptr, add, add_dtype, dx, dx_dtype};
    e = product<kOpCol, kOpRow>(p, s);
    if (e != hipSuccess) return e;
  }
  if (dw_gu) {
    FfnProduct p = {{x, nullptr, H, H}, {dgu, nullptr, 2 * I, 2 * I}, 0, 0, T, H, 2 * I,
                    nullptr, nullptr, 0, dw_gu, dw_dtype};
    e = product<kOpCol, kOpCol>(p, s);
    if (e != hipSuccess) return e;
  }
  if (dw_dn) {
    FfnProduct p = {{h, nullptr, I, I}, {dy, nullptr, H, H}, 0, 0, T, I, H,
                    nullptr, nullptr, 0, dw_dn, dw_dtype};
    e = product<kOpCol, kOpCol>(p, s);
    if (e != hipSuccess) return e;
  }
  if (db_gu) {
    e = col_sums(dgu, T, 2 * I, part, db_gu, dw_dtype, s);
    if (e != hipSuccess) return e;
  }
  return db_dn ? col_sums(dy, T, H, part, db_dn, dw_dtype, s) : hipSuccess;
}

}  // namespace moe4
