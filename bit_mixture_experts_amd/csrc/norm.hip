// The root-mean-square norm with the residual stream's addition in front of it, in bf16 and,
// or, MXFP8, and its backward pass; the MXFP8 quantiser; sums over rows of partial results.
//
// All of them are bound by HBM: every element is read and written once, and held in registers
// between the row's sum of squares and its output.
#include "internal.hpp"
#include "mx.hpp"

namespace moe4 {
namespace {

// 8 elements of a row in registers as they lie in memory: bf16 (16 bytes) or fp32 (32 bytes)
template <int DT>
struct Raw8 {
  u32x4 r[DT == MOE4_DTYPE_F32 ? 2 : 1];
  // column c of a row whose resource is rs; zeros past its end
  __device__ __forceinline__ void load(rsrc_t rs, int c) {
    if constexpr (DT == MOE4_DTYPE_F32) {
      r[0] = buf_load_b128(rs, 4 * c);
      r[1] = buf_load_b128(rs, 4 * c + 16);
    } else {
      r[0] = buf_load_b128(rs, 2 * c);
    }
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE4_DTYPE_F32) {
        v[i] = __uint_as_float(r[0][i]);
        v[4 + i] = __uint_as_float(r[1][i]);
      } else {
        v[2 * i] = bf16lo(r[0][i]);
        v[2 * i + 1] = bf16hi(r[0][i]);
      }
    }
  }
  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE4_DTYPE_F32) {
        r[0][i] = __float_as_uint(v[i]);
        r[1][i] = __float_as_uint(v[4 + i]);
      } else {
        r[0][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      }
    }
  }
  // stores past the row's end are dropped
  __device__ __forceinline__ void store(rsrc_t rs, int c) const {
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    if constexpr (DT == MOE4_DTYPE_F32) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, r[0]), rs, 4 * c, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, r[1]), rs, 4 * c + 16, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, r[0]), rs, 2 * c, 0, 0);
    }
  }
};

template <int DT>
__device__ __forceinline__ rsrc_t row_rsrc(const void* p, int64_t row, int H) {
  constexpr int es = DT == MOE4_DTYPE_F32 ? 4 : 2;
  return make_rsrc_uniform(static_cast<const uint8_t*>(p) + row * H * es, (uint32_t)H * es);
}

// fp32 sum over the wave, in every lane: DPP and permlane steps, no LDS round trip
__device__ __forceinline__ float wave_sum_f32(float x) {
  auto dpp = [](float v, auto ctl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctl)::value,
                                                      0xF, 0xF, false));
  };
  x += dpp(x, std::integral_constant<int, 0xB1>{});    // quad_perm [1,0,3,2]
  x += dpp(x, std::integral_constant<int, 0x4E>{});    // quad_perm [2,3,0,1]
  x += dpp(x, std::integral_constant<int, 0x141>{});   // row_half_mirror
  x += dpp(x, std::integral_constant<int, 0x140>{});   // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// sum over the W waves of a row, in every lane; slot alternates between calls so that one
// barrier a call is enough
template <int W>
__device__ __forceinline__ float row_sum(float x, float (&red)[2][W], int slot) {
  x = wave_sum_f32(x);
  if constexpr (W == 1) return x;
  if (lane_id() == 0) red[slot][wave_id()] = x;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) s += red[slot][i];
  return s;
}

// One pass: the row stays in registers between its sum of squares and its outputs. Bound by HBM:
// 4096 x 2880, fp32 x and bf16 stream in, sum, bf16 and MXFP8 out (130 MB): 26.7 us, 4.9 TB/s,
// the rate of a large copy on this card; one row of 2048: 2.2 us, a launch.
//
// Shapes: W waves of a row, each lane NV chunks of 8 columns (W * NV * 512 columns at most).
// W == 1 puts four rows into a workgroup and needs no barrier: for many rows. More waves a
// row shorten a row's own latency: for few rows, and for rows past one wave's registers.
template <int W>
constexpr int kNormThreads = W == 1 ? 256 : 64 * W;

struct NormArgs {
  const void *x, *res;
  void* sum;
  const void* w;
  int w_dtype;
  int T, H;
  float eps;
  uint16_t* out;
  uint8_t *q, *qs;
  float* rstd;
};

// DX, DR: types of x and of the residual stream (0: no residual; the row is x itself)
template <int DX, int DR, int W, int NV>
__global__ __launch_bounds__(kNormThreads<W>) void k_add_rmsnorm(const NormArgs a) {
  constexpr int kRows = W == 1 ? 4 : 1;
  __shared__ float red[2][W];
  const int tid = W == 1 ? lane_id() : threadIdx.x;
  const int w0 = W == 1 ? __builtin_amdgcn_readfirstlane(wave_id()) : 0;
  auto col = [&](int i) { return (i * W * 64 + tid) * 8; };
  // the weight stays in registers over the rows of the workgroup, as it lies in memory
  Raw8<MOE4_DTYPE_BF16> wb[NV];
  const bool wf = a.w_dtype == MOE4_DTYPE_F32;
  const rsrc_t rw = make_rsrc_uniform(a.w, (uint32_t)a.H * (wf ? 4 : 2));
  if (!wf) {
#pragma unroll
    for (int i = 0; i < NV; ++i) wb[i].load(rw, col(i));
  }
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + w0; row < a.T; row += (int64_t)gridDim.x * kRows) {
    Raw8<DX> x[NV];
    Raw8<DR == 0 ? DX : DR> r[NV];
    const rsrc_t rx = row_rsrc<DX>(a.x, row, a.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i].load(rx, col(i));
    if constexpr (DR != 0) {
      const rsrc_t rr = row_rsrc<DR>(a.res, row, a.H);
#pragma unroll
      for (int i = 0; i < NV; ++i) r[i].load(rr, col(i));
    }
    // The row is normalised as the stream holds it: the sum is rounded to the stream's type
    // first, so that the backward pass and the next layer see the row that was normalised.
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8];
      x[i].get(v);
      if constexpr (DR != 0) {
        float u[8];
        r[i].get(u);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += u[k];
        r[i].set(v);
        r[i].get(v);
      } else {
        r[i] = x[i];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[k], v[k], ss);
    }
    if constexpr (DR != 0) {
      if (a.sum) {
        const rsrc_t rs = row_rsrc<DR>(a.sum, row, a.H);
#pragma unroll
        for (int i = 0; i < NV; ++i) r[i].store(rs, col(i));
      }
    }
    ss = row_sum<W>(ss, red, slot);
    slot ^= 1;
    const float rstd = rsqrtf(ss / (float)a.H + a.eps);
    if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8], w[8];
      r[i].get(v);
      if (wf) {
        Raw8<MOE4_DTYPE_F32> t;
        t.load(rw, col(i));
        t.get(w);
      } else {
        wb[i].get(w);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] * rstd * w[k];
      if (a.out) {
        Raw8<MOE4_DTYPE_BF16> o;
        o.set(v);
        o.store(row_rsrc<MOE4_DTYPE_BF16>(a.out, row, a.H), col(i));
      }
      if (a.q) {
        uint32_t byte;
        const u32x2 q = mx_quantize8(v, byte);
        if (col(i) < a.H) {
          *reinterpret_cast<u32x2*>(a.q + row * a.H + col(i)) = q;
          if ((tid & 3) == 0) a.qs[row * (a.H / 32) + col(i) / 32] = (uint8_t)byte;
        }
      }
    }
  }
}

struct NormBwdArgs {
  const void *dy, *s, *w, *dres;
  int w_dtype;
  const float* rstd;
  int T, H;
  void* dx;
  float* part;   // [gridDim.x][H] or null
};

// n = s * rstd;  p = w * dy;  dx = rstd * (p - n * mean(p * n)) (+ dres);  dw = sum_t dy * n.
// The workgroup sums its rows' dw in registers, in row order, and its waves' sums through LDS;
// k_sum_rows joins the workgroups' sums. Bound by HBM: 8191 x 2880 in bf16 with dres (189 MB):
// 38.6 us, 4.9 TB/s, and 4.7 us for the join.
template <int DY, int DS, int DX, int W, int NV>
__global__ __launch_bounds__(kNormThreads<W>) void k_add_rmsnorm_bwd(const NormBwdArgs a) {
  constexpr int kRows = W == 1 ? 4 : 1;
  __shared__ float red[2][W];
  const int tid = W == 1 ? lane_id() : threadIdx.x;
  const int w0 = W == 1 ? __builtin_amdgcn_readfirstlane(wave_id()) : 0;
  auto col = [&](int i) { return (i * W * 64 + tid) * 8; };
  Raw8<MOE4_DTYPE_BF16> wb[NV];
  const bool wf = a.w_dtype == MOE4_DTYPE_F32;
  const rsrc_t rw = make_rsrc_uniform(a.w, (uint32_t)a.H * (wf ? 4 : 2));
  if (!wf) {
#pragma unroll
    for (int i = 0; i < NV; ++i) wb[i].load(rw, col(i));
  }
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = 0.0f;
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + w0; row < a.T; row += (int64_t)gridDim.x * kRows) {
    Raw8<DY> y[NV];
    Raw8<DS> s[NV];
    Raw8<DX> e[NV];
    const rsrc_t ry = row_rsrc<DY>(a.dy, row, a.H), rs = row_rsrc<DS>(a.s, row, a.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) y[i].load(ry, col(i));
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i].load(rs, col(i));
    if (a.dres) {
      const rsrc_t re = row_rsrc<DX>(a.dres, row, a.H);
#pragma unroll
      for (int i = 0; i < NV; ++i) e[i].load(re, col(i));
    }
    const float rstd = a.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float g[8], n[8], w[8];
      y[i].get(g);
      s[i].get(n);
      if (wf) {
        Raw8<MOE4_DTYPE_F32> t;
        t.load(rw, col(i));
        t.get(w);
      } else {
        wb[i].get(w);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        n[k] *= rstd;
        dot = fmaf(g[k] * w[k], n[k], dot);
        dw[i][k] = fmaf(g[k], n[k], dw[i][k]);
      }
    }
    dot = row_sum<W>(dot, red, slot);
    slot ^= 1;
    const float mean = dot / (float)a.H;
    const rsrc_t ro = row_rsrc<DX>(a.dx, row, a.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float g[8], n[8], w[8];
      y[i].get(g);
      s[i].get(n);
      if (wf) {
        Raw8<MOE4_DTYPE_F32> t;
        t.load(rw, col(i));
        t.get(w);
      } else {
        wb[i].get(w);
      }
      float o[8] = {};
      if (a.dres) e[i].get(o);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = fmaf(rstd, g[k] * w[k] - n[k] * rstd * mean, o[k]);
      Raw8<DX> st;
      st.set(o);
      st.store(ro, col(i));
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * a.H;
  if constexpr (W == 1) {
    // four waves hold the same columns: wave by wave into LDS
    __shared__ __attribute__((aligned(16))) float sum[NV * 512];
    for (int w = 0; w < 4; ++w) {
      if (w0 == w) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = i * 512 + k * 64 + tid;   // a lane's own slots, conflict-free
            dw[i][k] += w ? sum[c] : 0.0f;
            sum[c] = dw[i][k];
          }
      }
      __syncthreads();
    }
    if (w0 != 3) return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col(i) < a.H) {
      *reinterpret_cast<f32x4*>(part + col(i)) = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
      *reinterpret_cast<f32x4*>(part + col(i) + 4) = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
}

// out[c] = sum over the P rows of part [P][N], in fp32 in a fixed order: thread (y, x) takes
// rows y, y + 32, ... of column 32 blockIdx + x, and the 32 sums of a column meet in LDS. 1024 x
// 2880: 4.7 us, mostly its launch and one round trip.
__global__ __launch_bounds__(1024) void k_sum_rows(const float* part, int P, int N, void* out,
                                                   int dtype) {
  __shared__ float red[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + x;
  float s = 0.0f;
  if (c < N) {
#pragma unroll 8
    for (int p = y; p < P; p += 32) s += part[(int64_t)p * N + c];
  }
  red[y][x] = s;
  __syncthreads();
  if (y == 0 && c < N) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][x];
    if (dtype == MOE4_DTYPE_F32) static_cast<float*>(out)[c] = t;
    else static_cast<uint16_t*>(out)[c] = f32_to_bf16(t);
  }
}

// 8 values a lane, four lanes a block (the maximum by two quad permutes). Bound by HBM: 16384 x
// 4096 from bf16 (203 MB): 36.4 us, 5.6 TB/s.
template <int DT>
__global__ __launch_bounds__(256) void k_quantize_mxfp8(const void* v, int64_t n8, uint8_t* q,
                                                        uint8_t* s) {
  constexpr int es = DT == MOE4_DTYPE_F32 ? 4 : 2;
  // n8 (a multiple of 4) chunks of 8 values; the lanes of a quad take one block, so they
  // leave the loop together
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(v) + i * 8 * es);
    Raw8<DT> r;
    r.r[0] = p[0];
    if constexpr (DT == MOE4_DTYPE_F32) r.r[1] = p[1];
    float x[8];
    r.get(x);
    uint32_t byte;
    *reinterpret_cast<u32x2*>(q + i * 8) = mx_quantize8(x, byte);
    if ((threadIdx.x & 3) == 0) s[i >> 2] = (uint8_t)byte;
  }
}

// Waves of a row: each lane holds at most 32 columns (the registers of the operands of one
// row, at four waves a SIMD), and a row of few goes over four waves. Us in bf16, forward /
// backward with dweight, at 1, 2, 4 and 16 waves:
//   1 x 2048      2.9 / 6.2   2.8 / 5.1   2.4 / 4.5   3.2 / 5.6
//   512 x 2048    3.8 / 8.2   3.9 / 8.2   3.2 / 7.6   5.5 / 8.9
//   512 x 512     2.6 / 5.8   3.5 / 6.3   2.9 / 5.7   5.2 / 7.9
//   2047 x 1024   4.1 / 7.9   5.2 / 11.1  4.9 / 9.9   13 / 18    (one wave would do from here on)
//   8192 x 1024   11.5 / 17   13.8 / 22   12.4 / 18   43 / 60
//   8192 x 2880               29.6 / 34   29.6 / 35   46 / 62
//   1 x 8192                              3.3 / 6.0   3.4 / 5.8
//   8192 x 8192                           97 / 112    96 / 109
constexpr int64_t kManyRows = 2048;
int norm_waves(int64_t T, int H) {
  if (H > 8192) return 16;
  if (H > 4096 || (T < kManyRows && H > 512)) return 4;
  return H > 2048 ? 2 : 1;
}
// workgroups: enough waves for every CU's latency to be covered, each with several rows. Us with at
// most 512, 1024, 2048, 4096 and 8192: 8192 x 2880 32.2, 30.2, 29.6, 29.5, 29.2; 65536 x 2880 353, 274,
// 287, 290, 284; 16 waves a row, 8192 x 16384 199, 200, 198, 196, 189.
int norm_blocks(int64_t T, int W) {
  const int64_t rows = W == 1 ? (T + 3) / 4 : T;
  const int64_t most = W == 16 ? 512 : 2048;
  return (int)(rows < most ? rows : most);
}
// the backward's workgroups each leave a row of partial sums: fewer of them. Us with at most 256,
// 512, 1024, 2048 and 4096: 8192 x 2880 47.7, 34.2, 34.5, 38.5, 44.9; 65536 x 2880 428, 313, 294, 321,
// 316; 16 waves a row, 8192 x 16384 199, 206, 218, 249, 310.
int norm_bwd_blocks(int64_t T, int W) {
  const int64_t rows = W == 1 ? (T + 3) / 4 : T;
  const int64_t most = W == 16 ? 256 : 1024;
  return (int)(rows < most ? rows : most);
}

template <int DX, int DR, int W, int NV>
hipError_t run_norm(const NormArgs& a, hipStream_t s) {
  k_add_rmsnorm<DX, DR, W, NV><<<norm_blocks(a.T, W), kNormThreads<W>, 0, s>>>(a);
  return hipGetLastError();
}
template <int DY, int DS, int DX, int W, int NV>
hipError_t run_norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  k_add_rmsnorm_bwd<DY, DS, DX, W, NV><<<norm_bwd_blocks(a.T, W), kNormThreads<W>, 0, s>>>(a);
  return hipGetLastError();
}

// f(waves, chunks) for the smallest instance that holds H columns
template <typename F>
hipError_t pick_shape(int64_t T, int H, F f) {
  const int W = norm_waves(T, H), nv = (H + 512 * W - 1) / (512 * W);
#define MOE4_NORM(w, n) return f(std::integral_constant<int, w>{}, std::integral_constant<int, n>{})
  if (W == 1) {
    if (nv <= 1) MOE4_NORM(1, 1);
    if (nv <= 2) MOE4_NORM(1, 2);
    MOE4_NORM(1, 4);
  }
  if (W == 2) {
    if (nv <= 3) MOE4_NORM(2, 3);
    MOE4_NORM(2, 4);
  }
  if (W == 4) {
    if (nv <= 1) MOE4_NORM(4, 1);
    if (nv <= 2) MOE4_NORM(4, 2);
    MOE4_NORM(4, 4);
  }
  MOE4_NORM(16, 2);
#undef MOE4_NORM
}

constexpr int B = MOE4_DTYPE_BF16, F = MOE4_DTYPE_F32;

}  // namespace

hipError_t launch_sum_rows(const float* part, int P, int N, void* out, int dtype, hipStream_t s) {
  k_sum_rows<<<(N + 31) / 32, 1024, 0, s>>>(part, P, N, out, dtype);
  return hipGetLastError();
}

hipError_t launch_add_rmsnorm(const void* x, int x_dtype, const void* res, int res_dtype, void* sum,
                              const void* w, int w_dtype, int T, int H, float eps, uint16_t* out,
                              uint8_t* q, uint8_t* qs, float* rstd, hipStream_t s) {
  const NormArgs a = {x, res, sum, w, w_dtype, T, H, eps, out, q, qs, rstd};
  return pick_shape(T, H, [&](auto wc, auto nc) {
    constexpr int W = decltype(wc)::value, N = decltype(nc)::value;
    if (!res) return x_dtype == F ? run_norm<F, 0, W, N>(a, s) : run_norm<B, 0, W, N>(a, s);
    if (x_dtype == F)
      return res_dtype == F ? run_norm<F, F, W, N>(a, s) : run_norm<F, B, W, N>(a, s);
    return res_dtype == F ? run_norm<B, F, W, N>(a, s) : run_norm<B, B, W, N>(a, s);
  });
}

// For this T or any smaller one: from kManyRows on a row of 512 < H <= 2048 goes to one wave,
// and four rows to a workgroup, so fewer workgroups leave sums than just below it.
size_t add_rmsnorm_ws_bytes(int64_t T, int H) {
  const int own = norm_bwd_blocks(T, norm_waves(T, H));
  const int64_t few = T < kManyRows ? T : kManyRows - 1;
  const int below = norm_bwd_blocks(few, norm_waves(few, H));
  return (size_t)(own > below ? own : below) * H * 4;
}

hipError_t launch_add_rmsnorm_backward(const void* dy, int dy_dtype, const void* sv, int s_dtype,
                                       const void* w, int w_dtype, const float* rstd,
                                       const void* dres, int T, int H, void* dx, int dx_dtype,
                                       float* dw, void* ws, hipStream_t st) {
  if (T == 0) return launch_zero_i32(reinterpret_cast<int32_t*>(dw), H, st);
  const NormBwdArgs a = {dy, sv, w, dres, w_dtype, rstd, T, H, dx,
                         dw ? static_cast<float*>(ws) : nullptr};
  hipError_t e = pick_shape(T, H, [&](auto wc, auto nc) {
    constexpr int W = decltype(wc)::value, N = decltype(nc)::value;
    if (dy_dtype == F) {
      if (s_dtype == F)
        return dx_dtype == F ? run_norm_bwd<F, F, F, W, N>(a, st) : run_norm_bwd<F, F, B, W, N>(a, st);
      return dx_dtype == F ? run_norm_bwd<F, B, F, W, N>(a, st) : run_norm_bwd<F, B, B, W, N>(a, st);
    }
    if (s_dtype == F)
      return dx_dtype == F ? run_norm_bwd<B, F, F, W, N>(a, st) : run_norm_bwd<B, F, B, W, N>(a, st);
    return dx_dtype == F ? run_norm_bwd<B, B, F, W, N>(a, st) : run_norm_bwd<B, B, B, W, N>(a, st);
  });
  if (e != hipSuccess || !dw) return e;
  return launch_sum_rows(a.part, norm_bwd_blocks(T, norm_waves(T, H)), H, dw, F, st);
}

hipError_t launch_quantize_mxfp8(const void* x, int x_dtype, int64_t n, uint8_t* q, uint8_t* qs,
                                 hipStream_t s) {
  const int64_t n8 = n / 8, blocks = (n8 + 255) / 256;
  const int grid = (int)(blocks < 16384 ? blocks : 16384);
  if (x_dtype == F) k_quantize_mxfp8<F><<<grid, 256, 0, s>>>(x, n8, q, qs);
  else k_quantize_mxfp8<B><<<grid, 256, 0, s>>>(x, n8, q, qs);
  return hipGetLastError();
}

}  // namespace moe4
