// What stands between two blocks of a model that norms each block's output before it joins the
// residual stream, and the stream in front of the next block:
//   n = b * rstd(b) * w_post;  s = res_scale * residual + block_scale * gate * n  (rounded to the
//   stream's type);  y = s * rstd(s) * w_pre  as bf16, MXFP8 or MXFP4
// and its backward pass. Every element is read and written once; a row stays in registers over both
// of its reductions.
#include "internal.hpp"
#include "mx.hpp"
#include "rows.hpp"

namespace moe4 {
namespace {

// 8 columns of a weight that is bf16 or fp32: bf16 stays in registers over the rows, unless LEAN
template <int NV, bool LEAN = false>
struct RowWeight {
  Raw8<MOE4_DTYPE_BF16> raw[LEAN ? 1 : NV];
  rsrc_t r;
  bool f32;
  __device__ __forceinline__ void init(const void* w, int dtype, int H) {
    f32 = dtype == MOE4_DTYPE_F32;
    r = make_rsrc_uniform(w, w ? (uint32_t)H * (f32 ? 4 : 2) : 0u);
  }
  __device__ __forceinline__ void load(int i, int c) {
    if (!LEAN && !f32) raw[i].load(r, c);
  }
  __device__ __forceinline__ void get(int i, int c, float* w) const {
    if (f32) {
      Raw8<MOE4_DTYPE_F32> t;
      t.load(r, c);
      t.get(w);
    } else if constexpr (LEAN) {
      Raw8<MOE4_DTYPE_BF16> t;
      t.load(r, c);
      t.get(w);
    } else {
      raw[i].get(w);
    }
  }
};

// the sum of 8 squares, in pairs: three additions deep, not eight
__device__ __forceinline__ float squares8(const float* v) {
  float p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = fmaf(v[2 * i], v[2 * i], v[2 * i + 1] * v[2 * i + 1]);
  return (p[0] + p[1]) + (p[2] + p[3]);
}

struct JoinNormArgs {
  const void *b, *res;
  float res_scale, block_scale;
  const float* gate;
  const void *wo, *wi;
  int wo_dtype, wi_dtype;
  int T, H;
  float eps;
  void* sum;
  float *ro, *ri;
  uint16_t* out;
  uint8_t *q, *qs;
  bool q4;
};

// DB, DS: types of the block's output and of the stream.
template <int DB, int DS, int W, int NV>
__global__ __launch_bounds__(kNormThreads<W>) void k_join_norm(const JoinNormArgs a) {
  constexpr int kRows = W == 1 ? 4 : 1;
  __shared__ float red[2][W];
  const int tid = W == 1 ? lane_id() : threadIdx.x;
  const int w0 = W == 1 ? __builtin_amdgcn_readfirstlane(wave_id()) : 0;
  auto col = [&](int i) { return (i * W * 64 + tid) * 8; };
  RowWeight<NV> wo, wi;
  wo.init(a.wo, a.wo_dtype, a.H);
  wi.init(a.wi, a.wi_dtype, a.H);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    wo.load(i, col(i));
    wi.load(i, col(i));
  }
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + w0; row < a.T; row += (int64_t)gridDim.x * kRows) {
    Raw8<DB> b[NV];
    Raw8<DS> r[NV];
    const rsrc_t rb = row_rsrc<DB>(a.b, row, a.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) b[i].load(rb, col(i));
    // (no residual: a resource of no bytes, which reads as zeros)
    const rsrc_t rr = a.res ? row_rsrc<DS>(a.res, row, a.H) : make_rsrc_uniform(a.b, 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) r[i].load(rr, col(i));
    float c = a.block_scale * (a.gate ? a.gate[row] : 1.0f);
    if (a.wo) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v[8];
        b[i].get(v);
        ss += squares8(v);
      }
      ss = row_sum<W>(ss, red, slot);
      slot ^= 1;
      const float ro = rsqrtf(ss / (float)a.H + a.eps);
      if (a.ro && tid == 0) a.ro[row] = ro;
      c *= ro;
    }
    // the row that the second norm sees is the one that the stream holds, rounded to its type
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8], u[8], w[8];
      b[i].get(v);
      r[i].get(u);
      if (a.wo) wo.get(i, col(i), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // (b * rstd first: b * w_post may leave fp32's range where their product with rstd does not)
        v[k] *= c;
        u[k] = fmaf(a.res_scale, u[k], a.wo ? v[k] * w[k] : v[k]);
      }
      r[i].set(u);
      r[i].get(u);
      ss += squares8(u);
    }
    if (a.sum) {
      const rsrc_t rs = row_rsrc<DS>(a.sum, row, a.H);
#pragma unroll
      for (int i = 0; i < NV; ++i) r[i].store(rs, col(i));
    }
    if (!a.wi) continue;
    ss = row_sum<W>(ss, red, slot);
    slot ^= 1;
    const float ri = rsqrtf(ss / (float)a.H + a.eps);
    if (a.ri && tid == 0) a.ri[row] = ri;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8], w[8];
      r[i].get(v);
      wi.get(i, col(i), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] * ri * w[k];
      if (a.out) {
        Raw8<MOE4_DTYPE_BF16> o;
        o.set(v);
        o.store(row_rsrc<MOE4_DTYPE_BF16>(a.out, row, a.H), col(i));
      }
      if (a.q) {
        uint32_t byte;
        if (a.q4) {
          const uint32_t q = mx4_quantize8(v, byte);
          if (col(i) < a.H)
            *reinterpret_cast<uint32_t*>(a.q + row * (a.H / 2) + col(i) / 2) = q;
        } else {
          const u32x2 q = mx_quantize8(v, byte);
          if (col(i) < a.H) *reinterpret_cast<u32x2*>(a.q + row * a.H + col(i)) = q;
        }
        if (col(i) < a.H && (tid & 3) == 0) a.qs[row * (a.H / 32) + col(i) / 32] = (uint8_t)byte;
      }
    }
  }
}

struct JoinNormBwdArgs {
  const void *dy, *s, *b, *ds;
  const void *wo, *wi;
  int wo_dtype, wi_dtype;
  const float *gate, *ro, *ri;
  float res_scale, block_scale;
  int T, H;
  void *db, *dres;
  float* dgate;
  float* part;   // [gridDim.x][2][H]: dw_post, dw_pre; or null
};

// With t = s * rstd_pre, m = b * rstd_post (m = b without w_post):
//   dS = rstd_pre * (w_pre dy - t mean(w_pre dy t)) + ds;   dres = res_scale dS
//   q = w_post dS (dS without);  D = sum_h q m;             dgate = block_scale D
//   db = block_scale gate rstd_post (q - m D / H)           (without w_post: block_scale gate dS)
//   dw_post = block_scale sum_t gate dS m;                  dw_pre = sum_t dy t
// One pass: dS stays in registers between the two reductions. The workgroup sums its rows' dw in
// registers, in row order, and its waves' sums through LDS; k_sum_rows joins the workgroups'. At
// sixteen waves a row a lane has 128 registers, which both sums and four operands do not fit: there
// dy, s and the weights are read again after the first reduction (from the caches).
template <int DY, int DS, int DB, int W, int NV>
__global__ __launch_bounds__(kNormThreads<W>) void k_join_norm_bwd(const JoinNormBwdArgs a) {
  constexpr int kRows = W == 1 ? 4 : 1;
  constexpr bool kLean = W == 16;
  __shared__ float red[2][W];
  const int tid = W == 1 ? lane_id() : threadIdx.x;
  const int w0 = W == 1 ? __builtin_amdgcn_readfirstlane(wave_id()) : 0;
  auto col = [&](int i) { return (i * W * 64 + tid) * 8; };
  RowWeight<NV, kLean> wo, wi;
  wo.init(a.wo, a.wo_dtype, a.H);
  wi.init(a.wi, a.wi_dtype, a.H);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    wo.load(i, col(i));
    wi.load(i, col(i));
  }
  float dwo[NV][8], dwi[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dwo[i][k] = dwi[i][k] = 0.0f;
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + w0; row < a.T; row += (int64_t)gridDim.x * kRows) {
    Raw8<DY> y[NV];
    Raw8<DS> s[NV], e[NV];
    Raw8<DB> b[NV];
    const rsrc_t ry = a.wi ? row_rsrc<DY>(a.dy, row, a.H) : make_rsrc_uniform(a.b, 0);
    const rsrc_t rs = a.wi ? row_rsrc<DS>(a.s, row, a.H) : make_rsrc_uniform(a.b, 0);
    const rsrc_t re = a.ds ? row_rsrc<DS>(a.ds, row, a.H) : make_rsrc_uniform(a.b, 0);
    const rsrc_t rb = row_rsrc<DB>(a.b, row, a.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      y[i].load(ry, col(i));
      s[i].load(rs, col(i));
    }
    if constexpr (!kLean) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        e[i].load(re, col(i));
        b[i].load(rb, col(i));
      }
    }
    const float ri = a.wi ? a.ri[row] : 0.0f, ro = a.wo ? a.ro[row] : 1.0f;
    const float c = a.block_scale * (a.gate ? a.gate[row] : 1.0f);
    float mean = 0.0f;
    if (a.wi) {
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float g[8], t[8], w[8];
        y[i].get(g);
        s[i].get(t);
        wi.get(i, col(i), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          t[k] *= ri;
          dot = fmaf(g[k] * w[k], t[k], dot);
          dwi[i][k] = fmaf(g[k], t[k], dwi[i][k]);
        }
      }
      mean = row_sum<W>(dot, red, slot) / (float)a.H;
      slot ^= 1;
    }
    if constexpr (kLean) {
      // (the empty asm keeps the compiler from taking the values of the first reading)
      asm volatile("" ::: "memory");
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        y[i].load(ry, col(i));
        s[i].load(rs, col(i));
        e[i].load(re, col(i));
        b[i].load(rb, col(i));
      }
    }
    float d[NV][8];   // dS, then what db is made of
    float along = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float g[8], t[8], w[8], m[8];
      e[i].get(d[i]);
      if (a.wi) {
        y[i].get(g);
        s[i].get(t);
        wi.get(i, col(i), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[i][k] = fmaf(ri, g[k] * w[k] - t[k] * ri * mean, d[i][k]);
      }
      if (a.dres) {
        Raw8<DS> st;
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = a.res_scale * d[i][k];
        st.set(t);
        st.store(row_rsrc<DS>(a.dres, row, a.H), col(i));
      }
      b[i].get(m);
      if (a.wo) wo.get(i, col(i), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] *= ro;
        if (a.wo) {
          dwo[i][k] = fmaf(c * d[i][k], m[k], dwo[i][k]);
          d[i][k] *= w[k];
        }
        along = fmaf(d[i][k], m[k], along);
      }
    }
    float inner = 0.0f;
    if (a.wo || a.dgate) {
      along = row_sum<W>(along, red, slot);
      slot ^= 1;
      if (a.dgate && tid == 0) a.dgate[row] = a.block_scale * along;
      if (a.wo) inner = along / (float)a.H;
    }
    const rsrc_t ro_ = row_rsrc<DB>(a.db, row, a.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float m[8];
      b[i].get(m);
#pragma unroll
      for (int k = 0; k < 8; ++k) d[i][k] = c * ro * (a.wo ? d[i][k] - m[k] * ro * inner : d[i][k]);
      Raw8<DB> st;
      st.set(d[i]);
      st.store(ro_, col(i));
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.H;
  if constexpr (W == 1) {
    // four waves hold the same columns: wave by wave into LDS
    __shared__ __attribute__((aligned(16))) float sum[2 * NV * 512];
    for (int w = 0; w < 4; ++w) {
      if (w0 == w) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = i * 512 + k * 64 + tid;   // a lane's own slots, conflict-free
            dwo[i][k] += w ? sum[c] : 0.0f;
            sum[c] = dwo[i][k];
            dwi[i][k] += w ? sum[NV * 512 + c] : 0.0f;
            sum[NV * 512 + c] = dwi[i][k];
          }
      }
      __syncthreads();
    }
    if (w0 != 3) return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col(i) < a.H) {
      float* const o = part + col(i);
      *reinterpret_cast<f32x4*>(o) = f32x4{dwo[i][0], dwo[i][1], dwo[i][2], dwo[i][3]};
      *reinterpret_cast<f32x4*>(o + 4) = f32x4{dwo[i][4], dwo[i][5], dwo[i][6], dwo[i][7]};
      *reinterpret_cast<f32x4*>(o + a.H) = f32x4{dwi[i][0], dwi[i][1], dwi[i][2], dwi[i][3]};
      *reinterpret_cast<f32x4*>(o + a.H + 4) = f32x4{dwi[i][4], dwi[i][5], dwi[i][6], dwi[i][7]};
    }
}

// A workgroup to a row (us, us with at most 2048 workgroups: 4096 rows of 2880 25, 28, 16384 83, 100), but
// for the widest rows, whose workgroups keep their weights (4096 of 16384: 135, 120 with 512).
int join_blocks(int64_t T, int W) {
  const int64_t rows = W == 1 ? (T + 3) / 4 : T;
  const int64_t most = W == 16 ? 512 : 1 << 20;
  return (int)(rows < most ? rows : most);
}
// the backward's workgroups each leave two rows of partial sums: fewer of them
int join_bwd_blocks(int64_t T, int W) {
  const int64_t rows = W == 1 ? (T + 3) / 4 : T;
  const int64_t most = W == 16 ? 256 : 1024;
  return (int)(rows < most ? rows : most);
}

constexpr int B = MOE4_DTYPE_BF16, F = MOE4_DTYPE_F32;

}  // namespace

hipError_t launch_join_norm(const void* b, int b_dtype, const void* res, int s_dtype,
                            float res_scale, float block_scale, const float* gate,
                            const void* w_post, int post_dtype, const void* w_pre, int pre_dtype,
                            int T, int H, float eps, void* sum, float* ro, float* ri,
                            uint16_t* out, uint8_t* q, uint8_t* qs, bool q4, hipStream_t s) {
  const JoinNormArgs a = {b, res, res_scale, block_scale, gate, w_post, w_pre, post_dtype,
                          pre_dtype, T, H, eps, sum, ro, ri, out, q, qs, q4};
  return pick_shape(T, H, [&](auto wc, auto nc) {
    constexpr int W = decltype(wc)::value, N = decltype(nc)::value;
    auto run = [&](auto* k) {
      k<<<join_blocks(T, W), kNormThreads<W>, 0, s>>>(a);
      return hipGetLastError();
    };
    if (b_dtype == F) return s_dtype == F ? run(&k_join_norm<F, F, W, N>) : run(&k_join_norm<F, B, W, N>);
    return s_dtype == F ? run(&k_join_norm<B, F, W, N>) : run(&k_join_norm<B, B, W, N>);
  });
}

// For this T or any smaller one: from kManyRows on a row of 512 < H <= 2048 goes to one wave,
// and four rows to a workgroup, so fewer workgroups leave sums than just below it.
size_t join_norm_ws_bytes(int64_t T, int H) {
  const int own = join_bwd_blocks(T, norm_waves(T, H));
  const int64_t few = T < kManyRows ? T : kManyRows - 1;
  const int below = join_bwd_blocks(few, norm_waves(few, H));
  return (size_t)(own > below ? own : below) * H * 8;
}

hipError_t launch_join_norm_backward(const void* dy, int dy_dtype, const void* sv, int s_dtype,
                                     const void* b, int b_dtype, const void* ds, float res_scale,
                                     float block_scale, const float* gate, const void* w_post,
                                     int post_dtype, const void* w_pre, int pre_dtype,
                                     const float* ro, const float* ri, int T, int H, void* db,
                                     void* dres, float* dgate, float* dw_post, float* dw_pre,
                                     void* ws, hipStream_t st) {
  if (T == 0) {
    for (float* p : {dw_post, dw_pre})
      if (hipError_t e = p ? launch_zero_i32(reinterpret_cast<int32_t*>(p), H, st) : hipSuccess;
          e != hipSuccess)
        return e;
    return hipSuccess;
  }
  const bool sums = dw_post || dw_pre;
  const JoinNormBwdArgs a = {dy, sv, b, ds, w_post, w_pre, post_dtype, pre_dtype, gate, ro, ri,
                             res_scale, block_scale, T, H, db, dres, dgate,
                             sums ? static_cast<float*>(ws) : nullptr};
  hipError_t e = pick_shape(T, H, [&](auto wc, auto nc) {
    constexpr int W = decltype(wc)::value, N = decltype(nc)::value;
    auto run = [&](auto* k) {
      k<<<join_bwd_blocks(T, W), kNormThreads<W>, 0, st>>>(a);
      return hipGetLastError();
    };
    if (dy_dtype == F) {
      if (s_dtype == F)
        return b_dtype == F ? run(&k_join_norm_bwd<F, F, F, W, N>) : run(&k_join_norm_bwd<F, F, B, W, N>);
      return b_dtype == F ? run(&k_join_norm_bwd<F, B, F, W, N>) : run(&k_join_norm_bwd<F, B, B, W, N>);
    }
    if (s_dtype == F)
      return b_dtype == F ? run(&k_join_norm_bwd<B, F, F, W, N>) : run(&k_join_norm_bwd<B, F, B, W, N>);
    return b_dtype == F ? run(&k_join_norm_bwd<B, B, F, W, N>) : run(&k_join_norm_bwd<B, B, B, W, N>);
  });
  if (e != hipSuccess || !sums) return e;
  const int P = join_bwd_blocks(T, norm_waves(T, H));
  // both halves of the sums in one launch, or the half that is wanted: [P][2][H]
  if (dw_post && dw_pre) return launch_sum_rows2(a.part, P, 2 * H, dw_post, F, H, dw_pre, st);
  return launch_sum_rows_of(dw_post ? a.part : a.part + H, P, 2 * H, H, dw_post ? dw_post : dw_pre, F, st);
}

}  // namespace moe4
