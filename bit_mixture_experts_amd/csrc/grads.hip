// The global norm of a list of gradients, and clipping by it.
//
// The list travels in the kernels' arguments, kGradBatch tensors to a launch, so nothing is
// copied to the device and a captured graph holds the list by value. Work is dealt in chunks
// of kGradChunk elements of one tensor. Squares are summed in fp64 (an fp32 square overflows from
// 1.9e19 on and vanishes below 1e-23): the norm is right to fp32 for any finite gradients, an
// infinity where it passes fp32's range, and the fp64 adds hide behind the loads.
//
// Bound by HBM. 88 million fp32 values in 48 tensors (352 MB): squares 81-92 us, 4.1 TB/s; scaling
// to another place 108-115 us, 6.3 TB/s, part of its reads from the caches. Fp64 partial sums, at most
// 2048 a launch (1024 left CUs idle between chunks: 88 us; chunks of half the size 86), are added
// up by every scaling workgroup for itself, which saves a launch while they are few.
#include "internal.hpp"
#include "common.hpp"

namespace moe4 {
namespace {

constexpr int kGradBatch = 128, kGradChunk = 8192, kGradParts = 2048;
// The most partial sums that every scaling workgroup adds up for itself; more of them are joined by
// a launch first, since their number grows with the list and so does that of the workgroups. Us
// by themselves and joined: 2 tensors, 10 sums 6.5 and 8.1; 64, 1024 sums 21.9 and 23.7; 257, 4112
// sums 83.4 and 83.3; 512, 8192 sums 190 and 182; 6144, 12288 sums 700 and 640; 32768 tensors of
// 20 elements 2954 and 2068.
constexpr int kScaleParts = kGradParts;

struct GradBatch {
  const void* in[kGradBatch];
  void* out[kGradBatch];
  int64_t numel[kGradBatch];
  int32_t first[kGradBatch];   // the tensor's first chunk
  uint8_t f32[kGradBatch];
  int32_t n, chunks;
};
static_assert(sizeof(GradBatch) <= 4000, "fits a kernel's arguments");

__device__ __forceinline__ int tensor_of(const GradBatch& b, int chunk) {
  int lo = 0, hi = b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  if (lane_id() == 0) red[wave_id()] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

// f(index, 4-byte or 2-byte values) over the 16-byte pieces of a chunk
template <typename T, int PER, typename F4, typename F1>
__device__ __forceinline__ void walk(const T* p, int64_t n, F4 whole, F1 single) {
  constexpr int kPieces = kGradChunk / PER / 256;
  if (n >= kGradChunk) {
    u32x4 v[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      v[i] = reinterpret_cast<const u32x4*>(p)[i * 256 + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) whole(i * 256 + threadIdx.x, v[i]);
  } else {
    const int np = (int)(n / PER);
    for (int i = threadIdx.x; i < np; i += 256) whole(i, reinterpret_cast<const u32x4*>(p)[i]);
    for (int i = np * PER + threadIdx.x; i < n; i += 256) single(i);
  }
}

__global__ __launch_bounds__(256) void k_grad_squares(const GradBatch b, double* part) {
  __shared__ double red[4];
  double s = 0.0;
  for (int c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const int t = __builtin_amdgcn_readfirstlane(tensor_of(b, c));
    const int64_t at = (int64_t)(c - b.first[t]) * kGradChunk, n = b.numel[t] - at;
    auto add = [&](float v) { s = fma((double)v, (double)v, s); };
    if (b.f32[t]) {
      const float* p = static_cast<const float*>(b.in[t]) + at;
      walk<float, 4>(p, n, [&](int, u32x4 v) {
#pragma unroll
        for (int k = 0; k < 4; ++k) add(__uint_as_float(v[k]));
      }, [&](int i) { add(p[i]); });
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(b.in[t]) + at;
      walk<uint16_t, 8>(p, n, [&](int, u32x4 v) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          add(bf16lo(v[k]));
          add(bf16hi(v[k]));
        }
      }, [&](int i) { add(bf16_to_f32(p[i])); });
    }
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// the sum of the squares from the partial sums, in the same order wherever it is taken
__device__ __forceinline__ double total_squares(const double* part, int nparts, double* red) {
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < nparts; i += 256) s += part[i];
  return block_sum(s, red);
}

__global__ __launch_bounds__(256) void k_grad_norm(const double* part, int nparts, float* norm) {
  __shared__ double red[4];
  const double s = total_squares(part, nparts, red);
  if (threadIdx.x == 0) norm[0] = (float)sqrt(s);
}

__global__ __launch_bounds__(256) void k_grad_join(const double* part, int nparts, double* total) {
  __shared__ double red[4];
  const double s = total_squares(part, nparts, red);
  if (threadIdx.x == 0) total[0] = s;
}

// out = g * min(1, max_norm / (norm + 1e-6)), rounded once to the gradient's type. The norm is the
// fp32 one that is written, or, where finite gradients pass fp32's range, the fp64 one. A norm that
// is no finite number leaves the gradients as they are: the caller reads it and drops the step.
__global__ __launch_bounds__(256) void k_grad_scale(const GradBatch b, const double* part,
                                                    int nparts, const float* norm_in,
                                                    float max_norm, float* norm_out) {
  __shared__ double red[4];
  const double exact = norm_in ? (double)norm_in[0] : sqrt(total_squares(part, nparts, red));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) norm_out[0] = (float)exact;
  const double norm = __builtin_isfinite((float)exact) ? (double)(float)exact : exact;
  const double k = (double)max_norm / (norm + 1e-6);
  const bool clip = k < 1.0 && __builtin_isfinite(norm);
  // a factor below fp32's normal range would hold few bits: it goes in two, the second exact
  const bool tiny = clip && k < 0x1p-126;
  const float coef = clip ? (float)(tiny ? k * 0x1p126 : k) : 1.0f, down = tiny ? 0x1p-126f : 1.0f;
  auto scaled = [&](float g) { return g * coef * down; };
  // back to front: what the norm's pass read last is still in the caches
  for (int c = b.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int t = __builtin_amdgcn_readfirstlane(tensor_of(b, c));
    if (!clip && b.in[t] == b.out[t]) continue;
    const int64_t at = (int64_t)(c - b.first[t]) * kGradChunk, n = b.numel[t] - at;
    if (b.f32[t]) {
      const float* p = static_cast<const float*>(b.in[t]) + at;
      float* o = static_cast<float*>(b.out[t]) + at;
      walk<float, 4>(p, n, [&](int i, u32x4 v) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = __float_as_uint(scaled(__uint_as_float(v[q])));
        reinterpret_cast<u32x4*>(o)[i] = v;
      }, [&](int i) { o[i] = scaled(p[i]); });
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(b.in[t]) + at;
      uint16_t* o = static_cast<uint16_t*>(b.out[t]) + at;
      walk<uint16_t, 8>(p, n, [&](int i, u32x4 v) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = pack_bf16x2(scaled(bf16lo(v[q])), scaled(bf16hi(v[q])));
        reinterpret_cast<u32x4*>(o)[i] = v;
      }, [&](int i) { o[i] = f32_to_bf16(scaled(bf16_to_f32(p[i]))); });
    }
  }
}

int grad_blocks(int chunks) { return chunks < kGradParts ? chunks : kGradParts; }

// f(batch, blocks) for every launch's worth of the list; empty tensors are left out
template <typename F>
hipError_t each_batch(const void* const* in, void* const* out, const int64_t* numel,
                      const int32_t* dtype, int n, F f) {
  GradBatch b;
  b.n = b.chunks = 0;
  hipError_t e = hipSuccess;
  for (int i = 0; i <= n && e == hipSuccess; ++i) {
    if (i == n || b.n == kGradBatch) {
      if (b.n) e = f(b, grad_blocks(b.chunks));
      b.n = b.chunks = 0;
      if (i == n) break;
    }
    if (numel[i] == 0) continue;
    b.in[b.n] = in[i];
    b.out[b.n] = out ? out[i] : const_cast<void*>(in[i]);
    b.numel[b.n] = numel[i];
    b.first[b.n] = b.chunks;
    b.f32[b.n] = dtype[i] == MOE4_DTYPE_F32;
    b.chunks += (int)((numel[i] + kGradChunk - 1) / kGradChunk);
    ++b.n;
  }
  return e;
}

hipError_t squares(const void* const* in, const int64_t* numel, const int32_t* dtype, int n,
                   double* part, int* nparts, hipStream_t s) {
  *nparts = 0;
  return each_batch(in, nullptr, numel, dtype, n, [&](const GradBatch& b, int blocks) {
    k_grad_squares<<<blocks, 256, 0, s>>>(b, part + *nparts);
    *nparts += blocks;
    return hipGetLastError();
  });
}

}  // namespace

size_t grad_ws_bytes(int64_t n) {
  return align_up((size_t)((n + kGradBatch - 1) / kGradBatch) * kGradParts * 8 + 8, 256);
}
int64_t grad_most_numel() { return (int64_t)kGradChunk << 23; }

hipError_t launch_grad_norm(const void* const* in, const int64_t* numel, const int32_t* dtype,
                            int n, float* norm, void* ws, hipStream_t s) {
  int parts = 0;
  hipError_t e = squares(in, numel, dtype, n, static_cast<double*>(ws), &parts, s);
  if (e != hipSuccess) return e;
  k_grad_norm<<<1, 256, 0, s>>>(static_cast<double*>(ws), parts, norm);
  return hipGetLastError();
}

hipError_t launch_clip_grads(const void* const* in, void* const* out, const int64_t* numel,
                             const int32_t* dtype, int n, float max_norm, const float* norm_in,
                             float* norm_out, void* ws, hipStream_t s) {
  int parts = 0;
  hipError_t e = hipSuccess;
  double* part = static_cast<double*>(ws);
  if (!norm_in) {
    e = squares(in, numel, dtype, n, part, &parts, s);
    if (e != hipSuccess) return e;
    if (parts > kScaleParts) {
      k_grad_join<<<1, 256, 0, s>>>(part, parts, part + parts);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      part += parts;
      parts = 1;
    }
  }
  bool first = true;
  e = each_batch(in, out, numel, dtype, n, [&](const GradBatch& b, int blocks) {
    k_grad_scale<<<blocks, 256, 0, s>>>(b, part, parts, norm_in, max_norm,
                                        first ? norm_out : nullptr);
    first = false;
    return hipGetLastError();
  });
  if (e != hipSuccess || !first || !norm_out) return e;
  // nothing to scale: the norm is 0 (or the one given)
  GradBatch b;
  b.n = b.chunks = 0;
  k_grad_scale<<<1, 256, 0, s>>>(b, part, 0, norm_in, max_norm, norm_out);
  return hipGetLastError();
}

}  // namespace moe4
