// The MXFP4 quantiser: e2m1 codes in blocks of 32 along a row, one e8m0 scale per block, and, where
// they are asked for, the values that the codes stand for.
#include "internal.hpp"
#include "mx.hpp"
#include "rows.hpp"

namespace moe4 {
namespace {

// 8 values a lane, four lanes a block (the maximum by two quad permutes). Bound by HBM.
template <int DT>
__global__ __launch_bounds__(256) void k_quantize_mxfp4(const void* v, int64_t n8, uint32_t* q,
                                                        uint8_t* s, u32x4* val) {
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
    const uint32_t w = mx4_quantize8(x, byte);
    q[i] = w;
    if ((threadIdx.x & 3) == 0) s[i >> 2] = (uint8_t)byte;
    if (val) {
      const u32x4 nan = {0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
      val[i] = byte == kMxNanScale ? nan : mx4_bf16x8(w, byte);
    }
  }
}

}  // namespace

hipError_t launch_quantize_mxfp4(const void* x, int x_dtype, int64_t n, uint8_t* q, uint8_t* qs,
                                 uint16_t* values, hipStream_t s) {
  const int64_t n8 = n / 8, blocks = (n8 + 255) / 256;
  const int grid = (int)(blocks < 16384 ? blocks : 16384);
  auto* const qw = reinterpret_cast<uint32_t*>(q);
  auto* const val = reinterpret_cast<u32x4*>(values);
  if (x_dtype == MOE4_DTYPE_F32)
    k_quantize_mxfp4<MOE4_DTYPE_F32><<<grid, 256, 0, s>>>(x, n8, qw, qs, val);
  else
    k_quantize_mxfp4<MOE4_DTYPE_BF16><<<grid, 256, 0, s>>>(x, n8, qw, qs, val);
  return hipGetLastError();
}

}  // namespace moe4
