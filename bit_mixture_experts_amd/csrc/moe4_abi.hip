// C ABI of libmoe4: argument validation (synchronous, before anything is
// enqueued) and dispatch to the kernel launchers. Every refusal names the
// first offending argument; nothing falls back to another computation
// (project page "experts4bit-qlora", "Do not use this when" and "Limitations --
// qlora-fused-moe-experts": counts or loud refusals, never a silent fallback;
// a base whose epilogue differs from the kernel's is refused).
#include <stdarg.h>
#include <stdio.h>

#include <mutex>

#include "internal.hpp"

namespace {

// Scratch of moe4_expert_forward_noalloc: file-scope device memory, one copy
// on every GPU the library runs on, held until the process ends. In host code
// `scratch` names a host-side stand-in: its device address comes from
// hipGetSymbolAddress, once per device (scratch_of_current_device).
constexpr size_t kNoAllocScratchBytes = (size_t)16 << 20;
static_assert(MOE4_NOALLOC_SCRATCH_BYTES == kNoAllocScratchBytes, "moe4.h states the size");
static __device__ __align__(256) uint8_t scratch[kNoAllocScratchBytes];
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch[kMaxDevices] = {};

thread_local char g_err[512] = "";
thread_local int g_variant = 0;
thread_local hipEvent_t const* g_events = nullptr;

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

int ok() {
  g_err[0] = '\0';
  return MOE4_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

#define REQUIRE_PTR(p, name)                                            \
  do {                                                                  \
    if ((p) == nullptr) return fail(MOE4_EINVAL, "%s is NULL", name);   \
  } while (0)
#define REQUIRE_ALIGN(p, a, name)                                                   \
  do {                                                                              \
    if ((p) != nullptr && !aligned((p), (a)))                                       \
      return fail(MOE4_EALIGN, "%s is not %d-byte aligned", name, (int)(a));        \
  } while (0)

int launched(hipError_t e, const char* what) {
  if (e != hipSuccess)
    return fail(MOE4_EDEVICE, "%s: HIP launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

// Shared checks of a moe4_experts descriptor.
int check_experts(const moe4_experts* ex) {
  if (ex == nullptr) return fail(MOE4_EINVAL, "moe4_experts is NULL");
  if (ex->format != MOE4_FMT_NF4 && ex->format != MOE4_FMT_MXFP4 &&
      ex->format != MOE4_FMT_NF4_DQ)
    return fail(MOE4_EINVAL, "moe4_experts.format %s (%d)", ex->format ? "unknown" : "unset",
                ex->format);
  if (ex->gu_layout != MOE4_GU_HALVES && ex->gu_layout != MOE4_GU_INTERLEAVED)
    return fail(MOE4_EINVAL, "moe4_experts.gu_layout %s (%d)",
                ex->gu_layout ? "unknown" : "unset", ex->gu_layout);
  if (ex->act != MOE4_ACT_SWIGLU && ex->act != MOE4_ACT_SWIGLU_CLAMPED)
    return fail(MOE4_EINVAL, "moe4_experts.act %s (%d)", ex->act ? "unknown" : "unset", ex->act);
  if (ex->variant != MOE4_VARIANT_AUTO && ex->variant != MOE4_VARIANT_SKINNY &&
      ex->variant != MOE4_VARIANT_TILED)
    return fail(MOE4_EINVAL, "moe4_experts.variant unknown (%d)", ex->variant);
  if (ex->E < 1 || ex->E > 1024)
    return fail(MOE4_ESHAPE, "moe4_experts.E = %d outside [1, 1024]", ex->E);
  if (ex->H <= 0 || ex->I <= 0)
    return fail(MOE4_ESHAPE, "moe4_experts.H = %d, I = %d must be positive", ex->H, ex->I);
  const int blk = ex->format == MOE4_FMT_MXFP4 ? 32 : 64;
  if (ex->H % blk)
    return fail(MOE4_ESHAPE, "moe4_experts.H = %d is not a multiple of %d", ex->H, blk);
  if (ex->I % blk)
    return fail(MOE4_ESHAPE, "moe4_experts.I = %d is not a multiple of %d", ex->I, blk);
  if ((int64_t)ex->E * 2 * ex->I * ex->H > ((int64_t)1 << 40))
    return fail(MOE4_ESHAPE, "moe4_experts: stack of %lld weights is beyond the supported 2^40",
                (long long)ex->E * 2 * ex->I * ex->H);
  // the GEMM kernels address one expert's matrix with 32-bit byte offsets
  if ((int64_t)ex->I * ex->H >= ((int64_t)1 << 31) - ((int64_t)1 << 24))
    return fail(MOE4_ESHAPE, "moe4_experts: I*H = %lld; one expert's packed matrix must stay "
                "under 2 GiB", (long long)ex->I * ex->H);
  // the GEMM kernels address an activation tile (up to 320 rows of K = H or
  // 2I bf16 values) and an output tile (up to 320 rows of H fp32 values) with
  // 32-bit byte offsets
  {
    const int64_t kmax = ex->H > 2 * (int64_t)ex->I ? ex->H : 2 * (int64_t)ex->I;
    if (320 * 4 * kmax >= ((int64_t)1 << 31) - ((int64_t)1 << 24))
      return fail(MOE4_ESHAPE, "moe4_experts: max(H, 2I) = %lld; a 320-row fp32 tile "
                  "must stay under 2 GiB", (long long)kmax);
  }
  REQUIRE_PTR(ex->gu_q, "moe4_experts.gu_q");
  REQUIRE_PTR(ex->gu_s, "moe4_experts.gu_s");
  REQUIRE_PTR(ex->dn_q, "moe4_experts.dn_q");
  REQUIRE_PTR(ex->dn_s, "moe4_experts.dn_s");
  REQUIRE_ALIGN(ex->gu_q, 16, "moe4_experts.gu_q");
  REQUIRE_ALIGN(ex->dn_q, 16, "moe4_experts.dn_q");
  if (ex->format == MOE4_FMT_NF4) {
    REQUIRE_ALIGN(ex->gu_s, 4, "moe4_experts.gu_s");
    REQUIRE_ALIGN(ex->dn_s, 4, "moe4_experts.dn_s");
  }
  if (ex->format == MOE4_FMT_NF4_DQ) {
    REQUIRE_PTR(ex->gu_s2, "moe4_experts.gu_s2");
    REQUIRE_PTR(ex->dn_s2, "moe4_experts.dn_s2");
    REQUIRE_PTR(ex->gu_soff, "moe4_experts.gu_soff");
    REQUIRE_PTR(ex->dn_soff, "moe4_experts.dn_soff");
    REQUIRE_PTR(ex->dq_book, "moe4_experts.dq_book");
    REQUIRE_ALIGN(ex->gu_s2, 4, "moe4_experts.gu_s2");
    REQUIRE_ALIGN(ex->dn_s2, 4, "moe4_experts.dn_s2");
    REQUIRE_ALIGN(ex->gu_soff, 4, "moe4_experts.gu_soff");
    REQUIRE_ALIGN(ex->dn_soff, 4, "moe4_experts.dn_soff");
    REQUIRE_ALIGN(ex->dq_book, 4, "moe4_experts.dq_book");
  } else if (ex->gu_s2 || ex->dn_s2 || ex->gu_soff || ex->dn_soff || ex->dq_book) {
    return fail(MOE4_EINVAL, "moe4_experts: double-quantised absmax fields given for format %d",
                ex->format);
  }
  REQUIRE_ALIGN(ex->gu_bias, 2, "moe4_experts.gu_bias");
  REQUIRE_ALIGN(ex->dn_bias, 2, "moe4_experts.dn_bias");
  if (ex->act == MOE4_ACT_SWIGLU_CLAMPED) {
    if (!(ex->act_limit > 0.0f) || !(ex->act_alpha > 0.0f))
      return fail(MOE4_EINVAL,
                  "moe4_experts.act_alpha/act_limit must be positive for the clamped GLU "
                  "(got %g, %g)",
                  (double)ex->act_alpha, (double)ex->act_limit);
  }
  if ((ex->lora_A == nullptr) != (ex->lora_B == nullptr))
    return fail(MOE4_EINVAL, "moe4_experts.lora_A and lora_B must be given together");
  if (ex->lora_A) {
    if (ex->lora_r < 1 || ex->lora_r > 64)
      return fail(MOE4_ESHAPE, "moe4_experts.lora_r = %d outside [1, 64]", ex->lora_r);
    REQUIRE_ALIGN(ex->lora_A, 16, "moe4_experts.lora_A");
    REQUIRE_ALIGN(ex->lora_B, 2, "moe4_experts.lora_B");
    if (ex->H % 8) return fail(MOE4_ESHAPE, "LoRA needs H %% 8 == 0 (H = %d)", ex->H);
  }
  return MOE4_OK;
}

// Device address of `scratch` on the current device, looked up on the first
// call per device (with that device current) and kept.
int scratch_of_current_device(void* stream, void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess)
    return fail(MOE4_EDEVICE, "moe4_expert_forward_noalloc: hipGetDevice failed: %s",
                hipGetErrorString(e));
  if (stream != nullptr) {
    int sdev = -1;
    e = hipStreamGetDevice(static_cast<hipStream_t>(stream), &sdev);
    if (e != hipSuccess)
      return fail(MOE4_EINVAL, "moe4_expert_forward_noalloc: stream: %s", hipGetErrorString(e));
    if (sdev != dev)
      return fail(MOE4_EINVAL,
                  "moe4_expert_forward_noalloc: stream is on device %d, the current device is %d",
                  sdev, dev);
  }
  if (dev < 0 || dev >= kMaxDevices)
    return fail(MOE4_EDEVICE, "moe4_expert_forward_noalloc: device %d beyond the %d supported",
                dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch[dev] == nullptr) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || p == nullptr)
      return fail(MOE4_EDEVICE, "moe4_expert_forward_noalloc: device %d: scratch address: %s",
                  dev, hipGetErrorString(e));
    g_scratch[dev] = p;
  }
  *out = g_scratch[dev];
  return MOE4_OK;
}

int check_ws(void* ws, size_t ws_bytes, size_t need, const char* fn) {
  if (need == 0) return MOE4_OK;
  if (ws == nullptr || ws_bytes < need)
    return fail(MOE4_EWORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn,
                ws ? ws_bytes : (size_t)0, need);
  if (!aligned(ws, 256)) return fail(MOE4_EALIGN, "%s: ws is not 256-byte aligned", fn);
  return MOE4_OK;
}

}  // namespace

extern "C" {

int moe4_quantize_nf4(const float* w, int64_t n, int32_t blocksize, uint8_t* packed,
                      float* absmax, void* stream) {
  if (blocksize != 64) return fail(MOE4_EUNSUPPORTED, "blocksize = %d; NF4 uses 64", blocksize);
  if (n < 0 || n % 64) return fail(MOE4_ESHAPE, "n = %lld is not a non-negative multiple of 64",
                                   (long long)n);
  if (n == 0) return ok();
  REQUIRE_PTR(w, "w");
  REQUIRE_PTR(packed, "packed");
  REQUIRE_PTR(absmax, "absmax");
  REQUIRE_ALIGN(w, 16, "w");
  REQUIRE_ALIGN(packed, 4, "packed");
  REQUIRE_ALIGN(absmax, 4, "absmax");
  return launched(moe4::launch_quantize_nf4(w, n, packed, absmax, (hipStream_t)stream),
                  "moe4_quantize_nf4");
}

int moe4_decode_mxfp4(const uint8_t* blocks, const uint8_t* scales, int64_t R, int64_t K,
                      uint16_t* out, void* stream) {
  if (R < 0 || K < 0 || K % 32)
    return fail(MOE4_ESHAPE, "R = %lld, K = %lld: need R >= 0 and K a non-negative multiple of 32",
                (long long)R, (long long)K);
  if (R == 0 || K == 0) return ok();
  REQUIRE_PTR(blocks, "blocks");
  REQUIRE_PTR(scales, "scales");
  REQUIRE_PTR(out, "out");
  REQUIRE_ALIGN(blocks, 16, "blocks");
  REQUIRE_ALIGN(out, 16, "out");
  return launched(moe4::launch_decode_mxfp4(blocks, scales, R, K, out, (hipStream_t)stream),
                  "moe4_decode_mxfp4");
}

int moe4_compress_absmax(const float* absmax, int64_t n, const float* book, uint8_t* code,
                         float* absmax2, float* offset, void* ws, size_t ws_bytes,
                         void* stream) {
  if (n < 0) return fail(MOE4_ESHAPE, "n = %lld is negative", (long long)n);
  if (n == 0) return ok();
  REQUIRE_PTR(absmax, "absmax");
  REQUIRE_PTR(book, "book");
  REQUIRE_PTR(code, "code");
  REQUIRE_PTR(absmax2, "absmax2");
  REQUIRE_PTR(offset, "offset");
  REQUIRE_ALIGN(absmax, 4, "absmax");
  REQUIRE_ALIGN(book, 4, "book");
  REQUIRE_ALIGN(code, 4, "code");
  REQUIRE_ALIGN(absmax2, 4, "absmax2");
  REQUIRE_ALIGN(offset, 4, "offset");
  if (ws == nullptr || ws_bytes < (size_t)MOE4_DQ_WS_BYTES)
    return fail(MOE4_EWORKSPACE, "moe4_compress_absmax: workspace of %zu bytes given, %d needed",
                ws ? ws_bytes : (size_t)0, (int)MOE4_DQ_WS_BYTES);
  if (!aligned(ws, 8)) return fail(MOE4_EALIGN, "moe4_compress_absmax: ws is not 8-byte aligned");
  return launched(moe4::launch_dq_compress(absmax, n, book, code, absmax2, offset, ws,
                                           (hipStream_t)stream),
                  "moe4_compress_absmax");
}

int moe4_expand_absmax(const uint8_t* code, const float* absmax2, const float* offset,
                       const float* book, int64_t n, float* out, void* stream) {
  if (n < 0) return fail(MOE4_ESHAPE, "n = %lld is negative", (long long)n);
  if (n == 0) return ok();
  REQUIRE_PTR(code, "code");
  REQUIRE_PTR(absmax2, "absmax2");
  REQUIRE_PTR(offset, "offset");
  REQUIRE_PTR(book, "book");
  REQUIRE_PTR(out, "out");
  REQUIRE_ALIGN(absmax2, 4, "absmax2");
  REQUIRE_ALIGN(offset, 4, "offset");
  REQUIRE_ALIGN(book, 4, "book");
  REQUIRE_ALIGN(out, 4, "out");
  return launched(moe4::launch_dq_expand(code, absmax2, offset, book, n, out,
                                         (hipStream_t)stream),
                  "moe4_expand_absmax");
}

int moe4_convert_mxfp4_nf4(const uint8_t* blocks, const uint8_t* scales, int64_t R, int64_t K,
                           uint8_t* packed, float* absmax, void* stream) {
  if (R < 0 || K < 0 || K % 64)
    return fail(MOE4_ESHAPE, "R = %lld, K = %lld: need R >= 0 and K a non-negative multiple of 64",
                (long long)R, (long long)K);
  if (R == 0 || K == 0) return ok();
  REQUIRE_PTR(blocks, "blocks");
  REQUIRE_PTR(scales, "scales");
  REQUIRE_PTR(packed, "packed");
  REQUIRE_PTR(absmax, "absmax");
  REQUIRE_ALIGN(blocks, 16, "blocks");
  REQUIRE_ALIGN(packed, 16, "packed");
  REQUIRE_ALIGN(absmax, 4, "absmax");
  return launched(
      moe4::launch_convert_mxfp4_nf4(blocks, scales, R, K, packed, absmax, (hipStream_t)stream),
      "moe4_convert_mxfp4_nf4");
}

int moe4_route(const float* logits, int32_t T, int32_t E, int32_t k, int32_t renormalize,
               int32_t* topk_idx, float* topk_w, void* stream) {
  if (E < 1 || E > 1024) return fail(MOE4_ESHAPE, "E = %d outside [1, 1024]", E);
  if (k < 1 || k > E) return fail(MOE4_ESHAPE, "k = %d outside [1, E = %d]", k, E);
  if (T < 0 || (int64_t)T * k >= ((int64_t)1 << 31))
    return fail(MOE4_ESHAPE, "T = %d: need T >= 0 and T*k < 2^31", T);
  if (T == 0) return ok();
  REQUIRE_PTR(logits, "logits");
  REQUIRE_PTR(topk_idx, "topk_idx");
  REQUIRE_PTR(topk_w, "topk_w");
  REQUIRE_ALIGN(logits, 4, "logits");
  REQUIRE_ALIGN(topk_idx, 4, "topk_idx");
  REQUIRE_ALIGN(topk_w, 4, "topk_w");
  return launched(moe4::launch_route(logits, T, E, k, renormalize != 0, topk_idx, topk_w,
                                     (hipStream_t)stream),
                  "moe4_route");
}

int moe4_router_logits(const uint16_t* x, const uint16_t* wr, const float* bias, int32_t T,
                       int32_t H, int32_t E, float* logits, void* stream) {
  if (E < 1 || E > 1024) return fail(MOE4_ESHAPE, "E = %d outside [1, 1024]", E);
  if (H <= 0 || H % 8 || H >= (1 << 25))
    return fail(MOE4_ESHAPE, "H = %d must be a positive multiple of 8 below 2^25", H);
  if (T < 0) return fail(MOE4_ESHAPE, "T = %d is negative", T);
  if (T == 0) return ok();
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(wr, "wr");
  REQUIRE_PTR(logits, "logits");
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(wr, 16, "wr");
  REQUIRE_ALIGN(bias, 4, "bias");
  REQUIRE_ALIGN(logits, 4, "logits");
  return launched(moe4::launch_router_logits(x, wr, bias, T, H, E, logits, (hipStream_t)stream),
                  "moe4_router_logits");
}

int moe4_route_backward(const int32_t* topk_idx, const float* topk_w, const float* logits,
                        int32_t renormalize, const uint16_t* dout, const float* y_perm,
                        const int32_t* row_of_slot, int32_t T, int32_t k, int32_t E, int32_t H,
                        float* dw, float* dlogits, void* stream) {
  if (E < 1 || E > 1024) return fail(MOE4_ESHAPE, "E = %d outside [1, 1024]", E);
  if (k < 1 || k > E) return fail(MOE4_ESHAPE, "k = %d outside [1, E = %d]", k, E);
  if (T < 0 || (int64_t)T * k >= ((int64_t)1 << 31))
    return fail(MOE4_ESHAPE, "T = %d: need T >= 0 and T*k < 2^31", T);
  if (H <= 0 || H % 8) return fail(MOE4_ESHAPE, "H = %d must be a positive multiple of 8", H);
  if (!renormalize && T > 0) REQUIRE_PTR(logits, "logits (needed without renormalisation)");
  if (T == 0) return ok();
  REQUIRE_PTR(topk_idx, "topk_idx");
  REQUIRE_PTR(topk_w, "topk_w");
  REQUIRE_PTR(dout, "dout");
  REQUIRE_PTR(y_perm, "y_perm");
  REQUIRE_PTR(row_of_slot, "row_of_slot");
  REQUIRE_PTR(dw, "dw");
  REQUIRE_PTR(dlogits, "dlogits");
  REQUIRE_ALIGN(dout, 16, "dout");
  REQUIRE_ALIGN(y_perm, 16, "y_perm");
  REQUIRE_ALIGN(topk_idx, 4, "topk_idx");
  REQUIRE_ALIGN(topk_w, 4, "topk_w");
  REQUIRE_ALIGN(logits, 4, "logits");
  REQUIRE_ALIGN(row_of_slot, 4, "row_of_slot");
  REQUIRE_ALIGN(dw, 4, "dw");
  REQUIRE_ALIGN(dlogits, 4, "dlogits");
  return launched(moe4::launch_route_backward(topk_idx, topk_w, logits, renormalize != 0, dout,
                                              y_perm, row_of_slot, T, k, E, H, dw, dlogits,
                                              (hipStream_t)stream),
                  "moe4_route_backward");
}

int moe4_permute(const int32_t* topk_idx, int32_t T, int32_t k, int32_t E, int32_t* offsets,
                 int32_t* slot_of_row, int32_t* row_of_slot, const uint16_t* x,
                 const float* row_scale, int32_t H, uint16_t* x_perm, void* ws, size_t ws_bytes,
                 void* stream) {
  if (E < 1 || E > 1024) return fail(MOE4_ESHAPE, "E = %d outside [1, 1024]", E);
  if (k < 1 || k > E) return fail(MOE4_ESHAPE, "k = %d outside [1, E = %d]", k, E);
  if (T < 0 || (int64_t)T * k >= ((int64_t)1 << 31))
    return fail(MOE4_ESHAPE, "T = %d: need T >= 0 and T*k < 2^31", T);
  REQUIRE_PTR(offsets, "offsets");
  if (T > 0) {
    REQUIRE_PTR(topk_idx, "topk_idx");
    REQUIRE_PTR(slot_of_row, "slot_of_row");
    REQUIRE_PTR(row_of_slot, "row_of_slot");
  }
  if (x != nullptr) {
    if (H <= 0 || H % 8) return fail(MOE4_ESHAPE, "H = %d must be a positive multiple of 8", H);
    if (T > 0) REQUIRE_PTR(x_perm, "x_perm");
    REQUIRE_ALIGN(x, 16, "x");
    REQUIRE_ALIGN(x_perm, 16, "x_perm");
  } else if (row_scale != nullptr) {
    return fail(MOE4_EINVAL, "row_scale given without x");
  }
  const size_t need = moe4::permute_ws_bytes(T, k, E);
  int rc = check_ws(ws, ws_bytes, need, "moe4_permute");
  if (rc) return rc;
  if (T == 0) {
    // every expert is empty: offsets = 0 (a fill kernel, so the call can be
    // captured into a HIP graph)
    return launched(moe4::launch_zero_i32(offsets, E + 1, (hipStream_t)stream), "moe4_permute");
  }
  return launched(moe4::launch_permute(topk_idx, T, k, E, offsets, slot_of_row, row_of_slot, x,
                                       row_scale, H, x_perm, ws, (hipStream_t)stream),
                  "moe4_permute");
}

int moe4_gather_rows(const uint16_t* x, int32_t T, int32_t k, int32_t H,
                     const int32_t* slot_of_row, const float* row_scale, uint16_t* x_perm,
                     void* stream) {
  if (k < 1 || k > 1024) return fail(MOE4_ESHAPE, "k = %d outside [1, 1024]", k);
  if (T < 0 || (int64_t)T * k >= ((int64_t)1 << 31))
    return fail(MOE4_ESHAPE, "T = %d: need T >= 0 and T*k < 2^31", T);
  if (H <= 0 || H % 8) return fail(MOE4_ESHAPE, "H = %d must be a positive multiple of 8", H);
  if (T > 0) {
    REQUIRE_PTR(x, "x");
    REQUIRE_PTR(slot_of_row, "slot_of_row");
    REQUIRE_PTR(x_perm, "x_perm");
  }
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(x_perm, 16, "x_perm");
  REQUIRE_ALIGN(row_scale, 4, "row_scale");
  return launched(moe4::launch_gather(x, T, k, H, slot_of_row, row_scale, x_perm,
                                      (hipStream_t)stream),
                  "moe4_gather_rows");
}

int moe4_route_permute(const float* logits, int32_t T, int32_t E, int32_t k,
                       int32_t renormalize, int32_t* topk_idx, float* topk_w, int32_t* offsets,
                       int32_t* slot_of_row, int32_t* row_of_slot, const uint16_t* x, int32_t H,
                       uint16_t* x_perm, void* ws, size_t ws_bytes, void* stream) {
  if (E < 1 || E > 1024) return fail(MOE4_ESHAPE, "E = %d outside [1, 1024]", E);
  if (k < 1 || k > E) return fail(MOE4_ESHAPE, "k = %d outside [1, E = %d]", k, E);
  if (T < 0 || (int64_t)T * k >= ((int64_t)1 << 31))
    return fail(MOE4_ESHAPE, "T = %d: need T >= 0 and T*k < 2^31", T);
  REQUIRE_PTR(offsets, "offsets");
  if (T > 0) {
    REQUIRE_PTR(logits, "logits");
    REQUIRE_PTR(topk_idx, "topk_idx");
    REQUIRE_PTR(topk_w, "topk_w");
    REQUIRE_PTR(slot_of_row, "slot_of_row");
    REQUIRE_PTR(row_of_slot, "row_of_slot");
    REQUIRE_ALIGN(logits, 4, "logits");
    REQUIRE_ALIGN(topk_idx, 4, "topk_idx");
    REQUIRE_ALIGN(topk_w, 4, "topk_w");
  }
  if (x != nullptr) {
    if (H <= 0 || H % 8) return fail(MOE4_ESHAPE, "H = %d must be a positive multiple of 8", H);
    if (T > 0) REQUIRE_PTR(x_perm, "x_perm");
    REQUIRE_ALIGN(x, 16, "x");
    REQUIRE_ALIGN(x_perm, 16, "x_perm");
  }
  const size_t need = moe4::permute_ws_bytes(T, k, E);
  int rc = check_ws(ws, ws_bytes, need, "moe4_route_permute");
  if (rc) return rc;
  if (T == 0)
    return launched(moe4::launch_zero_i32(offsets, E + 1, (hipStream_t)stream),
                    "moe4_route_permute");
  return launched(moe4::launch_route_permute(logits, T, E, k, renormalize != 0, topk_idx, topk_w,
                                             offsets, slot_of_row, row_of_slot, x, H, x_perm, ws,
                                             (hipStream_t)stream),
                  "moe4_route_permute");
}

}  // extern "C"

namespace {

// Argument checks of the expert forward (both entry points).
int check_forward(const moe4_experts* ex, const uint16_t* x_perm, const int32_t* offsets,
                  int32_t rows, float* y_perm, float* save_gu, float* save_xa) {
  int rc = check_experts(ex);
  if (rc) return rc;
  if (rows < 0) return fail(MOE4_ESHAPE, "rows = %d is negative", rows);
  if (save_xa && !ex->lora_A) return fail(MOE4_EINVAL, "save_xa given without LoRA adapters");
  if (ex->H % 8) return fail(MOE4_ESHAPE, "H = %d must be a multiple of 8", ex->H);
  REQUIRE_PTR(offsets, "offsets");
  if (rows > 0) {
    REQUIRE_PTR(x_perm, "x_perm");
    REQUIRE_PTR(y_perm, "y_perm");
  }
  REQUIRE_ALIGN(x_perm, 16, "x_perm");
  REQUIRE_ALIGN(y_perm, 16, "y_perm");
  REQUIRE_ALIGN(save_gu, 4, "save_gu");
  REQUIRE_ALIGN(save_xa, 4, "save_xa");
  return MOE4_OK;
}

}  // namespace

extern "C" {

int moe4_expert_forward_noalloc(const moe4_experts* ex, const uint16_t* x_perm,
                                const int32_t* offsets, int32_t rows, float* y_perm,
                                float* save_gu, float* save_xa, void* stream) {
  g_variant = 0;
  int rc = check_forward(ex, x_perm, offsets, rows, y_perm, save_gu, save_xa);
  if (rc) return rc;
  const size_t need = moe4::forward_ws_bytes(*ex, rows);
  if (need > kNoAllocScratchBytes)
    return fail(MOE4_EWORKSPACE,
                "moe4_expert_forward_noalloc: this call needs %zu bytes of scratch, beyond the "
                "%zu the library holds per device (moe4_expert_forward takes a workspace)",
                need, kNoAllocScratchBytes);
  void* ws = nullptr;
  rc = scratch_of_current_device(stream, &ws);
  if (rc) return rc;
  int variant = 0;
  hipError_t e = moe4::launch_expert_forward(*ex, x_perm, offsets, rows, y_perm, save_gu,
                                             save_xa, ws, &variant, moe4::LaunchEvents{g_events},
                                             (hipStream_t)stream);
  rc = launched(e, "moe4_expert_forward_noalloc");
  if (rc == MOE4_OK) g_variant = variant;
  return rc;
}

int moe4_expert_forward(const moe4_experts* ex, const uint16_t* x_perm, const int32_t* offsets,
                        int32_t rows, float* y_perm, float* save_gu, float* save_xa,
                        void* ws, size_t ws_bytes, void* stream) {
  g_variant = 0;
  int rc = check_forward(ex, x_perm, offsets, rows, y_perm, save_gu, save_xa);
  if (rc) return rc;
  rc = check_ws(ws, ws_bytes, moe4::forward_ws_bytes(*ex, rows), "moe4_expert_forward");
  if (rc) return rc;
  int variant = 0;
  hipError_t e = moe4::launch_expert_forward(*ex, x_perm, offsets, rows, y_perm, save_gu,
                                             save_xa, ws, &variant, moe4::LaunchEvents{g_events},
                                             (hipStream_t)stream);
  rc = launched(e, "moe4_expert_forward");
  if (rc == MOE4_OK) g_variant = variant;
  return rc;
}

int moe4_expert_forward_gather(const moe4_experts* ex, const uint16_t* x, int32_t T, int32_t k,
                               const int32_t* slot_of_row, const int32_t* offsets, int32_t rows,
                               float* y_perm, float* save_gu, void* ws, size_t ws_bytes,
                               void* stream) {
  g_variant = 0;
  int rc = check_experts(ex);
  if (rc) return rc;
  if (ex->lora_A)
    return fail(MOE4_EUNSUPPORTED,
                "moe4_expert_forward_gather: the adapter path takes x_perm (moe4_expert_forward)");
  if (k < 1) return fail(MOE4_ESHAPE, "k = %d must be >= 1", k);
  if (T < 0 || (int64_t)T * k >= ((int64_t)1 << 31))
    return fail(MOE4_ESHAPE, "T = %d: need T >= 0 and T*k < 2^31", T);
  if (rows != T * k) return fail(MOE4_ESHAPE, "rows = %d must be T*k = %d", rows, T * k);
  if (ex->H % 8) return fail(MOE4_ESHAPE, "H = %d must be a multiple of 8", ex->H);
  if ((int64_t)T * ex->H * 2 >= ((int64_t)1 << 29))
    return fail(MOE4_ESHAPE, "x of T = %d rows of H = %d exceeds 2^29 bytes (gathered rows are "
                "addressed with 32-bit offsets); use moe4_permute + moe4_expert_forward", T, ex->H);
  REQUIRE_PTR(offsets, "offsets");
  if (rows > 0) {
    REQUIRE_PTR(x, "x");
    REQUIRE_PTR(slot_of_row, "slot_of_row");
    REQUIRE_PTR(y_perm, "y_perm");
  }
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(y_perm, 16, "y_perm");
  REQUIRE_ALIGN(save_gu, 4, "save_gu");
  rc = check_ws(ws, ws_bytes, moe4::forward_ws_bytes(*ex, rows), "moe4_expert_forward_gather");
  if (rc) return rc;
  int variant = 0;
  const moe4::GatherRows ga{x, slot_of_row, k, T};
  hipError_t e = moe4::launch_expert_forward(*ex, nullptr, offsets, rows, y_perm, save_gu,
                                             nullptr, ws, &variant, moe4::LaunchEvents{g_events},
                                             (hipStream_t)stream, &ga);
  rc = launched(e, "moe4_expert_forward_gather");
  if (rc == MOE4_OK) g_variant = variant;
  return rc;
}

int moe4_combine(const float* y_perm, const int32_t* row_of_slot, const float* topk_w,
                 int32_t T, int32_t k, int32_t H, void* out, int32_t out_dtype, void* stream) {
  if (out_dtype != MOE4_DTYPE_BF16 && out_dtype != MOE4_DTYPE_F32)
    return fail(MOE4_EINVAL, "out_dtype %s (%d)", out_dtype ? "unknown" : "unset", out_dtype);
  if (k < 1) return fail(MOE4_ESHAPE, "k = %d must be >= 1", k);
  if (T < 0 || (int64_t)T * k >= ((int64_t)1 << 31))
    return fail(MOE4_ESHAPE, "T = %d: need T >= 0 and T*k < 2^31", T);
  if (H <= 0 || H % 8) return fail(MOE4_ESHAPE, "H = %d must be a positive multiple of 8", H);
  if (T == 0) return ok();
  REQUIRE_PTR(y_perm, "y_perm");
  REQUIRE_PTR(row_of_slot, "row_of_slot");
  REQUIRE_PTR(out, "out");
  REQUIRE_ALIGN(y_perm, 16, "y_perm");
  REQUIRE_ALIGN(out, 16, "out");
  REQUIRE_ALIGN(topk_w, 4, "topk_w");
  return launched(moe4::launch_combine(y_perm, row_of_slot, topk_w, T, k, H, out,
                                       out_dtype == MOE4_DTYPE_F32, (hipStream_t)stream),
                  "moe4_combine");
}

int moe4_expert_backward(const moe4_experts* ex, const uint16_t* x_perm, const int32_t* offsets,
                         int32_t rows, const float* save_gu, const float* save_xa,
                         const uint16_t* dy_perm, float* dx_perm, float* dA, float* dB,
                         void* ws, size_t ws_bytes, void* stream) {
  g_variant = 0;
  int rc = check_experts(ex);
  if (rc) return rc;
  if (rows < 0) return fail(MOE4_ESHAPE, "rows = %d is negative", rows);
  REQUIRE_PTR(offsets, "offsets");
  if (rows > 0) {
    REQUIRE_PTR(save_gu, "save_gu");
    REQUIRE_PTR(dy_perm, "dy_perm");
    REQUIRE_PTR(dx_perm, "dx_perm");
  }
  if (ex->lora_A) {
    REQUIRE_PTR(dA, "dA");
    REQUIRE_PTR(dB, "dB");
    if (rows > 0) {
      REQUIRE_PTR(x_perm, "x_perm");
      REQUIRE_PTR(save_xa, "save_xa");
    }
  } else if (dA || dB) {
    return fail(MOE4_EINVAL, "dA/dB given without LoRA adapters");
  }
  REQUIRE_ALIGN(x_perm, 16, "x_perm");
  REQUIRE_ALIGN(dy_perm, 16, "dy_perm");
  REQUIRE_ALIGN(dx_perm, 16, "dx_perm");
  REQUIRE_ALIGN(save_gu, 4, "save_gu");
  REQUIRE_ALIGN(save_xa, 4, "save_xa");
  REQUIRE_ALIGN(dA, 4, "dA");
  REQUIRE_ALIGN(dB, 4, "dB");
  rc = check_ws(ws, ws_bytes, moe4::backward_ws_bytes(*ex, rows), "moe4_expert_backward");
  if (rc) return rc;
  int variant = 0;
  hipError_t e = moe4::launch_expert_backward(*ex, x_perm, offsets, rows, save_gu, save_xa,
                                              dy_perm, dx_perm, dA, dB, ws, &variant,
                                              moe4::LaunchEvents{g_events}, (hipStream_t)stream);
  rc = launched(e, "moe4_expert_backward");
  if (rc == MOE4_OK) g_variant = variant;
  return rc;
}

}  // extern "C"

namespace {

constexpr int64_t kByteSpan = ((int64_t)1 << 31) - ((int64_t)1 << 24);   // 32-bit byte offsets

#define REQUIRE_DTYPE(d, name)                                                          \
  do {                                                                                  \
    if ((d) != MOE4_DTYPE_BF16 && (d) != MOE4_DTYPE_F32)                                \
      return fail(MOE4_EINVAL, "%s %s (%d)", name, (d) ? "unknown" : "unset", (int)(d)); \
  } while (0)

int check_norm_shape(int32_t T, int32_t H) {
  if (T < 0) return fail(MOE4_ESHAPE, "T = %d is negative", T);
  if (H < 8 || H > 16384 || H % 8)
    return fail(MOE4_ESHAPE, "H = %d must be a multiple of 8 in [8, 16384]", H);
  return MOE4_OK;
}

int check_ffn(const moe4_ffn* f) {
  if (f == nullptr) return fail(MOE4_EINVAL, "moe4_ffn is NULL");
  if (f->format != MOE4_FFN_BF16 && f->format != MOE4_FFN_MXFP8)
    return fail(MOE4_EINVAL, "moe4_ffn.format %s (%d)", f->format ? "unknown" : "unset", f->format);
  if (f->gu_layout != MOE4_GU_HALVES && f->gu_layout != MOE4_GU_INTERLEAVED)
    return fail(MOE4_EINVAL, "moe4_ffn.gu_layout %s (%d)", f->gu_layout ? "unknown" : "unset",
                f->gu_layout);
  if (f->act != MOE4_ACT_SWIGLU && f->act != MOE4_ACT_SWIGLU_CLAMPED)
    return fail(MOE4_EINVAL, "moe4_ffn.act %s (%d)", f->act ? "unknown" : "unset", f->act);
  if (f->variant != MOE4_VARIANT_AUTO && f->variant != MOE4_VARIANT_SKINNY &&
      f->variant != MOE4_VARIANT_TILED)
    return fail(MOE4_EINVAL, "moe4_ffn.variant unknown (%d)", f->variant);
  const int mx = f->format == MOE4_FFN_MXFP8, blk = mx ? 32 : 8;
  if (f->H <= 0 || f->H % blk)
    return fail(MOE4_ESHAPE, "moe4_ffn.H = %d is not a positive multiple of %d", f->H, blk);
  if (f->I <= 0 || f->I % blk)
    return fail(MOE4_ESHAPE, "moe4_ffn.I = %d is not a positive multiple of %d", f->I, blk);
  const int64_t wide = f->H > 2 * (int64_t)f->I ? f->H : 2 * (int64_t)f->I;
  if (2 * (int64_t)f->I * f->H * (mx ? 1 : 2) >= kByteSpan)
    return fail(MOE4_ESHAPE, "moe4_ffn: 2*I*H = %lld; a weight must stay under 2 GiB",
                (long long)(2 * (int64_t)f->I * f->H));
  if (256 * 2 * wide >= kByteSpan)
    return fail(MOE4_ESHAPE, "moe4_ffn: max(H, 2I) = %lld; 256 rows must stay under 2 GiB",
                (long long)wide);
  REQUIRE_PTR(f->w_gu, "moe4_ffn.w_gu");
  REQUIRE_PTR(f->w_dn, "moe4_ffn.w_dn");
  REQUIRE_ALIGN(f->w_gu, 16, "moe4_ffn.w_gu");
  REQUIRE_ALIGN(f->w_dn, 16, "moe4_ffn.w_dn");
  if (mx) {
    REQUIRE_PTR(f->gu_s, "moe4_ffn.gu_s");
    REQUIRE_PTR(f->dn_s, "moe4_ffn.dn_s");
    REQUIRE_ALIGN(f->gu_s, 4, "moe4_ffn.gu_s");
    REQUIRE_ALIGN(f->dn_s, 4, "moe4_ffn.dn_s");
  } else if (f->gu_s || f->dn_s) {
    return fail(MOE4_EINVAL, "moe4_ffn: scales given for bf16 weights");
  }
  REQUIRE_ALIGN(f->gu_bias, 16, "moe4_ffn.gu_bias");
  REQUIRE_ALIGN(f->dn_bias, 16, "moe4_ffn.dn_bias");
  if (f->act == MOE4_ACT_SWIGLU_CLAMPED && (!(f->act_limit > 0.0f) || !(f->act_alpha > 0.0f)))
    return fail(MOE4_EINVAL,
                "moe4_ffn.act_alpha/act_limit must be positive for the clamped GLU (got %g, %g)",
                (double)f->act_alpha, (double)f->act_limit);
  return MOE4_OK;
}

int check_ffn_tokens(const moe4_ffn* f, int32_t T) {
  if (T < 0) return fail(MOE4_ESHAPE, "T = %d is negative", T);
  if (f->variant == MOE4_VARIANT_SKINNY && T > 1 << 20)
    return fail(MOE4_ESHAPE, "T = %d: the skinny variant takes at most 2^20 tokens", T);
  const int64_t wide = f->H > f->I ? f->H : f->I;
  if (f->format == MOE4_FFN_MXFP8 && T * (wide / 32) >= kByteSpan)
    return fail(MOE4_ESHAPE, "T = %d: the activations' scales must stay under 2 GiB", T);
  // workgroups of the smallest tiles, 256 threads each, in one 32-bit launch
  if (((int64_t)T + 127) / 128 * ((2 * wide + 127) / 128) >= (int64_t)1 << 23)
    return fail(MOE4_ESHAPE, "T = %d with max(H, I) = %lld is beyond one launch", T,
                (long long)wide);
  return MOE4_OK;
}

int check_grads(const void* const* grads, void* const* outs, const int64_t* numel,
                const int32_t* dtype, int32_t n) {
  if (n < 0 || n > 1 << 20) return fail(MOE4_ESHAPE, "n = %d outside [0, 2^20]", n);
  if (n == 0) return MOE4_OK;
  REQUIRE_PTR(grads, "grads");
  REQUIRE_PTR(numel, "numel");
  REQUIRE_PTR(dtype, "dtype");
  for (int i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] > moe4::grad_most_numel())
      return fail(MOE4_ESHAPE, "numel[%d] = %lld outside [0, 2^36]", i, (long long)numel[i]);
    if (dtype[i] != MOE4_DTYPE_BF16 && dtype[i] != MOE4_DTYPE_F32)
      return fail(MOE4_EINVAL, "dtype[%d] %s (%d)", i, dtype[i] ? "unknown" : "unset", dtype[i]);
    if (numel[i] == 0) continue;
    if (grads[i] == nullptr || (outs && outs[i] == nullptr))
      return fail(MOE4_EINVAL, "%s[%d] is NULL", grads[i] ? "outs" : "grads", i);
    if (!aligned(grads[i], 16) || (outs && !aligned(outs[i], 16)))
      return fail(MOE4_EALIGN, "%s[%d] is not 16-byte aligned",
                  aligned(grads[i], 16) ? "outs" : "grads", i);
  }
  return MOE4_OK;
}

}  // namespace

extern "C" {

int moe4_add_rmsnorm(const void* x, int32_t x_dtype, const void* residual, int32_t res_dtype,
                     void* sum_out, const void* weight, int32_t w_dtype, int32_t T, int32_t H,
                     float eps, uint16_t* out, uint8_t* out_q, uint8_t* out_s, float* rstd,
                     void* stream) {
  int rc = check_norm_shape(T, H);
  if (rc) return rc;
  REQUIRE_DTYPE(x_dtype, "x_dtype");
  REQUIRE_DTYPE(w_dtype, "w_dtype");
  if (residual) REQUIRE_DTYPE(res_dtype, "res_dtype");
  if (!(eps >= 0.0f)) return fail(MOE4_EINVAL, "eps = %g must not be negative", (double)eps);
  if (sum_out && !residual && T > 0)
    return fail(MOE4_EINVAL, "sum_out given without a residual");
  if ((out_q == nullptr) != (out_s == nullptr))
    return fail(MOE4_EINVAL, "out_q and out_s must be given together");
  if (out_q && H % 32)
    return fail(MOE4_ESHAPE, "H = %d must be a multiple of 32 for an MXFP8 output", H);
  if (T == 0) return ok();
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(weight, "weight");
  if (!out && !out_q) return fail(MOE4_EINVAL, "out and out_q are both NULL");
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(residual, 16, "residual");
  REQUIRE_ALIGN(sum_out, 16, "sum_out");
  REQUIRE_ALIGN(weight, 16, "weight");
  REQUIRE_ALIGN(out, 16, "out");
  REQUIRE_ALIGN(out_q, 16, "out_q");
  REQUIRE_ALIGN(rstd, 4, "rstd");
  return launched(moe4::launch_add_rmsnorm(x, x_dtype, residual, res_dtype, sum_out, weight,
                                           w_dtype, T, H, eps, out, out_q, out_s, rstd,
                                           (hipStream_t)stream),
                  "moe4_add_rmsnorm");
}

size_t moe4_add_rmsnorm_workspace_size(int32_t T, int32_t H) {
  if (check_norm_shape(T, H) != MOE4_OK) return 0;
  ok();
  const size_t need = moe4::add_rmsnorm_ws_bytes(T, H);
  return need < 256 ? 256 : need;
}

int moe4_add_rmsnorm_backward(const void* dy, int32_t dy_dtype, const void* s, int32_t s_dtype,
                              const void* weight, int32_t w_dtype, const float* rstd,
                              const void* dres, int32_t T, int32_t H, void* dx, int32_t dx_dtype,
                              float* dweight, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_norm_shape(T, H);
  if (rc) return rc;
  REQUIRE_DTYPE(dy_dtype, "dy_dtype");
  REQUIRE_DTYPE(s_dtype, "s_dtype");
  REQUIRE_DTYPE(w_dtype, "w_dtype");
  REQUIRE_DTYPE(dx_dtype, "dx_dtype");
  if (T > 0) {
    REQUIRE_PTR(dy, "dy");
    REQUIRE_PTR(s, "s");
    REQUIRE_PTR(weight, "weight");
    REQUIRE_PTR(rstd, "rstd");
    REQUIRE_PTR(dx, "dx");
  }
  REQUIRE_ALIGN(dy, 16, "dy");
  REQUIRE_ALIGN(s, 16, "s");
  REQUIRE_ALIGN(weight, 16, "weight");
  REQUIRE_ALIGN(rstd, 4, "rstd");
  REQUIRE_ALIGN(dres, 16, "dres");
  REQUIRE_ALIGN(dx, 16, "dx");
  REQUIRE_ALIGN(dweight, 16, "dweight");
  if (dweight && T > 0) {
    rc = check_ws(ws, ws_bytes, moe4::add_rmsnorm_ws_bytes(T, H), "moe4_add_rmsnorm_backward");
    if (rc) return rc;
  }
  if (T == 0 && !dweight) return ok();
  return launched(moe4::launch_add_rmsnorm_backward(dy, dy_dtype, s, s_dtype, weight, w_dtype,
                                                    rstd, dres, T, H, dx, dx_dtype, dweight, ws,
                                                    (hipStream_t)stream),
                  "moe4_add_rmsnorm_backward");
}

int moe4_quantize_mxfp8(const void* x, int32_t x_dtype, int64_t R, int64_t K, uint8_t* q,
                        uint8_t* s, void* stream) {
  REQUIRE_DTYPE(x_dtype, "x_dtype");
  if (R < 0) return fail(MOE4_ESHAPE, "R = %lld is negative", (long long)R);
  if (K < 0 || K % 32)
    return fail(MOE4_ESHAPE, "K = %lld is not a non-negative multiple of 32", (long long)K);
  if (K && R > ((int64_t)1 << 40) / K)
    return fail(MOE4_ESHAPE, "R * K is beyond the supported 2^40");
  if (R == 0 || K == 0) return ok();
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(q, "q");
  REQUIRE_PTR(s, "s");
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(q, 16, "q");
  return launched(moe4::launch_quantize_mxfp8(x, x_dtype, R * K, q, s, (hipStream_t)stream),
                  "moe4_quantize_mxfp8");
}

size_t moe4_ffn_workspace_size(const moe4_ffn* f, int32_t T, int32_t backward) {
  if (check_ffn(f) != MOE4_OK || check_ffn_tokens(f, T) != MOE4_OK) return 0;
  ok();
  const size_t need = backward ? moe4::ffn_backward_ws_bytes(*f, T) : moe4::ffn_forward_ws_bytes(*f, T);
  return need < 256 ? 256 : need;
}

int moe4_ffn_forward(const moe4_ffn* f, const void* x, const uint8_t* x_s, int32_t T,
                     const void* residual, int32_t res_dtype, void* out, int32_t out_dtype,
                     float* save_gu, void* ws, size_t ws_bytes, void* stream) {
  g_variant = 0;
  int rc = check_ffn(f);
  if (rc) return rc;
  rc = check_ffn_tokens(f, T);
  if (rc) return rc;
  REQUIRE_DTYPE(out_dtype, "out_dtype");
  if (residual) REQUIRE_DTYPE(res_dtype, "res_dtype");
  if (x_s && f->format == MOE4_FFN_BF16)
    return fail(MOE4_EINVAL, "x_s given for a bf16 block");
  if (T == 0) return ok();
  REQUIRE_PTR(x, "x");
  if (f->format == MOE4_FFN_MXFP8) REQUIRE_PTR(x_s, "x_s");
  REQUIRE_PTR(out, "out");
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(x_s, 4, "x_s");
  REQUIRE_ALIGN(residual, 16, "residual");
  REQUIRE_ALIGN(out, 16, "out");
  REQUIRE_ALIGN(save_gu, 16, "save_gu");
  rc = check_ws(ws, ws_bytes, moe4::ffn_forward_ws_bytes(*f, T), "moe4_ffn_forward");
  if (rc) return rc;
  int variant = 0;
  hipError_t e = moe4::launch_ffn_forward(*f, x, x_s, T, residual, res_dtype, out, out_dtype,
                                          save_gu, ws, &variant, (hipStream_t)stream);
  rc = launched(e, "moe4_ffn_forward");
  if (rc == MOE4_OK) g_variant = variant;
  return rc;
}

int moe4_ffn_backward(const moe4_ffn* f, const uint16_t* x, int32_t T, const float* save_gu,
                      const uint16_t* dy, const void* dx_add, int32_t add_dtype, void* dx,
                      int32_t dx_dtype, void* dw_gu, void* dw_dn, void* db_gu, void* db_dn,
                      int32_t dw_dtype, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_ffn(f);
  if (rc) return rc;
  if (f->format != MOE4_FFN_BF16)
    return fail(MOE4_EUNSUPPORTED, "moe4_ffn_backward: bf16 blocks only (format %d)", f->format);
  rc = check_ffn_tokens(f, T);
  if (rc) return rc;
  if (dx) REQUIRE_DTYPE(dx_dtype, "dx_dtype");
  if (dx_add) {
    if (!dx && T > 0) return fail(MOE4_EINVAL, "dx_add given without dx");
    REQUIRE_DTYPE(add_dtype, "add_dtype");
  }
  const bool params = dw_gu || dw_dn || db_gu || db_dn;
  if (params) REQUIRE_DTYPE(dw_dtype, "dw_dtype");
  if (T > 0 && (dx || params)) {
    REQUIRE_PTR(dy, "dy");
    REQUIRE_PTR(save_gu, "save_gu");
    if (dw_gu) REQUIRE_PTR(x, "x");
  }
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(save_gu, 16, "save_gu");
  REQUIRE_ALIGN(dy, 16, "dy");
  REQUIRE_ALIGN(dx_add, 16, "dx_add");
  REQUIRE_ALIGN(dx, 16, "dx");
  REQUIRE_ALIGN(dw_gu, 16, "dw_gu");
  REQUIRE_ALIGN(dw_dn, 16, "dw_dn");
  REQUIRE_ALIGN(db_gu, 16, "db_gu");
  REQUIRE_ALIGN(db_dn, 16, "db_dn");
  hipStream_t s = (hipStream_t)stream;
  if (T == 0) {
    // no token: zero gradients (by a fill kernel, so that the call can be captured)
    const int words = dw_dtype == MOE4_DTYPE_F32 ? 1 : 2;   // elements of a 4-byte word
    const struct { void* p; int n; } z[] = {{dw_gu, 2 * f->I * f->H}, {dw_dn, f->H * f->I},
                                            {db_gu, 2 * f->I}, {db_dn, f->H}};
    for (const auto& q : z) {
      if (!q.p) continue;
      rc = launched(moe4::launch_zero_i32(static_cast<int32_t*>(q.p), q.n / words, s),
                    "moe4_ffn_backward");
      if (rc) return rc;
    }
    return ok();
  }
  if (!dx && !params) return ok();
  rc = check_ws(ws, ws_bytes, moe4::ffn_backward_ws_bytes(*f, T), "moe4_ffn_backward");
  if (rc) return rc;
  return launched(moe4::launch_ffn_backward(*f, x, T, save_gu, dy, dx_add, add_dtype, dx, dx_dtype,
                                            dw_gu, dw_dn, db_gu, db_dn, dw_dtype, ws, s),
                  "moe4_ffn_backward");
}

size_t moe4_grad_workspace_size(int32_t n) {
  if (n < 0 || n > 1 << 20) {
    fail(MOE4_ESHAPE, "moe4_grad_workspace_size: n = %d outside [0, 2^20]", n);
    return 0;
  }
  ok();
  return moe4::grad_ws_bytes(n);
}

int moe4_grad_norm(const void* const* grads, const int64_t* numel, const int32_t* dtype,
                   int32_t n, float* norm, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_grads(grads, nullptr, numel, dtype, n);
  if (rc) return rc;
  REQUIRE_PTR(norm, "norm");
  REQUIRE_ALIGN(norm, 4, "norm");
  rc = check_ws(ws, ws_bytes, moe4::grad_ws_bytes(n), "moe4_grad_norm");
  if (rc) return rc;
  return launched(moe4::launch_grad_norm(grads, numel, dtype, n, norm, ws, (hipStream_t)stream),
                  "moe4_grad_norm");
}

int moe4_clip_grads(const void* const* grads, void* const* outs, const int64_t* numel,
                    const int32_t* dtype, int32_t n, float max_norm, const float* norm_in,
                    float* norm_out, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_grads(grads, outs, numel, dtype, n);
  if (rc) return rc;
  if (!(max_norm > 0.0f)) return fail(MOE4_EINVAL, "max_norm = %g must be positive", (double)max_norm);
  REQUIRE_ALIGN(norm_in, 4, "norm_in");
  REQUIRE_ALIGN(norm_out, 4, "norm_out");
  if (!norm_in) {
    rc = check_ws(ws, ws_bytes, moe4::grad_ws_bytes(n), "moe4_clip_grads");
    if (rc) return rc;
  }
  return launched(moe4::launch_clip_grads(grads, outs, numel, dtype, n, max_norm, norm_in, norm_out,
                                          ws, (hipStream_t)stream),
                  "moe4_clip_grads");
}

int moe4_quantize_mxfp4(const void* x, int32_t x_dtype, int64_t R, int64_t K, uint8_t* blocks,
                        uint8_t* scales, uint16_t* values, void* stream) {
  REQUIRE_DTYPE(x_dtype, "x_dtype");
  if (R < 0) return fail(MOE4_ESHAPE, "R = %lld is negative", (long long)R);
  if (K < 0 || K % 32)
    return fail(MOE4_ESHAPE, "K = %lld is not a non-negative multiple of 32", (long long)K);
  if (K && R > ((int64_t)1 << 40) / K)
    return fail(MOE4_ESHAPE, "R * K is beyond the supported 2^40");
  if (R == 0 || K == 0) return ok();
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(blocks, "blocks");
  REQUIRE_PTR(scales, "scales");
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(blocks, 16, "blocks");
  REQUIRE_ALIGN(values, 16, "values");
  return launched(moe4::launch_quantize_mxfp4(x, x_dtype, R * K, blocks, scales, values,
                                              (hipStream_t)stream),
                  "moe4_quantize_mxfp4");
}

int moe4_join_norm(const void* b, int32_t b_dtype, const void* residual, int32_t s_dtype,
                   float res_scale, float block_scale, const float* gate, const void* w_post,
                   int32_t post_dtype, const void* w_pre, int32_t pre_dtype, int32_t T,
                   int32_t H, float eps, void* sum_out, float* rstd_post, float* rstd_pre,
                   uint16_t* out, uint8_t* out_q, uint8_t* out_s, int32_t q_format,
                   void* stream) {
  int rc = check_norm_shape(T, H);
  if (rc) return rc;
  REQUIRE_DTYPE(b_dtype, "b_dtype");
  REQUIRE_DTYPE(s_dtype, "s_dtype");
  if (w_post) REQUIRE_DTYPE(post_dtype, "post_dtype");
  if (w_pre) REQUIRE_DTYPE(pre_dtype, "pre_dtype");
  if (!(eps >= 0.0f)) return fail(MOE4_EINVAL, "eps = %g must not be negative", (double)eps);
  if ((out_q == nullptr) != (out_s == nullptr))
    return fail(MOE4_EINVAL, "out_q and out_s must be given together");
  if (out_q && q_format != MOE4_X_MXFP8 && q_format != MOE4_X_MXFP4)
    return fail(MOE4_EINVAL, "q_format %s (%d)", q_format ? "is neither MXFP8 nor MXFP4" : "unset",
                q_format);
  if (out_q && H % 32)
    return fail(MOE4_ESHAPE, "H = %d must be a multiple of 32 for an 8- or 4-bit output", H);
  if (T == 0) return ok();
  REQUIRE_PTR(b, "b");
  if (!w_pre && (out || out_q || rstd_pre))
    return fail(MOE4_EINVAL, "%s given without w_pre", out ? "out" : out_q ? "out_q" : "rstd_pre");
  if (!w_post && rstd_post) return fail(MOE4_EINVAL, "rstd_post given without w_post");
  if (!out && !out_q && !sum_out)
    return fail(MOE4_EINVAL, "sum_out, out and out_q are all NULL");
  if (w_pre && !out && !out_q) return fail(MOE4_EINVAL, "w_pre given, out and out_q both NULL");
  REQUIRE_ALIGN(b, 16, "b");
  REQUIRE_ALIGN(residual, 16, "residual");
  REQUIRE_ALIGN(gate, 4, "gate");
  REQUIRE_ALIGN(w_post, 16, "w_post");
  REQUIRE_ALIGN(w_pre, 16, "w_pre");
  REQUIRE_ALIGN(sum_out, 16, "sum_out");
  REQUIRE_ALIGN(rstd_post, 4, "rstd_post");
  REQUIRE_ALIGN(rstd_pre, 4, "rstd_pre");
  REQUIRE_ALIGN(out, 16, "out");
  REQUIRE_ALIGN(out_q, 16, "out_q");
  return launched(moe4::launch_join_norm(b, b_dtype, residual, s_dtype, res_scale, block_scale,
                                         gate, w_post, post_dtype, w_pre, pre_dtype, T, H, eps,
                                         sum_out, rstd_post, rstd_pre, out, out_q, out_s,
                                         q_format == MOE4_X_MXFP4, (hipStream_t)stream),
                  "moe4_join_norm");
}

size_t moe4_join_norm_workspace_size(int32_t T, int32_t H) {
  if (check_norm_shape(T, H) != MOE4_OK) return 0;
  ok();
  const size_t need = moe4::join_norm_ws_bytes(T, H);
  return need < 256 ? 256 : need;
}

int moe4_join_norm_backward(const void* dy, int32_t dy_dtype, const void* s, int32_t s_dtype,
                            const void* b, int32_t b_dtype, const void* ds, float res_scale,
                            float block_scale, const float* gate, const void* w_post,
                            int32_t post_dtype, const void* w_pre, int32_t pre_dtype,
                            const float* rstd_post, const float* rstd_pre, int32_t T, int32_t H,
                            void* db, void* dres, float* dgate, float* dw_post, float* dw_pre,
                            void* ws, size_t ws_bytes, void* stream) {
  int rc = check_norm_shape(T, H);
  if (rc) return rc;
  REQUIRE_DTYPE(s_dtype, "s_dtype");
  REQUIRE_DTYPE(b_dtype, "b_dtype");
  if (w_post) REQUIRE_DTYPE(post_dtype, "post_dtype");
  if (w_pre) {
    REQUIRE_DTYPE(pre_dtype, "pre_dtype");
    REQUIRE_DTYPE(dy_dtype, "dy_dtype");
  } else if (dy || s || rstd_pre || dw_pre) {
    return fail(MOE4_EINVAL, "%s given without w_pre",
                dy ? "dy" : s ? "s" : rstd_pre ? "rstd_pre" : "dw_pre");
  }
  if (!w_post && (rstd_post || dw_post))
    return fail(MOE4_EINVAL, "%s given without w_post", rstd_post ? "rstd_post" : "dw_post");
  if (T > 0) {
    if (w_pre) {
      REQUIRE_PTR(dy, "dy");
      REQUIRE_PTR(s, "s");
      REQUIRE_PTR(rstd_pre, "rstd_pre");
    } else {
      REQUIRE_PTR(ds, "ds");
    }
    if (w_post) REQUIRE_PTR(rstd_post, "rstd_post");
    REQUIRE_PTR(b, "b");
    REQUIRE_PTR(db, "db");
    if (db == dres) return fail(MOE4_EINVAL, "db and dres are the same memory");
  }
  REQUIRE_ALIGN(dy, 16, "dy");
  REQUIRE_ALIGN(s, 16, "s");
  REQUIRE_ALIGN(b, 16, "b");
  REQUIRE_ALIGN(ds, 16, "ds");
  REQUIRE_ALIGN(gate, 4, "gate");
  REQUIRE_ALIGN(w_post, 16, "w_post");
  REQUIRE_ALIGN(w_pre, 16, "w_pre");
  REQUIRE_ALIGN(rstd_post, 4, "rstd_post");
  REQUIRE_ALIGN(rstd_pre, 4, "rstd_pre");
  REQUIRE_ALIGN(db, 16, "db");
  REQUIRE_ALIGN(dres, 16, "dres");
  REQUIRE_ALIGN(dgate, 4, "dgate");
  REQUIRE_ALIGN(dw_post, 16, "dw_post");
  REQUIRE_ALIGN(dw_pre, 16, "dw_pre");
  if ((dw_post || dw_pre) && T > 0) {
    rc = check_ws(ws, ws_bytes, moe4::join_norm_ws_bytes(T, H), "moe4_join_norm_backward");
    if (rc) return rc;
  }
  if (T == 0 && !dw_post && !dw_pre) return ok();
  return launched(
      moe4::launch_join_norm_backward(dy, dy_dtype, s, s_dtype, b, b_dtype, ds, res_scale,
                                      block_scale, gate, w_post, post_dtype, w_pre, pre_dtype,
                                      rstd_post, rstd_pre, T, H, db, dres, dgate, dw_post, dw_pre,
                                      ws, (hipStream_t)stream),
      "moe4_join_norm_backward");
}

static int check_linear(const moe4_linear* l, int32_t T) {
  if (l == nullptr) return fail(MOE4_EINVAL, "moe4_linear is NULL");
  if (l->variant != MOE4_VARIANT_AUTO && l->variant != MOE4_VARIANT_SKINNY &&
      l->variant != MOE4_VARIANT_TILED)
    return fail(MOE4_EINVAL, "moe4_linear.variant unknown (%d)", l->variant);
  if (l->N <= 0 || l->N % 8)
    return fail(MOE4_ESHAPE, "moe4_linear.N = %d is not a positive multiple of 8", l->N);
  if (l->K <= 0 || l->K % 32)
    return fail(MOE4_ESHAPE, "moe4_linear.K = %d is not a positive multiple of 32", l->K);
  if ((int64_t)l->N * l->K / 2 >= kByteSpan)
    return fail(MOE4_ESHAPE, "moe4_linear: N * K = %lld; the codes must stay under 2 GiB",
                (long long)l->N * l->K);
  const int64_t wide = l->N > l->K ? l->N : l->K;
  if (256 * 4 * wide >= kByteSpan)
    return fail(MOE4_ESHAPE, "moe4_linear: max(N, K) = %lld; 256 rows must stay under 2 GiB",
                (long long)wide);
  REQUIRE_PTR(l->w_q, "moe4_linear.w_q");
  REQUIRE_PTR(l->w_s, "moe4_linear.w_s");
  REQUIRE_ALIGN(l->w_q, 16, "moe4_linear.w_q");
  REQUIRE_ALIGN(l->w_s, 4, "moe4_linear.w_s");
  REQUIRE_ALIGN(l->bias, 16, "moe4_linear.bias");
  if (T < 0) return fail(MOE4_ESHAPE, "T = %d is negative", T);
  if (l->variant == MOE4_VARIANT_SKINNY && T > 1 << 20)
    return fail(MOE4_ESHAPE, "T = %d: the skinny variant takes at most 2^20 tokens", T);
  if (T * (wide / 32) >= kByteSpan)
    return fail(MOE4_ESHAPE, "T = %d: the activations' scales must stay under 2 GiB", T);
  // workgroups of the smallest tiles (128 x 64), 256 threads each, in one 32-bit launch
  if (((int64_t)T + 63) / 64 * ((wide + 127) / 128) >= (int64_t)1 << 23)
    return fail(MOE4_ESHAPE, "T = %d with max(N, K) = %lld is beyond one launch", T, (long long)wide);
  return MOE4_OK;
}

size_t moe4_linear_workspace_size(const moe4_linear* l, int32_t T, int32_t backward) {
  if (check_linear(l, T) != MOE4_OK) return 0;
  ok();
  const size_t need = moe4::linear_ws_bytes(*l, T, backward != 0);
  return need < 256 ? 256 : need;
}

int moe4_linear_forward(const moe4_linear* l, const void* x, int32_t x_format,
                        const uint8_t* x_s, int32_t T, const void* residual, int32_t res_dtype,
                        void* out, int32_t out_dtype, void* ws, size_t ws_bytes, void* stream) {
  g_variant = 0;
  int rc = check_linear(l, T);
  if (rc) return rc;
  if (x_format != MOE4_X_BF16 && x_format != MOE4_X_MXFP8 && x_format != MOE4_X_MXFP4)
    return fail(MOE4_EINVAL, "x_format %s (%d)", x_format ? "unknown" : "unset", x_format);
  REQUIRE_DTYPE(out_dtype, "out_dtype");
  if (residual) REQUIRE_DTYPE(res_dtype, "res_dtype");
  if (x_s && x_format == MOE4_X_BF16) return fail(MOE4_EINVAL, "x_s given for bf16 activations");
  if (T == 0) return ok();
  REQUIRE_PTR(x, "x");
  if (x_format != MOE4_X_BF16) REQUIRE_PTR(x_s, "x_s");
  REQUIRE_PTR(out, "out");
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(x_s, 4, "x_s");
  REQUIRE_ALIGN(residual, 16, "residual");
  REQUIRE_ALIGN(out, 16, "out");
  rc = check_ws(ws, ws_bytes, moe4::linear_ws_bytes(*l, T, false), "moe4_linear_forward");
  if (rc) return rc;
  int variant = 0;
  hipError_t e = moe4::launch_linear_forward(*l, x, x_format, x_s, T, residual, res_dtype, out,
                                             out_dtype, ws, &variant, (hipStream_t)stream);
  rc = launched(e, "moe4_linear_forward");
  if (rc == MOE4_OK) g_variant = variant;
  return rc;
}

int moe4_linear_backward(const moe4_linear* l, const uint16_t* dy, int32_t T, const void* dx_add,
                         int32_t add_dtype, void* dx, int32_t dx_dtype, void* db,
                         int32_t db_dtype, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_linear(l, T);
  if (rc) return rc;
  if (dx) REQUIRE_DTYPE(dx_dtype, "dx_dtype");
  if (dx_add) {
    if (!dx && T > 0) return fail(MOE4_EINVAL, "dx_add given without dx");
    REQUIRE_DTYPE(add_dtype, "add_dtype");
  }
  if (db) REQUIRE_DTYPE(db_dtype, "db_dtype");
  if (T > 0 && (dx || db)) REQUIRE_PTR(dy, "dy");
  REQUIRE_ALIGN(dy, 16, "dy");
  REQUIRE_ALIGN(dx_add, 16, "dx_add");
  REQUIRE_ALIGN(dx, 16, "dx");
  REQUIRE_ALIGN(db, 16, "db");
  hipStream_t s = (hipStream_t)stream;
  if (T == 0)   // no token: a zero gradient (by a fill kernel, so that the call can be captured)
    return db ? launched(moe4::launch_zero_i32(static_cast<int32_t*>(db),
                                               db_dtype == MOE4_DTYPE_F32 ? l->N : l->N / 2, s),
                         "moe4_linear_backward")
              : ok();
  if (!dx && !db) return ok();
  rc = check_ws(ws, ws_bytes, moe4::linear_ws_bytes(*l, T, true), "moe4_linear_backward");
  if (rc) return rc;
  return launched(moe4::launch_linear_backward(*l, dy, T, dx_add, add_dtype, dx, dx_dtype, db,
                                               db_dtype, ws, s),
                  "moe4_linear_backward");
}

static int check_layer_decode(const moe4_experts* ex, int32_t T, int32_t k) {
  int rc = check_experts(ex);
  if (rc) return rc;
  if (ex->lora_A)
    return fail(MOE4_EUNSUPPORTED, "moe4_layer_decode: adapters (lora_A) take moe4_expert_forward");
  if (ex->variant == MOE4_VARIANT_TILED)
    return fail(MOE4_EUNSUPPORTED, "moe4_layer_decode: moe4_experts.variant TILED");
  // the width up to which the other calls decode both levels of the absmax in place; beyond it they
  // expand them into their workspace, which this one does not
  if (ex->format == MOE4_FMT_NF4_DQ && (ex->H > 16384 || ex->I > 16384))
    return fail(MOE4_EUNSUPPORTED, "moe4_layer_decode: double-quantised rows of H = %d, I = %d "
                "beyond 16384", ex->H, ex->I);
  // all rows of h (512 of I bf16 values) and all tokens stand in one buffer each, of 32-bit byte offsets
  if (ex->H > 1 << 20 || ex->I > 1 << 20)
    return fail(MOE4_ESHAPE, "moe4_layer_decode: H = %d, I = %d beyond 2^20", ex->H, ex->I);
  if (T < 0 || T > MOE4_LAYER_MOST_TOKENS)
    return fail(MOE4_ESHAPE, "T = %d outside [0, %d]", T, (int)MOE4_LAYER_MOST_TOKENS);
  if (k < 1 || k > ex->E) return fail(MOE4_ESHAPE, "k = %d outside [1, E = %d]", k, ex->E);
  if ((int64_t)T * k > MOE4_LAYER_MOST_SLOTS)
    return fail(MOE4_ESHAPE, "T * k = %lld beyond %d slots", (long long)T * k,
                (int)MOE4_LAYER_MOST_SLOTS);
  return MOE4_OK;
}

size_t moe4_layer_decode_workspace_size(const moe4_experts* ex, int32_t T, int32_t k) {
  if (check_layer_decode(ex, T, k) != MOE4_OK) return 0;
  ok();
  const size_t need = moe4::layer_decode_ws_bytes(*ex, T, k);
  return need < 256 ? 256 : need;
}

int moe4_layer_decode(const moe4_experts* ex, const uint16_t* x, const float* logits, int32_t T,
                      int32_t k, int32_t renormalize, const void* residual, int32_t res_dtype,
                      void* out, int32_t out_dtype, int32_t* topk_idx, float* topk_w, void* ws,
                      size_t ws_bytes, void* stream) {
  int rc = check_layer_decode(ex, T, k);
  if (rc) return rc;
  REQUIRE_DTYPE(out_dtype, "out_dtype");
  if (residual) REQUIRE_DTYPE(res_dtype, "res_dtype");
  if (T == 0) return ok();
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(logits, "logits");
  REQUIRE_PTR(out, "out");
  REQUIRE_ALIGN(x, 16, "x");
  REQUIRE_ALIGN(logits, 4, "logits");
  REQUIRE_ALIGN(residual, 16, "residual");
  REQUIRE_ALIGN(out, 16, "out");
  REQUIRE_ALIGN(topk_idx, 4, "topk_idx");
  REQUIRE_ALIGN(topk_w, 4, "topk_w");
  rc = check_ws(ws, ws_bytes, moe4::layer_decode_ws_bytes(*ex, T, k), "moe4_layer_decode");
  if (rc) return rc;
  return launched(moe4::launch_layer_decode(*ex, x, logits, T, k, renormalize, residual, res_dtype,
                                            out, out_dtype, topk_idx, topk_w, ws,
                                            (hipStream_t)stream),
                  "moe4_layer_decode");
}

size_t moe4_workspace_size(const moe4_experts* ex, int32_t T, int32_t k) {
  if (check_experts(ex) != MOE4_OK) return 0;
  if (T < 0 || k < 1 || k > ex->E || (int64_t)T * k >= ((int64_t)1 << 31)) {
    fail(MOE4_ESHAPE, "moe4_workspace_size: T = %d, k = %d invalid", T, k);
    return 0;
  }
  const int rows = T * k;
  size_t need = moe4::permute_ws_bytes(T, k, ex->E);
  const size_t f = moe4::forward_ws_bytes(*ex, rows);
  const size_t b = moe4::backward_ws_bytes(*ex, rows);
  if (f > need) need = f;
  if (b > need) need = b;
  ok();
  return need < 256 ? 256 : need;
}

int moe4_set_timing_events(void* const* events, int32_t n_events) {
  if (events == nullptr || n_events == 0) {
    g_events = nullptr;
    return ok();
  }
  if (n_events < 4) return fail(MOE4_EINVAL, "n_events = %d: need 0 or at least 4", n_events);
  g_events = reinterpret_cast<hipEvent_t const*>(events);
  return ok();
}

const char* moe4_last_error(void) { return g_err; }

int moe4_last_variant(void) { return g_variant; }

}  // extern "C"
