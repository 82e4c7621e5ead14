"""Thin Python binding of libmoe4 (ctypes). Same names as the C interface in
include/moe4.h; the functions only marshal torch tensors into pointers, sizes
and the current HIP stream. Every step of the layer runs in the library's HIP
kernels; nothing here computes.

Importing this module loads libmoe4.so and fails loudly when it is missing.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# MOE4_LIB_PATH names another build of the same library (the host-only ASan
# build that tests/test_abi_asan.py loads); by default the in-tree libmoe4.so
LIB_PATH = os.environ.get("MOE4_LIB_PATH") or os.path.join(_HERE, "libmoe4.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; build it with `python -m bit_mixture_experts_amd.build` "
        "or __graft_entry__.build()")

_lib = ctypes.CDLL(LIB_PATH)

MOE4_OK, MOE4_EINVAL, MOE4_EUNSUPPORTED, MOE4_ESHAPE = 0, -1, -2, -3
MOE4_EALIGN, MOE4_EWORKSPACE, MOE4_EDEVICE = -4, -5, -6
MOE4_FMT_NF4, MOE4_FMT_MXFP4, MOE4_FMT_NF4_DQ = 1, 2, 3
MOE4_DQ_WS_BYTES = 8192
MOE4_GU_HALVES, MOE4_GU_INTERLEAVED = 1, 2
MOE4_ACT_SWIGLU, MOE4_ACT_SWIGLU_CLAMPED = 1, 2
MOE4_VARIANT_AUTO, MOE4_VARIANT_SKINNY, MOE4_VARIANT_TILED = 0, 1, 2
MOE4_DTYPE_BF16, MOE4_DTYPE_F32 = 1, 2
MOE4_NOALLOC_SCRATCH_BYTES = 16 << 20
MOE4_FFN_BF16, MOE4_FFN_MXFP8 = 1, 2

# every symbol declared in include/moe4.h
EXPORTS = ("moe4_quantize_nf4", "moe4_compress_absmax", "moe4_expand_absmax",
           "moe4_decode_mxfp4", "moe4_convert_mxfp4_nf4",
           "moe4_router_logits", "moe4_route", "moe4_route_backward", "moe4_permute",
           "moe4_gather_rows", "moe4_route_permute", "moe4_expert_forward", "moe4_expert_forward_gather", "moe4_expert_forward_noalloc", "moe4_combine",
           "moe4_expert_backward",
           "moe4_add_rmsnorm", "moe4_add_rmsnorm_backward", "moe4_add_rmsnorm_workspace_size",
           "moe4_quantize_mxfp8", "moe4_ffn_forward", "moe4_ffn_backward",
           "moe4_ffn_workspace_size", "moe4_grad_norm", "moe4_clip_grads",
           "moe4_grad_workspace_size",
           "moe4_workspace_size", "moe4_set_timing_events", "moe4_last_error",
           "moe4_last_variant")


class Moe4Experts(ctypes.Structure):
    """Mirror of the C struct moe4_experts."""
    _fields_ = [
        ("format", ctypes.c_int32), ("E", ctypes.c_int32), ("H", ctypes.c_int32),
        ("I", ctypes.c_int32), ("gu_layout", ctypes.c_int32), ("act", ctypes.c_int32),
        ("act_alpha", ctypes.c_float), ("act_limit", ctypes.c_float),
        ("gu_q", ctypes.c_void_p), ("gu_s", ctypes.c_void_p),
        ("dn_q", ctypes.c_void_p), ("dn_s", ctypes.c_void_p),
        ("gu_bias", ctypes.c_void_p), ("dn_bias", ctypes.c_void_p),
        ("lora_A", ctypes.c_void_p), ("lora_B", ctypes.c_void_p),
        ("lora_r", ctypes.c_int32), ("lora_scale", ctypes.c_float),
        ("variant", ctypes.c_int32),
        ("gu_s2", ctypes.c_void_p), ("dn_s2", ctypes.c_void_p),
        ("gu_soff", ctypes.c_void_p), ("dn_soff", ctypes.c_void_p),
        ("dq_book", ctypes.c_void_p),
    ]


class Moe4Ffn(ctypes.Structure):
    """Mirror of the C struct moe4_ffn."""
    _fields_ = [
        ("format", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
        ("gu_layout", ctypes.c_int32), ("act", ctypes.c_int32),
        ("act_alpha", ctypes.c_float), ("act_limit", ctypes.c_float), ("variant", ctypes.c_int32),
        ("w_gu", ctypes.c_void_p), ("gu_s", ctypes.c_void_p),
        ("w_dn", ctypes.c_void_p), ("dn_s", ctypes.c_void_p),
        ("gu_bias", ctypes.c_void_p), ("dn_bias", ctypes.c_void_p),
    ]


_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_P = ctypes.POINTER(Moe4Experts)
_PF = ctypes.POINTER(Moe4Ffn)
_f32c = ctypes.c_float
_SIGS = {
    "moe4_quantize_nf4": ([_vp, _i64, _i32, _vp, _vp, _vp], ctypes.c_int),
    "moe4_decode_mxfp4": ([_vp, _vp, _i64, _i64, _vp, _vp], ctypes.c_int),
    "moe4_compress_absmax": ([_vp, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "moe4_expand_absmax": ([_vp, _vp, _vp, _vp, _i64, _vp, _vp], ctypes.c_int),
    "moe4_convert_mxfp4_nf4": ([_vp, _vp, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "moe4_route": ([_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp], ctypes.c_int),
    "moe4_router_logits": ([_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp], ctypes.c_int),
    "moe4_route_backward": ([_vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp,
                             _vp, _vp], ctypes.c_int),
    "moe4_permute": ([_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _sz, _vp],
                     ctypes.c_int),
    "moe4_gather_rows": ([_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp], ctypes.c_int),
    "moe4_route_permute": ([_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                            _vp, _vp, _sz, _vp], ctypes.c_int),
    "moe4_expert_forward": ([_P, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "moe4_expert_forward_noalloc": ([_P, _vp, _vp, _i32, _vp, _vp, _vp, _vp], ctypes.c_int),
    "moe4_expert_forward_gather": ([_P, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp],
                                   ctypes.c_int),
    "moe4_combine": ([_vp, _vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp], ctypes.c_int),
    "moe4_expert_backward": ([_P, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
                             ctypes.c_int),
    "moe4_add_rmsnorm": ([_vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _f32c, _vp, _vp, _vp,
                          _vp, _vp], ctypes.c_int),
    "moe4_add_rmsnorm_backward": ([_vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _vp,
                                   _i32, _vp, _vp, _sz, _vp], ctypes.c_int),
    "moe4_add_rmsnorm_workspace_size": ([_i32, _i32], ctypes.c_size_t),
    "moe4_quantize_mxfp8": ([_vp, _i32, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "moe4_ffn_forward": ([_PF, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _sz, _vp],
                         ctypes.c_int),
    "moe4_ffn_backward": ([_PF, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp,
                           _i32, _vp, _sz, _vp], ctypes.c_int),
    "moe4_ffn_workspace_size": ([_PF, _i32, _i32], ctypes.c_size_t),
    "moe4_grad_norm": ([_vp, _vp, _vp, _i32, _vp, _vp, _sz, _vp], ctypes.c_int),
    "moe4_clip_grads": ([_vp, _vp, _vp, _vp, _i32, _f32c, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "moe4_grad_workspace_size": ([_i32], ctypes.c_size_t),
    "moe4_workspace_size": ([_P, _i32, _i32], ctypes.c_size_t),
    "moe4_set_timing_events": ([_vp, _i32], ctypes.c_int),
    "moe4_last_error": ([], ctypes.c_char_p),
    "moe4_last_variant": ([], ctypes.c_int),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes, _f.restype = _args, _res


class Moe4Error(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"moe4 status {code}: {msg}")
        self.code = code


def moe4_last_error():
    return _lib.moe4_last_error().decode()


def moe4_last_variant():
    return _lib.moe4_last_variant()


def _check(rc):
    if rc != MOE4_OK:
        raise Moe4Error(rc, moe4_last_error())


def _ptr(t, dtypes=None, name="tensor"):
    """Device pointer of a contiguous GPU tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must live on the GPU")
    if not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_U8 = (torch.uint8,)
_F32 = (torch.float32,)
_I32 = (torch.int32,)


class Experts:
    """Owns references to one layer's stack tensors and the C descriptor."""

    def __init__(self, fmt, gu_q, gu_s, dn_q, dn_s, *, gu_layout, act, E, H, I,
                 gu_bias=None, dn_bias=None, lora_A=None, lora_B=None, lora_scale=0.0,
                 act_alpha=1.702, act_limit=7.0, variant=MOE4_VARIANT_AUTO,
                 gu_s2=None, dn_s2=None, gu_soff=None, dn_soff=None, dq_book=None):
        """fmt MOE4_FMT_NF4_DQ: gu_s / dn_s are the u8 absmax codes and
        gu_s2, dn_s2, gu_soff, dn_soff, dq_book the rest of the nested absmax
        (see moe4_compress_absmax)."""
        sdt = _F32 if fmt == MOE4_FMT_NF4 else _U8
        self.tensors = (gu_q, gu_s, dn_q, dn_s, gu_bias, dn_bias, lora_A, lora_B,
                        gu_s2, dn_s2, gu_soff, dn_soff, dq_book)
        self.desc = Moe4Experts(
            format=fmt, E=E, H=H, I=I, gu_layout=gu_layout, act=act,
            act_alpha=act_alpha, act_limit=act_limit,
            gu_q=_ptr(gu_q, _U8, "gu_q"), gu_s=_ptr(gu_s, sdt, "gu_s"),
            dn_q=_ptr(dn_q, _U8, "dn_q"), dn_s=_ptr(dn_s, sdt, "dn_s"),
            gu_bias=_ptr(gu_bias, _BF16, "gu_bias"), dn_bias=_ptr(dn_bias, _BF16, "dn_bias"),
            lora_A=_ptr(lora_A, _BF16, "lora_A"), lora_B=_ptr(lora_B, _BF16, "lora_B"),
            lora_r=0 if lora_A is None else int(lora_A.shape[1]),
            lora_scale=lora_scale, variant=variant,
            gu_s2=_ptr(gu_s2, _F32, "gu_s2"), dn_s2=_ptr(dn_s2, _F32, "dn_s2"),
            gu_soff=_ptr(gu_soff, _F32, "gu_soff"), dn_soff=_ptr(dn_soff, _F32, "dn_soff"),
            dq_book=_ptr(dq_book, _F32, "dq_book"))
        self.E, self.H, self.I = E, H, I
        self.lora_r = self.desc.lora_r

    def with_variant(self, variant):
        d = Moe4Experts()
        ctypes.pointer(d)[0] = self.desc
        d.variant = variant
        out = object.__new__(Experts)
        out.__dict__.update(self.__dict__)
        out.desc = d
        return out


def moe4_quantize_nf4(w, packed, absmax, blocksize=64, stream=None):
    _check(_lib.moe4_quantize_nf4(_ptr(w, _F32, "w"), w.numel(), blocksize,
                                  _ptr(packed, _U8, "packed"), _ptr(absmax, _F32, "absmax"),
                                  _stream(stream)))


def moe4_compress_absmax(absmax, book, code, absmax2, offset, ws, stream=None):
    """absmax f32 [n] -> code u8 [n], absmax2 f32 [ceil(n/256)], offset f32 [1];
    ws: at least MOE4_DQ_WS_BYTES bytes of device scratch."""
    n = absmax.numel()
    if code.numel() != n or absmax2.numel() != (n + 255) // 256 or offset.numel() != 1:
        raise ValueError("compress_absmax: output sizes do not match n")
    _check(_lib.moe4_compress_absmax(_ptr(absmax, _F32, "absmax"), n, _ptr(book, _F32, "book"),
                                     _ptr(code, _U8, "code"), _ptr(absmax2, _F32, "absmax2"),
                                     _ptr(offset, _F32, "offset"), _ptr(ws, None, "ws"),
                                     ws.numel() * ws.element_size(), _stream(stream)))


def moe4_expand_absmax(code, absmax2, offset, book, out, stream=None):
    n = code.numel()
    if out.numel() != n or absmax2.numel() != (n + 255) // 256:
        raise ValueError("expand_absmax: sizes do not match")
    _check(_lib.moe4_expand_absmax(_ptr(code, _U8, "code"), _ptr(absmax2, _F32, "absmax2"),
                                   _ptr(offset, _F32, "offset"), _ptr(book, _F32, "book"), n,
                                   _ptr(out, _F32, "out"), _stream(stream)))


def moe4_decode_mxfp4(blocks, scales, out, stream=None):
    R = scales.numel() // scales.shape[-1] if scales.dim() else 0
    K = scales.shape[-1] * 32
    _check(_lib.moe4_decode_mxfp4(_ptr(blocks, _U8, "blocks"), _ptr(scales, _U8, "scales"),
                                  R, K, _ptr(out, _BF16, "out"), _stream(stream)))


def moe4_convert_mxfp4_nf4(blocks, scales, packed, absmax, stream=None):
    """blocks u8 [..., K/32, 16], scales u8 [..., K/32] -> packed u8 [..., K/2],
    absmax f32 [..., K/64]."""
    R = scales.numel() // scales.shape[-1] if scales.dim() else 0
    K = scales.shape[-1] * 32
    if packed.numel() != R * K // 2 or absmax.numel() != R * (K // 64):
        raise ValueError("packed / absmax do not match the MXFP4 stack's size")
    _check(_lib.moe4_convert_mxfp4_nf4(_ptr(blocks, _U8, "blocks"), _ptr(scales, _U8, "scales"),
                                       R, K, _ptr(packed, _U8, "packed"),
                                       _ptr(absmax, _F32, "absmax"), _stream(stream)))


def moe4_route(logits, k, topk_idx, topk_w, renormalize=True, stream=None):
    T, E = logits.shape
    _check(_lib.moe4_route(_ptr(logits, _F32, "logits"), T, E, k, int(bool(renormalize)),
                           _ptr(topk_idx, _I32, "topk_idx"), _ptr(topk_w, _F32, "topk_w"),
                           _stream(stream)))


def moe4_router_logits(x, wr, logits, bias=None, stream=None):
    """x bf16 [T, H], wr bf16 [E, H], bias f32 [E] or None -> logits f32 [T, E]."""
    T, H = x.shape
    E = wr.shape[0]
    if wr.shape[1] != H or tuple(logits.shape) != (T, E):
        raise ValueError("router_logits: x [T,H], wr [E,H] and logits [T,E] do not agree")
    _check(_lib.moe4_router_logits(_ptr(x, _BF16, "x"), _ptr(wr, _BF16, "wr"),
                                   _ptr(bias, _F32, "bias"), T, H, E,
                                   _ptr(logits, _F32, "logits"), _stream(stream)))


def moe4_route_backward(topk_idx, topk_w, dout, y_perm, row_of_slot, dw, dlogits,
                        logits=None, renormalize=True, stream=None):
    """dw f32 [T, k] and dlogits f32 [T, E] from the upstream gradient dout
    bf16 [T, H] and the slots' expert outputs y_perm f32 [T*k, H]."""
    T, k = topk_idx.shape
    E = dlogits.shape[1]
    H = dout.shape[1]
    _check(_lib.moe4_route_backward(_ptr(topk_idx, _I32, "topk_idx"), _ptr(topk_w, _F32, "topk_w"),
                                    _ptr(logits, _F32, "logits"), int(bool(renormalize)),
                                    _ptr(dout, _BF16, "dout"), _ptr(y_perm, _F32, "y_perm"),
                                    _ptr(row_of_slot, _I32, "row_of_slot"), T, k, E, H,
                                    _ptr(dw, _F32, "dw"), _ptr(dlogits, _F32, "dlogits"),
                                    _stream(stream)))


def moe4_permute(topk_idx, E, offsets, slot_of_row, row_of_slot, x=None, row_scale=None,
                 x_perm=None, ws=None, stream=None):
    T, k = topk_idx.shape
    H = 0 if x is None else x.shape[1]
    _check(_lib.moe4_permute(_ptr(topk_idx, _I32, "topk_idx"), T, k, E,
                             _ptr(offsets, _I32, "offsets"), _ptr(slot_of_row, _I32, "slot_of_row"),
                             _ptr(row_of_slot, _I32, "row_of_slot"), _ptr(x, _BF16, "x"),
                             _ptr(row_scale, _F32, "row_scale"), H,
                             _ptr(x_perm, _BF16, "x_perm"), _ptr(ws, None, "ws"),
                             0 if ws is None else ws.numel() * ws.element_size(),
                             _stream(stream)))


def moe4_gather_rows(x, k, slot_of_row, x_perm, row_scale=None, stream=None):
    """The row gather of moe4_permute on an existing permutation (slot_of_row)."""
    T, H = x.shape
    _check(_lib.moe4_gather_rows(_ptr(x, _BF16, "x"), T, k, H,
                                 _ptr(slot_of_row, _I32, "slot_of_row"),
                                 _ptr(row_scale, _F32, "row_scale"), _ptr(x_perm, _BF16, "x_perm"),
                                 _stream(stream)))


def moe4_route_permute(logits, k, topk_idx, topk_w, offsets, slot_of_row, row_of_slot, x=None,
                       x_perm=None, ws=None, renormalize=True, stream=None):
    """moe4_route then moe4_permute (no row_scale), one launch for small batches."""
    T, E = logits.shape
    H = 0 if x is None else x.shape[1]
    _check(_lib.moe4_route_permute(_ptr(logits, _F32, "logits"), T, E, k, int(bool(renormalize)),
                                   _ptr(topk_idx, _I32, "topk_idx"), _ptr(topk_w, _F32, "topk_w"),
                                   _ptr(offsets, _I32, "offsets"),
                                   _ptr(slot_of_row, _I32, "slot_of_row"),
                                   _ptr(row_of_slot, _I32, "row_of_slot"), _ptr(x, _BF16, "x"), H,
                                   _ptr(x_perm, _BF16, "x_perm"), _ptr(ws, None, "ws"),
                                   0 if ws is None else ws.numel() * ws.element_size(),
                                   _stream(stream)))


def moe4_expert_forward_gather(ex, x, k, slot_of_row, offsets, y_perm, save_gu=None, ws=None,
                               stream=None):
    """moe4_expert_forward on rows gathered from x [T, H] by the GEMM itself."""
    T = x.shape[0]
    _check(_lib.moe4_expert_forward_gather(ctypes.byref(ex.desc), _ptr(x, _BF16, "x"), T, k,
                                           _ptr(slot_of_row, _I32, "slot_of_row"),
                                           _ptr(offsets, _I32, "offsets"), T * k,
                                           _ptr(y_perm, _F32, "y_perm"),
                                           _ptr(save_gu, _F32, "save_gu"), _ptr(ws, None, "ws"),
                                           0 if ws is None else ws.numel() * ws.element_size(),
                                           _stream(stream)))


def moe4_expert_forward(ex, x_perm, offsets, y_perm, save_gu=None, save_xa=None, ws=None,
                        stream=None):
    _check(_lib.moe4_expert_forward(ctypes.byref(ex.desc), _ptr(x_perm, _BF16, "x_perm"),
                                    _ptr(offsets, _I32, "offsets"), x_perm.shape[0],
                                    _ptr(y_perm, _F32, "y_perm"), _ptr(save_gu, _F32, "save_gu"),
                                    _ptr(save_xa, _F32, "save_xa"), _ptr(ws, None, "ws"),
                                    0 if ws is None else ws.numel() * ws.element_size(),
                                    _stream(stream)))


def moe4_expert_forward_noalloc(ex, x_perm, offsets, y_perm, save_gu=None, save_xa=None,
                                stream=None):
    """moe4_expert_forward with the library's per-device scratch in place of a
    workspace (allocates nothing)."""
    _check(_lib.moe4_expert_forward_noalloc(
        ctypes.byref(ex.desc), _ptr(x_perm, _BF16, "x_perm"), _ptr(offsets, _I32, "offsets"),
        x_perm.shape[0], _ptr(y_perm, _F32, "y_perm"), _ptr(save_gu, _F32, "save_gu"),
        _ptr(save_xa, _F32, "save_xa"), _stream(stream)))


def moe4_combine(y_perm, row_of_slot, topk_w, out, k, stream=None):
    """out: bf16 [T, H] (rounded once) or float32 [T, H] (the fp32 sum)."""
    T, H = out.shape
    dt = MOE4_DTYPE_F32 if out.dtype == torch.float32 else MOE4_DTYPE_BF16
    _check(_lib.moe4_combine(_ptr(y_perm, _F32, "y_perm"), _ptr(row_of_slot, _I32, "row_of_slot"),
                             _ptr(topk_w, _F32, "topk_w"), T, k, H,
                             _ptr(out, _BF16 + _F32, "out"), dt, _stream(stream)))


def moe4_expert_backward(ex, x_perm, offsets, save_gu, save_xa, dy_perm, dx_perm, dA=None,
                         dB=None, ws=None, stream=None):
    _check(_lib.moe4_expert_backward(ctypes.byref(ex.desc), _ptr(x_perm, _BF16, "x_perm"),
                                     _ptr(offsets, _I32, "offsets"), dy_perm.shape[0],
                                     _ptr(save_gu, _F32, "save_gu"), _ptr(save_xa, _F32, "save_xa"),
                                     _ptr(dy_perm, _BF16, "dy_perm"), _ptr(dx_perm, _F32, "dx_perm"),
                                     _ptr(dA, _F32, "dA"), _ptr(dB, _F32, "dB"),
                                     _ptr(ws, None, "ws"),
                                     0 if ws is None else ws.numel() * ws.element_size(),
                                     _stream(stream)))


def moe4_set_timing_events(events):
    """events: a ctypes array of hipEvent_t handles (len >= 4), or None to stop.
    The caller keeps the array alive while timing is on."""
    if events is None:
        _check(_lib.moe4_set_timing_events(None, 0))
    else:
        _check(_lib.moe4_set_timing_events(ctypes.cast(events, ctypes.c_void_p), len(events)))


def moe4_workspace_size(ex, T, k):
    n = _lib.moe4_workspace_size(ctypes.byref(ex.desc), T, k)
    if n == 0:
        raise Moe4Error(MOE4_EINVAL, moe4_last_error())
    return n


# ---- the dense half of the block: norm, MXFP8, feed-forward block, gradient clipping.
# These check every size against the others (the kernels trust them) and that all tensors,
# and the stream, are on the current device.

_CODES = (torch.uint8, torch.float8_e4m3fn)
_SCALES = (torch.uint8, torch.float8_e8m0fnu)
_FLOATS = (torch.bfloat16, torch.float32)


_DT = {torch.bfloat16: MOE4_DTYPE_BF16, torch.float32: MOE4_DTYPE_F32}


def _dt(t):
    return 0 if t is None else _DT.get(t.dtype, 0)   # what is neither is refused as a pointer


class _Call:
    """Pointers of one call's tensors: shape, dtype, contiguity and device checked. A decode
    step's kernels are a few microseconds long, so the way without an error is kept short."""
    __slots__ = ("fn", "dev")

    def __init__(self, fn):
        self.fn = fn
        self.dev = -2   # none yet (a CPU tensor's is -1)

    def ptr(self, t, name, shape, dtypes):
        if t is None:
            return None
        try:
            dev = t.get_device()
        except AttributeError:
            raise TypeError(f"{name} must be a torch.Tensor") from None
        if dev != self.dev:
            self.place(t, name)
        if t.dtype not in dtypes or not t.is_contiguous():
            _ptr(t, dtypes, name)
        if t.shape != shape:
            raise ValueError(f"{self.fn}: {name} has shape {tuple(t.shape)}, expected {shape}")
        return t.data_ptr()

    def place(self, t, name):
        if not t.is_cuda:
            raise TypeError(f"{name} must live on the GPU")
        d = t.get_device()
        if self.dev >= 0 and d != self.dev:
            raise ValueError(f"{self.fn}: {name} is on device {d}, other tensors on {self.dev}")
        if d != torch.cuda.current_device():
            raise ValueError(f"{self.fn}: {name} is on device {d}, the current device is "
                             f"{torch.cuda.current_device()}")
        self.dev = d

    def ws(self, ws):
        if ws is None:
            return None, 0
        if ws.get_device() != self.dev:
            self.place(ws, "ws")
        if not ws.is_contiguous():
            _ptr(ws, None, "ws")
        return ws.data_ptr(), ws.nbytes

    def stream(self, stream):
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(max(self.dev, 0))
        d = getattr(stream, "device_index", self.dev)
        if d != self.dev:
            raise ValueError(f"{self.fn}: the stream is on device {d}, the tensors on {self.dev}")
        return _stream(stream)


def _int32(fn, **sizes):
    """Sizes that the C interface takes as int32 (ctypes would cut a larger one off silently)."""
    for name, v in sizes.items():
        if not -(1 << 31) <= v < 1 << 31:   # a negative one is for the C interface to refuse
            raise ValueError(f"{fn}: {name} = {v} outside int32")


def moe4_add_rmsnorm(x, weight, eps, residual=None, sum_out=None, out=None, out_q=None, out_s=None,
                     rstd=None, stream=None):
    """s = x + residual (rounded to the residual's type; sum_out), y = s * rstd * weight, as bf16
    (out) and, or, MXFP8 (out_q u8 or float8_e4m3fn [T, H], out_s u8 or float8_e8m0fnu [T, H/32]).
    x, residual bf16 or f32 [T, H]; weight bf16 or f32 [H]; rstd f32 [T]."""
    c = _Call("add_rmsnorm")
    T, H = sh = x.shape
    if T >> 31 or H >> 31:
        _int32(c.fn, T=T, H=H)
    if sum_out is not None and residual is not None and sum_out.dtype != residual.dtype:
        raise TypeError("sum_out must have the residual's dtype")
    ptr = c.ptr
    rc = _lib.moe4_add_rmsnorm(
        ptr(x, "x", sh, _FLOATS), _dt(x),
        None if residual is None else ptr(residual, "residual", sh, _FLOATS), _dt(residual),
        None if sum_out is None else ptr(sum_out, "sum_out", sh, _FLOATS),
        ptr(weight, "weight", (H,), _FLOATS), _dt(weight), T, H, eps,
        None if out is None else ptr(out, "out", sh, _BF16),
        None if out_q is None else ptr(out_q, "out_q", sh, _CODES),
        None if out_s is None else ptr(out_s, "out_s", (T, H // 32), _SCALES),
        None if rstd is None else ptr(rstd, "rstd", (T,), _F32), c.stream(stream))
    if rc:
        _check(rc)


def moe4_add_rmsnorm_workspace_size(T, H):
    _int32("add_rmsnorm_workspace_size", T=T, H=H)
    n = _lib.moe4_add_rmsnorm_workspace_size(T, H)
    if n == 0:
        raise Moe4Error(MOE4_ESHAPE, moe4_last_error())
    return n


def moe4_add_rmsnorm_backward(dy, s, weight, rstd, dx, dres=None, dweight=None, ws=None,
                              stream=None):
    """Gradient of moe4_add_rmsnorm: dx (of x and of the residual alike; dres, of dx's dtype, is
    added) and dweight f32 [H]. s: the forward's sum_out (its x without a residual)."""
    c = _Call("add_rmsnorm_backward")
    T, H = sh = s.shape
    if T >> 31 or H >> 31:
        _int32(c.fn, T=T, H=H)
    if dres is not None and dres.dtype != dx.dtype:
        raise TypeError("dres must have dx's dtype")
    ps = c.ptr(s, "s", sh, _FLOATS)
    pw, nw = c.ws(ws)
    _check(_lib.moe4_add_rmsnorm_backward(
        c.ptr(dy, "dy", sh, _FLOATS), _dt(dy), ps, _dt(s), c.ptr(weight, "weight", (H,), _FLOATS),
        _dt(weight), c.ptr(rstd, "rstd", (T,), _F32), c.ptr(dres, "dres", sh, _FLOATS), T, H,
        c.ptr(dx, "dx", sh, _FLOATS), _dt(dx), c.ptr(dweight, "dweight", (H,), _F32), pw, nw,
        c.stream(stream)))


def moe4_quantize_mxfp8(x, q, s, stream=None):
    """x bf16 or f32 [..., K] -> q (u8 or float8_e4m3fn) [..., K], s (u8 or float8_e8m0fnu)
    [..., K/32]."""
    c = _Call("quantize_mxfp8")
    sh = tuple(x.shape)
    if not sh:
        raise ValueError("quantize_mxfp8: x has no dimension")
    K = sh[-1]
    R = x.numel() // K if K else 0
    rc = _lib.moe4_quantize_mxfp8(c.ptr(x, "x", sh, _FLOATS), _dt(x), R, K,
                                  c.ptr(q, "q", sh, _CODES),
                                  c.ptr(s, "s", sh[:-1] + (K // 32,), _SCALES), c.stream(stream))
    if rc:
        _check(rc)


class Ffn:
    """Owns references to a dense feed-forward block's tensors and the C descriptor (moe4_ffn).
    fmt MOE4_FFN_BF16: w_gu bf16 [2I, H], w_dn bf16 [H, I]; MOE4_FFN_MXFP8: codes of the same
    shapes with scales gu_s [2I, H/32], dn_s [H, I/32] (moe4_quantize_mxfp8)."""

    def __init__(self, fmt, w_gu, w_dn, *, gu_layout, act, H, I, gu_s=None, dn_s=None,
                 gu_bias=None, dn_bias=None, act_alpha=1.702, act_limit=7.0,
                 variant=MOE4_VARIANT_AUTO):
        c = _Call("Ffn")
        _int32("Ffn", H=H, I=I)
        wdt = _CODES if fmt == MOE4_FFN_MXFP8 else _BF16
        self.tensors = (w_gu, w_dn, gu_s, dn_s, gu_bias, dn_bias)
        self.desc = Moe4Ffn(
            format=fmt, H=H, I=I, gu_layout=gu_layout, act=act, act_alpha=act_alpha,
            act_limit=act_limit, variant=variant,
            w_gu=c.ptr(w_gu, "w_gu", (2 * I, H), wdt),
            gu_s=c.ptr(gu_s, "gu_s", (2 * I, H // 32), _SCALES),
            w_dn=c.ptr(w_dn, "w_dn", (H, I), wdt),
            dn_s=c.ptr(dn_s, "dn_s", (H, I // 32), _SCALES),
            gu_bias=c.ptr(gu_bias, "gu_bias", (2 * I,), _BF16),
            dn_bias=c.ptr(dn_bias, "dn_bias", (H,), _BF16))
        self.H, self.I = H, I
        self.device = w_gu.get_device()
        self.ref = ctypes.byref(self.desc)

    def with_variant(self, variant):
        d = Moe4Ffn()
        ctypes.pointer(d)[0] = self.desc
        d.variant = variant
        out = object.__new__(Ffn)
        out.__dict__.update(self.__dict__)
        out.desc, out.ref = d, ctypes.byref(d)
        return out


def _ffn_call(fn, ffn):
    c = _Call(fn)
    c.place(ffn.tensors[0], "w_gu")
    return c


def moe4_ffn_workspace_size(ffn, T, backward=False):
    _int32("ffn_workspace_size", T=T)
    n = _lib.moe4_ffn_workspace_size(ffn.ref, T, int(bool(backward)))
    if n == 0:
        raise Moe4Error(MOE4_EINVAL, moe4_last_error())
    return n


def moe4_ffn_forward(ffn, x, out, x_s=None, residual=None, save_gu=None, ws=None, stream=None):
    """out [T, H] (bf16 or f32) = the block on x (bf16, or MXFP8 codes with scales x_s) +
    residual (bf16 or f32); save_gu f32 [T, 2I]: the pre-activations for the backward pass."""
    c = _ffn_call("ffn_forward", ffn)
    T, H = x.shape[0], ffn.H
    if T >> 31:
        _int32(c.fn, T=T)
    mx = ffn.desc.format == MOE4_FFN_MXFP8
    pw, nw = c.ws(ws)
    ptr, sh = c.ptr, (T, H)
    rc = _lib.moe4_ffn_forward(
        ffn.ref, ptr(x, "x", sh, _CODES if mx else _BF16),
        None if x_s is None else ptr(x_s, "x_s", (T, H // 32), _SCALES), T,
        None if residual is None else ptr(residual, "residual", sh, _FLOATS), _dt(residual),
        ptr(out, "out", sh, _FLOATS), _dt(out),
        None if save_gu is None else ptr(save_gu, "save_gu", (T, 2 * ffn.I), _F32), pw, nw,
        c.stream(stream))
    if rc:
        _check(rc)


def moe4_ffn_backward(ffn, x, save_gu, dy, dx=None, dx_add=None, dw_gu=None, dw_dn=None,
                      db_gu=None, db_dn=None, ws=None, stream=None):
    """Gradients of moe4_ffn_forward (bf16 blocks) from dy bf16 [T, H]: dx (bf16 or f32; dx_add is
    added), dw_gu, dw_dn, db_gu, db_dn (one dtype, bf16 or f32); each may be None."""
    c = _ffn_call("ffn_backward", ffn)
    T, H, I = dy.shape[0], ffn.H, ffn.I
    if T >> 31:
        _int32(c.fn, T=T)
    given = [t for t in (dw_gu, dw_dn, db_gu, db_dn) if t is not None]
    if any(t.dtype != given[0].dtype for t in given):
        raise TypeError("the weights' and biases' gradients must have one dtype")
    pw, nw = c.ws(ws)
    _check(_lib.moe4_ffn_backward(
        ffn.ref, c.ptr(x, "x", (T, H), _BF16), T, c.ptr(save_gu, "save_gu", (T, 2 * I), _F32),
        c.ptr(dy, "dy", (T, H), _BF16), c.ptr(dx_add, "dx_add", (T, H), _FLOATS), _dt(dx_add),
        c.ptr(dx, "dx", (T, H), _FLOATS), _dt(dx), c.ptr(dw_gu, "dw_gu", (2 * I, H), _FLOATS),
        c.ptr(dw_dn, "dw_dn", (H, I), _FLOATS), c.ptr(db_gu, "db_gu", (2 * I,), _FLOATS),
        c.ptr(db_dn, "db_dn", (H,), _FLOATS), _dt(given[0]) if given else 0, pw, nw,
        c.stream(stream)))


class GradList:
    """Owns references to a list of gradients (bf16 or f32, any shapes) and the host arrays that
    moe4_grad_norm and moe4_clip_grads read. outs: where moe4_clip_grads writes (same shapes and
    dtypes), None for in place. Build it anew when a gradient is another tensor. What
    moe4_clip_grads writes may overlap nothing else of the list (a gradient that is in it twice
    would be scaled by two workgroups at once): it refuses such a list."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = None if outs is None else list(outs)
        n = self.n = len(self.grads)
        if self.outs is not None and len(self.outs) != n:
            raise ValueError("GradList: outs and grads differ in length")
        c = _Call("GradList")
        self._in, self._numel = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)()
        self._dtype = (ctypes.c_int32 * n)()
        self._out = None if outs is None else (ctypes.c_void_p * n)()
        for i, g in enumerate(self.grads):
            self._in[i] = c.ptr(g, f"grads[{i}]", tuple(g.shape), _FLOATS)
            self._numel[i], self._dtype[i] = g.numel(), _dt(g)
            if self.outs is not None:
                self._out[i] = c.ptr(self.outs[i], f"outs[{i}]", tuple(g.shape), (g.dtype,))
        self.clash = self._overlap()

    def _overlap(self):
        """Where an output overlaps another output, or another entry's gradient: a message."""
        spans = []   # (first byte, end, entry, whether it is written)
        for i, g in enumerate(self.grads):
            size = g.numel() * g.element_size()
            if size == 0:
                continue
            out = self._in[i] if self._out is None else self._out[i]
            spans.append((out, out + size, i, True))
            if out != self._in[i]:
                spans.append((self._in[i], self._in[i] + size, i, False))
        spans.sort()
        end = {True: (0, 0), False: (0, 0)}   # the furthest byte written, read so far
        for a, b, i, written in spans:
            for w in (True, False) if written else (True,):
                if a < end[w][0]:
                    return f"outs[{i if written else end[w][1]}] overlaps entry {end[w][1] if written else i}"
            end[written] = max(end[written], (b, i))
        return None


def moe4_grad_workspace_size(grads):
    n = _lib.moe4_grad_workspace_size(grads.n)
    if n == 0:
        raise Moe4Error(MOE4_ESHAPE, moe4_last_error())
    return n


def _grad_call(fn, grads):
    c = _Call(fn)
    if grads.n:
        c.place(grads.grads[0], "grads[0]")
    return c


def moe4_grad_norm(grads, norm, ws, stream=None):
    """norm f32 [1]: the global norm of a GradList."""
    c = _grad_call("grad_norm", grads)
    pw, nw = c.ws(ws)
    _check(_lib.moe4_grad_norm(grads._in, grads._numel, grads._dtype, grads.n,
                               c.ptr(norm, "norm", (1,), _F32), pw, nw, c.stream(stream)))


def moe4_clip_grads(grads, max_norm, norm_out=None, ws=None, norm_in=None, stream=None):
    """Scales a GradList by min(1, max_norm / (norm + 1e-6)); the norm is norm_in where given,
    else the list's own; norm_out f32 [1] takes the norm used."""
    c = _grad_call("clip_grads", grads)
    if grads.clash:
        raise ValueError(f"clip_grads: {grads.clash}")
    pw, nw = c.ws(ws)
    _check(_lib.moe4_clip_grads(grads._in, grads._out, grads._numel, grads._dtype, grads.n,
                                max_norm, c.ptr(norm_in, "norm_in", (1,), _F32),
                                c.ptr(norm_out, "norm_out", (1,), _F32), pw, nw,
                                c.stream(stream)))
