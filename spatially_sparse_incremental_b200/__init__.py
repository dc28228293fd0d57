"""Python binding of libsige (the C ABI in include/sige.h).

Argument marshalling only: every step of the sparse layer runs in the CUDA
kernels of ``libsige.so``; torch supplies device memory and streams.  The
functions carry the ABI's names and raise ``SigeError`` on any non-OK status.
There is no fallback: if the library is missing, importing a call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsige.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_CAPACITY, ERR_TIMEOUT, ERR_WORKSPACE = 0, -1, -2, -3, -4, -5, -6
CALL_REDUCE_MASK, CALL_SPARSE_CONV, CALL_CONV_FUSED, CALL_DENSE_CONV, CALL_RESBLOCK = 0, 1, 2, 3, 4
U8, F32, BF16 = 0, 1, 2
NHWC, NCHW = 0, 1
WORKSPACE_HEADER = 256
MAX_SCALES = 8

_DT = {torch.uint8: U8, torch.float32: F32, torch.bfloat16: BF16}


class SigeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class TensorDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("h", ctypes.c_int32), ("w", ctypes.c_int32), ("c", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32)]


class ConvDesc(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("stride", ctypes.c_int32), ("pad", ctypes.c_int32),
                ("c_in", ctypes.c_int32), ("c_out", ctypes.c_int32), ("block", ctypes.c_int32)]


class LayerExt(ctypes.Structure):
    _fields_ = [("transposed", ctypes.c_int32), ("output_padding", ctypes.c_int32),
                ("spade_gamma", ctypes.c_void_p), ("spade_beta", ctypes.c_void_p), ("act", ctypes.c_int32)]


class QCacheDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("h", ctypes.c_int32), ("w", ctypes.c_int32), ("c", ctypes.c_int32),
                ("format", ctypes.c_int32), ("group", ctypes.c_int32)]


ACT_NONE, ACT_SILU, ACT_LEAKY = 0, 1, 2
Q_S8, Q_E4M3, Q_S4 = 0, 1, 2


class ScaleDesc(ctypes.Structure):
    _fields_ = [("h", ctypes.c_int32), ("w", ctypes.c_int32), ("block", ctypes.c_int32),
                ("capacity", ctypes.c_int32)]


# Every symbol include/sige.h declares, with its ctypes signature.
_vp, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_TD, _CD, _SD = ctypes.POINTER(TensorDesc), ctypes.POINTER(ConvDesc), ctypes.POINTER(ScaleDesc)
_LE = ctypes.POINTER(LayerExt)
_QD = ctypes.POINTER(QCacheDesc)
SIGNATURES = {
    "sige_reduce_mask_workspace_bytes": (_sz, [_TD, _i32, _SD]),
    "sige_reduce_mask": (_i32, [_vp, _vp, _TD, _f32, _i32, _i32, _SD, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sige_reduce_mask_px": (_i32, [_vp, _vp, _TD, _f32, _i32, _i32, _SD, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sige_reduce_mask_static": (_i32, [_vp, _vp, _TD, _f32, _i32, _i32, _SD, _vp, _vp, _vp]),
    "sige_gather": (_i32, [_vp, _TD, _CD, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _vp]),
    "sige_sparse_conv": (_i32, [_vp, _CD, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _sz, _vp]),
    "sige_scatter": (_i32, [_vp, _CD, _vp, _vp, _i32, _vp, _vp, _vp, _TD, _vp]),
    "sige_conv_fused": (_i32, [_vp, _TD, _vp, _vp, _CD, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _TD,
                               _vp, _sz, _vp]),
    "sige_resblock_step_workspace_bytes": (_sz, [_TD, _i32]),
    "sige_resblock_step": (_i32, [_vp, _vp, _TD, _f32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
                                  _i32, _vp, _vp, _vp, _sz, _vp]),
    "sige_conv_fused_ext": (_i32, [_vp, _TD, _vp, _vp, _CD, _LE, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _TD, _vp,
                                   _sz, _vp]),
    "sige_dense_conv": (_i32, [_vp, _TD, _vp, _vp, _CD, _vp, _vp, _i32, _vp, _vp, _TD, _vp, _sz, _vp]),
    "sige_groupnorm_affine": (_i32, [_vp, _TD, _i32, _vp, _vp, _f32, _vp, _vp, _vp]),
    "sige_resblock_fused": (_i32, [_vp, _TD, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _vp,
                                   _vp, _vp, _sz, _vp]),
    "sige_restore_tiles": (_i32, [_vp, _vp, _TD, _i32, _vp, _vp, _i32, _vp]),
    "sige_download_tiles_bytes": (_sz, [_TD, _i32, _i32]),
    "sige_download_tiles": (_i32, [_vp, _TD, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp]),
    "sige_conv_workspace_bytes": (_sz, [_CD, _i32, _i32, _i32, _i32]),
    "sige_get_error": (_i32, [_vp, _vp]),
    "sige_get_device_error": (_i32, [_vp, _vp]),
    "sige_workspace_bytes": (_sz, [_i32, _CD, _i32]),
    "sige_set_wait_cycles": (_i32, [ctypes.c_int64]),
    "sige_conv_path": (_i32, [_CD, _i32]),
    "sige_conv_schedule": (_i32, [_CD, _i32, _i32, _i32, _vp, _i32]),
    "sige_attention_core": (_i32, [_vp, _TD, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _i32, _i32, _vp, _vp]),
    "sige_attention_path": (_i32, [_TD, _i32, _i32]),
    "sige_qcache_code_bytes": (_sz, [_QD]),
    "sige_qcache_scales": (_sz, [_QD]),
    "sige_qcache_write": (_i32, [_vp, _TD, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _QD, _vp]),
    "sige_qcache_read": (_i32, [_vp, _vp, _QD, _i32, _vp, _vp, _i32, _vp, _TD, _vp]),
    "sige_qlinear": (_i32, [_vp, _vp, _QD, _vp, _vp, _QD, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _TD, _vp, _sz, _vp]),
    "sige_qlinear_path": (_i32, [_i32]),
    "sige_attention_qcache": (_i32, [_vp, _TD, _vp, _vp, _QD, _vp, _vp, _QD, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp,
                                     _sz, _vp]),
    "sige_attention_qcache_path": (_i32, [_i32, _i32]),
    "sige_launch_count": (ctypes.c_uint64, []),
    "sige_status_string": (ctypes.c_char_p, [_i32]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libsige.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().sige_status_string(int(status)).decode()
    except Exception:  # library missing
        return "status"


def _check(st: int, what: str):
    if st != OK:
        raise SigeError(st, what)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def tensor_desc(t: torch.Tensor, layout: int = NHWC) -> TensorDesc:
    if t.dim() != 4:
        raise ValueError("expected a 4-d tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if layout == NHWC:
        n, h, w, c = t.shape
    else:
        n, c, h, w = t.shape
    return TensorDesc(n, h, w, c, _DT[t.dtype], layout)


def conv_desc(kernel, stride, pad, c_in, c_out, block) -> ConvDesc:
    return ConvDesc(kernel, stride, pad, c_in, c_out, block)


def zeros_workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled device workspace (16-byte aligned, as torch allocations are)."""
    return torch.zeros(max(int(nbytes), WORKSPACE_HEADER), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ calls

def sige_reduce_mask_workspace_bytes(desc: TensorDesc, scales) -> int:
    arr = (ScaleDesc * len(scales))(*[ScaleDesc(*s) for s in scales])
    return int(lib().sige_reduce_mask_workspace_bytes(ctypes.byref(desc), len(scales), arr))


def _host_counts(n, want):
    return (ctypes.c_int32 * n)() if want else None


def sige_reduce_mask(a_orig, a_edit, threshold, scales, dilate=1, layout=NHWC, idx=None, counts=None,
                     workspace=None, stream=None, host_counts=False):
    """Difference mask -> per-scale active-tile lists.  ``scales`` is a list of
    (h, w, block, capacity).  Returns (idx [sum(capacity), 2] int32, counts
    [n_scales] int32, workspace); all on the device, nothing synchronised.
    With ``host_counts=True`` the call also copies the counts to the host
    (the library synchronises the stream) and returns them as a fourth item,
    a list of ints."""
    desc = tensor_desc(a_orig, layout)
    arr = (ScaleDesc * len(scales))(*[ScaleDesc(*s) for s in scales])
    dev = a_orig.device
    if idx is None:
        idx = torch.empty((max(1, sum(s[3] for s in scales)), 2), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty(len(scales), dtype=torch.int32, device=dev)
    need = int(lib().sige_reduce_mask_workspace_bytes(ctypes.byref(desc), len(scales), arr))
    if workspace is None:
        workspace = zeros_workspace(need, dev)
    hc = _host_counts(len(scales), host_counts)
    st = lib().sige_reduce_mask(_ptr(a_orig), _ptr(a_edit), ctypes.byref(desc), float(threshold), int(dilate),
                                len(scales), arr, _ptr(idx), _ptr(counts), hc, _ptr(workspace),
                                workspace.numel(), _stream(stream))
    _check(st, "sige_reduce_mask")
    if host_counts:
        return idx, counts, workspace, [int(v) for v in hc]
    return idx, counts, workspace


def sige_reduce_mask_px(a_orig, a_edit, threshold, scales, radius=1, layout=NHWC, idx=None, counts=None,
                        workspace=None, stream=None, host_counts=False):
    """As sige_reduce_mask, with the mask dilated by ``radius`` pixels at each
    scale before tiling (no tile dilation)."""
    desc = tensor_desc(a_orig, layout)
    arr = (ScaleDesc * len(scales))(*[ScaleDesc(*s) for s in scales])
    dev = a_orig.device
    if idx is None:
        idx = torch.empty((max(1, sum(s[3] for s in scales)), 2), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty(len(scales), dtype=torch.int32, device=dev)
    need = int(lib().sige_reduce_mask_workspace_bytes(ctypes.byref(desc), len(scales), arr))
    if workspace is None:
        workspace = zeros_workspace(need, dev)
    hc = _host_counts(len(scales), host_counts)
    st = lib().sige_reduce_mask_px(_ptr(a_orig), _ptr(a_edit), ctypes.byref(desc), float(threshold), int(radius),
                                   len(scales), arr, _ptr(idx), _ptr(counts), hc, _ptr(workspace),
                                   workspace.numel(), _stream(stream))
    _check(st, "sige_reduce_mask_px")
    if host_counts:
        return idx, counts, workspace, [int(v) for v in hc]
    return idx, counts, workspace


def sige_reduce_mask_static(a_orig, a_edit, threshold, scales, dilate=1, layout=NHWC, idx=None, counts=None,
                            stream=None):
    """sige_reduce_mask for callers that cannot allocate a workspace: the
    library's built-in 64 KB scratch is used instead (calls on one device must
    not overlap).  Returns (idx, counts)."""
    desc = tensor_desc(a_orig, layout)
    arr = (ScaleDesc * len(scales))(*[ScaleDesc(*s) for s in scales])
    dev = a_orig.device
    if idx is None:
        idx = torch.empty((max(1, sum(s[3] for s in scales)), 2), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty(len(scales), dtype=torch.int32, device=dev)
    st = lib().sige_reduce_mask_static(_ptr(a_orig), _ptr(a_edit), ctypes.byref(desc), float(threshold),
                                       int(dilate), len(scales), arr, _ptr(idx), _ptr(counts), _stream(stream))
    _check(st, "sige_reduce_mask_static")
    return idx, counts


def sige_gather(x, cd: ConvDesc, idx, count, capacity, gn_scale=None, gn_shift=None, silu=False,
                blocks=None, stream=None):
    xd = tensor_desc(x)
    bin_ = (cd.block - 1) * cd.stride + cd.kernel
    if blocks is None:
        blocks = torch.empty((max(capacity, 1), x.shape[0], bin_, bin_, cd.c_in), dtype=x.dtype, device=x.device)
    st = lib().sige_gather(_ptr(x), ctypes.byref(xd), ctypes.byref(cd), _ptr(idx), _ptr(count), int(capacity),
                           _ptr(gn_scale), _ptr(gn_shift), int(bool(silu)), _ptr(blocks), _stream(stream))
    _check(st, "sige_gather")
    return blocks


def sige_sparse_conv(blocks, cd: ConvDesc, weight, count, capacity, batch=1, out_blocks=None, workspace=None,
                     stream=None):
    if out_blocks is None:
        out_blocks = torch.empty((max(capacity, 1), batch, cd.block, cd.block, cd.c_out), dtype=torch.float32,
                                 device=blocks.device)
    if workspace is None:
        workspace = zeros_workspace(sige_conv_workspace_bytes(cd, batch, capacity, 0, 0), blocks.device)
    st = lib().sige_sparse_conv(_ptr(blocks), ctypes.byref(cd), _DT[blocks.dtype], int(batch), _ptr(weight),
                                _ptr(count), int(capacity), _ptr(out_blocks), _ptr(workspace), workspace.numel(),
                                _stream(stream))
    _check(st, "sige_sparse_conv")
    return out_blocks


def sige_scatter(out_blocks, cd: ConvDesc, idx, count, capacity, y, bias=None, residual=None, stream=None):
    yd = tensor_desc(y)
    st = lib().sige_scatter(_ptr(out_blocks), ctypes.byref(cd), _ptr(idx), _ptr(count), int(capacity),
                            _ptr(bias), _ptr(residual), _ptr(y), ctypes.byref(yd), _stream(stream))
    _check(st, "sige_scatter")
    return y


def sige_conv_fused(x, weight, bias, cd: ConvDesc, idx, count, capacity, y, gn_scale=None, gn_shift=None,
                    silu=False, residual=None, workspace=None, stream=None):
    xd, yd = tensor_desc(x), tensor_desc(y)
    if workspace is None:
        workspace = zeros_workspace(sige_conv_workspace_bytes(cd, x.shape[0], capacity, y.shape[1], y.shape[2]),
                                    x.device)
    st = lib().sige_conv_fused(_ptr(x), ctypes.byref(xd), _ptr(weight), _ptr(bias), ctypes.byref(cd), _ptr(idx),
                               _ptr(count), int(capacity), _ptr(gn_scale), _ptr(gn_shift), int(bool(silu)),
                               _ptr(residual), _ptr(y), ctypes.byref(yd), _ptr(workspace), workspace.numel(),
                               _stream(stream))
    _check(st, "sige_conv_fused")
    return y


def conv_out_hw(cd: ConvDesc, H: int, W: int, transposed=False, output_padding=0):
    if transposed:
        return ((H - 1) * cd.stride - 2 * cd.pad + cd.kernel + output_padding,
                (W - 1) * cd.stride - 2 * cd.pad + cd.kernel + output_padding)
    return (H + 2 * cd.pad - cd.kernel) // cd.stride + 1, (W + 2 * cd.pad - cd.kernel) // cd.stride + 1


def sige_conv_fused_ext(x, weight, bias, cd: ConvDesc, y=None, idx=None, count=None, capacity=0, gn_scale=None,
                        gn_shift=None, transposed=False, output_padding=0, spade_gamma=None, spade_beta=None,
                        act=ACT_NONE, residual=None, workspace=None, stream=None):
    """A GauGAN-style layer (transposed conv and / or SPADE-style modulated
    input) on the listed tiles of y, or on every tile when ``idx`` is None."""
    N, H, W, _ = x.shape
    Ho, Wo = conv_out_hw(cd, H, W, transposed, output_padding)
    if y is None:
        y = torch.empty((N, Ho, Wo, cd.c_out), dtype=x.dtype, device=x.device)
    xd, yd = tensor_desc(x), tensor_desc(y)
    if workspace is None:
        workspace = zeros_workspace(sige_conv_workspace_bytes(cd, N, max(capacity, 1), Ho, Wo), x.device)
    ext = LayerExt(int(bool(transposed)), int(output_padding), None if spade_gamma is None else spade_gamma.data_ptr(),
                   None if spade_beta is None else spade_beta.data_ptr(), int(act))
    st = lib().sige_conv_fused_ext(_ptr(x), ctypes.byref(xd), _ptr(weight), _ptr(bias), ctypes.byref(cd),
                                   ctypes.byref(ext), _ptr(idx), _ptr(count), int(capacity), _ptr(gn_scale),
                                   _ptr(gn_shift), _ptr(residual), _ptr(y), ctypes.byref(yd), _ptr(workspace),
                                   workspace.numel(), _stream(stream))
    _check(st, "sige_conv_fused_ext")
    return y


def sige_dense_conv(x, weight, bias, cd: ConvDesc, y=None, gn_scale=None, gn_shift=None, silu=False,
                    residual=None, workspace=None, stream=None):
    N, H, W, _ = x.shape
    Ho = (H + 2 * cd.pad - cd.kernel) // cd.stride + 1
    Wo = (W + 2 * cd.pad - cd.kernel) // cd.stride + 1
    if y is None:
        y = torch.empty((N, Ho, Wo, cd.c_out), dtype=x.dtype, device=x.device)
    xd, yd = tensor_desc(x), tensor_desc(y)
    if workspace is None:
        workspace = zeros_workspace(sige_conv_workspace_bytes(cd, N, 0, Ho, Wo), x.device)
    st = lib().sige_dense_conv(_ptr(x), ctypes.byref(xd), _ptr(weight), _ptr(bias), ctypes.byref(cd),
                               _ptr(gn_scale), _ptr(gn_shift), int(bool(silu)), _ptr(residual), _ptr(y),
                               ctypes.byref(yd), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "sige_dense_conv")
    return y


def sige_resblock_fused(x_edit, w1, b1, gn1, w2, b2, gn2, idx, count, capacity, y1, out, block=8,
                        workspace=None, stream=None):
    """The res block on the active tiles in one launch: y1 and out (the caches,
    NHWC bf16) are updated in place at the listed 8x8 tiles.  ``gn1`` / ``gn2``
    are (scale, shift) pairs from sige_groupnorm_affine; biases may be None."""
    xd = tensor_desc(x_edit)
    if workspace is None:
        workspace = zeros_workspace(WORKSPACE_HEADER, x_edit.device)
    st = lib().sige_resblock_fused(_ptr(x_edit), ctypes.byref(xd), _ptr(w1), _ptr(b1), _ptr(gn1[0]), _ptr(gn1[1]),
                                   _ptr(w2), _ptr(b2), _ptr(gn2[0]), _ptr(gn2[1]), int(block), _ptr(idx),
                                   _ptr(count), int(capacity), _ptr(y1), _ptr(out), _ptr(workspace),
                                   workspace.numel(), _stream(stream))
    _check(st, "sige_resblock_fused")
    return y1, out


def sige_resblock_step_workspace_bytes(x, block=8) -> int:
    xd = tensor_desc(x)
    return int(lib().sige_resblock_step_workspace_bytes(ctypes.byref(xd), int(block)))


def sige_resblock_step(x_orig, x_edit, threshold, w1, b1, gn1, w2, b2, gn2, y1, out, capacity, dilate=1, block=8,
                       idx=None, count=None, workspace=None, stream=None):
    """Mask, tile list and the fused res block in one launch.  Returns (idx,
    count) on the device; y1 and out are updated in place."""
    xd = tensor_desc(x_edit)
    dev = x_edit.device
    if idx is None:
        idx = torch.empty((max(int(capacity), 1), 2), dtype=torch.int32, device=dev)
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = zeros_workspace(sige_resblock_step_workspace_bytes(x_edit, block), dev)
    st = lib().sige_resblock_step(_ptr(x_orig), _ptr(x_edit), ctypes.byref(xd), float(threshold), int(dilate),
                                  _ptr(w1), _ptr(b1), _ptr(gn1[0]), _ptr(gn1[1]), _ptr(w2), _ptr(b2), _ptr(gn2[0]),
                                  _ptr(gn2[1]), int(block), _ptr(idx), _ptr(count), int(capacity), _ptr(y1),
                                  _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "sige_resblock_step")
    return idx, count


def sige_groupnorm_affine(x, groups, gamma, beta, eps=1e-5, scale=None, shift=None, stream=None):
    xd = tensor_desc(x)
    if scale is None:
        scale = torch.empty((x.shape[0], x.shape[3]), dtype=torch.float32, device=x.device)
    if shift is None:
        shift = torch.empty_like(scale)
    st = lib().sige_groupnorm_affine(_ptr(x), ctypes.byref(xd), int(groups), _ptr(gamma), _ptr(beta), float(eps),
                                     _ptr(scale), _ptr(shift), _stream(stream))
    _check(st, "sige_groupnorm_affine")
    return scale, shift


def sige_restore_tiles(src, dst, block, idx, count, capacity, stream=None):
    """dst[n, h0+i, w0+j, :] = src[n, h0+i, w0+j, :] for the listed tiles (in-image
    pixels, i, j < block); every other element of dst is left as it is."""
    if src.shape != dst.shape or src.dtype != dst.dtype:
        raise ValueError("src and dst must have the same shape and dtype")
    d = tensor_desc(dst)
    st = lib().sige_restore_tiles(_ptr(src), _ptr(dst), ctypes.byref(d), int(block), _ptr(idx), _ptr(count),
                                  int(capacity), _stream(stream))
    _check(st, "sige_restore_tiles")
    return dst


def sige_download_tiles_bytes(y, block, capacity) -> int:
    d = tensor_desc(y)
    return int(lib().sige_download_tiles_bytes(ctypes.byref(d), int(block), int(capacity)))


def sige_download_tiles(y, block, idx, count, capacity, host_y, staging=None, host_staging=None, stream=None):
    """host_y[n, h0+i, w0+j, :] = y[n, h0+i, w0+j, :] for the listed tiles of the
    device tensor y (in-image pixels, i, j < block); every other element of the
    host tensor host_y is left as it is.  Returns once host_y is complete."""
    if tuple(host_y.shape) != tuple(y.shape) or host_y.dtype != y.dtype or host_y.device.type != "cpu":
        raise ValueError("host_y must be a host tensor of y's shape and dtype")
    if not host_y.is_contiguous():
        raise ValueError("host_y must be contiguous")
    nbytes = sige_download_tiles_bytes(y, block, capacity)
    if staging is None:
        staging = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=y.device)
    if host_staging is None:
        host_staging = torch.empty(max(nbytes, 16), dtype=torch.uint8).pin_memory()
    if staging.numel() * staging.element_size() < nbytes or host_staging.numel() * host_staging.element_size() < nbytes:
        raise ValueError("staging buffers smaller than sige_download_tiles_bytes")
    d = tensor_desc(y)
    st = lib().sige_download_tiles(_ptr(y), ctypes.byref(d), int(block), _ptr(idx), _ptr(count), int(capacity),
                                   _ptr(staging), ctypes.c_void_p(host_staging.data_ptr()),
                                   ctypes.c_void_p(host_y.data_ptr()), _stream(stream))
    _check(st, "sige_download_tiles")
    return host_y


def sige_conv_workspace_bytes(cd: ConvDesc, batch: int, capacity: int, out_h: int, out_w: int) -> int:
    return int(lib().sige_conv_workspace_bytes(ctypes.byref(cd), int(batch), int(capacity), int(out_h), int(out_w)))


def sige_get_error(workspace, stream=None) -> int:
    return int(lib().sige_get_error(_ptr(workspace), _stream(stream)))


def sige_get_device_error(workspace, stream=None) -> int:
    return int(lib().sige_get_device_error(_ptr(workspace), _stream(stream)))


def sige_workspace_bytes(which_call: int, cd: ConvDesc | None, capacity: int) -> int:
    return int(lib().sige_workspace_bytes(int(which_call), None if cd is None else ctypes.byref(cd),
                                          int(capacity)))


def sige_set_wait_cycles(cycles: int) -> None:
    """Bound of the device waits that report SIGE_ERR_TIMEOUT (0: the kernels'
    own bounds), for launches enqueued from now on, process-wide."""
    _check(lib().sige_set_wait_cycles(int(cycles)), "sige_set_wait_cycles")


def sige_conv_path(cd: ConvDesc, dtype: torch.dtype) -> int:
    return int(lib().sige_conv_path(ctypes.byref(cd), _DT[dtype]))


def sige_attention_path(q, dv: int, heads: int) -> int:
    """Which kernel sige_attention_core runs for queries like ``q`` (an NHWC
    tensor), value width dv and this head count: 1 = tcgen05 tensor cores,
    0 = CUDA cores; negative = a sige_status."""
    qd = tensor_desc(q)
    return int(lib().sige_attention_path(ctypes.byref(qd), int(dv), int(heads)))


def sige_attention_core(q, k, v, heads: int, idx, count, capacity: int, block: int, o=None, stream=None):
    """Attention at the tokens under the tile list: q [N, H, W, D] bf16, k
    [N, Lk, D], v [N, Lk, Dv] (a [N, H, W, *] map is viewed as [N, H*W, *]),
    o [N, H, W, Dv] written at those tokens only (zeros elsewhere when
    allocated here)."""
    N, H, W, D = q.shape
    kk = k.reshape(N, -1, D)
    vv = v.reshape(N, kk.shape[1], -1)
    if o is None:
        o = torch.zeros((N, H, W, vv.shape[2]), dtype=q.dtype, device=q.device)
    qd = tensor_desc(q)
    st = lib().sige_attention_core(_ptr(q), ctypes.byref(qd), _ptr(kk), _ptr(vv), int(kk.shape[1]),
                                   int(vv.shape[2]), int(heads), _ptr(idx), _ptr(count), int(capacity), int(block),
                                   _ptr(o), _stream(stream))
    _check(st, "sige_attention_core")
    return o


def sige_attention_sparse(x, idx, count, capacity: int, block: int, wq, wo, bo, heads: int, k_map, v_map, y,
                          wk=None, wv=None, residual=None, workspace=None, stream=None):
    """One attention layer with pruned queries, in place into the cached output
    ``y`` [N, H, W, Co]: q = x Wq at the tokens under the tile list (sparse 1x1
    conv), the cached key / value maps ``k_map`` [N, H, W, D] / ``v_map``
    updated there from x when ``wk`` / ``wv`` are given (self-attention; a
    cross-attention caller passes the context's key / value sequences
    [N, Lc, *] and no ``wk`` / ``wv``), the attention step, and
    y = o Wo + bo (+ residual) at those tokens (sparse 1x1 conv).  Weights
    are 1x1 conv weights [c_out][1][1][c_in] (the transposed projection
    matrices).  With caches built from the original map and an edit confined to
    the listed tiles, the keys and values equal those of the whole edited map."""
    N, H, W, C = x.shape
    D, Dv, Co = wq.shape[0], v_map.shape[-1], wo.shape[0]
    cd_q = conv_desc(1, 1, 0, C, D, block)
    if workspace is None:
        need = max(sige_conv_workspace_bytes(conv_desc(1, 1, 0, ci, co, block), N, capacity, 0, 0)
                   for ci, co in ((C, D), (C, Dv), (Dv, Co)))
        workspace = zeros_workspace(need, x.device)
    q = torch.empty((N, H, W, D), dtype=x.dtype, device=x.device)
    sige_conv_fused(x, wq, None, cd_q, idx, count, capacity, q, workspace=workspace, stream=stream)
    if wk is not None:
        sige_conv_fused(x, wk, None, cd_q, idx, count, capacity, k_map, workspace=workspace, stream=stream)
    if wv is not None:
        sige_conv_fused(x, wv, None, conv_desc(1, 1, 0, C, Dv, block), idx, count, capacity, v_map,
                        workspace=workspace, stream=stream)
    o = torch.empty((N, H, W, Dv), dtype=x.dtype, device=x.device)
    sige_attention_core(q, k_map, v_map, heads, idx, count, capacity, block, o, stream)
    sige_conv_fused(o, wo, bo, conv_desc(1, 1, 0, Dv, Co, block), idx, count, capacity, y, residual=residual,
                    workspace=workspace, stream=stream)
    return y


# ------------------------------------------------------------------ quantised cache

_QFMT = {"s8": Q_S8, "e4m3": Q_E4M3, "s4": Q_S4}
_QSTORE = {"s8": torch.int8, "e4m3": torch.float8_e4m3fn, "s4": torch.uint8}


_INT32_MAX = 0x7FFFFFFF


def _too_large(what: str, *numbers):
    """The library's sizes are int32 (ctypes would drop the upper bits)."""
    return ValueError(f"{what}: a size of {max(numbers)} does not fit 32 bits")


class QCache:
    """A quantised NHWC map: ``codes`` [N, H, W, C] (int8 for "s8", float8_e4m3fn
    for "e4m3"; uint8 [N, H, W, C / 2] for "s4": two 4-bit codes a byte, the even
    channel in the low half) and ``scales`` float32 [N, H, W, C / group]; a
    code stands for code * scale.  A view of the two tensors: nothing is
    copied or kept."""
    __slots__ = ("codes", "scales", "format", "shape", "desc")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, format: str):
        fmt = _QFMT.get(format)
        if fmt is None:
            raise ValueError(f"unknown format {format!r}: one of {sorted(_QFMT)}")
        if codes.dtype is not _QSTORE[format] or scales.dtype is not torch.float32:
            raise ValueError(f"{format} codes are {_QSTORE[format]}, scales are torch.float32")
        if codes.dim() != 4 or scales.dim() != 4:
            raise ValueError("expected codes and scales [N, H, W, *] of one map")
        n, h, w, c = codes.shape
        sn, sh, sw, ng = scales.shape
        if n != sn or h != sh or w != sw:
            raise ValueError("expected codes and scales [N, H, W, *] of one map")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("expected contiguous codes and scales")
        if fmt == Q_S4:
            c *= 2
        if ng < 1 or c % ng:
            raise ValueError(f"{ng} scales a pixel do not divide {c} channels")
        if n | h | w | c > _INT32_MAX:
            raise _too_large("QCache", n, h, w, c)
        self.codes, self.scales, self.format, self.shape = codes, scales, format, (n, h, w, c)
        self.desc = QCacheDesc(n, h, w, c, fmt, c // ng)

    @property
    def group(self) -> int:
        return self.desc.group


def qcache_empty(n: int, h: int, w: int, c: int, format: str = "s8", group: int | None = None,
                 device="cuda") -> QCache:
    """An uninitialised cache of that map (``group`` None: one scale a pixel)."""
    group = c if group is None else group
    if group < 1 or c % group or (format == "s4" and group % 2):
        raise ValueError(f"a group of {group} does not fit {c} channels of {format}")
    codes = torch.empty((n, h, w, c // 2 if format == "s4" else c), dtype=_QSTORE[format], device=device)
    return QCache(codes, torch.empty((n, h, w, c // group), dtype=torch.float32, device=device), format)


def sige_qcache_code_bytes(cd: QCacheDesc) -> int:
    return int(lib().sige_qcache_code_bytes(ctypes.byref(cd)))


def sige_qcache_scales(cd: QCacheDesc) -> int:
    return int(lib().sige_qcache_scales(ctypes.byref(cd)))


def _device_index(what: str, *tensors) -> int:
    """Index of the CUDA device that all the given tensors (None: left out) are on."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError(f"{what}: expected tensors on a CUDA device")
                if dev is not None:
                    raise ValueError(f"{what}: tensors on different devices (cuda:{dev} and cuda:{d})")
                dev = d
    return dev


class _Launch:
    """Makes device ``dev`` and ``stream`` (None: that device's current stream)
    current for a call and gives the stream's handle: the library launches on
    the current device, and a workspace or an output allocated meanwhile
    belongs to that stream.  An argument that was allocated on another stream is
    the caller's to keep until the call has run, as under torch.cuda.stream."""
    __slots__ = ("ctx", "dev", "stream")

    def __init__(self, dev: int, stream):
        self.dev, self.stream, self.ctx = dev, stream, None

    def __enter__(self):
        st = self.stream
        if st is None:
            if self.dev != torch._C._cuda_getDevice():
                self.ctx = torch.cuda.device(self.dev)
                self.ctx.__enter__()
            return torch._C._cuda_getCurrentRawStream(self.dev)
        if not isinstance(st, torch.cuda.Stream):
            st = torch.cuda.ExternalStream(int(st), device=self.dev)
        if st.device.index != self.dev:
            raise ValueError(f"the stream is on {st.device}, the tensors on cuda:{self.dev}")
        self.ctx = torch.cuda.stream(st)
        self.ctx.__enter__()
        return st.cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _addr(t):
    return None if t is None else t.data_ptr()


def _map_desc(what: str, t, shape) -> TensorDesc:
    """Descriptor of a contiguous NHWC map of that shape."""
    if t.shape != shape:
        raise ValueError(f"{what}: a map of shape {tuple(t.shape)} does not fit, {tuple(shape)} is expected")
    if not t.is_contiguous() or t.dtype not in _DT:
        raise ValueError(f"{what}: expected a contiguous bf16 or float32 map")
    n, h, w, c = shape
    if n | h | w | c > _INT32_MAX:
        raise _too_large(what, *shape)
    return TensorDesc(n, h, w, c, _DT[t.dtype], NHWC)


def _f32(what: str, t, shape):
    if t is not None and (t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{what}: expected a contiguous float32 tensor of shape {tuple(shape)}")


def _tile_args(what: str, idx, count, capacity, block):
    """(block, idx, count, capacity) of the C call; idx None: every pixel."""
    if idx is None:
        return 1, None, None, 0
    if count is None or idx.dtype != torch.int32 or count.dtype != torch.int32 or not idx.is_contiguous() or \
            count.numel() < 1:
        raise ValueError(f"{what}: the tile list is a contiguous int32 [capacity, 2] with an int32 count")
    if capacity > 0 and idx.numel() < 2 * capacity:
        raise ValueError(f"{what}: the list holds {idx.numel() // 2} tiles, fewer than its capacity {capacity}")
    if block > _INT32_MAX or capacity > _INT32_MAX:
        raise _too_large(what, block, capacity)
    # (a tensor without elements has no address, and a list of no address is every
    # pixel to the library: any other stands for it, nothing is read there)
    return block, idx.data_ptr() or 8, count.data_ptr(), capacity


def sige_qcache_write(x, cache: QCache, idx=None, count=None, capacity=0, block=1, gn_scale=None, gn_shift=None,
                      silu=False, stream=None) -> QCache:
    """Quantise the NHWC map ``x`` (bf16 or float32) into ``cache``, in place, at
    the pixels under the tile list or, with ``idx`` None, at every pixel."""
    what = "sige_qcache_write"
    xd = _map_desc(what, x, cache.shape)
    if gn_scale is not None or gn_shift is not None:
        _f32(what + ": gn_scale", gn_scale, (xd.n, xd.c))
        _f32(what + ": gn_shift", gn_shift, (xd.n, xd.c))
    b, i, c, cap = _tile_args(what, idx, count, capacity, block)
    dev = _device_index(what, x, cache.codes, cache.scales, idx, count, gn_scale, gn_shift)
    with _Launch(dev, stream) as st:
        _check(lib().sige_qcache_write(x.data_ptr(), xd, _addr(gn_scale), _addr(gn_shift),
                                       1 if silu else 0, b, i, c, cap, cache.codes.data_ptr(), cache.scales.data_ptr(),
                                       cache.desc, st), what)
    return cache


def sige_qcache_read(cache: QCache, y=None, idx=None, count=None, capacity=0, block=1, dtype=torch.bfloat16,
                     stream=None) -> torch.Tensor:
    """What the cache stands for, into ``y`` [N, H, W, C] (bf16 or float32) at the
    pixels under the tile list or at every pixel; other pixels keep their bytes
    (zeros where ``y`` is allocated here, as ``dtype``)."""
    what = "sige_qcache_read"
    b, i, c, cap = _tile_args(what, idx, count, capacity, block)
    dev = _device_index(what, cache.codes, cache.scales, y, idx, count)
    with _Launch(dev, stream) as st:
        if y is None:
            y = (torch.empty if idx is None else torch.zeros)(cache.shape, dtype=dtype, device=cache.codes.device)
        yd = _map_desc(what, y, cache.shape)
        _check(lib().sige_qcache_read(cache.codes.data_ptr(), cache.scales.data_ptr(), cache.desc, b, i, c,
                                      cap, y.data_ptr(), yd, st), what)
    return y


def sige_qlinear(a: QCache, w: QCache, bias=None, y=None, idx=None, count=None, capacity=0, block=1, residual=None,
                 dtype=torch.bfloat16, workspace=None, stream=None) -> torch.Tensor:
    """y = a w^T (8-bit integers, one scale per token and per output channel)
    + bias + residual at the tokens under the tile list or at every token.
    ``a``: an "s8" cache [N, H, W, C] with one scale a pixel; ``w``: an "s8"
    cache [C_out, 1, 1, C] with one scale a row."""
    what = "sige_qlinear"
    n, h, wd, _ = a.shape
    shape = (n, h, wd, w.shape[0])
    _f32("sige_qlinear: bias", bias, (shape[3],))
    b, i, c, cap = _tile_args(what, idx, count, capacity, block)
    dev = _device_index(what, a.codes, a.scales, w.codes, w.scales, bias, y, idx, count, residual, workspace)
    with _Launch(dev, stream) as st:
        if y is None:
            y = (torch.empty if idx is None else torch.zeros)(shape, dtype=dtype, device=a.codes.device)
        if residual is not None and (residual.shape != y.shape or residual.dtype != y.dtype or
                                     not residual.is_contiguous()):
            raise ValueError("sige_qlinear: the residual is a contiguous tensor of y's shape and dtype")
        yd = _map_desc(what, y, shape)
        if workspace is None:
            workspace = zeros_workspace(WORKSPACE_HEADER, a.codes.device)
        _check(lib().sige_qlinear(a.codes.data_ptr(), a.scales.data_ptr(), a.desc, w.codes.data_ptr(),
                                  w.scales.data_ptr(), w.desc, _addr(bias), b, i, c, cap, _addr(residual),
                                  y.data_ptr(), yd, workspace.data_ptr(), workspace.nbytes, st), what)
    return y


def sige_qlinear_path(c: int) -> int:
    return int(lib().sige_qlinear_path(int(c)))


def sige_attention_qcache(q, k: QCache, v: QCache, heads: int, o=None, idx=None, count=None, capacity=0, block=1,
                          key_counts=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of the tokens of ``q`` [N, H, W, D] (bf16) under the tile list,
    or of every token, over the key and value caches ``k`` [N, h, w, D] and
    ``v`` [N, h, w, Dv] (h * w keys; a context sequence is [N, keys, 1, *]),
    into ``o`` [N, H, W, Dv].  ``key_counts``: int32 [N], the valid keys of each
    item (0: its tokens get zeros)."""
    what = "sige_attention_qcache"
    if key_counts is not None and (key_counts.dtype != torch.int32 or key_counts.numel() != q.shape[0] or
                                   not key_counts.is_contiguous()):
        raise ValueError("sige_attention_qcache: key_counts is a contiguous int32 tensor of one count per item")
    qs = q.shape
    if len(qs) != 4 or q.dtype != torch.bfloat16:
        raise ValueError("sige_attention_qcache: q is a bf16 map [N, H, W, D]")
    qd = _map_desc(what, q, qs)
    if heads > _INT32_MAX:
        raise _too_large(what, heads)
    shape = (qs[0], qs[1], qs[2], v.shape[3])
    if o is not None and (o.shape != shape or o.dtype != torch.bfloat16 or not o.is_contiguous()):
        raise ValueError(f"sige_attention_qcache: o is a contiguous bf16 tensor of shape {shape}")
    b, i, c, cap = _tile_args(what, idx, count, capacity, block)
    dev = _device_index(what, q, k.codes, k.scales, v.codes, v.scales, o, idx, count, key_counts, workspace)
    with _Launch(dev, stream) as st:
        if o is None:
            o = (torch.empty if idx is None else torch.zeros)(shape, dtype=torch.bfloat16, device=q.device)
        if workspace is None:
            workspace = zeros_workspace(WORKSPACE_HEADER, q.device)
        _check(lib().sige_attention_qcache(q.data_ptr(), qd, k.codes.data_ptr(), k.scales.data_ptr(),
                                           k.desc, v.codes.data_ptr(), v.scales.data_ptr(),
                                           v.desc, _addr(key_counts), heads, b, i, c, cap, o.data_ptr(),
                                           workspace.data_ptr(), workspace.nbytes, st), what)
    return o


def sige_attention_qcache_path(dh: int, dvh: int) -> int:
    return int(lib().sige_attention_qcache_path(int(dh), int(dvh)))


def _range(t):
    a = t.data_ptr()
    return a, a + t.numel() * t.element_size()


def _overlap(a, b) -> bool:
    return a[0] < b[1] and b[0] < a[1]


def _check_sparse_q(what, x, idx, count, wq, wo, bo, heads, k_map, v_map, y, wk, wv, residual, key_counts, workspace):
    """Everything that a step of sige_attention_sparse_q would refuse, before the
    first step: once the caches are updated there is no way back.  Descriptors of
    x and y, and the device's index."""
    xd = _map_desc(what, x, x.shape)
    N, H, W, C = x.shape
    ks, vs, rows = k_map.shape, v_map.shape, wo.shape[0]
    D, Dv = ks[3], vs[3]
    for name, w, r, c in (("wq", wq, D, C), ("wk", wk, D, C), ("wv", wv, Dv, C), ("wo", wo, rows, Dv)):
        if w is not None and (w.format != "s8" or w.shape != (r, 1, 1, c) or w.desc.group != c or c > 131071):
            raise ValueError(f'{what}: {name} is an "s8" cache [{r}, 1, 1, {c}] with one scale a row')
    if ks[0] != N or vs[0] != N or ks[1] * ks[2] != vs[1] * vs[2] or (wk is not None and ks[:3] != (N, H, W)) or \
            (wv is not None and vs[:3] != (N, H, W)):
        raise ValueError(f"{what}: keys {ks} and values {vs} do not fit a map {(N, H, W, C)}")
    if heads < 1 or D % heads or Dv % heads:
        raise ValueError(f"{what}: {heads} heads do not divide {D} and {Dv} channels")
    dh, dvh, kg, vg = D // heads, Dv // heads, k_map.desc.group, v_map.desc.group
    if kg % dh or vg % dvh or dh > 256 or dvh > 256:
        raise ValueError(f"{what}: heads of {dh} and {dvh} channels, scales of {kg} and {vg}: a scale covers whole heads of up to "
                         "256 channels")
    if key_counts is not None and (key_counts.dtype != torch.int32 or key_counts.numel() != N or not key_counts.is_contiguous()):
        raise ValueError(f"{what}: key_counts is a contiguous int32 tensor of one count per item")
    yd = _map_desc(what, y, (N, H, W, rows))
    _f32(what, bo, (rows,))
    if residual is not None and (residual.dtype != y.dtype or residual.shape != y.shape or not residual.is_contiguous()):
        raise ValueError(f"{what}: the residual is a contiguous tensor of y's shape and dtype")
    at = _range(y)
    for t in (wo.codes, wo.scales, bo, residual, workspace, idx, count):
        if t is not None and _overlap(at, _range(t)):
            raise ValueError(f"{what}: y shares memory with an operand")
    if wk is not None or wv is not None:
        kv = sorted(_range(t) for t in (k_map.codes, k_map.scales, v_map.codes, v_map.scales))
        if any(_overlap(a, b) for a, b in zip(kv, kv[1:])):
            raise ValueError(f"{what}: the key and value caches share memory")
    if workspace is not None and (workspace.nbytes < WORKSPACE_HEADER or workspace.data_ptr() % 16):
        raise ValueError(f"{what}: a workspace of {WORKSPACE_HEADER} bytes, 16-byte aligned, is expected")
    tensors = [x, y, idx, count, bo, residual, key_counts, workspace]
    for c in (wq, wk, wv, wo, k_map, v_map):
        if c is not None:
            tensors += (c.codes, c.scales)
    return xd, yd, _device_index(what, *tensors)


def sige_attention_sparse_q(x, idx, count, capacity: int, block: int, wq: QCache, wo: QCache, bo, heads: int,
                            k_map: QCache, v_map: QCache, y, wk: QCache | None = None, wv: QCache | None = None,
                            residual=None, key_counts=None, workspace=None, stream=None):
    """sige_attention_sparse with everything it keeps in codes: the tokens under
    the tile list of ``x`` [N, H, W, C] are quantised (one scale a token), the
    projections run in 8-bit integers (weights: "s8" caches [c_out, 1, 1, c_in]),
    the key and value caches ``k_map`` / ``v_map`` (any format) are updated at
    those tokens when ``wk`` / ``wv`` are given (self-attention; else they are
    the context's), and y = o Wo + bo (+ residual) at those tokens of the
    cached output ``y``.  Queries, keys, values and the step's output are rounded
    to bf16 between the calls, as in sige_attention_sparse.  A call that is
    refused leaves caches and output as they were."""
    what = "sige_attention_sparse_q"
    tiles = _tile_args(what, idx, count, capacity, block)
    xd, yd, index = _check_sparse_q(what, x, idx, count, wq, wo, bo, heads, k_map, v_map, y, wk, wv, residual, key_counts,
                                    workspace)
    L, dev = lib(), x.device
    n, h, w = xd.n, xd.h, xd.w
    D, Dv = k_map.shape[3], v_map.shape[3]

    def bf16(c):
        return torch.empty((n, h, w, c), dtype=torch.bfloat16, device=dev), TensorDesc(n, h, w, c, BF16, NHWC)

    def write(t, td, cache):
        _check(L.sige_qcache_write(t.data_ptr(), td, None, None, 0, *tiles, cache.codes.data_ptr(), cache.scales.data_ptr(), cache.desc,
                                   st), what)
        return cache

    def linear(a, wt, bias, res, out, od):
        _check(L.sige_qlinear(a.codes.data_ptr(), a.scales.data_ptr(), a.desc, wt.codes.data_ptr(), wt.scales.data_ptr(), wt.desc,
                              _addr(bias), *tiles, _addr(res), out.data_ptr(), od, workspace.data_ptr(), workspace.nbytes, st), what)

    with _Launch(index, stream) as st:
        if workspace is None:
            workspace = zeros_workspace(WORKSPACE_HEADER, dev)
        xq = write(x, xd, qcache_empty(n, h, w, xd.c, device=dev))
        q, qd = bf16(D)
        linear(xq, wq, None, None, q, qd)
        for wt, cache in ((wk, k_map), (wv, v_map)):
            if wt is not None:
                t, td = bf16(cache.shape[3])
                linear(xq, wt, None, None, t, td)
                write(t, td, cache)
        o, od = bf16(Dv)
        _check(L.sige_attention_qcache(q.data_ptr(), qd, k_map.codes.data_ptr(), k_map.scales.data_ptr(), k_map.desc,
                                       v_map.codes.data_ptr(), v_map.scales.data_ptr(), v_map.desc, _addr(key_counts), heads,
                                       *tiles, o.data_ptr(), workspace.data_ptr(), workspace.nbytes, st), what)
        linear(write(o, od, qcache_empty(n, h, w, Dv, device=dev)), wo, bo, residual, y, yd)
    return y


SCHEDULE_FIELDS = ("layout", "T", "tile_groups", "splits", "units", "split_sum", "unit_cols", "weight_stages",
                   "halo_bytes", "reduce_scatter_bytes", "cout_tiles", "k_chunks", "cluster_for_sparse",
                   "halo_offset", "smem_bytes")


def sige_conv_schedule(cd: ConvDesc, tiles: int, grid: int, cluster: int) -> dict:
    """Work decomposition of the tensor-core conv for ``tiles`` active tiles
    (times batch) on a launch of ``grid`` CTAs in clusters of ``cluster``;
    host-only.  Keys are SCHEDULE_FIELDS."""
    out = (ctypes.c_int32 * len(SCHEDULE_FIELDS))()
    _check(lib().sige_conv_schedule(ctypes.byref(cd), int(tiles), int(grid), int(cluster),
                                    ctypes.cast(out, ctypes.c_void_p), len(SCHEDULE_FIELDS)), "sige_conv_schedule")
    return dict(zip(SCHEDULE_FIELDS, (int(v) for v in out)))


def sige_launch_count() -> int:
    return int(lib().sige_launch_count())
