"""ctypes binding over libwhtq.so (C ABI in include/whtq.h).

Argument marshalling only: tensors are checked for device, dtype, layout and
shape, their pointers and the current HIP stream are handed to the library,
and every step of the computation runs in the library's HIP kernels.  There
is no CPU fallback: importing this module fails if the library is missing.
"""
import ctypes
import dataclasses
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.environ.get("WHTQ_LIB", os.path.join(_HERE, "libwhtq.so"))

if not os.path.exists(lib_path):
    raise ImportError(
        f"libwhtq.so not found at {lib_path}; build it with `python -m wht_adapters_amd.build`")
_lib = ctypes.CDLL(lib_path)

_i64, _int, _vp, _f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float


class _Cache(ctypes.Structure):  # whtq_kv_cache
    _fields_ = [("k", _vp), ("v", _vp), ("k_scales", _vp), ("v_scales", _vp), ("sign_bits", _vp),
                ("num_pages", _i64), ("page_size", _i64), ("kv_heads", _i64), ("dim", _i64),
                ("k_stride", _i64 * 3), ("v_stride", _i64 * 3), ("ks_stride", _i64 * 2), ("vs_stride", _i64 * 2),
                ("format", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class _Rope(ctypes.Structure):  # whtq_rope
    _fields_ = [("cos", _vp), ("sin", _vp), ("positions", _vp), ("ld", _i64), ("max_position", _i64),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class _Norm(ctypes.Structure):  # whtq_qk_norm
    _fields_ = [("q", _vp), ("k", _vp), ("q_head", _i64), ("k_head", _i64), ("dtype", ctypes.c_int32), ("eps", _f32)]


_cache_p, _rope_p, _i64_p = ctypes.POINTER(_Cache), ctypes.POINTER(_Rope), ctypes.POINTER(_i64)
_norm_p = ctypes.POINTER(_Norm)

_SIG = {
    "wht_batched": [_vp, _int, _vp, _int, _i64, _i64, _i64, _i64, _vp, _int, _int, _vp],
    "rht_quantize_rtn": [_vp, _int, _i64, _i64, _i64, _vp, _int, _int, _vp, _vp, _vp],
    "rht_dequantize_inverse": [_vp, _vp, _i64, _i64, _vp, _int, _int, _vp, _int, _i64, _vp],
    "qwha_adapter_forward": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _i64, _i64, _vp, _int,
                             _i64, _vp],
    "harp_rotate": [_vp, _vp, _int, _i64, _i64, _i64, _i64, _vp, _int, _vp, _int, _vp, _int, _vp],
    "qwha_csr_transpose": [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp],
    "harp_build_blocks": [_vp, _int, _vp, _i64, _vp, _int, _vp, _vp, _int, _vp],
    "qwha_permute_values": [_vp, _int, _vp, _i64, _vp, _vp],
    "qwha_adapter_backward_input": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _i64, _i64, _vp, _int,
                                    _i64, _vp],
    "qwha_adapter_grad_values": [_vp, _vp, _int, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64,
                                 _vp],
    "rht_lowbit_gemv": [_vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _int, _int, _vp, _i64, _vp],
    "qwha_init_error_coeffs": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _int, _vp, _i64, _vp],
    "qwha_init_gram": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _int, _vp],
    "qwha_init_channel_errors": [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp],
    "qwha_init_allocate": [_vp, _i64, _i64, _i64, _int, _int, _vp],
    "qwha_init_select": [_vp, _i64, _i64, _i64, _vp, _vp, _vp],
    "qwha_init_refine": [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp],
    "whtq_stream_probe": [_vp, _i64, _vp, _i64, _vp],
    "qwha_adapter_grad_values_noalloc": [_vp, _vp, _int, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp,
                                         _vp],
    "qwha_forward_plan": [_i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp],
    "qwha_adapter_forward_planned": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _i64, _i64, _vp, _i64,
                                     _vp, _int, _i64, _vp],
    "kv_append": [_cache_p, _vp, _i64_p, _vp, _i64_p, _int, _i64, _vp, _rope_p, _vp, _i64_p, _i64, _vp, _i64_p, _vp],
    "kv_attention_sinks": [_cache_p, _vp, _i64_p, _int, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _f32,
                           _int, _i64, _i64, _vp, _i64_p, _vp, _vp, _i64, _vp],
    "kv_append_norm": [_cache_p, _vp, _i64_p, _vp, _i64_p, _int, _i64, _vp, _norm_p, _rope_p, _vp, _i64_p, _i64, _vp,
                       _i64_p, _vp],
    "qk_norm_rope": [_vp, _i64_p, _i64, _vp, _i64_p, _i64, _int, _i64, _i64, _norm_p, _rope_p, _vp, _i64_p, _vp, _i64_p,
                     _vp],
    "qk_norm_rope_backward": [_vp, _i64_p, _vp, _i64_p, _i64, _vp, _i64_p, _vp, _i64_p, _i64, _int, _i64, _i64, _norm_p,
                              _rope_p, _vp, _i64_p, _vp, _i64_p, _vp, _vp, _vp, _i64, _vp],
    "token_logprobs": [_vp, _int, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _vp],
    "token_logprobs_backward": [_vp, _int, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp],
    "kv_gather": [_cache_p, _i64, _vp, _vp, _i64_p, _vp, _i64_p, _int, _vp],
    "kv_attention": [_cache_p, _vp, _i64_p, _int, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _f32,
                     _int, _i64, _vp, _i64_p, _vp, _vp, _i64, _vp],
}
for _name, _args in _SIG.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _int
_lib.qwha_grad_values_workspace_bytes.argtypes = [_i64, _i64, _i64]
_lib.qwha_grad_values_workspace_bytes.restype = _i64
_lib.qwha_forward_plan_bytes.argtypes = [_i64, _i64, _i64, _i64]
_lib.qwha_forward_plan_bytes.restype = _i64
_lib.kv_attention_workspace_bytes.argtypes = [_cache_p, _i64, _i64, _i64, _i64, _i64, _i64]
_lib.kv_attention_workspace_bytes.restype = _i64
_lib.kv_attention_sinks_workspace_bytes.argtypes = [_cache_p, _i64, _i64, _i64, _i64, _i64, _i64, _i64]
_lib.kv_attention_sinks_workspace_bytes.restype = _i64
_lib.qk_norm_rope_backward_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _norm_p]
_lib.qk_norm_rope_backward_workspace_bytes.restype = _i64
_lib.token_logprobs_workspace_bytes.argtypes = [_i64, _i64, _i64]
_lib.token_logprobs_workspace_bytes.restype = _i64
_lib.whtq_status_string.argtypes = [_int]
_lib.whtq_status_string.restype = ctypes.c_char_p
_lib.whtq_last_hip_error.restype = _int
_lib.whtq_abi_version.restype = _int

F32, BF16, F16, I8 = 0, 1, 2, 3
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16, torch.int8: I8}
SIGN_NONE, SIGN_BEFORE, SIGN_AFTER = 0, 1, 2
_SIGN_MODES = {"none": SIGN_NONE, "before": SIGN_BEFORE, "after": SIGN_AFTER}


class WhtqError(RuntimeError):
    def __init__(self, fn, status):
        msg = _lib.whtq_status_string(status).decode()
        if status == 4:
            msg += f" (hipError {_lib.whtq_last_hip_error()})"
        super().__init__(f"{fn}: {msg} [status {status}]")
        self.status = status


def abi_version():
    return _lib.whtq_abi_version()


def raw():
    """The ctypes library handle (for callers that marshal pointers themselves)."""
    return _lib


def _check(fn, status):
    if status != 0:
        raise WhtqError(fn, status)


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need_cuda(name, t):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")


def _rows_ld(name, t):
    """(rows, n, ld) of a 2-D tensor with unit stride along the last dim."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with a contiguous last dimension")
    rows, n = t.shape
    # a single row's stride is meaningless (torch may report 0 or 1 for it)
    return rows, n, (t.stride(0) if rows > 1 else n)


def _sign_ptr(signs, n, device):
    if signs is None:
        return ctypes.c_void_p(0)
    _need_cuda("signs", signs)
    if signs.dtype not in (torch.int32, torch.uint32) or signs.numel() * 32 < n or not signs.is_contiguous():
        raise ValueError("signs must be a contiguous int32/uint32 bitmask of ceil(n/32) words")
    if signs.device != device:
        raise ValueError("signs must be on the same device")
    return _ptr(signs)


def wht_batched(x, out=None, *, signs=None, sign_mode="none", normalize=True, out_dtype=None):
    """y = Hn(S x) ('before'), Hn x ('none') or S Hn x ('after') along the last dim."""
    _need_cuda("x", x)
    rows, n, ldx = _rows_ld("x", x)
    if out is None:
        out = torch.empty((rows, n), dtype=out_dtype or x.dtype, device=x.device)
    _need_cuda("out", out)
    r2, n2, ldy = _rows_ld("out", out)
    if (r2, n2) != (rows, n):
        raise ValueError("out shape mismatch")
    mode = _SIGN_MODES[sign_mode]
    with torch.cuda.device(x.device):
        _check("wht_batched", _lib.wht_batched(
            _ptr(x), _DT[x.dtype], _ptr(out), _DT[out.dtype], rows, n, ldx, ldy,
            _sign_ptr(signs, n, x.device), mode, int(bool(normalize)), _stream(x)))
    return out


def rht_quantize_rtn(w, signs, bits, group, codes=None, scales=None):
    """Returns (codes uint8 [rows, n*bits/8], scales float16 [rows, n/group])."""
    _need_cuda("w", w)
    rows, n, ldw = _rows_ld("w", w)
    if codes is None:
        codes = torch.empty((rows, n * bits // 8), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty((rows, max(1, n // group)), dtype=torch.float16, device=w.device)
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    with torch.cuda.device(w.device):
        _check("rht_quantize_rtn", _lib.rht_quantize_rtn(
            _ptr(w), _DT[w.dtype], rows, n, ldw, _sign_ptr(signs, n, w.device), bits, group,
            _ptr(codes), _ptr(scales), _stream(w)))
    return codes, scales


def rht_dequantize_inverse(codes, scales, signs, bits, group, n, out=None, out_dtype=torch.bfloat16):
    """out = S Hn (q * s) for codes/scales written by rht_quantize_rtn."""
    _need_cuda("codes", codes)
    rows = codes.shape[0]
    if codes.dtype != torch.uint8 or scales.dtype != torch.float16:
        raise ValueError("codes must be uint8 and scales float16")
    if codes.shape != (rows, n * bits // 8) or scales.shape != (rows, n // group):
        raise ValueError("codes / scales shape mismatch")
    if out is None:
        out = torch.empty((rows, n), dtype=out_dtype, device=codes.device)
    r2, n2, ldo = _rows_ld("out", out)
    if (r2, n2) != (rows, n):
        raise ValueError("out shape mismatch")
    with torch.cuda.device(codes.device):
        _check("rht_dequantize_inverse", _lib.rht_dequantize_inverse(
            _ptr(codes), _ptr(scales), rows, n, _sign_ptr(signs, n, codes.device), bits, group,
            _ptr(out), _DT[out.dtype], ldo, _stream(codes)))
    return out


def rht_lowbit_gemv(x, codes, scales, signs, bits, group, out=None):
    """y = x W_hat^T for W_hat the rows rht_dequantize_inverse would decode from
    (codes, scales); x [tokens, n] bf16, y [tokens, rows] bf16."""
    _need_cuda("x", x)
    tokens, n, ldx = _rows_ld("x", x)
    rows = codes.shape[0]
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16")
    if codes.dtype != torch.uint8 or scales.dtype != torch.float16:
        raise ValueError("codes must be uint8 and scales float16")
    if codes.shape != (rows, n * bits // 8) or scales.shape != (rows, n // group):
        raise ValueError("codes / scales shape mismatch")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    if codes.device != x.device or scales.device != x.device:
        raise ValueError("x, codes and scales must be on one device")
    if out is None:
        out = torch.empty((tokens, rows), dtype=torch.bfloat16, device=x.device)
    _need_cuda("out", out)
    t2, r2, ldy = _rows_ld("out", out)
    if (t2, r2) != (tokens, rows) or out.dtype != torch.bfloat16:
        raise ValueError("out must be bfloat16 [tokens, rows]")
    with torch.cuda.device(x.device):
        _check("rht_lowbit_gemv", _lib.rht_lowbit_gemv(
            _ptr(x), tokens, ldx, _ptr(codes), _ptr(scales), rows, n, _sign_ptr(signs, n, x.device),
            bits, group, _ptr(out), ldy, _stream(x)))
    return out


def qwha_forward_plan(tokens, d_in, row_ptr, d_out, nnz, out=None):
    """The forward's per-chunk bookkeeping for a fixed support (row_ptr), as
    a uint8 device tensor to pass as `plan` to qwha_adapter_forward (built on
    row_ptr's stream; valid for this token count and device).  `out`: a
    contiguous uint8 buffer of at least qwha_forward_plan_bytes to reuse."""
    _need_cuda("row_ptr", row_ptr)
    if row_ptr.dtype != torch.int32 or not row_ptr.is_contiguous() or row_ptr.numel() != d_out + 1:
        raise ValueError("row_ptr must be contiguous int32 with d_out + 1 entries")
    with torch.cuda.device(row_ptr.device):
        nb = _lib.qwha_forward_plan_bytes(tokens, d_in, d_out, nnz)
        if nb < 0:
            raise ValueError("invalid sizes for a forward plan")
        if out is None:
            plan = torch.empty(max(int(nb), 256), dtype=torch.uint8, device=row_ptr.device)
        else:
            _need_cuda("out", out)
            if out.dtype != torch.uint8 or not out.is_contiguous() or out.numel() < nb:
                raise ValueError("out must be a contiguous uint8 buffer of qwha_forward_plan_bytes or more")
            plan = out
        _check("qwha_forward_plan", _lib.qwha_forward_plan(
            tokens, d_in, _ptr(row_ptr), d_out, nnz, _ptr(plan), plan.numel(), _stream(row_ptr)))
    return plan


def qwha_adapter_forward(x, row_ptr, col_idx, vals, d_out, out=None, plan=None):
    """y = (x Hn) F^T with F [d_out x d_in] in CSR (int32 row_ptr / col_idx);
    `plan` from qwha_forward_plan skips the per-chunk bookkeeping."""
    _need_cuda("x", x)
    tokens, d_in, ldx = _rows_ld("x", x)
    for nm, t in (("row_ptr", row_ptr), ("col_idx", col_idx), ("vals", vals)):
        _need_cuda(nm, t)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    if row_ptr.dtype != torch.int32 or col_idx.dtype != torch.int32:
        raise ValueError("row_ptr and col_idx must be int32")
    if row_ptr.numel() != d_out + 1:
        raise ValueError("row_ptr must have d_out + 1 entries")
    nnz = col_idx.numel()
    if vals.numel() != nnz:
        raise ValueError("vals and col_idx must have the same length")
    if out is None:
        # rows of 16 bytes or more need a 16-byte row stride: pad the storage to a multiple of 8
        width = d_out if d_out < 8 else -(-d_out // 8) * 8
        out = torch.empty((tokens, width), dtype=x.dtype, device=x.device)[:, :d_out]
    r2, n2, ldy = _rows_ld("out", out)
    if (r2, n2) != (tokens, d_out):
        raise ValueError("out shape mismatch")
    with torch.cuda.device(x.device):
        if plan is None:
            _check("qwha_adapter_forward", _lib.qwha_adapter_forward(
                _ptr(x), _DT[x.dtype], tokens, d_in, ldx, _ptr(row_ptr), _ptr(col_idx), _ptr(vals),
                _DT[vals.dtype], d_out, nnz, _ptr(out), _DT[out.dtype], ldy, _stream(x)))
        else:
            _need_cuda("plan", plan)
            if plan.dtype != torch.uint8 or not plan.is_contiguous():
                raise ValueError("plan must be a contiguous uint8 tensor from qwha_forward_plan")
            _check("qwha_adapter_forward_planned", _lib.qwha_adapter_forward_planned(
                _ptr(x), _DT[x.dtype], tokens, d_in, ldx, _ptr(row_ptr), _ptr(col_idx), _ptr(vals),
                _DT[vals.dtype], d_out, nnz, _ptr(plan), plan.numel(), _ptr(out), _DT[out.dtype], ldy,
                _stream(x)))
    return out


def harp_rotate(x, blocks, radices=(16, 16, 16), signs=None, precondition=True, out=None):
    """y = stages(Hn S x) (precondition) or stages(x); blocks float32 or float16, stage-major."""
    _need_cuda("x", x)
    _need_cuda("blocks", blocks)
    tokens, d, ldx = _rows_ld("x", x)
    if blocks.dtype not in (torch.float32, torch.float16) or not blocks.is_contiguous():
        raise ValueError("blocks must be contiguous float32 or float16")
    rad = (ctypes.c_int32 * len(radices))(*[int(b) for b in radices])
    if out is None:
        out = torch.empty_like(x)
    r2, d2, ldy = _rows_ld("out", out)
    if (r2, d2) != (tokens, d) or out.dtype != x.dtype:
        raise ValueError("out shape or dtype mismatch")
    with torch.cuda.device(x.device):
        _check("harp_rotate", _lib.harp_rotate(
            _ptr(x), _ptr(out), _DT[x.dtype], tokens, d, ldx, ldy, _sign_ptr(signs, d, x.device),
            int(bool(precondition)), rad, len(radices), _ptr(blocks), _DT[blocks.dtype], _stream(x)))
    return out


def _csr_dev(**ts):
    for nm, t in ts.items():
        _need_cuda(nm, t)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")


def qwha_csr_transpose(row_ptr, col_idx, d_in):
    """CSR of F^T from the CSR of F (host helper; numpy int32 arrays in and out).
    Returns (t_row_ptr [d_in + 1], t_col_idx [nnz], t_perm [nnz])."""
    import numpy as np
    rp = np.ascontiguousarray(row_ptr, dtype=np.int32)
    ci = np.ascontiguousarray(col_idx, dtype=np.int32)
    d_out, nnz = rp.size - 1, ci.size
    t_rp = np.empty(d_in + 1, np.int32)
    t_ci = np.empty(max(nnz, 1), np.int32)
    t_pm = np.empty(max(nnz, 1), np.int32)
    _check("qwha_csr_transpose", _lib.qwha_csr_transpose(
        rp.ctypes.data_as(_vp), ci.ctypes.data_as(_vp), d_out, d_in, nnz, t_rp.ctypes.data_as(_vp),
        t_ci.ctypes.data_as(_vp), t_pm.ctypes.data_as(_vp)))
    return t_rp, t_ci[:nnz], t_pm[:nnz]


def qwha_permute_values(vals, perm, out=None):
    """out[j] = vals[perm[j]] on the device (F's values in F^T's entry order)."""
    _csr_dev(vals=vals, perm=perm)
    if perm.dtype != torch.int32:
        raise ValueError("perm must be int32")
    if out is None:
        out = torch.empty(perm.numel(), dtype=vals.dtype, device=vals.device)
    _csr_dev(out=out)
    if out.numel() != perm.numel() or out.dtype != vals.dtype:
        raise ValueError("out must match perm's length and vals' dtype")
    with torch.cuda.device(vals.device):
        _check("qwha_permute_values", _lib.qwha_permute_values(
            _ptr(vals), _DT[vals.dtype], _ptr(perm), perm.numel(), _ptr(out), _stream(vals)))
    return out


def qwha_adapter_backward_input(dy, t_row_ptr, t_col_idx, t_vals, d_in=4096, out=None):
    """dx = (dy F) Hn from the CSR of F^T (t_row_ptr [d_in + 1], t_col_idx, t_vals)."""
    _need_cuda("dy", dy)
    tokens, d_out, lddy = _rows_ld("dy", dy)
    _csr_dev(t_row_ptr=t_row_ptr, t_col_idx=t_col_idx, t_vals=t_vals)
    if t_row_ptr.dtype != torch.int32 or t_col_idx.dtype != torch.int32:
        raise ValueError("t_row_ptr and t_col_idx must be int32")
    if t_row_ptr.numel() != d_in + 1:
        raise ValueError("t_row_ptr must have d_in + 1 entries")
    nnz = t_col_idx.numel()
    if t_vals.numel() != nnz:
        raise ValueError("t_vals and t_col_idx must have the same length")
    if out is None:
        out = torch.empty((tokens, d_in), dtype=dy.dtype, device=dy.device)
    r2, n2, lddx = _rows_ld("out", out)
    if (r2, n2) != (tokens, d_in):
        raise ValueError("out shape mismatch")
    with torch.cuda.device(dy.device):
        _check("qwha_adapter_backward_input", _lib.qwha_adapter_backward_input(
            _ptr(dy), _DT[dy.dtype], tokens, d_out, lddy, _ptr(t_row_ptr), _ptr(t_col_idx), _ptr(t_vals),
            _DT[t_vals.dtype], d_in, nnz, _ptr(out), _DT[out.dtype], lddx, _stream(dy)))
    return out


def qwha_grad_values_workspace_bytes(tokens, d_in, nnz):
    return int(_lib.qwha_grad_values_workspace_bytes(tokens, d_in, nnz))


def qwha_adapter_grad_values(x, dy, row_ptr, col_idx, out=None, workspace=None):
    """dc[e] = sum_t dy[t, row(e)] (x Hn)[t, col_idx[e]] in float32, CSR entry order."""
    _need_cuda("x", x)
    _need_cuda("dy", dy)
    tokens, d_in, ldx = _rows_ld("x", x)
    t2, d_out, lddy = _rows_ld("dy", dy)
    if t2 != tokens:
        raise ValueError("x and dy must have the same number of tokens")
    _csr_dev(row_ptr=row_ptr, col_idx=col_idx)
    if row_ptr.dtype != torch.int32 or col_idx.dtype != torch.int32:
        raise ValueError("row_ptr and col_idx must be int32")
    if row_ptr.numel() != d_out + 1:
        raise ValueError("row_ptr must have d_out + 1 entries")
    nnz = col_idx.numel()
    if out is None:
        out = torch.empty(nnz, dtype=torch.float32, device=x.device)
    _csr_dev(out=out)
    if out.dtype != torch.float32 or out.numel() != nnz:
        raise ValueError("out must be float32 with nnz entries")
    need = qwha_grad_values_workspace_bytes(tokens, d_in, nnz)
    if need < 0:
        raise WhtqError("qwha_grad_values_workspace_bytes", 2)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _csr_dev(workspace=workspace)
    wbytes = workspace.numel() * workspace.element_size()
    with torch.cuda.device(x.device):
        _check("qwha_adapter_grad_values", _lib.qwha_adapter_grad_values(
            _ptr(x), _ptr(dy), _DT[x.dtype], tokens, d_in, d_out, ldx, lddy, _ptr(row_ptr), _ptr(col_idx),
            nnz, _ptr(out), _ptr(workspace), wbytes, _stream(x)))
    return out


def qwha_adapter_grad_values_noalloc(x, dy, row_ptr, col_idx, out=None):
    """qwha_adapter_grad_values with the library's fixed per-GPU scratch array
    instead of a workspace (the library call allocates nothing; `out` is the
    caller's).  Calls that overlap on one GPU race."""
    _need_cuda("x", x)
    _need_cuda("dy", dy)
    tokens, d_in, ldx = _rows_ld("x", x)
    t2, d_out, lddy = _rows_ld("dy", dy)
    if t2 != tokens:
        raise ValueError("x and dy must have the same number of tokens")
    _csr_dev(row_ptr=row_ptr, col_idx=col_idx)
    if row_ptr.dtype != torch.int32 or col_idx.dtype != torch.int32:
        raise ValueError("row_ptr and col_idx must be int32")
    if row_ptr.numel() != d_out + 1:
        raise ValueError("row_ptr must have d_out + 1 entries")
    nnz = col_idx.numel()
    if out is None:
        out = torch.empty(nnz, dtype=torch.float32, device=x.device)
    _csr_dev(out=out)
    if out.dtype != torch.float32 or out.numel() != nnz:
        raise ValueError("out must be float32 with nnz entries")
    with torch.cuda.device(x.device):
        _check("qwha_adapter_grad_values_noalloc", _lib.qwha_adapter_grad_values_noalloc(
            _ptr(x), _ptr(dy), _DT[x.dtype], tokens, d_in, d_out, ldx, lddy, _ptr(row_ptr), _ptr(col_idx),
            nnz, _ptr(out), _stream(x)))
    return out


def harp_build_blocks(params, radices, d, scales=None, mixers=None, out=None, out_dtype=torch.float32):
    """Blocks Q(theta) G for harp_rotate from float32 parameters, or int8 codes
    with per-stage float32 scales; mixers float32 (stage-major) or None for Sylvester."""
    _need_cuda("params", params)
    if params.dtype not in (torch.float32, torch.int8) or not params.is_contiguous():
        raise ValueError("params must be contiguous float32 or int8")
    if params.dtype == torch.int8:
        _need_cuda("scales", scales)
        if scales.dtype != torch.float32 or scales.numel() != len(radices):
            raise ValueError("int8 params need float32 scales, one per stage")
    if mixers is not None:
        _need_cuda("mixers", mixers)
        if mixers.dtype != torch.float32 or not mixers.is_contiguous():
            raise ValueError("mixers must be contiguous float32")
    nblk = sum(d * int(b) for b in radices)
    if out is None:
        out = torch.empty(nblk, dtype=out_dtype, device=params.device)
    if out.numel() != nblk or not out.is_contiguous():
        raise ValueError("out must be contiguous with sum(d * b_t) elements")
    rad = (ctypes.c_int32 * len(radices))(*[int(b) for b in radices])
    with torch.cuda.device(params.device):
        _check("harp_build_blocks", _lib.harp_build_blocks(
            _ptr(params), _DT[params.dtype], _ptr(scales), d, rad, len(radices), _ptr(mixers), _ptr(out),
            _DT[out.dtype], _stream(params)))
    return out


# ------------------------------------------------------------ QWHA initialisation

QWHA_INIT_MAX_SUPPORT = 128


def _f32_rows(name, t):
    _need_cuda(name, t)
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32")
    return _rows_ld(name, t)


def qwha_init_error_coeffs(w, codes, scales, signs, bits, group, out=None):
    """F_dense = (W - Q(W)) Hn, float32 [rows, n], Q the RHT + RTN round trip of
    the stored codes / scales."""
    _need_cuda("w", w)
    rows, n, ldw = _rows_ld("w", w)
    if codes.shape != (rows, n * bits // 8) or scales.shape != (rows, n // group):
        raise ValueError("codes / scales shape mismatch")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    if out is None:
        out = torch.empty((rows, n), dtype=torch.float32, device=w.device)
    r2, n2, ldf = _f32_rows("out", out)
    if (r2, n2) != (rows, n):
        raise ValueError("out must be [rows, n]")
    with torch.cuda.device(w.device):
        _check("qwha_init_error_coeffs", _lib.qwha_init_error_coeffs(
            _ptr(w), _DT[w.dtype], rows, n, ldw, _ptr(codes), _ptr(scales), _sign_ptr(signs, n, w.device),
            bits, group, _ptr(out), ldf, _stream(w)))
    return out


def qwha_init_gram(x, g=None, accumulate=False, z=None):
    """G (+)= (x Hn)^T (x Hn), float32 [n, n]; z is the [tokens, n] float32
    workspace that receives x Hn.  Returns g."""
    _need_cuda("x", x)
    tokens, n, ldx = _rows_ld("x", x)
    if g is None:
        if accumulate:
            raise ValueError("accumulate needs g")
        g = torch.empty((n, n), dtype=torch.float32, device=x.device)
    if g.shape != (n, n) or g.dtype != torch.float32 or not g.is_contiguous():
        raise ValueError("g must be contiguous float32 [n, n]")
    if z is None:
        z = torch.empty((max(tokens, 1), n), dtype=torch.float32, device=x.device)
    if z.dtype != torch.float32 or not z.is_contiguous() or z.numel() < tokens * n:
        raise ValueError("z must be contiguous float32 with tokens * n elements")
    with torch.cuda.device(x.device):
        _check("qwha_init_gram", _lib.qwha_init_gram(
            _ptr(x), _DT[x.dtype], tokens, n, ldx, _ptr(z), _ptr(g), int(bool(accumulate)), _stream(x)))
    return g


def qwha_init_channel_errors(f, g, p=None, err=None):
    """(P = F G float32 [rows, n], err float32 [rows]) with err_o = sqrt(F[o] G F[o]^T)."""
    rows, n, ldf = _f32_rows("f", f)
    if g.shape != (n, n) or g.dtype != torch.float32 or not g.is_contiguous():
        raise ValueError("g must be contiguous float32 [n, n]")
    if p is None:
        p = torch.empty((rows, n), dtype=torch.float32, device=f.device)
    if err is None:
        err = torch.empty(rows, dtype=torch.float32, device=f.device)
    if p.shape != (rows, n) or p.dtype != torch.float32 or not p.is_contiguous():
        raise ValueError("p must be contiguous float32 [rows, n]")
    if err.shape != (rows,) or err.dtype != torch.float32:
        raise ValueError("err must be float32 [rows]")
    with torch.cuda.device(f.device):
        _check("qwha_init_channel_errors", _lib.qwha_init_channel_errors(
            _ptr(f), rows, n, ldf, _ptr(g), _ptr(p), _ptr(err), _stream(f)))
    return p, err


def qwha_init_allocate(err, n, total, floor, cap):
    """Host call: int32 row_ptr [rows + 1] of the per-channel budgets."""
    e = err.detach().to("cpu", torch.float32).contiguous()
    rows = e.numel()
    row_ptr = torch.empty(rows + 1, dtype=torch.int32)
    _check("qwha_init_allocate", _lib.qwha_init_allocate(
        _ptr(e), rows, n, int(total), int(floor), int(cap), _ptr(row_ptr)))
    return row_ptr


def qwha_init_select(f, row_ptr, col_idx=None):
    """int32 col_idx: per row the budget's largest |F| columns (ties to the lower
    column), ascending.  row_ptr: int32 device [rows + 1]."""
    rows, n, ldf = _f32_rows("f", f)
    _need_cuda("row_ptr", row_ptr)
    if row_ptr.dtype != torch.int32 or row_ptr.shape != (rows + 1,) or not row_ptr.is_contiguous():
        raise ValueError("row_ptr must be contiguous int32 [rows + 1]")
    # the size check reads row_ptr[-1] on the host, which a stream under
    # graph capture does not allow: there the caller's col_idx is trusted
    capturing = torch.cuda.is_current_stream_capturing()
    if col_idx is None:
        col_idx = torch.empty(int(row_ptr[-1].item()), dtype=torch.int32, device=f.device)
    _need_cuda("col_idx", col_idx)
    if col_idx.dtype != torch.int32 or not col_idx.is_contiguous():
        raise ValueError("col_idx must be contiguous int32")
    if not capturing and col_idx.numel() < int(row_ptr[-1].item()):
        raise ValueError("col_idx must hold row_ptr[-1] entries")
    with torch.cuda.device(f.device):
        _check("qwha_init_select", _lib.qwha_init_select(
            _ptr(f), rows, n, ldf, _ptr(row_ptr), _ptr(col_idx), _stream(f)))
    return col_idx


def qwha_init_refine(g, p, row_ptr, col_idx, vals=None):
    """float32 vals (CSR order) solving G[E][E] c = P[o][E] per row."""
    n = g.shape[0]
    if g.shape != (n, n) or g.dtype != torch.float32 or not g.is_contiguous():
        raise ValueError("g must be contiguous float32 [n, n]")
    rows = p.shape[0]
    if p.shape != (rows, n) or p.dtype != torch.float32 or not p.is_contiguous():
        raise ValueError("p must be contiguous float32 [rows, n]")
    for name, t in (("g", g), ("p", p), ("row_ptr", row_ptr), ("col_idx", col_idx)):
        _need_cuda(name, t)
    if row_ptr.dtype != torch.int32 or row_ptr.shape != (rows + 1,) or col_idx.dtype != torch.int32:
        raise ValueError("row_ptr / col_idx must be int32, row_ptr [rows + 1]")
    if not (row_ptr.is_contiguous() and col_idx.is_contiguous()):
        raise ValueError("row_ptr and col_idx must be contiguous")
    if vals is None:
        vals = torch.empty(col_idx.numel(), dtype=torch.float32, device=g.device)
    _need_cuda("vals", vals)
    if vals.dtype != torch.float32 or vals.numel() != col_idx.numel() or not vals.is_contiguous():
        raise ValueError("vals must be contiguous float32 with one entry per column index")
    if not torch.cuda.is_current_stream_capturing() and col_idx.numel() < int(row_ptr[-1].item()):
        raise ValueError("col_idx and vals must hold row_ptr[-1] entries")  # (not checked under graph capture)
    with torch.cuda.device(g.device):
        _check("qwha_init_refine", _lib.qwha_init_refine(
            _ptr(g), n, _ptr(p), rows, _ptr(row_ptr), _ptr(col_idx), _ptr(vals), _stream(g)))
    return vals


def qwha_initialize(w, codes, scales, signs, bits, group, x, total, floor, cap):
    """The whole initialisation of one layer through the calls above:
    returns (row_ptr int32, col_idx int32, vals float32) on w's device, plus
    the channel errors.  The budget allocation waits for the errors on the
    host (one device-to-host copy of rows floats)."""
    f = qwha_init_error_coeffs(w, codes, scales, signs, bits, group)
    g = qwha_init_gram(x)
    p, err = qwha_init_channel_errors(f, g)
    row_ptr = qwha_init_allocate(err, f.shape[1], total, floor, cap).to(w.device)
    col_idx = qwha_init_select(f, row_ptr)
    vals = qwha_init_refine(g, p, row_ptr, col_idx)
    return row_ptr, col_idx, vals, err


# ------------------------------------------------------------ paged key/value cache

@dataclasses.dataclass(frozen=True, eq=False)
class KVCache:
    """A paged cache of keys and values (include/whtq.h, whtq_kv_cache).

    k, v: [pages, kv_heads, page_size, dim] bfloat16 or float16, or uint8
    [pages, kv_heads, page_size, dim / 2] INT4 codes with float16 k_scales,
    v_scales [pages, kv_heads, page_size] and a sign bitmask (dim / 32 words,
    or None).  Any strides with a contiguous last dimension that the header's
    alignment allows (a transposed [pages, page_size, kv_heads, dim] too).
    The tensors stay the caller's.  Their addresses are read when the KVCache
    is made: other tensors need a new one (dataclasses.replace), and these must
    keep their storage (no resize_ or set_)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scales: Optional[torch.Tensor] = None
    v_scales: Optional[torch.Tensor] = None
    signs: Optional[torch.Tensor] = None

    def __post_init__(self):
        for nm, t in (("k", self.k), ("v", self.v)):
            _need_cuda(nm, t)
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{nm} must be [pages, kv_heads, page_size, dim] with a contiguous last dimension")
        if self.k.shape != self.v.shape or self.k.dtype != self.v.dtype or self.k.device != self.v.device:
            raise ValueError("k and v must have one shape, dtype and device")
        c = _Cache()
        int4 = self.k.dtype == torch.uint8
        if not int4 and self.k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("k and v must be bfloat16, float16 or uint8 (INT4 codes)")
        c.num_pages, c.kv_heads, c.page_size, c.dim = self.k.shape
        c.k, c.v = self.k.data_ptr(), self.v.data_ptr()
        c.k_stride[:], c.v_stride[:] = self.k.stride()[:3], self.v.stride()[:3]
        c.format = int(int4)
        if int4:
            c.dim = 2 * self.k.shape[3]
            for nm, t in (("k_scales", self.k_scales), ("v_scales", self.v_scales)):
                _need_cuda(nm, t)
                if t.dtype != torch.float16 or t.shape != self.k.shape[:3] or t.stride(2) != 1:
                    raise ValueError(f"{nm} must be float16 [pages, kv_heads, page_size] with contiguous offsets")
                if t.device != self.k.device:
                    raise ValueError(f"{nm} must be on k's device")
            c.k_scales, c.v_scales = self.k_scales.data_ptr(), self.v_scales.data_ptr()
            c.ks_stride[:], c.vs_stride[:] = self.k_scales.stride()[:2], self.v_scales.stride()[:2]
            c.sign_bits = _sign_ptr(self.signs, c.dim, self.k.device).value
        else:
            if self.k_scales is not None or self.v_scales is not None or self.signs is not None:
                raise ValueError("scales and signs belong to INT4 caches")
            c.dtype = _DT[self.k.dtype]
        self.__dict__.update(_c=c, int4=int4, dim=c.dim, kv_heads=c.kv_heads, page_size=c.page_size,
                             _scale=c.dim ** -0.5, _dev=self.k.get_device())


def kv_cache_alloc(num_pages, page_size, kv_heads, dim, *, int4=False, dtype=torch.bfloat16, signs=None, device="cuda"):
    """A zero-filled KVCache: 16-bit pages, or INT4 codes with scales."""
    if not int4:
        shape = (num_pages, kv_heads, page_size, dim)
        return KVCache(*(torch.zeros(shape, dtype=dtype, device=device) for _ in range(2)))
    codes = [torch.zeros((num_pages, kv_heads, page_size, dim // 2), dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.zeros((num_pages, kv_heads, page_size), dtype=torch.float16, device=device) for _ in range(2)]
    return KVCache(*codes, *scales, signs)


_NORM_DT = frozenset((torch.float32, torch.bfloat16, torch.float16))
_CLEAR_Q, _CLEAR_K = 0x100, 0x200  # WHTQ_CLEAR_Q, WHTQ_CLEAR_K
_pair = functools.lru_cache(maxsize=1024)(lambda a, b: (_i64 * 2)(a, b))  # strides as the library takes them
_raw_stream = torch._C._cuda_getCurrentRawStream


def _rows_like(t):
    """A new contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _on_device(dev, f, *args):
    """f(*args, stream) on device `dev`'s current stream."""
    if torch.cuda.current_device() == dev:
        return f(*args, _raw_stream(dev))
    with torch.cuda.device(dev):
        return f(*args, _raw_stream(dev))


def _head_rows(name, t, cache, tokens, heads, dtype):
    return _dense_rows(name, t, cache._dev, "the cache's", cache.dim, tokens, heads, dtype)


def _dense_rows(name, t, dev, whose, dim, tokens, heads, dtype):
    """Strides of a [tokens, heads, dim] tensor with contiguous head vectors."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on {whose} device")
    shape, st = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != dim or st[2] != 1:
        raise ValueError(f"{name} must be [tokens, heads, {dim}] with a contiguous last dimension")
    if shape[0] != tokens or shape[1] != heads:
        raise ValueError(f"{name} must have {tokens} tokens and {heads} heads")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    # the stride of a dimension of one entry is meaningless
    return _pair(st[0] if tokens > 1 else 0, st[1] if heads > 1 else 0)


def _rows_dtype(name, t, cache):
    """The type of a call's rows: a 16-bit cache's own, or either with INT4."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a [tokens, heads, dim] tensor")
    dtype = t.dtype
    if dtype is not cache.k.dtype and not (cache.int4 and dtype in (torch.bfloat16, torch.float16)):
        raise ValueError(f"{name} must be {'bfloat16 or float16' if cache.int4 else cache.k.dtype}")
    return dtype


def _ints(name, t, dtype, dev, n, whose="the cache's"):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or t.shape != (n,) or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{n}] tensor on {whose} device")
    return t.data_ptr()


def _rope_arg(cos, sin, positions, rot_dim, interleaved, tokens, dev, whose):
    """The rotation of a call, or None without tables and positions."""
    if cos is None and sin is None and positions is None:
        return None
    for nm, t in (("cos", cos), ("sin", sin)):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.dim() != 2 or t.get_device() != dev:
            raise ValueError(f"{nm} must be a float32 [positions, rot_dim / 2] tensor with a contiguous last "
                             f"dimension on {whose} device")
    (rows, half), (ld, one) = cos.shape, cos.stride()
    if one != 1:
        raise ValueError("cos and sin must have a contiguous last dimension")
    if sin.shape != (rows, half) or sin.stride() != (ld, 1):
        raise ValueError("cos and sin must have one shape and layout")
    rot = 2 * half if rot_dim is None else int(rot_dim)
    if rot > 2 * half:
        raise ValueError("cos and sin must hold rot_dim / 2 entries a row")
    return _Rope(cos.data_ptr(), sin.data_ptr(), _ints("positions", positions, torch.int32, dev, tokens, whose),
                 ld if rows > 1 else -(-half // 4) * 4, rows, rot, 1 if interleaved else 0)


def _norm_arg(q_norm, k_norm, eps, heads, kv_heads, dim, dev, whose):
    """The norms of a call: weights [dim], or [heads, dim] for one a head."""
    q_p, q_head = _norm_weight("q_norm", q_norm, heads, dim, dev, whose)
    k_p, k_head = _norm_weight("k_norm", k_norm, kv_heads, dim, dev, whose)
    if q_norm is not None and k_norm is not None and q_norm.dtype is not k_norm.dtype:
        raise ValueError("q_norm and k_norm must have one dtype")
    return _Norm(q_p, k_p, q_head, k_head, _DT[(k_norm if q_norm is None else q_norm).dtype], eps)


def _norm_weight(name, t, heads, dim, dev, whose):
    if t is None:
        return 0, 0
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype not in _NORM_DT:
        raise ValueError(f"{name} must be a float32, bfloat16 or float16 tensor on {whose} device")
    shape, st = t.shape, t.stride()
    if (shape != (dim,) and shape != (heads, dim)) or st[-1] != 1:
        raise ValueError(f"{name} must be [{dim}] or [{heads}, {dim}] with a contiguous last dimension")
    # (a stride of 0 says that all heads share one vector)
    return t.data_ptr(), 0 if len(shape) == 1 else st[0] if heads > 1 else dim


def kv_append(cache, k, v, slots, *, q=None, cos=None, sin=None, positions=None, rot_dim=None, interleaved=False,
              q_out=None, q_norm=None, k_norm=None, norm_eps=1e-6):
    """Rotates new keys (and queries) by their positions and writes keys and
    values [tokens, kv_heads, dim] into the cache's slots (int64 [tokens];
    outside the cache: not written).  cos, sin: float32 [positions, rot_dim /
    2] tables, or None for no rotation; positions: int32 [tokens].  q_norm,
    k_norm: weights of norms of each head vector before the rotation, [dim] or
    [heads, dim] (x / sqrt(mean x^2 + norm_eps) * weight; None: no norm).
    Returns the rotated queries (q_out, q's shape; q_out=q rotates in place).  A
    token whose position lies outside the tables is not written anywhere: its
    rows of a q_out allocated here are undefined."""
    dtype = _rows_dtype("k", k, cache)
    tokens, dev = k.shape[0], cache._dev
    ks = _head_rows("k", k, cache, tokens, cache.kv_heads, dtype)
    vs = _head_rows("v", v, cache, tokens, cache.kv_heads, dtype)
    slots_p = _ints("slots", slots, torch.int64, dev, tokens)
    rope = _rope_arg(cos, sin, positions, rot_dim, interleaved, tokens, dev, "the cache's")
    qs = qos = q_p = qo_p = None
    heads = 0
    if q is not None:
        heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
        qs = _head_rows("q", q, cache, tokens, heads, dtype)
        if q_out is None:
            q_out = _rows_like(q)
        qos = _head_rows("q_out", q_out, cache, tokens, heads, dtype)
        q_p, qo_p = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if q_norm is None and k_norm is None:
        _check("kv_append", _on_device(dev, _lib.kv_append, cache._c, k.data_ptr(), ks, v.data_ptr(), vs, _DT[dtype],
                                       tokens, slots_p, rope, q_p, qs, heads, qo_p, qos))
        return q_out
    if q is None and q_norm is not None:
        raise ValueError("q_norm needs q")
    norm = _norm_arg(q_norm, k_norm, norm_eps, heads, cache.kv_heads, cache.dim, dev, "the cache's")
    _check("kv_append_norm", _on_device(dev, _lib.kv_append_norm, cache._c, k.data_ptr(), ks, v.data_ptr(), vs, _DT[dtype],
                                        tokens, slots_p, norm, rope, q_p, qs, heads, qo_p, qos))
    return q_out


def _qk_call(q, k, q_norm, k_norm, norm_eps, cos, sin, positions, rot_dim, interleaved):
    """What qk_norm_rope and its backward pass have in common: sizes, strides, norms and rotation."""
    for nm, t in (("q", q), ("k", k)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.get_device() < 0:
            raise ValueError(f"{nm} must be a [tokens, heads, dim] device tensor")
    dtype, dev = q.dtype, q.get_device()
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q must be bfloat16 or float16")
    tokens, heads, dim = q.shape
    kv_heads = k.shape[1]
    if q_norm is None or k_norm is None:
        raise ValueError("q_norm and k_norm must be given")
    rows = lambda name, t, h: _dense_rows(name, t, dev, "q's", dim, tokens, h, dtype)
    norm = _norm_arg(q_norm, k_norm, norm_eps, heads, kv_heads, dim, dev, "q's")
    rope = _rope_arg(cos, sin, positions, rot_dim, interleaved, tokens, dev, "q's")
    return dtype, dev, tokens, heads, kv_heads, dim, rows, rows("q", q, heads), rows("k", k, kv_heads), norm, rope


def qk_norm_rope(q, k, *, q_norm, k_norm, norm_eps=1e-6, cos=None, sin=None, positions=None, rot_dim=None,
                 interleaved=False, q_out=None, k_out=None):
    """Norms of each head vector of q [tokens, heads, dim] and k [tokens,
    kv_heads, dim] with weights [dim] or [heads, dim], then their rotation, as
    in kv_append, into dense rows.  Returns (q_out, k_out); q_out=q and k_out=k
    work in place.  A token whose position lies outside the tables (-1 for
    padding) leaves its rows of a given q_out or k_out as they are; of those
    allocated here they are 0."""
    dtype, dev, tokens, heads, kv_heads, dim, rows, qs, ks, norm, rope = _qk_call(
        q, k, q_norm, k_norm, norm_eps, cos, sin, positions, rot_dim, interleaved)
    norm.dtype |= (_CLEAR_Q if q_out is None else 0) | (_CLEAR_K if k_out is None else 0)
    q_out = _rows_like(q) if q_out is None else q_out
    k_out = _rows_like(k) if k_out is None else k_out
    qos, kos = rows("q_out", q_out, heads), rows("k_out", k_out, kv_heads)
    _check("qk_norm_rope", _on_device(dev, _lib.qk_norm_rope, q.data_ptr(), qs, heads, k.data_ptr(), ks, kv_heads,
                                      _DT[dtype], dim, tokens, norm, rope, q_out.data_ptr(), qos, k_out.data_ptr(), kos))
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, *, q_norm, k_norm, norm_eps=1e-6, cos=None, sin=None, positions=None,
                          rot_dim=None, interleaved=False, dq=None, dk=None, workspace=None):
    """The gradients of qk_norm_rope's inputs from those of its outputs and the
    same inputs: (dq, dk, dq_norm, dk_norm), the weights' in float32 and their
    shape.  dq and dk may be any rows of q's and k's shapes, dq_out and dk_out
    among them.  A token outside the tables adds nothing to the weights'
    gradients; its rows of a given dq or dk stay as they are, of those allocated
    here they are 0.  workspace: a tensor of
    qk_norm_rope_backward_workspace_bytes, allocated here if not given."""
    dtype, dev, tokens, heads, kv_heads, dim, rows, qs, ks, norm, rope = _qk_call(
        q, k, q_norm, k_norm, norm_eps, cos, sin, positions, rot_dim, interleaved)
    for nm, t in (("q_norm", q_norm), ("k_norm", k_norm)):
        if t.dim() == 2 and t.shape[0] > 1 and t.stride(0) == 0:
            raise ValueError(f"{nm} is one vector expanded over the heads: pass it as [dim], its gradient is one vector too")
    dqos, dkos = rows("dq_out", dq_out, heads), rows("dk_out", dk_out, kv_heads)
    norm.dtype |= (_CLEAR_Q if dq is None else 0) | (_CLEAR_K if dk is None else 0)
    dq = _rows_like(q) if dq is None else dq
    dk = _rows_like(k) if dk is None else dk
    dqs, dks = rows("dq", dq, heads), rows("dk", dk, kv_heads)
    dwq, dwk = (torch.empty_like(t, dtype=torch.float32, memory_format=torch.contiguous_format) for t in (q_norm, k_norm))
    if workspace is None:
        need = _bytes(dev, _lib.qk_norm_rope_backward_workspace_bytes, heads, kv_heads, dim, tokens, norm)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_p, wbytes = _workspace(workspace, dev, "q's")
    _check("qk_norm_rope_backward", _on_device(
        dev, _lib.qk_norm_rope_backward, dq_out.data_ptr(), dqos, q.data_ptr(), qs, heads, dk_out.data_ptr(), dkos,
        k.data_ptr(), ks, kv_heads, _DT[dtype], dim, tokens, norm, rope, dq.data_ptr(), dqs, dk.data_ptr(), dks,
        dwq.data_ptr(), dwk.data_ptr(), ws_p, wbytes))
    return dq, dk, dwq, dwk


def qk_norm_rope_backward_workspace_bytes(q, k, *, q_norm, k_norm):
    norm = _norm_arg(q_norm, k_norm, 0.0, q.shape[1], k.shape[1], q.shape[2], q.get_device(), "q's")
    with torch.cuda.device(q.device):
        return int(_lib.qk_norm_rope_backward_workspace_bytes(q.shape[1], k.shape[1], q.shape[2], q.shape[0], norm))


def _bytes(dev, f, *args):
    """f(*args), a workspace's size on device `dev`."""
    if torch.cuda.current_device() == dev:
        return f(*args)
    with torch.cuda.device(dev):
        return f(*args)


def _workspace(t, dev, whose):
    """(address, bytes) of a workspace tensor or None."""
    if t is None:
        return 0, 0
    if not isinstance(t, torch.Tensor) or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"workspace must be a contiguous tensor on {whose} device")
    return t.data_ptr(), t.numel() * t.element_size()


def kv_gather(cache, slots, *, dtype=None, k_out=None, v_out=None):
    """(k, v) [tokens, kv_heads, dim]: what the cache's slots (int64 [tokens])
    stand for; zeros for a slot outside the cache.  dtype: an INT4 cache's
    output type (bfloat16 by default)."""
    dev = cache._dev
    tokens = slots.numel() if isinstance(slots, torch.Tensor) else 0
    slots_p = _ints("slots", slots, torch.int64, dev, tokens)
    if dtype is None:
        dtype = torch.bfloat16 if cache.int4 else cache.k.dtype
    elif dtype is not cache.k.dtype and not (cache.int4 and dtype in (torch.bfloat16, torch.float16)):
        raise ValueError(f"dtype must be {'bfloat16 or float16' if cache.int4 else cache.k.dtype}")
    heads, shape = cache.kv_heads, (tokens, cache.kv_heads, cache.dim)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=cache.k.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=cache.k.device)
    ks = _head_rows("k_out", k_out, cache, tokens, heads, dtype)
    vs = _head_rows("v_out", v_out, cache, tokens, heads, dtype)
    _check("kv_gather", _on_device(dev, _lib.kv_gather, cache._c, tokens, slots_p, k_out.data_ptr(), ks, v_out.data_ptr(),
                                   vs, _DT[dtype]))
    return k_out, v_out


def kv_attention_workspace_bytes(cache, q_tokens, heads, seqs, max_q_len, max_kv_len, window=0, sinks=0):
    with torch.cuda.device(cache._dev):
        return int(_lib.kv_attention_sinks_workspace_bytes(cache._c, q_tokens, heads, seqs, max_q_len, max_kv_len, window,
                                                           sinks))


def kv_attention(cache, q, q_start, kv_len, block_table, *, max_q_len, max_kv_len, scale=None, causal=True, window=0, sinks=0,
                 out=None, lse=None, workspace=None):
    """Attention of new tokens q [tokens, heads, dim] over their sequences'
    pages.  q_start: int32 [seqs + 1]; kv_len: int32 [seqs] (keys, the new
    tokens' included); block_table: int32 [seqs, width].  max_q_len and
    max_kv_len bound the lengths (host numbers).  scale: 1 / sqrt(dim) by
    default; window: 0, or how many of the latest keys a query sees; sinks: how
    many of a sequence's first keys it sees as well.  lse: a float32 [tokens, heads] tensor to fill.  workspace: a uint8 tensor of
    kv_attention_workspace_bytes, allocated here if not given."""
    dtype = _rows_dtype("q", q, cache)
    dev = cache._dev
    tokens, heads, _ = q.shape
    qs = _head_rows("q", q, cache, tokens, heads, dtype)
    if not isinstance(kv_len, torch.Tensor):
        raise ValueError("kv_len must be a tensor")
    seqs = kv_len.numel()
    start_p = _ints("q_start", q_start, torch.int32, dev, seqs + 1)
    kv_p = _ints("kv_len", kv_len, torch.int32, dev, seqs)
    if not isinstance(block_table, torch.Tensor) or block_table.dtype is not torch.int32 or block_table.dim() != 2 or \
            block_table.get_device() != dev:
        raise ValueError("block_table must be an int32 [seqs, width] tensor on the cache's device")
    (rows, width), (ts, t1) = block_table.shape, block_table.stride()
    if rows != seqs or (width > 1 and t1 != 1):
        raise ValueError("block_table must have a row per sequence and a contiguous last dimension")
    if heads % cache.kv_heads:
        raise ValueError("q's heads must be a multiple of the cache's")
    if out is None:
        out = _rows_like(q)
    outs = _head_rows("out", out, cache, tokens, heads, dtype)
    lse_p = None
    if lse is not None:
        if not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float32 or lse.shape != (tokens, heads) or \
                not lse.is_contiguous() or lse.get_device() != dev:
            raise ValueError("lse must be a contiguous float32 [tokens, heads] tensor on the cache's device")
        lse_p = lse.data_ptr()
    if workspace is None:
        need = _bytes(dev, _lib.kv_attention_sinks_workspace_bytes, cache._c, tokens, heads, seqs, max_q_len, max_kv_len,
                      window, sinks)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_p, wbytes = _workspace(workspace, dev, "the cache's")
    _check("kv_attention", _on_device(
        dev, _lib.kv_attention_sinks, cache._c, q.data_ptr(), qs, _DT[dtype], tokens, heads, seqs, start_p, kv_p,
        block_table.data_ptr(), ts if seqs > 1 else width, width, max_q_len, max_kv_len,
        cache._scale if scale is None else scale, 1 if causal else 0, window, sinks, out.data_ptr(), outs, lse_p, ws_p, wbytes))
    return out


class TokenLogprobs:
    """Of rows of logits: float32 [rows] logprob (None without targets), lse
    and entropy; top_logprob float32 and top_id int64 [rows, top] (None for top
    = 0).  row_ref (a logit near the row's largest) and row_sum (of the
    exponentials relative to it) are for the gradient."""
    __slots__ = ("_buf", "_at", "_n", "_of", "_targets", "top_logprob", "top_id")

    def __init__(self, buf, at, rows, vocab, scale, targets, top_logprob, top_id):
        self._buf, self._at, self._n, self._of, self._targets = buf, at, rows, (vocab, scale), targets
        self.top_logprob, self.top_id = top_logprob, top_id

    def _row(self, i):  # parts of one tensor, taken out when they are asked for
        return self._buf[self._at + i * self._n:self._at + (i + 1) * self._n]

    lse = property(lambda self: self._row(0))
    row_ref = property(lambda self: self._row(1))
    row_sum = property(lambda self: self._row(2))
    entropy = property(lambda self: self._row(3))
    logprob = property(lambda self: self._row(4) if self._targets else None)

    def _ptr(self, i):
        return self._buf.data_ptr() + 4 * (self._at + i * self._n)


def _logits(name, t, dev=None, shape=None):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.get_device() < 0 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a [rows, vocab] device tensor with a contiguous last dimension")
    if t.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    if dev is not None and (t.get_device() != dev or t.shape != shape):
        raise ValueError(f"{name} must have the logits' shape and device")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _row_floats(name, t, rows, dev):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.shape != (rows,) or not t.is_contiguous() or \
            t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous float32 [{rows}] tensor on the logits' device")
    return t.data_ptr()


# Bytes of scratch that the results of token_logprobs may hold on to.  A tensor of its own costs a call 2 us (8 rows of
# 131072, 20 tokens, 9760 bytes: 18.4 us against 16.6), but results are kept, and a few long rows have megabytes of it.
_SCRATCH_BESIDE = 16384


def token_logprobs_workspace_bytes(rows, vocab, top=0, device="cuda"):
    with torch.cuda.device(device):
        return int(_lib.token_logprobs_workspace_bytes(rows, vocab, top))


def token_logprobs(logits, targets=None, *, top=0, scale=1.0, workspace=None):
    """Log probabilities under softmax(scale * logits) of logits [rows, vocab]:
    of targets (int64 [rows]; one outside the vocabulary gives 0), the `top`
    (at most 32) likeliest tokens of each row (equal logits: the lower index
    first) and the entropy, in one pass.  workspace: a tensor of
    token_logprobs_workspace_bytes, allocated here if not given.  Returns
    TokenLogprobs."""
    ld = _logits("logits", logits)
    (rows, vocab), dev = logits.shape, logits.get_device()
    t_p = None
    if targets is not None:
        t_p = _ints("targets", targets, torch.int64, dev, rows, "the logits'")
    top_logprob = top_id = top_lp = top_ip = None
    if top > 0:
        top_logprob = torch.empty((rows, top), dtype=torch.float32, device=logits.device)
        top_id = torch.empty((rows, top), dtype=torch.int64, device=logits.device)
        top_lp, top_ip = top_logprob.data_ptr(), top_id.data_ptr()
    need = _bytes(dev, _lib.token_logprobs_workspace_bytes, rows, vocab, top) if workspace is None else 0
    if need > _SCRATCH_BESIDE:
        workspace = torch.empty(need, dtype=torch.uint8, device=logits.device)
        need = 0
    # a small workspace and the results in one tensor
    at = max(need, 0) // 4
    buf = torch.empty(at + 5 * rows, dtype=torch.float32, device=logits.device)
    ws_p, wbytes = _workspace(workspace, dev, "the logits'") if need <= 0 else (buf.data_ptr(), need)
    r = TokenLogprobs(buf, at, rows, vocab, scale, t_p is not None, top_logprob, top_id)
    _check("token_logprobs", _on_device(
        dev, _lib.token_logprobs, logits.data_ptr(), _DT[logits.dtype], rows, vocab, ld, scale, t_p,
        None if t_p is None else r._ptr(4), r._ptr(0), r._ptr(1), r._ptr(2), r._ptr(3), top, top_lp, top_ip, ws_p, wbytes))
    return r


def token_logprobs_backward(logits, targets, result, dlogprob=None, dentropy=None, *, scale=1.0, out=None):
    """The gradient of the logits for float32 [rows] gradients of `result`'s
    logprob and entropy (either may be None), `result` being token_logprobs's of
    the same logits, targets and scale (one of another shape or scale is
    refused, other values are not noticed).  out: a tensor of the logits' shape and
    type (out=logits works in place)."""
    ld = _logits("logits", logits)
    (rows, vocab), dev = logits.shape, logits.get_device()
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    ldd = _logits("out", out, dev, logits.shape)
    if out.dtype is not logits.dtype:
        raise ValueError("out must have the logits' dtype")
    t_p = _ints("targets", targets, torch.int64, dev, rows, "the logits'") if targets is not None else None
    of = lambda name, t: _row_floats(name, t, rows, dev) if t is not None else None
    if not isinstance(result, TokenLogprobs) or result._n != rows or result._of != (vocab, scale) or \
            result._buf.get_device() != dev:
        raise ValueError("result must be token_logprobs's of these logits and this scale")
    _check("token_logprobs_backward", _on_device(
        dev, _lib.token_logprobs_backward, logits.data_ptr(), _DT[logits.dtype], rows, vocab, ld, scale, t_p,
        result._ptr(1), result._ptr(2), result._ptr(3), of("dlogprob", dlogprob), of("dentropy", dentropy), out.data_ptr(), ldd))
    return out


def stream_probe(src, dst):
    """Measurement helper: read all bytes of `src` and write all bytes of `dst`
    with a plain 16-byte streaming kernel (the "% achievable" reference)."""
    _need_cuda("src", src)
    _need_cuda("dst", dst)
    if not (src.is_contiguous() and dst.is_contiguous()):
        raise ValueError("src and dst must be contiguous")
    ib, ob = src.numel() * src.element_size(), dst.numel() * dst.element_size()
    with torch.cuda.device(src.device):
        _check("whtq_stream_probe", _lib.whtq_stream_probe(_ptr(src), ib, _ptr(dst), ob, _stream(src)))
    return dst
