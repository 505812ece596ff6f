"""Quantized-linear hot path for AMD MI355X (gfx950): Python binding of libpql.

Argument marshalling only: every step of quantize / dequantize / qgemm /
qlinear runs in the HIP kernels of ``libpql.so`` (declared in
``include/pql.h``).  torch supplies device memory and the current stream.
There is no CPU fallback: if the library is missing, every call raises.

    import precision_quantized_linear_amd as pql
    wq = pql.quantize(w, "mxfp8", "weight")      # once, at load
    y = pql.qlinear(x, wq)                        # every call: quantize x, GEMM

A layer of experts (``moe_route``, ``moe_plan``, ``moe_qgemm``, ``swiglu_quantize``,
``moe_combine``, and all of them after the router as ``moe_mlp``) is for inference like the
rest: no call records a gradient.  So is the cache of keys and values with the attention over it
(``rope``, ``kv_slots``, ``kv_append``, ``kv_read``, ``kv_attention``; ``kv.py``).
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpql.so")

# MX exponent bytes per packed chunk (one chunk = 128 bytes of codes along K).
MX_CHUNK = {"mxfp8": 4, "mxfp4": 8}

SCHEMES = {"fp8_tensor": 0, "fp8_row": 1, "fp8_block128": 2, "mxfp8": 3, "mxfp4": 4,
           "w4a16_asym": 5, "w4a16_sym": 6, "int8_row": 7, "mxfp4_dual": 8}
STATIC_SCHEMES = ("fp8_tensor", "fp8_block128")
ROLES = {"activation": 0, "weight": 1}
OPS = {"quantize": 0, "dequantize": 1, "qgemm": 2, "qlinear": 3}

PQL_OK, PQL_ERR_INVALID_ARGUMENT, PQL_ERR_UNSUPPORTED, PQL_ERR_WORKSPACE, PQL_ERR_HIP = range(5)

_lib = None


class PqlError(RuntimeError):
    """A HIP runtime failure reported by libpql."""


def lib() -> ctypes.CDLL:
    """Load libpql.so (built in-tree by ``precision_quantized_linear_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; run `python -m precision_quantized_linear_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        i64, sz, vp, ci = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
        L.pql_version.restype = ci
        L.pql_last_error.restype = ctypes.c_char_p
        L.pql_kernel_name.restype = ctypes.c_char_p
        L.pql_kernel_name.argtypes = [ci, ci, ci, i64, i64, i64]
        L.pql_quantized_sizes.argtypes = [ci, ci, i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.pql_workspace_size.argtypes = [ci, ci, ci, i64, i64, i64, ctypes.POINTER(sz)]
        L.pql_quantize.argtypes = [ci, ci, vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]
        L.pql_dequantize.argtypes = [ci, ci, vp, vp, vp, i64, i64, vp, i64, vp]
        L.pql_qgemm.argtypes = [ci, vp, vp, vp, vp, vp, i64, i64, i64, vp, i64, vp]
        L.pql_qlinear.argtypes = [ci, vp, i64, i64, i64, vp, vp, vp, i64, vp, i64, vp, sz, vp]
        f32 = ctypes.c_float
        L.pql_quantize_static.argtypes = [ci, ci, vp, i64, i64, i64, vp, vp, vp]
        L.pql_qgemm_ex.argtypes = [ci, vp, vp, vp, vp, vp, i64, i64, i64, f32, vp, vp, i64, vp]
        L.pql_qlinear_ex.argtypes = [ci, vp, i64, i64, i64, vp, vp, vp, vp, i64, f32, vp, vp, i64, vp, sz, vp]
        L.pql_layout_sizes.argtypes = [ci, ci, ci, i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.pql_repack.argtypes = [ci, ci, ci, ci, vp, vp, vp, vp, i64, i64, vp]
        L.pql_qlinear_noalloc.argtypes = [ci, vp, i64, i64, i64, vp, vp, vp, vp, i64, f32, vp, vp, i64, vp]
        L.pql_noalloc_scratch_bytes.restype = sz
        L.pql_moe_kernel_name.restype = ctypes.c_char_p
        L.pql_moe_kernel_name.argtypes = [ci, ci, i64, i64, i64, i64, i64]
        L.pql_moe_route.argtypes = [ci, ci, vp, i64, i64, i64, vp, i64, i64, i64, ci, ci, f32, vp, vp, vp]
        L.pql_moe_plan_workspace.argtypes = [i64, i64, i64, ctypes.POINTER(sz)]
        L.pql_moe_plan.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]
        L.pql_moe_qgemm.argtypes = [ci, vp, vp, i64, ci, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, i64, vp]
        L.pql_swiglu_quantize.argtypes = [ci, vp, i64, i64, i64, vp, vp, vp, vp]
        L.pql_moe_combine.argtypes = [vp, i64, i64, vp, vp, i64, i64, i64, vp, i64, vp, i64, vp]
        L.pql_rope.argtypes = [ci, vp, i64, i64, i64, i64, i64, vp, vp, i64, f32, vp, i64, i64, vp]
        L.pql_kv_sizes.argtypes = [ci, i64, i64, i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.pql_kv_slots.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, vp, vp, vp]
        L.pql_kv_append.argtypes = [ci, vp, i64, i64, vp, i64, i64, i64, vp, ci, vp, vp, i64, f32, vp, vp, vp, vp, i64,
                                    i64, i64, i64, vp]
        L.pql_kv_read.argtypes = [ci, vp, vp, vp, vp, i64, i64, i64, i64, vp, i64, vp, i64, i64, vp, i64, i64, vp]
        L.pql_kv_attention_workspace.argtypes = [ci, i64, i64, i64, i64, i64, i64, i64, ctypes.POINTER(sz)]
        L.pql_kv_attention.argtypes = [ci, vp, i64, i64, i64, i64, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, vp, i64,
                                       i64, i64, ci, i64, f32, vp, i64, i64, vp, vp, sz, vp]
        L.pql_kv_kernel_name.restype = ctypes.c_char_p
        L.pql_kv_kernel_name.argtypes = [ci, i64, i64, i64, i64, i64, i64, i64]
        for f in ("pql_rope", "pql_kv_sizes", "pql_kv_slots", "pql_kv_append", "pql_kv_read",
                  "pql_kv_attention_workspace", "pql_kv_attention", "pql_moe_route", "pql_moe_plan_workspace", "pql_moe_plan", "pql_moe_qgemm", "pql_swiglu_quantize",
                  "pql_moe_combine", "pql_quantized_sizes", "pql_workspace_size", "pql_quantize", "pql_dequantize",
                  "pql_qgemm", "pql_qlinear", "pql_quantize_static", "pql_qgemm_ex", "pql_qlinear_ex",
                  "pql_qlinear_noalloc", "pql_layout_sizes", "pql_repack"):
            getattr(L, f).restype = ci
        _lib = L
    return _lib


def _check(status: int, what: str) -> None:
    if status == PQL_OK:
        return
    msg = f"{what}: {lib().pql_last_error().decode()}"
    if status in (PQL_ERR_INVALID_ARGUMENT, PQL_ERR_WORKSPACE):
        raise ValueError(msg)
    if status == PQL_ERR_UNSUPPORTED:
        raise NotImplementedError(msg)
    raise PqlError(msg)


def _scheme(s) -> int:
    if isinstance(s, int):
        return s
    if s not in SCHEMES:
        raise ValueError(f"unknown scheme {s!r}; supported: {sorted(SCHEMES)}")
    return SCHEMES[s]


def _role(r) -> int:
    if isinstance(r, int):
        return r
    if r not in ROLES:
        raise ValueError(f"unknown role {r!r}")
    return ROLES[r]


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


@dataclass
class QTensor:
    """A quantized [rows, cols] tensor in the canonical layout of include/pql.h."""
    scheme: str
    role: str
    rows: int
    cols: int
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor | None = None

    @property
    def device(self):
        return self.codes.device


def quantized_sizes(scheme, role, rows: int, cols: int):
    c, s, z = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().pql_quantized_sizes(_scheme(scheme), _role(role), rows, cols,
                                     ctypes.byref(c), ctypes.byref(s), ctypes.byref(z)), "quantized_sizes")
    return c.value, s.value, z.value


def workspace_size(op, scheme, role="activation", M=0, N=0, K=0) -> int:
    b = ctypes.c_size_t()
    _check(lib().pql_workspace_size(OPS[op] if isinstance(op, str) else op, _scheme(scheme), _role(role),
                                    M, N, K, ctypes.byref(b)), "workspace_size")
    return b.value


def kernel_name(op, scheme, role="activation", M=0, N=0, K=0) -> str:
    return lib().pql_kernel_name(OPS[op] if isinstance(op, str) else op, _scheme(scheme), _role(role),
                                 M, N, K).decode()


def _alloc_q(scheme: str, role: str, rows: int, cols: int, device) -> QTensor:
    cb, sb, zb = quantized_sizes(scheme, role, rows, cols)
    if scheme.startswith("w4a16"):
        codes = torch.empty((rows, cols // 8), dtype=torch.int32, device=device)
        scales = torch.empty((cols // 128, rows), dtype=torch.bfloat16, device=device)   # group-major
        zeros = torch.empty((cols // 128, rows), dtype=torch.uint8, device=device)
    elif scheme == "int8_row":
        codes = torch.empty((rows, cols), dtype=torch.int8, device=device)
        scales = torch.empty((rows,), dtype=torch.float32, device=device)
        zeros = None
    elif scheme == "mxfp4_dual":   # fine exponents, then coarse fp32 scales, in one byte buffer
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        scales = torch.empty((sb,), dtype=torch.uint8, device=device)
        zeros = None
    else:
        codes = torch.empty((rows, cols if scheme != "mxfp4" else cols // 2), dtype=torch.uint8, device=device)
        if scheme in ("mxfp8", "mxfp4"):
            c = MX_CHUNK[scheme]
            scales = torch.empty((-(-cols // (32 * c)), rows, c), dtype=torch.uint8, device=device)
        elif scheme == "fp8_tensor":
            scales = torch.empty((1,), dtype=torch.float32, device=device)
        elif scheme == "fp8_row":
            scales = torch.empty((rows,), dtype=torch.float32, device=device)
        elif role == "activation":
            scales = torch.empty((rows, cols // 128), dtype=torch.float32, device=device)
        else:
            scales = torch.empty((rows // 128, cols // 128), dtype=torch.float32, device=device)
        zeros = None
    assert codes.numel() * codes.element_size() == cb and scales.numel() * scales.element_size() == sb
    return QTensor(scheme, role, rows, cols, codes, scales, zeros)


def _as_2d_bf16(x: torch.Tensor) -> torch.Tensor:
    if x.dtype != torch.bfloat16:
        raise ValueError("expected a bfloat16 tensor")
    if not x.is_cuda:
        raise ValueError("expected a tensor on a HIP device")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit stride along K")
    return x


def quantize(x: torch.Tensor, scheme: str, role: str = "activation", workspace: torch.Tensor | None = None,
             out: QTensor | None = None) -> QTensor:
    """Quantize a bf16 [rows, K] tensor (activation: rows = tokens; weight: rows = out channels).
    ``out`` reuses the buffers of an earlier result of the same scheme, role and shape."""
    x = _as_2d_bf16(x)
    rows, cols = x.shape
    if out is not None:
        _check_qtensor(out, "out")
        if (out.scheme, out.role, out.rows, out.cols) != (scheme, role, rows, cols):
            raise ValueError("out does not match the scheme, role and shape")
        if out.device != x.device:
            raise ValueError(f"out is on {out.device}, x on {x.device}")
        q = out
    else:
        q = _alloc_q(scheme, role, rows, cols, x.device)
    wsb = workspace_size("quantize", scheme, role)
    if wsb and workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    _check(lib().pql_quantize(_scheme(scheme), _role(role), x.data_ptr(), rows, cols, x.stride(0),
                              q.codes.data_ptr(), q.scales.data_ptr(), _ptr(q.zeros), _ptr(workspace),
                              0 if workspace is None else workspace.numel() * workspace.element_size(),
                              _stream(x.device)), "quantize")
    return q


def quantize_static(x: torch.Tensor, scheme: str, role: str, scales: torch.Tensor,
                    out: QTensor | None = None) -> QTensor:
    """FP8 quantization with supplied (static, calibrated) fp32 scales in the scheme's
    canonical scale layout (fp8_tensor: [1]; fp8_block128: [rows, K/128] activations,
    [rows/128, K/128] weights).  The result holds ``scales`` itself."""
    if scheme not in STATIC_SCHEMES:
        raise NotImplementedError(f"static scales are defined for {STATIC_SCHEMES} only, not {scheme!r}")
    x = _as_2d_bf16(x)
    rows, cols = x.shape
    if scales.dtype != torch.float32 or not scales.is_contiguous() or scales.device != x.device:
        raise ValueError("scales must be a contiguous float32 tensor on the input's device")
    q = out if out is not None else _alloc_q(scheme, role, rows, cols, x.device)
    if scales.numel() != q.scales.numel():
        raise ValueError(f"expected {q.scales.numel()} scales, got {scales.numel()}")
    _check(lib().pql_quantize_static(_scheme(scheme), _role(role), x.data_ptr(), rows, cols, x.stride(0),
                                     scales.data_ptr(), q.codes.data_ptr(), _stream(x.device)), "quantize_static")
    return QTensor(scheme, role, rows, cols, q.codes, scales.reshape(q.scales.shape), None)


def _bias_ptr(bias, n: int, device):
    if bias is None:
        return None
    if bias.dtype != torch.bfloat16 or bias.shape != (n,) or not bias.is_contiguous() or bias.device != device:
        raise ValueError(f"bias must be a contiguous bfloat16 [{n}] tensor on the weight's device")
    return bias.data_ptr()


def _check_out(out: torch.Tensor, rows: int, cols: int, device, what: str = "out") -> None:
    """The C ABI sees only a pointer and a row stride, so the binding checks the rest:
    a bf16 [rows, cols] view on ``device`` with unit column stride and a row stride of
    at least ``cols`` (a view into a wider buffer is fine)."""
    if not isinstance(out, torch.Tensor):
        raise ValueError(f"{what} must be a torch tensor")
    if out.dtype != torch.bfloat16:
        raise ValueError(f"{what} must be bfloat16, not {out.dtype}")
    if out.dim() != 2 or tuple(out.shape) != (rows, cols):
        raise ValueError(f"{what} must have shape ({rows}, {cols}), not {tuple(out.shape)}")
    if rows and (out.stride(1) != 1 or out.stride(0) < cols):
        raise ValueError(f"{what} needs unit column stride and a row stride >= {cols} "
                         f"(strides {tuple(out.stride())})")
    if out.device != torch.device(device):
        raise ValueError(f"{what} is on {out.device}, the operands on {device}")


def _check_qtensor(q: QTensor, what: str) -> None:
    if not isinstance(q, QTensor):
        raise ValueError(f"{what} must be a QTensor")
    bufs = [q.codes, q.scales] + ([q.zeros] if q.zeros is not None else [])
    if any(b.device != q.codes.device for b in bufs):
        raise ValueError(f"{what}: codes, scales and zero-points must be on one device")


def _on_device(device) -> None:
    if (device if isinstance(device, torch.device) else torch.device(device)).type != "cuda":
        raise ValueError(f"operands must be on a HIP device, not {device}")


def dequantize(q: QTensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [rows, cols] = bf16(decode(code) * scale)."""
    _check_qtensor(q, "q")
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=torch.bfloat16, device=q.device)
    _check_out(out, q.rows, q.cols, q.device)
    _on_device(q.device)
    _check(lib().pql_dequantize(_scheme(q.scheme), _role(q.role), q.codes.data_ptr(), q.scales.data_ptr(),
                                _ptr(q.zeros), q.rows, q.cols, out.data_ptr(), out.stride(0),
                                _stream(q.device)), "dequantize")
    return out


def qgemm(a, w: QTensor, out: torch.Tensor | None = None, alpha: float = 1.0,
          bias: torch.Tensor | None = None) -> torch.Tensor:
    """C[M, N] = alpha * (A_hat * W_hat^T) + bias on quantized operands (W4A16: ``a`` is the
    bf16 activation).  ``alpha`` and ``bias`` (bf16 [N]) are the fused epilogue of the FP8
    and int8 schemes."""
    _check_qtensor(w, "w")
    if w.role != "weight":
        raise ValueError("the second operand must be a quantized weight")
    if isinstance(a, QTensor):
        _check_qtensor(a, "a")
        if a.role != "activation":
            raise ValueError("the first operand must be a quantized activation")
        if a.scheme != w.scheme:
            raise ValueError("activation and weight schemes differ")
        if w.scheme.startswith("w4a16"):
            raise ValueError("W4A16 takes the bf16 activation itself, not a quantized one")
        if a.device != w.device:
            raise ValueError(f"activation on {a.device}, weight on {w.device}")
        M, K = a.rows, a.cols
        a_ptr, as_ptr = a.codes.data_ptr(), a.scales.data_ptr()
    else:
        if not w.scheme.startswith("w4a16"):
            raise ValueError(f"{w.scheme} needs a quantized activation (pql.quantize(x, scheme, 'activation'))")
        a = _as_2d_bf16(a)
        if a.device != w.device:
            raise ValueError(f"activation on {a.device}, weight on {w.device}")
        if a.stride(0) != a.shape[1]:
            a = a.contiguous()
        M, K = a.shape
        a_ptr, as_ptr = a.data_ptr(), None
    if K != w.cols:
        raise ValueError(f"K mismatch: {K} vs {w.cols}")
    if out is None:
        out = torch.empty((M, w.rows), dtype=torch.bfloat16, device=w.device)
    _check_out(out, M, w.rows, w.device)
    _on_device(w.device)
    _check(lib().pql_qgemm_ex(_scheme(w.scheme), a_ptr, as_ptr, w.codes.data_ptr(), w.scales.data_ptr(),
                              _ptr(w.zeros), M, w.rows, K, float(alpha), _bias_ptr(bias, w.rows, w.device),
                              out.data_ptr(), out.stride(0), _stream(w.device)), "qgemm")
    return out


def qlinear(x: torch.Tensor, w: QTensor, out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, alpha: float = 1.0, bias: torch.Tensor | None = None,
            act_scales: torch.Tensor | None = None) -> torch.Tensor:
    """The quantized linear layer's forward: flatten x[..., K] to 2-D, quantize it with the
    weight's scheme (activation rule), GEMM against ``w``, restore the leading shape.
    ``out``, if given, is the 2-D [M, N] bf16 output (a view with a wider row stride is
    accepted).
    ``alpha`` / ``bias`` are the fused epilogue; ``act_scales`` (fp32, the scheme's
    activation scale layout) makes the activation scales static (fp8_tensor and
    fp8_block128)."""
    _check_qtensor(w, "w")
    if w.role != "weight":
        raise ValueError("w must be a quantized weight")
    lead = x.shape[:-1]
    x2 = x.reshape(-1, x.shape[-1])
    if x2.stride(-1) != 1 or (w.scheme.startswith("w4a16") and x2.stride(0) != x2.shape[1]):
        x2 = x2.contiguous()
    x2 = _as_2d_bf16(x2)
    M, K = x2.shape
    if K != w.cols:
        raise ValueError(f"K mismatch: {K} vs {w.cols}")
    if x2.device != w.device:
        raise ValueError(f"input on {x2.device}, weight on {w.device}")
    if out is None:
        out = torch.empty((M, w.rows), dtype=torch.bfloat16, device=x.device)
    _check_out(out, M, w.rows, w.device)
    if act_scales is not None:
        if w.scheme not in STATIC_SCHEMES:
            raise NotImplementedError(f"static activation scales are defined for {STATIC_SCHEMES} only")
        want = 1 if w.scheme == "fp8_tensor" else M * (K // 128)
        if (act_scales.dtype != torch.float32 or not act_scales.is_contiguous()
                or act_scales.device != x2.device):
            raise ValueError("act_scales must be a contiguous float32 tensor on the input's device")
        if act_scales.numel() != want:
            raise ValueError(f"{w.scheme} takes {want} activation scales, got {act_scales.numel()}")
    wsb = workspace_size("qlinear", w.scheme, "activation", M, w.rows, K)
    if wsb and workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    if workspace is not None and (workspace.device != x2.device or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the input's device")
    _on_device(w.device)
    _check(lib().pql_qlinear_ex(_scheme(w.scheme), x2.data_ptr(), M, K, x2.stride(0), _ptr(act_scales),
                                w.codes.data_ptr(), w.scales.data_ptr(), _ptr(w.zeros), w.rows, float(alpha),
                                _bias_ptr(bias, w.rows, x.device), out.data_ptr(), out.stride(0),
                                _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
                                _stream(x.device)), "qlinear")
    return out.reshape(*lead, w.rows)


LAYOUTS = {"canonical": 0, "packed": 1}


def layout_sizes(scheme, role, layout, rows: int, cols: int):
    c, s, z = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().pql_layout_sizes(_scheme(scheme), _role(role), LAYOUTS[layout], rows, cols,
                                  ctypes.byref(c), ctypes.byref(s), ctypes.byref(z)), "layout_sizes")
    return c.value, s.value, z.value


def _dual_coarse_offset(rows, cols):
    return (rows * (cols // 32) + 255) // 256 * 256


def _canonical_shapes(scheme, role, rows, cols):
    """(scales dtype, scales shape, zeros shape or None) of the canonical layout."""
    if scheme == "mxfp4_dual":
        return torch.uint8, (_dual_coarse_offset(rows, cols) + 4 * rows * (cols // 512),), None
    if scheme in MX_CHUNK:
        return torch.uint8, (rows, cols // 32), None
    if scheme.startswith("w4a16"):
        return torch.bfloat16, (rows, cols // 128), (rows, cols // 128)
    return None, None, None     # the same bytes as the packed layout


def _repack(scheme, role, rows, cols, frm, to, scales_in, zeros_in, scales_out, zeros_out, device):
    _check(lib().pql_repack(_scheme(scheme), _role(role), LAYOUTS[frm], LAYOUTS[to], scales_in.data_ptr(),
                            _ptr(zeros_in), scales_out.data_ptr(), _ptr(zeros_out), rows, cols, _stream(device)),
           "repack")


def to_canonical(q: QTensor):
    """(codes, scales, zeros) of ``q`` in the canonical layout, as device tensors; the
    scales (and W4A16 zero-points) are rearranged on the device by pql_repack."""
    _check_qtensor(q, "q")
    _on_device(q.device)
    dt, shape, zshape = _canonical_shapes(q.scheme, q.role, q.rows, q.cols)
    if dt is None:
        return q.codes, q.scales, q.zeros
    scales = torch.empty(shape, dtype=dt, device=q.device)
    zeros = torch.empty(zshape, dtype=torch.uint8, device=q.device) if zshape else None
    _repack(q.scheme, q.role, q.rows, q.cols, "packed", "canonical", q.scales, q.zeros, scales, zeros, q.device)
    return q.codes, scales, zeros


def from_canonical(scheme: str, role: str, rows: int, cols: int, codes: torch.Tensor, scales: torch.Tensor,
                   zeros: torch.Tensor | None = None) -> QTensor:
    """A QTensor (packed layout) from device tensors in the canonical layout; codes are
    used as they are, scales (and W4A16 zero-points) are rearranged on the device."""
    _on_device(codes.device)
    q = _alloc_q(scheme, role, rows, cols, codes.device)
    cb, sb, zb = layout_sizes(scheme, role, "canonical", rows, cols)
    for t, nb, what in ((codes, cb, "codes"), (scales, sb, "scales"), (zeros, zb, "zeros")):
        if t is None:
            if nb:
                raise ValueError(f"{scheme} needs {what}")
            continue
        if t.device != codes.device or not t.is_contiguous() or t.numel() * t.element_size() != nb:
            raise ValueError(f"{what} must be a contiguous tensor of {nb} bytes on {codes.device}")
    q.codes = codes.view(q.codes.dtype).reshape(q.codes.shape)
    _repack(scheme, role, rows, cols, "canonical", "packed", scales, zeros, q.scales, q.zeros, codes.device)
    return q


def from_numpy(q: dict, device) -> QTensor:
    """Upload a quantized tensor given as NumPy arrays in the canonical layout (MX
    exponents [rows, cols / 32], W4A16 scales and zero-points [rows, cols / 128]); the
    arrays go up as they are and pql_repack rearranges them into the packed layout on
    the device."""
    import numpy as np
    scheme = q["scheme"]

    def up(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(device)

    codes = up(np.asarray(q["codes"]).view(np.uint8))
    if scheme == "mxfp4_dual":      # one canonical buffer: fine [rows, cols/32], then coarse [rows, cols/512]
        off = _dual_coarse_offset(q["rows"], q["cols"])
        buf = np.zeros(off + 4 * q["rows"] * (q["cols"] // 512), np.uint8)
        fine = np.ascontiguousarray(q["scales"], np.uint8).reshape(-1)
        buf[:fine.size] = fine
        buf[off:] = np.ascontiguousarray(q["coarse"], np.float32).reshape(-1).view(np.uint8)
        scales = up(buf)
    else:
        scales = up(np.asarray(q["scales"]).view(np.uint8))
    zeros = up(np.asarray(q["zeros"]).view(np.uint8)) if q.get("zeros") is not None else None
    return from_canonical(scheme, q["role"], q["rows"], q["cols"], codes, scales, zeros)


def to_numpy(q: QTensor) -> dict:
    """Download a quantized tensor into NumPy arrays in the canonical layout: pql_repack
    rearranges the scales (and W4A16 zero-points) on the device, then the bytes come down
    as they are.  The packed device bytes of MX exponents are also returned, under
    "scales_packed"."""
    import numpy as np
    codes, scales, zeros = to_canonical(q)
    np_dtype = {torch.uint8: np.uint8, torch.int8: np.int8, torch.int32: np.uint32, torch.float32: np.float32,
                torch.bfloat16: np.uint16}

    def down(t):
        return t.contiguous().view(torch.uint8).cpu().numpy().view(np_dtype[t.dtype]).reshape(t.shape)

    out = {"scheme": q.scheme, "role": q.role, "rows": q.rows, "cols": q.cols,
           "codes": down(codes), "scales": down(scales), "zeros": None if zeros is None else down(zeros)}
    if q.scheme in MX_CHUNK:
        out["scales_packed"] = down(q.scales)
    if q.scheme == "mxfp4_dual":    # split the canonical buffer into its two levels
        buf, off = out["scales"], _dual_coarse_offset(q.rows, q.cols)
        out["scales"] = buf[:q.rows * (q.cols // 32)].reshape(q.rows, q.cols // 32).copy()
        out["coarse"] = buf[off:].view(np.float32).reshape(q.rows, q.cols // 512).copy()
        out["scales_packed"] = down(q.scales)
    return out


def qlinear_noalloc(x: torch.Tensor, w: QTensor, out: torch.Tensor, alpha: float = 1.0,
                    bias: torch.Tensor | None = None, act_scales: torch.Tensor | None = None) -> torch.Tensor:
    """``qlinear`` that allocates nothing, for code under HIP graph capture or loops that must
    not allocate: x is a 2-D bf16 [M, K] tensor (W4A16: contiguous), ``out`` the caller's bf16
    [M, N] output.  The activation's codes and scales live in the library's static device
    buffer (``noalloc_scratch_bytes()``); calls overlapping in time on one device race."""
    _check_qtensor(w, "w")
    if w.role != "weight":
        raise ValueError("w must be a quantized weight")
    x = _as_2d_bf16(x)
    M, K = x.shape
    if K != w.cols:
        raise ValueError(f"K mismatch: {K} vs {w.cols}")
    if x.device != w.device:
        raise ValueError(f"input on {x.device}, weight on {w.device}")
    _check_out(out, M, w.rows, w.device)
    if act_scales is not None:
        if w.scheme not in STATIC_SCHEMES:
            raise NotImplementedError(f"static activation scales are defined for {STATIC_SCHEMES} only")
        want = 1 if w.scheme == "fp8_tensor" else M * (K // 128)
        if act_scales.dtype != torch.float32 or not act_scales.is_contiguous() or act_scales.device != x.device \
                or act_scales.numel() != want:
            raise ValueError(f"act_scales must be {want} contiguous float32 values on the input's device")
    _check(lib().pql_qlinear_noalloc(_scheme(w.scheme), x.data_ptr(), M, K, x.stride(0), _ptr(act_scales),
                                     w.codes.data_ptr(), w.scales.data_ptr(), _ptr(w.zeros), w.rows, float(alpha),
                                     _bias_ptr(bias, w.rows, x.device), out.data_ptr(), out.stride(0),
                                     _stream(x.device)), "qlinear_noalloc")
    return out


def noalloc_scratch_bytes() -> int:
    return int(lib().pql_noalloc_scratch_bytes())


# ---------------------------------------------------------------- experts
MOE_SCORES = {"softmax": 0, "sigmoid": 1}
MOE_GROUP_SCORES = {"max": 0, "top2": 1}
MOE_SCHEMES = ("fp8_row", "fp8_block128")
_LOGIT_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


@dataclass
class MoePlan:
    """The assignments i = token * top_k + j of a batch, grouped by expert (include/pql.h,
    pql_moe_plan): int32 ``offsets`` [n_experts + 1], ``order`` [tokens * top_k] (position to
    assignment) and ``slots`` [tokens * top_k] (assignment to position, -1 for none)."""
    tokens: int
    top_k: int
    n_experts: int
    offsets: torch.Tensor
    order: torch.Tensor
    slots: torch.Tensor

    @property
    def device(self):
        return self.offsets.device


def _call(fn, what: str, device, *args) -> None:
    """One launch on the device's current stream, with that device current."""
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)   # current_stream() without building a Stream object
    if torch.cuda.current_device() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != PQL_OK:
        _check(status, what)


def _check_rows(t, name: str, rows: int, cols: int, device) -> int:
    """The row stride of a bf16 [rows, cols] operand with unit column stride on ``device``."""
    if type(t) is torch.Tensor and t.dtype is torch.bfloat16 and t.device == device and t.dim() == 2:
        (r, c), (ld, unit) = t.shape, t.stride()
        if r == rows and c == cols:
            if rows <= 1 and (unit == 1 or cols == 1):
                return cols
            if unit == 1 and ld >= cols:
                return ld
    _check_out(t, rows, cols, device, name)   # names what is wrong
    return t.stride(0) if rows > 1 else cols


def _check_vector(t, name: str, dtype, n: int, device) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the operands on {device}")


def _check_plan(plan, device, *fields) -> None:
    """A plan on ``device``, with the sizes of the ``fields`` that the caller hands to the library."""
    if not isinstance(plan, MoePlan):
        raise ValueError("plan must be a MoePlan")
    for f in fields:
        n = plan.n_experts + 1 if f == "offsets" else plan.tokens * plan.top_k
        _check_vector(getattr(plan, f), "plan." + f, torch.int32, n, device)


def _check_moe_scheme(scheme: str) -> None:
    if scheme not in MOE_SCHEMES:
        raise NotImplementedError(f"defined for the schemes {MOE_SCHEMES}, not {scheme!r}")


def moe_route(logits: torch.Tensor, top_k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
              n_groups: int = 1, top_groups: int = 1, group_score: str = "top2", renormalize: bool = True,
              scale: float = 1.0):
    """The ``top_k`` experts of each token, best first, and their weights: int32 and float32
    [T, top_k] from router logits [T, E] (fp32, bf16 or fp16; any row stride from E on).

    ``score``: "softmax" or "sigmoid".  ``bias`` (float32 [E]) is added to the scores for the
    choice alone.  With ``n_groups`` > 1 only the ``top_groups`` best groups of E / n_groups
    consecutive experts take part (``group_score``: a group's "max" choice, or the sum of its
    "top2").  Ties go to the lowest index.  ``renormalize`` divides the weights by their sum,
    ``scale`` multiplies them.  Unavailable experts (-inf) and broken rows (NaN, +inf): see
    include/pql.h, pql_moe_route."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _LOGIT_TYPES:
        raise ValueError("logits must be a float32, bfloat16 or float16 tensor")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-D with unit stride along the experts")
    if score not in MOE_SCORES:
        raise ValueError(f"unknown score {score!r}; supported: {sorted(MOE_SCORES)}")
    if group_score not in MOE_GROUP_SCORES:
        raise ValueError(f"unknown group score {group_score!r}; supported: {sorted(MOE_GROUP_SCORES)}")
    T, E = logits.shape
    device = logits.device
    if bias is not None:
        _check_vector(bias, "bias", torch.float32, E, device)
    _on_device(device)
    k = int(top_k)
    room = min(max(k, 0), E)   # a k outside 1 .. E is the library's to refuse, not the allocator's
    ids = torch.empty((T, room), dtype=torch.int32, device=device)
    weights = torch.empty((T, room), dtype=torch.float32, device=device)
    ld = logits.stride(0) if T > 1 else E
    _call(lib().pql_moe_route, "moe_route", device, MOE_SCORES[score], _LOGIT_TYPES[logits.dtype], logits.data_ptr(), T,
          E, ld, _ptr(bias), k, n_groups, top_groups, MOE_GROUP_SCORES[group_score], bool(renormalize), scale,
          ids.data_ptr(), weights.data_ptr())
    return ids, weights


@functools.lru_cache(maxsize=4096)
def _plan_workspace(T: int, k: int, n_experts: int) -> int:
    wsb = ctypes.c_size_t()
    _check(lib().pql_moe_plan_workspace(T, k, n_experts, ctypes.byref(wsb)), "moe_plan")
    return wsb.value


def moe_plan(ids: torch.Tensor, n_experts: int, workspace: torch.Tensor | None = None) -> MoePlan:
    """Group the assignments of int32 ids [T, top_k] by expert (stable).  Ids outside
    0 .. n_experts - 1 take no part: experts held elsewhere, or none."""
    if not isinstance(ids, torch.Tensor) or ids.dtype != torch.int32 or ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 [T, top_k] tensor")
    T, k = ids.shape
    device = ids.device
    _on_device(device)
    wsb = _plan_workspace(T, k, n_experts)
    P = T * k
    ws_at = (2 * P + n_experts + 1 + 3) // 4 * 4                 # one allocation for the plan and the workspace
    buf = torch.empty(ws_at + (0 if workspace is not None else wsb // 4), dtype=torch.int32, device=device)
    if workspace is None:
        ws, wsn = buf.data_ptr() + 4 * ws_at, wsb
    else:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the ids' device")
        ws, wsn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    order, slots, offsets, _ = buf.split((P, P, n_experts + 1, buf.numel() - 2 * P - n_experts - 1))
    plan = MoePlan(T, k, n_experts, offsets, order, slots)
    at = buf.data_ptr()
    _call(lib().pql_moe_plan, "moe_plan", device, ids.data_ptr(), T, k, n_experts, at + 8 * P, at, at + 4 * P, ws, wsn)
    return plan


def moe_qgemm(a: QTensor, w: QTensor, plan: MoePlan, gather: bool = False,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """Each expert's product of its rows with its own weight: bf16 [T * top_k, N] in expert
    order (rows from plan.offsets[-1] on are left as they were).

    ``w`` is the quantized [n_experts * N, K] stack of the experts' weights.  ``gather``: ``a``
    has one row per token, which its assignments share; otherwise one row per position."""
    _check_qtensor(a, "a")
    _check_qtensor(w, "w")
    _check_plan(plan, w.device, "offsets", "order")
    if a.role != "activation" or w.role != "weight":
        raise ValueError("moe_qgemm takes a quantized activation and a quantized weight")
    if a.scheme != w.scheme:
        raise ValueError("activation and weight schemes differ")
    _check_moe_scheme(w.scheme)
    if a.device != w.device:
        raise ValueError(f"activation on {a.device}, weight on {w.device}")
    if a.cols != w.cols:
        raise ValueError(f"K mismatch: {a.cols} vs {w.cols}")
    if w.rows % plan.n_experts:
        raise ValueError(f"{w.rows} weight rows do not divide into {plan.n_experts} experts")
    P, N = plan.tokens * plan.top_k, w.rows // plan.n_experts
    if a.rows != (plan.tokens if gather else P):
        raise ValueError(f"expected an activation of {plan.tokens if gather else P} rows, got {a.rows}")
    device = w.device
    if out is None:
        out, ldc = torch.empty((P, N), dtype=torch.bfloat16, device=device), N
    else:
        ldc = _check_rows(out, "out", P, N, device)
    _on_device(device)
    _call(lib().pql_moe_qgemm, "moe_qgemm", device, SCHEMES[w.scheme], a.codes.data_ptr(), a.scales.data_ptr(), a.rows,
          gather, w.codes.data_ptr(), w.scales.data_ptr(), plan.offsets.data_ptr(), plan.order.data_ptr(), plan.tokens,
          plan.top_k, plan.n_experts, N, w.cols, out.data_ptr(), ldc)
    return out


def moe_kernel_name(scheme, T: int, top_k: int, n_experts: int, N: int, K: int, gather: bool = False) -> str:
    return lib().pql_moe_kernel_name(_scheme(scheme), int(gather), T, top_k, n_experts, N, K).decode()


def swiglu_quantize(x: torch.Tensor, scheme: str, plan: MoePlan | None = None, out: QTensor | None = None) -> QTensor:
    """silu(gate) * up of a bf16 [rows, 2 F] tensor (gate half first), quantized as a [rows, F]
    activation in the same pass.  With ``plan`` the rows from plan.offsets[-1] on are left as
    they were.  ``out`` reuses the buffers of an earlier result of the same shape."""
    x = _as_2d_bf16(x)
    _check_moe_scheme(scheme)
    rows, cols = x.shape[0], x.shape[1] // 2
    if x.shape[1] != 2 * cols:
        raise ValueError("expected gate and up halves of equal width")
    if plan is not None:
        _check_plan(plan, x.device, "offsets")
        if rows != plan.tokens * plan.top_k:
            raise ValueError(f"expected the plan's {plan.tokens * plan.top_k} rows, got {rows}")
    if out is not None:
        _check_qtensor(out, "out")
        if (out.scheme, out.role, out.rows, out.cols) != (scheme, "activation", rows, cols):
            raise ValueError("out does not match the scheme, role and shape")
        if out.device != x.device:
            raise ValueError(f"out is on {out.device}, x on {x.device}")
        q = out
    else:
        # as _alloc_q lays them out; a width that does not divide is the library's to refuse
        codes = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
        scales = torch.empty((rows,) if scheme == "fp8_row" else (rows, cols // 128), dtype=torch.float32, device=x.device)
        q = QTensor(scheme, "activation", rows, cols, codes, scales)
    _call(lib().pql_swiglu_quantize, "swiglu_quantize", x.device, SCHEMES[scheme], x.data_ptr(), rows, cols,
          x.stride(0) if rows > 1 else 2 * cols, None if plan is None else plan.offsets.data_ptr() + 4 * plan.n_experts,
          q.codes.data_ptr(), q.scales.data_ptr())
    return q


def moe_combine(y: torch.Tensor, plan: MoePlan, weights: torch.Tensor, add: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """Back to tokens: out[t] = add[t] + sum_j weights[t, j] * y[slot of (t, j)], bf16 [T, N],
    summed in fp32.  ``add`` (a shared expert's output, a residual) may be ``out`` itself."""
    _check_plan(plan, None)
    T, P, device = plan.tokens, plan.tokens * plan.top_k, plan.slots.device
    _check_plan(plan, device, "slots")
    if not isinstance(y, torch.Tensor) or y.dim() != 2:
        raise ValueError("y must be a 2-D tensor")
    N = y.shape[1]
    ldy = _check_rows(y, "y", P, N, device)
    _check_vector(weights, "weights", torch.float32, P, device)
    if weights.dim() != 2 or weights.shape[0] != T:
        raise ValueError(f"weights must be [{T}, {plan.top_k}], not {tuple(weights.shape)}")
    ldadd = N if add is None else _check_rows(add, "add", T, N, device)
    if out is None:
        out, ldo = torch.empty((T, N), dtype=torch.bfloat16, device=device), N
    else:
        ldo = _check_rows(out, "out", T, N, device)
    _on_device(device)
    _call(lib().pql_moe_combine, "moe_combine", device, y.data_ptr(), P, ldy, plan.slots.data_ptr(), weights.data_ptr(),
          T, plan.top_k, N, _ptr(add), ldadd, out.data_ptr(), ldo)
    return out


def moe_mlp(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w_in: QTensor, w_out: QTensor,
            n_experts: int, add: torch.Tensor | None = None) -> torch.Tensor:
    """A layer of gated experts on bf16 x [T, K]: plan, quantize, product with ``w_in``
    ([n_experts * 2 F, K]: gate rows, then up rows, of each expert), gated activation with its
    quantization, product with ``w_out`` ([n_experts * N, F]), weighted sum to [T, N]."""
    x = _as_2d_bf16(x)
    _check_qtensor(w_in, "w_in")
    _check_qtensor(w_out, "w_out")
    _check_moe_scheme(w_in.scheme)
    if w_in.scheme != w_out.scheme:
        raise ValueError("the two weights' schemes differ")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
        raise ValueError(f"ids must be [{x.shape[0]}, top_k]")
    with torch.cuda.device(x.device):
        plan = moe_plan(ids, n_experts)
        h = moe_qgemm(quantize(x, w_in.scheme), w_in, plan, gather=True)
        y = moe_qgemm(swiglu_quantize(h, w_in.scheme, plan), w_out, plan)
        return moe_combine(y, plan, weights, add=add)


from .kv import (KV_HEAD_DIMS, KV_SCHEMES, ROPE_LAYOUTS, KVCache, Rope, kv_append, kv_attention,   # noqa: E402,F401
                 kv_attention_workspace, kv_cache, kv_kernel_name, kv_read, kv_sizes, kv_slots, rope, rope_freqs)
