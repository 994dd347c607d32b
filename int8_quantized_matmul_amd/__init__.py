"""LLM.int8() mixed-precision decomposed int8 matmul for AMD MI355X (gfx950).

Thin Python binding over the C ABI of libi8mm.so (include/i8mm.h). Each
function checks tensor placement, dtype and shape, allocates outputs with
torch on the tensors' device, and passes raw device pointers plus torch's
current HIP stream to the library. Every step of the computation runs in the
library's HIP kernels; there is no CPU or PyTorch fallback: without the
built library the first call raises ImportError.

Page tags: [DIGEST] "LLM.int8(): 8-bit Matrix Multiplication for Transformers
at Scale" (paper-graph-ui digest), "The Full LLM.int8() Algorithm".
"""

from __future__ import annotations

import array
import ctypes
import operator
from typing import Dict, Optional, Sequence, Tuple

import torch

from . import _native

__all__ = [
    "quantize_colwise_weights",
    "detect_outlier_cols",
    "quantize_rowwise",
    "int8_mixed_matmul",
    "outlier_matmul",
    "int8_gemm_i32",
    "forward",
    "forward_tensorwise",
    "forward_zeropoint",
    "forward_noalloc",
    "forward_decode",
    "forward_inline_quant",
    "INLINE_QUANT_MIN_ROWS",
    "NOALLOC_SCRATCH_BYTES",
    "pack_fp16_weights",
    "fp16_gemm",
    "quantize_tensorwise",
    "quantize_weights_tensorwise",
    "quantize_rowwise_zeropoint",
    "quantize_colwise_weights_zeropoint",
    "zeropoint_matmul",
    "SCHEMES",
    "quantize_weights",
    "variant_forward",
    "layer_norm",
    "layer_norm_backward",
    "lora_forward",
    "lora_backward",
    "LORA_MAX_RANK",
    "clip_grad_norm",
    "forward_workspace",
    "forward_workspace_views",
    "x_o_stride",
    "weight_panels_shape",
    "panels_to_rows",
    "version",
    "library_path",
    "I8MMError",
]


class _LazyLib:
    """Loads libi8mm.so on first use, so that the build module can be imported
    before the library exists. Any call without the library raises ImportError."""

    def __getattr__(self, name):
        return getattr(_native.load(), name)


_lib = _LazyLib()

# Bytes of the forward workspace's leading accumulator (I8MM_FORWARD_ACC_BYTES).
ACC_BYTES = _native.header_define("I8MM_FORWARD_ACC_BYTES")
# Bytes of the static device scratch behind forward_noalloc (I8MM_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = _native.header_define("I8MM_NOALLOC_SCRATCH_BYTES")
# Fewest rows forward_inline_quant takes (I8MM_INLINE_QUANT_MIN_ROWS).
INLINE_QUANT_MIN_ROWS = _native.header_define("I8MM_INLINE_QUANT_MIN_ROWS")
# Largest rank of the adapters (I8MM_LORA_MAX_RANK).
LORA_MAX_RANK = _native.header_define("I8MM_LORA_MAX_RANK")


class I8MMError(RuntimeError):
    """A libi8mm entry point returned an error status."""


def _check(status: int, what: str) -> None:
    if status != 0:
        msg = _lib.i8mm_status_string(status).decode()
        raise I8MMError(f"{what}: {msg} (status {status})")


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    return t.data_ptr()


def x_o_stride(h: int) -> int:
    """Row stride (elements) of the gathered outlier columns X_O: room for |O| = h."""
    return (h + 31) // 32 * 32


def weight_panels_shape(h: int, o: int) -> Tuple[int, int, int]:
    """Shape of the quantised weights in the library's panel layout: the code
    W_i8[k, j] sits at Wq[k // 64, j, k % 64] (h / 64 panels of 64 reduction
    rows, each column's 64 codes contiguous)."""
    if h % 64 != 0:
        raise ValueError(f"h must be a multiple of 64 (got {h})")
    return (h // 64, o, 64)


def panels_to_rows(Wq: torch.Tensor) -> torch.Tensor:
    """The codes of a panel-layout Wq as W_i8 transposed, [o, h] (a copy, for
    inspection and tests; the products read the panel layout directly)."""
    p, o, _ = Wq.shape
    return Wq.permute(1, 0, 2).reshape(o, p * 64)


def version() -> str:
    return _lib.i8mm_version().decode()


def library_path() -> str:
    return _native.loaded_path()


def quantize_colwise_weights(W: torch.Tensor, Wq: Optional[torch.Tensor] = None,
                             c_w: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Load-time conversion: W fp16 [h, o] -> (Wq int8 [h/64, o, 64] panel
    layout, c_w fp32 [o])."""
    h, o = W.shape
    shape = weight_panels_shape(h, o)
    if Wq is None:
        Wq = torch.empty(shape, dtype=torch.int8, device=W.device)
    if c_w is None:
        c_w = torch.empty((o,), dtype=torch.float32, device=W.device)
    st = _lib.i8mm_quantize_colwise_weights(
        _dev(W, "W", torch.float16), h, o, _dev(Wq, "Wq", torch.int8, shape),
        _dev(c_w, "c_w", torch.float32, (o,)), _stream(W))
    _check(st, "quantize_colwise_weights")
    return Wq, c_w


def detect_outlier_cols(X: torch.Tensor, alpha: float = 6.0, mask: Optional[torch.Tensor] = None,
                        idx: Optional[torch.Tensor] = None, n_out: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """O = {j : max_i |X_ij| >= alpha} as (mask int32 view of uint32 [ceil(h/32)],
    idx int32 [h] (first |O| valid, ascending), n_out int32 [1]) on the device."""
    s, h = X.shape
    nw = (h + 31) // 32
    dev = X.device
    if mask is None:
        mask = torch.empty((nw,), dtype=torch.int32, device=dev)
    if idx is None:
        idx = torch.empty((h,), dtype=torch.int32, device=dev)
    if n_out is None:
        n_out = torch.empty((1,), dtype=torch.int32, device=dev)
    st = _lib.i8mm_detect_outlier_cols(
        _dev(X, "X", torch.float16), s, h, float(alpha), _dev(mask, "mask", torch.int32, (nw,)),
        _dev(idx, "idx", torch.int32, (h,)), _dev(n_out, "n_out", torch.int32, (1,)), _stream(X))
    _check(st, "detect_outlier_cols")
    return mask, idx, n_out


def quantize_rowwise(X: torch.Tensor, mask: torch.Tensor, idx: torch.Tensor, n_out: torch.Tensor,
                     Xq: Optional[torch.Tensor] = None, c_x: Optional[torch.Tensor] = None,
                     X_O: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Row-wise absmax int8 over the non-outlier columns: (Xq int8 [s, h] with
    O columns 0, c_x fp32 [s], X_O fp16 [s, x_o_stride(h)] gathered outliers)."""
    s, h = X.shape
    dev = X.device
    ldo = x_o_stride(h) if X_O is None else X_O.shape[1]
    if Xq is None:
        Xq = torch.empty((s, h), dtype=torch.int8, device=dev)
    if c_x is None:
        c_x = torch.empty((s,), dtype=torch.float32, device=dev)
    if X_O is None:
        X_O = torch.empty((s, ldo), dtype=torch.float16, device=dev)
    st = _lib.i8mm_quantize_rowwise(
        _dev(X, "X", torch.float16), s, h, _dev(mask, "mask", torch.int32),
        _dev(idx, "idx", torch.int32), _dev(n_out, "n_out", torch.int32, (1,)),
        _dev(Xq, "Xq", torch.int8, (s, h)), _dev(c_x, "c_x", torch.float32, (s,)),
        _dev(X_O, "X_O", torch.float16, (s, ldo)), ldo, _stream(X))
    _check(st, "quantize_rowwise")
    return Xq, c_x, X_O


def _weights_ptr(W: Optional[torch.Tensor], h: int, o: int) -> Optional[int]:
    """Pointer of the resident fp16 W, or None (outlier rows rebuilt from Wq / c_w)."""
    return None if W is None else _dev(W, "W", torch.float16, (h, o))


def _bias_ptr(bias: Optional[torch.Tensor], o: int) -> Optional[int]:
    """Pointer of the fp16 layer bias [o], or None (no bias)."""
    return None if bias is None else _dev(bias, "bias", torch.float16, (o,))


def int8_mixed_matmul(Xq: torch.Tensor, c_x: torch.Tensor, X_O: torch.Tensor, idx: torch.Tensor,
                      n_out: torch.Tensor, Wq: torch.Tensor, c_w: torch.Tensor, W: Optional[torch.Tensor],
                      C: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C fp16 [s, o] = fp16(C_i32 / (c_x ⊗ c_w) + X_O W[idx, :] [+ bias]). With W
    None no fp16 copy of the weights is needed: W[idx, :] is rebuilt as
    fp16(W_i8 * fl32(1 / c_w)). bias: fp16 [o] or None."""
    s, h = Xq.shape
    o = Wq.shape[1]
    if C is None:
        C = torch.empty((s, o), dtype=torch.float16, device=Xq.device)
    st = _lib.i8mm_int8_mixed_matmul(
        _dev(Xq, "Xq", torch.int8), _dev(c_x, "c_x", torch.float32, (s,)),
        _dev(X_O, "X_O", torch.float16), X_O.shape[1], _dev(idx, "idx", torch.int32),
        _dev(n_out, "n_out", torch.int32, (1,)), _dev(Wq, "Wq", torch.int8, weight_panels_shape(h, o)),
        _dev(c_w, "c_w", torch.float32, (o,)), _weights_ptr(W, h, o), _bias_ptr(bias, o),
        s, h, o, _dev(C, "C", torch.float16, (s, o)), _stream(Xq))
    _check(st, "int8_mixed_matmul")
    return C


def outlier_matmul(X_O: torch.Tensor, idx: torch.Tensor, n_out: torch.Tensor, W: torch.Tensor,
                   C_O: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C_O fp32 [s, o] = X_O W[idx, :] (the fp16 outlier product alone)."""
    s, ldo = X_O.shape
    h, o = W.shape
    if C_O is None:
        C_O = torch.empty((s, o), dtype=torch.float32, device=X_O.device)
    st = _lib.i8mm_outlier_matmul(
        _dev(X_O, "X_O", torch.float16), ldo, _dev(idx, "idx", torch.int32),
        _dev(n_out, "n_out", torch.int32, (1,)), _dev(W, "W", torch.float16), s, h, o,
        _dev(C_O, "C_O", torch.float32, (s, o)), _stream(X_O))
    _check(st, "outlier_matmul")
    return C_O


def int8_gemm_i32(Xq: torch.Tensor, Wq: torch.Tensor, C: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C_i32 int32 [s, o] = Xq W_i8 exactly (same main loop as the mixed product)."""
    s, h = Xq.shape
    o = Wq.shape[1]
    if C is None:
        C = torch.empty((s, o), dtype=torch.int32, device=Xq.device)
    st = _lib.i8mm_int8_gemm_i32(
        _dev(Xq, "Xq", torch.int8), _dev(Wq, "Wq", torch.int8, weight_panels_shape(h, o)), s, h, o,
        _dev(C, "C", torch.int32, (s, o)), _stream(Xq))
    _check(st, "int8_gemm_i32")
    return C


def pack_fp16_weights(W: torch.Tensor, Wp: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Load-time packing for the dense fp16 baseline: W fp16 [h, o] -> Wp fp16
    [h/32, o, 32] (W[k, j] at Wp[k // 32, j, k % 32])."""
    h, o = W.shape
    if h % 32 != 0:
        raise ValueError(f"h must be a multiple of 64 (got {h})")
    shape = (h // 32, o, 32)
    if Wp is None:
        Wp = torch.empty(shape, dtype=torch.float16, device=W.device)
    st = _lib.i8mm_pack_fp16_weights(_dev(W, "W", torch.float16), h, o, _dev(Wp, "Wp", torch.float16, shape),
                                     _stream(W))
    _check(st, "pack_fp16_weights")
    return Wp


def fp16_gemm(X: torch.Tensor, Wp: torch.Tensor, C: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dense fp16 baseline C fp16 [s, o] = fp16(X W) (fp32 accumulation) from packed Wp."""
    s, h = X.shape
    o = Wp.shape[1]
    if C is None:
        C = torch.empty((s, o), dtype=torch.float16, device=X.device)
    st = _lib.i8mm_fp16_gemm(_dev(X, "X", torch.float16), _dev(Wp, "Wp", torch.float16, (h // 32, o, 32)),
                             s, h, o, _dev(C, "C", torch.float16, (s, o)), _stream(X))
    _check(st, "fp16_gemm")
    return C


# ---------------------------------------------------------------- quantiser variants (Table 1)

def quantize_weights_tensorwise(W: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Tensor-wise absmax for W: (Wq int8 panels, c_w fp32 [o] all equal to the
    one constant 127 / max |W|)."""
    h, o = W.shape
    Wq = torch.empty(weight_panels_shape(h, o), dtype=torch.int8, device=W.device)
    c_w = torch.empty((o,), dtype=torch.float32, device=W.device)
    st = _lib.i8mm_quantize_weights_tensorwise(_dev(W, "W", torch.float16), h, o, _dev(Wq, "Wq", torch.int8),
                                               _dev(c_w, "c_w", torch.float32), _stream(W))
    _check(st, "quantize_weights_tensorwise")
    return Wq, c_w


def quantize_tensorwise(X: torch.Tensor, mask: torch.Tensor, idx: torch.Tensor, n_out: torch.Tensor
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Tensor-wise absmax for X over the non-outlier columns: (Xq, c_x [s] all
    equal, X_O), laid out as by quantize_rowwise."""
    s, h = X.shape
    dev = X.device
    ldo = x_o_stride(h)
    Xq = torch.empty((s, h), dtype=torch.int8, device=dev)
    c_x = torch.empty((s,), dtype=torch.float32, device=dev)
    X_O = torch.empty((s, ldo), dtype=torch.float16, device=dev)
    st = _lib.i8mm_quantize_tensorwise(
        _dev(X, "X", torch.float16), s, h, _dev(mask, "mask", torch.int32), _dev(idx, "idx", torch.int32),
        _dev(n_out, "n_out", torch.int32, (1,)), _dev(Xq, "Xq", torch.int8), _dev(c_x, "c_x", torch.float32),
        _dev(X_O, "X_O", torch.float16), ldo, _stream(X))
    _check(st, "quantize_tensorwise")
    return Xq, c_x, X_O


def quantize_colwise_weights_zeropoint(W: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor,
                                                                 torch.Tensor]:
    """Zeropoint quantisation of the columns of W (load time): (Wq int8 panels,
    nd_w fp32 [o], zp_w int32 [o], colsum_w int32 [o])."""
    h, o = W.shape
    dev = W.device
    Wq = torch.empty(weight_panels_shape(h, o), dtype=torch.int8, device=dev)
    nd_w = torch.empty((o,), dtype=torch.float32, device=dev)
    zp_w = torch.empty((o,), dtype=torch.int32, device=dev)
    cs_w = torch.empty((o,), dtype=torch.int32, device=dev)
    st = _lib.i8mm_quantize_colwise_weights_zeropoint(
        _dev(W, "W", torch.float16), h, o, _dev(Wq, "Wq", torch.int8), _dev(nd_w, "nd_w", torch.float32),
        _dev(zp_w, "zp_w", torch.int32), _dev(cs_w, "colsum_w", torch.int32), _stream(W))
    _check(st, "quantize_colwise_weights_zeropoint")
    return Wq, nd_w, zp_w, cs_w


def quantize_rowwise_zeropoint(X: torch.Tensor, mask: torch.Tensor, idx: torch.Tensor, n_out: torch.Tensor
                               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Zeropoint quantisation of the rows of X over the non-outlier columns:
    (Xq int8 [s, h], nd_x fp32 [s], zp_x int32 [s], rowsum_x int32 [s], X_O)."""
    s, h = X.shape
    dev = X.device
    ldo = x_o_stride(h)
    Xq = torch.empty((s, h), dtype=torch.int8, device=dev)
    nd_x = torch.empty((s,), dtype=torch.float32, device=dev)
    zp_x = torch.empty((s,), dtype=torch.int32, device=dev)
    rs_x = torch.empty((s,), dtype=torch.int32, device=dev)
    X_O = torch.empty((s, ldo), dtype=torch.float16, device=dev)
    st = _lib.i8mm_quantize_rowwise_zeropoint(
        _dev(X, "X", torch.float16), s, h, _dev(mask, "mask", torch.int32), _dev(idx, "idx", torch.int32),
        _dev(n_out, "n_out", torch.int32, (1,)), _dev(Xq, "Xq", torch.int8), _dev(nd_x, "nd_x", torch.float32),
        _dev(zp_x, "zp_x", torch.int32), _dev(rs_x, "rowsum_x", torch.int32), _dev(X_O, "X_O", torch.float16), ldo,
        _stream(X))
    _check(st, "quantize_rowwise_zeropoint")
    return Xq, nd_x, zp_x, rs_x, X_O


def zeropoint_matmul(Xq: torch.Tensor, nd_x: torch.Tensor, zp_x: torch.Tensor, rowsum_x: torch.Tensor,
                     X_O: torch.Tensor, idx: torch.Tensor, n_out: torch.Tensor, Wq: torch.Tensor,
                     nd_w: torch.Tensor, zp_w: torch.Tensor, colsum_w: torch.Tensor, W: torch.Tensor,
                     C: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C fp16 [s, o] = fp16(C' / (nd_x ⊗ nd_w) + X_O W[idx, :] [+ bias]), C' the
    product of the zero-point-shifted codes over the non-outlier columns."""
    s, h = Xq.shape
    o = Wq.shape[1]
    if C is None:
        C = torch.empty((s, o), dtype=torch.float16, device=Xq.device)
    st = _lib.i8mm_zeropoint_matmul(
        _dev(Xq, "Xq", torch.int8), _dev(nd_x, "nd_x", torch.float32, (s,)), _dev(zp_x, "zp_x", torch.int32, (s,)),
        _dev(rowsum_x, "rowsum_x", torch.int32, (s,)), _dev(X_O, "X_O", torch.float16), X_O.shape[1],
        _dev(idx, "idx", torch.int32), _dev(n_out, "n_out", torch.int32, (1,)),
        _dev(Wq, "Wq", torch.int8, weight_panels_shape(h, o)), _dev(nd_w, "nd_w", torch.float32, (o,)),
        _dev(zp_w, "zp_w", torch.int32, (o,)), _dev(colsum_w, "colsum_w", torch.int32, (o,)),
        _dev(W, "W", torch.float16, (h, o)), _bias_ptr(bias, o), s, h, o, _dev(C, "C", torch.float16, (s, o)),
        _stream(Xq))
    _check(st, "zeropoint_matmul")
    return C


SCHEMES = ("tensor", "row", "vector", "zeropoint")


def quantize_weights(W: torch.Tensor, scheme: str) -> Tuple[torch.Tensor, ...]:
    """Load-time weights for one quantiser scheme: (Wq, c_w) for "tensor" and
    "row" (one constant) and "vector" (per column); (Wq, nd_w, zp_w, colsum_w)
    for "zeropoint"."""
    if scheme in ("tensor", "row"):
        return quantize_weights_tensorwise(W)
    if scheme == "vector":
        return quantize_colwise_weights(W)
    if scheme == "zeropoint":
        return quantize_colwise_weights_zeropoint(W)
    raise ValueError(f"unknown scheme {scheme!r}; one of {SCHEMES}")


def variant_forward(X: torch.Tensor, qw: Tuple[torch.Tensor, ...], W: torch.Tensor, scheme: str,
                    alpha: float = 6.0, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One forward of a quantiser scheme (Table 1) as a sequence of C-ABI
    calls: detection at alpha (inf: no decomposition), the scheme's row
    quantiser, then its product. qw comes from quantize_weights(W, scheme)."""
    mask, idx, n_out = detect_outlier_cols(X, alpha)
    if scheme == "zeropoint":
        Xq, nd_x, zp_x, rs_x, X_O = quantize_rowwise_zeropoint(X, mask, idx, n_out)
        Wq, nd_w, zp_w, cs_w = qw
        return zeropoint_matmul(Xq, nd_x, zp_x, rs_x, X_O, idx, n_out, Wq, nd_w, zp_w, cs_w, W, bias=bias)
    if scheme == "tensor":
        Xq, c_x, X_O = quantize_tensorwise(X, mask, idx, n_out)
    elif scheme in ("row", "vector"):
        Xq, c_x, X_O = quantize_rowwise(X, mask, idx, n_out)
    else:
        raise ValueError(f"unknown scheme {scheme!r}; one of {SCHEMES}")
    Wq, c_w = qw
    return int8_mixed_matmul(Xq, c_x, X_O, idx, n_out, Wq, c_w, W, bias=bias)


def forward_workspace(s: int, h: int, device, zeropoint: bool = False) -> torch.Tensor:
    """A zero-filled device workspace (uint8) for forward() and
    forward_tensorwise() (zeropoint=True: sized for forward_zeropoint(),
    which also serves the others). Its leading accumulator must start at
    zero; every one-call forward leaves it zero again."""
    n = (_lib.i8mm_forward_zeropoint_workspace_bytes if zeropoint else _lib.i8mm_forward_workspace_bytes)(s, h)
    if n == 0:
        raise I8MMError(f"invalid shape for the forward workspace: s={s}, h={h}")
    return torch.zeros((n,), dtype=torch.uint8, device=device)


def forward_workspace_views(workspace: torch.Tensor, s: int, h: int) -> Dict[str, torch.Tensor]:
    """Typed views of the intermediates that forward() leaves in its workspace."""
    offs = (ctypes.c_size_t * 7)()
    ldo = ctypes.c_int64()
    _check(_lib.i8mm_forward_workspace_layout(s, h, offs, ctypes.byref(ldo)), "forward_workspace_layout")
    nw = (h + 31) // 32
    l = ldo.value

    def view(i, nbytes, dtype, shape):
        return workspace[offs[i]:offs[i] + nbytes].view(dtype).view(shape)

    acc_words = ACC_BYTES // 4
    return {
        "acc": view(0, ACC_BYTES, torch.int32, (acc_words,)),
        "mask": view(1, 4 * nw, torch.int32, (nw,)),
        "idx": view(2, 4 * h, torch.int32, (h,)),
        "n_out": view(3, 4, torch.int32, (1,)),
        "Xq": view(4, s * h, torch.int8, (s, h)),
        "c_x": view(5, 4 * s, torch.float32, (s,)),
        "X_O": view(6, 2 * s * l, torch.float16, (s, l)),
    }


def forward(X: torch.Tensor, Wq: torch.Tensor, c_w: torch.Tensor, W: Optional[torch.Tensor],
            alpha: float = 6.0, workspace: Optional[torch.Tensor] = None,
            C: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The whole per-forward path: detect -> quantise rows -> decomposed product.
    W is the resident fp16 weight matrix, or None (outlier rows rebuilt from
    Wq / c_w); bias is the fp16 layer bias [o], or None."""
    s, h = X.shape
    o = Wq.shape[1]
    if workspace is None:
        workspace = forward_workspace(s, h, X.device)
    if C is None:
        C = torch.empty((s, o), dtype=torch.float16, device=X.device)
    need = _lib.i8mm_forward_workspace_bytes(s, h)
    if workspace.numel() < need or workspace.dtype != torch.uint8:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    st = _lib.i8mm_forward(
        _dev(X, "X", torch.float16), s, h, o, float(alpha), _dev(Wq, "Wq", torch.int8, weight_panels_shape(h, o)),
        _dev(c_w, "c_w", torch.float32, (o,)), _weights_ptr(W, h, o), _bias_ptr(bias, o),
        _dev(workspace, "workspace", torch.uint8), _dev(C, "C", torch.float16, (s, o)), _stream(X))
    _check(st, "forward")
    return C


def forward_tensorwise(X: torch.Tensor, Wq: torch.Tensor, c_w: torch.Tensor, W: Optional[torch.Tensor],
                       alpha: float = 6.0, workspace: Optional[torch.Tensor] = None,
                       C: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """forward() with tensor-wise absmax for X (one constant over the columns
    not in O): Table 1's tensor-wise scheme with weights from
    quantize_weights_tensorwise (or quantize_weights(W, "tensor"))."""
    s, h = X.shape
    o = Wq.shape[1]
    if workspace is None:
        workspace = forward_workspace(s, h, X.device)
    if C is None:
        C = torch.empty((s, o), dtype=torch.float16, device=X.device)
    need = _lib.i8mm_forward_workspace_bytes(s, h)
    if workspace.numel() < need or workspace.dtype != torch.uint8:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    st = _lib.i8mm_forward_tensorwise(
        _dev(X, "X", torch.float16), s, h, o, float(alpha), _dev(Wq, "Wq", torch.int8, weight_panels_shape(h, o)),
        _dev(c_w, "c_w", torch.float32, (o,)), _weights_ptr(W, h, o), _bias_ptr(bias, o),
        _dev(workspace, "workspace", torch.uint8), _dev(C, "C", torch.float16, (s, o)), _stream(X))
    _check(st, "forward_tensorwise")
    return C


def forward_zeropoint(X: torch.Tensor, qw: Tuple[torch.Tensor, ...], W: torch.Tensor, alpha: float = 6.0,
                      workspace: Optional[torch.Tensor] = None, C: Optional[torch.Tensor] = None,
                      bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The one-call forward of the zeropoint vector-wise scheme: qw = (Wq,
    nd_w, zp_w, colsum_w) from quantize_weights(W, "zeropoint"); W (fp16) is
    required for the outlier rows. The workspace must come from
    forward_workspace(s, h, device, zeropoint=True) or be as large."""
    s, h = X.shape
    Wq, nd_w, zp_w, cs_w = qw
    o = Wq.shape[1]
    if workspace is None:
        workspace = forward_workspace(s, h, X.device, zeropoint=True)
    if C is None:
        C = torch.empty((s, o), dtype=torch.float16, device=X.device)
    need = _lib.i8mm_forward_zeropoint_workspace_bytes(s, h)
    if workspace.numel() < need or workspace.dtype != torch.uint8:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    st = _lib.i8mm_forward_zeropoint(
        _dev(X, "X", torch.float16), s, h, o, float(alpha), _dev(Wq, "Wq", torch.int8, weight_panels_shape(h, o)),
        _dev(nd_w, "nd_w", torch.float32, (o,)), _dev(zp_w, "zp_w", torch.int32, (o,)),
        _dev(cs_w, "colsum_w", torch.int32, (o,)), _dev(W, "W", torch.float16, (h, o)), _bias_ptr(bias, o),
        _dev(workspace, "workspace", torch.uint8), _dev(C, "C", torch.float16, (s, o)), _stream(X))
    _check(st, "forward_zeropoint")
    return C


def forward_decode(X: torch.Tensor, Wq: torch.Tensor, c_w: torch.Tensor, W: Optional[torch.Tensor],
                   alpha: float = 6.0, workspace: Optional[torch.Tensor] = None,
                   C: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """forward() in one kernel launch for s <= 16 rows (i8mm_forward_decode);
    the workspace receives the same intermediates as forward()'s."""
    s, h = X.shape
    o = Wq.shape[1]
    if workspace is None:
        workspace = forward_workspace(s, h, X.device)
    if C is None:
        C = torch.empty((s, o), dtype=torch.float16, device=X.device)
    need = _lib.i8mm_forward_workspace_bytes(s, h)
    if workspace.numel() < need or workspace.dtype != torch.uint8:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    st = _lib.i8mm_forward_decode(
        _dev(X, "X", torch.float16), s, h, o, float(alpha), _dev(Wq, "Wq", torch.int8, weight_panels_shape(h, o)),
        _dev(c_w, "c_w", torch.float32, (o,)), _weights_ptr(W, h, o), _bias_ptr(bias, o),
        _dev(workspace, "workspace", torch.uint8), _dev(C, "C", torch.float16, (s, o)), _stream(X))
    _check(st, "forward_decode")
    return C


def forward_inline_quant(X: torch.Tensor, Wq: torch.Tensor, c_w: torch.Tensor, W: Optional[torch.Tensor],
                         alpha: float = 6.0, workspace: Optional[torch.Tensor] = None,
                         C: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """forward() with the int8 codes of X made inside the product kernel
    and never stored (i8mm_forward_inline_quant; s >= INLINE_QUANT_MIN_ROWS).
    The workspace receives the outlier set, c_x and X_O; its Xq region is
    not written."""
    s, h = X.shape
    o = Wq.shape[1]
    if workspace is None:
        workspace = forward_workspace(s, h, X.device)
    if C is None:
        C = torch.empty((s, o), dtype=torch.float16, device=X.device)
    need = _lib.i8mm_forward_workspace_bytes(s, h)
    if workspace.numel() < need or workspace.dtype != torch.uint8:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    st = _lib.i8mm_forward_inline_quant(
        _dev(X, "X", torch.float16), s, h, o, float(alpha), _dev(Wq, "Wq", torch.int8, weight_panels_shape(h, o)),
        _dev(c_w, "c_w", torch.float32, (o,)), _weights_ptr(W, h, o), _bias_ptr(bias, o),
        _dev(workspace, "workspace", torch.uint8), _dev(C, "C", torch.float16, (s, o)), _stream(X))
    _check(st, "forward_inline_quant")
    return C


def forward_noalloc(X: torch.Tensor, Wq: torch.Tensor, c_w: torch.Tensor, W: Optional[torch.Tensor],
                    alpha: float = 6.0, C: torch.Tensor = None, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """forward() over the library's static device scratch instead of a
    workspace: the call allocates nothing on the device when C is given
    (for graph capture and loops that must not allocate). Raises I8MMError
    (status -5) when the shape needs more than NOALLOC_SCRATCH_BYTES of
    workspace. Calls on one GPU share the scratch and must not overlap."""
    s, h = X.shape
    o = Wq.shape[1]
    if C is None:
        C = torch.empty((s, o), dtype=torch.float16, device=X.device)
    st = _lib.i8mm_forward_noalloc(
        _dev(X, "X", torch.float16), s, h, o, float(alpha), _dev(Wq, "Wq", torch.int8, weight_panels_shape(h, o)),
        _dev(c_w, "c_w", torch.float32, (o,)), _weights_ptr(W, h, o), _bias_ptr(bias, o),
        _dev(C, "C", torch.float16, (s, o)), _stream(X))
    _check(st, "forward_noalloc")
    return C


def calib_mfma_i8(codes: torch.Tensor, iters: int, out: torch.Tensor) -> int:
    """Measurement calibration (not the method): enqueues a stream of int8
    MFMAs on register-resident operands, len(out) / 256 blocks of four
    wavefronts, 32 * iters MFMAs per wavefront. codes: int8, 65536 per block;
    out: int32, 256 per block. Returns the integer operations performed."""
    blocks = out.numel() // 256
    if blocks < 1 or out.numel() != blocks * 256:
        raise ValueError("out must hold a positive multiple of 256 int32")
    st = _lib.i8mm_calib_mfma_i8(_dev(codes, "codes", torch.int8, (blocks * 65536,)), blocks, iters,
                                 _dev(out, "out", torch.int32, (blocks * 256,)), _stream(codes))
    _check(st, "calib_mfma_i8")
    return blocks * 4 * 32 * iters * 65536


# ---------------------------------------------------------------- around an adapted layer
#
# These calls run in a few microseconds on the GPU while tokens are decoded,
# so what they do on the host is kept short: one look at each tensor, none at
# the outputs that they allocate themselves.

_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}   # i8mm_dtype
_LORA_TYPES = (torch.float16, torch.bfloat16)


def _matrix(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: int) -> Tuple[int, int]:
    """(pointer, row stride) of a GPU matrix whose columns are adjacent; what
    the C ABI cannot see is checked here."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device or t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on cuda:{device} "
                         f"(got {t.dtype} of shape {tuple(t.shape)} on {t.device})")
    if shape[0] <= 1:                   # the stride of a single row says nothing, no row has no strides
        ld, step = shape[1], t.stride(1) if shape[0] else 1
    else:
        ld, step = t.stride()
    if (step != 1 and shape[1] > 1) or ld < shape[1]:
        raise ValueError(f"{name} must have adjacent columns and rows that do not overlap (strides {t.stride()})")
    return t.data_ptr(), ld


def _dense(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: int) -> int:
    """The pointer of a contiguous GPU tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} of shape {tuple(shape)} on cuda:{device} "
                         f"(got {t.dtype} of shape {tuple(t.shape)} on {t.device})")
    return t.data_ptr()


def _gpu_of(t: torch.Tensor, name: str, types) -> int:
    """The index of the GPU that t is on, which has to be the current one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    device = t.get_device()
    if device != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current GPU, cuda:{torch.cuda.current_device()} (got {t.device})")
    if t.dtype not in types:
        raise ValueError(f"{name} must be one of {tuple(types)} (got {t.dtype})")
    return device


def _rows_of(X: torch.Tensor, types) -> Tuple[int, int, int, int, int]:
    """(device, rows, columns, pointer, row stride) of the matrix X that a call goes by."""
    device = _gpu_of(X, "X", types)
    if X.dim() != 2:
        raise ValueError(f"X must be a matrix (got shape {tuple(X.shape)})")
    s, h = X.shape
    return (device, s, h) + _matrix(X, "X", X.dtype, X.shape, device)


def _raw_stream(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)


def _scratch(nbytes: int, what: str, workspace: Optional[torch.Tensor], device: torch.device) -> torch.Tensor:
    """The caller's workspace, checked, or a new one."""
    if nbytes == 0:
        raise I8MMError(f"{what}: invalid shape")
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or workspace.numel() < nbytes or not workspace.is_contiguous() \
            or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {nbytes} bytes on {device}")
    return workspace


def _norm_weight(weight: torch.Tensor, X: torch.Tensor, h: int, device: int) -> Tuple[int, int]:
    """(pointer, i8mm_dtype) of a norm's weight, which is of X's type or fp32."""
    wt = getattr(weight, "dtype", None)
    if wt is not X.dtype and wt is not torch.float32:
        raise ValueError(f"weight must be {X.dtype} or torch.float32 (got {wt})")
    return _dense(weight, "weight", wt, (h,), device), _DTYPES[wt]


def layer_norm(X: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
               Y: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
               rstd: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Layer norm of the rows of X [s, h] (fp16, bf16 or fp32; rows may be
    strided): (Y = (X - mean) rstd weight + bias of X's type, mean fp32 [s],
    rstd fp32 [s]). weight and bias [h] are of X's type or fp32. Y may be X."""
    dev, s, h, x, ldx = _rows_of(X, _DTYPES)
    w, wt = _norm_weight(weight, X, h, dev)
    b = None if bias is None else _dense(bias, "bias", weight.dtype, (h,), dev)
    if Y is None:
        Y = X.new_empty((s, h))
        y, ldy = Y.data_ptr(), h
    else:
        y, ldy = _matrix(Y, "Y", X.dtype, X.shape, dev)
    if mean is None:
        mean = X.new_empty(s, dtype=torch.float32)
        m = mean.data_ptr()
    else:
        m = _dense(mean, "mean", torch.float32, (s,), dev)
    if rstd is None:
        rstd = X.new_empty(s, dtype=torch.float32)
        r = rstd.data_ptr()
    else:
        r = _dense(rstd, "rstd", torch.float32, (s,), dev)
    st = _lib.i8mm_layer_norm(x, ldx, _DTYPES[X.dtype], s, h, w, b, wt, eps, y, ldy, m, r, _raw_stream(dev))
    _check(st, "layer_norm")
    return Y, mean, rstd


def layer_norm_backward_workspace(s: int, h: int) -> int:
    """Bytes of workspace that layer_norm_backward needs."""
    return _lib.i8mm_layer_norm_backward_workspace_bytes(s, h)


def layer_norm_backward(dY: torch.Tensor, X: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, param_grads: bool = True, dX: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The gradients of layer_norm for dY, with its mean and rstd: (dX of X's
    type, d_weight fp32 [h], d_bias fp32 [h]); the last two are None if
    param_grads is false (a frozen norm). A workspace, if given, is a uint8
    tensor of layer_norm_backward_workspace(s, h) bytes or more."""
    dev, s, h, x, ldx = _rows_of(X, _DTYPES)
    w, wt = _norm_weight(weight, X, h, dev)
    dy, lddy = _matrix(dY, "dY", X.dtype, X.shape, dev)
    m, r = _dense(mean, "mean", torch.float32, (s,), dev), _dense(rstd, "rstd", torch.float32, (s,), dev)
    if dX is None:
        dX = X.new_empty((s, h))
        dx, lddx = dX.data_ptr(), h
    else:
        dx, lddx = _matrix(dX, "dX", X.dtype, X.shape, dev)
    d_weight = d_bias = dw = db = ws = None
    if param_grads:
        d_weight, d_bias = X.new_empty(h, dtype=torch.float32), X.new_empty(h, dtype=torch.float32)
        workspace = _scratch(layer_norm_backward_workspace(s, h), "layer_norm_backward", workspace, X.device)
        dw, db, ws = d_weight.data_ptr(), d_bias.data_ptr(), workspace.data_ptr()
    st = _lib.i8mm_layer_norm_backward(dy, lddy, x, ldx, _DTYPES[X.dtype], s, h, w, wt, m, r, dx, lddx, dw, db, ws,
                                       _raw_stream(dev))
    _check(st, "layer_norm_backward")
    return dX, d_weight, d_bias


def _adapters(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, ids: torch.Tensor, scale: torch.Tensor, s: int, h: int,
              dev: int):
    """(G, r, o, and the pointers of the adapters, the ids and the factors)."""
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError(f"A and B must be [adapters, rank, features] (got {tuple(A.shape)}, {tuple(B.shape)})")
    G, r, _ = A.shape
    o = B.shape[2]
    return G, r, o, _dense(A, "A", X.dtype, (G, r, h), dev), _dense(B, "B", X.dtype, (G, r, o), dev), \
        _dense(ids, "ids", torch.int32, (s,), dev), _dense(scale, "scale", torch.float32, (G,), dev)


def lora_forward_workspace(s: int, h: int, o: int, r: int) -> int:
    """Bytes of workspace that lora_forward needs."""
    return _lib.i8mm_lora_forward_workspace_bytes(s, h, o, r)


def lora_forward(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, ids: torch.Tensor, scale: torch.Tensor,
                 base: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                 T: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Low-rank adapters beside a shared projection: row i of X [s, h] (fp16 or
    bf16) carries adapter g = ids[i] (int32 [s]; none if outside [0, G)), and
    Y_i = base_i + scale_g T_i B_g with T_i = X_i A_g^T. A [G, r, h] and
    B [G, r, o] are of X's type, scale is fp32 [G]; base [s, o] is the
    projection's output (None: zeros) and may be passed as Y too. Returns
    (Y of X's type, T fp32 [s, r], which lora_backward reads). A workspace, if
    given, is a uint8 tensor of lora_forward_workspace(s, h, o, r) bytes or
    more."""
    dev, s, h, x, ldx = _rows_of(X, _LORA_TYPES)
    G, r, o, a, b, i, f = _adapters(X, A, B, ids, scale, s, h, dev)
    bp, ldb = (None, 0) if base is None else _matrix(base, "base", X.dtype, (s, o), dev)
    if Y is None:
        Y = X.new_empty((s, o))
        y, ldy = Y.data_ptr(), o
    else:
        y, ldy = _matrix(Y, "Y", X.dtype, (s, o), dev)
    if T is None:
        T = X.new_empty((s, r), dtype=torch.float32)
        t = T.data_ptr()
    else:
        t = _dense(T, "T", torch.float32, (s, r), dev)
    workspace = _scratch(lora_forward_workspace(s, h, o, r), "lora_forward", workspace, X.device)
    st = _lib.i8mm_lora_forward(x, ldx, a, b, _DTYPES[X.dtype], G, r, i, f, bp, ldb, s, h, o, y, ldy, t,
                                workspace.data_ptr(), _raw_stream(dev))
    _check(st, "lora_forward")
    return Y, T


def lora_backward_workspace(s: int, h: int, o: int, r: int, n_adapters: int) -> int:
    """Bytes of workspace that lora_backward needs."""
    return _lib.i8mm_lora_backward_workspace_bytes(s, h, o, r, n_adapters)


def lora_backward(dY: torch.Tensor, X: torch.Tensor, T: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                  ids: torch.Tensor, scale: torch.Tensor, base: Optional[torch.Tensor] = None,
                  input_grad: bool = True, dX: Optional[torch.Tensor] = None, dA: Optional[torch.Tensor] = None,
                  dB: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                  ) -> Tuple[Optional[torch.Tensor], torch.Tensor, torch.Tensor]:
    """The gradients of lora_forward for dY [s, o], with its T: (dX [s, h] of
    X's type, dA fp32 [G, r, h], dB fp32 [G, r, o]; zero for an adapter that
    no row carries). base [s, h] is the gradient that reaches X through the
    projection itself (None: zeros) and may be passed as dX too; dX is None
    if input_grad is false. A workspace, if given, is a uint8 tensor of
    lora_backward_workspace(s, h, o, r, G) bytes or more."""
    dev, s, h, x, ldx = _rows_of(X, _LORA_TYPES)
    G, r, o, a, b, i, f = _adapters(X, A, B, ids, scale, s, h, dev)
    dy, lddy = _matrix(dY, "dY", X.dtype, (s, o), dev)
    t = _dense(T, "T", torch.float32, (s, r), dev)
    bp = dx = None
    ldb = lddx = 0
    if not input_grad:
        dX = None
    else:
        if base is not None:
            bp, ldb = _matrix(base, "base", X.dtype, (s, h), dev)
        if dX is None:
            dX = X.new_empty((s, h))
        dx, lddx = _matrix(dX, "dX", X.dtype, (s, h), dev)
    if dA is None:
        dA = X.new_empty((G, r, h), dtype=torch.float32)
    if dB is None:
        dB = X.new_empty((G, r, o), dtype=torch.float32)
    workspace = _scratch(lora_backward_workspace(s, h, o, r, G), "lora_backward", workspace, X.device)
    st = _lib.i8mm_lora_backward(dy, lddy, x, ldx, t, a, b, _DTYPES[X.dtype], G, r, i, f, bp, ldb, s, h, o, dx, lddx,
                                 _dense(dA, "dA", torch.float32, (G, r, h), dev),
                                 _dense(dB, "dB", torch.float32, (G, r, o), dev), workspace.data_ptr(),
                                 _raw_stream(dev))
    _check(st, "lora_backward")
    return dX, dA, dB


def _tensor_table(tensors, name: str, device: int):
    """(pointers, element counts, i8mm_dtypes) of contiguous tensors on the
    device, as host arrays; written as maps, since a model has hundreds."""
    T = torch.Tensor
    if not set(map(T.get_device, tensors)) <= {device} or not all(map(T.is_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous tensors on the current GPU, cuda:{device}")
    try:
        types = array.array("i", map(_DTYPES.__getitem__, map(operator.attrgetter("dtype"), tensors)))
    except KeyError as e:
        raise ValueError(f"{name} must be fp16, bf16 or fp32 (got {e.args[0]})") from None
    return array.array("Q", map(T.data_ptr, tensors)), array.array("q", map(T.numel, tensors)), types


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The global norm N over all gradients (contiguous tensors on the current
    GPU, each fp16, bf16 or fp32), as fp32 [1] on the GPU, and the gradients
    times min(1, max_norm / (N + 1e-6)): in place, or into the tensors of
    `out`, each of its gradient's size and type. max_norm = inf leaves them as
    they are, whatever N is but NaN."""
    grads = list(grads)
    n = len(grads)
    dev = torch.cuda.current_device()
    device = torch.device("cuda", dev)
    pointers, numels, types = _tensor_table(grads, "grads", dev)
    out_pointers = None
    if out is not None:
        out_pointers, out_numels, out_types = _tensor_table(list(out), "out", dev)
        if out_numels != numels or out_types != types:
            raise ValueError("out must hold a tensor of each gradient's size and type, in their order")
    at = numels.buffer_info()[0]
    workspace = _scratch(_lib.i8mm_clip_grad_norm_workspace_bytes(at, n), "clip_grad_norm", workspace, device)
    total = torch.empty(1, dtype=torch.float32, device=device)
    st = _lib.i8mm_clip_grad_norm(pointers.buffer_info()[0], out_pointers.buffer_info()[0] if out_pointers else None,
                                  at, types.buffer_info()[0], n, max_norm, workspace.data_ptr(), total.data_ptr(),
                                  _raw_stream(dev))
    _check(st, "clip_grad_norm")
    return total
