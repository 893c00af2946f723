"""Python binding of libvq (include/vq.h, vq_i8.h, vq_experts.h): argument
marshalling only.

Every computation runs in the CUDA kernels behind the C ABI; this module only
turns torch tensors into pointers, sizes and the current CUDA stream.  There
is no fallback: if ``libvq.so`` is missing or fails to load, every call raises.

Names follow the C ABI: ``dequant``, ``gemv``, ``gemv_multi``, ``gemv_rht``,
``rht``, ``gemm``, ``repack_tile4``, ``encode``, ``hessian``, plus the
workspace size queries.  A ``Layer`` holds the device tensors of one
quantised layer (packed index streams in row order or in the tiled order,
fp16 codebooks, optional fp16 scale and bias, optional fp16 output bias).

Beside them stand layers in 8-bit integers (``Int8Layer``, ``quant_i8``,
``gemm_i8``, ``linear_i8``) and the experts of a mixture (``Experts``,
``group_rows``, ``gemm_experts``, ``combine_rows``).  Those calls check their
tensors' types, shapes, strides and device and raise ``ValueError``, and run on
their tensors' device whatever the current one is.
"""
from __future__ import annotations

import ctypes as C
import os
import re
import threading
from dataclasses import dataclass, field
from typing import List, Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libvq.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "vq.h")
HEADER_I8 = os.path.join(os.path.dirname(HERE), "include", "vq_i8.h")
HEADER_EXPERTS = os.path.join(os.path.dirname(HERE), "include", "vq_experts.h")

VQ_OK, VQ_ERR_INVALID_ARG, VQ_ERR_UNSUPPORTED, VQ_ERR_ALIGNMENT = 0, 1, 2, 3
VQ_ERR_WORKSPACE, VQ_ERR_CUDA, VQ_ERR_TIMEOUT = 4, 5, 6
VQ_BF16, VQ_FP16, VQ_FP32 = 0, 1, 2
VQ_IDX_ROWS, VQ_IDX_TILE4 = 0, 1
_LAYOUT = {"rows": VQ_IDX_ROWS, "tile4": VQ_IDX_TILE4}

_DTYPE = {torch.bfloat16: VQ_BF16, torch.float16: VQ_FP16, torch.float32: VQ_FP32}


class VQError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str, cuda_error: int = 0):
        super().__init__(f"{fn}: {msg} (status {status}"
                         + (f", cudaError {cuda_error})" if status == VQ_ERR_CUDA else ")"))
        self.status = status
        self.cuda_error = cuda_error


class _Desc(C.Structure):
    _fields_ = [
        ("out_features", C.c_int32), ("in_features", C.c_int32),
        ("vec_dim", C.c_int32), ("n_books", C.c_int32), ("log2k", C.c_int32 * 2),
        ("idx", C.c_void_p * 2), ("idx_row_words", C.c_int64 * 2),
        ("codebook", C.c_void_p * 2), ("scale", C.c_void_p), ("bias", C.c_void_p),
        ("idx_layout", C.c_int32), ("reserved", C.c_int32), ("out_bias", C.c_void_p),
    ]


class _EncDesc(C.Structure):
    _fields_ = [
        ("out_features", C.c_int32), ("in_features", C.c_int32),
        ("vec_dim", C.c_int32), ("n_books", C.c_int32), ("log2k", C.c_int32 * 2),
        ("w", C.c_void_p), ("ldw", C.c_int64),
        ("codebook", C.c_void_p * 2),
        ("idx", C.c_void_p * 2), ("idx_row_words", C.c_int64 * 2),
        ("h", C.c_void_p), ("ldh", C.c_int64),
    ]


class _I8Desc(C.Structure):
    _fields_ = [
        ("out_features", C.c_int32), ("in_features", C.c_int32),
        ("w", C.c_void_p), ("ldw", C.c_int64), ("scale", C.c_void_p), ("out_bias", C.c_void_p),
    ]


class _ExpertsDesc(C.Structure):
    _fields_ = [
        ("layer", _Desc), ("n_experts", C.c_int32), ("reserved", C.c_int32),
        ("idx_stride", C.c_int64 * 2), ("codebook_stride", C.c_int64 * 2),
        ("scale_stride", C.c_int64), ("bias_stride", C.c_int64), ("out_bias_stride", C.c_int64),
    ]


_lock = threading.Lock()
_lib = None


def exported_names(header: str = HEADER) -> List[str]:
    """Function names a header declares (VQ_API ...)."""
    with open(header) as fh:
        text = fh.read()
    return re.findall(r"VQ_API\s+[\w\s\*]+?\b(vq_\w+)\s*\(", text)


def lib():
    """Load libvq.so (raises if it is missing: there is no other code path)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libvq.so not found at {LIB_PATH}; build it with "
                                   "`python bit_packed_index_b200/build.py`")
            L = C.CDLL(LIB_PATH)
            P, I32, I64, SZ = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
            L.vq_dequant.argtypes = [P, P, I64, P]
            L.vq_gemv_workspace_size.argtypes = [P, I32, C.POINTER(SZ)]
            L.vq_gemv.argtypes = [P, P, C.c_int, I32, I64, P, C.c_int, I64, P, SZ, P]
            L.vq_gemv_noalloc.argtypes = [P, P, C.c_int, I32, I64, P, C.c_int, I64, P]
            L.vq_gemm_workspace_size.argtypes = [P, I32, C.c_int, C.POINTER(SZ)]
            L.vq_gemm.argtypes = [P, P, C.c_int, I32, I64, P, C.c_int, I64, P, SZ, P]
            L.vq_repack_tile4.argtypes = [P, C.POINTER(P), C.POINTER(I64), P]
            L.vq_gemv_multi_workspace_size.argtypes = [P, I32, I32, C.POINTER(SZ)]
            L.vq_gemv_multi.argtypes = [P, I32, P, C.c_int, I32, I64, P, C.c_int, P, P, SZ, P]
            L.vq_rht.argtypes = [P, C.c_int, I32, I32, I64, P, I32, P, C.c_int, I64, P]
            L.vq_gemv_rht_workspace_size.argtypes = [P, I32, C.POINTER(SZ)]
            L.vq_gemv_rht.argtypes = [P, P, P, P, C.c_int, I32, I64, P, C.c_int, I64, P, SZ, P]
            L.vq_hessian_workspace_size.argtypes = [I32, I32, C.POINTER(SZ)]
            L.vq_hessian.argtypes = [P, C.c_int, I32, I32, I64, P, I64, P, SZ, P]
            L.vq_encode_workspace_size.argtypes = [P, C.POINTER(SZ)]
            L.vq_encode.argtypes = [P, P, SZ, P]
            L.vq_quant_i8.argtypes = [P, C.c_int, I32, I32, I64, P, I64, P, P]
            L.vq_gemm_i8_workspace_size.argtypes = [P, I32, C.POINTER(SZ)]
            L.vq_gemm_i8.argtypes = [P, P, I64, P, I32, P, C.c_int, I64, P, SZ, P]
            L.vq_linear_i8_workspace_size.argtypes = [P, I32, C.POINTER(SZ)]
            L.vq_linear_i8.argtypes = [P, P, C.c_int, I32, I64, P, C.c_int, I64, P, SZ, P]
            L.vq_group_rows.argtypes = [P, I32, I32, I64, I32, P, P, P, P]
            L.vq_gemm_experts_workspace_size.argtypes = [P, I32, C.POINTER(SZ)]
            L.vq_gemm_experts.argtypes = [P, P, C.c_int, I32, I64, P, P, I32, P, C.c_int, I64, P, SZ, P]
            L.vq_combine_rows.argtypes = [P, C.c_int, I32, I32, I64, P, P, I64, I32, I32, P, C.c_int, I64, P]
            for fn in ("vq_quant_i8", "vq_gemm_i8_workspace_size", "vq_gemm_i8",
                       "vq_linear_i8_workspace_size", "vq_linear_i8", "vq_group_rows",
                       "vq_gemm_experts_workspace_size", "vq_gemm_experts", "vq_combine_rows"):
                getattr(L, fn).restype = C.c_int
            for fn in ("vq_dequant", "vq_gemv_workspace_size", "vq_gemv", "vq_gemv_noalloc",
                       "vq_gemm_workspace_size", "vq_gemm", "vq_repack_tile4",
                       "vq_encode_workspace_size", "vq_encode", "vq_gemv_multi_workspace_size",
                       "vq_gemv_multi", "vq_rht", "vq_gemv_rht_workspace_size", "vq_gemv_rht",
                       "vq_hessian_workspace_size", "vq_hessian"):
                getattr(L, fn).restype = C.c_int
            L.vq_status_string.argtypes = [C.c_int]
            L.vq_status_string.restype = C.c_char_p
            L.vq_last_cuda_error.restype = C.c_int
            L.vq_abi_version.restype = C.c_int
            L.vq_kernel_launches.restype = C.c_uint64
            _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != VQ_OK:
        L = lib()
        raise VQError(fn, status, L.vq_status_string(status).decode(),
                      L.vq_last_cuda_error() if status == VQ_ERR_CUDA else 0)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


@dataclass
class Layer:
    """Device tensors of one quantised layer (see include/vq.h)."""
    out_features: int
    in_features: int
    vec_dim: int
    log2k: List[int]
    idx: List[torch.Tensor]            # int32 views of uint32 words: [N][row_words] in row
                                       # order, [ceil(nvec/4)][tile_words] tiled
    codebooks: List[torch.Tensor]      # float16 [K][d]
    scale: Optional[torch.Tensor] = None   # float16 [N]
    bias: Optional[torch.Tensor] = None    # float16 [N]
    layout: str = "rows"               # "rows" or "tile4"
    out_bias: Optional[torch.Tensor] = None   # float16 [N], added to y after the product
    _desc: Optional[_Desc] = field(default=None, repr=False)

    @property
    def n_books(self) -> int:
        return len(self.log2k)

    @property
    def device(self) -> torch.device:
        return self.idx[0].device

    def desc(self) -> _Desc:
        if self._desc is None:
            d = _Desc()
            d.out_features, d.in_features = self.out_features, self.in_features
            d.vec_dim, d.n_books = self.vec_dim, self.n_books
            for m in range(self.n_books):
                d.log2k[m] = self.log2k[m]
                d.idx[m] = self.idx[m].data_ptr()
                d.idx_row_words[m] = self.idx[m].stride(0) if self.idx[m].shape[1] > 0 else 0
                d.codebook[m] = self.codebooks[m].data_ptr()
            d.scale = None if self.scale is None else self.scale.data_ptr()
            d.bias = None if self.bias is None else self.bias.data_ptr()
            d.idx_layout = _LAYOUT[self.layout]
            d.out_bias = None if self.out_bias is None else self.out_bias.data_ptr()
            self._desc = d
        return self._desc

    @classmethod
    def from_host(cls, out_features: int, in_features: int, vec_dim: int, log2k: Sequence[int],
                  idx_words: Sequence, codebooks: Sequence, scale=None, bias=None,
                  device="cuda", out_bias=None) -> "Layer":
        """From numpy arrays: uint32 streams, fp16-bit (uint16) codebooks, scale,
        bias and output bias."""
        import numpy as np

        def words(a):
            a = np.ascontiguousarray(a, np.uint32).view(np.int32)
            return torch.from_numpy(a).to(device)

        def halves(a):
            if a is None:
                return None
            a = np.ascontiguousarray(a, np.uint16).view(np.int16)
            return torch.from_numpy(a).to(device).view(torch.float16)

        return cls(out_features, in_features, vec_dim, list(log2k),
                   [words(w) for w in idx_words], [halves(c) for c in codebooks],
                   halves(scale), halves(bias), out_bias=halves(out_bias))

    @classmethod
    def from_synth(cls, data, device="cuda", layout: str = "rows") -> "Layer":
        """From generated host data (row-order streams); layout="tile4" converts
        them on the device with vq_repack_tile4."""
        s = data.spec
        layer = cls.from_host(s.out_features, s.in_features, s.d, s.log2k, data.idx_words,
                              data.codebooks, data.scale, data.bias, device,
                              getattr(data, "out_bias", None))
        if layout == "tile4":
            layer = repack_tile4(layer)
        elif layout != "rows":
            raise ValueError(f"unknown index layout {layout!r}")
        return layer

    def nbytes(self) -> int:
        n = sum(t.numel() * t.element_size() for t in self.idx + self.codebooks)
        for t in (self.scale, self.bias, self.out_bias):
            n += 0 if t is None else t.numel() * 2
        return n


def tile4_words(out_features: int, log2k: int) -> int:
    """Smallest tile stride (32-bit words) of the tiled order: N records of 4 fields."""
    return -(-(out_features * 4 * log2k) // 128) * 4


def repack_tile4(layer: Layer, tile_words: Optional[Sequence[int]] = None) -> Layer:
    """The same layer with its index streams in the tiled order (vq_repack_tile4);
    codebooks, scale and bias are shared with ``layer``."""
    if layer.layout != "rows":
        raise ValueError("repack_tile4 needs a row-order layer")
    nvec = -(-layer.in_features // layer.vec_dim)
    ntile = -(-nvec // 4)
    tw = [tile4_words(layer.out_features, b) if tile_words is None else int(tile_words[m])
          for m, b in enumerate(layer.log2k)]
    dst = [torch.empty((ntile, w), dtype=torch.int32, device=layer.device) for w in tw]
    ptrs = (C.c_void_p * 2)(*([t.data_ptr() for t in dst] + [0] * (2 - len(dst))))
    words = (C.c_int64 * 2)(*(tw + [0] * (2 - len(tw))))
    _check("vq_repack_tile4", lib().vq_repack_tile4(C.byref(layer.desc()), ptrs, words,
                                                    C.c_void_p(_stream(layer.device))))
    return Layer(layer.out_features, layer.in_features, layer.vec_dim, list(layer.log2k), dst,
                 layer.codebooks, layer.scale, layer.bias, layout="tile4", out_bias=layer.out_bias)


def dequant(layer: Layer, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """W_hat, float16 [N][Kin] (or into ``out``, whose row stride is honoured)."""
    if out is None:
        out = torch.empty((layer.out_features, layer.in_features), dtype=torch.float16,
                          device=layer.device)
    ldw = out.stride(0) if out.dim() == 2 and out.shape[0] > 0 else layer.in_features
    _check("vq_dequant", lib().vq_dequant(C.byref(layer.desc()), _ptr(out), ldw,
                                          C.c_void_p(_stream(layer.device))))
    return out


def gemv_workspace_size(layer: Layer, batch: int) -> int:
    n = C.c_size_t(0)
    _check("vq_gemv_workspace_size", lib().vq_gemv_workspace_size(C.byref(layer.desc()), batch,
                                                                  C.byref(n)))
    return n.value


def gemm_workspace_size(layer: Layer, m: int, x_dtype=torch.bfloat16) -> int:
    n = C.c_size_t(0)
    _check("vq_gemm_workspace_size", lib().vq_gemm_workspace_size(
        C.byref(layer.desc()), m, _DTYPE[x_dtype], C.byref(n)))
    return n.value


def _workspace(nbytes: int, device, given: Optional[torch.Tensor]):
    if nbytes == 0:
        return None, 0
    if given is not None:
        return given, given.numel() * given.element_size()
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, nbytes


def gemv(layer: Layer, x: torch.Tensor, out_dtype=torch.bfloat16,
         out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [B][N] = x [B][Kin] . W_hat^T for B <= 16 (x bf16 or fp16 on the device)."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    batch = x.shape[0]
    if out is None:
        out = torch.empty((batch, layer.out_features), dtype=out_dtype, device=layer.device)
    ws, ws_bytes = _workspace(gemv_workspace_size(layer, batch), layer.device, workspace)
    ldx = x.stride(0) if batch > 1 else max(x.shape[1], layer.in_features)
    ldy = out.stride(0) if batch > 1 else max(out.shape[1], layer.out_features)
    _check("vq_gemv", lib().vq_gemv(C.byref(layer.desc()), _ptr(x), _DTYPE[x.dtype], batch, ldx,
                                    _ptr(out), _DTYPE[out.dtype], ldy, _ptr(ws), ws_bytes,
                                    C.c_void_p(_stream(layer.device))))
    return out


NOALLOC_SCRATCH_BYTES = 8 << 20


def gemv_noalloc(layer: Layer, x: torch.Tensor, out_dtype=torch.bfloat16,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """vq_gemv without a workspace, for callers that cannot allocate device
    memory where they run the layer: the split-K scratch is a fixed
    NOALLOC_SCRATCH_BYTES array inside the library (see vq_gemv_noalloc in
    include/vq.h).  Pass ``out`` to keep the call free of allocations."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    batch = x.shape[0]
    if out is None:
        out = torch.empty((batch, layer.out_features), dtype=out_dtype, device=layer.device)
    ldx = x.stride(0) if batch > 1 else max(x.shape[1], layer.in_features)
    ldy = out.stride(0) if batch > 1 else max(out.shape[1], layer.out_features)
    _check("vq_gemv_noalloc", lib().vq_gemv_noalloc(
        C.byref(layer.desc()), _ptr(x), _DTYPE[x.dtype], batch, ldx, _ptr(out),
        _DTYPE[out.dtype], ldy, C.c_void_p(_stream(layer.device))))
    return out


def gemm(layer: Layer, x: torch.Tensor, out_dtype=torch.bfloat16,
         out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M][N] = x [M][Kin] . W_hat^T on the tensor cores (x bf16 or fp16)."""
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, layer.out_features), dtype=out_dtype, device=layer.device)
    ws, ws_bytes = _workspace(gemm_workspace_size(layer, m, x.dtype), layer.device, workspace)
    ldx = x.stride(0) if m > 1 else max(x.shape[1], layer.in_features)
    ldy = out.stride(0) if m > 1 else max(out.shape[1], layer.out_features)
    _check("vq_gemm", lib().vq_gemm(C.byref(layer.desc()), _ptr(x), _DTYPE[x.dtype], m, ldx,
                                    _ptr(out), _DTYPE[out.dtype], ldy, _ptr(ws), ws_bytes,
                                    C.c_void_p(_stream(layer.device))))
    return out


def _desc_array(layers: Sequence[Layer]):
    arr = (C.c_void_p * len(layers))(*[C.addressof(l.desc()) for l in layers])
    return arr


def gemv_multi_workspace_size(layers: Sequence[Layer], batch: int) -> int:
    n = C.c_size_t(0)
    _check("vq_gemv_multi_workspace_size",
           lib().vq_gemv_multi_workspace_size(_desc_array(layers), len(layers), batch, C.byref(n)))
    return n.value


def gemv_multi(layers: Sequence[Layer], x: torch.Tensor, out_dtype=torch.bfloat16,
               outs: Optional[Sequence[torch.Tensor]] = None,
               workspace: Optional[torch.Tensor] = None) -> List[torch.Tensor]:
    """y_l [B][N_l] = x [B][Kin] . W_hat_l^T for layers sharing x (vq_gemv_multi);
    tiled 2^16-book layers at batch 1 run as one table launch."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    batch = x.shape[0]
    dev = layers[0].device
    if outs is None:
        outs = [torch.empty((batch, l.out_features), dtype=out_dtype, device=dev) for l in layers]
    ws, ws_bytes = _workspace(gemv_multi_workspace_size(layers, batch), dev, workspace)
    ldx = x.stride(0) if batch > 1 else max(x.shape[1], layers[0].in_features)
    ys = (C.c_void_p * len(layers))(*[o.data_ptr() for o in outs])
    ldy = (C.c_int64 * len(layers))(*[o.stride(0) if batch > 1 else max(o.shape[1], l.out_features)
                                      for o, l in zip(outs, layers)])
    _check("vq_gemv_multi", lib().vq_gemv_multi(_desc_array(layers), len(layers), _ptr(x), _DTYPE[x.dtype],
                                                batch, ldx, ys, _DTYPE[outs[0].dtype], ldy, _ptr(ws),
                                                ws_bytes, C.c_void_p(_stream(dev))))
    return list(outs)


def rht(x: torch.Tensor, signs: torch.Tensor, inverse: bool = False, out_dtype=None,
        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Randomized Hadamard transform of the rows of x (vq_rht); `signs` holds
    the sign bits as int32 words (bit t set -> -1)."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    rows, n = x.shape
    if out is None:
        out = torch.empty((rows, n), dtype=out_dtype or x.dtype, device=x.device)
    ld_in = x.stride(0) if rows > 1 else max(n, 1)
    ld_out = out.stride(0) if rows > 1 else max(n, 1)
    _check("vq_rht", lib().vq_rht(_ptr(x), _DTYPE[x.dtype], rows, n, ld_in, _ptr(signs), int(inverse),
                                  _ptr(out), _DTYPE[out.dtype], ld_out, C.c_void_p(_stream(x.device))))
    return out


def gemv_rht_workspace_size(layer: Layer, batch: int) -> int:
    n = C.c_size_t(0)
    _check("vq_gemv_rht_workspace_size",
           lib().vq_gemv_rht_workspace_size(C.byref(layer.desc()), batch, C.byref(n)))
    return n.value


def gemv_rht(layer: Layer, signs_in: torch.Tensor, signs_out: torch.Tensor, x: torch.Tensor,
             out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = U^T (W~ (V x)) for a layer whose streams encode the rotated W~ (vq_gemv_rht)."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    batch = x.shape[0]
    if out is None:
        out = torch.empty((batch, layer.out_features), dtype=out_dtype, device=layer.device)
    ws, ws_bytes = _workspace(gemv_rht_workspace_size(layer, batch), layer.device, workspace)
    ldx = x.stride(0) if batch > 1 else max(x.shape[1], layer.in_features)
    ldy = out.stride(0) if batch > 1 else max(out.shape[1], layer.out_features)
    _check("vq_gemv_rht", lib().vq_gemv_rht(C.byref(layer.desc()), _ptr(signs_in), _ptr(signs_out), _ptr(x),
                                            _DTYPE[x.dtype], batch, ldx, _ptr(out), _DTYPE[out.dtype], ldy,
                                            _ptr(ws), ws_bytes, C.c_void_p(_stream(layer.device))))
    return out


def hessian_workspace_size(n_tokens: int, d: int) -> int:
    nb = C.c_size_t(0)
    _check("vq_hessian_workspace_size", lib().vq_hessian_workspace_size(n_tokens, d, C.byref(nb)))
    return nb.value


def hessian(x: torch.Tensor, out: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h = 2 X^T X / n + 0.01 mean(diag) I (float32 [d][d]) of activations x
    (bf16 or fp16 [n_tokens][d] on the device), through vq_hessian."""
    n, d = x.shape
    if out is None:
        out = torch.empty((d, d), dtype=torch.float32, device=x.device)
    ws, ws_bytes = _workspace(hessian_workspace_size(n, d), x.device, workspace)
    ldx = x.stride(0) if n > 1 else max(d, 1)
    _check("vq_hessian", lib().vq_hessian(_ptr(x), _DTYPE[x.dtype], n, d, ldx, _ptr(out), out.stride(0),
                                          _ptr(ws), ws_bytes, C.c_void_p(_stream(x.device))))
    return out


def row_words(in_features: int, vec_dim: int, log2k: int) -> int:
    """Smallest row stride (32-bit words) of a row-order stream."""
    nvec = -(-in_features // vec_dim)
    return -(-(nvec * log2k) // 128) * 4


def _encode_desc(w: torch.Tensor, codebooks, log2k, vec_dim: int, idx,
                 hessian: Optional[torch.Tensor] = None) -> _EncDesc:
    d = _EncDesc()
    d.out_features, d.in_features = w.shape[0], w.shape[1]
    d.vec_dim, d.n_books = vec_dim, len(log2k)
    d.w = w.data_ptr() if w.numel() else None
    d.ldw = w.stride(0) if w.shape[0] > 1 else max(w.shape[1], 1)   # ldw >= Kin
    for m, b in enumerate(log2k):
        d.log2k[m] = b
        d.codebook[m] = codebooks[m].data_ptr()
        d.idx[m] = idx[m].data_ptr() if idx[m].numel() else None
        d.idx_row_words[m] = idx[m].shape[1]
    if hessian is not None:
        if hessian.dtype != torch.float32 or hessian.dim() != 2 or hessian.stride(1) != 1:
            raise ValueError("the Hessian must be a row-major float32 matrix")
        d.h = hessian.data_ptr()
        d.ldh = hessian.stride(0)
    return d


def encode_workspace_size(out_features: int, in_features: int, log2k: Sequence[int],
                          vec_dim: int, hessian: bool = False) -> int:
    d = _EncDesc()
    d.out_features, d.in_features, d.vec_dim, d.n_books = out_features, in_features, vec_dim, len(log2k)
    d.ldw = max(in_features, 1)
    if hessian:                        # any aligned non-null pointer: only sizes are read
        d.h = 256
        d.ldh = max(in_features, 1)
    for m, b in enumerate(log2k):
        d.log2k[m] = int(b)
        d.idx_row_words[m] = row_words(in_features, vec_dim, int(b))
    n = C.c_size_t(0)
    _check("vq_encode_workspace_size", lib().vq_encode_workspace_size(C.byref(d), C.byref(n)))
    return n.value


def encode(w: torch.Tensor, codebooks: Sequence[torch.Tensor], log2k: Sequence[int], vec_dim: int,
           workspace: Optional[torch.Tensor] = None, hessian: Optional[torch.Tensor] = None) -> Layer:
    """Nearest-centroid encoding of W (float16 [N][Kin] on the device) against
    one book, or two as a greedy residual cascade (vq_encode): a row-order
    Layer holding the packed streams and the given codebooks (no scale or
    bias).  With ``hessian`` (float32 [Kin][Kin] on the device, e.g. from
    ``hessian()``) the distance is the Hessian-weighted (v-c)^T H_v (v-c)."""
    if w.dtype != torch.float16 or w.dim() != 2 or (w.shape[0] > 1 and w.stride(1) != 1):
        raise ValueError("w must be a row-major float16 matrix")
    log2k = [int(b) for b in log2k]
    books = [c.contiguous() for c in codebooks[:len(log2k)]]
    idx = [torch.empty((w.shape[0], row_words(w.shape[1], vec_dim, b)), dtype=torch.int32,
                       device=w.device) for b in log2k]
    d = _encode_desc(w, books, log2k, vec_dim, idx, hessian)
    n = C.c_size_t(0)
    _check("vq_encode_workspace_size", lib().vq_encode_workspace_size(C.byref(d), C.byref(n)))
    ws, ws_bytes = _workspace(n.value, w.device, workspace)
    _check("vq_encode", lib().vq_encode(C.byref(d), _ptr(ws), ws_bytes, C.c_void_p(_stream(w.device))))
    return Layer(w.shape[0], w.shape[1], vec_dim, log2k, idx, books)


# ---------------------------------------------------------------------------
# Layers in 8-bit integers (include/vq_i8.h).
# ---------------------------------------------------------------------------
# A small call takes the GPU a few microseconds, so the checks here are kept
# cheap: one pass over plain attributes, and a message only when one fails.
_IN16 = {torch.bfloat16: VQ_BF16, torch.float16: VQ_FP16}
_INT8 = {torch.int8: 0}
_INT32 = {torch.int32: 0}
_FLOAT32 = {torch.float32: VQ_FP32}


def _refuse(t, name: str, want: str):
    have = (f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}" if isinstance(t, torch.Tensor)
            else type(t).__name__)
    raise ValueError(f"{name} must be {want}; it is {have}")


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _matrix(t: torch.Tensor, name: str, types, index: int, cols: int = -1) -> int:
    """Row stride of a row-major matrix of one of `types` on CUDA device `index`."""
    shape = t.shape
    if len(shape) == 2 and t.dtype in types and index >= 0 and t.get_device() == index and cols in (-1, shape[1]):
        rows, n = shape
        if n <= 1 or t.stride(1) == 1:
            if rows <= 1:
                return n or 1
            ld = t.stride(0)
            if ld >= n:
                return ld
    _refuse(t, name, f"a row-major matrix{'' if cols < 0 else f' of {cols} columns'} of "
                     f"{' or '.join(map(str, types))} on {f'cuda:{index}' if index >= 0 else 'a CUDA device'}, "
                     "its rows apart")


def _vector(t: torch.Tensor, name: str, dtype, n: int, index: int):
    if (len(t.shape) != 1 or t.dtype != dtype or t.shape[0] != n or t.get_device() != index
            or (n > 1 and t.stride(0) != 1)):
        _refuse(t, name, f"a contiguous vector of {n} {dtype} on cuda:{index}")


def _output(out, rows: int, cols: int, dtype, like: torch.Tensor, index: int):
    if out is None:
        if dtype not in _DTYPE:
            raise ValueError(f"unsupported output type {dtype}")
        return like.new_empty((rows, cols), dtype=dtype), cols or 1
    ld = _matrix(out, "out", _DTYPE, index, cols)
    if out.shape[0] != rows:
        _refuse(out, "out", f"{rows} x {cols}")
    return out, ld


def _scratch(nbytes: int, like: torch.Tensor, index: int, given: Optional[torch.Tensor]):
    """Pointer, size and owner of a call's workspace (the caller's holds a
    status word that the caller clears; see include/vq_i8.h)."""
    if given is not None:
        if given.get_device() != index or not given.is_contiguous():
            _refuse(given, "workspace", f"contiguous, on cuda:{index}")
        return given.data_ptr(), given.numel() * given.element_size(), given
    if nbytes == 0:
        return 0, 0, None
    t = like.new_empty(nbytes, dtype=torch.uint8)
    return t.data_ptr(), nbytes, t


def _accepted(size_fn: str, ref: int, rules: str):
    """Refuse a description that no call would accept (host-only: the size of a call without rows)."""
    status = getattr(lib(), size_fn)(ref, 0, C.byref(C.c_size_t(0)))
    if status != VQ_OK:
        raise ValueError(f"{rules} ({status_string(status)})")


_functions = {}


def _run(name: str, index: int, *args):
    """lib().<name>(*args, the current stream of device `index`) with that device current."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(lib(), name)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != VQ_OK:
        _check(name, status)


class Int8Layer:
    """A linear layer in 8-bit integers: weight int8 [N][Kin] (rows 16-byte
    aligned, a stride that is a multiple of 16), one float32 scale per output
    channel, optional float16 output bias.  ``quantise`` makes one from a
    float16 or bfloat16 matrix."""

    def __init__(self, weight: torch.Tensor, scale: torch.Tensor, out_bias: Optional[torch.Tensor] = None):
        self.device, self.index = weight.device, weight.get_device()
        ld = _matrix(weight, "weight", _INT8, self.index)
        n, k = weight.shape
        _vector(scale, "scale", torch.float32, n, self.index)
        if out_bias is not None:
            _vector(out_bias, "out_bias", torch.float16, n, self.index)
        self.weight, self.scale, self.out_bias = weight, scale, out_bias
        self.out_features, self.in_features = n, k
        d = _I8Desc()
        d.out_features, d.in_features = n, k
        d.w, d.ldw = weight.data_ptr(), ld if n > 1 else -(-max(k, 1) // 16) * 16
        d.scale = scale.data_ptr()
        d.out_bias = None if out_bias is None else out_bias.data_ptr()
        self._desc = d
        self._ref = C.addressof(d)
        self._sizes = {}
        _accepted("vq_gemm_i8_workspace_size", self._ref, "weight rows must start on 16 bytes and hold at most 131071 values")

    @classmethod
    def quantise(cls, w: torch.Tensor, out_bias: Optional[torch.Tensor] = None) -> "Int8Layer":
        """From W [N][Kin] (float16 or bfloat16, on the device), row by row (vq_quant_i8)."""
        q, scale = quant_i8(w)
        return cls(q, scale, out_bias)

    def nbytes(self) -> int:
        return self.weight.shape[0] * (self.weight.shape[1] + 4 + (0 if self.out_bias is None else 2))

    def _bytes(self, fn: str, m: int) -> int:
        """Workspace bytes of vq_<fn>_i8 for m rows (a function of the sizes alone, so kept)."""
        n = self._sizes.get((fn, m))
        if n is None:
            size, name = C.c_size_t(0), f"vq_{fn}_i8_workspace_size"
            _check(name, getattr(lib(), name)(self._ref, m, C.byref(size)))
            n = self._sizes[(fn, m)] = size.value
        return n


def gemm_i8_workspace_size(layer: Int8Layer, m: int) -> int:
    return layer._bytes("gemm", m)


def linear_i8_workspace_size(layer: Int8Layer, m: int) -> int:
    return layer._bytes("linear", m)


def quant_i8(x: torch.Tensor, out: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None):
    """(q, scale): the rows of x (bf16 or fp16 [m][n]) as int8 with one float32
    scale each (vq_quant_i8).  A new q has rows padded to 16 bytes, as gemm_i8
    and Int8Layer want them."""
    index = x.get_device()
    ldx = _matrix(x, "x", _IN16, index)
    m, n = x.shape
    if out is None:
        ldq = -(-(n or 1) // 16) * 16
        out = x.new_empty((m, ldq), dtype=torch.int8)
        if ldq != n:
            out = out[:, :n]
    else:
        ldq = _matrix(out, "out", _INT8, index, n)
        if out.shape[0] != m:
            _refuse(out, "out", f"{m} x {n}")
    if scale is None:
        scale = x.new_empty(m, dtype=torch.float32)
    else:
        _vector(scale, "scale", torch.float32, m, index)
    _run("vq_quant_i8", index, x.data_ptr(), _DTYPE[x.dtype], m, n, ldx, out.data_ptr(), ldq, scale.data_ptr())
    return out, scale


def gemm_i8(layer: Int8Layer, q: torch.Tensor, q_scale: torch.Tensor, out_dtype=torch.bfloat16,
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [m][N] = (q . W^T) * scale * q_scale + bias for rows that quant_i8 made (vq_gemm_i8)."""
    index = layer.index
    ldq = _matrix(q, "q", _INT8, index, layer.in_features)
    m = q.shape[0]
    if m <= 1:
        ldq = -(-ldq // 16) * 16
    _vector(q_scale, "q_scale", torch.float32, m, index)
    out, ldy = _output(out, m, layer.out_features, out_dtype, q, index)
    ws, n, keep = _scratch(layer._bytes("gemm", m), q, index, workspace)
    _run("vq_gemm_i8", index, layer._ref, q.data_ptr(), ldq, q_scale.data_ptr(), m, out.data_ptr(), _DTYPE[out.dtype],
         ldy, ws, n)
    return out


def linear_i8(layer: Int8Layer, x: torch.Tensor, out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [m][N] of bf16 or fp16 activations x [m][Kin]: quant_i8 and gemm_i8 in one call (vq_linear_i8)."""
    index = layer.index
    ldx = _matrix(x, "x", _IN16, index, layer.in_features)
    m = x.shape[0]
    out, ldy = _output(out, m, layer.out_features, out_dtype, x, index)
    ws, n, keep = _scratch(layer._bytes("linear", m), x, index, workspace)
    _run("vq_linear_i8", index, layer._ref, x.data_ptr(), _DTYPE[x.dtype], m, ldx, out.data_ptr(), _DTYPE[out.dtype],
         ldy, ws, n)
    return out


# ---------------------------------------------------------------------------
# The experts of a mixture (include/vq_experts.h).
# ---------------------------------------------------------------------------
class Experts:
    """Codebook-indexed experts of one shape, stacked: ``idx[m]`` int32
    [E][N][row_words] (row order) or [E][tiles][tile_words] (tiled),
    ``codebooks[m]`` float16 [E][K][d] or [1][K][d] (one book for all), scale,
    bias and out_bias float16 [E][N] or [1][N].  ``from_layers`` stacks
    ``Layer`` objects; ``layer(e)`` is expert e as a ``Layer`` on the same
    memory (index words that are columns of a wider array are copied: a layer's
    last row has to own the whole distance between two rows)."""

    def __init__(self, out_features: int, in_features: int, vec_dim: int, log2k: Sequence[int],
                 idx: Sequence[torch.Tensor], codebooks: Sequence[torch.Tensor], scale: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, layout: str = "rows", out_bias: Optional[torch.Tensor] = None):
        _need(layout in _LAYOUT, f"unknown index layout {layout!r}")
        _need(1 <= len(log2k) <= 2 and len(idx) == len(log2k) == len(codebooks),
              "one or two books, an index stream and a codebook each")
        _need(idx[0].dim() == 3 and idx[0].is_cuda, "idx must be stacked streams on a CUDA device")
        _need(1 <= vec_dim <= 16 and all(1 <= int(b) <= 16 for b in log2k), "vec_dim and log2k must lie in 1..16")
        dev, e = idx[0].device, idx[0].shape[0]
        _need(e >= 1, "at least one expert")
        nvec = -(-in_features // vec_dim)
        stream_rows = out_features if layout == "rows" else -(-nvec // 4)
        D = _ExpertsDesc()
        d = D.layer
        d.out_features, d.in_features, d.vec_dim, d.n_books = out_features, in_features, vec_dim, len(log2k)
        d.idx_layout = _LAYOUT[layout]
        for m, b in enumerate(log2k):
            t, c = idx[m], codebooks[m]
            _need(t.dtype == torch.int32 and t.device == dev and tuple(t.shape[:2]) == (e, stream_rows)
                  and (t.shape[2] <= 1 or t.stride(2) == 1),
                  f"idx[{m}] must be int32 [{e}][{stream_rows}][words], its words contiguous, on {dev}")
            _need(c.dtype == torch.float16 and c.device == dev and c.dim() == 3 and c.shape[0] in (1, e)
                  and tuple(c.shape[1:]) == (1 << int(b), vec_dim) and c[0].is_contiguous(),
                  f"codebooks[{m}] must be float16 [{e} or 1][{1 << int(b)}][{vec_dim}], each book contiguous, on {dev}")
            d.log2k[m], d.idx[m], d.codebook[m] = int(b), t.data_ptr(), c.data_ptr()
            d.idx_row_words[m] = t.stride(1) if stream_rows > 1 and t.shape[2] > 0 else t.shape[2]
            words = row_words(in_features, vec_dim, int(b)) if layout == "rows" else tile4_words(out_features, int(b))
            _need(words <= t.shape[2] <= d.idx_row_words[m] or stream_rows == 0 or t.shape[1] == 0,
                  f"idx[{m}] needs {words} words a row, and rows that do not overlap")
            D.idx_stride[m] = t.stride(0) if e > 1 and t.numel() > 0 else 0
            D.codebook_stride[m] = c.stride(0) if c.shape[0] > 1 else 0
        for name, t in (("scale", scale), ("bias", bias), ("out_bias", out_bias)):
            if t is None:
                continue
            _need(t.dtype == torch.float16 and t.device == dev and t.dim() == 2 and t.shape[0] in (1, e)
                  and t.shape[1] == out_features and (out_features <= 1 or t.stride(1) == 1),
                  f"{name} must be float16 [{e} or 1][{out_features}] on {dev}")
            setattr(d, name, t.data_ptr())
            setattr(D, name + "_stride", t.stride(0) if t.shape[0] > 1 else 0)
        D.n_experts = e
        _accepted("vq_gemm_experts_workspace_size", C.addressof(D), "every expert's streams and books must start on 16 "
                  "bytes, index rows be a multiple of 4 words apart, and experts number at most 1024")
        self.n_experts, self.out_features, self.in_features, self.vec_dim = e, out_features, in_features, vec_dim
        self.log2k, self.layout, self.device, self.index = [int(b) for b in log2k], layout, dev, idx[0].get_device()
        self.idx, self.codebooks = list(idx), list(codebooks)
        self.scale, self.bias, self.out_bias = scale, bias, out_bias
        self._desc = D
        self._ref = C.addressof(D)
        self._sizes = {}

    @classmethod
    def from_layers(cls, layers: Sequence[Layer]) -> "Experts":
        """Stack layers of one shape, layout and device (their tensors are copied)."""
        _need(len(layers) >= 1, "at least one layer")
        a = layers[0]
        shape = lambda l: (l.out_features, l.in_features, l.vec_dim, list(l.log2k), l.layout, l.device,
                           [tuple(t.shape) for t in l.idx], l.scale is None, l.bias is None, l.out_bias is None)
        _need(all(shape(l) == shape(a) for l in layers), "the layers must have one shape, layout and device")
        books = []
        for m in range(a.n_books):
            size = a.codebooks[m].numel()
            # every book starts on 16 bytes
            flat = torch.zeros((len(layers), -(-size // 8) * 8), dtype=torch.float16, device=a.device)
            for e, l in enumerate(layers):
                flat[e, :size] = l.codebooks[m].reshape(-1)
            books.append(flat.as_strided((len(layers), 1 << a.log2k[m], a.vec_dim), (flat.shape[1], a.vec_dim, 1)))
        stack = lambda ts: None if ts[0] is None else torch.stack(ts)
        return cls(a.out_features, a.in_features, a.vec_dim, a.log2k,
                   [torch.stack([l.idx[m] for l in layers]) for m in range(a.n_books)], books,
                   stack([l.scale for l in layers]), stack([l.bias for l in layers]), a.layout,
                   stack([l.out_bias for l in layers]))

    def layer(self, e: int) -> Layer:
        at = lambda t: None if t is None else t[e if t.shape[0] > 1 else 0]
        whole = lambda t: t if t.stride(0) == t.shape[1] else t.clone(memory_format=torch.contiguous_format)
        return Layer(self.out_features, self.in_features, self.vec_dim, list(self.log2k), [whole(t[e]) for t in self.idx],
                     [at(c) for c in self.codebooks], at(self.scale), at(self.bias), layout=self.layout,
                     out_bias=at(self.out_bias))

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   self.idx + self.codebooks + [v for v in (self.scale, self.bias, self.out_bias) if v is not None])


def group_rows(ids: torch.Tensor, n_experts: int, offsets: Optional[torch.Tensor] = None,
               rows: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None):
    """(offsets [E+1], rows [T * top_k], pos [T][top_k]) of the picks ids (int32
    [T][top_k]) in the order of their experts (vq_group_rows)."""
    index = ids.get_device()
    ld = _matrix(ids, "ids", _INT32, index)
    t, k = ids.shape
    if offsets is None:
        offsets = ids.new_empty(max(n_experts, 0) + 1)
    else:
        _vector(offsets, "offsets", torch.int32, n_experts + 1, index)
    if rows is None:
        rows = ids.new_empty(t * k)
    else:
        _vector(rows, "rows", torch.int32, t * k, index)
    if pos is None:
        pos = ids.new_empty((t, k))
    elif pos.dtype != torch.int32 or pos.get_device() != index or pos.shape != ids.shape or not pos.is_contiguous():
        _refuse(pos, "pos", "contiguous int32 of ids' shape")
    _run("vq_group_rows", index, ids.data_ptr(), t, k, ld, n_experts, offsets.data_ptr(), rows.data_ptr(),
         pos.data_ptr())
    return offsets, rows, pos


def gemm_experts_workspace_size(experts: Experts, m: int) -> int:
    n = experts._sizes.get(m)                 # a function of the sizes alone, so kept
    if n is None:
        size = C.c_size_t(0)
        _check("vq_gemm_experts_workspace_size",
               lib().vq_gemm_experts_workspace_size(experts._ref, m, C.byref(size)))
        n = experts._sizes[m] = size.value
    return n


def gemm_experts(experts: Experts, x: torch.Tensor, offsets: torch.Tensor, rows: Optional[torch.Tensor] = None,
                 out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [m][N]: rows offsets[e] .. offsets[e+1]-1 are the products of their
    rows of x with expert e (vq_gemm_experts).  Grouped row r reads x[rows[r]],
    or x[r] without ``rows``; m is the length of ``rows``, else of x.  Rows
    behind the last group are not written."""
    index = experts.index
    ldx = _matrix(x, "x", _IN16, index, experts.in_features)
    _vector(offsets, "offsets", torch.int32, experts.n_experts + 1, index)
    m = x_rows = x.shape[0]
    rows_ptr = None
    if rows is not None:
        _vector(rows, "rows", torch.int32, rows.numel(), index)
        m, rows_ptr = rows.shape[0], rows.data_ptr()
    out, ldy = _output(out, m, experts.out_features, out_dtype, x, index)
    ws, n, keep = _scratch(gemm_experts_workspace_size(experts, m), x, index, workspace)
    _run("vq_gemm_experts", index, experts._ref, x.data_ptr(), _DTYPE[x.dtype], x_rows, ldx, rows_ptr,
         offsets.data_ptr(), m, out.data_ptr(), _DTYPE[out.dtype], ldy, ws, n)
    return out


def combine_rows(z: torch.Tensor, pos: torch.Tensor, weight: torch.Tensor, out_dtype=torch.bfloat16,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [T][n] = sum_j weight[t][j] z[pos[t][j]] over a token's picks (vq_combine_rows)."""
    index = z.get_device()
    ldz = _matrix(z, "z", _DTYPE, index)
    z_rows, n = z.shape
    _matrix(pos, "pos", _INT32, index)
    t, k = pos.shape
    if not pos.is_contiguous():
        _refuse(pos, "pos", "contiguous")
    ldw = _matrix(weight, "weight", _FLOAT32, index, k)
    if weight.shape[0] != t:
        _refuse(weight, "weight", f"{t} x {k}")
    out, ldy = _output(out, t, n, out_dtype, z, index)
    _run("vq_combine_rows", index, z.data_ptr(), _DTYPE[z.dtype], z_rows, n, ldz, pos.data_ptr(), weight.data_ptr(),
         ldw, t, k, out.data_ptr(), _DTYPE[out.dtype], ldy)
    return out


def kernel_launches() -> int:
    """Kernels this library has launched in this process (host counter)."""
    return int(lib().vq_kernel_launches())


def abi_version() -> int:
    return lib().vq_abi_version()


def status_string(status: int) -> str:
    return lib().vq_status_string(status).decode()
