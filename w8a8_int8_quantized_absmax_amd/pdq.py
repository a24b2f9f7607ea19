"""Thin Python binding of libpdq (include/pdq.h), same names without the prefix.

Argument marshalling only: every computation runs in the HIP kernels behind
the C ABI.  PyTorch provides device memory (outputs are allocated with
torch.empty on the input's device) and the stream (the current stream).
There is no fallback: if libpdq.so is missing or a call fails, an exception
is raised.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import re

import torch

LIB_PATH = os.environ.get("PDQ_LIB") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                      "libpdq.so")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pdq.h")

F32, BF16, F16 = 0, 1, 2
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}

_vp, _i64, _f32, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int32, ctypes.c_size_t

SIGNATURES = {
    "pdq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "pdq_quantize_weight": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "pdq_calibrate_static": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "pdq_linear_prefill": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _i64,
                                          _vp, _vp, _vp, _i64, _vp, _vp]),
    "pdq_linear_decode": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _f32, _i32, _vp, _vp,
                                         _vp, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp]),
    "pdq_quantize_per_token": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "pdq_gemm_per_token": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp,
                                          _vp]),
    "pdq_quantize_static": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _f32, _i32, _vp, _vp,
                                           _vp]),
    "pdq_gemm_static": (ctypes.c_int, [_vp, _i64, _i64, _f32, _i32, _vp, _vp, _vp, _vp, _i64, _vp,
                                       _i64, _vp, _vp]),
    "pdq_quantize_per_token_asym": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp,
                                                   _vp]),
    "pdq_gemm_per_token_asym": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp,
                                               _i64, _vp, _vp]),
    "pdq_linear_prefill_asym": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                               _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "pdq_calibrate_static_sym": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "pdq_quantize_static_sym": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _f32, _vp, _vp, _vp]),
    "pdq_linear_static_sym": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _i64,
                                             _vp, _vp, _i64, _vp, _vp, _vp]),
    "pdq_calibrate_zeropoint": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "pdq_quantize_zeropoint": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _f32, _i32, _vp, _vp, _vp]),
    "pdq_linear_zeropoint": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _f32, _i32, _vp, _vp, _vp, _vp,
                                            _i64, _vp, _vp, _i64, _vp, _vp, _vp]),
    "pdq_silu_mul_quantize_per_token": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _i64, _i64, _i64, _vp, _vp,
                                                       _vp, _i64, _vp]),
    "pdq_linear_prefill_silu_mul": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _i64, _i64, _i64, _vp, _vp, _vp,
                                                   _i64, _vp, _vp, _vp, _i64, _vp, _vp]),
    "pdq_linear_int8_outlier_workspace": (_sz, [_i64, _i64, _i64, _i64]),
    "pdq_weight_bytes": (_sz, [_i64, _i64]),
    "pdq_act_bytes": (_sz, [_i64, _i64]),
    "pdq_gemm_kernel": (ctypes.c_int, [_i64, _i64]),
    "pdq_skinny_channels": (ctypes.c_int, [_i64, _i64]),
    "pdq_pack_int8": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _vp]),
    "pdq_unpack_int8": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i64, _vp]),
    "pdq_linear_int8_outlier": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _f32, _vp, _vp,
                                               _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp,
                                               _i64, _vp, _sz, _vp, _vp]),
    "pdq_noalloc_scratch_bytes": (_sz, []),
    "pdq_linear_int8_outlier_noalloc": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _f32, _vp, _vp,
                                                       _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp,
                                                       _i64, _vp, _vp]),
    "pdq_kv_append": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _i64,
                                     ctypes.c_int, _vp, _vp, _vp, _i64, _vp]),
    "pdq_kv_attention_workspace": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "pdq_kv_attention": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _f32, _f32, _i64, _vp, _vp,
                                        _vp, _i64, _vp, _vp, _sz, _vp]),
    "pdq_fp8_bytes": (_sz, [_i64, _i64]),
    "pdq_fp8_scale_pitch": (_i64, [_i64]),
    "pdq_quantize_weight_fp8": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp]),
    "pdq_pack_weight_fp8": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "pdq_quantize_fp8": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "pdq_gemm_fp8": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, ctypes.c_int, _vp, _i64, _vp, ctypes.c_int, _i64,
                                    _vp]),
    "pdq_gemm_fp8_tile": (ctypes.c_int, [_i64, _i64, _i64, ctypes.c_int]),
    "pdq_linear_fp8_workspace": (_sz, [_i64, _i64]),
    "pdq_linear_fp8": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, ctypes.c_int, _vp, _i64, _vp,
                                      ctypes.c_int, _i64, _vp, _sz, _vp]),
    "pdq_route_workspace": (_sz, [_i64, _i64]),
    "pdq_route_experts": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                         _vp]),
    "pdq_experts_fp8_workspace": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "pdq_experts_fp8": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
}

_lib = None


class PdqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")


def header_functions(path: str = HEADER) -> list[str]:
    """Names of the functions include/pdq.h declares."""
    text = open(path).read()
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(pdq_\w+)\s*\(", text, flags=re.M)))


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                               "(python -m w8a8_int8_quantized_absmax_amd.build_lib)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pdq_status_string(status).decode()


def _call(name: str, *args) -> None:
    st = getattr(lib(), name)(*args)
    if st != 0:
        raise PdqError(name, st)


def _p(t):
    if t is None:
        return None
    return ctypes.c_void_p((t.data if isinstance(t, Codes) else t).data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check_mat(t: torch.Tensor, name: str, dtypes=_DT):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2 or (t.numel() > 0 and t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit stride in the last dimension")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")


def _ld(t: torch.Tensor) -> int:
    """Row pitch in elements (a single or empty row has no meaningful stride)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


# ---------------------------------------------------------------------------

def weight_bytes(n: int, k: int) -> int:
    """Bytes of the packed INT8 weight of N output channels x K (include/pdq.h)."""
    return int(lib().pdq_weight_bytes(n, k))


def act_bytes(m: int, k: int) -> int:
    """Bytes of the packed INT8 activation codes of M rows x K (include/pdq.h)."""
    return int(lib().pdq_act_bytes(m, k))


def unpack(buf: torch.Tensor, rows: int, k: int, padded: bool = False):
    """The codes [rows, k] of a packed INT8 matrix (weight or activations) as a host int8 array.

    Layout (include/pdq.h): 1024-byte blocks of 16 rows x 64 K values, block
    (g, s) at (g * ceil(K / 64) + s) * 1024, row r at r * 64 in it, its
    16-byte chunk c at position c ^ ((r >> 2) & 3).  padded: the whole
    [16 ceil(rows / 16), 64 ceil(k / 64)] matrix, padding included.
    """
    import numpy as np

    ng, kt = (rows + 15) // 16, (k + 63) // 64
    b = buf.detach().cpu().numpy()[:ng * kt * 1024].reshape(ng, kt, 16, 4, 16)
    r = np.arange(16)[:, None]
    pos = np.arange(4)[None, :] ^ ((r >> 2) & 3)  # [r, c] -> position of chunk c
    out = b[:, :, r, pos, :]                      # [ng, kt, 16, 4, 16], chunks in K order
    out = out.transpose(0, 2, 1, 3, 4).reshape(ng * 16, kt * 64)
    return out if padded else out[:rows, :k]


unpack_weight = unpack


def gemm_kernel(m: int, n: int) -> str:
    """The GEMM kernel the library runs for M activation rows x N channels: "skinny" or "tiled"."""
    return {0: "skinny", 1: "tiled"}.get(int(lib().pdq_gemm_kernel(m, n)), "none")


def pack_int8(x: torch.Tensor) -> torch.Tensor:
    """A plain int8 [rows, K] device matrix -> its packed image (pdq_weight_bytes(rows, K) bytes), the
    layout every GEMM takes its weight and activation codes in."""
    _check_mat(x, "x", (torch.int8,))
    rows, k = x.shape
    out = torch.empty(weight_bytes(rows, k), dtype=torch.int8, device=x.device)
    _call("pdq_pack_int8", _p(x), rows, k, _ld(x), _p(out), _stream(x.device))
    return out


def unpack_int8(packed: torch.Tensor, rows: int, k: int, out=None) -> torch.Tensor:
    """The packed image of an int8 [rows, K] matrix -> the plain [rows, K] int8 matrix on the device."""
    dst = out if out is not None else torch.empty((rows, k), dtype=torch.int8, device=packed.device)
    _call("pdq_unpack_int8", _p(packed), rows, k, _p(dst), _ld(dst), _stream(packed.device))
    return dst


def skinny_channels(m: int, n: int) -> int:
    """Weight channels per workgroup of the skinny kernel for M rows x N channels (16 .. 64)."""
    return int(lib().pdq_skinny_channels(m, n))


class Codes:
    """INT8 activation codes of a [rows, k] matrix in the packed layout (include/pdq.h).

    data: contiguous int8 device tensor of at least act_bytes(rows, k) bytes.
    """

    __slots__ = ("data", "rows", "k")

    def __init__(self, data: torch.Tensor, rows: int, k: int):
        if not data.is_cuda or data.dtype != torch.int8 or not data.is_contiguous():
            raise ValueError("packed codes must be a contiguous int8 device tensor")
        if data.numel() < act_bytes(rows, k):
            raise ValueError(f"{data.numel()} bytes cannot hold packed {rows} x {k} codes "
                             f"({act_bytes(rows, k)} needed)")
        self.data, self.rows, self.k = data, int(rows), int(k)

    @classmethod
    def empty(cls, rows: int, k: int, device) -> "Codes":
        return cls(torch.empty(max(act_bytes(rows, k), 1), dtype=torch.int8, device=device), rows, k)

    @property
    def shape(self):
        return (self.rows, self.k)

    def unpack(self, padded: bool = False):
        """Host int8 array [rows, k] (padded: with the zero padding rows and K values)."""
        return unpack(self.data, self.rows, self.k, padded)


def _codes_out(xq, m: int, k: int, device) -> Codes:
    if xq is None:
        return Codes.empty(m, k, device)
    if isinstance(xq, Codes):
        if xq.shape != (m, k):
            raise ValueError(f"codes of shape {xq.shape} given for a {m} x {k} activation")
        return xq
    return Codes(xq, m, k)


def _codes_in(xq) -> Codes:
    if not isinstance(xq, Codes):
        raise ValueError("xq must be packed activation codes (a Codes object)")
    return xq


def _check_weight(wq: torch.Tensor, n: int, k: int):
    if not wq.is_cuda or wq.dtype != torch.int8 or not wq.is_contiguous():
        raise ValueError("wq must be a contiguous int8 device tensor (a packed weight)")
    if wq.numel() < weight_bytes(n, k):
        raise ValueError(f"wq holds {wq.numel()} bytes, a packed {n} x {k} weight needs {weight_bytes(n, k)}")


def quantize_weight(w: torch.Tensor):
    """Per-output-channel symmetric INT8 weight -> (packed wq int8, w_scale f32 [N], colsum i32 [N])."""
    _check_mat(w, "w")
    n, k = w.shape
    wq = torch.empty(weight_bytes(n, k), dtype=torch.int8, device=w.device)
    ws = torch.empty(n, dtype=torch.float32, device=w.device)
    cs = torch.empty(n, dtype=torch.int32, device=w.device)
    _call("pdq_quantize_weight", _p(w), _DT[w.dtype], n, k, _ld(w), _p(wq), _p(ws), _p(cs),
          _stream(w.device))
    return wq, ws, cs


def minmax_state(device) -> torch.Tensor:
    """A fresh MinMax observer state {+INF, -INF}."""
    return torch.tensor([float("inf"), float("-inf")], dtype=torch.float32, device=device)


def calibrate_static(x: torch.Tensor, minmax: torch.Tensor, finalize: bool = False):
    """Update the MinMax state with batch x; if finalize, return (a_scale, a_zp) device tensors."""
    _check_mat(x, "x")
    m, k = x.shape
    s = z = None
    if finalize:
        s = torch.empty(1, dtype=torch.float32, device=x.device)
        z = torch.empty(1, dtype=torch.int32, device=x.device)
    _call("pdq_calibrate_static", _p(x), _DT[x.dtype], m, k, _ld(x), _p(minmax), _p(s), _p(z),
          _stream(x.device))
    return (s, z) if finalize else None


def linear_prefill(x, wq, w_scale, bias=None, want_acc: bool = False, out=None):
    """Per-token dynamic symmetric W8A8 linear -> dict(y bf16, xq, x_scale[, acc])."""
    _check_mat(x, "x")
    m, k = x.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    xq = Codes.empty(m, k, x.device)
    xs = torch.empty(m, dtype=torch.float32, device=x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    acc = torch.empty((m, n), dtype=torch.int32, device=x.device) if want_acc else None
    _call("pdq_linear_prefill", _p(x), _DT[x.dtype], m, k, _ld(x), _p(wq), _p(w_scale), _p(bias),
          n, _p(xq), _p(xs), _p(y), _ld(y), _p(acc), _stream(x.device))
    return dict(y=y, xq=xq, x_scale=xs, acc=acc)


def linear_prefill_asym(x, wq, w_scale, colsum, bias=None, want_acc: bool = False, out=None):
    """Per-token dynamic asymmetric W8A8 linear -> dict(y bf16, xq, x_scale, x_zp[, acc])."""
    _check_mat(x, "x")
    m, k = x.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    xq = Codes.empty(m, k, x.device)
    xs = torch.empty(m, dtype=torch.float32, device=x.device)
    xz = torch.empty(m, dtype=torch.int32, device=x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    acc = torch.empty((m, n), dtype=torch.int32, device=x.device) if want_acc else None
    _call("pdq_linear_prefill_asym", _p(x), _DT[x.dtype], m, k, _ld(x), _p(wq), _p(w_scale), _p(colsum),
          _p(bias), n, _p(xq), _p(xs), _p(xz), _p(y), _ld(y), _p(acc), _stream(x.device))
    return dict(y=y, xq=xq, x_scale=xs, x_zp=xz, acc=acc)


def quantize_per_token_asym(x, xq=None, x_scale=None, x_zp=None):
    """Per-token dynamic asymmetric INT8 -> (xq packed Codes [M,K], x_scale f32 [M], x_zp i32 [M])."""
    _check_mat(x, "x")
    m, k = x.shape
    xq = _codes_out(xq, m, k, x.device)
    xs = x_scale if x_scale is not None else torch.empty(m, dtype=torch.float32, device=x.device)
    xz = x_zp if x_zp is not None else torch.empty(m, dtype=torch.int32, device=x.device)
    _call("pdq_quantize_per_token_asym", _p(x), _DT[x.dtype], m, k, _ld(x), _p(xq), _p(xs), _p(xz),
          _stream(x.device))
    return xq, xs, xz


def gemm_per_token_asym(xq, x_scale, x_zp, wq, w_scale, colsum, bias=None, want_acc: bool = False, out=None):
    """INT8 GEMM + per-token zero-point correction + dequant epilogue -> dict(y bf16[, acc])."""
    xq = _codes_in(xq)
    m, k = xq.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    dev = xq.data.device
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    acc = torch.empty((m, n), dtype=torch.int32, device=dev) if want_acc else None
    _call("pdq_gemm_per_token_asym", _p(xq), _p(x_scale), _p(x_zp), m, k, _p(wq), _p(w_scale), _p(colsum),
          _p(bias), n, _p(y), _ld(y), _p(acc), _stream(dev))
    return dict(y=y, acc=acc)


def linear_decode(x, a_scale: float, a_zp: int, wq, w_scale, colsum, bias=None,
                  sat_count=None, want_acc: bool = False, out=None, xq=None):
    """Per-tensor static asymmetric W8A8 linear -> dict(y bf16, xq[, acc])."""
    _check_mat(x, "x")
    m, k = x.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    xq = _codes_out(xq, m, k, x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    acc = torch.empty((m, n), dtype=torch.int32, device=x.device) if want_acc else None
    _call("pdq_linear_decode", _p(x), _DT[x.dtype], m, k, _ld(x), float(a_scale), int(a_zp),
          _p(wq), _p(w_scale), _p(colsum), _p(bias), n, _p(xq), _p(y), _ld(y), _p(acc),
          _p(sat_count), _stream(x.device))
    return dict(y=y, xq=xq, acc=acc)


def calibrate_static_sym(x: torch.Tensor, minmax: torch.Tensor, finalize: bool = False):
    """Update the MinMax state with batch x; if finalize, return the tensor-wise absmax scale (device [1])."""
    _check_mat(x, "x")
    m, k = x.shape
    s = torch.empty(1, dtype=torch.float32, device=x.device) if finalize else None
    _call("pdq_calibrate_static_sym", _p(x), _DT[x.dtype], m, k, _ld(x), _p(minmax), _p(s), _stream(x.device))
    return s


def quantize_static_sym(x, a_scale: float, xq=None, sat_count=None):
    """Static tensor-wise symmetric INT8 -> xq packed Codes [M,K]."""
    _check_mat(x, "x")
    m, k = x.shape
    xq = _codes_out(xq, m, k, x.device)
    _call("pdq_quantize_static_sym", _p(x), _DT[x.dtype], m, k, _ld(x), float(a_scale), _p(xq),
          _p(sat_count), _stream(x.device))
    return xq


def linear_static_sym(x, a_scale: float, wq, w_scale, bias=None, sat_count=None, want_acc: bool = False,
                      out=None, xq=None):
    """Static tensor-wise symmetric W8A8 linear -> dict(y bf16, xq[, acc])."""
    _check_mat(x, "x")
    m, k = x.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    xq = _codes_out(xq, m, k, x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    acc = torch.empty((m, n), dtype=torch.int32, device=x.device) if want_acc else None
    _call("pdq_linear_static_sym", _p(x), _DT[x.dtype], m, k, _ld(x), float(a_scale), _p(wq), _p(w_scale),
          _p(bias), n, _p(xq), _p(y), _ld(y), _p(acc), _p(sat_count), _stream(x.device))
    return dict(y=y, xq=xq, acc=acc)


def calibrate_zeropoint(x: torch.Tensor, minmax: torch.Tensor, finalize: bool = False):
    """Update the MinMax state with batch x; if finalize, return the 254-level zero-point grid's (S, Z) device tensors."""
    _check_mat(x, "x")
    m, k = x.shape
    s = z = None
    if finalize:
        s = torch.empty(1, dtype=torch.float32, device=x.device)
        z = torch.empty(1, dtype=torch.int32, device=x.device)
    _call("pdq_calibrate_zeropoint", _p(x), _DT[x.dtype], m, k, _ld(x), _p(minmax), _p(s), _p(z),
          _stream(x.device))
    return (s, z) if finalize else None


def quantize_zeropoint(x, a_scale: float, a_zp: int, xq=None, sat_count=None):
    """Static tensor-wise zero-point INT8 (254 levels) -> xq packed Codes [M,K]."""
    _check_mat(x, "x")
    m, k = x.shape
    xq = _codes_out(xq, m, k, x.device)
    _call("pdq_quantize_zeropoint", _p(x), _DT[x.dtype], m, k, _ld(x), float(a_scale), int(a_zp), _p(xq),
          _p(sat_count), _stream(x.device))
    return xq


def linear_zeropoint(x, a_scale: float, a_zp: int, wq, w_scale, colsum, bias=None, sat_count=None,
                     want_acc: bool = False, out=None, xq=None):
    """Static tensor-wise zero-point W8A8 linear (254 levels) -> dict(y bf16, xq[, acc])."""
    _check_mat(x, "x")
    m, k = x.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    xq = _codes_out(xq, m, k, x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    acc = torch.empty((m, n), dtype=torch.int32, device=x.device) if want_acc else None
    _call("pdq_linear_zeropoint", _p(x), _DT[x.dtype], m, k, _ld(x), float(a_scale), int(a_zp), _p(wq),
          _p(w_scale), _p(colsum), _p(bias), n, _p(xq), _p(y), _ld(y), _p(acc), _p(sat_count), _stream(x.device))
    return dict(y=y, xq=xq, acc=acc)


def int8_outlier_workspace_bytes(m: int, n: int, k: int, max_outliers: int) -> int:
    return int(lib().pdq_linear_int8_outlier_workspace(m, n, k, max_outliers))


def linear_int8_outlier(x, threshold: float, wq, w_scale, w16, bias=None, max_outliers: int = 64,
                        want_acc: bool = False, workspace=None, out=None):
    """LLM.int8() vector-wise INT8 + 16-bit outlier decomposition -> dict(y, xq, x_scale, idx, count[, acc])."""
    _check_mat(x, "x")
    _check_mat(w16, "w16")
    m, k = x.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    dev = x.device
    max_outliers = min(max_outliers, k)
    xq = Codes.empty(m, k, dev)
    xs = torch.empty(m, dtype=torch.float32, device=dev)
    idx = torch.empty(max(max_outliers, 1), dtype=torch.int32, device=dev)
    cnt = torch.empty(1, dtype=torch.int32, device=dev)
    y = out if out is not None else torch.empty((m, n), dtype=x.dtype, device=dev)
    acc = torch.empty((m, n), dtype=torch.int32, device=dev) if want_acc else None
    need = int8_outlier_workspace_bytes(m, n, k, max_outliers)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _call("pdq_linear_int8_outlier", _p(x), _DT[x.dtype], m, k, _ld(x), float(threshold), _p(wq),
          _p(w_scale), _p(w16), _ld(w16), _p(bias), n, _p(y), _ld(y), _p(xq), _p(xs), _p(idx),
          _p(cnt), max_outliers, _p(workspace), workspace.numel(), _p(acc), _stream(dev))
    return dict(y=y, xq=xq, x_scale=xs, idx=idx, count=cnt, acc=acc)


def linear_int8_outlier_noalloc(x, threshold: float, wq, w_scale, w16, bias=None, max_outliers: int = 64,
                                want_acc: bool = False, out=None, xq=None, x_scale=None, idx=None, count=None):
    """linear_int8_outlier on the library's own scratch instead of a workspace (the
    call itself allocates nothing; outputs not given are allocated here)."""
    _check_mat(x, "x")
    _check_mat(w16, "w16")
    m, k = x.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    dev = x.device
    max_outliers = min(max_outliers, k)
    xq = _codes_out(xq, m, k, dev)
    xs = x_scale if x_scale is not None else torch.empty(m, dtype=torch.float32, device=dev)
    idx = idx if idx is not None else torch.empty(max(max_outliers, 1), dtype=torch.int32, device=dev)
    cnt = count if count is not None else torch.empty(1, dtype=torch.int32, device=dev)
    y = out if out is not None else torch.empty((m, n), dtype=x.dtype, device=dev)
    acc = torch.empty((m, n), dtype=torch.int32, device=dev) if want_acc else None
    _call("pdq_linear_int8_outlier_noalloc", _p(x), _DT[x.dtype], m, k, _ld(x), float(threshold), _p(wq),
          _p(w_scale), _p(w16), _ld(w16), _p(bias), n, _p(y), _ld(y), _p(xq), _p(xs), _p(idx),
          _p(cnt), max_outliers, _p(acc), _stream(dev))
    return dict(y=y, xq=xq, x_scale=xs, idx=idx, count=cnt, acc=acc)


def noalloc_scratch_bytes() -> int:
    return int(lib().pdq_noalloc_scratch_bytes())


def quantize_per_token(x, xq=None, x_scale=None):
    """Per-token dynamic symmetric INT8 -> (xq packed Codes [M,K], x_scale f32 [M])."""
    _check_mat(x, "x")
    m, k = x.shape
    xq = _codes_out(xq, m, k, x.device)
    xs = x_scale if x_scale is not None else torch.empty(m, dtype=torch.float32, device=x.device)
    _call("pdq_quantize_per_token", _p(x), _DT[x.dtype], m, k, _ld(x), _p(xq), _p(xs), _stream(x.device))
    return xq, xs


_HALF = (torch.bfloat16, torch.float16)


def _check_gate_up(gate, up):
    _check_mat(gate, "gate", _HALF)
    _check_mat(up, "up", _HALF)
    if up.shape != gate.shape or up.dtype != gate.dtype:
        raise ValueError("gate and up must have the same shape and dtype")
    return gate.shape


def silu_mul_quantize_per_token(gate, up, xq=None, x_scale=None, h=None):
    """h = SiLU(gate) * up (rounded to gate's 16-bit dtype) quantized per token
    -> (xq packed Codes [M,K], x_scale f32 [M]).  h: optional [M,K] tensor of
    that dtype that also receives the product."""
    m, k = _check_gate_up(gate, up)
    xq = _codes_out(xq, m, k, gate.device)
    xs = x_scale if x_scale is not None else torch.empty(m, dtype=torch.float32, device=gate.device)
    if h is not None:
        _check_mat(h, "h", (gate.dtype,))
        if h.shape != gate.shape:
            raise ValueError("h must have gate's shape")
    _call("pdq_silu_mul_quantize_per_token", _p(gate), _p(up), _DT[gate.dtype], m, k, _ld(gate), _ld(up),
          _p(xq), _p(xs), _p(h), _ld(h) if h is not None else 0, _stream(gate.device))
    return xq, xs


def linear_prefill_silu_mul(gate, up, wq, w_scale, bias=None, want_acc: bool = False, out=None):
    """Down projection of h = SiLU(gate) * up, per-token dynamic symmetric W8A8
    -> dict(y bf16, xq, x_scale[, acc]); K is the intermediate size."""
    m, k = _check_gate_up(gate, up)
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    xq = Codes.empty(m, k, gate.device)
    xs = torch.empty(m, dtype=torch.float32, device=gate.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=gate.device)
    acc = torch.empty((m, n), dtype=torch.int32, device=gate.device) if want_acc else None
    _call("pdq_linear_prefill_silu_mul", _p(gate), _p(up), _DT[gate.dtype], m, k, _ld(gate), _ld(up), _p(wq),
          _p(w_scale), _p(bias), n, _p(xq), _p(xs), _p(y), _ld(y), _p(acc), _stream(gate.device))
    return dict(y=y, xq=xq, x_scale=xs, acc=acc)


def gemm_per_token(xq, x_scale, wq, w_scale, bias=None, want_acc: bool = False, out=None):
    """INT8 GEMM + per-token/per-channel dequant epilogue -> dict(y bf16[, acc])."""
    xq = _codes_in(xq)
    m, k = xq.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    dev = xq.data.device
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    acc = torch.empty((m, n), dtype=torch.int32, device=dev) if want_acc else None
    _call("pdq_gemm_per_token", _p(xq), _p(x_scale), m, k, _p(wq), _p(w_scale), _p(bias), n, _p(y),
          _ld(y), _p(acc), _stream(dev))
    return dict(y=y, acc=acc)


def quantize_static(x, a_scale: float, a_zp: int, xq=None, sat_count=None):
    """Per-tensor static asymmetric INT8 -> xq packed Codes [M,K]."""
    _check_mat(x, "x")
    m, k = x.shape
    xq = _codes_out(xq, m, k, x.device)
    _call("pdq_quantize_static", _p(x), _DT[x.dtype], m, k, _ld(x), float(a_scale), int(a_zp), _p(xq),
          _p(sat_count), _stream(x.device))
    return xq


def gemm_static(xq, a_scale: float, a_zp: int, wq, w_scale, colsum, bias=None, want_acc: bool = False,
                out=None):
    """INT8 GEMM + zero-point correction + dequant epilogue -> dict(y bf16[, acc])."""
    xq = _codes_in(xq)
    m, k = xq.shape
    n = w_scale.shape[0]
    _check_weight(wq, n, k)
    dev = xq.data.device
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    acc = torch.empty((m, n), dtype=torch.int32, device=dev) if want_acc else None
    _call("pdq_gemm_static", _p(xq), m, k, float(a_scale), int(a_zp), _p(wq), _p(w_scale), _p(colsum),
          _p(bias), n, _p(y), _ld(y), _p(acc), _stream(dev))
    return dict(y=y, acc=acc)


# ---- the INT8 key/value cache ---------------------------------------------

class _KVCacheC(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("pages", _i64), ("heads", _i32),
                ("page", _i32), ("dim", _i32)]


class _KVBatchC(ctypes.Structure):
    _fields_ = [("page_table", _vp), ("ldt", _i64), ("seq_len", _vp), ("cu_q", _vp), ("batch", _i32),
                ("max_pages", _i32)]


def _check_dense(t, name, dtype, shape=None):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} device tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(shape)} needed")


class _Fixed:
    """Objects whose calls go by the addresses and sizes that were checked when they were made: an attribute set afterwards
    would change neither.  (In place their tensors may change; what makes such an object sets it by _put.)  A copy is made
    of _parts, the constructor's arguments: its addresses are its own."""

    __slots__ = ()

    def __reduce__(self):
        return type(self), self._parts()

    def __setattr__(self, name, value):
        raise AttributeError(f"{type(self).__name__}.{name} cannot be set: its calls go by what it was made of; make another")

    def __delattr__(self, name):
        raise AttributeError(f"{type(self).__name__}.{name} cannot be deleted")

    def _put(self, **values):
        for name, value in values.items():
            object.__setattr__(self, name, value)


class KVCache(_Fixed):
    """A pool of pages of the INT8 key/value cache (include/pdq.h, pdq_kv_cache).

    k [pages, heads, page, dim] and v [pages, heads, page / 4, dim, 4] int8,
    k_scale and v_scale [pages, heads] float32, all contiguous on one device.
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "pages", "heads", "page", "dim", "device", "index", "_c", "_ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if k.dim() != 4:
            raise ValueError("k must be [pages, heads, page, dim]")
        pages, heads, page, dim = k.shape
        _check_dense(k, "k", torch.int8)
        _check_dense(v, "v", torch.int8, (pages, heads, page // 4, dim, 4))
        _check_dense(k_scale, "k_scale", torch.float32, (pages, heads))
        _check_dense(v_scale, "v_scale", torch.float32, (pages, heads))
        if not k.device == v.device == k_scale.device == v_scale.device:
            raise ValueError("the cache's tensors must be on one device")
        c = _KVCacheC(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, heads, page, dim)
        self._put(k=k, v=v, k_scale=k_scale, v_scale=v_scale, pages=pages, heads=heads, page=page, dim=dim, device=k.device,
                  index=k.get_device(), _c=c, _ref=ctypes.byref(c))

    def _parts(self):
        return self.k, self.v, self.k_scale, self.v_scale

    @classmethod
    def empty(cls, pages: int, heads: int, dim: int, page: int = 64, device="cuda") -> "KVCache":
        return cls(torch.empty((pages, heads, page, dim), dtype=torch.int8, device=device),
                   torch.empty((pages, heads, page // 4, dim, 4), dtype=torch.int8, device=device),
                   torch.empty((pages, heads), dtype=torch.float32, device=device),
                   torch.empty((pages, heads), dtype=torch.float32, device=device))


class KVBatch(_Fixed):
    """The sequences of a call (include/pdq.h, pdq_kv_batch): page_table int32
    [batch, max_pages], seq_len int32 [batch] (the new tokens included), cu_q int32
    [batch + 1] row offsets of the new tokens, or None: one row a sequence.  The
    tensors are read when the calls run on the device, so that a program may
    update them in place between calls (or between replays of a graph)."""

    __slots__ = ("page_table", "seq_len", "cu_q", "batch", "device", "index", "_c", "_ref")

    def __init__(self, page_table: torch.Tensor, seq_len: torch.Tensor, cu_q: torch.Tensor | None = None):
        _check_mat(page_table, "page_table", (torch.int32,))
        batch, max_pages = page_table.shape
        _check_dense(seq_len, "seq_len", torch.int32, (batch,))
        if cu_q is not None:
            _check_dense(cu_q, "cu_q", torch.int32, (batch + 1,))
        if page_table.device != seq_len.device or (cu_q is not None and cu_q.device != seq_len.device):
            raise ValueError("the batch's tensors must be on one device")
        c = _KVBatchC(page_table.data_ptr(), _ld(page_table), seq_len.data_ptr(),
                      cu_q.data_ptr() if cu_q is not None else None, batch, max_pages)
        self._put(page_table=page_table, seq_len=seq_len, cu_q=cu_q, batch=batch, device=seq_len.device,
                  index=seq_len.get_device(), _c=c, _ref=ctypes.byref(c))

    def _parts(self):
        return self.page_table, self.seq_len, self.cu_q


def _check_kv_rows(t, name, cache, heads=None, dtype=None):
    """A [tokens, heads, dim] operand, the heads of a row side by side -> its row pitch."""
    if t.get_device() != cache.index:
        raise ValueError(f"{name}, the cache and the batch must be on one device")
    if t.dtype not in _HALF or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    shape, dim = t.shape, cache.dim
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} of shape {tuple(shape)} given, [tokens, "
                         f"{heads if heads is not None else 'heads'}, {dim}] needed")
    rows, each, _ = shape
    pitch, head, one = t.stride()
    if rows and (one != 1 or (each > 1 and head != dim)):
        raise ValueError(f"{name}: the heads of a row must lie side by side")
    return pitch if rows > 1 else each * dim


def _dense2(t):
    """Whether a 2-D tensor is contiguous (is_contiguous() costs more than the strides)."""
    return t.stride() == (t.shape[1], 1) or t.is_contiguous()


_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _kv_call(fn, index: int, *args) -> None:
    """A key/value call on the current stream of device `index`, with that device current.  These calls run once a
    layer and token, where the host's microseconds count: the raw stream is asked for, no stream object made."""
    if index != _current_device():
        with torch.cuda.device(index):
            return _kv_call(fn, index, *args)
    st = getattr(_lib or lib(), fn)(*args, _raw_stream(index))
    if st != 0:
        raise PdqError(fn, st)


def kv_append(k, v, cache: KVCache, batch: KVBatch, q=None, cos=None, sin=None, interleaved: bool = False,
              q_out=None):
    """Rotates k (and q) by position, codes k and v with one scale a page and head,
    and writes them into the cache -> the rotated q (None without q).

    k, v: [tokens, heads, dim] bf16 or f16; q: [tokens, hq, dim]; cos, sin: float32
    [positions, rot / 2] (None: no rotation); q_out: where the rotated q goes (q itself
    for in place)."""
    index = cache.index
    if batch.index != index:
        raise ValueError("the cache and the batch must be on one device")
    ldk = _check_kv_rows(k, "k", cache, cache.heads)
    tokens, dtype = k.shape[0], k.dtype
    ldv = _check_kv_rows(v, "v", cache, cache.heads, dtype)
    if v.shape[0] != tokens:
        raise ValueError("k and v must have the same rows")
    if (cos is None) != (sin is None) or (q is not None and cos is None):
        raise ValueError("a rotation needs both tables, and q is there to be rotated")
    positions = rot = hq = ldq = ldqo = 0
    if cos is not None:
        if (cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.dim() != 2 or cos.shape != sin.shape
                or cos.get_device() != index or sin.get_device() != index or not _dense2(cos) or not _dense2(sin)):
            raise ValueError("cos and sin must be contiguous float32 [positions, rot / 2] on k's device")
        positions, rot = cos.shape
        rot *= 2
    if q is not None:
        ldq = _check_kv_rows(q, "q", cache, None, dtype)
        if q.shape[0] != tokens:
            raise ValueError("q and k must have the same rows")
        hq = q.shape[1]
        if q_out is None:
            q_out = q.new_empty((tokens, hq, cache.dim))
            ldqo = hq * cache.dim
        else:
            ldqo = _check_kv_rows(q_out, "q_out", cache, hq, dtype)
            if q_out.shape[0] != tokens:
                raise ValueError("q_out and q must have the same rows")
    elif q_out is not None:
        raise ValueError("q_out without q")
    _kv_call("pdq_kv_append", index, k.data_ptr(), v.data_ptr(), q.data_ptr() if q is not None else None, _DT[dtype],
             tokens, hq, ldk, ldv, ldq, cos.data_ptr() if cos is not None else None,
             sin.data_ptr() if sin is not None else None, positions, rot, 1 if interleaved else 0, cache._ref, batch._ref,
             q_out.data_ptr() if q_out is not None else None, ldqo)
    return q_out


@functools.lru_cache(maxsize=4096)
def kv_attention_workspace_bytes(tokens: int, batch: int, hq: int, heads: int, dim: int) -> int:
    return int(lib().pdq_kv_attention_workspace(tokens, batch, hq, heads, dim))


def kv_attention(q, cache: KVCache, batch: KVBatch, scale: float | None = None, softcap: float = 0.0,
                 window: int = 0, alibi_slopes=None, prefix_len=None, want_lse: bool = False, out=None, lse=None,
                 workspace=None):
    """Attention of the new rows q [tokens, hq, dim] over the cache -> dict(y of q's
    shape and dtype, lse float32 [tokens, hq] or None).

    scale: 1 / sqrt(dim) by default; softcap > 0: scores capped by softcap *
    tanh(z / softcap); window > 0: the last window keys; alibi_slopes float32 [hq]:
    slope * (key - row) added, the signed distance (keys ahead of a row, which only
    prefix_len shows, gain by a positive slope); prefix_len int32 [batch]: tokens that
    every row sees.  A batch that mixes single rows with a prompt's chunk is faster as
    two calls, the second's cu_q beginning behind the first's rows."""
    index = cache.index
    if batch.index != index:
        raise ValueError("the cache and the batch must be on one device")
    ldq = _check_kv_rows(q, "q", cache)
    tokens, hq, dim = q.shape
    if alibi_slopes is not None:
        _check_dense(alibi_slopes, "alibi_slopes", torch.float32, (hq,))
        if alibi_slopes.get_device() != index:
            raise ValueError("alibi_slopes must be on q's device")
    if prefix_len is not None:
        _check_dense(prefix_len, "prefix_len", torch.int32, (batch.batch,))
        if prefix_len.get_device() != index:
            raise ValueError("prefix_len must be on q's device")
    if out is None:
        y = q.new_empty((tokens, hq, dim))  # half the time of torch.empty with a dtype and a device
        ldy = hq * dim
    else:
        y = out
        ldy = _check_kv_rows(y, "out", cache, hq, q.dtype)
        if y.shape[0] != tokens:
            raise ValueError("out and q must have the same rows")
    if lse is not None:
        _check_dense(lse, "lse", torch.float32, (tokens, hq))
        if lse.get_device() != index:
            raise ValueError("lse must be on q's device")
    elif want_lse:
        lse = q.new_empty((tokens, hq), dtype=torch.float32)
    size = 0
    if workspace is None:
        size = kv_attention_workspace_bytes(tokens, batch.batch, hq, cache.heads, dim)
        if size:
            workspace = q.new_empty(size // 2)  # 16-bit values; size is a multiple of 256
    else:
        _check_dense(workspace, "workspace", torch.uint8)
        if workspace.get_device() != index:
            raise ValueError("workspace must be on q's device")
        size = workspace.numel()
    _kv_call("pdq_kv_attention", index, q.data_ptr(), _DT[q.dtype], tokens, hq, ldq, cache._ref, batch._ref,
             dim ** -0.5 if scale is None else float(scale), float(softcap), int(window),
             alibi_slopes.data_ptr() if alibi_slopes is not None else None,
             prefix_len.data_ptr() if prefix_len is not None else None, y.data_ptr(), ldy,
             lse.data_ptr() if lse is not None else None, workspace.data_ptr() if size else None, size)
    return dict(y=y, lse=lse)


# ---- 8-bit floating-point products, routing and experts -------------------

E8M0, SCALE_F32 = 0, 1
_SCORES = {"softmax": 0, "sigmoid": 1}


def fp8_bytes(rows: int, k: int) -> int:
    """Bytes of the packed FP8 codes of a [rows, k] matrix (include/pdq.h)."""
    return int(lib().pdq_fp8_bytes(rows, k))


@functools.lru_cache(maxsize=4096)
def _fp8_sizes(rows: int, k: int):
    """Bytes of packed codes, scales in a row of them."""
    return int(lib().pdq_fp8_bytes(rows, k)), int(lib().pdq_fp8_scale_pitch(k))


def _fp8_unpack(data: torch.Tensor, count: int, n: int, k: int) -> torch.Tensor:
    """Packed codes (include/pdq.h) -> [count, n, k] e4m3 on their device."""
    blocks = data[:count * fp8_bytes(n, k)].view(count, (n + 15) // 16, (k + 127) // 128 * 2, 4, 16, 16)
    rows = blocks.permute(0, 1, 4, 2, 3, 5).reshape(count, (n + 15) // 16 * 16, -1)
    return rows[:, :n, :k].contiguous().view(torch.float8_e4m3fn)


class WeightFP8(_Fixed):
    """FP8 weights with a scale for each block of 128 x 128 (include/pdq.h): one [n, k]
    matrix, or a stack of them with the leading dimensions `lead`.

    data: packed codes, uint8; scale: e8m0 (torch.float8_e8m0fnu) or float32, [*lead,
    ceil(n / 128), pitch].  quantize_weight_fp8 and pack_weight_fp8 make them."""

    __slots__ = ("data", "scale", "lead", "n", "k", "scale_type", "device", "index", "at", "scale_at")

    def __init__(self, data: torch.Tensor, scale: torch.Tensor, n: int, k: int):
        if scale.dtype not in (torch.float8_e8m0fnu, torch.float32):
            raise ValueError(f"scale: unsupported dtype {scale.dtype}")
        _check_dense(scale, "scale", scale.dtype)
        _check_dense(data, "data", torch.uint8)
        size, pitch = _fp8_sizes(n, k)
        if scale.dim() < 2 or scale.shape[-1] != pitch or scale.shape[-2] != (n + 127) // 128:
            raise ValueError(f"scale of shape {tuple(scale.shape)} given for {n} x {k} weights")
        count = scale.numel() // max(1, scale.shape[-1] * scale.shape[-2])
        if data.numel() < count * size:
            raise ValueError(f"data holds {data.numel()} bytes, {count} packed {n} x {k} weights need {count * size}")
        if data.device != scale.device:
            raise ValueError("the weight's tensors must be on one device")
        self._put(data=data, scale=scale, n=int(n), k=int(k), lead=tuple(scale.shape[:-2]),
                  scale_type=SCALE_F32 if scale.dtype == torch.float32 else E8M0, device=data.device,
                  index=data.get_device(), at=data.data_ptr(), scale_at=scale.data_ptr())

    def _parts(self):
        return self.data, self.scale, self.n, self.k

    @property
    def shape(self):
        return (*self.lead, self.n, self.k)

    def codes(self) -> torch.Tensor:
        """The e4m3 codes [*lead, n, k], row-major."""
        count = 1
        for d in self.lead:
            count *= d
        return _fp8_unpack(self.data, count, self.n, self.k).view(self.shape)

    def scales(self) -> torch.Tensor:
        """The block scales [*lead, ceil(n / 128), ceil(k / 128)], float32."""
        return self.scale.float()[..., :(self.k + 127) // 128]


class _CodesFP8Parts:  # (what quantize_fp8 fills: a plain attribute costs the host a third of _put's)
    __slots__ = ("buffer", "rows", "k", "size", "pitch", "index")


class CodesFP8(_Fixed, _CodesFP8Parts):
    """FP8 activation codes of a [rows, k] matrix, packed, and their groups' e8m0 scales behind them,
    in one buffer (16-byte aligned)."""

    __slots__ = ()

    def __init__(self, buffer: torch.Tensor, rows: int, k: int):
        size, pitch = _fp8_sizes(rows, k)
        if not buffer.is_cuda or not buffer.is_contiguous() or buffer.nbytes < size + rows * pitch:
            raise ValueError(f"packed {rows} x {k} codes with their scales need a contiguous device tensor of "
                             f"{size + rows * pitch} bytes")
        self._put(buffer=buffer, rows=rows, k=k, size=size, pitch=pitch, index=buffer.get_device())

    def _parts(self):
        return self.buffer, self.rows, self.k

    @property
    def shape(self):
        return (self.rows, self.k)

    @property
    def data(self) -> torch.Tensor:
        """The packed codes, uint8."""
        return self.buffer.view(-1).view(torch.uint8)[:self.size]

    @property
    def scale(self) -> torch.Tensor:
        """The groups' scales [rows, pitch], torch.float8_e8m0fnu."""
        flat = self.buffer.view(-1).view(torch.uint8)[self.size:self.size + self.rows * self.pitch]
        return flat.view(torch.float8_e8m0fnu).view(self.rows, self.pitch)

    def codes(self) -> torch.Tensor:
        """The e4m3 codes [rows, k], row-major."""
        return _fp8_unpack(self.data, 1, self.rows, self.k)[0]

    def values(self) -> torch.Tensor:
        """What the codes and scales stand for, float32 [rows, k]."""
        return self.codes().float() * self.scale.float().repeat_interleave(128, 1)[:, :self.k]


def _codes_fp8(like, m, k, index):
    """New codes of a [m, k] matrix, in like's dtype (a new tensor of another one costs the host more)."""
    size, pitch = _fp8_sizes(m, k)
    c = _CodesFP8Parts()
    c.buffer, c.rows, c.k = like.new_empty((size + m * pitch + 3) // like.element_size() + 1), m, k
    c.size, c.pitch, c.index = size, pitch, index
    c.__class__ = CodesFP8
    return c


def _stack_shape(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() < 2:
        raise ValueError(f"{name} must be [..., n, k]")
    count = 1
    for d in t.shape[:-2]:
        count *= d
    return count, t.shape[-2], t.shape[-1]


def quantize_weight_fp8(w: torch.Tensor) -> WeightFP8:
    """Weights [..., n, k] of f32, bf16 or f16 -> FP8 with a power of two as scale for each block
    of 128 x 128."""
    count, n, k = _stack_shape(w, "w")
    if w.dtype not in _DT:
        raise ValueError(f"w: unsupported dtype {w.dtype}")
    if not w.is_contiguous() and not (w.dim() == 2 and w.stride(1) == 1):
        raise ValueError("w must be contiguous, or 2-D with unit stride in the last dimension")
    size, pitch = _fp8_sizes(n, k)
    data = torch.empty(count * size, dtype=torch.uint8, device=w.device)
    scale = torch.empty((*w.shape[:-2], (n + 127) // 128, pitch), dtype=torch.float8_e8m0fnu, device=w.device)
    ld = _ld(w) if w.dim() == 2 else k
    _kv_call("pdq_quantize_weight_fp8", w.get_device(), w.data_ptr(), _DT[w.dtype], count, n, k, ld, n * k, data.data_ptr(),
             scale.data_ptr())
    return WeightFP8(data, scale, n, k)


def pack_weight_fp8(codes: torch.Tensor, scale: torch.Tensor) -> WeightFP8:
    """Codes [..., n, k] (torch.float8_e4m3fn) and block scales [..., ceil(n / 128), ceil(k / 128)]
    (float32 or torch.float8_e8m0fnu), as a checkpoint holds them -> the packed weight."""
    count, n, k = _stack_shape(codes, "codes")
    _check_dense(codes, "codes", torch.float8_e4m3fn)
    if scale.dtype not in (torch.float8_e8m0fnu, torch.float32):
        raise ValueError(f"scale: unsupported dtype {scale.dtype}")
    _check_dense(scale, "scale", scale.dtype, (*codes.shape[:-2], (n + 127) // 128, (k + 127) // 128))
    if scale.device != codes.device:
        raise ValueError("codes and scale must be on one device")
    size, pitch = _fp8_sizes(n, k)
    data = torch.empty(count * size, dtype=torch.uint8, device=codes.device)
    out = torch.empty((*codes.shape[:-2], (n + 127) // 128, pitch), dtype=scale.dtype, device=codes.device)
    _kv_call("pdq_pack_weight_fp8", codes.get_device(), codes.data_ptr(), scale.data_ptr(),
             SCALE_F32 if scale.dtype == torch.float32 else E8M0, count, n, k, data.data_ptr(), out.data_ptr())
    return WeightFP8(data, out, n, k)


def quantize_fp8(x: torch.Tensor) -> CodesFP8:
    """Activations [m, k] -> FP8 codes with a power of two as scale for each row and group of 128."""
    _check_mat(x, "x")
    m, k = x.shape
    index = x.get_device()
    q = _codes_fp8(x, m, k, index)
    at = q.buffer.data_ptr()
    _kv_call("pdq_quantize_fp8", index, x.data_ptr(), _DT[x.dtype], m, k, _ld(x), at, at + q.size)
    return q


def _rows(t, name, kind, dtypes):
    """_check_mat for what is called once a layer and token -> the row pitch."""
    if t.dim() != 2 or kind not in dtypes or not t.is_cuda:
        _check_mat(t, name, dtypes)
    pitch, one = t.stride()
    if one != 1:
        _check_mat(t, name, dtypes)
    return pitch if t.shape[0] > 1 else t.shape[1]


def _fp8_operands(w, k, index, bias, m, out, dtype, like):
    """The checks that linear_fp8 and gemm_fp8 share -> y, its row pitch."""
    if type(w) is not WeightFP8 or w.lead:
        raise ValueError("w must be one FP8 weight (a WeightFP8 without leading dimensions)")
    if w.k != k or w.index != index:
        raise ValueError(f"a [{w.n}, {w.k}] weight on device {w.index} does not fit activations of {k} on device {index}")
    if bias is not None:
        _check_dense(bias, "bias", torch.float32, (w.n,))
        if bias.get_device() != index:
            raise ValueError("bias must be on the weight's device")
    if out is None:
        if dtype is like.dtype and dtype in _HALF:
            return like.new_empty((m, w.n)), w.n
        if dtype not in _HALF:
            raise ValueError(f"unsupported output dtype {dtype}")
        return like.new_empty((m, w.n), dtype=dtype), w.n
    _check_mat(out, "out", _HALF)
    if tuple(out.shape) != (m, w.n) or out.get_device() != index:
        raise ValueError(f"out must be [{m}, {w.n}] on the weight's device")
    return out, _ld(out)


@functools.lru_cache(maxsize=4096)
def linear_fp8_workspace_bytes(m: int, k: int) -> int:
    return int(lib().pdq_linear_fp8_workspace(m, k))


def linear_fp8(x, w: WeightFP8, bias=None, out=None, dtype=None, workspace=None):
    """y = x W^T (+ bias) on FP8 codes -> dict(y): x [m, k] f32, bf16 or f16, coded within the call.
    (quantize_fp8 and gemm_fp8: codes for several weights.)

    y is f16 for f16 x, else bf16, or of `dtype`."""
    kind = x.dtype
    ldx = _rows(x, "x", kind, _DT)
    m, k = x.shape
    index = x.get_device()
    y, ldy = _fp8_operands(w, k, index, bias, m, out, dtype or (torch.bfloat16 if kind is torch.float32 else kind), x)
    size, at = linear_fp8_workspace_bytes(m, k), None
    if size or workspace is not None:
        workspace, size = _workspace(workspace, size, x, index)
        at = workspace.data_ptr()
    _kv_call("pdq_linear_fp8", index, x.data_ptr(), _DT[kind], m, k, ldx, w.at, w.scale_at, w.scale_type,
             bias.data_ptr() if bias is not None else None, w.n, y.data_ptr(), _DT[y.dtype], ldy, at, size)
    return {"y": y}


def gemm_fp8(xq: CodesFP8, w: WeightFP8, bias=None, out=None, dtype=torch.bfloat16):
    """The product of linear_fp8 on codes that are there already -> dict(y)."""
    if type(xq) is not CodesFP8:
        raise ValueError("xq must be FP8 activation codes (a CodesFP8 object)")
    m, k, index = xq.rows, xq.k, xq.index
    y, ldy = _fp8_operands(w, k, index, bias, m, out, dtype, xq.buffer)
    at = xq.buffer.data_ptr()
    _kv_call("pdq_gemm_fp8", index, at, at + xq.size, m, k, w.at, w.scale_at, w.scale_type,
             bias.data_ptr() if bias is not None else None, w.n, y.data_ptr(), _DT[y.dtype], ldy)
    return {"y": y}


def gemm_fp8_tile(m: int, n: int, k: int, scale_type: int = E8M0) -> int:
    """Rows of a tile where gemm_fp8 runs the tiled kernel, 0 where it runs the one for few rows."""
    return int(lib().pdq_gemm_fp8_tile(m, n, k, scale_type))


class _RouteRuleC(ctypes.Structure):
    _fields_ = [("score", _i32), ("k", _i32), ("groups", _i32), ("top_groups", _i32), ("group_score", _i32),
                ("renormalize", _i32), ("scale", _f32)]


class _RoutingC(ctypes.Structure):
    _fields_ = [("ids", _vp), ("weights", _vp), ("offsets", _vp), ("rows", _vp), ("tokens", _i64), ("experts", _i64),
                ("k", _i64)]


class _ExpertsC(ctypes.Structure):
    _fields_ = [("gate_up", _vp), ("gate_up_scale", _vp), ("down", _vp), ("down_scale", _vp), ("scale_t", ctypes.c_int),
                ("experts", _i64), ("hidden", _i64), ("inner", _i64)]


class _RoutingParts:
    __slots__ = ("_tensors", "_buffer", "tokens", "experts", "k", "index", "_at", "_c")


class Routing(_Fixed, _RoutingParts):
    """The experts of each token (include/pdq.h, pdq_route_experts): ids int32 and weights float32
    [tokens, k]; the rows token * k + slot sorted by expert: offsets int32 [experts + 1], rows int32
    [tokens * k]."""

    __slots__ = ()

    def __init__(self, ids: torch.Tensor, weights: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor):
        if ids.dim() != 2 or offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError("ids must be [tokens, k], offsets [experts + 1]")
        tokens, k = ids.shape
        _check_dense(ids, "ids", torch.int32)
        _check_dense(weights, "weights", torch.float32, (tokens, k))
        _check_dense(offsets, "offsets", torch.int32)
        _check_dense(rows, "rows", torch.int32, (tokens * k,))
        if not ids.device == weights.device == offsets.device == rows.device:
            raise ValueError("the routing's tensors must be on one device")
        tensors = (ids, weights, offsets, rows)
        self._put(_tensors=tensors, _buffer=None, tokens=tokens, experts=offsets.shape[0] - 1, k=k, index=ids.get_device(),
                  _at=tuple(t.data_ptr() for t in tensors), _c=None)

    def _ref(self):
        if self._c is None:
            self._put(_c=_RoutingC(*self._at, self.tokens, self.experts, self.k))
        return ctypes.byref(self._c)

    def _parts(self):
        return self._all()

    def _all(self):
        if self._tensors is None:  # parts of route_experts' one buffer, as tensors when they are asked for
            n, e = self.tokens * self.k, self.experts + 1
            ids, weights, rows, offsets, _ = self._buffer.split((n, n, n, e, self._buffer.shape[0] - 3 * n - e))
            self._put(_tensors=(ids.view(self.tokens, self.k), weights.view(torch.float32).view(self.tokens, self.k),
                                offsets, rows))
        return self._tensors

    @property
    def ids(self) -> torch.Tensor:
        return self._all()[0]

    @property
    def weights(self) -> torch.Tensor:
        return self._all()[1]

    @property
    def offsets(self) -> torch.Tensor:
        return self._all()[2]

    @property
    def rows(self) -> torch.Tensor:
        return self._all()[3]


@functools.lru_cache(maxsize=4096)
def route_workspace_bytes(tokens: int, experts: int) -> int:
    return int(lib().pdq_route_workspace(tokens, experts))


@functools.lru_cache(maxsize=256)
def _rule_struct(score, k, groups, top_groups, group_score, renormalize, scale):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    for v in (k, groups, top_groups, group_score):
        if not -2 ** 31 <= v < 2 ** 31:  # (the C struct's fields would lose the upper bits)
            raise ValueError(f"{v} in a routing rule")
    c = _RouteRuleC(_SCORES[score], k, groups, top_groups, group_score, renormalize, scale)
    return c, ctypes.byref(c)


def _route_rule(score, k, groups, top_groups, group_score, renormalize, scale):
    """The rule as a C struct, kept by the values alone: an object that is passed for one (a tensor) may change."""
    if not (type(k) is type(groups) is type(top_groups) is type(group_score) is int and type(scale) is float):
        k, groups, top_groups, group_score = map(operator.index, (k, groups, top_groups, group_score))
        scale = float(scale)
    return _rule_struct(score, k, groups, top_groups, group_score, 1 if renormalize else 0, scale)


def route_experts(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
                  group_score: int = 1, renormalize: bool = True, scale: float = 1.0, workspace=None) -> Routing:
    """The k experts of each token from the router's logits [tokens, experts] (f32, bf16 or f16), and
    the tokens sorted by expert.

    score: "softmax" or "sigmoid"; bias float32 [experts]: added for the choice alone; groups,
    top_groups, group_score: only the best top_groups of `groups` runs of experts take part, by the sum
    of their group_score largest; renormalize: a token's weights sum to 1, times scale."""
    kind = logits.dtype
    ldl = _rows(logits, "logits", kind, _DT)
    tokens, experts = logits.shape
    index = logits.get_device()
    if bias is not None:
        _check_dense(bias, "bias", torch.float32, (experts,))
        if bias.get_device() != index:
            raise ValueError("bias must be on logits' device")
    k = operator.index(k)
    if not 1 <= k <= experts:
        raise ValueError(f"k = {k} of {experts} experts")
    rule = _route_rule(score, k, groups, top_groups, group_score, renormalize, scale)
    n = tokens * k
    used = (3 * n + experts + 1 + 63) // 64 * 64
    size = route_workspace_bytes(tokens, experts)
    if workspace is None:  # behind the outputs, in one buffer
        buffer = logits.new_empty(used + size // 4, dtype=torch.int32)
        at = buffer.data_ptr()
        ws = at + 4 * used
    else:
        workspace, size = _workspace(workspace, size, logits, index)
        buffer = logits.new_empty(used, dtype=torch.int32)
        at = buffer.data_ptr()
        ws = workspace.data_ptr()
    offsets = at + 12 * n
    _kv_call("pdq_route_experts", index, logits.data_ptr(), _DT[kind], tokens, experts, ldl,
             bias.data_ptr() if bias is not None else None, rule[1], at, at + 4 * n, offsets, at + 8 * n, ws, size)
    r = _RoutingParts()
    r._tensors, r._buffer, r.tokens, r.experts, r.k, r.index = None, buffer, tokens, experts, k, index
    r._at, r._c = (at, at + 4 * n, offsets, at + 8 * n), None
    r.__class__ = Routing
    return r


def _workspace(workspace, size, like, index):
    """The caller's workspace, or a new one."""
    if workspace is None:
        return (like.new_empty(size // like.element_size()) if size else None), size
    _check_dense(workspace, "workspace", torch.uint8)
    if workspace.get_device() != index:
        raise ValueError("the workspace must be on the call's device")
    return workspace, workspace.numel()


@functools.lru_cache(maxsize=4096)
def experts_fp8_workspace_bytes(tokens: int, k: int, experts: int, hidden: int, inner: int) -> int:
    return int(lib().pdq_experts_fp8_workspace(tokens, k, experts, hidden, inner))


def experts_fp8(x, routing: Routing, gate_up: WeightFP8, down: WeightFP8, out=None, workspace=None):
    """The experts' layer -> dict(y of x's shape and dtype): each token's chosen gated MLPs on FP8
    weights, weighted and summed.

    x: [tokens, hidden] bf16 or f16; gate_up: a WeightFP8 [experts, 2, inner, hidden]; down:
    [experts, hidden, inner], both with scales of one type."""
    kind = x.dtype
    ldx = _rows(x, "x", kind, _HALF)
    tokens, hidden = x.shape
    index = x.get_device()
    experts, inner = routing.experts, gate_up.n
    if gate_up.lead != (experts, 2) or down.lead != (experts,) or gate_up.k != hidden or down.n != hidden or down.k != inner:
        raise ValueError(f"weights of shapes {gate_up.shape} and {down.shape} given, [{experts}, 2, inner, {hidden}] and "
                         f"[{experts}, {hidden}, inner] needed")
    if gate_up.scale_type != down.scale_type:
        raise ValueError("the weights' scales must be of one type")
    if routing.tokens != tokens:
        raise ValueError(f"the routing of {routing.tokens} tokens given for {tokens}")
    if not index == routing.index == gate_up.index == down.index:
        raise ValueError("x, the routing and the weights must be on one device")
    if out is None:
        y, ldy = x.new_empty((tokens, hidden)), hidden
    else:
        y = out
        _check_mat(y, "out", (kind,))
        if y.shape != x.shape or y.get_device() != index:
            raise ValueError("out must have x's shape and device")
        ldy = _ld(y)
    size = experts_fp8_workspace_bytes(tokens, routing.k, experts, hidden, inner)
    workspace, size = _workspace(workspace, size, x, index)
    c = _ExpertsC(gate_up.at, gate_up.scale_at, down.at, down.scale_at, gate_up.scale_type, experts, hidden, inner)
    _kv_call("pdq_experts_fp8", index, x.data_ptr(), _DT[kind], ldx, routing._ref(), ctypes.byref(c), y.data_ptr(),
             ldy, workspace.data_ptr() if size else None, size)
    return {"y": y}
