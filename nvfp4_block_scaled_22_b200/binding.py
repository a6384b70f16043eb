"""Thin ctypes binding of libnvfp4.so (the C ABI in include/nvfp4.h).

Argument marshalling only: every step of the NVFP4 path runs in the CUDA
kernels of libnvfp4.so.  PyTorch supplies device memory and streams.  There
is no CPU fallback -- loading fails loudly if the library is missing.

Function names follow the C ABI (``nvfp4_quantize`` ...), taking torch
tensors instead of raw pointers.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# The in-tree build; NVFP4_LIBRARY may name another build of the same C ABI
# (for example one compiled with a different pipeline geometry).
LIB_PATH = os.environ.get("NVFP4_LIBRARY") or os.path.join(HERE, "libnvfp4.so")

SF_SWIZZLED = 0
SF_LINEAR = 1

OP_QUANTIZE, OP_DEQUANTIZE, OP_GEMM, OP_GROUPED_GEMM, OP_QUANTIZE_GATHER, OP_ATTENTION = range(6)

STATUS_NAMES = {
    0: "NVFP4_OK", 1: "NVFP4_ERR_INVALID_ARG", 2: "NVFP4_ERR_ALIGNMENT", 3: "NVFP4_ERR_SHAPE",
    4: "NVFP4_ERR_NONFINITE", 5: "NVFP4_ERR_RANGE", 6: "NVFP4_ERR_WORKSPACE",
    7: "NVFP4_ERR_TIMEOUT", 8: "NVFP4_ERR_UNSUPPORTED_DEVICE", 9: "NVFP4_ERR_CUDA",
}

# Symbols the header declares; the library must export every one.
EXPORTED = (
    "nvfp4_codes_bytes", "nvfp4_scales_bytes", "nvfp4_workspace_bytes", "nvfp4_quantize",
    "nvfp4_global_scale", "nvfp4_quantize_gather", "nvfp4_dequantize", "nvfp4_gemm",
    "nvfp4_grouped_gemm", "nvfp4_grouped_gemm_out_scale", "nvfp4_check_status",
    "nvfp4_status_string", "nvfp4_version",
    "nvfp4_launch_count", "nvfp4_set_wait_limit_cycles", "nvfp4_set_gemm_pairs",
    "nvfp4_quantize_noalloc", "nvfp4_quantize_rht", "nvfp4_quantize_t", "nvfp4_quantize_2d",
    "nvfp4_quantize_sr", "nvfp4_mx_scales_bytes", "nvfp4_quantize_mx", "nvfp4_dequantize_mx",
    "nvfp4_gemm_mx", "nvfp4_moe_combine", "nvfp4_dequantize_fp8", "nvfp4_quantize_swiglu",
    "nvfp4_attention_decode", "nvfp4_gather_rows", "nvfp4_rope_inv_freq", "nvfp4_rope_table",
    "nvfp4_rope", "nvfp4_kv_write", "nvfp4_kv_read", "nvfp4_attention_paged_scratch_bytes",
    "nvfp4_attention_decode_paged",
)

ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "bands": 3, "ramp": 4}


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class CTensor(C.Structure):
    """Mirror of ``nvfp4_tensor``."""
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("global_", C.c_void_p),
                ("rows", C.c_int64), ("cols", C.c_int64), ("sf_layout", C.c_int32)]


_lib = None


def lib() -> C.CDLL:
    """Load libnvfp4.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libnvfp4.so not built at {LIB_PATH}; run "
                              "python -m nvfp4_block_scaled_22_b200.build")
        L = C.CDLL(LIB_PATH)
        i64, i32, vp, sz = C.c_int64, C.c_int32, C.c_void_p, C.c_size_t
        T = C.POINTER(CTensor)
        sig = {
            "nvfp4_codes_bytes": (sz, [i64, i64]),
            "nvfp4_scales_bytes": (sz, [i64, i64, i32]),
            "nvfp4_workspace_bytes": (sz, [i32, i64, i64, i64, i32]),
            "nvfp4_quantize": (C.c_int, [vp, i64, T, i32, vp, sz, vp]),
            "nvfp4_global_scale": (C.c_int, [vp, i64, i64, i64, vp, vp, sz, vp]),
            "nvfp4_quantize_gather": (C.c_int, [vp, i64, i64, vp, T, i32, vp, sz, vp]),
            "nvfp4_dequantize": (C.c_int, [T, vp, i64, vp]),
            "nvfp4_gemm": (C.c_int, [T, T, vp, i64, vp, sz, vp]),
            "nvfp4_grouped_gemm": (C.c_int, [i32, vp, vp, T, T, vp, i64, vp, i64, vp, sz, vp]),
            "nvfp4_grouped_gemm_out_scale": (C.c_int, [i32, vp, vp, T, T, vp, i64, vp, i64, vp, vp,
                                                       sz, vp]),
            "nvfp4_check_status": (C.c_int, [vp, vp]),
            "nvfp4_status_string": (C.c_char_p, [C.c_int]),
            "nvfp4_version": (i32, []),
            "nvfp4_launch_count": (i64, []),
            "nvfp4_gather_rows": (C.c_int, [T, vp, T, vp, sz, vp]),
            "nvfp4_set_wait_limit_cycles": (C.c_longlong, [C.c_longlong]),
            "nvfp4_set_gemm_pairs": (i32, [i32]),
            "nvfp4_quantize_noalloc": (C.c_int, [vp, i64, T, i32, vp]),
            "nvfp4_quantize_rht": (C.c_int, [vp, i64, C.c_uint32, T, i32, vp, sz, vp]),
            "nvfp4_quantize_t": (C.c_int, [vp, i64, i32, C.c_uint32, T, i32, vp, sz, vp]),
            "nvfp4_quantize_2d": (C.c_int, [vp, i64, T, T, i32, vp, sz, vp]),
            "nvfp4_quantize_sr": (C.c_int, [vp, i64, i32, i32, C.c_uint32, C.c_uint64, T, i32, vp,
                                            sz, vp]),
            "nvfp4_mx_scales_bytes": (sz, [i64, i64, i32]),
            "nvfp4_quantize_mx": (C.c_int, [vp, i64, T, vp, sz, vp]),
            "nvfp4_dequantize_mx": (C.c_int, [T, vp, i64, vp]),
            "nvfp4_gemm_mx": (C.c_int, [T, T, vp, i64, vp, sz, vp]),
            "nvfp4_moe_combine": (C.c_int, [vp, i64, i64, vp, vp, i64, i32, i64, vp, i64, vp]),
            "nvfp4_dequantize_fp8": (C.c_int, [T, vp, i64, vp, vp]),
            "nvfp4_quantize_swiglu": (C.c_int, [vp, i64, T, vp, sz, vp]),
            "nvfp4_attention_decode": (C.c_int, [vp, i64, i32, T, T, i32, C.c_float, vp, i64, vp, sz,
                                                 vp]),
            "nvfp4_rope_inv_freq": (C.c_int, [i32, C.c_double, i32, C.c_double, C.c_double, C.c_double,
                                              C.c_double, vp]),
            "nvfp4_rope_table": (C.c_int, [vp, i32, i64, i64, C.c_double, vp, vp]),
            "nvfp4_rope": (C.c_int, [vp, i64, i64, i64, i32, i32, vp, vp, i64, i32, i32, i32, vp, i64,
                                     i64, vp, sz, vp]),
            "nvfp4_kv_write": (C.c_int, [vp, i64, i64, vp, i64, i64, i64, i32, i32, vp, T, T, vp, vp,
                                         i64, i32, i32, vp, sz, vp]),
            "nvfp4_kv_read": (C.c_int, [T, T, vp, i64, vp, i64, vp, i64, vp, sz, vp]),
            "nvfp4_attention_paged_scratch_bytes": (sz, [i32, i32, i32]),
            "nvfp4_attention_decode_paged": (C.c_int, [vp, i64, i64, i32, i32, T, T, i32, vp, i64, i32,
                                                       vp, i32, C.c_float, vp, i64, i64, vp, vp, sz,
                                                       vp, sz, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(st: int, where: str):
    if st != 0:
        raise NVFP4Error(st, where)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


# ------------------------------------------------------------------ sizes
def nvfp4_codes_bytes(rows: int, cols: int) -> int:
    return int(lib().nvfp4_codes_bytes(rows, cols))


def nvfp4_scales_bytes(rows: int, cols: int, layout: int = SF_SWIZZLED) -> int:
    return int(lib().nvfp4_scales_bytes(rows, cols, layout))


def nvfp4_workspace_bytes(op: int, a=0, b=0, c=0, groups=0) -> int:
    return int(lib().nvfp4_workspace_bytes(op, a, b, c, groups))


# ---------------------------------------------------------- tensor types
class NVFP4Tensor:
    """Device NVFP4 tensor: packed codes, block scales and the tensor scale.

    ``codes`` uint8 [rows, cols/2], ``scales`` uint8 [scales_bytes],
    ``global_scale`` float32 [1]; all on one CUDA device."""

    def __init__(self, codes, scales, global_scale, rows, cols, layout):
        self.codes, self.scales, self.global_scale = codes, scales, global_scale
        self.rows, self.cols, self.layout = rows, cols, layout

    @classmethod
    def empty(cls, rows: int, cols: int, layout: int = SF_SWIZZLED, device="cuda",
              global_scale=None):
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        scales = torch.empty(nvfp4_scales_bytes(rows, cols, layout), dtype=torch.uint8,
                             device=device)
        if global_scale is None:
            global_scale = torch.zeros(1, dtype=torch.float32, device=device)
        return cls(codes, scales, global_scale, rows, cols, layout)

    def c_struct(self) -> CTensor:
        return CTensor(_ptr(self.codes), _ptr(self.scales), _ptr(self.global_scale),
                       self.rows, self.cols, self.layout)

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


class MXFP4Tensor(NVFP4Tensor):
    """Device MXFP4 tensor: packed codes and UE8M0 scales (one per 32
    values); no tensor scale."""

    @classmethod
    def empty(cls, rows: int, cols: int, layout: int = SF_SWIZZLED, device="cuda"):
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        scales = torch.empty(lib().nvfp4_mx_scales_bytes(rows, cols, layout), dtype=torch.uint8,
                             device=device)
        return cls(codes, scales, None, rows, cols, layout)


class Workspace:
    """Zero-initialised device workspace (status word + scratch)."""

    def __init__(self, device="cuda", nbytes: int | None = None):
        if nbytes is None:
            # room for the split-K slices of small-M GEMMs (a smaller
            # workspace only turns the split off)
            nbytes = max(max(nvfp4_workspace_bytes(op) for op in range(5)), 32 << 20)
        self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


_default_ws: dict[int, Workspace] = {}


def default_workspace(device=None) -> Workspace:
    """The device's workspace of calls that are given none, made by the first
    of them.  Make it before a CUDA graph is captured (by a call outside, or by
    this one): made inside, each replay fills it anew, and with that clears
    what the replays before recorded."""
    dev = torch.device(device or "cuda")
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    if idx not in _default_ws:
        ws = Workspace(torch.device("cuda", idx))
        # filled before a call on another stream uses it
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(idx).synchronize()
        _default_ws[idx] = ws
    return _default_ws[idx]


# ------------------------------------------------------------ operations
def nvfp4_quantize(x: torch.Tensor, out: NVFP4Tensor | None = None, layout: int = SF_SWIZZLED,
                   global_supplied: bool = False, workspace: Workspace | None = None,
                   stream=None) -> NVFP4Tensor:
    """Two-level NVFP4 quantization of a 2-D BF16 CUDA tensor (row pitch
    x.stride(0)).  With ``global_supplied`` the tensor scale already in
    ``out.global_scale`` is used."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if out is None:
        out = NVFP4Tensor.empty(rows, cols, layout, x.device)
    ws = workspace or default_workspace(x.device)
    t = out.c_struct()
    _check(lib().nvfp4_quantize(x.data_ptr(), x.stride(0), C.byref(t), int(global_supplied),
                                ws.ptr, ws.nbytes, _stream(stream)), "nvfp4_quantize")
    return out


def nvfp4_quantize_rht(x: torch.Tensor, sign_mask: int, out: NVFP4Tensor | None = None,
                       layout: int = SF_SWIZZLED, global_supplied: bool = False,
                       workspace: Workspace | None = None, stream=None) -> NVFP4Tensor:
    """Quantize after the 16x16 random Hadamard transform of every block
    (``sign_mask`` bit j negates value j of each block before the transform)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if out is None:
        out = NVFP4Tensor.empty(rows, cols, layout, x.device)
    ws = workspace or default_workspace(x.device)
    t = out.c_struct()
    _check(lib().nvfp4_quantize_rht(x.data_ptr(), x.stride(0), sign_mask, C.byref(t),
                                    int(global_supplied), ws.ptr, ws.nbytes, _stream(stream)),
           "nvfp4_quantize_rht")
    return out


def nvfp4_quantize_t(x: torch.Tensor, out: NVFP4Tensor | None = None, layout: int = SF_SWIZZLED,
                     sign_mask: int | None = None, global_supplied: bool = False,
                     workspace: Workspace | None = None, stream=None) -> NVFP4Tensor:
    """NVFP4 of x^T from a row-major BF16 x (x.shape = (R, C) gives a C x R
    tensor).  With ``sign_mask`` the blocks are Hadamard-transformed first."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows_x, cols_x = x.shape
    if out is None:
        out = NVFP4Tensor.empty(cols_x, rows_x, layout, x.device)
    ws = workspace or default_workspace(x.device)
    t = out.c_struct()
    rht = 0 if sign_mask is None else 1
    _check(lib().nvfp4_quantize_t(x.data_ptr(), x.stride(0), rht, sign_mask or 0, C.byref(t),
                                  int(global_supplied), ws.ptr, ws.nbytes, _stream(stream)),
           "nvfp4_quantize_t")
    return out


def nvfp4_quantize_2d(w: torch.Tensor, out: NVFP4Tensor | None = None,
                      out_t: NVFP4Tensor | None = None, transposed: bool = False,
                      layout: int = SF_SWIZZLED, global_supplied: bool = False,
                      workspace: Workspace | None = None, stream=None):
    """16x16-block quantization of a BF16 weight; with ``transposed`` (or an
    ``out_t``) also returns W^T's NVFP4 tensor holding the same values."""
    assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.stride(1) == 1
    rows, cols = w.shape
    if out is None:
        out = NVFP4Tensor.empty(rows, cols, layout, w.device)
    if out_t is None and transposed:
        out_t = NVFP4Tensor.empty(cols, rows, layout, w.device)
    ws = workspace or default_workspace(w.device)
    t = out.c_struct()
    tt = out_t.c_struct() if out_t is not None else None
    _check(lib().nvfp4_quantize_2d(w.data_ptr(), w.stride(0), C.byref(t),
                                   C.byref(tt) if tt is not None else None, int(global_supplied),
                                   ws.ptr, ws.nbytes, _stream(stream)), "nvfp4_quantize_2d")
    return (out, out_t) if out_t is not None else out


def nvfp4_quantize_sr(x: torch.Tensor, seed: int, out: NVFP4Tensor | None = None,
                      transposed: bool = False, sign_mask: int | None = None,
                      layout: int = SF_SWIZZLED, global_supplied: bool = False,
                      workspace: Workspace | None = None, stream=None) -> NVFP4Tensor:
    """Quantize with stochastically rounded codes (Philox draws keyed by
    ``seed``); ``transposed`` gives NVFP4 of x^T, ``sign_mask`` applies the
    Hadamard transform first."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if out is None:
        out = (NVFP4Tensor.empty(cols, rows, layout, x.device) if transposed
               else NVFP4Tensor.empty(rows, cols, layout, x.device))
    ws = workspace or default_workspace(x.device)
    t = out.c_struct()
    _check(lib().nvfp4_quantize_sr(x.data_ptr(), x.stride(0), int(transposed),
                                   0 if sign_mask is None else 1, sign_mask or 0, seed, C.byref(t),
                                   int(global_supplied), ws.ptr, ws.nbytes, _stream(stream)),
           "nvfp4_quantize_sr")
    return out


def nvfp4_quantize_mx(x: torch.Tensor, out: MXFP4Tensor | None = None, layout: int = SF_SWIZZLED,
                      workspace: Workspace | None = None, stream=None) -> MXFP4Tensor:
    """MXFP4 quantization (block 32, UE8M0 scales) of a 2-D BF16 tensor."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if out is None:
        out = MXFP4Tensor.empty(rows, cols, layout, x.device)
    ws = workspace or default_workspace(x.device)
    t = out.c_struct()
    _check(lib().nvfp4_quantize_mx(x.data_ptr(), x.stride(0), C.byref(t), ws.ptr, ws.nbytes,
                                   _stream(stream)), "nvfp4_quantize_mx")
    return out


def nvfp4_dequantize_mx(t: MXFP4Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty((t.rows, t.cols), dtype=torch.bfloat16, device=t.codes.device)
    ct = t.c_struct()
    _check(lib().nvfp4_dequantize_mx(C.byref(ct), out.data_ptr(), out.stride(0), _stream(stream)),
           "nvfp4_dequantize_mx")
    return out


def nvfp4_gemm_mx(a: MXFP4Tensor, w: MXFP4Tensor, out: torch.Tensor | None = None,
                  workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """D = A_hat * W_hat^T for MXFP4 operands (BF16 out)."""
    if out is None:
        out = torch.empty((a.rows, w.rows), dtype=torch.bfloat16, device=a.codes.device)
    ws = workspace or default_workspace(a.codes.device)
    ta, tw = a.c_struct(), w.c_struct()
    _check(lib().nvfp4_gemm_mx(C.byref(ta), C.byref(tw), out.data_ptr(), out.stride(0), ws.ptr,
                               ws.nbytes, _stream(stream)), "nvfp4_gemm_mx")
    return out


def nvfp4_moe_combine(expert_out: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = bf16(sum_k weights[t,k] * expert_out[slots[t,k]])."""
    assert expert_out.dtype == torch.bfloat16 and expert_out.stride(1) == 1
    assert slots.dtype == torch.int32 and weights.dtype == torch.float32
    tokens, topk = slots.shape
    hidden = expert_out.shape[1]
    if out is None:
        out = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=expert_out.device)
    _check(lib().nvfp4_moe_combine(expert_out.data_ptr(), expert_out.stride(0), expert_out.shape[0],
                                   slots.contiguous().data_ptr(), weights.contiguous().data_ptr(),
                                   tokens, topk, hidden, out.data_ptr(), out.stride(0),
                                   _stream(stream)), "nvfp4_moe_combine")
    return out


def nvfp4_dequantize_fp8(t: NVFP4Tensor, out: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                         stream=None):
    """NVFP4 -> E4M3 bytes (uint8) and the per-tensor factor RN(8/g)."""
    if out is None:
        out = torch.empty((t.rows, t.cols), dtype=torch.uint8, device=t.codes.device)
    if scale is None:
        scale = torch.zeros(1, dtype=torch.float32, device=t.codes.device)
    ct = t.c_struct()
    _check(lib().nvfp4_dequantize_fp8(C.byref(ct), out.data_ptr(), out.stride(0), scale.data_ptr(),
                                      _stream(stream)), "nvfp4_dequantize_fp8")
    return out, scale


def nvfp4_attention_decode(q: torch.Tensor, k: NVFP4Tensor, v: NVFP4Tensor, heads_kv: int,
                           scale: float | None = None, out: torch.Tensor | None = None,
                           workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """One decode step of grouped-query attention read straight from an
    NVFP4 KV cache: q BF16 [heads_q x 128]; k, v NVFP4 [tokens x heads_kv *
    128] in the linear scale layout.  Returns BF16 [heads_q x 128].  The
    softmax scale defaults to 1 / sqrt(128)."""
    assert q.dtype == torch.bfloat16 and q.dim() == 2 and q.stride(1) == 1
    heads_q = q.shape[0]
    if scale is None:
        scale = 128 ** -0.5
    if out is None:
        out = torch.empty((heads_q, 128), dtype=torch.bfloat16, device=q.device)
    need = nvfp4_workspace_bytes(OP_ATTENTION, k.rows, heads_q, heads_kv)
    ws = workspace or default_workspace(q.device)
    if ws.nbytes < need:
        ws = Workspace(q.device, need)
    tk, tv = k.c_struct(), v.c_struct()
    _check(lib().nvfp4_attention_decode(q.data_ptr(), q.stride(0), heads_q, C.byref(tk), C.byref(tv),
                                        heads_kv, float(scale), out.data_ptr(), out.stride(0), ws.ptr,
                                        ws.nbytes, _stream(stream)), "nvfp4_attention_decode")
    return out


# -------------------------------------------------------- paged KV cache
# These calls are made for every layer of every generated token, so that the
# host's time counts: the checks are plain comparisons, and the current device
# and stream are asked of torch's own bindings (a few hundred ns, against 7 us
# through torch.cuda.current_stream()).
def _require(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _current_stream(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)


def _new(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """torch.empty((rows, cols)) at 0.9 us less."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


@contextlib.contextmanager
def _switched(device, stream):
    """The tensors' device and the given stream made current, so that outputs
    and scratch belong to the stream the kernels run on."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                # 0 and 1 (cudaStreamLegacy) are the default stream; torch
                # takes a null handle for "any stream of the pool"
                stream = (torch.cuda.default_stream(device) if int(stream) in (0, 1)
                          else torch.cuda.ExternalStream(int(stream), device=device))
            elif stream.device_index != _current_device():
                raise ValueError(f"stream is not on cuda:{_current_device()}, the device of the first argument")
            with torch.cuda.stream(stream):
                yield


def _workspace_of(workspace, device):
    if workspace is None:
        workspace = _default_ws.get(device.index) or default_workspace(device)
    elif workspace.buf.device != device:
        raise ValueError(f"workspace is not on {device}, the device of the first argument")
    return workspace


def _pool_error(name, t, device):
    """What is wrong with a cache's tensor."""
    if t.layout != SF_LINEAR:
        raise ValueError(f"{name}: the cache needs the linear scale layout")
    for part, x, dtype, n in (("codes", t.codes, torch.uint8, t.rows * (t.cols // 2)),
                              ("scales", t.scales, torch.uint8, t.rows * (t.cols // 16)),
                              ("global_scale", t.global_scale, torch.float32, 1)):
        if x.dtype != dtype or x.numel() != n or not x.is_contiguous():
            raise ValueError(f"{name}.{part}: {dtype} of {n} elements, contiguous")
        if x.device != device:
            raise ValueError(f"{name} is not on {device}, the device of the first argument")


def _pool_struct(name, t: NVFP4Tensor, device):
    """C struct of a cache's tensor; its buffers hold what the C ABI is told
    (which cannot see their sizes)."""
    codes, scales, g, rows, cols, at = t.codes, t.scales, t.global_scale, t.rows, t.cols, device.index
    if (t.layout != SF_LINEAR or codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8
            or g.dtype is not torch.float32 or codes.numel() != rows * (cols // 2)
            or scales.numel() != rows * (cols // 16) or g.numel() != 1 or codes.get_device() != at
            or scales.get_device() != at or g.get_device() != at or not codes.is_contiguous()
            or not scales.is_contiguous()):
        _pool_error(name, t, device)
    return CTensor(codes.data_ptr(), scales.data_ptr(), g.data_ptr(), rows, cols, SF_LINEAR)


def _check_index(name, t, device, n):
    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.dim() != 1 or t.shape[0] != n
            or not t.is_contiguous()):
        raise ValueError(f"{name}: int32, one dimension of {n}, contiguous")
    if t.get_device() != device.index:
        raise ValueError(f"{name} is not on {device}, the device of the first argument")


def _check_table(table, device):
    if table.dtype is not torch.float32 or table.dim() != 3 or table.shape[2] != 2 or not table.is_contiguous():
        raise ValueError("table: float32 [positions, rotary_dim / 2, 2], contiguous")
    if table.get_device() != device.index:
        raise ValueError(f"table is not on {device}, the device of the first argument")


def _check_heads(name, t, shape, device):
    """A BF16 CUDA tensor of rows of heads, values of a head contiguous."""
    if t.dtype != torch.bfloat16 or t.dim() != 3 or not t.is_cuda or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name}: BF16 CUDA, three dimensions, innermost contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is not on {device}, the device of the first argument")


def nvfp4_rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: str = "plain",
                        factor: float = 1.0, original_positions: float = 0.0, low: float = 1.0,
                        high: float = 32.0) -> torch.Tensor:
    """Rotary frequencies, float64 [rotary_dim / 2] on the host.  ``scaling``:
    plain, linear, ntk, bands or ramp (see nvfp4_rope_inv_freq in the header)."""
    _require(scaling in ROPE_SCALINGS, f"scaling: one of {', '.join(ROPE_SCALINGS)}")
    out = torch.empty(max(int(rotary_dim) // 2, 0), dtype=torch.float64)
    _check(lib().nvfp4_rope_inv_freq(rotary_dim, base, ROPE_SCALINGS[scaling], factor,
                                     original_positions, low, high, out.data_ptr()),
           "nvfp4_rope_inv_freq")
    return out


def nvfp4_rope_table(inv_freq: torch.Tensor, positions: int, magnitude: float = 1.0, first: int = 0,
                     device="cuda", stream=None) -> torch.Tensor:
    """(cos, sin) * magnitude of positions first .. first + positions - 1:
    float32 [positions, rotary_dim / 2, 2], the ``table`` of nvfp4_rope and
    nvfp4_kv_write."""
    _require(inv_freq.dtype == torch.float64 and inv_freq.dim() == 1, "inv_freq: float64, one dimension")
    device = inv_freq.device if inv_freq.is_cuda else torch.device(device)
    with _switched(device, stream):
        f = inv_freq.to(torch.device("cuda", _current_device())).contiguous()
        out = torch.empty((positions, f.numel(), 2), dtype=torch.float32, device=f.device)
        _check(lib().nvfp4_rope_table(f.data_ptr(), 2 * f.numel(), first, positions, magnitude,
                                      out.data_ptr(), _current_stream(f.device.index)), "nvfp4_rope_table")
    return out


def nvfp4_rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, interleaved: bool = False,
               inverse: bool = False, out: torch.Tensor | None = None,
               workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """Rotary positions of a BF16 tensor [tokens, heads, head_dim] (any token
    and head strides): the first 2 * table.shape[1] values of each head are
    rotated, the rest copied.  ``inverse`` gives the gradient of x from that
    of the output.  ``out`` may be x itself; tokens at position -1 keep what
    ``out`` holds there."""
    _check_heads("x", x, None, None)
    device = x.device
    if stream is not None or device.index != _current_device():
        with _switched(device, stream):
            return nvfp4_rope(x, positions, table, interleaved, inverse, out, workspace)
    tokens, heads, dim = x.shape
    _check_table(table, device)
    _check_index("positions", positions, device, tokens)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check_heads("out", out, x.shape, device)
    ws = _workspace_of(workspace, device)
    x_token, x_head, _ = x.stride()
    out_token, out_head, _ = out.stride()
    rows, pairs, _ = table.shape
    st = lib().nvfp4_rope(x.data_ptr(), x_token, x_head, tokens, heads, dim, positions.data_ptr(),
                          table.data_ptr(), rows, 2 * pairs, interleaved, inverse, out.data_ptr(),
                          out_token, out_head, ws.ptr, ws.nbytes, _current_stream(device.index))
    if st != 0:
        raise NVFP4Error(st, "nvfp4_rope")
    return out


def nvfp4_kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: NVFP4Tensor,
                   v_cache: NVFP4Tensor, positions: torch.Tensor | None = None,
                   table: torch.Tensor | None = None, interleaved: bool = False,
                   workspace: Workspace | None = None, stream=None) -> None:
    """Quantize k and v (BF16 [tokens, heads, head_dim]) into rows ``slots``
    (int32, -1 = none) of the cache, under the caches' own tensor scales.
    With a ``table`` the keys are rotated to ``positions`` first."""
    _check_heads("k", k, None, None)
    device = k.device
    if stream is not None or device.index != _current_device():
        with _switched(device, stream):
            return nvfp4_kv_write(k, v, slots, k_cache, v_cache, positions, table, interleaved, workspace)
    _check_heads("v", v, k.shape, device)
    tokens, heads, dim = k.shape
    _check_index("slots", slots, device, tokens)
    tk, tv = _pool_struct("k_cache", k_cache, device), _pool_struct("v_cache", v_cache, device)
    at, rows, pairs, pos = 0, 0, 0, 0
    if table is not None:
        _check_table(table, device)
        _check_index("positions", positions, device, tokens)
        rows, pairs, _ = table.shape
        at, pos = table.data_ptr(), positions.data_ptr()
    ws = _workspace_of(workspace, device)
    k_token, k_head, _ = k.stride()
    v_token, v_head, _ = v.stride()
    st = lib().nvfp4_kv_write(k.data_ptr(), k_token, k_head, v.data_ptr(), v_token, v_head, tokens, heads,
                              dim, slots.data_ptr(), tk, tv, pos, at, rows, 2 * pairs, interleaved, ws.ptr,
                              ws.nbytes, _current_stream(device.index))
    if st != 0:
        raise NVFP4Error(st, "nvfp4_kv_write")


def nvfp4_kv_read(k_cache: NVFP4Tensor, v_cache: NVFP4Tensor, slots: torch.Tensor,
                  out: tuple[torch.Tensor, torch.Tensor] | None = None,
                  workspace: Workspace | None = None, stream=None):
    """Rows ``slots`` (int32, -1 = zeros) of the cache as BF16 [rows, heads *
    head_dim] pairs (k, v), restored as nvfp4_dequantize restores them."""
    if not slots.is_cuda:
        raise ValueError("slots: int32 CUDA [rows]")
    device = slots.device
    if stream is not None or device.index != _current_device():
        with _switched(device, stream):
            return nvfp4_kv_read(k_cache, v_cache, slots, out, workspace)
    rows, cols = slots.numel(), k_cache.cols
    _check_index("slots", slots, device, rows)
    tk, tv = _pool_struct("k_cache", k_cache, device), _pool_struct("v_cache", v_cache, device)
    if out is None:
        out = (_new(rows, cols, torch.bfloat16, device), _new(rows, cols, torch.bfloat16, device))
    else:
        for t in out:
            if t.dtype != torch.bfloat16 or t.shape != (rows, cols) or (cols > 1 and t.stride(1) != 1):
                raise ValueError("out: two BF16 [rows, heads * head_dim], innermost contiguous")
            if t.device != device:
                raise ValueError(f"out is not on {device}, the device of the first argument")
    yk, yv = out
    ws = _workspace_of(workspace, device)
    st = lib().nvfp4_kv_read(tk, tv, slots.data_ptr(), rows, yk.data_ptr(), yk.stride(0), yv.data_ptr(),
                             yv.stride(0), ws.ptr, ws.nbytes, _current_stream(device.index))
    if st != 0:
        raise NVFP4Error(st, "nvfp4_kv_read")
    return out


_scratch_bytes: dict[tuple[int, int, int], int] = {}     # by the head counts and head size


def nvfp4_attention_decode_paged(q: torch.Tensor, k_cache: NVFP4Tensor, v_cache: NVFP4Tensor,
                                 heads_kv: int, block_table: torch.Tensor, seq_lens: torch.Tensor,
                                 page_size: int, scale: float | None = None,
                                 out: torch.Tensor | None = None, return_lse: bool = False,
                                 workspace: Workspace | None = None, stream=None):
    """Decode attention of a batch over the paged cache: q BF16 [sequences,
    heads_q, head_dim], block_table int32 [sequences, pages], seq_lens int32
    [sequences].  Returns BF16 of q's shape, with ``return_lse`` also the
    float32 [sequences, heads_q] log of the summed exponentials.  The softmax
    scale defaults to 1 / sqrt(head_dim)."""
    _check_heads("q", q, None, None)
    device = q.device
    if stream is not None or device.index != _current_device():
        with _switched(device, stream):
            return nvfp4_attention_decode_paged(q, k_cache, v_cache, heads_kv, block_table, seq_lens, page_size,
                                                scale, out, return_lse, workspace)
    sequences, heads_q, dim = q.shape
    tk, tv = _pool_struct("k_cache", k_cache, device), _pool_struct("v_cache", v_cache, device)
    if heads_kv <= 0 or k_cache.cols != heads_kv * dim:
        raise ValueError("the cache's columns are heads_kv * head_dim")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != sequences:
        raise ValueError("block_table: int32 [sequences, pages]")
    pages, (table_row, table_page) = block_table.shape[1], block_table.stride()
    if pages > 1 and table_page != 1:
        raise ValueError("block_table: innermost contiguous")
    if block_table.device != device:
        raise ValueError(f"block_table is not on {device}, the device of the first argument")
    _check_index("seq_lens", seq_lens, device, sequences)
    if scale is None:
        scale = dim ** -0.5
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_heads("out", out, q.shape, device)
    lse = _new(sequences, heads_q, torch.float32, device) if return_lse else None
    # scratch of the call's own, from the allocator of the stream (or the
    # graph being captured): calls on two streams do not share it
    need = _scratch_bytes.get((heads_q, heads_kv, dim))
    if need is None:
        need = int(lib().nvfp4_attention_paged_scratch_bytes(heads_q, heads_kv, dim))
        _scratch_bytes[heads_q, heads_kv, dim] = need
    scratch = _new(1, need, torch.uint8, device)
    ws = _workspace_of(workspace, device)
    q_seq, q_head, _ = q.stride()
    out_seq, out_head, _ = out.stride()
    st = lib().nvfp4_attention_decode_paged(
        q.data_ptr(), q_seq, q_head, sequences, heads_q, tk, tv, heads_kv, block_table.data_ptr(), table_row,
        pages, seq_lens.data_ptr(), page_size, scale, out.data_ptr(), out_seq, out_head,
        0 if lse is None else lse.data_ptr(), ws.ptr, ws.nbytes, scratch.data_ptr(), need,
        _current_stream(device.index))
    if st != 0:
        raise NVFP4Error(st, "nvfp4_attention_decode_paged")
    return (out, lse) if return_lse else out


def nvfp4_quantize_swiglu(gate_up: torch.Tensor, out: NVFP4Tensor | None = None,
                          layout: int = SF_SWIZZLED, workspace: Workspace | None = None,
                          stream=None) -> NVFP4Tensor:
    """NVFP4 of silu(gate) * up for gate_up = [gate | up] (BF16, rows x 2I)."""
    assert gate_up.dtype == torch.bfloat16 and gate_up.dim() == 2 and gate_up.stride(1) == 1
    rows, two_i = gate_up.shape
    if out is None:
        out = NVFP4Tensor.empty(rows, two_i // 2, layout, gate_up.device)
    ws = workspace or default_workspace(gate_up.device)
    t = out.c_struct()
    _check(lib().nvfp4_quantize_swiglu(gate_up.data_ptr(), gate_up.stride(0), C.byref(t), ws.ptr,
                                       ws.nbytes, _stream(stream)), "nvfp4_quantize_swiglu")
    return out


def nvfp4_gather_rows(src: NVFP4Tensor, gather: torch.Tensor, out: NVFP4Tensor | None = None,
                      layout: int = SF_SWIZZLED, workspace: Workspace | None = None,
                      stream=None) -> NVFP4Tensor:
    """Out row r = source row gather[r] (codes and scales), -1 = zero row;
    the tensor scale is copied.  gather: int32 CUDA tensor."""
    assert gather.dtype == torch.int32 and gather.is_cuda
    if out is None:
        out = NVFP4Tensor.empty(gather.numel(), src.cols, layout, src.codes.device)
    ws = workspace or default_workspace(src.codes.device)
    cs, co = src.c_struct(), out.c_struct()
    _check(lib().nvfp4_gather_rows(C.byref(cs), gather.data_ptr(), C.byref(co), ws.ptr, ws.nbytes,
                                   _stream(stream)), "nvfp4_gather_rows")
    return out


def nvfp4_global_scale(x: torch.Tensor, out: torch.Tensor | None = None,
                       workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    if out is None:
        out = torch.zeros(1, dtype=torch.float32, device=x.device)
    ws = workspace or default_workspace(x.device)
    _check(lib().nvfp4_global_scale(x.data_ptr(), x.stride(0), x.shape[0], x.shape[1],
                                    out.data_ptr(), ws.ptr, ws.nbytes, _stream(stream)),
           "nvfp4_global_scale")
    return out


def nvfp4_quantize_gather(x: torch.Tensor, gather: torch.Tensor, out: NVFP4Tensor | None = None,
                          layout: int = SF_SWIZZLED, global_supplied: bool = False,
                          workspace: Workspace | None = None, stream=None) -> NVFP4Tensor:
    """Quantize rows x[gather[r]] (gather int32 CUDA, -1 = zero row)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    assert gather.dtype == torch.int32 and gather.is_contiguous()
    rows, cols = gather.numel(), x.shape[1]
    if out is None:
        out = NVFP4Tensor.empty(rows, cols, layout, x.device)
    ws = workspace or default_workspace(x.device)
    t = out.c_struct()
    _check(lib().nvfp4_quantize_gather(x.data_ptr(), x.stride(0), x.shape[0], gather.data_ptr(),
                                       C.byref(t), int(global_supplied), ws.ptr, ws.nbytes,
                                       _stream(stream)), "nvfp4_quantize_gather")
    return out


def nvfp4_dequantize(t: NVFP4Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty((t.rows, t.cols), dtype=torch.bfloat16, device=t.codes.device)
    ct = t.c_struct()
    _check(lib().nvfp4_dequantize(C.byref(ct), out.data_ptr(), out.stride(0), _stream(stream)),
           "nvfp4_dequantize")
    return out


def nvfp4_gemm(a: NVFP4Tensor, w: NVFP4Tensor, out: torch.Tensor | None = None,
               workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """D = A * W^T on the FP4 tensor cores, BF16 [a.rows, w.rows]."""
    if out is None:
        out = torch.empty((a.rows, w.rows), dtype=torch.bfloat16, device=a.codes.device)
    ws = workspace or default_workspace(a.codes.device)
    ca, cw = a.c_struct(), w.c_struct()
    _check(lib().nvfp4_gemm(C.byref(ca), C.byref(cw), out.data_ptr(), out.stride(0), ws.ptr,
                            ws.nbytes, _stream(stream)), "nvfp4_gemm")
    return out


def nvfp4_grouped_gemm(slot_offsets: torch.Tensor, group_rows: torch.Tensor, a: NVFP4Tensor,
                       w: NVFP4Tensor, w_globals: torch.Tensor, n: int,
                       out: torch.Tensor | None = None, workspace: Workspace | None = None,
                       stream=None) -> torch.Tensor:
    """Grouped D_g = A_g * W_g^T over expert slots (see nvfp4_grouped_gemm in
    the header).  slot_offsets/group_rows int32 CUDA, w_globals float32 CUDA."""
    groups = group_rows.numel()
    if out is None:
        out = torch.empty((a.rows, n), dtype=torch.bfloat16, device=a.codes.device)
    ws = workspace or default_workspace(a.codes.device)
    ca, cw = a.c_struct(), w.c_struct()
    _check(lib().nvfp4_grouped_gemm(groups, slot_offsets.data_ptr(), group_rows.data_ptr(),
                                    C.byref(ca), C.byref(cw), w_globals.data_ptr(), n,
                                    out.data_ptr(), out.stride(0), ws.ptr, ws.nbytes,
                                    _stream(stream)), "nvfp4_grouped_gemm")
    return out


def nvfp4_grouped_gemm_out_scale(slot_offsets: torch.Tensor, group_rows: torch.Tensor,
                                 a: NVFP4Tensor, w: NVFP4Tensor, w_globals: torch.Tensor, n: int,
                                 out: torch.Tensor | None = None,
                                 out_global: torch.Tensor | None = None,
                                 workspace: Workspace | None = None, stream=None):
    """nvfp4_grouped_gemm that also writes the NVFP4 tensor scale of its BF16
    output over the real rows into out_global (float32 CUDA, one element).
    Returns (out, out_global)."""
    groups = group_rows.numel()
    if out is None:
        out = torch.empty((a.rows, n), dtype=torch.bfloat16, device=a.codes.device)
    if out_global is None:
        out_global = torch.empty(1, dtype=torch.float32, device=a.codes.device)
    ws = workspace or default_workspace(a.codes.device)
    ca, cw = a.c_struct(), w.c_struct()
    _check(lib().nvfp4_grouped_gemm_out_scale(groups, slot_offsets.data_ptr(), group_rows.data_ptr(),
                                              C.byref(ca), C.byref(cw), w_globals.data_ptr(), n,
                                              out.data_ptr(), out.stride(0), out_global.data_ptr(),
                                              ws.ptr, ws.nbytes, _stream(stream)),
           "nvfp4_grouped_gemm_out_scale")
    return out, out_global


def nvfp4_check_status(workspace: Workspace | None = None, stream=None) -> int:
    """Synchronise, return and clear the workspace status word (0 = OK)."""
    ws = workspace or default_workspace()
    return int(lib().nvfp4_check_status(ws.ptr, _stream(stream)))


def nvfp4_status_string(status: int) -> str:
    return lib().nvfp4_status_string(status).decode()


def nvfp4_launch_count() -> int:
    return int(lib().nvfp4_launch_count())


def nvfp4_set_wait_limit_cycles(cycles: int) -> int:
    return int(lib().nvfp4_set_wait_limit_cycles(cycles))


def nvfp4_set_gemm_pairs(enable: bool) -> bool:
    return bool(lib().nvfp4_set_gemm_pairs(int(enable)))
