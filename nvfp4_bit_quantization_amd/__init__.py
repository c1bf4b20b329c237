"""Python binding of libnvfp4.so: NVFP4 quantisation and the NVFP4 GEMM on
MI355X (gfx950).

The functions named like the C ABI (``nvfp4_quantize``, ``nvfp4_dequantize``,
``nvfp4_gemm``, ...) only marshal arguments: torch supplies device memory and
the current HIP stream, every step of the computation runs in the library's
HIP kernels.  Importing this package fails loudly when the library has not
been built (``python -m nvfp4_bit_quantization_amd.build``); there is no CPU
fallback.

Method: NVFP4 pretraining news page (zubnet.ai), paragraph 2 -- blocks of 16
E2M1 values with an E4M3 scale each, an FP32 scale per tensor, 1D blocks for
activations/gradients and 16x16 blocks for weights, stochastic rounding for
gradients, a 16-point randomised Hadamard transform on the weight-gradient
inputs.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import List, Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")

# enums (include/nvfp4.h)
NVFP4_OK = 0
ROW_1D, COL_1D, TWO_D, TWO_D_T = 0, 1, 2, 3
RTN, SR = 0, 1
AMAX_GIVEN = 1  # nvfp4_quant_output.flags
SCALE_1D16, SCALE_2D16 = 0, 1
F32, BF16 = 0, 1
LAYOUTS = {"row": ROW_1D, "col": COL_1D, "2d": TWO_D, "2d_t": TWO_D_T}
ROUNDINGS = {"rtn": RTN, "sr": SR}


class Nvfp4Error(RuntimeError):
    pass


class nvfp4_tensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("global_scale", ctypes.c_void_p),
                ("amax", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("scale_kind", ctypes.c_int32), ("rht", ctypes.c_int32)]


class mxfp4_tensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class nvfp4_quant_output(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rounding", ctypes.c_int32), ("rht", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("sr_seed", ctypes.c_uint64), ("rht_seed", ctypes.c_uint64),
                ("out", nvfp4_tensor)]


class nvfp4_quant_job(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld_x", ctypes.c_int64),
                ("outs", ctypes.POINTER(nvfp4_quant_output)), ("n_outs", ctypes.c_int32)]


class nvfp4_layernorm_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "residual", "weight", "bias", "y", "sum", "mean", "rstd", "amax")] + [
        (n, ctypes.c_int64) for n in ("rows", "cols", "ld_x", "ld_residual", "ld_y", "ld_sum")] + [
        (n, ctypes.c_int32) for n in ("x_dtype", "y_dtype", "w_dtype")] + [("eps", ctypes.c_float)]


class nvfp4_layernorm_backward_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dy", "x", "weight", "mean", "rstd", "dsum", "dx", "dweight", "dbias",
                                               "amax")] + [
        (n, ctypes.c_int64) for n in ("rows", "cols", "ld_dy", "ld_x", "ld_dsum", "ld_dx")] + [
        (n, ctypes.c_int32) for n in ("x_dtype", "y_dtype", "w_dtype")]


class nvfp4_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class nvfp4_attention_shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("q_len", ctypes.c_int64), ("k_len", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("window", ctypes.c_int64), ("cu_q", ctypes.c_void_p),
                ("cu_k", ctypes.c_void_p), ("total_q", ctypes.c_int64), ("total_k", ctypes.c_int64),
                ("scale", ctypes.c_float)]


class nvfp4_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "m", "v", "m_scale", "v_scale", "copy", "amax")] + [
        ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
        ("state_bits", ctypes.c_int32), ("weight_decay", ctypes.c_float)]


class nvfp4_adamw_config(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_float), ("rounding", ctypes.c_int32), ("step", ctypes.c_int64),
                ("seed", ctypes.c_uint64), ("grad_scale", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libnvfp4.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("libnvfp4.so is not built: run `python -m nvfp4_bit_quantization_amd.build` "
                          "(expected at %s)" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.nvfp4_quantize.restype = i32
    L.nvfp4_quantize.argtypes = [P, i64, i64, i64, ctypes.POINTER(nvfp4_quant_output), i32, P, ctypes.c_size_t, P]
    L.nvfp4_quantize_batch.restype = i32
    L.nvfp4_quantize_batch.argtypes = [ctypes.POINTER(nvfp4_quant_job), i32, P, ctypes.c_size_t, P]
    L.nvfp4_quantize_noalloc.restype = i32
    L.nvfp4_quantize_noalloc.argtypes = [P, i64, i64, i64, ctypes.POINTER(nvfp4_quant_output), i32, P]
    L.nvfp4_workspace_bytes.restype = ctypes.c_size_t
    L.nvfp4_workspace_bytes.argtypes = []
    L.nvfp4_dequantize.restype = i32
    L.nvfp4_dequantize.argtypes = [ctypes.POINTER(nvfp4_tensor), P, i64, P]
    L.nvfp4_gemm.restype = i32
    L.nvfp4_gemm.argtypes = [ctypes.POINTER(nvfp4_tensor), ctypes.POINTER(nvfp4_tensor), P, ctypes.c_int32, i64, P,
                             ctypes.c_size_t, P]
    L.nvfp4_gemm_amax.restype = i32
    L.nvfp4_gemm_amax.argtypes = [ctypes.POINTER(nvfp4_tensor), ctypes.POINTER(nvfp4_tensor), P, i64, P,
                                  ctypes.c_size_t, P, P, ctypes.c_uint64, P]
    L.nvfp4_gemm_workspace_bytes.restype = ctypes.c_size_t
    L.nvfp4_gemm_workspace_bytes.argtypes = []
    L.nvfp4_rht_sign_mask.restype = ctypes.c_uint16
    L.nvfp4_rht_sign_mask.argtypes = [ctypes.c_uint64]
    L.nvfp4_status_string.restype = ctypes.c_char_p
    L.nvfp4_status_string.argtypes = [i32]
    L.nvfp4_codec_selftest.restype = i32
    L.nvfp4_codec_selftest.argtypes = [i32, P, P, P, i64, P]
    L.mxfp4_quantize.restype = i32
    L.mxfp4_quantize.argtypes = [P, i64, i64, i64, ctypes.c_int32, ctypes.POINTER(mxfp4_tensor), P]
    L.mxfp4_dequantize.restype = i32
    L.mxfp4_dequantize.argtypes = [ctypes.POINTER(mxfp4_tensor), P, i64, P]
    L.mxfp4_gemm.restype = i32
    L.mxfp4_gemm.argtypes = [ctypes.POINTER(mxfp4_tensor), ctypes.POINTER(mxfp4_tensor), P, ctypes.c_int32, i64, P]
    A = ctypes.POINTER
    L.nvfp4_layernorm.restype = i32
    L.nvfp4_layernorm.argtypes = [P, P]  # the structures by address, or packed
    L.nvfp4_layernorm_backward.restype = i32
    L.nvfp4_layernorm_backward.argtypes = [P, P, ctypes.c_size_t, P]
    L.nvfp4_layernorm_backward_workspace_bytes.restype = ctypes.c_size_t
    L.nvfp4_layernorm_backward_workspace_bytes.argtypes = [i64, i64]
    L.nvfp4_attention.restype = i32
    L.nvfp4_attention.argtypes = [P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.nvfp4_attention_workspace_bytes.restype = ctypes.c_size_t
    L.nvfp4_attention_workspace_bytes.argtypes = [P]
    L.nvfp4_attention_backward.restype = i32
    L.nvfp4_attention_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.nvfp4_attention_backward_workspace_bytes.restype = ctypes.c_size_t
    L.nvfp4_attention_backward_workspace_bytes.argtypes = [P]
    L.nvfp4_adamw.restype = i32
    L.nvfp4_adamw.argtypes = [A(nvfp4_adamw_tensor), i64, A(nvfp4_adamw_config), P]
    _lib = L
    return L


def _check(status: int, what: str):
    if status != NVFP4_OK:
        raise Nvfp4Error("%s failed: %d (%s)" % (what, status, lib().nvfp4_status_string(status).decode()))


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _on_stream(stream):
    """Context under which the conveniences allocate: the stream the library
    will launch on.  torch's caching allocator then hands a freed block (the
    temporary quantise workspace) to later allocations on that same stream
    only, i.e. after the kernels that use it; memory taken on another stream
    could be reused while those kernels still run."""
    import contextlib
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


# ---------------------------------------------------------------------------
# quantised tensors held in torch device memory
# ---------------------------------------------------------------------------
@dataclass
class QTensor:
    codes: "object"         # torch.uint8 [rows][cols/2]
    scales: "object"        # torch.uint8, 1D [rows][cols/16] or 2D [rows/16][cols/16]
    global_scale: "object"  # torch.float32 [1]
    amax: "object"          # torch.float32 [1]
    rows: int
    cols: int
    scale_kind: int
    rht: int = 0

    def c_struct(self) -> nvfp4_tensor:
        return nvfp4_tensor(self.codes.data_ptr(), self.scales.data_ptr(), self.global_scale.data_ptr(),
                            self.amax.data_ptr(), self.rows, self.cols, self.scale_kind, self.rht)


def empty_qtensor(rows: int, cols: int, scale_kind: int, device="cuda", rht: int = 0) -> QTensor:
    import torch
    sshape = (rows, cols // 16) if scale_kind == SCALE_1D16 else (rows // 16, cols // 16)
    return QTensor(codes=torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                   scales=torch.empty(sshape, dtype=torch.uint8, device=device),
                   global_scale=torch.empty(1, dtype=torch.float32, device=device),
                   amax=torch.empty(1, dtype=torch.float32, device=device),
                   rows=rows, cols=cols, scale_kind=scale_kind, rht=rht)


@dataclass
class QuantSpec:
    """One requested output of nvfp4_quantize."""
    layout: int = ROW_1D
    rounding: int = RTN
    rht: bool = False
    sr_seed: int = 0
    rht_seed: int = 0
    amax_given: bool = False  # the output's amax tensor already holds its maximum (nvfp4_gemm_amax)

    @staticmethod
    def of(layout="row", rounding="rtn", rht=False, sr_seed=0, rht_seed=0, amax_given=False) -> "QuantSpec":
        return QuantSpec(LAYOUTS.get(layout, layout), ROUNDINGS.get(rounding, rounding), bool(rht), sr_seed, rht_seed,
                         bool(amax_given))


def output_shape(rows: int, cols: int, layout: int):
    """(rows, cols, scale_kind) of the stored output for an input [rows][cols]."""
    if layout == ROW_1D:
        return rows, cols, SCALE_1D16
    if layout == COL_1D:
        return cols, rows, SCALE_1D16
    if layout == TWO_D:
        return rows, cols, SCALE_2D16
    if layout == TWO_D_T:
        return cols, rows, SCALE_2D16
    raise ValueError(layout)


def new_workspace(device="cuda", jobs=1):
    """A quantise workspace (one per stream), for `jobs` jobs of a batch."""
    import torch
    return torch.empty(jobs * lib().nvfp4_workspace_bytes() // 4, dtype=torch.float32, device=device)


# ---------------------------------------------------------------------------
# C ABI entry points (argument marshalling only)
# ---------------------------------------------------------------------------
def nvfp4_quantize(x, specs: Sequence[QuantSpec], outs: Sequence[QTensor], workspace, stream=None) -> List[QTensor]:
    """Quantise the bf16 device tensor x [rows][cols] (row stride x.stride(0))
    into 1 or 2 outputs (see include/nvfp4.h)."""
    assert len(specs) == len(outs) and 1 <= len(specs) <= 2
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    arr = (nvfp4_quant_output * len(specs))()
    for i, (s, o) in enumerate(zip(specs, outs)):
        arr[i] = nvfp4_quant_output(s.layout, s.rounding, int(s.rht), AMAX_GIVEN if s.amax_given else 0, s.sr_seed,
                                    s.rht_seed, o.c_struct())
    st = lib().nvfp4_quantize(ctypes.c_void_p(x.data_ptr()), x.shape[0], x.shape[1], x.stride(0), arr, len(specs),
                              ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(),
                              _stream(stream))
    _check(st, "nvfp4_quantize")
    return list(outs)


def nvfp4_quantize_batch(jobs, workspace, stream=None):
    """Several independent nvfp4_quantize calls enqueued together (see
    include/nvfp4.h).  jobs: a sequence of (x, specs, outs); workspace: at
    least len(jobs) * nvfp4_workspace_bytes() bytes (new_workspace(len(jobs)))."""
    import torch
    arrs = []
    jarr = (nvfp4_quant_job * len(jobs))()
    for j, (x, specs, outs) in enumerate(jobs):
        assert len(specs) == len(outs) and 1 <= len(specs) <= 2
        assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
        arr = (nvfp4_quant_output * len(specs))()
        for i, (s, o) in enumerate(zip(specs, outs)):
            arr[i] = nvfp4_quant_output(s.layout, s.rounding, int(s.rht), AMAX_GIVEN if s.amax_given else 0,
                                        s.sr_seed, s.rht_seed, o.c_struct())
        arrs.append(arr)  # kept alive until the call returns
        jarr[j] = nvfp4_quant_job(x.data_ptr(), x.shape[0], x.shape[1], x.stride(0),
                                  ctypes.cast(arr, ctypes.POINTER(nvfp4_quant_output)), len(specs))
    st = lib().nvfp4_quantize_batch(jarr, len(jobs), ctypes.c_void_p(workspace.data_ptr()),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "nvfp4_quantize_batch")
    return [list(outs) for _, _, outs in jobs]


def nvfp4_quantize_noalloc(x, specs: Sequence[QuantSpec], outs: Sequence[QTensor], stream=None) -> List[QTensor]:
    """nvfp4_quantize with the library's static scratch instead of a
    workspace (allocates nothing; calls overlapping on one GPU race)."""
    assert len(specs) == len(outs) and 1 <= len(specs) <= 2
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    arr = (nvfp4_quant_output * len(specs))()
    for i, (s, o) in enumerate(zip(specs, outs)):
        arr[i] = nvfp4_quant_output(s.layout, s.rounding, int(s.rht), AMAX_GIVEN if s.amax_given else 0, s.sr_seed,
                                    s.rht_seed, o.c_struct())
    st = lib().nvfp4_quantize_noalloc(ctypes.c_void_p(x.data_ptr()), x.shape[0], x.shape[1], x.stride(0), arr,
                                      len(specs), _stream(stream))
    _check(st, "nvfp4_quantize_noalloc")
    return list(outs)


def nvfp4_dequantize(q: QTensor, y, stream=None):
    """y[r][c] = (e(code) * s_b) / S for the stored orientation of q (fp32)."""
    import torch
    assert y.dtype == torch.float32 and y.stride(1) == 1
    t = q.c_struct()
    _check(lib().nvfp4_dequantize(ctypes.byref(t), ctypes.c_void_p(y.data_ptr()), y.stride(0), _stream(stream)),
           "nvfp4_dequantize")
    return y


def nvfp4_gemm(a: QTensor, b: QTensor, c, workspace=None, stream=None):
    """C[M][N] = A^ B^T / (S_A S_B) into the fp32 or bf16 device tensor c.
    `workspace` (from new_gemm_workspace) enables the stream-K path."""
    import torch
    dt = F32 if c.dtype == torch.float32 else BF16 if c.dtype == torch.bfloat16 else None
    if dt is None:
        raise TypeError("c must be float32 or bfloat16")
    assert c.stride(1) == 1
    ta, tb = a.c_struct(), b.c_struct()
    wp = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p(0)
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().nvfp4_gemm(ctypes.byref(ta), ctypes.byref(tb), ctypes.c_void_p(c.data_ptr()), dt, c.stride(0),
                            wp, wb, _stream(stream)), "nvfp4_gemm")
    return c


def nvfp4_gemm_amax(a: QTensor, b: QTensor, c, amax_plain=None, amax_rht_col=None, rht_seed: int = 0,
                    workspace=None, stream=None):
    """nvfp4_gemm into the bf16 tensor c that also folds max |c| into the
    float32 device tensor amax_plain[0] and the RHT-domain maximum of c's
    16-row groups (signs from rht_seed) into amax_rht_col[0] (atomic maxima:
    initialise them, e.g. to 0)."""
    import torch
    if c.dtype != torch.bfloat16:
        raise TypeError("c must be bfloat16")
    assert c.stride(1) == 1
    ta, tb = a.c_struct(), b.c_struct()
    p = (lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0))
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().nvfp4_gemm_amax(ctypes.byref(ta), ctypes.byref(tb), ctypes.c_void_p(c.data_ptr()), c.stride(0),
                                 p(workspace), wb, p(amax_plain), p(amax_rht_col), rht_seed, _stream(stream)),
           "nvfp4_gemm_amax")
    return c


def nvfp4_gemm_workspace_bytes() -> int:
    return lib().nvfp4_gemm_workspace_bytes()


def new_gemm_workspace(device="cuda"):
    """A zero-filled GEMM workspace (one per stream)."""
    import torch
    return torch.zeros(lib().nvfp4_gemm_workspace_bytes(), dtype=torch.uint8, device=device)


def gemm_workspace_timed_out(workspace) -> bool:
    """True if a stream-K call on this workspace hit its wait limit (the
    outputs of that call are invalid; reset_gemm_workspace before reuse)."""
    return bool(workspace[4096:4100].view(__import__("torch").int32).item() != 0)


def reset_gemm_workspace(workspace):
    """Zero-fill a GEMM workspace again (needed after a timed-out call)."""
    workspace.zero_()
    return workspace


def nvfp4_workspace_bytes() -> int:
    return lib().nvfp4_workspace_bytes()


def nvfp4_rht_sign_mask(seed: int) -> int:
    return lib().nvfp4_rht_sign_mask(seed)


def nvfp4_status_string(status: int) -> str:
    return lib().nvfp4_status_string(status).decode()


def nvfp4_codec_selftest(which: int, x, u16, out, stream=None):
    p = (lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0))
    _check(lib().nvfp4_codec_selftest(which, p(x), p(u16), p(out), out.numel(), _stream(stream)),
           "nvfp4_codec_selftest")
    return out


# ---------------------------------------------------------------------------
# conveniences (allocation + one call)
# ---------------------------------------------------------------------------
def quantize(x, specs: Sequence[QuantSpec], workspace=None, stream=None) -> List[QTensor]:
    """Allocate the outputs for `specs` (and, if none is given, a workspace)
    on the stream the call runs on, and quantise x into them."""
    with _on_stream(stream):
        if workspace is None:
            workspace = new_workspace(x.device)
        outs = []
        for s in specs:
            r, c, k = output_shape(x.shape[0], x.shape[1], s.layout)
            outs.append(empty_qtensor(r, c, k, x.device, rht=int(s.rht)))
    return nvfp4_quantize(x, specs, outs, workspace, stream)


def dequantize(q: QTensor, stream=None):
    import torch
    with _on_stream(stream):
        y = torch.empty((q.rows, q.cols), dtype=torch.float32, device=q.codes.device)
    return nvfp4_dequantize(q, y, stream)


def gemm(a: QTensor, b: QTensor, out_dtype="f32", workspace=None, stream=None):
    import torch
    dt = torch.float32 if out_dtype == "f32" else torch.bfloat16
    with _on_stream(stream):
        c = torch.empty((a.rows, b.rows), dtype=dt, device=a.codes.device)
    return nvfp4_gemm(a, b, c, workspace, stream)


# ---------------------------------------------------------------------------
# MXFP4 (OCP MX v1.0: 32-element blocks, E8M0 scales, no per-tensor scale)
# ---------------------------------------------------------------------------
@dataclass
class MXTensor:
    codes: "object"   # torch.uint8 [rows][cols/2]
    scales: "object"  # torch.uint8 [rows][cols/32] (E8M0)
    rows: int
    cols: int

    def c_struct(self) -> mxfp4_tensor:
        return mxfp4_tensor(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.cols)


def empty_mxtensor(rows: int, cols: int, device="cuda") -> MXTensor:
    import torch
    return MXTensor(codes=torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                    scales=torch.empty((rows, cols // 32), dtype=torch.uint8, device=device), rows=rows, cols=cols)


def mxfp4_quantize(x, layout, out: MXTensor, stream=None) -> MXTensor:
    """MXFP4-quantise the bf16 device tensor x [rows][cols] into out
    (layout ROW_1D: out is rows x cols; COL_1D: out is x^T)."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    t = out.c_struct()
    _check(lib().mxfp4_quantize(ctypes.c_void_p(x.data_ptr()), x.shape[0], x.shape[1], x.stride(0),
                                LAYOUTS.get(layout, layout), ctypes.byref(t), _stream(stream)), "mxfp4_quantize")
    return out


def mxfp4_dequantize(q: MXTensor, y, stream=None):
    """y = e(code) * 2^(scale - 127) as fp32."""
    import torch
    assert y.dtype == torch.float32 and y.stride(1) == 1
    t = q.c_struct()
    _check(lib().mxfp4_dequantize(ctypes.byref(t), ctypes.c_void_p(y.data_ptr()), y.stride(0), _stream(stream)),
           "mxfp4_dequantize")
    return y


def mxfp4_gemm(a: MXTensor, b: MXTensor, c, stream=None):
    """C[M][N] = A^ B^T into the fp32 or bf16 device tensor c."""
    import torch
    dt = F32 if c.dtype == torch.float32 else BF16 if c.dtype == torch.bfloat16 else None
    if dt is None:
        raise TypeError("c must be float32 or bfloat16")
    assert c.stride(1) == 1
    ta, tb = a.c_struct(), b.c_struct()
    _check(lib().mxfp4_gemm(ctypes.byref(ta), ctypes.byref(tb), ctypes.c_void_p(c.data_ptr()), dt, c.stride(0),
                            _stream(stream)), "mxfp4_gemm")
    return c


def mx_quantize(x, layout="row", stream=None) -> MXTensor:
    """Allocate the output and MXFP4-quantise x."""
    layout = LAYOUTS.get(layout, layout)
    r, c = (x.shape[0], x.shape[1]) if layout == ROW_1D else (x.shape[1], x.shape[0])
    with _on_stream(stream):
        out = empty_mxtensor(r, c, x.device)
    return mxfp4_quantize(x, layout, out, stream)


def mx_gemm(a: MXTensor, b: MXTensor, out_dtype="f32", stream=None):
    import torch
    dt = torch.float32 if out_dtype == "f32" else torch.bfloat16
    with _on_stream(stream):
        c = torch.empty((a.rows, b.rows), dtype=dt, device=a.codes.device)
    return mxfp4_gemm(a, b, c, stream)


# ---------------------------------------------------------------------------
# training operators: layer norm, attention, AdamW (see include/nvfp4.h)
#
# Their smallest calls take less time on the GPU than Python needs to describe
# them, so arguments are packed straight into the C structures' layout, outputs
# that were allocated here are not looked over again, and the stream's handle
# is taken without a stream object.
# ---------------------------------------------------------------------------
_NORM = struct.Struct("@9P6q3if")
_NORM_GRAD = struct.Struct("@10P6q3i4x")
_SHAPE = struct.Struct("@3q4iq2P2qf4x")
_HEADS = struct.Struct("@P3q")


def _dtype(t) -> int:
    name = str(t.dtype)
    if name == "torch.bfloat16":
        return BF16
    if name == "torch.float32":
        return F32
    raise TypeError("float32 or bfloat16 is wanted, not %s" % name)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _scratch(t, device):
    """Checks a workspace, whose size is taken from its elements: each has to be memory of its own."""
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on device %d is wanted" % device)


def _raw_stream(stream, device_index) -> int:
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(device_index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _floats(rows, cols, device):
    """A new contiguous float32 [rows][cols] (the quickest of torch's ways)."""
    import torch
    return torch.empty_strided((rows, cols), (cols, 1), dtype=torch.float32, device=device)


def _on_device(t, what) -> int:
    if not t.is_cuda:
        raise ValueError("%s: a device tensor is wanted" % what)
    return t.get_device()


def _matrix(t, shape, device, what, dtype=None):
    """Checks that t is a device tensor of a [rows][cols] shape with contiguous rows."""
    if t.get_device() != device or t.shape != shape:
        raise ValueError("%s: a tensor of shape %s on device %d is wanted" % (what, tuple(shape), device))
    if t.stride(1) != 1 and shape[1] > 1:
        raise ValueError("%s: contiguous rows are wanted" % what)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s: %s is wanted, not %s" % (what, dtype, t.dtype))


def _row_stride(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _vector(t, n, device, what, dtype=None):
    if t.dim() != 1 or t.numel() != n or t.get_device() != device or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s: a contiguous vector of %d elements on device %d is wanted" % (what, n, device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s: %s is wanted, not %s" % (what, dtype, t.dtype))


def _layernorm_inputs(x, weight, bias, residual, amax):
    """(rows, cols, device) of the checked inputs of a layer norm."""
    device = _on_device(x, "x")
    if x.dim() != 2:
        raise ValueError("x: [rows][cols] is wanted")
    shape = x.shape
    if x.stride(1) != 1 and shape[1] > 1:
        raise ValueError("x: contiguous rows are wanted")
    if residual is not None:
        _matrix(residual, shape, device, "residual", x.dtype)
    _vector(weight, shape[1], device, "weight")
    if bias is not None:
        _vector(bias, shape[1], device, "bias", weight.dtype)
    if amax is not None:
        import torch
        _vector(amax, 1, device, "amax", torch.float32)
    return shape, device


def _layernorm(x, weight, bias, eps, y, mean, rstd, residual, total, amax, shape, device, stream):
    a = _NORM.pack(x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(bias), y.data_ptr(), _ptr(total), mean, rstd,
                   _ptr(amax), shape[0], shape[1], _row_stride(x), 0 if residual is None else _row_stride(residual),
                   _row_stride(y), 0 if total is None else _row_stride(total), _dtype(x), _dtype(y), _dtype(weight), eps)
    _check(lib().nvfp4_layernorm(a, _raw_stream(stream, device)), "nvfp4_layernorm")


def nvfp4_layernorm(x, weight, bias, eps, y, mean, rstd, residual=None, sum=None, amax=None, stream=None):
    """y = layer norm of x (or of x + residual, which goes to sum) over the rows of [rows][cols], with the rows' mean
    and 1 / standard deviation; *amax is raised to max |y|."""
    import torch
    shape, device = _layernorm_inputs(x, weight, bias, residual, amax)
    _matrix(y, shape, device, "y")
    if sum is not None:
        _matrix(sum, shape, device, "sum", x.dtype)
    _vector(mean, shape[0], device, "mean", torch.float32)
    _vector(rstd, shape[0], device, "rstd", torch.float32)
    _layernorm(x, weight, bias, eps, y, mean.data_ptr(), rstd.data_ptr(), residual, sum, amax, shape, device, stream)
    return y


def layernorm(x, weight, bias=None, eps=1e-5, residual=None, amax=None, out_dtype=None, stream=None):
    """Allocates and computes (y, mean, rstd, sum): y of x's dtype or `out_dtype`; sum is x + residual, or None."""
    if stream is not None:
        with _on_stream(stream):
            return layernorm(x, weight, bias, eps, residual, amax, out_dtype)
    import torch
    shape, device = _layernorm_inputs(x, weight, bias, residual, amax)
    y = torch.empty_like(x, dtype=out_dtype, memory_format=torch.contiguous_format)
    mean, rstd = _floats(2, shape[0], x.device).unbind()
    total = None if residual is None else torch.empty_like(x, memory_format=torch.contiguous_format)
    _layernorm(x, weight, bias, eps, y, mean.data_ptr(), rstd.data_ptr(), residual, total, amax, shape, device, None)
    return y, mean, rstd, total


def _layernorm_backward_inputs(dy, x, weight, mean, rstd, dsum, amax):
    import torch
    device = _on_device(x, "x")
    if x.dim() != 2:
        raise ValueError("x: [rows][cols] is wanted")
    shape = x.shape
    if x.stride(1) != 1 and shape[1] > 1:
        raise ValueError("x: contiguous rows are wanted")
    _matrix(dy, shape, device, "dy")
    if dsum is not None:
        _matrix(dsum, shape, device, "dsum", x.dtype)
    _vector(weight, shape[1], device, "weight")
    _vector(mean, shape[0], device, "mean", torch.float32)
    _vector(rstd, shape[0], device, "rstd", torch.float32)
    if amax is not None:
        _vector(amax, 1, device, "amax", torch.float32)
    return shape, device


def _layernorm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, dsum, amax, workspace, shape, device, stream):
    a = _NORM_GRAD.pack(dy.data_ptr(), x.data_ptr(), weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _ptr(dsum),
                        dx.data_ptr(), _ptr(dweight), _ptr(dbias), _ptr(amax), shape[0], shape[1], _row_stride(dy),
                        _row_stride(x), 0 if dsum is None else _row_stride(dsum), _row_stride(dx), _dtype(x), _dtype(dy),
                        _dtype(weight))
    _check(lib().nvfp4_layernorm_backward(a, _ptr(workspace), _nbytes(workspace), _raw_stream(stream, device)),
           "nvfp4_layernorm_backward")


def nvfp4_layernorm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, dsum=None, amax=None, workspace=None,
                             stream=None):
    """dx, dweight and dbias (each of the two may be None) of a layer norm of x; dsum is added to dx."""
    import torch
    shape, device = _layernorm_backward_inputs(dy, x, weight, mean, rstd, dsum, amax)
    _matrix(dx, shape, device, "dx", x.dtype)
    for t, what in ((dweight, "dweight"), (dbias, "dbias")):
        if t is not None:
            _vector(t, shape[1], device, what, torch.float32)
    if workspace is not None:
        _scratch(workspace, device)
    _layernorm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, dsum, amax, workspace, shape, device, stream)
    return dx


def layernorm_backward(dy, x, weight, mean, rstd, dsum=None, amax=None, workspace=None, stream=None):
    """Allocates and computes (dx, dweight, dbias)."""
    if stream is not None:
        with _on_stream(stream):
            return layernorm_backward(dy, x, weight, mean, rstd, dsum, amax, workspace)
    import torch
    shape, device = _layernorm_backward_inputs(dy, x, weight, mean, rstd, dsum, amax)
    dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    dweight, dbias = _floats(2, shape[1], x.device).unbind()
    if workspace is None:
        workspace = _floats(1, lib().nvfp4_layernorm_backward_workspace_bytes(*shape) // 4, x.device)
    else:
        _scratch(workspace, device)
    _layernorm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, dsum, amax, workspace, shape, device, None)
    return dx, dweight, dbias


def _heads(t, shape) -> bytes:
    """The C form of [batch][tokens][heads][dim], or of packed [tokens][heads][dim]."""
    st = t.stride()  # of a dimension of one element: anything, and not used
    return _HEADS.pack(t.data_ptr(), st[0] if len(shape) == 4 and shape[0] > 1 else 0,
                       st[-3] if shape[-3] > 1 else shape[-2] * shape[-1], st[-2] if shape[-2] > 1 else 0)


def _attention_inputs(q, k, v, causal, window, scale, cu_q, cu_k, max_q, max_k):
    """(C shape, heads, query tokens, device) of the checked inputs of an attention call."""
    import torch
    packed = cu_q is not None
    if packed != (cu_k is not None) or (packed and (max_q is None or max_k is None)):
        raise ValueError("packed sequences need cu_q, cu_k, max_q and max_k")
    bf16, device, dims = torch.bfloat16, q.get_device(), 3 if packed else 4
    for t, what in ((q, "q"), (k, "k"), (v, "v")):
        if t.dtype != bf16:
            raise TypeError("%s: bfloat16 is wanted, not %s" % (what, t.dtype))
        if t.dim() != dims or device < 0 or t.get_device() != device:
            raise ValueError("%s: a device tensor [%stokens][heads][dim] is wanted" % (what, "" if packed else "batch]["))
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("%s: a contiguous last dimension is wanted" % what)
    sq, sk = q.shape, k.shape
    if v.shape != sk or sk[-1] != sq[-1] or (not packed and sk[0] != sq[0]):
        raise ValueError("q, k and v do not fit: %s, %s, %s" % (tuple(sq), tuple(sk), tuple(v.shape)))
    if scale is None:
        scale = sq[-1] ** -0.5
    if not packed:
        b, nq, h, d = sq
        nk = sk[1]
        return _SHAPE.pack(b, nq, nk, h, sk[2], d, causal, window, 0, 0, b * nq, b * nk, scale), sq, sk, h, b * nq, device
    n = cu_q.shape[0]
    _vector(cu_q, n, device, "cu_q", torch.int32)
    _vector(cu_k, n, device, "cu_k", torch.int32)
    return (_SHAPE.pack(n - 1, max_q, max_k, sq[1], sk[1], sq[2], causal, window, cu_q.data_ptr(), cu_k.data_ptr(), sq[0],
                        sk[0], scale), sq, sk, sq[1], sq[0], device)


def _as(t, shape, device, what):
    import torch
    if t.shape != shape or t.dtype != torch.bfloat16 or t.get_device() != device or (t.stride(-1) != 1 and shape[-1] > 1):
        raise ValueError("%s: a bfloat16 tensor of shape %s on device %d is wanted" % (what, tuple(shape), device))


def _lse(lse, heads, tokens, device):
    import torch
    if lse.shape != (heads, tokens) or lse.dtype != torch.float32 or lse.get_device() != device or not lse.is_contiguous():
        raise ValueError("lse: a contiguous float32 tensor of shape %s on device %d is wanted" % ((heads, tokens), device))


def nvfp4_attention(q, k, v, o, lse, causal=True, window=0, scale=None, cu_q=None, cu_k=None, max_q=None, max_k=None,
                    workspace=None, stream=None):
    """o = softmax(scale q k^T) v and lse [heads][all queries] for [batch][tokens][heads][dim] tensors, or packed
    [tokens][heads][dim] ones with cu_q, cu_k (int32 [batch + 1], device) and the longest lengths max_q, max_k.
    workspace: new_attention_workspace's, where one is needed.  Tokens of no packed sequence are not written."""
    s, sq, sk, heads, tokens, device = _attention_inputs(q, k, v, causal, window, scale, cu_q, cu_k, max_q, max_k)
    _as(o, sq, device, "o")
    _lse(lse, heads, tokens, device)
    if workspace is not None:
        _scratch(workspace, device)
    _check(lib().nvfp4_attention(s, _heads(q, sq), _heads(k, sk), _heads(v, sk), _heads(o, sq), lse.data_ptr(),
                                 _ptr(workspace), _nbytes(workspace), _raw_stream(stream, device)), "nvfp4_attention")
    return o


def attention(q, k, v, causal=True, window=0, scale=None, cu_q=None, cu_k=None, max_q=None, max_k=None, workspace=None,
              stream=None):
    """Allocates and computes (o, lse).  Rows of tokens that belong to no packed sequence are left uninitialised: a buffer
    that a maximum is taken of later is better passed to nvfp4_attention, with zeros there."""
    if stream is not None:
        with _on_stream(stream):
            return attention(q, k, v, causal, window, scale, cu_q, cu_k, max_q, max_k, workspace)
    import torch
    s, sq, sk, heads, tokens, device = _attention_inputs(q, k, v, causal, window, scale, cu_q, cu_k, max_q, max_k)
    L = lib()
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = _floats(heads, tokens, q.device)
    if workspace is None:
        need = L.nvfp4_attention_workspace_bytes(s)
        if need:
            workspace = _floats(1, need // 4, q.device)
    else:
        _scratch(workspace, device)
    _check(L.nvfp4_attention(s, _heads(q, sq), _heads(k, sk), _heads(v, sk), _heads(o, sq), lse.data_ptr(), _ptr(workspace),
                             _nbytes(workspace), _raw_stream(None, device)), "nvfp4_attention")
    return o, lse


def _attention_backward(s, d_o, q, k, v, o, lse, dq, dk, dv, workspace, sq, sk, stream):
    _check(lib().nvfp4_attention_backward(s, _heads(q, sq), _heads(k, sk), _heads(v, sk), _heads(o, sq), lse.data_ptr(),
                                          _heads(d_o, sq), _heads(dq, sq), _heads(dk, sk), _heads(dv, sk),
                                          _ptr(workspace), _nbytes(workspace), stream), "nvfp4_attention_backward")


def nvfp4_attention_backward(d_o, q, k, v, o, lse, dq, dk, dv, workspace, causal=True, window=0, scale=None, cu_q=None,
                             cu_k=None, max_q=None, max_k=None, stream=None):
    """dq, dk and dv of nvfp4_attention with the same arguments.  dq may be o, dk and dv may be k and v."""
    s, sq, sk, heads, tokens, device = _attention_inputs(q, k, v, causal, window, scale, cu_q, cu_k, max_q, max_k)
    for t, shape, what in ((d_o, sq, "d_o"), (o, sq, "o"), (dq, sq, "dq"), (dk, sk, "dk"), (dv, sk, "dv")):
        _as(t, shape, device, what)
    _lse(lse, heads, tokens, device)
    if workspace is not None:
        _scratch(workspace, device)
    _attention_backward(s, d_o, q, k, v, o, lse, dq, dk, dv, workspace, sq, sk, _raw_stream(stream, device))
    return dq, dk, dv


def new_attention_workspace(q, k, v, causal=True, window=0, scale=None, cu_q=None, cu_k=None, max_q=None, max_k=None):
    """A workspace of nvfp4_attention and nvfp4_attention_backward for these arguments (one per stream)."""
    import torch
    s = _attention_inputs(q, k, v, causal, window, scale, cu_q, cu_k, max_q, max_k)[0]
    need = max(lib().nvfp4_attention_backward_workspace_bytes(s), lib().nvfp4_attention_workspace_bytes(s))
    return torch.empty(need, dtype=torch.uint8, device=q.device)


def attention_backward(d_o, q, k, v, o, lse, causal=True, window=0, scale=None, cu_q=None, cu_k=None, max_q=None,
                       max_k=None, workspace=None, stream=None):
    """Allocates and computes (dq, dk, dv); rows of tokens that belong to no packed sequence are left uninitialised."""
    if stream is not None:
        with _on_stream(stream):
            return attention_backward(d_o, q, k, v, o, lse, causal, window, scale, cu_q, cu_k, max_q, max_k, workspace)
    import torch
    s, sq, sk, heads, tokens, device = _attention_inputs(q, k, v, causal, window, scale, cu_q, cu_k, max_q, max_k)
    _as(d_o, sq, device, "d_o")
    _as(o, sq, device, "o")
    _lse(lse, heads, tokens, device)
    dense = torch.contiguous_format
    dq, dk, dv = torch.empty_like(q, memory_format=dense), torch.empty_like(k, memory_format=dense), torch.empty_like(
        v, memory_format=dense)
    if workspace is None:
        workspace = _floats(1, lib().nvfp4_attention_backward_workspace_bytes(s) // 4, q.device)
    else:
        _scratch(workspace, device)
    _attention_backward(s, d_o, q, k, v, o, lse, dq, dk, dv, workspace, sq, sk, _raw_stream(None, device))
    return dq, dk, dv


@dataclass
class AdamWTensor:
    """One tensor of an AdamW step: param and grad float32 or bfloat16; m, v float32 (32-bit states), or uint8 with
    their block scales (8-bit states: v holds sqrt(v)); copy: bfloat16, or None; amax: float32 [1], or None."""
    param: "object"
    grad: "object"
    m: "object"
    v: "object"
    m_scale: "object" = None
    v_scale: "object" = None
    weight_decay: float = 0.0
    copy: "object" = None
    amax: "object" = None

    def c_struct(self) -> nvfp4_adamw_tensor:
        import torch
        n, bits = self.param.numel(), 8 if self.m.dtype == torch.uint8 else 32
        state = torch.uint8 if bits == 8 else torch.float32
        wanted = [(self.param, n, None, "param"), (self.grad, n, None, "grad"), (self.m, n, state, "m"),
                  (self.v, n, state, "v"), (self.copy, n, torch.bfloat16, "copy"), (self.amax, 1, torch.float32, "amax")]
        if bits == 8:
            blocks = (n + 31) // 32
            wanted += [(self.m_scale, blocks, torch.uint8, "m_scale"), (self.v_scale, blocks, torch.uint8, "v_scale")]
            if self.m_scale is None or self.v_scale is None:
                raise ValueError("8-bit states need m_scale and v_scale")
        elif self.m_scale is not None or self.v_scale is not None:
            raise ValueError("32-bit states have no scales")
        for t, size, dtype, what in wanted:
            if t is None:
                continue
            if t.numel() != size or not t.is_contiguous() or not t.is_cuda or t.device != self.param.device:
                raise ValueError("%s: a contiguous device tensor of %d elements is wanted" % (what, size))
            if dtype is not None and t.dtype != dtype:
                raise TypeError("%s: %s is wanted, not %s" % (what, dtype, t.dtype))
        return nvfp4_adamw_tensor(self.param.data_ptr(), self.grad.data_ptr(), self.m.data_ptr(), self.v.data_ptr(),
                                  _ptr(self.m_scale), _ptr(self.v_scale), _ptr(self.copy), _ptr(self.amax), n,
                                  _dtype(self.param), _dtype(self.grad), bits, self.weight_decay)


def adamw_tensor(param, grad, state_bits=32, weight_decay=0.0, copy=None, amax=None) -> AdamWTensor:
    """An AdamWTensor with new zero states of 32 or 8 bits."""
    import torch
    if state_bits not in (8, 32):
        raise ValueError("state_bits: 8 or 32 is wanted")
    n, device = param.numel(), param.device
    if state_bits == 32:
        m, v = (torch.zeros(param.shape, dtype=torch.float32, device=device) for _ in range(2))
        return AdamWTensor(param, grad, m, v, None, None, weight_decay, copy, amax)
    m, v = (torch.zeros(param.shape, dtype=torch.uint8, device=device) for _ in range(2))
    ms, vs = (torch.ones((n + 31) // 32, dtype=torch.uint8, device=device) for _ in range(2))
    return AdamWTensor(param, grad, m, v, ms, vs, weight_decay, copy, amax)


class AdamWList:
    """The tensors of an AdamW step with their descriptors laid out once; the buffers stay the same from step to step
    (a gradient's may be replaced by set_grad)."""

    def __init__(self, tensors: Sequence[AdamWTensor]):
        self.tensors = list(tensors)
        if not self.tensors:
            raise ValueError("no tensors")
        self.array = (nvfp4_adamw_tensor * len(self.tensors))(*[t.c_struct() for t in self.tensors])
        self.device = self.tensors[0].param.get_device()
        if any(t.param.get_device() != self.device for t in self.tensors):
            raise ValueError("the tensors are on several devices")
        self.eight_bit = any(t.state_bits == 8 for t in self.array)

    def set_grad(self, index: int, grad):
        t = self.tensors[index]
        if grad.get_device() != self.device:
            raise ValueError("grad: a tensor on device %d is wanted" % self.device)
        old, t.grad = t.grad, grad
        try:
            self.array[index] = t.c_struct()
        except Exception:
            t.grad = old
            raise


def adamw(tensors, lr, beta1=0.9, beta2=0.999, eps=1e-8, step=1, rounding=None, seed=0, grad_scale=None, stream=None):
    """One AdamW step (number `step`, from 1) of an AdamWList, or of a sequence of AdamWTensor.  rounding: "rtn" or
    "sr"; None: "sr" where any states have 8 bits, else "rtn".  To nearest, an 8-bit v does not follow its gradients (a
    step moves it by less than half of what its format resolves), and steps grow as the bias correction fades."""
    import torch
    if not isinstance(tensors, AdamWList):
        tensors = AdamWList(tensors)
    if grad_scale is not None:
        _vector(grad_scale, 1, tensors.device, "grad_scale", torch.float32)
    if rounding is None:
        rounding = SR if tensors.eight_bit else RTN
    c = nvfp4_adamw_config(lr, beta1, beta2, eps, ROUNDINGS.get(rounding, rounding), step, seed, _ptr(grad_scale))
    _check(lib().nvfp4_adamw(tensors.array, len(tensors.array), ctypes.byref(c), _raw_stream(stream, tensors.device)),
           "nvfp4_adamw")


def adamw_state_values(t: AdamWTensor):
    """(m, v) of a tensor as float32, whatever its states are held in."""
    import torch
    if t.m_scale is None:
        return t.m.clone(), t.v.clone()
    n = t.m.numel()
    m, r = (torch.repeat_interleave(torch.exp2(s.float() - 127), 32)[:n].view(c.shape) * c.view(torch.float8_e4m3fn).float()
            for c, s in ((t.m, t.m_scale), (t.v, t.v_scale)))
    return m, r * r
