"""Python binding of libmxgemm.so (C ABI in include/mxgemm.h).

Argument marshalling only: shapes, dtypes and devices of torch tensors are
checked, outputs are allocated with torch when not given, and the device
pointers plus the current HIP stream are handed to the library.  Every step of
the computation runs in the library's HIP kernels; there is no fallback.  If
the library has not been built, loading fails with MXGemmError.
"""
from __future__ import annotations

import ctypes
import os

import torch

E4M3 = 0
E5M2 = 1
E2M3 = 2
E3M2 = 3
E2M1 = 4
INT4 = 8
INT2 = 9
FMT_FP8_FP8 = 0
FMT_FP8_FP4 = 1
FMT_FP4_FP4 = 2
FMT_BF8_BF8 = 3
FMT_FP8_BF8 = 4
FMT_BF8_FP8 = 5
FMT_FP8_INT4 = 6
FMT_FP8_INT2 = 7
FMT_FP8_FP6 = 8
FMT_FP8_BF6 = 9

_FMT_ELEMS = {FMT_FP8_FP8: (E4M3, E4M3), FMT_FP8_FP4: (E4M3, E2M1), FMT_FP4_FP4: (E2M1, E2M1),
              FMT_BF8_BF8: (E5M2, E5M2), FMT_FP8_BF8: (E4M3, E5M2), FMT_BF8_FP8: (E5M2, E4M3),
              FMT_FP8_INT4: (E4M3, INT4), FMT_FP8_INT2: (E4M3, INT2), FMT_FP8_FP6: (E4M3, E2M3),
              FMT_FP8_BF6: (E4M3, E3M2)}

# output types and activations of the fused epilogue (MXG_OUT_*, MXG_ACT_*)
OUT_F32 = 0
OUT_BF16 = 1
OUT_F16 = 2
ACT_NONE = 0
ACT_GELU = 1
# kind of mxgemm_mfma_ceiling beside the FMT_* pairs
CEIL_FP16 = 16
# scores of expert_route (MXG_SCORE_*) and the largest K of an int8 product
GRAD_ANY_SCALE = 16
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
INT8_MAX_K = 131056
# codes that rmsnorm_quantize writes (MXG_QUANT_*)
QUANT_NONE = 0
QUANT_INT8 = 1
QUANT_FP8 = 2
QUANT_FP8_POW2 = 3
QUANT_MXFP8 = 4
_OUT_DTYPES = {OUT_F32: torch.float32, OUT_BF16: torch.bfloat16, OUT_F16: torch.float16}
_DTYPE_IDS = {t: i for i, t in _OUT_DTYPES.items()}

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxgemm.so")


class MXGemmError(RuntimeError):
    pass


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise MXGemmError("libmxgemm.so is not built (run __graft_entry__.build() or "
                          "python -m block_scaled_precision_mxgemm_amd.build): " + library_path)
    lib = ctypes.CDLL(library_path)
    p = ctypes.c_void_p
    i64 = ctypes.c_int64
    ci = ctypes.c_int
    lib.mxgemm_quantize.argtypes = [p, i64, i64, ci, p, p, p]
    lib.mxgemm_quantize.restype = ci
    lib.mxgemm_run.argtypes = [p, p, p, p, p, i64, i64, i64, ci, p]
    lib.mxgemm_run.restype = ci
    lib.mxgemm_run_dequant_fp16.argtypes = [p, p, p, p, p, i64, i64, i64, ci, p]
    lib.mxgemm_run_dequant_fp16.restype = ci
    lib.mxgemm_run_fused.argtypes = [p, p, p, p, p, i64, i64, i64, ci, p, ci, ci, p]
    lib.mxgemm_run_fused.restype = ci
    lib.mxgemm_epilogue.argtypes = [p, i64, i64, p, ci, ci, p, p]
    lib.mxgemm_epilogue.restype = ci
    lib.fp16gemm_run.argtypes = [p, p, p, i64, i64, i64, ci, p]
    lib.fp16gemm_run.restype = ci
    lib.mxgemm_mfma_ceiling.argtypes = [p, i64, p, i64, ci, i64, ci, p, p, p]
    lib.mxgemm_mfma_ceiling.restype = ci
    cf = ctypes.c_float
    lib.int8gemm_quantize.argtypes = [p, ci, i64, i64, p, p, p]
    lib.int8gemm_run.argtypes = [p, p, p, p, p, i64, i64, i64, p, ci, ci, p]
    lib.int8gemm_run_grouped.argtypes = [p, p, i64, p, p, p, i64, i64, i64, i64, p, p, ci, p, ci, ci, p]
    lib.expert_route.argtypes = [p, ci, i64, i64, ci, ci, p, ci, ci, ci, ci, cf, p, p, p]
    lib.expert_route_backward.argtypes = [p, ci, i64, i64, p, p, ci, ci, ci, cf, p, p]
    lib.expert_plan.argtypes = [p, i64, ci, i64, p, p, p, p, p]
    lib.expert_combine.argtypes = [p, ci, i64, i64, p, p, i64, ci, p, ci, p]
    lib.expert_combine_backward.argtypes = [p, ci, p, ci, i64, i64, p, p, i64, ci, p, p, p]
    lib.fp8gemm_quantize.argtypes = [p, ci, i64, i64, i64, ci, ci, p, p, p]
    lib.fp8gemm_run.argtypes = [p, p, p, p, p, i64, i64, i64, p, ci, ci, p]
    lib.fp8gemm_run_grouped.argtypes = [p, p, i64, p, p, p, i64, i64, i64, i64, p, p, ci, p, ci, ci, p]
    lib.fp8gemm_weight_grad.argtypes = [p, ci, i64, i64, p, p, i64, p, ci, p, p]
    lib.fp8gemm_weight_grad_grouped.argtypes = [p, ci, i64, i64, p, p, i64, i64, i64, p, p, ci, p, ci, p, p]
    lib.rmsnorm_quantize.argtypes = [p, p, ci, p, ci, i64, i64, cf, p, p, ci, p, p, p, p]
    lib.rmsnorm_backward.argtypes = [p, p, p, ci, p, ci, p, i64, i64, p, p, p, p]
    lib.fp8gemm_weight_grad_workspace.argtypes = [i64, i64, i64, i64]
    lib.rmsnorm_backward_workspace.argtypes = [i64, i64]
    for name in ("fp8gemm_quantize", "fp8gemm_run", "fp8gemm_run_grouped", "fp8gemm_weight_grad",
                 "fp8gemm_weight_grad_grouped", "rmsnorm_quantize", "rmsnorm_backward"):
        getattr(lib, name).restype = ci
    for name in ("fp8gemm_weight_grad_workspace", "rmsnorm_backward_workspace"):
        getattr(lib, name).restype = i64
    for name in ("int8gemm_quantize", "int8gemm_run", "int8gemm_run_grouped", "expert_route", "expert_route_backward",
                 "expert_plan", "expert_combine", "expert_combine_backward"):
        getattr(lib, name).restype = ci
    lib.expert_plan_workspace.argtypes = [i64, ci, i64]
    lib.expert_plan_workspace.restype = i64
    lib.mxgemm_device_supported.argtypes = []
    lib.mxgemm_device_supported.restype = ci
    lib.mxgemm_status_string.argtypes = [ci]
    lib.mxgemm_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = _load().mxgemm_status_string(rc).decode()
        raise MXGemmError("%s failed: status %d (%s)" % (what, rc, msg))


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev_u8(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(name + " must be a GPU tensor")
    if t.dtype in (torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu):
        t = t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(name + " must hold uint8 codes")
    if not t.is_contiguous():
        raise ValueError(name + " must be contiguous")
    return t


def _row_bytes(K: int, elem: int) -> int:
    if elem in (E2M1, INT4):
        return K // 2
    if elem == INT2:
        return K // 4
    if elem in (E2M3, E3M2):
        return K // 4 * 3
    return K


def mxgemm_device_supported() -> bool:
    rc = _load().mxgemm_device_supported()
    if rc < 0:
        _check(-rc, "mxgemm_device_supported")
    return rc == 1


def mxgemm_quantize(x: torch.Tensor, elem: int = E4M3, q: torch.Tensor | None = None,
                    s: torch.Tensor | None = None, stream=None):
    """Quantize fp32 rows (rows x K, K contiguous) to (codes, scales), uint8 tensors."""
    if x.dtype != torch.float32 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D float32 GPU tensor")
    rows, K = x.shape
    if q is None:
        q = torch.empty((rows, _row_bytes(K, elem)), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty((rows, K // 32), dtype=torch.uint8, device=x.device)
    q = _dev_u8(q, "q")
    s = _dev_u8(s, "s")
    if q.shape != (rows, _row_bytes(K, elem)) or s.shape != (rows, K // 32):
        raise ValueError("output shapes do not match x")
    rc = _load().mxgemm_quantize(x.data_ptr(), rows, K, elem, q.data_ptr(), s.data_ptr(), _stream(stream))
    _check(rc, "mxgemm_quantize")
    return q, s


def _mx_args(a_q, a_s, b_q, b_s, fmt, out, out_dtype=torch.float32):
    if fmt not in _FMT_ELEMS:
        raise ValueError("unknown fmt %r" % (fmt,))
    ea, eb = _FMT_ELEMS[fmt]
    a_q = _dev_u8(a_q, "a_q")
    a_s = _dev_u8(a_s, "a_s")
    b_q = _dev_u8(b_q, "b_q")
    b_s = _dev_u8(b_s, "b_s")
    M, nb = a_s.shape
    N = b_s.shape[0]
    K = nb * 32
    if a_q.shape != (M, _row_bytes(K, ea)) or b_q.shape != (N, _row_bytes(K, eb)) or b_s.shape != (N, nb):
        raise ValueError("operand shapes disagree: A %s/%s, B %s/%s" %
                         (tuple(a_q.shape), tuple(a_s.shape), tuple(b_q.shape), tuple(b_s.shape)))
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a_q.device)
    if out.dtype != out_dtype or out.shape != (M, N) or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous M x N %s GPU tensor" % (out_dtype,))
    return a_q, a_s, b_q, b_s, out, M, N, K


def _bias_arg(bias, N):
    if bias is None:
        return None
    if bias.dtype != torch.float32 or not bias.is_cuda or bias.shape != (N,) or not bias.is_contiguous():
        raise ValueError("bias must be a contiguous float32 GPU tensor of N values")
    return bias


def mxgemm_run(a_q, a_s, b_q, b_s, fmt: int = FMT_FP8_FP8, out: torch.Tensor | None = None, stream=None):
    """C = (A * 2^sA)(B * 2^sB)^T in fp32; A: M x K codes, B: N x K codes."""
    a_q, a_s, b_q, b_s, out, M, N, K = _mx_args(a_q, a_s, b_q, b_s, fmt, out)
    rc = _load().mxgemm_run(a_q.data_ptr(), a_s.data_ptr(), b_q.data_ptr(), b_s.data_ptr(), out.data_ptr(),
                            M, N, K, fmt, _stream(stream))
    _check(rc, "mxgemm_run")
    return out


def mxgemm_run_fused(a_q, a_s, b_q, b_s, fmt: int = FMT_FP8_FP8, bias: torch.Tensor | None = None,
                     act: int = ACT_NONE, out_type: int = OUT_F32, out: torch.Tensor | None = None, stream=None):
    """mxgemm_run with the output step fused into the GEMM: C = out_type(act(A B^T + bias)).
    bias: N float32 values or None; act: ACT_NONE / ACT_GELU; out_type: OUT_F32 /
    OUT_BF16 / OUT_F16 (the output tensor's dtype float32 / bfloat16 / float16)."""
    if out_type not in _OUT_DTYPES:
        raise ValueError("unknown out_type %r" % (out_type,))
    a_q, a_s, b_q, b_s, out, M, N, K = _mx_args(a_q, a_s, b_q, b_s, fmt, out, _OUT_DTYPES[out_type])
    bias = _bias_arg(bias, N)
    rc = _load().mxgemm_run_fused(a_q.data_ptr(), a_s.data_ptr(), b_q.data_ptr(), b_s.data_ptr(), out.data_ptr(),
                                  M, N, K, fmt, None if bias is None else bias.data_ptr(), act, out_type,
                                  _stream(stream))
    _check(rc, "mxgemm_run_fused")
    return out


def mxgemm_epilogue(x: torch.Tensor, bias: torch.Tensor | None = None, act: int = ACT_NONE,
                    out_type: int = OUT_F32, out: torch.Tensor | None = None, stream=None):
    """The same output step as a separate pass over an fp32 M x N matrix x."""
    if x.dtype != torch.float32 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D float32 GPU tensor")
    if out_type not in _OUT_DTYPES:
        raise ValueError("unknown out_type %r" % (out_type,))
    M, N = x.shape
    if out is None:
        out = torch.empty((M, N), dtype=_OUT_DTYPES[out_type], device=x.device)
    if out.dtype != _OUT_DTYPES[out_type] or out.shape != (M, N) or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous M x N %s GPU tensor" % (_OUT_DTYPES[out_type],))
    bias = _bias_arg(bias, N)
    rc = _load().mxgemm_epilogue(x.data_ptr(), M, N, None if bias is None else bias.data_ptr(), act, out_type,
                                 out.data_ptr(), _stream(stream))
    _check(rc, "mxgemm_epilogue")
    return out


def mxgemm_run_dequant_fp16(a_q, a_s, b_q, b_s, fmt: int = FMT_FP8_FP8, out: torch.Tensor | None = None,
                            stream=None):
    """Ablation: dequantize to fp16 in registers, then fp16 MFMA (fp8 x fp8 only)."""
    a_q, a_s, b_q, b_s, out, M, N, K = _mx_args(a_q, a_s, b_q, b_s, fmt, out)
    rc = _load().mxgemm_run_dequant_fp16(a_q.data_ptr(), a_s.data_ptr(), b_q.data_ptr(), b_s.data_ptr(),
                                         out.data_ptr(), M, N, K, fmt, _stream(stream))
    _check(rc, "mxgemm_run_dequant_fp16")
    return out


def fp16gemm_run(a: torch.Tensor, b: torch.Tensor, b_is_nk: bool, out: torch.Tensor | None = None, stream=None):
    """fp16 GEMM with fp32 output. a: M x K; b: N x K if b_is_nk else K x N."""
    for name, t in (("a", a), ("b", b)):
        if t.dtype not in (torch.float16, torch.int16, torch.uint16) or not t.is_cuda or not t.is_contiguous():
            raise ValueError(name + " must be a contiguous fp16 GPU tensor")
    M, K = a.shape
    N = b.shape[0] if b_is_nk else b.shape[1]
    if (b.shape[1] if b_is_nk else b.shape[0]) != K:
        raise ValueError("inner dimensions disagree")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=a.device)
    if out.dtype != torch.float32 or out.shape != (M, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous M x N float32 tensor")
    rc = _load().fp16gemm_run(a.data_ptr(), b.data_ptr(), out.data_ptr(), M, N, K, 1 if b_is_nk else 0,
                              _stream(stream))
    _check(rc, "fp16gemm_run")
    return out


def mxgemm_mfma_ceiling(ops: torch.Tensor, scales: torch.Tensor | None, kind: int, iters: int, workgroups: int,
                        out: torch.Tensor | None = None, clocks: torch.Tensor | None = None, stream=None):
    """Measurement helper: run `iters` rounds of the large GEMM's 32-MFMA
    compute phase per wave on fragments taken from the bytes of `ops` (and
    scale registers from `scales`), `workgroups` workgroups of 8 waves, no
    memory traffic.  kind: an FMT_* pair or CEIL_FP16.  Returns `out`
    (workgroups * 512 floats).  Flops: workgroups * 8 * iters * 32 * 65536
    (CEIL_FP16: workgroups * 8 * iters * 64 * 16384).  clocks (optional,
    workgroups * 2 int32): shader cycles and 100 MHz ticks of each
    workgroup's first wave over its MFMA loop."""
    if not ops.is_cuda or not ops.is_contiguous():
        raise ValueError("ops must be a contiguous GPU tensor")
    if scales is not None and (not scales.is_cuda or not scales.is_contiguous()):
        raise ValueError("scales must be a contiguous GPU tensor")
    if out is None:
        out = torch.empty(workgroups * 512, dtype=torch.float32, device=ops.device)
    if out.dtype != torch.float32 or out.numel() < workgroups * 512 or not out.is_contiguous():
        raise ValueError("out must hold workgroups * 512 contiguous floats")
    if clocks is not None and (clocks.dtype != torch.int32 or clocks.numel() < 2 * workgroups
                               or not clocks.is_contiguous()):
        raise ValueError("clocks must hold workgroups * 2 contiguous int32")
    rc = _load().mxgemm_mfma_ceiling(ops.data_ptr(), ops.numel() * ops.element_size(),
                                     None if scales is None else scales.data_ptr(),
                                     0 if scales is None else scales.numel() * scales.element_size(),
                                     kind, iters, workgroups, out.data_ptr(),
                                     None if clocks is None else clocks.data_ptr(), _stream(stream))
    _check(rc, "mxgemm_mfma_ceiling")
    return out


# ---- int8 products and experts ----------------------------------------------


def _arg(t, name: str, dtypes, shape=None, dim: int | None = None, like: torch.Tensor | None = None) -> torch.Tensor:
    """A contiguous GPU tensor of one of `dtypes`, of the shape or number of
    dimensions given, on the device of `like`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(name + " must be a GPU tensor")
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, not %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if dim is not None and t.dim() != dim:
        raise ValueError("%s must have %d dimensions" % (name, dim))
    if not t.is_contiguous():
        raise ValueError(name + " must be contiguous")
    if like is not None and t.device != like.device:
        raise ValueError("%s is on %s, the other operands on %s" % (name, t.device, like.device))
    return t


def _new(shape, dtype, device: torch.device, stream=None, make=torch.empty) -> torch.Tensor:
    """A tensor for a call on `stream`: it is made there, since memory of the
    current stream's pool may still be in use by work queued on that one."""
    if stream is None:
        return make(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(*shape, dtype=dtype, device=device)


def _out(t, name: str, dtype, shape, like: torch.Tensor, stream=None) -> torch.Tensor:
    if t is not None:
        return _arg(t, name, (dtype,), shape, like=like)
    if stream is not None:
        return _new(shape, dtype, like.device, stream)
    return torch.empty(*shape, dtype=dtype, device=like.device)


def _on16(t: torch.Tensor, stream) -> torch.Tensor:
    """The values where the library takes them: at a multiple of 16 bytes.  Others
    (one expert's row of E x N scales, with N not a multiple of 4) are copied on
    the call's stream."""
    if t.data_ptr() & 15 == 0:
        return t
    if stream is None:
        return t.clone()
    with torch.cuda.stream(stream):
        return t.clone()


_FLOATS = tuple(_DTYPE_IDS)


def _ptr(t):
    return None if t is None else t.data_ptr()


# Without Stream and device objects around them, where this torch has them (2
# us less per call, of about 9): the current stream's handle, the current device.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name: str, device: torch.device, stream, *args):
    """An entry point on the operands' own device; without a stream, on that
    device's current one."""
    index = device.index
    if _current_device() != index:
        with torch.cuda.device(device):
            return _call(name, device, stream, *args)
    rc = getattr(_lib or _load(), name)(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, name)


def int8gemm_quantize(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None, stream=None):
    """Quantize rows (rows x K of float32, bfloat16 or float16, K a multiple of
    16) to (int8 codes, fp32 scale per row): tokens, or the N x K weights of a
    layer with a scale per output channel."""
    x = _arg(x, "x", _FLOATS, dim=2)
    rows, K = x.shape
    q = _out(q, "q", torch.int8, (rows, K), x, stream)
    s = _out(s, "s", torch.float32, (rows,), x, stream)
    _call("int8gemm_quantize", x.device, stream, x.data_ptr(), _DTYPE_IDS[x.dtype], rows, K, q.data_ptr(), s.data_ptr())
    return q, s


def int8gemm_run(a_q, a_s, b_q, b_s, bias: torch.Tensor | None = None, act: int = ACT_NONE, out_type: int = OUT_F32,
                 out: torch.Tensor | None = None, stream=None):
    """C = out_type(act(a_s[i] b_s[j] sum_k a_q[i][k] b_q[j][k] + bias[j])); a_q: M x K,
    b_q: N x K int8; a_s: M, b_s: N float32 scales per token and per channel."""
    if out_type not in _OUT_DTYPES:
        raise ValueError("unknown out_type %r" % (out_type,))
    a_q = _arg(a_q, "a_q", (torch.int8,), dim=2)
    M, K = a_q.shape
    b_q = _arg(b_q, "b_q", (torch.int8,), dim=2, like=a_q)
    N = b_q.shape[0]
    if b_q.shape[1] != K:
        raise ValueError("inner dimensions disagree: a_q %s, b_q %s" % (tuple(a_q.shape), tuple(b_q.shape)))
    a_s = _arg(a_s, "a_s", (torch.float32,), (M,), like=a_q)
    b_s = _on16(_arg(b_s, "b_s", (torch.float32,), (N,), like=a_q), stream)
    if bias is not None:
        bias = _on16(_arg(bias, "bias", (torch.float32,), (N,), like=a_q), stream)
    out = _out(out, "out", _OUT_DTYPES[out_type], (M, N), a_q, stream)
    _call("int8gemm_run", a_q.device, stream, a_q.data_ptr(), a_s.data_ptr(), b_q.data_ptr(), b_s.data_ptr(),
          out.data_ptr(), M, N, K, _ptr(bias), act, out_type)
    return out


def int8gemm_run_grouped(a_q, a_s, b_q, b_s, offsets, index: torch.Tensor | None = None, index_div: int = 1,
                         bias: torch.Tensor | None = None, act: int = ACT_NONE, out_type: int = OUT_F32,
                         out: torch.Tensor | None = None, stream=None):
    """The products of E experts: rows offsets[e] .. offsets[e+1]-1 of the result
    with b_q[e] (E x N x K), b_s[e] and bias[e] (E x N).  Row p takes row
    index[p] // index_div of a_q, or row p without an index.  offsets (E + 1)
    and index are int32 tensors, as expert_plan gives them.  Rows outside the
    offsets are left as they were; without `out` they hold nothing defined."""
    if out_type not in _OUT_DTYPES:
        raise ValueError("unknown out_type %r" % (out_type,))
    a_q = _arg(a_q, "a_q", (torch.int8,), dim=2)
    rows_a, K = a_q.shape
    b_q = _arg(b_q, "b_q", (torch.int8,), dim=3, like=a_q)
    E, N = b_q.shape[:2]
    if b_q.shape[2] != K:
        raise ValueError("inner dimensions disagree: a_q %s, b_q %s" % (tuple(a_q.shape), tuple(b_q.shape)))
    a_s = _arg(a_s, "a_s", (torch.float32,), (rows_a,), like=a_q)
    b_s = _on16(_arg(b_s, "b_s", (torch.float32,), (E, N), like=a_q), stream)
    offsets = _arg(offsets, "offsets", (torch.int32,), (E + 1,), like=a_q)
    rows = rows_a
    if index is not None:
        index = _arg(index, "index", (torch.int32,), dim=1, like=a_q)
        rows = index.shape[0]
    if bias is not None:
        bias = _on16(_arg(bias, "bias", (torch.float32,), (E, N), like=a_q), stream)
    out = _out(out, "out", _OUT_DTYPES[out_type], (rows, N), a_q, stream)
    _call("int8gemm_run_grouped", a_q.device, stream, a_q.data_ptr(), a_s.data_ptr(), rows_a, b_q.data_ptr(),
          b_s.data_ptr(), out.data_ptr(), rows, N, K, E, offsets.data_ptr(), _ptr(index), index_div, _ptr(bias), act,
          out_type)
    return out


def expert_route(logits, k: int, score: int = SCORE_SOFTMAX, bias: torch.Tensor | None = None, groups: int = 1,
                 top_groups: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
                 ids: torch.Tensor | None = None, weights: torch.Tensor | None = None, stream=None):
    """The k experts of each token (T x E logits) and their weights: (ids T x k
    int32, weights T x k float32).  bias (E float32) counts for the choice
    alone; with groups > 1 only the top_groups groups with the largest sum of
    their group_top largest scores (of experts that can be chosen) are chosen
    from.  Experts with a logit of -inf are not chosen; missing choices are -1
    with weight 0.  No autograd graph is recorded (as in all calls here): the
    gradient of the weights is expert_route_backward."""
    logits = _arg(logits, "logits", _FLOATS, dim=2)
    T, E = logits.shape
    if bias is not None:
        bias = _arg(bias, "bias", (torch.float32,), (E,), like=logits)
    if not 1 <= k <= E:
        raise ValueError("k must be 1 .. %d" % E)
    ids = _out(ids, "ids", torch.int32, (T, k), logits, stream)
    weights = _out(weights, "weights", torch.float32, (T, k), logits, stream)
    _call("expert_route", logits.device, stream, logits.data_ptr(), _DTYPE_IDS[logits.dtype], T, E, k, score, _ptr(bias),
          groups, top_groups, group_top, int(renormalize), scale, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def expert_route_backward(logits, ids, d_weights, score: int = SCORE_SOFTMAX, renormalize: bool = True,
                          scale: float = 1.0, d_logits: torch.Tensor | None = None, stream=None):
    """Gradient of the logits (T x E, in their type) from that of expert_route's
    weights (T x k float32), the choice `ids` held."""
    logits = _arg(logits, "logits", _FLOATS, dim=2)
    T, E = logits.shape
    ids = _arg(ids, "ids", (torch.int32,), dim=2, like=logits)
    k = ids.shape[1]
    if ids.shape[0] != T:
        raise ValueError("ids must have %d rows" % T)
    d_weights = _arg(d_weights, "d_weights", (torch.float32,), (T, k), like=logits)
    d_logits = _out(d_logits, "d_logits", logits.dtype, (T, E), logits, stream)
    _call("expert_route_backward", logits.device, stream, logits.data_ptr(), _DTYPE_IDS[logits.dtype], T, E,
          ids.data_ptr(), d_weights.data_ptr(), k, score, int(renormalize), scale, d_logits.data_ptr())
    return d_logits


def expert_plan(ids, experts: int, offsets: torch.Tensor | None = None, order: torch.Tensor | None = None,
                position: torch.Tensor | None = None, stream=None):
    """Slots (token * k + choice) sorted by expert, from ids (T x k int32; values
    outside 0 .. experts-1 are slots without an expert): (offsets E + 1, order
    T * k, position T x k), int32.  order[p] is the slot in row p, -1 behind the
    last expert's rows; position[t][j] is the slot's row, or -1."""
    ids = _arg(ids, "ids", (torch.int32,), dim=2)
    T, k = ids.shape
    need = _load().expert_plan_workspace(T, k, experts)
    if need < 0:
        _check(1, "expert_plan")
    n = T * k
    if offsets is None and order is None and position is None:
        # one allocation for the three (2 us less than three)
        offsets, order, position = _new((experts + 1 + 2 * n,), torch.int32, ids.device, stream).split_with_sizes(
            (experts + 1, n, n))
        position = position.view(T, k)
    else:
        offsets = _out(offsets, "offsets", torch.int32, (experts + 1,), ids, stream)
        order = _out(order, "order", torch.int32, (n,), ids, stream)
        position = _out(position, "position", torch.int32, (T, k), ids, stream)
    workspace = _new((need,), torch.uint8, ids.device, stream) if need else None
    _call("expert_plan", ids.device, stream, ids.data_ptr(), T, k, experts, offsets.data_ptr(), order.data_ptr(),
          position.data_ptr(), _ptr(workspace))
    return offsets, order, position


def _combine_args(y, position, weights):
    y = _arg(y, "y", _FLOATS, dim=2)
    position = _arg(position, "position", (torch.int32,), dim=2, like=y)
    T, k = position.shape
    weights = _arg(weights, "weights", (torch.float32,), (T, k), like=y)
    return y, position, weights, y.shape[0], y.shape[1], T, k


def expert_combine(y, position, weights, out_type: int | None = None, out: torch.Tensor | None = None, stream=None):
    """out[t] = sum_j weights[t][j] y[position[t][j]] (y: rows x N; position: T x k
    int32, values outside the rows add nothing; weights: T x k float32), summed
    in fp32, in out_type (y's type unless given).  No autograd graph is recorded:
    the gradient is expert_combine_backward."""
    y, position, weights, rows, N, T, k = _combine_args(y, position, weights)
    out_type = _DTYPE_IDS[y.dtype] if out_type is None else out_type
    if out_type not in _OUT_DTYPES:
        raise ValueError("unknown out_type %r" % (out_type,))
    out = _out(out, "out", _OUT_DTYPES[out_type], (T, N), y, stream)
    _call("expert_combine", y.device, stream, y.data_ptr(), _DTYPE_IDS[y.dtype], rows, N, position.data_ptr(),
          weights.data_ptr(), T, k, out.data_ptr(), out_type)
    return out


def expert_combine_backward(d_out, y, position, weights, d_y: torch.Tensor | None = None,
                            d_weights: torch.Tensor | None = None, stream=None):
    """Gradients (d_y in y's type, d_weights T x k float32) of expert_combine from
    that of its result.  Rows of d_y that no position names are left as they
    were; without `d_y` they are zero.  `d_y` may be y itself."""
    y, position, weights, rows, N, T, k = _combine_args(y, position, weights)
    d_out = _arg(d_out, "d_out", _FLOATS, (T, N), like=y)
    if d_y is None:
        d_y = _new((rows, N), y.dtype, y.device, stream, torch.zeros)
    d_y = _arg(d_y, "d_y", (y.dtype,), (rows, N), like=y)
    d_weights = _out(d_weights, "d_weights", torch.float32, (T, k), y, stream)
    _call("expert_combine_backward", y.device, stream, d_out.data_ptr(), _DTYPE_IDS[d_out.dtype], y.data_ptr(),
          _DTYPE_IDS[y.dtype], rows, N, position.data_ptr(), weights.data_ptr(), T, k, d_y.data_ptr(),
          d_weights.data_ptr())
    return d_y, d_weights


# ---- E4M3 products with a scale per block of 128 -------------------------------


def _blocks(d: int) -> int:
    return (d + 127) // 128


def _codes_arg(t, name: str, dim: int, like: torch.Tensor | None = None, shape=None) -> torch.Tensor:
    """E4M3 codes: uint8, or float8_e4m3fn taken as its bytes."""
    if isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    return _arg(t, name, (torch.uint8,), shape, dim, like)


def fp8gemm_quantize(x: torch.Tensor, block_rows: int = 1, pow2: bool = False, q: torch.Tensor | None = None,
                     s: torch.Tensor | None = None, stream=None):
    """Quantize rows (rows x K or E x rows x K of float32, bfloat16 or float16, K a
    multiple of 16) to (E4M3 codes as uint8, fp32 scales): one per row and 128
    columns (block_rows 1: activations) or per 128 x 128 block (block_rows 128:
    weights).  pow2: scales that are powers of two, as fp8gemm_weight_grad takes
    them without another rounding."""
    x = _arg(x, "x", _FLOATS)
    if x.dim() not in (2, 3):
        raise ValueError("x must have 2 or 3 dimensions")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    rows, K = x.shape[-2:]
    E = x.shape[0] if x.dim() == 3 else 1
    lead = tuple(x.shape[:-2])
    q = _out(q, "q", torch.uint8, lead + (rows, K), x, stream)
    s = _out(s, "s", torch.float32, lead + (-(-rows // block_rows), _blocks(K)), x, stream)
    _call("fp8gemm_quantize", x.device, stream, x.data_ptr(), _DTYPE_IDS[x.dtype], E, rows, K, block_rows, int(pow2),
          q.data_ptr(), s.data_ptr())
    return q, s


def fp8gemm_run(a_q, a_s, b_q, b_s, bias: torch.Tensor | None = None, act: int = ACT_NONE, out_type: int = OUT_F32,
                out: torch.Tensor | None = None, stream=None):
    """C = out_type(act(sum_b a_s[i][b] b_s[j // 128][b] sum_{k in block b} a_q[i][k] b_q[j][k]
    + bias[j])), blocks of 128 columns; a_q: M x K, b_q: N x K E4M3 codes; a_s: M x KB,
    b_s: NB x KB float32 (KB, NB the blocks of K and N)."""
    if out_type not in _OUT_DTYPES:
        raise ValueError("unknown out_type %r" % (out_type,))
    a_q = _codes_arg(a_q, "a_q", 2)
    M, K = a_q.shape
    b_q = _codes_arg(b_q, "b_q", 2, a_q)
    N = b_q.shape[0]
    if b_q.shape[1] != K:
        raise ValueError("inner dimensions disagree: a_q %s, b_q %s" % (tuple(a_q.shape), tuple(b_q.shape)))
    a_s = _arg(a_s, "a_s", (torch.float32,), (M, _blocks(K)), like=a_q)
    b_s = _arg(b_s, "b_s", (torch.float32,), (_blocks(N), _blocks(K)), like=a_q)
    if bias is not None:
        bias = _on16(_arg(bias, "bias", (torch.float32,), (N,), like=a_q), stream)
    out = _out(out, "out", _OUT_DTYPES[out_type], (M, N), a_q, stream)
    _call("fp8gemm_run", a_q.device, stream, a_q.data_ptr(), a_s.data_ptr(), b_q.data_ptr(), b_s.data_ptr(),
          out.data_ptr(), M, N, K, _ptr(bias), act, out_type)
    return out


def fp8gemm_run_grouped(a_q, a_s, b_q, b_s, offsets, index: torch.Tensor | None = None, index_div: int = 1,
                        bias: torch.Tensor | None = None, act: int = ACT_NONE, out_type: int = OUT_F32,
                        out: torch.Tensor | None = None, stream=None):
    """The products of E experts: rows offsets[e] .. offsets[e+1]-1 of the result
    with b_q[e] (E x N x K), b_s[e] (E x NB x KB) and bias[e] (E x N).  offsets, index,
    index_div and rows outside the offsets as for int8gemm_run_grouped."""
    if out_type not in _OUT_DTYPES:
        raise ValueError("unknown out_type %r" % (out_type,))
    a_q = _codes_arg(a_q, "a_q", 2)
    rows_a, K = a_q.shape
    b_q = _codes_arg(b_q, "b_q", 3, a_q)
    E, N = b_q.shape[:2]
    if b_q.shape[2] != K:
        raise ValueError("inner dimensions disagree: a_q %s, b_q %s" % (tuple(a_q.shape), tuple(b_q.shape)))
    a_s = _arg(a_s, "a_s", (torch.float32,), (rows_a, _blocks(K)), like=a_q)
    b_s = _arg(b_s, "b_s", (torch.float32,), (E, _blocks(N), _blocks(K)), like=a_q)
    offsets = _arg(offsets, "offsets", (torch.int32,), (E + 1,), like=a_q)
    rows = rows_a
    if index is not None:
        index = _arg(index, "index", (torch.int32,), dim=1, like=a_q)
        rows = index.shape[0]
    if bias is not None:
        bias = _on16(_arg(bias, "bias", (torch.float32,), (E, N), like=a_q), stream)
    out = _out(out, "out", _OUT_DTYPES[out_type], (rows, N), a_q, stream)
    _call("fp8gemm_run_grouped", a_q.device, stream, a_q.data_ptr(), a_s.data_ptr(), rows_a, b_q.data_ptr(),
          b_s.data_ptr(), out.data_ptr(), rows, N, K, E, offsets.data_ptr(), _ptr(index), index_div, _ptr(bias), act,
          out_type)
    return out


def _grad_workspace(rows: int, N: int, K: int, E: int, device: torch.device, stream):
    need = (_lib or _load()).fp8gemm_weight_grad_workspace(rows, N, K, E)
    if need < 0:
        _check(1, "fp8gemm_weight_grad")
    return _new((need,), torch.uint8, device, stream) if need else None


def fp8gemm_weight_grad(d_c, a_q, a_s, out_type: int = OUT_F32, out: torch.Tensor | None = None, stream=None,
                        any_scale: bool = False):
    """Gradient of fp8gemm_run's weights (N x K) from that of its result (d_c: M x N
    of float32, bfloat16 or float16) and the activations' codes (a_q: M x K, a_s: M x
    KB): sum_m d_c[m][n] a_s[m][k // 128] a_q[m][k], in fp32.  The products a_s a_q are
    rounded to bfloat16, which leaves them as they are when the scales are powers
    of two; any_scale: the scales, of any kind, are applied in fp32, which takes longer
    (8192 x 4096 x 4096 of bfloat16 1.2 ms, 0.23 without).  (The gradient of the activations is fp8gemm_run of the quantized d_c with
    the transposed weights and scales.)"""
    if out_type not in _OUT_DTYPES:
        raise ValueError("unknown out_type %r" % (out_type,))
    d_c = _arg(d_c, "d_c", _FLOATS, dim=2)
    M, N = d_c.shape
    a_q = _codes_arg(a_q, "a_q", 2, d_c)
    K = a_q.shape[1]
    if a_q.shape[0] != M:
        raise ValueError("rows disagree: d_c %s, a_q %s" % (tuple(d_c.shape), tuple(a_q.shape)))
    a_s = _arg(a_s, "a_s", (torch.float32,), (M, _blocks(K)), like=d_c)
    out = _out(out, "out", _OUT_DTYPES[out_type], (N, K), d_c, stream)
    workspace = _grad_workspace(M, N, K, 1, d_c.device, stream)
    _call("fp8gemm_weight_grad", d_c.device, stream, d_c.data_ptr(),
          _DTYPE_IDS[d_c.dtype] + (GRAD_ANY_SCALE if any_scale else 0), M, N, a_q.data_ptr(), a_s.data_ptr(), K,
          out.data_ptr(), out_type, _ptr(workspace))
    return out


def fp8gemm_weight_grad_grouped(d_c, a_q, a_s, offsets, index: torch.Tensor | None = None, index_div: int = 1,
                                out_type: int = OUT_F32, out: torch.Tensor | None = None, stream=None,
                                any_scale: bool = False):
    """Gradients of the weights of E experts (E x N x K): that of expert e from rows
    offsets[e] .. offsets[e+1]-1 of d_c (rows x N), row p against row index[p] //
    index_div of a_q and a_s, or row p without an index.  Zeros for an expert without
    rows; a row whose index is outside a_q makes its expert's gradient NaN.  any_scale
    as for fp8gemm_weight_grad."""
    if out_type not in _OUT_DTYPES:
        raise ValueError("unknown out_type %r" % (out_type,))
    d_c = _arg(d_c, "d_c", _FLOATS, dim=2)
    rows, N = d_c.shape
    a_q = _codes_arg(a_q, "a_q", 2, d_c)
    rows_a, K = a_q.shape
    a_s = _arg(a_s, "a_s", (torch.float32,), (rows_a, _blocks(K)), like=d_c)
    offsets = _arg(offsets, "offsets", (torch.int32,), dim=1, like=d_c)
    E = offsets.shape[0] - 1
    if E < 1:
        raise ValueError("offsets must have an entry per expert and one more")
    if index is not None:
        index = _arg(index, "index", (torch.int32,), (rows,), like=d_c)
    elif rows_a < rows:
        raise ValueError("a_q has %d rows, d_c %d" % (rows_a, rows))
    out = _out(out, "out", _OUT_DTYPES[out_type], (E, N, K), d_c, stream)
    workspace = _grad_workspace(rows, N, K, E, d_c.device, stream)
    _call("fp8gemm_weight_grad_grouped", d_c.device, stream, d_c.data_ptr(),
          _DTYPE_IDS[d_c.dtype] + (GRAD_ANY_SCALE if any_scale else 0), rows, N, a_q.data_ptr(), a_s.data_ptr(), rows_a, K,
          E, offsets.data_ptr(), _ptr(index), index_div, out.data_ptr(), out_type, _ptr(workspace))
    return out


# ---- root-mean-square norm with an 8-bit output ----------------------------------


def rmsnorm_quantize(x, weight, residual: torch.Tensor | None = None, quant: int = QUANT_FP8, eps: float = 1e-6,
                     with_y: bool = False, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                     h: torch.Tensor | None = None, y: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                     stream=None):
    """h = x + residual (x without one); y = h / sqrt(mean(h^2) + eps) * weight; codes
    and scales of y: (q, s, h, y, rstd).  x, residual: rows x K of float32, bfloat16
    or float16, weight: K of any of them.  quant: QUANT_INT8 (q int8, s per row),
    QUANT_FP8 / QUANT_FP8_POW2 (q uint8, s rows x KB: fp8gemm_run), QUANT_MXFP8 (q, s
    uint8, s rows x K / 32: mxgemm_run) or QUANT_NONE (q and s are None, y is given).
    y, in x's type, only with_y (or when passed); h may be x or residual; rstd (rows
    float32) is what rmsnorm_backward takes."""
    x = _arg(x, "x", _FLOATS, dim=2)
    rows, K = x.shape
    weight = _arg(weight, "weight", _FLOATS, (K,), like=x)
    if quant not in (QUANT_NONE, QUANT_INT8, QUANT_FP8, QUANT_FP8_POW2, QUANT_MXFP8):
        raise ValueError("unknown quant %r" % (quant,))
    if residual is not None:
        residual = _arg(residual, "residual", (x.dtype,), (rows, K), like=x)
        h = _out(h, "h", x.dtype, (rows, K), x, stream)
    elif h is not None:
        raise ValueError("h is written only with a residual")
    if quant == QUANT_NONE:
        if q is not None or s is not None:
            raise ValueError("q and s are written only with a quant")
    else:
        q = _out(q, "q", torch.int8 if quant == QUANT_INT8 else torch.uint8, (rows, K), x, stream)
        if quant == QUANT_MXFP8:
            s = _out(s, "s", torch.uint8, (rows, K // 32), x, stream)
        else:
            s = _out(s, "s", torch.float32, (rows,) if quant == QUANT_INT8 else (rows, _blocks(K)), x, stream)
    if y is not None or with_y or quant == QUANT_NONE:
        y = _out(y, "y", x.dtype, (rows, K), x, stream)
    rstd = _out(rstd, "rstd", torch.float32, (rows,), x, stream)
    _call("rmsnorm_quantize", x.device, stream, x.data_ptr(), _ptr(residual), _DTYPE_IDS[x.dtype], weight.data_ptr(),
          _DTYPE_IDS[weight.dtype], rows, K, eps, _ptr(h), _ptr(y), quant, _ptr(q), _ptr(s), rstd.data_ptr())
    return q, s, x if h is None else h, y, rstd


def rmsnorm_backward(d_y, h, weight, rstd, d_h: torch.Tensor | None = None, d_x: torch.Tensor | None = None,
                     d_weight: torch.Tensor | None = None, stream=None):
    """Gradients (d_x in h's type, of x and of the residual alike; d_weight K float32)
    of rmsnorm_quantize's y from d_y, with h and rstd as it gave them.  d_h: the
    gradient that h gets besides, added to d_x.  d_x may be d_h.  The rounding
    to codes counts as the identity."""
    h = _arg(h, "h", _FLOATS, dim=2)
    rows, K = h.shape
    d_y = _arg(d_y, "d_y", (h.dtype,), (rows, K), like=h)
    weight = _arg(weight, "weight", _FLOATS, (K,), like=h)
    rstd = _arg(rstd, "rstd", (torch.float32,), (rows,), like=h)
    if d_h is not None:
        d_h = _arg(d_h, "d_h", (h.dtype,), (rows, K), like=h)
    need = (_lib or _load()).rmsnorm_backward_workspace(rows, K)
    if need < 0:
        _check(1, "rmsnorm_backward")
    d_x = _out(d_x, "d_x", h.dtype, (rows, K), h, stream)
    d_weight = _out(d_weight, "d_weight", torch.float32, (K,), h, stream)
    workspace = _new((need,), torch.uint8, h.device, stream) if need else None
    _call("rmsnorm_backward", h.device, stream, d_y.data_ptr(), h.data_ptr(), _ptr(d_h), _DTYPE_IDS[h.dtype],
          weight.data_ptr(), _DTYPE_IDS[weight.dtype], rstd.data_ptr(), rows, K, d_x.data_ptr(), d_weight.data_ptr(),
          _ptr(workspace))
    return d_x, d_weight


def raw_library():
    """The loaded ctypes library (for ABI-level tests)."""
    return _load()
