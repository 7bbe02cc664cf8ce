"""B200 (sm_100a) QLoRA quantized linear layer: NF4 + Double Quantization, dequantization,
and the LoRA-augmented forward/backward through the frozen dequantized weight.

The Python functions below carry the names of the C entry points of libqlora.so
(include/qlora.h).  They only marshal arguments: they allocate outputs with
torch (device memory), pass raw pointers and the current CUDA stream, and check
the returned status.  Every step of the computation runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback.

`stream=` runs a call on another stream than the current one.  What the caller passes
has to be ready for that stream, and what comes back is complete when it is (as for any
work on a stream of one's own: wait_stream before and after).  Workspaces and outputs that
the call allocates belong to that stream; the outputs are also marked as used by the
current one.
"""
from __future__ import annotations

import contextlib
import ctypes
from ctypes import byref, c_float, c_size_t, c_uint32
from dataclasses import dataclass
from functools import lru_cache

import torch

from ._lib import (QLORA_DTYPE_BF16, QLORA_DTYPE_F16, QLORA_DTYPE_F32, TIMER_KINDS, NF4WeightC, QloraError,
                   check, lib)

__all__ = [
    "NF4Weight", "QloraError", "CODEBOOKS", "qlora_nf4_sizes", "qlora_nf4_codebook", "qlora_codebook_values",
    "qlora_quantize_nf4_dq",
    "qlora_quantize_nf4_dq_noalloc",
    "qlora_dequantize", "qlora_quantize_int8_absmax", "qlora_dequantize_int8_absmax", "qlora_merge_lora", "qlora_linear_workspace_size", "qlora_linear_fwd", "qlora_linear_fwd_multi", "qlora_linear_bwd",
    "qlora_adapters_workspace_size", "qlora_linear_fwd_adapters", "qlora_linear_bwd_adapters",
    "qlora_distill_topk_fwd", "qlora_distill_topk_bwd",
    "qlora_read_device_errors", "qlora_selftest_bounded_wait", "qlora_launch_count", "qlora_timing_enable", "qlora_timing_read",
]


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# The caching allocator hands out a block again in the order of the stream that it was allocated on, so memory that
# the kernels on another stream than the current one use has to come from there: another call could have it
# while they still run.  Calls without `stream` use torch.empty itself.
def _on(stream):
    """A context in which torch allocates for `stream`."""
    if stream.cuda_stream == torch.cuda.current_stream().cuda_stream:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream))


def _for_current(t: torch.Tensor, stream) -> torch.Tensor:
    """An output allocated on `stream`, marked as used by the current stream, to which it is returned."""
    current = torch.cuda.current_stream(t.device)
    if stream.cuda_stream != current.cuda_stream:
        t.record_stream(current)
    return t


def _scratch(stream):
    """torch.empty for memory that only the kernels on `stream` use."""
    def empty(*shape, **kw):
        with _on(stream):
            return torch.empty(*shape, **kw)
    return empty


def _outputs(stream):
    """torch.empty for what the kernels on `stream` write and the call returns."""
    def empty(*shape, **kw):
        with _on(stream):
            t = torch.empty(*shape, **kw)
        return _for_current(t, stream)
    return empty


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, dtype, name: str, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _dtype_code(dtype) -> int:
    if dtype == torch.bfloat16:
        return QLORA_DTYPE_BF16
    if dtype == torch.float16:
        return QLORA_DTYPE_F16
    if dtype == torch.float32:
        return QLORA_DTYPE_F32
    raise TypeError("output dtype must be torch.bfloat16, torch.float16 or torch.float32")


@dataclass
class NF4Weight:
    """The stored buffers of a 4-bit quantized weight (device tensors) and its shape.

    With double quantization (the default) the block constants are c1_codes, c2 and mu and
    `c1` is None; without it `c1` holds the fp32 block absmax values and the other three are
    None.  `codebook` is "nf4" or "uniform4" (the uniform 4-bit grid NF4 is compared with)."""
    codes: torch.Tensor                 # uint8 [N*K/2]
    c1_codes: torch.Tensor | None       # uint8 [N*K/64]  (FP8 E4M3 bit patterns)
    c2: torch.Tensor | None             # fp32 [ceil(N*K/64/256)]
    mu: torch.Tensor | None             # fp32 [1]
    N: int
    K: int
    codebook: str = "nf4"
    c1: torch.Tensor | None = None      # fp32 [N*K/64] when double quantization is off
    compute_dtype: torch.dtype = torch.bfloat16   # or torch.float16: W_hat, activations, adapters

    def c_struct(self) -> NF4WeightC:
        p = lambda t: t.data_ptr() if t is not None else None
        return NF4WeightC(self.codes.data_ptr(), p(self.c1_codes), p(self.c2), p(self.mu), self.N, self.K,
                          64, 256, CODEBOOKS[self.codebook], _dtype_code(self.compute_dtype), p(self.c1))

    _BUFFERS = ("codes", "c1_codes", "c2", "mu", "c1")

    def state_dict(self) -> dict:
        """Host copies of the stored buffers plus the shape and settings that give them meaning:
        a checkpoint of the frozen quantized weight (torch.save can write it as is)."""
        d = {"N": self.N, "K": self.K, "codebook": self.codebook, "blocksize": 64, "blocksize2": 256,
             "compute_dtype": str(self.compute_dtype).replace("torch.", "")}
        for name in self._BUFFERS:
            t = getattr(self, name)
            d[name] = None if t is None else t.detach().to("cpu", copy=True)
        return d

    @classmethod
    def from_state_dict(cls, d: dict, device="cuda") -> "NF4Weight":
        """Rebuild a weight from state_dict() output: the buffers are copied to `device` byte for byte
        after their sizes are checked against the shape."""
        N, K = int(d["N"]), int(d["K"])
        if d.get("blocksize", 64) != 64 or d.get("blocksize2", 256) != 256:
            raise ValueError("only blocksize 64 and blocksize2 256 are defined")
        dtype = {"bfloat16": torch.bfloat16, "float16": torch.float16}[d["compute_dtype"]]
        ref = cls.empty(N, K, device, d["codebook"], d.get("c1") is None, dtype)
        for name in cls._BUFFERS:
            t, src = getattr(ref, name), d.get(name)
            if (t is None) != (src is None):
                raise ValueError(f"buffer {name!r} does not match the stored settings")
            if t is not None:
                if src.dtype != t.dtype or src.numel() != t.numel():
                    raise ValueError(f"buffer {name!r}: expected {t.numel()} x {t.dtype}, got "
                                     f"{src.numel()} x {src.dtype}")
                t.copy_(src.reshape(t.shape))
        return ref

    @staticmethod
    def empty(N: int, K: int, device="cuda", codebook: str = "nf4", double_quant: bool = True,
              compute_dtype: torch.dtype = torch.bfloat16) -> "NF4Weight":
        if codebook not in CODEBOOKS:
            raise ValueError(f"codebook must be one of {sorted(CODEBOOKS)}")
        if compute_dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("compute_dtype must be torch.bfloat16 or torch.float16")
        s = qlora_nf4_sizes(N, K)
        codes = torch.empty(s["codes"], dtype=torch.uint8, device=device)
        if not double_quant:
            return NF4Weight(codes, None, None, None, N, K, codebook,
                             torch.empty(s["c1_codes"], dtype=torch.float32, device=device), compute_dtype)
        return NF4Weight(codes,
                         torch.empty(s["c1_codes"], dtype=torch.uint8, device=device),
                         torch.empty(s["c2"] // 4, dtype=torch.float32, device=device),
                         torch.empty(1, dtype=torch.float32, device=device), N, K, codebook, None, compute_dtype)


CODEBOOKS = {"nf4": 0, "uniform4": 1}


def qlora_nf4_sizes(N: int, K: int, blocksize: int = 64, blocksize2: int = 256) -> dict:
    a, b, c, d = c_size_t(), c_size_t(), c_size_t(), c_size_t()
    check(lib().qlora_nf4_sizes(N, K, blocksize, blocksize2, byref(a), byref(b), byref(c), byref(d)),
          "qlora_nf4_sizes")
    return {"codes": a.value, "c1_codes": b.value, "c2": c.value, "workspace": d.value}


def qlora_nf4_codebook():
    """(values[16], thresholds[15]) of the library, as Python float lists."""
    v = (c_float * 16)()
    t = (c_float * 15)()
    check(lib().qlora_nf4_codebook(v, t), "qlora_nf4_codebook")
    return list(v), list(t)


def qlora_codebook_values(codebook: str = "nf4"):
    """(values[16], thresholds[15]) of a codebook ("nf4" or "uniform4")."""
    v = (c_float * 16)()
    t = (c_float * 15)()
    check(lib().qlora_codebook_values(CODEBOOKS[codebook], v, t), "qlora_codebook_values")
    return list(v), list(t)


def qlora_quantize_nf4_dq(W: torch.Tensor, blocksize: int = 64, blocksize2: int = 256,
                          out: NF4Weight | None = None, workspace: torch.Tensor | None = None,
                          stream=None, codebook: str = "nf4", double_quant: bool = True,
                          compute_dtype: torch.dtype = torch.bfloat16) -> NF4Weight:
    """Quantize W (bf16 [N, K]); `codebook`, `double_quant` and `compute_dtype` apply when `out`
    is None (otherwise `out` carries them)."""
    _need(W, torch.bfloat16, "W")
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N, K]")
    N, K = W.shape
    sizes = qlora_nf4_sizes(N, K, blocksize, blocksize2)
    if out is None:
        with _on(stream) if stream is not None else contextlib.nullcontext():
            out = NF4Weight.empty(N, K, W.device, codebook, double_quant, compute_dtype)
        for name in out._BUFFERS if stream is not None else ():
            if getattr(out, name) is not None:
                _for_current(getattr(out, name), stream)
    if workspace is None:
        empty = torch.empty if stream is None else _scratch(stream)
        workspace = empty(sizes["workspace"], dtype=torch.uint8, device=W.device)
    ws = out.c_struct()
    check(lib().qlora_quantize_nf4_dq(_ptr(W), N, K, blocksize, blocksize2, byref(ws), _ptr(workspace),
                                      workspace.numel(), _stream(stream)), "qlora_quantize_nf4_dq")
    return out


def qlora_quantize_nf4_dq_noalloc(W: torch.Tensor, out: NF4Weight, stream=None) -> NF4Weight:
    """Quantize into caller-allocated `out` using the library's static device scratch (no
    workspace, no allocation in the call).  At most 67,108,864 weights; calls that overlap on
    the GPU race on the shared scratch."""
    _need(W, torch.bfloat16, "W")
    N, K = W.shape
    ws = out.c_struct()
    check(lib().qlora_quantize_nf4_dq_noalloc(_ptr(W), N, K, 64, 256, byref(ws), _stream(stream)),
          "qlora_quantize_nf4_dq_noalloc")
    return out


def qlora_dequantize(w: NF4Weight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    empty = torch.empty if stream is None else _outputs(stream)
    if out is None:
        out = empty(w.N, w.K, dtype=w.compute_dtype, device=w.codes.device)
    _need(out, w.compute_dtype, "out", (w.N, w.K))
    ws = w.c_struct()
    check(lib().qlora_dequantize(byref(ws), _ptr(out), _stream(stream)), "qlora_dequantize")
    return out


def qlora_quantize_int8_absmax(W: torch.Tensor, blocksize: int = 64, codes: torch.Tensor | None = None,
                               alpha: torch.Tensor | None = None, stream=None):
    """Blockwise absmax INT8 of a bf16 tensor: alpha = 127 / max|x| per block of
    `blocksize` consecutive elements, codes = round half away from zero of x * alpha.
    Returns (codes int8 shaped like W, alpha fp32 [W.numel() // blocksize])."""
    _need(W, torch.bfloat16, "W")
    n = W.numel()
    empty = torch.empty if stream is None else _outputs(stream)
    if codes is None:
        codes = empty(W.shape, dtype=torch.int8, device=W.device)
    if alpha is None:
        alpha = empty(max(n // blocksize, 1), dtype=torch.float32, device=W.device)
    _need(codes, torch.int8, "codes", tuple(W.shape))
    _need(alpha, torch.float32, "alpha")
    if blocksize <= 0 or alpha.numel() * blocksize != n:
        raise ValueError(f"alpha must hold {n // blocksize} scales")
    check(lib().qlora_quantize_int8_absmax(_ptr(W), n, blocksize, _ptr(codes), _ptr(alpha), _stream(stream)),
          "qlora_quantize_int8_absmax")
    return codes, alpha


def qlora_dequantize_int8_absmax(codes: torch.Tensor, alpha: torch.Tensor, blocksize: int = 64,
                                 dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x_hat = code / alpha per block, rounded to `dtype` (bf16, fp16 or fp32)."""
    _need(codes, torch.int8, "codes")
    _need(alpha, torch.float32, "alpha")
    if blocksize <= 0 or alpha.numel() * blocksize != codes.numel():
        raise ValueError(f"alpha must hold codes.numel() / blocksize = {codes.numel() // max(blocksize, 1)} scales")
    empty = torch.empty if stream is None else _outputs(stream)
    if out is None:
        out = empty(codes.shape, dtype=dtype, device=codes.device)
    _need(out, dtype, "out", tuple(codes.shape))
    check(lib().qlora_dequantize_int8_absmax(_ptr(codes), _ptr(alpha), codes.numel(), blocksize, _ptr(out),
                                             _dtype_code(dtype), _stream(stream)), "qlora_dequantize_int8_absmax")
    return out


def qlora_merge_lora(w: NF4Weight, A: torch.Tensor, B: torch.Tensor, r: int, alpha: float,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """W_merged = bf16(W_hat + (alpha / r) B A) for inference; requantize it with
    qlora_quantize_nf4_dq to serve the merged model in 4 bits."""
    _need(A, w.compute_dtype, "A", (r, w.K))
    _need(B, w.compute_dtype, "B", (w.N, r))
    empty = torch.empty if stream is None else _outputs(stream)
    if out is None:
        out = empty(w.N, w.K, dtype=w.compute_dtype, device=w.codes.device)
    _need(out, w.compute_dtype, "out", (w.N, w.K))
    ws = w.c_struct()
    check(lib().qlora_merge_lora(byref(ws), _ptr(A), _ptr(B), r, float(alpha), _ptr(out), _stream(stream)),
          "qlora_merge_lora")
    return out


def qlora_linear_workspace_size(M: int, N: int, K: int, r: int) -> int:
    n = c_size_t()
    check(lib().qlora_linear_workspace_size(M, N, K, r, byref(n)), "qlora_linear_workspace_size")
    return n.value


def _workspace(M, N, K, r, device, workspace, stream):
    need = qlora_linear_workspace_size(M, N, K, r)
    if workspace is None:
        empty = torch.empty if stream is None else _scratch(stream)
        workspace = empty(max(need, 16), dtype=torch.uint8, device=device)
    return workspace


def qlora_linear_fwd(w: NF4Weight, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, r: int,
                     alpha: float, y_dtype=None, save_U: bool = True,
                     out: torch.Tensor | None = None, U_out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """Y = X W_hat^T + (alpha/r) (X A^T) B^T.  Returns (Y, U) with U fp32 [M,r] (or None).
    X, A, B are in the weight's compute dtype; Y is in it too unless y_dtype is torch.float32."""
    M = X.shape[0]
    y_dtype = w.compute_dtype if y_dtype is None else y_dtype
    _need(X, w.compute_dtype, "X", (M, w.K))
    _need(A, w.compute_dtype, "A", (r, w.K))
    _need(B, w.compute_dtype, "B", (w.N, r))
    empty = torch.empty if stream is None else _outputs(stream)
    if out is None:
        out = empty(M, w.N, dtype=y_dtype, device=X.device)
    _need(out, y_dtype, "Y", (M, w.N))
    if save_U and U_out is None:
        U_out = empty(M, r, dtype=torch.float32, device=X.device)
    if U_out is not None:
        _need(U_out, torch.float32, "U", (M, r))
    workspace = _workspace(M, w.N, w.K, r, X.device, workspace, stream)
    ws = w.c_struct()
    check(lib().qlora_linear_fwd(byref(ws), _ptr(X), M, _ptr(A), _ptr(B), r, c_float(alpha), _ptr(out),
                                 _dtype_code(y_dtype), _ptr(U_out), _ptr(workspace), workspace.numel(),
                                 _stream(stream)), "qlora_linear_fwd")
    return out, U_out


def qlora_linear_fwd_multi(w: NF4Weight, X: torch.Tensor, A_all: torch.Tensor, B_all: torch.Tensor,
                           adapter_idx: torch.Tensor, r: int, alpha: float, y_dtype=None,
                           save_U: bool = False, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None):
    """One base, many adapters (M <= 16 tokens): Y[m] = X[m] W_hat^T + (alpha/r) (X[m] A_a^T) B_a^T
    with a = adapter_idx[m] (-1: base only).  A_all [n, r, K], B_all [n, N, r] bf16; adapter_idx
    int32 [M] on the device.  Returns (Y, U or None)."""
    M = X.shape[0]
    n_ad = A_all.shape[0]
    y_dtype = w.compute_dtype if y_dtype is None else y_dtype
    _need(X, w.compute_dtype, "X", (M, w.K))
    _need(A_all, w.compute_dtype, "A_all", (n_ad, r, w.K))
    _need(B_all, w.compute_dtype, "B_all", (n_ad, w.N, r))
    _need(adapter_idx, torch.int32, "adapter_idx", (M,))
    empty = torch.empty if stream is None else _outputs(stream)
    if out is None:
        out = empty(M, w.N, dtype=y_dtype, device=X.device)
    _need(out, y_dtype, "Y", (M, w.N))
    U = empty(M, r, dtype=torch.float32, device=X.device) if save_U else None
    workspace = _workspace(M, w.N, w.K, r, X.device, workspace, stream)
    ws = w.c_struct()
    check(lib().qlora_linear_fwd_multi(byref(ws), _ptr(X), M, _ptr(A_all), _ptr(B_all), n_ad, _ptr(adapter_idx),
                                       r, c_float(alpha), _ptr(out), _dtype_code(y_dtype), _ptr(U),
                                       _ptr(workspace), workspace.numel(), _stream(stream)),
          "qlora_linear_fwd_multi")
    return out, U


def qlora_linear_bwd(w: NF4Weight, X: torch.Tensor, dY: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                     r: int, alpha: float, U_saved: torch.Tensor | None = None, need_dX: bool = True,
                     dx_dtype=None, dX: torch.Tensor | None = None,
                     dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """(dX, dA, dB) of <dY, Y> through the frozen W_hat.  dX is None when need_dX is False."""
    M = X.shape[0]
    dx_dtype = w.compute_dtype if dx_dtype is None else dx_dtype
    _need(X, w.compute_dtype, "X", (M, w.K))
    _need(dY, w.compute_dtype, "dY", (M, w.N))
    _need(A, w.compute_dtype, "A", (r, w.K))
    _need(B, w.compute_dtype, "B", (w.N, r))
    if U_saved is not None:
        _need(U_saved, torch.float32, "U_saved", (M, r))
    empty = torch.empty if stream is None else _outputs(stream)
    if need_dX and dX is None:
        dX = empty(M, w.K, dtype=dx_dtype, device=X.device)
    if dX is not None:
        _need(dX, dx_dtype, "dX", (M, w.K))
    if dA is None:
        dA = empty(r, w.K, dtype=torch.float32, device=X.device)
    if dB is None:
        dB = empty(w.N, r, dtype=torch.float32, device=X.device)
    _need(dA, torch.float32, "dA", (r, w.K))
    _need(dB, torch.float32, "dB", (w.N, r))
    workspace = _workspace(M, w.N, w.K, r, X.device, workspace, stream)
    ws = w.c_struct()
    check(lib().qlora_linear_bwd(byref(ws), _ptr(X), _ptr(dY), M, _ptr(A), _ptr(B), r, c_float(alpha),
                                 _ptr(U_saved), _ptr(dX), _dtype_code(dx_dtype), _ptr(dA), _ptr(dB),
                                 _ptr(workspace), workspace.numel(), _stream(stream)), "qlora_linear_bwd")
    return dX, dA, dB


# The calls below are short next to a Python function call, so their checks read each attribute once and
# hand ctypes plain integers.
_DTYPE_CODES = {torch.bfloat16: QLORA_DTYPE_BF16, torch.float16: QLORA_DTYPE_F16, torch.float32: QLORA_DTYPE_F32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # the current stream without a Stream object


def _need_on(t: torch.Tensor, dtype, name: str, shape, dev: int) -> int:
    """_need, and on CUDA device `dev`, the current one, where the library launches; returns the address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, dtype, name, shape)
    raise ValueError(f"{name} must be on the current CUDA device cuda:{dev}, got {t.device}")


def _device_of(t: torch.Tensor, name: str) -> int:
    """The CUDA device of t, which has to be the current one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")
    return dev


def _stream_on(stream, dev: int) -> int:
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


@lru_cache(maxsize=256)
def qlora_adapters_workspace_size(M: int, N: int, K: int, r: int, n_adapters: int) -> int:
    n = c_size_t()
    check(lib().qlora_adapters_workspace_size(M, N, K, r, n_adapters, byref(n)), "qlora_adapters_workspace_size")
    return n.value


def _adapter_args(w, X, A_all, B_all, adapter_idx, scales, workspace, dev, stream):
    """Checks of both directions; returns (M, n_adapters, r, addresses in C order, workspace)."""
    if not isinstance(A_all, torch.Tensor):
        raise TypeError("A_all must be a torch.Tensor")
    if A_all.dim() != 3:
        raise ValueError("A_all must be 3-D [n_adapters, r, K]")
    M, (n, r, _), dt = X.shape[0], A_all.shape, w.compute_dtype
    at = (_need_on(X, dt, "X", (M, w.K), dev), _need_on(A_all, dt, "A_all", (n, r, w.K), dev),
          _need_on(B_all, dt, "B_all", (n, w.N, r), dev), _need_on(adapter_idx, torch.int32, "adapter_idx", (M,), dev),
          _need_on(scales, torch.float32, "scales", (n,), dev))
    if w.codes.get_device() != dev:
        raise ValueError(f"the weight must be on the current CUDA device cuda:{dev}, got {w.codes.device}")
    if workspace is None:
        empty = torch.empty if stream is None else _scratch(stream)
        workspace = empty(qlora_adapters_workspace_size(M, w.N, w.K, r, n), dtype=torch.uint8, device=X.device)
    elif not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    elif workspace.get_device() != dev or not workspace.is_contiguous() or workspace.dtype != torch.uint8:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on the current CUDA device cuda:{dev}")
    return M, n, r, at, workspace


def qlora_linear_fwd_adapters(w: NF4Weight, X: torch.Tensor, A_all: torch.Tensor, B_all: torch.Tensor,
                              adapter_idx: torch.Tensor, scales: torch.Tensor, y_dtype=None, save_U: bool = True,
                              out: torch.Tensor | None = None, U_out: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, stream=None):
    """The adapters of many requests over one base, any number of tokens: Y[m] = X[m] W_hat^T +
    s_a (X[m] A_a^T) B_a^T with a = adapter_idx[m] (negative: base only) and s_a = scales[a].
    A_all [n, r, K] and B_all [n, N, r] in the compute dtype (smaller ranks zero-padded to r),
    adapter_idx int32 [M], scales fp32 [n], all on the current device.  Returns (Y, U) with U fp32
    [M, r] (or None)."""
    dev = _device_of(X, "X")
    M, n, r, at, workspace = _adapter_args(w, X, A_all, B_all, adapter_idx, scales, workspace, dev, stream)
    y_dtype = w.compute_dtype if y_dtype is None else y_dtype
    empty = torch.empty if stream is None else _outputs(stream)
    if out is None:
        out = empty((M, w.N), dtype=y_dtype, device=X.device)
    y_at = _need_on(out, y_dtype, "Y", (M, w.N), dev)
    if save_U and U_out is None:
        U_out = empty((M, r), dtype=torch.float32, device=X.device)
    u_at = None if U_out is None else _need_on(U_out, torch.float32, "U", (M, r), dev)
    check(lib().qlora_linear_fwd_adapters(byref(w.c_struct()), at[0], M, at[1], at[2], n, at[3], r, at[4], y_at,
                                          _dtype_code(y_dtype), u_at, workspace.data_ptr(), workspace.numel(),
                                          _stream_on(stream, dev)), "qlora_linear_fwd_adapters")
    return out, U_out


def qlora_linear_bwd_adapters(w: NF4Weight, X: torch.Tensor, dY: torch.Tensor, A_all: torch.Tensor,
                              B_all: torch.Tensor, adapter_idx: torch.Tensor, scales: torch.Tensor,
                              U_saved: torch.Tensor | None = None, need_dX: bool = True, dx_dtype=None,
                              dX: torch.Tensor | None = None, dA: torch.Tensor | None = None,
                              dB: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """(dX, dA_all, dB_all) of <dY, Y> of qlora_linear_fwd_adapters: dA_all fp32 [n, r, K] and dB_all
    fp32 [n, N, r] hold every adapter's gradient over its own tokens.  dX is None when need_dX is False."""
    dev = _device_of(X, "X")
    M, n, r, at, workspace = _adapter_args(w, X, A_all, B_all, adapter_idx, scales, workspace, dev, stream)
    dx_dtype = w.compute_dtype if dx_dtype is None else dx_dtype
    dy_at = _need_on(dY, w.compute_dtype, "dY", (M, w.N), dev)
    u_at = None if U_saved is None else _need_on(U_saved, torch.float32, "U_saved", (M, r), dev)
    empty = torch.empty if stream is None else _outputs(stream)
    if need_dX and dX is None:
        dX = empty((M, w.K), dtype=dx_dtype, device=X.device)
    dx_at = None if dX is None else _need_on(dX, dx_dtype, "dX", (M, w.K), dev)
    if dA is None:
        dA = empty((n, r, w.K), dtype=torch.float32, device=X.device)
    if dB is None:
        dB = empty((n, w.N, r), dtype=torch.float32, device=X.device)
    da_at = _need_on(dA, torch.float32, "dA", (n, r, w.K), dev)
    db_at = _need_on(dB, torch.float32, "dB", (n, w.N, r), dev)
    check(lib().qlora_linear_bwd_adapters(byref(w.c_struct()), at[0], dy_at, M, at[1], at[2], n, at[3], r, at[4], u_at,
                                          dx_at, _dtype_code(dx_dtype), da_at, db_at, workspace.data_ptr(),
                                          workspace.numel(), _stream_on(stream, dev)), "qlora_linear_bwd_adapters")
    return dX, dA, dB


def _rows(t: torch.Tensor, name: str, dev: int, shape=None):
    """A 2-D tensor of a library dtype on CUDA device `dev` whose rows are contiguous; returns (dtype
    code, row stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.bfloat16, torch.float16 or torch.float32, got {t.dtype}")
    size = t.shape
    if len(size) != 2 or (shape is not None and size != shape):
        raise ValueError(f"{name} must be 2-D{'' if shape is None else f' of shape {tuple(shape)}'}, "
                         f"got {tuple(size)}")
    M, V = size
    ld, one = t.stride()
    if M <= 1:
        ld = max(V, 1)
    if t.get_device() != dev or (V > 1 and one != 1) or ld < V:
        raise ValueError(f"{name} must be a tensor on the current CUDA device with contiguous rows")
    return code, ld


def _topk_args(logits, teacher_idx, teacher_logits, dev):
    z_code, ld = _rows(logits, "logits", dev)
    if not isinstance(teacher_idx, torch.Tensor):
        raise TypeError("teacher_idx must be a torch.Tensor")
    if not isinstance(teacher_logits, torch.Tensor):
        raise TypeError("teacher_logits must be a torch.Tensor")
    if teacher_idx.dim() != 2:
        raise ValueError("teacher_idx must be a 2-D tensor [M, k]")
    k = teacher_idx.shape[1]
    shape, t_dtype = (logits.shape[0], k), teacher_logits.dtype
    t_code = _DTYPE_CODES.get(t_dtype)
    if t_code is None:
        raise TypeError(f"teacher_logits must be torch.bfloat16, torch.float16 or torch.float32, got {t_dtype}")
    return (z_code, ld, k, t_code, _need_on(teacher_idx, torch.int32, "teacher_idx", shape, dev),
            _need_on(teacher_logits, t_dtype, "teacher_logits", shape, dev))


def qlora_distill_topk_fwd(logits: torch.Tensor, teacher_idx: torch.Tensor, teacher_logits: torch.Tensor,
                           temperature: float = 1.0, loss: torch.Tensor | None = None,
                           lse: torch.Tensor | None = None, stream=None):
    """Distillation loss of each row from a teacher's top logits: T^2 KL(p || q), p the softmax of the
    row's k teacher logits over T and q the student's over the whole vocabulary.  logits [M, V] (bf16,
    fp16 or fp32, rows contiguous), teacher_idx int32 [M, k] (-1: no entry), teacher_logits [M, k].
    Returns (loss, lse), fp32 [M]; the backward takes lse."""
    dev = _device_of(logits, "logits")
    z_code, ld, k, t_code, i_at, t_at = _topk_args(logits, teacher_idx, teacher_logits, dev)
    M, V = logits.shape
    empty = torch.empty if stream is None else _outputs(stream)
    if loss is None:
        loss = empty(M, dtype=torch.float32, device=logits.device)
    if lse is None:
        lse = empty(M, dtype=torch.float32, device=logits.device)
    check(lib().qlora_distill_topk_fwd(logits.data_ptr(), z_code, ld, M, V, i_at, t_at, t_code, k, temperature,
                                       _need_on(loss, torch.float32, "loss", (M,), dev),
                                       _need_on(lse, torch.float32, "lse", (M,), dev), _stream_on(stream, dev)),
          "qlora_distill_topk_fwd")
    return loss, lse


def qlora_distill_topk_bwd(logits: torch.Tensor, teacher_idx: torch.Tensor, teacher_logits: torch.Tensor,
                           lse: torch.Tensor, dloss: torch.Tensor, temperature: float = 1.0, d_dtype=None,
                           dlogits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """d(sum_m dloss[m] loss[m]) / d logits, in d_dtype (the logits' dtype when None): the dY of the
    output projection's backward.  `dlogits` may be `logits` itself."""
    dev = _device_of(logits, "logits")
    z_code, ld, k, t_code, i_at, t_at = _topk_args(logits, teacher_idx, teacher_logits, dev)
    M, V = logits.shape
    lse_at = _need_on(lse, torch.float32, "lse", (M,), dev)
    dloss_at = _need_on(dloss, torch.float32, "dloss", (M,), dev)
    empty = torch.empty if stream is None else _outputs(stream)
    if dlogits is None:
        dlogits = empty((M, V), dtype=logits.dtype if d_dtype is None else d_dtype, device=logits.device)
    elif d_dtype is not None and dlogits.dtype != d_dtype:
        raise TypeError(f"dlogits must be {d_dtype}, got {dlogits.dtype}")
    d_code, ldd = _rows(dlogits, "dlogits", dev, (M, V))
    check(lib().qlora_distill_topk_bwd(logits.data_ptr(), z_code, ld, M, V, i_at, t_at, t_code, k, temperature,
                                       lse_at, dloss_at, dlogits.data_ptr(), d_code, ldd, _stream_on(stream, dev)),
          "qlora_distill_topk_bwd")
    return dlogits


def qlora_read_device_errors(clear: bool = True, stream=None) -> int:
    """Synchronize and return the device error flags (1: timeout, 2: non-finite weight,
    4: an index out of range)."""
    f = c_uint32()
    lib().qlora_read_device_errors(_stream(stream), 1 if clear else 0, byref(f))
    return f.value


def qlora_selftest_bounded_wait(limit_us: int, device=None, stream=None):
    """Run the bounded-wait self-test (a wait that nothing completes, limited to `limit_us`);
    returns (completed, aborted) as read back from the device.  The timeout device flag is
    left set for qlora_read_device_errors."""
    result = torch.zeros(2, dtype=torch.int32, device=device or torch.device("cuda"))
    check(lib().qlora_selftest_bounded_wait(int(limit_us), _ptr(result), _stream(stream)),
          "qlora_selftest_bounded_wait")
    r = result.cpu().tolist()
    return bool(r[0]), bool(r[1])


def qlora_launch_count() -> int:
    return int(lib().qlora_launch_count())


def qlora_timing_enable(on: bool = True) -> None:
    check(lib().qlora_timing_enable(1 if on else 0), "qlora_timing_enable")


def qlora_timing_read(kind: str, reset: bool = False):
    """(timed units, total device ms) recorded for one kind since the last reset."""
    n = ctypes.c_uint64()
    ms = ctypes.c_double()
    check(lib().qlora_timing_read(TIMER_KINDS[kind], byref(n), byref(ms), 1 if reset else 0),
          "qlora_timing_read")
    return int(n.value), float(ms.value)
