"""Torch-facing binding of the C ABI: tensors in, tensors out.

PyTorch supplies device memory and the current stream; the arithmetic of every
step runs in libqlora_b200.so. Functions mirror the C entry points:

    quantize(W, double_quant)              -> NF4Weight        (nf4_quantize)
    dequantize(w)                          -> bf16 tensor      (nf4_dequantize)
    linear_fwd(w, X, L1, L2, scale)        -> (Y, T)           (qlora_linear_fwd)
    linear_bwd(w, X, dY, L1, L2, scale, T) -> (dX, dL1, dL2)   (qlora_linear_bwd)
    layer_error_rank(Ws, K, double_quant)  -> (err, order, keep) (nf4_layer_error_rank)

Between the linears, 8-bit linears, and linears grouped by expert:

    rms_norm_fwd(x, weight, eps, residual, fp8)       -> (y, h, rstd)   (qlora_rms_norm_fwd)
    rms_norm_bwd(dy, h, rstd, weight, dh)             -> (dx, dw)       (qlora_rms_norm_bwd)
    fp8_quantize_rows(X)                              -> FP8Rows        (fp8_quantize_rows)
    fp8_quantize_weight(W)                            -> FP8Weight      (fp8_quantize_weight)
    fp8_linear_fwd(w, X), fp8_linear_bwd(w, dY)       -> Y, dX          (fp8_linear_fwd, fp8_linear_bwd)
    grouped_linear_fwd(W, X, offsets)                 -> Y              (qlora_grouped_linear_fwd)
    grouped_linear_bwd(W, X, dY, offsets)             -> (dX, dW)       (qlora_grouped_linear_bwd)
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import List, Optional, Sequence, Tuple

import torch

from . import _lib
from ._lib import DTYPE_BF16, DTYPE_F32, NF4QConfig, QLoraWeight, check


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _need(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class Workspace:
    """A grow-only device scratch buffer per (device, stream), zeroed at allocation
    (its first 4 bytes are the library's sticky device status word). Calls on
    different streams get different buffers, so they may run at the same time."""

    _bufs = {}

    @classmethod
    def get(cls, nbytes: int, device: torch.device) -> torch.Tensor:
        dev = torch.device(device)
        idx = dev.index if dev.index is not None else torch.cuda.current_device()
        key = (idx, torch.cuda.current_stream(idx).cuda_stream)
        buf = cls._bufs.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=dev)
            cls._bufs[key] = buf
        return buf

    @classmethod
    def status_word(cls, index: int) -> torch.Tensor:
        """The status word of the calls that need no other workspace, one per device:
        calls on any stream, and captured ones, may share it."""
        buf = cls._bufs.get((index, None))
        if buf is None:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("make one 8-bit or grouped call on this device before capturing one: the first "
                                   "call sets up the device's status word")
            buf = torch.zeros(256, dtype=torch.uint8, device=torch.device("cuda", index))
            torch.cuda.current_stream(index).synchronize()
            buf = cls._bufs.setdefault((index, None), buf)     # (another thread may have been first)
        return buf

    @classmethod
    def all(cls, index: int):
        return [b for (i, _), b in cls._bufs.items() if i == index]


def read_status(ws: torch.Tensor) -> int:
    return _lib.load().qlora_read_status(ctypes.c_void_p(ws.data_ptr()), ctypes.c_void_p(_stream()))


def reset_status(ws: torch.Tensor) -> None:
    """Clears the status word and the tile counters / block flags after it (an
    interrupted GEMM can leave those set)."""
    check(_lib.load().qlora_reset_workspace(ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(),
                                            ctypes.c_void_p(_stream())), "reset_status")


@dataclasses.dataclass
class NF4Weight:
    """An NF4 (or protected bf16) frozen weight stored out x in."""
    out: int
    inp: int
    double_quant: bool
    codes: Optional[torch.Tensor] = None
    absmax: Optional[torch.Tensor] = None
    absmax_q: Optional[torch.Tensor] = None
    absmax2: Optional[torch.Tensor] = None
    w_bf16: Optional[torch.Tensor] = None

    @property
    def is_bf16(self) -> bool:
        return self.w_bf16 is not None

    @staticmethod
    def protected(W: torch.Tensor) -> "NF4Weight":
        _need(W, torch.bfloat16, "W")
        return NF4Weight(W.shape[0], W.shape[1], False, w_bf16=W)

    def c_struct(self) -> QLoraWeight:
        s = QLoraWeight()
        s.out, s.in_ = self.out, self.inp
        s.q = NF4QConfig(64, 1 if self.double_quant else 0, 256)
        s.is_bf16 = 1 if self.is_bf16 else 0
        s.codes = _ptr(self.codes)
        s.absmax = _ptr(self.absmax)
        s.absmax_q = _ptr(self.absmax_q)
        s.absmax2 = _ptr(self.absmax2)
        s.w_bf16 = _ptr(self.w_bf16)
        return s


def quantize(W: torch.Tensor, double_quant: bool = False, keep_absmax: bool = False,
             codes: Optional[torch.Tensor] = None, absmax: Optional[torch.Tensor] = None) -> NF4Weight:
    """NF4-quantize a 2-D bf16 or fp32 CUDA tensor stored out x in. `codes` and
    `absmax` may be given as preallocated outputs (no double quant)."""
    if W.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("W must be bf16 or fp32")
    _need(W, W.dtype, "W")
    lib = _lib.load()
    out, inp = W.shape
    n = W.numel()
    nb = (n + 63) // 64
    dev = W.device
    if codes is None:
        codes = torch.empty((n + 1) // 2, dtype=torch.uint8, device=dev)
    elif codes.numel() < (n + 1) // 2 or codes.dtype != torch.uint8 or not codes.is_contiguous():
        raise ValueError("codes: need a contiguous uint8 tensor of (numel + 1) // 2 bytes")
    if absmax is None:
        absmax = torch.empty(nb, dtype=torch.float32, device=dev) if (not double_quant or keep_absmax) else None
    elif absmax.numel() < nb or absmax.dtype != torch.float32 or not absmax.is_contiguous():
        raise ValueError("absmax: need a contiguous fp32 tensor of one value per 64 weights")
    absmax_q = torch.empty(nb, dtype=torch.uint8, device=dev) if double_quant else None
    absmax2 = torch.empty((nb + 255) // 256, dtype=torch.float32, device=dev) if double_quant else None
    ws = Workspace.get(lib.nf4_quantize_workspace_size(n), dev)
    check(lib.nf4_quantize(_ptr(W), DTYPE_BF16 if W.dtype == torch.bfloat16 else DTYPE_F32, out, inp,
                           NF4QConfig(64, 1 if double_quant else 0, 256), _ptr(codes), _ptr(absmax),
                           _ptr(absmax_q), _ptr(absmax2), _ptr(ws), ws.numel(), _stream()), "nf4_quantize")
    return NF4Weight(out, inp, double_quant, codes=codes, absmax=absmax, absmax_q=absmax_q, absmax2=absmax2)


def quantize_batch(Ws: Sequence[torch.Tensor], double_quant: bool = False, keep_absmax: bool = False,
                   outs: Optional[Sequence[NF4Weight]] = None) -> list:
    """quantize() for up to 512 bf16 matrices in one launch (same bits per matrix).
    `outs` may supply preallocated weights (same shapes and settings)."""
    lib = _lib.load()
    L = len(Ws)
    for i, W in enumerate(Ws):
        _need(W, torch.bfloat16, f"W[{i}]")
    dev = Ws[0].device
    if outs is None:
        outs = []
        for W in Ws:
            n = W.numel()
            nb = (n + 63) // 64
            outs.append(NF4Weight(
                W.shape[0], W.shape[1], double_quant,
                codes=torch.empty((n + 1) // 2, dtype=torch.uint8, device=dev),
                absmax=torch.empty(nb, dtype=torch.float32, device=dev) if (not double_quant or keep_absmax) else None,
                absmax_q=torch.empty(nb, dtype=torch.uint8, device=dev) if double_quant else None,
                absmax2=torch.empty((nb + 255) // 256, dtype=torch.float32, device=dev) if double_quant else None))
    ptrs = (ctypes.c_void_p * L)(*[W.data_ptr() for W in Ws])
    numel = (ctypes.c_int64 * L)(*[W.numel() for W in Ws])

    def arr(name):
        return (ctypes.c_void_p * L)(*[(_ptr(getattr(o, name)) or 0) for o in outs])

    ws = Workspace.get(lib.nf4_quantize_workspace_size(0), dev)
    check(lib.nf4_quantize_batch(L, ptrs, numel, DTYPE_BF16, NF4QConfig(64, 1 if double_quant else 0, 256),
                                 arr("codes"), arr("absmax"), arr("absmax_q"), arr("absmax2"), _ptr(ws), ws.numel(),
                                 _stream()), "nf4_quantize_batch")
    return list(outs)


def dequantize(w: NF4Weight) -> torch.Tensor:
    lib = _lib.load()
    out = torch.empty((w.out, w.inp), dtype=torch.bfloat16, device=w.codes.device)
    cs = w.c_struct()
    check(lib.nf4_dequantize(ctypes.byref(cs), _ptr(out), _stream()), "nf4_dequantize")
    return out


def quantize_residual(W: torch.Tensor, w1: NF4Weight, double_quant: bool = False,
                      keep_absmax: bool = False) -> NF4Weight:
    """Second NF4 stage of W over the first stage w1: quantizes
    R = fp32_rn(W - fp32_rn(c1 a1)) as quantize() would quantize an fp32 tensor."""
    _need(W, torch.bfloat16, "W")
    if tuple(W.shape) != (w1.out, w1.inp):
        raise ValueError("W must have the first stage's shape")
    lib = _lib.load()
    dev = W.device
    n = W.numel()
    nb = (n + 63) // 64
    o = NF4Weight(w1.out, w1.inp, double_quant,
                  codes=torch.empty((n + 1) // 2, dtype=torch.uint8, device=dev),
                  absmax=torch.empty(nb, dtype=torch.float32, device=dev) if (not double_quant or keep_absmax) else None,
                  absmax_q=torch.empty(nb, dtype=torch.uint8, device=dev) if double_quant else None,
                  absmax2=torch.empty((nb + 255) // 256, dtype=torch.float32, device=dev) if double_quant else None)
    ws = Workspace.get(lib.nf4_quantize_residual_workspace_size(n), dev)
    cs = w1.c_struct()
    check(lib.nf4_quantize_residual(_ptr(W), ctypes.byref(cs), NF4QConfig(64, 1 if double_quant else 0, 256),
                                    _ptr(o.codes), _ptr(o.absmax), _ptr(o.absmax_q), _ptr(o.absmax2), _ptr(ws),
                                    ws.numel(), _stream()), "nf4_quantize_residual")
    return o


def dequantize_two_stage(w1: NF4Weight, w2: NF4Weight) -> torch.Tensor:
    """bf16_rn(fp32_rn(v1 + v2)) of two NF4 stages, stored out x in."""
    lib = _lib.load()
    out = torch.empty((w1.out, w1.inp), dtype=torch.bfloat16, device=w1.codes.device)
    c1, c2 = w1.c_struct(), w2.c_struct()
    check(lib.nf4_dequantize_two_stage(ctypes.byref(c1), ctypes.byref(c2), _ptr(out), _stream()),
          "nf4_dequantize_two_stage")
    return out


def lora_merge(w: NF4Weight, L1: torch.Tensor, L2: torch.Tensor, scale: float) -> torch.Tensor:
    """bf16 [out x in] = W_hat + scale (L1 L2)^T (a negative scale unmerges)."""
    _need(L1, torch.bfloat16, "L1")
    _need(L2, torch.bfloat16, "L2")
    lib = _lib.load()
    dev = L1.device
    out = torch.empty((w.out, w.inp), dtype=torch.bfloat16, device=dev)
    cs = w.c_struct()
    check(lib.qlora_lora_merge(ctypes.byref(cs), _ptr(L1), _ptr(L2), L1.shape[1], float(scale), _ptr(out), _stream()),
          "qlora_lora_merge")
    return out


def lora_merge_requantize(w: NF4Weight, L1: torch.Tensor, L2: torch.Tensor, scale: float,
                          double_quant: bool = False, keep_absmax: bool = False) -> NF4Weight:
    """The merged weight W_hat + scale (L1 L2)^T, NF4-quantized as quantize() would."""
    _need(L1, torch.bfloat16, "L1")
    _need(L2, torch.bfloat16, "L2")
    lib = _lib.load()
    dev = L1.device
    n = w.out * w.inp
    nb = (n + 63) // 64
    o = NF4Weight(w.out, w.inp, double_quant,
                  codes=torch.empty((n + 1) // 2, dtype=torch.uint8, device=dev),
                  absmax=torch.empty(nb, dtype=torch.float32, device=dev) if (not double_quant or keep_absmax) else None,
                  absmax_q=torch.empty(nb, dtype=torch.uint8, device=dev) if double_quant else None,
                  absmax2=torch.empty((nb + 255) // 256, dtype=torch.float32, device=dev) if double_quant else None)
    ws = Workspace.get(lib.qlora_lora_merge_requantize_workspace_size(w.out, w.inp), dev)
    cs = w.c_struct()
    check(lib.qlora_lora_merge_requantize(ctypes.byref(cs), _ptr(L1), _ptr(L2), L1.shape[1], float(scale),
                                          NF4QConfig(64, 1 if double_quant else 0, 256), _ptr(o.codes),
                                          _ptr(o.absmax), _ptr(o.absmax_q), _ptr(o.absmax2), _ptr(ws), ws.numel(),
                                          _stream()), "qlora_lora_merge_requantize")
    return o


def linear_fwd(w: NF4Weight, X: torch.Tensor, L1: torch.Tensor, L2: torch.Tensor, scale: float,
               save_T: bool = True, Y: Optional[torch.Tensor] = None,
               T: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Y = X W^T + s (X L1) L2. With T given (from lora_down), X L1 is not
    recomputed and T is returned as is."""
    for t, nm in ((X, "X"), (L1, "L1"), (L2, "L2")):
        _need(t, torch.bfloat16, nm)
    lib = _lib.load()
    M, r = X.shape[0], L1.shape[1]
    dev = X.device
    if Y is None:
        Y = torch.empty((M, w.out), dtype=torch.bfloat16, device=dev)
    ws = Workspace.get(lib.qlora_fwd_workspace_size(M, w.out, w.inp, r), dev)
    cs = w.c_struct()
    if T is not None:
        _need(T, torch.bfloat16, "T")
        check(lib.qlora_linear_fwd_t(ctypes.byref(cs), _ptr(X), M, _ptr(T), _ptr(L2), r, float(scale), _ptr(Y),
                                     _ptr(ws), ws.numel(), _stream()), "qlora_linear_fwd_t")
        return Y, T
    T = torch.empty((M, r), dtype=torch.bfloat16, device=dev) if save_T else None
    check(lib.qlora_linear_fwd(ctypes.byref(cs), _ptr(X), M, _ptr(L1), _ptr(L2), r, float(scale), _ptr(Y), _ptr(T),
                               _ptr(ws), ws.numel(), _stream()), "qlora_linear_fwd")
    return Y, T


def lora_down(X: torch.Tensor, L1: torch.Tensor, T: Optional[torch.Tensor] = None) -> torch.Tensor:
    """T = X L1 (bf16 [M x r]): the LoRA down-projection alone, for overlapping it
    with other work; pass the result to linear_fwd(..., T=T)."""
    _need(X, torch.bfloat16, "X")
    _need(L1, torch.bfloat16, "L1")
    lib = _lib.load()
    M, r = X.shape[0], L1.shape[1]
    dev = X.device
    if T is None:
        T = torch.empty((M, r), dtype=torch.bfloat16, device=dev)
    ws = Workspace.get(lib.qlora_lora_down_workspace_size(M, X.shape[1], r), dev)
    check(lib.qlora_lora_down(_ptr(X), M, X.shape[1], _ptr(L1), r, _ptr(T), _ptr(ws), ws.numel(), _stream()),
          "qlora_lora_down")
    return T


def linear_bwd(w: NF4Weight, X: torch.Tensor, dY: torch.Tensor, L1: torch.Tensor, L2: torch.Tensor, scale: float,
               T: Optional[torch.Tensor] = None, need_dX: bool = True):
    for t, nm in ((X, "X"), (dY, "dY"), (L1, "L1"), (L2, "L2")):
        _need(t, torch.bfloat16, nm)
    lib = _lib.load()
    M, r = X.shape[0], L1.shape[1]
    dev = X.device
    dX = torch.empty((M, w.inp), dtype=torch.bfloat16, device=dev) if need_dX else None
    dL1 = torch.empty((w.inp, r), dtype=torch.float32, device=dev)
    dL2 = torch.empty((r, w.out), dtype=torch.float32, device=dev)
    ws = Workspace.get(lib.qlora_bwd_workspace_size(M, w.out, w.inp, r), dev)
    cs = w.c_struct()
    check(lib.qlora_linear_bwd(ctypes.byref(cs), _ptr(X), _ptr(dY), M, _ptr(L1), _ptr(L2), r, float(scale), _ptr(T),
                               _ptr(dX), _ptr(dL1), _ptr(dL2), _ptr(ws), ws.numel(), _stream()), "qlora_linear_bwd")
    return dX, dL1, dL2


def layer_error_rank(Ws: Sequence[torch.Tensor], K: int, double_quant: bool = False):
    lib = _lib.load()
    L = len(Ws)
    for i, W in enumerate(Ws):
        _need(W, torch.bfloat16, f"W[{i}]")
    dev = Ws[0].device
    ptrs = (ctypes.c_void_p * L)(*[W.data_ptr() for W in Ws])
    numel = (ctypes.c_int64 * L)(*[W.numel() for W in Ws])
    err = torch.empty(L, dtype=torch.float64, device=dev)
    order = torch.empty(L, dtype=torch.int32, device=dev)
    keep = torch.empty(L, dtype=torch.uint8, device=dev)
    ws = Workspace.get(lib.nf4_layer_error_rank_workspace_size(L, numel), dev)
    check(lib.nf4_layer_error_rank(L, ptrs, numel, DTYPE_BF16, NF4QConfig(64, 1 if double_quant else 0, 256), K,
                                   _ptr(err), _ptr(order), _ptr(keep), _ptr(ws), ws.numel(), _stream()),
          "nf4_layer_error_rank")
    return err, order, keep


def layer_error_rank_budget(Ws: Sequence[torch.Tensor], budget_bytes: int, double_quant: bool = False):
    """layer_error_rank with K from a memory budget: the longest prefix of the
    ranking whose bf16 copies add at most budget_bytes to the NF4 storage.
    Returns (err, order, keep, K) with K a one-element device int32 tensor."""
    lib = _lib.load()
    L = len(Ws)
    for i, W in enumerate(Ws):
        _need(W, torch.bfloat16, f"W[{i}]")
    dev = Ws[0].device
    ptrs = (ctypes.c_void_p * L)(*[W.data_ptr() for W in Ws])
    numel = (ctypes.c_int64 * L)(*[W.numel() for W in Ws])
    err = torch.empty(L, dtype=torch.float64, device=dev)
    order = torch.empty(L, dtype=torch.int32, device=dev)
    keep = torch.empty(L, dtype=torch.uint8, device=dev)
    K = torch.empty(1, dtype=torch.int32, device=dev)
    ws = Workspace.get(lib.nf4_layer_error_rank_workspace_size(L, numel), dev)
    check(lib.nf4_layer_error_rank_budget(L, ptrs, numel, DTYPE_BF16, NF4QConfig(64, 1 if double_quant else 0, 256),
                                          int(budget_bytes), _ptr(err), _ptr(order), _ptr(keep), _ptr(K), _ptr(ws),
                                          ws.numel(), _stream()), "nf4_layer_error_rank_budget")
    return err, order, keep, K


def k_from_fraction(num: int, den: int, n_layers: int) -> int:
    """K = round half up of (num / den) * n_layers (host only)."""
    k = ctypes.c_int32(0)
    check(_lib.load().nf4_k_from_fraction(int(num), int(den), int(n_layers), ctypes.byref(k)), "nf4_k_from_fraction")
    return int(k.value)


def quantize_error_rank(Ws: Sequence[torch.Tensor], K: int, double_quant: bool = False, keep_absmax: bool = False,
                        outs: Optional[Sequence[NF4Weight]] = None):
    """The allocation pass fused with the quantization: one read of every matrix
    gives (err, order, keep) as layer_error_rank and every layer's NF4Weight as
    quantize. `outs` may supply preallocated weights (same shapes and settings)."""
    lib = _lib.load()
    L = len(Ws)
    for i, W in enumerate(Ws):
        _need(W, torch.bfloat16, f"W[{i}]")
    dev = Ws[0].device
    if outs is None:
        outs = []
        for W in Ws:
            n = W.numel()
            nb = n // 64
            outs.append(NF4Weight(
                W.shape[0], W.shape[1], double_quant,
                codes=torch.empty(n // 2, dtype=torch.uint8, device=dev),
                absmax=torch.empty(nb, dtype=torch.float32, device=dev) if (not double_quant or keep_absmax) else None,
                absmax_q=torch.empty(nb, dtype=torch.uint8, device=dev) if double_quant else None,
                absmax2=torch.empty((nb + 255) // 256, dtype=torch.float32, device=dev) if double_quant else None))
    ptrs = (ctypes.c_void_p * L)(*[W.data_ptr() for W in Ws])
    numel = (ctypes.c_int64 * L)(*[W.numel() for W in Ws])
    arr = lambda name: (ctypes.c_void_p * L)(*[_ptr(getattr(w, name)) for w in outs])
    err = torch.empty(L, dtype=torch.float64, device=dev)
    order = torch.empty(L, dtype=torch.int32, device=dev)
    keep = torch.empty(L, dtype=torch.uint8, device=dev)
    ws = Workspace.get(lib.nf4_layer_error_rank_workspace_size(L, numel), dev)
    check(lib.nf4_quantize_error_rank(L, ptrs, numel, DTYPE_BF16, NF4QConfig(64, 1 if double_quant else 0, 256), K,
                                      arr("codes"), arr("absmax"), arr("absmax_q"), arr("absmax2"),
                                      _ptr(err), _ptr(order), _ptr(keep), _ptr(ws), ws.numel(), _stream()),
          "nf4_quantize_error_rank")
    return err, order, keep, list(outs)


def rank_errors(err: torch.Tensor, K: int):
    """(order, keep) of per-layer errors already on the device (fp64): the ranking
    step alone, (error desc, index asc), NaN first."""
    _need(err, torch.float64, "err")
    lib = _lib.load()
    L = err.numel()
    order = torch.empty(L, dtype=torch.int32, device=err.device)
    keep = torch.empty(L, dtype=torch.uint8, device=err.device)
    check(lib.nf4_rank_errors(L, _ptr(err), int(K), _ptr(order), _ptr(keep), _stream()), "nf4_rank_errors")
    return order, keep


# ------------------------------------------------------------------ norm, 8-bit and grouped linears

_F8, _BF16, _F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _blocks(n: int) -> int:
    return (n + 127) >> 7


def _check(t: torch.Tensor, dtype, shape: Optional[tuple], name: str, device: Optional[int] = None):
    """t is a contiguous CUDA tensor of this dtype, shape (None: any 2-D one) and device."""
    if not (t.is_cuda and t.dtype is dtype and t.is_contiguous() and
            (t.dim() == 2 if shape is None else t.shape == shape)):
        _need(t, dtype, name)
        raise ValueError(f"{name} must be 2-D" if shape is None else
                         f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"every tensor of a call must be on one device: {name} is on cuda:{t.get_device()}, "
                         f"not cuda:{device}")


def _check_weight_vector(w: torch.Tensor, H: int, device: int) -> int:
    if w.dtype is _BF16:
        _check(w, _BF16, (H,), "weight", device)
        return DTYPE_BF16
    if w.dtype is not _F32:
        raise ValueError("weight must be bf16 or fp32")
    _check(w, _F32, (H,), "weight", device)
    return DTYPE_F32


@dataclasses.dataclass(frozen=True)
class FP8Rows:
    """Rows in e4m3: codes float8_e4m3fn [M, in], scale fp32 [M, ceil(in / 128)]; a value
    is its code times its block's scale. Checked once, when made."""
    codes: torch.Tensor
    scale: torch.Tensor

    def __post_init__(self):
        _check(self.codes, _F8, None, "codes")
        M, n = self.codes.shape
        _check(self.scale, _F32, (M, _blocks(n)), "scale", self.codes.get_device())


@dataclasses.dataclass(frozen=True)
class FP8Weight:
    """A frozen weight in e4m3, stored out x in: codes float8_e4m3fn [out, in], or
    [experts, out, in], with a scale for each 128 x 128 block, fp32
    [(experts,) ceil(out / 128), ceil(in / 128)]. Checked once, when made."""
    codes: torch.Tensor
    scale: torch.Tensor

    def __post_init__(self):
        shape = self.codes.shape
        if len(shape) not in (2, 3):
            raise ValueError("codes must be [out, in] or [experts, out, in]")
        _check(self.codes, _F8, shape, "codes")
        _check(self.scale, _F32, (*shape[:-2], _blocks(shape[-2]), _blocks(shape[-1])), "scale",
               self.codes.get_device())

    @property
    def out(self) -> int:
        return self.codes.shape[-2]

    @property
    def inp(self) -> int:
        return self.codes.shape[-1]


def _new_rows(M: int, n: int, device) -> FP8Rows:
    r = object.__new__(FP8Rows)
    r.__dict__.update(codes=torch.empty(M, n, dtype=_F8, device=device),
                      scale=torch.empty(M, _blocks(n), dtype=_F32, device=device))
    return r


def _status_ptr(device: int) -> int:
    buf = Workspace._bufs.get((device, None))
    return (Workspace.status_word(device) if buf is None else buf).data_ptr()


def _expert_weight(W, device: int) -> Tuple[_lib.ExpertWeight, int, int, int]:
    """(descriptor, experts, out, in) of an FP8Weight or a bf16 tensor [(experts,) out, in]."""
    if isinstance(W, FP8Weight):
        t = W.codes
        if t.get_device() != device:
            raise ValueError(f"every tensor of a call must be on one device: the weight is on {t.device}, "
                             f"not cuda:{device}")
        shape = t.shape
        E, o, i = shape if len(shape) == 3 else (1, *shape)
        return _lib.ExpertWeight(E, o, i, 0, t.data_ptr(), W.scale.data_ptr(), None), E, o, i
    t, shape = W, W.shape
    _check(t, _BF16, shape, "W", device)
    E, o, i = shape if len(shape) == 3 else (1, *shape)
    return _lib.ExpertWeight(E, o, i, 1, None, None, t.data_ptr()), E, o, i


def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                 fp8: bool = False):
    """(y, h, rstd): h = bf16(x + residual) (x itself without a residual), rstd = 1 /
    sqrt(mean(h^2) + eps) per row, y = h rstd weight. y is bf16, or FP8Rows with fp8=True
    (quantized from the fp32 value). x: bf16 [M, H] with H % 8 == 0; weight: bf16 or fp32 [H]."""
    _check(x, _BF16, None, "x")
    dev = x.get_device()
    if _device() != dev:
        with torch.cuda.device(dev):
            return rms_norm_fwd(x, weight, eps, residual, fp8)
    M, H = x.shape
    wt = _check_weight_vector(weight, H, dev)
    if residual is None:
        h, rp, hp = x, None, None
    else:
        _check(residual, _BF16, x.shape, "residual", dev)
        h = torch.empty_like(x)
        rp, hp = residual.data_ptr(), h.data_ptr()
    rstd = torch.empty(M, dtype=_F32, device=x.device)
    if fp8:
        y = _new_rows(M, H, x.device)
        yp, qp, sp = None, y.codes.data_ptr(), y.scale.data_ptr()
    else:
        y = torch.empty_like(x)
        yp, qp, sp = y.data_ptr(), None, None
    check(_lib.load().qlora_rms_norm_fwd(x.data_ptr(), rp, weight.data_ptr(), wt, M, H, eps, hp, yp, qp, sp,
                                         rstd.data_ptr(), _raw_stream(dev)), "qlora_rms_norm_fwd")
    return y, h, rstd


def rms_norm_bwd(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                 dh: Optional[torch.Tensor] = None, need_dw: bool = True):
    """(dx, dw) from the gradient of y and, with dh, the one that reaches h itself: dx (bf16) is
    the gradient of x and of the residual alike, dw (fp32 [H]; None with need_dw=False) the
    weight's. h and rstd are rms_norm_fwd's. An 8-bit y counts as not rounded."""
    _check(dy, _BF16, None, "dy")
    dev = dy.get_device()
    if _device() != dev:
        with torch.cuda.device(dev):
            return rms_norm_bwd(dy, h, rstd, weight, dh, need_dw)
    M, H = dy.shape
    _check(h, _BF16, dy.shape, "h", dev)
    if dh is not None:
        _check(dh, _BF16, dy.shape, "dh", dev)
    _check(rstd, _F32, (M,), "rstd", dev)
    wt = _check_weight_vector(weight, H, dev)
    lib = _lib.load()
    dx = torch.empty_like(dy)
    dw, ws, nbytes = None, None, 0
    if need_dw:
        dw = torch.empty(H, dtype=_F32, device=dy.device)
        nbytes = lib.qlora_rms_norm_bwd_workspace_size(M, H)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device)   # this call's alone
    check(lib.qlora_rms_norm_bwd(dy.data_ptr(), _ptr(dh), h.data_ptr(), rstd.data_ptr(), weight.data_ptr(), wt, M, H,
                                 dx.data_ptr(), _ptr(dw), _ptr(ws), nbytes, _raw_stream(dev)), "qlora_rms_norm_bwd")
    return dx, dw


def fp8_quantize_rows(X: torch.Tensor) -> FP8Rows:
    """e4m3 codes of bf16 rows [M, in] with a scale for each 128 values (in % 16 == 0)."""
    _check(X, _BF16, None, "X")
    dev = X.get_device()
    if _device() != dev:
        with torch.cuda.device(dev):
            return fp8_quantize_rows(X)
    M, inp = X.shape
    q = _new_rows(M, inp, X.device)
    check(_lib.load().fp8_quantize_rows(X.data_ptr(), M, inp, q.codes.data_ptr(), q.scale.data_ptr(),
                                        _raw_stream(dev)), "fp8_quantize_rows")
    return q


def fp8_quantize_weight(W: torch.Tensor) -> FP8Weight:
    """e4m3 codes of a bf16 or fp32 weight [out, in] or [experts, out, in] with a scale for each
    128 x 128 block. A non-finite weight is reported by status()."""
    if W.dtype not in (_BF16, _F32):
        raise ValueError("W must be bf16 or fp32")
    _need(W, W.dtype, "W")
    if W.dim() not in (2, 3):
        raise ValueError("W must be [out, in] or [experts, out, in]")
    dev = W.get_device()
    if _device() != dev:
        with torch.cuda.device(dev):
            return fp8_quantize_weight(W)
    o, i = W.shape[-2:]
    ws = Workspace.status_word(dev)
    codes = torch.empty(W.shape, dtype=_F8, device=W.device)
    scale = torch.empty((*W.shape[:-2], _blocks(o), _blocks(i)), dtype=_F32, device=W.device)
    check(_lib.load().fp8_quantize_weight(W.data_ptr(), DTYPE_BF16 if W.dtype is _BF16 else DTYPE_F32,
                                          W.shape[0] if W.dim() == 3 else 1, o, i, codes.data_ptr(), scale.data_ptr(),
                                          ws.data_ptr(), ws.numel(), _raw_stream(dev)), "fp8_quantize_weight")
    return FP8Weight(codes, scale)


def _rows_of(rows, eight_bit: bool, cols: int, name: str):
    """(tensor, scale or None, device) of a product's rows: FP8Rows, or bf16, which is quantized
    where the weight is 8 bit."""
    if isinstance(rows, FP8Rows):
        if not eight_bit:
            raise ValueError(f"{name}: FP8Rows need an FP8Weight")
        t, sc = rows.codes, rows.scale
        dev = t.get_device()
    else:
        _check(rows, _BF16, None, name)
        t, sc, dev = rows, None, rows.get_device()
    if t.shape[1] != cols:
        raise ValueError(f"{name} must have {cols} columns, got {t.shape[1]}")
    return t, sc, dev


def _output(t: Optional[torch.Tensor], shape: tuple, dtype, dev: int, name: str, *inputs) -> torch.Tensor:
    """A new output, or the caller's, which may not share memory with an input (the first one has the
    device)."""
    if t is None:
        return torch.empty(*shape, dtype=dtype, device=inputs[0].device)
    _check(t, dtype, shape, name, dev)
    a, b = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
    for i in inputs:
        if i is not None and i.data_ptr() < b and a < i.data_ptr() + i.numel() * i.element_size():
            raise ValueError(f"{name} may not overlap an input of the call")
    return t


def _sides(W) -> Tuple[int, int]:
    """(out, in) of an FP8Weight or a bf16 tensor [(experts,) out, in]."""
    if isinstance(W, FP8Weight):
        return W.out, W.inp
    if W.dim() not in (2, 3):
        raise ValueError("W must be [out, in] or [experts, out, in]")
    return W.shape[-2:]


def _parts(W) -> tuple:
    return (W.codes, W.scale) if isinstance(W, FP8Weight) else (W,)


def fp8_linear_fwd(w: FP8Weight, X, Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = X W^T (bf16 [M, out]) with e4m3 weight and rows. X: FP8Rows, or bf16 [M, in], which is
    quantized first."""
    if not isinstance(w, FP8Weight) or w.codes.dim() != 2:
        raise ValueError("w must be an FP8Weight [out, in]")
    x, sx, dev = _rows_of(X, True, w.inp, "X")
    if _device() != dev:
        with torch.cuda.device(dev):
            return fp8_linear_fwd(w, X, Y)
    cs = _expert_weight(w, dev)[0]
    lib = _lib.load()
    M = x.shape[0]
    if sx is None and M > _FP8_BF16_ROWS:
        q = fp8_quantize_rows(x)
        x, sx = q.codes, q.scale
    ws = _status_ptr(dev)
    Y = _output(Y, (M, w.out), _BF16, dev, "Y", x, sx, w.codes, w.scale)
    check(lib.fp8_linear_fwd(ctypes.byref(cs), x.data_ptr(), _ptr(sx), M, Y.data_ptr(), ws, 256,
                             _raw_stream(dev)), "fp8_linear_fwd")
    return Y


# Rows up to which fp8_linear_fwd takes bf16 and quantizes within its kernel (fp8_linear_bf16_rows()).
_FP8_BF16_ROWS = 2


def fp8_linear_bwd(w: FP8Weight, dY, dX: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX = dY W (bf16 [M, in]), the gradient through the frozen weight. dY: FP8Rows, or bf16
    [M, out], which is quantized first."""
    if not isinstance(w, FP8Weight) or w.codes.dim() != 2:
        raise ValueError("w must be an FP8Weight [out, in]")
    d, sd, dev = _rows_of(dY, True, w.out, "dY")
    if _device() != dev:
        with torch.cuda.device(dev):
            return fp8_linear_bwd(w, dY, dX)
    cs = _expert_weight(w, dev)[0]
    if sd is None:
        q = fp8_quantize_rows(d)
        d, sd = q.codes, q.scale
    ws = _status_ptr(dev)
    dX = _output(dX, (d.shape[0], w.inp), _BF16, dev, "dX", d, sd, w.codes, w.scale)
    check(_lib.load().fp8_linear_bwd(ctypes.byref(cs), d.data_ptr(), sd.data_ptr(), d.shape[0], dX.data_ptr(),
                                     ws, 256, _raw_stream(dev)), "fp8_linear_bwd")
    return dX


def grouped_linear_fwd(W, X, offsets: torch.Tensor, Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y (bf16 [M, out]): rows offsets[e]:offsets[e + 1] of X go through expert e, Y_e = X_e W_e^T.
    W: bf16 [experts, out, in] with bf16 X [M, in], or an FP8Weight with FP8Rows (bf16 X is
    quantized first). offsets: int32 [experts + 1] on the device, ascending within 0 .. M; rows
    outside every group are not written (pass Y to keep what is in them)."""
    eight = isinstance(W, FP8Weight)
    x, sx, dev = _rows_of(X, eight, _sides(W)[1], "X")
    if _device() != dev:
        with torch.cuda.device(dev):
            return grouped_linear_fwd(W, X, offsets, Y)
    cs, E, o, _ = _expert_weight(W, dev)
    _check(offsets, torch.int32, (E + 1,), "offsets", dev)
    if eight and sx is None:
        q = fp8_quantize_rows(x)
        x, sx = q.codes, q.scale
    ws = _status_ptr(dev)
    Y = _output(Y, (x.shape[0], o), _BF16, dev, "Y", x, sx, *_parts(W), offsets)
    check(_lib.load().qlora_grouped_linear_fwd(ctypes.byref(cs), x.data_ptr(), _ptr(sx), x.shape[0],
                                               offsets.data_ptr(), Y.data_ptr(), ws, 256,
                                               _raw_stream(dev)), "qlora_grouped_linear_fwd")
    return Y


def grouped_linear_bwd(W, X: Optional[torch.Tensor], dY, offsets: torch.Tensor, need_dX: bool = True,
                       need_dW: bool = True, dX: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None):
    """(dX, dW) of grouped_linear_fwd: dX_e = dY_e W_e (bf16 [M, in]; rows outside every group are
    not written) and dW_e = dY_e^T X_e (fp32 [experts, out, in], zero for an expert without rows;
    bf16 weights only: an FP8Weight is frozen, pass need_dW=False). X may be None without dW."""
    eight = isinstance(W, FP8Weight)
    if not need_dX and not need_dW:
        raise ValueError("need_dX or need_dW must be true")
    if need_dW and eight:
        raise ValueError("an FP8Weight is frozen: pass need_dW=False")
    d, sd, dev = _rows_of(dY, eight, _sides(W)[0], "dY")
    if _device() != dev:
        with torch.cuda.device(dev):
            return grouped_linear_bwd(W, X, dY, offsets, need_dX, need_dW, dX, dW)
    cs, E, o, i = _expert_weight(W, dev)
    _check(offsets, torch.int32, (E + 1,), "offsets", dev)
    M = d.shape[0]
    xp = None
    if need_dW:
        if X is None:
            raise ValueError("X is needed for dW")
        _check(X, _BF16, (M, i), "X", dev)
        xp = X.data_ptr()
    if eight and sd is None:
        q = fp8_quantize_rows(d)
        d, sd = q.codes, q.scale
    ws = _status_ptr(dev)
    dX = _output(dX, (M, i), _BF16, dev, "dX", d, sd, *_parts(W), offsets, X if need_dW else None) if need_dX else None
    dW = _output(dW, (E, o, i), _F32, dev, "dW", d, X, *_parts(W), offsets, dX) if need_dW else None
    check(_lib.load().qlora_grouped_linear_bwd(ctypes.byref(cs), xp, d.data_ptr(), _ptr(sd), M, offsets.data_ptr(),
                                               _ptr(dX), _ptr(dW), ws, 256, _raw_stream(dev)),
          "qlora_grouped_linear_bwd")
    return dX, dW


def status() -> int:
    """First nonzero device status word among this device's workspaces (one per
    stream the library was called on, and one for the calls that share it);
    synchronizes."""
    idx = torch.cuda.current_device()
    dev = torch.device("cuda", idx)
    if (idx, None) in Workspace._bufs:
        torch.cuda.synchronize(idx)      # that word is every stream's
    for ws in Workspace.all(idx) or [Workspace.get(256, dev)]:
        st = read_status(ws)
        if st:
            return st
    return 0
