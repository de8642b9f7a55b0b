"""B200 (sm_100a) frozen-base NF4 + double-quant LoRA linear layer.

A thin Python binding over the C ABI of libqlora_nf4.so (include/qlora_nf4.h).
The functions below carry the C names and only marshal torch tensors to raw
device pointers and sizes; every step of the computation runs in the
library's CUDA kernels.  If the library is missing, importing the binding
functions raises: there is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _capi

__all__ = ["NF4Weight", "QLORA_QT_NF4", "QLORA_QT_FP4", "QLORA_FMT_BLOCK128", "QLORA_FMT_NO_DQ",
           "QLORA_FMT_CODES_AFTER_DQ", "qlora_packed_bytes", "qlora_packed_bytes_fmt", "qlora_nf4_codebook",
           "qlora_codebook",
           "qlora_quantize_nf4_dq", "qlora_dequant",
           "qlora_lora_merge_requant",
           "qlora_workspace_bytes", "qlora_lora_linear_fwd", "qlora_lora_linear_fwd_static_ws",
           "qlora_lora_linear_bwd_dx", "qlora_lora_grad_AB",
           "qlora_sync_status", "qlora_set_wait_limit_ns", "qlora_probe_wait_timeout", "Q80Weight",
           "qlora_q8_0_packed_bytes", "qlora_quantize_q8_0", "qlora_dequant_q8_0", "qlora_q8_0_lora_linear_fwd",
           "qlora_q8_0_lora_linear_bwd_dx",
           "qlora_embed_fwd", "qlora_embed_nf4_fwd", "qlora_embed_q8_0_fwd", "qlora_embed_grad_workspace_bytes",
           "qlora_embed_grad", "AdamWTensor", "AdamWPlan", "qlora_adamw_plan_init", "qlora_adamw_step",
           "qlora_grad_norm", "qlora_adam8_encode", "qlora_adam8_decode", "QloraError"]

QloraError = _capi.QloraError


def _lib():
    return _capi.load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    # the raw handle of the current stream: building a torch.cuda.Stream object takes longer than a small kernel
    raw = torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) if stream is None else stream.cuda_stream
    return ctypes.c_void_p(raw)


def _need(t, dtype, shape, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected contiguous cuda {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


QLORA_QT_NF4, QLORA_QT_FP4 = _capi.QT_NF4, _capi.QT_FP4
QLORA_FMT_BLOCK128, QLORA_FMT_NO_DQ, QLORA_FMT_CODES_AFTER_DQ = (_capi.FMT_BLOCK128, _capi.FMT_NO_DQ,
                                                                 _capi.FMT_CODES_AFTER_DQ)


@dataclass
class NF4Weight:
    """Packed 4-bit weight: device buffers owned by this object (codes, first-level scales,
    second-level steps), the quant type whose 16 levels the codes index (NF4 by default, or
    FP4) and the storage format of the scales (QLORA_FMT_* flags, 0 = blocks of 64 with
    double quantization).  Without double quantization `scales` holds float32 absmaxes and
    `scales2` is an empty tensor."""
    n_out: int
    n_in: int
    codes: torch.Tensor
    scales: torch.Tensor
    scales2: torch.Tensor
    quant_type: int = QLORA_QT_NF4
    format: int = 0

    @classmethod
    def empty(cls, n_out: int, n_in: int, device="cuda", quant_type: int = QLORA_QT_NF4,
              format: int = 0) -> "NF4Weight":
        numel = n_out * n_in
        nb = numel // (128 if format & QLORA_FMT_BLOCK128 else 64)
        if format & QLORA_FMT_NO_DQ:
            scales = torch.empty(nb, dtype=torch.float32, device=device)
            scales2 = torch.empty(0, dtype=torch.float32, device=device)
        else:
            scales = torch.empty(nb, dtype=torch.uint8, device=device)
            scales2 = torch.empty((nb + 255) // 256, dtype=torch.float32, device=device)
        return cls(n_out, n_in, torch.empty(numel // 2, dtype=torch.uint8, device=device), scales, scales2,
                   int(quant_type), int(format))

    def c_struct(self) -> _capi.Nf4WeightC:
        s2 = self.scales2.data_ptr() if self.scales2.numel() else None
        return _capi.Nf4WeightC(self.n_out, self.n_in, self.codes.data_ptr(), self.scales.data_ptr(), s2,
                                int(self.quant_type), int(self.format))


def qlora_packed_bytes(numel: int) -> int:
    return int(_lib().qlora_packed_bytes(int(numel)))


def qlora_packed_bytes_fmt(numel: int, format: int) -> int:
    return int(_lib().qlora_packed_bytes_fmt(int(numel), int(format)))


def qlora_nf4_codebook() -> list[float]:
    buf = (ctypes.c_float * 16)()
    _capi.check("qlora_nf4_codebook", _lib().qlora_nf4_codebook(buf))
    return list(buf)


def qlora_codebook(quant_type: int) -> list[float]:
    buf = (ctypes.c_float * 16)()
    _capi.check("qlora_codebook", _lib().qlora_codebook(int(quant_type), buf))
    return list(buf)


def qlora_quantize_nf4_dq(W: torch.Tensor, weight: NF4Weight, stream=None) -> None:
    _need(W, torch.float32, (weight.n_out, weight.n_in), "W")
    s = weight.c_struct()
    _capi.check("qlora_quantize_nf4_dq", _lib().qlora_quantize_nf4_dq(_ptr(W), ctypes.byref(s), _stream(stream)))


def qlora_dequant(weight: NF4Weight, out: torch.Tensor, stream=None) -> None:
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out must be float32 or bfloat16")
    _need(out, out.dtype, (weight.n_out, weight.n_in), "out")
    s = weight.c_struct()
    _capi.check("qlora_dequant", _lib().qlora_dequant(ctypes.byref(s), _ptr(out), int(out.dtype == torch.bfloat16),
                                                      _stream(stream)))


def qlora_lora_merge_requant(weight: NF4Weight, A, B, r: int, scaling: float, W_scratch: torch.Tensor,
                             out: NF4Weight, stream=None) -> None:
    """Merge the adapter into the base and quantize again into `out` (may be `weight`);
    W_scratch is a float32 [n_out, n_in] device tensor that receives the merged base."""
    _need(W_scratch, torch.float32, (weight.n_out, weight.n_in), "W_scratch")
    if (out.n_out, out.n_in) != (weight.n_out, weight.n_in):
        raise ValueError("out must have the shape of weight")
    if r:
        _need(A, torch.bfloat16, (r, weight.n_in), "A")
        _need(B, torch.bfloat16, (weight.n_out, r), "B")
    s_in, s_out = weight.c_struct(), out.c_struct()
    _capi.check("qlora_lora_merge_requant",
                _lib().qlora_lora_merge_requant(ctypes.byref(s_in), _ptr(A) if r else None, _ptr(B) if r else None,
                                                int(r), float(scaling), _ptr(W_scratch), ctypes.byref(s_out),
                                                _stream(stream)))


def qlora_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return int(_lib().qlora_workspace_bytes(int(M), int(N), int(K), int(r)))


def qlora_lora_linear_fwd(weight: NF4Weight, X, A, B, r: int, scaling: float, Y, U_save=None, ws=None,
                          stream=None) -> None:
    M = X.shape[0]
    _need(X, torch.bfloat16, (M, weight.n_in), "X")
    _need(Y, torch.bfloat16, (M, weight.n_out), "Y")
    if r:
        _need(A, torch.bfloat16, (r, weight.n_in), "A")
        _need(B, torch.bfloat16, (weight.n_out, r), "B")
    if U_save is not None:
        _need(U_save, torch.bfloat16, (M, r), "U_save")
    s = weight.c_struct()
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _capi.check("qlora_lora_linear_fwd", _lib().qlora_lora_linear_fwd(
        ctypes.byref(s), _ptr(X), M, _ptr(A), _ptr(B), int(r), float(scaling), _ptr(Y), _ptr(U_save), _ptr(ws),
        wsb, _stream(stream)))


def qlora_lora_linear_fwd_static_ws(weight: NF4Weight, X, A, B, r: int, scaling: float, Y, U_save=None,
                                    stream=None) -> None:
    """qlora_lora_linear_fwd with the library's static device scratch (no workspace argument)."""
    M = X.shape[0]
    _need(X, torch.bfloat16, (M, weight.n_in), "X")
    _need(Y, torch.bfloat16, (M, weight.n_out), "Y")
    if r:
        _need(A, torch.bfloat16, (r, weight.n_in), "A")
        _need(B, torch.bfloat16, (weight.n_out, r), "B")
    if U_save is not None:
        _need(U_save, torch.bfloat16, (M, r), "U_save")
    s = weight.c_struct()
    _capi.check("qlora_lora_linear_fwd_static_ws", _lib().qlora_lora_linear_fwd_static_ws(
        ctypes.byref(s), _ptr(X), M, _ptr(A), _ptr(B), int(r), float(scaling), _ptr(Y), _ptr(U_save),
        _stream(stream)))


def qlora_lora_linear_bwd_dx(weight: NF4Weight, dY, A, B, r: int, scaling: float, dX, G_save=None, ws=None,
                             stream=None) -> None:
    M = dY.shape[0]
    _need(dY, torch.bfloat16, (M, weight.n_out), "dY")
    _need(dX, torch.bfloat16, (M, weight.n_in), "dX")
    if r:
        _need(A, torch.bfloat16, (r, weight.n_in), "A")
        _need(B, torch.bfloat16, (weight.n_out, r), "B")
    if G_save is not None:
        _need(G_save, torch.bfloat16, (M, r), "G_save")
    s = weight.c_struct()
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _capi.check("qlora_lora_linear_bwd_dx", _lib().qlora_lora_linear_bwd_dx(
        ctypes.byref(s), _ptr(dY), M, _ptr(A), _ptr(B), int(r), float(scaling), _ptr(dX), _ptr(G_save), _ptr(ws),
        wsb, _stream(stream)))


def qlora_lora_grad_AB(X, dY, U, G, r: int, scaling: float, dA, dB, accumulate: bool = False,
                       stream=None) -> None:
    M, K = X.shape
    N = dY.shape[1]
    _need(X, torch.bfloat16, (M, K), "X")
    _need(dY, torch.bfloat16, (M, N), "dY")
    _need(U, torch.bfloat16, (M, r), "U")
    _need(G, torch.bfloat16, (M, r), "G")
    _need(dA, torch.float32, (r, K), "dA")
    _need(dB, torch.float32, (N, r), "dB")
    _capi.check("qlora_lora_grad_AB", _lib().qlora_lora_grad_AB(
        _ptr(X), _ptr(dY), _ptr(U), _ptr(G), M, N, K, int(r), float(scaling), _ptr(dA), _ptr(dB),
        int(bool(accumulate)), _stream(stream)))


def qlora_sync_status(stream=None) -> None:
    _capi.check("qlora_sync_status", _lib().qlora_sync_status(_stream(stream)))


def qlora_set_wait_limit_ns(ns: int) -> None:
    """Time after which a kernel pipeline wait gives up on the current device (default 2e9 ns)."""
    _capi.check("qlora_set_wait_limit_ns", _lib().qlora_set_wait_limit_ns(int(ns)))


def qlora_probe_wait_timeout(stream=None) -> None:
    """Enqueue the self-test kernel whose wait runs out; the next sync reports QLORA_ERR_TIMEOUT."""
    _capi.check("qlora_probe_wait_timeout", _lib().qlora_probe_wait_timeout(_stream(stream)))


# ----------------------------------------------------------------------------- Q8_0 route

@dataclass
class Q80Weight:
    """Q8_0 weight: int8 codes [n_out, n_in] and an fp16 scale per 32 weights (device)."""
    n_out: int
    n_in: int
    q: torch.Tensor
    d: torch.Tensor

    @classmethod
    def empty(cls, n_out: int, n_in: int, device="cuda") -> "Q80Weight":
        return cls(n_out, n_in, torch.empty(n_out * n_in, dtype=torch.int8, device=device),
                   torch.empty(n_out * n_in // 32, dtype=torch.float16, device=device))

    def c_struct(self) -> _capi.Q80WeightC:
        return _capi.Q80WeightC(self.n_out, self.n_in, self.q.data_ptr(), self.d.data_ptr())


def qlora_q8_0_packed_bytes(numel: int) -> int:
    return int(_lib().qlora_q8_0_packed_bytes(int(numel)))


def qlora_quantize_q8_0(W: torch.Tensor, weight: Q80Weight, stream=None) -> None:
    _need(W, torch.float32, (weight.n_out, weight.n_in), "W")
    s = weight.c_struct()
    _capi.check("qlora_quantize_q8_0", _lib().qlora_quantize_q8_0(_ptr(W), ctypes.byref(s), _stream(stream)))


def qlora_dequant_q8_0(weight: Q80Weight, out: torch.Tensor, stream=None) -> None:
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out must be float32 or bfloat16")
    _need(out, out.dtype, (weight.n_out, weight.n_in), "out")
    s = weight.c_struct()
    _capi.check("qlora_dequant_q8_0", _lib().qlora_dequant_q8_0(ctypes.byref(s), _ptr(out),
                                                                int(out.dtype == torch.bfloat16), _stream(stream)))


def qlora_q8_0_lora_linear_fwd(weight: Q80Weight, X, A, B, r: int, scaling: float, Y, U_save=None, ws=None,
                               stream=None) -> None:
    M = X.shape[0]
    _need(X, torch.bfloat16, (M, weight.n_in), "X")
    _need(Y, torch.bfloat16, (M, weight.n_out), "Y")
    if r:
        _need(A, torch.bfloat16, (r, weight.n_in), "A")
        _need(B, torch.bfloat16, (weight.n_out, r), "B")
    if U_save is not None:
        _need(U_save, torch.bfloat16, (M, r), "U_save")
    s = weight.c_struct()
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _capi.check("qlora_q8_0_lora_linear_fwd", _lib().qlora_q8_0_lora_linear_fwd(
        ctypes.byref(s), _ptr(X), M, _ptr(A), _ptr(B), int(r), float(scaling), _ptr(Y), _ptr(U_save), _ptr(ws),
        wsb, _stream(stream)))


def qlora_q8_0_lora_linear_bwd_dx(weight: Q80Weight, dY, A, B, r: int, scaling: float, dX, G_save=None, ws=None,
                                  stream=None) -> None:
    M = dY.shape[0]
    _need(dY, torch.bfloat16, (M, weight.n_out), "dY")
    _need(dX, torch.bfloat16, (M, weight.n_in), "dX")
    if r:
        _need(A, torch.bfloat16, (r, weight.n_in), "A")
        _need(B, torch.bfloat16, (weight.n_out, r), "B")
    if G_save is not None:
        _need(G_save, torch.bfloat16, (M, r), "G_save")
    s = weight.c_struct()
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _capi.check("qlora_q8_0_lora_linear_bwd_dx", _lib().qlora_q8_0_lora_linear_bwd_dx(
        ctypes.byref(s), _ptr(dY), M, _ptr(A), _ptr(B), int(r), float(scaling), _ptr(dX), _ptr(G_save), _ptr(ws),
        wsb, _stream(stream)))


# ----------------------------------------------------------------------------- embedding

def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _on(t, dev: int, name: str) -> None:
    """The calls launch on the current device: a tensor has to be contiguous and live there."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor on the current device cuda:{dev}, got strides {t.stride()} on "
                         f"{t.device}")


def _ids_bytes(ids, dev: int) -> int:
    if ids.dtype is torch.int64:
        size = 8
    elif ids.dtype is torch.int32:
        size = 4
    else:
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.dim() != 1:
        raise ValueError(f"ids must be [T], got {tuple(ids.shape)}")
    _on(ids, dev, "ids")
    return size


def _is_bf16(t, shape, dev: int, name: str) -> int:
    """1 for a bfloat16 tensor of that shape on the device, 0 for a float32 one; else an error."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev or not t.is_contiguous():
        _on(t, dev, name)
    if t.dtype is torch.bfloat16:
        return 1
    if t.dtype is torch.float32:
        return 0
    raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def qlora_embed_fwd(table: torch.Tensor, ids: torch.Tensor, scale: float, Y: torch.Tensor, stream=None) -> None:
    """Y [T, H] = scale * table[ids] from a float32 or bfloat16 table [V, H]."""
    dev = torch.cuda.current_device()
    if table.dim() != 2:
        raise ValueError("table must be [V, H]")
    V, H = table.shape
    T = ids.numel()
    idb, tb, yb = _ids_bytes(ids, dev), _is_bf16(table, (V, H), dev, "table"), _is_bf16(Y, (T, H), dev, "Y")
    st = _lib().qlora_embed_fwd(table.data_ptr(), tb, V, H, ids.data_ptr(), idb, T, scale, Y.data_ptr(), yb, _raw_stream(stream, dev))
    if st:
        _capi.check("qlora_embed_fwd", st)


def _embed_packed(name, f, weight, codes, ids, scale, Y, stream):
    dev = torch.cuda.current_device()
    T = ids.numel()
    idb, yb = _ids_bytes(ids, dev), _is_bf16(Y, (T, weight.n_in), dev, "Y")
    _on(codes, dev, "codes")
    st = f(ctypes.byref(weight.c_struct()), ids.data_ptr(), idb, T, scale, Y.data_ptr(), yb, _raw_stream(stream, dev))
    if st:
        _capi.check(name, st)


def qlora_embed_nf4_fwd(weight: NF4Weight, ids: torch.Tensor, scale: float, Y: torch.Tensor, stream=None) -> None:
    """Y [T, n_in] = scale * the dequantized rows `ids` of a packed 4-bit table, as float32 or bfloat16."""
    _embed_packed("qlora_embed_nf4_fwd", _lib().qlora_embed_nf4_fwd, weight, weight.codes, ids, scale, Y, stream)


def qlora_embed_q8_0_fwd(weight: Q80Weight, ids: torch.Tensor, scale: float, Y: torch.Tensor, stream=None) -> None:
    """Y [T, n_in] = scale * the dequantized rows `ids` of a Q8_0 table, as float32 or bfloat16."""
    _embed_packed("qlora_embed_q8_0_fwd", _lib().qlora_embed_q8_0_fwd, weight, weight.q, ids, scale, Y, stream)


def qlora_embed_grad_workspace_bytes(T: int, V: int, H: int) -> int:
    return int(_lib().qlora_embed_grad_workspace_bytes(int(T), int(V), int(H)))


def qlora_embed_grad(ids: torch.Tensor, dY: torch.Tensor, scale: float, dE: torch.Tensor, padding_id: int = -1,
                     accumulate: bool = False, ws=None, stream=None) -> None:
    """dE [V, H] = scale * the sum of dY's rows by token id (added to dE with accumulate); dY and dE are
    float32 or bfloat16, `ws` a scratch tensor of qlora_embed_grad_workspace_bytes(T, V, H)."""
    dev = torch.cuda.current_device()
    if dE.dim() != 2:
        raise ValueError("dE must be [V, H]")
    V, H = dE.shape
    T = ids.numel()
    idb, yb, eb = _ids_bytes(ids, dev), _is_bf16(dY, (T, H), dev, "dY"), _is_bf16(dE, (V, H), dev, "dE")
    if ws is not None:
        _on(ws, dev, "ws")
    st = _lib().qlora_embed_grad(
        ids.data_ptr(), idb, T, dY.data_ptr(), yb, V, H, scale, padding_id, dE.data_ptr(), eb, 1 if accumulate else 0,
        None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size(), _raw_stream(stream, dev))
    if st:
        _capi.check("qlora_embed_grad", st)


# ----------------------------------------------------------------------------- optimizer

@dataclass
class AdamWTensor:
    """One trained tensor of an AdamW plan: contiguous device buffers owned by the caller.

    param: float32 or bfloat16, updated in place; None with a grad alone makes a tensor that only counts in
    qlora_grad_norm.  exp_avg / exp_avg_sq: float32 m and v, or int8 / uint8 codes with their float32 block
    steps exp_avg_step / exp_avg_sq_step [ceil(numel / 256)] (8-bit states; all zeros is the start).
    param_bf16: bfloat16 copy written beside a float32 param (the A or B that the layer reads).  lr_scale
    multiplies the step's learning rate for this tensor."""
    param: torch.Tensor | None
    grad: torch.Tensor
    exp_avg: torch.Tensor | None = None
    exp_avg_sq: torch.Tensor | None = None
    exp_avg_step: torch.Tensor | None = None
    exp_avg_sq_step: torch.Tensor | None = None
    param_bf16: torch.Tensor | None = None
    lr_scale: float = 1.0
    weight_decay: float = 0.0

    @classmethod
    def zeros(cls, param: torch.Tensor, grad: torch.Tensor, bits: int = 32, **kw) -> "AdamWTensor":
        """The tensor with zero states of 32 or 8 bits."""
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32")
        n, dev = param.numel(), param.device
        if bits == 32:
            return cls(param, grad, *(torch.zeros(n, dtype=torch.float32, device=dev) for _ in range(2)), **kw)
        return cls(param, grad, torch.zeros(n, dtype=torch.int8, device=dev),
                   torch.zeros(n, dtype=torch.uint8, device=dev),
                   *(torch.zeros((n + 255) // 256, dtype=torch.float32, device=dev) for _ in range(2)), **kw)

    def c_struct(self) -> _capi.AdamWTensorC:
        if self.grad is None:
            raise ValueError("grad is required")
        dev, n = torch.cuda.current_device(), self.grad.numel()
        flags = _capi.OPT_GRAD_BF16 if _flat(self.grad, n, dev, _FLOATS, "grad") is torch.bfloat16 else 0
        if self.param is None:
            if self.exp_avg is not None or self.exp_avg_sq is not None or self.param_bf16 is not None:
                raise ValueError("a tensor without param has a grad alone")
            return _capi.AdamWTensorC(None, None, self.grad.data_ptr(), None, None, None, None, n, 0.0, 0.0,
                                      flags | _capi.OPT_GRAD_ONLY, 0)
        if _flat(self.param, n, dev, _FLOATS, "param") is torch.bfloat16:
            flags |= _capi.OPT_PARAM_BF16
        m_step = v_step = copy = None
        if _flat(self.exp_avg, n, dev, _FIRST, "exp_avg") is torch.int8:
            flags |= _capi.OPT_STATE_8BIT
            _flat(self.exp_avg_sq, n, dev, _CODES, "exp_avg_sq")
            nb = (n + 255) // 256
            _flat(self.exp_avg_step, nb, dev, _F32, "exp_avg_step")
            _flat(self.exp_avg_sq_step, nb, dev, _F32, "exp_avg_sq_step")
            m_step, v_step = self.exp_avg_step.data_ptr(), self.exp_avg_sq_step.data_ptr()
        else:
            _flat(self.exp_avg_sq, n, dev, _F32, "exp_avg_sq")
        if self.param_bf16 is not None:
            _flat(self.param_bf16, n, dev, _BF16, "param_bf16")
            copy = self.param_bf16.data_ptr()
        return _capi.AdamWTensorC(self.param.data_ptr(), copy, self.grad.data_ptr(), self.exp_avg.data_ptr(),
                                  self.exp_avg_sq.data_ptr(), m_step, v_step, n, self.lr_scale, self.weight_decay, flags, 0)


_F32, _BF16, _FLOATS = (torch.float32,), (torch.bfloat16,), (torch.float32, torch.bfloat16)
_FIRST, _CODES = (torch.float32, torch.int8), (torch.uint8,)


def _flat(t, n: int, dev: int, dtypes, name: str):
    """The type of a contiguous tensor of n elements on the device; an error for any other."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype not in dtypes or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {' or '.join(map(str, dtypes))} of {n} elements on cuda:{dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.dtype


@dataclass
class AdamWPlan:
    """A list of tensors prepared for qlora_adamw_step and qlora_grad_norm; keeps the buffers it names and the
    device buffer alive.  The calls go to the addresses of the time it was made: a field of an AdamWTensor that is
    assigned anew (a gradient that is allocated each step) does not change the plan, so fill the same buffers
    or make another plan.  Made by qlora_adamw_plan_init, whose stream the buffer belongs to: a plan that is used on
    another stream has to live until that work is done, like the tensors it names.  The buffer holds scratch of the
    norm and of a counted step: calls on one plan must not overlap in time."""
    tensors: list
    buffer: torch.Tensor
    c_plan: _capi.AdamWPlanC
    held: tuple = ()


def qlora_adamw_plan_init(tensors, stream=None) -> AdamWPlan:
    tensors = list(tensors)
    if not tensors:
        raise ValueError("a plan needs a tensor")
    dev = torch.cuda.current_device()
    arr = (_capi.AdamWTensorC * len(tensors))(*(t.c_struct() for t in tensors))
    nbytes = _lib().qlora_adamw_plan_bytes(arr, len(tensors))
    # from the pool of the stream that fills it: a block of the current stream's pool may still be written there
    with torch.cuda.stream(stream):
        buffer = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device="cuda")
    held = tuple(x for t in tensors for x in vars(t).values() if isinstance(x, torch.Tensor))
    plan = AdamWPlan(tensors, buffer, _capi.AdamWPlanC(), held)
    _capi.check("qlora_adamw_plan_init", _lib().qlora_adamw_plan_init(arr, len(tensors), buffer.data_ptr(), buffer.numel(),
                                                                      ctypes.byref(plan.c_plan), _raw_stream(stream, dev)))
    return plan


def _scalar(t, dtype, dev: int, name: str):
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != 1 or t.get_device() != dev:
        raise ValueError(f"{name}: expected one {dtype} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def qlora_adamw_step(plan: AdamWPlan, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999,
                     eps: float = 1e-8, grad_scale=None, lr_dev=None, step_dev=None, stream=None) -> None:
    """Step number `step` (from 1; 0 with a device counter step_dev) over the plan's tensors."""
    dev = torch.cuda.current_device()
    _on(plan.buffer, dev, "plan")
    st = _lib().qlora_adamw_step(
        ctypes.byref(plan.c_plan), lr, beta1, beta2, eps, step, _scalar(grad_scale, torch.float32, dev, "grad_scale"),
        _scalar(lr_dev, torch.float32, dev, "lr_dev"), _scalar(step_dev, torch.int64, dev, "step_dev"), _raw_stream(stream, dev))
    if st:
        _capi.check("qlora_adamw_step", st)


def qlora_grad_norm(plan: AdamWPlan, max_norm: float, out: torch.Tensor, stream=None) -> None:
    """out [2] float32 = the norm of the plan's gradients and the clip coefficient (pass out[1:2] as grad_scale)."""
    dev = torch.cuda.current_device()
    _flat(out, 2, dev, _F32, "out")
    _on(plan.buffer, dev, "plan")
    st = _lib().qlora_grad_norm(ctypes.byref(plan.c_plan), max_norm, out.data_ptr(), _raw_stream(stream, dev))
    if st:
        _capi.check("qlora_grad_norm", st)


def _adam8(codes, steps, x):
    dev, n = torch.cuda.current_device(), codes.numel()
    kind = _capi.ADAM8_SECOND if _flat(codes, n, dev, (torch.int8, torch.uint8), "codes") is torch.uint8 else _capi.ADAM8_FIRST
    _flat(steps, (n + 255) // 256, dev, _F32, "steps")
    _flat(x, n, dev, _F32, "x")
    return kind, n, dev


def qlora_adam8_encode(x: torch.Tensor, codes: torch.Tensor, steps: torch.Tensor, stream=None) -> None:
    """8-bit state of float32 moments x: m into int8 codes, or v into uint8 codes (of its root), with block steps."""
    kind, n, dev = _adam8(codes, steps, x)
    st = _lib().qlora_adam8_encode(x.data_ptr(), kind, codes.data_ptr(), steps.data_ptr(), n, _raw_stream(stream, dev))
    if st:
        _capi.check("qlora_adam8_encode", st)


def qlora_adam8_decode(codes: torch.Tensor, steps: torch.Tensor, x: torch.Tensor, stream=None) -> None:
    """The float32 moments that an 8-bit state stands for: m from int8 codes, v from uint8 codes."""
    kind, n, dev = _adam8(codes, steps, x)
    st = _lib().qlora_adam8_decode(codes.data_ptr(), kind, steps.data_ptr(), x.data_ptr(), n, _raw_stream(stream, dev))
    if st:
        _capi.check("qlora_adam8_decode", st)
