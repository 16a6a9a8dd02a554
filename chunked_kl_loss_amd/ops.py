"""Operators around the loss: the top-K teacher cache, the embedding table and
its gradient, activations in 8 bits and the RMS norm that saves its input so.

Argument marshalling over include/ckl.h, as in _binding.  Leading dimensions
are rows; tensors are contiguous and on one GPU.  Calls run on that GPU's
current stream."""
from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import CKL_TEACHER_LOGITS, _dtype_code, _empty, _ptr, check, load_library

ACT_BLOCK = 32  # columns that share an exponent (CKL_ACT_BLOCK)

_TOKEN_BYTES = {torch.int32: 4, torch.int64: 8}


def _check(device, **tensors) -> None:
    for name, t in tensors.items():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if t.device != device:
            raise ValueError(f"{name} must be on {device}, not {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _call(device, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream.  The library launches on the current GPU: the tensors'
    own is made current where it is not."""
    index = device.index
    if index == torch.cuda.current_device():
        # (the raw handle: a Stream object costs as much as a launch)
        check(fn(*args, torch._C._cuda_getCurrentRawStream(index)))
    else:
        with torch.cuda.device(device):
            check(fn(*args, torch._C._cuda_getCurrentRawStream(index)))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name: str, *sizes) -> int:
    out = ctypes.c_size_t(0)
    check(getattr(load_library(), name)(*sizes, ctypes.byref(out)))
    return out.value


def _workspace(device, name: str, *sizes):
    n = _workspace_bytes(name, *sizes)
    return (_empty(n, torch.uint8, device) if n else None), n


def _rows(t) -> int:
    """Rows of t [..., d]."""
    d = t.shape[-1]
    return t.numel() // d if d else 0


# ----------------------------------------------------------- teacher top-K --
def teacher_topk(logits, K: int, mask=None, teacher_form: int = CKL_TEACHER_LOGITS):
    """The sparse teacher that the loss reads, from full logits [..., V] (bf16 or fp32): returns
    (idx int32 [..., K], values float32 [..., K], lse float32 [...]), the K largest logits of a row in
    descending order (equal ones by index) and the row's log-sum-exp.  teacher_form 0: values are the logits;
    1: log-probabilities, logit - lse.  Rows whose mask (uint8 / bool [...]) is 0 are not read and get idx
    0 .. K-1, values 0, lse 0."""
    if logits.dim() < 1:
        raise ValueError("logits must be [..., V]")
    K = int(K)
    lead, V = logits.shape[:-1], logits.shape[-1]
    T, dev = _rows(logits), logits.device
    _check(dev, logits=logits)
    if mask is not None:
        _check(dev, mask=mask)
        if mask.shape != lead or mask.dtype not in (torch.uint8, torch.bool):
            raise ValueError("mask must be a uint8/bool tensor of the logits' leading shape")
    code = _dtype_code(logits.dtype)
    lib = load_library()
    ws, ws_bytes = _workspace(dev, "ckl_topk_workspace_size", T, V, K)
    idx = _empty((*lead, K), torch.int32, dev)
    values = _empty((*lead, K), torch.float32, dev)
    lse = _empty(lead, torch.float32, dev)
    _call(dev, lib.ckl_teacher_topk, _ptr(logits), code, T, V, K, teacher_form, _ptr(mask), _ptr(idx), _ptr(values),
          _ptr(lse), _ptr(ws), ws_bytes)
    return idx, values, lse


# --------------------------------------------------------------- embedding --
def _token_bytes(tokens) -> int:
    if tokens.dtype not in _TOKEN_BYTES:
        raise TypeError("tokens must be int32 or int64")
    return _TOKEN_BYTES[tokens.dtype]


def embedding_forward(W, tokens, scale: float = 1.0, v_offset: int = 0):
    """scale * W[tokens - v_offset] as [*tokens.shape, d] in W's dtype; a zero row for a token outside
    [v_offset, v_offset + V) (padding, or another shard's)."""
    if W.dim() != 2:
        raise ValueError("W must be [V, d]")
    dev = W.device
    _check(dev, W=W, tokens=tokens)
    nb, code = _token_bytes(tokens), _dtype_code(W.dtype)
    V, d = W.shape
    out = _empty((*tokens.shape, d), W.dtype, dev)
    lib = load_library()
    _call(dev, lib.ckl_embedding_forward, _ptr(W), code, V, d, v_offset, _ptr(tokens), nb, tokens.numel(), scale,
          _ptr(out))
    return out


def embedding_backward(dY, tokens, V: int, scale: float = 1.0, v_offset: int = 0, dw_dtype=None, add_to=None):
    """dW[v] = scale * the sum of dY [..., d] over the positions of token v + v_offset, as [V, d] in dw_dtype
    (default float32).  add_to: a [V, d] gradient (the tied head's) the sums are added to in place; it is
    returned, and rows without a token are not touched."""
    if dY.dim() < 1 or dY.shape[:-1] != tokens.shape:
        raise ValueError("dY must be [*tokens.shape, d]")
    dev, d = dY.device, dY.shape[-1]
    _check(dev, dY=dY, tokens=tokens)
    nb, code = _token_bytes(tokens), _dtype_code(dY.dtype)
    if add_to is not None:
        _check(dev, add_to=add_to)
        if add_to.shape != (V, d):
            raise ValueError("add_to must be [V, d]")
        if dw_dtype is not None and dw_dtype != add_to.dtype:
            raise TypeError("dw_dtype differs from add_to's")
        dW, dw_code = add_to, _dtype_code(add_to.dtype)
    else:
        dw_dtype = torch.float32 if dw_dtype is None else dw_dtype
        dw_code = _dtype_code(dw_dtype)
    T = tokens.numel()
    lib = load_library()
    ws, ws_bytes = _workspace(dev, "ckl_embedding_workspace_size", T, d, V)
    if add_to is None:
        dW = _empty((V, d), dw_dtype, dev)
    _call(dev, lib.ckl_embedding_backward, _ptr(dY), code, T, d, _ptr(tokens), nb, V, v_offset, scale, _ptr(dW),
          dw_code, int(add_to is not None), _ptr(ws), ws_bytes)
    return dW


# ------------------------------------------------- 8-bit activations, norm --
def _check_codes(codes, exps):
    if codes.dim() < 1 or codes.dtype != torch.int8 or exps.dtype != torch.uint8:
        raise TypeError("codes must be int8 and exps uint8")
    if exps.shape != (*codes.shape[:-1], -(-codes.shape[-1] // ACT_BLOCK)):
        raise ValueError("exps must be [..., ceil(d / 32)] for codes [..., d]")


def _check_weight(weight, d):
    if weight.shape != (d,):
        raise ValueError("weight must be [d]")
    return _dtype_code(weight.dtype)


def _codes_for(lead, d, dev):
    return (_empty((*lead, d), torch.int8, dev), _empty((*lead, -(-d // ACT_BLOCK)), torch.uint8, dev))


def act_encode(x):
    """x [..., d] (bf16 or fp32) in 8 bits: (codes int8 [..., d], exps uint8 [..., ceil(d / 32)]).  A code stands
    for code * 2^(E - 127) with the E of its 32 columns: within max|x| / 127.5 of x over them."""
    if x.dim() < 1:
        raise ValueError("x must be [..., d]")
    dev, d = x.device, x.shape[-1]
    _check(dev, x=x)
    code = _dtype_code(x.dtype)
    codes, exps = _codes_for(x.shape[:-1], d, dev)
    lib = load_library()
    _call(dev, lib.ckl_act_encode, _ptr(x), code, _rows(x), d, _ptr(codes), _ptr(exps))
    return codes, exps


def act_decode(codes, exps, rstd=None, weight=None, dtype=torch.bfloat16):
    """The values the codes stand for (exact in bf16 and fp32); with rstd [...] and weight [d], the RMS norm's
    output rebuilt from them: value * rstd * weight, rounded once."""
    dev = codes.device
    _check(dev, codes=codes, exps=exps)
    _check_codes(codes, exps)
    lead, d = codes.shape[:-1], codes.shape[-1]
    if (rstd is None) != (weight is None):
        raise ValueError("rstd and weight go together")
    w_code = 0
    if rstd is not None:
        _check(dev, rstd=rstd, weight=weight)
        w_code = _check_weight(weight, d)
        if rstd.shape != lead or rstd.dtype != torch.float32:
            raise ValueError("rstd must be a float32 tensor of the rows' shape")
    code = _dtype_code(dtype)
    out = _empty(codes.shape, dtype, dev)
    lib = load_library()
    _call(dev, lib.ckl_act_decode, _ptr(codes), _ptr(exps), _rows(codes), d, _ptr(rstd), _ptr(weight), w_code,
          _ptr(out), code)
    return out


def norm_forward(x, weight, eps: float = 1e-6, save: bool = True):
    """RMS norm over the last dimension: (y, codes, exps, rstd) with y = x * rstd * weight in x's dtype and x in
    8 bits for norm_backward; save=False: y alone is computed and the others are None."""
    if x.dim() < 1:
        raise ValueError("x must be [..., d]")
    dev, lead, d = x.device, x.shape[:-1], x.shape[-1]
    _check(dev, x=x, weight=weight)
    code, w_code = _dtype_code(x.dtype), _check_weight(weight, d)
    y = _empty(x.shape, x.dtype, dev)
    codes = exps = rstd = None
    if save:
        codes, exps = _codes_for(lead, d, dev)
        rstd = _empty(lead, torch.float32, dev)
    lib = load_library()
    _call(dev, lib.ckl_norm_forward, _ptr(x), code, _rows(x), d, _ptr(weight), w_code, eps, _ptr(y), _ptr(codes),
          _ptr(exps), _ptr(rstd))
    return y, codes, exps, rstd


def norm_backward(dy, codes, exps, rstd, weight):
    """Gradients (dx in dy's dtype, dweight in weight's) of the norm from what norm_forward saved."""
    dev = dy.device
    _check(dev, dy=dy, codes=codes, exps=exps, rstd=rstd, weight=weight)
    _check_codes(codes, exps)
    lead, d = codes.shape[:-1], codes.shape[-1]
    if dy.shape != codes.shape:
        raise ValueError("dy must have the codes' shape")
    if rstd.shape != lead or rstd.dtype != torch.float32:
        raise ValueError("rstd must be a float32 tensor of the rows' shape")
    code, w_code = _dtype_code(dy.dtype), _check_weight(weight, d)
    T = _rows(codes)
    lib = load_library()
    ws, ws_bytes = _workspace(dev, "ckl_norm_workspace_size", T, d)
    dx = _empty(dy.shape, dy.dtype, dev)
    dweight = _empty(d, weight.dtype, dev)
    _call(dev, lib.ckl_norm_backward, _ptr(dy), code, T, d, _ptr(codes), _ptr(exps), _ptr(rstd), _ptr(weight), w_code,
          _ptr(dx), _ptr(dweight), _ptr(ws), ws_bytes)
    return dx, dweight
