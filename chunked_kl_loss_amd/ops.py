"""Operators around the loss: the top-K teacher cache, log probabilities of given
tokens (from logits, and from states and head), the embedding table and its
gradient, activations in 8 bits and the RMS norm that saves its input so,
dropout, and the RMS norm with the residual's addition.

Argument marshalling over include/ckl.h, as in _binding.  Leading dimensions
are rows; tensors are contiguous and on one GPU.  The library takes arrays from
a 16-byte boundary: an input that begins off one (a slice of rows of an odd
width) is copied first.  Calls run on that GPU's current stream.  Small calls are bound by this layer, so it does little: one
pass over the arguments, the outputs, the call."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _binding
from ._binding import (CKL_BF16, CKL_F32, CKL_QUANT_E4M3, CKL_QUANT_INT8, CKL_TEACHER_LOGITS, check,
                       load_library)

ACT_BLOCK = 32  # columns that share an exponent (CKL_ACT_BLOCK)

_CODES = {torch.bfloat16: CKL_BF16, torch.float32: CKL_F32}
_TOKEN_BYTES = {torch.int32: 4, torch.int64: 8}


def _code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}; use torch.bfloat16 or torch.float32")
    return code


def _token_bytes(tokens) -> int:
    nb = _TOKEN_BYTES.get(tokens.dtype)
    if nb is None:
        raise TypeError("tokens must be int32 or int64")
    return nb


def _check(names, *tensors):
    """The device of the tensors, which must be contiguous and on one GPU."""
    device = tensors[0].device
    for name, t in zip(names, tensors):
        if t.device != device or not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor on {device if device.type == 'cuda' else 'a GPU'}, "
                             f"not on {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return device


def _aligned(t):
    return t.clone() if t.data_ptr() & 15 else t


def _new(shape, dtype, device):
    t = torch.empty(shape, dtype=dtype, device=device)
    if _binding.FILL_BYTE is not None and t.numel() > 0:
        t.view(-1).view(torch.uint8).fill_(int(_binding.FILL_BYTE))
    return t


def _like(t):
    """_new of the shape and type of a contiguous tensor (a third cheaper)."""
    t = torch.empty_like(t)
    if _binding.FILL_BYTE is not None and t.numel() > 0:
        t.view(-1).view(torch.uint8).fill_(int(_binding.FILL_BYTE))
    return t


def _call(device, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream.  The library launches on the current GPU: the tensors'
    own is made current where it is not."""
    index = device.index
    if index == torch._C._cuda_getDevice():  # (torch.cuda.current_device without its checks: there are GPU tensors)
        # (the raw handle: a Stream object costs as much as a launch)
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        check(status)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name: str, *sizes) -> int:
    out = ctypes.c_size_t(0)
    check(getattr(load_library(), name)(*sizes, ctypes.byref(out)))
    return out.value


def _workspace(device, name: str, *sizes):
    """A workspace (None where the call needs none), its address and its bytes."""
    n = _workspace_bytes(name, *sizes)
    if not n:
        return None, None, 0
    ws = _new(n, torch.uint8, device)
    return ws, ws.data_ptr(), n


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
    if mask is None:
        dev, mask_ptr = _check(("logits",), logits), None
    else:
        dev, mask_ptr = _check(("logits", "mask"), logits, mask), mask.data_ptr()
        if mask.shape != lead or mask.dtype not in (torch.uint8, torch.bool):
            raise ValueError("mask must be a uint8/bool tensor of the logits' leading shape")
    T, code = _rows(logits), _code(logits.dtype)
    logits = _aligned(logits)
    ws, ws_ptr, ws_bytes = _workspace(dev, "ckl_topk_workspace_size", T, V, K)
    idx = _new((*lead, K), torch.int32, dev)
    values = _new((*lead, K), torch.float32, dev)
    lse = _new(lead, torch.float32, dev)
    _call(dev, load_library().ckl_teacher_topk, logits.data_ptr(), code, T, V, K, teacher_form, mask_ptr,
          idx.data_ptr(), values.data_ptr(), lse.data_ptr(), ws_ptr, ws_bytes)
    return idx, values, lse


# ----------------------------------------------- log probabilities of tokens --
def _check_rows_args(tokens, mask, lead, what):
    """Checks of per-row arguments; the mask's address."""
    if tokens.shape != lead:
        raise ValueError(f"tokens must have the leading shape of {what}")
    if mask is None:
        return None
    if mask.shape != lead or mask.dtype not in (torch.uint8, torch.bool):
        raise ValueError(f"mask must be a uint8/bool tensor of the leading shape of {what}")
    return mask.data_ptr()


def _check_row_floats(lead, **rows):
    for name, t in rows.items():
        if t is not None and (t.shape != lead or t.dtype != torch.float32):
            raise ValueError(f"{name} must be a float32 tensor of the rows' shape")


def _given(**tensors):
    """Names and tensors of those that are not None, for _check."""
    there = {name: t for name, t in tensors.items() if t is not None}
    return tuple(there), *there.values()


def _ptr(t):
    return None if t is None else t.data_ptr()


def token_logprobs_forward(logits, tokens, top: int = 0, mask=None):
    """From logits [..., V] (bf16 or fp32): (logprob, entropy, lse: float32 [...], top_idx int32 and top_logprob
    float32 [..., top]).  logprob is that of tokens [...] (int32 / int64; 0 for a token outside [0, V)), entropy
    that of the row's softmax, top_idx the most likely columns in descending order (equal ones by index).  Rows
    whose mask (uint8 / bool [...]) is 0 are not read and get 0 (top_idx 0 .. top-1)."""
    if logits.dim() < 1:
        raise ValueError("logits must be [..., V]")
    top = int(top)
    lead, V = logits.shape[:-1], logits.shape[-1]
    dev = _check(*_given(logits=logits, tokens=tokens, mask=mask))
    mask_ptr = _check_rows_args(tokens, mask, lead, "logits")
    T, code, nb = tokens.numel(), _code(logits.dtype), _token_bytes(tokens)
    logits = _aligned(logits)
    ws, ws_ptr, ws_bytes = _workspace(dev, "ckl_logprob_workspace_size", T, V, top)
    logprob, entropy, lse = (_new(lead, torch.float32, dev) for _ in range(3))
    top_idx = _new((*lead, top), torch.int32, dev)
    top_logprob = _new((*lead, top), torch.float32, dev)
    _call(dev, load_library().ckl_token_logprobs, logits.data_ptr(), code, T, V, tokens.data_ptr(), nb, top, mask_ptr,
          logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), top_idx.data_ptr(), top_logprob.data_ptr(), ws_ptr,
          ws_bytes)
    return logprob, entropy, lse, top_idx, top_logprob


def token_logprobs_backward(dlogprob, dentropy, logits, tokens, lse, entropy, mask=None):
    """Gradient of the logits, in their type, from those of logprob and entropy (float32 [...]; either may be None)
    and what token_logprobs_forward returned.  Rows that are masked or have no gradient get zeros."""
    lead, V = logits.shape[:-1], logits.shape[-1]
    dev = _check(*_given(logits=logits, tokens=tokens, lse=lse, entropy=entropy, mask=mask, dlogprob=dlogprob,
                         dentropy=dentropy))
    mask_ptr = _check_rows_args(tokens, mask, lead, "logits")
    _check_row_floats(lead, lse=lse, entropy=entropy, dlogprob=dlogprob, dentropy=dentropy)
    T, code, nb = tokens.numel(), _code(logits.dtype), _token_bytes(tokens)
    logits = _aligned(logits)
    dlogits = _like(logits)
    _call(dev, load_library().ckl_token_logprobs_backward, logits.data_ptr(), code, T, V, tokens.data_ptr(), nb,
          mask_ptr, lse.data_ptr(), entropy.data_ptr(), _ptr(dlogprob), _ptr(dentropy), dlogits.data_ptr())
    return dlogits


def _check_head(H, W):
    if H.dim() < 1 or W.dim() != 2 or H.shape[-1] != W.shape[1] or H.dtype != W.dtype:
        raise ValueError("H [..., d] and W [V, d] must share d and dtype")


def head_logprobs_forward(H, W, tokens, mask=None, chunk: int = 2048):
    """(logprob, entropy, lse: float32 [...]) of the logits H W^T, which are never stored: H [..., d] and W [V, d]
    (bf16 or fp32), tokens and mask [...] as for token_logprobs_forward.  Masked rows are not computed."""
    _check_head(H, W)
    lead = H.shape[:-1]
    dev = _check(*_given(H=H, W=W, tokens=tokens, mask=mask))
    mask_ptr = _check_rows_args(tokens, mask, lead, "H")
    T, code, nb = tokens.numel(), _code(H.dtype), _token_bytes(tokens)
    V, d = W.shape
    H, W = _aligned(H), _aligned(W)
    ws, ws_ptr, ws_bytes = _workspace(dev, "ckl_head_workspace_size", T, d, V, chunk, code, code, CKL_F32,
                                      int(mask is not None), 0)
    logprob, entropy, lse = (_new(lead, torch.float32, dev) for _ in range(3))
    _call(dev, load_library().ckl_head_logprobs, H.data_ptr(), W.data_ptr(), code, T, d, V, tokens.data_ptr(), nb,
          mask_ptr, chunk, logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), ws_ptr, ws_bytes)
    return logprob, entropy, lse


def head_logprobs_backward(dlogprob, dentropy, H, W, tokens, lse, entropy, mask=None, chunk: int = 2048, dh_dtype=None,
                           dw_dtype=None, need_dh: bool = True, need_dw: bool = True):
    """Gradients (dH in dh_dtype, default H's; dW in dw_dtype, default float32) from those of logprob and entropy
    (float32 [...]; either may be None) and what head_logprobs_forward returned.  The logits are multiplied again.
    need_dh / need_dw False: that gradient is not computed and None."""
    _check_head(H, W)
    if not (need_dh or need_dw):
        return None, None
    lead = H.shape[:-1]
    dev = _check(*_given(H=H, W=W, tokens=tokens, lse=lse, entropy=entropy, mask=mask, dlogprob=dlogprob,
                         dentropy=dentropy))
    mask_ptr = _check_rows_args(tokens, mask, lead, "H")
    _check_row_floats(lead, lse=lse, entropy=entropy, dlogprob=dlogprob, dentropy=dentropy)
    T, code, nb = tokens.numel(), _code(H.dtype), _token_bytes(tokens)
    V, d = W.shape
    dh_dtype = H.dtype if dh_dtype is None else dh_dtype
    dw_dtype = torch.float32 if dw_dtype is None else dw_dtype
    H, W = _aligned(H), _aligned(W)
    ws, ws_ptr, ws_bytes = _workspace(dev, "ckl_head_workspace_size", T, d, V, chunk, code, _code(dh_dtype),
                                      _code(dw_dtype), int(mask is not None), 1)
    dH = (_like(H) if dh_dtype == H.dtype else _new(H.shape, dh_dtype, dev)) if need_dh else None
    dW = _new(W.shape, dw_dtype, dev) if need_dw else None
    _call(dev, load_library().ckl_head_logprobs_backward, H.data_ptr(), W.data_ptr(), code, T, d, V,
          tokens.data_ptr(), nb, mask_ptr, chunk, lse.data_ptr(), entropy.data_ptr(), _ptr(dlogprob), _ptr(dentropy),
          _ptr(dH), _code(dh_dtype), _ptr(dW), _code(dw_dtype), ws_ptr, ws_bytes)
    return dH, dW


# --------------------------------------------------------------- embedding --
def embedding_forward(W, tokens, scale: float = 1.0, v_offset: int = 0):
    """scale * W[tokens - v_offset] as [*tokens.shape, d] in W's dtype; a zero row for a token outside
    [v_offset, v_offset + V) (padding, or another shard's)."""
    if W.dim() != 2:
        raise ValueError("W must be [V, d]")
    dev = _check(("W", "tokens"), W, tokens)
    nb, code = _token_bytes(tokens), _code(W.dtype)
    V, d = W.shape
    W = _aligned(W)
    out = _new((*tokens.shape, d), W.dtype, dev)
    _call(dev, load_library().ckl_embedding_forward, W.data_ptr(), code, V, d, v_offset, tokens.data_ptr(), nb,
          tokens.numel(), scale, out.data_ptr())
    return out


def embedding_backward(dY, tokens, V: int, scale: float = 1.0, v_offset: int = 0, dw_dtype=None, add_to=None):
    """dW[v] = scale * the sum of dY [..., d] over the positions of token v + v_offset, as [V, d] in dw_dtype
    (default float32).  add_to: a [V, d] gradient (the tied head's, from a 16-byte boundary) the sums are added to
    in place; it is returned, and rows without a token are not touched."""
    if dY.dim() < 1 or dY.shape[:-1] != tokens.shape:
        raise ValueError("dY must be [*tokens.shape, d]")
    d = dY.shape[-1]
    if add_to is None:
        dev = _check(("dY", "tokens"), dY, tokens)
        dw_dtype = torch.float32 if dw_dtype is None else dw_dtype
    else:
        dev = _check(("dY", "tokens", "add_to"), dY, tokens, add_to)
        if add_to.shape != (V, d):
            raise ValueError("add_to must be [V, d]")
        if dw_dtype is not None and dw_dtype != add_to.dtype:
            raise TypeError("dw_dtype differs from add_to's")
        dw_dtype = add_to.dtype
    nb, code, dw_code = _token_bytes(tokens), _code(dY.dtype), _code(dw_dtype)
    T = tokens.numel()
    dY = _aligned(dY)
    ws, ws_ptr, ws_bytes = _workspace(dev, "ckl_embedding_workspace_size", T, d, V)
    dW = _new((V, d), dw_dtype, dev) if add_to is None else add_to
    _call(dev, load_library().ckl_embedding_backward, dY.data_ptr(), code, T, d, tokens.data_ptr(), nb, V, v_offset,
          scale, dW.data_ptr(), dw_code, int(add_to is not None), ws_ptr, ws_bytes)
    return dW


# ------------------------------------------------- 8-bit activations, norm --
def _check_codes(codes, exps):
    if codes.dim() < 1 or codes.dtype != torch.int8 or exps.dtype != torch.uint8:
        raise TypeError("codes must be int8 and exps uint8")
    if exps.shape != (*codes.shape[:-1], -(-codes.shape[-1] // ACT_BLOCK)):
        raise ValueError("exps must be [..., ceil(d / 32)] for codes [..., d]")


def _check_rstd(rstd, lead):
    if rstd.shape != lead or rstd.dtype != torch.float32:
        raise ValueError("rstd must be a float32 tensor of the rows' shape")


def _weight_code(weight, d) -> int:
    if weight.shape != (d,):
        raise ValueError("weight must be [d]")
    return _code(weight.dtype)


def act_encode(x):
    """x [..., d] (bf16 or fp32) in 8 bits: (codes int8 [..., d], exps uint8 [..., ceil(d / 32)]).  A code stands
    for code * 2^(E - 127) with the E of its 32 columns: within max|x| / 127.5 of x over them."""
    if x.dim() < 1:
        raise ValueError("x must be [..., d]")
    dev, shape, code = _check(("x",), x), x.shape, _code(x.dtype)
    d, x = shape[-1], _aligned(x)
    codes = _new(shape, torch.int8, dev)
    exps = _new((*shape[:-1], -(-d // ACT_BLOCK)), torch.uint8, dev)
    _call(dev, load_library().ckl_act_encode, x.data_ptr(), code, _rows(x), d, codes.data_ptr(), exps.data_ptr())
    return codes, exps


def act_decode(codes, exps, rstd=None, weight=None, dtype=torch.bfloat16):
    """The values the codes stand for (exact in bf16 and fp32); with rstd [...] and weight [d], the RMS norm's
    output rebuilt from them: value * rstd * weight, rounded once."""
    if (rstd is None) != (weight is None):
        raise ValueError("rstd and weight go together")
    code, rstd_ptr, weight_ptr, w_code = _code(dtype), None, None, 0
    if rstd is None:
        dev = _check(("codes", "exps"), codes, exps)
        _check_codes(codes, exps)
    else:
        dev = _check(("codes", "exps", "rstd", "weight"), codes, exps, rstd, weight)
        _check_codes(codes, exps)
        _check_rstd(rstd, codes.shape[:-1])
        weight = _aligned(weight)
        rstd_ptr, weight_ptr, w_code = rstd.data_ptr(), weight.data_ptr(), _weight_code(weight, codes.shape[-1])
    codes = _aligned(codes)
    out = _new(codes.shape, dtype, dev)
    _call(dev, load_library().ckl_act_decode, codes.data_ptr(), exps.data_ptr(), _rows(codes), codes.shape[-1],
          rstd_ptr, weight_ptr, w_code, out.data_ptr(), code)
    return out


def norm_forward(x, weight, eps: float = 1e-6, save: bool = True):
    """RMS norm over the last dimension: (y, codes, exps, rstd) with y = x * rstd * weight in x's dtype and x in
    8 bits for norm_backward; save=False: y alone is computed and the others are None."""
    if x.dim() < 1:
        raise ValueError("x must be [..., d]")
    dev, shape, code = _check(("x", "weight"), x, weight), x.shape, _code(x.dtype)
    d = shape[-1]
    w_code = _weight_code(weight, d)
    x, weight = _aligned(x), _aligned(weight)
    y = _new(shape, x.dtype, dev)
    if save:
        codes = _new(shape, torch.int8, dev)
        exps = _new((*shape[:-1], -(-d // ACT_BLOCK)), torch.uint8, dev)
        rstd = _new(shape[:-1], torch.float32, dev)
        saved = codes.data_ptr(), exps.data_ptr(), rstd.data_ptr()
    else:
        codes = exps = rstd = None
        saved = None, None, None
    _call(dev, load_library().ckl_norm_forward, x.data_ptr(), code, _rows(x), d, weight.data_ptr(), w_code, eps,
          y.data_ptr(), *saved)
    return y, codes, exps, rstd


def norm_backward(dy, codes, exps, rstd, weight):
    """Gradients (dx in dy's dtype, dweight in weight's) of the norm from what norm_forward saved."""
    dev = _check(("dy", "codes", "exps", "rstd", "weight"), dy, codes, exps, rstd, weight)
    _check_codes(codes, exps)
    shape = codes.shape
    if dy.shape != shape:
        raise ValueError("dy must have the codes' shape")
    _check_rstd(rstd, shape[:-1])
    d, T, code = shape[-1], _rows(codes), _code(dy.dtype)
    w_code = _weight_code(weight, d)
    dy, codes, weight = _aligned(dy), _aligned(codes), _aligned(weight)
    ws, ws_ptr, ws_bytes = _workspace(dev, "ckl_norm_workspace_size", T, d)
    dx = _new(shape, dy.dtype, dev)
    dweight = _new(weight.shape, weight.dtype, dev)
    _call(dev, load_library().ckl_norm_backward, dy.data_ptr(), code, T, d, codes.data_ptr(), exps.data_ptr(),
          rstd.data_ptr(), weight.data_ptr(), w_code, dx.data_ptr(), dweight.data_ptr(), ws_ptr, ws_bytes)
    return dx, dweight


# The same for autograd, with all that is saved in one tensor (rstd, codes from a 16-byte boundary, exps): a norm
# of a few rows costs what its host does, and two tensors fewer to make and to keep take 132 us to 113
# (257 x 520 fp32, forward and backward).
def _norm_saved(T, d):
    codes = (4 * T + 15) & ~15
    return codes, codes + T * d, codes + T * (d + -(-d // ACT_BLOCK))


def norm_forward_saving(x, weight, eps: float, mask=None):
    """norm_forward as (y, saved); rows whose mask is 0 are saved as rows of zeros (norm_drop_rows)."""
    if x.dim() < 1:
        raise ValueError("x must be [..., d]")
    dev, d, code = _check(("x", "weight"), x, weight), x.shape[-1], _code(x.dtype)
    if mask is not None:
        _check(("x", "mask"), x, mask)
    w_code, T = _weight_code(weight, d), _rows(x)
    x, weight = _aligned(x), _aligned(weight)
    codes, exps, size = _norm_saved(T, d)
    y = _new(x.shape, x.dtype, dev)
    saved = _new(size, torch.uint8, dev)
    at = saved.data_ptr()
    _call(dev, load_library().ckl_norm_forward, x.data_ptr(), code, T, d, weight.data_ptr(), w_code, eps, y.data_ptr(),
          at + codes, at + exps, at)
    if mask is not None:
        norm_drop_rows(saved[exps:].view(T, -(-d // ACT_BLOCK)), saved[:4 * T].view(torch.float32), mask)
    return y, saved


def norm_drop_rows(exps, rstd, mask) -> None:
    """Rows of exps [T, ...] and rstd [T] whose mask [T] is 0 become those of zeros: a row that nothing reads may
    hold infinities or NaN, which a gradient of zero would not keep out of the weight's gradient."""
    drop = mask == 0
    exps.masked_fill_(drop[:, None], 1)
    rstd.masked_fill_(drop, 0.0)


def norm_backward_saved(dy, saved, weight):
    """norm_backward from what norm_forward_saving saved for rows of dy's shape and type."""
    dev, d, T = dy.device, dy.shape[-1], _rows(dy)
    dy, weight = _aligned(dy), _aligned(weight)
    codes, exps, _ = _norm_saved(T, d)
    ws, ws_ptr, ws_bytes = _workspace(dev, "ckl_norm_workspace_size", T, d)
    dx = _new(dy.shape, dy.dtype, dev)
    dweight = _new(weight.shape, weight.dtype, dev)
    at = saved.data_ptr()
    _call(dev, load_library().ckl_norm_backward, dy.data_ptr(), _CODES[dy.dtype], T, d, at + codes, at + exps, at,
          weight.data_ptr(), _CODES[weight.dtype], dx.data_ptr(), dweight.data_ptr(), ws_ptr, ws_bytes)
    return dx, dweight


# ---------------------------------------- dropout, norm behind a residual's sum --
def _drop_args(p, seed, offset, device):
    """p, seed, offset and the state's address for the library."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be from 0 to 1")
    offset = int(offset)
    if not 0 <= offset < 2 ** 64:
        raise ValueError("offset must be from 0 to 2^64 - 1")
    if isinstance(seed, torch.Tensor):
        if seed.shape != (2,) or seed.dtype != torch.int64 or not seed.is_contiguous() or seed.device != device:
            raise ValueError("seed must be an integer or an int64 tensor [2], (seed, offset), on the inputs' GPU")
        return p, 0, offset, seed.data_ptr()
    seed = int(seed)
    if not 0 <= seed < 2 ** 64:
        raise ValueError("seed must be from 0 to 2^64 - 1")
    return p, seed, offset, None


def dropout_forward(x, p: float, seed=0, offset: int = 0):
    """x * 1 / (1 - p) where kept, 0 elsewhere, with a mask that is a function of (seed, offset, element): p is taken
    to the nearest multiple of 2^-16.  The gradient is the same call on the incoming one.  seed: an integer, or an
    int64 tensor (seed, offset) on the GPU that is read when the kernel runs, its offset added to this one: a
    captured call then draws anew when the tensor changes."""
    dev, code = _check(("x",), x), _code(x.dtype)
    args = _drop_args(p, seed, offset, dev)
    x = _aligned(x)
    out = _like(x)
    _call(dev, load_library().ckl_dropout, x.data_ptr(), code, x.numel(), *args, out.data_ptr())
    return out


def _check_branch(x, residual, weight):
    if x.dim() < 1 or residual.shape != x.shape:
        raise ValueError("x and residual must be [..., d] of one shape")
    dev = _check(("x", "residual", "weight"), x, residual, weight)
    return dev, _code(x.dtype), _code(residual.dtype), _weight_code(weight, x.shape[-1])


def add_norm_forward(x, residual, weight, eps: float = 1e-6, p: float = 0.0, seed=0, offset: int = 0,
                     save: bool = True):
    """(y, h, rstd): h = residual + dropout(x) in the residual's type (x's, or float32 with x in bf16), y = h * rstd *
    weight in x's, rstd float32 [...] of h for add_norm_backward (None with save=False).  p, seed, offset as for
    dropout_forward."""
    dev, code, r_code, w_code = _check_branch(x, residual, weight)
    args = _drop_args(p, seed, offset, dev)
    x, residual, weight = _aligned(x), _aligned(residual), _aligned(weight)
    y, h = _like(x), _like(residual)
    rstd = _new(x.shape[:-1], torch.float32, dev) if save else None
    _call(dev, load_library().ckl_add_norm_forward, x.data_ptr(), code, residual.data_ptr(), r_code, _rows(x),
          x.shape[-1], weight.data_ptr(), w_code, eps, *args, h.data_ptr(), y.data_ptr(), _ptr(rstd))
    return y, h, rstd


def add_norm_backward(dy, dh, h, rstd, weight, p: float = 0.0, seed=0, offset: int = 0):
    """Gradients (dx in dy's type, dresidual in h's, dweight in weight's) from those of y and h (dh may be None), h and
    rstd.  Without dropout and with one type, dx is dresidual itself."""
    if dy.shape != h.shape or (dh is not None and (dh.shape != h.shape or dh.dtype != h.dtype)):
        raise ValueError("dy and dh must have h's shape, and dh its type")
    dev = _check(*_given(dy=dy, h=h, rstd=rstd, weight=weight, dh=dh))
    _check_rstd(rstd, h.shape[:-1])
    _weight_code(weight, h.shape[-1])
    _code(dy.dtype), _code(h.dtype)
    return add_norm_backward_saved(dy, dh, h, rstd, weight, _drop_args(p, seed, offset, dev))


def add_norm_backward_saved(dy, dh, h, rstd, weight, args):
    """add_norm_backward from what a forward call checked: args are its _drop_args."""
    dev, d, T = h.device, h.shape[-1], _rows(h)
    code, r_code, w_code = _CODES[dy.dtype], _CODES[h.dtype], _CODES[weight.dtype]
    dy, h, weight = _aligned(dy), _aligned(h), _aligned(weight)
    dh = None if dh is None else _aligned(dh)
    ws, ws_ptr, ws_bytes = _workspace(dev, "ckl_add_norm_workspace_size", T, d)
    dresidual = _like(h)
    dx = _like(dy) if args[0] > 0.0 or code != r_code else None
    dweight = _like(weight)
    _call(dev, load_library().ckl_add_norm_backward, dy.data_ptr(), code, _ptr(dh), r_code, T, d, h.data_ptr(),
          rstd.data_ptr(), weight.data_ptr(), w_code, *args, _ptr(dx), dresidual.data_ptr(), dweight.data_ptr(),
          ws_ptr, ws_bytes)
    return (dresidual if dx is None else dx), dresidual, dweight


_FORMS = {"int8": CKL_QUANT_INT8, "e4m3": CKL_QUANT_E4M3}


def add_norm_quant(x, residual, weight, eps: float = 1e-6, form: str = "int8"):
    """The norm behind a residual's addition with its output in 8 bits: (codes, scales, h), without a gradient (one that
    is asked for is an error, tangents are refused).  form "int8":
    codes int8 [..., d] and scales uint8 [..., ceil(d / 32)] as act_encode writes them, for act_decode; "e4m3":
    codes float8_e4m3fn [..., d] that stand for code * scale, scales float32 [...]."""
    if form not in _FORMS:
        raise ValueError("form must be 'int8' or 'e4m3'")
    dev, code, r_code, w_code = _check_branch(x, residual, weight)
    x, residual, weight = _aligned(x), _aligned(residual), _aligned(weight)
    d, lead = x.shape[-1], x.shape[:-1]
    h = _like(residual)
    if form == "int8":
        codes, scales = _new(x.shape, torch.int8, dev), _new((*lead, -(-d // ACT_BLOCK)), torch.uint8, dev)
    else:
        codes, scales = _new(x.shape, torch.float8_e4m3fn, dev), _new(lead, torch.float32, dev)
    _call(dev, load_library().ckl_add_norm_quant, x.data_ptr(), code, residual.data_ptr(), r_code, _rows(x), d,
          weight.data_ptr(), w_code, eps, _FORMS[form], h.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return codes, scales, h
