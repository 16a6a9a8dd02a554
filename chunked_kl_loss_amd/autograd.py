"""torch.autograd wrappers.

ChunkedKLLoss: the forward saves (H, W, idx, tlogit, mask, lse) and the
backward recomputes the logit tiles inside libckl.

FusedChunkedKLLoss: one library call in the forward computes the loss and the
fp32 gradients of the loss itself (no recompute); the backward multiplies them
by the incoming gradient and rounds them once to the dtypes of H and W, in the
library (ckl_scale_cast).  When neither H nor W needs a gradient the forward
computes the loss alone.

ChunkedKLLoss8Bit: as ChunkedKLLoss, but the backward's hidden states are
rebuilt from 8 bits per value, and it multiplies their logits once more for
their log-sum-exp; with a norm before the head, the norm's input is what is
saved, once for the norm's gradient and the head's.

Embedding and RMSNorm8Bit: the embedding by a table of the head's shape, and the
norm that saves its input in 8 bits."""
from __future__ import annotations

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _binding, ops


class ChunkedKLLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, idx, tlogit, mask=None, chunk: int = 2048, teacher_form: int = 0):
        loss, lse, _ = _binding.forward(H, W, idx, tlogit, mask, chunk=chunk, teacher_form=teacher_form)
        ctx.save_for_backward(H, W, idx, tlogit, lse, mask if mask is not None else torch.empty(0))
        ctx.has_mask = mask is not None
        ctx.chunk = chunk
        ctx.teacher_form = teacher_form
        return loss[0]

    @staticmethod
    def backward(ctx, grad):
        need_h, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if not (need_h or need_w):
            return None, None, None, None, None, None, None
        H, W, idx, tlogit, lse, mask = ctx.saved_tensors
        mask = mask if ctx.has_mask else None
        g = grad.reshape(1).to(torch.float32)
        dH, dW = _binding.backward(H, W, idx, tlogit, mask, lse, g, chunk=ctx.chunk,
                                   dh_dtype=H.dtype, dw_dtype=W.dtype, teacher_form=ctx.teacher_form)
        return (dH if need_h else None), (dW if need_w else None), None, None, None, None, None


class FusedChunkedKLLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, idx, tlogit, mask=None, chunk: int = 2048, teacher_form: int = 0,
                dw_group_rows: int = 0):
        need_h, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        ctx.dtypes = (H.dtype, W.dtype)
        if not (need_h or need_w):
            loss, _, _ = _binding.forward(H, W, idx, tlogit, mask, chunk=chunk, teacher_form=teacher_form)
            ctx.save_for_backward(torch.empty(0, device=H.device), torch.empty(0, device=H.device))
            return loss[0]
        # gradients of the loss itself, kept in fp32 until the incoming
        # gradient is known
        loss, _, _, dH, dW = _binding.forward_backward(H, W, idx, tlogit, mask, None, chunk=chunk,
                                                       dh_dtype=torch.float32, dw_dtype=torch.float32,
                                                       teacher_form=teacher_form, dw_group_rows=dw_group_rows)
        ctx.save_for_backward(dH if need_h else torch.empty(0, device=H.device),
                              dW if need_w else torch.empty(0, device=H.device))
        return loss[0]

    @staticmethod
    def backward(ctx, grad):
        dH32, dW32 = ctx.saved_tensors
        h_dtype, w_dtype = ctx.dtypes
        g = grad.reshape(1).to(torch.float32)
        dH = dW = None
        if ctx.needs_input_grad[0]:
            dH = _binding.scale_cast(dH32, torch.empty(dH32.shape, dtype=h_dtype, device=dH32.device), g)
        if ctx.needs_input_grad[1]:
            dW = _binding.scale_cast(dW32, torch.empty(dW32.shape, dtype=w_dtype, device=dW32.device), g)
        return dH, dW, None, None, None, None, None, None


class ChunkedKLLoss8Bit(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, idx, tlogit, mask, chunk, teacher_form, norm_weight, norm_eps):
        need = any(ctx.needs_input_grad)
        rstd = codes = exps = None
        dtype = H.dtype
        if norm_weight is not None:
            H, codes, exps, rstd = ops.norm_forward(H, norm_weight, norm_eps, save=need)
        elif need:
            codes, exps = ops.act_encode(H)
        loss, _, _ = _binding.forward(H, W, idx, tlogit, mask, chunk=chunk, teacher_form=teacher_form)
        if need:
            if norm_weight is not None and mask is not None:
                ops.norm_drop_rows(exps, rstd, mask)
            ctx.save_for_backward(codes, exps, rstd, norm_weight, W, idx, tlogit, mask)
        ctx.chunk, ctx.teacher_form, ctx.dtype = chunk, teacher_form, dtype
        return loss[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        codes, exps, rstd, norm_weight, W, idx, tlogit, mask = ctx.saved_tensors
        H = ops.act_decode(codes, exps, rstd, norm_weight, dtype=ctx.dtype)
        # The log-sum-exp of these states, not of the exact ones: with theirs a row's probabilities would add up to
        # exp(difference), which outweighs p - q where the student is sure (4096 x 2048 bf16 states, a teacher whose
        # logits are 0.1 away: dH off by 0.49 of its norm at a top probability of 0.989, by 21 at 0.9998; so by 0.01).
        _, lse, _ = _binding.forward(H, W, idx, tlogit, mask, chunk=ctx.chunk, teacher_form=ctx.teacher_form)
        g = grad.reshape(1).to(torch.float32)
        dH, dW = _binding.backward(H, W, idx, tlogit, mask, lse, g, chunk=ctx.chunk, dh_dtype=ctx.dtype,
                                   dw_dtype=W.dtype, teacher_form=ctx.teacher_form)
        dnorm = None
        if norm_weight is not None and (ctx.needs_input_grad[0] or ctx.needs_input_grad[7]):
            dH, dnorm = ops.norm_backward(dH, codes, exps, rstd, norm_weight)
        need = ctx.needs_input_grad
        return (dH if need[0] else None, dW if need[1] else None, None, None, None, None, None,
                dnorm if need[7] else None, None)


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, W, tokens, scale: float = 1.0):
        ctx.save_for_backward(tokens)
        ctx.V, ctx.dtype, ctx.scale = W.shape[0], W.dtype, scale
        return ops.embedding_forward(W, tokens, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        (tokens,) = ctx.saved_tensors
        dW = ops.embedding_backward(grad.contiguous(), tokens, ctx.V, ctx.scale, dw_dtype=ctx.dtype)
        return dW, None, None


class RMSNorm8Bit(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps: float = 1e-6, mask=None):
        y, saved = ops.norm_forward_saving(x, weight, eps, mask)
        ctx.save_for_backward(saved, weight)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        saved, weight = ctx.saved_tensors
        dx, dweight = ops.norm_backward_saved(grad.contiguous(), saved, weight)
        return dx, dweight, None, None


def _needs_function(requires_grad: bool) -> bool:
    """Whether a call whose inputs require a gradient or not has to go through its Function: where a gradient is
    asked for, and in a forward-mode context, where the Function refuses tangents (the raw call would drop them)."""
    return forward_ad._current_level >= 0 or (requires_grad and torch.is_grad_enabled())


def embedding(W, tokens, scale: float = 1.0):
    """scale * W[tokens], differentiable with respect to the table W [V, d] (the output head's, when tied).
    tokens: int32 / int64 of any shape; a token outside [0, V) gives a zero row and no gradient."""
    W, tokens = W.contiguous(), tokens.contiguous()
    if not _needs_function(W.requires_grad):
        return ops.embedding_forward(W, tokens, scale)
    return Embedding.apply(W, tokens, scale)


def _norm(x, weight, eps, mask=None):
    """rms_norm_8bit; with a mask [T], rows of x [T, d] that are masked out add nothing to the weight's gradient
    whatever they hold (their gradients have to be zero)."""
    x, weight = x.contiguous(), weight.contiguous()
    if not _needs_function(x.requires_grad or weight.requires_grad):
        return ops.norm_forward(x, weight, eps, save=False)[0]
    return RMSNorm8Bit.apply(x, weight, eps, mask)


def rms_norm_8bit(x, weight, eps: float = 1e-6):
    """RMS norm of the last dimension, differentiable with respect to x [..., d] and weight [d].  The output is
    that of the exact x; the backward pass reads x from 8 bits (ops.act_encode), so that the norm keeps d bytes a
    row instead of x."""
    return _norm(x, weight, eps)


def chunked_kl_loss(H, W, idx, tlogit, mask=None, chunk: int = 2048, fused: bool = False, teacher_form: int = 0,
                    dw_group_rows: int = 0, save_8bit: bool = False, norm_weight=None, norm_eps: float = 1e-6):
    """Mean forward KL(teacher || student) over unmasked rows, differentiable
    with respect to H and W.  fused=True computes the gradients together with
    the loss (one pass over the logits; it keeps the logit gradients of up to
    dw_group_rows rows, 0 = the library default of min(16384, 8 chunks), so
    a smaller value holds less memory and updates dW more often).
    teacher_form 1: tlogit holds truncated teacher log-probabilities, used as
    given (teacher mass below one).

    save_8bit=True: the loss is that of the exact H, but the backward pass
    rebuilds H from 8 bits per value (ops.act_encode), so that d bytes a row are
    kept from forward to backward instead of H, and gives the gradient at the
    rebuilt H (it multiplies the logits once more for their log-sum-exp:
    32768 x 2880 over 201088 words 149 ms a step, 121 without).  norm_weight [d] (with
    save_8bit): H is the input of an RMS norm before the head, whose input is
    saved instead, once for both; differentiable with respect to norm_weight
    too.  fused=True keeps gradients instead of H, so there save_8bit goes with
    norm_weight only.  Masked rows of H may hold anything.

    Leading batch dimensions are flattened into rows: H [..., d], idx and
    tlogit [..., K], mask [...].  The library takes contiguous tensors, int32
    indices and fp32 teacher values: other layouts and integer / float types
    are converted here (no copy when they already match; H and W keep their
    dtype, which selects the bf16 or fp32 path)."""
    d, K = H.shape[-1], idx.shape[-1]
    if idx.shape[:-1] != H.shape[:-1] or tlogit.shape != idx.shape or (mask is not None and mask.shape != H.shape[:-1]):
        raise ValueError("H [..., d], idx and tlogit [..., K] and mask [...] must share their leading dimensions")
    H, W = H.reshape(-1, d).contiguous(), W.contiguous()
    idx = idx.reshape(-1, K).to(torch.int32).contiguous()
    tlogit = tlogit.reshape(-1, K).to(torch.float32).contiguous()
    if mask is not None:
        mask = mask.reshape(-1).contiguous()
    if norm_weight is not None and not save_8bit:
        raise ValueError("norm_weight needs save_8bit=True: the norm saves its input in 8 bits")
    if fused and save_8bit:
        if norm_weight is None:
            raise ValueError("fused=True keeps no hidden states: save_8bit there needs norm_weight")
        H = _norm(H, norm_weight, norm_eps, mask)
    if save_8bit and not fused:
        nw = None if norm_weight is None else norm_weight.contiguous()
        if not torch.is_grad_enabled():  # nothing is saved (a Function sees the leaves' requires_grad all the same)
            H = H if nw is None else _norm(H, nw, norm_eps)
            return ChunkedKLLoss.apply(H, W, idx, tlogit, mask, chunk, teacher_form)
        return ChunkedKLLoss8Bit.apply(H, W, idx, tlogit, mask, chunk, teacher_form, nw, norm_eps)
    if fused:
        return FusedChunkedKLLoss.apply(H, W, idx, tlogit, mask, chunk, teacher_form, dw_group_rows)
    return ChunkedKLLoss.apply(H, W, idx, tlogit, mask, chunk, teacher_form)
