"""Fused chunked forward-KL distillation loss for AMD MI355X (gfx950).

The loss of a student output head against a sparse cached top-K teacher,
computed by hand-written HIP kernels behind the C ABI in include/ckl.h:

    loss, lse, _ = forward(H, W, idx, tlogit, mask, chunk)
    dH, dW = backward(H, W, idx, tlogit, mask, lse, grad_loss, chunk)

or, in one call without recomputing the logits,

    loss, lse, _, dH, dW = forward_backward(H, W, idx, tlogit, mask, grad_loss, chunk)

or, through autograd, ``chunked_kl_loss(H, W, idx, tlogit, mask, chunk, fused=False)``.

Around the loss: ``teacher_topk`` makes the sparse teacher from full logits;
``embedding`` is the lookup in a table of the head's shape, whose gradient
``embedding_backward`` can add to the head's; ``act_encode`` / ``act_decode``
hold activations in 8 bits, and ``rms_norm_8bit`` is a norm that saves its
input so.  Between a model's last block and the loss: ``dropout``, whose mask is
formed again instead of stored, ``add_rms_norm`` and ``add_norm_quant``, the norm
with the residual's addition; ``head_logprobs`` and ``token_logprobs``, the log
probabilities of given tokens from states and head or from logits.
"""
from ._binding import (  # noqa: F401
    CKL_BF16,
    CKL_F32,
    CklError,
    Problem,
    backward,
    backward_plan,
    forward,
    forward_backward,
    fused_plan,
    scale_cast,
    load_library,
    make_problem,
    shard_combine,
    shard_forward,
    timing_enable,
    timing_read,
    workspace_size,
)
from .autograd import (  # noqa: F401
    AddNormQuant,
    AddRMSNorm,
    ChunkedKLLoss,
    ChunkedKLLoss8Bit,
    Dropout,
    Embedding,
    FusedChunkedKLLoss,
    HeadLogprobs,
    RMSNorm8Bit,
    TokenLogprobs,
    add_norm_quant,
    add_rms_norm,
    chunked_kl_loss,
    dropout,
    embedding,
    head_logprobs,
    rms_norm_8bit,
    token_logprobs,
)
from .ops import (  # noqa: F401
    act_decode,
    act_encode,
    add_norm_backward,
    add_norm_forward,
    dropout_forward,
    embedding_backward,
    embedding_forward,
    head_logprobs_backward,
    head_logprobs_forward,
    norm_backward,
    norm_forward,
    teacher_topk,
    token_logprobs_backward,
    token_logprobs_forward,
)
