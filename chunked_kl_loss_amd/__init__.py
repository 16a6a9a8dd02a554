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
input so.
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
    ChunkedKLLoss,
    ChunkedKLLoss8Bit,
    Embedding,
    FusedChunkedKLLoss,
    RMSNorm8Bit,
    chunked_kl_loss,
    embedding,
    rms_norm_8bit,
)
from .ops import (  # noqa: F401
    act_decode,
    act_encode,
    embedding_backward,
    embedding_forward,
    norm_backward,
    norm_forward,
    teacher_topk,
)
