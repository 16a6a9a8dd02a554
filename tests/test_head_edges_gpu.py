"""Gradients of log probabilities from states and head on the GPU, cut into blocks of rows and of words."""
import math

import pytest
import torch

import chunked_kl_loss_amd as ckl
from tests.test_head_gpu import check, inputs
from tests.test_logprob_gpu import DT, gen, normal, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,chunk", [(3000, 72, 5000, 100), (2999, 264, 3001, 64), (5000, 64, 1100, 700),
                                         (1025, 520, 9000, 300)])
def test_gradients_in_blocks_of_rows_and_words(T, d, V, chunk, dtype, masked):
    H, W, tok = inputs(T, d, V, DT[dtype], 3)
    mask = (torch.rand(T, generator=gen(1)) < 0.6) if masked else None
    if masked:
        H[~mask] = math.nan
    check(H, W, tok, mask, chunk=chunk)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V,chunk", [(3000, 72, 5000, 100), (5000, 64, 1100, 700), (1500, 72, 300, 256)])
def test_gradients_of_either_type_in_blocks(T, d, V, chunk, dtype, masked):
    H, W, tok = (t.cuda() for t in inputs(T, d, V, DT[dtype], 5))
    mask = (torch.rand(T, generator=gen(1)) < 0.6).cuda() if masked else None
    lp, ent, lse = ckl.head_logprobs_forward(H, W, tok, mask)
    a, b = normal((T,), torch.float32, 1).cuda(), normal((T,), torch.float32, 2, 0.3).cuda()

    def grads(**kw):
        return ckl.head_logprobs_backward(a, b, H, W, tok, lse, ent, mask, chunk, **kw)
    dh, dw = grads(dh_dtype=torch.float32)
    for _ in range(2):
        dh16, dw16 = grads(dh_dtype=torch.bfloat16, dw_dtype=torch.bfloat16)
        assert same_bits(dh16, dh.bfloat16()) and same_bits(dw16, dw.bfloat16())
    assert same_bits(grads(dh_dtype=torch.float32, need_dw=False)[0], dh)
    if masked:
        assert not dh[~mask].any()


@pytest.mark.parametrize("share", [0.0, 0.1, 1.0])
def test_blocks_past_the_last_kept_row(share):
    # whole blocks of rows hold no kept one
    T, d, V = 3000, 72, 3000
    H, W, tok = inputs(T, d, V, torch.bfloat16, 7)
    mask = torch.arange(T) >= T * (1 - share)
    H[~mask] = math.nan
    check(H, W, tok, mask, chunk=100)
