"""Log probabilities of given tokens, from logits and from states and head, without a GPU: what the C ABI refuses on
the host (nothing is launched), workspaces, and what the Python layer refuses before any call."""
import ctypes

import pytest
import torch

import chunked_kl_loss_amd as ckl
from tests.test_operators_abi import BIG, INV, P, UNS, WSP, lib, size  # noqa: F401


def rows(lib, z=P[0], dtype=1, T=4, V=1000, tok=P[1], nb=8, top=5, mask=P[2], lp=P[3], ent=P[4], lse=P[5], idx=P[6],  # noqa: F811
         val=P[7], ws=P[8], ws_bytes=BIG):
    return lib.ckl_token_logprobs(z, dtype, T, V, tok, nb, top, mask, lp, ent, lse, idx, val, ws, ws_bytes, None)


def rows_b(lib, z=P[0], dtype=1, T=4, V=1000, tok=P[1], nb=8, mask=P[2], lse=P[3], ent=P[4], a=P[5], b=P[6], dz=P[7]):  # noqa: F811
    return lib.ckl_token_logprobs_backward(z, dtype, T, V, tok, nb, mask, lse, ent, a, b, dz, None)


def head(lib, H=P[0], W=P[1], dtype=1, T=4, d=64, V=1000, tok=P[2], nb=8, mask=P[3], chunk=64, lp=P[4], ent=P[5],  # noqa: F811
         lse=P[6], ws=P[7], ws_bytes=BIG):
    return lib.ckl_head_logprobs(H, W, dtype, T, d, V, tok, nb, mask, chunk, lp, ent, lse, ws, ws_bytes, None)


def head_b(lib, H=P[0], W=P[1], dtype=1, T=4, d=64, V=1000, tok=P[2], nb=8, mask=P[3], chunk=64, lse=P[4], ent=P[5],  # noqa: F811
           a=P[6], b=P[7], dH=P[8], ht=1, dW=P[9], wt=0, ws=P[10], ws_bytes=BIG):
    return lib.ckl_head_logprobs_backward(H, W, dtype, T, d, V, tok, nb, mask, chunk, lse, ent, a, b, dH, ht, dW, wt, ws,
                                          ws_bytes, None)


TOKENS = [(dict(nb=2), INV), (dict(tok=P[11] + 4), INV), (dict(nb=4, tok=P[11] + 2), INV), (dict(tok=None), INV),
          (dict(dtype=2), INV), (dict(T=-1), INV), (dict(T=4000001), UNS), (dict(V=0), INV), (dict(V=4000001), UNS),
          (dict(ent=None), INV), (dict(ent=P[11] + 2), INV), (dict(lse=P[11] + 1), INV)]


@pytest.mark.parametrize("kw,status", TOKENS + [
    (dict(top=-1), INV), (dict(top=1001), INV), (dict(V=9000, top=4097), UNS), (dict(T=2000000, V=5000, top=4096), UNS),
    (dict(z=None), INV), (dict(lp=None), INV), (dict(lse=None), INV), (dict(idx=None), INV), (dict(val=None), INV),
    (dict(z=P[0] + 2), INV), (dict(ws=P[8] + 8), INV), (dict(idx=P[6] + 2), INV), (dict(V=201088, top=100, ws=None), WSP),
    (dict(V=201088, top=100, ws_bytes=16), WSP), (dict(lp=P[4]), INV), (dict(lse=P[0]), INV), (dict(idx=P[1]), INV),
    (dict(val=P[2]), INV), (dict(V=201088, top=100, ws=P[3]), INV)])
def test_token_logprobs_refusals(lib, kw, status):  # noqa: F811
    assert rows(lib, **kw) == status
    assert lib.ckl_last_error()


@pytest.mark.parametrize("kw,status", TOKENS + [
    (dict(z=None), INV), (dict(lse=None), INV), (dict(dz=None), INV), (dict(z=P[0] + 8), INV), (dict(dz=P[7] + 2), INV),
    (dict(a=P[5] + 2), INV), (dict(b=P[6] + 2), INV), (dict(dz=P[0]), INV), (dict(dz=P[3]), INV), (dict(dz=P[2]), INV)])
def test_token_logprobs_backward_refusals(lib, kw, status):  # noqa: F811
    assert rows_b(lib, **kw) == status
    assert lib.ckl_last_error()


@pytest.mark.parametrize("kw,status", TOKENS + [
    (dict(d=12), INV), (dict(d=0), INV), (dict(d=65544), UNS), (dict(chunk=0), INV), (dict(H=None), INV), (dict(W=None), INV),
    (dict(lp=None), INV), (dict(lse=None), INV), (dict(H=P[0] + 8), INV), (dict(W=P[1] + 2), INV), (dict(lp=P[4] + 2), INV),
    (dict(ws=None), WSP), (dict(ws_bytes=64), WSP), (dict(ws=P[7] + 4), INV), (dict(lp=P[0]), INV), (dict(ent=P[6]), INV),
    (dict(lse=P[2]), INV), (dict(ws=P[3]), INV)])
def test_head_logprobs_refusals(lib, kw, status):  # noqa: F811
    assert head(lib, **kw) == status
    assert lib.ckl_last_error()


@pytest.mark.parametrize("kw,status", TOKENS + [
    (dict(d=12), INV), (dict(chunk=-3), INV), (dict(ht=2), INV), (dict(wt=2), INV), (dict(H=None), INV), (dict(W=None), INV),
    (dict(lse=None), INV), (dict(dH=None, dW=None), INV), (dict(dH=P[8] + 8), INV), (dict(dW=P[9] + 4), INV),
    (dict(a=P[6] + 1), INV), (dict(ws=None), WSP), (dict(ws_bytes=64), WSP), (dict(dH=P[0]), INV), (dict(dW=P[1]), INV),
    (dict(dH=P[9]), INV), (dict(ws=P[8]), INV), (dict(dW=P[7]), INV)])
def test_head_logprobs_backward_refusals(lib, kw, status):  # noqa: F811
    assert head_b(lib, **kw) == status
    assert lib.ckl_last_error()


def test_nothing_to_do(lib):  # noqa: F811
    assert rows(lib, T=0, z=None, tok=None, lp=None, ent=None, lse=None, idx=None, val=None, ws=None) == 0
    assert rows_b(lib, T=0, z=None, tok=None, lse=None, ent=None, dz=None) == 0
    assert head(lib, T=0, H=None, tok=None, lp=None, ent=None, lse=None, ws=None) == 0
    assert size(lib.ckl_head_workspace_size, 0, 64, 1000, 64, 1, 1, 0, 1, 1) == 0


def test_workspaces(lib):  # noqa: F811
    ws = lib.ckl_logprob_workspace_size
    assert size(ws, 1, 201088, 0) == 0 and size(ws, 1, 2048, 64) == 0 and size(ws, 4096, 201088, 100) == 0 and 0 < size(ws, 1, 201088, 100) < 1 << 20
    assert ws(1, 10, 11, ctypes.byref(ctypes.c_size_t())) == INV and ws(1, 10, 1, None) == INV
    hw = lib.ckl_head_workspace_size
    # the forward keeps per-row arrays; a mask adds a copy of the states
    plain, masked = (size(hw, 32768, 2880, 201088, 2048, 1, 1, 0, m, 0) for m in (0, 1))
    assert plain < 4 << 20 and 32768 * 2880 * 2 <= masked - plain < 32768 * 2880 * 2 + (1 << 20)
    # the backward holds about chunk x V gradients, W^T of a block of them, and dH and H^T besides; an fp32 dW only
    # where there are several blocks of rows, or the inputs are fp32 and dW is bf16
    small, large = (size(hw, 32768, 2880, 201088, c, 1, 1, 0, 0, 1) for c in (512, 4096))
    assert small < large < 1.1 * (32768 * 2880 * 6 + 4096 * 201088 * 2 + 201088 * 2880 * 2)
    add = [size(hw, T, 2880, 201088, 2048, t, 1, 1, 0, 1) - size(hw, T, 2880, 201088, 2048, t, 1, 0, 0, 1)
           for T, t in ((2048, 1), (32768, 1), (2048, 0))]
    assert add == [0, 201088 * 2880 * 4, 201088 * 2880 * 4]
    for bad in ((4, 64, 1000, 64, 1, 1, 0, 2, 0), (4, 64, 1000, 64, 1, 1, 0, 0, 2), (4, 64, 1000, 0, 1, 1, 0, 0, 0),
                (4, 60, 1000, 64, 1, 1, 0, 0, 0), (4, 64, 1000, 64, 3, 1, 0, 0, 0)):
        assert hw(*bad, ctypes.byref(ctypes.c_size_t())) == INV
    assert hw(4, 64, 1000, 64, 1, 1, 0, 0, 0, None) == INV


def test_python_layer_refuses():
    z, tok = torch.zeros(4, 9), torch.zeros(4, dtype=torch.int64)
    H, W = torch.zeros(4, 16), torch.zeros(9, 16)
    for call in (lambda: ckl.token_logprobs(z, tok), lambda: ckl.head_logprobs(H, W, tok)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="share d"):
        ckl.head_logprobs(H, W[:, :8], tok)
    with pytest.raises(ValueError, match="share d"):
        ckl.head_logprobs(H, W.bfloat16(), tok)
    with pytest.raises(ValueError):
        ckl.token_logprobs(torch.zeros(()), torch.zeros((), dtype=torch.int64))
