"""The operators around the loss without a GPU: sizes and buffers the C ABI
refuses on the host (nothing is launched), and what the Python layer refuses
before any call."""
import ctypes
import os

import pytest
import torch

import chunked_kl_loss_amd as ckl
from chunked_kl_loss_amd import _binding as B

INV, UNS, WSP = B.CKL_ERR_INVALID_ARG, B.CKL_ERR_UNSUPPORTED, B.CKL_ERR_WORKSPACE
FAR = 1 << 34  # buffers this far apart never overlap
P = [(1 << 40) + i * FAR for i in range(12)]  # never dereferenced: every call below fails its checks
BIG = 1 << 33


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from chunked_kl_loss_amd import build
        build.build()
    return B.load_library()


def size(fn, *args):
    out = ctypes.c_size_t(0)
    B.check(fn(*args, ctypes.byref(out)))
    return out.value


def topk(lib, logits=P[0], dtype=1, T=4, V=1000, K=10, form=0, mask=P[1], idx=P[2], val=P[3], lse=P[4], ws=P[5],
         ws_bytes=BIG):
    return lib.ckl_teacher_topk(logits, dtype, T, V, K, form, mask, idx, val, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(T=4000001), UNS), (dict(V=0), INV), (dict(V=4000001), UNS), (dict(K=0), INV),
    (dict(K=1001), INV), (dict(V=9000, K=4097), UNS), (dict(T=2000000, V=5000, K=4096), UNS), (dict(dtype=2), INV),
    (dict(form=2), INV), (dict(logits=None), INV), (dict(idx=None), INV), (dict(val=None), INV), (dict(lse=None), INV),
    (dict(logits=P[0] + 2), INV), (dict(idx=P[2] + 4), INV), (dict(lse=P[4] + 2), INV), (dict(ws=P[5] + 8), INV),
    (dict(V=201088, ws=None), WSP), (dict(V=201088, ws_bytes=16), WSP),
    (dict(idx=P[3]), INV), (dict(idx=P[0]), INV), (dict(lse=P[1]), INV), (dict(V=201088, ws=P[2]), INV),
])
def test_topk_refusals(lib, kw, status):
    assert topk(lib, **kw) == status
    assert lib.ckl_last_error()


def test_topk_workspace(lib):
    assert size(lib.ckl_topk_workspace_size, 4096, 201088, 100) == 0   # rows enough: no segments
    one = size(lib.ckl_topk_workspace_size, 1, 201088, 100)
    assert 0 < one < 1 << 20
    assert size(lib.ckl_topk_workspace_size, 0, 201088, 100) == 0
    assert lib.ckl_topk_workspace_size(1, 10, 11, ctypes.byref(ctypes.c_size_t())) == INV
    assert lib.ckl_topk_workspace_size(1, 10, 1, None) == INV


def emb_f(lib, W=P[0], dtype=1, V=100, d=64, off=0, tok=P[1], nb=8, T=10, out=P[2]):
    return lib.ckl_embedding_forward(W, dtype, V, d, off, tok, nb, T, 1.0, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(T=4000001), UNS), (dict(V=0), INV), (dict(V=4000001), UNS), (dict(d=12), INV),
    (dict(d=0), INV), (dict(d=65544), UNS), (dict(off=-1), INV), (dict(dtype=3), INV), (dict(nb=2), INV),
    (dict(W=None), INV), (dict(tok=None), INV), (dict(out=None), INV), (dict(W=P[0] + 8), INV),
    (dict(tok=P[1] + 4), INV), (dict(tok=P[1] + 2, nb=4), INV), (dict(out=P[0]), INV), (dict(out=P[1]), INV),
])
def test_embedding_forward_refusals(lib, kw, status):
    assert emb_f(lib, **kw) == status
    assert lib.ckl_last_error()


def emb_b(lib, dY=P[0], dtype=1, T=10, d=64, tok=P[1], nb=8, V=100, off=0, dW=P[2], dwt=0, acc=0, ws=P[3],
          ws_bytes=BIG):
    return lib.ckl_embedding_backward(dY, dtype, T, d, tok, nb, V, off, 1.0, dW, dwt, acc, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(V=0), INV), (dict(d=12), INV), (dict(off=-1), INV), (dict(dtype=3), INV),
    (dict(dwt=2), INV), (dict(acc=2), INV), (dict(nb=1), INV), (dict(dY=None), INV), (dict(tok=None), INV),
    (dict(dW=None), INV), (dict(dW=None, T=0), INV), (dict(dY=P[0] + 4), INV), (dict(dW=P[2] + 4), INV),
    (dict(tok=P[1] + 4), INV), (dict(T=1000, ws=None), WSP), (dict(T=1000, ws_bytes=64), WSP),
    (dict(dW=P[0]), INV), (dict(T=1000, ws=P[1]), INV), (dict(T=1000, ws=P[2]), INV),
])
def test_embedding_backward_refusals(lib, kw, status):
    assert emb_b(lib, **kw) == status
    assert lib.ckl_last_error()


@pytest.mark.parametrize("T", [1, 64, 4096, 8192, 8193, 300000, 4000000])
@pytest.mark.parametrize("V", [1, 511, 512, 262143, 262144, 4000000])
def test_embedding_workspace_grows_with_rows_only(lib, T, V):
    n = size(lib.ckl_embedding_workspace_size, T, 64, V)
    # (a prompt of up to 256 tokens needs none)
    assert (0 if T <= 256 else 8 * T) <= n <= 200 * T + (1 << 16)


def test_small_refusals_of_the_8bit_calls(lib):
    enc = lambda x=P[0], t=1, T=4, d=64, c=P[1], e=P[2]: lib.ckl_act_encode(x, t, T, d, c, e, None)  # noqa: E731
    for kw in (dict(T=-1), dict(d=12), dict(t=2), dict(x=None), dict(c=None), dict(e=None), dict(x=P[0] + 8),
               dict(c=P[1] + 4), dict(c=P[0]), dict(e=P[1])):
        assert enc(**kw) == INV
    assert enc(d=65544) == UNS

    def dec(c=P[0], e=P[1], T=4, d=64, r=None, w=None, wt=0, o=P[4], ot=1):
        return lib.ckl_act_decode(c, e, T, d, r, w, wt, o, ot, None)
    for kw in (dict(T=-1), dict(d=4), dict(c=None), dict(e=None), dict(o=None), dict(ot=5), dict(wt=5), dict(r=P[2]),
               dict(w=P[3]), dict(c=P[0] + 8), dict(o=P[4] + 8), dict(o=P[0]), dict(r=P[2] + 2, w=P[3]),
               dict(r=P[2], w=P[3] + 4), dict(r=P[2], w=P[4])):
        assert dec(**kw) == INV

    def nf(x=P[0], t=1, T=4, d=64, w=P[1], wt=1, eps=1e-6, y=P[2], c=P[3], e=P[4], r=P[5]):
        return lib.ckl_norm_forward(x, t, T, d, w, wt, eps, y, c, e, r, None)
    for kw in (dict(T=-1), dict(d=20), dict(t=4), dict(wt=4), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(x=None), dict(w=None), dict(y=None), dict(c=None), dict(e=None),
               dict(r=None), dict(c=None, e=None), dict(x=P[0] + 2), dict(r=P[5] + 1), dict(y=P[0]), dict(c=P[2]),
               dict(r=P[1])):
        assert nf(**kw) == INV

    def nb(dy=P[0], t=1, T=4, d=64, c=P[1], e=P[2], r=P[3], w=P[4], wt=1, dx=P[5], dw=P[6], ws=P[7], n=BIG):
        return lib.ckl_norm_backward(dy, t, T, d, c, e, r, w, wt, dx, dw, ws, n, None)
    for kw in (dict(T=-1), dict(d=20), dict(t=4), dict(wt=4), dict(dy=None), dict(c=None), dict(e=None), dict(r=None),
               dict(w=None), dict(dx=None), dict(dw=None), dict(T=0, dw=None), dict(dy=P[0] + 2), dict(dw=P[6] + 8),
               dict(dx=P[0]), dict(dw=P[5]), dict(ws=P[0])):
        assert nb(**kw) == INV
    assert nb(ws=None) == WSP and nb(n=0) == WSP


def test_calls_without_rows_touch_nothing(lib):
    assert topk(lib, T=0, logits=None, mask=None, idx=None, val=None, lse=None, ws=None, ws_bytes=0) == B.CKL_OK
    assert emb_f(lib, T=0, W=None, tok=None, out=None) == B.CKL_OK
    assert lib.ckl_act_encode(None, 1, 0, 64, None, None, None) == B.CKL_OK
    assert lib.ckl_act_decode(None, None, 0, 64, None, None, 0, None, 1, None) == B.CKL_OK
    assert lib.ckl_norm_forward(None, 1, 0, 64, None, 1, 1e-6, None, None, None, None, None) == B.CKL_OK


def test_python_layer_refuses_host_tensors_and_mismatches():
    x, w = torch.zeros(4, 64), torch.ones(64)
    tok = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: ckl.teacher_topk(x, 3), lambda: ckl.embedding(x, tok), lambda: ckl.embedding_forward(x, tok),
                 lambda: ckl.embedding_backward(x, tok, 10), lambda: ckl.act_encode(x),
                 lambda: ckl.act_decode(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)),
                 lambda: ckl.norm_forward(x, w), lambda: ckl.rms_norm_8bit(x, w),
                 lambda: ckl.norm_backward(x, x, x, w, w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        ckl.embedding_backward(x, torch.zeros(5, dtype=torch.int64), 10)
    idx, tl = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="save_8bit"):
        ckl.chunked_kl_loss(x, x, idx, tl, norm_weight=w)
    with pytest.raises(ValueError, match="norm_weight"):
        ckl.chunked_kl_loss(x, x, idx, tl, fused=True, save_8bit=True)
