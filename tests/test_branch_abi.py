"""Dropout and the RMS norm with the residual's addition without a GPU: what the C ABI refuses on the host, what the
Python layer refuses before any call, and the generator that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_kl_loss_amd as ckl
from chunked_kl_loss_amd import _binding as B
from tests.philox import keep_mask, philox4x32
from tests.test_operators_abi import BIG, INV, P, UNS, WSP, lib, size  # noqa: F401


def test_philox_known_answers():
    # the answers that the authors publish with the algorithm
    for c, k, want in [
            ([0] * 4, [0] * 2, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
            ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
            ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
             [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])]:
        assert [int(x[0]) for x in philox4x32([np.array([v]) for v in c], k)] == want


def test_keep_mask_shares():
    for p in (0.0, 0.1, 0.5, 1.0):
        keep, scale = keep_mask(1 << 16, p, 1, 2)
        q = 1 - round(p * 65536) / 65536
        assert abs(keep.mean() - q) < 6 * (q * (1 - q) / (1 << 16)) ** 0.5 + 1e-12
        assert scale == (1 / q if q else 0.0)


def drop(lib, x=P[0], dtype=1, n=100, p=0.5, seed=1, offset=0, state=None, out=P[1]):  # noqa: F811
    return lib.ckl_dropout(x, dtype, n, p, seed, offset, state, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INV), (dict(n=(1 << 36) + 1), UNS), (dict(dtype=2), INV), (dict(p=-0.1), INV), (dict(p=1.1), INV),
    (dict(p=float("nan")), INV), (dict(x=None), INV), (dict(out=None), INV), (dict(x=P[0] + 2), INV),
    (dict(out=P[1] + 8), INV), (dict(out=P[0]), INV), (dict(out=P[0] + 192), INV), (dict(state=P[2] + 4), INV),
    (dict(state=P[1] + 16), INV)])
def test_dropout_refusals(lib, kw, status):  # noqa: F811
    assert drop(lib, **kw) == status
    assert lib.ckl_last_error()


def fwd(lib, x=P[0], xt=1, res=P[1], rt=1, T=4, d=64, w=P[2], wt=1, eps=1e-6, p=0.1, seed=1, off=0, state=None,  # noqa: F811
        h=P[3], y=P[4], rstd=P[5]):
    return lib.ckl_add_norm_forward(x, xt, res, rt, T, d, w, wt, eps, p, seed, off, state, h, y, rstd, None)


def bwd(lib, dy=P[0], xt=1, dh=P[1], rt=1, T=4, d=64, h=P[2], rstd=P[3], w=P[4], wt=1, p=0.1, seed=1, off=0,  # noqa: F811
        state=None, dx=P[5], dr=P[6], dw=P[7], ws=P[8], ws_bytes=BIG):
    return lib.ckl_add_norm_backward(dy, xt, dh, rt, T, d, h, rstd, w, wt, p, seed, off, state, dx, dr, dw, ws,
                                     ws_bytes, None)


def quant(lib, x=P[0], xt=1, res=P[1], rt=1, T=4, d=64, w=P[2], wt=1, eps=1e-6, form=1, h=P[3], codes=P[4],  # noqa: F811
          scales=P[5]):
    return lib.ckl_add_norm_quant(x, xt, res, rt, T, d, w, wt, eps, form, h, codes, scales, None)


SIZES = [(dict(T=-1), INV), (dict(T=4000001), UNS), (dict(d=0), INV), (dict(d=12), INV), (dict(d=65544), UNS),
         (dict(xt=2), INV), (dict(rt=-1), INV), (dict(wt=3), INV), (dict(xt=0, rt=1), UNS), (dict(w=None), INV),
         (dict(w=P[9] + 2), INV), (dict(h=None), INV)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(eps=-1.0), INV), (dict(eps=float("inf")), INV), (dict(p=2.0), INV), (dict(x=None), INV), (dict(res=None), INV),
    (dict(y=None), INV), (dict(x=P[0] + 8), INV), (dict(h=P[3] + 8), INV), (dict(rstd=P[5] + 2), INV), (dict(h=P[1]), INV),
    (dict(y=P[0]), INV), (dict(y=P[3]), INV), (dict(rstd=P[2]), INV), (dict(state=P[4]), INV), (dict(state=P[6] + 1), INV)])
def test_add_norm_forward_refusals(lib, kw, status):  # noqa: F811
    assert fwd(lib, **kw) == status
    assert lib.ckl_last_error()


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(p=-1.0), INV), (dict(dy=None), INV), (dict(rstd=None), INV), (dict(dr=None), INV), (dict(dw=None), INV),
    (dict(dx=None), INV), (dict(dx=None, p=0.0, rt=0), INV), (dict(dx=P[6]), INV), (dict(dr=P[1]), INV), (dict(dr=P[2]), INV),
    (dict(dw=P[4]), INV), (dict(ws=None), WSP), (dict(ws_bytes=64), WSP), (dict(ws=P[8] + 4), INV), (dict(ws=P[0]), INV),
    (dict(rstd=P[3] + 1), INV)])
def test_add_norm_backward_refusals(lib, kw, status):  # noqa: F811
    assert bwd(lib, **kw) == status
    assert lib.ckl_last_error()


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(form=0), INV), (dict(form=3), INV), (dict(codes=None), INV), (dict(scales=None), INV), (dict(codes=P[4] + 8), INV),
    (dict(form=2, scales=P[5] + 2), INV), (dict(codes=P[3]), INV), (dict(scales=P[2]), INV), (dict(h=P[0]), INV)])
def test_add_norm_quant_refusals(lib, kw, status):  # noqa: F811
    assert quant(lib, **kw) == status
    assert lib.ckl_last_error()


def test_nothing_to_do(lib):  # noqa: F811
    assert drop(lib, n=0, x=None, out=None) == 0
    assert fwd(lib, T=0, x=None, res=None, h=None, y=None, rstd=None) == 0
    assert quant(lib, T=0, x=None, res=None, h=None, codes=None, scales=None) == 0
    assert size(lib.ckl_add_norm_workspace_size, 0, 64) == 0
    assert 0 < size(lib.ckl_add_norm_workspace_size, 4000000, 64) < 1 << 22
    assert lib.ckl_add_norm_workspace_size(4, 64, None) == INV
    assert lib.ckl_add_norm_workspace_size(4, 12, ctypes.byref(ctypes.c_size_t())) == INV


def test_python_layer_refuses():
    x, w = torch.zeros(4, 16), torch.zeros(16)
    for call in (lambda: ckl.dropout(x, 0.5), lambda: ckl.add_rms_norm(x, x, w), lambda: ckl.add_norm_quant(x, x, w)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="one shape"):
        ckl.add_rms_norm(x, x[:2], w)
    with pytest.raises(ValueError, match="form"):
        ckl.add_norm_quant(x, x, w, form="e5m2")
    from chunked_kl_loss_amd import ops
    cpu = torch.device("cpu")
    for bad in (dict(p=-0.1), dict(p=1.5), dict(seed=-1), dict(seed=2 ** 64), dict(offset=-1), dict(offset=2 ** 64),
                dict(seed=torch.zeros(2)), dict(seed=torch.zeros(3, dtype=torch.int64)),
                dict(seed=torch.zeros(2, dtype=torch.int64, device="meta"))):
        with pytest.raises(ValueError):
            ops._drop_args(**{**dict(p=0.5, seed=0, offset=0), **bad}, device=cpu)
