"""Dropout and the RMS norm with the residual's addition on the GPU against plain computations.

Dropout is compared bit for bit with Philox4x32-10 written in numpy.  Elsewhere tolerances count roundings: EPS is
one fp32 rounding relative to the value, a sum of n terms in any order is within n EPS of the sum of magnitudes, and
a result in type t is rounded once more, by at most HALF[t] of its value."""
import math

import numpy as np
import pytest
import torch

import chunked_kl_loss_amd as ckl
from tests.philox import keep_mask

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
PAIRS = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")]


def normal(shape, dtype, seed, std=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float32) * std).to(dtype)


def same_bits(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.contiguous().reshape(-1).view(torch.uint8),
                                                                     b.contiguous().reshape(-1).view(torch.uint8))


def dropped(x, p, seed, offset):
    """x (any float tensor on the CPU) after dropout, each element rounded once from an fp32 product."""
    keep, scale = keep_mask(x.numel(), p, seed, offset)
    y = np.where(keep, x.float().numpy().reshape(-1) * np.float32(scale), np.float32(0))
    return torch.from_numpy(y.astype(np.float32)).view(x.shape).to(x.dtype), torch.from_numpy(keep).view(x.shape)


def test_offsets_past_32_bits():
    # the last rows lie more than 2^32 elements behind the first
    T, d, p = 2_900_000, 1512, 0.3
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    last, dlast = normal((2, d), torch.bfloat16, 1), normal((2, d), torch.bfloat16, 2)
    x[-2:] = last.cuda()
    keep, scale = keep_mask(2 * d, p, 7, 9, (T - 2) * d)

    def drop(t):
        return torch.where(torch.from_numpy(keep).view(2, d), t.float() * scale, 0.0).bfloat16()
    y = ckl.dropout(x, p, 7, 9)
    assert same_bits(y[-2:].cpu(), drop(last)) and not y[:-2].any()
    del y
    w = (1 + normal((d,), torch.float32, 3, 0.1)).bfloat16().cuda()
    y, h, rstd = ckl.add_norm_forward(x, x, w, 1e-6, p, 7, 9)
    hl = (last.float() + torch.where(torch.from_numpy(keep).view(2, d), last.float() * scale, 0.0)).bfloat16()
    want = ckl.add_norm_forward(torch.zeros_like(hl).cuda(), hl.cuda(), w)
    for got, v in zip((y, h, rstd), want):
        assert same_bits(got[-2:], v)
    assert not y[:-2].any() and not h[:-2].any() and (rstd[:-2] == rstd[0]).all()
    del y, want
    x.zero_()
    x[-2:] = dlast.cuda()
    dx, dres, dw = ckl.add_norm_backward(x, None, h, rstd, w, p, 7, 9)
    _, small, dw2 = ckl.add_norm_backward(dlast.cuda(), None, hl.cuda(), rstd[-2:].contiguous(), w)
    assert same_bits(dres[-2:], small) and not dres[:-2].any() and not dx[:-2].any()
    # (dx is scaled before dres is rounded: three roundings between the two)
    assert ((dx[-2:].cpu() != 0) == (torch.from_numpy(keep).view(2, d) & (small.cpu() != 0))).all()
    assert ((dx[-2:].cpu().double() - drop(small.cpu()).double()).abs() <= 2 ** -6 * drop(small.cpu()).double().abs()).all()
    # (a workgroup may hold both rows or each its own: sums of two terms)
    assert ((dw.double() - dw2.double()).abs() <= 2 ** -6 * dw2.double().abs() + 1e-6).all()
    del x, h, dx, dres
    z = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    z[-2:] = last.cuda()
    for form in ("int8", "e4m3"):
        codes, scales, h = ckl.add_norm_quant(z, z, w, form=form)
        small = ckl.add_norm_quant(last.cuda(), last.cuda(), w, form=form)
        for got, v in zip((codes, scales, h), small):
            assert same_bits(got[-2:], v)
        assert not codes[:-2].view(torch.uint8).any()
        del codes, scales, h


# ---------------------------------------------------------------- dropout --
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,p,seed,offset", [
    (1, 0.5, 0, 0), (7, 0.5, 1, 0), (8, 0.25, 2, 3), (9, 0.1, 3, 0), (8191, 0.1, 4, 1), (8192, 0.1, 5, 1),
    (8193, 0.9, 6, 1), (77 * 1003, 0.25, 2 ** 64 - 1, 2 ** 64 - 1), (1 << 20, 0.1, 2 ** 40 + 5, 2 ** 33),
    (100, 0.0, 9, 0), (100, 1.0, 9, 0), (5000, 1e-6, 9, 0), (5000, 1 - 1e-6, 9, 0)])
def test_dropout(n, p, seed, offset, dtype):
    x = normal((n,), DT[dtype], n)
    want, keep = dropped(x, p, seed, offset)
    xg = x.cuda().requires_grad_(True)
    y = ckl.dropout(xg, p, seed=seed, offset=offset)
    dy = normal((n,), DT[dtype], n + 1)
    (dx,) = torch.autograd.grad(y, (xg,), dy.cuda())
    assert same_bits(y.detach().cpu(), want)
    assert same_bits(dx.cpu(), dropped(dy, p, seed, offset)[0])
    with torch.no_grad():
        assert same_bits(ckl.dropout(xg, p, seed, offset), y)
    state = torch.tensor([seed, offset - 1 if offset else 0], dtype=torch.uint64).view(torch.int64).cuda()
    assert same_bits(ckl.dropout(xg, p, state, 1 if offset else 0), y)  # the same numbers from device memory


def test_dropout_share_and_independence():
    # 2^22 elements: the share kept is within 6 standard deviations, as are those of two offsets and of two seeds at once
    n, p = 1 << 22, 0.3
    x = torch.ones(n, device="cuda")
    a = ckl.dropout(x, p, 1, 0) != 0
    q = 1 - round(p * 65536) / 65536
    assert abs(float(a.double().mean()) - q) < 6 * math.sqrt(q * (1 - q) / n)
    for b in (ckl.dropout(x, p, 1, 1) != 0, ckl.dropout(x, p, 2, 0) != 0, torch.roll(a, 1), torch.roll(a, 8)):
        both = float((a & b).double().mean())
        assert abs(both - q * q) < 6 * math.sqrt(q * q * (1 - q * q) / n)


def test_dropped_elements_may_hold_anything():
    keep = torch.from_numpy(keep_mask(4000, 0.5, 3, 0)[0])
    x = torch.where(keep, 1.0, torch.tensor([math.nan, math.inf, -math.inf, 1e38]).repeat(1000))
    y = ckl.dropout(x.cuda(), 0.5, 3).cpu()
    assert torch.equal(y, torch.where(keep, 2.0, 0.0))


def test_dropout_shapes_strides_and_offsets():
    x = normal((6, 50, 33), torch.bfloat16, 1).cuda()
    t = x.transpose(0, 2)
    assert same_bits(ckl.dropout(t, 0.2, 5), ckl.dropout(t.contiguous(), 0.2, 5))
    s = x.view(-1)[3:1003]  # begins off a 16-byte boundary
    assert same_bits(ckl.dropout(s, 0.2, 5), ckl.dropout(s.clone(), 0.2, 5))
    for empty in (torch.empty(0, device="cuda"), torch.empty(3, 0, 8, device="cuda")):
        assert ckl.dropout(empty, 0.5).shape == empty.shape
    e = torch.ones(1, 1, device="cuda", requires_grad=True)
    y = ckl.dropout(e.expand(400, 8), 0.5, 4)  # the gradient of a broadcast input is summed
    y.sum().backward()
    assert float(e.grad) == float(y.sum())


# ------------------------------------------------------ norm behind a branch --
def reference(x, res, w, eps, p, seed, offset):
    """h before its rounding, the mask and the scale, in 64 bits."""
    keep, scale = keep_mask(x.numel(), p, seed, offset)
    m = torch.from_numpy(keep).view(x.shape).double() * float(np.float32(scale))
    return res.double() + torch.where(m > 0, x.double() * m, torch.zeros_like(m)), m


def check_forward(x, res, w, eps, p, seed, offset, y, h):
    h64, m = reference(x, res, w, eps, p, seed, offset)
    d = x.shape[-1]
    # the product with the scale and the sum round once each
    tol = EPS * ((x.double() * m).abs() + h64.abs() * 2) + HALF[h.dtype] * h64.abs() + 1e-37
    assert ((h.double() - h64).abs() <= tol).all()
    hd = h.double()
    r = 1 / torch.sqrt((hd * hd).mean(-1, keepdim=True) + eps)
    y64 = hd * r * w.double()
    # half of the sum of squares' d + 4 roundings, the root, its inverse, two products, the rounding to y's type
    tol = y64.abs() * ((d + 4) * EPS / 2 + 6 * EPS + HALF[y.dtype]) + 1e-37
    assert ((y.double() - y64).abs() <= tol).all()
    return hd, r, m


def check_backward(dy, dh, hd, r, w, m, dx, dres, dw):
    T, d = hd.reshape(-1, hd.shape[-1]).shape
    n, g = hd * r, dy.double() * w.double()
    base = torch.zeros_like(g) if dh is None else dh.double()
    c, cabs = (g * n).mean(-1, keepdim=True), (g * n).abs().mean(-1, keepdim=True)
    d64 = base + r * (g - n * c)
    rel = (d + 4) * EPS / 2 + 6 * EPS  # that of r, as above
    err = r * (g.abs() * (rel + 4 * EPS) + n.abs() * (c.abs() * (3 * rel + 6 * EPS) + cabs * (d + 8) * EPS))
    err = err + EPS * (base.abs() + d64.abs() * 2) + 1e-37
    assert ((dres.double() - d64).abs() <= err + HALF[dres.dtype] * d64.abs()).all()
    dx64 = d64 * m
    assert ((dx.double() - dx64).abs() <= (err * m + EPS * dx64.abs()) + HALF[dx.dtype] * dx64.abs()).all()
    assert (dx[m == 0] == 0).all()
    dw64 = (dy.double() * n).reshape(T, d).sum(0)
    mag = (dy.double() * n).abs().reshape(T, d).sum(0)
    assert ((dw.double() - dw64).abs() <= mag * ((T + 70) * EPS + rel + 2 * EPS) + HALF[dw.dtype] * dw64.abs() + 1e-37).all()


@pytest.mark.parametrize("types", PAIRS, ids=lambda t: "-".join(t))
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 16), (5, 64), (33, 72), (257, 128), (100, 136), (65, 256), (9, 264),
                                 (257, 512), (31, 520), (300, 1000), (64, 2880), (3, 8192), (5, 16384), (3, 20480),
                                 (2, 32768), (3, 65536), (2050, 64), (1300, 2056)])
def test_add_rms_norm(T, d, p, types):
    xt, rt = DT[types[0]], DT[types[1]]
    x, res = normal((T, d), xt, T + d, 0.5), normal((T, d), rt, T + d + 1, 2.0)
    w = (1 + normal((d,), torch.float32, d, 0.2)).to(xt)
    dy, dh = normal((T, d), xt, 5), normal((T, d), rt, 6)
    X, R, W = (t.cuda().requires_grad_(True) for t in (x, res, w))
    y, h = ckl.add_rms_norm(X, R, W, 1e-5, p, seed=11, offset=7)
    assert y.dtype == xt and h.dtype == rt
    hd, r, m = check_forward(x, res, w, 1e-5, p, 11, 7, y.detach().cpu(), h.detach().cpu())
    dx, dr, dw = torch.autograd.grad((y, h), (X, R, W), (dy.cuda(), dh.cuda()))
    check_backward(dy, dh, hd, r, w, m, dx.cpu(), dr.cpu(), dw.cpu())
    with torch.no_grad():
        assert all(same_bits(a, b) for a, b in zip(ckl.add_rms_norm(X, R, W, 1e-5, p, 11, 7), (y, h)))


@pytest.mark.parametrize("types", PAIRS, ids=lambda t: "-".join(t))
def test_one_output_only(types):
    # the loss may depend on y alone or on h alone
    xt, rt = DT[types[0]], DT[types[1]]
    T, d = 37, 200
    x, res, w = normal((T, d), xt, 1), normal((T, d), rt, 2), (1 + normal((d,), torch.float32, 3, 0.2)).to(xt)
    X, R, W = (t.cuda().requires_grad_(True) for t in (x, res, w))
    y, h = ckl.add_rms_norm(X, R, W, 1e-6, 0.25, 3, 1)
    hd, r, m = check_forward(x, res, w, 1e-6, 0.25, 3, 1, y.detach().cpu(), h.detach().cpu())
    dy, dh = normal((T, d), xt, 5), normal((T, d), rt, 6)
    dx, dr, dw = torch.autograd.grad(y, (X, R, W), dy.cuda(), retain_graph=True)
    check_backward(dy, None, hd, r, w, m, dx.cpu(), dr.cpu(), dw.cpu())
    dx, dr, dw = torch.autograd.grad(h, (X, R, W), dh.cuda(), allow_unused=True)
    check_backward(torch.zeros_like(dy), dh, hd, r, w, m, dx.cpu(), dr.cpu(), dw.cpu())
    assert not dw.any()


def test_gradients_against_differences():
    # values: at most 300 terms of about 1, each with 4 roundings.  The norm's third derivative along u is below 15
    # (|u| / |h|)^3 |y| a row, here 6 rows of 15 * 0.7 * 24, and enters with step^2 / 6.
    T, d, step = 6, 24, 4e-3
    tol = 300 * 4 * EPS / step + step ** 2 / 6 * 6 * 15 * 0.7 * 24
    x, res, w = normal((T, d), torch.float32, 1), normal((T, d), torch.float32, 2), 1 + normal((d,), torch.float32, 3, 0.2)
    a, b = normal((T, d), torch.float64, 4), normal((T, d), torch.float64, 5)
    X, R, W = (t.cuda().requires_grad_(True) for t in (x, res, w))

    def value(x, r, w):
        y, h = ckl.add_rms_norm(x, r, w, 1e-5, 0.25, 9)
        return (y.double() * a.cuda()).sum() + (h.double() * b.cuda()).sum()
    grads = torch.autograd.grad(value(X, R, W), (X, R, W))
    for k, (t, g) in enumerate(zip((x, res, w), grads)):
        for i in range(5):
            u = normal(t.shape, torch.float32, 20 + i)
            at = [[s + (e * u if j == k else 0) for j, s in enumerate((x, res, w))] for e in (step, -step)]
            hi, lo = (float(value(*(s.cuda() for s in p))) for p in at)
            got = float((g.double().cpu() * u.double()).sum())
            assert abs((hi - lo) / (2 * step) - got) < tol


def test_rows_of_zeros_and_special_values():
    T, d = 8, 96
    x, res, w = torch.zeros(T, d), torch.zeros(T, d), torch.ones(d)
    res[1], res[2, 5], res[3, 6], res[4], res[5] = 1e-30, math.inf, math.nan, 3e18, -1e-20
    X, R, W = (t.cuda().requires_grad_(True) for t in (x, res, w))
    y, h = ckl.add_rms_norm(X, R, W, 1e-6)
    assert same_bits(h.detach().cpu(), res)
    y = y.detach().cpu()
    assert not y[0].any() and torch.isfinite(y[[0, 1, 4, 5]]).all() and torch.isnan(y[3]).all()
    assert torch.allclose(y[4], torch.ones(d), rtol=1e-5) and not torch.isfinite(y[2]).all()
    # (no eps: a row of zeros is 0 / 0)
    assert torch.isnan(ckl.add_rms_norm(X[:1], R[:1], W, 0.0)[0]).all()


@pytest.mark.parametrize("types", PAIRS, ids=lambda t: "-".join(t))
def test_branches_of_strided_broadcast_and_empty_inputs(types):
    xt, rt = DT[types[0]], DT[types[1]]
    x, res, w = normal((3, 40, 4), xt, 1).cuda(), normal((4, 3, 40), rt, 2).cuda(), normal((80,), xt, 3).cuda()[::2]
    t = x.permute(2, 0, 1)
    got, want = ckl.add_rms_norm(t, res, w), ckl.add_rms_norm(t.contiguous(), res, w.contiguous())
    assert all(same_bits(a, b) for a, b in zip(got, want)) and got[0].shape == (4, 3, 40)
    e = torch.empty(0, 40, dtype=xt, device="cuda", requires_grad=True)
    W = w.contiguous().requires_grad_(True)
    y, h = ckl.add_rms_norm(e, torch.empty(0, 40, dtype=rt, device="cuda"), W)
    dx, dw = torch.autograd.grad((y, h), (e, W), (torch.zeros_like(y), torch.zeros_like(h)))
    assert y.shape == h.shape == dx.shape == (0, 40) and not dw.any()
    r = normal((1, 40), rt, 4).cuda().requires_grad_(True)  # one residual for all rows: its gradient is the rows' sum
    y, h = ckl.add_rms_norm(t.reshape(12, 40), r.expand(12, 40), w)
    (dr,) = torch.autograd.grad(h, (r,), torch.ones_like(h))
    assert torch.equal(dr, torch.full_like(dr, 12.0))


# ----------------------------------------------------------------- 8 bits --
@pytest.mark.parametrize("types", PAIRS, ids=lambda t: "-".join(t))
@pytest.mark.parametrize("T,d", [(1, 8), (5, 40), (33, 72), (257, 512), (31, 520), (16, 2880), (3, 20480), (2, 65536)])
def test_add_norm_quant(T, d, types):
    xt, rt = DT[types[0]], DT[types[1]]
    x, res = normal((T, d), xt, T + d, 0.5).cuda(), normal((T, d), rt, T + d + 1, 2.0).cuda()
    res[T // 2, d // 2] = 90.0  # a column that stands out
    w = (1 + normal((d,), torch.float32, d, 0.2)).cuda()
    _, want_h = ckl.add_rms_norm(x, res, w)
    codes, scales, h = ckl.add_norm_quant(x, res, w, form="int8")
    assert same_bits(h, want_h)
    hd = h.double().cpu()
    y = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-6) * w.double().cpu()
    # y before its coding: half of the sum of squares' d + 4 roundings and four more; a code is within half a step
    rel = (d + 4) * EPS / 2 + 4 * EPS
    held = ckl.act_decode(codes, scales, dtype=torch.float32).double().cpu()
    blocks = torch.nn.functional.pad(y, (0, -d % 32)).view(T, -1, 32).abs().amax(2, keepdim=True)
    step = torch.exp2(torch.floor(torch.log2(blocks * (1 + 2 * rel) / 127.5)) + 1).expand(-1, -1, 32).reshape(T, -1)[:, :d]
    assert ((held - y).abs() <= step / 2 + rel * y.abs()).all()
    near = torch.exp2(torch.floor(torch.log2(blocks / 127.5)) + 1 + 127)[:, :, 0]
    border = (torch.log2(blocks / 127.5) - torch.log2(blocks / 127.5).round()).abs()[:, :, 0] < 2 * rel
    assert ((scales.cpu().double() == torch.log2(near)) | border).all()  # the smallest power of two that will do
    codes, scales, h = ckl.add_norm_quant(x, res, w, form="e4m3")
    assert same_bits(h, want_h) and codes.dtype == torch.float8_e4m3fn
    top = y.abs().amax(1)
    assert ((scales.double().cpu() - top / 448).abs() <= top / 448 * (rel + EPS)).all()
    c = codes.cpu().double()
    q = y / scales.double().cpu()[:, None]
    # three bits behind the first: half a step is 2^-4 of the power of two below, at least half of 2^-9
    half = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 4)
    assert ((c - q).abs() <= half + (rel + 2 * EPS) * q.abs()).all() and (c.abs().amax(1) == 448).all()


@pytest.mark.parametrize("types", PAIRS, ids=lambda t: "-".join(t))
@pytest.mark.parametrize("T,d", [(400, 64), (300, 520), (200, 2880), (7, 20480), (3, 65536)])
def test_codes_carry_one_rounding_of_the_norm(T, d, types):
    # whatever d: y is not rounded before its int8 code; e4m3: to fp32 once, and its quotient once more
    xt, rt = DT[types[0]], DT[types[1]]
    x, res = normal((T, d), xt, T + d, 0.5).cuda(), normal((T, d), rt, T + d + 1, 2.0).cuda()
    w = (1 + normal((d,), torch.float32, d, 0.2)).cuda()
    codes, scales, h = ckl.add_norm_quant(x, res, w, form="int8")
    hd = h.double()
    y = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + float(np.float32(1e-6))) * w.double()
    step = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :d]
    assert ((codes.double() * step - y).abs() <= step * (0.5 + 1e-9)).all()
    codes, scales, _ = ckl.add_norm_quant(x, res, w, form="e4m3")
    top = y.abs().amax(1)
    assert ((scales.double() - top / 448).abs() <= top / 448 * 2.01 * EPS).all()
    q = y / scales.double()[:, None]
    half = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 4)
    assert ((codes.double() - q).abs() <= half + 2.01 * EPS * q.abs()).all()


def test_codes_are_those_of_the_rounded_quotients():
    # values that are exact through the norm: h of one magnitude a row, the weight shapes it
    T, d = 64, 64
    h = torch.where(torch.rand(T, d, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0)
    h = h * torch.exp2(torch.randint(-20, 20, (T, 1)).float())
    w = normal((d,), torch.float32, 2)
    # r = 1 / |h| is a power of two: y = +-w exactly
    zero = torch.zeros(T, d).cuda()
    codes, scales, _ = ckl.add_norm_quant(zero, h.cuda(), w.cuda(), eps=0.0, form="e4m3")
    y = torch.sign(h) * w
    want = (w.abs().max() / 448).expand(T)
    assert same_bits(scales.cpu(), want.contiguous())
    assert same_bits(codes.cpu(), (y / want[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn))
    codes, scales, _ = ckl.add_norm_quant(zero, h.cuda(), w.cuda(), eps=0.0, form="int8")
    assert all(same_bits(a, b) for a, b in zip((codes, scales), ckl.act_encode(y.cuda())))


def test_quant_of_zeros_and_special_values():
    T, d = 6, 64
    x, res, w = torch.zeros(T, d).cuda(), torch.zeros(T, d), torch.ones(d).cuda()
    res[1, 3], res[2, 40], res[3] = math.nan, math.inf, 1e-30
    res = res.cuda()
    codes, scales, h = ckl.add_norm_quant(x, res, w, form="e4m3")
    assert torch.isnan(scales[1:3]).all() and not codes.float()[[0, 1, 2]].any()
    assert float(scales[0]) == 2.0 ** -126 and torch.isfinite(scales[3])
    codes, scales, h = ckl.add_norm_quant(x, res, w, form="int8")
    assert (scales[1] == 255).all() and (scales[2] == 255).any() and (scales[0] == 1).all() and not codes[0].any()
    for form in ("int8", "e4m3"):
        c, s, h = ckl.add_norm_quant(x[:0], res[:0], w, form=form)
        assert c.shape == h.shape == (0, d)


# ------------------------------------------------- captures, streams, tangents --
def test_captured_step_draws_anew_when_the_state_moves():
    T, d = 130, 200
    w = (1 + normal((d,), torch.float32, 3, 0.2)).cuda()
    state = torch.zeros(2, dtype=torch.int64, device="cuda")

    def run(x, res, dy, seed):
        X, R, W = (t.detach().requires_grad_(True) for t in (x, res, w))
        y, h = ckl.add_rms_norm(X, R, W, 1e-6, 0.3, seed, 5)
        z = ckl.dropout(y, 0.2, seed, 6)
        return [z.detach(), h.detach(), *torch.autograd.grad((z, h), (X, R, W), (dy, dy))]
    ins = [normal((T, d), torch.float32, s).cuda() for s in (1, 2, 4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*ins, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(*ins, state)
    seen = []
    for seed, offset in ((5, 0), (5, 1), (6, 1), (5, 0)):
        state.copy_(torch.tensor([seed, offset]))
        for i, t in enumerate(ins):
            t.copy_(normal((T, d), torch.float32, 40 + i))
        plain = [t.clone() for t in run(*ins, torch.tensor([seed, offset]).cuda())]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(outs, plain))
        seen.append(outs[0].clone())
    assert same_bits(seen[0], seen[3]) and not any(same_bits(seen[0], s) for s in seen[1:3])


def test_state_may_move_before_the_backward_pass():
    x = torch.ones(4000, device="cuda", requires_grad=True)
    state = torch.tensor([3, 4], device="cuda")
    y = ckl.dropout(x, 0.5, state)
    z, _ = ckl.add_rms_norm(x.view(50, 80), torch.zeros(50, 80, device="cuda"), torch.ones(80, device="cuda"), p=0.5,
                            seed=state)
    state += 7
    (dx,) = torch.autograd.grad(y, (x,), torch.ones_like(y))
    assert same_bits(dx, y.detach())
    (dx,) = torch.autograd.grad(z, (x,), torch.ones_like(z))
    assert torch.equal(dx.view(50, 80) == 0, z.detach() == 0)


def test_two_streams_at_once():
    def run(seed):
        x, r = normal((4000, 520), torch.bfloat16, seed).cuda(), normal((4000, 520), torch.bfloat16, seed + 1).cuda()
        w = normal((520,), torch.bfloat16, 3).cuda().requires_grad_(True)
        x.requires_grad_(True)

        def go():
            y, h = ckl.add_rms_norm(x, r, w, 1e-6, 0.1, seed)
            return [y.detach(), h.detach(), *torch.autograd.grad((y, h), (x, w), (r, r))]
        return go
    jobs = [run(1), run(30)]
    want = [[t.clone() for t in j()] for j in jobs]
    torch.cuda.synchronize()
    got, streams = [], [torch.cuda.Stream() for _ in jobs]
    for s, j in zip(streams, jobs):
        with torch.cuda.stream(s):
            got.append(j())
    torch.cuda.synchronize()
    assert all(same_bits(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_forward_mode_tangents_are_refused():
    fw = torch.autograd.forward_ad
    x, w = normal((4, 16), torch.float32, 2).cuda(), normal((16,), torch.float32, 3).cuda()
    with fw.dual_level():
        d = fw.make_dual(x, torch.ones_like(x))
        for call in (lambda: ckl.dropout(d, 0.5), lambda: ckl.add_rms_norm(d, x, w), lambda: ckl.add_rms_norm(x, d, w)):
            with torch.no_grad(), pytest.raises(NotImplementedError, match="jvp"):
                call()


def test_neighbours_stay_untouched():
    import ctypes

    from chunked_kl_loss_amd import _binding as B
    lib = B.load_library()
    T, d = 9, 40
    x, r, w = (normal(s, torch.float32, i).cuda() for i, s in enumerate(((T, d), (T, d), (d,))))
    n = T * d
    bufs = {k: torch.full((n + 64,), -7.0, device="cuda") for k in ("h", "y", "dx", "dr")}
    rstd, dw = torch.full((T + 64,), -7.0, device="cuda"), torch.full((d + 64,), -7.0, device="cuda")
    need = ctypes.c_size_t(0)
    B.check(lib.ckl_add_norm_workspace_size(T, d, ctypes.byref(need)))
    ws = torch.full((need.value + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    at = {k: b.data_ptr() + 64 for k, b in bufs.items()}
    B.check(lib.ckl_add_norm_forward(x.data_ptr(), 0, r.data_ptr(), 0, T, d, w.data_ptr(), 0, 1e-6, 0.5, 1, 2, None,
                                     at["h"], at["y"], rstd.data_ptr() + 64, None))
    B.check(lib.ckl_add_norm_backward(x.data_ptr(), 0, None, 0, T, d, at["h"], rstd.data_ptr() + 64, w.data_ptr(), 0,
                                      0.5, 1, 2, None, at["dx"], at["dr"], dw.data_ptr() + 64, ws.data_ptr(),
                                      need.value, None))
    drop = torch.full((1003 + 64,), -7.0, device="cuda")
    src = normal((1003,), torch.float32, 9).cuda()
    B.check(lib.ckl_dropout(src.data_ptr(), 0, 1003, 0.5, 1, 2, None, drop.data_ptr() + 64, None))
    torch.cuda.synchronize()
    for b, m in [(b, n) for b in bufs.values()] + [(rstd, T), (dw, d), (drop, 1003)]:
        assert (b[:16] == -7).all() and (b[16 + m:] == -7).all() and not (b[16:16 + m] == -7).any()
    assert (ws[need.value:] == 0xAB).all()


def test_second_derivatives_are_refused():
    x, w = normal((4, 16), torch.float32, 2).cuda().requires_grad_(True), normal((16,), torch.float32, 3).cuda()
    z, tok = normal((4, 9), torch.float32, 4).cuda().requires_grad_(True), torch.zeros(4, dtype=torch.int64, device="cuda")
    head = normal((9, 16), torch.float32, 5).cuda()
    for f, leaf in ((lambda: ckl.add_rms_norm(x, x.detach(), w)[0], x), (lambda: ckl.token_logprobs(z, tok)[1], z),
                    (lambda: ckl.head_logprobs(x, head, tok)[0], x)):
        (g,) = torch.autograd.grad(f().sum(), (leaf,), create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.sum().backward()
    v = normal((4, 16), torch.float32, 6).cuda().requires_grad_(True)
    y = ckl.dropout(x, 0.5, 3)  # linear: its gradient can be differentiated
    (g,) = torch.autograd.grad(y, (x,), v, create_graph=True)
    (gg,) = torch.autograd.grad(g, (v,), x.detach())
    assert same_bits(gg, y.detach())


def test_one_tensor_as_branch_and_residual():
    T, d = 9, 64
    w = (1 + normal((d,), torch.float32, 3, 0.2)).cuda()
    x = normal((T, d), torch.float32, 1).cuda().requires_grad_(True)
    y, h = ckl.add_rms_norm(x, x, w)
    assert same_bits(h.detach(), x.detach() + x.detach())
    dy = normal((T, d), torch.float32, 2).cuda()
    (y * dy).sum().backward()
    a, b = (x.detach().clone().requires_grad_(True) for _ in range(2))
    (ckl.add_rms_norm(a, b, w)[0] * dy).sum().backward()
    assert torch.equal(x.grad, a.grad + b.grad) and a.grad.data_ptr() != b.grad.data_ptr()
