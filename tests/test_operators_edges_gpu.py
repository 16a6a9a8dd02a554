"""The operators around the loss on the GPU where their inputs are unusual: logits of a mask's size, students that
are sure and close to their teacher, tensors off a 16-byte boundary, garbage in masked rows, ids at the ends of
their type, forward-mode tangents, and what lies around the workspaces and outputs.

References are plain 64-bit computations.  Tolerances count roundings: EPS is one fp32 rounding relative to the
value, a sum of n terms in any order is within n EPS of the sum of magnitudes, and a result in type t is rounded
once more, by at most HALF[t] of its value."""
import ctypes
import math

import pytest
import torch

import chunked_kl_loss_amd as ckl
from chunked_kl_loss_amd import _binding as B
from tests.test_operators_gpu import DT, EPS, HALF, check_topk, loss_inputs, normal, same_bits

pytestmark = pytest.mark.gpu


# ---------------------------------------------- logits of a mask's magnitude --
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", [0, 1])
@pytest.mark.parametrize("T", [3, 1030])
def test_topk_of_logits_far_from_zero(T, form, dtype):
    # several segments to a row (T = 3), whole rows to a workgroup (T = 1030)
    V, K = 9001, 33
    far = [f * m for m in (5e9, 1e10, 1e12, 1e20, 6e29, 1e31) for f in (-1.0, 1.0)] + [-7e7, 7e7, -3e9, 2e8]
    for i, m in enumerate(far):
        z = normal((T, V), torch.float32, 40 + i, 2.0)
        z[0, :] = m                      # a whole row
        z[1, :8] = m                     # the first columns that one thread sees
        z[2, :2048:3] = m                # some of the columns of every thread's first vector
        z[2, 8500:8700] = m              # and of a later segment
        check_topk(z.to(DT[dtype]), K, form)


# ------------------------------------------------------ forward-mode tangents --
def test_forward_mode_tangents_are_refused_not_lost():
    fw = torch.autograd.forward_ad
    W, tok = normal((50, 16), torch.float32, 1).cuda(), torch.tensor([1, -1, 49, 7], device="cuda")
    x, w = normal((4, 16), torch.float32, 2).cuda(), normal((16,), torch.float32, 3).cuda()
    idx, tl = torch.arange(2, device="cuda", dtype=torch.int32).repeat(4, 1), normal((4, 2), torch.float32, 4).cuda()
    kl = ckl.chunked_kl_loss
    calls = [lambda W, x, w: ckl.embedding(W, tok, 2.0), lambda W, x, w: ckl.rms_norm_8bit(x, w),
             lambda W, x, w: kl(x, W, idx, tl), lambda W, x, w: kl(x, W, idx, tl, save_8bit=True),
             lambda W, x, w: kl(x, W, idx, tl, save_8bit=True, norm_weight=w),
             lambda W, x, w: kl(x, W, idx, tl, fused=True, save_8bit=True, norm_weight=w)]
    uses = ["W", "xw", "Wx", "Wx", "Wxw", "Wxw"]
    plain = [f(W, x, w) for f in calls]
    with fw.dual_level():
        dual = {n: fw.make_dual(t, torch.ones_like(t)) for n, t in (("W", W), ("x", x), ("w", w))}
        for f, names, want in zip(calls, uses, plain):
            for grad_mode in (True, False):
                with torch.set_grad_enabled(grad_mode):
                    for n in names:
                        args = dict(W=W, x=x, w=w)
                        args[n] = dual[n]
                        with pytest.raises(NotImplementedError, match="jvp"):
                            f(**args)
                    got = f(W, x, w)  # without a tangent as ever
                    assert not got.requires_grad and same_bits(got, want)


# ------------------------------------- the loss's gradient from 8-bit states --
def sure_student(dtype, lean, big, d=256, T=200, V=4000, K=50, noise=0.1):
    """States that lean on one word a row, a teacher that is the student's logits and a little noise, a mask."""
    W = normal((V, d), torch.float32, 1, d ** -0.5)
    word = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(2))
    H = lean * W[word] + normal((T, d), torch.float32, 3)
    if big > 1:  # a few large columns, as residual streams have them
        H[:, [5, 100]] *= big
        W[:, [5, 100]] /= big
    H, W = H.to(dtype), W.to(dtype)
    teacher = H.double() @ W.double().t() + noise * normal((T, V), torch.float64, 4)
    vals, idx = torch.topk(teacher, K, 1)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(5)) < 0.8
    return H, W, idx.int(), vals.float(), mask


def loss_gradient(h, W, idx, vals, mask, half):
    """Of the mean KL at states h, in 64 bits: (dH, dW) with a bound on each element's error.  half: one rounding of
    G and of the results."""
    T, d = h.shape
    V = W.shape[0]
    z = h @ W.t()
    lse = torch.logsumexp(z, 1, keepdim=True)
    q = torch.zeros_like(z).scatter_(1, idx.long(), torch.softmax(vals.double(), 1))
    p = torch.exp(z - lse)
    s = mask.double()[:, None] / mask.sum()
    G = s * (p - q)
    # a logit is a sum of d products; the log-sum-exp adds V exponentials and rounds with its size, and carries its
    # largest logit's error; an exponential is good to 2^-22 and to the rounding of its argument; q likewise
    e_z = 2 * d * EPS * (h.abs() @ W.abs().t())
    e_lse = (p * e_z).sum(1, keepdim=True) + (V + 8) * EPS + 4 * EPS * lse.abs()
    e_p = p * (e_z + e_lse + 4 * EPS * (z - lse).abs() + 2.0 ** -22)
    e_q = q * (64 * EPS + 4 * EPS * vals.abs().max())
    e_G = s * (e_p + e_q) + G.abs() * half + 4 * EPS * s * (p + q)
    dH, dW = G @ W, G.t() @ h
    e_H = e_G @ W.abs() + (V + 8) * EPS * (G.abs() @ W.abs())
    e_W = e_G.t() @ h.abs() + (T + 8) * EPS * (G.abs().t() @ h.abs())
    return dH, e_H + dH.abs() * half, dW, e_W + dW.abs() * half


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lean,big", [(0, 1), (9, 1), (12, 1), (15, 1), (15, 30), (40, 1)])
def test_gradient_from_saved_states_of_a_sure_student(lean, big, dtype):
    t = DT[dtype]
    H, W, idx, vals, mask = sure_student(t, lean, big)
    Hp, Wp = H.cuda().requires_grad_(True), W.cuda().requires_grad_(True)
    args = idx.cuda(), vals.cuda(), mask.cuda()
    ckl.chunked_kl_loss(Hp, Wp, *args, chunk=128, save_8bit=True).backward()
    held = ckl.act_decode(*ckl.act_encode(H.cuda()), dtype=t).double().cpu()
    dH, e_H, dW, e_W = loss_gradient(held, W.double(), idx, vals, mask, HALF[t] * (1 + 2.0 ** -6))
    assert ((Hp.grad.double().cpu() - dH).abs() <= e_H).all()
    assert ((Wp.grad.double().cpu() - dW).abs() <= e_W).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lean,big", [(0, 1), (12, 1), (15, 1), (15, 30)])
def test_gradient_through_the_norm_of_a_sure_student(lean, big, dtype):
    t = DT[dtype]
    X, W, idx, vals, mask = sure_student(t, lean, big)
    W = (W.float() * (X.double() ** 2).mean().sqrt()).to(t)  # logits of the same size behind the norm
    nw = (1 + normal((X.shape[1],), torch.float32, 9, 0.1)).to(t)
    leaves = [v.cuda().requires_grad_(True) for v in (X, W, nw)]
    ckl.chunked_kl_loss(leaves[0], leaves[1], idx.cuda(), vals.cuda(), mask.cuda(), chunk=128, save_8bit=True,
                        norm_weight=leaves[2]).backward()
    _, codes, exps, rstd = ckl.norm_forward(X.cuda(), nw.cuda())
    h = ckl.act_decode(codes, exps, rstd, nw.cuda(), dtype=t).double().cpu()
    half = HALF[t] * (1 + 2.0 ** -6)
    dH, e_H, dW, e_W = loss_gradient(h, W.double(), idx, vals, mask, half)
    assert ((leaves[1].grad.double().cpu() - dW).abs() <= e_W).all()
    # the norm's own gradient, linear in dH: its error passes through, and the norm's sums add theirs
    r, w = rstd.double().cpu()[:, None], nw.double()
    n = ckl.act_decode(codes, exps, dtype=torch.float32).double().cpu() * r
    dX = r * (dH * w - n * (dH * w * n).mean(1, keepdim=True))
    e_X = r * (e_H * w.abs() + n.abs() * (e_H * w.abs() * n.abs()).mean(1, keepdim=True))
    mag = r * ((dH * w).abs() + n.abs() * (dH * w * n).abs().mean(1, keepdim=True))
    assert ((leaves[0].grad.double().cpu() - dX).abs() <= e_X + mag * 240 * EPS + dX.abs() * half).all()
    dn = (dH * n).sum(0)
    e_n = (e_H * n.abs()).sum(0) + (len(X) + 56) * EPS * (dH * n).abs().sum(0) + dn.abs() * half
    assert ((leaves[2].grad.double().cpu() - dn).abs() <= e_n).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_saved_states_are_the_direct_calls_with_their_own_lse(norm, masked, dtype):
    X, W, idx, tl, mask = loss_inputs(dtype=DT[dtype], seed=20)
    mask = mask if masked else None
    nw = (1 + normal((72,), torch.float32, 9, 0.2)).to(DT[dtype]).cuda() if norm else None
    leaves = [t.clone().requires_grad_(True) for t in (X, W)] + ([nw.clone().requires_grad_(True)] if norm else [])
    kw = dict(chunk=128, save_8bit=True, norm_weight=leaves[2] if norm else None)
    loss = ckl.chunked_kl_loss(leaves[0], leaves[1], idx, tl, mask, **kw)
    (3.0 * loss).backward()
    g = torch.tensor([3.0], device="cuda")
    if norm:
        y, codes, exps, rstd = ckl.norm_forward(X, nw)
        held = ckl.act_decode(codes, exps, rstd, nw, dtype=X.dtype)
    else:
        y, (codes, exps) = X, ckl.act_encode(X)
        held = ckl.act_decode(codes, exps, dtype=X.dtype)
    plain, _, _ = ckl.forward(y, W, idx, tl, mask, chunk=128)
    assert same_bits(loss.detach().reshape(1), plain)  # the loss is that of the exact states
    with torch.no_grad():
        assert same_bits(ckl.chunked_kl_loss(leaves[0], leaves[1], idx, tl, mask, **kw).reshape(1), plain)
    _, lse, _ = ckl.forward(held, W, idx, tl, mask, chunk=128)
    dH, dW = ckl.backward(held, W, idx, tl, mask, lse, g, chunk=128, dh_dtype=X.dtype, dw_dtype=W.dtype)
    want = [*ckl.norm_backward(dH, codes, exps, rstd, nw)] if norm else [dH]
    want.insert(1, dW)
    for leaf, ref in zip(leaves, want):
        assert same_bits(leaf.grad, ref)
    if norm:  # only the norm's weight asked for
        only = nw.clone().requires_grad_(True)
        (3.0 * ckl.chunked_kl_loss(X, W, idx, tl, mask, chunk=128, save_8bit=True, norm_weight=only)).backward()
        assert same_bits(only.grad, want[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_masked_rows_may_hold_anything(norm, fused, dtype):
    # a masked row contributes nothing, whatever the padding of a batch left in it
    if fused and not norm:
        pytest.skip("the one-call loss keeps no hidden states")
    X, W, idx, tl, mask = loss_inputs(dtype=DT[dtype], seed=30)
    nw = (1 + normal((72,), torch.float32, 9, 0.2)).to(DT[dtype]).cuda()

    def grads(x, m):
        leaves = [x.clone().requires_grad_(True), W.clone().requires_grad_(True), nw.clone().requires_grad_(True)]
        loss = ckl.chunked_kl_loss(leaves[0], leaves[1], idx, tl, m, chunk=128, fused=fused, save_8bit=True,
                                   norm_weight=leaves[2] if norm else None)
        loss.backward()
        return [loss.detach(), *(v.grad for v in leaves[:3 if norm else 2])]
    for m in (mask, mask.to(torch.uint8), torch.zeros_like(mask)):
        want = grads(X, m)
        for bad in (math.nan, math.inf, -math.inf, torch.finfo(X.dtype).max, 0.0):
            x = X.clone()
            x[m == 0, ::2] = bad
            got = grads(x, m)
            assert not got[1][m == 0].any()
            for a, b in zip(got, want):
                assert same_bits(a, b)
    for off in (mask.cpu(), mask.float()):
        with pytest.raises(ValueError):
            ckl.chunked_kl_loss(X.clone().requires_grad_(True), W, idx, tl, off, chunk=128, fused=fused,
                                save_8bit=True, norm_weight=nw if norm else None)


# ------------------------------------------------------ off a 16-byte boundary --
def off_by(t, n):
    """t's values in a contiguous tensor that begins n elements behind a 16-byte boundary."""
    flat = torch.full((t.numel() + n,), math.nan if t.is_floating_point() else 1, dtype=t.dtype, device="cuda")
    flat[n:] = t.reshape(-1)
    out = flat[n:].view(t.shape)
    assert out.is_contiguous() and out.data_ptr() % 16 == n * t.element_size() % 16
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_topk_of_row_slices(dtype):
    # rows of an odd vocabulary begin anywhere: a slice of them is contiguous all the same
    for T, V, K in ((5, 333, 7), (9, 50021, 40)):
        z = normal((T, V), DT[dtype], V, 2.0).cuda()
        mask = torch.tensor([True, False, True] * 3, device="cuda")[:T]
        whole = ckl.teacher_topk(z, K, mask, 1)
        for i in range(T):
            for part in (slice(i, i + 1), slice(i, T)):
                for a, b in zip(ckl.teacher_topk(z[part], K, mask[part], 1), whole):
                    # a log-sum-exp (here below 13) may move by its roundings where the split is another one, and
                    # the values (below 25) with it: twice check_topk's bound
                    if a.dtype == torch.int32:
                        assert torch.equal(a, b[part])
                    else:
                        torch.testing.assert_close(a, b[part], rtol=0, atol=2 * (V / 256 + 40 + 4 + 26 + 50) * EPS)
        one = ckl.teacher_topk(z.view(1, T, V)[:, -1], K)
        assert torch.equal(one[0][0], ckl.teacher_topk(z, K)[0][-1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 3])
def test_inputs_off_a_boundary(n, dtype):
    t, T, V, d = DT[dtype], 300, 77, 40
    W, x, dy = (normal(s, t, i).cuda() for i, s in enumerate(((V, d), (T, d), (T, d))))
    w = (1 + normal((d,), torch.float32, 4, 0.1)).to(t).cuda()
    tok = torch.randint(-1, V + 1, (T,), generator=torch.Generator().manual_seed(1)).cuda()
    o = lambda v: off_by(v, n)  # noqa: E731
    assert same_bits(ckl.embedding_forward(o(W), o(tok), 2.0), ckl.embedding_forward(W, tok, 2.0))
    assert same_bits(ckl.embedding_backward(o(dy), o(tok), V), ckl.embedding_backward(dy, tok, V))
    codes, exps = ckl.act_encode(x)
    for a, b in zip(ckl.act_encode(o(x)), (codes, exps)):
        assert same_bits(a, b)
    y, _, _, rstd = want = ckl.norm_forward(x, w)
    for a, b in zip(ckl.norm_forward(o(x), o(w)), want):
        assert same_bits(a, b)
    assert same_bits(ckl.act_decode(o(codes), o(exps), o(rstd), o(w), dtype=t),
                     ckl.act_decode(codes, exps, rstd, w, dtype=t))
    dx, dw = ckl.norm_backward(dy, codes, exps, rstd, w)
    for a, b in zip(ckl.norm_backward(o(dy), o(codes), o(exps), o(rstd), o(w)), (dx, dw)):
        assert same_bits(a, b)
    # through autograd, with a gradient that begins off a boundary (a slice of a larger one)
    X, Wt = o(x).requires_grad_(True), o(w).requires_grad_(True)
    out = ckl.rms_norm_8bit(X, Wt)
    assert same_bits(out.detach(), y)
    for a, b in zip(torch.autograd.grad(out, (X, Wt), o(dy)), (dx, dw)):
        assert same_bits(a, b)
    E = o(W).requires_grad_(True)
    got, = torch.autograd.grad(ckl.embedding(E, o(tok), 2.0), E, o(dy))
    assert same_bits(got, ckl.embedding_backward(dy, tok, V, 2.0, dw_dtype=t))
    # what is written in place cannot be a copy
    with pytest.raises(B.CklError, match="aligned"):
        ckl.embedding_backward(dy, tok, V, add_to=o(torch.zeros(V, d, device="cuda")))


# ------------------------------------------------------ ids at their type's ends --
@pytest.mark.parametrize("T", [9, 300, 9000])
def test_ids_and_offsets_at_the_ends_of_their_type(T):
    V, d, big = 100, 16, 2 ** 63 - 1
    W, dY = normal((V, d), torch.float32, 1).cuda(), normal((T, d), torch.float32, 2).cuda()
    for off, inside in ((big - V, [0, V - 1]), (2 ** 62, [5]), (0, [0, V - 1])):
        tok = [-2 ** 63, -2 ** 63 + 1, -1, big, -2 ** 63 + off % 2, big - 1]
        tok = [t for t in tok if not off <= t < off + V] + [off + i for i in inside]
        tok = torch.tensor((tok * T)[:T], device="cuda")
        at = torch.tensor([t - off if off <= t < off + V else -1 for t in tok.tolist()], device="cuda")
        assert same_bits(ckl.embedding_forward(W, tok, 2.0, v_offset=off), ckl.embedding_forward(W, at, 2.0))
        assert same_bits(ckl.embedding_backward(dY, tok, V, 2.0, v_offset=off), ckl.embedding_backward(dY, at, V, 2.0))
    for off in (big, big - V + 1):
        with pytest.raises(B.CklError, match="v_offset"):
            ckl.embedding_forward(W, tok, v_offset=off)
        with pytest.raises(B.CklError, match="v_offset"):
            ckl.embedding_backward(dY, tok, V, v_offset=off)


# ------------------------------------------- around workspaces and outputs --
class Guarded:
    """Arrays between guard bytes, from a 16-byte boundary that is not a page's."""

    def __init__(self):
        self.buffers = []

    def __call__(self, shape, dtype, fill=0xAB):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 2 * 4096,), 0xAB, dtype=torch.uint8, device="cuda")
        body = buf[4112:4112 + n]
        body.fill_(fill)
        self.buffers.append((buf, n))
        return body.view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.buffers:
            assert (buf[:4112] == 0xAB).all() and (buf[4112 + n:] == 0xAB).all()


def workspace(guarded, fn, *sizes):
    need = ctypes.c_size_t(0)
    B.check(fn(*sizes, ctypes.byref(need)))
    return guarded((need.value,), torch.uint8, 0xFF), need.value


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,K", [(1, 201088, 4096), (3, 8200, 100), (7, 50021, 1000), (1030, 301, 17)])
def test_topk_writes_its_own_arrays_only(T, V, K, dtype):
    lib, g = B.load_library(), Guarded()
    z = g((T, V), DT[dtype])
    z.copy_(normal((T, V), DT[dtype], T + V, 2.0))
    idx, val, lse = g((T, K), torch.int32), g((T, K), torch.float32), g((T,), torch.float32)
    ws, n = workspace(g, lib.ckl_topk_workspace_size, T, V, K)
    assert (n > 0) == (V > 50000)  # several segments to a row
    B.check(lib.ckl_teacher_topk(z.data_ptr(), int(dtype == "bf16"), T, V, K, 0, None, idx.data_ptr(), val.data_ptr(),
                                 lse.data_ptr(), ws.data_ptr(), n, None))
    g.check()
    for a, b in zip((idx, val, lse), ckl.teacher_topk(z.clone(), K)):
        assert same_bits(a, b)


@pytest.mark.parametrize("add", [0, 1])
@pytest.mark.parametrize("dtype,grad", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,V,d", [(200, 333, 40), (257, 333, 40), (8193, 333, 8), (70001, 50, 2056), (300, 1, 16)])
def test_embedding_grad_writes_its_own_arrays_only(T, V, d, dtype, grad, add):
    lib, g = B.load_library(), Guarded()
    dY, tok = g((T, d), DT[dtype]), g((T,), torch.int64)
    dY.copy_(normal((T, d), DT[dtype], T))
    tok.copy_(torch.randint(-2, V + 2, (T,), generator=torch.Generator().manual_seed(T)))
    dW = g((V, d), DT[grad], 0)
    ws, n = workspace(g, lib.ckl_embedding_workspace_size, T, d, V)
    B.check(lib.ckl_embedding_backward(dY.data_ptr(), int(dtype == "bf16"), T, d, tok.data_ptr(), 8, V, 0, 1.5,
                                       dW.data_ptr(), int(grad == "bf16"), add, ws.data_ptr(), n, None))
    g.check()
    want = ckl.embedding_backward(dY.clone(), tok.clone(), V, 1.5, dw_dtype=DT[grad])
    assert torch.equal(dW, want)  # (added to zeros: the same sums)


@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,d", [(1, 8), (1025, 72), (2050, 520), (5, 8200), (3, 32776)])
def test_norm_writes_its_own_arrays_only(T, d, dtype, wtype):
    lib, g = B.load_library(), Guarded()
    t, bf, wbf, nb = DT[dtype], int(dtype == "bf16"), int(wtype == "bf16"), -(-d // 32)
    x, dy, w = g((T, d), t), g((T, d), t), g((d,), DT[wtype])
    for i, v in enumerate((x, dy, w)):
        v.copy_(normal(tuple(v.shape), v.dtype, i))
    y, codes, exps, rstd = g((T, d), t), g((T, d), torch.int8), g((T, nb), torch.uint8), g((T,), torch.float32)
    B.check(lib.ckl_norm_forward(x.data_ptr(), bf, T, d, w.data_ptr(), wbf, 1e-6, y.data_ptr(), codes.data_ptr(),
                                 exps.data_ptr(), rstd.data_ptr(), None))
    dx, dw, out = g((T, d), t), g((d,), DT[wtype]), g((T, d), t)
    ws, n = workspace(g, lib.ckl_norm_workspace_size, T, d)
    B.check(lib.ckl_norm_backward(dy.data_ptr(), bf, T, d, codes.data_ptr(), exps.data_ptr(), rstd.data_ptr(),
                                  w.data_ptr(), wbf, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), n, None))
    B.check(lib.ckl_act_decode(codes.data_ptr(), exps.data_ptr(), T, d, rstd.data_ptr(), w.data_ptr(), wbf,
                               out.data_ptr(), bf, None))
    g.check()
    for a, b in zip((y, codes, exps, rstd), ckl.norm_forward(x.clone(), w.clone())):
        assert same_bits(a, b)
    for a, b in zip((dx, dw), ckl.norm_backward(dy.clone(), codes.clone(), exps.clone(), rstd.clone(), w.clone())):
        assert same_bits(a, b)
    assert same_bits(out, ckl.act_decode(codes.clone(), exps.clone(), rstd.clone(), w.clone(), dtype=t))


# --------------------------------------------------------------- captured --
@pytest.mark.parametrize("fused", [False, True])
def test_masked_gradients_replay_with_new_inputs(fused):
    # the norm before the loss with a mask, forward and backward in one graph
    def inputs(seed):
        X, W, idx, tl, mask = loss_inputs(seed=seed)
        X[~mask, ::3] = math.nan
        return [X, W, idx, tl, mask, (1 + normal((72,), torch.float32, seed + 5, 0.1)).cuda()]

    def grads(X, W, idx, tl, mask, nw):
        leaves = [v.detach().requires_grad_(True) for v in (X, W, nw)]
        loss = ckl.chunked_kl_loss(leaves[0], leaves[1], idx, tl, mask, chunk=128, fused=fused, save_8bit=True,
                                   norm_weight=leaves[2])
        return [loss.detach(), *torch.autograd.grad(loss, leaves)]
    ins = inputs(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads(*ins)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = grads(*ins)
    for seed in (1, 40, 80, 40):
        for a, b in zip(ins, inputs(seed)):
            a.copy_(b)
        want = [t.clone() for t in grads(*inputs(seed))]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert bool(torch.isfinite(a).all()) and same_bits(a, b)
