"""Log probabilities and entropies from hidden states and head on the GPU, their gradients, and a step that uses all
of what lies between a model's last block and its training signal.

H and W hold small whole numbers times a power of two, so that every logit is exact in fp32 whatever the order of its
sum: the rows are then held to the tolerances of logits that are given (tests/test_logprob_gpu.py).  Gradients: G
rounded once to the inputs' type, sums of V or T terms in fp32, one rounding to the outputs' type."""
import math

import pytest
import torch

import chunked_kl_loss_amd as ckl
from tests.test_logprob_gpu import DT, EPS, HALF, dz_reference, gen, normal, rows_reference, same_bits, some_tokens, within

pytestmark = pytest.mark.gpu


def grid(shape, dtype, seed, step, most=8):
    return (torch.randint(-most, most + 1, shape, generator=gen(seed)).float() * step).to(dtype)


def inputs(T, d, V, dtype, seed=0):
    # logits of a standard deviation near 2: steps are powers of two
    hs = 0.25
    ws = 2.0 ** round(math.log2(2.0 / (4.9 * hs * 4.9 * math.sqrt(d))))
    H, W = grid((T, d), dtype, seed, hs), grid((V, d), dtype, seed + 1, ws)
    return H, W, some_tokens(T, V, seed + 2)


def check(H, W, tok, mask=None, chunk=2048, train=True, out_types=None):
    T, V = H.shape[0], W.shape[0]
    dtype = H.dtype
    Hg, Wg = H.cuda().requires_grad_(train), W.cuda().requires_grad_(train)
    m = None if mask is None else mask.cuda()
    logprob, entropy = ckl.head_logprobs(Hg, Wg, tok.cuda(), mask=m, chunk=chunk)
    H64, W64 = H.double().cuda(), W.double().cuda()
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    H64 = torch.where(keep.cuda()[:, None], H64, 0.0)  # (masked rows may hold anything)
    z = (H64 @ W64.t()).cpu()
    r = rows_reference(z, tok, mask)
    assert within(logprob.detach(), r["logprob"], r["tol_lp"] + 4 * EPS * r["lse"].abs())
    assert within(entropy.detach(), r["entropy"], r["tol_ent"])
    if not train:
        return
    a, b = normal((T,), torch.float32, 3), normal((T,), torch.float32, 4, 0.3)
    a[::5], b[::5] = 0.0, 0.0   # rows without a gradient
    dH, dW = torch.autograd.grad((logprob, entropy), (Hg, Wg), (a.cuda(), b.cuda()))
    G, tol = dz_reference(z, tok, r, a, b)
    G[~keep], tol[~keep] = 0.0, 0.0
    G, tol = G.cuda(), tol.cuda()
    if dtype == torch.bfloat16:
        tol = tol + HALF[dtype] * G.abs()
    for got, op, mag, n in ((dH, G @ W64, (tol + (V + 8) * EPS * G.abs()) @ W64.abs(), V),
                            (dW, G.t() @ H64, (tol + (T + 8) * EPS * G.abs()).t() @ H64.abs(), T)):
        assert got.dtype == dtype
        assert within(got, op, mag + HALF[dtype] * op.abs() + 1e-37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,V", [(1, 8, 1), (1, 16, 700), (3, 72, 255), (8, 64, 257), (16, 200, 5003), (33, 520, 1000),
                                   (64, 72, 4100), (65, 64, 513), (128, 136, 300), (129, 128, 1030), (255, 64, 256),
                                   (257, 264, 2049), (300, 72, 1500), (700, 64, 900)])
def test_sizes(T, d, V, dtype):
    check(*inputs(T, d, V, DT[dtype], T + V))


@pytest.mark.parametrize("T", [1, 2, 5, 16, 31, 32, 33, 64, 100])
def test_few_rows_of_a_large_head(T):
    check(*inputs(T, 320, 20011, torch.bfloat16, T), train=T in (1, 33))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunk", [1, 256, 300, 100000, 2 ** 62])
def test_chunks(chunk, dtype):
    check(*inputs(600, 72, 1500, DT[dtype], 1), chunk=chunk)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("share", [None, 0.98, 0.5])
def test_more_rows_than_a_launch_takes(share, dtype):
    T = 17000
    H, W, tok = inputs(T, 16, 300, DT[dtype], 1)
    mask = None if share is None else torch.rand(T, generator=gen(2)) < share
    check(H, W, tok, mask, chunk=4096)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,chunk", [(8192, 500, 2048), (6001, 600, 512), (3000, 64, 1 << 20)])
def test_many_rows_of_few_words(T, V, chunk, dtype):
    check(*inputs(T, 136, V, DT[dtype], 1), chunk=chunk)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["some", "all", "none", "one", "packed"])
def test_masks_and_tokens_outside(kind, dtype):
    T, V = 700, 900
    H, W, tok = inputs(T, 64, V, DT[dtype], 5)
    tok[::4] = torch.tensor([-1, -100, V, 2 ** 31, 2 ** 40, -2 ** 63, 2 ** 63 - 1]).repeat(T)[:len(tok[::4])]
    mask = {"some": torch.rand(T, generator=gen(1)) < 0.6, "all": torch.ones(T, dtype=torch.bool),
            "none": torch.zeros(T, dtype=torch.uint8), "one": torch.arange(T) == 444,
            "packed": torch.arange(T) % 350 > 80}[kind]
    H[~mask.bool()] = math.nan  # masked rows may hold anything
    check(H, W, tok, mask, chunk=256)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,d,V,chunk", [(200, 72, 3001, 1), (200, 264, 20001, 20), (31, 328, 12345, 40),
                                         (513, 72, 9000, 200)])
def test_few_rows_in_blocks_of_words(T, d, V, chunk, masked):
    H, W, tok = inputs(T, d, V, torch.bfloat16, 3)
    mask = (torch.rand(T, generator=gen(1)) < 0.6) if masked else None
    check(H, W, tok, mask, chunk=chunk)


def test_one_block_of_millions_of_rows():
    check(*inputs(2_200_000, 8, 8, torch.bfloat16, 3), chunk=2 ** 40)


def test_larger_products():
    check(*inputs(512, 512, 30011, torch.bfloat16, 3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_random_states_agree_with_logits_in_memory(dtype):
    # z in fp32 carries d roundings of its products' magnitudes
    T, d, V = 70, 256, 3001
    H, W, tok = normal((T, d), DT[dtype], 1), normal((V, d), DT[dtype], 2, d ** -0.5), some_tokens(T, V, 3)
    z = H.double() @ W.double().t()
    off = float((d * 2 * EPS * (H.double().abs() @ W.double().abs().t())).max())
    r = rows_reference(z, tok)
    lp, ent, lse = ckl.head_logprobs_forward(H.cuda(), W.cuda(), tok.cuda())
    assert within(lse, r["lse"], r["tol_lse"] + off) and within(lp, r["logprob"], r["tol_lp"] + 2 * off)
    # |d entropy| <= off * sum q |log q + entropy| <= off * 2 entropy
    assert within(ent, r["entropy"], r["tol_ent"] + off * 2 * r["entropy"])


def test_only_the_gradients_asked_for():
    H, W, tok = (t.cuda() for t in inputs(300, 64, 900, torch.bfloat16, 5))
    lp, ent, lse = ckl.head_logprobs_forward(H, W, tok)
    a = normal((300,), torch.float32, 1).cuda()
    both = ckl.head_logprobs_backward(a, a, H, W, tok, lse, ent)
    dh, none = ckl.head_logprobs_backward(a, a, H, W, tok, lse, ent, need_dw=False)
    assert none is None and same_bits(dh, both[0])
    none, dw = ckl.head_logprobs_backward(a, a, H, W, tok, lse, ent, need_dh=False)
    assert none is None and same_bits(dw, both[1]) and dw.dtype == torch.float32
    assert ckl.head_logprobs_backward(a, a, H, W, tok, lse, ent, need_dh=False, need_dw=False) == (None, None)
    zero = torch.zeros_like(a)
    for got, want in (((a, None), (a, zero)), ((None, a), (zero, a)), ((None, None), (zero, zero))):
        x, y = (ckl.head_logprobs_backward(*g, H, W, tok, lse, ent) for g in (got, want))
        assert same_bits(x[0], y[0]) and same_bits(x[1], y[1])
    h32 = ckl.head_logprobs_backward(a, a, H, W, tok, lse, ent, dh_dtype=torch.float32, dw_dtype=torch.bfloat16)
    assert same_bits(h32[0].bfloat16(), both[0]) and same_bits(h32[1], both[1].bfloat16())
    Wp = W.clone().requires_grad_(True)  # a frozen body
    (dw,) = torch.autograd.grad(ckl.head_logprobs(H, Wp, tok)[0], (Wp,), a)
    assert same_bits(dw, ckl.head_logprobs_backward(a, None, H, W, tok, lse, ent, dw_dtype=torch.bfloat16)[1])


def test_the_cross_entropy_is_the_loss_of_a_sure_teacher():
    T, d, V = 300, 72, 1500
    H, W, tok = (t.cuda() for t in inputs(T, d, V, torch.bfloat16, 9))
    loss, lse, rows = ckl.forward(H, W, tok[:, None].int().contiguous(), torch.zeros(T, 1, device="cuda"), want_row_loss=True)
    lp, ent, lse2 = ckl.head_logprobs_forward(H, W, tok)
    assert torch.allclose(-lp, rows, atol=1e-5, rtol=1e-6) and torch.allclose(lse, lse2, atol=1e-5, rtol=1e-6)


def test_gradients_against_differences():
    # third derivatives: step^2 / 6 of 30 times the rows' |dz|^3 a row, dz = step H dW below 1
    T, d, V, step = 5, 16, 40, 1e-2
    H, W, tok = normal((T, d), torch.float32, 1), normal((V, d), torch.float32, 2, 0.4), some_tokens(T, V, 3)
    a, b = normal((T,), torch.float64, 3), normal((T,), torch.float64, 4)

    def value(H, W):
        lp, ent = ckl.head_logprobs(H, W, tok.cuda())
        return (lp.double() * a.cuda() + ent.double() * b.cuda()).sum()
    Hg, Wg = H.cuda().requires_grad_(True), W.cuda().requires_grad_(True)
    grads = torch.autograd.grad(value(Hg, Wg), (Hg, Wg))
    r = rows_reference(H.double() @ W.double().t(), tok)
    off = float((d * 2 * EPS * (H.double().abs() @ W.double().abs().t())).max())
    noise = float((a.abs() * (r["tol_lp"] + 2 * off) + b.abs() * (r["tol_ent"] + 2 * off * r["entropy"])).sum())
    for k, g in enumerate(grads):
        for i in range(4):
            u = normal(g.shape, torch.float32, 20 + i)
            u = u / ((u @ W.t()) if k == 0 else (H @ u.t())).abs().max()  # logits move by at most 1
            p, m = ([t + (s * u if j == k else 0) for j, t in enumerate((H, W))] for s in (step, -step))
            diff = float(value(p[0].cuda(), p[1].cuda()) - value(m[0].cuda(), m[1].cuda())) / (2 * step)
            got = float((g.double().cpu() * u.double()).sum())
            assert abs(diff - got) < noise / step + step ** 2 / 6 * 30 * float(a.abs().sum() + 4 * b.abs().sum())


def test_layouts_and_empty_batches():
    H, W, tok = inputs(24, 64, 300, torch.bfloat16, 2)
    H, W, tok = H.view(4, 6, 64).cuda(), W.cuda(), tok.view(4, 6).cuda()
    mask = torch.rand(4, 6, generator=gen(1)).cuda() < 0.5
    lp, ent = ckl.head_logprobs(H, W, tok, mask)
    flat = ckl.head_logprobs(H.view(24, 64), W, tok.view(24), mask.view(24))
    assert lp.shape == (4, 6) and same_bits(lp.view(24), flat[0]) and same_bits(ent.view(24), flat[1])
    got = ckl.head_logprobs(H.transpose(0, 1), W.t().contiguous().t(), tok.t(), mask.t())
    assert same_bits(got[0], lp.t().contiguous()) and same_bits(got[1], ent.t().contiguous())
    one = ckl.head_logprobs(H[1, 2], W, tok[1, 2])
    assert one[0].shape == ()
    for mk in (None, mask[:0]):
        e, w = H[:0].clone().requires_grad_(True), W.clone().requires_grad_(True)
        lp, ent = ckl.head_logprobs(e, w, tok[:0], mk)
        dh, dw = torch.autograd.grad((lp, ent), (e, w), (torch.zeros_like(lp), torch.zeros_like(ent)))
        assert lp.shape == (0, 6) and dh.shape == e.shape and not dw.any()
    lp, ent = ckl.head_logprobs(H.requires_grad_(True), W, tok)
    (dh,) = torch.autograd.grad(lp.sum(), (H,))  # a gradient with stride 0
    (want,) = torch.autograd.grad(ckl.head_logprobs(H, W, tok)[0], (H,), torch.ones(4, 6, device="cuda"))
    assert same_bits(dh, want)


def test_neighbours_and_rows_past_the_last():
    # nothing behind H's last row or W's is read into a result, nothing around the outputs written
    import ctypes

    from chunked_kl_loss_amd import _binding as B
    lib = B.load_library()
    for T, d, V, dt in ((5, 72, 301, torch.bfloat16), (130, 64, 257, torch.bfloat16), (131, 40, 130, torch.float32)):
        H, W, tok = inputs(T, d, V, dt, 1)
        Hb, Wb = torch.full((T + 300, d), math.nan, dtype=dt, device="cuda"), torch.full((V + 300, d), math.nan, dtype=dt,
                                                                                        device="cuda")
        Hb[:T], Wb[:V] = H.cuda(), W.cuda()
        want = ckl.head_logprobs_forward(H.cuda(), W.cuda(), tok.cuda())
        a = normal((T,), torch.float32, 1).cuda()
        wdh, wdw = ckl.head_logprobs_backward(a, a, H.cuda(), W.cuda(), tok.cuda(), want[2], want[1])
        code, tk = int(dt == torch.bfloat16), tok.cuda()
        rows = [torch.full((T + 64,), -7.0, device="cuda") for _ in range(3)]
        dH = torch.full((T * d + 64,), -7.0, dtype=dt, device="cuda")
        dW = torch.full((V * d + 64,), -7.0, device="cuda")
        at = [r.data_ptr() + 64 for r in rows]
        for which in (0, 1):
            need = ctypes.c_size_t(0)
            B.check(lib.ckl_head_workspace_size(T, d, V, 100, code, code, 0, 0, which, ctypes.byref(need)))
            ws = torch.full((need.value + 64,), 0xFF, dtype=torch.uint8, device="cuda")
            if which == 0:
                B.check(lib.ckl_head_logprobs(Hb.data_ptr(), Wb.data_ptr(), code, T, d, V, tk.data_ptr(), 8, None, 100,
                                              *at, ws.data_ptr(), need.value, None))
            else:
                B.check(lib.ckl_head_logprobs_backward(
                    Hb.data_ptr(), Wb.data_ptr(), code, T, d, V, tk.data_ptr(), 8, None, 100, at[2], at[1],
                    a.data_ptr(), a.data_ptr(), dH.data_ptr() + 16 * dH.element_size(), code, dW.data_ptr() + 64, 0,
                    ws.data_ptr(), need.value, None))
            torch.cuda.synchronize()
            assert (ws[need.value:] == 0xFF).all()
        for b, n, w in [(r, T, x) for r, x in zip(rows, want)] + [(dH, T * d, wdh), (dW, V * d, wdw)]:
            assert (b[:16] == -7).all() and (b[16 + n:] == -7).all()
            assert torch.allclose(b[16:16 + n].float(), w.reshape(-1).float(), rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("T,d,V,chunk", [(40, 2880, 800_000, 2048), (2900, 64, 800_000, 1 << 20), (3, 8, 4_000_000, 1)])
def test_offsets_past_32_bits(T, d, V, chunk):
    # W, or the block of logit gradients, holds more than 2^31 elements; the last holds the most words there are
    H = grid((T, d), torch.bfloat16, 1, 0.25).cuda()
    gen_cuda = torch.Generator("cuda")
    gen_cuda.manual_seed(2)
    step = 2.0 ** round(math.log2(2.0 / (4.9 * 0.25 * 4.9 * math.sqrt(d))))
    W = torch.randint(-8, 9, (V, d), generator=gen_cuda, device="cuda", dtype=torch.int8).bfloat16() * step
    tok = some_tokens(T, V, 3)
    tok[-1] = V - 1
    rows = torch.tensor(sorted({0, 1, T // 2, T - 2, T - 1}))
    tok = tok.cuda()
    lp, ent, lse = ckl.head_logprobs_forward(H, W, tok)
    a, b = normal((T,), torch.float32, 3), normal((T,), torch.float32, 4, 0.3)
    dH, dW = ckl.head_logprobs_backward(a.cuda(), b.cuda(), H, W, tok, lse, ent, chunk=chunk, dw_dtype=torch.bfloat16)
    # some rows over all words, by blocks of words
    blocks = range(0, V, 50_000)
    z = torch.cat([(H[rows].double() @ W[v:v + 50_000].double().t()).cpu() for v in blocks], 1)
    r = rows_reference(z, tok.cpu()[rows])
    assert within(lse[rows], r["lse"], r["tol_lse"])
    assert within(lp[rows], r["logprob"], r["tol_lp"] + 4 * EPS * r["lse"].abs())
    assert within(ent[rows], r["entropy"], r["tol_ent"])
    G, tol = dz_reference(z, tok.cpu()[rows], r, a[rows], b[rows])
    tol = tol + (HALF[torch.bfloat16] + (V + 8) * EPS) * G.abs()
    want, off = torch.zeros(len(rows), d, dtype=torch.float64), torch.zeros(len(rows), d, dtype=torch.float64)
    for v in blocks:
        part = W[v:v + 50_000].double()
        want += (G[:, v:v + 50_000].cuda() @ part).cpu()
        off += (tol[:, v:v + 50_000].cuda() @ part.abs()).cpu()
    assert within(dH[rows], want, off + HALF[torch.bfloat16] * want.abs())
    # all rows over some words
    words = torch.cat([torch.arange(3), torch.arange(V // 2, V // 2 + 300), torch.arange(V - 300, V)])
    at = torch.full((V,), -1)
    at[words] = torch.arange(len(words))
    z = (H.double() @ W[words.cuda()].double().t()).cpu()
    # (4,000,000 terms a sum: tolerances of 9.4e-4 and, with a mean distance of 10 from the maximum, 0.027)
    r = dict(lse=lse.double().cpu(), entropy=ent.double().cpu(), tol_lse=torch.full((T,), 1e-3), tol_ent=torch.full((T,), 3e-2))
    inside = (tok.cpu() >= 0) & (tok.cpu() < V)
    mapped = torch.where(inside, at[torch.where(inside, tok.cpu(), 0)], -1)
    G, tol = dz_reference(z, mapped, r, torch.where(inside, a, 0.0), b)
    G = G - torch.where(inside & (mapped < 0), a.double(), 0.0)[:, None] * torch.exp(z - r["lse"][:, None])
    tol = tol + (HALF[torch.bfloat16] + (T + 8) * EPS) * G.abs() + 1e-3 * a.abs().double()[:, None] * torch.exp(z - r["lse"][:, None])
    want = G.t().cuda() @ H.double()
    assert within(dW[words.cuda()], want, tol.t().cuda() @ H.double().abs() + HALF[torch.bfloat16] * want.abs() + 1e-37)


# ------------------------------------------------------- all of it, used together --
def full_step(x, res, nw, W, tok, idx, tl, mask, state, adv):
    """A branch's output behind dropout, the residual's sum and the norm into the head: distillation, a policy term
    with a weight for each token, and a bonus on the entropy."""
    x, res, nw, W = (t.detach().requires_grad_(True) for t in (x, res, nw, W))
    y, h = ckl.add_rms_norm(x, res, nw, 1e-6, 0.2, state, 3)
    lp, ent = ckl.head_logprobs(y, W, tok, mask, chunk=256)
    kl = ckl.chunked_kl_loss(y, W, idx, tl, mask, chunk=256)
    loss = kl - (adv * lp).sum() / 100 - 0.01 * ent.mean() + 1e-3 * h.float().square().mean()
    return [loss.detach(), lp.detach(), ent.detach(), h.detach(), *torch.autograd.grad(loss, (x, res, nw, W))]


def full_inputs(seed, T=330, d=72, V=700, K=9, dtype=torch.float32):
    teacher = normal((T, V), torch.float32, seed + 7, 2.0).cuda()
    idx, tl, _ = ckl.teacher_topk(teacher, K)
    return [normal((T, d), dtype, seed, 0.5).cuda(), normal((T, d), dtype, seed + 1).cuda(),
            (1 + normal((d,), torch.float32, seed + 2, 0.1)).to(dtype).cuda(), normal((V, d), dtype, seed + 3, 0.2).cuda(),
            some_tokens(T, V, seed + 4).cuda(), idx, tl, (torch.rand(T, generator=gen(seed + 5)) < 0.7).cuda(),
            torch.tensor([seed, 11]).cuda(), normal((T,), torch.float32, seed + 6).cuda()]


def test_a_step_of_all_of_them_against_64_bits():
    from tests.philox import keep_mask
    ins = full_inputs(1)
    got = full_step(*ins)
    x, res, nw, W, tok, idx, tl, mask, state, adv = (t.cpu() for t in ins)
    x, res, nw, W, tl, adv = (t.double().requires_grad_(t.is_floating_point()) for t in (x, res, nw, W, tl, adv))
    keep, scale = keep_mask(x.numel(), 0.2, int(state[0]), int(state[1]) + 3)
    h = res + x * torch.from_numpy(keep).view(x.shape).double() * scale
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * nw
    logq = torch.log_softmax(y @ W.t(), 1)
    lp = torch.where(mask, logq.gather(1, tok[:, None])[:, 0], 0.0)
    ent = torch.where(mask, -(logq.exp() * logq).sum(1), 0.0)
    p = torch.softmax(tl, 1)
    kl = (torch.where(mask, (p * (torch.log_softmax(tl, 1) - logq.gather(1, idx.long()))).sum(1), 0.0)).sum() / mask.sum()
    loss = kl - (adv * lp).sum() / 100 - 0.01 * ent.mean() + 1e-3 * h.square().mean()
    want = [loss, lp, ent, h, *torch.autograd.grad(loss, (x, res, nw, W))]
    # fp32 throughout: at most 700 + 330 + 72 roundings a sum on the way, of magnitudes within 30 of the largest result
    for g, w in zip(got, want):
        assert (g.double().cpu() - w).abs().max() <= 1102 * EPS * 30 * w.abs().max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_step_of_all_of_them(dtype):
    ins = full_inputs(1, dtype=DT[dtype])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        full_step(*ins)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = full_step(*ins)
    for seed in (1, 40, 80, 40):
        new = full_inputs(seed, dtype=DT[dtype])
        for a, b in zip(ins, new):
            a.copy_(b)
        want = [t.clone() for t in full_step(*new)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        # (the loss is a sum by torch; what the library computes is the same bits)
        assert torch.allclose(outs[0], want[0], rtol=1e-5)
        assert all(same_bits(a, b) for a, b in zip(outs[1:], want[1:]))


def test_two_streams_at_once():
    ins = [full_inputs(s, T=900, dtype=torch.bfloat16) for s in (1, 30)]
    want = [[t.clone() for t in full_step(*i)] for i in ins]
    torch.cuda.synchronize()
    got, streams = [], [torch.cuda.Stream() for _ in ins]
    for s, i in zip(streams, ins):
        with torch.cuda.stream(s):
            got.append(full_step(*i))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(same_bits(a, b) for a, b in zip(g[1:], w[1:]))


@pytest.mark.parametrize("kind", ["one", "two", "rising"])
def test_tokens_that_repeat(kind):
    # many rows of one token: their states are added to one row of dW in a fixed order
    T, V = 1300, 900
    H, W, tok = inputs(T, 72, V, torch.bfloat16, 5)
    tok = {"one": torch.full((T,), 511), "two": torch.where(torch.arange(T) % 3 == 0, 256, 255),
           "rising": torch.arange(T) % V}[kind]
    check(H, W, tok, chunk=512)
    got = [ckl.head_logprobs_backward(normal((T,), torch.float32, 1).cuda(), None, H.cuda(), W.cuda(), tok.cuda(),
                                      *ckl.head_logprobs_forward(H.cuda(), W.cuda(), tok.cuda())[2:0:-1]) for _ in range(2)]
    assert same_bits(got[0][0], got[1][0]) and same_bits(got[0][1], got[1][1])


def test_gradients_lose_no_more_than_their_outputs_rounding():
    # a row's token has its largest entry of G as a rule; in bf16 it would cost dH and dW as much again as their rounding
    T, d, V = 400, 256, 3001
    H, W, tok = normal((T, d), torch.bfloat16, 1), normal((V, d), torch.bfloat16, 2, d ** -0.5), some_tokens(T, V, 3)
    a = normal((T,), torch.float32, 4)
    Hg, Wg = H.cuda().requires_grad_(True), W.cuda().requires_grad_(True)
    lp, _ = ckl.head_logprobs(Hg, Wg, tok.cuda())
    got = torch.autograd.grad(lp, (Hg, Wg), a.cuda())
    q = torch.softmax(H.double() @ W.double().t(), 1)
    G = -q * a.double()[:, None]
    G[torch.arange(T), tok] += a.double()
    for g, w in zip(got, (G @ W.double(), G.t() @ H.double())):
        off = float((g.double().cpu() - w).norm()), float((w.to(torch.bfloat16).double() - w).norm())
        assert off[0] < 1.1 * off[1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 100, 300])
@pytest.mark.parametrize("words", [(0, 1), (0, 256), (3, 260), (512, 513), (899, 900), (768, 900), (0, 900)])
def test_a_nan_in_the_head_reaches_every_row(words, T, dtype):
    H, W, tok = inputs(T, 64, 900, DT[dtype], 3)
    W[words[0]:words[1], 7] = math.nan
    for t in ckl.head_logprobs_forward(H.cuda(), W.cuda(), tok.clamp(0, 899).cuda()):
        assert t.isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [8, 100, 304])
def test_a_state_that_is_not_finite_stays_in_its_row(T, dtype):
    H, W, tok = inputs(T, 64, 900, DT[dtype], 3)
    want = ckl.head_logprobs_forward(H.cuda(), W.cuda(), tok.cuda())
    bad = torch.arange(T) % 8 == 3
    H[bad, 5] = torch.tensor([math.nan, math.inf, -math.inf]).to(H.dtype).repeat(T)[:int(bad.sum())]
    tok[bad] = 7
    W[::9, 5] = 0.0  # infinity times zero
    clean = ckl.head_logprobs_forward(torch.where(bad[:, None], 0.0, H.float()).to(H.dtype).cuda(), W.cuda(), tok.cuda())
    for t, w in zip(ckl.head_logprobs_forward(H.cuda(), W.cuda(), tok.cuda()), clean):
        assert t[bad].isnan().all() and same_bits(t[~bad], w[~bad])
    assert all(not w.isnan().any() for w in want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [8, 100, 304])
def test_logits_that_overflow_to_minus_infinity_count_for_nothing(T, dtype):
    # a row's logits are a column of W: H holds one 2^100 a row, W the logits times 2^-100, and -2^60 for -infinity
    V = 900
    z = grid((8, V), torch.float32, 1, 0.25)
    gone = torch.zeros(8, V, dtype=torch.bool)
    for r, (a, b) in enumerate([(0, 0), (0, 300), (0, 899), (1, 900), (768, 900), (897, 900), (256, 512), (0, 900)]):
        gone[r, a:b] = True
    W = torch.where(gone, -2.0 ** 60, z * 2.0 ** -100).t().contiguous().to(DT[dtype])
    H = torch.zeros(T, 8, dtype=DT[dtype])
    H[torch.arange(T), torch.arange(T) % 8] = 2.0 ** 100
    z = torch.where(gone, -math.inf, z.double())[torch.arange(T) % 8]
    tok = torch.randint(0, V, (T,), generator=gen(2))
    lp, ent, lse = (t.cpu() for t in ckl.head_logprobs_forward(H.cuda(), W.cuda(), tok.cuda()))
    some = torch.arange(T) % 8 != 7
    r = rows_reference(z[some], tok[some])
    there = r["logprob"] > -math.inf
    assert (lp[some][~there] == -math.inf).all()
    assert within(lp[some][there], r["logprob"][there], (r["tol_lp"] + 4 * EPS * r["lse"].abs())[there])
    assert within(ent[some], r["entropy"], r["tol_ent"])
    assert (lse[~some] == -math.inf).all() and (lp[~some] == -math.inf).all() and (ent[~some] == 0).all()
