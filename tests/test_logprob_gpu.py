"""Log probabilities of given tokens with entropy and alternatives, from logits, on the GPU against plain 64-bit
computations.

Tolerances count roundings: EPS is one fp32 rounding relative to the value, a sum of n terms in any order is within
n EPS of the sum of magnitudes, and a result in type t is rounded once more, by at most HALF[t] of its value.  A
term exp(x - m) carries at most 2^-22 (its argument's rounding times the argument, which the exponential outweighs,
and the exponential's)."""
import math

import numpy as np
import pytest
import torch

import chunked_kl_loss_amd as ckl

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=gen(seed), dtype=torch.float32) * std).to(dtype)


def same_bits(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.contiguous().reshape(-1).view(torch.uint8),
                                                                     b.contiguous().reshape(-1).view(torch.uint8))


def rows_reference(z, tokens, mask=None):
    """From logits [T, V] in 64 bits (finite or -inf, a finite one in every row): lse, log probability of the tokens,
    entropy, and the tolerances of the three for a sum of V terms by 256 threads or more."""
    T, V = z.shape
    top = z.max(1).values
    u = torch.exp(z - top[:, None])
    s = u.sum(1)
    gap = (torch.where(u > 0, top[:, None] - z, 0.0) * u).sum(1) / s  # the mean distance from the maximum
    lse = top + torch.log(s)
    inside = (tokens >= 0) & (tokens < V)
    zt = z.gather(1, torch.where(inside, tokens, 0).long()[:, None])[:, 0]
    logprob = torch.where(inside, zt - lse, 0.0)
    entropy = torch.log(s) + gap
    tau = (V / 256 + 40) * EPS + 2.0 ** -22
    tol_lse = tau + 2 * EPS * lse.abs()
    tol_lp = torch.where(inside & torch.isfinite(zt), tol_lse + 2 * EPS * logprob.abs().clamp(max=1e30), 0.0)
    # ln s and ln 2 e / s: sums of V terms about a reference within 4 of the maximum, and four roundings of each
    tol_ent = tau * (1 + 2 * (gap + 4)) + 4 * EPS * (torch.log(s).abs() + gap + 8)
    if mask is not None:
        keep = mask.bool()
        for t in (lse, logprob, entropy, tol_lse, tol_lp, tol_ent):
            t[~keep] = 0.0
    return dict(lse=lse, logprob=logprob, entropy=entropy, tol_lse=tol_lse, tol_lp=tol_lp, tol_ent=tol_ent)


def within(got, want, tol):
    got, want = got.double().cpu(), want.cpu()
    fin = torch.isfinite(want)
    return bool((got[~fin] == want[~fin]).all() and ((got - want).abs()[fin] <= tol.cpu()[fin]).all())


def top_reference(z, top):
    return torch.from_numpy(np.stack([np.lexsort((np.arange(z.shape[1]), -r))[:top] for r in z.numpy()]).astype(np.int32))


def dz_reference(z, tokens, r, a, b):
    """The logits' gradient in 64 bits and its tolerance before the rounding to its type."""
    lq = z - r["lse"][:, None]
    q = torch.exp(lq)
    lqf = torch.where(q > 0, lq, 0.0)
    inside = (tokens >= 0) & (tokens < z.shape[1])
    a = torch.where(inside, a.double(), 0.0)[:, None]
    b, ent = b.double()[:, None], r["entropy"][:, None]
    dz = -q * (a + b * (lqf + ent))
    rows = inside.nonzero()[:, 0]
    dz[rows, tokens[rows].long()] += a[rows, 0]
    # q: the argument's rounding (twice |log q| + |lse|) and the exponential's; the bracket: six roundings
    rel = r["tol_lse"][:, None] + (2 * lqf.abs() + r["lse"].abs()[:, None] + 4) * 2.0 ** -23
    mag = a.abs() + b.abs() * (lqf.abs() + ent)
    tol = q * (mag * (rel + 6 * EPS) + b.abs() * (r["tol_ent"] + r["tol_lse"])[:, None] + 6 * EPS * mag) + a.abs() * EPS * 2
    return dz, tol + 1e-37


def check(z, tokens, top=0, mask=None, train=True, a=None, b=None):
    T, V = z.shape
    dtype = z.dtype
    Z = z.cuda().requires_grad_(train)
    m = None if mask is None else mask.cuda()
    logprob, entropy, idx, val = ckl.token_logprobs(Z, tokens.cuda(), top=top, mask=m)
    z64 = z.double()
    r = rows_reference(z64, tokens, mask)
    assert logprob.dtype == entropy.dtype == val.dtype == torch.float32 and idx.dtype == torch.int32
    assert within(logprob.detach(), r["logprob"], r["tol_lp"])
    assert within(entropy.detach(), r["entropy"], r["tol_ent"])
    assert (entropy >= 0).all() and idx.shape == val.shape == (T, top)
    if top:
        want = top_reference(z64, top)
        lv = z64.gather(1, want.long()) - r["lse"][:, None]
        if mask is not None:
            want[~mask.bool()], lv[~mask.bool()] = torch.arange(top, dtype=torch.int32), 0.0
        assert torch.equal(idx.cpu(), want)
        assert within(val, lv, r["tol_lse"][:, None] + 2 * EPS * lv.abs().clamp(max=1e30))
        with torch.no_grad():  # with and without alternatives: sums in another order
            lp0, ent0, _, _ = ckl.token_logprobs(Z, tokens.cuda(), mask=m)
        assert within(lp0, r["logprob"], r["tol_lp"]) and within(ent0, r["entropy"], r["tol_ent"])
    if train:
        a = normal((T,), torch.float32, 3) if a is None else a
        b = normal((T,), torch.float32, 4, 0.3) if b is None else b
        (dz,) = torch.autograd.grad((logprob, entropy), (Z,), (a.cuda(), b.cuda()))
        want, tol = dz_reference(z64, tokens, r, a, b)
        if mask is not None:
            want[~mask.bool()], tol[~mask.bool()] = 0.0, 0.0
        assert dz.dtype == dtype and dz.shape == (T, V)
        assert within(dz, want, tol + HALF[dtype] * want.abs())
    return logprob, entropy


def some_tokens(T, V, seed, kind=torch.int64):
    return torch.randint(0, V, (T,), generator=gen(seed)).to(kind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,top", [(1, 1, 1), (1, 1, 0), (2, 2, 1), (1, 7, 7), (3, 9, 0), (3, 33, 5), (5, 2041, 0),
                                     (5, 2048, 1), (5, 2049, 20), (2, 8185, 0), (2, 8193, 3), (7, 4099, 1),
                                     (2, 50021, 1000), (1, 201088, 20), (3, 201088, 0), (1, 120001, 4096),
                                     (1100, 301, 17), (2100, 303, 0), (1030, 9000, 1025), (600, 5003, 0),
                                     (3, 64, 64), (9, 5003, 64), (9, 5003, 65), (9, 2047, 64), (9, 16385, 7), (2, 201088, 64), (2, 201088, 200)])
def test_sizes(T, V, top, dtype):
    z = normal((T, V), DT[dtype], 7 * T + V, 3.0)
    tok = some_tokens(T, V, V, torch.int32 if T % 2 else torch.int64)
    z[torch.arange(T), tok.long()] += 6.0
    check(z, tok, top, train=T * V <= 700000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 9, 15, 17])
def test_rows_shorter_than_two_vectors(V, dtype):
    for T in (1, 2, 5):
        check(normal((T, V), DT[dtype], V + T, 3.0), some_tokens(T, V, T), min(V, 3))


@pytest.mark.parametrize("top", [0, 9])
@pytest.mark.parametrize("T", [2, 1300])
def test_masks_and_tokens_outside(T, top):
    V = 1003
    mask = torch.rand(T, generator=gen(1)) < 0.6
    mask[0], mask[1] = True, False
    z = normal((T, V), torch.bfloat16, 3, 2.0)
    tok = some_tokens(T, V, 5)
    tok[::3] = torch.tensor([-1, -100, V, 2 ** 31, 2 ** 40, -2 ** 63, 2 ** 63 - 1]).repeat(T)[:len(tok[::3])]
    check(z, tok, top, mask)
    check(z, tok, top, torch.zeros(T, dtype=torch.uint8))
    check(z, tok.clamp(-2 ** 31, 2 ** 31 - 1).int(), top, mask)
    bad = z.clone()
    bad[~mask] = math.nan  # rows that are masked are not read
    Z = bad.cuda().requires_grad_(True)
    lp, ent, _, _ = ckl.token_logprobs(Z, tok.cuda(), top, mask.cuda())
    (dz,) = torch.autograd.grad((lp, ent), (Z,), (torch.ones_like(lp), torch.ones_like(ent)))
    assert torch.isfinite(lp).all() and torch.isfinite(dz).all() and not dz[~mask.cuda()].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [0, 40])
def test_forbidden_tokens_and_masks_of_the_lowest_value(top, dtype):
    V = 9001
    low = torch.finfo(DT[dtype]).min
    for fill in (-math.inf, low, -1e9, -7e7, -1e4):
        z = normal((6, V), torch.float32, 8, 2.0).to(DT[dtype])
        z[0, 1:] = fill                      # one column left
        z[1, ::2] = fill
        z[2, :V - 60] = fill                 # the last ones left
        z[3, 5:] = fill
        z[4, 100:8300] = fill
        tok = torch.tensor([0, 1, V - 1, 4000, 7, 3])
        # sums near -inf or the lowest value: their gap is infinite only where their weight is zero
        check(z, tok, top)


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("T", [4, 2100])
def test_rows_without_a_distribution(T, top):
    V = 600
    z = normal((T, V), torch.float32, 1)
    z[0] = -math.inf
    z[1, 3] = math.nan
    z[2, 5] = math.inf
    tok = torch.full((T,), 7)
    Z = z.cuda().requires_grad_(True)
    lp, ent, idx, val = ckl.token_logprobs(Z, tok.cuda(), top)
    assert float(lp[0].detach()) == -math.inf and float(ent[0].detach()) == 0
    assert torch.isnan(lp[1]) and torch.isnan(ent[1])
    assert float(lp[2].detach()) == -math.inf and torch.isnan(ent[2])
    assert torch.isfinite(lp[3:]).all() and torch.isfinite(ent[3:]).all()
    (dz,) = torch.autograd.grad((lp, ent), (Z,), (torch.ones_like(lp), torch.ones_like(ent)))
    assert not dz[0].any() and torch.isnan(dz[1]).all() and torch.isfinite(dz[3:]).all()
    # rows whose results nobody used have no gradient, whatever they hold
    lp, ent, _, _ = ckl.token_logprobs(Z, tok.cuda(), top)
    (dz,) = torch.autograd.grad(lp[3:].sum(), (Z,))
    assert torch.isfinite(dz).all() and not dz[:3].any()


@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("m", [-1e31, -6e29, -1e10, -3e8, 2e8, 7e7, 1e12, 6e29])
def test_logits_far_from_zero(m, top):
    V = 9001
    z = normal((4, V), torch.float32, 2, 2.0)
    z[0] = m                 # a whole row: the entropy is ln V
    z[1, :8] = m
    z[2, :2048:3] = m
    z[2, 8500:8700] = m
    z[3, ::2] = -abs(m)
    tok = torch.tensor([5, 4, 9, 10])
    # where all that counts is equal, differences vanish; lse and log probability round at m's size
    check(z, tok, top, train=False)


@pytest.mark.parametrize("rising", [False, True])
def test_order_of_the_columns(rising):
    # a reference that moves all along the row, and one that never does
    V = 30001
    z = torch.linspace(0, 90, V)[None].repeat(3, 1)
    z = z if rising else z.flip(1)
    check(z.contiguous(), torch.tensor([0, V // 2, V - 1]), 7)


@pytest.mark.parametrize("top", [1, 12, 13, 64, 70])
@pytest.mark.parametrize("T", [2, 1100])
@pytest.mark.parametrize("kind", ["equal", "few", "rising", "falling", "zeros", "comb"])
def test_ties_and_orders(kind, T, top):
    V = 5001
    if kind == "equal":
        z = torch.full((T, V), 1.25)
    elif kind == "few":
        z = torch.randint(0, 4, (T, V), generator=gen(5)).float()
    elif kind == "zeros":  # -0 and +0 are one value
        z = torch.where(torch.rand(T, V, generator=gen(6)) < 0.5, -0.0, 0.0)
        z[:, 4000] = 1.0
    elif kind == "comb":  # a few lanes hold all that is wanted
        z = torch.zeros(T, V)
        z[:, ::512] = 3.0 + torch.arange(len(range(0, V, 512))) / 8
    else:
        z = torch.arange(V, dtype=torch.float32).expand(T, V) / 64
        z = z if kind == "rising" else z.flip(1)
    check(z.contiguous(), some_tokens(T, V, 1), top, train=False)


def test_sure_and_diffuse_rows():
    # entropies from 1e-9 to ln V: absolute tolerances hold at both ends
    V = 4001
    z = torch.zeros(6, V)
    for i, t in enumerate((0.0, 1.0, 5.0, 12.0, 20.0, 32.0)):
        z[i, 17] = t
    check(z, torch.full((6,), 17), 2)


@pytest.mark.parametrize("only", ["logprob", "entropy"])
def test_one_output_only(only):
    T, V = 40, 700
    z, tok = normal((T, V), torch.float32, 1, 2.0), some_tokens(T, V, 2)
    Z = z.cuda().requires_grad_(True)
    lp, ent, _, _ = ckl.token_logprobs(Z, tok.cuda())
    g = normal((T,), torch.float32, 3)
    (dz,) = torch.autograd.grad(lp if only == "logprob" else ent, (Z,), g.cuda())
    zero = torch.zeros(T)
    r = rows_reference(z.double(), tok)
    want, tol = dz_reference(z.double(), tok, r, g if only == "logprob" else zero, zero if only == "logprob" else g)
    assert within(dz, want, tol + EPS * want.abs())


def test_gradients_against_differences():
    # the tolerance: values carry the tolerances of the rows, and the third derivatives step^2 / 6 of at most 30 |u|^3
    T, V, step = 4, 50, 1e-2
    z, tok = normal((T, V), torch.float32, 1, 1.5), some_tokens(T, V, 2)
    a, b = normal((T,), torch.float64, 3), normal((T,), torch.float64, 4)

    def value(z):
        lp, ent, _, _ = ckl.token_logprobs(z, tok.cuda())
        return (lp.double() * a.cuda() + ent.double() * b.cuda()).sum()
    Z = z.cuda().requires_grad_(True)
    (dz,) = torch.autograd.grad(value(Z), (Z,))
    r = rows_reference(z.double(), tok)
    noise = float((a.abs() * r["tol_lp"] + b.abs() * r["tol_ent"]).sum())
    for i in range(6):
        u = normal((T, V), torch.float32, 20 + i)
        u = u / u.abs().max()
        diff = float(value((z + step * u).cuda()) - value((z - step * u).cuda())) / (2 * step)
        got = float((dz.double().cpu() * u.double()).sum())
        assert abs(diff - got) < noise / step + step ** 2 / 6 * 30 * float(a.abs().sum() + 4 * b.abs().sum())


def test_layouts():
    z = normal((3, 7, 40), torch.bfloat16, 1, 2.0).cuda()
    tok = some_tokens(21, 40, 2).view(3, 7).cuda()
    mask = torch.rand(3, 7, generator=gen(1)).cuda() < 0.5
    lp, ent, idx, val = ckl.token_logprobs(z, tok, 4, mask)
    flat = ckl.token_logprobs(z.view(21, 40), tok.view(21), 4, mask.view(21))
    assert idx.shape == (3, 7, 4) and all(same_bits(a.reshape(b.shape), b) for a, b in zip((lp, ent, idx, val), flat))
    t = z.transpose(0, 1)  # strided
    got = ckl.token_logprobs(t, tok.t(), 4, mask.t())
    assert all(same_bits(a, b.transpose(0, 1).contiguous()) for a, b in zip(got, (lp, ent, idx, val)))
    one = ckl.token_logprobs(z[0, 0], tok[0, 0], 2)
    assert one[0].shape == () and one[2].shape == (2,)
    odd = normal((30, 41), torch.float32, 5).cuda()
    tk = some_tokens(30, 41, 3).cuda()
    got, want = ckl.token_logprobs(odd[1:], tk[1:], 3), ckl.token_logprobs(odd[1:].clone(), tk[1:], 3)
    assert all(same_bits(a, b) for a, b in zip(got, want))  # begins off a 16-byte boundary
    e = z[:0].requires_grad_(True)
    lp, ent, idx, val = ckl.token_logprobs(e, tok[:0], 2)
    (d,) = torch.autograd.grad((lp, ent), (e,), (torch.zeros_like(lp), torch.zeros_like(ent)))
    assert lp.shape == (0, 7) and idx.shape == (0, 7, 2) and d.shape == e.shape
    # the gradient of one row of logits for many tokens
    r = normal((1, 40), torch.float32, 6).cuda().requires_grad_(True)
    lp, _, _, _ = ckl.token_logprobs(r.expand(21, 40), tok.view(21))
    (d,) = torch.autograd.grad(lp.sum(), (r,))
    assert abs(float(d.sum())) < 1e-4


def test_agrees_with_the_teacher_of_the_same_logits():
    z = normal((50, 3001), torch.bfloat16, 4, 3.0).cuda()
    idx, val, lse = ckl.teacher_topk(z, 30, teacher_form=1)
    tok = idx[:, 3].contiguous()
    lp, ent, tidx, tval = ckl.token_logprobs(z, tok, 30)
    assert torch.equal(idx, tidx) and same_bits(lp, tval[:, 3].contiguous())
    assert torch.allclose(val, tval, atol=(3001 / 256 + 40) * EPS * 4, rtol=4 * EPS)


def test_offsets_past_32_bits():
    # the last rows lie more than 2^31 elements behind the first
    T, V = 11000, 200001
    z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    last = normal((2, V), torch.bfloat16, 1, 3.0)
    z[-2:] = last.cuda()
    tok = torch.zeros(T, dtype=torch.int64, device="cuda")
    tok[-2:] = torch.tensor([V - 1, 5])
    r = rows_reference(last.double(), tok[-2:].cpu())
    for top in (0, 3):
        lp, ent, lse, idx, val = ckl.token_logprobs_forward(z, tok, top)
        assert within(lp[-2:], r["logprob"], r["tol_lp"]) and within(ent[-2:], r["entropy"], r["tol_ent"])
        assert (lp[:-2] - lp[0]).abs().max() == 0 and abs(float(lp[0]) + math.log(V)) < 1e-4
        if top:
            assert torch.equal(idx[-2:].cpu(), top_reference(last.double(), top))
    a, b = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    a[-2:], b[-2:] = 1.5, -0.5
    dz = ckl.token_logprobs_backward(a, b, z, tok, lse, ent)
    del z
    want, tol = dz_reference(last.double(), tok[-2:].cpu(), r, a[-2:].cpu(), b[-2:].cpu())
    assert within(dz[-2:], want, tol + HALF[torch.bfloat16] * want.abs())
    assert not dz[:-2].any()


# ------------------------------------------------- captures, streams, tangents --
def steps(seed, T=300, V=5003, top=6):
    z = normal((T, V), torch.bfloat16, seed, 2.0).cuda()
    return z, some_tokens(T, V, seed + 1).cuda(), (torch.rand(T, generator=gen(seed + 2)) < 0.7).cuda()


def step(z, tok, mask, top=6):
    Z = z.detach().requires_grad_(True)
    lp, ent, idx, val = ckl.token_logprobs(Z, tok, top, mask)
    lp0, ent0, _, _ = ckl.token_logprobs(Z, tok, 0, mask)
    (dz,) = torch.autograd.grad((lp, ent, lp0), (Z,), (lp.detach(), ent.detach(), ent0.detach()))
    return [lp.detach(), ent.detach(), idx, val, lp0.detach(), dz]


@pytest.mark.parametrize("T", [2, 300])
def test_captured_step_replays_with_new_inputs(T):
    ins = steps(1, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*ins)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*ins)
    for seed in (1, 50, 90, 50):
        new = steps(seed, T)
        for a, b in zip(ins, new):
            a.copy_(b)
        want = [t.clone() for t in step(*new)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(outs, want))


def test_two_streams_at_once():
    ins = [steps(s, 3) for s in (1, 30)] + [steps(60, 900)]
    want = [[t.clone() for t in step(*i)] for i in ins]
    torch.cuda.synchronize()
    got, streams = [], [torch.cuda.Stream() for _ in ins]
    for s, i in zip(streams, ins):
        with torch.cuda.stream(s):
            got.append(step(*i))
    torch.cuda.synchronize()
    assert all(same_bits(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_forward_mode_tangents_are_refused():
    fw = torch.autograd.forward_ad
    z, tok = normal((4, 16), torch.float32, 2).cuda(), torch.zeros(4, dtype=torch.int64, device="cuda")
    w = normal((9, 16), torch.float32, 3).cuda()
    with fw.dual_level():
        d = fw.make_dual(z, torch.ones_like(z))
        for call in (lambda: ckl.token_logprobs(d, tok), lambda: ckl.head_logprobs(d, w, tok)):
            with torch.no_grad(), pytest.raises(NotImplementedError, match="jvp"):
                call()


def test_neighbours_stay_untouched():
    import ctypes

    from chunked_kl_loss_amd import _binding as B
    lib = B.load_library()
    for T, V, top, dt in ((3, 20001, 5, torch.float32), (3, 20001, 70, torch.float32), (9, 333, 5, torch.bfloat16), (5, 1001, 0, torch.float32)):
        z, tok = normal((T, V), dt, 1).cuda(), some_tokens(T, V, 2).cuda()
        code = int(dt == torch.bfloat16)
        rows = [torch.full((T + 64,), -7.0, device="cuda") for _ in range(3)]
        idx = torch.full((T * top + 64,), -7, dtype=torch.int32, device="cuda")
        val = torch.full((T * top + 64,), -7.0, device="cuda")
        dz = torch.full((T * V + 64,), -7.0, dtype=dt, device="cuda")
        need = ctypes.c_size_t(0)
        B.check(lib.ckl_logprob_workspace_size(T, V, top, ctypes.byref(need)))
        ws = torch.full((need.value + 64,), 0xAB, dtype=torch.uint8, device="cuda")
        at = [r.data_ptr() + 64 for r in rows]
        B.check(lib.ckl_token_logprobs(z.data_ptr(), code, T, V, tok.data_ptr(), 8, top, None, *at, idx.data_ptr() + 64,
                                       val.data_ptr() + 64, ws.data_ptr(), need.value, None))
        B.check(lib.ckl_token_logprobs_backward(z.data_ptr(), code, T, V, tok.data_ptr(), 8, None, at[2], at[1], at[0],
                                                at[1], dz.data_ptr() + 16 * dz.element_size(), None))
        torch.cuda.synchronize()
        for b, n in [(r, T) for r in rows] + [(idx, T * top), (val, T * top), (dz, T * V)]:
            assert (b[:16] == -7).all() and (b[16 + n:] == -7).all() and not (b[16:16 + n] == -7).any()
        assert (ws[need.value:] == 0xAB).all()
