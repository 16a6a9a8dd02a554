"""The operators around the loss on the GPU against plain 64-bit computations:
the top-K teacher, the embedding and its gradient, 8-bit activations and the
norm that saves them, and one step that uses all of them.

Tolerances count roundings.  EPS is one fp32 rounding relative to the value; a
sum of n terms in any order is within n EPS of the sum of magnitudes; a result
in type t is rounded once more, by at most HALF[t] of its value."""
import math

import numpy as np
import pytest
import torch

import chunked_kl_loss_amd as ckl
from chunked_kl_loss_amd import _binding as B
from chunked_kl_loss_amd import ops

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


# ----------------------------------------------------------- teacher top-K --
def topk_reference(z, K, form, mask):
    """z: float tensor on the CPU.  Order: NaN first, then descending, equal values by index."""
    z64 = z.double().numpy()
    T, V = z64.shape
    key = np.where(np.isnan(z64), np.inf, z64)
    idx = np.empty((T, K), np.int32)
    for t in range(T):
        idx[t] = np.lexsort((np.arange(V), -key[t], ~np.isnan(z64[t])))[:K]
    val = np.take_along_axis(z64, idx.astype(np.int64), 1)
    lse = torch.logsumexp(torch.from_numpy(z64), 1).numpy()
    if form == 1:
        with np.errstate(invalid="ignore"):
            val = np.where(val == -np.inf, -np.inf, val - lse[:, None])
    if mask is not None:
        m = mask.numpy().astype(bool)
        idx[~m], val[~m], lse[~m] = np.arange(K), 0.0, 0.0
    return idx, val, lse


def check_topk(z, K, form=0, mask=None):
    idx, val, lse = ckl.teacher_topk(z.cuda(), K, None if mask is None else mask.cuda(), form)
    torch.cuda.synchronize()
    ridx, rval, rlse = topk_reference(z, K, form, mask)
    np.testing.assert_array_equal(idx.cpu().numpy(), ridx)
    V = z.shape[-1]
    # log-sum-exp: the sum's terms carry at most 2^-22 each (argument and exponential), a thread adds at most
    # V / 256 + 8 of them, 32 merges follow; the logarithm and its sum with the maximum round once each
    tol = (V / 256 + 40) * EPS + 2.0 ** -22 + 2 * EPS * np.abs(np.nan_to_num(rlse, posinf=0, neginf=0))
    got = lse.double().cpu().numpy()
    fin = np.isfinite(rlse)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(rlse))
    np.testing.assert_array_equal(got[~fin & ~np.isnan(rlse)], rlse[~fin & ~np.isnan(rlse)])
    assert (np.abs(got - rlse)[fin] <= tol[fin]).all()
    gv = val.double().cpu().numpy()
    if form == 0:
        np.testing.assert_array_equal(gv, rval)
    else:
        fv = np.isfinite(rval)
        np.testing.assert_array_equal(np.isnan(gv), np.isnan(rval))
        np.testing.assert_array_equal(gv[~fv & ~np.isnan(rval)], rval[~fv & ~np.isnan(rval)])
        bound = np.broadcast_to(tol[:, None], gv.shape) + 2 * EPS * np.abs(np.where(fv, rval, 0))
        assert (np.abs(gv - rval)[fv] <= bound[fv]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (1, 7, 7), (3, 33, 5), (2, 2048, 2048), (5, 2049, 100), (7, 4099, 1),
                                   (2, 50021, 1000), (1, 201088, 100), (1, 120001, 4096), (3, 8200, 4096),
                                   (1100, 301, 17), (1030, 9000, 1025)])
def test_topk_sizes(T, V, K, dtype):
    check_topk(normal((T, V), DT[dtype], 7 * T + V, 3.0), K, form=(T + V) % 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 9])
def test_topk_rows_shorter_than_a_vector(V, dtype):
    for T in (1, 2, 5):
        check_topk(normal((T, V), DT[dtype], V + T, 3.0), V, form=T % 2)


@pytest.mark.parametrize("T", [2, 1300])
@pytest.mark.parametrize("form", [0, 1])
def test_topk_masks(T, form):
    mask = torch.rand(T, generator=gen(1)) < 0.6
    mask[0], mask[1] = True, False
    z = normal((T, 5003), torch.bfloat16, 3, 2.0)
    check_topk(z, 33, form, mask)
    check_topk(z, 33, form, torch.zeros(T, dtype=torch.uint8))


@pytest.mark.parametrize("T", [1, 1030])
@pytest.mark.parametrize("kind", ["equal", "few", "rising", "falling", "zeros"])
def test_topk_ties_and_orders(T, kind):
    V, K = 9001, 700
    if kind == "equal":
        z = torch.full((T, V), 1.25)
    elif kind == "few":
        z = torch.randint(0, 4, (T, V), generator=gen(5)).float()
    elif kind == "zeros":  # -0 and +0 are one value
        z = torch.where(torch.rand(T, V, generator=gen(6)) < 0.5, -0.0, 0.0)
        z[:, 4000] = 1.0
    else:
        z = torch.arange(V, dtype=torch.float32).expand(T, V) / 64
        z = z if kind == "rising" else z.flip(1)
    check_topk(z.contiguous(), K, form=0)


def test_topk_infinities_and_nan():
    V, K = 6007, 40
    z = normal((8, V), torch.float32, 9)
    z[0, :] = -math.inf
    z[1, 5:] = -math.inf                      # fewer finite logits than K
    z[2, 17] = math.inf
    z[3, 4000] = math.nan
    z[3, 3] = math.nan
    z[4, ::3] = -math.inf
    z[5, :] = -3.0e38
    z[6, :] = torch.finfo(torch.float32).min  # masks of the lowest value
    z[6, 77] = 2.0
    z[7, 10], z[7, 9] = math.inf, math.inf
    check_topk(z, K, form=0)
    check_topk(z[[0, 1, 3, 4, 5, 6]], K, form=1)
    big = torch.cat([z] * 200)                # whole rows to a workgroup
    check_topk(big[:1100], K, form=0)


@pytest.mark.parametrize("K", [40, 700, 1100])
@pytest.mark.parametrize("T", [2, 1030])
def test_topk_rows_of_mostly_special_values(T, K):
    # thousands of NaN or infinite logits: the range of keys reaches the last one
    z = normal((T, 9001), torch.float32, 3)
    z[:, ::2] = math.nan
    check_topk(z, K)
    z[:, ::2] = math.inf
    check_topk(z, K)
    z[:, 1::4] = math.nan
    check_topk(z, K)
    z[:, ::2] = -math.inf
    check_topk(z.bfloat16(), K)
    z = normal((T, 6000), torch.float32, 4)   # one tile, fewer finite logits than K
    z[:, 30:] = -math.inf
    check_topk(z, K)


def test_topk_shapes_and_repeatability():
    z = normal((2, 3, 1001), torch.bfloat16, 4).cuda()
    mask = torch.tensor([[1, 0, 1], [1, 1, 0]], dtype=torch.uint8).cuda()
    a = ckl.teacher_topk(z, 8, mask, 1)
    assert [tuple(t.shape) for t in a] == [(2, 3, 8), (2, 3, 8), (2, 3)]
    b = ckl.teacher_topk(z.view(6, -1), 8, mask.view(-1), 1)
    for x, y in zip(a, b):
        assert same_bits(x.reshape(y.shape), y)
    e = ckl.teacher_topk(z[:0], 8)
    assert tuple(e[0].shape) == (0, 3, 8) and tuple(e[2].shape) == (0, 3)
    with pytest.raises(ValueError):
        ckl.teacher_topk(z.transpose(1, 2), 2)
    with pytest.raises(TypeError):
        ckl.teacher_topk(z.half(), 2)
    with pytest.raises(B.CklError):
        ckl.teacher_topk(z, 1002)


# --------------------------------------------------------------- embedding --
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,d", [(1, 1, 8), (3, 5, 16), (64, 100, 520), (1000, 3001, 2880), (5, 7, 65536),
                                   (70001, 50, 24)])
def test_embedding_forward(T, V, d, dtype):
    W = normal((V, d), DT[dtype], 1)
    tok = torch.randint(-2, V + 2, (T,), generator=gen(2))
    scale = 3.25
    out = ckl.embedding_forward(W.cuda(), tok.cuda(), scale).double().cpu()
    inside = (tok >= 0) & (tok < V)
    ref = torch.where(inside[:, None], W.double()[tok.clamp(0, V - 1)] * scale, 0.0)
    assert (out - ref).abs().le(ref.abs() * (HALF[DT[dtype]] * (1 + 2 * EPS) + 2 * EPS)).all()
    again = ckl.embedding_forward(W.cuda(), tok.int().cuda(), scale).double().cpu()
    assert torch.equal(out, again)


def test_embedding_shapes_and_shards():
    W = normal((1000, 64), torch.float32, 1).cuda()
    tok = torch.randint(0, 1000, (4, 9), generator=gen(2)).cuda()
    whole = ckl.embedding_forward(W, tok, 2.0)
    assert whole.shape == (4, 9, 64) and torch.equal(whole, W[tok] * 2)
    parts = [ckl.embedding_forward(W[a:b].contiguous(), tok, 2.0, v_offset=a) for a, b in ((0, 333), (333, 1000))]
    assert torch.equal(parts[0] + parts[1], whole)
    assert ckl.embedding_forward(W, tok[:0]).shape == (0, 9, 64)
    for bad in (tok.short(), tok.float()):
        with pytest.raises(TypeError):
            ckl.embedding_forward(W, bad)
    with pytest.raises(ValueError):
        ckl.embedding_forward(W.t(), tok)
    with pytest.raises(B.CklError):
        ckl.embedding_forward(W[:, :12].contiguous(), tok)


def tokens_of(kind, T, V, seed):
    if kind == "uniform":
        return torch.randint(0, V, (T,), generator=gen(seed))
    if kind == "zipf":
        u = torch.rand(T, generator=gen(seed), dtype=torch.float64)
        return (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp(0, V - 1)
    if kind == "one":
        return torch.full((T,), V - 1)
    if kind == "none":
        return torch.full((T,), -100)
    t = tokens_of("zipf", T, V, seed)  # half of the positions outside the table, on both sides
    r = torch.rand(T, generator=gen(seed + 1))
    return torch.where(r < 0.25, -1 - t, torch.where(r < 0.5, V + t, t))


def check_embedding_grad(T, V, d, kind, dtype, grad, add, scale=1.5, off=0, tok_dtype=torch.int64):
    dY = normal((T, d), DT[dtype], T + d)
    tok = tokens_of(kind, T, V, T + V)
    old = normal((V, d), DT[grad], 11) if add else None
    dev_old = None if old is None else old.cuda()
    out = ckl.embedding_backward(dY.cuda(), (tok + off).to(tok_dtype).cuda(), V, scale, off, DT[grad], dev_old)
    if add:
        assert out is dev_old
    got = out.double().cpu()
    inside = (tok >= 0) & (tok < V)
    at = tok[inside]
    ref = torch.zeros(V, d, dtype=torch.float64).index_add_(0, at, dY.double()[inside]) * scale
    mag = torch.zeros(V, d, dtype=torch.float64).index_add_(0, at, dY.double()[inside].abs()) * scale
    n = torch.zeros(V, dtype=torch.float64).index_add_(0, at, torch.ones(len(at), dtype=torch.float64))
    if add:
        ref, mag = ref + old.double(), mag + old.double().abs()
        untouched = n == 0
        assert same_bits(out.cpu()[untouched], old[untouched])
    # a token's n terms, the scale and the old value: n + 2 roundings of sums, then the result's own
    tol = (n[:, None] + 2) * EPS * mag + HALF[DT[grad]] * ref.abs() * (1 + 2.0 ** -6)
    assert (got - ref).abs().le(tol).all(), ((got - ref).abs() - tol).max()
    return out


@pytest.mark.parametrize("kind", ["uniform", "zipf", "one", "none", "padded"])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 64, 65, 1000, 4097, 8192, 8193, 20000])
def test_embedding_grad_lengths(T, kind):
    check_embedding_grad(T, 1000, 24, kind, "bf16", "f32", add=T % 2 == 0)
    check_embedding_grad(T, 513, 64, kind, "f32", "bf16", add=T % 2 == 1, tok_dtype=torch.int32)


@pytest.mark.parametrize("kind", ["zipf", "one", "padded"])
@pytest.mark.parametrize("T", [127, 255, 256, 257, 272, 513])
def test_embedding_grad_where_the_way_changes(T, kind):
    # up to 256 positions in one launch, ranked beyond; every type, several workgroups to a row
    for dtype, grad in (("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")):
        check_embedding_grad(T, 300, 2056, kind, dtype, grad, add=dtype == grad, tok_dtype=torch.int32)
        check_embedding_grad(T, 300, 8, kind, dtype, grad, add=dtype != grad)


def test_embedding_grad_of_one_token_many_times():
    # one run through hundreds of chunks, and one that ends with the last chunk
    check_embedding_grad(70000, 5, 520, "one", "bf16", "f32", add=True)
    check_embedding_grad(65536, 1, 16, "uniform", "f32", "bf16", add=False)


@pytest.mark.parametrize("V", [1, 2, 511, 512, 32000, 262143, 262144, 300000])
@pytest.mark.parametrize("T", [300, 12345, 70000])
def test_embedding_grad_vocabularies(T, V):
    check_embedding_grad(T, V, 8, "zipf", "f32", "f32", add=False)
    check_embedding_grad(T, V, 8, "padded", "bf16", "f32", add=True)


@pytest.mark.parametrize("d", [8, 16, 520, 2880, 16384])
@pytest.mark.parametrize("dtype,grad", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_embedding_grad_widths_and_types(d, dtype, grad):
    for T, kind in ((37, "zipf"), (9000, "padded")):
        if T * d < 60_000_000:
            for add in (False, True):
                check_embedding_grad(T, 400, d, kind, dtype, grad, add)


def test_embedding_grad_long_and_large():
    check_embedding_grad(300000, 5000, 16, "zipf", "bf16", "f32", add=True)
    # more than 2^31 elements of dW: rows past every 32-bit offset
    V, d = 1_100_000, 2048
    tok = torch.tensor([0, V - 1, V - 1, 1_048_577, V, 5])
    dY = normal((6, d), torch.bfloat16, 2)
    dW = torch.zeros((V, d), dtype=torch.bfloat16, device="cuda")
    ckl.embedding_backward(dY.cuda(), tok.cuda(), V, 2.0, add_to=dW)
    assert torch.equal(dW[0].cpu(), dY[0] * 2) and torch.equal(dW[1_048_577].cpu(), dY[3] * 2)
    assert torch.equal(dW[V - 1].cpu(), ((dY[1].float() + dY[2].float()) * 2).bfloat16())
    assert int((dW != 0).any(dim=1).sum()) == 4
    out = ckl.embedding_forward(dW, tok.cuda())
    assert torch.equal(out[1], dW[V - 1]) and int(out[4].count_nonzero()) == 0


def test_embedding_grad_empty_shards_and_repeats():
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    dY0 = torch.zeros(0, 16, device="cuda")
    assert not ckl.embedding_backward(dY0, none, 30).any()
    old = normal((30, 16), torch.float32, 3).cuda()
    assert same_bits(ckl.embedding_backward(dY0, none, 30, add_to=old.clone()), old)
    # shards hold the rows of the whole gradient, bit for bit
    dY, tok = normal((9000, 40), torch.bfloat16, 5).cuda(), tokens_of("zipf", 9000, 1000, 6).cuda()
    whole = ckl.embedding_backward(dY, tok, 1000, 0.5)
    parts = [ckl.embedding_backward(dY, tok, b - a, 0.5, v_offset=a) for a, b in ((0, 17), (17, 700), (700, 1000))]
    torch.testing.assert_close(torch.cat(parts), whole, rtol=1e-5, atol=1e-4)
    for _ in range(3):
        assert same_bits(ckl.embedding_backward(dY, tok, 1000, 0.5), whole)
    check_embedding_grad(9000, 700, 40, "padded", "bf16", "f32", add=True, off=17)
    with pytest.raises(ValueError):
        ckl.embedding_backward(dY, tok, 1000, add_to=torch.zeros(999, 40, device="cuda"))
    with pytest.raises(TypeError):
        ckl.embedding_backward(dY, tok, 1000, dw_dtype=torch.bfloat16, add_to=torch.zeros(1000, 40, device="cuda"))
    with pytest.raises(B.CklError):
        ckl.embedding_backward(dY, tok, 0)


def test_embedding_autograd_against_differences():
    # linear in W, so a difference quotient is the derivative up to rounding: with integers it is exact
    W = torch.randint(-8, 9, (50, 16), generator=gen(1)).float().cuda().requires_grad_(True)
    tok = torch.randint(-1, 51, (3, 21), generator=gen(2)).cuda()
    dY = torch.randint(-4, 5, (3, 21, 16), generator=gen(3)).float().cuda()
    step = torch.randint(-2, 3, (50, 16), generator=gen(4)).float().cuda()
    f = lambda w: float((ckl.embedding(w, tok, scale=2.0) * dY).double().sum())  # noqa: E731
    (ckl.embedding(W, tok, scale=2.0) * dY).sum().backward()
    with torch.no_grad():
        assert f(W + step) - f(W - step) == 2 * float((W.grad * step).double().sum())
    Wb = W.detach().bfloat16().requires_grad_(True)
    ckl.embedding(Wb, tok.t(), scale=2.0).sum().backward()  # tokens of another order, bf16 gradient
    count = torch.bincount(tok[(tok >= 0) & (tok < 50)], minlength=50).float()
    assert Wb.grad.dtype == torch.bfloat16
    assert torch.equal(Wb.grad.float(), (2 * count)[:, None].expand(50, 16))


# ------------------------------------------------- 8-bit activations, norm --
def encode_reference(x):
    """The definition in 64 bits: codes, exponents and the values they stand for."""
    x = x.double().reshape(-1, x.shape[-1])
    T, d = x.shape
    nb = -(-d // 32)
    codes, exps, held = torch.zeros(T, d), torch.zeros(T, nb), torch.zeros(T, d, dtype=torch.float64)
    for b in range(nb):
        s = slice(32 * b, min(d, 32 * b + 32))
        block = x[:, s]
        top = block.abs().amax(1)
        bad = ~torch.isfinite(block).all(1)
        top = torch.where(bad, 1.0, top)
        _, e = torch.frexp(top)                       # top = m 2^e, m in [1/2, 1)
        e = torch.where(top == 0, -10000, e - 7)
        e = torch.where(top >= 127.5 * torch.exp2(e.double()), e + 1, e).clamp(-126, 121)
        step = torch.exp2(e.double())
        c = torch.round(torch.where(bad[:, None], 0.0, block) / step[:, None]).clamp(-127, 127)
        codes[:, s], exps[:, b] = c.float(), torch.where(bad, 255, e + 127).float()
        held[:, s] = torch.where(bad[:, None], math.nan, c * step[:, None])
    return codes.to(torch.int8), exps.to(torch.uint8), held


def check_codes(x):
    codes, exps = ckl.act_encode(x.cuda())
    rc, re, held = encode_reference(x)
    assert torch.equal(codes.cpu().reshape(rc.shape), rc) and torch.equal(exps.cpu().reshape(re.shape), re)
    for t in (torch.float32, torch.bfloat16):
        got = ckl.act_decode(codes, exps, dtype=t).double().cpu().reshape(held.shape)
        assert torch.equal(torch.nan_to_num(got, nan=1e300), torch.nan_to_num(held, nan=1e300))
    return codes, exps, held


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (1, 32), (3, 40), (257, 24), (1000, 520), (33, 2880), (2, 65536), (20001, 8)])
def test_codes_sizes(T, d, dtype):
    x = normal((T, d), DT[dtype], T + d) * torch.exp(normal((d,), torch.float32, 3)).to(DT[dtype])
    _, _, held = check_codes(x)
    top = torch.nn.functional.pad(x.double().abs(), (0, -d % 32)).view(T, -1, 32).amax(2)
    bound = top.repeat_interleave(32, 1)[:, :d] / 127.5
    assert (held - x.double()).abs().le(bound).all()


def test_codes_at_borders():
    rows = []
    for e in (-149, -140, -133, -127, -126, -120, -60, -6, 0, 5, 60, 120, 127):
        for top in (1.0, 1.9921874, 1.9921875, 1.9921876, 1.999, 1.5):
            r = torch.linspace(-1, 1, 32, dtype=torch.float64) * (top * 2.0 ** e)
            r[31], r[30] = top * 2.0 ** e, -top * 2.0 ** e
            rows.append(r)
    x = torch.stack(rows).float()
    x = torch.where(torch.isinf(x), torch.finfo(torch.float32).max, x)
    check_codes(x)
    check_codes(torch.nan_to_num(x.bfloat16(), posinf=1e38, neginf=-1e38))
    half = (torch.arange(-127, 128).float() + 0.5).clamp(-127, 127)[:224].view(7, 32)  # ties to even
    half[:, 0] = 127
    check_codes(half)
    check_codes(torch.zeros(2, 64))
    bad = normal((5, 104), torch.float32, 1)
    bad[0, 3], bad[1, 40], bad[2, 103], bad[3, 96] = math.nan, math.inf, -math.inf, math.nan
    check_codes(bad)
    check_codes(bad.bfloat16())
    assert ckl.act_encode(torch.zeros(2, 0, 40, device="cuda"))[1].shape == (2, 0, 2)


def norm_reference(x, w, dy, eps, held):
    x, w, dy = x.double(), w.double(), dy.double()
    r = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    n = held * r
    gw = dy * w
    c = (gw * n).mean(1, keepdim=True)
    dx = r * (gw - n * c)
    mag = r * (gw.abs() + n.abs() * (gw * n).abs().mean(1, keepdim=True))
    return x * r * w, r[:, 0], dx, mag, (dy * n).sum(0), (dy * n).abs().sum(0)


@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 24), (1025, 64), (257, 520), (2050, 2880), (5, 8192), (5, 8200),
                                 (3, 16392), (3, 32776), (2, 65536)])
def test_norm(T, d, dtype, wtype):
    t, eps = DT[dtype], 1e-5
    x = normal((T, d), t, T + d) * torch.exp(normal((d,), torch.float32, 3, 0.5)).to(t)
    w, dy = (1 + normal((d,), torch.float32, 4, 0.2)).to(DT[wtype]), normal((T, d), t, 5)
    y, codes, exps, rstd = ckl.norm_forward(x.cuda(), w.cuda(), eps)
    rc, re, held = encode_reference(x)
    assert torch.equal(codes.cpu(), rc) and torch.equal(exps.cpu(), re)
    ry, rr, rdx, mag, rdw, wmag = norm_reference(x, w, dy, eps, held)
    # the mean of squares: a thread adds at most 64 terms, 6 + 16 more across the workgroup; half of that relative
    # error in rstd, and its own roundings
    k = 48 * EPS
    assert (rstd.double().cpu() - rr).abs().le(k * rr).all()
    assert (y.double().cpu() - ry).abs().le(ry.abs() * (k + 3 * EPS + HALF[t] * (1 + 2 * k))).all()
    y2, *rest = ckl.norm_forward(x.cuda(), w.cuda(), eps, save=False)
    assert same_bits(y2, y) and rest == [None, None, None]
    again = ckl.act_decode(codes, exps, rstd, w.cuda(), dtype=t).double().cpu()
    ref = held * rr[:, None] * w.double()
    assert (again - ref).abs().le(ref.abs() * (k + 3 * EPS + HALF[t] * (1 + 2 * k))).all()
    dx, dw = ckl.norm_backward(dy.cuda(), codes, exps, rstd, w.cuda())
    assert dx.dtype == t and dw.dtype == DT[wtype]
    # rstd enters three times; the mean of dy w n has the same number of terms as the mean of squares
    assert (dx.double().cpu() - rdx).abs().le(mag * (3 * k + 96 * EPS) + rdx.abs() * HALF[t] * (1 + 2.0 ** -6)).all()
    assert (dw.double().cpu() - rdw).abs().le(wmag * (k + (T + 8) * EPS) + rdw.abs() * HALF[DT[wtype]] * (1 + 2.0 ** -6)).all()
    for _ in range(2):
        a, b = ckl.norm_backward(dy.cuda(), codes, exps, rstd, w.cuda())
        assert same_bits(a, dx) and same_bits(b, dw)


def test_norm_rows_of_zeros_nan_and_none():
    x = normal((4, 72), torch.float32, 1)
    x[1] = 0
    x[2, 5] = math.nan
    w = torch.ones(72)
    y, codes, exps, rstd = ckl.norm_forward(x.cuda(), w.cuda(), 1e-6)
    assert not y[1].any() and torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3]]).all()
    dx, _ = ckl.norm_backward(torch.ones(4, 72, device="cuda"), codes, exps, rstd, w.cuda())
    assert torch.isnan(dx[2]).all() and torch.isfinite(dx[[0, 1, 3]]).all()
    assert torch.equal(dx[1], torch.full((72,), 1000.0, device="cuda").mul(1 / (1e-6 ** 0.5 * 1000))) or \
        torch.allclose(dx[1], torch.full((72,), 1e3, device="cuda"), rtol=1e-6)
    e = torch.zeros(0, 72, device="cuda")
    y, codes, exps, rstd = ckl.norm_forward(e, w.cuda())
    dx, dw = ckl.norm_backward(e, codes, exps, rstd, w.cuda())
    assert y.shape == dx.shape == (0, 72) and not dw.any()


@pytest.mark.parametrize("lead,d", [((1,), 8), ((3,), 24), ((5, 7), 520), ((0,), 72), ((2, 0), 8), ((13,), 8200)])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f32", "bf16")])
def test_norm_autograd_is_the_direct_calls(lead, d, dtype, wtype):
    # what is saved lies in one tensor, at offsets that depend on the rows: the same bits all the same
    x, dy = normal((*lead, d), DT[dtype], 1).cuda(), normal((*lead, d), DT[dtype], 2).cuda()
    w = normal((d,), DT[wtype], 3).cuda()
    y, codes, exps, rstd = ckl.norm_forward(x, w, 1e-5)
    dx, dw = ckl.norm_backward(dy, codes, exps, rstd, w)
    X, Wt = x.clone().requires_grad_(), w.clone().requires_grad_()
    out = ckl.rms_norm_8bit(X, Wt, 1e-5)
    assert same_bits(out.detach(), y)
    for _ in range(2):  # the saved tensor outlives a backward pass that retains it
        a, b = torch.autograd.grad(out, (X, Wt), dy, retain_graph=True)
        assert same_bits(a, dx) and same_bits(b, dw)
    only, = torch.autograd.grad(ckl.rms_norm_8bit(X, w, 1e-5), (X,), dy)
    assert same_bits(only, dx)
    only, = torch.autograd.grad(ckl.rms_norm_8bit(x, Wt, 1e-5), (Wt,), dy)
    assert same_bits(only, dw)
    one = torch.ones((), dtype=DT[dtype], device="cuda").expand(*lead, d)  # a gradient with strides of zero
    a, b = torch.autograd.grad(out, (X, Wt), one)
    dx, dw = ckl.norm_backward(one.contiguous(), codes, exps, rstd, w)
    assert same_bits(a, dx) and same_bits(b, dw)


def test_norm_gradient_against_differences():
    # x on the codes' grid: the 8-bit form is exact, so the gradient is that of the norm itself
    T, d = 5, 72
    x = torch.randint(-127, 128, (T, d), generator=gen(1)).float()
    x[:, ::32] = 127
    w = 1 + normal((d,), torch.float32, 2, 0.3)
    dy = normal((T, d), torch.float32, 3)
    X = x.cuda().requires_grad_(True)
    Wt = w.cuda().requires_grad_(True)
    (ckl.rms_norm_8bit(X, Wt, eps=1e-3) * dy.cuda()).sum().backward()

    def f(x64, w64):
        r = 1.0 / torch.sqrt((x64 * x64).mean(1, keepdim=True) + 1e-3)
        return float((x64 * r * w64 * dy.double()).sum())
    ux, uw = normal((T, d), torch.float64, 4), normal((d,), torch.float64, 5)
    h = 1e-4
    num = (f(x.double() + h * ux, w.double() + h * uw) - f(x.double() - h * ux, w.double() - h * uw)) / (2 * h)
    ana = float((X.grad.double().cpu() * ux).sum() + (Wt.grad.double().cpu() * uw).sum())
    # terms of both sums are of order 1, sums of 72 in fp32; the quotient's own error is h^2 and 1e-16 / h
    size = float((X.grad.double().cpu() * ux).abs().sum() + (Wt.grad.double().cpu() * uw).abs().sum())
    assert abs(num - ana) <= 200 * EPS * size + 1e-7


# ------------------------------------------------------- use by the loss --
def loss_inputs(T=300, d=72, V=1500, K=20, dtype=torch.bfloat16, seed=0):
    H, W = normal((T, d), dtype, seed).cuda(), normal((V, d), dtype, seed + 1, d ** -0.5).cuda()
    idx, tl, _ = ckl.teacher_topk(normal((T, V), torch.bfloat16, seed + 2, 2.0).cuda(), K)
    mask = (torch.rand(T, generator=gen(seed + 3)) < 0.7).cuda()
    return H, W, idx, tl, mask


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("masked", [False, True])
def test_loss_with_saved_8bit_states(dtype, masked):
    H, W, idx, tl, mask = loss_inputs(dtype=DT[dtype])
    mask = mask if masked else None
    Hp, Wp = H.clone().requires_grad_(True), W.clone().requires_grad_(True)
    loss = ckl.chunked_kl_loss(Hp, Wp, idx, tl, mask, chunk=128, save_8bit=True)
    plain, lse, _ = ckl.forward(H, W, idx, tl, mask, chunk=128)
    assert same_bits(loss.detach().reshape(1), plain)  # the loss is that of the exact states
    (3.0 * loss).backward()
    held = ckl.act_decode(*ckl.act_encode(H), dtype=H.dtype)
    dH, dW = ckl.backward(held, W, idx, tl, mask, lse, torch.tensor([3.0], device="cuda"), chunk=128,
                          dh_dtype=H.dtype, dw_dtype=W.dtype)
    assert same_bits(Hp.grad, dH) and same_bits(Wp.grad, dW)
    exact_h, exact_w = ckl.backward(H, W, idx, tl, mask, lse, torch.tensor([3.0], device="cuda"), chunk=128)
    # states off by at most 1/127.5 of their block's maximum (3 to 4 of their size): logits off by about a percent
    for got, ref in ((Hp.grad, exact_h), (Wp.grad, exact_w)):
        assert (got.double() - ref.double()).norm() <= 0.05 * ref.double().norm()
    with torch.no_grad():
        assert same_bits(ckl.chunked_kl_loss(Hp, Wp, idx, tl, mask, chunk=128, save_8bit=True).reshape(1), plain)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_loss_with_the_norm_before_the_head(dtype):
    X, W, idx, tl, mask = loss_inputs(dtype=DT[dtype], seed=20)
    nw = (1 + normal((72,), torch.float32, 9, 0.2)).to(DT[dtype]).cuda()
    leaves = [t.clone().requires_grad_(True) for t in (X, W, nw)]
    loss = ckl.chunked_kl_loss(leaves[0], leaves[1], idx, tl, mask, chunk=128, save_8bit=True, norm_weight=leaves[2],
                               norm_eps=1e-5)
    y, codes, exps, rstd = ckl.norm_forward(X, nw, 1e-5)
    plain, lse, _ = ckl.forward(y, W, idx, tl, mask, chunk=128)
    assert same_bits(loss.detach().reshape(1), plain)
    loss.backward()
    h = ckl.act_decode(codes, exps, rstd, nw, dtype=X.dtype)
    dH, dW = ckl.backward(h, W, idx, tl, mask, lse, None, chunk=128, dh_dtype=X.dtype, dw_dtype=W.dtype)
    dX, dn = ckl.norm_backward(dH, codes, exps, rstd, nw)
    for leaf, ref in zip(leaves, (dX, dW, dn)):
        assert same_bits(leaf.grad, ref)
    # the one-call loss behind the same norm: same loss, gradients up to the 8-bit states
    fused = [t.clone().requires_grad_(True) for t in (X, W, nw)]
    lf = ckl.chunked_kl_loss(fused[0], fused[1], idx, tl, mask, chunk=128, fused=True, save_8bit=True,
                             norm_weight=fused[2], norm_eps=1e-5)
    lf.backward()
    assert abs(float(lf) - float(loss)) <= 1e-5 * abs(float(loss))
    for a, b in zip(fused, leaves):
        assert (a.grad.double() - b.grad.double()).norm() <= 0.05 * b.grad.double().norm()
    # only some gradients asked for
    only = nw.clone().requires_grad_(True)
    ckl.chunked_kl_loss(X, W, idx, tl, mask, chunk=128, save_8bit=True, norm_weight=only, norm_eps=1e-5).backward()
    assert same_bits(only.grad, dn)


@pytest.mark.parametrize("norm", [False, True])
def test_loss_without_a_backward_pass_saves_nothing(norm, monkeypatch):
    X, W, idx, tl, mask = loss_inputs(seed=21)
    nw = (1 + normal((72,), torch.float32, 9, 0.2)).cuda().requires_grad_(True) if norm else None
    leaves = [t.clone().requires_grad_(True) for t in (X, W)]
    loss = ckl.chunked_kl_loss(*leaves, idx, tl, mask, chunk=128, save_8bit=True, norm_weight=nw)
    forward, saves = ops.norm_forward, []
    monkeypatch.setattr(ops, "act_encode", lambda x: saves.append("encode"))
    monkeypatch.setattr(ops, "norm_forward", lambda x, w, eps, save=True: saves.append(save) or forward(x, w, eps, save))
    with torch.no_grad():
        again = ckl.chunked_kl_loss(*leaves, idx, tl, mask, chunk=128, save_8bit=True, norm_weight=nw)
    assert saves == [False] * norm and not again.requires_grad
    assert same_bits(again, loss.detach())


def dense_step(emb, nw, tok, teacher, K, scale, eps, mask):
    """The whole step in 64 bits on the CPU: tied embedding, norm, head, KL against the top-K teacher."""
    x = torch.where((tok >= 0)[:, None], emb[tok.clamp(min=0)] * scale, torch.zeros((), dtype=torch.float64))
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * nw
    logq = torch.log_softmax(y @ emb.t(), 1)
    vals, idx = torch.topk(teacher, K, 1)
    p = torch.softmax(vals, 1)
    rows = (p * (torch.log(p) - torch.gather(logq, 1, idx))).sum(1)
    return (rows * mask).sum() / mask.sum()


@pytest.mark.parametrize("fused", [False, True])
def test_a_training_step_of_a_tied_model(fused):
    T, d, V, K, scale, eps = 260, 64, 900, 16, 8.0, 1e-5
    emb, nw = normal((V, d), torch.float32, 1, d ** -0.5), 1 + normal((d,), torch.float32, 2, 0.2)
    tok = tokens_of("zipf", T, V, 3)
    tok[::13] = -1
    teacher = normal((T, V), torch.float32, 4, 2.0)
    mask = tok >= 0
    E, N = emb.cuda().requires_grad_(True), nw.cuda().requires_grad_(True)
    idx, vals, _ = ckl.teacher_topk(teacher.cuda(), K, mask.cuda())
    x = ckl.embedding(E, tok.cuda(), scale)
    loss = ckl.chunked_kl_loss(x, E, idx, vals, mask.cuda(), chunk=64, fused=fused, save_8bit=True, norm_weight=N,
                               norm_eps=eps)
    loss.backward()
    e64, n64 = emb.double().requires_grad_(True), nw.double().requires_grad_(True)
    ref = dense_step(e64, n64, tok, teacher.double(), K, scale, eps, mask.double())
    ref.backward()
    assert abs(float(loss) - float(ref)) <= 1e-5 * abs(float(ref))
    for got, want in ((E.grad, e64.grad), (N.grad, n64.grad)):
        assert (got.double().cpu() - want).norm() <= 0.03 * want.norm()  # the norm's input in 8 bits
    # by hand, the embedding's share added to the head's gradient: the same sum
    with torch.no_grad():
        y, codes, exps, rstd = ckl.norm_forward(ckl.embedding_forward(E, tok.cuda(), scale), N, eps)
        _, _, _, dH, dW = ckl.forward_backward(y, E, idx, vals, mask.cuda(), chunk=64)
        dX, _ = ckl.norm_backward(dH, codes, exps, rstd, N)
        total = ckl.embedding_backward(dX, tok.cuda(), V, scale, add_to=dW)
        assert total is dW
        assert (total.double().cpu() - e64.grad).norm() <= 0.03 * e64.grad.norm()


def step(z, W, tok, nw, dW):
    """The operators as a training loop without autograd calls them."""
    idx, vals, lse = ckl.teacher_topk(z, 12, teacher_form=1)
    x = ckl.embedding_forward(W, tok, 8.0)
    y, codes, exps, rstd = ckl.norm_forward(x, nw)
    loss, s, _ = ckl.forward(y, W, idx, vals, None, chunk=256, teacher_form=1)
    dH, dW2 = ckl.backward(ckl.act_decode(codes, exps, rstd, nw), W, idx, vals, None, s, None, chunk=256,
                           teacher_form=1)
    dx, dn = ckl.norm_backward(dH, codes, exps, rstd, nw)
    dW.copy_(dW2)
    ckl.embedding_backward(dx, tok, W.shape[0], 8.0, add_to=dW)
    return idx, vals, lse, loss, dx, dn, dW


def step_inputs(seed, T, V=700, d=64):
    return (normal((T, V), torch.bfloat16, seed, 2.0).cuda(), normal((V, d), torch.bfloat16, seed + 1, d ** -0.5).cuda(),
            tokens_of("padded", T, V, seed + 2).cuda(), (1 + normal((d,), torch.float32, seed + 3, 0.1)).cuda(),
            torch.zeros(V, d, device="cuda"))


@pytest.mark.parametrize("T", [5, 600, 9000])
def test_captured_step_replays_with_new_inputs(T):
    ins = step_inputs(1, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*ins)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*ins)
    for seed in (1, 50, 90, 50):
        new = step_inputs(seed, T)
        for a, b in zip(ins[:4], new[:4]):
            a.copy_(b)
        want = [t.clone() for t in step(*new)]   # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert same_bits(a, b)


def test_captured_gradients_replay_with_new_inputs():
    # forward and backward through autograd in one graph; the leaves have no other graph alive
    T, d, V, K = 300, 72, 500, 9

    def inputs(seed):
        idx, vals, _ = ckl.teacher_topk(normal((T, V), torch.bfloat16, seed, 2.0).cuda(), K)
        return [normal((V, d), torch.bfloat16, seed + 1, 0.2).cuda(), tokens_of("padded", T, V, seed + 2).cuda(),
                (1 + normal((d,), torch.bfloat16, seed + 3, 0.1)).cuda(), idx, vals]

    def grads(W, tok, nw, idx, vals):
        W, nw = W.detach().requires_grad_(True), nw.detach().requires_grad_(True)
        x = ckl.embedding(W, tok, 4.0)
        loss = ckl.chunked_kl_loss(x, W, idx, vals, chunk=128, save_8bit=True, norm_weight=nw)
        more = ckl.rms_norm_8bit(x, nw).float().sum()
        return [loss.detach(), *torch.autograd.grad(loss + 0.01 * more, (W, nw))]
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
        new = inputs(seed)
        for a, b in zip(ins, new):
            a.copy_(b)
        want = grads(*new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert same_bits(a, b)


def test_streams_and_concurrent_calls():
    ins = [step_inputs(s, 3000) for s in (1, 30)]
    want = [[t.clone() for t in step(*i)] for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = []
    for s, i in zip(streams, ins):
        with torch.cuda.stream(s):
            got.append(step(*i))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert same_bits(x, y)


def test_outputs_and_neighbours_stay_untouched():
    # results written into the middle of larger buffers: nothing around them changes
    lib = B.load_library()
    T, V, K, d = 9, 333, 5, 40
    z = normal((T, V), torch.float32, 1).cuda()
    buf = torch.full((T * K + 64,), -7, dtype=torch.int32, device="cuda")
    val, lse = torch.full((T * K + 64,), -7.0, device="cuda"), torch.full((T + 64,), -7.0, device="cuda")
    import ctypes
    need = ctypes.c_size_t(0)
    B.check(lib.ckl_topk_workspace_size(T, V, K, ctypes.byref(need)))
    ws = torch.full((need.value + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    B.check(lib.ckl_teacher_topk(z.data_ptr(), 0, T, V, K, 0, None, buf.data_ptr() + 64, val.data_ptr() + 64,
                                 lse.data_ptr() + 64, ws.data_ptr(), need.value, None))
    torch.cuda.synchronize()
    for t in (buf, val):
        assert (t[:16] == -7).all() and (t[16 + T * K:] == -7).all() and not (t[16:16 + T * K] == -7).any()
    assert (lse[:16] == -7).all() and (lse[16 + T:] == -7).all() and (ws[need.value:] == 0xAB).all()
    x = normal((T, d), torch.float32, 2).cuda()
    codes = torch.full((T * d + 64,), 99, dtype=torch.int8, device="cuda")
    exps = torch.full((T * 2 + 64,), 99, dtype=torch.uint8, device="cuda")
    B.check(lib.ckl_act_encode(x.data_ptr(), 0, T, d, codes.data_ptr() + 32, exps.data_ptr() + 31, None))
    torch.cuda.synchronize()
    rc, re, _ = encode_reference(x.cpu())
    assert torch.equal(codes[32:32 + T * d].cpu().view(T, d), rc) and torch.equal(exps[31:31 + 2 * T].cpu().view(T, 2), re)
    assert (codes[:32] == 99).all() and (codes[32 + T * d:] == 99).all()
    assert (exps[:31] == 99).all() and (exps[31 + 2 * T:] == 99).all()
