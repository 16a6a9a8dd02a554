"""Log probabilities from states and head on the GPU: logits far from zero, gradients cut into blocks of rows and of
words, and more elements than a launch has threads."""
import math

import pytest
import torch

import chunked_kl_loss_amd as ckl
from tests.test_head_gpu import check, grid, inputs
from tests.test_logprob_gpu import DT, EPS, gen, normal, rows_reference, same_bits, some_tokens, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("base", [128, -128])
@pytest.mark.parametrize("T,V", [(3, 3001), (40, 1500), (100, 5003), (300, 2049)])
def test_log_probabilities_of_logits_far_from_zero(T, V, base, dtype):
    # one column adds 2^14 or its negative to all logits: multiples of 2^-6 below 2^15, exact in fp32
    d = 16
    H, W = grid((T, d), DT[dtype], 1, 0.25), grid((V, d), DT[dtype], 2, 2.0 ** -4)
    H[:, 0], W[:, 0] = 128, base
    tok = some_tokens(T, V, 3)
    z = H.double() @ W.double().t()
    r = rows_reference(z, tok)
    s = r["lse"] - z.max(1).values
    lp, ent, lse = ckl.head_logprobs_forward(H.cuda(), W.cuda(), tok.cuda())
    # (z - m) - ln s: the sum's tolerance (tests/test_logprob_gpu.py), and a rounding of each difference, of the
    # logarithm, of log2 e and of ln 2
    tol = (V / 256 + 40) * EPS + 2.0 ** -22 + 6 * EPS * (r["logprob"].abs() + 2 * s + 1)
    assert within(lp, r["logprob"], tol)
    assert within(ent, r["entropy"], r["tol_ent"])
    # ln 2 (m + log2 s): a rounding of m, of the sum, of the product and of either constant
    assert within(lse, r["lse"], tol + 6 * EPS * r["lse"].abs())


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


# A launch of 2^32 threads or more loses those past its low 32 bits without an error.
V_WIDE, D_WIDE = 65600, 65536  # their product is past 2^32


@pytest.fixture
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_a_zero_gradient_of_more_elements_than_a_launch_has_threads(room):
    V, d = V_WIDE, D_WIDE
    W = torch.ones(V, d, dtype=torch.bfloat16, device="cuda")
    H = torch.ones(0, d, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, device="cuda")
    _, dW = ckl.head_logprobs_backward(none, none, H, W, none.long(), none, none)
    assert float(dW.amax()) == float(dW.amin()) == 0


def test_a_rounded_gradient_of_more_elements_than_a_launch_has_threads(room):
    V, d = V_WIDE, D_WIDE
    g = torch.Generator("cuda")
    g.manual_seed(1)
    W = torch.empty(V, d, device="cuda").normal_(0.0, 2.0 ** -8, generator=g)
    H = torch.zeros(2, d, device="cuda")
    H[:, :4], H[:, -4:] = 1.0, 2.0
    tok = torch.tensor([V - 1, 3], device="cuda")
    lp, ent, lse = ckl.head_logprobs_forward(H, W, tok)
    a = torch.tensor([8.0, -2.0], device="cuda")
    _, dW = ckl.head_logprobs_backward(a, None, H, W, tok, lse, ent, need_dh=False, dw_dtype=torch.bfloat16)
    for words in (slice(0, 40), slice(V // 2, V // 2 + 40), slice(V - 40, V)):
        z = H.double() @ W[words].double().t()
        G = -torch.exp(z - lse.double()[:, None]) * a.double()[:, None]
        for i in range(2):
            at = int(tok[i]) - words.start
            if 0 <= at < 40:
                G[i, at] += a[i].double()
        want = G.t() @ H.double()
        # z: 8 products of at most 2^-5 (|z| < 1) that sum up in fp32, lse its tolerance: relative 2^-18 of G; one rounding
        assert ((dW[words].double() - want).abs() <= (2.0 ** -18 + 2.0 ** -8) * (G.abs().t() @ H.double()) + 1e-37).all()
    assert not dW[:, 4:-4].any()


def test_packed_states_of_more_pieces_than_a_launch_has_threads(room):
    T, d, V = 524_400, 65536, 8  # T d / 8 is past 2^32
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GiB")
    H = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    last = inputs(200, d, V, torch.bfloat16, 1)
    H[-200:] = last[0].cuda()
    W = last[1].cuda()
    tok = torch.zeros(T, dtype=torch.int64, device="cuda")
    tok[-200:] = last[2].cuda()
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[3] = False
    lp, ent, lse = ckl.head_logprobs_forward(H, W, tok, mask)
    want = ckl.head_logprobs_forward(last[0].cuda(), W, last[2].cuda())
    assert float(lp[3]) == 0 and (lp[:-200][torch.arange(T - 200, device="cuda") != 3] == lp[0]).all()
    z = last[0].double() @ last[1].double().t()
    r = rows_reference(z, last[2])
    for got, w, key, tol in zip((lp, ent, lse), want, ("logprob", "entropy", "lse"), ("tol_lp", "tol_ent", "tol_lse")):
        t = r[tol] + 4 * EPS * r["lse"].abs()
        assert within(got[-200:], r[key], t) and within(w, r[key], t)
