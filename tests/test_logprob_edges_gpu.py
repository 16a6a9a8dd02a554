"""Log probabilities of given tokens from logits on the GPU, where plain formulas lose: logits far from zero whose
differences are ordinary.  The log-sum-exp rounds at its own size there; what is taken from differences does not have
to."""
import pytest
import torch

import chunked_kl_loss_amd as ckl
from tests.test_logprob_gpu import DT, EPS, HALF, normal, rows_reference, some_tokens, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("base", [1e4, -3e4, 4e6])
@pytest.mark.parametrize("T,V,top", [(5, 3001, 0), (5, 3001, 7), (3, 1500, 7), (2, 30001, 70), (1100, 5003, 70),
                                     (1, 120001, 1025)])
def test_entropies_of_logits_far_from_zero(T, V, top, base):
    z = (base + normal((T, V), torch.float32, T + V, 3.0).double()).float()
    z[:, V // 2:] += 8.0  # a reference that moves while much has been added up behind it
    tok = some_tokens(T, V, 1)
    _, ent, _, _, _ = ckl.token_logprobs_forward(z.cuda(), tok.cuda(), top)
    r = rows_reference(z.double(), tok)
    assert within(ent, r["entropy"], r["tol_ent"])


@pytest.mark.parametrize("base", [1e4, -3e4, 4e6])
@pytest.mark.parametrize("T,V,top", [(5, 3001, 0), (5, 3001, 7), (3, 1500, 7), (2, 30001, 70), (1100, 5003, 70),
                                     (1, 120001, 1025)])
def test_log_probabilities_of_logits_far_from_zero(T, V, top, base):
    z = (base + normal((T, V), torch.float32, T + V, 3.0).double()).float()
    tok = some_tokens(T, V, 1)
    z[torch.arange(T), tok] += 6.0
    lp, ent, lse, idx, val = ckl.token_logprobs_forward(z.cuda(), tok.cuda(), top)
    z64 = z.double()
    r = rows_reference(z64, tok)
    s = r["lse"] - z64.max(1).values  # ln of the sum behind the maximum

    def tol(logprob, s):
        # (z - m) - ln s: the sum's tolerance (tests/test_logprob_gpu.py), one rounding of each difference and of the
        # logarithm, whose reference m lies within 4 of the maximum
        return (V / 256 + 40) * EPS + 2.0 ** -22 + 4 * EPS * (logprob.abs() + 2 * s + 8)
    assert within(lp, r["logprob"], tol(r["logprob"], s))
    assert within(ent, r["entropy"], r["tol_ent"])
    assert within(lse, r["lse"], r["tol_lse"])
    if top:
        lv = z64.gather(1, idx.cpu().long()) - r["lse"][:, None]
        assert within(val, lv, tol(lv, s[:, None]))
        assert ((idx == tok.cuda()[:, None]) <= (val == lp[:, None])).all()  # the token among them: the same number


@pytest.mark.parametrize("top", [0, 3, 70])
@pytest.mark.parametrize("fill", [-1e31, 3e8, torch.finfo(torch.float32).min])
def test_a_row_of_one_far_value_is_uniform(fill, top):
    V = 4001
    z = torch.full((2, V), fill)
    z[1, 10:] = -torch.inf
    tok = torch.tensor([5, 6])
    lp, ent, lse, idx, val = ckl.token_logprobs_forward(z.cuda(), tok.cuda(), top)
    # the sum is a whole number, exact; one rounding of its logarithm
    want = -torch.log(torch.tensor([V, 10], dtype=torch.float64))
    assert within(lp, want, 4 * EPS * want.abs())
    if top:
        assert within(val[:, :3], want[:, None].expand(2, 3), (4 * EPS * want.abs())[:, None].expand(2, 3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_forbidden_tokens(dtype):
    # none, but where one is the given token: that of its own log probability, which the formula leaves it
    T, V = 4, 1003
    z = normal((T, V), DT[dtype], 1, 2.0)
    z[:, ::3] = -torch.inf
    tok = torch.tensor([0, 1, 3, 999])
    Z = z.cuda().requires_grad_(True)
    lp, ent, _, _ = ckl.token_logprobs(Z, tok.cuda())
    (dz,) = torch.autograd.grad((lp, ent), (Z,), (torch.full_like(lp, 1.5), torch.full_like(ent, 0.5)))
    dz, gone = dz.double().cpu(), torch.isinf(z)
    own = torch.zeros_like(gone)
    own[torch.arange(T), tok] = True
    assert (dz[gone & own] == 1.5).all() and int((gone & own).sum()) == 3 and not dz[gone & ~own].any()
    q = torch.softmax(z.double(), 1)
    logq = torch.where(gone, 0.0, torch.log_softmax(z.double(), 1))
    want = 1.5 * own - q * (1.5 + 0.5 * (logq - (q * logq).sum(1, keepdim=True)))
    # sums and arguments: as in the log probabilities' tolerance; one rounding
    tau = ((V / 256 + 40) * EPS + 2.0 ** -20) * 10
    assert ((dz - want).abs() <= tau * (q + EPS) + HALF[DT[dtype]] * want.abs()).all()
