"""Log probabilities of given tokens from logits on the GPU, where plain formulas lose: logits far from zero whose
differences are ordinary.  The log-sum-exp rounds at its own size there; what is taken from differences does not have
to."""
import pytest
import torch

import chunked_kl_loss_amd as ckl
from tests.test_logprob_gpu import EPS, normal, rows_reference, some_tokens, within

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
