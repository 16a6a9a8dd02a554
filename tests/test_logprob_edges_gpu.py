"""Log probabilities of given tokens from logits on the GPU, where plain formulas lose: logits far from zero whose
differences are ordinary."""
import pytest
import torch

import chunked_kl_loss_amd as ckl
from tests.test_logprob_gpu import normal, rows_reference, some_tokens, within

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
