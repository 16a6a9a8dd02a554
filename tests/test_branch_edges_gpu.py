"""What the operators behind a branch refuse on the GPU."""
import pytest
import torch

import chunked_kl_loss_amd as ckl
from tests.test_branch_gpu import DT, PAIRS, normal, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("types", PAIRS, ids=lambda t: "-".join(t))
@pytest.mark.parametrize("leaf", [0, 1, 2])
def test_the_norm_in_8_bits_says_that_it_has_no_gradient(leaf, types, form):
    # its h is the residual stream: a loss behind it must not lose that without a word
    T, d = 5, 72
    ins = [normal((T, d), DT[types[0]], 1).cuda(), normal((T, d), DT[types[1]], 2).cuda(),
           normal((d,), torch.float32, 3).cuda()]
    want = ckl.add_norm_quant(*ins, form=form)
    assert not any(t.requires_grad for t in want)
    ins[leaf].requires_grad_(True)
    got = ckl.add_norm_quant(*ins, form=form)
    assert all(same_bits(a.detach(), b) for a, b in zip(got, want))
    with pytest.raises(NotImplementedError, match="add_norm_quant has no gradient"):
        got[2].float().sum().backward()
    if form == "e4m3":
        codes, scales, _ = ckl.add_norm_quant(*ins, form=form)
        with pytest.raises(NotImplementedError, match="add_norm_quant has no gradient"):
            (codes.float() * scales[:, None]).sum().backward()
    assert ins[leaf].grad is None
    with torch.no_grad():
        got = ckl.add_norm_quant(*ins, form=form)
    assert all(same_bits(a, b) for a, b in zip(got, want)) and not any(t.requires_grad for t in got)


def test_the_norm_in_8_bits_refuses_tangents():
    fw = torch.autograd.forward_ad
    x, w = normal((4, 16), torch.float32, 2).cuda(), normal((16,), torch.float32, 3).cuda()
    with fw.dual_level():
        d = fw.make_dual(x, torch.ones_like(x))
        for form in ("int8", "e4m3"):
            for args in ((d, x, w), (x, d, w)):
                with torch.no_grad(), pytest.raises(NotImplementedError, match="jvp"):
                    ckl.add_norm_quant(*args, form=form)
