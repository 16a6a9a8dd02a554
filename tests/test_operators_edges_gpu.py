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
from tests.test_operators_gpu import DT, EPS, check_topk, normal, same_bits

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
