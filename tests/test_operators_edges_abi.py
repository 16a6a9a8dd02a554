"""Calls of the operators around the loss that the C ABI refuses on the host, past those of test_operators_abi.py
(nothing is launched: every call below fails its checks)."""
import pytest

from chunked_kl_loss_amd import _binding as B
from tests.test_operators_abi import emb_b, emb_f, lib  # noqa: F401


@pytest.mark.parametrize("off", [2 ** 63 - 1, 2 ** 63 - 100])
def test_table_ends_past_the_largest_id(lib, off):  # noqa: F811
    # (a token near the other end of its type would come out inside the table)
    for call in (emb_f, emb_b):
        assert call(lib, off=off, V=100) == B.CKL_ERR_INVALID_ARG
        assert b"v_offset" in lib.ckl_last_error()
