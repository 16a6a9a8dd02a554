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


def test_more_threads_than_a_launch_takes(lib):  # noqa: F811
    # 32 elements a thread; a grid of 2^32 threads or more would lose those past its low 32 bits without an error
    for T, d in ((4_000_000, 65536), (2 ** 21, 65536), (4_000_000, 34360)):
        assert emb_f(lib, T=T, d=d) == B.CKL_ERR_UNSUPPORTED
        assert b"2^37" in lib.ckl_last_error()
    assert emb_f(lib, T=2 ** 21 - 1, d=65536, nb=3) == B.CKL_ERR_INVALID_ARG and b"token_bytes" in lib.ckl_last_error()
