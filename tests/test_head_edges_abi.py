"""What the backward pass of log probabilities from states and head holds, without a GPU."""
import pytest

from tests.test_operators_abi import lib, size  # noqa: F401

SHAPES = [(1_000_000, 512, 32000), (131072, 2880, 201088), (32768, 2880, 201088), (32768, 1024, 50264),
          (2048, 2880, 201088), (16, 2880, 201088), (8192, 512, 1000), (4_000_000, 64, 1000), (20, 64, 4_000_000)]
PARTS = 340 << 20  # dH's parts of one block of rows: a tile of 256 x 320 fp32 for each quarter of 256 compute units


def backward(lib, T, d, V, chunk, dt=1, dh=1, dw=1, masked=0):  # noqa: F811
    return size(lib.ckl_head_workspace_size, T, d, V, chunk, dt, dh, dw, masked, 1)


@pytest.mark.parametrize("dt", [1, 0])
@pytest.mark.parametrize("masked", [0, 1])
@pytest.mark.parametrize("T,d,V", SHAPES)
def test_chunk_bounds_what_grows_with_rows_and_words(lib, T, d, V, masked, dt):  # noqa: F811
    e = 2 if dt else 4
    for chunk in (16, 64, 256, 1024, 2048, 8192):
        G = (max(chunk, 256) + 256) * (V + 512) * e     # of the logits' gradients (fp32: half, and half their transpose)
        states = (T + 512) * d * e * (1 + masked)       # H's transpose, and its packed rows
        head = (V + 512) * d * e                        # the transpose of a block of words
        sums = (T + 8) * d * 4 + V * d * 4              # dH and dW in fp32
        for dh, dw in ((0, 0), (1, 1)):
            assert backward(lib, T, d, V, chunk, dt, dh, dw, masked) <= G + states + head + sums + PARTS + 64 * T + (8 << 20)


@pytest.mark.parametrize("out", [0, 1])
@pytest.mark.parametrize("masked", [0, 1])
@pytest.mark.parametrize("T,d,V", SHAPES[:4])
def test_a_smaller_chunk_does_not_hold_more(lib, T, d, V, masked, out):  # noqa: F811
    # but for sums in fp32 that outputs in bf16 (and a packed dH) need once rows and words are cut; blocks and parts are
    # whole tiles, a few of them more
    once = (T * d * 4 if out or masked else 0) + (V * d * 4 if out else 0)
    at = [backward(lib, T, d, V, 8192 >> i, dh=out, dw=out, masked=masked) for i in range(10)]
    assert all(b <= a + once + (64 << 20) for i, a in enumerate(at) for b in at[i + 1:])
