"""Sizes next to and beyond 31 bits (no GPU: refusals come before anything is
queued)."""
import ctypes

import pytest

from sparse_mixture_experts_03_b200 import moe

BAD, UNSUP = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
INT_MAX = 2 ** 31 - 1


def product(R=4, n=64, k=128, G=1):
    counts = ctypes.c_void_p(256) if G > 1 else None
    return moe.lib().moe_matmul_fp8(None, None, None, None, counts, R, G, n, k, moe.MOE_BF16, None,
                                    None, None)


# The kernel rounds R and k up to 128 and n up to 256, in 32 bits: 2^31 must not
# be reached.
@pytest.mark.parametrize("sizes", [dict(k=INT_MAX - 15), dict(k=INT_MAX - 111), dict(R=INT_MAX, n=1, k=16),
                                   dict(R=INT_MAX - 126, n=1, k=16), dict(R=1, n=INT_MAX, k=16),
                                   dict(R=1, n=INT_MAX - 254, k=16)])
def test_sizes_whose_tiles_pass_31_bits_are_refused(sizes):
    assert product(**sizes) == UNSUP


@pytest.mark.parametrize("sizes", [dict(k=INT_MAX - 127), dict(R=INT_MAX - 127, n=1, k=16),
                                   dict(R=1, n=INT_MAX - 255, k=16)])
def test_the_largest_sizes_are_taken(sizes):
    assert product(**sizes) == BAD  # the missing pointers, checked after the sizes
