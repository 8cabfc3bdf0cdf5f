"""Sizes next to and beyond 31 bits (no GPU: refusals come before anything is
queued)."""
import ctypes

import pytest
import torch

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

def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda n: moe.quantize_rows(meta(n, 16)),
    lambda n: moe.swiglu_quantize_rows(meta(n, 32)),
    lambda n: moe.quantize_weight(meta(n, 16)),
    lambda n: moe.quantize_weight(meta(n, 1, 16)),
    lambda n: moe.quantize_weight(meta(1, n)),
    lambda n: moe.matmul_fp8(meta(n, 16, dtype=moe.E4M3), meta(1, n, dtype=torch.float32),
                             meta(1, 16, dtype=moe.E4M3), meta(1, 1, dtype=torch.float32)),
    lambda n: moe.matmul_fp8(meta(1, 16, dtype=moe.E4M3), meta(1, 1, dtype=torch.float32),
                             meta(n, 16, dtype=moe.E4M3),
                             meta((n + 127) // 128, 1, dtype=torch.float32)),
])
def test_sizes_beyond_a_c_int_are_refused(monkeypatch, call):
    """2^32 + 16 rows are not 16 rows."""
    class Library:
        def __getattr__(self, name):
            return lambda *args: pytest.fail(f"{name} was reached with {args}")
    monkeypatch.setattr(moe, "lib", lambda: Library())
    monkeypatch.setattr(moe, "_on_current", lambda name, t, s: (0, 0))
    for n in (2 ** 31, 2 ** 32 + 16):
        with pytest.raises(ValueError, match="2\\^31"):
            call(n)
