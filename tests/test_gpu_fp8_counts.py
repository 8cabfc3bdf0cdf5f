"""Counts of the grouped 8-bit product that ask for more rows than there are."""
import pytest
import torch

from sparse_mixture_experts_03_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
R, N, K = 100, 64, 128


def operands(G):
    g = torch.Generator(device=DEV).manual_seed(G)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    return (*moe.quantize_rows(randn(R, K)), *moe.quantize_weight(randn(G, N, K)))


@pytest.mark.parametrize("counts", [[R + 1], [R + 50], [2 ** 31 - 1], [0, R + 1, 0], [-3, 0, R + 1],
                                    [0, 2 ** 31 - 1, -7], [0] * 40 + [R + 1], [R, 1], [R, 0, 0, 1],
                                    [2 ** 31 - 1] * 256])
def test_one_count_too_many_is_cut_and_reported(counts):
    a, sa, b, sb = operands(len(counts))
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    guard = torch.full((R + 50, N), 3.0, device=DEV)
    moe.matmul_fp8(a, sa, b, sb, c, y=guard[:R], status_ws=ws)
    assert moe.device_status(ws)[0] == moe.MOE_ERR_DEVICE
    assert bool((guard[R:] == 3.0).all())
    # the rows that there are belong to the first group that asks for any
    first = next(g for g, n in enumerate(counts) if n > 0)
    want = moe.matmul_fp8(a, sa, b[first], sb[first], out_dtype=torch.float32)
    assert torch.equal(guard[:R], want)


@pytest.mark.parametrize("counts", [[R], [R - 1], [0, R, 0], [-5, R], [0, 0], [40, 60], [0] * 40 + [R]])
def test_counts_that_fit_are_not_reported(counts):
    a, sa, b, sb = operands(len(counts))
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    moe.matmul_fp8(a, sa, b, sb, c, status_ws=ws)
    assert moe.device_status(ws)[0] == moe.MOE_OK
