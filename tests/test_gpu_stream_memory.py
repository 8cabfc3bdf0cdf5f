"""Calls for another stream that allocate what they return, while freed memory
of the same sizes still has work queued on the current stream."""
import pytest
import torch

from sparse_mixture_experts_03_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).bfloat16()


def rows():
    x = randn(96, 1024)
    return lambda **kw: moe.quantize_rows(x, **kw)


def swiglu():
    x = randn(96, 2048)
    return lambda **kw: moe.swiglu_quantize_rows(x, **kw)


def weight():
    W = randn(2, 640, 1024)
    return lambda **kw: moe.quantize_weight(W, **kw)


def product():
    ops = (*moe.quantize_rows(randn(96, 1024)), *moe.quantize_weight(randn(640, 1024, seed=1)))
    return lambda **kw: moe.matmul_fp8(*ops, **kw)


def few():
    E, k, d, I = 16, 4, 512, 256
    args = (randn(4, d), randn(E, d, seed=1, scale=d ** -0.5),
            randn(E, 2 * I, d, seed=2, scale=d ** -0.5), randn(E, d, I, seed=3, scale=I ** -0.5))
    return lambda **kw: moe.forward_few(*args, None, k, 4, 2, I, 0, **kw)


def flat(out):
    return [t.view(torch.uint8) for t in (out if isinstance(out, tuple) else (out,))]


@pytest.mark.parametrize("make", [rows, swiglu, weight, product, few])
def test_freed_memory_with_work_behind_it(make):
    call = make()
    want = [t.clone() for t in flat(call())]
    sizes = [t.numel() for t in want]
    if make is few:
        sizes.append(moe.few_workspace_bytes(4, 512, 16, 4, 256, 0))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(4_000_000)  # what follows on this stream starts 2 ms later
        tmp = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xFF) for n in sizes]
        del tmp
        got = call(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(flat(got), want))


@pytest.mark.parametrize("make", [rows, product, few])
def test_results_are_not_reused_while_the_current_stream_reads_them(make):
    call = make()
    want = [t.clone() for t in flat(call())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = flat(call(stream=side))
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(4_000_000)
        copies = [t.clone() for t in got]  # read here, 2 ms later
        sizes = [t.numel() for t in got]
        del got
        with torch.cuda.stream(side):  # the next owner of such memory writes at once
            junk = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xFF) for n in sizes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))
        del junk
