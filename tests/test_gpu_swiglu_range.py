"""SwiGLU rows whose gate is far below zero: silu is tiny, but as long as fp32
holds its sigmoid and the up value is large, h is an ordinary number."""
import pytest
import torch

from sparse_mixture_experts_03_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
FLOOR = 2.0 ** -100


@pytest.mark.parametrize("up", [2.0 ** 60, 2.0 ** 90, 2.0 ** 120])
def test_far_negative_gates(up):
    # exp(88.5) = 2.7e38 is the last step of bf16 below fp32's largest number
    gates = torch.tensor([-1.0, -20.0, -60.0, -80.0, -87.0, -87.5, -88.0, -88.5, 3.0, 88.5],
                         device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    u = torch.randn(gates.numel(), 256, generator=gen, device=DEV)
    u *= torch.where(gates[:, None] < 0, up, 1.0)  # h stays below fp32's largest number
    gu = torch.cat([gates[:, None].expand(-1, 256), u], 1).bfloat16().contiguous()
    q, s = moe.swiglu_quantize_rows(gu)
    g, u = gu.double().split(256, 1)
    h = g * torch.sigmoid(g) * u
    # the error of h: 2^-22 (4 + |g|), from the rounded argument of the
    # exponential (|g| log2 e 2^-24), ex2.approx, the reciprocal and the products
    slack = 2.0 ** -22 * (4 + gates.double().abs())
    A = h.view(-1, 2, 128).abs().amax(2).clamp(min=FLOOR)
    assert bool(((s.t().double() - A / 448).abs() <= (slack + 2.0 ** -22)[:, None] * A / 448).all())
    t = h / (A / 448).repeat_interleave(128, 1)
    _, e = torch.frexp(t)
    half = torch.ldexp(torch.ones_like(t), (e - 4).clamp(min=-9)) / 2
    assert bool(((q.double() - t).abs() <= half + 2 * slack[:, None] * t.abs() + 2.0 ** -40).all())


def test_gates_beyond_fp32s_exponential():
    """exp(-g) is infinite: silu is zero whatever the up value is, and a far
    positive gate is its own silu."""
    gates = torch.tensor([-89.0, -1e30, 1e30], device=DEV)
    gu = torch.cat([gates[:, None].expand(-1, 128), torch.full((3, 128), 2.0, device=DEV)], 1).bfloat16()
    q, s = moe.swiglu_quantize_rows(gu.contiguous())
    assert not q[:2].double().any()
    assert bool((q[2].double() == 448).all())
    want = 2 * gu[2, 0].double() / 448
    # the reciprocal (an ulp) and one rounding of the scale
    assert abs(float(s[0, 2]) - float(want)) <= 2.0 ** -22 * float(want)
