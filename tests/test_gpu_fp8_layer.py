"""The layer on 8-bit weights: refusals, and what its callers can ask of it."""
import pytest
import torch

from sparse_mixture_experts_03_b200.fp8 import Fp8MoE

pytestmark = pytest.mark.gpu
DEV = "cuda"
E, D, I, S, K, G, TG = 16, 512, 256, 2, 4, 4, 2


def randn(*shape, seed=0, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)


def make(S=S, I=I, D=D, seed=0, **kw):
    sh = None
    if S:
        sh = torch.cat([randn(2 * S * I * D, seed=seed + 3, scale=D ** -0.5),
                        randn(S * I * D, seed=seed + 4, scale=I ** -0.5)])
    w = dict(W_router=randn(E, D, seed=seed, scale=D ** -0.5),
             W_gate_up=randn(E, 2 * I, D, seed=seed + 1, scale=D ** -0.5),
             W_down=randn(E, D, I, seed=seed + 2, scale=I ** -0.5), W_shared=sh)
    w.update(kw)
    return Fp8MoE(**w, k=K, n_group=G, topk_group=TG, inter=I, n_shared=S)


def test_wrong_types_and_shapes_are_refused_at_every_batch_size():
    with pytest.raises(TypeError):
        make(W_router=randn(E, D, dtype=torch.float32))
    with pytest.raises(TypeError):
        make(expert_bias=randn(E))
    layer = make()
    for T in (4, 40):
        for x, error in [(randn(T, D, dtype=torch.float32), TypeError),
                         (randn(T, D + 256), ValueError), (randn(T, D - 256), ValueError),
                         (randn(T, 2 * D)[:, ::2], ValueError), (randn(T, D).cpu(), ValueError)]:
            with pytest.raises(error):
                layer(x)
        assert layer(randn(T, D)).shape == (T, D)
