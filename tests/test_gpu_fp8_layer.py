"""The layer on 8-bit weights: refusals, and what its callers can ask of it."""
import pytest
import torch

from sparse_mixture_experts_03_b200 import moe
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


def test_status_of_a_call():
    layer = make()
    ws = torch.full((layer.workspace_bytes(1100),), 0xAB, dtype=torch.uint8, device=DEV)
    for T in (1, 8, 9, 300, 1100, 5):  # whatever the last batch left in the workspace
        x = randn(T, D, seed=T)
        y = layer(x, workspace=ws)
        assert moe.device_status(ws)[0] == moe.MOE_OK
        assert torch.equal(y, layer(x))


def test_a_steps_error_is_seen(monkeypatch):
    layer, x = make(), randn(40, D)
    ws = torch.zeros(layer.workspace_bytes(40), dtype=torch.uint8, device=DEV)
    disp = moe.dispatch(x, layer.W_router, K, G, TG)
    status = torch.zeros(256, dtype=torch.uint8, device=DEV)
    layer.experts(disp.x_perm, disp.w_perm, disp.counts, status)
    assert moe.device_status(status)[0] == moe.MOE_OK
    layer.experts(disp.x_perm, disp.w_perm, disp.counts + 1, status)
    assert moe.device_status(status)[0] == moe.MOE_ERR_DEVICE

    dispatch = moe.dispatch

    def too_many(*args, **kw):  # the rows that there are still go to some expert
        out = dispatch(*args, **kw)
        out.counts[0] += 40 * K
        return out
    good = layer(x, workspace=ws)
    monkeypatch.setattr(moe, "dispatch", too_many)
    layer(x, workspace=ws)
    assert moe.device_status(ws)[0] == moe.MOE_ERR_DEVICE
    monkeypatch.setattr(moe, "dispatch", dispatch)
    assert torch.equal(layer(x, workspace=ws), good)  # and the next call starts anew
    assert moe.device_status(ws)[0] == moe.MOE_OK


def test_workspaces_that_do_not_fit_are_refused():
    layer = make()
    for T in (4, 40):
        x = randn(T, D)
        with pytest.raises(moe.MoeError):
            layer(x, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
        with pytest.raises(moe.MoeError):  # not aligned
            layer(x, workspace=torch.empty(1 << 22, dtype=torch.uint8, device=DEV)[16:])
        with pytest.raises(ValueError):
            layer(x, workspace=torch.empty(1 << 22, dtype=torch.uint8))


def test_a_captured_call_with_its_workspace():
    layer = make()
    for T in (5, 40):
        x = randn(T, D, seed=T)
        ws = torch.empty(layer.workspace_bytes(T), dtype=torch.uint8, device=DEV)
        layer(x, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = layer(x, ws)
        for seed in (1, 2):
            x.copy_(randn(T, D, seed=seed))
            g.replay()
            assert torch.equal(y, layer(x))
            assert moe.device_status(ws)[0] == moe.MOE_OK
        del g


def wide(q, s):
    """The values that codes [..., n, k] and their block scales stand for."""
    n, k = q.shape[-2:]
    return q.double() * s.double().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]


def layer64(layer, x, idx, w):
    """The layer in 64 bits on its 8-bit weights, for a given routing."""
    silu = torch.nn.functional.silu
    ffn = lambda gu, dn, v: (silu(v @ gu[:dn.shape[1]].t()) * (v @ gu[dn.shape[1]:].t())) @ dn.t()
    X = x.double()
    y = torch.zeros_like(X)
    if layer.n_shared:
        y += ffn(wide(*layer.shared_gate_up), wide(*layer.shared_down), X)
    gu, dn = wide(layer.W_gate_up, layer.s_gate_up), wide(layer.W_down, layer.s_down)
    for e in range(layer.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        y[t] += w[t, j, None].double() * ffn(gu[e], dn[e], X[t])
    return y


def check_tokens(layer, x):
    """Every token by itself: rounding a row to e4m3 is off by at most r = 2^-4 /
    sqrt(3) of its norm (half a step either way, evenly); x's error reaches h
    through gate (|silu'| <= 1.1) and up, 2.1 r, and h has its own, r.  A token
    that lost one of its k experts is off by far more than 3.1 r = 0.11.  In
    the one call x stays 16-bit and h is rounded to bf16."""
    y = layer(x)
    idx, w = moe.route(x, layer.W_router, K, G, TG)
    ref = layer64(layer, x, idx.long(), w)
    err = (y.double() - ref).norm(dim=1) / ref.norm(dim=1)
    assert float(err.max()) <= (5e-3 if len(x) <= layer.few else 3.1 * 2.0 ** -4 / 3 ** 0.5)


@pytest.mark.parametrize("T", [1, 8, 40, 300])
@pytest.mark.parametrize("inter,n_shared", [(192, 1), (80, 3), (208, 2), (64, 0), (256, 2)])
def test_every_token_at_odd_expert_sizes(inter, n_shared, T):
    check_tokens(make(S=n_shared, I=inter, seed=T), randn(T, D, seed=T + 9))


@pytest.mark.parametrize("inter", [192, 256])  # without the one call, and with it
def test_no_tokens(inter):
    layer = make(I=inter, S=1)
    assert (layer.few == 0) == (inter == 192)
    for ws in (None, torch.zeros(layer.workspace_bytes(0), dtype=torch.uint8, device=DEV)):
        y = layer(randn(0, D), ws)
        assert y.shape == (0, D) and y.dtype == torch.float32
