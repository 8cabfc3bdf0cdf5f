"""What the layer on 8-bit weights refuses (no GPU: the library's calls are
replaced by ones that must not be reached, or by ones that make nothing)."""
import pytest
import torch

from sparse_mixture_experts_03_b200 import fp8, moe

E, D, I, S, K = 8, 256, 128, 2, 2
BF, F32 = torch.bfloat16, torch.float32


def weights(**kw):
    w = dict(W_router=torch.zeros(E, D, dtype=BF), W_gate_up=torch.zeros(E, 2 * I, D, dtype=BF),
             W_down=torch.zeros(E, D, I, dtype=BF), W_shared=torch.zeros(3 * S * I * D, dtype=BF),
             k=K, n_group=1, topk_group=1, inter=I, n_shared=S)
    w.update(kw)
    return w


def reached(*args, **kw):
    raise AssertionError("a call of the library was reached")


@pytest.fixture
def no_library(monkeypatch):
    for name in ("quantize_rows", "swiglu_quantize_rows", "matmul_fp8", "forward_few", "dispatch",
                 "combine"):
        monkeypatch.setattr(moe, name, reached)


@pytest.fixture
def quantised(no_library, monkeypatch):
    """Weights are taken, nothing is computed."""
    def quantize_weight(W, q=None, scales=None, **kw):
        n, k = W.shape[-2:]
        shape = (*W.shape[:-2], -(-n // 128), -(-k // 128))
        return (torch.zeros(W.shape, dtype=moe.E4M3) if q is None else q,
                torch.zeros(shape) if scales is None else scales)
    monkeypatch.setattr(moe, "quantize_weight", quantize_weight)


@pytest.mark.parametrize("bad,error", [
    (dict(W_router=torch.zeros(E, D)), TypeError),                      # a router in fp32
    (dict(W_router=torch.zeros(E, D).half()), TypeError),
    (dict(W_router=torch.zeros(E * D, dtype=BF)), ValueError),
    (dict(W_router=torch.zeros(D, E, dtype=BF).t()), ValueError),       # not contiguous
    (dict(W_router=torch.zeros(E + 1, D, dtype=BF)), ValueError),       # more experts than weights
    (dict(expert_bias=torch.zeros(E, dtype=BF)), TypeError),
    (dict(expert_bias=torch.zeros(E - 1)), ValueError),
    (dict(expert_bias=torch.zeros(2 * E)[::2]), ValueError),
    (dict(W_gate_up=torch.zeros(E, I, D, dtype=BF)), ValueError),
    (dict(W_gate_up=torch.zeros(E, 2 * I, 2 * D, dtype=BF)), ValueError),
    (dict(W_gate_up=torch.zeros(E, 2 * I, D, dtype=torch.float16)), TypeError),
    (dict(W_down=torch.zeros(E, I, D, dtype=BF)), ValueError),
    (dict(W_down=torch.zeros(E, D, I, dtype=torch.float64)), TypeError),
    (dict(W_shared=torch.zeros(3 * S * I * D + 128, dtype=BF)), ValueError),
    (dict(W_shared=torch.zeros(3 * S * I * D, dtype=torch.float16)), TypeError),
    (dict(W_shared=None), ValueError),
    (dict(n_shared=0), ValueError),
    (dict(W_router=torch.zeros(E, 128, dtype=BF), W_gate_up=torch.zeros(E, 2 * I, 128, dtype=BF),
          W_down=torch.zeros(E, 128, I, dtype=BF), W_shared=torch.zeros(3 * S * I * 128, dtype=BF)),
     ValueError),                                                       # d is no multiple of 256
    (dict(W_gate_up=torch.zeros(E, 2 * I, D, dtype=BF, device="meta")), ValueError),
])
def test_weights_are_checked(quantised, bad, error):
    with pytest.raises(error):
        fp8.Fp8MoE(**weights(**bad))


@pytest.mark.parametrize("kw", [dict(), dict(W_down=torch.zeros(E, D, I), expert_bias=torch.zeros(E)),
                                dict(W_shared=None, n_shared=0),
                                dict(W_shared=torch.zeros(3 * S * I, D, dtype=BF))])
def test_weights_that_fit_are_taken(quantised, kw):
    layer = fp8.Fp8MoE(**weights(**kw))
    assert (layer.E, layer.d) == (E, D)


@pytest.mark.parametrize("T", [4, 40])  # the one call, and the steps
@pytest.mark.parametrize("make,error", [
    (lambda T: torch.zeros(T, D), TypeError),                  # fp32 tokens
    (lambda T: torch.zeros(T, D).half(), TypeError),
    (lambda T: torch.zeros(T, D + 256, dtype=BF), ValueError),  # wider than the router's rows
    (lambda T: torch.zeros(T, D - 16, dtype=BF), ValueError),
    (lambda T: torch.zeros(T * D, dtype=BF), ValueError),
    (lambda T: torch.zeros(1, T, D, dtype=BF), ValueError),
    (lambda T: torch.zeros(T, D, dtype=BF, device="meta"), ValueError),
    (lambda T: torch.zeros(T, D, dtype=BF), ValueError),       # not on a CUDA device
])
def test_tokens_are_checked_before_a_path_is_chosen(quantised, make, error, T):
    layer = fp8.Fp8MoE(**weights())
    with pytest.raises(error):
        layer(make(T))


def test_every_step_is_given_the_workspace(quantised, monkeypatch):
    """Dispatch first, which clears the status words; then the steps that set them."""
    seen = []

    def take(name, key, out):
        def call(*args, **kw):
            seen.append((name, kw.get(key)))
            return out
        monkeypatch.setattr(moe, name, call)
    t = torch.zeros(1)
    take("dispatch", "workspace", moe.Dispatched(t, t, t, t, t, t))
    take("matmul_fp8", "status_ws", t)
    take("combine", "status_ws", t)
    take("forward_few", "workspace", t)
    for name in ("quantize_rows", "swiglu_quantize_rows"):
        monkeypatch.setattr(moe, name, lambda *a, **kw: (t, t))
    monkeypatch.setattr(moe, "_on_current", lambda *a: (0, 0))
    layer = fp8.Fp8MoE(**weights())
    ws = torch.zeros(layer.workspace_bytes(40), dtype=torch.uint8)
    layer(torch.zeros(40, D, dtype=BF), ws)
    assert [n for n, _ in seen] == ["dispatch"] + 4 * ["matmul_fp8"] + ["combine"]
    assert all(w is ws for _, w in seen)
    seen.clear()
    layer(torch.zeros(4, D, dtype=BF), workspace=ws)
    assert seen == [("forward_few", ws)]
    for bad in (ws.int(), ws[::2], ws.to("meta")):
        with pytest.raises((TypeError, ValueError)):
            layer(torch.zeros(40, D, dtype=BF), bad)


@pytest.mark.parametrize("inter", [I, 192])  # with the one call, and without
def test_workspace_of_a_batch_holds_smaller_ones(quantised, inter):
    w = weights(W_gate_up=torch.zeros(E, 2 * inter, D, dtype=BF), inter=inter,
                W_down=torch.zeros(E, D, inter, dtype=BF),
                W_shared=torch.zeros(3 * S * inter * D, dtype=BF))
    layer = fp8.Fp8MoE(**w)
    sizes = [layer.workspace_bytes(T) for T in range(200)]
    assert sizes == sorted(sizes) and sizes[0] >= 256
    for T in range(1, 200):
        need = (moe.few_workspace_bytes(T, D, E, K, inter, S) if T <= layer.few
                else moe.lib().moe_dispatch_workspace_bytes(T, E, K))
        assert sizes[T] >= need


@pytest.mark.parametrize("inter,n_shared", [(192, 1), (16, 1), (80, 3), (48, 2), (128, 1)])
def test_shared_experts_of_any_size_that_routed_ones_may_have(quantised, inter, n_shared):
    SI = n_shared * inter
    layer = fp8.Fp8MoE(**weights(inter=inter, n_shared=n_shared,
                                 W_gate_up=torch.zeros(E, 2 * inter, D, dtype=BF),
                                 W_down=torch.zeros(E, D, inter, dtype=BF),
                                 W_shared=torch.zeros(3 * SI * D, dtype=BF)))
    up, s_up = layer.shared_gate_up
    down, s_down = layer.shared_down
    assert up.shape == (2 * SI, D) and s_up.shape == (-(-2 * SI // 128), D // 128)
    assert down.shape == (D, SI) and s_down.shape == (D // 128, -(-SI // 128))
    assert up.data_ptr() == layer.W_shared.data_ptr()
    assert s_up.data_ptr() == layer.s_shared.data_ptr()
    assert s_down.data_ptr() == s_up.data_ptr() + 4 * s_up.numel()


@pytest.mark.parametrize("inter", [I, 192])  # with the one call, and without
@pytest.mark.parametrize("out", [F32, BF])
def test_no_tokens(quantised, monkeypatch, inter, out):
    monkeypatch.setattr(moe, "_on_current", lambda *a: (0, 0))
    layer = fp8.Fp8MoE(**weights(inter=inter, W_gate_up=torch.zeros(E, 2 * inter, D, dtype=BF),
                                 W_down=torch.zeros(E, D, inter, dtype=BF), out_dtype=out,
                                 W_shared=torch.zeros(3 * S * inter * D, dtype=BF)))
    y = layer(torch.zeros(0, D, dtype=BF))
    assert y.shape == (0, D) and y.dtype == out
