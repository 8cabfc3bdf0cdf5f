"""Refusals of the 8-bit entry points and of the layer for a few tokens (no
GPU: every one of them comes before anything is queued)."""
import ctypes

import pytest
import torch

from sparse_mixture_experts_03_b200 import moe

BAD, UNSUP, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK


def test_rows_and_weights_refuse_bad_arguments():
    L = moe.lib()
    rows = lambda R, d, dt: L.moe_quantize_rows(None, R, d, dt, None, None, None)
    assert rows(4, 128, 7) == BAD
    assert rows(-1, 128, moe.MOE_BF16) == BAD
    assert rows(4, 0, moe.MOE_BF16) == BAD
    assert rows(4, 120, moe.MOE_BF16) == UNSUP       # d % 16
    assert rows(4, 196608 + 16, moe.MOE_BF16) == UNSUP
    assert rows(4, 128, moe.MOE_BF16) == BAD         # no pointers
    assert rows(0, 128, moe.MOE_F32) == OK
    sw = lambda R, I, dt: L.moe_swiglu_quantize_rows(None, None, R, I, dt, None, None, None)
    assert sw(4, 128, moe.MOE_F32) == UNSUP          # bf16 rows only
    assert sw(4, 24, moe.MOE_BF16) == UNSUP
    assert sw(4, 128, moe.MOE_BF16) == BAD
    assert sw(0, 128, moe.MOE_BF16) == OK
    wt = lambda G, n, k, dt: L.moe_quantize_weight(None, G, n, k, dt, None, None, None)
    assert wt(1, 8, 24, moe.MOE_BF16) == UNSUP
    assert wt(1, 0, 16, moe.MOE_BF16) == BAD
    assert wt(-1, 8, 16, moe.MOE_BF16) == BAD
    assert wt(2 ** 30, 2 ** 30, 16, moe.MOE_BF16) == UNSUP  # more blocks than a grid has
    assert wt(1, 8, 16, 5) == BAD
    assert wt(1, 8, 16, moe.MOE_F32) == BAD
    assert wt(0, 8, 16, moe.MOE_F32) == OK


def test_product_refuses_bad_arguments():
    f = lambda R=4, G=1, n=64, k=128, dt=moe.MOE_BF16, counts=None: moe.lib().moe_matmul_fp8(
        None, None, None, None, counts, R, G, n, k, dt, None, None, None)
    assert f(R=-1) == BAD and f(n=0) == BAD and f(k=0) == BAD
    assert f(G=0) == BAD and f(G=257, counts=ctypes.c_void_p(256)) == BAD
    assert f(dt=3) == BAD
    assert f(G=2) == BAD                              # groups without counts
    assert f(k=136) == UNSUP                          # k % 16
    assert f(R=2 ** 31 - 1, n=2 ** 31 - 1) == UNSUP   # tiles beyond 32 bits
    assert f() == BAD                                 # no pointers
    assert f(R=0) == OK


def _few(T=4, d=256, E=8, k=2, G=1, TG=1, I=128, S=0, dt=moe.MOE_BF16, out=moe.MOE_F32, gate=0,
         W_sh=None, s=(None, None, None), ws=None, wsb=0):
    return moe.lib().moe_forward_few(None, None, None, None, W_sh, *s, T, d, E, k, G, TG, I, S, dt,
                                     out, gate, None, None, None, None, ws, wsb, None)


def test_few_refuses_bad_arguments():
    p = ctypes.c_void_p(256)
    assert _few(dt=moe.MOE_F32) == UNSUP and _few(dt=9) == BAD
    assert _few(T=17) == UNSUP and _few(T=-1) == BAD
    assert _few(d=128) == UNSUP and _few(I=192) == UNSUP
    assert _few(S=65, W_sh=p) == UNSUP
    assert _few(E=300) == BAD and _few(k=9) == BAD and _few(E=8, G=3) == BAD
    assert _few(k=5, E=8, G=2, TG=1) == BAD
    assert _few(out=4) == BAD
    assert _few(S=1) == BAD and _few(W_sh=p) == BAD   # shared count and weights disagree
    assert _few(s=(p, None, None)) == BAD             # scales of some weights only
    assert _few(S=1, W_sh=p, s=(p, p, None)) == BAD
    assert _few(s=(p, p, p)) == BAD
    assert _few() == moe.MOE_ERR_WORKSPACE
    assert _few(ws=p, wsb=64) == moe.MOE_ERR_WORKSPACE
    assert _few(gate=2, ws=p, wsb=1 << 30) == BAD
    assert _few(T=0, ws=p, wsb=1 << 30) == OK
    assert _few(ws=p, wsb=1 << 30) == BAD             # no pointers


def test_few_sizes():
    assert moe.few_max_tokens(2048, 64, 6, 1536, 4) == 16
    assert moe.few_max_tokens(7168, 64, 6, 1536, 4) == 8    # operand B of 16 tokens does not fit
    assert moe.few_max_tokens(32768, 64, 6, 1536, 4) == 0
    assert moe.few_max_tokens(2048, 64, 6, 1500, 4) == 0
    n = moe.few_workspace_bytes(16, 2048, 64, 6, 1536, 4)
    # h of 68 entries and the slots
    assert n >= 68 * 16 * 1536 * 2 + 16 * 10 * 2048 * 4
    with pytest.raises(moe.MoeError):
        moe.few_workspace_bytes(17, 2048, 64, 6, 1536, 4)


def test_tensors_are_checked_before_their_pointers():
    bf = torch.zeros(4, 256, dtype=torch.bfloat16)
    for call in (lambda: moe.quantize_rows(bf), lambda: moe.quantize_weight(bf),
                 lambda: moe.swiglu_quantize_rows(bf)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        moe.quantize_rows(bf.half())
    with pytest.raises(ValueError):
        moe.quantize_rows(bf[0])
    with pytest.raises(ValueError):
        moe.swiglu_quantize_rows(bf[:, :255])
    q = torch.zeros(4, 256, dtype=moe.E4M3)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.matmul_fp8(q, q, q, q)
    want = moe._want  # noqa: SLF001
    with pytest.raises(ValueError):
        want("t", bf, (4, 255), torch.bfloat16, bf)
    with pytest.raises(TypeError):
        want("t", bf, (4, 256), torch.float32, bf)
    want("t", bf, (4, 256), torch.bfloat16, bf)
