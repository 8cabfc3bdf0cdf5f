"""The layer for a few tokens (moe.forward_few) against the fp64 oracle, and
against formulas in fp64 for the rounding bound."""
import numpy as np
import pytest
import torch

import oracle
from sparse_mixture_experts_03_b200 import moe
from tests import parity

pytestmark = pytest.mark.gpu
DEV = "cuda"

# T, d, E, k, n_group, topk_group, inter, n_shared
SHAPES = [
    (1, 256, 8, 2, 1, 1, 128, 0),
    (3, 256, 16, 4, 4, 2, 256, 2),
    (8, 512, 64, 6, 8, 4, 384, 4),
    (9, 256, 64, 8, 8, 4, 128, 1),
    (16, 768, 32, 6, 4, 3, 640, 3),
    (16, 256, 4, 4, 1, 1, 1152, 0),      # every expert takes every token
    (5, 1280, 256, 8, 32, 8, 128, 1),    # many experts, an odd number of row pieces
    (2, 2048, 64, 6, 8, 4, 1536, 4),     # the workloads' layer
    (3, 4096, 4, 2, 1, 1, 2304, 1),      # rows longer than one pass makes operand B of
    (11, 2560, 6, 3, 3, 2, 2688, 0),
    (8, 7168, 2, 1, 1, 1, 128, 0),       # the least room for the ring
]


class Layer:
    def __init__(self, shape, fp8, seed=0):
        self.T, self.d, self.E, self.k, self.G, self.TG, self.I, self.S = shape
        T, d, E, I, S = self.T, self.d, self.E, self.I, self.S
        g = torch.Generator(device=DEV).manual_seed(seed)
        rn = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device=DEV) * scale).bfloat16()
        self.x, self.Wr = rn(T, d), rn(E, d, scale=d ** -0.5)
        gu, dn = rn(E, 2 * I, d, scale=d ** -0.5), rn(E, d, I, scale=I ** -0.5)
        sgu, sdn = rn(2 * S * I, d, scale=d ** -0.5), rn(d, S * I, scale=I ** -0.5)
        self.scales = None
        wide = [t.double() for t in (gu, dn, sgu, sdn)]
        if fp8:
            (gu, a), (dn, b) = moe.quantize_weight(gu), moe.quantize_weight(dn)
            wide[:2] = [self.values(gu, a), self.values(dn, b)]
            c = None
            if S:
                (sgu, c0), (sdn, c1) = moe.quantize_weight(sgu), moe.quantize_weight(sdn)
                wide[2:] = [self.values(sgu, c0), self.values(sdn, c1)]
                c = torch.cat([c0.flatten(), c1.flatten()])
            self.scales = (a, b, c)
        self.gu, self.dn = gu, dn
        self.sh = None
        if S:
            u8 = torch.uint8
            self.sh = torch.cat([sgu.flatten().view(u8), sdn.flatten().view(u8)]).view(sgu.dtype)
        self.wide = wide

    @staticmethod
    def values(q, s):
        return q.double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)

    def run(self, **kw):
        idx = torch.empty(self.T, self.k, dtype=torch.int32, device=DEV)
        w = torch.empty(self.T, self.k, dtype=torch.float32, device=DEV)
        kw.setdefault("scales", self.scales)
        y = moe.forward_few(self.x, self.Wr, self.gu, self.dn, self.sh, self.k, self.G, self.TG,
                            self.I, self.S, topk_idx=idx, topk_w=w, **kw)
        return y, idx, w

    def oracle(self, forced_idx=None, **kw):
        c = lambda t: t.cpu().contiguous()
        sh = torch.cat([self.wide[2].flatten(), self.wide[3].flatten()]) if self.S else None
        return oracle.forward(c(self.x.double()), c(self.Wr.double()), c(self.wide[0]),
                              c(self.wide[1]), None if sh is None else c(sh), self.k, self.G,
                              self.TG, self.I, self.S, forced_idx=forced_idx, **kw)

    def bound(self, idx, w):
        """How far y may be off in fp64 terms, worst case: the sums of the
        pre-activations (fp32, at most d + 16 roundings of the sum of
        magnitudes), silu (a few ulp), h rounded to bf16 (2^-8), the down sums
        (fp32) and the gate weight (2e-5 absolute covers a near-equal score)."""
        d, I, S = self.d, self.I, self.S
        eps = 2.0 ** -23  # the tensor core may truncate
        out = torch.zeros(self.T, d, dtype=torch.float64, device=DEV)
        for t in range(self.T):
            x = self.x[t].double()
            parts = [(self.wide[0][e], self.wide[1][e], float(p), I)
                     for e, p in zip(idx[t].tolist(), w[t].tolist())]
            if S:
                parts.append((self.wide[2], self.wide[3], 1.0, S * I))
            for gu, dn, p, F in parts:
                pre, mag = gu @ x, gu.abs() @ x.abs()
                dp = (d + 16) * eps * mag
                g, u = pre[:F], pre[F:]
                sig = torch.sigmoid(g)
                h = g * sig * u
                dh = 1.1 * dp[:F] * (u.abs() + dp[F:]) + (g * sig).abs() * dp[F:] + \
                    (8 + g.abs()) * 2.0 ** -23 * h.abs()
                dh = dh + 2.0 ** -8 * (h.abs() + dh)
                m = dn.abs() @ h.abs()
                out[t] += p * (dn.abs() @ dh + (I + 16) * eps * m) + 2e-5 * (dn @ h).abs()
                out[t] += (S + self.k + 2) * eps * p * m
        return out


def check(layer, y, idx, w, gate="sigmoid", bias=None):
    score = {"score_func": gate, "bias": None if bias is None else bias.cpu().numpy()}
    ref = oracle.route(layer.x.cpu(), layer.Wr.cpu(), layer.k, layer.G, layer.TG, **score)
    rep = parity.check_routing(idx.cpu().numpy(), w.cpu().numpy(), ref, layer.G, layer.TG, layer.E)
    forced = ref.idx.copy()
    for t in rep.mismatched_tokens:
        forced[t] = idx[t].cpu().numpy()
    y_ref, ri, rw = layer.oracle(forced_idx=forced, **score)
    y_ref = torch.from_numpy(y_ref).to(DEV)
    tol = layer.bound(torch.from_numpy(ri), torch.from_numpy(rw))
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (y_ref.abs() + tol)
    diff = (y.double() - y_ref).abs()
    assert bool((diff <= tol).all())
    # the rounding of h alone is about 2^-9 of y (0.2%); of a bf16 y as much again
    assert float(diff.norm() / y_ref.norm()) <= 5e-3


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_few_tokens(shape, fp8, out):
    layer = Layer(shape, fp8, seed=sum(shape))
    ws = torch.full((moe.few_workspace_bytes(*(shape[i] for i in (0, 1, 2, 3, 6, 7))),), 0xAB,
                    dtype=torch.uint8, device=DEV)  # whatever the workspace held before
    y, idx, w = layer.run(out_dtype=out, workspace=ws)
    assert moe.device_status(ws)[0] == moe.MOE_OK
    check(layer, y, idx, w)
    y2, idx2, w2 = layer.run(out_dtype=out, workspace=ws)
    assert torch.equal(y, y2) and torch.equal(idx, idx2) and torch.equal(w, w2)


@pytest.mark.parametrize("gate,biased", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_gates(gate, biased):
    layer = Layer((7, 256, 32, 4, 4, 2, 128, 1), False, seed=5)
    bias = 0.3 * torch.randn(32, device=DEV) if biased else None
    y, idx, w = layer.run(gate=gate, expert_bias=bias)
    check(layer, y, idx, w, gate, bias)


def test_equals_the_layer_for_any_number_of_tokens():
    """The same routing as moe.forward, and outputs that differ by its extra
    rounding of the experts' outputs only (both are within 5e-3 of fp64)."""
    layer = Layer((12, 512, 64, 6, 8, 4, 256, 2), False, seed=8)
    y, idx, w = layer.run()
    idx2, w2 = torch.empty_like(idx), torch.empty_like(w)
    y2 = moe.forward(layer.x, layer.Wr, layer.gu, layer.dn, layer.sh, 6, 8, 4, 256, 2,
                     topk_idx=idx2, topk_w=w2)
    assert torch.equal(idx, idx2)
    assert float((y - y2).norm() / y2.norm()) <= 1e-2


def test_no_tokens_and_all_sizes_of_batch():
    layer = Layer((16, 256, 16, 4, 4, 2, 128, 1), False, seed=2)
    full, idx, _ = layer.run()
    for T in (0, 1, 7, 8, 9, 15):
        y = moe.forward_few(layer.x[:T], layer.Wr, layer.gu, layer.dn, layer.sh, 4, 4, 2, 128, 1)
        # a token's sums do not depend on the others of the batch
        assert y.shape == (T, 256) and torch.equal(y, full[:T])


def test_nan_in_one_token_stays_there():
    layer = Layer((6, 256, 16, 4, 4, 2, 128, 1), False, seed=4)
    full, _, _ = layer.run()
    layer.x[2, 17] = float("nan")
    y, idx, _ = layer.run()
    keep = torch.arange(6, device=DEV) != 2
    assert y[2].isnan().all() and torch.equal(y[keep], full[keep])
    assert bool(((idx >= 0) & (idx < 16)).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_graph_and_two_streams(fp8):
    shape = (4, 512, 32, 6, 4, 2, 256, 2)
    a, b = Layer(shape, fp8, seed=1), Layer(shape, fp8, seed=2)
    want = [l.run()[0] for l in (a, b)]
    torch.cuda.synchronize()
    # two calls at once, a workspace each
    streams = [torch.cuda.Stream() for _ in range(2)]
    sizes = [shape[i] for i in (0, 1, 2, 3, 6, 7)]
    ws = [torch.empty(moe.few_workspace_bytes(*sizes), dtype=torch.uint8, device=DEV)
          for _ in range(2)]
    ys = [torch.empty_like(want[0]) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for l, s, w, y in zip((a, b), streams, ws, ys):
            l.run(stream=s, workspace=w, y=y)
    torch.cuda.synchronize()
    assert all(moe.device_status(w)[0] == moe.MOE_OK for w in ws)
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])
    # captured and replayed, with new inputs
    y, idx, w = torch.empty_like(want[0]), torch.empty(4, 6, dtype=torch.int32, device=DEV), None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.forward_few(a.x, a.Wr, a.gu, a.dn, a.sh, 6, 4, 2, 256, 2, scales=a.scales, y=y,
                        topk_idx=idx, workspace=ws[0])
    for x in (a.x.clone(), b.x.clone(), a.x.clone()):
        a.x.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, a.run()[0])
    del g


def test_side_stream_without_a_workspace():
    """What the call allocates for work on another stream is not reused before
    that work is done."""
    layer = Layer((4, 512, 32, 6, 4, 2, 256, 2), False, seed=1)
    want = layer.run()[0]
    s = torch.cuda.Stream()
    n = moe.few_workspace_bytes(4, 512, 32, 6, 256, 2)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s):
            torch.cuda._sleep(1000000)  # the call starts later than what follows here
        y = layer.run(stream=s)[0]
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2)]
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del junk


def test_refusals_on_the_gpu():
    layer = Layer((4, 256, 16, 4, 4, 2, 128, 1), False)
    with pytest.raises(TypeError):
        layer.run(scales=(layer.Wr.float(), layer.Wr.float(), None))  # 16-bit weights, scales
    with pytest.raises(ValueError):
        layer.run(y=torch.empty(4, 255, device=DEV))
    with pytest.raises(ValueError):
        moe.forward_few(layer.x.cpu(), layer.Wr, layer.gu, layer.dn, layer.sh, 4, 4, 2, 128, 1)
    with pytest.raises(ValueError):
        moe.forward_few(layer.x[:, ::2], layer.Wr, layer.gu, layer.dn, layer.sh, 4, 4, 2, 128, 1)
    with pytest.raises(moe.MoeError):
        layer.run(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    x17 = torch.zeros(17, 256, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(moe.MoeError):
        moe.forward_few(x17, layer.Wr, layer.gu, layer.dn, layer.sh, 4, 4, 2, 128, 1)
