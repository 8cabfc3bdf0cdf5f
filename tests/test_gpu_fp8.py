"""8-bit rows, weights and products against their definitions in 64 bits."""
import pytest
import torch

from sparse_mixture_experts_03_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
FLOOR = 2.0 ** -100
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def nearest_e4m3(t):
    """The e4m3 value next to each fp64 value of at most 448, ties to even:
    steps of 2^(e - 3) from 2^-6 on, of 2^-9 below."""
    _, e = torch.frexp(t)
    step = torch.ldexp(torch.ones_like(t), (e - 4).clamp(min=-9))
    return torch.round(t / step) * step


def row_blocks(x):
    """(codes as fp64 values, scales fp64 [blocks, R]) of fp64 rows."""
    q, s = torch.empty_like(x), []
    for c in range(0, x.shape[1], 128):
        A = x[:, c:c + 128].abs().amax(1).clamp(min=FLOOR)
        q[:, c:c + 128] = nearest_e4m3(x[:, c:c + 128] * 448 / A[:, None])
        s.append(A / 448)
    return q, torch.stack(s)


def randn(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def scales_equal(got, want):
    # one fp32 rounding of the quotient A / 448 (and of a product with a weight)
    return bool(((got.double() - want).abs() <= 2.0 ** -24 * want).all())


# ---------------------------------------------------------------- rows

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,d", [(1, 16), (1, 2048), (7, 128), (8, 144), (9, 256), (65, 2064),
                                 (300, 1040), (1, 196608), (3, 6144), (64, 6160)])
def test_rows_are_exact(R, d, dt):
    x = randn(R, d, seed=R + d, dtype=torch.float32)
    x[:, ::5] *= 30
    x = x.to(DT[dt])
    q, s = moe.quantize_rows(x)
    want_q, want_s = row_blocks(x.double())
    assert torch.equal(q.double(), want_q)
    assert scales_equal(s, want_s)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_on_borders(dt):
    """Values half way between two codes, where a quotient that is a little off
    picks the wrong one: all code midpoints times each block maximum."""
    codes = torch.arange(127, device=DEV, dtype=torch.uint8).view(moe.E4M3).double()
    mid = (codes[1:] + codes[:-1]) / 2
    A = torch.tensor([448, 1, 1.5, 1.75, 3, 5.5, 7, 100, 2.0 ** -90 * 1.25, 2.0 ** 110 * 1.625],
                     device=DEV, dtype=torch.float64)
    x = torch.zeros(A.numel(), 256, device=DEV, dtype=torch.float64)
    x[:, :126] = mid * A[:, None] / 448
    x[:, 126] = A
    x[:, 128:254] = -mid * A[:, None] / 448
    x[:, 254] = -A
    x = x.to(DT[dt])  # some are now next to a midpoint instead of on it
    q, s = moe.quantize_rows(x)
    want_q, want_s = row_blocks(x.double())
    assert torch.equal(q.double(), want_q)
    assert scales_equal(s, want_s)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_of_extreme_values(dt):
    x = randn(8, 384, seed=3, dtype=torch.float32)
    x[0] = 0
    x[1] *= 2.0 ** -110                 # below the floor of the scale
    x[2] *= 1e-38
    x[3] = x[3].sign() * 3.38e38        # 448 x would overflow
    x[4, 0] = 3.3e38
    x[5, 200] = float("inf")
    x[6, 5] = float("nan")
    x[7, 383] = -float("inf")
    x = x.to(DT[dt])
    q, s = moe.quantize_rows(x)
    want_q, want_s = row_blocks(x.double())
    bad = torch.zeros(8, 384, dtype=torch.bool, device=DEV)
    bad[5, 128:256] = bad[6, :128] = bad[7, 256:] = True
    assert q.double()[bad].isnan().all()
    assert torch.equal(q.double()[~bad], want_q[~bad])
    bad_s = torch.zeros(3, 8, dtype=torch.bool, device=DEV)
    bad_s[1, 5] = bad_s[0, 6] = bad_s[2, 7] = True
    assert s[bad_s].isnan().all()
    assert scales_equal(s[~bad_s], want_s[~bad_s])


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("R,inter", [(1, 128), (13, 400), (130, 1536), (20, 6160)])
def test_swiglu_rows(R, inter, weighted):
    gu = randn(R, 2 * inter, seed=R, dtype=torch.float32) * 3
    gu[0, :inter] = -90.0                # silu underflows towards zero
    gu = gu.bfloat16()
    w = torch.rand(R, device=DEV) if weighted else None
    q, s = moe.swiglu_quantize_rows(gu, w)
    g, u = gu.double().split(inter, 1)
    h = g * torch.sigmoid(g) * u
    # h in fp32 is off by a few roundings and by the exponential's error, which
    # grows with |g|: 2^-22 (4 + |g|) of h covers ex2.approx (2 ulp), its
    # argument's rounding (|g| log2 e 2^-24) and the divide (2 ulp)
    slack = 2.0 ** -22 * (4 + g.abs())
    worst = float(slack.max())
    want_s = row_blocks(h)[1]
    f = w.double()[None] if weighted else 1.0
    assert bool(((s.double() - want_s * f).abs() <= (worst + 2.0 ** -22) * want_s * f).all())
    # a code is the nearest one to a quotient that is off by that much
    A = want_s.t().repeat_interleave(128, 1)[:, :inter]
    t = h / A
    _, e = torch.frexp(t)
    half = torch.ldexp(torch.ones_like(t), (e - 4).clamp(min=-9)) / 2
    assert bool(((q.double() - t).abs() <= half + 2 * worst * t.abs() + 2.0 ** -40).all())


# ---------------------------------------------------------------- weights

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(16, 16), (128, 128), (200, 144), (3, 129, 272), (2, 1000, 1040)])
def test_weights_are_exact(shape, dt):
    W = randn(*shape, seed=len(shape), dtype=DT[dt])
    W.view(-1, shape[-1])[0, 0] = 40.0
    q, s = moe.quantize_weight(W)
    W3 = W.double().view(-1, *shape[-2:])
    G, n, k = W3.shape
    want_q, want_s = torch.empty_like(W3), torch.empty_like(s, dtype=torch.float64).view(G, (n + 127) // 128, -1)
    for i in range(0, n, 128):
        for j in range(0, k, 128):
            part = W3[:, i:i + 128, j:j + 128]
            A = part.abs().amax((1, 2)).clamp(min=FLOOR)
            want_q[:, i:i + 128, j:j + 128] = nearest_e4m3(part * 448 / A[:, None, None])
            want_s[:, i // 128, j // 128] = A / 448
    assert torch.equal(q.double(), want_q.view(q.shape))
    assert scales_equal(s, want_s.view(s.shape))


def test_nothing_to_quantize():
    q, s = moe.quantize_rows(torch.empty(0, 256, device=DEV))
    assert q.shape == (0, 256) and s.shape == (2, 0)
    q, s = moe.quantize_weight(torch.empty(0, 5, 256, device=DEV))
    assert q.shape == (0, 5, 256) and s.shape == (0, 1, 2)


# ---------------------------------------------------------------- products

def operands(R, G, n, k, seed=0):
    a, sa = moe.quantize_rows(randn(R, k, seed=seed))
    b, sb = moe.quantize_weight(randn(G, n, k, seed=seed + 1))
    # scales as a checkpoint may have them: any positive numbers
    g = torch.Generator(device=DEV).manual_seed(seed + 2)
    return a, sa * (0.5 + torch.rand(sa.shape, generator=g, device=DEV)), b, sb


def product64(a, sa, b, sb, counts):
    """(y, sum of magnitudes) in fp64; NaN behind the last group."""
    A = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :a.shape[1]]
    n, k = b.shape[-2:]
    B = b.double() * sb.double().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]
    y = torch.full((a.shape[0], n), float("nan"), dtype=torch.float64, device=DEV)
    mag, r = y.clone(), 0
    for e, c in enumerate(counts):
        c = min(max(c, 0), a.shape[0] - r)
        y[r:r + c] = A[r:r + c] @ B[e].t()
        mag[r:r + c] = A[r:r + c].abs() @ B[e].abs().t()
        r += c
    return y, mag


def check_product(y, want, mag, k, fill=None):
    """Every addition of the k products and of the blocks' sums may lose one
    unit of the last of 24 bits (2^-23, the tensor core may truncate) of at
    most the sum of magnitudes; a block's scale and its product with the sum
    are three roundings more; y is rounded once."""
    out = 2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24
    tol = (k + (k + 127) // 128 + 8) * 2.0 ** -23 * mag + out * want.abs()
    done = ~want.isnan()
    assert bool(((y.double() - want).abs() <= tol)[done].all())
    if fill is not None:
        assert bool((y[~done] == fill).all())


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("R,n,k", [(1, 1, 16), (1, 2048, 1536), (3, 100, 144), (64, 257, 256),
                                   (128, 128, 128), (129, 320, 400), (500, 1000, 1040),
                                   (2000, 2050, 272), (5001, 2048, 400), (9000, 1001, 272),
                                   # several CTAs per tile
                                   (64, 2048, 6144), (5, 100, 4096), (200, 66, 2064),
                                   (1, 129, 16400), (128, 1000, 1104),
                                   # between the widths
                                   (64, 6200, 512), (1024, 1100, 800), (700, 300, 2064)])
def test_dense_product(R, n, k, out):
    a, sa, b, sb = operands(R, 1, n, k, seed=R + n + k)
    y = moe.matmul_fp8(a, sa, b[0], sb[0], out_dtype=DT[out])
    want, mag = product64(a, sa, b, sb, [R])
    check_product(y, want, mag, k)
    assert torch.equal(y, moe.matmul_fp8(a, sa, b, sb, out_dtype=DT[out]))  # bit for bit


@pytest.mark.parametrize("counts,n,k,R", [
    ([5, 0, 1, 130, 0], 96, 128, 136),           # empty groups, the last one too
    ([0, 0, 0], 64, 256, 10),                    # no rows at all
    ([127, 128, 129, 256, 257], 256, 160, 900),  # tile edges; rows behind the last group
    ([1] * 200, 72, 96, 200),                    # many groups of one row
    ([3, -4, 2], 40, 64, 5),                     # a negative count is an empty group
    ([700, 1, 33], 1300, 512, 734),
    # CTA pairs: 256-row tiles, some with rows of the first CTA only
    ([1000, 0, 300, 2000, 57, 1500], 2100, 144, 5000),
    ([256, 1, 128, 4000, 129, 700, 2], 2050, 272, 5216),
])
def test_grouped_product(counts, n, k, R):
    a, sa, b, sb = operands(R, len(counts), n, k, seed=R)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    for dt in (torch.bfloat16, torch.float32):
        y = torch.full((R, n), 7.0, dtype=dt, device=DEV)
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        moe.matmul_fp8(a, sa, b, sb, c, y=y, status_ws=ws)
        want, mag = product64(a, sa, b, sb, counts)
        check_product(y, want, mag, k, fill=7.0)
        assert moe.device_status(ws)[0] == moe.MOE_OK


def test_product_of_too_many_rows_is_cut_and_reported():
    R, counts = 100, [60, 60, 2 ** 31 - 1, 5]
    a, sa, b, sb = operands(R, 4, 64, 128)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    guard = torch.full((R + 50, 64), 3.0, device=DEV)
    moe.matmul_fp8(a, sa, b, sb, c, y=guard[:R], status_ws=ws)
    want, mag = product64(a, sa, b, sb, counts)
    check_product(guard[:R], want, mag, 128)
    assert bool((guard[R:] == 3.0).all())
    assert moe.device_status(ws)[0] == moe.MOE_ERR_DEVICE
    moe.clear_device_status(ws)
    assert moe.device_status(ws)[0] == moe.MOE_OK


def test_product_keeps_nan_and_large_scales_in_their_rows():
    a, sa, b, sb = operands(40, 1, 64, 256)
    sa[1, 3] = float("nan")
    sa[0, 7] = 1e30
    y = moe.matmul_fp8(a, sa, b[0], sb[0], out_dtype=torch.float32)
    assert y[3].isnan().all()
    keep = torch.arange(40, device=DEV) != 3
    want, mag = product64(a[keep], sa[:, keep], b, sb, [39])
    check_product(y[keep], want, mag, 256)


def test_product_on_a_side_stream_and_in_a_graph():
    R, n, k, counts = 300, 200, 384, [100, 0, 150]
    a, sa, b, sb = operands(R, 3, n, k, seed=9)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    y0 = moe.matmul_fp8(a, sa, b, sb, c, y=torch.zeros(R, n, dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y1 = torch.zeros_like(y0)
    s.wait_stream(torch.cuda.current_stream())
    moe.matmul_fp8(a, sa, b, sb, c, y=y1, stream=s)
    s.synchronize()
    assert torch.equal(y0, y1)
    x = randn(R, k, seed=9)
    g = torch.cuda.CUDAGraph()
    y2 = torch.zeros_like(y0)
    with torch.cuda.graph(g):
        q, sq = moe.quantize_rows(x)
        moe.matmul_fp8(q, sq, b, sb, c, y=y2)
    for seed in (9, 10):
        x.copy_(randn(R, k, seed=seed))
        c.copy_(torch.tensor([counts, [20, 250, 30]][seed - 9], dtype=torch.int32))
        y2.zero_()
        g.replay()
        want = torch.zeros_like(y0)
        moe.matmul_fp8(*moe.quantize_rows(x), b, sb, c, y=want)
        torch.cuda.synchronize()
        assert torch.equal(y2, want)
    del g


def test_refusals_on_the_gpu():
    a, sa, b, sb = operands(8, 2, 32, 128)
    c = torch.tensor([4, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        moe.matmul_fp8(randn(8, 128), sa, b, sb, c)
    with pytest.raises(ValueError):
        moe.matmul_fp8(a, sa.t().contiguous(), b, sb, c)        # scales lie [block][row]
    with pytest.raises(TypeError):
        moe.matmul_fp8(a, sa, b, sb, c.long())
    with pytest.raises(ValueError):
        moe.matmul_fp8(a, sa, b, sb, c[:1])
    with pytest.raises(moe.MoeError):
        moe.matmul_fp8(a, sa, b, sb)                            # two groups without counts
    with pytest.raises(ValueError):
        moe.matmul_fp8(a, sa, b, sb, c, status_ws=torch.zeros(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        moe.matmul_fp8(a, sa, b, sb, c, out_dtype=torch.float16)
    with pytest.raises(moe.MoeError):
        moe.quantize_rows(randn(4, 24))                         # d % 16
    with pytest.raises(ValueError):
        moe.quantize_rows(randn(4, 256)[:, :128])               # not contiguous
    base = torch.zeros(4 * 128 + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(moe.MoeError):
        moe.quantize_rows(base[4:4 + 512].view(4, 128))         # 8-byte aligned rows


def test_offsets_beyond_32_bits():
    """Rows and codes whose byte offsets pass 2^32, from the last rows."""
    R, d = 1_100_000, 2048  # 4.5 GB of bf16, 2.25 GB of codes
    x = torch.zeros(R, d, dtype=torch.bfloat16, device=DEV)
    x[-3:] = randn(3, d, seed=1)
    q, s = moe.quantize_rows(x)
    want_q, want_s = row_blocks(x[-3:].double())
    assert torch.equal(q[-3:].double(), want_q) and scales_equal(s[:, -3:], want_s)
    del x
    b, sb = moe.quantize_weight(randn(1, 2064, d, seed=2))  # y: 2.27e9 values
    y = moe.matmul_fp8(q, s, b[0], sb[0])
    want, mag = product64(q[-3:], s[:, -3:].contiguous(), b, sb, [3])
    check_product(y[-3:], want, mag, d)
    assert not y[:128].any()


# ---------------------------------------------------------------- the layer on 8-bit weights

def fp8_layer(E=16, k=4, G=4, TG=2, d=512, I=256, S=2, seed=0, **kw):
    from sparse_mixture_experts_03_b200.fp8 import Fp8MoE
    Wr = randn(E, d, seed=seed).mul_(d ** -0.5)
    gu = randn(E, 2 * I, d, seed=seed + 1).mul_(d ** -0.5)
    dn = randn(E, d, I, seed=seed + 2).mul_(I ** -0.5)
    sh = None
    if S:
        sh = torch.cat([randn(2 * S * I * d, seed=seed + 3).mul_(d ** -0.5),
                        randn(S * I * d, seed=seed + 4).mul_(I ** -0.5)])
    return Fp8MoE(Wr, gu, dn, sh, k, G, TG, I, S, **kw)


def layer64(layer, x, idx, w):
    """The layer in fp64 on its 8-bit weights, for a given routing."""
    wide = lambda q, s: q.double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)
    I, SI = layer.inter, layer.n_shared * layer.inter
    ffn = lambda gu, dn, F, v: (torch.nn.functional.silu(v @ gu[:F].t()) * (v @ gu[F:].t())) @ dn.t()
    X = x.double()
    y = torch.zeros_like(X)
    if SI:
        y += ffn(wide(*layer.shared_gate_up), wide(*layer.shared_down), SI, X)
    gu, dn = wide(layer.W_gate_up, layer.s_gate_up), wide(layer.W_down, layer.s_down)
    for e in range(layer.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            y[t] += w[t, j, None].double() * ffn(gu[e], dn[e], I, X[t])
    return y


@pytest.mark.parametrize("T,S,out", [(1, 2, torch.float32), (8, 2, torch.bfloat16),
                                     (9, 2, torch.float32), (300, 2, torch.bfloat16),
                                     (1100, 0, torch.float32), (33, 1, torch.float32)])
def test_layer_on_8bit_weights(T, S, out):
    layer = fp8_layer(S=S, out_dtype=out, seed=T)
    x = randn(T, 512, seed=T + 9)
    y = layer(x)
    idx, w = moe.route(x, layer.W_router, layer.k, layer.n_group, layer.topk_group)
    ref = layer64(layer, x, idx.long(), w)
    assert y.dtype == out and y.shape == (T, 512)
    # Up to 8 tokens only h and y are rounded, to bf16.  Above, rows are rounded
    # to e4m3: an error spread evenly over half a step either way is at most r =
    # 2^-4 / sqrt(3) of the norm; x's reaches h through gate (|silu'| <= 1.1) and
    # up, 2.1 r, and h has its own, r.
    tol = 5e-3 if T <= layer.few else 3.1 * 2.0 ** -4 / 3 ** 0.5
    assert float((y.double() - ref).norm() / ref.norm()) <= tol
    assert torch.equal(y, layer(x))


def test_layer_of_no_tokens_and_in_a_graph():
    layer = fp8_layer(seed=3)
    assert layer(randn(0, 512)).shape == (0, 512)
    for T in (5, 40):
        x = randn(T, 512, seed=T)
        g = torch.cuda.CUDAGraph()
        layer(x)  # the libraries' first calls are not captured
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            y = layer(x)
        for seed in (1, 2):
            x.copy_(randn(T, 512, seed=seed))
            g.replay()
            want = layer(x)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
        del g
