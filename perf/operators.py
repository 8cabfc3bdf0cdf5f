"""Workloads of the layer's 8-bit operators and of its form for a few tokens.

Four operators: 8-bit rows (one scale per 128 columns of a row, plain or of a
SwiGLU), 8-bit weights (one scale per 128 x 128 block), the 8-bit product over
expert groups, and the whole layer for a few tokens.  `run` computes each in
plain torch, or with `own` through the package's entry points.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
FLOOR = 2.0 ** -100  # blocks of smaller values are scaled as if their largest were this
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# The layer of the repository's workloads: d 2048, 64 experts of 1536, 6 chosen, 8 groups of
# which 4 are kept, 4 shared experts.
LAYER = {"d": 2048, "experts": 64, "k": 6, "groups": 8, "kept": 4, "inter": 1536, "shared": 4}


def listed():
    return [
        # one token's hidden state on its way to a product: latency
        {"name": "rows_one_token", "op": "rows", "rows": 1, "d": 2048, "dtype": "bf16"},
        # the dispatched rows of a 4096-token prefill (6 per token)
        {"name": "rows_prefill", "op": "rows", "rows": 24576, "d": 2048, "dtype": "bf16"},
        # the expert hidden states of a 64-token decode step, gate weights folded in
        {"name": "swiglu_decode", "op": "swiglu", "rows": 384, "inter": 1536, "weighted": True},
        # the same behind a prefill of an odd length
        {"name": "swiglu_prefill", "op": "swiglu", "rows": 24581, "inter": 1536, "weighted": False},
        # a layer's down projections, once when a checkpoint is loaded
        {"name": "weight_experts", "op": "weight", "experts": 64, "n": 2048, "k": 1536, "dtype": "bf16"},
        # one fp32 master weight with ragged edges
        {"name": "weight_ragged", "op": "weight", "experts": 1, "n": 1000, "k": 1040, "dtype": "f32"},
        # the shared experts' down projection of a decode step: few rows, long reduction
        {"name": "product_shared_decode", "op": "product", "rows": 64, "experts": 1, "n": 2048, "k": 6144, "out": "bf16", "seg": "whole"},
        # the down projections of a 64-token decode step: about 6 rows each, some experts idle
        {"name": "product_decode", "op": "product", "rows": 384, "experts": 64, "n": 2048, "k": 1536, "out": "bf16", "seg": "even"},
        # the down projections of a prefill whose load is uneven
        {"name": "product_prefill", "op": "product", "rows": 24576, "experts": 64, "n": 2048, "k": 1536, "out": "bf16", "seg": "uneven"},
        # interactive decoding: one sequence
        {"name": "few_one_token", "op": "few", "tokens": 1, "weights": "bf16", **LAYER},
        # a small batch on 8-bit weights
        {"name": "few_five_tokens_fp8", "op": "few", "tokens": 5, "weights": "fp8", **LAYER},
        # the largest batch of the form: most experts touched
        {"name": "few_sixteen_tokens", "op": "few", "tokens": 16, "weights": "bf16", **LAYER},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "swiglu", "weight", "product", "product", "few", "few"])
    if op == "rows":
        return {"op": op, "rows": _log(rng, 1, 20000), "d": 16 * _log(rng, 4, 140), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "swiglu":
        return {"op": op, "rows": _log(rng, 1, 20000), "inter": 16 * _log(rng, 8, 100), "weighted": rng.random() < 0.5}
    if op == "weight":
        return {"op": op, "experts": _log(rng, 1, 32), "n": _log(rng, 64, 2100), "k": 16 * _log(rng, 4, 128), "dtype": rng.choice(["bf16", "f32"])}
    if op == "product":
        experts = rng.choice([1, 1, 8, 16, 40, 64])
        seg = "whole" if experts == 1 else rng.choice(["even", "uneven"])
        return {"op": op, "rows": _log(rng, 1, 16000), "experts": experts, "n": _log(rng, 64, 2048), "k": 16 * _log(rng, 4, 96),
                "out": rng.choice(["bf16", "bf16", "f32"]), "seg": seg}
    groups, per = rng.choice([(1, 8), (4, 4), (8, 4), (8, 8)])
    kept = rng.randint(max(1, groups // 2), groups)
    return {"op": op, "tokens": rng.randint(1, 16), "weights": rng.choice(["bf16", "fp8"]), "d": 256 * rng.randint(1, 8), "experts": groups * per,
            "k": rng.randint(1, min(8, kept * per)), "groups": groups, "kept": kept, "inter": 128 * rng.randint(1, 12), "shared": rng.choice([0, 1, 2, 4])}


# ---------------------------------------------------------------- inputs

def _blocks(n):
    return -(-n // 128)


def _pad(t, dim):
    """t with zeros behind it up to whole blocks of 128 along dim."""
    extra = -t.shape[dim] % 128
    if not extra:
        return t
    shape = list(t.shape)
    shape[dim] = extra
    return torch.cat([t, t.new_zeros(shape)], dim)


def _weight_blocks(W):
    """[G, n, k] as (e4m3 codes, fp32 scales per 128 x 128 block)."""
    G, n, k = W.shape
    wide = W.double() if W.dtype == torch.float32 else W.float()
    t = _pad(_pad(wide, 1), 2).view(G, _blocks(n), 128, _blocks(k), 128)
    A = t.abs().amax((2, 4)).clamp(min=FLOOR)
    q = (t * 448 / A[:, :, None, :, None]).view(G, _blocks(n) * 128, -1)[:, :n, :k].to(E4M3)
    return q.contiguous(), (A.float() / 448).contiguous()


def _row_blocks(x, w=None):
    """[R, d] as (e4m3 codes, fp32 scales [blocks of d, R])."""
    R, d = x.shape
    wide = x.double() if x.dtype == torch.float32 else x.float()
    t = _pad(wide, 1).view(R, _blocks(d), 128)
    A = t.abs().amax(2).clamp(min=FLOOR)
    q = (t * 448 / A[:, :, None]).view(R, -1)[:, :d].to(E4M3)
    s = A.float() / 448
    if w is not None:
        s = s * w[:, None]
    return q.contiguous(), s.t().contiguous()


def _segments(case, g):
    """Rows of each expert, on the host: the batch's sizes as a router leaves them."""
    R, E = case["rows"], case["experts"]
    if case["seg"] == "whole":
        return [R]
    p = torch.ones(E, device="cuda") if case["seg"] == "even" else torch.rand(E, generator=g, device="cuda").pow(3) + 0.02
    got = torch.multinomial(p, R, replacement=True, generator=g)
    return torch.bincount(got, minlength=E).tolist()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)

    op, s = case["op"], {"case": case}
    if op == "rows":
        s["x"] = randn(case["rows"], case["d"], dtype=torch.float32)
        s["x"][:, ::97] *= 12.0  # a few large channels
        s["x"] = s["x"].to(TYPES[case["dtype"]])
    elif op == "swiglu":
        s["gu"] = randn(case["rows"], 2 * case["inter"])
        s["w"] = torch.rand(case["rows"], generator=g, device="cuda") if case["weighted"] else None
    elif op == "weight":
        s["W"] = randn(case["experts"], case["n"], case["k"], scale=case["k"] ** -0.5, dtype=TYPES[case["dtype"]])
    elif op == "product":
        counts = _segments(case, g)
        s["a"], s["sa"] = _row_blocks(randn(case["rows"], case["k"]))
        s["b"], s["sb"] = _weight_blocks(randn(case["experts"], case["n"], case["k"], scale=case["k"] ** -0.5))
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        s["most"] = max(counts)  # a batch's plan has its longest segment
    else:
        d, E, inter, S = case["d"], case["experts"], case["inter"], case["shared"]
        s["x"] = randn(case["tokens"], d)
        s["router"] = randn(E, d, scale=d ** -0.5)
        gate_up, down = randn(E, 2 * inter, d, scale=d ** -0.5), randn(E, d, inter, scale=inter ** -0.5)
        sh_gu, sh_dn = randn(1, 2 * S * inter, d, scale=d ** -0.5), randn(1, d, S * inter, scale=inter ** -0.5)
        if case["weights"] == "fp8":
            (gate_up, s["s_gate_up"]), (down, s["s_down"]) = _weight_blocks(gate_up), _weight_blocks(down)
            if S:
                (sh_gu, a), (sh_dn, b) = _weight_blocks(sh_gu), _weight_blocks(sh_dn)
                s["s_shared"] = torch.cat([a.flatten(), b.flatten()])
        s["gate_up"], s["down"] = gate_up, down
        s["shared"] = torch.cat([sh_gu.flatten().view(torch.uint8), sh_dn.flatten().view(torch.uint8)]).view(sh_gu.dtype) if S else None
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    if op == "rows":
        return _row_blocks(state["x"])
    if op == "swiglu":
        gate, up = state["gu"].float().chunk(2, 1)
        h = gate / (1 + torch.exp(-gate)) * up
        return _row_blocks_f32(h, state["w"])
    if op == "weight":
        return _weight_blocks(state["W"])
    if op == "product":
        return _plain_product(state)
    return _plain_few(state)


def _row_blocks_f32(h, w):
    """_row_blocks of values that were computed in 32 bits."""
    R, d = h.shape
    t = _pad(h, 1).view(R, _blocks(d), 128)
    A = t.abs().amax(2).clamp(min=FLOOR)
    q = (t * 448 / A[:, :, None]).view(R, -1)[:, :d].to(E4M3)
    s = A / 448
    if w is not None:
        s = s * w[:, None]
    return q.contiguous(), s.t().contiguous()


def _wide(q, s, dtype=torch.float32):
    """The values that 8-bit weights [..., n, k] and their block scales stand for."""
    n, k = q.shape[-2:]
    s = s.to(dtype).repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]
    return q.to(dtype) * s


def _padded(state):
    """(expert, place in the expert's segment) of each row."""
    counts = state["counts"].long()
    expert = torch.repeat_interleave(torch.arange(counts.numel(), device="cuda"), counts, output_size=state["case"]["rows"])
    first = counts.cumsum(0) - counts
    return expert, torch.arange(expert.numel(), device="cuda") - first[expert]


def _product(state, dtype):
    case = state["case"]
    a = state["a"].to(dtype) * state["sa"].t().to(dtype).repeat_interleave(128, 1)[:, :case["k"]]
    b = _wide(state["b"], state["sb"], dtype)
    if case["experts"] == 1:
        return a @ b[0].t()
    expert, place = _padded(state)
    rows = a.new_zeros(case["experts"], state["most"], case["k"])
    rows[expert, place] = a
    return torch.bmm(rows, b.transpose(1, 2))[expert, place]


def _plain_product(state):
    return _product(state, torch.float32).to(TYPES[state["case"]["out"]])


def _choose(logits, case):
    """The k experts of each token inside its kept groups, ties to the lower index, and their weights."""
    T, E = logits.shape
    best = logits.view(T, case["groups"], -1).amax(2)
    kept = torch.zeros_like(best, dtype=torch.bool)
    kept.scatter_(1, best.sort(dim=1, descending=True, stable=True)[1][:, :case["kept"]], True)
    masked = logits.masked_fill(~kept.repeat_interleave(E // case["groups"], 1), -math.inf)
    idx = masked.sort(dim=1, descending=True, stable=True)[1][:, :case["k"]]
    w = 1 / (1 + torch.exp(-logits.gather(1, idx)))
    return idx, w / w.sum(1, keepdim=True)


def _plain_few(state):
    case = state["case"]
    S, inter, d = case["shared"], case["inter"], case["d"]
    x = state["x"].float()
    # which expert is next is a matter of 64 bits where two are close
    idx, w = _choose(state["x"].double() @ state["router"].double().t(), case)
    gu, dn = _taken(state, "gate_up", idx), _taken(state, "down", idx)
    hid = torch.matmul(gu, x[:, None, :, None]).squeeze(3)
    h = hid[..., :inter] / (1 + torch.exp(-hid[..., :inter])) * hid[..., inter:]
    y = (torch.matmul(dn, h[..., None]).squeeze(3) * w.float()[..., None]).sum(1)
    if S:
        sh_gu, sh_dn = _shared(state, torch.float32)
        hid = x @ sh_gu.t()
        h = hid[:, :S * inter] / (1 + torch.exp(-hid[:, :S * inter])) * hid[:, S * inter:]
        y = y + h @ sh_dn.t()
    return y.to(torch.bfloat16), idx.int(), w.float()


def _taken(state, name, idx):
    """The chosen experts' weights of each token, in 32 bits."""
    W = state[name]
    if state["case"]["weights"] == "fp8":
        return _wide(W.view(torch.uint8)[idx].view(E4M3), state["s_" + name][idx])
    return W[idx].float()


def _shared(state, dtype):
    case = state["case"]
    S, inter, d = case["shared"], case["inter"], case["d"]
    gu, dn = state["shared"][:2 * S * inter * d].view(2 * S * inter, d), state["shared"][2 * S * inter * d:].view(d, S * inter)
    if case["weights"] == "fp8":
        n = 2 * S * inter // 128 * (d // 128)
        s = state["s_shared"]
        return _wide(gu, s[:n].view(-1, d // 128), dtype), _wide(dn, s[n:].view(d // 128, -1), dtype)
    return gu.to(dtype), dn.to(dtype)


def _own(op, state):
    from sparse_mixture_experts_03_b200 import moe

    case = state["case"]
    if op == "rows":
        return moe.quantize_rows(state["x"])
    if op == "swiglu":
        return moe.swiglu_quantize_rows(state["gu"], state["w"])
    if op == "weight":
        return moe.quantize_weight(state["W"])
    if op == "product":
        counts = None if case["experts"] == 1 else state["counts"]
        return moe.matmul_fp8(state["a"], state["sa"], state["b"], state["sb"], counts, out_dtype=TYPES[case["out"]])
    T, k = case["tokens"], case["k"]
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, dtype=torch.float32, device="cuda")
    scales = (state["s_gate_up"], state["s_down"], state.get("s_shared")) if case["weights"] == "fp8" else None
    y = moe.forward_few(state["x"], state["router"], state["gate_up"], state["down"], state["shared"], k, case["groups"], case["kept"],
                        case["inter"], case["shared"], scales=scales, out_dtype=torch.bfloat16, topk_idx=idx, topk_w=w)
    return y, idx, w


# ---------------------------------------------------------------- the cost, and 64 bits

def work(case):
    op = case["op"]
    size = 2 if case.get("dtype") == "bf16" else 4
    if op == "rows":
        n = case["rows"] * case["d"]
        return {"bytes": n * size + n + 4 * case["rows"] * _blocks(case["d"]), "flops": 3 * n}
    if op == "swiglu":
        n = case["rows"] * case["inter"]
        return {"bytes": 4 * n + n + 4 * case["rows"] * (_blocks(case["inter"]) + case["weighted"]), "flops": 8 * n}
    if op == "weight":
        n = case["experts"] * case["n"] * case["k"]
        return {"bytes": n * size + n + 4 * case["experts"] * _blocks(case["n"]) * _blocks(case["k"]), "flops": 3 * n}
    if op == "product":
        R, E, n, k = case["rows"], case["experts"], case["n"], case["k"]
        used = E * (1 - (1 - 1 / E) ** R)  # experts with rows, if the router is fair
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": R * k + used * n * k + R * n * out + 4 * (R + used * _blocks(n)) * _blocks(k), "flops": 2 * R * n * k}
    T, d, E, inter, S = case["tokens"], case["d"], case["experts"], case["inter"], case["shared"]
    used = E * (1 - (1 - case["k"] / E) ** T) + S
    each = 3 * inter * d
    return {"bytes": used * each * (2 if case["weights"] == "bf16" else 1) + 2 * E * d + 4 * T * d + 8 * T * case["k"],
            "flops": 2 * T * (case["k"] + S) * each + 2 * T * E * d}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rows":
        return _exact_rows(s["x"].double(), None)
    if op == "swiglu":
        gu = s["gu"].double()
        g, u = gu[:, :case["inter"]], gu[:, case["inter"]:]
        return _exact_rows(g * torch.sigmoid(g) * u, s["w"])
    if op == "weight":
        W = s["W"].double()
        q, sc = torch.empty_like(W), W.new_empty(case["experts"], _blocks(case["n"]), _blocks(case["k"]))
        for i in range(sc.shape[1]):
            for j in range(sc.shape[2]):
                part = W[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                top = part.abs().flatten(1).max(1).values.clamp(min=FLOOR)
                sc[:, i, j] = top / 448
                q[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128] = _nearest(part * 448 / top[:, None, None])
        return q, sc
    if op == "product":
        R, n, k = case["rows"], case["n"], case["k"]
        y, first = torch.empty(R, n, dtype=torch.float64, device="cuda"), 0
        for e, c in enumerate(s["counts"].tolist()):
            A, B = s["a"][first:first + c].double(), s["b"][e].double()
            y[first:first + c] = 0
            for j in range(_blocks(k)):
                part = A[:, 128 * j:128 * j + 128] @ B[:, 128 * j:128 * j + 128].t()
                scale = s["sa"][j, first:first + c].double()[:, None] * s["sb"][e, :, j].double().repeat_interleave(128)[:n]
                y[first:first + c] += part * scale
            first += c
        return y
    return _exact_few(case, s)


def _nearest(t):
    """The e4m3 value next to each, ties to the even one, in 64 bits: three bits behind the leading one, the smallest step 2^-9."""
    _, e = torch.frexp(t)
    step = torch.ldexp(torch.ones_like(t), (e - 4).clamp(min=-9))
    return torch.round(t / step) * step


def _exact_rows(x, w):
    R, d = x.shape
    q, s = torch.empty_like(x), x.new_empty(_blocks(d), R)
    for b in range(_blocks(d)):
        part = x[:, 128 * b:128 * b + 128]
        top = part.abs().max(1).values.clamp(min=FLOOR)
        s[b] = top / 448
        q[:, 128 * b:128 * b + 128] = _nearest(part * 448 / top[:, None])
    return q, s if w is None else s * w.double()


def _exact_few(case, s):
    T, k, E, inter, S = case["tokens"], case["k"], case["experts"], case["inter"], case["shared"]
    per = E // case["groups"]
    x = s["x"].double()
    logits = x @ s["router"].double().t()
    rows, chosen, weights = [], [], []

    def ffn(gu, dn, v, rows_n):
        hid = gu @ v
        return dn @ (hid[:rows_n] * torch.sigmoid(hid[:rows_n]) * hid[rows_n:])

    sh = _shared(s, torch.float64) if S else None
    for t in range(T):
        l = logits[t].tolist()
        groups = sorted(range(case["groups"]), key=lambda g: (-max(l[g * per:(g + 1) * per]), g))[:case["kept"]]
        pick = sorted((e for g in groups for e in range(g * per, (g + 1) * per)), key=lambda e: (-l[e], e))[:k]
        score = [1 / (1 + math.exp(-l[e])) for e in pick]
        y = torch.zeros_like(x[t])
        for e, p in zip(pick, score):
            gu, dn = s["gate_up"][e], s["down"][e]
            gu = _wide(gu, s["s_gate_up"][e], torch.float64) if case["weights"] == "fp8" else gu.double()
            dn = _wide(dn, s["s_down"][e], torch.float64) if case["weights"] == "fp8" else dn.double()
            y += p / sum(score) * ffn(gu, dn, x[t], inter)
        if S:
            y += ffn(*sh, x[t], S * inter)
        rows.append(y)
        chosen.append(pick)
        weights.append([p / sum(score) for p in score])
    return torch.stack(rows), torch.tensor(chosen, dtype=torch.int32, device="cuda"), torch.tensor(weights, dtype=torch.float64, device="cuda")
