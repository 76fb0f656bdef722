"""Cases of the 8-bit float and expert-grouped products, with their plain forms.

Four operators of the library:

  f8_quantize      rows of f32/bf16/f16 to e4m3 with one power-of-two scale per
                   128 columns
  f8_mm            y = x W^T, both e4m3 with f32 scales (x: per row and 128
                   columns; W: per 128 x 128 block)
  mm_grouped       y[r] = x[r] W_e^T for the rows r of group e, groups given by
                   offsets on the device; bf16, f16, or e4m3 with block scales
  moe_experts_f8   the experts of a mixture-of-experts layer for given routes:
                   quantise, gate and up products, SwiGLU, quantise, down
                   product, weighted sum into the residual

The plain forms are elementary torch operations in 32 bits; ``exact`` is the
definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the FFN input of one decoded token, hidden 2048
        dict(name="quantize_1x2048_bf16", op="f8_quantize", rows=1, cols=2048, type="bf16"),
        # the activations of a dense FFN of width 14336 for 4096 prompt tokens
        dict(name="quantize_4096x14336_bf16", op="f8_quantize", rows=4096, cols=14336,
             type="bf16"),
        # f32 hidden states (the library's own residual type), a ragged batch
        dict(name="quantize_517x2064_f32", op="f8_quantize", rows=517, cols=2064, type="f32"),
        # one decoded token through a 4096 x 4096 projection: latency
        dict(name="f8_mm_1x4096x4096", op="f8_mm", tokens=1, rows=4096, cols=4096, out="bf16"),
        # a serving batch of odd size through the dense FFN's gate
        dict(name="f8_mm_37x14336x4096", op="f8_mm", tokens=37, rows=14336, cols=4096,
             out="bf16"),
        # 4096 prompt tokens through the dense FFN's gate: the tensor cores' rate
        dict(name="f8_mm_4096x14336x4096", op="f8_mm", tokens=4096, rows=14336, cols=4096,
             out="bf16"),
        # one token's eight experts, bf16 gate rows: eight groups of one row
        dict(name="grouped_bf16_8rows", op="mm_grouped", type="bf16", out="bf16", experts=128,
             n_rows=8, rows=768, cols=2048, spread="spaced"),
        # 512 tokens, top-8 of 64 experts, uneven groups, e4m3 gate rows
        dict(name="grouped_f8_4096rows", op="mm_grouped", type="f8", out="bf16", experts=64,
             n_rows=4096, rows=1024, cols=2048, spread="uneven"),
        # a long prompt over few large f16 experts
        dict(name="grouped_f16_16384rows", op="mm_grouped", type="f16", out="f16", experts=8,
             n_rows=16384, rows=4096, cols=4096, spread="uneven"),
        # one decoded token of a layer of hidden 2048, 128 experts, top-8
        dict(name="moe_1token", op="moe_experts_f8", tokens=1, hidden=2048, expert_dim=768,
             experts=128, top_k=8, type="bf16"),
        # 512 tokens, hidden 2048, 64 experts, top-8: every expert is read, few rows each
        dict(name="moe_512tokens", op="moe_experts_f8", tokens=512, hidden=2048, expert_dim=1024,
             experts=64, top_k=8, type="bf16"),
        # a prompt of 4096 tokens
        dict(name="moe_4096tokens", op="moe_experts_f8", tokens=4096, hidden=2048,
             expert_dim=768, experts=128, top_k=8, type="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["f8_quantize", "f8_mm", "f8_mm", "mm_grouped", "mm_grouped",
                     "moe_experts_f8", "moe_experts_f8"])
    if op == "f8_quantize":
        return dict(op=op, rows=_log(rng, 1, 4096), cols=_log(rng, 64, 14336),
                    type=rng.choice(["f32", "bf16", "f16"]))
    if op == "f8_mm":
        return dict(op=op, tokens=_log(rng, 1, 4096), rows=_log(rng, 100, 14336),
                    cols=16 * _log(rng, 8, 256), out=rng.choice(["bf16", "f16", "f32"]))
    if op == "mm_grouped":
        kind = rng.choice(["bf16", "f16", "f8"])
        return dict(op=op, type=kind, out=rng.choice(["bf16", "f16", "f32"]),
                    experts=_log(rng, 1, 128), n_rows=_log(rng, 1, 8192),
                    rows=_log(rng, 100, 2048), cols=16 * _log(rng, 8, 128),
                    spread=rng.choice(["even", "uneven", "spaced"]))
    experts = _log(rng, 4, 128)
    return dict(op=op, tokens=_log(rng, 1, 2048), hidden=128 * rng.randint(2, 16),
                expert_dim=128 * rng.randint(1, 8), experts=experts,
                top_k=rng.randint(1, min(experts, 8)), type=rng.choice(["bf16", "f16"]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, n, k, dtype):
    """Rows of a residual stream: unit normal, some channels 8 times larger."""
    x = torch.randn(n, k, generator=g, device="cuda")
    loud = torch.rand(k, generator=g, device="cuda") < 0.01
    return torch.where(loud, 8.0 * x, x).to(dtype)


def _block_weights(g, e, n, k):
    """e4m3 matrices with one f32 scale per 128 x 128 block, as a checkpoint
    holds them: the block's largest magnitude becomes 448."""
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    q = torch.empty(e, n, k, dtype=F8, device="cuda")
    s = torch.empty(e, nb, kb, device="cuda")
    for i in range(e):
        w = torch.zeros(nb * BLOCK, kb * BLOCK, device="cuda")
        w[:n, :k] = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
        t = w.view(nb, BLOCK, kb, BLOCK)
        s[i] = t.abs().amax(dim=(1, 3)) / 448.0
        q[i] = (t / s[i][:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n, :k].to(F8)
    return q, s


def _sizes(g, case):
    """Rows of each group, as routing leaves them."""
    e, n = case["experts"], case["n_rows"]
    if case["spread"] == "even":
        return [n // e + (1 if i < n % e else 0) for i in range(e)]
    if case["spread"] == "spaced":  # one row in each of n groups, evenly spaced
        sizes = [0] * e
        for i in range(n):
            sizes[i * e // n % e if n < e else i % e] += 1
        return sizes
    p = torch.exp(torch.randn(e, generator=g, device="cuda"))
    p[torch.rand(e, generator=g, device="cuda") < 0.1] = 0.0  # experts with no rows
    if float(p.sum()) == 0.0:
        p[0] = 1.0
    pick = torch.multinomial(p, n, replacement=True, generator=g)
    return torch.bincount(pick, minlength=e).tolist()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op == "f8_quantize":
        x = _activations(g, case["rows"], case["cols"], TYPES[case["type"]])
        st.update(x=x, q=torch.empty(x.shape, dtype=F8, device="cuda"),
                  s=torch.empty(x.shape[0], -(-x.shape[1] // BLOCK), device="cuda"))
    elif op == "f8_mm":
        w, ws = _block_weights(g, 1, case["rows"], case["cols"])
        xq, xs = _plain_quantize(_activations(g, case["tokens"], case["cols"], torch.float32))
        st.update(w=w[0], ws=ws[0], xq=xq, xs=xs,
                  y=torch.empty(case["tokens"], case["rows"], dtype=TYPES[case["out"]],
                                device="cuda"))
    elif op == "mm_grouped":
        e, n, k = case["experts"], case["rows"], case["cols"]
        sizes = _sizes(g, case)
        offsets = [0]
        for c in sizes:
            offsets.append(offsets[-1] + c)
        x = _activations(g, case["n_rows"], k, torch.float32)
        if case["type"] == "f8":
            w, ws = _block_weights(g, e, n, k)
            x, xs = _plain_quantize(x)
            st.update(w=w, ws=ws, x=x, xs=xs)
        else:
            dt = TYPES[case["type"]]
            w = torch.empty(e, n, k, dtype=dt, device="cuda")
            for i in range(e):
                w[i] = (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).to(dt)
            st.update(w=w, ws=None, x=x.to(dt), xs=None)
        st.update(sizes=sizes, host_offsets=offsets,
                  offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                  y=torch.empty(case["n_rows"], n, dtype=TYPES[case["out"]], device="cuda"))
    else:
        t, h, f, e, k = (case[i] for i in ("tokens", "hidden", "expert_dim", "experts", "top_k"))
        for name, n, c in (("gate", f, h), ("up", f, h), ("down", h, f)):
            st[name], st[name + "_s"] = _block_weights(g, e, n, c)
        dt = TYPES[case["type"]]
        logits = torch.randn(t, e, generator=g, device="cuda")
        logits = logits + 0.5 * torch.randn(e, generator=g, device="cuda")  # uneven load
        top, idx = torch.topk(torch.softmax(logits, -1), k, dim=-1)
        st.update(x=_activations(g, t, h, dt), idx=idx.to(torch.int32),
                  w=top / top.sum(-1, keepdim=True),
                  residual=torch.randn(t, h, generator=g, device="cuda").to(dt),
                  out=torch.empty(t, h, dtype=dt, device="cuda"))
        if own:
            import moe_ffn_gb300 as qm
            shape = qm.moe_shape(h, f, e, k, t, qm.E4M3, qm.E4M3, qm.E4M3)
            st.update(shape=shape, wsp=torch.empty(qm.moe_experts_f8_workspace_size(shape),
                                                   dtype=torch.uint8, device="cuda"))
    return st


# -------------------------------------------------------------- plain forms
def _plain_quantize(x):
    n, k = x.shape
    kb = -(-k // BLOCK)
    p = torch.zeros(n, kb * BLOCK, device=x.device)
    p[:, :k] = x.float()
    p = p.view(n, kb, BLOCK)
    a = p.abs().amax(-1)
    m, ex = torch.frexp(a)  # a = m * 2^ex, 0.5 <= m < 1; 448 = 0.875 * 2^9
    ex = torch.where(m > 0.875, ex - 8, ex - 9).clamp(min=-126)
    s = torch.where(a > 0, torch.ldexp(torch.ones_like(a), ex), torch.ones_like(a))
    q = (p / s[:, :, None]).to(F8)
    return q.view(n, kb * BLOCK)[:, :k].contiguous(), s


def _plain_rows(q, s):
    """Scaled values of e4m3 rows with one scale per 128 columns."""
    return q.float() * s.repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]


def _plain_matrix(q, s):
    """Scaled values of an e4m3 matrix with one scale per 128 x 128 block."""
    n, k = q.shape
    if n % BLOCK == 0 and k % BLOCK == 0:
        v = q.float().view(n // BLOCK, BLOCK, k // BLOCK, BLOCK) * s[:, None, :, None]
        return v.view(n, k)
    full = s.repeat_interleave(BLOCK, dim=0)[:n]
    return q.float() * full.repeat_interleave(BLOCK, dim=1)[:, :k]


def _plain_moe(st):
    k, e = st["top_k"], st["experts"]
    x = _plain_rows(*_plain_quantize(st["x"]))
    flat = st["idx"].reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    sizes = torch.bincount(flat, minlength=e).tolist()
    y = torch.empty(flat.numel(), st["hidden"], device=x.device)
    at = 0
    for i, c in enumerate(sizes):
        if c == 0:
            continue
        pairs = order[at:at + c]
        at += c
        xe = x[pairs // k]
        gate = xe @ _plain_matrix(st["gate"][i], st["gate_s"][i]).T
        up = xe @ _plain_matrix(st["up"][i], st["up_s"][i]).T
        a = gate / (1.0 + torch.exp(-gate)) * up
        y[pairs] = _plain_rows(*_plain_quantize(a)) @ _plain_matrix(st["down"][i],
                                                                   st["down_s"][i]).T
    add = (y.view(-1, k, st["hidden"]) * st["w"][:, :, None]).sum(1)
    return (st["residual"].float() + add).to(st["out"].dtype)


def _run_plain(st):
    op = st["op"]
    if op == "f8_quantize":
        return _plain_quantize(st["x"])
    if op == "f8_mm":
        y = _plain_rows(st["xq"], st["xs"]) @ _plain_matrix(st["w"], st["ws"]).T
        return y.to(st["y"].dtype)
    if op == "mm_grouped":
        at, parts = 0, []
        for i, c in enumerate(st["sizes"]):
            if c == 0:
                continue
            if st["type"] == "f8":
                x = _plain_rows(st["x"][at:at + c], st["xs"][at:at + c])
                parts.append(x @ _plain_matrix(st["w"][i], st["ws"][i]).T)
            else:
                parts.append(st["x"][at:at + c].float() @ st["w"][i].float().T)
            at += c
        return torch.cat(parts).to(st["y"].dtype)
    return _plain_moe(st)


# ------------------------------------------------------------ the library's
def _run_own(st):
    import moe_ffn_gb300 as qm
    kinds = {torch.float32: qm.F32, torch.bfloat16: qm.BF16, torch.float16: qm.F16}
    op = st["op"]
    if op == "f8_quantize":
        qm.f8_quantize(kinds[st["x"].dtype], st["x"], st["rows"], st["cols"], st["q"], st["s"])
        return st["q"], st["s"]
    if op == "f8_mm":
        qm.f8_mm(st["w"], st["ws"], st["rows"], st["cols"], st["xq"], st["xs"], st["tokens"],
                 kinds[st["y"].dtype], st["y"])
        return st["y"]
    if op == "mm_grouped":
        kind = qm.E4M3 if st["type"] == "f8" else kinds[st["w"].dtype]
        qm.mm_grouped(kind, st["w"], st["ws"], st["experts"], st["rows"], st["cols"], st["x"],
                      st["xs"], st["n_rows"], st["offsets"], kinds[st["y"].dtype], st["y"])
        return st["y"]
    qm.moe_experts_f8(st["gate"], st["gate_s"], st["up"], st["up_s"], st["down"], st["down_s"],
                      st["shape"], kinds[st["x"].dtype], st["x"], st["idx"], st["w"],
                      st["residual"], st["out"], st["wsp"])
    return st["out"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------------- work
def _active(case):
    """Groups that have rows, as expected of the case's spread."""
    e, n = case["experts"], case["n_rows"]
    if case["spread"] == "uneven":
        return 0.9 * e * (1.0 - (1.0 - 1.0 / e) ** n)
    return min(e, n)


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2, "f8": 1}
    if op == "f8_quantize":
        n, k = case["rows"], case["cols"]
        return {"bytes": n * k * (size[case["type"]] + 1) + 4 * n * -(-k // BLOCK),
                "flops": 2 * n * k}
    if op == "f8_mm":
        m, n, k = case["tokens"], case["rows"], case["cols"]
        kb = -(-k // BLOCK)
        return {"bytes": n * k + 4 * kb * -(-n // BLOCK) + m * (k + 4 * kb)
                + m * n * size[case["out"]], "flops": 2 * m * n * k}
    if op == "mm_grouped":
        m, n, k = case["n_rows"], case["rows"], case["cols"]
        return {"bytes": int(_active(case) * n * k + m * k) * size[case["type"]]
                + m * n * size[case["out"]], "flops": 2 * m * n * k}
    t, h, f, e, k = (case[i] for i in ("tokens", "hidden", "expert_dim", "experts", "top_k"))
    active = e * (1.0 - (1.0 - k / e) ** t)
    return {"bytes": int(active * 3 * h * f) + 3 * t * h * size[case["type"]] + 8 * t * k,
            "flops": 6 * t * k * h * f}


# ------------------------------------------------------------------- exact
def _e4m3(v):
    """Nearest e4m3 value of each element, ties to the even significand."""
    a = v.abs()
    ex = torch.floor(torch.log2(torch.clamp(a, min=2.0 ** -30)))
    ex = torch.where(torch.exp2(ex) > a, ex - 1, ex)
    ex = torch.where(torch.exp2(ex + 1) <= a, ex + 1, ex)
    step = torch.exp2(torch.clamp(ex, min=-6.0) - 3.0)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def _quantized64(x):
    """(codes as values, scales) of 64-bit rows, by the definition."""
    n, k = x.shape
    q = torch.empty_like(x)
    scales = torch.empty(n, -(-k // BLOCK), dtype=torch.float64, device=x.device)
    for b in range(scales.shape[1]):
        blk = x[:, b * BLOCK:(b + 1) * BLOCK]
        top = blk.abs().amax(1)
        ex = torch.ceil(torch.log2(torch.clamp(top, min=2.0 ** -140) / 448.0))
        ex = torch.where(448.0 * torch.exp2(ex - 1) >= top, ex - 1, ex)
        ex = torch.where(448.0 * torch.exp2(ex) < top, ex + 1, ex)
        s = torch.where(top > 0, torch.exp2(torch.clamp(ex, min=-126.0)), torch.ones_like(top))
        scales[:, b] = s
        q[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3(blk / s[:, None])
    return q, scales


def _product64(xq, xs, w, ws):
    """sum over 128-column blocks of xs * ws * (codes' product)."""
    n, k = w.shape
    y = torch.zeros(xq.shape[0], n, dtype=torch.float64, device=xq.device)
    if xq.shape[0] <= 64:
        wd = w.double()
        for b in range(-(-k // BLOCK)):
            cols = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
            row_scale = ws[:, b].double().repeat_interleave(BLOCK)[:n]
            y += xs[:, b:b + 1].double() * ((xq[:, cols].double() @ wd[:, cols].T) * row_scale)
        return y
    # the same sums with the scales inside them: one product per matrix
    col = torch.arange(k, device=w.device) // BLOCK
    row = torch.arange(n, device=w.device) // BLOCK
    return (xq.double() * xs.double()[:, col]) @ (w.double() * ws.double()[row][:, col]).T


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "f8_quantize":
        return _quantized64(st["x"].double())
    if op == "f8_mm":
        return _product64(st["xq"], st["xs"], st["w"], st["ws"])
    if op == "mm_grouped":
        y = torch.empty(case["n_rows"], case["rows"], dtype=torch.float64, device="cuda")
        off = st["host_offsets"]
        for i in range(case["experts"]):
            rows = slice(off[i], off[i + 1])
            if off[i] == off[i + 1]:
                continue
            if case["type"] == "f8":
                y[rows] = _product64(st["x"][rows], st["xs"][rows], st["w"][i], st["ws"][i])
            else:
                y[rows] = st["x"][rows].double() @ st["w"][i].double().T
        return y
    out = st["residual"].double()
    xq, xs = _quantized64(st["x"].double())
    for i in range(case["experts"]):
        tok, slot = torch.nonzero(st["idx"] == i, as_tuple=True)
        if tok.numel() == 0:
            continue
        gate = _product64(xq[tok], xs[tok], st["gate"][i], st["gate_s"][i])
        up = _product64(xq[tok], xs[tok], st["up"][i], st["up_s"][i])
        aq, a_s = _quantized64(gate / (1.0 + torch.exp(-gate)) * up)
        y = _product64(aq, a_s, st["down"][i], st["down_s"][i])
        out.index_add_(0, tok, y * st["w"][tok, slot].double()[:, None])
    return out
