"""Cases of the steps around a mixture-of-experts layer's products, and of
products with 4-bit weights, with their plain forms.

Operators of the library:

  moe_route, moe_route_backward      router logits to the top-k experts and
                                     their softmax weights; the gradient of the
                                     logits
  moe_permute                        tokens sorted by expert: each token's row
                                     copied to the rows of its experts' groups
                                     (its gradient is moe_combine without
                                     weights)
  moe_combine, moe_combine_backward  the rows of a token's experts weighted and
                                     added to its residual; gradients of the
                                     rows and of the weights
  w4_mm, w4_mm_grouped               y = x W^T with 4-bit W, a scale and
                                     optionally a zero point per 32, 64 or 128
                                     columns of a row; one matrix, or a stack
                                     with ragged groups of rows

The plain forms are elementary torch operations in 32 bits; ``exact`` is the
definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token's routing, 128 experts: latency
        dict(name="route_1x128", op="route", tokens=1, experts=128, top_k=8, type="f32",
             renorm=True, train=False, masked=False),
        # a training batch's routing and its gradient, weights not renormalised
        dict(name="route_train_16384x128", op="route", tokens=16384, experts=128, top_k=8,
             type="bf16", renorm=False, train=True, masked=False),
        # one decoded token copied to its eight experts' rows: latency
        dict(name="permute_1x2048", op="permute", tokens=1, cols=2048, experts=128, top_k=8,
             type="bf16", pad=0.0, train=False),
        # a prompt of 4096 tokens sorted by expert
        dict(name="permute_4096x2048", op="permute", tokens=4096, cols=2048, experts=128, top_k=8,
             type="bf16", pad=0.0, train=False),
        # an odd batch in f32 with padded slots, and the gradient of its rows
        dict(name="permute_train_517x2064", op="permute", tokens=517, cols=2064, experts=64,
             top_k=6, type="f32", pad=0.1, train=True),
        # one decoded token's expert outputs added up, into the library's f32 residual: latency
        dict(name="combine_1x2048", op="combine", tokens=1, cols=2048, experts=128, top_k=8,
             type="bf16", out="f32", pad=0.0, train=False),
        # the same for a prompt of 4096 tokens, bf16 throughout
        dict(name="combine_4096x2048", op="combine", tokens=4096, cols=2048, experts=128, top_k=8,
             type="bf16", out="bf16", pad=0.0, train=False),
        # a training batch: the sum, the gradients of the rows and of the weights
        dict(name="combine_train_4096x2048", op="combine", tokens=4096, cols=2048, experts=64,
             top_k=8, type="bf16", out="bf16", pad=0.0, train=True),
        # one decoded token through a 4096 x 4096 projection
        dict(name="w4_1x4096x4096", op="w4_mm", tokens=1, rows=4096, cols=4096, group=128,
             zeros=True, scale="f16", type="bf16", out="bf16"),
        # five requests decoded together through the dense FFN's gate, symmetric weights
        dict(name="w4_5x14336x4096", op="w4_mm", tokens=5, rows=14336, cols=4096, group=64,
             zeros=False, scale="f16", type="f16", out="f16"),
        # one token's eight experts, gate rows: eight groups of one row
        dict(name="w4_grouped_8rows", op="w4_mm_grouped", experts=128, n_rows=8, rows=768,
             cols=2048, group=128, zeros=True, scale="bf16", type="bf16", out="bf16",
             spread="spaced"),
        # 512 tokens, top-8 of 64 experts, uneven groups
        dict(name="w4_grouped_4096rows", op="w4_mm_grouped", experts=64, n_rows=4096, rows=1024,
             cols=2048, group=128, zeros=True, scale="bf16", type="bf16", out="bf16",
             spread="uneven"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "permute", "combine", "combine", "w4_mm", "w4_mm", "w4_mm_grouped",
                     "w4_mm_grouped"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "route":
        experts = _log(rng, 4, 512)
        return dict(op=op, tokens=_log(rng, 1, 4096), experts=experts,
                    top_k=rng.randint(1, min(experts, 16)), type=kind,
                    renorm=rng.random() < 0.5, train=rng.random() < 0.5,
                    masked=rng.random() < 0.3)
    if op in ("permute", "combine"):
        experts = _log(rng, 4, 512)
        case = dict(op=op, tokens=_log(rng, 1, 2048), cols=_log(rng, 64, 2500), experts=experts,
                    top_k=rng.randint(1, min(experts, 8)), type=kind,
                    pad=rng.choice([0.0, 0.0, 0.2]), train=rng.random() < 0.5)
        if op == "combine":
            case["out"] = rng.choice([kind, "f32"])
        return case
    group = rng.choice([32, 64, 128])
    case = dict(op=op, group=group, zeros=rng.random() < 0.5,
                scale=rng.choice(["f32", "bf16", "f16"]), type=kind,
                out=rng.choice([kind, "f32"]))
    if op == "w4_mm":
        return dict(case, tokens=_log(rng, 1, 64), rows=_log(rng, 100, 8192),
                    cols=group * max(1, _log(rng, 64, 4096) // group))
    return dict(case, experts=_log(rng, 1, 128), n_rows=_log(rng, 1, 1024),
                rows=_log(rng, 100, 1024), cols=group * max(1, _log(rng, 128, 2048) // group),
                spread=rng.choice(["even", "uneven", "spaced"]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, n, k, dtype):
    """Rows of a residual stream: unit normal, some channels 8 times larger."""
    x = torch.randn(n, k, generator=g, device="cuda")
    loud = torch.rand(k, generator=g, device="cuda") < 0.01
    return torch.where(loud, 8.0 * x, x).to(dtype)


def _w4(g, e, n, k, group, zeros, dtype):
    """A stack of normal matrices rounded to 4 bits: codes (two to a byte, the
    even column in the low half), scales, and zero points (or None: 8)."""
    q = torch.empty(e, n, k // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(e, n, k // group, dtype=dtype, device="cuda")
    z = torch.empty(e, n, k // group, dtype=torch.uint8, device="cuda") if zeros else None
    for i in range(e):
        w = (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).view(n, -1, group)
        if zeros:
            lo, hi = w.amin(-1).clamp(max=0.0), w.amax(-1).clamp(min=0.0)
            s[i] = ((hi - lo) / 15.0).to(dtype)
            zero = torch.round(-lo / s[i].float()).clamp(0, 15)
            z[i] = zero.to(torch.uint8)
        else:
            s[i] = (w.abs().amax(-1) / 7.0).to(dtype)
            zero = torch.full_like(w[:, :, 0], 8.0)
        c = (torch.round(w / s[i].float()[:, :, None]) + zero[:, :, None]).clamp(0, 15)
        c = c.to(torch.uint8).view(n, k)
        q[i] = c[:, 0::2] | (c[:, 1::2] << 4)
    return q, s, z


def _routes(g, t, e, k):
    """Distinct experts of each token, unevenly loaded, and their weights."""
    logits = torch.randn(t, e, generator=g, device="cuda")
    logits = logits + 0.5 * torch.randn(e, generator=g, device="cuda")
    top, idx = torch.topk(torch.softmax(logits, -1), k, dim=-1)
    return idx.to(torch.int32), top / top.sum(-1, keepdim=True)


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


def _new(n, k, kind):
    return torch.zeros(n, k, dtype=kind if isinstance(kind, torch.dtype) else TYPES[kind],
                       device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op in ("w4_mm", "w4_mm_grouped"):
        grouped = op == "w4_mm_grouped"
        n, k = case["rows"], case["cols"]
        m = case["n_rows"] if grouped else case["tokens"]
        q, s, z = _w4(g, case["experts"] if grouped else 1, n, k, case["group"], case["zeros"],
                      TYPES[case["scale"]])
        sizes = _sizes(g, case) if grouped else [m]
        offsets = [0]
        for c in sizes:
            offsets.append(offsets[-1] + c)
        st.update(w=q, s=s, z=z, sizes=sizes, x=_activations(g, m, k, TYPES[case["type"]]),
                  offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                  y=_new(m, n, case["out"]))
        return st
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if op == "route":
        logits = 1.5 * torch.randn(t, e, generator=g, device="cuda")
        logits = logits + 0.5 * torch.randn(e, generator=g, device="cuda")
        if case["masked"]:  # experts that a token may not take; one is always left
            off = torch.rand(t, e, generator=g, device="cuda") < 0.5
            off[:, 0] = False
            logits = logits.masked_fill(off, -math.inf)
        st.update(logits=logits.to(TYPES[case["type"]]),
                  idx=_new(t, k, torch.int32), w=_new(t, k, "f32"))
        if case["train"]:
            st.update(grad_w=torch.randn(t, k, generator=g, device="cuda"),
                      grad_logits=_new(t, e, case["type"]))
        return st
    idx, w = _routes(g, t, e, k)
    if case["pad"]:
        idx[torch.rand(t, k, generator=g, device="cuda") < case["pad"]] = -1
    h, dt = case["cols"], TYPES[case["type"]]
    if op == "permute":
        st.update(x=_activations(g, t, h, dt), idx=idx, rows=_new(t * k, h, dt),
                  offsets=_new(1, e + 1, torch.int32)[0], pos=_new(t, k, torch.int32))
        if case["train"]:
            st.update(grad_rows=torch.randn(t * k, h, generator=g, device="cuda").to(dt),
                      grad_x=_new(t, h, dt))
        if own:
            import moe_ffn_gb300 as qm
            st["ws"] = torch.empty(qm.moe_permute_workspace_size(t, e, k), dtype=torch.uint8,
                                   device="cuda")
        return st
    # combine: the rows lie as a sort by expert leaves them
    flat = idx.reshape(-1).long()
    order = torch.argsort(torch.where(flat < 0, e, flat), stable=True)
    pos = torch.empty_like(flat)
    pos[order] = torch.arange(t * k, device="cuda")
    pos[flat < 0] = -1
    st.update(y=torch.randn(t * k, h, generator=g, device="cuda").to(dt), w=w,
              pos=pos.to(torch.int32).view(t, k),
              residual=torch.randn(t, h, generator=g, device="cuda").to(TYPES[case["out"]]),
              out_=_new(t, h, case["out"]))
    if case["train"]:
        st.update(grad_out=torch.randn(t, h, generator=g, device="cuda").to(TYPES[case["out"]]),
                  grad_y=_new(t * k, h, dt), grad_w=_new(t, k, "f32"))
    return st


# -------------------------------------------------------------- plain forms
def _plain_route(st):
    x, k = st["logits"].float(), st["top_k"]
    e = torch.exp(x - x.amax(-1, keepdim=True))
    idx = torch.argsort(x, dim=-1, descending=True, stable=True)[:, :k]
    top = torch.gather(e, 1, idx)
    w = top / (top if st["renorm"] else e).sum(-1, keepdim=True)
    if not st["train"]:
        return idx.to(torch.int32), w
    d = st["grad_w"]
    c = (w * d).sum(-1, keepdim=True)
    if st["renorm"]:
        grad = torch.zeros_like(x).scatter_(1, idx, w * (d - c))
    else:
        p = e / e.sum(-1, keepdim=True)
        grad = p * (torch.zeros_like(x).scatter_(1, idx, d) - c)
    return idx.to(torch.int32), w, grad.to(st["logits"].dtype)


def _plain_permute(st):
    t, k, e = st["tokens"], st["top_k"], st["experts"]
    flat = st["idx"].reshape(-1).long()
    order = torch.argsort(torch.where(flat < 0, e, flat), stable=True)
    count = (flat[:, None] == torch.arange(e, device=flat.device)).sum(0)
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(count, 0)
    pos = torch.empty_like(flat)
    pos[order] = torch.arange(t * k, device=flat.device)
    pos = torch.where(flat < 0, -1, pos)
    rows = st["x"][order // k] * (torch.arange(t * k, device=flat.device) < offsets[e])[:, None]
    got = (rows, offsets.to(torch.int32), pos.to(torch.int32).view(t, k))
    if not st["train"]:
        return got
    g = st["grad_rows"].float()[pos.clamp(min=0)] * (pos >= 0)[:, None]
    return got + (g.view(t, k, -1).sum(1).to(st["x"].dtype),)


def _plain_combine(st):
    t, k = st["tokens"], st["top_k"]
    pos, live = st["pos"].long().clamp(min=0), st["pos"] >= 0
    w = torch.where(live, st["w"], 0.0)
    y = st["y"].float()[pos]
    out = (st["residual"].float() + (y * w[:, :, None]).sum(1)).to(st["out_"].dtype)
    if not st["train"]:
        return out
    g = st["grad_out"].float()
    grad_y = torch.zeros(t * k, st["cols"], device=g.device)
    grad_y[pos[live]] = (g[:, None, :] * w[:, :, None])[live]
    grad_w = torch.where(live, (y * g[:, None, :]).sum(-1), 0.0)
    return out, grad_y.to(st["y"].dtype), grad_w


def _plain_codes(q):
    return torch.stack((q & 15, q >> 4), -1).view(q.shape[0], -1)


def _plain_w4(st):
    at, parts = 0, []
    for i, c in enumerate(st["sizes"]):
        if c == 0:
            continue
        q = _plain_codes(st["w"][i]).float().view(st["rows"], -1, st["group"])
        z = st["z"][i].float()[:, :, None] if st["zeros"] else 8.0
        w = ((q - z) * st["s"][i].float()[:, :, None]).view(st["rows"], -1)
        parts.append(st["x"][at:at + c].float() @ w.T)
        at += c
    return torch.cat(parts).to(st["y"].dtype)


PLAIN = {"route": _plain_route, "permute": _plain_permute, "combine": _plain_combine,
         "w4_mm": _plain_w4, "w4_mm_grouped": _plain_w4}


# ------------------------------------------------------------ the library's
def _run_own(st):
    import moe_ffn_gb300 as qm
    kinds = {torch.float32: qm.F32, torch.bfloat16: qm.BF16, torch.float16: qm.F16}
    op = st["op"]
    if op == "w4_mm":
        qm.w4_mm(st["w"], kinds[st["s"].dtype], st["s"], st["z"], st["group"], st["rows"],
                 st["cols"], kinds[st["x"].dtype], st["x"], st["tokens"], kinds[st["y"].dtype],
                 st["y"])
        return st["y"]
    if op == "w4_mm_grouped":
        qm.w4_mm_grouped(st["w"], kinds[st["s"].dtype], st["s"], st["z"], st["group"],
                         st["experts"], st["rows"], st["cols"], kinds[st["x"].dtype], st["x"],
                         st["n_rows"], st["offsets"], kinds[st["y"].dtype], st["y"])
        return st["y"]
    t, e, k = st["tokens"], st["experts"], st["top_k"]
    if op == "route":
        kind = kinds[st["logits"].dtype]
        qm.moe_route(kind, st["logits"], t, e, k, st["idx"], st["w"], renormalize=st["renorm"])
        if not st["train"]:
            return st["idx"], st["w"]
        qm.moe_route_backward(kind, st["logits"], t, e, k, st["idx"], st["w"], st["grad_w"],
                              st["grad_logits"], renormalize=st["renorm"])
        return st["idx"], st["w"], st["grad_logits"]
    if op == "permute":
        kind = kinds[st["x"].dtype]
        qm.moe_permute(kind, st["x"], t, st["cols"], st["idx"], e, k, st["rows"], st["offsets"],
                       st["pos"], st["ws"])
        got = (st["rows"], st["offsets"], st["pos"])
        if not st["train"]:
            return got
        qm.moe_combine(kind, st["grad_rows"], t * k, st["cols"], st["pos"], None, t, k, kind, None,
                       st["grad_x"])
        return got + (st["grad_x"],)
    ykind, okind = kinds[st["y"].dtype], kinds[st["out_"].dtype]
    qm.moe_combine(ykind, st["y"], t * k, st["cols"], st["pos"], st["w"], t, k, okind,
                   st["residual"], st["out_"])
    if not st["train"]:
        return st["out_"]
    qm.moe_combine_backward(ykind, st["y"], t * k, st["cols"], st["pos"], st["w"], t, k, okind,
                            st["grad_out"], st["grad_y"], st["grad_w"])
    return st["out_"], st["grad_y"], st["grad_w"]


def run(state):
    return _run_own(state) if own else PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work
def _active(case):
    """Groups that have rows, as expected of the case's spread."""
    e, n = case["experts"], case["n_rows"]
    if case["spread"] == "uneven":
        return 0.9 * e * (1.0 - (1.0 - 1.0 / e) ** n)
    return min(e, n)


def work(case):
    op, size = case["op"], SIZE[case["type"]]
    if op in ("w4_mm", "w4_mm_grouped"):
        grouped = op == "w4_mm_grouped"
        n, k = case["rows"], case["cols"]
        m = case["n_rows"] if grouped else case["tokens"]
        per = k // 2 + k // case["group"] * (SIZE[case["scale"]] + int(case["zeros"]))
        return {"bytes": int((_active(case) if grouped else 1) * n * per) + m * k * size
                + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if op == "route":
        return {"bytes": t * e * size * (2 if case["train"] else 1)
                + t * k * (12 if case["train"] else 8), "flops": 5 * t * e}
    h = case["cols"]
    live = int(t * k * (1.0 - case["pad"]))
    if op == "permute":
        train = (live + t) * h * size if case["train"] else 0
        return {"bytes": (t + live) * h * size + 8 * t * k + 4 * e + train,
                "flops": live * h if case["train"] else t * k}
    osize = SIZE[case["out"]]
    train = live * h * size + t * h * osize + 4 * t * k if case["train"] else 0
    return {"bytes": live * h * size + 2 * t * h * osize + 8 * t * k + train,
            "flops": (5 if case["train"] else 2) * live * h}


# ------------------------------------------------------------------- exact
def _exact_route(st):
    x, k = st["logits"].double(), st["top_k"]
    t = x.shape[0]
    idx = torch.sort(-x, dim=-1, stable=True).indices[:, :k]
    row = torch.arange(t, device=x.device)[:, None]
    p = torch.softmax(x, -1)
    w = p[row, idx]
    if st["renorm"]:
        w = torch.softmax(x[row, idx], -1)
    if not st["train"]:
        return idx.to(torch.int32), w
    # the Jacobian of the weights, column by column of the selected experts
    d = st["grad_w"].double()
    grad = torch.zeros_like(x)
    for s in range(k):
        ds = d[:, s] * w[:, s]
        if st["renorm"]:
            for j in range(k):
                grad[row[:, 0], idx[:, j]] += ds * ((1.0 if j == s else 0.0) - w[:, j])
        else:
            grad -= ds[:, None] * p
            grad[row[:, 0], idx[:, s]] += ds
    return idx.to(torch.int32), w, grad


def _exact_permute(st):
    t, k, e = st["tokens"], st["top_k"], st["experts"]
    idx = st["idx"].reshape(-1).tolist()
    groups = [[] for _ in range(e)]
    for p, x in enumerate(idx):
        if 0 <= x < e:
            groups[x].append(p)
    offsets, pos, order = [0], [-1] * (t * k), []
    for group in groups:
        for p in group:
            pos[p] = len(order)
            order.append(p)
        offsets.append(len(order))
    at = torch.tensor(order, dtype=torch.int64, device="cuda")
    rows = torch.zeros(t * k, st["cols"], dtype=torch.float64, device="cuda")
    rows[:len(order)] = st["x"].double()[at // k]
    whole = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (offsets, pos)]
    got = (rows, whole[0], whole[1].view(t, k))
    if not st["train"]:
        return got
    grad = torch.zeros(t, st["cols"], dtype=torch.float64, device="cuda")
    grad.index_add_(0, at // k, st["grad_rows"][:len(order)].double())
    return got + (grad,)


def _exact_combine(st):
    t, k = st["tokens"], st["top_k"]
    out = st["residual"].double()
    y, w = st["y"].double(), st["w"].double()
    grad_y, grad_w = torch.zeros_like(y), torch.zeros_like(w)
    g = st["grad_out"].double() if st["train"] else None
    for s in range(k):
        tok = torch.nonzero(st["pos"][:, s] >= 0)[:, 0]
        r = st["pos"][tok, s].long()
        out[tok] += w[tok, s][:, None] * y[r]
        if st["train"]:
            grad_y[r] = w[tok, s][:, None] * g[tok]
            grad_w[tok, s] = (y[r] * g[tok]).sum(-1)
    return (out, grad_y, grad_w) if st["train"] else out


def _exact_w4(st):
    k, at = st["cols"], 0
    col = torch.arange(k, device="cuda")
    y = torch.empty(st["x"].shape[0], st["rows"], dtype=torch.float64, device="cuda")
    for i, c in enumerate(st["sizes"]):
        if c == 0:
            continue
        byte = st["w"][i][:, col // 2].to(torch.int32)
        code = torch.where(col % 2 == 1, byte // 16, byte % 16)
        z = st["z"][i][:, col // st["group"]].to(torch.int32) if st["zeros"] else 8
        w = (code - z).double() * st["s"][i][:, col // st["group"]].double()
        y[at:at + c] = st["x"][at:at + c].double() @ w.T
        at += c
    return y


EXACT = {"route": _exact_route, "permute": _exact_permute, "combine": _exact_combine,
         "w4_mm": _exact_w4, "w4_mm_grouped": _exact_w4}


def exact(case, seed):
    st = prepare(case, seed)
    return EXACT[case["op"]](st)
