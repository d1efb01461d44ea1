"""Rows sorted by expert, the experts' MLP on them and 8-bit integer experts: cases, inputs, plain forms.

Without a capacity ("dropless"), the rows of all experts lie one after the other in one [n, m] buffer:
expert j has the rows offsets[j] .. offsets[j + 1] - 1, its routes in route-priority order (all
tokens' route 0 in token order, then route 1, and so on).  A route with expert -1 (a padded token, an
expert that lives elsewhere) gets no row.

Operators (a case's "op"):
  sort      the routes ordered by expert, and the tokens' rows copied there (times the gate or not)
  combine   the way back: y[t] = sum over the token's routes of gate * row; "train": also its gradient
            (rows and gates) and the gradient of the way in (tokens and gates)
  ffn       the expert MLP on sorted rows, bf16; "train": it also keeps the pre-activation.  The hidden
            and the pre-activation are outputs, stored in bf16; the second product reads the stored hidden
  ffn_bwd   its gradient, from the stored hidden and pre-activation
  product   sorted rows of 8-bit integers times 8-bit weights, a scale for each row and each output channel
  ffn8      tokens quantised to 8-bit integers straight into their sorted rows, then the expert MLP on
            8-bit operands; the hidden, bf16, is quantised by rows in between

8-bit rows: scale = amax / 127, code = round(x * (127 / amax)) to nearest even, in fp32; zeros with
scale 1 where amax < 2^-100.
"""

import math

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of a fine-grained layer: latency
        dict(name="sort 1 token e256", op="sort", s=1, e=256, k=8, m=7168, dtype="bf16", weighted=False, pad=0),
        # the largest batch of the load sweep, its last tokens padding
        dict(name="sort 65536 e64", op="sort", s=65536, e=64, k=2, m=4096, dtype="bf16", weighted=False, pad=500),
        # serving: the weighted way back of a prefill batch, top-3
        dict(name="combine 8192 e16", op="combine", s=8192, e=16, k=3, m=2048, dtype="bf16", train=False, pad=0),
        # training: fine-grained top-8, an odd batch, both ways' gradients
        dict(name="combine train 8191 e256", op="combine", s=8191, e=256, k=8, m=2048, dtype="bf16", train=True,
             pad=0),
        # a few decoded tokens on small gated experts: latency
        dict(name="ffn 5 tokens e64 swiglu", op="ffn", s=5, e=64, k=4, m=1024, h=704, act="swiglu", train=False,
             pad=0),
        # the training forward of a 16-expert top-3 layer
        dict(name="ffn train e16 gelu", op="ffn", s=8192, e=16, k=3, m=2048, h=4096, act="gelu", train=True, pad=0),
        # its gradient
        dict(name="ffn_bwd e16 gelu", op="ffn_bwd", s=8192, e=16, k=3, m=2048, h=4096, act="gelu", pad=0),
        # many small gated experts, uneven, some tokens padding
        dict(name="ffn_bwd e64 swiglu", op="ffn_bwd", s=4100, e=64, k=8, m=1024, h=512, act="swiglu", pad=77),
        # one token through one dense 8-bit projection: the weights' bytes
        dict(name="product 1 row 4096x8192", op="product", s=1, e=1, k=1, cols=4096, n=8192, out="bf16", bias=False,
             pad=0),
        # uneven experts of a prefill chunk, a width that ends inside a tile, fp32 results
        dict(name="product e16 2000x2048x1048", op="product", s=2000, e=16, k=2, cols=2048, n=1048, out="f32",
             bias=True, pad=0),
        # 16 decoded tokens, top-8 of 256 fine-grained experts: the chosen experts' bytes
        dict(name="ffn8 decode e256 swiglu", op="ffn8", s=16, e=256, k=8, m=7168, h=2048, act="swiglu", pad=0),
        # a full layer of 8 GELU experts over 8192 tokens, top-2
        dict(name="ffn8 8192 e8 gelu", op="ffn8", s=8192, e=8, k=2, m=4096, h=8192, act="gelu", pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sort", "combine", "ffn", "ffn_bwd", "product", "ffn8"))
    pad = rng.choice((0, 0, 0.03, 0.3))
    if op in ("sort", "combine"):
        e = rng.choice((1, 4, 16, 60, 64, 128, 256, 512))
        k = rng.randint(1, min(e, 8))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        m = 8 * _log(rng, 8, 900)
        s = max(1, min(_log(rng, 1, 65536), (1 << 27) // (m * k), (1 << 23) // e))
        c = dict(op=op, s=s, e=e, k=k, m=m, dtype=dtype, pad=int(s * pad))
        c["weighted" if op == "sort" else "train"] = rng.random() < 0.5
        return c
    e = rng.choice((1, 2, 8, 16, 60, 64, 128))
    k = rng.randint(1, min(e, 8))
    act = rng.choice(("relu", "gelu", "swiglu"))
    if op in ("ffn", "ffn_bwd"):
        m, h = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 512)
        m = max(64, min(m, (1 << 27) // (e * h) // 8 * 8))
        s = max(1, min(_log(rng, 1, 16384), (1 << 37) // (m * h * k), (1 << 28) // ((m + h) * k)))
        c = dict(op=op, s=s, e=e, k=k, m=m, h=h, act=act, pad=int(s * pad))
        if op == "ffn":
            c["train"] = rng.random() < 0.5
        return c
    m, h = 16 * _log(rng, 4, 320), 16 * _log(rng, 4, 512)
    m = max(64, min(m, (1 << 28) // (e * h) // 16 * 16))
    s = max(1, min(_log(rng, 1, 16384), (1 << 37) // (m * h * k), (1 << 28) // ((m + h) * k)))
    if op == "product":
        n = h + rng.choice((0, 8))
        return dict(op=op, s=s, e=e, k=k, cols=m, n=n, out=rng.choice(("bf16", "f32")), bias=rng.random() < 0.5,
                    pad=int(s * pad))
    return dict(op=op, s=s, e=e, k=k, m=m, h=h, act=act, pad=int(s * pad))


def _routes(case, seed):
    """The chosen experts [k, s] of random tokens, some experts more popular than others; the last
    `pad` tokens have none."""
    s, e, k = case["s"], case["e"], case["k"]
    gen = torch.Generator().manual_seed(seed * 2 + 1)
    like = torch.rand((s, e), generator=gen).neg_().add_(1.0).log_().neg_().log_().neg_()   # Gumbel: random top-k
    like += torch.randn(e, generator=gen) * 0.5
    idx = like.topk(k, dim=1).indices.t().contiguous().int()
    if case["pad"]:
        idx[:, s - case["pad"]:] = -1
    return idx


def _counts(idx, e):
    return torch.bincount(idx[idx >= 0].flatten().long(), minlength=e)


def work(case):
    op, s, e, k = case["op"], case["s"], case["e"], case["k"]
    rows = (s - case["pad"]) * k
    if op in ("sort", "combine"):
        b = case["m"] * (2 if case["dtype"] == "bf16" else 4)
        live = s - case["pad"]
        if op == "sort":
            return {"bytes": s * k * 12 + 4 * e + live * b + rows * (b + (4 if case["weighted"] else 0)),
                    "flops": rows * case["m"] if case["weighted"] else rows}
        fwd = s * b + rows * (b + 8)
        if not case["train"]:
            return {"bytes": fwd, "flops": 2 * rows * case["m"]}
        # y; d_rows and d_gates from dy and the rows; d_x and the way in's d_gates from d_in and x
        return {"bytes": fwd + s * b + rows * (2 * b + 12) + rows * (b + 12) + 2 * s * b,
                "flops": 9 * rows * case["m"]}
    counts = _counts(_routes(case, 0), e)
    used = int((counts > 0).sum())
    if op == "product":
        kk, n = case["cols"], case["n"]
        return {"bytes": used * n * (kk + 4) + rows * (kk + 4 + n * (2 if case["out"] == "bf16" else 4)),
                "flops": 2 * rows * n * kk}
    m, h, mats = case["m"], case["h"], 3 if case["act"] == "swiglu" else 2
    if op == "ffn8":
        return {"bytes": used * mats * m * h + s * m * 2 + rows * m * 2, "flops": 2 * rows * m * h * mats}
    pre = h * (mats - 1)
    if op == "ffn":
        return {"bytes": 2 * (used * mats * m * h + rows * (2 * m + h + (pre if case["train"] else 0))),
                "flops": 2 * rows * m * h * mats}
    return {"bytes": 2 * (used * mats * m * h + e * mats * m * h + rows * (3 * m + h + pre)),
            "flops": 4 * rows * m * h * mats}


# ------------------------------------------------------------------ inputs
def _rows_of(idx, e):
    """Plain form of the sort: rows [k, s], offsets [e + 1], source [k * s] (-1 behind the last row)."""
    k, s = idx.shape
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, e, flat)
    source = torch.argsort(key, stable=True)
    at = torch.empty_like(source)
    at[source] = torch.arange(k * s, device=idx.device)
    counts = torch.zeros(e + 1, dtype=torch.long, device=idx.device).index_add_(0, key, torch.ones_like(key))[:e]
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    live = torch.arange(k * s, device=idx.device) < offsets[-1]
    rows = torch.where(flat < 0, -1, at).view(k, s)
    return rows.int(), offsets.int(), torch.where(live, source, -1).int()


def _weights(gen, shape, dev):
    """bf16 weights of variance 1 / (the last dimension)."""
    w = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    step = max(1, (1 << 27) // (shape[1] * shape[2]))
    for j in range(0, shape[0], step):
        part = w[j:j + step]
        part.copy_(torch.randn(part.shape, generator=gen, device=dev).mul_(shape[2] ** -0.5))
    return w


def _weights8(gen, shape, dev):
    """8-bit weights of variance 1 / (the last dimension) and their scale for each output channel."""
    q = torch.empty(shape, dtype=torch.int8, device=dev)
    scale = torch.empty(shape[:2], device=dev)
    step = max(1, (1 << 27) // (shape[1] * shape[2]))
    for j in range(0, shape[0], step):
        part = q[j:j + step]
        w = torch.randn(part.shape, generator=gen, device=dev).mul_(shape[2] ** -0.5)
        q[j:j + step], scale[j:j + step] = _quantize(w)
    return q, scale


def _tokens(gen, s, m, dev):
    """Activations: a few channels and tokens much larger than the rest."""
    x = torch.randn((s, m), generator=gen, device=dev)
    x *= torch.exp(torch.randn(m, generator=gen, device=dev) * 0.4)
    return x.mul_(torch.exp(torch.randn((s, 1), generator=gen, device=dev) * 0.3))


def prepare(case, seed):
    dev, op = "cuda", case["op"]
    gen = torch.Generator(device=dev).manual_seed(seed)
    s, e, k = case["s"], case["e"], case["k"]
    idx = _routes(case, seed)
    st = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=dev), "idx": idx.to(dev), "n": s * k}
    st["counts"] = _counts(idx, e).tolist()   # the plain forms' loop over experts
    gates = torch.rand((s, k), generator=gen, device=dev) + 0.05
    st["gates"] = (gates / gates.sum(1, keepdim=True)).t().contiguous()
    st["rows"], st["offsets"], st["source"] = _rows_of(st["idx"], e)
    n = s * k
    if op in ("sort", "combine"):
        m, dt = case["m"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["x"] = _tokens(gen, s, m, dev).to(dt)
        st["xs"] = torch.zeros((n, m), dtype=dt, device=dev)
        if op == "combine":
            st["xs"] = torch.randn((n, m), generator=gen, device=dev).to(dt)
            st["y"] = torch.zeros((s, m), dtype=dt, device=dev)
            if case["train"]:
                st["dy"] = torch.randn((s, m), generator=gen, device=dev).to(dt)
                st["d_in"] = torch.randn((n, m), generator=gen, device=dev).to(dt)   # gradient of the way in's rows
                st["d_xs"] = torch.zeros((n, m), dtype=dt, device=dev)
                st["dx"] = torch.zeros((s, m), dtype=dt, device=dev)
                st["d_gates"], st["d_gates_in"] = torch.zeros((2, k, s), device=dev).unbind(0)
        return st
    if op == "product":
        st["a"] = _quantize(_tokens(gen, n, case["cols"], dev))
        st["w"] = _weights8(gen, (e, case["n"], case["cols"]), dev)
        st["b"] = torch.randn((e, case["n"]), generator=gen, device=dev).mul_(0.1).bfloat16() if case["bias"] else None
        st["out"] = torch.zeros((n, case["n"]), dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32,
                                device=dev)
        return st
    m, h, act = case["m"], case["h"], case["act"]
    wide = 2 * h if act == "swiglu" else h
    make = _weights8 if op == "ffn8" else _weights
    st["w1"] = make(gen, (e, h, m), dev)
    st["w3"] = make(gen, (e, h, m), dev) if act == "swiglu" else None
    st["w2"] = make(gen, (e, m, h), dev)
    st["b1"] = st["b2"] = None
    if act != "swiglu":
        st["b1"] = torch.randn((e, h), generator=gen, device=dev).mul_(0.1).bfloat16()
        st["b2"] = torch.randn((e, m), generator=gen, device=dev).mul_(0.1).bfloat16()
    st["out"] = torch.zeros((n, m), dtype=torch.bfloat16, device=dev)
    if op == "ffn8":
        st["x"] = _tokens(gen, s, m, dev).bfloat16()
        st["q"] = torch.zeros((n, m), dtype=torch.int8, device=dev)
        st["scale"] = torch.zeros(n, device=dev)
        return st
    st["x"] = _tokens(gen, n, m, dev).bfloat16()
    st["hid"] = torch.zeros((n, h), dtype=torch.bfloat16, device=dev)
    st["pre"] = torch.zeros((n, wide), dtype=torch.bfloat16, device=dev)
    if op == "ffn_bwd":
        _plain_ffn(st, st["hid"], st["pre"], None)   # what the training forward kept
        st["d_out"] = torch.randn((n, m), generator=gen, device=dev).bfloat16()
        st["dx"] = torch.zeros((n, m), dtype=torch.bfloat16, device=dev)
        for name in ("w1", "w2", "b1", "b2") if act != "swiglu" else ("w1", "w3", "w2"):
            st["d_" + name] = torch.zeros_like(st[name])
    return st


# --------------------------------------------------------------- one pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _space(st, name, n):
    """A buffer of n bytes that the program keeps with its plan."""
    if name not in st:
        st[name] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st[name]


def _run_own(st):
    import combine_moe_gate_gb300 as M

    case, status, op = st["case"], st["status"], st["case"]["op"]
    e, n = case["e"], st["n"]
    if op == "sort":
        if "out_rows" not in st:
            st["out_rows"], st["out_offsets"], st["out_source"] = map(torch.empty_like, (st["rows"], st["offsets"],
                                                                                         st["source"]))
        ws = _space(st, "ws", M.moe_sort_workspace_size(case["s"], e, case["k"]))
        M.moe_sort_routes(st["idx"], e, st["out_rows"], st["out_offsets"], ws, status, source=st["out_source"])
        M.moe_encode_sorted(st["x"], st["out_rows"], st["xs"], status, gates=st["gates"] if case["weighted"] else None)
        return {"rows": st["out_rows"], "offsets": st["out_offsets"], "source": st["out_source"], "xs": st["xs"]}
    if op == "combine":
        M.moe_decode_sorted(st["xs"], st["rows"], st["y"], status, gates=st["gates"])
        if not case["train"]:
            return {"y": st["y"]}
        M.moe_decode_sorted_bwd(st["dy"], st["xs"], st["rows"], st["gates"], st["d_xs"], st["d_gates"], status)
        M.moe_encode_sorted_bwd(st["d_in"], st["rows"], st["dx"], status, x=st["x"], gates=st["gates"],
                                d_gates=st["d_gates_in"])
        return {name: st[name] for name in ("y", "d_xs", "d_gates", "dx", "d_gates_in")}
    if op == "product":
        (aq, asc), (wq, wsc) = st["a"], st["w"]
        ws = _space(st, "ws", M.moe_product_int8_workspace_size(e, n, case["cols"], case["n"]))
        M.moe_product_int8(aq, asc, st["offsets"], wq, wsc, st["b"], ws, st["out"], status)
        return st["out"]
    m, h, act = case["m"], case["h"], case["act"]
    if op == "ffn8":
        ws = _space(st, "ws", M.moe_expert_ffn_int8_workspace_size(act, e, n, m, h))
        M.moe_quantize_rows_int8(st["x"], st["q"], st["scale"], status, rows=st["rows"])
        w3 = st["w3"] or (None, None)
        M.moe_expert_ffn_int8(st["q"], st["scale"], st["offsets"], *st["w1"], st["b1"], *w3, *st["w2"], st["b2"], act,
                              ws, st["out"], status)
        return st["out"]
    if op == "ffn":
        M.moe_expert_ffn_sorted(st["x"], st["offsets"], st["w1"], st["b1"], st["w3"], st["w2"], st["b2"], act,
                                st["hid"], st["out"], status, pre=st["pre"] if case["train"] else None)
        return {name: st[name] for name in (("out", "hid", "pre") if case["train"] else ("out",))}
    ws = _space(st, "ws", M.moe_expert_ffn_sorted_bwd_workspace_size(act, e, n, m, h))
    M.moe_expert_ffn_sorted_bwd(st["x"], st["hid"], st["pre"], st["offsets"], st["w1"], st["w3"], st["w2"], act,
                                st["d_out"], ws, st["dx"], st["d_w1"], st.get("d_w3"), st["d_w2"], st.get("d_b1"),
                                st.get("d_b2"), status)
    return {name: st[name] for name in ("dx", "d_w1", "d_w3", "d_w2", "d_b1", "d_b2") if name in st}


def _quantize(x):
    """fp32 rows -> 8-bit codes and a scale for each row."""
    amax = x.abs().amax(-1)
    live = amax >= 2.0 ** -100
    scale = torch.where(live, amax / 127.0, 1.0)
    inv = torch.where(live, 127.0 / amax, 0.0)
    return (x * inv[..., None]).round_().to(torch.int8), scale


def _act(a, b, act):
    if act == "relu":
        return torch.clamp(a, min=0.0)
    if act == "gelu":
        return a * 0.5 * (1.0 + torch.erf(a * 0.5 ** 0.5))
    return a / (1.0 + torch.exp(-a)) * b


def _experts(st):
    """(expert, its first row, its end) of the experts that have rows."""
    at = 0
    for j, c in enumerate(st["counts"]):
        if c:
            yield j, at, at + c
        at += c


def _plain_ffn(st, hid, pre, out):
    act = st["case"]["act"]
    for j, lo, hi in _experts(st):
        x = st["x"][lo:hi].float()
        a, b = x @ st["w1"][j].float().t(), None
        if st["b1"] is not None:
            a += st["b1"][j].float()
        if act == "swiglu":
            b = x @ st["w3"][j].float().t()
        if pre is not None:
            pre[lo:hi] = a if b is None else torch.cat((a, b), 1)
        hid[lo:hi] = _act(a, b, act)
        if out is not None:
            y = hid[lo:hi].float() @ st["w2"][j].float().t()
            out[lo:hi] = y if st["b2"] is None else y + st["b2"][j].float()


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    e, n, s, k = case["e"], st["n"], case["s"], case["k"]
    if op == "sort":
        rows, offsets, source = _rows_of(st["idx"], e)
        live = (source >= 0)[:, None]
        at = source.clamp(min=0).long()
        xs = st["x"].float()[at % s]
        if case["weighted"]:
            xs = xs * st["gates"].view(-1)[at][:, None]
        return {"rows": rows, "offsets": offsets, "source": source,
                "xs": torch.where(live, xs, 0.0).to(st["x"].dtype)}
    if op == "combine":
        rows, dt = st["rows"], st["x"].dtype
        live = rows >= 0
        at = rows.clamp(min=0).long()
        xs = st["xs"].float()
        g = torch.where(live, st["gates"], 0.0)
        y = torch.zeros((s, case["m"]), device=xs.device)
        for r in range(k):
            y += g[r][:, None] * xs[at[r]]
        out = {"y": y.to(dt)}
        if not case["train"]:
            return out
        dy, x, d_in = st["dy"].float(), st["x"].float(), st["d_in"].float()
        d_xs = torch.zeros((n + 1, case["m"]), device=xs.device)   # the last row takes the routes without one
        d_gates, d_gates_in, dx = torch.zeros_like(g), torch.zeros_like(g), torch.zeros_like(x)
        to = torch.where(live, rows, n).long()
        for r in range(k):
            d_xs[to[r]] = g[r][:, None] * dy
            d_gates[r] = (dy * xs[at[r]]).sum(1) * live[r]
            dx += g[r][:, None] * d_in[at[r]]
            d_gates_in[r] = (x * d_in[at[r]]).sum(1) * live[r]
        out.update(d_xs=d_xs[:n].to(dt), d_gates=d_gates, dx=dx.to(dt), d_gates_in=d_gates_in)
        return out
    if op == "product":
        (aq, asc), (wq, wsc) = st["a"], st["w"]
        out = torch.zeros_like(st["out"])
        for j, lo, hi in _experts(st):
            y = (aq[lo:hi].float() @ wq[j].float().t()) * asc[lo:hi, None] * wsc[j]
            out[lo:hi] = y if st["b"] is None else y + st["b"][j].float()
        return out
    act = case["act"]
    if op == "ffn8":
        q, scale = _quantize(st["x"].float())
        token = st["source"].clamp(min=0).long() % s
        out = torch.zeros_like(st["out"])
        for j, lo, hi in _experts(st):
            x, sx = q[token[lo:hi]].float(), scale[token[lo:hi], None]
            a, b = (x @ st["w1"][0][j].float().t()) * sx * st["w1"][1][j], None
            if st["b1"] is not None:
                a += st["b1"][j].float()
            if act == "swiglu":
                b = (x @ st["w3"][0][j].float().t()) * sx * st["w3"][1][j]
            hq, hs = _quantize(_act(a, b, act).bfloat16().float())
            y = (hq.float() @ st["w2"][0][j].float().t()) * hs[:, None] * st["w2"][1][j]
            out[lo:hi] = y if st["b2"] is None else y + st["b2"][j].float()
        return out
    if op == "ffn":
        out, hid = torch.zeros_like(st["out"]), torch.zeros_like(st["hid"])
        pre = torch.zeros_like(st["pre"]) if case["train"] else None
        _plain_ffn(st, hid, pre, out)
        return {"out": out, "hid": hid, "pre": pre} if case["train"] else {"out": out}
    h = case["h"]
    res = {"dx": torch.zeros_like(st["dx"])}
    for name in ("d_w1", "d_w3", "d_w2", "d_b1", "d_b2"):
        if name in st:
            res[name] = torch.zeros_like(st[name])
    for j, lo, hi in _experts(st):
        x, hid, pre = st["x"][lo:hi].float(), st["hid"][lo:hi].float(), st["pre"][lo:hi].float()
        do = st["d_out"][lo:hi].float()
        dh = do @ st["w2"][j].float()
        res["d_w2"][j] = do.t() @ hid
        if act == "swiglu":
            a, b = pre[:, :h], pre[:, h:]
            sg = 1.0 / (1.0 + torch.exp(-a))
            da, db = dh * b * sg * (1.0 + a * (1.0 - sg)), dh * a * sg
            res["d_w3"][j] = db.t() @ x
            dx = da @ st["w1"][j].float() + db @ st["w3"][j].float()
        else:
            if act == "relu":
                da = dh * (pre > 0)
            else:
                cdf = 0.5 * (1.0 + torch.erf(pre * 0.5 ** 0.5))
                da = dh * (cdf + pre * torch.exp(-0.5 * pre * pre) * (2.0 * math.pi) ** -0.5)
            dx = da @ st["w1"][j].float()
            res["d_b1"][j] = da.sum(0)
            res["d_b2"][j] = do.sum(0)
        res["d_w1"][j] = da.t() @ x
        res["dx"][lo:hi] = dx
    return res


# ---------------------------------------------------- the operators in 64 bits
def _exact_sort(idx, e):
    """Row of each route, offsets and source, expert by expert."""
    k, s = idx.shape
    flat = idx.flatten().long()
    rows = torch.full((k * s,), -1, device=idx.device)
    source = torch.full((k * s,), -1, device=idx.device)
    offsets = [0]
    for j in range(e):
        mine = torch.nonzero(flat == j).flatten()   # ascending: route-priority order
        to = torch.arange(len(mine), device=idx.device) + offsets[-1]
        rows[mine] = to
        source[to] = mine
        offsets.append(offsets[-1] + len(mine))
    return rows.view(k, s).int(), torch.tensor(offsets, device=idx.device).int(), source.int(), offsets


def _exact_quantize(x):
    """Values that the 8-bit rows stand for, as (codes, scales), the fp32 steps of the definition in 64 bits."""
    amax = x.abs().amax(-1, keepdim=True)
    scale, inv = (amax / 127.0).float().double(), (127.0 / amax).float().double()
    code = torch.round((x * inv).float().double())
    none = amax < 2.0 ** -100
    return torch.where(none, 0.0, code), torch.where(none, 1.0, scale)


def _exact_act(a, b, act):
    if act == "relu":
        return torch.nn.functional.relu(a)
    return torch.nn.functional.gelu(a) if act == "gelu" else torch.nn.functional.silu(a) * b


def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e12 and case["op"] not in ("sort", "combine"):
        return None   # more than the card's 64-bit units do in the time
    st = prepare(case, seed)
    op, s, e, k, n = case["op"], case["s"], case["e"], case["k"], st["n"]
    rows, offsets, source, off = _exact_sort(st["idx"], e)
    if op == "sort":
        xs = torch.zeros((n, case["m"]), dtype=torch.float64, device="cuda")
        for r in range(k):
            for t0 in range(0, s, 16384):
                at = rows[r, t0:t0 + 16384].long()
                part = st["x"][t0:t0 + 16384].double()
                if case["weighted"]:
                    part = part * st["gates"][r, t0:t0 + 16384, None].double()
                xs[at[at >= 0]] = part[at >= 0]
        return {"rows": rows, "offsets": offsets, "source": source, "xs": xs}
    if op == "combine":
        m = case["m"]
        pad = torch.zeros((1, m), dtype=torch.float64, device="cuda")
        xs = torch.cat((st["xs"].double(), pad))            # row n: what a route without a row reads
        at = torch.where(rows < 0, n, rows).long()
        gates = st["gates"].double()
        res = {"y": torch.einsum("ks,ksm->sm", gates, xs[at]) if n * m < 1 << 24 else
               sum(gates[r, :, None] * xs[at[r]] for r in range(k))}
        if case["train"]:
            dy, x, d_in = st["dy"].double(), st["x"].double(), torch.cat((st["d_in"].double(), pad))
            res["d_gates"] = torch.stack([torch.einsum("sm,sm->s", dy, xs[at[r]]) for r in range(k)])
            res["d_gates_in"] = torch.stack([torch.einsum("sm,sm->s", x, d_in[at[r]]) for r in range(k)])
            res["dx"] = sum(gates[r, :, None] * d_in[at[r]] for r in range(k))
            d_xs = torch.zeros_like(xs)
            for r in range(k):
                d_xs[at[r]] = gates[r, :, None] * dy
            res["d_xs"] = d_xs[:n]
        return res
    act = case.get("act")
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    if op == "product":
        (aq, asc), (wq, wsc) = st["a"], st["w"]
        for j in range(e):
            mine = slice(off[j], off[j + 1])
            vals = aq[mine].double() * asc[mine, None].double()
            out[mine] = vals @ (wq[j].double() * wsc[j, :, None].double()).t()
            if st["b"] is not None:
                out[mine] += st["b"][j].double()
        return out
    if op == "ffn8":
        q, sc = _exact_quantize(st["x"].double())
        x = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        live = source[source >= 0].long() % s
        x[:len(live)] = (q * sc)[live]
        for j in range(e):
            mine = slice(off[j], off[j + 1])
            if off[j] == off[j + 1]:
                continue
            up = x[mine] @ (st["w1"][0][j].double() * st["w1"][1][j, :, None].double()).t()
            if st["b1"] is not None:
                up += st["b1"][j].double()
            side = x[mine] @ (st["w3"][0][j].double() * st["w3"][1][j, :, None].double()).t() if act == "swiglu" else None
            hq, hs = _exact_quantize(_exact_act(up, side, act).bfloat16().double())
            out[mine] = (hq * hs) @ (st["w2"][0][j].double() * st["w2"][1][j, :, None].double()).t()
            if st["b2"] is not None:
                out[mine] += st["b2"][j].double()
        return out
    if op == "ffn":
        hid = torch.zeros(st["hid"].shape, dtype=torch.float64, device="cuda")
        pre = torch.zeros(st["pre"].shape, dtype=torch.float64, device="cuda")
        for j in range(e):
            mine = slice(off[j], off[j + 1])
            x = st["x"][mine].double()
            up = x @ st["w1"][j].double().t()
            if act == "swiglu":
                side = x @ st["w3"][j].double().t()
                pre[mine, :case["h"]], pre[mine, case["h"]:] = up, side
            else:
                up, side = up + st["b1"][j].double(), None
                pre[mine] = up
            hid[mine] = _exact_act(up, side, act)
            out[mine] = hid[mine].bfloat16().double() @ st["w2"][j].double().t()
            if st["b2"] is not None:
                out[mine] += st["b2"][j].double()
        return {"out": out, "hid": hid, "pre": pre} if case["train"] else {"out": out}
    # the gradient by differentiating the MLP from its pre-activation on
    h = case["h"]
    res = {name: torch.zeros(st[name].shape, dtype=torch.float64, device="cuda")
           for name in ("dx", "d_w1", "d_w3", "d_w2", "d_b1", "d_b2") if name in st}
    for j in range(e):
        mine = slice(off[j], off[j + 1])
        x, d_out = st["x"][mine].double(), st["d_out"][mine].double()
        pre = st["pre"][mine].double().requires_grad_(True)
        with torch.enable_grad():
            hid = _exact_act(pre[:, :h], pre[:, h:], act) if act == "swiglu" else _exact_act(pre, None, act)
            (d_pre,) = torch.autograd.grad(hid, pre, d_out @ st["w2"][j].double())
        res["d_w2"][j] = torch.einsum("rm,rh->mh", d_out, st["hid"][mine].double())
        if act == "swiglu":
            both = torch.cat((st["w1"][j], st["w3"][j])).double()
            res["dx"][mine] = d_pre @ both
            grads = d_pre.t() @ x
            res["d_w1"][j], res["d_w3"][j] = grads[:h], grads[h:]
        else:
            res["dx"][mine] = d_pre @ st["w1"][j].double()
            res["d_w1"][j] = d_pre.t() @ x
            res["d_b1"][j], res["d_b2"][j] = d_pre.sum(0), d_out.sum(0)
    return res
