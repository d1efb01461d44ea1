"""The routing and 4-bit expert operators, as a program calls them: cases, inputs, plain forms.

Operators (a case's "op"):
  route      scores of router logits (softmax or sigmoid), a balance bias that selects but does not
             weigh, group-limited top-k, renormalised and scaled gates
  route_bwd  its gradient with respect to the logits
  quantize   bf16 rows to microscaled 4-bit floats (e2m1 codes with block scales) and back
  product    the grouped product of 4-bit rows with 4-bit weights, over each expert's kept rows
  ffn        the expert MLP on 4-bit operands: the rows quantised, both products, the hidden
             quantised in between

Formats: "mx" has blocks of 32 with one power-of-two scale (e8m0); "nv" has blocks of 16 with one
e4m3 scale and one fp32 factor per expert.  Block scales are stored in tiles of 128 rows x 4 blocks
(32 rows of 16 bytes: row r, block b at (r % 32) * 16 + (r / 32) * 4 + b), row tiles outermost.
"""

import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a fine-grained layer being decoded: latency of the router
        dict(name="route 1 token e256 sigmoid", op="route", s=1, e=256, k=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, scale=2.5, norm=True, dtype="f32", masked=0),
        # a prefill batch of the same layer
        dict(name="route 16384 e256 sigmoid", op="route", s=16384, e=256, k=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, scale=2.5, norm=True, dtype="f32", masked=0),
        # the largest sweep batch, top-2 softmax on bf16 logits, a few experts masked out
        dict(name="route 65536 e64 softmax", op="route", s=65536, e=64, k=2, score="softmax", bias=False,
             groups=1, topk_groups=1, group_top=1, scale=1.0, norm=True, dtype="bf16", masked=5),
        # training: the fine-grained layer's router gradient
        dict(name="route_bwd 16384 e256 sigmoid", op="route_bwd", s=16384, e=256, k=8, score="sigmoid",
             scale=2.5, norm=True, dtype="f32"),
        # training with raw softmax gates; odd sizes, so rows start off the 16-byte grid
        dict(name="route_bwd 8191 e60 softmax", op="route_bwd", s=8191, e=60, k=4, score="softmax",
             scale=1.0, norm=False, dtype="bf16"),
        # the rows of an expert buffer before a 4-bit layer, some experts partly filled
        dict(name="quantize nv 8x2048x4096", op="quantize", fmt="nv", e=8, c=2048, cols=4096, fill="ragged"),
        # a handful of decoded tokens; the last scale tile is partly used in both directions
        dict(name="quantize mx 1x37x2080", op="quantize", fmt="mx", e=1, c=37, cols=2080, fill="full"),
        # one dense 4-bit projection over a prefill chunk
        dict(name="product nv 1x4096x4096x8192", op="product", fmt="nv", e=1, c=4096, k=4096, n=8192,
             bias=False, fill="full"),
        # many experts, few uneven rows each, a width that ends inside a tile
        dict(name="product mx 16x300x2048x1056", op="product", fmt="mx", e=16, c=300, k=2048, n=1056,
             bias=True, fill="ragged"),
        # 16 decoded tokens over 256 fine-grained experts, top-8: the weights' bytes count
        dict(name="ffn decode nv e256 swiglu", op="ffn", fmt="nv", e=256, c=16, m=7168, h=2048, act="swiglu",
             fill="routed", tokens=16, topk=8),
        # a full layer of 8 GELU experts over 8192 tokens, top-2
        dict(name="ffn nv e8 gelu", op="ffn", fmt="nv", e=8, c=2048, m=4096, h=8192, act="gelu",
             fill="ragged", tokens=0, topk=0),
        # the smallest layer
        dict(name="ffn mx e4 relu", op="ffn", fmt="mx", e=4, c=64, m=64, h=160, act="relu",
             fill="ragged", tokens=0, topk=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route", "route_bwd", "quantize", "product", "ffn", "ffn"))
    if op in ("route", "route_bwd"):
        e = rng.choice((8, 16, 60, 64, 96, 128, 160, 256, 384, 512))
        s = max(1, min(_log(rng, 1, 65536), (1 << 24) // e))
        k = rng.randint(1, min(e, 10))
        c = dict(op=op, s=s, e=e, k=k, score=rng.choice(("softmax", "sigmoid")),
                 scale=rng.choice((1.0, 2.5)), norm=rng.random() < 0.7, dtype=rng.choice(("f32", "bf16")))
        if op == "route":
            groups = rng.choice([g for g in (1, 1, 2, 4, 8) if e % g == 0 and e // g >= 2])
            keep = rng.choice([t for t in (1, 2, 3, 4, 8) if t <= groups and t * (e // groups) >= k])
            c.update(bias=rng.random() < 0.6, groups=groups, topk_groups=keep,
                     group_top=rng.choice((1, 2)), masked=rng.choice((0, 0, 3)))
        return c
    fmt = rng.choice(("mx", "nv"))
    if op == "quantize":
        cols = 32 * _log(rng, 1, 512)
        c = _log(rng, 1, 16384)
        e = rng.choice((1, 1, 3, 8, 16))
        c = max(1, min(c, (1 << 26) // (cols * e)))
        return dict(op=op, fmt=fmt, e=e, c=c, cols=cols, fill=rng.choice(("full", "ragged")))
    e = rng.choice((1, 2, 4, 8, 16, 32))
    c = _log(rng, 1, 4096)
    if op == "product":
        k, n = 32 * _log(rng, 2, 256), 32 * _log(rng, 2, 256)
        c = max(1, min(c, (1 << 37) // (k * n * e)))
        return dict(op=op, fmt=fmt, e=e, c=c, k=k, n=n, bias=rng.random() < 0.5,
                    fill=rng.choice(("full", "ragged")))
    m, h = 32 * _log(rng, 2, 224), 32 * _log(rng, 2, 256)
    c = max(1, min(c, (1 << 38) // (m * h * e * 3)))
    return dict(op=op, fmt=fmt, e=e, c=c, m=m, h=h, act=rng.choice(("relu", "gelu", "swiglu")),
                fill=rng.choice(("full", "ragged")), tokens=0, topk=0)


def _kept(case, seed):
    """Kept rows of each expert, as a list."""
    e, c = case["e"], case["c"]
    if case["fill"] == "full":
        return [c] * e
    g = torch.Generator().manual_seed(seed)
    if case["fill"] == "routed":   # tokens choosing topk different experts each
        counts = [0] * e
        for _ in range(case["tokens"]):
            for j in torch.randperm(e, generator=g)[: case["topk"]].tolist():
                counts[j] += 1
        return counts
    lo = torch.rand(e, generator=g)
    counts = [min(c, int(c * (0.5 + float(v)))) for v in lo]   # half of the experts are full
    if e > 2:
        counts[1] = 0   # and one has nothing
    return counts


def _blk(fmt):
    return 32 if fmt == "mx" else 16


def work(case):
    op = case["op"]
    if op == "route":
        b = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["s"] * (case["e"] * b + case["k"] * 8) + (4 * case["e"] if case["bias"] else 0),
                "flops": 4 * case["s"] * case["e"]}
    if op == "route_bwd":
        b = 4 if case["dtype"] == "f32" else 2
        whole = case["score"] == "softmax" and not case["norm"]   # the sum over all logits
        read = case["e"] if whole else case["k"]
        return {"bytes": case["s"] * (read * b + case["e"] * 4 + case["k"] * 8),
                "flops": case["s"] * (4 * read + 8 * case["k"])}
    blk = _blk(case["fmt"])
    unit = 0.5 + 1.0 / blk
    rows = sum(_kept(case, 0))
    if op == "quantize":
        n = rows * case["cols"]
        return {"bytes": n * (2 + unit) + n * (unit + 2), "flops": 4 * n}
    used = sum(1 for r in _kept(case, 0) if r)
    if op == "product":
        k, n = case["k"], case["n"]
        return {"bytes": used * n * k * unit + rows * (k * unit + 2 * n), "flops": 2 * rows * n * k}
    m, h, mats = case["m"], case["h"], 3 if case["act"] == "swiglu" else 2
    return {"bytes": used * mats * m * h * unit + rows * m * 4, "flops": 2 * rows * m * h * mats}


# ----------------------------------------------------------- 4-bit storage
def _tile_scales(sc):
    """[b, rows, blocks] scale bytes -> [b, bytes] in 128 x 4 tiles; zeros after the last block."""
    b, r, n = sc.shape
    rt, nt = -(-r // 128), -(-n // 4)
    full = torch.zeros((b, rt * 128, nt * 4), dtype=torch.uint8, device=sc.device)
    full[:, :r, :n] = sc
    return full.view(b, rt, 4, 32, nt, 4).permute(0, 1, 4, 3, 2, 5).reshape(b, -1).contiguous()


def _untile_scales(t, r, n):
    b = t.shape[0]
    rt, nt = -(-r // 128), -(-n // 4)
    return t.view(b, rt, nt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(b, rt * 128, nt * 4)[:, :r, :n]


def _codes(x, fmt, g):
    """fp32 [b, rows, cols] -> e2m1 codes (uint8, one per value) and scale bytes [b, rows, blocks]."""
    b, r, c = x.shape
    xb = x.view(b, r, c // _blk(fmt), _blk(fmt))
    amax = xb.abs().amax(-1)
    if fmt == "mx":
        exp = (amax.view(torch.int32) >> 23) & 255
        sc = torch.where(amax == 0, 127, (exp - 2).clamp(min=0))
        inv = ((254 - sc) << 23).view(torch.float32)
        sc = sc.to(torch.uint8)
    else:
        gb = torch.ones((b, 1, 1), device=x.device) if g is None else g.view(b, 1, 1)
        s8 = (amax / (gb * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s8.float() * gb
        inv = torch.where(s > 0, 1.0 / s, 0.0)
        sc = s8.view(torch.uint8)
    y = xb * inv[..., None]
    a = y.abs()
    q = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    q = (q + (y < 0).to(torch.uint8) * 8).to(torch.uint8)
    return q.view(b, r, c), sc


def _pack(q):
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous()


_pairs = {}


def _values(packed, sc_tiled, fmt, g):
    """Packed codes and tiled scales -> the fp32 values they stand for."""
    b, r, half = packed.shape
    dev, blk = packed.device, _blk(fmt)
    if dev not in _pairs:
        v = torch.tensor(E2M1 + tuple(-t for t in E2M1), device=dev)
        i = torch.arange(256, device=dev)
        _pairs[dev] = torch.stack((v[i & 15], v[i >> 4]), -1)   # byte -> its two values
    out = _pairs[dev].index_select(0, packed.view(-1).int()).view(b, r, 2 * half // blk, blk)
    sc = _untile_scales(sc_tiled, r, 2 * half // blk)
    if fmt == "mx":
        n = sc.int()   # 2^(n - 127); the smallest is a subnormal number
        s = torch.where(n == 0, 1 << 22, n << 23).to(torch.int32).view(torch.float32)
    else:
        s = sc.contiguous().view(torch.float8_e4m3fn).float()
        if g is not None:
            s = s * g.view(b, 1, 1)
    return out.mul_(s[..., None]).view(b, r, 2 * half)


def _weight(gen, e, n, k, fmt, dev):
    """Random [e, n, k] weights of variance 1/k, quantised: codes, tiled scales, per-expert factors."""
    q = torch.empty((e, n, k // 2), dtype=torch.uint8, device=dev)
    sc = torch.empty((e, -(-n // 128) * 128 * (-(-(k // _blk(fmt)) // 4) * 4)), dtype=torch.uint8, device=dev)
    g = torch.empty(e, device=dev) if fmt == "nv" else None
    step = max(1, (1 << 27) // (n * k))
    for j in range(0, e, step):
        w = torch.randn((min(step, e - j), n, k), generator=gen, device=dev).mul_(k ** -0.5)
        if g is not None:
            g[j:j + step] = w.abs().amax((1, 2)) / (6.0 * 448.0)
        c, s = _codes(w, fmt, None if g is None else g[j:j + step])
        q[j:j + step], sc[j:j + step] = _pack(c), _tile_scales(s)
    return q, sc, g


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    op = case["op"]
    if op in ("route", "route_bwd"):
        s, e, k = case["s"], case["e"], case["k"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        # tokens differ in what they prefer, experts in how often they are preferred
        logits = torch.randn((s, e), generator=gen, device=dev) * 1.5
        logits += torch.randn(e, generator=gen, device=dev) * 0.5 - 0.5
        st["idx"] = torch.empty((k, s), dtype=torch.int32, device=dev)
        if op == "route":
            for j in range(case["masked"]):
                logits[:, (j * 7 + 1) % e] = -math.inf
            if case["masked"]:
                logits[s // 2] = -math.inf   # a token with no expert left
            st["bias"] = torch.randn(e, generator=gen, device=dev) * 0.05 if case["bias"] else None
            st["gates"] = torch.empty((k, s), device=dev)
        else:
            order = torch.rand((s, e), generator=gen, device=dev).add_(logits.sigmoid()).argsort(1, descending=True)
            st["idx"] = order[:, :k].t().contiguous().int()
            st["d_gates"] = torch.randn((k, s), generator=gen, device=dev)
            st["d_logits"] = torch.empty((s, e), device=dev)
        st["logits"] = logits.to(dt)
        return st
    fmt, e, c = case["fmt"], case["e"], case["c"]
    kept = _kept(case, seed)
    st["counts"] = torch.tensor(kept, dtype=torch.int32, device=dev)
    st["c_dev"] = torch.tensor([c], dtype=torch.int32, device=dev)
    cols = case["cols"] if op == "quantize" else case["k"] if op == "product" else case["m"]
    # activations: a few channels and rows much larger than the rest
    x = torch.randn((e, c, cols), generator=gen, device=dev)
    x *= torch.exp(torch.randn(cols, generator=gen, device=dev) * 0.5)
    x *= torch.exp(torch.randn((e, c, 1), generator=gen, device=dev) * 0.3)
    st["src"] = x.to(torch.bfloat16)
    # the calibrated factors of a serving program: about each expert's largest value / (6 * 448)
    spread = torch.rand((2, e), generator=gen, device=dev) * 0.5 + 0.75
    st["g"] = 12.0 / (6.0 * 448.0) * spread[0].contiguous() if fmt == "nv" else None
    if op == "quantize":
        st["values"] = torch.zeros((e, c, cols), device=dev)
        return st
    if op == "product":
        n = case["n"]
        st["w"] = _weight(gen, e, n, cols, fmt, dev)
        st["b"] = torch.randn((e, n), generator=gen, device=dev).mul_(0.1).bfloat16() if case["bias"] else None
        q, sc = _codes(st["src"].float(), fmt, st["g"])
        st["a"] = (_pack(q), _tile_scales(sc), st["g"])
        st["out"] = torch.zeros((e, c, n), dtype=torch.bfloat16, device=dev)
        return st
    m, h, act = case["m"], case["h"], case["act"]
    st["w1"] = _weight(gen, e, h, m, fmt, dev)
    st["w3"] = _weight(gen, e, h, m, fmt, dev) if act == "swiglu" else (None, None, None)
    st["w2"] = _weight(gen, e, m, h, fmt, dev)
    st["b1"] = st["b2"] = None
    if act != "swiglu":
        st["b1"] = torch.randn((e, h), generator=gen, device=dev).mul_(0.1).bfloat16()
        st["b2"] = torch.randn((e, m), generator=gen, device=dev).mul_(0.1).bfloat16()
    st["gh"] = 6.0 / (6.0 * 448.0) * spread[1].contiguous() if fmt == "nv" else None
    st["out"] = torch.zeros((e, c, m), dtype=torch.bfloat16, device=dev)
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

    case, status = st["case"], st["status"]
    op = case["op"]
    if op == "route":
        M.moe_route_topk(st["logits"], st["bias"], case["k"], st["idx"], st["gates"], status,
                         score=case["score"], groups=case["groups"], topk_groups=case["topk_groups"],
                         group_top=case["group_top"], scale=case["scale"],
                         flags=M.MOE_FLAG_NORMALIZE_GATES if case["norm"] else 0)
        return {"idx": st["idx"], "gates": st["gates"]}
    if op == "route_bwd":
        M.moe_route_bwd(st["logits"], st["idx"], st["d_gates"], st["d_logits"], status, score=case["score"],
                        scale=case["scale"], flags=M.MOE_FLAG_NORMALIZE_GATES if case["norm"] else 0)
        return st["d_logits"]
    fmt, e, c = case["fmt"], case["e"], case["c"]
    counts, c_dev = st["counts"], st["c_dev"]
    if op == "product":
        aq, asc, ag = st["a"]
        wq, wsc, wg = st["w"]
        M.moe_product_fp4(aq, asc, ag, counts, c_dev, wq, wsc, wg, st["b"], fmt, st["out"], status)
        return st["out"]
    cols = st["src"].shape[2]
    q = _space(st, "q", e * c * cols // 2).view(e, c, cols // 2)
    sc = _space(st, "sc", e * M.moe_fp4_scale_bytes(fmt, c, cols)).view(e, -1)
    M.moe_quantize_fp4(st["src"], fmt, q, sc, status, global_scale=st["g"], counts=counts, c_dev=c_dev)
    if op == "quantize":
        M.moe_dequantize_fp4(q, sc, fmt, st["values"], status, global_scale=st["g"], counts=counts, c_dev=c_dev)
        return st["values"]
    m, h, act = case["m"], case["h"], case["act"]
    ws = _space(st, "ws", M.moe_expert_ffn_fp4_workspace_size(fmt, act, e, c, m, h))
    M.moe_expert_ffn_fp4(q, sc, st["g"], st["gh"], counts, c_dev, *st["w1"], st["b1"], *st["w3"], *st["w2"],
                         st["b2"], fmt, act, ws, st["out"], status)
    return st["out"]


def _scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - top)
    width = 1 << (x.shape[1] - 1).bit_length()
    t = torch.nn.functional.pad(p, (0, width - x.shape[1]))
    while t.shape[1] > 1:   # the sum by adjacent pairs
        t = t[:, 0::2] + t[:, 1::2]
    return torch.where(top == -math.inf, 0.0, p / t)


def _in_order(v):
    """Descending order with ties to the lower index."""
    return torch.sort(v, dim=1, descending=True, stable=True)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route":
        x, k, groups = st["logits"].float(), case["k"], case["groups"]
        sc = _scores(x, case["score"])
        choice = sc if st["bias"] is None else sc + st["bias"]
        choice = torch.where((x == -math.inf) | choice.isnan(), -math.inf, choice)
        order = _in_order(choice)[1]
        if groups > 1:
            s, e = x.shape
            best = choice.view(s, groups, e // groups).sort(2, descending=True)[0]
            gv = best[..., 0]
            if case["group_top"] == 2:
                gv = torch.where(best[..., 1] > -math.inf, best[..., 0] + best[..., 1], gv)
            keep = _in_order(gv)[1][:, : case["topk_groups"]]
            kept = torch.zeros((s, groups), dtype=torch.uint8, device=x.device).scatter_(1, keep, 1)
            inside = kept.repeat_interleave(e // groups, 1)
            order = order.gather(1, _in_order(inside.gather(1, order))[1])
        idx = order[:, :k]
        g = sc.gather(1, idx)
        if case["norm"]:
            total = g.sum(1, keepdim=True)
            g = torch.where(total == 0, 0.0, g / total)
        return {"idx": idx.t().int().contiguous(), "gates": (g * case["scale"]).t().contiguous()}
    if op == "route_bwd":
        x, idx = st["logits"].float(), st["idx"].t().long()
        sc = _scores(x, case["score"])
        g, dg, scale = sc.gather(1, idx), st["d_gates"].t(), case["scale"]
        d = torch.zeros_like(x)
        if case["norm"]:
            total = g.sum(1, keepdim=True)
            gn = torch.where(total == 0, 0.0, g / total)
            back = dg - (dg * gn).sum(1, keepdim=True)
            if case["score"] == "softmax":
                return d.scatter_(1, idx, scale * gn * back)
            return d.scatter_(1, idx, scale * gn * back * (1.0 - g))
        if case["score"] == "sigmoid":
            return d.scatter_(1, idx, scale * dg * g * (1.0 - g))
        return d.scatter_(1, idx, scale * dg * g) - sc * (scale * (dg * g).sum(1, keepdim=True))
    fmt, e, c = case["fmt"], case["e"], case["c"]
    rows = torch.minimum(st["counts"], st["c_dev"])
    live = torch.arange(c, device="cuda")[None, :, None] < rows[:, None, None]
    if op == "product":
        aq, asc, ag = st["a"]
        wq, wsc, wg = st["w"]
        y = torch.bmm(_values(aq, asc, fmt, ag), _values(wq, wsc, fmt, wg).transpose(1, 2))
        if st["b"] is not None:
            y = y + st["b"].float()[:, None]
        return torch.where(live, y, 0.0).bfloat16()
    q, sc = _codes(torch.where(live, st["src"].float(), 0.0), fmt, st["g"])
    x = _values(_pack(q), _tile_scales(sc), fmt, st["g"])
    if op == "quantize":
        return x
    hid = torch.bmm(x, _values(*st["w1"][:2], fmt, st["w1"][2]).transpose(1, 2))
    if st["b1"] is not None:
        hid = hid + st["b1"].float()[:, None]
    if case["act"] == "relu":
        hid = hid.clamp(min=0.0)
    elif case["act"] == "gelu":
        hid = 0.5 * hid * (1.0 + torch.erf(hid * math.sqrt(0.5)))
    else:
        up = torch.bmm(x, _values(*st["w3"][:2], fmt, st["w3"][2]).transpose(1, 2))
        hid = hid / (1.0 + torch.exp(-hid)) * up
    q, sc = _codes(hid, fmt, st["gh"])
    hid = _values(_pack(q), _tile_scales(sc), fmt, st["gh"])
    y = torch.bmm(hid, _values(*st["w2"][:2], fmt, st["w2"][2]).transpose(1, 2))
    if st["b2"] is not None:
        y = y + st["b2"].float()[:, None]
    return torch.where(live, y, 0.0).bfloat16()


# ------------------------------------------------------- 64-bit definition
def _near(v, grid):
    """Nearest of the ascending `grid` (ties to the even position), for v >= 0."""
    hi = torch.searchsorted(grid, v.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - v, v - grid[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return torch.where(take_hi, grid[hi], grid[lo])


def _exact_round(x, fmt, g):
    """The values that the 4-bit form of x [rows, cols] stands for, in 64 bits."""
    blk, dev = _blk(fmt), x.device
    v = x.view(x.shape[0], -1, blk)
    amax = v.abs().amax(2, keepdim=True)
    if fmt == "mx":
        p = torch.frexp(torch.where(amax > 0, amax, 1.0))[1] - 1   # floor(log2)
        s = torch.ldexp(torch.ones_like(amax), (p - 2).clamp(min=-127))
    else:
        man = torch.arange(8, device=dev, dtype=torch.float64) / 8
        grid = torch.cat([man * 2.0 ** -6] + [(1 + man) * 2.0 ** p for p in range(-6, 9)])[:-1]
        s = _near((amax / (6.0 * g)).clamp(max=448.0), grid) * g
    s = torch.where(s > 0, s, torch.inf)
    f = torch.tensor(E2M1, device=dev, dtype=torch.float64)
    y = _near((v.abs() / s).clamp(max=6.0), f) * torch.where(torch.isinf(s), 0.0, s)
    return (torch.sign(v) * y).view(x.shape)


def _exact_weight(w, j, fmt, cols):
    q, sc, g = w
    by = q[j].long()
    c = torch.stack((by & 15, by >> 4), -1).view(by.shape[0], -1)
    f = torch.tensor(E2M1, device=q.device, dtype=torch.float64)
    v = f[c & 7] * (1.0 - 2.0 * (c >> 3))
    b = torch.arange(cols // _blk(fmt), device=q.device)
    r = torch.arange(by.shape[0], device=q.device)[:, None]
    nt = -(-b.numel() // 4)
    s = sc[j][((r // 128) * nt + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4].long()
    if fmt == "mx":
        s = torch.ldexp(torch.ones_like(s, dtype=torch.float64), s - 127)
    else:
        ex, man = s >> 3, (s & 7).double()
        s = torch.where(ex > 0, torch.ldexp(8 + man, ex - 10), man * 2.0 ** -9) * g[j].double()
    return (v.view(by.shape[0], -1, _blk(fmt)) * s[..., None]).view(by.shape[0], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_bwd"):
        x = st["logits"].double()
        s, e = x.shape
        k, scale = case["k"], case["scale"]
        p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1))
        if op == "route_bwd":
            idx = st["idx"].t().long()
            leaf = x.clone().requires_grad_()
            p = torch.sigmoid(leaf) if case["score"] == "sigmoid" else torch.softmax(leaf, 1)
            g = p.gather(1, idx)
            if case["norm"]:
                g = g / g.sum(1, keepdim=True)
            (g * scale * st["d_gates"].t().double()).sum().backward()
            return leaf.grad
        want = p if st["bias"] is None else p + st["bias"].double()
        want = want.masked_fill(x == -math.inf, -1e30)
        gs = e // case["groups"]
        top = want.view(s, -1, gs).topk(min(case["group_top"], gs), 2)[0]
        val = torch.where(top[..., :1] > -1e29, torch.where(top > -1e29, top, 0.0).sum(2, keepdim=True), -1e30)
        place = (-val[..., 0]).argsort(dim=1, stable=True).argsort(dim=1)
        out = (place >= case["topk_groups"]).repeat_interleave(gs, 1)
        idx = (-want.masked_fill(out, -2e30)).argsort(dim=1, stable=True)[:, :k]
        g = p.gather(1, idx)
        if case["norm"]:
            g = torch.nan_to_num(g / g.sum(1, keepdim=True))
        return {"idx": None, "gates": (g * scale).t()}   # near ties may order differently in 64 bits
    fmt, kept = case["fmt"], _kept(case, seed)
    g = [None] * case["e"] if st["g"] is None else st["g"].tolist()
    wide = st["src"].shape[2] if op == "quantize" else case["n"] if op == "product" else case["m"]
    out = torch.zeros((case["e"], case["c"], wide), dtype=torch.float64, device="cuda")
    for j, r in enumerate(kept):
        if r == 0:
            continue
        x = _exact_round(st["src"][j, :r].double(), fmt, g[j])
        if op == "quantize":
            out[j, :r] = x
        elif op == "product":
            y = x @ _exact_weight(st["w"], j, fmt, case["k"]).t()
            out[j, :r] = y if st["b"] is None else y + st["b"][j].double()
        else:
            hid = x @ _exact_weight(st["w1"], j, fmt, case["m"]).t()
            if st["b1"] is not None:
                hid = hid + st["b1"][j].double()
            if case["act"] == "relu":
                hid = torch.relu(hid)
            elif case["act"] == "gelu":
                hid = torch.nn.functional.gelu(hid)
            else:
                hid = torch.nn.functional.silu(hid) * (x @ _exact_weight(st["w3"], j, fmt, case["m"]).t())
            hid = _exact_round(hid, fmt, None if st["gh"] is None else float(st["gh"][j]))
            y = hid @ _exact_weight(st["w2"], j, fmt, case["h"]).t()
            out[j, :r] = y if st["b2"] is None else y + st["b2"][j].double()
    return out
