"""Whole layers on rows sorted by expert: routing, order, experts and way back together, forward and
gradient, padded batches, other streams, captured graphs; bf16 and 8-bit integer experts.

Compared with 64 bits by the root mean square.  A rounding to bf16 is off by at most 2^-8 of the value,
and a product or sum with independent terms passes relative errors of that kind on as they are: with r
roundings on the way the error stays below r * 2^-8 of the result's root mean square.  (Forward: hidden,
expert output, y.  Gradient: those, d_out, d_pre, d_xs and the gradient itself; the 8-bit layer also has
its codes, half a step of 1 / 127 of a row's largest value, here at most 6 of its root mean square:
6 / 254 for the tokens, the weights being taken as quantised, and again for the hidden, at most 12.)"""

import pytest
import torch

import combine_moe_gate_gb300 as M

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
STEP = 2.0 ** -8


def inputs(s, m, e, h, act, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF)

    swiglu = act == "swiglu"
    return dict(x=r(s, m), logits=torch.randn((s, e), generator=g, device="cuda"), w1=r(e, h, m, scale=m ** -0.5),
                w3=r(e, h, m, scale=m ** -0.5) if swiglu else None, w2=r(e, m, h, scale=h ** -0.5),
                b1=None if swiglu else r(e, h), b2=None if swiglu else r(e, m), dy=r(s, m))


def plain(p, act, idx, w):
    """The layer and its gradients in 64 bits, with the selection idx [k, s] (-1: none) taken as it is."""
    d = {n: None if t is None else t.double() for n, t in w.items()}
    leaves = {n: d[n].clone().requires_grad_(True) for n in ("w1", "w3", "w2", "b1", "b2") if d[n] is not None}
    x, logits = p["x"].double().requires_grad_(True), p["logits"].double().requires_grad_(True)
    score = torch.sigmoid(logits)
    live = idx >= 0
    pick = score.gather(1, idx.clamp(min=0).t().long()).t() * live
    gates = pick / pick.sum(0).clamp(min=1e-300) * 2.0
    y = 0
    for r in range(idx.shape[0]):
        rows = []
        for t in range(idx.shape[1]):
            j = int(idx[r, t])
            if j < 0:
                rows.append(torch.zeros_like(x[t]))
                continue
            a = leaves["w1"][j] @ x[t]
            if act == "swiglu":
                hid = torch.nn.functional.silu(a) * (leaves["w3"][j] @ x[t])
            else:
                a = a + leaves["b1"][j]
                hid = torch.relu(a) if act == "relu" else torch.nn.functional.gelu(a)
            o = leaves["w2"][j] @ hid
            rows.append(o if act == "swiglu" else o + leaves["b2"][j])
        y = y + gates[r, :, None] * torch.stack(rows)
    names = list(leaves)
    grads = torch.autograd.grad(y, [x, logits] + [leaves[n] for n in names], p["dy"].double())
    return y.detach(), dict(zip(["d_x", "d_logits"] + ["d_" + n for n in names], grads))


def off(got, want):
    return ((got.double() - want).square().mean() / want.square().mean().clamp(min=1e-300)).sqrt().item()


OPT = dict(score="sigmoid", scale=2.0)


@pytest.mark.parametrize("act", ["relu", "gelu", "swiglu"])
@pytest.mark.parametrize("s,k,padded", [(1, 1, 0), (45, 3, 0), (64, 2, 9)])
def test_layer_and_gradient(s, k, padded, act):
    m, e, h = 64, 6, 96
    p = inputs(s, m, e, h, act)
    padding = torch.arange(s, device="cuda") >= s - padded if padded else None
    B = M.alloc_layer_sorted(s, m, e, k, h, act, train=True)
    y = M.run_layer_sorted(p["x"], p["logits"], None, p["w1"], p["b1"], p["w3"], p["w2"], p["b2"], act, k, B,
                           padding=padding, **OPT)
    G = M.alloc_grads_sorted(s, k, p["w1"], p["w3"], p["w2"], act)
    M.run_layer_sorted_bwd(p["dy"], p["logits"], p["w1"], p["w3"], p["w2"], act, B, G, padding=padding, **OPT)
    assert B.status.item() == 0
    if padded:
        assert (B.idx[:, s - padded:] == -1).all() and (y[s - padded:] == 0).all()
        assert (G.d_x[s - padded:] == 0).all() and (G.d_logits[s - padded:] == 0).all()
    want, grads = plain(p, act, B.idx, p)
    assert off(y, want) < 3 * STEP
    for name, g in grads.items():
        assert off(getattr(G, name), g) < 7 * STEP, name


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("s,k,padded", [(1, 2, 0), (4, 2, 0), (70, 3, 11)])
def test_layer_on_8_bit_experts(s, k, padded, act):
    m, e, h = 128, 6, 80
    p = inputs(s, m, e, h, act)
    padding = torch.arange(s, device="cuda") >= s - padded if padded else None
    q = {n: M.quantize_weights_int8(p[n]) if p[n] is not None else None for n in ("w1", "w3", "w2")}
    B = M.alloc_layer_sorted(s, m, e, k, h, act, int8=True)
    y = M.run_layer_int8(p["x"], p["logits"], None, q["w1"], p["b1"], q["w3"], q["w2"], p["b2"], act, k, B,
                         padding=padding, **OPT)
    assert B.status.item() == 0
    w = dict(p)
    for n, t in q.items():
        if t is not None:
            w[n] = t.q.double() * t.scale.double()[..., None]
    want, _ = plain(p, act, B.idx, w)
    assert off(y, want) < 3 * STEP + 6 / 254 + 12 / 254
    if padded:
        assert (y[s - padded:] == 0).all()


def test_captured_layers_follow_their_inputs():
    """Forward and gradient captured once and replayed on other inputs: the bits of eager calls."""
    s, m, e, k, h, act = 100, 64, 8, 2, 128, "swiglu"
    p, p2 = inputs(s, m, e, h, act, 1), inputs(s, m, e, h, act, 2)
    B, G = M.alloc_layer_sorted(s, m, e, k, h, act, train=True), M.alloc_grads_sorted(s, k, p["w1"], p["w3"], p["w2"], act)
    q = {n: M.quantize_weights_int8(p[n]) for n in ("w1", "w3", "w2")}
    B8 = M.alloc_layer_sorted(s, m, e, k, h, act, int8=True)

    def step(p, B, G, B8):
        M.run_layer_sorted(p["x"], p["logits"], None, p["w1"], None, p["w3"], p["w2"], None, act, k, B, **OPT)
        M.run_layer_sorted_bwd(p["dy"], p["logits"], p["w1"], p["w3"], p["w2"], act, B, G, **OPT)
        M.run_layer_int8(p["x"], p["logits"], None, q["w1"], None, q["w3"], q["w2"], None, act, k, B8, **OPT)

    step(p, B, G, B8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(p, B, G, B8)
    for n, t in p.items():
        if t is not None and n not in ("w1", "w3", "w2"):
            t.copy_(p2[n])
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (B.y, B8.y, G.d_x, G.d_logits, G.d_w1, G.d_w3, G.d_w2)]
    B, G = M.alloc_layer_sorted(s, m, e, k, h, act, train=True), M.alloc_grads_sorted(s, k, p["w1"], p["w3"], p["w2"], act)
    B8 = M.alloc_layer_sorted(s, m, e, k, h, act, int8=True)
    step(p, B, G, B8)
    for a, b in zip(got, (B.y, B8.y, G.d_x, G.d_logits, G.d_w1, G.d_w3, G.d_w2)):
        assert torch.equal(a, b)


def test_two_layers_on_two_streams():
    s, m, e, k, h, act = 300, 128, 8, 2, 256, "gelu"
    runs, alone = [], []
    for seed in (1, 2):
        p = inputs(s, m, e, h, act, seed)
        pad = torch.arange(s, device="cuda") % 7 == seed
        args = (p["x"], p["logits"], None, p["w1"], p["b1"], p["w3"], p["w2"], p["b2"], act, k)
        B = M.alloc_layer_sorted(s, m, e, k, h, act)
        alone.append(M.run_layer_sorted(*args, B, padding=pad, **OPT).clone())
        runs.append((args, pad))
    streams = [torch.cuda.Stream() for _ in runs]
    out = [[M.alloc_layer_sorted(s, m, e, k, h, act) for _ in range(4)] for _ in runs]
    torch.cuda.synchronize()
    for i in range(4):   # both streams have work at the same time
        for st, bufs, (args, pad) in zip(streams, out, runs):
            M.run_layer_sorted(*args, bufs[i], padding=pad, stream=st, **OPT)
    torch.cuda.synchronize()
    for bufs, want in zip(out, alone):
        for B in bufs:
            assert torch.equal(B.y, want) and B.status.item() == 0


def test_what_padded_tokens_hold_does_not_matter():
    """NaN in the padded tokens' x, logits and dy: the bits of zeros there."""
    s, m, e, k, h, act = 90, 64, 6, 3, 96, "swiglu"
    padding = torch.arange(s, device="cuda") % 5 == 2
    got = []
    for fill in (0.0, float("nan")):
        p = inputs(s, m, e, h, act, 3)
        for n in ("x", "logits", "dy"):
            p[n][padding] = fill
        args = (p["x"], p["logits"], None, p["w1"], None, p["w3"], p["w2"], None, act, k)
        B, G = M.alloc_layer_sorted(s, m, e, k, h, act, train=True), M.alloc_grads_sorted(s, k, p["w1"], p["w3"], p["w2"], act)
        M.run_layer_sorted(*args, B, padding=padding, **OPT)
        M.run_layer_sorted_bwd(p["dy"], p["logits"], p["w1"], p["w3"], p["w2"], act, B, G, padding=padding, **OPT)
        B8 = M.alloc_layer_sorted(s, m, e, k, h, act, int8=True)
        q = {n: M.quantize_weights_int8(p[n]) for n in ("w1", "w3", "w2")}
        M.run_layer_int8(p["x"], p["logits"], None, q["w1"], None, q["w3"], q["w2"], None, act, k, B8, padding=padding, **OPT)
        assert B.status.item() == 0 and B8.status.item() == 0
        assert (G.d_x[padding] == 0).all() and (G.d_logits[padding] == 0).all() and (B.y[padding] == 0).all()
        got.append([B.y, B8.y, G.d_x, G.d_logits, G.d_w1, G.d_w3, G.d_w2])
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)
