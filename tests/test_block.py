"""A block of a model end to end (block.py), its router's gradient, and the forward
with a given routing, on the GPU."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import blocks as B
from oracle import moe as O
from tests._util import oracle_args, rel_l2

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def m():
    import __graft_entry__

    __graft_entry__.build()
    import mixture_experts_layer_index_gb300 as mod

    return mod


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _dev(inp):
    return {k: (v.to(DEV) if v is not None else None) for k, v in inp.items()}


@pytest.mark.parametrize("quant,T,path", [("bf16", 70, "grouped"), ("fp8_tensor", 5, "route_direct"),
                                          ("fp8_tensor", 70, "grouped"), ("fp8_block", 6, "route_direct"),
                                          ("fp8_block", 70, "grouped"), ("mxfp8", 70, "grouped")])
def test_given_routing_equals_own_routing(m, quant, T, path):
    wl = W.Workload("t", T, 16, 4, 256, 128, quant, 5)
    d = _dev(W.make_inputs(wl))
    p = m.problem(T, 16, 4, 256, 128, quant, {"grouped": m.MOE_PATH_GROUPED, "route_direct": m.MOE_PATH_ROUTE_DIRECT}[path])
    ids, w = torch.empty(T, 4, dtype=torch.int32, device=DEV), torch.empty(T, 4, device=DEV)
    m.moe_route(d["scores"], T, 16, 4, ids, w)
    y = [torch.full((T, 256), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ws = torch.empty(m.moe_workspace_size(p), dtype=torch.uint8, device=DEV)
    m.moe_forward(p, d["x"], d["scores"], d["w1"], d["w2"], d["w1_scale"], d["w2_scale"], y[0], ws)
    m.moe_forward_routed(p, None, d["x"], ids, w, d["w1"], d["w2"], d["w1_scale"], d["w2_scale"], y[1], ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    assert torch.equal(y[0], y[1])
    v = m.moe_forward_views(p, ws)
    at = v.ids - ws.data_ptr()
    assert torch.equal(ws[at:at + T * 16].view(torch.int32).view(T, 4), ids)
    # an id that is no expert is reported and adds nothing
    bad, w0 = ids.clone(), w.clone()
    bad[2, 1], bad[3, 0] = 16, -3
    w0[2, 1] = w0[3, 0] = 0
    z = [torch.empty_like(y[0]) for _ in range(2)]
    m.moe_forward_routed(p, None, d["x"], bad, w, d["w1"], d["w2"], d["w1_scale"], d["w2_scale"], z[0], ws)
    assert m.moe_read_device_status(ws) == m.MOE_ERR_DEVICE_BOUNDS
    m.moe_forward_routed(p, None, d["x"], ids, w0, d["w1"], d["w2"], d["w1_scale"], d["w2_scale"], z[1], ws)
    # per-tensor FP8 scales h by its maximum over all routes, the ones that add nothing among them
    keep = [t for t in range(T) if t not in (2, 3)]
    if quant != "fp8_tensor":
        assert torch.equal(z[0], z[1])
    else:
        assert rel_l2(_f64(z[0])[keep], _f64(z[1])[keep]) <= 2e-2
    with pytest.raises(m.MoeError):
        m.moe_forward_routed(p, None, d["x"], None, w, d["w1"], d["w2"], d["w1_scale"], d["w2_scale"], z[0], ws)


def _block(m, quant, T, E, k, H, I, rule, gate=True, shared=0, seed=3):
    from mixture_experts_layer_index_gb300.block import Block

    wl = W.Workload("b", T, E, k, H, I, quant, seed)
    inp = W.make_inputs(wl)
    g = torch.Generator().manual_seed(seed)
    router = (torch.randn(E, H, generator=g) / H ** 0.5).to(torch.bfloat16).to(DEV), torch.randn(E, generator=g).to(DEV) * 0.1
    norms = [(1 + 0.2 * torch.randn(H, generator=g)).to(DEV) for _ in range(2)] + [
        (0.5 + 0.2 * torch.randn(H, generator=g)).to(DEV) if gate else None]
    sh = None
    if shared:
        s = _dev(W.make_inputs(W.Workload("s", 1, shared, 1, H, I, quant, seed + 1)))
        sh = (shared, s["w1"], s["w2"], s["w1_scale"], s["w2_scale"])
    d = _dev(inp)
    b = Block(T, E, k, H, I, quant, (d["w1"], d["w2"], d["w1_scale"], d["w2_scale"]), router, norms, rule, sh)
    h = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    o = (0.5 * torch.randn(T, H, generator=g)).to(torch.bfloat16).to(DEV)
    return b, inp, h, o


@pytest.mark.parametrize("quant,T", [("bf16", 1), ("bf16", 90), ("fp8_tensor", 3), ("fp8_block", 90)])
@pytest.mark.parametrize("rule", [dict(), dict(score="sigmoid", n_group=4, topk_group=2, group_best=2, scale=2.0)])
def test_block_against_the_oracle(m, quant, T, rule):
    E, k, H, I = 16, 4, 256, 128
    b, inp, h, o = _block(m, quant, T, E, k, H, I, rule)
    h1, o1 = b.forward(h, o)
    assert b.status() == m.MOE_OK
    post, pre, gate = b.norms
    ref_h, ref_x, mag_h, mag_x = B.norm(_f64(h), _f64(o), {"kind": "channel", "values": _f64(gate)}, _f64(post), None,
                                        _f64(pre), None, "rms", "rms", 1e-6, 1.0, 1.0)
    assert np.all(np.abs(_f64(h1) - ref_h) <= 2.0 ** -8 * np.abs(ref_h) + 32 * 2.0 ** -23 * mag_h)
    assert np.all(np.abs(_f64(b.x) - ref_x) <= 2.0 ** -8 * np.abs(ref_x) + 64 * 2.0 ** -23 * mag_x)
    # from here on, from the x the block computed
    logits, _, mag = B.linear(_f64(b.x), _f64(b.router[0]), _f64(b.router[1]), None, "none", 1.0)
    assert np.all(np.abs(_f64(b.logits) - logits) <= (H / 8 + 16) * 2.0 ** -23 * mag)
    ids, w, margin = B.route(_f64(b.logits), k, **rule)
    sure = margin > 16 * 2.0 ** -23
    assert np.array_equal(b.ids.cpu().numpy()[sure], ids[sure])
    assert np.all(np.abs(_f64(b.w) - w)[sure] <= 2e-5 * np.abs(w[sure]))
    # the experts: the oracle routes by softmax over the selected scores, so log w of the selected
    # experts as scores gives it this routing, with weights w / sum(w)
    args = list(oracle_args(inp))
    args[0] = b.x.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)
    got_ids, got_w = b.ids.cpu().numpy(), _f64(b.w)
    scores = np.full((T, E), -1e4, dtype=np.float32)
    np.put_along_axis(scores, got_ids.astype(np.int64), np.log(got_w).astype(np.float32), 1)
    args[1] = scores
    y = O.forward(*args, k, quant)["y"] * got_w.sum(axis=1, keepdims=True)
    assert rel_l2(_f64(o1), y) <= (1e-2 if quant == "bf16" else 2e-2)


def test_block_with_shared_experts_chains_in_a_graph(m):
    b, _, h, o = _block(m, "bf16", 33, 16, 4, 256, 128, dict(score="sigmoid"), gate=False, shared=1)
    h1, o1 = (t.clone() for t in b.forward(h, o))
    h2, o2 = (t.clone() for t in b.forward(h1, o1))
    torch.cuda.synchronize()
    hg, og = h1.clone(), o1.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(hg, og)
    b.h_out.zero_(), b.o_out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.h_out, h2) and torch.equal(b.o_out, o2) and b.status() == m.MOE_OK


@pytest.mark.parametrize("rule", [dict(scale=1.5), dict(score="sigmoid", n_group=2, topk_group=1), dict(renormalise=False)])
def test_router_gradient_by_differentiation(m, rule):
    T, E, k, H = 50, 16, 4, 256
    b, _, h, o = _block(m, "bf16", T, E, k, H, 128, rule)
    b.forward(h, o)
    g = torch.Generator().manual_seed(9)
    dw = torch.randn(T, k, generator=g).to(DEV)
    dh = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    got = b.router_gradient(o, dw, dh)
    ids = b.ids.long()
    v = {n: t.double().requires_grad_() for n, t in dict(h=h, o=o, post=b.norms[0], pre=b.norms[1], gate=b.norms[2],
                                                        wr=b.router[0], br=b.router[1]).items()}

    def rms(x, w):
        return x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * w

    h1 = v["h"] + v["gate"] * rms(v["o"], v["post"])
    logits = rms(h1, v["pre"]) @ v["wr"].t() + v["br"]
    p = torch.sigmoid(logits) if rule.get("score") == "sigmoid" else torch.softmax(logits, 1)
    w = p.gather(1, ids)
    if rule.get("renormalise", True):
        w = w / w.sum(1, keepdim=True)
    ((rule.get("scale", 1.0) * w * dw.double()).sum() + (h1 * dh.double()).sum()).backward()
    # h', x, dlogits and dx are rounded to bf16 on the way (2^-8 each at most, 2^-9 on average)
    for name, t in (("dh", "h"), ("d_o", "o"), ("router_weight", "wr"), ("router_bias", "br"), ("post_weight", "post"),
                    ("pre_weight", "pre"), ("gate", "gate")):
        assert rel_l2(_f64(getattr(got, name)), _f64(v[t].grad)) <= 2e-2, name


def test_a_router_learns_a_given_routing(m):
    # gradient descent on the router's logits layer until its weights match a target's
    T, E, k, H = 256, 8, 8, 256
    b, _, h, o = _block(m, "bf16", T, E, k, H, 128, dict(score="sigmoid"))
    target = torch.softmax(torch.randn(E, generator=torch.Generator().manual_seed(1)), 0).to(DEV)
    master_w, master_b = b.router[0].float(), b.router[1].clone()
    losses = []
    for _ in range(40):
        b.forward(h, o)
        d = b.w - target[b.ids.long()]
        losses.append(float(d.square().sum()))
        grad = b.router_gradient(o, 2 * d)
        master_w -= 0.02 * grad.router_weight.float()
        master_b -= 0.02 * grad.router_bias
        b.router[0].copy_(master_w)
        b.router[1].copy_(master_b)
    assert losses[-1] < 0.2 * losses[0], losses[::8]
