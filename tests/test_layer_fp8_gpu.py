"""The norm, quantisation, the 8-bit experts and the 8-bit shared expert together, as a layer
uses them, against the float64 oracle stage by stage: each stage from what the device
computed before it, so that a value next to a rounding border counts once. Errors in the
2-norm are held to the roundings of a stage, half a step each at its worst: 2^-8 in bf16, 2^-4 in e4m3."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import f64
from oracle import fp8 as ofp8, linear as olinear, norm as onorm, route_scored as oscored

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_top_router_amd")
ops = moe.ops
BF = torch.bfloat16


def _bytes(q):
    return q.view(torch.uint8).cpu().numpy()


def _rel(got, want):
    return np.linalg.norm(np.asarray(got, np.float64) - want) / np.linalg.norm(want)


def _rows(q, s):
    return ofp8.row_values(_bytes(q), s.cpu().numpy())


def _stack(pair):
    q, s = pair
    return [ofp8.weight_values(_bytes(q[e]), s[e].cpu().numpy()) for e in range(len(q))]


def _make(T, E, k, H, I, Is, seed, **kw):
    g = torch.Generator("cuda").manual_seed(seed)

    def n(shape, fan):
        return (torch.randn(shape, generator=g, device="cuda") * fan ** -0.5).to(BF)
    gate, w1, w3, w2 = n((E, H), H), n((E, H, I), H), n((E, H, I), H), n((E, I, H), I)
    shared = (n((H, Is), H), n((H, Is), H), n((Is, H), Is)) if Is else None
    gain = 1 + 0.2 * torch.randn((H,), generator=g, device="cuda")
    layer = moe.MoELayer(T, H, E, k, I, w1, w3, w2, align=32, gate_w=gate, shared=shared,
                         router=moe.Router(num_groups=4, top_groups=2), norm=gain, fp8=True, **kw)
    x, res = n((T, H), 1), n((T, H), 0.25)
    return layer, x, res, gate, gain, (w1, w3, w2)


@pytest.mark.parametrize("T, E, k, Is, fast", [(1, 16, 4, 256, False), (70, 32, 4, 384, False),
                                               (300, 8, 2, 0, True), (520, 16, 4, 128, True)])
def test_layer(T, E, k, Is, fast):
    print("CASE fp8 layer", T, E, k, Is, fast, flush=True)
    H, I = 384, 256
    layer, x, res, gate, gain, (w1, w3, w2) = _make(T, E, k, H, I, Is, T, fp8_fast=fast)
    out = layer(x, residual=res).clone()
    torch.cuda.synchronize()
    assert torch.equal(layer.total, (x.float() + res.float()).to(BF))
    y = onorm.rms_norm(f64(layer.total), gain.double().cpu().numpy(), 1e-6)
    xq = _rows(*layer.xq)
    assert _rel(f64(layer.normed), y) <= 2.0 ** -8 and _rel(xq, y) <= 2.0 ** -4
    logits, _ = olinear.linear(f64(layer.normed), f64(gate))
    assert _rel(layer.logits.cpu().numpy(), logits) <= 1e-5
    idx, w = oscored.route(layer.logits.cpu().numpy(), k, None, "sigmoid", 4, 2, "top2", True, 1.0)
    assert (layer.topk_idx.cpu().numpy() == idx).all()

    # the weights are those of the quantiser, which hold the given ones to half a step
    for pair, given in ((layer.w1q, w1), (layer.w3q, w3), (layer.w2q, w2)):
        for e, v in enumerate(_stack(pair)):
            assert _rel(v, f64(given[e]).T) <= 2.0 ** -4
    w1v, w3v, w2v = _stack(layer.w1q), _stack(layer.w3q), _stack(layer.w2q)
    h, off = _rows(layer.h, layer.h_scale), layer.L.offsets.cpu().numpy()
    dst = layer.L.dst_row.cpu().numpy()
    want = np.zeros((T, H))
    for e in range(E):
        t, s = np.nonzero(idx == e)
        if not len(t):
            continue
        rows = off[e] + np.arange(len(t))
        assert (dst[t, s] == rows).all()
        assert _rel(h[rows], olinear.act(xq[t] @ w1v[e].T, "silu") * (xq[t] @ w3v[e].T)) <= 2.0 ** -4
        y = h[rows] @ w2v[e].T
        assert _rel(f64(layer.y)[rows], y) <= 2.0 ** -8 + 2.0 ** -12
        want[t] += w[t, s][:, None] * y
    if Is:
        hs = _rows(*layer.shared_h)
        (s1,), (s3,) = _stack(layer.shared_w1), _stack(layer.shared_w3)
        assert _rel(hs, olinear.act(xq @ s1.T, "silu") * (xq @ s3.T)) <= 2.0 ** -4
        q, s = layer.shared_w2
        want += hs @ ofp8.weight_values(_bytes(q), s.cpu().numpy()).T
    # y, the combine and the output each rounded once
    assert _rel(f64(out), want) <= 3 * 2.0 ** -8
    again = layer(x, residual=res)
    assert torch.equal(again, out)


def test_layer_without_norm_quantises_its_rows_and_is_replayed():
    T, H, E, I = 64, 256, 8, 128
    g = torch.Generator("cuda").manual_seed(3)
    w1, w3, w2 = (torch.randn(s, generator=g, device="cuda").mul_(0.06).to(BF)
                  for s in ((E, H, I), (E, H, I), (E, I, H)))
    layer = moe.MoELayer(T, H, E, 2, I, w1, w3, w2, fp8=True)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF)
    logits = torch.randn((T, E), generator=g, device="cuda")
    out = layer(x, logits).clone()
    q, s = ops.quantize_fp8(x)
    assert torch.equal(q.view(torch.uint8), layer.xq[0].view(torch.uint8)) and torch.equal(s, layer.xq[1])
    # against the bf16 layer: both operands of two products in e4m3, h in between
    bf = moe.MoELayer(T, H, E, 2, I, w1, w3, w2)(x, logits)
    assert _rel(f64(out), f64(bf)) <= 5 * 2.0 ** -4
    with pytest.raises(ValueError, match="norm"):
        layer(x, logits, residual=x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = layer(x, logits)
    for k in range(3):
        x.copy_(torch.randn((T, H), generator=g, device="cuda").to(BF))
        logits.copy_(torch.randn((T, E), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = kept.clone()
        assert torch.equal(got, layer(x, logits)), k


def test_norm_beside_the_bf16_experts():
    T, H, E, I = 33, 256, 8, 128
    g = torch.Generator("cuda").manual_seed(4)
    w1, w3, w2 = (torch.randn(s, generator=g, device="cuda").mul_(0.06).to(BF)
                  for s in ((E, H, I), (E, H, I), (E, I, H)))
    gain = torch.rand((H,), generator=g, device="cuda")
    x, res = (torch.randn((T, H), generator=g, device="cuda").to(BF) for _ in range(2))
    logits = torch.randn((T, E), generator=g, device="cuda")
    normed = moe.MoELayer(T, H, E, 2, I, w1, w3, w2, norm=gain, eps=1e-5)
    plain = moe.MoELayer(T, H, E, 2, I, w1, w3, w2)
    y, _, _, total = ops.rms_norm(x, gain, residual=res, eps=1e-5)
    assert torch.equal(normed(x, logits, residual=res), plain(y, logits))
    assert torch.equal(normed.total, total)
    y = ops.rms_norm(x, gain, eps=1e-5)[0]
    assert torch.equal(normed(x, logits), plain(y, logits))


def test_training_step_of_the_norm_against_differences():
    """A loss through norm and router projection: the gradients of the calls against the
    change of the loss, computed in float64, along random directions."""
    T, H, E = 40, 128, 16
    g = torch.Generator("cuda").manual_seed(5)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, gain, gate, dl = n(T, H), 1 + 0.2 * n(H), (n(E, H) * H ** -0.5).to(BF), n(T, E)
    y, _, _, _ = ops.rms_norm(x, gain, eps=1e-5)
    dy = (dl.double() @ gate.double()).float()
    dx, dg = ops.rms_norm_backward(dy, x, gain, eps=1e-5)
    xs, gs, ws, ds = (v.double().cpu().numpy() for v in (x, gain, gate.float(), dl))
    loss = lambda a, b: ((onorm.rms_norm(a, b, 1e-5) @ ws.T) * ds).sum()  # noqa: E731
    r = np.random.default_rng(6)
    for _ in range(4):
        e, f = r.normal(size=xs.shape), r.normal(size=gs.shape)
        got = (dx.double().cpu().numpy() * e).sum(), (dg.double().cpu().numpy() * f).sum()
        d = 1e-5
        num = ((loss(xs + d * e, gs) - loss(xs - d * e, gs)) / (2 * d),
               (loss(xs, gs + d * f) - loss(xs, gs - d * f)) / (2 * d))
        size = (np.abs(dx.double().cpu().numpy() * e).sum(), np.abs(dg.double().cpu().numpy() * f).sum())
        for a, b, m in zip(got, num, size):
            assert abs(a - b) <= 2.0 ** -16 * m + 1e-6
