"""The router projection, the scored router, the experts, a shared expert and
gradient clipping together, as a layer uses them: forward through MoELayer
against the float64 oracle, and one training step through the library's calls
against autograd in float64. Each 16-bit rounding on a path is off by at most
half a step, 2^-8 of the value: errors (in the 2-norm) are held to the number
of roundings on the longest path, each taken at its worst."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import bf16 as obf16, linear as olinear, route_scored as oscored
from gpu_util import f64

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_top_router_amd")
ops = moe.ops
BF = torch.bfloat16


def _weights(gen, E, H, I, Is):
    def n(shape, fan):
        return (torch.randn(shape, generator=gen, device="cuda") * fan ** -0.5).to(BF)
    return (n((E, H), H), n((E, H, I), H), n((E, H, I), H), n((E, I, H), I),
            (n((H, Is), H), n((H, Is), H), n((Is, H), Is)))


def _rel(got, want):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("T,E,k,groups,top,score,renorm", [
    (1, 16, 4, 4, 2, "sigmoid", True), (77, 32, 4, 8, 3, "sigmoid", True),
    (500, 24, 3, 1, 1, "softmax", False),
])
def test_layer_with_gate_scored_router_and_shared_expert(T, E, k, groups, top, score, renorm):
    print("CASE layer", T, E, k, groups, top, score, flush=True)
    H, I, Is = 256, 128, 384
    gen = torch.Generator("cuda").manual_seed(T)
    gate, w1, w3, w2, shared = _weights(gen, E, H, I, Is)
    bias = torch.randn((E,), generator=gen, device="cuda") * 0.1
    layer = moe.MoELayer(T, H, E, k, I, w1, w3, w2, align=32, gate_w=gate, shared=shared,
                         router=moe.Router(score, bias, groups, top, "top2", renorm, 2.0))
    x = torch.randn((T, H), generator=gen, device="cuda").to(BF)
    out = layer(x).clone()
    torch.cuda.synchronize()

    xs = f64(x)
    logits, _ = olinear.linear(xs, f64(gate))
    assert np.abs(layer.logits.cpu().numpy() - logits).max() <= \
        (H + 160) * 2.0 ** -23 * (np.abs(xs) @ np.abs(f64(gate)).T).max()
    # the choice on the logits the layer computed
    idx, w = oscored.route(layer.logits.cpu().numpy(), k, bias.cpu().numpy(), score, groups, top,
                           "top2", renorm, 2.0)
    assert (layer.topk_idx.cpu().numpy() == idx).all()

    def expert(rows, a, b, c):
        h = obf16.round_to_bf16(olinear.act(rows @ a, "silu") * (rows @ b))
        return h @ c
    want = expert(xs, *(f64(t) for t in shared))
    for e in range(E):
        t, s = np.nonzero(idx == e)
        if len(t):
            y = obf16.round_to_bf16(expert(xs[t], f64(w1[e]), f64(w3[e]), f64(w2[e])))
            want[t] += w[t, s][:, None] * y
    # roundings: h (where the device's fp32 falls on the other side), y, the combine, the output
    assert _rel(f64(out), want) <= 4 * 2.0 ** -8
    # and again: the shared product took `out` as its residual, nothing is left over
    again = layer(x)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


def test_layer_takes_logits_or_a_gate():
    gen = torch.Generator("cuda").manual_seed(0)
    gate, w1, w3, w2, _ = _weights(gen, 8, 128, 128, 128)
    x = torch.randn((16, 128), generator=gen, device="cuda").to(BF)
    logits = torch.randn((16, 8), generator=gen, device="cuda")
    with_gate = moe.MoELayer(16, 128, 8, 2, 128, w1, w3, w2, gate_w=gate)
    plain = moe.MoELayer(16, 128, 8, 2, 128, w1, w3, w2)
    with pytest.raises(ValueError):
        with_gate(x, logits)
    with pytest.raises(ValueError):
        plain(x)
    got = with_gate(x)
    want = plain(x, with_gate.logits)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("softmax", False)])
def test_one_training_step(score, renorm):
    T, H, I, E, k = 192, 256, 128, 16, 4
    gen = torch.Generator("cuda").manual_seed(5)
    gate, w1, w3, w2, _ = _weights(gen, E, H, I, 128)
    x = torch.randn((T, H), generator=gen, device="cuda").to(BF)
    G = torch.randn((T, H), generator=gen, device="cuda").to(BF)

    logits = ops.linear(x, gate, out_dtype=torch.float32)
    idx, w = ops.route_scored(logits, k, None, score, 4, 2, "top2", renorm, 1.5)
    L = ops.layout(idx, E, align=32)
    xp = ops.permute(x, L.dst_row, L.src_row, L.offsets, L.m_cap)
    h, gu = ops.grouped_gate_up_save(xp, L.offsets, L.local_counts, ops.pack_weights(w1),
                                     ops.pack_weights(w3))
    y = ops.grouped_down(h, L.offsets, L.local_counts, ops.pack_weights(w2))
    out = ops.combine(y, L.dst_row, w)

    dy, dw = ops.combine_backward(G, y, L.dst_row, w, grad_y=torch.zeros_like(y))
    dlogits = ops.route_scored_backward(logits, idx, dw, score, renorm, 1.5)
    dx_gate, dgate, _ = ops.linear_backward(dlogits, x, gate)
    dgu = ops.grouped_down_backward(dy, gu, L.offsets, L.local_counts, w2)
    dw2 = ops.grouped_down_wgrad(h, dy, L.offsets, L.local_counts)
    dw1, dw3 = ops.grouped_gate_up_wgrad(xp, dgu, L.offsets, L.local_counts)
    dxp = ops.grouped_gate_up_backward(dgu, L.offsets, L.local_counts, w1, w3)
    dx = ops.permute_backward(dxp, L.dst_row)
    raw = [t.clone() for t in (dgate, dw1, dw3, dw2)]
    norm = ops.clip_grad_norm([dgate, dw1, dw3, dw2], 1.0)
    torch.cuda.synchronize()

    # the same step in float64, the choice taken from the device
    leaf = [t.detach().cpu().double().requires_grad_() for t in (x, gate, w1, w3, w2)]
    X, Wg, W1, W3, W2 = leaf
    ll = X @ Wg.t()
    chosen = idx.cpu().long()
    p = torch.sigmoid(ll) if score == "sigmoid" else torch.softmax(ll, dim=1)
    ww = p.gather(1, chosen)
    ww = 1.5 * (ww / ww.sum(dim=1, keepdim=True) if renorm else ww)
    res = torch.zeros((T, H), dtype=torch.float64)
    for e in range(E):
        t, s = torch.nonzero(chosen == e, as_tuple=True)
        hh = torch.nn.functional.silu(X[t] @ W1[e]) * (X[t] @ W3[e])
        res = res.index_add(0, t, ww[t, s][:, None] * (hh @ W2[e]))
    grads = torch.autograd.grad((res * G.cpu().double()).sum(), leaf)
    u = 2.0 ** -8
    assert _rel(f64(out), res.detach()) <= 3 * u                   # h, y, out
    # dy, gu, dgu, then dxp and dx; the router's part: y, dlogits as read, dx
    assert _rel(f64(dx) + f64(dx_gate), grads[0]) <= 5 * u
    for got, want, n in zip(raw, grads[1:], (3, 4, 4, 3)):  # roundings up to each gradient
        assert _rel(f64(got), want) <= n * u
    total = np.sqrt(sum(float((f64(t) ** 2).sum()) for t in raw))
    assert abs(norm.item() - total) <= 2.0 ** -22 * total and total > 1
    for got, r in zip((dgate, dw1, dw3, dw2), raw):
        assert np.abs(f64(got) - f64(r) / (total + 1e-6)).max() <= \
            (u + 2.0 ** -22) * np.abs(f64(r)).max() / total
