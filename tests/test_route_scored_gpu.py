"""GPU parity of the scored router against the float64 oracle: equal experts,
weights and gradients within their roundings."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import route_scored as oscored

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_top_router_amd")
ops = moe.ops

U = 2.0 ** -24  # half a step of fp32, relative

# (T, E, k, groups, top_groups): every lane layout, odd sizes, the limits
SHAPES = [
    (1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (3, 7, 7, 1, 1), (257, 60, 4, 1, 1), (33, 64, 8, 8, 3),
    (65, 160, 6, 8, 3), (129, 256, 8, 8, 4), (17, 66, 5, 6, 2), (40, 18, 3, 9, 4),
    (31, 256, 16, 1, 1), (50, 384, 8, 1, 1), (9, 1024, 16, 64, 3), (5, 1023, 16, 33, 2),
    (7, 1000, 12, 5, 2), (21, 64, 8, 64, 9), (6, 16, 16, 2, 2), (1000, 128, 8, 1, 1),
    # more tokens than get a wavefront each
    (2100, 256, 8, 8, 4), (2500, 128, 8, 1, 1), (2200, 60, 4, 6, 2), (3001, 33, 7, 1, 1),
    (2057, 500, 16, 4, 3),
]


def _same(got, want, slack=0.0):
    """Within one fp32 rounding of the float64 value (and of its smallest steps)."""
    got = got.cpu().double().numpy()
    tol = U * (1 + 1e-6) * np.abs(want) + 2.0 ** -149 + slack
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def _check(logits, k, bias, score, groups, top_groups, rank, renorm, scale):
    idx, w = ops.route_scored(logits, k, bias, score, groups, top_groups, rank, renorm, scale)
    torch.cuda.synchronize()
    ln = logits.cpu().numpy()
    want_idx, want_w = oscored.route(ln, k, None if bias is None else bias.cpu().numpy(), score,
                                     groups, top_groups, rank, renorm, np.float32(scale).item())
    assert (idx.cpu().numpy() == want_idx).all()
    # A weight in fp32: expf (2 half steps), 1 + e and its reciprocal (2), a sum across at
    # most 64 lanes (6, on top of its terms' 4), the quotient and the scale (2): 16 half steps.
    # The softmax's arguments are rounded differences, |l - max| half steps for the term
    # and, weighted by the terms, for the sum, which takes up to 38 additions if over all experts.
    half_steps = 16.0
    if score == "softmax":
        l = oscored._clean(ln)
        sel = np.take_along_axis(l, want_idx.astype(np.int64), axis=1)
        with np.errstate(invalid="ignore"):
            far = np.where(sel == -np.inf, 0.0,
                           np.abs(sel - (sel if renorm else l).max(axis=1, keepdims=True)))
            every = np.where(l == -np.inf, 0.0, np.abs(l - l.max(axis=1, keepdims=True)))
        p = oscored.scores(ln, score)
        mean = (p * np.where(p > 0, every, 0.0)).sum(axis=1, keepdims=True)
        # where fp64 takes over (|l - max| above 80) nothing of this is lost: 80 at most
        half_steps = 16 + np.minimum(far, 80) + \
            (np.minimum(far, 80).max(axis=1, keepdims=True) if renorm else 38 + mean)
    _same(w, want_w, np.abs(want_w) * half_steps * U)
    return idx


def _check_grad(logits, idx, k, score, renorm, scale, seed=0):
    T = logits.shape[0]
    g = torch.randn((T, k), generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    out = ops.route_scored_backward(logits, idx, g, score, renorm, scale)
    torch.cuda.synchronize()
    ln, gn = logits.cpu().numpy(), g.cpu().double().numpy()
    want = oscored.route_backward(ln, idx.cpu().numpy(), gn, score, renorm,
                                  np.float32(scale).item())
    big = abs(scale) * np.abs(gn).max(axis=1, keepdims=True, initial=0.0)
    if score == "softmax" and not renorm:
        # p in fp32: expf (2 half steps), its argument's rounding (|l - max| half steps,
        # twice: numerator and, at most as much, the sum), the sum's at most 22 additions
        # in sequence, and 6 products and quotients; times |g| + |inner| <= 2 max|g|
        l = oscored._clean(ln)
        with np.errstate(invalid="ignore"):
            far = np.where(l == -np.inf, 0.0, np.abs(l - l.max(axis=1, keepdims=True)))
        p = oscored.scores(ln, score)
        slack = 2 * big * p * (32 + 2 * far) * U
    else:
        slack = 1e-13 * k * big  # fp64 sums of k terms, before the one rounding
    _same(out, want, slack)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_weights_and_gradient(shape, score):
    T, E, k, groups, top = shape
    print("CASE route_scored", shape, score, flush=True)
    gen = torch.Generator("cuda").manual_seed(T * 1009 + E)
    logits = torch.randn((T, E), generator=gen, device="cuda") * 2
    bias = torch.randn((E,), generator=gen, device="cuda") * 0.1
    for rank in ("top2", "max"):
        for b in (None, bias):
            for renorm, scale in ((True, 2.5), (False, 1.0)):
                idx = _check(logits, k, b, score, groups, top, rank, renorm, scale)
    for renorm in (True, False):
        _check_grad(logits, idx, k, score, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_masked_experts_and_values_that_are_not_finite(score):
    inf, nan = float("inf"), float("nan")
    rows = torch.zeros((12, 32))
    rows[1] = -inf
    rows[2] = nan
    rows[3, 5] = inf
    rows[4, ::2] = -inf
    rows[5, 7], rows[5, 9] = nan, 3.0
    rows[6] = 200.0   # saturated sigmoids tie
    rows[7] = torch.arange(32) * 1e30
    rows[8] = -torch.arange(32) * 1e30
    rows[9] = torch.finfo(torch.float32).min
    rows[10] = torch.tensor([1.0, -0.0, 0.0, 1.0] * 8)
    rows[11, 31] = -100.0
    logits = rows.cuda()
    bias = torch.zeros(32)
    bias[3], bias[4], bias[8] = inf, -inf, nan
    for b in (None, torch.zeros(32).cuda(), bias.cuda()):
        for groups, top in ((1, 1), (4, 2), (32, 9), (8, 8)):
            for renorm in (True, False):
                idx = _check(logits, 6, b, score, groups, top, "top2", renorm, 1.5)
    for renorm in (True, False):
        _check_grad(logits, idx, 6, score, renorm, 1.5)


def test_close_scores_are_told_apart_as_in_64_bits():
    # logits one fp32 step apart near 16: their sigmoids are 1 - 1.1e-7, equal in fp32,
    # and a bias that differs by fractions of an fp32 step of the score
    T, E = 64, 64
    gen = torch.Generator("cuda").manual_seed(3)
    steps = torch.randint(0, 50, (T, E), generator=gen, device="cuda")
    logits = 16.0 + steps.float() * 2.0 ** -19
    bias = torch.randint(0, 3, (E,), generator=gen, device="cuda").float() * 2.0 ** -33
    for groups, top in ((1, 1), (8, 3)):
        for score in ("sigmoid", "softmax"):
            for b in (None, bias):
                # (sums of two would tie to within fp64's own rounding here)
                _check(logits, 8, b, score, groups, top, "max", True, 1.0)


@pytest.mark.parametrize("T,E,k,groups,top", [(40, 256, 8, 1, 1), (2100, 256, 8, 8, 4),
                                              (17000, 128, 7, 1, 1), (17000, 256, 8, 8, 4),
                                              (4200, 500, 16, 4, 2), (9000, 60, 4, 6, 2)])
def test_ties_between_experts_of_different_lanes(T, E, k, groups, top):
    """Logits on a coarse grid: most tokens have ties among the chosen and at the border."""
    print("CASE ties", T, E, k, groups, top, flush=True)
    gen = torch.Generator("cuda").manual_seed(T + E)
    logits = torch.round(torch.randn((T, E), generator=gen, device="cuda") * 4) / 4
    bias = torch.round(torch.randn((E,), generator=gen, device="cuda") * 2) / 8
    for score in ("sigmoid", "softmax"):
        # one expert's value decides a group's rank: sums of two different pairs that agree
        # but for fp64's own rounding are no ties
        for b in (None, bias):
            _check(logits, k, b if score == "sigmoid" else None, score, groups, top, "max", True, 1.0)


def test_repeated_and_foreign_ids_in_the_backward():
    logits = torch.randn((5, 20), generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    idx = torch.tensor([[3, 3, 3, 1], [-1, 20, 4, 4], [-5, -1, 99, 20], [0, 19, 0, 19],
                        [7, 8, 9, 7]], dtype=torch.int32, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _check_grad(logits, idx, 4, score, renorm, 1.0)


def test_unaligned_rows_and_given_outputs():
    base = torch.randn((40 * 128 + 1,), generator=torch.Generator("cuda").manual_seed(5),
                       device="cuda")
    logits = base[1:].view(40, 128)  # 4 bytes past a 16-byte boundary
    idx = torch.full((41, 8), -7, dtype=torch.int32, device="cuda")
    w = torch.full((41, 8), -7.0, device="cuda")
    ops.route_scored(logits, 8, topk_idx=idx[:40], topk_w=w[:40])
    want, _ = oscored.route(logits.cpu().numpy(), 8)
    assert (idx[:40].cpu().numpy() == want).all()
    assert (idx[40] == -7).all() and (w[40] == -7).all()
    _check_grad(logits, idx[:40].contiguous(), 8, "softmax", False, 1.0)


def test_plain_router_agrees():
    logits = torch.randn((4096, 128), generator=torch.Generator("cuda").manual_seed(6),
                         device="cuda")
    idx, w = ops.route(logits, 8)
    idx2, w2 = ops.route_scored(logits, 8, score="softmax")
    assert torch.equal(idx, idx2)
    assert torch.allclose(w, w2, rtol=1e-5, atol=0)


def test_empty_batch_and_refusals():
    z = torch.empty((0, 32), device="cuda")
    idx, w = ops.route_scored(z, 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    assert ops.route_scored_backward(z, idx, w).shape == (0, 32)
    x = torch.zeros((4, 32), device="cuda")
    with pytest.raises(TypeError):
        ops.route_scored(x.double(), 4)
    with pytest.raises(ValueError):
        ops.route_scored(x.t(), 4)
    with pytest.raises(ValueError):
        ops.route_scored(x, 4, score="cosine")
    with pytest.raises(ValueError):
        ops.route_scored(x, 4, bias=torch.zeros(31, device="cuda"))
    with pytest.raises(ValueError):
        ops.route_scored(x.cpu(), 4)
    with pytest.raises(moe.MoEError):
        ops.route_scored(x, 17)
    with pytest.raises(moe.MoEError):
        ops.route_scored(x, 4, num_groups=5)


def test_captured_call_replays_on_new_logits():
    logits = torch.zeros((300, 256), device="cuda")
    bias = torch.zeros((256,), device="cuda")
    g = torch.ones((300, 8), device="cuda")
    idx = torch.empty((300, 8), dtype=torch.int32, device="cuda")
    w, grad = torch.empty((300, 8), device="cuda"), torch.empty((300, 256), device="cuda")

    def step():
        ops.route_scored(logits, 8, bias, "sigmoid", 8, 4, topk_idx=idx, topk_w=w)
        ops.route_scored_backward(logits, idx, g, out=grad)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    gen = torch.Generator("cuda").manual_seed(7)
    for rep in range(3):
        logits.copy_(torch.randn((300, 256), generator=gen, device="cuda"))
        bias.copy_(torch.randn((256,), generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (idx, w, grad)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (idx, w, grad)))


@pytest.mark.parametrize("E,k", [(8, 7), (8, 8), (9, 8), (16, 15), (16, 16), (32, 16)])
@pytest.mark.parametrize("T", [3, 2100])
def test_empty_rows_where_nearly_every_expert_is_chosen(T, E, k):
    """Rows of -inf or NaN alone, with no expert left over or one: all scores are
    0, so the lowest ids in order, also beside rows that are not empty."""
    print("CASE empty rows", T, E, k, flush=True)
    logits = torch.randn((T, E), generator=torch.Generator("cuda").manual_seed(E), device="cuda")
    logits[0::3] = float("-inf")
    logits[1::6] = float("nan")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _check(logits, k, None, score, 1, 1, "max", renorm, 1.0)


@pytest.mark.parametrize("groups,top", [(1, 1), (8, 3)])
def test_scores_below_the_normal_range_are_told_apart_as_in_64_bits(groups, top):
    """Softmax scores of a few smallest steps of fp32, far below the first expert's."""
    print("CASE tiny scores", groups, top, flush=True)
    gen = torch.Generator("cuda").manual_seed(11)
    logits = -98.0 - 5.5 * torch.rand((2100, 64), generator=gen, device="cuda")
    logits[:, 5] = 0.0
    for renorm in (True, False):
        _check(logits, 8, None, "softmax", groups, top, "max", renorm, 1.0)
    _check(logits, 8, torch.zeros(64, device="cuda"), "softmax", groups, top, "max", True, 1.0)


def test_arguments_past_32_bits_are_refused():
    x = torch.zeros((4, 32), device="cuda")
    for bad in (dict(top_k=2 ** 32 + 4), dict(num_groups=2 ** 32 + 1),
                dict(num_groups=1 - 2 ** 32), dict(top_groups=2 ** 32 + 1)):
        with pytest.raises(ValueError):
            ops.route_scored(x, **{"top_k": 4, **bad})


@pytest.mark.parametrize("B", [64.0, 1e4, 1e6])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_ranks_whose_two_values_cancel(B, score):
    """Biases +B and -B inside each group: a rank is the sum of two values that are
    rounded at B's size and leave one of the scores' size."""
    T, E, groups, top = 100_000, 16, 8, 4
    print("CASE cancel", B, score, flush=True)
    gen = torch.Generator("cuda").manual_seed(int(B))
    logits = torch.randn((T, E), generator=gen, device="cuda")
    bias = torch.tensor([B, -B], device="cuda").repeat(E // 2)
    _check(logits, 4, bias, score, groups, top, "top2", True, 1.0)
    # one expert far above its group's other one, and a group of -inf beside
    bias = torch.tensor([B, -1.0, B, -B, 0.5, -0.5, -float("inf"), 3.0] * 2, device="cuda")
    _check(logits, 4, bias, score, groups, top, "top2", True, 1.0)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[4] < s[3] and s[1] >= 2 * s[3]],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_close_group_ranks_are_told_apart_as_in_64_bits(shape, score):
    """The best two of each group differ between groups by a few 2^-20 in the logits: ranks
    from equal down to 2^-43 apart (pairs of equal sum), far above fp64's own rounding."""
    T, E, k, groups, top = shape
    print("CASE close ranks", shape, score, flush=True)
    gen = torch.Generator("cuda").manual_seed(T + E)
    size = E // groups
    logits = torch.randn((T, groups, size), generator=gen, device="cuda") * 0.2 - 3
    best = torch.rand((T, groups, size), generator=gen, device="cuda").topk(2, dim=2).indices
    steps = torch.randint(0, 8, (T, groups, 2), generator=gen, device="cuda").float() * 2.0 ** -20
    logits.scatter_(2, best, 1.5 + steps)
    logits = logits.view(T, E).contiguous()
    # one value for a group: sums of the same two scores stay equal in any order
    bias = torch.randint(0, 4, (groups,), generator=gen, device="cuda").float() * 2.0 ** -21
    for b in (None, bias.repeat_interleave(size).contiguous()):
        for renorm in (True, False):
            _check(logits, k, b, score, groups, top, "top2", renorm, 1.0)


@pytest.mark.parametrize("E,k", [(8, 2), (64, 8), (256, 8), (500, 16), (1024, 4)])
@pytest.mark.parametrize("far", [3.0, 12.0, 18.0, 60.0])
def test_softmax_gradient_of_a_confident_token(E, k, far):
    """One expert holds nearly all of a token: dl_e = p_e (g_e (1 - p_e) - the others' g_i p_i),
    every term of which p's own relative error bounds (g_e - inner would cancel)."""
    T = 300
    print("CASE confident", E, k, far, flush=True)
    gen = torch.Generator("cuda").manual_seed(E + int(far))
    logits = torch.randn((T, E), generator=gen, device="cuda") - far
    best = torch.randint(0, E, (T, 1), generator=gen, device="cuda")
    logits.scatter_(1, best, 0.5)
    logits[1::3, 0] = logits[2::3, E - 1] = 0.5  # also two that share a token
    idx, _ = ops.route_scored(logits, k, score="softmax", renormalise=False)
    idx[0, 1] = idx[0, 0]  # and one that is named twice
    g = torch.randn((T, k), generator=gen, device="cuda")
    out = ops.route_scored_backward(logits, idx, g, "softmax", False, 1.5)
    torch.cuda.synchronize()
    l, gn, ix = logits.cpu().double().numpy(), g.cpu().double().numpy(), idx.cpu().long().numpy()
    p = oscored.scores(l, "softmax")
    G = np.zeros((T, E))
    np.add.at(G, (np.arange(T)[:, None], ix), gn)
    # 1 - p_e: the sum of the other scores
    rest = np.stack([np.delete(p, e, axis=1).sum(axis=1) for e in range(E)], axis=1)
    inner = G * p
    others = np.stack([np.delete(inner, e, axis=1).sum(axis=1) for e in range(E)], axis=1)
    want = 1.5 * p * (G * rest - others)
    # (summed without e: as a total less e's own, 1 + 1e-26 - 1, the others would be lost)
    size = np.stack([np.delete(np.abs(inner), e, axis=1).sum(axis=1) for e in range(E)], axis=1)
    size = 1.5 * p * (np.abs(G) * rest + size)
    size[0] += 1.5 * p[0] * p[0] * np.abs(gn[0]).max() * 2  # (the two named alike may cancel)
    # each score: 32 half steps and 2 of |l - max|, as in _check_grad; two scores to a term,
    # and the sum of the others, off by no more; the rest of the products 8
    away = np.abs(l - l.max(axis=1, keepdims=True))
    half_steps = 3 * 32 + 2 * away + 4 * away.max(axis=1, keepdims=True) + 8
    _same(out, want, size * half_steps * U + 2.0 ** -126)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_weights_are_rounded_once(shape):
    """Sigmoid weights, and renormalised softmax ones: fp64 up to half a step of fp32."""
    T, E, k, groups, top = shape
    print("CASE weights", shape, flush=True)
    gen = torch.Generator("cuda").manual_seed(T * 31 + E)
    logits = torch.randn((T, E), generator=gen, device="cuda") * 3
    for score, renorm, scale in (("sigmoid", True, 2.5), ("sigmoid", False, 1.0),
                                 ("softmax", True, 16.0), ("sigmoid", True, 0.3)):
        idx, w = ops.route_scored(logits, k, None, score, groups, top, "max", renorm, scale)
        torch.cuda.synchronize()
        want = oscored.weights(logits.cpu().numpy(), idx.cpu().numpy(), score, renorm,
                               np.float32(scale).item())
        _same(w, want)
