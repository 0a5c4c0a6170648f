"""GPU parity of the gradient norm and clipping against float64."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_top_router_amd")
ops = moe.ops

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def f64(t):
    return t.detach().cpu().double().numpy()


def _grads(gen, specs, std=0.05):
    """specs: (numel, dtype, offset into a larger buffer in elements)."""
    out = []
    for n, dtype, off in specs:
        base = (torch.randn((n + off,), generator=gen, device="cuda") * std).to(dtype)
        out.append(base[off:])
    return out


def _want(grads, max_norm):
    total = math.fsum(float((f64(g) ** 2).sum()) for g in grads)
    norm = math.sqrt(total)
    ratio = max_norm / (norm + 1e-6)
    coef = np.float32(1.0 if ratio >= 1 else ratio)
    # the product of two fp32 values is exact in float64 but for its last bits: rounding it
    # to fp32 and then to the type is what the call does
    return total, norm, [torch.from_numpy((f64(g) * np.float64(coef)).astype(np.float32)).to(g.dtype)
                         for g in grads]


CASES = {
    "one": [(1, F32, 0)],
    "odd": [(7, BF, 0), (9, FP, 1), (5, F32, 3), (0, BF, 0), (4097, BF, 1)],
    "chunks": [(32768, BF, 0), (32769, FP, 0), (16384, F32, 0), (16385, F32, 1), (65537, BF, 8)],
    "many": [(1 + 37 * i, (BF, FP, F32)[i % 3], i % 4) for i in range(300)],
    "long": [(40_000_003, BF, 0), (3_000_001, F32, 0), (10, FP, 0)],
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("bound", [0.5, 1e6])
def test_norm_and_scaled_gradients(name, bound):
    print("CASE clip", name, bound, flush=True)
    gen = torch.Generator("cuda").manual_seed(len(name))
    grads = _grads(gen, CASES[name], 5.0 if name == "one" else 0.05)
    total, norm, want = _want(grads, bound)
    s = ops.grad_sumsq(grads)
    out = [torch.full_like(g, 3.0) for g in grads]
    got = ops.clip_grads(grads, s, bound, out=out)
    torch.cuda.synchronize()
    # fp64 sums of fewer than 2^26 terms: 2^-53 each at most
    assert abs(s.item() - total) <= 2.0 ** -26 * total
    assert abs(got.item() - norm) <= (2.0 ** -24 + 2.0 ** -25) * norm
    for o, w in zip(out, want):
        o = o.cpu()
        # the coefficient comes from a sum in another order: it may round to the next fp32
        # (and the product to the next value of the type, a smallest subnormal at least)
        step = torch.finfo(o.dtype).eps * np.abs(f64(w)) + torch.finfo(o.dtype).smallest_normal * \
            torch.finfo(o.dtype).eps
        assert (np.abs(f64(o) - f64(w)) <= step).all()
        if o.numel():
            assert (o == w).float().mean() >= (0.9 if o.numel() > 100 and o.dtype != F32 else 0.0)
    # in place, both calls at once
    got2 = ops.clip_grad_norm(grads, bound)
    torch.cuda.synchronize()
    assert torch.equal(got, got2) and all(torch.equal(a, b) for a, b in zip(grads, out))


def test_values_around_views_are_left_alone():
    base = torch.ones((1000,), dtype=BF, device="cuda")
    ops.clip_grad_norm([base[3:500], base[501:999]], 0.1)
    torch.cuda.synchronize()
    edge = [0, 1, 2, 500, 999]
    assert (base[edge] == 1).all()
    base[edge] = 0
    assert base.float().max().item() < 0.01


def test_same_sum_every_time_and_a_tensor_twice():
    gen = torch.Generator("cuda").manual_seed(2)
    grads = _grads(gen, CASES["long"])
    a = [ops.grad_sumsq(grads) for _ in range(3)]
    b = ops.grad_sumsq(grads + grads)
    torch.cuda.synchronize()
    assert a[0].item() == a[1].item() == a[2].item()
    assert abs(b.item() - 2 * a[0].item()) <= 2.0 ** -26 * b.item()


def test_extremes():
    big = torch.full((100,), 3e38, device="cuda")
    s = ops.grad_sumsq([big])
    torch.cuda.synchronize()
    assert abs(s.item() - 100 * float(np.float32(3e38)) ** 2) <= 1e-12 * s.item()
    n = ops.clip_grad_norm([big], 1.0)  # 3e39 does not fit fp32: the norm says so, the scale holds
    torch.cuda.synchronize()
    assert n.item() == math.inf and torch.allclose(big, torch.full_like(big, 0.1), rtol=1e-5)
    tiny = torch.full((64,), 2.0 ** -140, device="cuda")
    s = ops.grad_sumsq([tiny])
    torch.cuda.synchronize()
    assert s.item() == 64 * 2.0 ** -280
    zero = torch.zeros((9,), dtype=FP, device="cuda")
    assert ops.clip_grad_norm([zero], 0.0).item() == 0 and not zero.any()
    for bad, same in ((float("inf"), lambda t: t[1].isnan() and t[0] == 0),
                      (float("nan"), lambda t: t.isnan().all())):
        t = torch.tensor([1.0, bad], device="cuda")
        n = ops.clip_grad_norm([t], 1.0)
        torch.cuda.synchronize()
        assert not math.isfinite(n.item()) and same(t)
    keep = torch.tensor([3.0, 4.0], device="cuda")
    assert ops.clip_grad_norm([keep], math.inf).item() == 5.0 and keep.tolist() == [3.0, 4.0]


def test_empty_tensors():
    e = torch.empty((0, 4), dtype=BF, device="cuda")
    n = ops.clip_grad_norm([e], 1.0)
    assert n.item() == 0.0


def test_sums_of_two_shares_added():
    # two ranks holding different parameters: their sums added, then each clips its own
    gen = torch.Generator("cuda").manual_seed(3)
    a, b = _grads(gen, [(5000, BF, 0)]), _grads(gen, [(7000, F32, 0)])
    both = [t.clone() for t in a + b]
    s = ops.grad_sumsq(a) + ops.grad_sumsq(b)
    na, nb = ops.clip_grads(a, s, 0.7), ops.clip_grads(b, s, 0.7)
    n = ops.clip_grad_norm(both, 0.7)
    torch.cuda.synchronize()
    assert na.item() == nb.item() and abs(n.item() - na.item()) <= 2.0 ** -23 * n.item()
    assert abs(math.sqrt(sum(float((f64(t) ** 2).sum()) for t in a + b)) - 0.7) < 0.7 * 2.0 ** -7


def test_refusals():
    t = torch.ones((8, 8), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        ops.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        ops.clip_grad_norm([t.cpu()], 1.0)
    with pytest.raises(TypeError):
        ops.clip_grad_norm([t.double()], 1.0)
    with pytest.raises(ValueError):
        ops.clip_grad_norm([t.t()[:4]], 1.0)
    with pytest.raises(ValueError):
        ops.clip_grad_norm([t], 1.0, out=[torch.ones((64,), dtype=BF, device="cuda")])
    with pytest.raises(TypeError):
        ops.clip_grad_norm([t], 1.0, out=[t.half()])
    with pytest.raises(moe.MoEError):
        ops.clip_grad_norm([t], -1.0)
    with pytest.raises(moe.MoEError):
        ops.clip_grad_norm([t, t], 1.0)
    with pytest.raises(TypeError):
        ops.clip_grads([t], torch.zeros((1,), device="cuda"), 1.0)


def test_captured_call_replays():
    gen = torch.Generator("cuda").manual_seed(4)
    grads = _grads(gen, [(5001, BF, 0), (70000, F32, 0), (33, FP, 1)])
    out = [torch.empty_like(g) for g in grads]
    norm = torch.empty((1,), device="cuda")

    def step():
        ops.clip_grad_norm(grads, 0.3, out=out, norm=norm)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        for g in grads:
            g.copy_(torch.randn(g.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out + [norm]]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, out + [norm]))


@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_no_bound_leaves_gradients_of_an_infinite_norm(bad):
    for dtype in (BF, FP, F32):
        t = torch.tensor([1.0, bad, -3.0], dtype=dtype, device="cuda")
        out = torch.zeros_like(t)
        n = ops.clip_grad_norm([t], math.inf, out=[out])
        m = ops.clip_grad_norm([t], math.inf)
        torch.cuda.synchronize()
        assert n.item() == m.item() == math.inf
        assert t.tolist() == out.tolist() == [1.0, bad, -3.0]
    t = torch.tensor([1.0, math.nan], device="cuda")  # a NaN norm reaches every element
    assert math.isnan(ops.clip_grad_norm([t], math.inf).item()) and t.isnan().all()
