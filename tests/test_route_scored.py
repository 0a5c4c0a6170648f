"""Scored routing on the CPU: the oracle against hand-computed choices and its
gradient against differences of its own weights; the library's refusals, which
return before any launch."""
from __future__ import annotations

import ctypes as C
import os

import numpy as np
import pytest

from oracle import route as oroute, route_scored as oscored

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "combine_top_router_amd", "libmoe.so")


def test_groups_bias_and_ties_by_hand():
    # sigmoid(0) = .5 everywhere; the bias decides. Groups {0,1} {2,3} {4,5}.
    logits = np.zeros((1, 6), np.float32)
    bias = np.array([.3, 0, .2, .2, .1, .1], np.float32)
    # two largest: .3, .4, .2 above 1 -> groups 1 and 0 stay; then .3, .2, .2
    idx, w = oscored.route(logits, 3, bias, num_groups=3, top_groups=2, scale=6.0)
    assert idx.tolist() == [[0, 2, 3]] and np.allclose(w, 2.0)
    # largest alone: group 0 (.3), group 1 (.2)
    idx, _ = oscored.route(logits, 2, bias, num_groups=3, top_groups=1, group_rank="max")
    assert idx.tolist() == [[0, 1]]
    # nothing but ties: the lowest groups, the lowest ids
    idx, _ = oscored.route(logits, 4, None, num_groups=3, top_groups=2)
    assert idx.tolist() == [[0, 1, 2, 3]]


def test_renormalised_softmax_without_bias_is_the_plain_router():
    logits = np.random.default_rng(0).standard_normal((50, 24)).astype(np.float32)
    idx, w = oscored.route(logits, 5, score="softmax")
    assert (idx == oroute.select(logits, 5)).all()
    assert np.allclose(w, oroute.weights(logits, idx), atol=1e-15)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_oracle_gradient_against_differences(score, renorm):
    r = np.random.default_rng(1)
    l = r.standard_normal((4, 9))
    idx, _ = oscored.route(l, 3, score=score)
    g = r.standard_normal((4, 3))
    got = oscored.route_backward(l, idx, g, score, renorm, 2.5)
    lf = l.astype(np.float32).astype(np.float64)  # the oracle reads fp32 logits
    h = 2.0 ** -9
    for e in range(9):
        # steps that fp32 holds exactly enough: the step itself is recomputed
        up, dn = (lf + 0).astype(np.float32), (lf + 0).astype(np.float32)
        up[:, e] += np.float32(h)
        dn[:, e] -= np.float32(h)
        step = up[:, e].astype(np.float64) - dn[:, e].astype(np.float64)
        f = lambda x: (oscored.weights(x, idx, score, renorm, 2.5) * g).sum(axis=1)  # noqa: E731
        # second-order differences: error h^2/6 |f'''| <= 2^-18 * 2.5 * sum|g| < 1e-4
        assert np.allclose((f(up) - f(dn)) / step, got[:, e], atol=1e-4)


def test_empty_rows_have_zero_weights_and_gradients():
    l = np.full((2, 4), -np.inf, np.float32)
    l[1, 2] = np.nan
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            idx, w = oscored.route(l, 2, score=score, renormalise=renorm)
            assert idx.tolist() == [[0, 1], [0, 1]] and not w.any()
            assert not oscored.route_backward(l, idx, np.ones((2, 2)), score, renorm).any()


@pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")
@pytest.mark.parametrize("bad", [
    dict(num_tokens=-1), dict(num_experts=0), dict(num_experts=1025), dict(top_k=0),
    dict(top_k=17), dict(score=2), dict(score=-1), dict(num_groups=0), dict(num_groups=3),
    dict(num_experts=130, num_groups=65), dict(top_groups=0), dict(top_groups=5),
    dict(top_groups=1, num_groups=8, top_k=5), dict(group_rank=2), dict(renormalise=2),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(num_tokens=1 << 31),
])
def test_bad_route_descriptors_are_refused(bad):
    from combine_top_router_amd import _lib
    lib = _lib.load()
    p = dict(num_tokens=16, num_experts=32, top_k=4, score=1, num_groups=4, top_groups=2,
             group_rank=1, renormalise=1, scale=1.0)
    p.update(bad)
    d = _lib.RouteDesc(*(p[f] for f, _ in _lib.RouteDesc._fields_))
    fake = C.c_void_p(1 << 20)  # never dereferenced
    assert lib.moe_route_scored(C.byref(d), fake, fake, fake, fake, None) == 1
    assert lib.moe_route_scored_backward(C.byref(d), fake, fake, fake, fake, None) == 1


@pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")
def test_null_pointers_and_empty_batches():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    d = _lib.RouteDesc(16, 32, 4, 1, 4, 2, 1, 1, 1.0)
    fake = C.c_void_p(1 << 20)
    assert lib.moe_route_scored(None, fake, fake, fake, fake, None) == 1
    for i in (0, 2, 3):
        args = [fake] * 4
        args[i] = None
        assert lib.moe_route_scored(C.byref(d), *args, None) == 1
    for i in range(4):
        args = [fake] * 4
        args[i] = None
        assert lib.moe_route_scored_backward(C.byref(d), *args, None) == 1
    d.num_tokens = 0
    assert lib.moe_route_scored(C.byref(d), None, None, None, None, None) == 0
    assert lib.moe_route_scored_backward(C.byref(d), None, None, None, None, None) == 0


@pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")
def test_more_tokens_than_a_launch_has_lanes_for_are_refused():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    d = _lib.RouteDesc(1 << 26, 8, 1, 1, 1, 1, 1, 1, 1.0)
    fake = C.c_void_p(1 << 20)  # never dereferenced
    assert lib.moe_route_scored(C.byref(d), fake, fake, fake, fake, None) == 1
    assert lib.moe_route_scored_backward(C.byref(d), fake, fake, fake, fake, None) == 1
