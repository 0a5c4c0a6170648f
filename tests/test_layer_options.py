"""What MoELayer refuses at its construction, before anything is on a GPU."""
import math

import pytest

torch = pytest.importorskip("torch")
from combine_top_router_amd import MoELayer, Router  # noqa: E402

T, H, E, K, I, IS = 16, 128, 8, 2, 128, 64
BF = torch.bfloat16


def _layer(**kw):
    w = torch.zeros((E, H, I), dtype=BF)
    return MoELayer(T, H, E, K, I, w, w, torch.zeros((E, I, H), dtype=BF), **kw)


def _z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("gate,error", [
    (_z(H, E), ValueError), (_z(E, H + 8), ValueError), (_z(E + 1, H), ValueError),
    (_z(E, H, dtype=torch.float32), TypeError), ("gate", TypeError),
    (_z(E, H, dtype=BF).to("meta"), ValueError),
])
def test_gate(gate, error):
    with pytest.raises(error, match="gate_w"):
        _layer(gate_w=gate)


@pytest.mark.parametrize("router,error,what", [
    ("sigmoid", TypeError, "router"), (Router(score="cosine"), ValueError, "router.score"),
    (Router(group_rank="sum"), ValueError, "router.group_rank"),
    (Router(num_groups=3), ValueError, "router.num_groups"),
    (Router(num_groups=0), ValueError, "router.num_groups"),
    (Router(num_groups=4, top_groups=5), ValueError, "router.top_groups"),
    (Router(top_groups=0), ValueError, "router.top_groups"),
    (Router(num_groups=8, top_groups=1), ValueError, "top_k"),
    (Router(scale=math.inf), ValueError, "router.scale"),
    (Router(scale=math.nan), ValueError, "router.scale"),
    (Router(bias=_z(E)), TypeError, "router.bias"),
    (Router(bias=_z(E + 1, dtype=torch.float32)), ValueError, "router.bias"),
    (Router(bias=_z(E, dtype=torch.float32).to("meta")), ValueError, "router.bias"),
])
def test_router(router, error, what):
    with pytest.raises(error, match=what):
        _layer(router=router)


@pytest.mark.parametrize("shared,error,what", [
    ((_z(H, IS), _z(H, IS)), ValueError, "shared"),
    ((_z(H, IS), _z(H, IS), _z(H, IS)), ValueError, "shared w2"),
    ((_z(H, IS), _z(H, IS + 8), _z(IS, H)), ValueError, "shared w3"),
    ((_z(H + 8, IS), _z(H, IS), _z(IS, H)), ValueError, "shared w1"),
    ((None, _z(H, IS), _z(IS, H)), TypeError, "shared w1"),
    ((_z(H, IS), _z(H, IS, dtype=torch.float16), _z(IS, H)), TypeError, "shared w3"),
])
def test_shared(shared, error, what):
    with pytest.raises(error, match=what):
        _layer(shared=shared)
