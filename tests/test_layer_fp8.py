"""What MoELayer refuses of its norm and 8-bit options, before anything is on a GPU."""
import math

import pytest

torch = pytest.importorskip("torch")
from combine_top_router_amd import MoELayer  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def _layer(H=128, I=128, **kw):
    w = torch.zeros((8, H, I), dtype=BF)
    return MoELayer(16, H, 8, 2, I, w, w, torch.zeros((8, I, H), dtype=BF), **kw)


@pytest.mark.parametrize("norm,error", [
    (torch.ones(128, dtype=BF), TypeError), (torch.ones(129), ValueError), ("ones", TypeError),
    (torch.ones(128).to("meta"), ValueError),
])
def test_norm(norm, error):
    with pytest.raises(error, match="norm"):
        _layer(norm=norm)


@pytest.mark.parametrize("eps", [math.nan, math.inf, -1e-6])
def test_eps(eps):
    with pytest.raises(ValueError, match="eps"):
        _layer(norm=torch.ones(128), eps=eps)


def test_fp8():
    with pytest.raises(ValueError, match="gathers"):
        _layer(fp8=True, gather=False)
    with pytest.raises(ValueError, match="fp8_fast"):
        _layer(fp8_fast=True)
    with pytest.raises(ValueError, match="multiples of 128"):
        _layer(H=192, fp8=True)
    with pytest.raises(ValueError, match="multiples of 128"):
        _layer(I=64, fp8=True)
    s = torch.zeros((128, 64), dtype=BF)
    with pytest.raises(ValueError, match="multiples of 128"):
        _layer(fp8=True, shared=(s, s, s.t().contiguous()))
