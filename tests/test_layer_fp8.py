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


@pytest.mark.parametrize("hidden", [16392, 20, 4])
def test_norm_of_a_width_that_its_call_refuses(hidden):
    with pytest.raises(ValueError, match="norm needs a hidden size"):
        _layer(H=hidden, norm=torch.ones(hidden))


@pytest.mark.parametrize("tokens,hidden", [(1 << 24, 128), (1 << 23, 256), ((1 << 31) // 384 + 1, 384)])
def test_fp8_of_more_rows_than_its_gather_reaches(tokens, hidden):
    w = torch.zeros((1, hidden, 128), dtype=BF)
    with pytest.raises(ValueError, match="tokens"):
        MoELayer(tokens, hidden, 1, 1, 128, w, w, torch.zeros((1, 128, hidden), dtype=BF), fp8=True)
