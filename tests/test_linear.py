"""The dense linear layer on the CPU: the oracle's gradients against
differences, and the library's refusals, which return before any launch."""
from __future__ import annotations

import ctypes as C
import os

import numpy as np
import pytest

from oracle import linear as olinear

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "combine_top_router_amd", "libmoe.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")


def test_forward_by_hand():
    y, z = olinear.linear([[1, 2]], [[3, 4], [5, -6]], [0.5, 1], "relu", [[10, 20]])
    assert z.tolist() == [[11.5, -6.0]] and y.tolist() == [[21.5, 20.0]]
    assert abs(olinear.act(np.array([1.0]), "gelu")[0] - 0.841344746068543) < 1e-12
    assert abs(olinear.act(np.array([1.0]), "silu")[0] - 0.731058578630005) < 1e-12


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu"])
def test_gradients_against_differences(name):
    r = np.random.default_rng(2)
    x, w, b, dy = (r.standard_normal(s) for s in ((3, 5), (4, 5), (4,), (3, 4)))
    f = lambda: (olinear.linear(x, w, b, name)[0] * dy).sum()  # noqa: E731
    _, z = olinear.linear(x, w, b, name)
    dx, dw, db, _ = olinear.linear_backward(dy, x, w, name, z)
    h = 1e-5
    for v, g in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(v.shape):
            v[i] += h
            up = f()
            v[i] -= 2 * h
            dn = f()
            v[i] += h
            # third derivatives are a few units: h^2 of them, and 1e-16 * 50 / h of rounding
            assert abs((up - dn) / (2 * h) - g[i]) < 1e-8


def _desc(**kw):
    from combine_top_router_amd import _lib
    p = dict(rows=16, inner=64, cols=32, dtype=0, w_order=0, act=0, y_f32=0, ldx=64, ldw=64,
             ldy=32, ldr=32, ldp=32)
    p.update(kw)
    return _lib.LinearDesc(*(p[f] for f, _ in _lib.LinearDesc._fields_))


@built
@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(inner=0), 1), (dict(cols=0), 1),
    (dict(inner=(1 << 20) + 8, ldx=1 << 21, ldw=1 << 21), 1), (dict(w_order=2), 1),
    (dict(act=4), 1), (dict(act=-1), 1), (dict(y_f32=2), 1), (dict(dtype=2), 2),
    (dict(dtype=7), 2), (dict(ldx=56), 1), (dict(ldw=56), 1), (dict(ldy=31), 1),
    (dict(ldx=(1 << 21) + 8), 1), (dict(inner=60), 2), (dict(ldx=68), 2), (dict(ldw=68), 2),
    (dict(w_order=1, cols=33, ldy=40, ldw=40), 2), (dict(w_order=1, ldw=24), 1),
    (dict(rows=(1 << 31) - 1, cols=1 << 20, ldy=1 << 20), 2),
])
def test_bad_linear_descriptors_are_refused(bad, status):
    from combine_top_router_amd import _lib
    lib = _lib.load()
    d = _desc(**bad)
    fake = C.c_void_p(1 << 20)  # never dereferenced
    big = 1 << 40
    assert lib.moe_linear_workspace_bytes(C.byref(d)) == 0
    assert lib.moe_linear_backward_workspace_bytes(C.byref(d)) == 0
    assert lib.moe_linear(C.byref(d), fake, fake, None, None, fake, None, fake, big, None) == status
    assert lib.moe_linear_backward(C.byref(d), fake, fake, fake, None, fake, fake, None, fake, big,
                                   None) == status


@built
def test_linear_argument_checks_launch_nothing():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    f, g, odd = C.c_void_p(1 << 20), C.c_void_p(2 << 20), C.c_void_p((1 << 20) + 8)
    big = 1 << 40

    def fwd(d=_desc(), x=f, w=f, bias=None, res=None, y=f, pre=None, ws=f, n=big):
        return lib.moe_linear(C.byref(d), x, w, bias, res, y, pre, ws, n, None)

    assert lib.moe_linear(None, f, f, None, None, f, None, f, big, None) == 1
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=odd), dict(w=odd),
               dict(res=f, d=_desc(ldr=24)), dict(pre=g, d=_desc(ldp=24)), dict(pre=f),
               dict(res=g, pre=g), dict(res=f, d=_desc(ldr=40)), dict(res=f, d=_desc(y_f32=1))):
        assert fwd(**kw) == 1, kw
    split = _desc(inner=8192, ldx=8192, ldw=8192)  # few outputs, a long reduction
    need = lib.moe_linear_workspace_bytes(C.byref(split))
    assert need > 0
    assert fwd(d=split, ws=None) == 1 and fwd(d=split, n=need - 1) == 1 and fwd(d=split, ws=odd) == 1
    assert fwd(d=_desc(rows=0), x=None, w=None, y=None, ws=None, n=0) == 0

    def bwd(d=_desc(), dy=f, x=f, w=f, pre=None, dx=f, dw=f, db=None, ws=f, n=big):
        return lib.moe_linear_backward(C.byref(d), dy, x, w, pre, dx, dw, db, ws, n, None)

    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(x=odd), dict(w=odd), dict(dx=odd),
               dict(dw=odd), dict(d=_desc(act=2)), dict(d=_desc(act=2, ldp=24), pre=g),
               dict(ws=None), dict(ws=odd), dict(n=15)):
        assert bwd(**kw) == 1, kw
    assert bwd(dx=None, dw=None) == 0  # nothing is wanted


@built
def test_workspace_does_not_depend_on_strides_or_types():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    for call in (lib.moe_linear_workspace_bytes, lib.moe_linear_backward_workspace_bytes):
        a = call(C.byref(_desc(inner=8192, ldx=8192, ldw=8192)))
        b = call(C.byref(_desc(inner=8192, ldx=9000, ldw=8200, ldy=64, act=3, dtype=1, y_f32=1)))
        assert a == b > 0


def test_a_rank_share_takes_no_shared_expert():
    torch = pytest.importorskip("torch")
    from combine_top_router_amd import MoELayer
    w = torch.zeros((4, 128, 128), dtype=torch.bfloat16)  # refused before anything is on a GPU
    with pytest.raises(ValueError, match="shared expert"):
        MoELayer(16, 128, 8, 2, 128, w, w, w, ep_size=2, local_rank=1, shared=(w[0], w[0], w[0]))


@built
def test_outputs_in_an_operand_are_refused():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    d = _desc()
    at = [C.c_void_p((i + 1) << 20) for i in range(8)]  # never dereferenced
    ws = C.c_void_p(1 << 30)

    def forward(x, w, bias, res, y, pre):
        return lib.moe_linear(C.byref(d), x, w, bias, res, y, pre, ws, 1 << 40, None)

    def backward(dy, x, w, pre, dx, dw, db):
        return lib.moe_linear_backward(C.byref(d), dy, x, w, pre, dx, dw, db, ws, 1 << 40, None)
    for out, operands in ((4, (0, 1, 2)), (5, (0, 1, 2, 3, 4))):
        for i in operands:
            args = at[:6]
            args[out] = args[i]
            assert forward(*args) == 1
    for out, operands in ((4, (0, 1, 2, 3)), (5, (0, 1, 2, 3, 4)), (6, (0, 1, 2, 3, 4, 5))):
        for i in operands:
            args = at[:7]
            args[out] = args[i]
            assert backward(*args) == 1


@built
def test_one_part_is_a_flag_beside_the_activation():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    for act in range(4):
        for call in (lib.moe_linear_workspace_bytes, lib.moe_linear_backward_workspace_bytes):
            long = dict(inner=8192, ldx=8192, ldw=8192)
            assert call(C.byref(_desc(act=act | 16, **long))) == call(C.byref(_desc(act=act, **long))) > 0
    for act in (4 | 16, 32, 16 - 32):
        assert lib.moe_linear_backward_workspace_bytes(C.byref(_desc(act=act))) == 0


@built
def test_products_of_more_tiles_than_a_launch_takes():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    # 2^34 outputs are taken, whatever their shape; 2^40 are not, nor 2^23 tiles (of 512
    # threads: 2^32, where a launch has fewer)
    for rows, cols in ((1 << 20, 1 << 14), (1 << 14, 1 << 20), (1 << 30, 16)):
        d = _desc(rows=rows, cols=cols, ldy=cols)
        assert lib.moe_linear_backward_workspace_bytes(C.byref(d)) > 0, (rows, cols)
    for rows, cols in ((1 << 20, 1 << 20), (1 << 30, 1 << 10), ((1 << 31) - 1, 8)):
        d = _desc(rows=rows, cols=cols, ldy=cols)
        assert lib.moe_linear(C.byref(d), C.c_void_p(1 << 20), C.c_void_p(1 << 21), None, None,
                              C.c_void_p(1 << 22), None, None, 0, None) == 2, (rows, cols)
