"""The 8-bit and norm calls without a GPU: the oracle's pins, and the refusals of the
C ABI, none of which reaches a kernel."""
import ctypes as C
import os

import numpy as np
import pytest

from oracle import fp8, norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "combine_top_router_amd", "libmoe.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")


def test_e4m3_values():
    v = fp8.VALUES
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0
    assert v[0xb8] == -1.0 and np.isnan(v[0x7f]) and np.isnan(v[0xff]) and v[0x80] == 0
    assert (np.diff(v[:127]) > 0).all()


def test_e4m3_rounding():
    v = fp8.VALUES[:127]
    assert (fp8.encode(v) == np.arange(127)).all()
    assert (fp8.encode(-v[1:]) == np.arange(1, 127) + 128).all()
    mid = (v[1:] + v[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert (fp8.encode(mid) == even).all()
    assert (fp8.encode(np.nextafter(mid, 0)) == np.arange(126)).all()
    assert (fp8.encode(np.nextafter(mid, 1e9)) == np.arange(1, 127)).all()
    assert fp8.encode(464.0) == 0x7e and fp8.encode(464.1) == 0x7f and fp8.encode(np.inf) == 0x7f
    assert fp8.encode(np.nan) & 0x7f == 0x7f


def test_e4m3_rounding_is_that_of_torch():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(1).normal(size=20000).astype(np.float32) * 60
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (got == fp8.encode(np.clip(x, -448, 448)))[np.abs(x) < 448].all()


def test_scales_by_hand():
    x = np.zeros((2, 200), np.float32)
    x[0, 3], x[0, 5], x[0, 130] = 448 * 4, 4, -2
    x[1, 199], x[1, 0] = np.inf, np.nan
    q, s = fp8.rows(x)
    assert s[0, 0] == 4 and s[0, 1] == np.float32(2) / np.float32(448)
    assert (s[1] == np.float32(2.0 ** -126)).all()
    d = fp8.decode(q)
    assert d[0, 3] == 448 and d[0, 5] == 1 and d[0, 130] == -448 and np.isnan(d[1, 199])
    assert np.isnan(d[1, 0]) and (d[1, 1:199] == 0).all()
    got = fp8.row_values(q, s)
    assert got[0, 3] == 1792 and got[0, 5] == 4 and abs(got[0, 130] + 2) < 1e-6


def test_weight_scales_are_the_blocks_largest():
    w = np.random.default_rng(2).normal(size=(130, 260)).astype(np.float32)
    q, s = fp8.weights(w)
    assert s.shape == (2, 3)
    assert s[1, 2] == np.abs(w[128:, 256:]).max() / np.float32(448)
    err = np.abs(fp8.weight_values(q, s) - w)
    step = np.repeat(np.repeat(s, 128, 0)[:130], 128, 1)[:, :260]
    assert (err <= np.maximum(np.abs(w) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 1e-6)).all()


def test_norm_gradient_by_differences():
    r = np.random.default_rng(3)
    h, dy, dt, g = r.normal(size=(3, 16)), r.normal(size=(3, 16)), r.normal(size=(3, 16)), r.normal(size=16)
    dh, dg = norm.rms_norm_backward(dy, h, g, 1e-3, dt)
    f = lambda h, g: (norm.rms_norm(h, g, 1e-3) * dy).sum() + (h * dt).sum()  # noqa: E731
    e = 1e-6
    for i in range(3):
        for j in range(16):
            d = np.zeros_like(h)
            d[i, j] = e
            assert abs((f(h + d, g) - f(h - d, g)) / (2 * e) - dh[i, j]) < 1e-7
    for j in range(16):
        d = np.zeros_like(g)
        d[j] = e
        assert abs((f(h, g + d) - f(h, g - d)) / (2 * e) - dg[j]) < 1e-7


def test_norm_by_hand():
    y = norm.rms_norm(np.array([[3.0, 4.0, 0.0, 0.0]]), np.array([1.0, 2.0, 1.0, 1.0]), 0.0)
    assert np.allclose(y, [[1.2, 3.2, 0, 0]])  # mean of the squares 6.25


# ---------------------------------------------------------------- refusals

def _norm_desc(**kw):
    from combine_top_router_amd._lib import NormDesc
    d = dict(rows=4, hidden=64, dtype=0, eps=1e-6, reserved=0, ldx=64, ldr=64, ldt=64, ldy=64)
    d.update(kw)
    return NormDesc(*(d[k] for k, _ in NormDesc._fields_))


@built
@pytest.mark.parametrize("bad, status", [
    (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(hidden=0), 1), (dict(reserved=1), 1),
    (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(dtype=3), 2), (dict(dtype=-1), 2), (dict(hidden=12), 2), (dict(hidden=16392), 2),
])
def test_bad_norm_descriptors_are_refused(bad, status):
    from combine_top_router_amd import _lib
    lib = _lib.load()
    d = _norm_desc(**bad)
    f = [C.c_void_p((i + 1) << 20) for i in range(8)]  # never dereferenced
    assert lib.moe_rms_norm(C.byref(d), *f[:7], None) == status
    assert lib.moe_rms_norm_backward_workspace_bytes(C.byref(d)) == 0
    assert lib.moe_rms_norm_backward(C.byref(d), *f[:7], 1 << 40, None) == status


@built
def test_norm_argument_checks_launch_nothing():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    at = [C.c_void_p((i + 1) << 20) for i in range(8)]
    odd = C.c_void_p((9 << 20) + 8)
    names = ("x", "res", "gain", "total", "y", "q", "scale")

    def fwd(d=None, **kw):
        a = dict(zip(names, at), **kw)
        return lib.moe_rms_norm(C.byref(d or _norm_desc()), *(a[n] for n in names), None)

    assert lib.moe_rms_norm(None, *at[:7], None) == 1
    for kw in (dict(x=None), dict(res=None), dict(q=None), dict(scale=None),
               dict(total=None, y=None, q=None, scale=None), *({n: odd} for n in names)):
        assert fwd(**kw) == 1, kw
    for ld in ("ldx", "ldr", "ldt", "ldy"):
        for v in (56, 68, (1 << 21) + 8):
            assert fwd(_norm_desc(**{ld: v})) == 1, (ld, v)
    for out, others in (("total", ("gain", "y")), ("y", ("gain",)),
                        ("q", ("x", "res", "gain", "total", "y")),
                        ("scale", ("x", "res", "gain", "total", "y", "q"))):
        for o in others:
            assert fwd(**{out: dict(zip(names, at))[o]}) == 1, (out, o)
    for out, ld in (("total", "ldt"), ("y", "ldy")):
        for o in ("x", "res"):  # in place, but rows apart
            assert fwd(_norm_desc(**{ld: 72}), **{out: dict(zip(names, at))[o]}) == 1, (out, o)
    assert fwd(_norm_desc(rows=0), x=None, y=None) == 0

    names2 = ("dy", "total", "gain", "dtotal", "dx", "dgain", "ws")

    def bwd(d=None, n=1 << 40, **kw):
        a = dict(zip(names2, at), **kw)
        return lib.moe_rms_norm_backward(C.byref(d or _norm_desc()), *(a[k] for k in names2), n, None)

    need = lib.moe_rms_norm_backward_workspace_bytes(C.byref(_norm_desc()))
    assert need > 0
    for kw in (dict(dy=None), dict(total=None), dict(ws=None), dict(n=need - 1),
               *({k: odd} for k in names2)):
        assert bwd(**kw) == 1, kw
    for out, others in (("dx", ("gain",)), ("dgain", ("dy", "total", "gain", "dtotal", "dx"))):
        for o in others:
            assert bwd(**{out: dict(zip(names2, at))[o]}) == 1, (out, o)
    for o in ("dy", "total", "dtotal"):
        assert bwd(_norm_desc(ldr=72), dx=dict(zip(names2, at))[o]) == 1, o
    assert bwd(dx=None, dgain=None) == 0
    assert bwd(_norm_desc(rows=0), dy=None, total=None, dgain=None) == 0


@built
def test_quantize_argument_checks_launch_nothing():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    x, q, s, odd = (C.c_void_p(v) for v in (1 << 20, 2 << 20, 3 << 20, (4 << 20) + 8))

    def rows(t=0, x=x, m=4, h=64, ld=64, q=q, s=s):
        return lib.moe_quantize_fp8(t, x, m, h, ld, q, s, None)

    for kw, status in ((dict(t=3), 2), (dict(h=12), 2), (dict(h=0), 1), (dict(h=1 << 21), 1),
                       (dict(m=-1), 1), (dict(m=1 << 31), 2), (dict(ld=56), 1), (dict(ld=68), 1),
                       (dict(x=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(x=odd), 1),
                       (dict(q=odd), 1), (dict(s=odd), 1), (dict(q=x), 1), (dict(s=x), 1),
                       (dict(s=q), 1)):
        assert rows(**kw) == status, kw
    assert rows(m=0, x=None, q=None, s=None) == 0

    def weights(t=0, w=x, n=2, k=64, c=64, order=0, q=q, s=s):
        return lib.moe_quantize_fp8_weights(t, w, n, k, c, order, q, s, None)

    for kw, status in ((dict(t=3), 2), (dict(k=24), 2), (dict(c=60, order=1), 2), (dict(order=2), 1),
                       (dict(n=-1), 1), (dict(n=65536), 1), (dict(k=0), 1), (dict(c=0), 1),
                       (dict(k=1 << 21), 1), (dict(w=None), 1), (dict(q=None), 1), (dict(s=None), 1),
                       (dict(w=odd), 1), (dict(q=odd), 1), (dict(s=odd), 1), (dict(q=x), 1),
                       (dict(s=x), 1), (dict(s=q), 1)):
        assert weights(**kw) == status, kw
    assert weights(n=0, w=None, q=None, s=None) == 0


def _linear_desc(**kw):
    from combine_top_router_amd._lib import LinearFp8Desc
    d = dict(rows=4, inner=128, cols=64, dtype=0, act=0, y_f32=0, reserved=0, ldy=64, ldr=64)
    d.update(kw)
    return LinearFp8Desc(*(d[k] for k, _ in LinearFp8Desc._fields_))


@built
@pytest.mark.parametrize("bad, status", [
    (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(inner=0), 1), (dict(inner=(1 << 20) + 16), 1),
    (dict(cols=0), 1), (dict(cols=(1 << 20) + 1), 1), (dict(act=4), 1), (dict(act=-1), 1),
    (dict(y_f32=2), 1), (dict(reserved=1), 1), (dict(ldy=63), 1), (dict(ldy=(1 << 21) + 1), 1),
    (dict(dtype=2), 2), (dict(inner=24), 2), (dict(rows=1 << 24, cols=1 << 20, ldy=1 << 20), 2),
    (dict(rows=(1 << 31) - 1, cols=128, ldy=128), 2),
])
def test_bad_linear_fp8_descriptors_are_refused(bad, status):
    from combine_top_router_amd import _lib
    lib = _lib.load()
    d = _linear_desc(**bad)
    f = [C.c_void_p((i + 1) << 20) for i in range(8)]  # never dereferenced
    assert lib.moe_linear_fp8_workspace_bytes(C.byref(d)) == 0
    assert lib.moe_linear_fp8(C.byref(d), *f, 1 << 40, None) == status


@built
def test_linear_fp8_argument_checks_launch_nothing():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    names = ("x", "xs", "w", "ws", "bias", "res", "y", "work")
    at = {n: C.c_void_p((i + 1) << 20) for i, n in enumerate(names)}
    odd = C.c_void_p((20 << 20) + 8)

    def call(d=None, n=1 << 40, **kw):
        a = dict(at, **kw)
        return lib.moe_linear_fp8(C.byref(d or _linear_desc()), *(a[k] for k in names), n, None)

    assert lib.moe_linear_fp8(None, *at.values(), 1 << 40, None) == 1
    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(x=odd),
               dict(w=odd), dict(y=at["res"], d=_linear_desc(ldr=72)),
               dict(y=at["res"], d=_linear_desc(y_f32=1)), dict(d=_linear_desc(ldr=63))):
        assert call(**kw) == 1, kw
    for n in ("x", "xs", "w", "ws", "bias"):
        assert call(y=at[n]) == 1, n
    assert call(d=_linear_desc(rows=0), x=None, w=None, y=None) == 0
    split = _linear_desc(rows=100, inner=8192, cols=128, ldy=128, ldr=128)
    need = lib.moe_linear_fp8_workspace_bytes(C.byref(split))
    assert need > 0
    assert call(d=split, work=None) == 1 and call(d=split, n=need - 1) == 1 and call(d=split, work=odd) == 1


def _grouped_desc(**kw):
    from combine_top_router_amd._lib import GroupedFp8Desc
    d = dict(m_cap=256, max_rows=256, num_tokens=64, num_groups=2, inner=128, cols=128, top_k=2, fast=0, reserved=0)
    d.update(kw)
    return GroupedFp8Desc(*(d[k] for k, _ in GroupedFp8Desc._fields_))


@built
def test_grouped_fp8_argument_checks_launch_nothing():
    from combine_top_router_amd import _lib
    lib = _lib.load()
    up = ("x", "xs", "src", "off", "cnt", "w1", "s1", "w3", "s3", "h", "hs")
    down = ("h", "hs", "off", "cnt", "w2", "s2", "y")
    odd = C.c_void_p((20 << 20) + 8)

    def call(fn, names, d=None, **kw):
        a = dict({n: C.c_void_p((i + 1) << 20) for i, n in enumerate(names)}, **kw)
        return fn(C.byref(d or _grouped_desc()), *(a[k] for k in names), None)

    for fn, names in ((lib.moe_grouped_gate_up_fp8, up), (lib.moe_grouped_down_fp8, down)):
        for bad, status in ((dict(m_cap=-1), 1), (dict(max_rows=-1), 1), (dict(num_groups=0), 1),
                            (dict(num_groups=1025), 1), (dict(inner=0), 1), (dict(cols=0), 1),
                            (dict(inner=(1 << 20) + 128), 1), (dict(cols=(1 << 20) + 128), 1),
                            (dict(fast=2), 1), (dict(reserved=1), 1),
                            (dict(inner=192), 2), (dict(cols=192), 2), (dict(m_cap=1 << 31), 2),
                            (dict(m_cap=(1 << 31) - 1, cols=1 << 20), 2)):
            assert call(fn, names, _grouped_desc(**bad)) == status, (fn, bad)
        assert fn(None, *[C.c_void_p(1 << 20)] * len(names), None) == 1
        for n in names:
            if n != "src":
                assert call(fn, names, **{n: None}) == 1, n
            if n not in ("src", "off", "cnt"):
                assert call(fn, names, **{n: odd}) == 1, n
        assert call(fn, names, _grouped_desc(m_cap=0)) == 0
        assert call(fn, names, _grouped_desc(max_rows=0)) == 0
    a = {n: C.c_void_p((i + 1) << 20) for i, n in enumerate(up)}
    for n in ("x", "xs", "w1", "s1", "w3", "s3"):
        assert call(lib.moe_grouped_gate_up_fp8, up, h=a[n]) == 1, n
        assert call(lib.moe_grouped_gate_up_fp8, up, hs=a[n]) == 1, n
    for bad, status in ((dict(top_k=0), 1), (dict(top_k=17), 1), (dict(num_tokens=-1), 1),
                        (dict(num_tokens=1 << 24), 2)):
        assert call(lib.moe_grouped_gate_up_fp8, up, _grouped_desc(**bad)) == status, bad
    assert call(lib.moe_grouped_gate_up_fp8, up, _grouped_desc(num_tokens=0)) == 0
    b = {n: C.c_void_p((i + 1) << 20) for i, n in enumerate(down)}
    for n in ("h", "hs", "w2", "s2"):
        assert call(lib.moe_grouped_down_fp8, down, y=b[n]) == 1, n
