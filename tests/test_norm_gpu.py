"""Root-mean-square norm, its gradients and quantisation on the GPU against the oracle.

u = 2^-24 (half a step of fp32). A row's sum of squares has no cancellation: a lane adds
up to 32 terms, then come 6 steps over the wavefront and up to 16 over wavefronts, 55
roundings with the squares'; the root halves them (28), and mean, eps, root, reciprocal,
two products add 6: 34 u at most, taken as 64 u = 2^-18 of the value."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import fp8, norm

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_top_router_amd")
ops = moe.ops

DEV = "cuda"
F32 = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# smallest step of a type, halved: what rounding costs near zero
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def rnd(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bytes_of(q):
    return q.view(torch.uint8).cpu().numpy()


def close(got, want, tol):
    got = np64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], np.broadcast_to(want, got.shape)[bad][:4])


def check_norm(x, gain, res, eps, y, q, s, total):
    dt = x.dtype
    h = x if res is None else (x.float() + res.float()).to(dt)
    if res is not None:
        assert torch.equal(total, h)
    else:
        assert total is None
    g = np.ones(x.shape[1]) if gain is None else np64(gain)
    want = norm.rms_norm(np64(h), g, eps)
    if y is not None:
        assert y.dtype == dt
        close(y, want, np.abs(want) * (HALF[dt] + F32 * (1 + HALF[dt])) + TINY[dt])
    if q is not None:
        n = -(-x.shape[1] // 128)
        amax = np.stack([np.abs(want[:, 128 * j:128 * j + 128]).max(axis=1) for j in range(n)], 1)
        ws = np.maximum(amax / 448, 2.0 ** -126)
        close(s, ws, ws * (F32 + 2.0 ** -23))
        step = np.repeat(np64(s), 128, axis=1)[:, :x.shape[1]]
        got = fp8.row_values(bytes_of(q), s.cpu().numpy())
        tol = np.maximum(np.abs(want) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -16) + np.abs(want) * 2 * F32
        assert (np.abs(got - want) <= tol).all()


SHAPES = [(1, 8), (3, 64), (5, 512), (7, 520), (4, 1000), (9, 1024), (2, 2048), (17, 2056),
          (3, 4104), (16, 7168), (5, 8200), (2, 16384), (700, 128), (1100, 2048), (1037, 4104),
          (900, 7168), (600, 16384)]


@pytest.mark.parametrize("rows, hidden", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_norm(rows, hidden, dtype):
    x, res = rnd((rows, hidden), dtype, 1), rnd((rows, hidden), dtype, 2, 2.0)
    gain = rnd((hidden,), torch.float32, 3, 0.3) + 1
    for r, g, wy, wq in ((res, gain, True, True), (None, gain, True, False), (res, None, False, True)):
        y, q, s, total = ops.rms_norm(x, g, residual=r, eps=1e-5, want_y=wy, want_fp8=wq)
        assert (y is not None) == wy and (q is not None) == wq
        check_norm(x, g, r, 1e-5, y, q, s, total)


def test_norm_fp8_is_that_of_the_unrounded_output():
    x, gain = rnd((37, 1416), torch.float32, 4), rnd((1416,), torch.float32, 5) + 1
    y, q, s, _ = ops.rms_norm(x, gain, want_fp8=True)
    wq, ws = fp8.rows(y.cpu().numpy())
    assert (s.cpu().numpy() == ws).all() and (bytes_of(q) == wq).all()
    q2, s2 = ops.quantize_fp8(y)
    assert torch.equal(s, s2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8))


@pytest.mark.parametrize("where", ["x", "residual", "both"])
@pytest.mark.parametrize("rows, hidden", [(3, 520), (300, 2056), (1200, 7168)])
def test_norm_in_place(where, rows, hidden):
    x, res, gain = rnd((rows, hidden), torch.bfloat16, 6), rnd((rows, hidden), torch.bfloat16, 7), None
    want = ops.rms_norm(x, gain, residual=res)
    a, b = x.clone(), res.clone()
    total, y = {"x": (a, None), "residual": (b, None), "both": (b, a)}[where]
    got = ops.rms_norm(a, gain, residual=b, total=total, y=y)
    assert torch.equal(got[3], want[3]) and torch.equal(got[0], want[0])


def test_norm_rows_apart_and_what_lies_between():
    H, M = 264, 50
    wide = rnd((M, 2 * H), torch.bfloat16, 8)
    x, res = wide[:, :H], wide[:, H:]
    out = torch.full((M + 1, 400), 7.0, dtype=torch.bfloat16, device=DEV)
    tot = torch.full((M + 1, 320), 7.0, dtype=torch.bfloat16, device=DEV)
    y, _, _, total = ops.rms_norm(x, None, residual=res, y=out[:M, 8:8 + H], total=tot[:M, :H])
    check_norm(x.contiguous(), None, res.contiguous(), 1e-6, y, None, None, total)
    assert (out[:, :8] == 7).all() and (out[:, 8 + H:] == 7).all() and (out[M] == 7).all()
    assert (tot[:, H:] == 7).all() and (tot[M] == 7).all()


def test_norm_of_nothing_and_of_odd_values():
    y, q, s, total = ops.rms_norm(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), want_fp8=True)
    assert y.shape == (0, 64) and q.shape == (0, 64) and s.shape == (0, 1) and total is None
    x = rnd((8, 384), torch.float32, 9)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4] = 2.0 ** -140
    x[5] = 1e30
    y, q, s, _ = ops.rms_norm(x, None, eps=0.0, want_fp8=True)
    assert torch.isnan(y[1]).all()  # 0 / 0: eps is the caller's
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 200]) and (y[3, :200] == 0).all()
    assert (y[5] == 0).all()  # squares past fp32
    d = fp8.decode(bytes_of(q))
    assert np.isnan(d[2]).all() and (s[2] == 2.0 ** -126).all()
    check_norm(x[6:], None, None, 0.0, y[6:], q[6:], s[6:], None)
    check_norm(x[:1], None, None, 0.0, y[:1], q[:1], s[:1], None)


@pytest.mark.parametrize("rows, hidden", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_norm_backward(rows, hidden, dtype):
    h, dy, dt = (rnd((rows, hidden), dtype, s) for s in (11, 12, 13))
    gain = rnd((hidden,), torch.float32, 14, 0.3) + 1
    for g, t in ((gain, dt), (None, None)):
        dx, dg = ops.rms_norm_backward(dy, h, g, eps=1e-5, dtotal=t)
        gg = np.ones(hidden) if g is None else np64(g)
        tt = 0.0 if t is None else np64(t)
        want, wdg = norm.rms_norm_backward(np64(dy), np64(h), gg, 1e-5, tt)
        hh = np64(h)
        xhat = hh * norm.rstd(hh, 1e-5)
        gdy = np.abs(np64(dy) * gg)
        size = norm.rstd(hh, 1e-5) * (gdy + np.abs(xhat) * (gdy * np.abs(xhat)).mean(axis=1, keepdims=True)) + np.abs(tt)
        # (34 u of rstd enters up to three times, and the second sum has its own 60 u)
        close(dx, want, np.abs(want) * HALF[dtype] + 4 * F32 * size + TINY[dtype])
        terms = np.abs(np64(dy) * xhat).sum(axis=0)
        close(dg, wdg, terms * F32 + np.abs(wdg) * 2.0 ** -24)


def test_norm_backward_parts_and_places():
    h, dy, dt = (rnd((130, 2056), torch.bfloat16, s) for s in (15, 16, 17))
    gain = rnd((2056,), torch.float32, 18)
    dx, dg = ops.rms_norm_backward(dy, h, gain, dtotal=dt)
    a, none = ops.rms_norm_backward(dy, h, gain, dtotal=dt, want_dgain=False)
    assert none is None and torch.equal(a, dx)
    none, b = ops.rms_norm_backward(dy, h, gain, dtotal=dt, want_dx=False)
    assert none is None and torch.equal(b, dg)
    for name in ("dy", "total", "dtotal"):
        t = dict(dy=dy.clone(), total=h.clone(), dtotal=dt.clone())
        got, b = ops.rms_norm_backward(t["dy"], t["total"], gain, dtotal=t["dtotal"], dx=t[name])
        assert torch.equal(got, dx) and torch.equal(b, dg), name
    e = torch.empty((0, 2056), dtype=torch.bfloat16, device=DEV)
    dx, dg = ops.rms_norm_backward(e, e, gain)
    assert dx.shape == (0, 2056) and (dg == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows, hidden", [(0, 64), (1, 8), (3, 128), (5, 1000), (33, 7168), (4100, 264)])
def test_quantize_rows(rows, hidden, dtype):
    x = rnd((rows, hidden), dtype, 20) * rnd((rows, 1), dtype, 21).abs().exp2()
    q, s = ops.quantize_fp8(x)
    wq, ws = fp8.rows(x.float().cpu().numpy())
    assert (s.cpu().numpy() == ws).all() and (bytes_of(q) == wq).all()


def test_quantize_odd_values():
    x = rnd((6, 264), torch.float32, 22)
    x[0] = 0
    x[1, 7], x[1, 8], x[1, 9] = float("nan"), float("inf"), float("-inf")
    x[2] *= 2.0 ** -130
    x[3] = torch.finfo(torch.float32).max
    x[4, 3] = 2.0 ** 100
    q, s = ops.quantize_fp8(x)
    wq, ws = fp8.rows(x.cpu().numpy())
    assert (s.cpu().numpy() == ws).all()
    d, w = fp8.decode(bytes_of(q)), fp8.decode(wq)
    assert (np.isnan(d) == np.isnan(w)).all() and (d[~np.isnan(w)] == w[~np.isnan(w)]).all()
    assert np.isnan(d[1, 7:10]).all() and np.isnan(d).sum() == 3


def test_quantize_rows_apart():
    x = rnd((40, 512), torch.float16, 23)[:, 128:392]
    q, s = ops.quantize_fp8(x)
    wq, ws = fp8.rows(x.float().cpu().numpy())
    assert (s.cpu().numpy() == ws).all() and (bytes_of(q) == wq).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n, N, K", [(1, 128, 128), (2, 136, 272), (1, 8, 16), (3, 256, 144), (1, 1000, 528)])
def test_quantize_weights(n, N, K, dtype):
    w = rnd((n, N, K), dtype, 24)
    want = [fp8.weights(m) for m in w.float().cpu().numpy()]
    for q, s in (ops.quantize_fp8_weights(w),
                 ops.quantize_fp8_weights(w.transpose(1, 2).contiguous(), transpose=True)):
        assert q.shape == (n, N, K) and s.shape == (n, -(-N // 128), -(-K // 128))
        for e in range(n):
            assert (s[e].cpu().numpy() == want[e][1]).all() and (bytes_of(q[e]) == want[e][0]).all()


def test_quantize_weights_of_odd_heights():
    w = rnd((37, 48), torch.bfloat16, 25)  # output-major: any number of outputs
    q, s = ops.quantize_fp8_weights(w)
    wq, ws = fp8.weights(w.float().cpu().numpy())
    assert q.shape == (37, 48) and (s.cpu().numpy() == ws).all() and (bytes_of(q) == wq).all()
    q, s = ops.quantize_fp8_weights(torch.empty((0, 32, 32), dtype=torch.bfloat16, device=DEV))
    assert q.shape == (0, 32, 32) and s.shape == (0, 1, 1)


def test_stream_and_graph():
    x, res = rnd((64, 7168), torch.bfloat16, 26), rnd((64, 7168), torch.bfloat16, 27)
    gain, dy = rnd((7168,), torch.float32, 28), rnd((64, 7168), torch.bfloat16, 29)

    def step():
        y, q, s, t = ops.rms_norm(x, gain, residual=res, want_fp8=True)
        return [y, q.view(torch.uint8), s, t, *ops.rms_norm_backward(dy, t, gain, dtotal=y),
                *(v.view(torch.uint8) for v in ops.quantize_fp8(t))]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for k in range(3):
        x.copy_(rnd((64, 7168), torch.bfloat16, 30 + k))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)), k


def test_refusals():
    x = rnd((4, 64), torch.bfloat16, 31)
    with pytest.raises(TypeError, match="bf16, fp16 or fp32"):
        ops.rms_norm(x.double())
    with pytest.raises(ValueError, match="needs a residual"):
        ops.rms_norm(x, total=torch.empty_like(x))
    with pytest.raises(TypeError, match="gain"):
        ops.rms_norm(x, x[0])
    with pytest.raises(ValueError, match="residual"):
        ops.rms_norm(x, residual=x[:3])
    with pytest.raises(moe.MoEError, match="MOE_ERR_UNSUPPORTED"):
        ops.rms_norm(x[:, :60].contiguous())
    with pytest.raises(moe.MoEError, match="MOE_ERR_ARG"):
        ops.rms_norm(x, want_y=False)
    with pytest.raises(moe.MoEError, match="MOE_ERR_ARG"):
        ops.rms_norm(x[:, 4:60])  # rows that start 8 bytes off
    with pytest.raises(ValueError, match="workspace"):
        ops.rms_norm_backward(x, x, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError, match="bf16, fp16 or fp32"):
        ops.quantize_fp8(x.to(torch.float8_e4m3fn))
    with pytest.raises(moe.MoEError, match="MOE_ERR_UNSUPPORTED"):
        ops.quantize_fp8_weights(x[:, :40].contiguous())
    with pytest.raises(ValueError, match="must be contiguous"):
        ops.quantize_fp8_weights(x.t())


def test_rows_past_32_bits():
    rows, hidden, few = 300000, 16384, 5  # 4.9e9 elements
    x = torch.zeros((rows, hidden), dtype=torch.bfloat16, device=DEV)
    x[-few:] = rnd((few, hidden), torch.bfloat16, 40)
    gain = rnd((hidden,), torch.float32, 41)
    y, q, s, _ = ops.rms_norm(x, gain, want_fp8=True)
    wy, wq, ws, _ = ops.rms_norm(x[-few:], gain, want_fp8=True)
    # (rows this wide take the same kernel whatever their number)
    assert torch.equal(y[-few:], wy) and torch.equal(q[-few:].view(torch.uint8), wq.view(torch.uint8))
    assert torch.equal(s[-few:], ws)
    del y, q, s
    q, s = ops.quantize_fp8(x)
    wq, ws = fp8.rows(x[-few:].float().cpu().numpy())
    assert (bytes_of(q[-few:]) == wq).all() and (s[-few:].cpu().numpy() == ws).all()
    del q, s
    dy = torch.zeros_like(x)
    dy[-few:] = rnd((few, hidden), torch.bfloat16, 42)
    dx, dg = ops.rms_norm_backward(dy, x, gain)
    wdx, wdg = ops.rms_norm_backward(dy[-few:], x[-few:], gain)
    assert torch.equal(dx[-few:], wdx)
    # the same terms dy xhat, added in the same order or another by at most `few` roundings each way
    h = np64(x[-few:])
    terms = np.abs(np64(dy[-few:]) * h * norm.rstd(h, 1e-6)).sum(axis=0)
    close(dg, np64(wdg), 2 * few * 2.0 ** -24 * terms)


def test_weights_past_32_bits():
    n, N, K = 1100, 2048, 2048  # 4.6e9 elements
    w = torch.zeros((n, N, K), dtype=torch.bfloat16, device=DEV)
    w[-1] = rnd((N, K), torch.bfloat16, 43)
    for turn in (False, True):
        q, s = ops.quantize_fp8_weights(w, transpose=turn)
        v = w[-1].t() if turn else w[-1]
        wq, ws = fp8.weights(v.float().cpu().numpy())
        assert (bytes_of(q[-1]) == wq).all() and (s[-1].cpu().numpy() == ws).all()
        del q, s
