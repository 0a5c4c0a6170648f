"""GPU parity of the dense linear layer and its gradients against the float64
oracle. Bounds: u is half a step of the 16-bit type; the products are exact in
fp32, a sum of K of them is off by at most K steps of 2^-23 of the sum of their
magnitudes; activations change an error by at most 1.13 (gelu's steepest slope)
and are evaluated in fp32 within 2^-20 of |z| (slopes: of 1)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import linear as olinear

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_top_router_amd")
ops = moe.ops

BF, FP = torch.bfloat16, torch.float16
HALF_STEP = {BF: 2.0 ** -8, FP: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {BF: 2.0 ** -133, FP: 2.0 ** -24, torch.float32: 2.0 ** -149}

# rows, inner, cols: single rows, odd and ragged sizes, every tile shape, split and not
SHAPES = [
    (1, 8, 1), (1, 64, 8), (3, 72, 5), (17, 7168, 256), (33, 136, 130), (64, 4096, 1000),
    (129, 264, 257), (300, 520, 520), (1000, 1024, 60), (513, 2056, 776), (2048, 512, 2048),
    (700, 64, 16), (5, 16, 4096), (4100, 200, 8), (256, 2048, 40), (1023, 4104, 300),
]
ACTS = ["none", "relu", "silu", "gelu"]


def f64(t):
    return t.detach().cpu().double().numpy()


def _close(got, want, tol, what):
    g = f64(got)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], g[bad][:4], want[bad][:4])


def _matrix(gen, rows, cols, dtype, pad=0, std=1.0):
    """Random [rows, cols]; with pad, a view of wider rows whose rest is NaN."""
    v = (torch.randn((rows, cols), generator=gen, device="cuda") * std).to(dtype)
    if not pad:
        return v
    wide = torch.full((rows + 1, cols + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:rows, :cols] = v
    return wide[:rows, :cols]


def _forward(gen, M, K, N, dtype, order, act, bias, res, keep, f32, pad=0, **kw):
    x = _matrix(gen, M, K, dtype, pad)
    w = _matrix(gen, N, K, dtype, pad, K ** -0.5) if order == "nk" else \
        _matrix(gen, K, N, dtype, pad, K ** -0.5).t()
    b = torch.randn((N,), generator=gen, device="cuda") if bias else None
    r = _matrix(gen, M, N, dtype, pad and pad + 1) if res else None
    pre = torch.empty((M, N), dtype=dtype, device="cuda") if keep else None
    y = ops.linear(x, w, b, act, r, torch.float32 if f32 else None, pre=pre, **kw)
    torch.cuda.synchronize()
    xs, ws = f64(x), f64(w)
    want, z = olinear.linear(xs, ws, None if b is None else f64(b), act, None if r is None else f64(r))
    mag = np.abs(xs) @ np.abs(ws).T
    ez = (K + 160) * 2.0 ** -23 * mag + 2.0 ** -23 * np.abs(z)  # up to 128 parts, and the bias
    t = torch.float32 if f32 else dtype
    ey = 1.13 * ez + 2.0 ** -20 * np.abs(z) + (2.0 ** -23 * (np.abs(want) + np.abs(z)))
    _close(y, want, ey + HALF_STEP[t] * (np.abs(want) + ey) + TINY[t], "y")
    if keep:
        _close(pre, z, ez + HALF_STEP[dtype] * (np.abs(z) + ez) + TINY[dtype], "pre")
    return x, w, b, r, y


def _backward(gen, M, K, N, dtype, order, act, f32, pad=0, bias=True, **kw):
    x = _matrix(gen, M, K, dtype, pad)
    w = _matrix(gen, N, K, dtype, pad, K ** -0.5) if order == "nk" else \
        _matrix(gen, K, N, dtype, pad, K ** -0.5).t()
    pre = _matrix(gen, M, N, dtype, pad and pad + 3) if act != "none" else None
    dy = _matrix(gen, M, N, torch.float32 if f32 else dtype, pad)
    dx, dw, db = ops.linear_backward(dy, x, w, act, pre, want_dbias=bias, **kw)
    torch.cuda.synchronize()
    assert dw.stride() == ((K, 1) if order == "nk" else (1, N)) or 1 in (K, N)
    xs, ws, dys = f64(x), f64(w), f64(dy)
    wx, ww, wb, dz = olinear.linear_backward(dys, xs, ws, act, None if pre is None else f64(pre))
    u = HALF_STEP[dtype]
    # dz as the matrix cores read it
    slope = 0.0 if act == "none" else 2.0 ** -20 * np.abs(dys)
    edz = slope + u * (np.abs(dz) + slope) + TINY[dtype]
    for got, want, other, n, what in ((dx, wx, np.abs(ws), N, "dx"),
                                      (dw.t(), ww.T, np.abs(xs), M, "dw")):
        if what == "dx":
            mag, e = (np.abs(dz) + edz) @ other, edz @ other
        else:
            mag, e = other.T @ (np.abs(dz) + edz), other.T @ edz
        e = e + (n + 160) * 2.0 ** -23 * mag
        _close(got, want, e + u * (np.abs(want) + e) + TINY[dtype], what)
    if bias:
        eb = (slope + (M / 8 + 16) * 2.0 ** -24 * np.abs(dz)).sum(axis=0)
        _close(db, wb, eb + 2.0 ** -24 * np.abs(wb) + 2.0 ** -149, "dbias")
    else:
        assert db is None
    return dx, dw, db


def _orders(N):
    return ["nk", "kn"] if N % 8 == 0 else ["nk"]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_forward(shape, dtype):
    M, K, N = shape
    gen = torch.Generator("cuda").manual_seed(M + K + N)
    for i, order in enumerate(_orders(N)):
        for j, act in enumerate(ACTS):
            print("CASE linear", shape, dtype, order, act, flush=True)
            f32 = (i + j) % 2 == 1
            _forward(gen, M, K, N, dtype, order, act, bias=j % 2 == 0, res=j >= 2,
                     keep=(i + j) % 3 == 0, f32=f32)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_backward(shape, dtype):
    M, K, N = shape
    gen = torch.Generator("cuda").manual_seed(M * 3 + K + N)
    for i, order in enumerate(_orders(N)):
        for j, act in enumerate(ACTS):
            print("CASE linear backward", shape, dtype, order, act, flush=True)
            _backward(gen, M, K, N, dtype, order, act, f32=(i + j) % 2 == 1, bias=j < 3)


@pytest.mark.parametrize("shape", [(4361, 2056, 4360), (6149, 2056, 6148), (1030, 2056, 4104),
                                   (1000, 4104, 2056), (2100, 4360, 4104)],
                         ids=lambda s: "x".join(map(str, s)))
def test_large_tiles_against_float64_on_the_device(shape):
    """The largest tiles, halved ones among them: the float64 products on the GPU."""
    M, K, N = shape
    gen = torch.Generator("cuda").manual_seed(K)
    for order in _orders(N):
        for dtype in (BF, FP):
            print("CASE large", shape, order, dtype, flush=True)
            u = HALF_STEP[dtype]
            x = _matrix(gen, M, K, dtype)
            w = _matrix(gen, N, K, dtype, 0, K ** -0.5) if order == "nk" else \
                _matrix(gen, K, N, dtype, 0, K ** -0.5).t()
            r, dy = _matrix(gen, M, N, dtype), _matrix(gen, M, N, dtype)
            b = torch.randn((N,), generator=gen, device="cuda")
            X, W, D = x.double(), w.double(), dy.double()
            XA, WA, DA = X.abs(), W.abs(), D.abs()

            def near(got, want, e, half):
                err = (got.double() - want).abs()
                assert bool((err <= e + half * (want.abs() + e) + TINY[got.dtype]).all())

            y = ops.linear(x, w, b, "none", r)
            z = X @ W.t() + b.double()
            e = (K + 160) * 2.0 ** -23 * (XA @ WA.t()) + 2.0 ** -22 * (z.abs() + r.double().abs())
            near(y, z + r.double(), e, u)
            y = ops.linear(x, w, out_dtype=torch.float32)
            near(y, X @ W.t(), (K + 160) * 2.0 ** -23 * (XA @ WA.t()), 2.0 ** -24)
            # dy is read as it is where its rows allow, or copied exactly
            dx, dw, db = ops.linear_backward(dy, x, w, want_dbias=True)
            near(dx, D @ W, (N + 160) * 2.0 ** -23 * (DA @ WA), u)
            near(dw, D.t() @ X, (M + 160) * 2.0 ** -23 * (DA.t() @ XA), u)
            near(db, D.sum(dim=0), (M / 8 + 16) * 2.0 ** -24 * DA.sum(dim=0), 2.0 ** -24)


@pytest.mark.parametrize("pad", [8, 24])
@pytest.mark.parametrize("shape", [(37, 72, 40), (300, 200, 264), (40, 4096, 128), (600, 64, 16)],
                         ids=lambda s: "x".join(map(str, s)))
def test_rows_lying_apart_with_nan_between(shape, pad):
    M, K, N = shape
    gen = torch.Generator("cuda").manual_seed(pad)
    for order in ("nk", "kn"):
        print("CASE strides", shape, pad, order, flush=True)
        _forward(gen, M, K, N, BF, order, "silu", True, True, True, False, pad)
        _backward(gen, M, K, N, BF, order, "gelu", False, pad)
        _backward(gen, M, K, N, FP, order, "none", False, pad)


def test_output_views_leave_their_surroundings_alone():
    gen = torch.Generator("cuda").manual_seed(9)
    x, w = _matrix(gen, 45, 64, BF), _matrix(gen, 33, 64, BF)
    plain = ops.linear(x, w)
    for cols in (40, 41):  # aligned rows and odd ones
        wide = torch.full((47, cols), 7.0, dtype=BF, device="cuda")
        pre = torch.full((47, cols), 7.0, dtype=BF, device="cuda")
        ops.linear(x, w, out=wide[1:46, :33], pre=pre[1:46, :33])
        torch.cuda.synchronize()
        for t in (wide, pre):
            assert torch.equal(t[1:46, :33], plain)
            t[1:46, :33] = 7.0
            assert (t == 7.0).all()


def test_residual_may_be_the_output():
    gen = torch.Generator("cuda").manual_seed(10)
    for M, K, N in ((70, 256, 96), (8, 8192, 64)):  # whole and split
        x, w, r = _matrix(gen, M, K, BF), _matrix(gen, N, K, BF, 0, K ** -0.5), _matrix(gen, M, N, BF)
        want = ops.linear(x, w, residual=r)
        ops.linear(x, w, residual=r, out=r)
        torch.cuda.synchronize()
        assert torch.equal(r, want)


def test_a_bad_row_or_column_stays_by_itself():
    gen = torch.Generator("cuda").manual_seed(11)
    for M, K, N in ((50, 72, 40), (300, 264, 300), (20, 4096, 64)):
        x, w = _matrix(gen, M, K, BF), _matrix(gen, N, K, BF, 0, K ** -0.5)
        want = ops.linear(x, w)
        x2, w2 = x.clone(), w.clone()
        x2[3], x2[-1, 0] = float("nan"), float("inf")
        w2[5] = float("nan")
        got = ops.linear(x2, w2)
        torch.cuda.synchronize()
        assert got[3].isnan().all() and got[:, 5].isnan().all()
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[3], keep[-1], keep[:, 5] = False, False, False
        assert torch.equal(got[keep], want[keep])
        dy = _matrix(gen, M, N, BF)
        dx, dw, _ = ops.linear_backward(dy, x, w)
        dy[3] = float("nan")
        dx2, _, _ = ops.linear_backward(dy, x, w, want_dw=False)
        torch.cuda.synchronize()
        assert dx2[3].isnan().all()
        dx2[3] = dx[3]
        assert torch.equal(dx2, dx)


def test_same_result_twice_and_from_a_dirty_workspace():
    gen = torch.Generator("cuda").manual_seed(12)
    x, w, dy = _matrix(gen, 24, 6144, BF), _matrix(gen, 200, 6144, BF), _matrix(gen, 24, 200, BF)
    y = ops.linear(x, w)
    ws = torch.full((ops.linear_workspace_bytes(x, w),), 255, dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0 and torch.equal(ops.linear(x, w, workspace=ws), y)
    a = ops.linear_backward(dy, x, w, want_dbias=True)
    ws = torch.full((ops.linear_backward_workspace_bytes(x, w),), 255, dtype=torch.uint8,
                    device="cuda")
    b = ops.linear_backward(dy, x, w, want_dbias=True, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rows_past_32_bit_offsets():
    M, K, N = 300_000, 8192, 24  # 4.9 GB of rows
    gen = torch.Generator("cuda").manual_seed(13)
    w = _matrix(gen, N, K, BF, 0, K ** -0.5)
    x = torch.zeros((M, K), dtype=BF, device="cuda")
    rows = [0, 1, 131071, 131072, 262143, 262144, 299_999]
    for r in rows:
        x[r] = torch.randn((K,), generator=gen, device="cuda").to(BF)
    y = ops.linear(x, w, out_dtype=torch.float32)
    torch.cuda.synchronize()
    want, _ = olinear.linear(f64(x[rows]), f64(w))
    mag = np.abs(f64(x[rows])) @ np.abs(f64(w)).T
    _close(y[rows], want, (K + 160) * 2.0 ** -23 * mag, "y")
    y[rows] = 0
    assert not y.any()
    dy = torch.zeros((M, N), dtype=BF, device="cuda")
    dy[rows] = torch.randn((len(rows), N), generator=gen, device="cuda").to(BF)
    dx, dw, _ = ops.linear_backward(dy, x, w)
    torch.cuda.synchronize()
    wx, ww, _, dz = olinear.linear_backward(f64(dy[rows]), f64(x[rows]), f64(w))
    ex = (N + 160) * 2.0 ** -23 * (np.abs(dz) @ np.abs(f64(w)))
    _close(dx[rows], wx, ex + 2.0 ** -8 * (np.abs(wx) + ex), "dx")
    ew = 200 * 2.0 ** -23 * (np.abs(dz).T @ np.abs(f64(x[rows])))
    _close(dw, ww, ew + 2.0 ** -8 * (np.abs(ww) + ew), "dw")
    dx[rows] = 0
    assert not dx.any()


def test_no_rows():
    x, w = torch.empty((0, 64), dtype=BF, device="cuda"), torch.ones((24, 64), dtype=BF, device="cuda")
    assert ops.linear(x, w).shape == (0, 24)
    for ww in (w, torch.ones((64, 24), dtype=BF, device="cuda").t()):
        dx, dw, db = ops.linear_backward(torch.empty((0, 24), dtype=BF, device="cuda"), x, ww,
                                         want_dbias=True)
        torch.cuda.synchronize()
        assert dx.shape == (0, 64) and dw.shape == (24, 64) and not dw.any() and not db.any()


def test_refusals():
    x, w = torch.zeros((4, 64), dtype=BF, device="cuda"), torch.zeros((8, 64), dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        ops.linear(x.float(), w)
    with pytest.raises(TypeError):
        ops.linear(x, w.half())
    with pytest.raises(TypeError):
        ops.linear(x, w, out_dtype=FP)
    with pytest.raises(ValueError):
        ops.linear(x, w, act="tanh")
    with pytest.raises(ValueError):
        ops.linear(x, w[:, :32])
    with pytest.raises(ValueError):
        ops.linear(x[:, ::2], w[:, ::2])
    with pytest.raises(ValueError):
        ops.linear(x, w, residual=torch.zeros((4, 9), dtype=BF, device="cuda"))
    with pytest.raises(TypeError):
        ops.linear(x, w, bias=torch.zeros((8,), dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        ops.linear(x[:1].expand(4, 64), w)
    with pytest.raises(ValueError):
        ops.linear(x.cpu(), w)
    with pytest.raises(moe.MoEError):
        ops.linear(x[:, :60].contiguous(), w[:, :60].contiguous())  # inner % 8
    with pytest.raises(ValueError):
        ops.linear_backward(torch.zeros((4, 8), dtype=BF, device="cuda"), x, w, act="silu")
    with pytest.raises(TypeError):
        ops.linear(x, w, workspace=torch.zeros((64,), device="cuda"))
    long = torch.zeros((4, 8192), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        ops.linear(long, long, workspace=torch.zeros((16,), dtype=torch.uint8, device="cuda"))


def test_two_graphs_replay_between_eager_calls():
    gen = torch.Generator("cuda").manual_seed(14)
    sets = []
    for M, K, N in ((16, 4096, 64), (300, 256, 512)):
        x, w, dy = _matrix(gen, M, K, BF), _matrix(gen, N, K, BF, 0, K ** -0.5), _matrix(gen, M, N, BF)
        pre = torch.empty((M, N), dtype=BF, device="cuda")

        def step(x=x, w=w, dy=dy, pre=pre):
            y = ops.linear(x, w, act="silu", pre=pre)
            return (y,) + ops.linear_backward(dy, x, w, "silu", pre, want_dbias=True)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        sets.append((graph, out, step, x))
    for rep in range(3):
        for graph, out, step, x in sets:
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
            want = [t.clone() for t in step()]
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("f32", [False, True])
def test_slopes_of_pre_activations_past_fp16(act, f32):
    """z outside fp16's range is stored as +-inf: its slope is 1 or 0, not NaN, and
    that of a NaN stays one (relu: z > 0 is false)."""
    inf, M, N, K = float("inf"), 9, 24, 16
    gen = torch.Generator("cuda").manual_seed(8)
    dy = torch.randn((M, N), generator=gen, device="cuda").to(torch.float32 if f32 else FP)
    x, w = _matrix(gen, M, K, FP), _matrix(gen, N, K, FP)
    z = torch.tensor([-inf, inf, -65504.0, 65504.0, -12.0, 12.0, -0.0, 1.0],
                     device="cuda").repeat(M, 3).to(FP)
    dx, dw, db = ops.linear_backward(dy, x, w, act, z, want_dbias=True)
    # and what the same finite slopes give
    z2 = z.clamp(-30000, 30000)
    dx2, dw2, db2 = ops.linear_backward(dy, x, w, act, z2, want_dbias=True)
    torch.cuda.synchronize()
    assert torch.isfinite(db).all()
    for a, b in ((dx, dx2), (dw, dw2), (db, db2)):
        assert torch.equal(a, b)
    assert not db[0::8].any() and torch.equal(db[1::8], ops.linear_backward(
        dy, x, w, want_dx=False, want_dw=False, want_dbias=True)[2][1::8])
    z[3, 5] = float("nan")
    db = ops.linear_backward(dy, x, w, act, z, False, False, True)[2]
    torch.cuda.synchronize()
    assert torch.isnan(db).nonzero().flatten().tolist() == ([] if act == "relu" else [5])


def test_sizes_past_32_bits_are_refused():
    x = torch.empty((1, 2 ** 32 + 8), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        ops.linear(x, x)


def _pairs(gen, rows, cols, along):
    """Random rows or columns, each twice in a row."""
    v = torch.randn((rows // 2, cols) if along == 0 else (rows, cols // 2), generator=gen, device="cuda")
    return v.repeat_interleave(2, dim=along)


def _cancelling(gen, M, K, N, dtype, act, f32):
    """dy, x, w, pre of which neighbouring rows' and columns' terms cancel but for 2^-6
    of them: what a 16-bit dz loses of the terms then shows in dx and in dw."""
    sign = 1.0 - 2.0 * ((torch.arange(M, device="cuda")[:, None] + torch.arange(N, device="cuda")) % 2)
    base = torch.randn((M // 2, N // 2), generator=gen, device="cuda")
    base = base.repeat_interleave(2, dim=0).repeat_interleave(2, dim=1)
    dy = sign * base + 2.0 ** -6 * torch.randn((M, N), generator=gen, device="cuda")
    x, w = _pairs(gen, M, K, 0).to(dtype), (_pairs(gen, N, K, 0) * K ** -0.5).to(dtype)
    pre = None
    if act != "none":
        pre = torch.randn((M // 2, N // 2), generator=gen, device="cuda").repeat_interleave(2, dim=0)
        pre = pre.repeat_interleave(2, dim=1).to(dtype)
    return dy.to(torch.float32 if f32 else dtype), x, w, pre


@pytest.mark.parametrize("shape", [(2, 8, 6), (64, 72, 64), (130, 136, 134), (1024, 64, 32),
                                   (16, 7168, 256), (1030, 520, 776), (2050, 2056, 1032)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_gradients_lose_no_more_of_dz_than_its_two_parts(shape, dtype):
    """dx and dw have their own rounding, and dz's are those of its second part: half a
    step of half a step, u^2 of it (and fp16's smallest steps)."""
    M, K, N = shape
    gen = torch.Generator("cuda").manual_seed(M + N)
    u = HALF_STEP[dtype]
    for order in _orders(N):
        for act, f32 in (("none", True), ("silu", False), ("gelu", True), ("relu", True)):
            print("CASE dz", shape, dtype, order, act, f32, flush=True)
            dy, x, w, pre = _cancelling(gen, M, K, N, dtype, act, f32)
            wm = w if order == "nk" else w.t().contiguous().t()
            dx, dw, _ = ops.linear_backward(dy, x, wm, act, pre)
            torch.cuda.synchronize()
            dys, xs, ws = f64(dy), f64(x), f64(w)
            wx, ww, _, dz = olinear.linear_backward(dys, xs, ws, act, None if pre is None else f64(pre))
            slope = 0.0 if act in ("none", "relu") else 2.0 ** -20 * np.abs(dys)
            edz = slope + u * u * np.abs(dz) + TINY[dtype]
            # twice the terms: sums of 2 n products, of magnitude dz and u dz
            for got, want, mag, e, n in ((dx, wx, np.abs(dz) @ np.abs(ws), edz @ np.abs(ws), N),
                                         (dw, ww, np.abs(dz).T @ np.abs(xs), edz.T @ np.abs(xs), M)):
                e = e + (2 * n + 160) * 2.0 ** -23 * (1 + u) * mag
                _close(got, want, e + u * (np.abs(want) + e) + TINY[dtype], "dx" if n == N else "dw")


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_dz_in_one_part_is_dz_rounded(dtype):
    gen = torch.Generator("cuda").manual_seed(21)
    for M, K, N in ((40, 72, 24), (300, 264, 257), (600, 512, 1024)):
        x, w = _matrix(gen, M, K, dtype), _matrix(gen, N, K, dtype, 0, K ** -0.5)
        dy = _matrix(gen, M, N, torch.float32)
        # (rounded before the call, dz is a 16-bit dy)
        want = ops.linear_backward(dy.to(dtype), x, w)
        got = ops.linear_backward(dy, x, w, dz16=True)
        two = ops.linear_backward(dy, x, w)
        torch.cuda.synchronize()
        for a, b, c in zip(got[:2], want[:2], two[:2]):
            assert torch.equal(a, b) and not torch.equal(a, c)
        _backward(gen, M, K, N, dtype, "nk", "silu", True, dz16=True)


def test_dz_past_fp16_is_an_infinity_in_its_row_and_column():
    M, K, N = 20, 64, 16
    gen = torch.Generator("cuda").manual_seed(22)
    x, w = _matrix(gen, M, K, FP).abs() + 1, _matrix(gen, N, K, FP).abs() + 1
    dy = _matrix(gen, M, N, torch.float32)
    dx, dw, _ = ops.linear_backward(dy, x, w)
    dy[3, 5] = 1e5
    for dz16 in (False, True):
        dx2, dw2, db = ops.linear_backward(dy, x, w, want_dbias=True, dz16=dz16)
        torch.cuda.synchronize()
        assert (dx2[3] == float("inf")).all() and (dw2[5] == float("inf")).all()
        assert torch.isfinite(db).all()
        if not dz16:
            dx2[3], dw2[5] = dx[3], dw[5]
            assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_activations_to_their_relative_error(act, dtype):
    """z known exactly (one product with 1): y within 2^-21 (1 + z^2 / 2) of itself for gelu,
    2^-21 (2 + |z|) for silu, also where it is small; slopes of the size of their two terms."""
    z = torch.cat([torch.linspace(-12.5, 12.5, 3001), torch.tensor([-0.0, 2.0 ** -14, -2.0 ** -14])])
    z = z.to(dtype).cuda()
    x = torch.zeros((z.numel(), 8), dtype=dtype, device="cuda")
    x[:, 3] = z
    w = torch.zeros((8, 8), dtype=dtype, device="cuda")
    w[:, 3] = 1.0
    zs = f64(z)[:, None]
    want = np.repeat(olinear.act(zs, act), 8, axis=1)
    rel = 2.0 ** -21 * (1 + zs * zs / 2 if act == "gelu" else 2 + np.abs(zs))
    for t in (torch.float32, dtype):
        y = ops.linear(x, w, act=act, out_dtype=t)
        torch.cuda.synchronize()
        _close(y, want, np.abs(want) * (rel + HALF_STEP[t]) * (1 + 2.0 ** -10) + TINY[t], str(t))
    # one row: dbias is dz itself, fp32
    n = z.numel() // 8 * 8
    dy, pre = torch.ones((1, n), device="cuda"), z[:n].view(1, n)
    _, _, db = ops.linear_backward(dy, x[:1], x[:n], act, pre, False, False, True)
    torch.cuda.synchronize()
    zs = f64(pre)[0]
    slope = olinear.act_slope(zs, act)
    if act == "gelu":
        two = olinear._phi(zs) + np.abs(zs) * np.exp(-zs * zs / 2) / np.sqrt(2 * np.pi)
        rel = 2.0 ** -21 * (1 + zs * zs / 2)
    else:
        s = 1 / (1 + np.exp(-zs))
        two, rel = s * (1 + np.abs(zs)), 2.0 ** -21 * (2 + np.abs(zs))
    _close(db, slope, two * (rel + 2.0 ** -22), "slope")


def test_a_product_of_2_to_the_34_outputs():
    M, K, N = 1 << 20, 64, 1 << 14  # 34 GB of outputs
    gen = torch.Generator("cuda").manual_seed(23)
    x, w = _matrix(gen, M, K, BF), _matrix(gen, N, K, BF, 0, K ** -0.5)
    y = ops.linear(x, w)
    rows = [0, 1, 255, 256, 131071, 131072, 524287, 524288, M - 257, M - 1]
    torch.cuda.synchronize()
    want, _ = olinear.linear(f64(x[rows]), f64(w))
    e = (K + 160) * 2.0 ** -23 * (np.abs(f64(x[rows])) @ np.abs(f64(w)).T)
    _close(y[rows], want, e + 2.0 ** -8 * (np.abs(want) + e), "y")
    # and as a gradient: dx of the same rows, dw from a few rows alone
    keep = y[rows].clone()
    y.zero_()
    y[rows] = keep
    dx, dw, _ = ops.linear_backward(y, x, w)
    torch.cuda.synchronize()
    wx, ww, _, dz = olinear.linear_backward(f64(keep), f64(x[rows]), f64(w))
    e = (N + 160) * 2.0 ** -23 * (np.abs(dz) @ np.abs(f64(w)))
    _close(dx[rows], wx, e + 2.0 ** -8 * (np.abs(wx) + e), "dx")
    e = 200 * 2.0 ** -23 * (np.abs(dz).T @ np.abs(f64(x[rows])))
    _close(dw, ww, e + 2.0 ** -8 * (np.abs(ww) + e), "dw")
    dx[rows] = 0
    assert not dx.any()


def _whole(gen, rows, cols, dtype, top):
    """Random whole numbers of at most `top`."""
    return torch.randint(-top, top + 1, (rows, cols), generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("shape", SHAPES + [(4361, 2056, 4360), (1030, 7176, 4104), (2048, 8192, 512)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_whole_numbers_exactly(shape, dtype):
    """Whole numbers whose sums fp32 holds (8192 terms of 3 * 3, of 900 * 2 with an fp32 dy's
    4361: below 2^24): every term counts once, however it is split, and the one rounding is to even."""
    M, K, N = shape
    gen = torch.Generator("cuda").manual_seed(K)
    for order in _orders(N):
        print("CASE whole", shape, dtype, order, flush=True)
        x, w = _whole(gen, M, K, dtype, 3), _whole(gen, N, K, dtype, 3)
        wm = w if order == "nk" else w.t().contiguous().t()
        b = _whole(gen, 1, N, torch.float32, 9)[0].contiguous()
        r = _whole(gen, M, N, dtype, 9)
        z = x.double() @ w.double().t() + b.double()
        y, pre = z.relu() + r.double(), torch.empty((M, N), dtype=dtype, device="cuda")
        assert torch.equal(ops.linear(x, wm, out_dtype=torch.float32), (z - b.double()).float())
        assert torch.equal(ops.linear(x, wm, b, "relu", r, pre=pre), y.to(dtype))
        assert torch.equal(pre, z.to(dtype))
        assert torch.equal(ops.linear(x, wm, b, "relu", r, torch.float32), y.float())
        # a 16-bit dy, and an fp32 one of more bits than one 16-bit part holds (900 * 2 of at
        # most 4361 terms; dx and dw past fp16's range are infinite on both sides)
        small = _whole(gen, M, N, dtype, 3)
        big = _whole(gen, M, N, torch.float32, 900)
        x, w = x.clamp(-2, 2), wm.clamp(-2, 2)
        for dy in (small, big):
            D = dy.double()
            dx, dw, db = ops.linear_backward(dy, x, w, want_dbias=True)
            torch.cuda.synchronize()
            assert torch.equal(dx, (D @ w.double()).to(dtype))
            assert torch.equal(dw, (D.t().contiguous() @ x.double()).to(dtype))
            assert torch.equal(db, D.sum(dim=0).float())


def test_activations_of_very_negative_values():
    """As above while the value is above 2^-118, and within 2^-118 below, down to -inf's side."""
    z = torch.cat([torch.linspace(-86.0, -12.5, 500), torch.linspace(-3e4, -86.0, 500)]).to(BF).cuda()
    x = torch.zeros((z.numel(), 8), dtype=BF, device="cuda")
    x[:, 0] = z
    w = torch.zeros((1, 8), dtype=BF, device="cuda")
    w[:, 0] = 1.0
    zs = f64(z)[:, None]
    for act in ("silu", "gelu"):
        y = ops.linear(x, w, act=act, out_dtype=torch.float32)
        torch.cuda.synchronize()
        with np.errstate(over="ignore"):
            want = olinear.act(zs, act)
        rel = 2.0 ** -21 * (1 + zs * zs / 2 if act == "gelu" else 2 + np.abs(zs)) + 2.0 ** -24
        _close(y, want, np.where(np.abs(want) > 2.0 ** -118, np.abs(want) * rel, 2.0 ** -118), act)
