"""Products of 8-bit operands on the GPU against the oracle's values.

u = 2^-24. With P = sum of |x w| over the reduction (in values): a run's 128 products are
exact in fp32's range and their sum takes at most 128 roundings of partial sums, 129 u P in
all; the scales' product, its product with the run's sum and the addition of up to 64 runs
(K <= 8192, split or not) add 66 u P. 2^-16 P = 256 u P bounds them.

A 16-bit output of more than 64 rows (grouped: of any), and gate/up with ``fast``, comes from the
matrix cores' 8-bit instruction, which cuts each of 8 neighbouring products to a multiple of 2^-13 2^E, E the largest sum
of the two factors' exponents, so that 2^E is at most the largest product: 7 products (the largest
keeps its bits: it has 7) lose less than 2^-13 2^E each, 7 * 2^-13 of the largest |x| times the
largest |w| among the eight, summed over the eights. silu, gelu: within 2^-21 (2 + |z|) and
2^-21 (1 + z^2 / 2) of the value, and their slope (at most 1.13) times z's error."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import fp8, linear as olinear

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_top_router_amd")
ops = moe.ops

DEV = "cuda"
SUM = 2.0 ** -16
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def rnd(shape, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bytes_of(q):
    return q.view(torch.uint8).cpu().numpy()


def row_operand(M, K, seed, std=1.0):
    """(q, scale, values); rows of very different sizes."""
    x = rnd((M, K), seed, std) * rnd((M, 1), seed + 1).exp2()
    q, s = ops.quantize_fp8(x)
    return q, s, fp8.row_values(bytes_of(q), s.cpu().numpy())


def weight_operand(N, K, seed, n=None):
    w = rnd((n or 1, N, K), seed, K ** -0.5)
    w = w * rnd((n or 1, 1, K), seed + 1).abs()
    q, s = ops.quantize_fp8_weights(w if n else w[0])
    if n:
        return q, s, [fp8.weight_values(bytes_of(q[e]), s[e].cpu().numpy()) for e in range(n)]
    return q, s, fp8.weight_values(bytes_of(q), s.cpu().numpy())


def close(got, want, tol):
    got = np64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def cut(xv, wv):
    """What the 8-bit instruction may lose: see above."""
    most = lambda v: np.abs(np.pad(v, ((0, 0), (0, -v.shape[1] % 8)))).reshape(len(v), -1, 8).max(axis=2)  # noqa: E731
    return 7 * 2.0 ** -13 * (most(xv) @ most(wv).T)


def check_linear(y, xv, wv, bias=None, act="none", res=None, exact=None):
    exact = (len(y) <= 64 or y.dtype == torch.float32) if exact is None else exact
    r = None if res is None else np64(res)
    want, z = olinear.linear(xv, wv, None if bias is None else np64(bias), act, r)
    size = np.abs(xv) @ np.abs(wv).T
    tol = SUM * (size + (0 if bias is None else np.abs(np64(bias)))) * 1.13
    if not exact:
        tol = tol + 1.13 * cut(xv, wv)
    a = olinear.act(z, act)
    if act in ("silu", "gelu"):
        tol = tol + np.abs(a) * 2.0 ** -21 * (2 + np.abs(z) if act == "silu" else 1 + z * z / 2) + 2.0 ** -118
    if r is not None:
        tol = tol + 2.0 ** -24 * (np.abs(a) + np.abs(r))
    close(y, want, tol * (1 + HALF[y.dtype]) + np.abs(want) * HALF[y.dtype] + TINY[y.dtype])


ROWS = [1, 2, 15, 16, 17, 32, 33, 64, 65, 96, 128, 130, 200, 256, 257, 400, 700]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("K, N", [(128, 128), (512, 136), (1040, 40), (16, 8), (2064, 640), (144, 1001)])
def test_linear(M, K, N):
    x, xs, xv = row_operand(M, K, M)
    w, ws, wv = weight_operand(N, K, K)
    check_linear(ops.linear_fp8(x, xs, w, ws), xv, wv)


@pytest.mark.parametrize("M, K, N", [(1, 7168, 100), (16, 4096, 512), (48, 8192, 48), (100, 8192, 128),
                                     (70, 4096, 512), (300, 7168, 264), (1023, 1024, 2304), (2048, 2048, 256)])
def test_linear_long_and_split(M, K, N):
    x, xs, xv = row_operand(M, K, 3)
    w, ws, wv = weight_operand(N, K, 5)
    check_linear(ops.linear_fp8(x, xs, w, ws), xv, wv)


@pytest.mark.parametrize("M", [1, 16, 20, 40, 64, 70])
@pytest.mark.parametrize("K, N", [(272, 6144), (1280, 6201), (128, 9000)])
def test_linear_few_rows_many_columns(M, K, N):
    x, xs, xv = row_operand(M, K, 25)
    w, ws, wv = weight_operand(N, K, 27)
    check_linear(ops.linear_fp8(x, xs, w, ws), xv, wv)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M, K, N", [(5, 256, 72), (40, 1040, 37), (150, 384, 264), (300, 272, 515), (90, 8192, 130)])
def test_linear_epilogues(act, out, M, K, N):
    x, xs, xv = row_operand(M, K, 7, 0.5)
    w, ws, wv = weight_operand(N, K, 9)
    bias = rnd((N,), 11)
    check_linear(ops.linear_fp8(x, xs, w, ws, bias=bias, act=act, out_dtype=out), xv, wv, bias, act)
    res = rnd((M, N), 12, dtype=torch.float16 if out == torch.float16 else torch.bfloat16)
    y = ops.linear_fp8(x, xs, w, ws, act=act, residual=res, out_dtype=out)
    check_linear(y, xv, wv, None, act, res)


def test_linear_whole_numbers_are_exact():
    # values and partial sums that fp32 and bf16 hold: nothing is rounded anywhere
    for M, K, N in ((3, 128, 16), (64, 512, 40), (200, 640, 300), (300, 4096, 128)):
        g = torch.Generator().manual_seed(M)
        xi = torch.randint(-1, 2, (M, K), generator=g) * (torch.rand((M, K), generator=g) < 0.05)
        wi = torch.randint(-2, 3, (N, K), generator=g)
        x, w = (t.float().to(torch.float8_e4m3fn).to(DEV) for t in (xi, wi))
        xs = torch.full((M, -(-K // 128)), 4.0, device=DEV)
        ws = torch.full((-(-N // 128), -(-K // 128)), 0.5, device=DEV)
        want = 2 * (xi @ wi.t())
        got = ops.linear_fp8(x, xs, w, ws, out_dtype=torch.float32)
        assert torch.equal(got.cpu(), want.float())


def test_every_scale_reaches_its_run_and_block():
    M, K, N = 150, 640, 400
    x = torch.ones((M, K), device=DEV).to(torch.float8_e4m3fn)
    w = torch.ones((N, K), device=DEV).to(torch.float8_e4m3fn)
    g = torch.Generator().manual_seed(1)
    xs = torch.randint(1, 9, (M, 5), generator=g).float().to(DEV)
    ws = torch.randint(1, 9, (4, 5), generator=g).float().to(DEV)
    want = 128 * (xs @ ws.repeat_interleave(128, 0)[:N].t())
    for m in (150, 64, 20, 5):
        got = ops.linear_fp8(x[:m], xs[:m], w, ws, out_dtype=torch.float32)
        assert torch.equal(got, want[:m])


def test_linear_places():
    M, K, N = 130, 272, 200
    x, xs, xv = row_operand(M, K, 13)
    w, ws, wv = weight_operand(N, K, 15)
    res = rnd((M, N), 16, dtype=torch.bfloat16)
    want = ops.linear_fp8(x, xs, w, ws, residual=res)
    a = res.clone()
    assert ops.linear_fp8(x, xs, w, ws, residual=a, out=a) is a and torch.equal(a, want)
    for pad, first in ((56, 8), (3, 1)):  # rows apart, 16-byte aligned and not
        big = torch.full((M + 1, N + pad), 7.0, dtype=torch.bfloat16, device=DEV)
        out = big[:M, first:first + N]
        ops.linear_fp8(x, xs, w, ws, residual=res, out=out)
        assert torch.equal(out, want)
        assert (big[:, :first] == 7).all() and (big[:, first + N:] == 7).all() and (big[M] == 7).all()
    assert ops.linear_fp8(x[:0], xs[:0], w, ws).shape == (0, N)


@pytest.mark.parametrize("M", [3, 40, 60, 200, 300])
def test_linear_nan_rows_stay_alone(M):
    K, N = 400, 264
    x, xs, xv = row_operand(M, K, 17)
    w, ws, wv = weight_operand(N, K, 19)
    clean = ops.linear_fp8(x, xs, w, ws)
    b = x.view(torch.uint8).clone()
    b[1, 5] = 0x7f
    y = ops.linear_fp8(b.view(torch.float8_e4m3fn), xs, w, ws)
    assert torch.isnan(y[1]).all()
    keep = [i for i in range(M) if i != 1]
    assert torch.equal(y[keep], clean[keep])
    s = xs.clone()
    s[2, 1] = float("inf")
    y = ops.linear_fp8(x, s, w, ws)
    keep = [i for i in range(M) if i != 2]
    assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[2]).any()


def test_linear_gradient_of_rows():
    """dx = dy w, the same product on the turned weights: they hold the same values."""
    M, K, N = 70, 384, 272
    w = rnd((N, K), 21, 0.1, torch.bfloat16)
    q, s = ops.quantize_fp8_weights(w)
    qt, st = ops.quantize_fp8_weights(w, transpose=True)
    assert torch.equal(qt.view(torch.uint8), q.view(torch.uint8).t()) and torch.equal(st, s.t())
    dy, ds, dv = row_operand(M, N, 22)
    wv = fp8.weight_values(bytes_of(q), s.cpu().numpy())
    dx = ops.linear_fp8(dy, ds, qt, st, out_dtype=torch.float32)
    check_linear(dx, dv, wv.T)
    # against differences of <dy, y> in the direction of one entry of x: y is linear in x
    xv = np64(rnd((M, K), 24))
    f = lambda x: ((x @ wv.T) * dv).sum()  # noqa: E731
    for m, k in ((0, 0), (69, 383), (12, 200)):
        e = np.zeros((M, K))
        e[m, k] = 0.5
        size = (np.abs(dv[m]) * np.abs(wv[:, k])).sum()
        assert abs((f(xv + e) - f(xv - e)) - float(dx[m, k])) <= SUM * size * 1.13 + 1e-9


# ---------------------------------------------------------------- grouped

def layout_of(counts, align):
    at = [0]
    for c in counts:
        at.append(at[-1] + -(-c // align) * align)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return i32(at), i32(counts), at


def check_h(h, hs, rows, xv, w1v, w3v, what, exact=True):
    g, u = xv @ w1v.T, xv @ w3v.T
    gs, us = np.abs(xv) @ np.abs(w1v).T, np.abs(xv) @ np.abs(w3v).T
    want = olinear.act(g, "silu") * u
    ge, ue = SUM * gs, SUM * us
    if not exact:
        ge, ue = ge + cut(xv, w1v), ue + cut(xv, w3v)
    err = 1.13 * (ge * np.abs(u) + ge * ue) + np.abs(olinear.act(g, "silu")) * ue \
        + np.abs(want) * 2.0 ** -20 * (2 + np.abs(g)) + 1e-37
    n = want.shape[1] // 128
    s = hs[rows].cpu().numpy().astype(np.float64)
    for j in range(n):
        c = np.s_[:, 128 * j:128 * j + 128]
        amax, most = np.abs(want[c]).max(axis=1), err[c].max(axis=1)
        ws = np.maximum(amax / 448, 2.0 ** -126)
        assert (np.abs(s[:, j] - ws) <= most / 448 + ws * 2.0 ** -23).all(), what
    got = fp8.row_values(bytes_of(h[rows]), s)
    step = np.repeat(s, 128, axis=1)
    tol = np.maximum((np.abs(want) + err) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -16) + err
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, bad.sum(), np.argwhere(bad)[:4])


COUNTS = [
    [1], [16], [17], [64], [65], [300],
    [0, 5, 0, 70, 33, 64, 0], [256, 257, 255], [513, 2, 0, 130, 48, 97], [0, 0], [31] * 40 + [0, 200],
]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("H, I, align", [(128, 128, 128), (384, 256, 16), (1024, 384, 1)])
@pytest.mark.parametrize("fast", [False, True])
def test_grouped(counts, H, I, align, fast):
    off, cnt, at = layout_of(counts, align)
    m_cap = at[-1] + 9
    E = len(counts)
    x, xs, xv = row_operand(m_cap, H, 31)
    w1, s1, w1v = weight_operand(I, H, 33, E)
    w3, s3, w3v = weight_operand(I, H, 35, E)
    w2, s2, w2v = weight_operand(H, I, 37, E)
    h = torch.full((m_cap, I), 0x55, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    hs = torch.full((m_cap, I // 128), -3.0, device=DEV)
    y = torch.full((m_cap, H), -7.0, dtype=torch.bfloat16, device=DEV)
    ops.grouped_gate_up_fp8(x, xs, off, cnt, w1, s1, w3, s3, h=h, h_scale=hs, fast=fast)
    ops.grouped_down_fp8(h, hs, off, cnt, w2, s2, out=y)
    left = np.ones(m_cap, bool)
    for e, c in enumerate(counts):
        rows = slice(at[e], at[e] + c)
        left[rows] = False
        if c:
            check_h(h, hs, rows, xv[rows], w1v[e], w3v[e], (e, c), not fast)
            hv = fp8.row_values(bytes_of(h[rows]), hs[rows].cpu().numpy())
            check_linear(y[rows], hv, w2v[e], exact=False)
    left = torch.from_numpy(left).to(DEV)
    assert (h.view(torch.uint8)[left] == 0x55).all() and (hs[left] == -3).all() and (y[left] == -7).all()


@pytest.mark.parametrize("counts", [[3, 0, 90, 17], [200, 40, 0, 300]], ids=str)
def test_grouped_gather_is_the_copy(counts):
    T, H, I, k = 320, 512, 256, 4
    off, cnt, at = layout_of(counts, 128)
    x, xs, _ = row_operand(T, H, 41)
    w1, s1, _ = weight_operand(I, H, 43, 4)
    w3, s3, _ = weight_operand(I, H, 45, 4)
    g = torch.Generator().manual_seed(7)
    src = torch.full((at[-1] + 5,), -1, dtype=torch.int32)
    for e, c in enumerate(counts):
        src[at[e]:at[e] + c] = (torch.randperm(T, generator=g)[:c] * k + e).to(torch.int32)
    src = src.to(DEV)
    tok = (src.clamp(min=0) // k).long()
    xp = x.view(torch.uint8)[tok].view(torch.float8_e4m3fn)
    valid = src >= 0
    want = ops.grouped_gate_up_fp8(xp, xs[tok], off, cnt, w1, s1, w3, s3)
    got = ops.grouped_gate_up_fp8(x, xs, off, cnt, w1, s1, w3, s3, src_row=src, top_k=k, max_rows=T)
    assert torch.equal(got[0].view(torch.uint8)[valid], want[0].view(torch.uint8)[valid])
    assert torch.equal(got[1][valid], want[1][valid])


def test_grouped_counts_that_do_not_fit():
    H = I = 128
    w1, s1, w1v = weight_operand(I, H, 51, 3)
    x, xs, xv = row_operand(100, H, 53)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    # a negative count and offset, a count past the end, more rows than max_rows
    for off, cnt, most, rows in (([0, 10, 90, 100], [-5, 8, 1000], 100, [(), range(10, 18), range(90, 100)]),
                                 ([-4, 20, 200, 300], [9, 80, 5], 70, [(), range(20, 90), ()])):
        h = torch.zeros((100, I), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        hs = torch.full((100, 1), -1.0, device=DEV)
        y = torch.full((100, H), -7.0, dtype=torch.bfloat16, device=DEV)
        ops.grouped_gate_up_fp8(x, xs, i32(off), i32(cnt), w1, s1, w1, s1, max_rows=most, h=h, h_scale=hs)
        ops.grouped_down_fp8(x, xs, i32(off), i32(cnt), w1, s1, max_rows=most, out=y)
        left = np.ones(100, bool)
        for e, r in enumerate(rows):
            r = list(r)
            left[r] = False
            if r:
                check_h(h, hs, r, xv[r], w1v[e], w1v[e], e)
                check_linear(y[r], xv[r], w1v[e], exact=False)
        left = torch.from_numpy(left).to(DEV)
        assert (hs[left] == -1).all() and (y[left] == -7).all()


@pytest.mark.parametrize("c", [10, 50, 100])
def test_grouped_nan_rows_stay_alone(c):
    H, I = 256, 128
    off, cnt, _ = layout_of([c], 1)
    x, xs, _ = row_operand(c, H, 61)
    w1, s1, _ = weight_operand(I, H, 63, 1)
    h0, hs0 = ops.grouped_gate_up_fp8(x, xs, off, cnt, w1, s1, w1, s1)
    b = x.view(torch.uint8).clone()
    b[3, 200] = 0xff
    h, hs = ops.grouped_gate_up_fp8(b.view(torch.float8_e4m3fn), xs, off, cnt, w1, s1, w1, s1)
    assert np.isnan(fp8.decode(bytes_of(h[3]))).all() and (hs[3] == 2.0 ** -126).all()
    keep = [i for i in range(c) if i != 3]
    assert torch.equal(h.view(torch.uint8)[keep], h0.view(torch.uint8)[keep]) and torch.equal(hs[keep], hs0[keep])


def test_stream_and_graph():
    x, xs, _ = row_operand(300, 512, 71)
    w, ws, _ = weight_operand(256, 512, 73, 2)
    off, cnt, at = layout_of([100, 30], 128)

    def step():
        h, hs = ops.grouped_gate_up_fp8(x, xs, off, cnt, w, ws, w, ws)
        return [ops.linear_fp8(x, xs, w[0], ws[0]), ops.linear_fp8(x[:8], xs[:8], w[1], ws[1]),
                *(t[r] for t in (h.view(torch.uint8), hs) for r in (slice(0, 100), slice(128, 158)))]

    want = [t.clone() for t in step()]
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
        new, s, _ = row_operand(300, 512, 80 + k)
        x.copy_(new)
        xs.copy_(s)
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)), k


def test_refusals():
    x, xs, _ = row_operand(4, 128, 91)
    w, ws, _ = weight_operand(64, 128, 93)
    with pytest.raises(TypeError, match="float8"):
        ops.linear_fp8(x.float(), xs, w, ws)
    with pytest.raises(ValueError, match="x_scale"):
        ops.linear_fp8(x, xs[:3], w, ws)
    with pytest.raises(ValueError, match="w_scale"):
        ops.linear_fp8(x, xs, w, ws.expand(2, 1).contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        ops.linear_fp8(x, xs, w.view(torch.uint8).t().contiguous().t().view(torch.float8_e4m3fn), ws)
    with pytest.raises(TypeError, match="residual"):
        ops.linear_fp8(x, xs, w, ws, residual=torch.zeros((4, 64), dtype=torch.float16, device=DEV))
    with pytest.raises(TypeError, match="out must be"):
        ops.linear_fp8(x, xs, w, ws, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="act"):
        ops.linear_fp8(x, xs, w, ws, act="tanh")
    off, cnt, _ = layout_of([4], 1)
    with pytest.raises(ValueError, match="stack"):
        ops.grouped_down_fp8(x, xs, off, cnt, w, ws)
    with pytest.raises(moe.MoEError, match="MOE_ERR_UNSUPPORTED"):
        ops.grouped_down_fp8(x, xs, off, cnt, w.unsqueeze(0), ws.unsqueeze(0))  # 64 columns
    with pytest.raises(ValueError, match="offsets"):
        ops.grouped_down_fp8(x, xs, off[:1], cnt, w.unsqueeze(0), ws.unsqueeze(0))


@pytest.mark.parametrize("M, K, N", [(40, 7168, 256), (300, 2048, 512), (300, 7168, 640)])
def test_error_on_normal_values(M, K, N):
    """fp32 outputs to 2e-6 of the norm (24-bit sums: 0.3 u sqrt(roundings) and cancellation; a
    plain fp32 product has 8e-7 at K = 8192); 16-bit ones have their rounding, at most half a step."""
    x, xs = ops.quantize_fp8(rnd((M, K), 95))
    w, ws = ops.quantize_fp8_weights(rnd((N, K), 96))
    want = fp8.row_values(bytes_of(x), xs.cpu().numpy()) @ fp8.weight_values(bytes_of(w), ws.cpu().numpy()).T
    for dt, most in ((torch.float32, 2e-6), (torch.bfloat16, HALF[torch.bfloat16]), (torch.float16, HALF[torch.float16])):
        y = np64(ops.linear_fp8(x, xs, w, ws, out_dtype=dt))
        assert np.linalg.norm(y - want) <= most * np.linalg.norm(want), dt


def far_rows(M, K, few, seed):
    """(q, scale, the last rows' values): zeros but for the last `few` rows."""
    q = torch.zeros((M, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    s = torch.zeros((M, -(-K // 128)), device=DEV)
    fq, fs, v = row_operand(few, K, seed)
    q.view(torch.uint8)[-few:] = fq.view(torch.uint8)
    s[-few:] = fs
    return q, s, v


@pytest.mark.parametrize("K, N", [(2048, 128), (128, 2048)])
def test_rows_past_32_bits(K, N):
    M, few = 2200000, 300  # 4.5e9 elements of x or of y
    x, xs, xv = far_rows(M, K, few, 70)
    w, ws, wv = weight_operand(N, K, 72)
    y = ops.linear_fp8(x, xs, w, ws)
    check_linear(y[-few:], xv, wv, exact=False)
    del y
    off = torch.tensor([0, M - few, M], dtype=torch.int32, device=DEV)
    cnt = torch.tensor([10, few], dtype=torch.int32, device=DEV)
    y = ops.grouped_down_fp8(x, xs, off, cnt, torch.stack([w.view(torch.uint8)] * 2).view(w.dtype), torch.stack([ws] * 2))
    check_linear(y[-few:], xv, wv, exact=False)
    del y
    w3, s3, v3 = weight_operand(N, K, 74, 2)
    h, hs = ops.grouped_gate_up_fp8(x, xs, off, cnt, torch.stack([w.view(torch.uint8)] * 2).view(w.dtype),
                                    torch.stack([ws] * 2), w3, s3)
    check_h(h[-few:], hs[-few:], slice(None), xv, wv, v3[1], "far rows")


@pytest.mark.parametrize("M", [16, 100])
def test_weights_past_32_bits(M):
    N, K, few = 1 << 20, 4352, 256  # 4.6e9 elements
    x, xs, xv = row_operand(M, K, 76)
    w = torch.zeros((N, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    ws = torch.zeros((N // 128, K // 128), device=DEV)
    lw, ls, wv = weight_operand(few, K, 80)
    w.view(torch.uint8)[-few:] = lw.view(torch.uint8)
    ws[-few // 128:] = ls
    y = ops.linear_fp8(x, xs, w, ws)
    assert (y[:, :-few] == 0).all()
    check_linear(y[:, -few:], xv, wv, exact=M <= 64)


def test_experts_past_32_bits():
    E, N, K, few = 520, 2048, 4096, 40  # 4.4e9 elements of each matrix stack
    x, xs, xv = row_operand(few, K, 82)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    cnt = torch.zeros(E, dtype=torch.int32, device=DEV)
    off[E], cnt[E - 1] = few, few
    w = [torch.zeros((E, N, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    s = [torch.zeros((E, N // 128, K // 128), device=DEV) for _ in range(2)]
    v = []
    for i in range(2):
        q, sc, val = weight_operand(N, K, 84 + 2 * i)
        w[i].view(torch.uint8)[-1], s[i][-1] = q.view(torch.uint8), sc
        v.append(val)
    h, hs = ops.grouped_gate_up_fp8(x, xs, off, cnt, w[0], s[0], w[1], s[1])
    check_h(h, hs, slice(None), xv, v[0], v[1], "last expert")
    y = ops.grouped_down_fp8(x, xs, off, cnt, w[0], s[0])
    check_linear(y, xv, v[0], exact=False)


def test_two_calls_at_once():
    """Split products on two streams, each with its own workspace, give what they give alone."""
    M, K, N = 70, 4096, 256
    w, ws, _ = weight_operand(N, K, 90)
    rows = [row_operand(M, K, 92 + 2 * i)[:2] for i in range(2)]
    assert ops.linear_fp8_workspace_bytes(rows[0][0], w) > 0
    alone = [ops.linear_fp8(*r, w, ws) for r in rows]
    streams = [torch.cuda.Stream() for _ in rows]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(6):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(ops.linear_fp8(*rows[i], w, ws))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, alone[i]) for y in got[i])
