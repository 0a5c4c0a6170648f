"""Every tile of the 8-bit products on the GPU, with each of its epilogues and with several
tiles to a workgroup, against the definition in 64 bits (on the GPU, for its size).

Bounds as in test_fp8_gemm_gpu.py: with P = sum of |x w| over the reduction, 2^-16 P for sums of 24 bits;
with ``fast`` 7 * 2^-13 of the largest |x| times the largest |w| among each eight besides; silu and
gelu within 2^-21 (2 + |z|) and 2^-21 (1 + z^2 / 2) of the value, their slope at most 1.13; half a step of
the output's type."""
from __future__ import annotations

import pytest
import torch

import fp8_sizes

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_top_router_amd")
ops = moe.ops

DEV, F8 = "cuda", torch.float8_e4m3fn
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SUM = 2.0 ** -16
HALF = {BF: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}


def rnd(shape, seed, std=1.0, dtype=F32):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def values(q, scale):
    """Rows of bytes and their scales in 64 bits; a matrix's with its scales repeated for the rows."""
    if len(scale) != len(q):
        scale = scale.repeat_interleave(128, dim=0)[:len(q)]
    return q.double() * scale.double().repeat_interleave(128, dim=1)[:, :q.shape[1]]


def row_operand(M, K, seed):
    x = rnd((M, K), seed, 0.5) * rnd((M, 1), seed + 1).exp2()
    q, s = ops.quantize_fp8(x)
    return q, s, values(q, s)


def weight_operand(N, K, seed):
    w = rnd((N, K), seed, K ** -0.5) * rnd((1, K), seed + 1).abs()
    q, s = ops.quantize_fp8_weights(w)
    return q, s, values(q, s)


def close(got, want, tol, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def sums(xv, wv, fast):
    """(the products' sums, what they may be off by)."""
    size = SUM * (xv.abs() @ wv.abs().T)
    if fast:
        most = lambda v: torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % 8)).unflatten(1, (-1, 8)).amax(2)  # noqa: E731
        size = size + 7 * 2.0 ** -13 * (most(xv) @ most(wv).T)
    return xv @ wv.T, size


ACTS = {"none": lambda z: z, "relu": torch.relu, "silu": lambda z: z * torch.sigmoid(z),
        "gelu": lambda z: z * torch.special.ndtr(z)}


def check(y, z, size, bias=None, act="none", res=None):
    if bias is not None:
        z, size = z + bias.double(), size + SUM * bias.double().abs()
    a, tol = ACTS[act](z), 1.13 * size
    if act in ("silu", "gelu"):
        tol = tol + a.abs() * 2.0 ** -21 * (2 + z.abs() if act == "silu" else 1 + z * z / 2) + 2.0 ** -118
    want = a
    if res is not None:
        want = a + res.double()
        tol = tol + 2.0 ** -24 * (a.abs() + res.double().abs())
    close(y, want, tol * (1 + HALF[y.dtype]) + want.abs() * HALF[y.dtype] + TINY[y.dtype], act)


@pytest.mark.parametrize("kind, case", [(k, c) for k in ("WALKS", "ODD_WALKS", "SINGLE", "SPLIT")
                                        for c in getattr(fp8_sizes, k)], ids=str)
def test_epilogues(kind, case):
    fast, _, _, M, K, N = case
    x, xs, xv = row_operand(M, K, 1)
    w, ws, wv = weight_operand(N, K, 3)
    z, size = sums(xv, wv, fast)
    del xv, wv
    call = lambda **kw: ops.linear_fp8(x, xs, w, ws, fast=fast, **kw)  # noqa: E731
    bias, res = rnd((N,), 5), rnd((M, N), 6, dtype=BF)

    check(call(), z, size)
    a = res.clone()
    assert call(residual=a, out=a) is a  # in place
    check(a, z, size, res=res)
    assert torch.equal(a, call(residual=res))
    check(call(bias=bias, act="gelu", out_dtype=F16), z, size, bias, "gelu")
    check(call(bias=bias, act="silu", residual=res, out_dtype=F32), z, size, bias, "silu", res)
    check(call(residual=res.to(F16), out_dtype=F16), z, size, res=res.to(F16))
    # rows that start 2 bytes off, and that lie apart: what lies between is left alone
    for first, pad in ((1, 2), (8, 8 + -N % 8)):
        big = torch.full((M + 1, N + first + pad), 7.0, dtype=BF, device=DEV)
        out = big[:M, first:first + N]
        call(bias=bias, act="relu", residual=res, out=out)
        check(out, z, size, bias, "relu", res)
        assert (big[:, :first] == 7).all() and (big[:, first + N:] == 7).all() and (big[M] == 7).all()


@pytest.mark.parametrize("case", fp8_sizes.WALKS + fp8_sizes.SPLIT, ids=str)
def test_nan_rows_stay_alone(case):
    fast, _, _, M, K, N = case
    x, xs, _ = row_operand(M, K, 7)
    w, ws, _ = weight_operand(N, K, 9)
    clean = ops.linear_fp8(x, xs, w, ws, fast=fast)
    b, s = x.view(torch.uint8).clone(), xs.clone()
    b[M // 2, K - 1] = 0x7f
    s[M - 1, 0] = float("inf")
    y = ops.linear_fp8(b.view(F8), s, w, ws, fast=fast)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[[M // 2, M - 1]] = False
    assert torch.isnan(y[M // 2]).all() and not torch.isfinite(y[M - 1]).any()
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("case", fp8_sizes.WALKS + fp8_sizes.SINGLE, ids=str)
def test_rows_do_not_depend_on_their_tile(case):
    """Runs enter in order whatever the tile: rows of a call are those of a call on them alone, where
    that has more than 64 rows and does not split the reduction either."""
    fast, _, _, M, K, N = case
    x, xs, _ = row_operand(M, K, 11)
    w, ws, _ = weight_operand(N, K, 13)
    assert K < 2048  # (at most 7 runs to a split of 2: none is taken at these sizes)
    whole = ops.linear_fp8(x, xs, w, ws, fast=fast, out_dtype=F32)
    for r in (slice(0, M // 2), slice(M // 3, M), slice(max(0, M - 300), M)):
        if ops.linear_fp8_workspace_bytes(x[r], w) == 0:
            assert torch.equal(ops.linear_fp8(x[r], xs[r], w, ws, fast=fast, out_dtype=F32), whole[r]), r


# ---------------------------------------------------------------- grouped

# 64 groups each. mixed: the large row tiles; small: those of 64 rows; ones: one past blocks and tiles
GROUPS = {
    "mixed": [0, 1, 17, 33, 161, 257, 513, 320] * 8,
    "small": [1, 17, 33, 48, 64, 0, 63, 49] * 8,
    "ones": [161, 321, 257, 97, 513, 241, 177, 305] * 8,
}


def layout_of(counts, align):
    at = [0]
    for c in counts:
        at.append(at[-1] + -(-c // align) * align)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return i32(at), i32(counts), at


def stack(n, N, K, seed):
    q = torch.empty((n, N, K), dtype=F8, device=DEV)
    s = torch.empty((n, N // 128, K // 128), device=DEV)
    for e in range(n):
        q[e], s[e] = ops.quantize_fp8_weights(rnd((N, K), seed + e, K ** -0.5))
    return q, s


def check_h(h, hs, xv, w1v, w3v, fast, what):
    (g, ge), (u, ue) = sums(xv, w1v, fast), sums(xv, w3v, fast)
    a = ACTS["silu"](g)
    want = a * u
    err = 1.13 * (ge * u.abs() + ge * ue) + a.abs() * ue + want.abs() * 2.0 ** -20 * (2 + g.abs()) + 1e-37
    blocks = lambda v: v.unflatten(1, (-1, 128)).amax(2)  # noqa: E731
    ws = (blocks(want.abs()) / 448).clamp(min=2.0 ** -126)
    close(hs, ws, blocks(err) / 448 + ws * 2.0 ** -23, what)
    step = hs.double().repeat_interleave(128, dim=1)
    tol = torch.maximum((want.abs() + err) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -16) + err
    close(values(h, hs), want, tol, what)


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_walks(groups, fast, gather):
    """Several tiles to each of 256 workgroups, groups and column tiles changing between them: gate/up has 9
    column tiles (1152), down 9 of which the last is half there (2176)."""
    counts, H, I, k = GROUPS[groups], 2176, 1152, 4
    E = len(counts)
    off, cnt, at = layout_of(counts, 16)
    m_cap, T = at[-1] + 3, 600
    least = sum(-(-c // 256) for c in counts) * 9
    assert least > 256, "several tiles to a workgroup"
    x, xs, xv = row_operand(T if gather else m_cap, H, 21)
    (w1, s1), (w3, s3), (w2, s2) = stack(E, I, H, 100), stack(E, I, H, 300), stack(E, H, I, 500)
    src, row = None, torch.arange(m_cap, device=DEV)
    if gather:
        g = torch.Generator().manual_seed(9)
        src = torch.full((m_cap,), -1, dtype=torch.int32)
        for e, c in enumerate(counts):
            src[at[e]:at[e] + c] = (torch.randperm(T, generator=g)[:c] * k + e % k).int()
        src = src.to(DEV)
        row = (src.clamp(min=0) // k).long()
    h = torch.full((m_cap, I), 0x55, dtype=torch.uint8, device=DEV).view(F8)
    hs = torch.full((m_cap, I // 128), -3.0, device=DEV)
    y = torch.full((m_cap, H), -7.0, dtype=BF, device=DEV)
    ops.grouped_gate_up_fp8(x, xs, off, cnt, w1, s1, w3, s3, src_row=src, top_k=k, max_rows=T if gather else None,
                            h=h, h_scale=hs, fast=fast)
    ops.grouped_down_fp8(h, hs, off, cnt, w2, s2, out=y, fast=fast)
    left = torch.ones(m_cap, dtype=torch.bool, device=DEV)
    xp, xsp = x.view(torch.uint8)[row], xs[row]
    for e, c in enumerate(counts):
        r = slice(at[e], at[e] + c)
        left[r] = False
        if not c:
            continue
        check_h(h[r], hs[r], xv[row[r]], values(w1[e], s1[e]), values(w3[e], s3[e]), fast, (e, c))
        z, size = sums(values(h[r], hs[r]), values(w2[e], s2[e]), fast)
        check(y[r], z, size)
        # the same bits as from a call of its own: another grid, other tiles
        o, n = layout_of([c], 1)[:2]
        own = lambda t: t[e:e + 1].clone()  # noqa: E731 (scales begin 16-byte aligned)
        h1, hs1 = ops.grouped_gate_up_fp8(xp[r].view(F8), xsp[r].clone(), o, n, w1[e:e + 1], own(s1), w3[e:e + 1],
                                          own(s3), fast=fast)
        assert torch.equal(h1.view(torch.uint8), h[r].view(torch.uint8)) and torch.equal(hs1, hs[r]), (e, c)
        y1 = ops.grouped_down_fp8(h[r], hs[r].clone(), o, n, w2[e:e + 1], own(s2), fast=fast)
        assert torch.equal(y1, y[r]), (e, c)
    assert (h.view(torch.uint8)[left] == 0x55).all() and (hs[left] == -3).all() and (y[left] == -7).all()


@pytest.mark.parametrize("K, N", [(2048, 128), (128, 2048)])
def test_fast_rows_past_32_bits(K, N):
    M, few = 2200000, 300  # 4.5e9 elements of x or of y
    x = torch.zeros((M, K), dtype=torch.uint8, device=DEV).view(F8)
    xs = torch.zeros((M, K // 128), device=DEV)
    q, s, xv = row_operand(few, K, 31)
    x[-few:], xs[-few:] = q, s
    w, ws, wv = weight_operand(N, K, 33)
    z, size = sums(xv, wv, True)
    y = ops.linear_fp8(x, xs, w, ws, fast=True)
    assert (y[:-few] == 0).all()
    check(y[-few:], z, size)
    off = torch.tensor([0, M - few, M], dtype=torch.int32, device=DEV)
    cnt = torch.tensor([10, few], dtype=torch.int32, device=DEV)
    w2, s2 = torch.stack([w.view(torch.uint8)] * 2).view(F8), torch.stack([ws] * 2)
    y = ops.grouped_down_fp8(x, xs, off, cnt, w2, s2, fast=True)
    check(y[-few:], z, size)
    del y
    h, hs = ops.grouped_gate_up_fp8(x, xs, off, cnt, w2, s2, w2, s2, fast=True)
    check_h(h[-few:], hs[-few:], xv, wv, wv, True, "far rows")
