"""Cases of the 8-bit operators and the root-mean-square norm, and their plain forms.

``run`` makes one pass of one operator on what ``prepare`` made. With ``own``
false it computes the operator from elementary torch operations in 32 bits;
with ``own`` true it makes the calls of ``combine_top_router_amd.ops``.
``exact`` computes the same outputs from the definitions in 64 bits.

Values in 8 bits are e4m3 (``torch.float8_e4m3fn``) with fp32 scales: a row's
for each 128 of its columns, a weight matrix's for each block of 128 x 128.

Operators (a case's ``op``):

  norm        the residual's addition, the root-mean-square norm, its output in
              the rows' type and/or in 8 bits with scales
  norm_grad   the gradients of the norm's rows and gain
  quant       rows or weights to 8 bits with scales
  linear      act(x w^T + bias) + residual on 8-bit operands
  gate_up     silu(x W1) * (x W3) of each expert's rows, 8-bit in and out
  down        h W2 of each expert's rows, 8-bit in, bf16 out
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
TOP = 448.0  # e4m3's largest value
LEAST = 2.0 ** -126


# ---------------------------------------------------------------- cases

def _norm(name, rows, hidden, dtype="bf16", residual=True, y=True, q=True, op="norm"):
    return dict(name=name, op=op, rows=rows, hidden=hidden, dtype=dtype, residual=residual, y=y,
                q=q)


def _linear(name, rows, inner, cols, out="bf16", bias=False, act="none", residual=False):
    return dict(name=name, op="linear", rows=rows, inner=inner, cols=cols, out=out, bias=bias,
                act=act, residual=residual)


def _experts(name, op, tokens, experts, local, top_k, hidden, inter, skew=0.0):
    return dict(name=name, op=op, tokens=tokens, experts=experts, local=local, top_k=top_k,
                hidden=hidden, inter=inter, skew=skew)


def listed():
    return [
        # before the experts of one decoding step: bf16 for the router, 8 bits for the experts
        _norm("norm decode", 16, 7168),
        # the same for the large batch of the benchmark's layer, 8 bits only
        _norm("norm large", 65536, 7168, y=False),
        # a ragged batch whose rows end inside a block of scales, no residual
        _norm("norm ragged", 8191, 4104, dtype="fp16", residual=False),
        # its backward in training, the residual stream's own gradient added
        _norm("norm grad", 16384, 7168, op="norm_grad"),
        # the activations of one GPU's share before a product
        dict(name="quant rows", op="quant", kind="rows", count=1, rows=8192, cols=7168,
             dtype="bf16"),
        # one share's expert matrices at load time, from math orientation
        dict(name="quant weights", op="quant", kind="weights", count=32, rows=7168, cols=2048,
             dtype="bf16"),
        # a shared expert's first products in one decoding step
        _linear("linear decode", 16, 7168, 4096),
        # a dense layer's first product on a ragged batch
        _linear("linear ragged", 1023, 4096, 14336, out="fp16", bias=True, act="gelu"),
        # a shared expert's down projection added to the routed experts' output
        _linear("linear large", 65536, 2048, 7168, residual=True),
        # the experts of one GPU's share in a decoding step of 128 sequences
        _experts("gate up decode", "gate_up", 128, 256, 32, 8, 7168, 2048),
        # the same share's batch of the benchmark
        _experts("gate up share", "gate_up", 8192, 256, 32, 8, 7168, 2048),
        # small experts, all on one GPU, routed with a strong skew
        _experts("down skew", "down", 8192, 128, 128, 8, 2048, 768, skew=1.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "quant", "linear", "linear", "gate_up", "down"])
    if op in ("norm", "norm_grad"):
        hidden = 8 * _log(rng, 8, 2048)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 65536 * 7168 // (4 if dtype == "fp32" or op == "norm_grad" else 2)
        y, q = rng.choice([(True, True), (True, False), (False, True)])
        return dict(op=op, rows=min(_log(rng, 1, 65536), most // hidden), hidden=hidden, dtype=dtype,
                    residual=rng.random() < 0.6, y=y, q=q)
    if op == "quant":
        kind = rng.choice(["rows", "weights"])
        rows, cols = _log(rng, 1, 16384), 8 * _log(rng, 8, 2048)
        if kind == "weights":
            rows = (rows + 15) // 16 * 16
        count = 1 if kind == "rows" else max(1, min(_log(rng, 1, 64), 2 ** 28 // (rows * cols)))
        return dict(op=op, kind=kind, count=count, rows=rows, cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "linear":
        while True:
            rows, inner, cols = _log(rng, 1, 65536), 16 * _log(rng, 4, 1024), _log(rng, 8, 16384)
            if rows * inner * cols <= 9e11 and rows * max(inner, cols) <= 4.5e8:
                break
        out = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return dict(op=op, rows=rows, inner=inner, cols=cols, out=out, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "silu", "gelu"]),
                    residual=out != "fp32" and rng.random() < 0.4)
    while True:
        experts = rng.choice([8, 16, 60, 64, 128, 256])
        local = rng.choice([experts, max(1, experts // 8)])
        top_k = min(experts, rng.choice([1, 2, 4, 8]))
        hidden, inter = 128 * _log(rng, 1, 56), 128 * _log(rng, 1, 56)
        tokens = _log(rng, 1, 16384)
        rows = tokens * top_k * local / experts
        if (local * hidden * inter <= 4.8e8 and rows * hidden * inter <= 1.3e11 and
                rows * max(hidden, inter) <= 2e8):
            break
    return dict(op=op, tokens=tokens, experts=experts, local=local, top_k=top_k, hidden=hidden,
                inter=inter, skew=rng.choice([0.0, 0.0, 0.6, 1.2]))


def _counts(case):
    """Rows of each local expert: every token to top_k of the experts, the popular ones more often."""
    c = case
    r = random.Random(c["tokens"] * 7919 + c["experts"] * 31 + c["top_k"])
    order = list(range(c["experts"]))
    r.shuffle(order)
    pull = [(1.0 + p) ** -c["skew"] for p in order]
    total = sum(pull)
    got = []
    for p in pull[:c["local"]]:
        mean = c["tokens"] * c["top_k"] * p / total
        n = int(round(r.gauss(mean, math.sqrt(mean)))) if mean > 30 else \
            sum(r.random() < mean / c["tokens"] for _ in range(c["tokens"]))
        got.append(max(0, min(c["tokens"], n)))
    if not any(got):
        got[0] = 1
    return got


def _offsets(counts, align=128):
    at = [0]
    for n in counts:
        at.append(at[-1] + (n + align - 1) // align * align)
    return at


# ---------------------------------------------------------------- inputs

def _padded(x, *dims):
    """x with the named dimensions filled up with zeros to multiples of 128."""
    pad = []
    for d in range(x.dim() - 1, -1, -1):
        pad += [0, -x.shape[d] % 128 if d - x.dim() in dims else 0]
    return torch.nn.functional.pad(x, pad)


def _to_8bit(v, amax):
    s = (amax / TOP).clamp(min=LEAST)
    return v * (1.0 / s), s


def _quant_rows(v):
    """(q, scales) of rows v [..., cols] in fp32."""
    b = _padded(v, -1).unflatten(-1, (-1, 128))
    q, s = _to_8bit(b, b.abs().amax(dim=-1, keepdim=True))
    return q.flatten(-2)[..., :v.shape[-1]].to(F8), s.squeeze(-1)


def _quant_weights(v):
    """(q, scales) of matrices v [..., N, K] in fp32."""
    b = _padded(v, -1, -2).unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    q, s = _to_8bit(b, b.abs().amax(dim=(-3, -1), keepdim=True))
    q = q.flatten(-4, -3).flatten(-2)[..., :v.shape[-2], :v.shape[-1]]
    return q.to(F8), s.squeeze(-1).squeeze(-2)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = case

    def normal(shape, dtype=torch.float32, std=1.0):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)

    def weights(n, cols, inner):
        w = torch.empty((n, cols, inner), device=DEV, dtype=F8)
        s = torch.empty((n, -(-cols // 128), -(-inner // 128)), device=DEV)
        for e in range(n):  # one matrix at a time: room
            w[e], s[e] = _quant_weights(normal((cols, inner), torch.bfloat16, inner ** -0.5).float())
        return w, s

    s = dict(case=c)
    if c["op"] in ("norm", "norm_grad"):
        t, shape = TYPES[c["dtype"]], (c["rows"], c["hidden"])
        s["x"] = normal(shape, t)
        s["gain"] = 1.0 + normal((c["hidden"],), std=0.2)
        s["residual"] = normal(shape, t, 2.0) if c["residual"] else None
        if c["op"] == "norm_grad":
            s["dy"] = normal(shape, t)
    elif c["op"] == "quant":
        shape = (c["rows"], c["cols"]) if c["kind"] == "rows" else (c["count"], c["rows"], c["cols"])
        s["x"] = torch.empty(shape, device=DEV, dtype=TYPES[c["dtype"]])
        for part in s["x"].view(-1, c["rows"], c["cols"]):
            part.copy_(normal(part.shape, std=1.0 if c["kind"] == "rows" else c["rows"] ** -0.5))
    elif c["op"] == "linear":
        M, K, N = c["rows"], c["inner"], c["cols"]
        s["x"], s["xs"] = _quant_rows(normal((M, K), torch.bfloat16).float())
        w, ws = weights(1, N, K)
        s["w"], s["ws"] = w[0], ws[0]
        s["bias"] = normal((N,), std=0.5) if c["bias"] else None
        s["residual"] = normal((M, N), TYPES[c["out"]]) if c["residual"] else None
    else:
        T, H, I, k = c["tokens"], c["hidden"], c["inter"], c["top_k"]
        counts = _counts(c)
        at = _offsets(counts)
        m_cap = max(1, at[-1])
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device=DEV)
        s["offsets"] = torch.tensor(at, dtype=torch.int32, device=DEV)
        if c["op"] == "gate_up":
            s["x"], s["xs"] = _quant_rows(normal((T, H), torch.bfloat16).float())
            s["w1"], s["s1"] = weights(len(counts), I, H)
            s["w3"], s["s3"] = weights(len(counts), I, H)
            src = torch.full((m_cap,), -1, dtype=torch.int32, device=DEV)
            for e, n in enumerate(counts):
                rows = torch.randperm(T, generator=g, device=DEV)[:n].sort().values
                src[at[e]:at[e] + n] = (rows * k + e % k).to(torch.int32)
            s["src_row"] = src
            s["h"] = torch.zeros((m_cap, I), device=DEV).to(F8)
            s["hs"] = torch.zeros((m_cap, I // 128), device=DEV)
        else:
            h = normal((m_cap, I), torch.bfloat16, 0.3).float()
            s["h"], s["hs"] = _quant_rows(h * normal((m_cap, 1)))
            s["w2"], s["s2"] = weights(len(counts), H, I)
            s["y"] = torch.zeros((m_cap, H), device=DEV, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "quant": _plain_quant,
            "linear": _plain_linear, "gate_up": _plain_gate_up, "down": _plain_down}[
                case["op"]](state, case)


def _run_own(s, c):
    from combine_top_router_amd import ops
    if c["op"] == "norm":
        return [t for t in ops.rms_norm(s["x"], s["gain"], residual=s["residual"], eps=1e-6,
                                        want_y=c["y"], want_fp8=c["q"]) if t is not None]
    if c["op"] == "norm_grad":
        return ops.rms_norm_backward(s["dy"], s["x"], s["gain"], eps=1e-6, dtotal=s["residual"])
    if c["op"] == "quant":
        if c["kind"] == "rows":
            return ops.quantize_fp8(s["x"])
        return ops.quantize_fp8_weights(s["x"], transpose=True)
    if c["op"] == "linear":
        return ops.linear_fp8(s["x"], s["xs"], s["w"], s["ws"], bias=s["bias"], act=c["act"],
                              residual=s["residual"], out_dtype=TYPES[c["out"]])
    if c["op"] == "gate_up":
        return ops.grouped_gate_up_fp8(s["x"], s["xs"], s["offsets"], s["counts"], s["w1"], s["s1"],
                                       s["w3"], s["s3"], src_row=s["src_row"], top_k=c["top_k"],
                                       max_rows=c["tokens"], h=s["h"], h_scale=s["hs"])
    return ops.grouped_down_fp8(s["h"], s["hs"], s["offsets"], s["counts"], s["w2"], s["s2"],
                                max_rows=c["tokens"], out=s["y"])


def _plain_norm(s, c):
    x = s["x"]
    out = []
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(x.dtype)
    v = x.float()
    y = v * (1.0 / ((v * v).mean(dim=1, keepdim=True) + 1e-6).sqrt()) * s["gain"]
    if c["y"]:
        out.append(y.to(x.dtype))
    if c["q"]:
        out += _quant_rows(y)
    return out + ([x] if s["residual"] is not None else [])


def _plain_norm_grad(s, c):
    v, dy = s["x"].float(), s["dy"].float()
    r = 1.0 / ((v * v).mean(dim=1, keepdim=True) + 1e-6).sqrt()
    xhat, gdy = v * r, dy * s["gain"]
    dx = r * (gdy - xhat * (gdy * xhat).mean(dim=1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return dx.to(s["x"].dtype), (dy * xhat).sum(dim=0)


def _plain_quant(s, c):
    if c["kind"] == "rows":
        return _quant_rows(s["x"].float())
    return _quant_weights(s["x"].float().transpose(1, 2).contiguous())


def _values(q, scale):
    """What 8-bit rows and their scales stand for, in fp32."""
    b = _padded(q.float(), -1).unflatten(-1, (-1, 128))
    return (b * scale.unsqueeze(-1)).flatten(-2)[..., :q.shape[-1]]


def _weight_values(q, scale):
    rows = scale.repeat_interleave(128, dim=-2)[..., :q.shape[-2], :]
    return _values(q, rows)


def _plain_linear(s, c):
    z = _values(s["x"], s["xs"]) @ _weight_values(s["w"], s["ws"]).t()
    if s["bias"] is not None:
        z = z + s["bias"]
    if c["act"] == "relu":
        z = z * (z > 0)
    elif c["act"] == "silu":
        z = z / (1.0 + (-z).exp())
    elif c["act"] == "gelu":
        z = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(TYPES[c["out"]])


def _plain_gate_up(s, c):
    counts = _counts(c)
    at = _offsets(counts)
    x = _values(s["x"], s["xs"])
    for e, n in enumerate(counts):  # the experts have rows of their own number
        rows = x[s["src_row"][at[e]:at[e] + n].long() // c["top_k"]]
        a = rows @ _weight_values(s["w1"][e], s["s1"][e]).t()
        b = rows @ _weight_values(s["w3"][e], s["s3"][e]).t()
        s["h"][at[e]:at[e] + n], s["hs"][at[e]:at[e] + n] = _quant_rows(a / (1.0 + (-a).exp()) * b)
    return s["h"], s["hs"]


def _plain_down(s, c):
    counts = _counts(c)
    at = _offsets(counts)
    for e, n in enumerate(counts):
        rows = slice(at[e], at[e] + n)
        s["y"][rows] = _values(s["h"][rows], s["hs"][rows]) @ \
            _weight_values(s["w2"][e], s["s2"][e]).t()
    return s["y"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    blocks = lambda n: -(-n // 128)  # noqa: E731
    if c["op"] in ("norm", "norm_grad"):
        n, b = c["rows"] * c["hidden"], size[c["dtype"]]
        if c["op"] == "norm_grad":
            return {"bytes": n * b * (4 if c["residual"] else 3) + 8 * c["hidden"], "flops": 12 * n}
        moved = n * b * (1 + 2 * c["residual"] + c["y"]) + 4 * c["hidden"]
        return {"bytes": moved + c["q"] * (n + 4 * c["rows"] * blocks(c["hidden"])), "flops": 6 * n}
    if c["op"] == "quant":
        n = c["count"] * c["rows"] * c["cols"]
        tall = c["rows"] if c["kind"] == "rows" else blocks(c["rows"])
        return {"bytes": n * (size[c["dtype"]] + 1) + 4 * c["count"] * tall * blocks(c["cols"]),
                "flops": 2 * n}
    if c["op"] == "linear":
        M, K, N = c["rows"], c["inner"], c["cols"]
        moved = M * (K + 4 * blocks(K)) + N * K + 4 * blocks(N) * blocks(K)
        moved += M * N * size[c["out"]] * (1 + c["residual"]) + 4 * N * c["bias"]
        return {"bytes": moved, "flops": 2 * M * N * K}
    H, I = c["hidden"], c["inter"]
    counts = _counts(c)
    rows, active = sum(counts), sum(n > 0 for n in counts)
    if c["op"] == "gate_up":
        tokens = min(rows, c["tokens"])  # a token's row is read once at least
        return {"bytes": max(1, tokens * (H + H // 32) + rows * (4 + I + I // 32) + 2 * active * H * I),
                "flops": 4 * rows * H * I}
    return {"bytes": max(1, rows * (I + I // 32 + 2 * H) + active * H * I), "flops": 2 * rows * H * I}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "quant": _exact_quant,
            "linear": _exact_linear, "gate_up": _exact_gate_up, "down": _exact_down}[
                case["op"]](s, case)


def _spread(scale, dim, size):
    """A scale for every element of a dimension of that size."""
    return scale.double().index_select(dim, torch.arange(size, device=scale.device) // 128)


def _exact_8bit(v):
    """Rows in units of their scale, not rounded to 8 bits, and the scales."""
    n = v.shape[1]
    s = torch.stack([v[:, a:a + 128].abs().max(dim=1).values for a in range(0, n, 128)], dim=1)
    s = torch.maximum(s / TOP, torch.full_like(s, LEAST))
    return v / _spread(s, 1, n), s


def _exact_norm(s, c):
    total, t = s["x"].double(), s["x"].dtype
    if s["residual"] is not None:
        total = total + s["residual"].double()
    # the norm is that of the rows as they are kept: summed in fp32, rounded to their type
    v = total.float().to(t).double()
    y = s["gain"].double() * v * torch.rsqrt(v.square().sum(dim=1, keepdim=True) / c["hidden"] + 1e-6)
    out = [y] if c["y"] else []
    if c["q"]:
        out += _exact_8bit(y)
    return out + ([total] if s["residual"] is not None else [])


def _exact_norm_grad(s, c):
    # the norm differentiated by autograd in 64 bits, some rows at a time
    gain = s["gain"].double().requires_grad_()
    dx, dgain = [], torch.zeros_like(gain)
    for v, dy in zip(s["x"].split(2048), s["dy"].split(2048)):
        v = v.double().requires_grad_()
        y = torch.nn.functional.rms_norm(v, (c["hidden"],), gain, 1e-6)
        a, b = torch.autograd.grad(y, (v, gain), dy.double())
        dx.append(a)
        dgain = dgain + b
    dx = torch.cat(dx)
    if s["residual"] is not None:
        dx += s["residual"].double()
    return dx, dgain


def _exact_quant(s, c):
    if c["kind"] == "rows":
        return _exact_8bit(s["x"].double())
    q = torch.empty((c["count"], c["cols"], c["rows"]), dtype=torch.float64, device=DEV)
    scales = []
    for e in range(c["count"]):
        w = s["x"][e].double()
        a = torch.stack([torch.stack([w[i:i + 128, j:j + 128].abs().max()
                                      for i in range(0, c["rows"], 128)])
                         for j in range(0, c["cols"], 128)])
        scales.append((a / TOP).clamp_min(LEAST))
        q[e] = w.t() / _spread(_spread(scales[-1], 0, c["cols"]), 1, c["rows"])
    return q, torch.stack(scales)


def _decoded(q, scale):
    return q.double() * _spread(scale, 1, q.shape[1])


def _decoded_weights(q, scale):
    return q.double() * _spread(_spread(scale, 0, q.shape[0]), 1, q.shape[1])


def _exact_linear(s, c):
    z = torch.nn.functional.linear(_decoded(s["x"], s["xs"]), _decoded_weights(s["w"], s["ws"]),
                                   None if s["bias"] is None else s["bias"].double())
    y = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
         "gelu": lambda v: v * torch.special.ndtr(v)}[c["act"]](z)
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_gate_up(s, c):
    h = torch.zeros(s["h"].shape, dtype=torch.float64, device=DEV)
    scale = torch.zeros(s["hs"].shape, dtype=torch.float64, device=DEV)
    token = torch.div(s["src_row"], c["top_k"], rounding_mode="floor").long()
    first = s["offsets"].tolist()
    for e, n in enumerate(s["counts"].tolist()):
        if n:
            at = torch.arange(first[e], first[e] + n, device=DEV)
            x = _decoded(s["x"][token[at]], s["xs"][token[at]])
            gate = x.matmul(_decoded_weights(s["w1"][e], s["s1"][e]).t())
            up = x.matmul(_decoded_weights(s["w3"][e], s["s3"][e]).t())
            h[at], scale[at] = _exact_8bit(torch.nn.functional.silu(gate) * up)
    return h, scale


def _exact_down(s, c):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    first = s["offsets"].tolist()
    for e, n in enumerate(s["counts"].tolist()):
        at = slice(first[e], first[e] + n)
        y[at] = _decoded(s["h"][at], s["hs"][at]).matmul(_decoded_weights(s["w2"][e], s["s2"][e]).t())
    return y
