"""Cases of the router, linear-layer and gradient-clipping operators, and their plain forms.

``run`` makes one pass of one operator on what ``prepare`` made. With ``own``
false it computes the operator from elementary torch operations in 32 bits
(64 where 32 would decide a choice or lose a long sum); with ``own`` true it
makes the calls of ``combine_top_router_amd.ops``. ``exact`` computes the same
outputs from the definitions in 64 bits.

Operators (a case's ``op``):

  route       experts and weights of each token from its router logits: softmax or sigmoid
              scores, an optional selection bias, optional groups of experts
  route_grad  the gradient of those weights with respect to the logits
  linear      act(x w^T + bias) + residual, optionally keeping the pre-activation
  linear_grad the gradients of x, w and bias
  clip        the norm of all gradients together, and the gradients scaled down to a bound
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _route(name, tokens, experts, top_k, score, bias, groups=1, top_groups=1, rank="top2",
           renorm=True, scale=1.0, op="route"):
    return dict(name=name, op=op, tokens=tokens, experts=experts, top_k=top_k, score=score,
                bias=bias, groups=groups, top_groups=top_groups, rank=rank, renorm=renorm,
                scale=scale)


def _linear(name, rows, inner, cols, dtype="bf16", order="nk", bias=False, act="none",
            residual=False, keep=False, f32=False, op="linear"):
    return dict(name=name, op=op, rows=rows, inner=inner, cols=cols, dtype=dtype, order=order,
                bias=bias, act=act, residual=residual, keep=keep, f32=f32)


def listed():
    return [
        # one decoding step of 16 sequences through a router with a balance bias and groups
        _route("route decode", 16, 256, 8, "sigmoid", True, 8, 4, scale=2.5),
        # a prefill batch through a plain softmax router whose weights are not renormalised
        _route("route softmax", 8191, 128, 8, "softmax", False, renorm=False),
        # the large-batch layer's router
        _route("route large", 65536, 256, 8, "sigmoid", True, 8, 4, scale=2.5),
        # its backward in training; a softmax without renormalisation reaches every logit
        _route("route grad", 65536, 256, 8, "softmax", False, renorm=False, op="route_grad"),
        # the router's projection for one decoding step: a handful of rows, fp32 logits
        _linear("gate decode", 16, 7168, 256, f32=True),
        # the same for the large batch: one read of the token rows
        _linear("gate large", 65536, 7168, 256, f32=True),
        # a shared expert's down projection added to the routed experts' output
        _linear("shared down", 8192, 2048, 7168, order="kn", residual=True),
        # a dense layer's first product on a ragged batch, its pre-activation kept for training
        _linear("dense in", 1023, 4096, 14336, dtype="fp16", bias=True, act="gelu", keep=True),
        # the router projection's backward: fp32 gradient of the logits, long reduction for w
        _linear("gate grad", 8192, 7168, 256, f32=True, op="linear_grad"),
        # the dense layer's backward
        _linear("dense grad", 4096, 4096, 14336, order="kn", bias=True, act="silu",
                op="linear_grad"),
        # a small model's gradients: many short tensors, where launches count
        dict(name="clip many", op="clip", kind="ragged", count=48, low=64, high=300000,
             dtype="mixed", bound=1.0),
        # the expert gradients of one GPU's share of a large layer, stacked as the layer holds them
        dict(name="clip share", op="clip", kind="experts", experts=32, hidden=7168, inter=2048,
             dtype="bf16", bound=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "linear", "linear", "linear_grad", "clip"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 6, 8])
        size = max(4, _log(rng, 8, 512) // groups)
        experts = groups * size
        top_groups = rng.randint(1, groups)
        # (one renormalised weight is a constant: its gradient is nothing but rounding)
        top_k = rng.randint(2 if op == "route_grad" else 1, min(16, top_groups * size))
        tokens = min(_log(rng, 1, 65536), 65536 * 256 // experts)
        score = rng.choice(["softmax", "sigmoid"])
        return {k: v for k, v in _route(
            None, tokens, experts, top_k, score, rng.random() < 0.6, groups, top_groups,
            rng.choice(["top2", "max"]), rng.random() < 0.7, rng.choice([1.0, 2.5, 16.0]),
            op).items() if k != "name"}
    if op in ("linear", "linear_grad"):
        while True:
            rows = _log(rng, 1, 65536)
            inner = 8 * _log(rng, 8, 2048)
            order = rng.choice(["nk", "kn"])
            cols = _log(rng, 8, 16384)
            if order == "kn":
                cols = (cols + 7) // 8 * 8
            if rows * inner * cols <= 2.4e11 and rows * max(inner, cols) <= 4.5e8:
                break
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        f32 = rng.random() < 0.3
        return {k: v for k, v in _linear(
            None, rows, inner, cols, dtype, order, rng.random() < 0.5,
            rng.choice(["none", "relu", "silu", "gelu"]), not f32 and rng.random() < 0.4,
            rng.random() < 0.3, f32, op).items() if k != "name"}
    return dict(op="clip", kind="ragged", count=rng.randint(1, 56), low=_log(rng, 1, 256),
                high=_log(rng, 1024, 4000000), dtype=rng.choice(["bf16", "fp16", "fp32", "mixed"]),
                bound=rng.choice([0.1, 1.0, 1e9]))


def _clip_sizes(case):
    """(shape, type) of each gradient tensor of a clip case."""
    if case["kind"] == "experts":
        e, h, i = case["experts"], case["hidden"], case["inter"]
        return [((e, h, i), "bf16"), ((e, h, i), "bf16"), ((e, i, h), "bf16"),
                ((e * 8, h), "bf16"), ((e * 8,), "fp32")]
    r = random.Random(case["count"] * 1000003 + case["high"])
    kinds = ["bf16", "fp16", "fp32"] if case["dtype"] == "mixed" else [case["dtype"]]
    return [((_log(r, case["low"], case["high"]),), r.choice(kinds))
            for _ in range(case["count"])]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(shape, dtype=torch.float32, std=1.0):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype) * std

    s = dict(case=case)
    if case["op"] in ("route", "route_grad"):
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        s["logits"] = normal((T, E), std=1.5)
        s["bias"] = normal((E,), std=0.1) if case["bias"] else None
        if case["op"] == "route_grad":
            s["topk_idx"] = s["logits"].topk(k, dim=1).indices.to(torch.int32).contiguous()
            s["grad_w"] = normal((T, k))
    elif case["op"] in ("linear", "linear_grad"):
        M, K, N = case["rows"], case["inner"], case["cols"]
        t = TYPES[case["dtype"]]
        s["x"] = normal((M, K), t)
        std = K ** -0.5
        s["w"] = normal((N, K), t, std) if case["order"] == "nk" else normal((K, N), t, std).t()
        if case["op"] == "linear":
            s["bias"] = normal((N,), std=0.5) if case["bias"] else None
            s["residual"] = normal((M, N), t) if case["residual"] else None
            s["pre"] = torch.empty((M, N), device=DEV, dtype=t) if case["keep"] else None
        else:
            s["dy"] = normal((M, N), torch.float32 if case["f32"] else t)
            s["pre"] = normal((M, N), t) if case["act"] != "none" else None
    else:
        s["grads"], s["outs"] = [], []
        for shape, t in _clip_sizes(case):
            s["grads"].append(normal(shape, TYPES[t], 0.02))
            s["outs"].append(torch.empty_like(s["grads"][-1]))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"route": _plain_route, "route_grad": _plain_route_grad, "linear": _plain_linear,
            "linear_grad": _plain_linear_grad, "clip": _plain_clip}[case["op"]](state, case)


def _run_own(s, c):
    from combine_top_router_amd import ops
    if c["op"] == "route":
        return ops.route_scored(s["logits"], c["top_k"], bias=s["bias"], score=c["score"],
                                num_groups=c["groups"], top_groups=c["top_groups"],
                                group_rank=c["rank"], renormalise=c["renorm"], scale=c["scale"])
    if c["op"] == "route_grad":
        return ops.route_scored_backward(s["logits"], s["topk_idx"], s["grad_w"],
                                         score=c["score"], renormalise=c["renorm"],
                                         scale=c["scale"])
    if c["op"] == "linear":
        out = ops.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"],
                         out_dtype=torch.float32 if c["f32"] else None, pre=s["pre"])
        return (out, s["pre"]) if c["keep"] else out
    if c["op"] == "linear_grad":
        dx, dw, dbias = ops.linear_backward(s["dy"], s["x"], s["w"], act=c["act"], pre=s["pre"],
                                            want_dbias=c["bias"])
        return (dx, dw, dbias) if c["bias"] else (dx, dw)
    norm = ops.clip_grad_norm(s["grads"], c["bound"], out=s["outs"])
    return [norm] + s["outs"]


# Scores and choices in 64 bits: two scores next to each other may differ by
# less than 32 bits hold once they have been through exp, and the choice
# between them is an integer.
def _plain_scores(logits, score):
    l = logits.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + (-l).exp())
    e = (l - l.max(dim=1, keepdim=True).values).exp()
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(s, c):
    T, E, G = c["tokens"], c["experts"], c["groups"]
    p = _plain_scores(s["logits"], c["score"])
    v = p if s["bias"] is None else p + s["bias"].double()
    if c["top_groups"] < G:
        r = v.view(T, G, E // G).sort(dim=2, descending=True).values
        r = r[:, :, 0] + r[:, :, 1] if c["rank"] == "top2" else r[:, :, 0]
        best = r.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=v.device).scatter(1, best, True)
        v = v.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    idx = v.sort(dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.to(torch.int32), (w * c["scale"]).float()


def _plain_route_grad(s, c):
    l, g, idx = s["logits"], s["grad_w"], s["topk_idx"].long()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + (-l.gather(1, idx)).exp())
        d = p * (1.0 - p)
        if c["renorm"]:
            total = p.sum(dim=1, keepdim=True)
            g = (g - (g * p).sum(dim=1, keepdim=True) / total) / total
        return torch.zeros_like(l).scatter(1, idx, c["scale"] * g * d)
    e = (l - l.max(dim=1, keepdim=True).values).exp()
    p = e / e.sum(dim=1, keepdim=True)
    q = p.gather(1, idx)
    if c["renorm"]:
        q = q / q.sum(dim=1, keepdim=True)
        inner = (q * g).sum(dim=1, keepdim=True)
        return torch.zeros_like(l).scatter(1, idx, c["scale"] * q * (g - inner))
    inner = (q * g).sum(dim=1, keepdim=True)
    return c["scale"] * p * (torch.zeros_like(l).scatter(1, idx, g) - inner)


def _plain_act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1.0 + (-z).exp())
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _plain_act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + (-z).exp())
        return p * (1.0 + z * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + \
        z * (-0.5 * z * z).exp() * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_linear(s, c):
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _plain_act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y if c["f32"] else y.to(s["x"].dtype)
    return (y, z.to(s["x"].dtype)) if c["keep"] else y


def _plain_linear_grad(s, c):
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _plain_act_slope(s["pre"].float(), c["act"])
    x, w = s["x"], s["w"]
    dx = (dz @ w.float()).to(x.dtype)
    if c["order"] == "nk":
        dw = (dz.t() @ x.float()).to(w.dtype)
    else:
        dw = (x.float().t() @ dz).to(w.dtype).t()
    return (dx, dw, dz.sum(dim=0)) if c["bias"] else (dx, dw)


def _plain_clip(s, c):
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for g in s["grads"]:  # a sum of up to half a billion squares: 64 bits
        total = total + g.double().square().sum()
    norm = total.sqrt()
    coef = (c["bound"] / (norm + 1e-6)).clamp(max=1.0).float()
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(g.float() * coef)
    return [norm.float().view(1)] + s["outs"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] in ("route", "route_grad"):
        T, E, k = c["tokens"], c["experts"], c["top_k"]
        b = E * 4 if c["bias"] else 0
        if c["op"] == "route":
            return {"bytes": T * E * 4 + b + T * k * 8, "flops": T * E * 4}
        # every logit only where the softmax over all of them matters
        reads = E if c["score"] == "softmax" and not c["renorm"] else k
        return {"bytes": T * (reads * 4 + k * 8 + E * 4), "flops": T * reads * 6}
    if c["op"] in ("linear", "linear_grad"):
        M, K, N = c["rows"], c["inner"], c["cols"]
        y = 4 if c["f32"] else 2
        if c["op"] == "linear":
            extra = M * N * 2 * (int(c["residual"]) + int(c["keep"])) + (N * 4 if c["bias"] else 0)
            return {"bytes": (M * K + N * K) * 2 + M * N * y + extra, "flops": 2 * M * N * K}
        extra = (M * N * 2 if c["act"] != "none" else 0) + (N * 4 if c["bias"] else 0)
        return {"bytes": 2 * (M * K + N * K) * 2 + M * N * y + extra, "flops": 4 * M * N * K}
    size = sum(math.prod(shape) * (4 if t == "fp32" else 2) for shape, t in _clip_sizes(c))
    count = sum(math.prod(shape) for shape, _ in _clip_sizes(c))
    return {"bytes": 2 * size + 4, "flops": 3 * count}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    return {"route": _exact_route, "route_grad": _exact_route_grad, "linear": _exact_linear,
            "linear_grad": _exact_linear_grad, "clip": _exact_clip}[c["op"]](s, c)


def _log_probability(logits, score):
    l = logits.double()
    return -torch.logaddexp(torch.zeros_like(l), -l) if score == "sigmoid" else \
        l - torch.logsumexp(l, dim=1, keepdim=True)


def _place(v):
    """How many of a row come before each value: larger ones, and equal ones further left."""
    out = torch.empty(v.shape, dtype=torch.int64, device=v.device)
    n = v.shape[1]
    left = torch.ones((n, n), dtype=torch.bool, device=v.device).tril(-1)  # [e, f]: f < e
    step = max(1, (1 << 27) // (n * n))
    for a in range(0, v.shape[0], step):
        x = v[a:a + step]
        before = (x[:, None, :] > x[:, :, None]) | ((x[:, None, :] == x[:, :, None]) & left)
        out[a:a + step] = before.sum(dim=2)
    return out


def _exact_route(s, c):
    T, E, G, k = c["tokens"], c["experts"], c["groups"], c["top_k"]
    logp = _log_probability(s["logits"], c["score"])
    v = logp.exp()
    if s["bias"] is not None:
        v = v + s["bias"].double()
    if c["top_groups"] < G:
        top = v.view(T * G, E // G)
        r = top.max(dim=1).values
        if c["rank"] == "top2":
            r = r + top.scatter(1, top.argmax(dim=1, keepdim=True), -math.inf).max(dim=1).values
        out = _place(r.view(T, G)) >= c["top_groups"]
        v = torch.where(out[:, :, None], -math.inf, v.view(T, G, E // G)).reshape(T, E)
    place = _place(v)
    rows, experts = torch.nonzero(place < k, as_tuple=True)
    idx = torch.empty((T, k), dtype=torch.int64, device=v.device)
    idx[rows, place[rows, experts]] = experts
    lw = torch.take_along_dim(logp, idx, dim=1)
    w = torch.softmax(lw, dim=1) if c["renorm"] else lw.exp()
    return idx.to(torch.int32), w * c["scale"]


def _exact_route_grad(s, c):
    # the weights as a function of the logits, differentiated by autograd in 64 bits
    l = s["logits"].double().requires_grad_()
    lw = _log_probability(l, c["score"]).gather(1, s["topk_idx"].long())
    w = torch.softmax(lw, dim=1) if c["renorm"] else lw.exp()
    return torch.autograd.grad((w * c["scale"] * s["grad_w"].double()).sum(), l)[0]


def _exact_linear(s, c):
    z = torch.nn.functional.linear(s["x"].double(), s["w"].double())
    if s["bias"] is not None:
        z += s["bias"].double()
    y = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
         "gelu": lambda v: v * torch.special.ndtr(v)}[c["act"]](z)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return (y, z) if c["keep"] else y


def _exact_linear_grad(s, c):
    dz = s["dy"].double()
    if c["act"] != "none":
        z = s["pre"].double().requires_grad_()
        y = {"relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
             "gelu": lambda v: v * torch.special.ndtr(v)}[c["act"]](z)
        dz = torch.autograd.grad(y, z, dz)[0]
    dx = dz.matmul(s["w"].double())
    dw = s["x"].double().t().contiguous().matmul(dz).t()
    return (dx, dw, dz.sum(dim=0)) if c["bias"] else (dx, dw)


def _exact_clip(s, c):
    total = math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"])
    norm = math.sqrt(total)
    coef = min(1.0, c["bound"] / (norm + 1e-6))
    return [torch.tensor([norm], dtype=torch.float64)] + [g.double() * coef for g in s["grads"]]
