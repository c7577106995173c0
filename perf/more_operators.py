"""Performance cases of the trainable and the 4-bit expert layer: the router,
the gated feed-forward block of experts with its backward pass, its 8-bit
activation checkpoints, and products with 4-bit weights.

``run`` computes each operator in plain torch operations (``own`` false) or
through the framework's entry points (``own`` true) on the same state.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # serving: the experts of one token
        _route("route one token", 1, 256, 8),
        # training: a long batch, and the gradient of its logits
        _route("route and gradient", 32768, 256, 8, grad=True),
        # serving: one token's eight rows, each with an expert of its own among 32 local ones
        _ffn("ffn one token", 8, 32, 7168, 2048, even=True),
        # prefill: 512 rows an expert on average, ragged
        _ffn("ffn rows", 16384, 32, 4096, 1024),
        # training: an odd number of sorted rows, gradients of the rows and of all weights
        _ffn("ffn and gradients", 8191, 8, 4096, 2048, grad=True),
        # training: a shared expert (dense) of odd sizes
        _ffn("shared ffn and gradients", 1023, 0, 2064, 1032, grad=True),
        # training: a batch's rows to 8 bits as it is saved, and back as the backward pass reads them
        {"name": "checkpoint rows", "op": "checkpoint", "rows": 16384, "hidden": 7168, "dtype": "bf16"},
        # training with 8-bit checkpoints: the block's forward and backward pass
        _ffn("ffn from checkpoints", 8191, 32, 4096, 1024, grad=True, checkpoint="mxfp8"),
        # serving: one token against a dense 4-bit weight
        _fourbit("4-bit one row", 1, 0, 4096, 4096),
        # serving: one token's gate and up projections, eight of 32 experts, and the activation
        _fourbit("4-bit gated token", 8, 32, 4096, 7168, gated=True, even=True),
        # serving: a step of 16 tokens, 128 rows over 32 experts
        _fourbit("4-bit step", 128, 32, 4096, 7168),
        # training: router, sort by expert, feed-forward and weighted sum, with all gradients
        {"name": "layer and gradients", "op": "layer", "tokens": 2047, "experts": 32, "top_k": 4, "hidden": 2048,
         "inter": 1024, "dtype": "bf16", "checkpoint": "mxfp8", "renormalize": True, "skew": 0.5},
    ]


def _route(name, tokens, experts, top_k, grad=False, dtype="fp32", renormalize=True, masked=False):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "grad": grad,
            "dtype": dtype, "renormalize": renormalize, "masked": masked}


def _ffn(name, rows, experts, hidden, inter, grad=False, checkpoint="bf16", skew=0.0, even=False):
    """experts 0: a dense block without offsets."""
    return {"name": name, "op": "ffn", "rows": rows, "experts": experts, "hidden": hidden, "inter": inter, "grad": grad,
            "checkpoint": checkpoint, "skew": skew, "even": even, "dtype": "bf16"}


def _fourbit(name, rows, experts, n, k, gated=False, out="bf16", skew=0.0, even=False):
    return {"name": name, "op": "fourbit", "rows": rows, "experts": experts, "n": n, "k": k, "gated": gated, "dtype": out,
            "skew": skew, "even": even}


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("route", "ffn", "ffn", "checkpoint", "fourbit", "layer"))
    skew = rng.choice((0.0, 0.5, 1.2))
    if op == "route":
        experts = _between(rng, 4, 512)
        return _route("", _between(rng, 1, (1 << 23) // experts), experts, rng.randint(1, min(16, experts)),
                      grad=rng.random() < 0.5, dtype=rng.choice(("bf16", "fp32")), renormalize=rng.random() < 0.5,
                      masked=rng.random() < 0.3)
    if op == "ffn":
        checkpoint = rng.choice(("bf16", "mxfp8"))
        unit = 32 if checkpoint == "mxfp8" else 8
        hidden, inter = unit * _between(rng, 2, 4096 // unit), unit * _between(rng, 2, 2048 // unit)
        grad = checkpoint == "mxfp8" or rng.random() < 0.5
        experts = rng.choice((0, _between(rng, 1, 64)))
        while experts * hidden * inter > 1 << 28:
            experts = (experts + 1) // 2
        rows = _between(rng, 1, 8191 if grad else 16384)
        return _ffn("", rows, experts, hidden, inter, grad=grad, checkpoint=checkpoint, skew=min(skew, 0.5))
    if op == "checkpoint":
        return {"name": "", "op": op, "rows": _between(rng, 1, 16384), "hidden": 32 * _between(rng, 1, 224),
                "dtype": rng.choice(("bf16", "bf16", "fp32"))}
    if op == "fourbit":
        experts, k = rng.choice((0, _between(rng, 1, 64))), 32 * _between(rng, 1, 224)
        gated = rng.random() < 0.4
        n = 2 * _between(rng, 8, 2048) if gated else _between(rng, 16, 8192)
        while experts * n * k > 1 << 29:
            experts = (experts + 1) // 2
        return _fourbit("", _between(rng, 1, 256), experts, n, k, gated=gated, out=rng.choice(("bf16", "bf16", "fp32")),
                        skew=skew)
    return {"name": "", "op": op, "tokens": _between(rng, 1, 2047), "experts": rng.randint(4, 32),
            "top_k": rng.randint(1, 4), "hidden": 32 * _between(rng, 2, 64), "inter": 32 * _between(rng, 2, 32),
            "dtype": "bf16", "checkpoint": rng.choice(("bf16", "mxfp8")), "renormalize": rng.random() < 0.5,
            "skew": min(skew, 0.5)}


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    st = {"op": op, "dtype": dt, "grad": case.get("grad", False), "checkpoint": case.get("checkpoint")}
    if op in ("route", "layer"):
        T, E = case["tokens"], case["experts"]
        st["top_k"], st["renormalize"] = case["top_k"], case["renormalize"]
        logits = torch.randn((T, E), generator=g, device="cuda") * 2
        if op == "layer":
            logits += _popularity(E, case["skew"]).log()
        if case.get("masked"):
            # experts that take no part in a step
            logits = logits.masked_fill(torch.rand((E,), generator=g, device="cuda") < 0.3, -math.inf)
        st["logits"] = logits.to(dt)
        st["grad_weights"] = torch.randn((T, case["top_k"]), generator=g, device="cuda") if st["grad"] else None
    if op == "layer":
        H, I, E = case["hidden"], case["inter"], case["experts"]
        st["x"], st["grad_y"] = _normal(g, (case["tokens"], H)), _normal(g, (case["tokens"], H))
        st["w1"], st["w2"] = _weight(g, (E, 2 * I, H)), _weight(g, (E, H, I))
    if op == "ffn":
        M, E, H, I = case["rows"], case["experts"], case["hidden"], case["inter"]
        st["offsets"] = _draw_offsets(case, g)
        many = (E,) if E else ()
        st["x"] = _normal(g, (M, H))
        st["w1"], st["w2"] = _weight(g, many + (2 * I, H)), _weight(g, many + (H, I))
        st["grad_y"] = _normal(g, (M, H)) if st["grad"] else None
    if op == "checkpoint":
        # rows of different magnitude, as a network's layers leave them
        size = torch.exp2(4 * torch.randn((case["rows"], 1), generator=g, device="cuda"))
        st["x"] = (torch.randn((case["rows"], case["hidden"]), generator=g, device="cuda") * size).to(dt)
    if op == "fourbit":
        M, E, N, K = case["rows"], case["experts"], case["n"], case["k"]
        st["offsets"], st["gated"] = _draw_offsets(case, g), case["gated"]
        st["x"] = _normal(g, (M, K))
        many = (E,) if E else ()
        codes = torch.empty((max(E, 1), N, K // 2), dtype=torch.uint8, device="cuda")
        steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        for e in range(max(E, 1)):
            v = torch.randn((N, K), generator=g, device="cuda") * 2
            c = (torch.bucketize(v.abs(), steps, out_int32=True) + 8 * (v < 0)).to(torch.uint8)
            codes[e] = c[:, ::2] | c[:, 1::2] << 4
        st["w"] = codes.view(many + (N, K // 2))
        middle = 127 - 1 - round(math.log2(K) / 2)
        exponents = torch.randint(middle - 1, middle + 2, many + (N, K // 32), generator=g, device="cuda")
        st["w_scales"] = exponents.to(torch.uint8).view(torch.float8_e8m0fnu)
    return st


def _normal(g, shape):
    return torch.randn(shape, generator=g, dtype=torch.bfloat16, device="cuda")


def _weight(g, shape):
    """Weights of deviation K^-1/2."""
    return _normal(g, shape) * (1 / math.sqrt(shape[-1]))


def _popularity(E, skew):
    return torch.arange(1, E + 1, dtype=torch.float32, device="cuda").pow(-skew)


def _draw_offsets(case, g):
    """Offsets of sorted rows over the experts; `even`: one row in each of evenly spaced experts."""
    M, E = case["rows"], case["experts"]
    if not E:
        return None
    if case["even"]:
        counts = torch.zeros(E, dtype=torch.int64, device="cuda")
        counts[:: E // M] = 1
    else:
        ids = torch.multinomial(_popularity(E, case["skew"]), M, replacement=True, generator=g)
        counts = torch.bincount(ids, minlength=E)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    from combine_route_mask_amd import experts as X, ffn as F, router as R
    op = st["op"]
    if op == "route":
        r = R.route_top_k(st["logits"], st["top_k"], renormalize=st["renormalize"])
        out = {"ids": r.ids, "weights": r.weights}
        if st["grad"]:
            out["grad"] = R.route_top_k_backward(st["logits"], r.ids, st["grad_weights"], renormalize=st["renormalize"])
        return out
    if op == "ffn":
        if not st["grad"]:
            return F.expert_ffn(st["x"], st["w1"], st["w2"], offsets=st["offsets"])
        y, saved = F.expert_ffn_forward(st["x"], st["w1"], st["w2"], offsets=st["offsets"], checkpoint=st["checkpoint"])
        dx, dw1, dw2 = F.expert_ffn_backward(st["grad_y"], saved, st["w1"], st["w2"], offsets=st["offsets"])
        return {"y": y, "grad_x": dx, "grad_w1": dw1, "grad_w2": dw2}
    if op == "checkpoint":
        c = F.checkpoint_rows(st["x"])
        return {"rows": c.rows, "scales": c.scales, "restored": F.restore_rows(c.rows, c.scales, dtype=st["dtype"])}
    if op == "fourbit":
        return F.expert_matmul_mxfp4(st["x"], st["w"], st["w_scales"], offsets=st["offsets"], gated=st["gated"],
                                     dtype=st["dtype"])
    x, logits, w1, w2 = (st[n].detach().requires_grad_() for n in ("x", "logits", "w1", "w2"))
    r = R.route_top_k(logits, st["top_k"], renormalize=st["renormalize"])
    s = X.expert_sort(r.ids[None], x[None], w1.shape[0])
    y = F.expert_ffn(s.rows, w1, w2, offsets=s.offsets, checkpoint=st["checkpoint"])
    out = X.expert_unsort(s.position, y, r.weights[None])[0]
    grads = torch.autograd.grad(out, (x, logits, w1, w2), st["grad_y"])
    return {"out": out.detach(), **dict(zip(("grad_x", "grad_logits", "grad_w1", "grad_w2"), grads))}


def _plain(st):
    op, dt = st["op"], st["dtype"]
    if op == "route":
        ids, weights, back = _routed(st["logits"].float(), st["top_k"], st["renormalize"])
        out = {"ids": ids.to(torch.int32), "weights": weights}
        if st["grad"]:
            out["grad"] = back(st["grad_weights"]).to(dt)
        return out
    if op == "ffn":
        y, back = _block(st["x"].float(), st["w1"], st["w2"], st["offsets"], st["checkpoint"])
        if not st["grad"]:
            return y.to(dt)
        dx, dw1, dw2 = back(st["grad_y"].float())
        return {"y": y.to(dt), "grad_x": dx.to(dt), "grad_w1": dw1.to(dt), "grad_w2": dw2.to(dt)}
    if op == "checkpoint":
        values, exponents = _mxfp8(st["x"].float())
        codes = (values.view(values.shape[0], -1, 32) * torch.exp2(-exponents)[:, :, None]).to(torch.float8_e4m3fn)
        scales = (exponents + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        return {"rows": codes.view_as(values), "scales": scales, "restored": values.to(dt)}
    if op == "fourbit":
        w = _mxfp4(st["w"], st["w_scales"])
        rows = _Rows(st["x"].shape[0], st["offsets"])
        y = rows.product(st["x"].float(), w if w.dim() == 3 else w[None])
        if st["gated"]:
            gate, up = y.chunk(2, dim=1)
            y = gate / (1 + torch.exp(-gate)) * up
        return y.to(dt)
    # the layer: pairs (token, choice) by expert, a stable order
    T, k, E = st["x"].shape[0], st["top_k"], st["w1"].shape[0]
    ids, weights, back_route = _routed(st["logits"].float(), k, st["renormalize"])
    key, order = torch.sort(ids.view(-1), stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device="cuda")).to(torch.int32)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device="cuda")
    y, back = _block(st["x"].float()[order // k], st["w1"], st["w2"], offsets, st["checkpoint"])
    each = y[place].view(T, k, -1)
    out = (each * weights[:, :, None]).sum(1)
    go = st["grad_y"].float()[:, None]
    grad_logits = back_route((each * go).sum(2))
    dx, dw1, dw2 = back((weights[:, :, None] * go).view(T * k, -1)[order])
    dx = dx[place].view(T, k, -1).sum(1)
    return {"out": out.to(dt), "grad_x": dx.to(dt), "grad_logits": grad_logits.to(dt),
            "grad_w1": dw1.to(dt), "grad_w2": dw2.to(dt)}


def _routed(logits, k, renormalize):
    """(ids, weights, gradient) of the k largest logits, equal ones by ascending index; an expert whose logit is
    -infinity is not chosen: its place holds the id E and the weight 0."""
    E = logits.shape[1]
    chosen, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    chosen, ids = chosen[:, :k], ids[:, :k]
    held = chosen > -math.inf
    top = torch.where(held[:, :1], chosen[:, :1], 0)
    e = torch.exp(chosen - top)
    full = torch.exp(logits - top)
    total = (e if renormalize else full).sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1)
    weights = e / total

    def back(grad):
        mean = (weights * grad).sum(1, keepdim=True)
        if renormalize:
            return torch.zeros_like(logits).scatter_(1, ids, weights * (grad - mean))
        return (-mean * (full / total)).scatter_add_(1, ids, weights * grad)

    return torch.where(held, ids, E), weights, back


def _block(x, w1, w2, offsets, checkpoint):
    """(y, gradient) of the gated block in 32 bits; the gradient is taken at what the checkpoint holds."""
    rows = _Rows(x.shape[0], offsets)
    w1, w2 = w1.float(), w2.float()
    dense = w1.dim() == 2
    if dense:
        w1, w2 = w1[None], w2[None]
    pre = rows.product(x, w1)
    gate, up = pre.chunk(2, dim=1)
    y = rows.product(gate / (1 + torch.exp(-gate)) * up, w2)

    def back(dy):
        xs, ps = (_mxfp8(x)[0], _mxfp8(pre)[0]) if checkpoint == "mxfp8" else (x, pre)
        gate, up = ps.chunk(2, dim=1)
        s = 1 / (1 + torch.exp(-gate))
        da = rows.product(dy, w2.transpose(1, 2))
        dpre = torch.cat([da * up * s * (1 + gate * (1 - s)), da * gate * s], dim=1)
        dw1, dw2 = rows.outer(dpre, xs), rows.outer(dy, gate * s * up)
        return rows.product(dpre, w1.transpose(1, 2)), dw1[0] if dense else dw1, dw2[0] if dense else dw2

    return y, back


class _Rows:
    """Sorted rows, and the same rows padded to the busiest expert's."""

    def __init__(self, M, offsets):
        if offsets is None:
            offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        m = torch.arange(M, device="cuda", dtype=torch.int32)
        self.E = offsets.numel() - 1
        e = torch.searchsorted(offsets[1:], m, right=True)
        self.most = int((offsets[1:] - offsets[:-1]).max())
        self.place = e * self.most + (m - offsets[e])

    def padded(self, x):
        full = torch.zeros((self.E * self.most, x.shape[1]), device="cuda")
        full[self.place] = x
        return full.view(self.E, self.most, -1)

    def product(self, x, w):
        """Each row times its expert's w [E, N, K]."""
        y = torch.bmm(self.padded(x), w.transpose(1, 2).contiguous())
        return y.view(self.E * self.most, -1)[self.place]

    def outer(self, a, b):
        """Sum over an expert's rows of a's row times b's: [E, N, K]."""
        return torch.bmm(self.padded(a).transpose(1, 2).contiguous(), self.padded(b))


def _mxfp8(x):
    """What MXFP8 holds of x, and the exponents: blocks of 32, the smallest power of two that keeps a block within
    448 as its scale."""
    b = x.view(x.shape[0], -1, 32)
    top = b.abs().amax(2)
    fraction, exponent = torch.frexp(top)
    # top = fraction * 2^exponent, 448 = 0.875 * 2^9
    e = torch.where(top > 0, exponent - 9 + (fraction > 0.875), -127).clamp(min=-127).float()
    codes = (b * torch.exp2(-e)[:, :, None]).to(torch.float8_e4m3fn).float()
    return (codes * torch.exp2(e)[:, :, None]).view_as(x), e


def _mxfp4(codes, scales):
    """The values [.., N, K] of two e2m1 codes a byte (the first in the low half) and a scale for 32."""
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    values = torch.cat([values, -values])
    w = torch.stack([values[(codes & 15).int()], values[(codes >> 4).int()]], dim=-1)
    w = w.view(scales.shape + (32,)) * torch.exp2(scales.view(torch.uint8).float() - 127)[..., None]
    return w.flatten(-2)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    item = 4 if case["dtype"] == "fp32" else 2
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        n = T * (item * E + 8 * k)
        return {"bytes": n + (T * (item * E + 4 * k) if case["grad"] else 0), "flops": 4 * T * E}
    if op == "checkpoint":
        n = case["rows"] * case["hidden"]
        return {"bytes": n * (2 * item + 33 / 32), "flops": 3 * n}
    if op == "fourbit":
        M, E, N, K = case["rows"], max(case["experts"], 1), case["n"], case["k"]
        busy = min(M, E) if case["even"] else E * (1 - (1 - 1 / E) ** M)
        return {"bytes": 2 * M * K + busy * N * K * 17 / 32 + item * M * N / (2 if case["gated"] else 1),
                "flops": 2 * M * N * K}
    H, I, E = case["hidden"], case["inter"], max(case["experts"], 1)
    if op == "ffn":
        M = case["rows"]
        busy = min(M, E) if case["even"] else E * (1 - (1 - 1 / E) ** M)
        n, f = 4 * M * H + 6 * busy * H * I, 6 * M * H * I
        if case["grad"]:
            # the gradients' rows in and out, and all weights' gradients
            n, f = n + 4 * M * H + 6 * E * H * I, 3 * f
        return {"bytes": n, "flops": f}
    T, k = case["tokens"], case["top_k"]
    M = T * k
    return {"bytes": 8 * T * H + 4 * T * E + 6 * E * H * I * 2, "flops": 18 * M * H * I}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op == "route":
        weights, grad = _exact_route(st["logits"].to(d), case, st["grad_weights"])[1:]
        return {"ids": None, "weights": weights, **({"grad": grad} if st["grad"] else {})}
    if op == "checkpoint":
        v, scale = _exact_mxfp8(st["x"].to(d))
        return {"rows": (v.view(v.shape[0], -1, 32) / scale[:, :, None]).view_as(v), "scales": scale, "restored": v}
    if op == "fourbit":
        M, N = case["rows"], case["n"]
        w, s = st["w"].view(-1, N, case["k"] // 2), st["w_scales"].view(torch.uint8).view(-1, N, case["k"] // 32)
        bounds = [0, M] if st["offsets"] is None else st["offsets"].tolist()
        y = torch.empty((M, N), dtype=d, device="cuda")
        for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
            if b > a:
                y[a:b] = st["x"][a:b].to(d) @ _exact_mxfp4(w[e], s[e]).t()
        if case["gated"]:
            y = y[:, : N // 2] * torch.sigmoid(y[:, : N // 2]) * y[:, N // 2:]
        return y
    if op == "ffn":
        M = case["rows"]
        bounds = [0, M] if st["offsets"] is None else st["offsets"].tolist()
        y, dx, dw1, dw2 = _exact_block(st["x"], st["w1"], st["w2"], bounds, case["checkpoint"],
                                       None if st["grad_y"] is None else st["grad_y"].to(d))
        return {"y": y, "grad_x": dx, "grad_w1": dw1, "grad_w2": dw2} if st["grad"] else y
    T, k, E, H = case["tokens"], case["top_k"], case["experts"], case["hidden"]
    ids, weights, _ = _exact_route(st["logits"].to(d), case, None)
    pair = torch.argsort(ids.view(-1) * (T * k) + torch.arange(T * k, device="cuda"))
    bounds = [0] + torch.bincount(ids.view(-1), minlength=E).cumsum(0).tolist()
    token = pair // k
    go = st["grad_y"].to(d)[token]
    w = weights.reshape(-1)[pair]
    y, dx, dw1, dw2 = _exact_block(st["x"][token], st["w1"], st["w2"], bounds, case["checkpoint"], go * w[:, None])
    gw = torch.empty(T * k, dtype=d, device="cuda")
    gw[pair] = (y * go).sum(1)
    zero = torch.zeros((T, H), dtype=d, device="cuda")
    return {"out": zero.index_add(0, token, y * w[:, None]), "grad_x": zero.index_add(0, token, dx),
            "grad_logits": _exact_route(st["logits"].to(d), case, gw.view(T, k))[2], "grad_w1": dw1, "grad_w2": dw2}


def _exact_route(logits, case, grad):
    """(ids, weights, gradient of the logits): a chosen expert has fewer than k before it."""
    k = case["top_k"]
    ids, left = [], logits.clone()
    for _ in range(k):
        # argmax of the first largest: compare, then the lowest index
        best = (left == left.amax(1, keepdim=True)).to(torch.int8).argmax(1, keepdim=True)
        ids.append(best)
        left.scatter_(1, best, -math.inf)
    ids = torch.cat(ids, dim=1)
    values = logits.gather(1, ids)
    among = values if case["renormalize"] else logits
    lse = torch.logsumexp(among, dim=1, keepdim=True)
    lse = torch.where(torch.isinf(lse), 0, lse)
    weights = torch.exp(values - lse)
    if grad is None:
        return ids, weights, None
    g = grad.to(torch.float64)
    p = torch.exp(logits - lse)
    chosen = torch.zeros_like(p).scatter_(1, ids, 1.0)
    spread = torch.zeros_like(p).scatter_(1, ids, g)
    mean = (weights * g).sum(1, keepdim=True)
    return ids, weights, p * ((spread - mean) * chosen if case["renormalize"] else spread - mean)


def _exact_block(x, w1, w2, bounds, checkpoint, dy):
    d = torch.float64
    M, H = x.shape
    dense = w1.dim() == 2
    w1, w2 = (w1[None], w2[None]) if dense else (w1, w2)
    I = w2.shape[2]
    y = torch.empty((M, H), dtype=d, device="cuda")
    dx, dw1, dw2 = (None,) * 3 if dy is None else (torch.empty_like(y), torch.zeros(w1.shape, dtype=d, device="cuda"),
                                                   torch.zeros(w2.shape, dtype=d, device="cuda"))
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if b <= a:
            continue
        xe, u, v = x[a:b].to(d), w1[e].to(d), w2[e].to(d)
        h = xe @ u.t()
        y[a:b] = (h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]) @ v.t()
        if dy is None:
            continue
        if checkpoint == "mxfp8":
            xe, h = _exact_mxfp8(xe)[0], _exact_mxfp8(h)[0]
        gate, up = h[:, :I], h[:, I:]
        s = torch.sigmoid(gate)
        da = dy[a:b] @ v
        dh = torch.cat([da * up * (s + gate * s * (1 - s)), da * gate * s], dim=1)
        dw2[e] = dy[a:b].t() @ (gate * s * up)
        dw1[e] = dh.t() @ xe
        dx[a:b] = dh @ u
    if dense and dy is not None:
        dw1, dw2 = dw1[0], dw2[0]
    return y, dx, dw1, dw2


def _exact_mxfp8(x):
    b = x.view(x.shape[0], -1, 32)
    top = b.abs().max(2, keepdim=True).values
    scale = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-127)), 2.0 ** -127)
    # e4m3: a step of 2^-3 of the value's power of two, and of 2^-9 below 2^-6
    v = b / scale
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step * scale).view_as(x), scale[:, :, 0]


def _exact_mxfp4(codes, exponents):
    """e2m1: sign, two bits of exponent, one of fraction; 0.5 below 1."""
    c = torch.stack([codes % 16, codes // 16], dim=2).view(codes.shape[0], -1).to(torch.float64)
    sign, c = 1 - 2 * torch.floor(c / 8), c % 8
    e, m = torch.floor(c / 2), c % 2
    v = sign * torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2)
    return (v.view(codes.shape[0], -1, 32) * torch.exp2(exponents.to(torch.float64) - 127)[:, :, None]).flatten(1)
