"""Performance cases of the operators around the exchange: tokens sorted by
expert and back (with weights and gradients), the 8-bit integer product over
experts, the gated activation with an int8 output, and the norm that makes
the next layer's 8-bit payload.

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
        # one token of a single-rank model: the latency of routing its row to its experts
        _sort("sort one token", 1, 1, 256, 8, 7168),
        # the receive regions of an 8-rank exchange of 64..128 tokens a rank, to expert order
        _sort("sort 8 ranks", 8, 128, 256, 8, 7168),
        # training: a long odd batch on one rank, and the gradient of its rows
        _sort("sort and gradient", 1, 8191, 128, 4, 4096, grad=True),
        # serving: a decode step of an 8-rank exchange, expert rows back to its slots
        _unsort("unsort step", 8, 16, 256, 8, 7168),
        # training: weighted rows back to an odd batch, gradients of rows and of weights
        _unsort("unsort and gradients", 1, 4095, 256, 8, 7168, grad=True),
        # serving: 8 tokens' 64 rows meet the gate and up weights of 32 local experts
        _product("product step", 64, 32, 4096, 7168),
        # prefill: 512 rows an expert on average, ragged
        _product("product rows", 16384, 32, 4096, 4096),
        # a dense 8-bit layer of odd sizes fed by the norm's int8 output
        {"name": "norm and dense product", "op": "dense", "rows": 1023, "n": 2055, "hidden": 2064, "dtype": "bf16"},
        # serving: one token's MXFP8 payload
        _norm("norm one token", 1, 7168, "mxfp8"),
        # the payload of a 64-rank exchange of 512 tokens a rank, DeepSeekFp8
        _norm("norm 64 ranks", 32768, 7168, "deepseek_fp8"),
        # serving: the whole expert layer of one rank for a step of 16 tokens
        _experts("experts step", 1, 16, 32, 8, 7168, 2048),
        # prefill: the whole expert layer of 8 ranks from their receive regions
        _experts("experts 8 ranks", 8, 256, 32, 4, 4096, 1024),
    ]


def _sort(name, ranks, tokens, experts, top_k, hidden, grad=False, dtype="bf16"):
    return {"name": name, "op": "sort", "ranks": ranks, "tokens": tokens, "experts": experts, "top_k": top_k,
            "hidden": hidden, "grad": grad, "dtype": dtype, "skew": 0.0}


def _unsort(name, ranks, tokens, experts, top_k, hidden, grad=False, dtype="bf16"):
    return dict(_sort(name, ranks, tokens, experts, top_k, hidden, grad, dtype), op="unsort")


def _product(name, rows, experts, n, k, out="bf16"):
    return {"name": name, "op": "product", "rows": rows, "experts": experts, "n": n, "k": k, "dtype": out, "skew": 0.0}


def _norm(name, rows, hidden, fmt, dtype="bf16"):
    return {"name": name, "op": "norm", "rows": rows, "hidden": hidden, "format": fmt, "dtype": dtype}


def _experts(name, ranks, tokens, experts, top_k, hidden, inter):
    return dict(_sort(name, ranks, tokens, experts, top_k, hidden), op="experts", inter=inter)


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("sort", "unsort", "product", "dense", "norm", "experts"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    skew = rng.choice((0.0, 0.5, 1.2))
    if op in ("sort", "unsort"):
        ranks = rng.choice((1, 1, 2, 4, 8, 16))
        epr = _between(rng, 1 if ranks >= 4 else 4, 256 // ranks)
        experts = ranks * epr if (ranks * epr) % 4 == 0 else ranks * ((epr + 3) // 4 * 4)
        k = min(experts, rng.randint(1, 8))
        hidden = 8 * _between(rng, 16, 896)
        # rows of all regions within 2^27 elements, so that plain gradients fit too
        most = max(1, min(8191, (1 << 27) // (hidden * ranks * max(ranks, k))))
        return dict(_sort("", ranks, _between(rng, 1, most), experts, k, hidden, grad=rng.random() < 0.5, dtype=dtype),
                    op=op, skew=skew)
    if op == "product":
        experts, n, k = _between(rng, 1, 64), _between(rng, 16, 4096), 16 * _between(rng, 4, 448)
        while experts * n * k > 1 << 30:
            experts = (experts + 1) // 2
        rows = _between(rng, 1, max(1, min(16384, (1 << 38) // (n * k))))
        return dict(_product("", rows, experts, n, k, dtype), skew=min(skew, 0.5))
    if op == "dense":
        return {"name": "", "op": op, "rows": _between(rng, 1, 4096), "n": _between(rng, 16, 4096),
                "hidden": 16 * _between(rng, 4, 448), "dtype": dtype}
    if op == "norm":
        fmt = rng.choice(("mxfp8", "deepseek_fp8"))
        return _norm("", _between(rng, 1, 32768), 128 * _between(rng, 1, 56), fmt, dtype)
    ranks = rng.choice((1, 2, 4, 8))
    experts = 4 * ranks * rng.randint(1, 8 // ranks)
    return dict(_experts("", ranks, _between(rng, 1, 512 // ranks), experts, rng.randint(1, 4), 128 * rng.randint(1, 32),
                         32 * rng.randint(1, 32)), skew=min(skew, 0.5))


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    st = {"op": op, "dtype": dt, "grad": case.get("grad", False)}
    if op in ("sort", "unsort", "experts"):
        _draw_routing(st, case, g)
        R, S, H, cap = st["ids"].shape[0], st["ids"].shape[1], case["hidden"], st["capacity"]
        if op != "unsort":
            st["rows"] = _normal(g, (R, S, H), dt)
        if op == "experts":
            E, I = case["experts"], case["inter"]
            st["w1"], st["s1"] = _weight(g, E, 2 * I, H)
            st["w2"], st["s2"] = _weight(g, E, H, I)
            st["most"] = int(_route(st["ids"], st["epr"], cap)[2].max())
        if op == "sort":
            st["sorted"] = torch.zeros((cap, H), dtype=dt, device="cuda")
            st["grad_sorted"] = _normal(g, (cap, H), dt) if st["grad"] else None
        if op == "unsort":
            st["position"], st["offsets"] = _route(st["ids"], st["epr"], cap)[:2]
            st["sorted"] = _normal(g, (cap, H), dt)
            if st["grad"]:
                st["grad_out"] = _normal(g, (R, S, H), dt)
                st["grad_sorted"] = torch.zeros((cap, H), dtype=dt, device="cuda")
        if op != "sort":
            # only slots that hold a token are written; the others stay zero
            st["out"] = torch.zeros((R, S, H), dtype=dt, device="cuda")
    elif op == "product":
        M, E, N, K = case["rows"], case["experts"], case["n"], case["k"]
        ids = torch.multinomial(_popularity(E, case["skew"]), M, replacement=True, generator=g)
        counts = torch.bincount(ids, minlength=E)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["most"] = int(counts.max())
        st["x"] = _codes(g, (M, K))
        st["sx"] = _scale(g, (M,), 1 / 32)
        st["w"], st["sw"] = _weight(g, E, N, K)
    else:
        M, H = case["rows"], case["hidden"]
        st["x"] = _normal(g, (M, H), dt)
        st["residual"] = (_normal(g, (M, H), torch.float32) * 4).to(dt)
        st["weight"] = (1 + 0.1 * _normal(g, (H,), torch.float32)).to(dt)
        st["eps"] = 1e-6
        if op == "dense":
            w, s = _weight(g, 1, case["n"], H)
            st["w"], st["sw"] = w[0], s[0]
        else:
            st["format"] = case["format"]
    return st


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, dtype=dtype, device="cuda")


def _scale(g, shape, mean):
    return (0.5 + torch.rand(shape, generator=g, device="cuda")) * mean


def _codes(g, shape):
    return (_normal(g, shape, torch.bfloat16) * 32).round_().clamp_(-127, 127).to(torch.int8)


def _weight(g, E, N, K):
    """Codes [E, N, K] and channel scales [E, N] of weights with deviation about K^-1/2."""
    return _codes(g, (E, N, K)), _scale(g, (E, N), 1 / (32 * math.sqrt(K)))


def _popularity(E, skew):
    return torch.arange(1, E + 1, dtype=torch.float32, device="cuda").pow(-skew)


def _draw_routing(st, case, g):
    """Top-k ids and softmax weights; for several ranks as a dispatch leaves them in the receive regions:
    slot src * T + t of a rank holds the token's ids if one of its experts lives there, else the id E."""
    R, T, E, k = case["ranks"], case["tokens"], case["experts"], case["top_k"]
    gumbel = -torch.log(-torch.log(torch.rand((R * T, E), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)))
    ids = (gumbel + _popularity(E, case["skew"]).log()).topk(k, dim=1).indices.to(torch.int32)
    weights = torch.softmax(_normal(g, (R * T, k), torch.float32), dim=1)
    epr = E // R
    if R > 1:
        # a source rank has between half and all of its T tokens
        n = torch.randint((T + 1) // 2, T + 1, (R, 1), generator=g, device="cuda")
        ids = torch.where((torch.arange(T, device="cuda") < n).view(R * T, 1), ids, E)
    rank = torch.arange(R, device="cuda").view(R, 1, 1)
    here = ((ids // epr)[None] == rank).any(dim=2, keepdim=True)
    st["ids"] = torch.where(here, ids[None], E).to(torch.int32).contiguous()
    st["weights"] = weights[None].expand(R, R * T, k).contiguous()
    st["epr"], st["capacity"] = epr, R * T * k


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    from combine_route_mask_amd import experts as X
    op = st["op"]
    if op == "sort":
        s = X.expert_sort(st["ids"], st["rows"], st["epr"], capacity=st["capacity"], out=st["sorted"])
        out = {"rows": s.rows, "position": s.position, "offsets": s.offsets}
        if st["grad"]:
            out["grad"] = X.expert_sort_backward(s.position, st["grad_sorted"])
        return out
    if op == "unsort":
        out = {"out": X.expert_unsort(st["position"], st["sorted"], st["weights"], out=st["out"], keep_empty=True)}
        if st["grad"]:
            out["grad_rows"], out["grad_weights"] = X.expert_unsort_backward(
                st["position"], st["grad_out"], st["sorted"], st["weights"], grad_rows=st["grad_sorted"])
        return out
    if op == "product":
        return X.expert_matmul(st["x"], st["sx"], st["w"], st["sw"], offsets=st["offsets"], dtype=st["dtype"])
    if op == "norm":
        n = X.add_rms_norm(st["x"], st["residual"], st["weight"], st["eps"], format=st["format"])
        return {"rows": n.rows, "scales": n.scales, "residual": n.residual}
    if op == "dense":
        n = X.add_rms_norm(st["x"], st["residual"], st["weight"], st["eps"], format="int8")
        return {"y": X.expert_matmul(n.rows, n.scales, st["w"], st["sw"]), "residual": n.residual}
    s = X.expert_sort(st["ids"], st["rows"], st["epr"], capacity=st["capacity"], quantize=True)
    h = X.expert_matmul(s.rows, s.scales, st["w1"], st["s1"], offsets=s.offsets)
    a = X.silu_mul_quantize(h, offsets=s.offsets)
    y = X.expert_matmul(a.rows, a.scales, st["w2"], st["s2"], offsets=s.offsets)
    return X.expert_unsort(s.position, y, st["weights"], out=st["out"], keep_empty=True)


def _plain(st):
    op, dt = st["op"], st["dtype"]
    if op == "sort":
        position, offsets, _, order = _route(st["ids"], st["epr"], st["capacity"])
        R, S, k = position.shape
        H = st["rows"].shape[2]
        held = torch.arange(st["capacity"], device="cuda") < offsets[-1]
        rows = torch.where(held[:, None], st["rows"].view(R * S, H)[order // k], 0)
        out = {"rows": rows, "position": position, "offsets": offsets}
        if st["grad"]:
            out["grad"] = _back(position, st["grad_sorted"].float(), None).to(dt)
        return out
    if op == "unsort":
        x, w, position = st["sorted"].float(), st["weights"], st["position"]
        out = {"out": _back(position, x, w).to(dt)}
        if st["grad"]:
            R, S, k = position.shape
            at, here = position.clamp(min=0).view(-1).long(), (position >= 0).view(-1)
            go = st["grad_out"].float().view(R * S, 1, -1)
            dots = (x[at].view(R * S, k, -1) * go).sum(2).view(-1)
            out["grad_weights"] = torch.where(here, dots, 0).view(R, S, k)
            g = (w.view(R * S, k, 1) * go).to(dt).view(R * S * k, -1)
            # pairs without a row write to a row behind the last, which is left out
            full = torch.zeros((x.shape[0] + 1, x.shape[1]), dtype=dt, device="cuda")
            full[torch.where(here, at, x.shape[0])] = g
            out["grad_rows"] = full[:-1]
        return out
    if op == "product":
        return _product_plain(st["x"], st["sx"], st["w"], st["sw"], st["offsets"], st["most"], dt)
    if op == "norm":
        y, residual = _normed(st)
        codes, scales = _blocks(y, st["format"])
        return {"rows": codes, "scales": scales, "residual": residual}
    if op == "dense":
        y, residual = _normed(st)
        q, s = _int8(y)
        acc = q @ st["w"].float().t()
        return {"y": (acc * s[:, None] * st["sw"]).to(torch.bfloat16), "residual": residual}
    position, offsets, _, order = _route(st["ids"], st["epr"], st["capacity"])
    R, S, k = position.shape
    q, s = _int8(st["rows"].view(R * S, -1)[order // k].float())
    h = _product_plain(q, s, st["w1"], st["s1"], offsets, st["most"], dt).float()
    gate, up = h.chunk(2, dim=1)
    q, s = _int8(gate / (1 + torch.exp(-gate)) * up)
    y = _product_plain(q, s, st["w2"], st["s2"], offsets, st["most"], dt)
    return _back(position, y.float(), st["weights"]).to(dt)


def _route(ids, epr, capacity):
    """(position [R, S, k], offsets [E + 1], counts [E], the pair of each sorted row): a pair is (slot, j), in
    expert order if its expert lives on the slot's rank."""
    R, S, k = ids.shape
    E = R * epr
    first = torch.arange(R, device="cuda", dtype=torch.int32).view(R, 1, 1) * epr
    key = torch.where((ids >= first) & (ids < first + epr), ids, E).view(-1)
    key_sorted, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key_sorted, torch.arange(E + 1, device="cuda", dtype=torch.int32)).to(torch.int32)
    place = torch.empty_like(key)
    place[order] = torch.arange(R * S * k, device="cuda", dtype=torch.int32)
    place = torch.where((key < E) & (place < capacity), place, -1)
    return place.view(R, S, k), offsets, offsets[1:] - offsets[:-1], order[:capacity]


def _back(position, x, w):
    """Sum over j of w * x[position], in 32 bits; no row adds nothing."""
    R, S, k = position.shape
    here = (position >= 0).view(R * S, k, 1)
    t = torch.where(here, x[position.clamp(min=0).view(-1).long()].view(R * S, k, -1), 0)
    if w is not None:
        t = t * w.view(R * S, k, 1)
    return t.sum(1).view(R, S, -1)


def _product_plain(x, sx, w, sw, offsets, most, dt):
    """Rows of each expert padded to the busiest one's, one batched product in 32 bits."""
    E, N, K = w.shape
    m = torch.arange(x.shape[0], device="cuda", dtype=torch.int32)
    e = torch.searchsorted(offsets[1:], m, right=True)
    held = e < E
    e = e.clamp(max=E - 1)
    place = torch.where(held, m - offsets[e], 0)
    # rows behind the last expert's go to a row of their own, which is left out
    padded = torch.zeros((E * most + 1, K), device="cuda")
    padded[torch.where(held, e * most + place, E * most)] = x.float()
    acc = torch.bmm(w.float(), padded[:-1].view(E, most, K).transpose(1, 2).contiguous())
    y = acc[e, :, place] * sx[:, None] * sw[e]
    return torch.where(held[:, None], y, 0).to(dt)


def _int8(x):
    """Codes (as 32-bit values) and scales of rows: scale = largest magnitude / 127."""
    s = x.abs().amax(1) / 127
    return torch.where(s[:, None] > 0, torch.round(x / s[:, None]), 0), s


def _normed(st):
    s = st["x"].float() + st["residual"].float()
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + st["eps"])
    return s * r * st["weight"].float(), s.to(st["dtype"])


def _blocks(y, fmt):
    """e4m3 codes and block scales: mxfp8 the smallest power of two that keeps a block of 32 within 448,
    deepseek_fp8 the largest magnitude of a block of 128 over 448."""
    M, H = y.shape
    n = 32 if fmt == "mxfp8" else 128
    b = y.view(M, H // n, n)
    top = b.abs().amax(2)
    if fmt == "mxfp8":
        fraction, exponent = torch.frexp(top)
        # top = fraction * 2^exponent, 448 = 0.875 * 2^9
        e = torch.where(top > 0, exponent - 9 + (fraction > 0.875), -127).clamp(min=-127)
        scale = torch.exp2(e.float())
        held = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        held = scale = top / 448
    codes = torch.where(scale[:, :, None] > 0, b / scale[:, :, None], 0).to(torch.float8_e4m3fn)
    return codes.view(M, H), held


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    item = 4 if case["dtype"] == "fp32" else 2
    if op in ("sort", "unsort", "experts"):
        R, T, E, k, H = case["ranks"], case["tokens"], case["experts"], case["top_k"], case["hidden"]
        tokens = R * T * (0.75 if R > 1 else 1.0)
        # a token reaches a rank unless all its experts live elsewhere
        away = math.prod((E - E // R - i) / (E - i) for i in range(k)) if R > 1 else 0.0
        slots, rows = tokens * R * (1 - away), tokens * k
        pairs = R * R * T * k
        if op == "sort":
            n, f = 8 * pairs + item * H * (slots + rows), 0
            if case["grad"]:
                n, f = n + item * H * (slots + rows), H * rows
            return {"bytes": n, "flops": f}
        if op == "unsort":
            n, f = 8 * pairs + item * H * (slots + rows), 2 * H * rows
            if case["grad"]:
                n, f = n + 4 * pairs + item * H * (slots + rows), f + 3 * H * rows
            return {"bytes": n, "flops": f}
        I = case["inter"]
        busy = E * (1 - (1 - 1 / E) ** rows)
        return {"bytes": 12 * pairs + 2 * item * H * slots + busy * (3 * H * I + 4 * (2 * I + H)),
                "flops": 6 * rows * H * I}
    if op == "product":
        M, E, N, K = case["rows"], case["experts"], case["n"], case["k"]
        busy = E * (1 - (1 - 1 / E) ** M)
        return {"bytes": M * (K + 4) + busy * N * (K + 4) + item * M * N, "flops": 2 * M * N * K}
    M, H = case["rows"], case["hidden"]
    if op == "norm":
        # both formats hold H / 32 bytes of scales a row
        return {"bytes": M * (3 * item * H + H + H / 32) + item * H, "flops": 6 * M * H}
    N = case["n"]
    return {"bytes": M * 3 * item * H + item * H + N * (H + 4) + 2 * M * N, "flops": 2 * M * N * H}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op in ("sort", "unsort", "experts"):
        ids, epr, cap = st["ids"].cpu(), st["epr"], st["capacity"]
        R, S, k = ids.shape
        # pairs (expert, slot of all ranks, j) of the experts that live on the slot's rank
        home = torch.div(ids, epr, rounding_mode="floor") == torch.arange(R).view(R, 1, 1)
        pair = home.view(-1).nonzero()[:, 0]
        pair = pair[torch.argsort(ids.view(-1)[pair].long() * (R * S * k) + pair)]
        slot, total = (pair // k).cuda(), pair.numel()
        wide = case["hidden"]
        if op == "sort":
            rows = torch.zeros((cap, wide), dtype=d, device="cuda")
            rows[:total] = st["rows"].view(R * S, wide)[slot].to(d)
            out = {"rows": rows, "position": None, "offsets": None}
            if st["grad"]:
                out["grad"] = torch.zeros((R * S, wide), dtype=d, device="cuda").index_add_(
                    0, slot, st["grad_sorted"][:total].to(d)).view(R, S, wide)
            return out
        w = st["weights"].view(-1)[pair.cuda()].to(d)
        if op == "unsort":
            x = st["sorted"][:total].to(d)
            zero = torch.zeros((R * S, wide), dtype=d, device="cuda")
            out = {"out": zero.index_add(0, slot, x * w[:, None]).view(R, S, wide)}
            if st["grad"]:
                go = st["grad_out"].view(R * S, wide)[slot].to(d)
                gw = torch.zeros(R * S * k, dtype=d, device="cuda")
                gw[pair.cuda()] = (x * go).sum(1)
                out["grad_weights"] = gw.view(R, S, k)
                out["grad_rows"] = torch.zeros((cap, wide), dtype=d, device="cuda")
                out["grad_rows"][:total] = go * w[:, None]
            return out
        expert = ids.view(-1)[pair]
        y = torch.empty((total, wide), dtype=d, device="cuda")
        x = st["rows"].view(R * S, wide)[slot].to(d)
        for e in range(case["experts"]):
            at = (expert == e).nonzero()[:, 0].cuda()
            if at.numel():
                h = _exact_linear(*_exact_int8(x[at]), st["w1"][e], st["s1"][e]).to(torch.bfloat16).to(d)
                a = h[:, : case["inter"]] * torch.sigmoid(h[:, : case["inter"]]) * h[:, case["inter"]:]
                y[at] = _exact_linear(*_exact_int8(a), st["w2"][e], st["s2"][e]).to(torch.bfloat16).to(d)
        zero = torch.zeros((R * S, wide), dtype=d, device="cuda")
        return zero.index_add_(0, slot, y * w[:, None]).view(R, S, wide)
    if op == "product":
        bounds = st["offsets"].tolist()
        y = torch.empty((case["rows"], case["n"]), dtype=d, device="cuda")
        for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
            if b > a:
                y[a:b] = _exact_linear(st["x"][a:b].to(d), st["sx"][a:b].to(d)[:, None], st["w"][e], st["sw"][e])
        return y
    s = st["x"].to(d) + st["residual"].to(d)
    y = s * torch.rsqrt(s.pow(2).mean(1, keepdim=True) + st["eps"]) * st["weight"].to(d)
    if op == "dense":
        return {"y": _exact_linear(*_exact_int8(y), st["w"], st["sw"]), "residual": s}
    size = 32 if case["format"] == "mxfp8" else 128
    blocks = y.view(y.shape[0], -1, size)
    top = blocks.abs().max(2, keepdim=True).values
    if case["format"] == "mxfp8":
        scale = torch.exp2(torch.ceil(torch.log2(top / 448)))
    else:
        scale = top / 448
    # e4m3: a step of 2^-3 of the value's power of two, and of 2^-9 below 2^-6
    v = blocks / scale
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return {"rows": (torch.round(v / step) * step).view_as(y), "scales": scale[:, :, 0], "residual": s}


def _exact_int8(x):
    s = x.abs().max(1, keepdim=True).values / 127
    return torch.round(x / s.clamp(min=1e-300)), s


def _exact_linear(q, s, w, sw):
    return (q @ w.to(torch.float64).t()) * s * sw.to(torch.float64)
