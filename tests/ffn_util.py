"""64-bit references of the trainable expert layer, written from the
definitions, and the bounds that the kernels' roundings allow.

fp32 sums on the matrix cores: each of n additions is off by at most one step,
2^-23 of the magnitudes' sum, in any order.  A rounding to bf16 is off by at
most 2^-8 of the value, to e4m3 by 2^-4 of it or half of 2^-9 of the scale."""
import numpy as np
import torch

U32, UBF = 2.0 ** -24, 2.0 ** -8


def ragged(rng, M, E, kind):
    """Offsets [E + 1] of M rows over E experts; some kinds leave rows behind the last expert's."""
    if kind == "even":
        counts = np.full(E, M // E)
    elif kind == "one":
        counts = np.zeros(E, int)
        counts[E // 2] = M
    elif kind == "single rows":
        counts = (np.arange(E) < M).astype(int)
    elif kind == "none":
        counts = np.zeros(E, int)
    else:
        counts = np.bincount(rng.integers(0, max(1, E - 1), size=max(0, M - 2)), minlength=E)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def bf16(rng, *shape, size=1.0):
    return (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * size).bfloat16()


def by_expert(offsets, M):
    """[(expert, first, last)] of the experts that have rows."""
    if offsets is None:
        return [(0, 0, M)] if M else []
    return [(e, int(a), int(b)) for e, (a, b) in enumerate(zip(offsets, offsets[1:])) if b > a]


def product(x, w, offsets, transposed=False):
    """(sum, bound of the fp32 sum's error, rows that have an expert) in float64."""
    x, w = x.double(), w.double()
    w = w if w.dim() == 3 else w[None]
    if not transposed:
        w = w.transpose(1, 2)
    M, K = x.shape
    y, mag = torch.zeros(M, w.shape[2], dtype=torch.float64), torch.zeros(M, w.shape[2], dtype=torch.float64)
    held = torch.zeros(M, dtype=torch.bool)
    for e, a, b in by_expert(offsets, M):
        y[a:b], mag[a:b] = x[a:b] @ w[e], x[a:b].abs() @ w[e].abs()
        held[a:b] = True
    return y, K * 2 * U32 * mag, held


def outer(a, b, offsets, E):
    """(sum, bound) of the weights' gradient [E, N, K] in float64."""
    a, b = a.double(), b.double()
    y = torch.zeros(E, a.shape[1], b.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(y)
    rows = torch.zeros(E, 1, 1, dtype=torch.float64)
    for e, lo, hi in by_expert(offsets, a.shape[0]):
        y[e], mag[e] = a[lo:hi].t() @ b[lo:hi], a[lo:hi].abs().t() @ b[lo:hi].abs()
        rows[e] = hi - lo
    return y, rows * 2 * U32 * mag


def silu(g):
    return g * torch.sigmoid(g)


def gated(pre, off):
    """(silu(gate) * up, bound) of products `pre` [M, 2 I] known to `off`: the slope of silu is at most 1.1, the
    formula's own error (2 |g| + 10) 2^-24."""
    I = pre.shape[1] // 2
    g, u, og, ou = pre[:, :I], pre[:, I:], off[:, :I], off[:, I:]
    y = silu(g) * u
    spread = 1.1 * og * (u.abs() + ou) + silu(g).abs() * ou
    return y, spread + (2 * g.abs() + 12) * U32 * (y.abs() + spread)


def gated_backward(d, off, pre):
    """(grad_pre, its bound, activation, its bound) for d = grad_out w known to `off` and exact `pre`."""
    I = pre.shape[1] // 2
    g, u = pre[:, :I], pre[:, I:]
    s = torch.sigmoid(g)
    y = g * s * u
    slope = s * (1 + g * (1 - s))
    # s is off by (|g| + 8) 2^-24 relative, 1 - s by as much of 1, g (1 - s) by |g| times that
    es = (g.abs() + 8) * U32
    du, dg = d * g * s, d * u * slope
    odu = off * (g * s).abs() + (es + 4 * U32) * du.abs()
    odg = off * (u * slope).abs() + d.abs() * u.abs() * (s * (g.abs() + 1) * (2 * es + 8 * U32) + 4 * U32)
    return torch.cat([dg, du], 1), torch.cat([odg, odu], 1) * 1.01, y, (es + 4 * U32) * y.abs()


def rounded(bound, ref, dtype=torch.bfloat16):
    """The bound of a value rounded to `dtype` behind an error `bound`."""
    u = UBF if dtype == torch.bfloat16 else U32
    return bound * (1 + u) + u * ref.abs() + 2.0 ** -133


def close(got, ref, bound, what):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {bad.nonzero()[0].tolist()}: "
        f"got {float(got[bad][0])}, want {float(ref[bad][0])} within {float(bound[bad][0]):.3g}")


def mx_scale(top):
    """The smallest power of two that keeps `top` within 448, as an exponent."""
    out = torch.full(top.shape, -127.0, dtype=torch.float64)
    some = top > 0
    out[some] = torch.ceil(torch.log2(top[some] / 448)).clamp(min=-127)
    return out


def mx_round(x, exponent):
    """x as e4m3 codes times 2^exponent of its block of 32."""
    b = x.double().view(x.shape[0], -1, 32)
    scale = torch.exp2(exponent)[:, :, None]
    v = b / scale
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step * scale).view(x.shape)


def half_values(rows, scales):
    """What fp16 rows with a scale for eight hold, in float64."""
    s = torch.exp2(scales.cpu().view(torch.uint8).double() - 127)
    return (rows.cpu().double().view(rows.shape[0], -1, 8) * s[:, :, None]).view(rows.shape)


def half_step(pre, off):
    """How far fp16 with a scale for eight may be from `pre` known to `off`: 2^-11 of the value, or half of fp16's
    least step, 2^-24, of a scale that the largest of the eight is below twice of."""
    top = (pre.abs() + off).view(pre.shape[0], -1, 8).amax(2, keepdim=True).expand(-1, -1, 8).reshape(pre.shape)
    return off + 2.0 ** -11 * (pre.abs() + off) + 2.0 ** -24 * top + 2.0 ** -149


def mx_values(rows, scales):
    """What MXFP8 codes and scales hold, in float64."""
    s = torch.exp2(scales.cpu().view(torch.uint8).double() - 127)
    return (rows.cpu().float().double().view(rows.shape[0], -1, 32) * s[:, :, None]).view(rows.shape)


E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def mxfp4_values(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    s = torch.exp2(scales.view(torch.uint8).double() - 127)
    return (E2M1[c].view(*s.shape, 32) * s[..., None]).flatten(-2)
