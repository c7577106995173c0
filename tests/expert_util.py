"""64-bit references of the expert layer's operators, on the CPU, written
from their definitions, and the bounds that the kernels' roundings allow.

A rounding is off by at most half a step: U32 = 2^-24 and UBF = 2^-8 relative
to the value for fp32 and bf16."""
import numpy as np
import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8


def unit(dtype):
    return UBF if dtype == torch.bfloat16 else 0.0


def sort_reference(ids, epr, capacity):
    """(position, offsets, counts, [(r, q) of each kept row]) of ids [R, S, k]."""
    R, S, k = ids.shape
    E = R * epr
    pairs = [(int(ids[r, q, j]), r, q, j) for r in range(R) for q in range(S) for j in range(k)
             if r * epr <= ids[r, q, j] < (r + 1) * epr]
    pairs.sort()
    position = np.full((R, S, k), -1, np.int32)
    counts = np.zeros(E, np.int32)
    for e, _, _, _ in pairs:
        counts[e] += 1
    offsets = np.minimum(np.concatenate([[0], np.cumsum(counts)]), capacity).astype(np.int32)
    for place, (_, r, q, j) in enumerate(pairs[:capacity]):
        position[r, q, j] = place
    return position, offsets, counts, [(r, q) for _, r, q, _ in pairs[:capacity]]


def draw_ids(rng, R, S, k, epr, local=0.7, odd=True):
    """Ids of which about `local` are on their rank; the rest elsewhere, with
    ids out of every range among them, and slots without any."""
    E = R * epr
    ids = rng.integers(0, E, size=(R, S, k))
    here = rng.random((R, S, k)) < local
    ids = np.where(here, np.arange(R)[:, None, None] * epr + rng.integers(0, epr, size=(R, S, k)), ids)
    if odd and S:
        bad = rng.random((R, S, k)) < 0.05
        ids[bad] = rng.choice([-1, E, E + 7, 2 ** 31 - 1, -2 ** 31], size=int(bad.sum()))
        ids[rng.random((R, S)) < 0.1] = E
    return ids.astype(np.int32)


def unsort_reference(position, rows, weights):
    """(sum, sum of magnitudes) over j of weights * rows[position], float64."""
    p = torch.as_tensor(position).long()
    R, S, k = p.shape
    x = rows.double().cpu()
    here = (p >= 0) & (p < x.shape[0])
    out = torch.zeros(R, S, x.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for j in range(k):
        h = here[:, :, j]
        t = x[p[:, :, j][h]]
        if weights is not None:
            t = t * weights[:, :, j].double().cpu()[h][:, None]
        out[h] += t
        mag[h] += t.abs()
    return out, mag


def check_close(got, ref, bound, what):
    got = got.double().cpu()
    err = (got - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err - bound)[bad].max()):.3g} "
        f"beyond its bound; first at {bad.nonzero()[0].tolist()}")


def check_int8(codes, scales, ref, rel, what):
    """codes * scale against rows `ref` [M, N] known to `rel` relative: the
    scale is amax / 127 (one division), a code within half a step of
    value / scale, taken through two more fp32 roundings (2^-15 at 127)."""
    top = ref.abs().amax(1)
    s = scales.double().cpu()
    assert bool(((s - top / 127).abs() <= (rel + 2 * U32) * top / 127 + 2.0 ** -149).all()), f"{what}: scales"
    q = codes.cpu().double()
    assert int(q.abs().max() if q.numel() else 0) <= 127, what
    bound = s[:, None] * (0.5 + 2.0 ** -15) + rel * ref.abs() + 2.0 ** -149
    check_close(q * s[:, None], ref, bound, what)


def bits(t):
    t = t.detach().contiguous().cpu()
    return t.view(torch.uint8).numpy()
