"""The plain form that the router's kernels are measured against, at rows whose
mask leaves fewer experts than places: ids, weights and gradient in 64 bits
against the definition, written row by row."""
import numpy as np
import pytest
import torch

from perf import more_operators as P
from tests.test_gpu_router import reference


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k,left", [(7, 6, 5, 4), (7, 6, 6, 1), (5, 16, 16, 9), (4, 4, 3, 0), (9, 40, 8, 40)])
def test_rows_with_fewer_experts_than_places(T, E, k, left, renormalize):
    rng = np.random.default_rng(E + left)
    x = torch.from_numpy(rng.standard_normal((T, E)) * 2)
    for t in range(T):
        x[t, torch.from_numpy(rng.permutation(E)[left:])] = -np.inf
    g = torch.from_numpy(rng.standard_normal((T, k)))
    ids, w, p = reference(x, k, renormalize, 1.0)
    got_ids, got_w, back = P._routed(x, k, renormalize)
    assert np.array_equal(got_ids.numpy(), ids)
    # 64-bit sums of at most 40 terms of size 1
    assert np.abs(got_w.numpy() - w).max() < 1e-14
    spread = np.zeros((T, E + 1))
    np.put_along_axis(spread, ids, g.numpy(), 1)
    mean = (w * g.numpy()).sum(1, keepdims=True)
    assert np.abs(back(g).numpy() - p * (spread[:, :E] - mean)).max() < 1e-13
