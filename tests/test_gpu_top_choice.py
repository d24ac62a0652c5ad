"""Alternatives on both sides of the limits of the rows that 16 waves take whole."""
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note
from tests.test_gpu_top import BF, F, check, make, ranked

pytestmark = pytest.mark.gpu

SIZES = [(16, 49153, 0), (17, 49153, 0), (16, 65536, 128), (17, 65536, 128), (3, 65537, 8), (3, 65537, 9), (16, 131072, 8),
         (17, 131072, 8), (16, 131073, 8), (2, 49152, 128)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V,k", SIZES)
def test_both_sides(dtype, T, V, k):
    note(f"top choice {dtype} {T} {V} {k}")
    x, y = make(T, V, dtype, T + V + k)
    out = L.lora_token_top(x, y, k, 0.9)
    live = ((y >= 0) & (y < V))[:, None]
    assert torch.equal(out[2], torch.where(live, ranked(x, k), -1))
    at = torch.tensor(sorted({0, 1, T - 1}), device=DEV)
    check(x[at], y[at], k, 0.9, tuple(t[at] for t in out))
    assert all(torch.equal(a, b) for a, b in zip(out, L.lora_token_top(x, y, k, 0.9)))
