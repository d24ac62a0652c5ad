"""Weights of the distillation's step: a masked row's is not used, whatever it is."""
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note
from tests.test_gpu_distill import make
from tests.test_gpu_top import BF, F

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
# by rows (4, 8 and 16 waves) and in pieces
SHAPES = [(9, 1001), (9, 40000), (130, 70003), (9, 70003)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V", SHAPES)
def test_weights_of_masked_rows(dtype, T, V):
    note(f"distill masked weights {dtype} {T} {V}")
    x, ids, logp = make(T, V, 6, dtype, seed=V)
    ids[5] = torch.tensor([V, -1, -7, 2 ** 31 - 1, -2 ** 31, V + 1], device=DEV, dtype=torch.int32)
    ids[7] = -1
    weights = torch.rand(T, device=DEV)
    weights[[2, 5, 7]] = 0.0
    loss, kl, dx = L.lora_distill_step(x, ids, logp, weights)
    assert bool(torch.isfinite(loss)) and not kl[[2, 5, 7]].any() and not dx[[2, 5, 7]].any()
    for bad in ((NAN, INF, -INF), (INF, INF, INF), (3e38, NAN, 1.0)):
        weights[[2, 5, 7]] = torch.tensor(bad, device=DEV)
        again = L.lora_distill_step(x, ids, logp, weights)
        assert all(torch.equal(a, b) for a, b in zip((loss, kl, dx), again)), bad
    weights[3] = NAN  # an unmasked row's counts
    assert bool(torch.isnan(L.lora_distill_step(x, ids, logp, weights)[0]))


def test_weights_of_rows_without_divergence():
    note("distill no divergence")
    # one token: its divergence is exactly 0, and NaN times that is not
    x, ids, logp = torch.zeros(3, 1, device=DEV), torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.zeros(3, 1, device=DEV)
    ids[1] = -1
    for weights, nan in (((1.0, NAN, 2.0), False), ((1.0, 1.0, NAN), True), ((INF, 1.0, 2.0), True)):
        loss, kl, _ = L.lora_distill_step(x, ids, logp, torch.tensor(weights, device=DEV))
        assert not kl.any() and bool(torch.isnan(loss)) == nan, weights
    # no column, no token
    x = torch.empty(3, 0, device=DEV)
    loss, _, _ = L.lora_distill_step(x, ids, logp, torch.tensor([NAN, INF, 1.0], device=DEV))
    assert float(loss) == 0
