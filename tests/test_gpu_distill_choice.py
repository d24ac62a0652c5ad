"""Distillation on both sides of every limit between rows whole and in pieces:
the divergence alone and the step choose for themselves."""
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note
from tests.test_gpu_distill import make
from tests.test_gpu_distill_precision import check
from tests.test_gpu_top import BF, F

pytestmark = pytest.mark.gpu

SIZES = [(BF, 3, 81920), (BF, 3, 81921), (BF, 143, 81921), (BF, 144, 81921), (BF, 103, 49153), (BF, 104, 49153),
         (BF, 3, 49152), (F, 3, 81920), (F, 3, 81921), (F, 143, 81921), (F, 144, 81921), (F, 63, 49153), (F, 64, 49153),
         (F, 3, 49152), (F, 70, 131071), (F, 70, 131072), (BF, 104, 262143), (BF, 104, 262144)]


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dtype,T,V", SIZES)
def test_both_sides(dtype, T, V, rest):
    note(f"distill choice {dtype} {T} {V} {rest}")
    x, ids, logp = make(6, V, 12, dtype, 1.3, seed=V)
    ids[2], logp[2] = ids[3], logp[3]
    at = torch.arange(T, device=DEV) % 6
    x, ids, logp = x[at], ids[at], logp[at]
    coef = torch.linspace(0.5, 1.5, 6, device=DEV)[at]
    kl, state = L.lora_distill_kl(x, ids, logp, 1.3, rest)
    assert torch.equal(kl, kl[:6][at]) and torch.equal(state, state[:6][at])
    check(x, ids, logp, 1.3, rest, coef, list(range(min(T, 6))))
