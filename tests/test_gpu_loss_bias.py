"""The exponentials of a row are off to either side: what one term is off by
averages out over a row and is not the same for all of them.

Logits between 8 and 16 below the largest one, which is 0: their differences
are exact. Each exponential's exponent (below 32 in units of log 2) is rounded
within 2^-20, to either side, and the exponential within one step; that step's
own leaning is allowed half of it, 2^-24. Over n terms the roundings leave at
most 2^-20 * 6 / sqrt(n) of it (six standard deviations, the bound taken for
one), over T rows their own rounding 2^-24 * 6 / sqrt(T) more."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu
H = 2.0 ** -24


@pytest.mark.parametrize("T,V", [(2048, 1000), (160, 60_000), (60, 60_000)])
def test_terms_do_not_lean(T, V):
    note(f"leaning {T} {V}")
    torch.manual_seed(T)
    x = -8 * (torch.rand(T, V, device=DEV) + 1)
    y = torch.zeros(T, dtype=torch.int32, device=DEV)
    x[:, 0] = 0.0
    x64 = x.double().cpu().numpy()
    e = np.exp(x64)
    t = e[:, 1:].sum(1)
    allowed = H + 2.0 ** -20 * 6 / np.sqrt(T * V) + H * 6 / np.sqrt(T)
    one = torch.ones(T, device=DEV)
    logp, _ = L.lora_token_logp(x, y)
    _, same, _ = L.lora_policy_step(x, y, one, one, one, 0.2, 0.2)
    for got in (logp, same):
        # d logp / d t = -1 / (1 + t): the relative error of t that the log probabilities show
        lean = ((got.double().cpu().numpy() + np.log1p(t)) * -(1 + t) / t).mean()
        rounding = np.abs(np.log1p(t) * (1 + t) / t).max()  # of logp, in the same units
        assert abs(lean) <= allowed * max(1.0, rounding), lean
    # the gradient's terms, with a sum of 2 and a coefficient of -2 that are exact
    stats = torch.tensor([[0.0, 2.0]], device=DEV).repeat(T, 1)
    dx = L.lora_logit_grad(x, y, stats, -2 * one).double().cpu().numpy()
    assert abs((dx[:, 1:] / e[:, 1:] - 1).mean()) <= allowed
