"""The policy loss's KL term exp(k) - k - 1 near k = 0, where it is k^2 / 2: its
own size is what it is off by, not that of k.

Below 1/2 it is a polynomial of k times k^2 (two roundings of the square, each
step of the polynomial's damped by k / 3, the last product: 4 roundings; its
remainder 2^-28), above a difference of two terms that are at most 6 times its
size, one of them within a step (2^-23), the other exact. The weight, the
coefficient and the loss are rounded once each."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu
H = 2.0 ** -24


def values():
    k = np.float32(10.0) ** np.arange(-12, 2, 0.25, dtype=np.float32)
    edge = np.float32([0.49999997, 0.5, 0.50000006, 0.25, 1.0])
    return np.concatenate([k, -k, edge, -edge])


def exact(k):
    """exp(k) - k - 1 in float64 by its series where the difference would cancel."""
    k = np.float64(k)
    if abs(k) > 1:
        return np.expm1(k) - k
    term, total = k, 0.0
    for n in range(2, 40):
        term = term * k / n
        total += term
    return total


def test_small_differences():
    note("policy kl")
    one, zero = torch.ones(1, device=DEV), torch.zeros(1, device=DEV)
    y = torch.zeros(1, dtype=torch.int32, device=DEV)
    for k in values():
        loss, coef = L.lora_policy_loss(zero, y, 5, zero, zero, one, 0.2, 0.2, zero + float(k), 0.25)
        want = 0.25 * exact(k)
        assert loss >= 0 and abs(float(loss) - want) <= (4 + 16 + 4) * H * want, k
        assert abs(float(coef) + 0.25 * np.expm1(np.float64(k))) <= 6 * H * abs(np.expm1(np.float64(k))), k


def test_the_steps_have_the_same_terms():
    note("policy kl, steps")
    k = torch.from_numpy(values()).to(DEV)
    T = len(k)
    for V in (50, 60_000):  # rows whole, and in pieces
        torch.manual_seed(V)
        x = torch.randn(T, V, device=DEV)
        y = torch.randint(0, V, (T,), dtype=torch.int32, device=DEV)
        lp, _ = L.lora_token_logp(x, y)
        one, zero = torch.ones(T, device=DEV), torch.zeros(T, device=DEV)
        ref = lp + 1e-4 * k.clamp(-1, 1)
        loss, logp, _ = L.lora_policy_step(x, y, lp, zero, one, 0.2, 0.2, ref, 1.0)
        d = (ref - logp).cpu().numpy()
        want = sum(exact(v) for v in d)
        assert abs(float(loss) - want) <= 24 * H * want
