"""Distillation of many long rows, by 16 and by 8 waves: a part of each row stays
in registers from the sum to the gradient, its beginning is read again. Bounds
as in test_gpu_distill_precision."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note
from tests.test_gpu_distill import make
from tests.test_gpu_distill_precision import check, tight
from tests.test_gpu_top import BF, F, close, f64

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def long_rows(T, V, k, dtype, seed):
    """T rows that repeat 10 of them."""
    x, ids, logp = make(10, V, k, dtype, seed=seed)
    ids[2], logp[2] = ids[3], logp[3]
    ids[4], logp[4] = ids[5], logp[5]
    at = torch.arange(T, device=DEV) % 10
    return x, ids, logp, at


LONG = [(120, 130003), (260, 130003)]


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V", LONG)
def test_many_long_rows(dtype, T, V, rest):
    note(f"distill many long {dtype} {T} {V} {rest}")
    x, ids, logp, at = long_rows(T, V, 24, dtype, 1)
    # tokens named twice, in the beginning and in the held end; one token, again and again
    ids[0, 5], ids[0, 9], ids[0, 23] = ids[0, 1], ids[0, 1], ids[0, 2]
    ids[1, 3], ids[1, 17] = V - 9, V - 9
    ids[6, 4], ids[6, 20] = 11, 11
    ids[8, 1:] = ids[8, 0]
    logp[8] = -4.0
    x, ids, logp = x[at], ids[at], logp[at]
    coef = torch.randn(10, device=DEV)[at]
    _, kl, dx = L.lora_distill_step(x, ids, logp, coef, 1.0, rest)
    assert torch.equal(kl, kl[:10][at]) and torch.equal(dx, dx[:10][at])
    check(x, ids, logp, 1.0, rest, coef, list(range(10)))


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V", LONG)
def test_undefined_values_in_many_long_rows(dtype, T, V, late):
    note(f"distill undefined long {dtype} {T} {V} {late}")
    x, ids, logp, at = long_rows(T, V, 6, dtype, 3)
    place = V - 5000 if late else 300  # in the end that registers hold, or where a row is read again
    ids[:, 5] = place
    other = place + 8 * 7 + 3
    while bool((ids == other).any()):
        other += 1
    x[0] = -INF                       # nothing left
    x[1, other] = INF
    x[2, place] = NAN
    x[3, other] = NAN
    x[4] = NAN
    ids[4] = -1                       # masked: not read
    x[5, place] = -INF                # a token of the teacher without probability
    named = torch.zeros(10, V, dtype=torch.bool, device=DEV).scatter_(1, ids.clamp(0, V - 1).long(), True)
    x[6] = torch.where(named[6], x[6], -INF)                          # only the teacher's tokens left
    x[7] = torch.where(named[7], x[7], torch.finfo(dtype).min)        # the same with the lowest value
    half = slice(0, V // 2) if late else slice(V // 2, V)
    x[8, half] = torch.where(named[8, half], x[8, half], -INF)        # half a vocabulary
    x, ids, logp = x[at], ids[at], logp[at]
    weights = torch.where(at < 8, 0.0, 1.0)
    for rest in (True, False):
        kl0, state = L.lora_distill_kl(x, ids, logp, 1.0, rest)
        dx0 = L.lora_distill_grad(x, ids, state, torch.ones(T, device=DEV), 1.0)
        _, kl1, dx1 = L.lora_distill_step(x, ids, logp, torch.ones(T, device=DEV), 1.0, rest)
        for kl, dx in ((kl0, dx0), (kl1, dx1)):
            assert torch.isnan(kl[:4]).all() and torch.isnan(dx[:4]).all()
            assert kl[4] == 0 and not dx[4].any()
            assert torch.isposinf(kl[5]) and torch.isfinite(dx[5:10]).all()
            assert bool(torch.isposinf(kl[6])) == rest
            assert not dx[6][~named[6]].any() and not dx[8, half][~named[8, half]].any()
            rows = [8, 9] if rest else [6, 7, 8, 9]
            pick = torch.tensor(rows, device=DEV)
            want, e_kl, wx, ex = tight(f64(x[pick]), ids[pick].cpu().numpy(), f64(logp[pick]), 1.0, rest,
                                       np.ones(len(rows)), dtype)
            close(f64(kl[pick]), want, e_kl)
            close(f64(dx[pick]), wx, ex)
            assert torch.equal(torch.nan_to_num(dx, 9.0), torch.nan_to_num(dx, 9.0)[:10][at])
        # a weight of zero drops what is infinite or undefined, also where the gradient takes the logits' place
        loss, kl, dx = L.lora_distill_step(x, ids, logp, weights, 1.0, rest)
        assert bool(torch.isfinite(loss)) and not dx[at < 8].any()
        y = x.clone()
        assert torch.equal(L.lora_distill_step(y, ids, logp, weights, 1.0, rest, dlogits=y)[2], dx)
