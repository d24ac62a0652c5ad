"""The policy step on both sides of where it changes its form, for both types:
rows taken whole by 4, 8 or 16 waves, and in pieces. Bounds as in the tests of
the losses."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from oracle import train_oracle as O
from tests.gpu_util import DEV, note
from tests.test_gpu_loss import BF, F, H, close, f64, grad_bounds, make, row_bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,T,V", [(BF, 79, 32769), (BF, 80, 32769), (BF, 5, 32768), (F, 47, 32769),
                                       (F, 48, 32769), (F, 5, 32768), (BF, 90, 20487), (BF, 90, 20488), (F, 50, 10243),
                                       (F, 50, 10244), (BF, 79, 128256), (F, 47, 128256)])
def test_either_side(dtype, T, V):
    note(f"policy forms {dtype} {T} {V}")
    torch.manual_seed(T + V)
    x, y = make(T, V, dtype, T + V, pad=1, shift=1)
    lp, _ = L.lora_token_logp(x, y)
    old, ref = lp + torch.randn(T, device=DEV) * 0.3, lp + torch.randn(T, device=DEV) * 0.5
    adv, w = torch.randn(T, device=DEV), torch.rand(T, device=DEV)
    masked = torch.from_numpy(O.masked(y.cpu().numpy(), V)).to(DEV)
    for t in (old, ref, adv, w):
        t[masked] = float("nan")
    args = (old, adv, w, 0.2, 0.3, ref, 0.1)
    loss, logp, dx = L.lora_policy_step(x, y, *args, grad_scale=0.5)
    x64, yn = f64(x), y.cpu().numpy()
    close(f64(logp), O.token_logp(x64, yn), row_bounds(x64, yn)[1], "logp")
    loss2, coef = L.lora_policy_loss(logp, y, V, *args)
    terms = np.abs(f64(w)) * (3 * np.abs(f64(adv)) + 1)
    assert abs(float(loss) - float(loss2)) <= 32 * H * np.nansum(terms)
    want, tol = grad_bounds(x64, yn, 0.5 * f64(coef), dtype)
    close(f64(dx), want, tol + 16 * H * np.abs(want), "dx")
    assert not dx[masked].any()
    L.lora_policy_step(x, y, *args, grad_scale=0.5, dlogits=x)
    assert torch.equal(x, dx)
