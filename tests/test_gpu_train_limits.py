"""The most rows that the losses take: a launch of 2^24 - 1 workgroups."""
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu


def test_most_rows():
    """Rows of two equal logits, every third masked: log probability -log 2, gradient half the coefficient. The
    last rows have others. All values but the logarithm are exact."""
    T = 2 ** 24 - 2
    note(f"rows {T}")
    x = torch.zeros(T, 2, dtype=torch.bfloat16, device=DEV)
    x[-2:, 0] = 1.0
    y = torch.ones(T, dtype=torch.int32, device=DEV)
    y[::3] = -1
    y[-2:] = 0
    live = y >= 0
    logp, stats = L.lora_token_logp(x, y)
    want = torch.where(live, -0.6931471805599453, 0.0).float()
    want[-2:] = -0.31326168751822286
    assert float((logp - want).abs().max()) <= 2.0 ** -22
    coef = torch.full((T,), -4.0, device=DEV)
    dx = L.lora_logit_grad(x, y, stats, coef)
    side = torch.where(live, 2.0, 0.0).to(torch.bfloat16)
    assert torch.equal(dx[:-2, 0], side[:-2]) and torch.equal(dx[:-2, 1], -side[:-2])
    assert float((dx[-2:, 0].float() + 4 * 0.2689414213699951).abs().max()) <= 4 * 0.27 * 2.0 ** -8
    # the steps: ratio 1 and advantage 4, and one pair
    one, zero = torch.ones(T, device=DEV), torch.zeros(T, device=DEV)
    loss, lp, got = L.lora_policy_step(x, y, logp, one * 4, one, 0.2, 0.2)
    assert torch.equal(lp, logp) and torch.equal(got, dx) and float(loss) == -4.0 * int(live.sum())
    off = torch.tensor([0, T - 1, T], dtype=torch.int32, device=DEV)
    _, seq, lp, _ = L.lora_pref_step(x, y, off, zero[:2], 0.1)
    assert torch.equal(lp, logp)
    total = float(logp[:-1].double().sum())
    assert abs(float(seq[0]) - total) <= abs(total) * 2.0 ** -23
    with pytest.raises(L.LoraError):
        L.lora_token_logp(x.new_zeros(2 ** 24, 2), y.new_zeros(2 ** 24))
