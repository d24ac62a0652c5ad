"""The example's distillation: it runs, and one step's gradients match the float64
derivative of the same model."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from examples.adapter_training import AdapterTrainer, distill, make_batch
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_example_runs(bits):
    note(f"distillation example {bits}")
    losses = distill(5, bits)
    assert len(losses) == 5 and np.isfinite(losses).all() and min(losses) > 0


def test_gradients_of_the_example_are_the_derivative():
    """float32 weights and activations, every product rounded to float32: the sums of at most 1000 terms are
    within about 1e-5 of the magnitudes, which cancel by far less than the factor of 100 allowed."""
    note("distillation example gradients")
    vocab, width, rank, pairs, k, tau = 300, 128, 8, 3, 12, 2.0
    t = AdapterTrainer(vocab, width, rank, dtype=torch.float32)
    teacher = AdapterTrainer(vocab, width, rank, dtype=torch.float32, seed=1)
    ids, targets, _ = make_batch(pairs, 30, vocab, DEV)
    top_ids, top_logp = teacher.top(ids, targets, k, tau)
    w = torch.rand(len(ids), device=DEV)
    x, logits = t.logits(ids)
    loss, kl, dlogits = L.lora_distill_step(logits, top_ids, top_logp, w, tau)
    t.backward(ids, x, dlogits)

    A, B, table = (v.double().cpu().requires_grad_() for v in t.weights)
    base, head = t.base.double().cpu(), t.head.double().cpu()
    e = table[ids.cpu().long()]
    lp = torch.log_softmax((e @ base + t.scale * (e @ A) @ B) @ head / tau, 1)
    live = (targets >= 0).cpu()
    at, lq = top_ids.cpu().long().clamp_min(0), top_logp.double().cpu()
    q = torch.exp(lq)
    named = torch.zeros(lp.shape, dtype=torch.bool).scatter_(1, at, True)
    q_r, l_r = 1 - q.sum(1), torch.logsumexp(lp.masked_fill(named, -torch.inf), 1)
    each = (q * (lq - lp.gather(1, at))).nan_to_num(0.0).sum(1) + q_r * (torch.log(q_r) - l_r)
    each = torch.where(live, each, 0.0)
    want = (w.double().cpu() * each).sum()
    assert abs(float(loss) - float(want.detach())) <= 1e-4 * (1 + abs(float(want.detach())))
    assert not kl[targets < 0].any()
    for got, v in zip(t.grads, torch.autograd.grad(want, (A, B, table))):
        assert float((got.double().cpu() - v).norm() / v.norm()) <= 1e-3
