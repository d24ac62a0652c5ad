"""The example that runs the training operators together: it learns, and one
step's gradients match the float64 derivative of the same model."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from examples.adapter_training import AdapterTrainer, make_batch, sequence_sums, train
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("loss", ["pref", "policy"])
def test_example_learns(loss, bits):
    note(f"example {loss} {bits}")
    losses, gains = train(loss, 24, bits)
    assert np.isfinite(losses).all()
    # the policy loss starts again near 0 with every new set of sampled log probabilities: its gains count
    assert loss == "policy" or losses[-1] < 0.5 * losses[0]
    assert min(gains) > 1.0, gains


def test_gradients_of_the_example_are_the_derivative():
    """float32 weights and activations, every product rounded to float32: the sums of at most 1000 terms are
    within about 1e-5 of the magnitudes, which cancel by far less than the factor of 100 allowed."""
    note("example gradients")
    vocab, width, rank, pairs = 300, 128, 8, 3
    t = AdapterTrainer(vocab, width, rank, dtype=torch.float32)
    ids, targets, offsets = make_batch(pairs, 30, vocab, DEV)
    ref = sequence_sums(t.logp(ids, targets), offsets) + torch.randn(2 * pairs, device=DEV)
    x, logits = t.logits(ids)
    loss, _, _, dlogits = L.lora_pref_step(logits, targets, offsets, ref, 0.1)
    t.backward(ids, x, dlogits)

    A, B, table = (w.double().cpu().requires_grad_() for w in t.weights)
    base, head = t.base.double().cpu(), t.head.double().cpu()
    e = table[ids.cpu().long()]
    y = e @ base + t.scale * (e @ A) @ B
    live = targets.cpu() >= 0
    lp = torch.log_softmax(y @ head, 1).gather(1, targets.cpu().long().clamp_min(0)[:, None])[:, 0]
    gain = (sequence_sums(torch.where(live, lp, 0.0), offsets.cpu()) - ref.double().cpu()).view(pairs, 2)
    want = -torch.nn.functional.logsigmoid(0.1 * (gain[:, 0] - gain[:, 1])).mean()
    assert abs(float(loss) - float(want.detach())) <= 1e-4
    for got, w in zip(t.grads, torch.autograd.grad(want, (A, B, table))):
        assert float((got.double().cpu() - w).norm() / w.norm()) <= 1e-3
