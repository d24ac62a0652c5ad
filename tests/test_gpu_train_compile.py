"""The losses as torch custom ops under tracing, with inputs that ask for a
gradient: torch's own checks of an op, and a compiled step against an eager
one, bit for bit."""
import pytest
import torch

import lora_rank_adapter_amd.torch_ops  # noqa: F401, registers the ops
from tests.gpu_util import DEV, note
from tests.test_gpu_loss import BF, F, make

pytestmark = pytest.mark.gpu
OPS = torch.ops.lora_amd
T, V = 37, 1003


def data(dtype):
    torch.manual_seed(2)
    x, y = make(T, V, dtype, 6)
    x[3] = 0
    x[3, y[3].long()] = 30.0  # a likely target
    off = torch.tensor([0, 9, 20, 20, 33], dtype=torch.int32, device=DEV)
    f = [torch.randn(T, device=DEV) * 0.3 - 4 for _ in range(2)]
    return x, y, off, torch.randn(4, device=DEV) * 3 - 30, f, torch.randn(T, device=DEV), torch.rand(T, device=DEV)


def test_opcheck_with_gradients():
    x, y, off, ref, f, adv, w = data(BF)
    lp, st = OPS.token_logp(x, y)
    cases = [
        (OPS.token_logp, (x.clone().requires_grad_(), y)),
        (OPS.logit_grad, (x, y, st, lp, lp)),
        (OPS.pref_loss, (lp.clone().requires_grad_(), off, ref, 0.1, 0.05)),
        (OPS.policy_loss, (lp.clone().requires_grad_(), y, V, f[0], adv, w, 0.2, 0.2, f[1], 0.1)),
    ]
    for op, args in cases:
        note(f"opcheck {op} with gradients")
        # not its tracing of the sum of all outputs, some of which have no gradient: the step below traces the losses
        torch.library.opcheck(op, args, test_utils=("test_schema", "test_autograd_registration", "test_faketensor"))


@pytest.mark.parametrize("dtype", [F, BF])
def test_traced_step_is_the_eager_one(dtype):
    note(f"traced losses {dtype}")
    x, y, off, ref, f, adv, w = data(dtype)

    def losses(x):
        logp, _ = OPS.token_logp(x, y)
        return OPS.pref_loss(logp, off, ref, 0.1, 0.05)[0] + OPS.policy_loss(logp, y, V, f[0], adv, w, 0.2, 0.2, f[1],
                                                                             0.1)[0]

    grads = []
    for call in (losses, torch.compile(losses, backend="aot_eager", fullgraph=True)):
        leaf = x.clone().requires_grad_()
        loss = call(leaf)
        loss.backward()
        grads.append((loss.detach(), leaf.grad))
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])
