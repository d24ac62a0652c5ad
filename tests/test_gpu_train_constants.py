"""The losses through autograd with inputs that ask for a gradient they do not
have, and with detached ones."""
import pytest
import torch

import lora_rank_adapter_amd.torch_ops  # noqa: F401, registers the ops
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu
OPS = torch.ops.lora_amd


def test_constants_say_so():
    note("loss constants")
    T = 12
    torch.manual_seed(0)
    logp, old, ref, adv, w = (torch.randn(T, device=DEV) for _ in range(5))
    y = torch.zeros(T, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 6, 12], dtype=torch.int32, device=DEV)

    def policy(old, adv, w, ref):
        leaf = logp.clone().requires_grad_()
        OPS.policy_loss(leaf, y, 5, old, adv, w, 0.2, 0.2, ref, 0.1)[0].backward()
        return leaf.grad

    given = [old, adv, w, ref]
    want = policy(*given)
    for i, name in enumerate(("old_logp", "advantages", "weights", "ref_logp")):
        asking = list(given)
        asking[i] = asking[i].clone().requires_grad_()
        with pytest.raises(RuntimeError, match=name):
            policy(*asking)
        asking[i] = asking[i].detach()
        assert torch.equal(policy(*asking), want)
        with torch.no_grad():  # nothing is asked for
            OPS.policy_loss(logp, y, 5, *[t.clone().requires_grad_() for t in given[:3]], 0.2, 0.2, None, 0.0)
    leaf = logp.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="ref_logp"):
        OPS.pref_loss(leaf, off, ref[:2].clone().requires_grad_(), 0.1, 0.0)[0].backward()
    OPS.pref_loss(leaf, off, ref[:2], 0.1, 0.0)[0].backward()
    assert leaf.grad.any()
