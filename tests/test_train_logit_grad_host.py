"""Refusals of the logit gradient with log probabilities, on the host."""
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.test_train_host import FAKE, by, m

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks (fake device pointers)")


def test_logit_grad_logp():
    lib = L.load_library()

    def g(x=m(8, 1000), y=FAKE, stats=FAKE, logp=FAKE, coef=FAKE, dx=m(8, 1000)):
        return lib.lora_logit_grad_logp(x and by(x), y, stats, logp, coef, None, 1.0, dx and by(dx), None)

    assert g(x=None) == -1 and g(dx=None) == -1 and g(y=None) == -1 and g(stats=None) == -1 and g(coef=None) == -1
    assert g(logp=None) == -1 and g(logp=None, x=m(0, 1000), dx=m(0, 1000)) == 0
    assert g(dx=m(8, 999)) == -2 and g(dx=m(8, 1000, 0)) == -3 and g(dx=m(8, 1000, sr=998)) == -4
    x, y, f = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError, match="logp"):
        L.lora_logit_grad(x, y, torch.zeros(4, 2), f, logp=torch.zeros(5))
    with pytest.raises(ValueError, match="GPU"):
        L.lora_logit_grad(x, y, torch.zeros(4, 2), f, logp=f)
