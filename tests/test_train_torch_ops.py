"""CPU checks of the training operators' torch custom ops: shapes on fake
tensors, the gradients' shapes and refusals, and that CPU tensors are refused."""
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from lora_rank_adapter_amd import torch_ops

OPS = torch.ops.lora_amd
BF, F = torch.bfloat16, torch.float32
T, V, D = 12, 50, 16


def test_fake_shapes():
    with FakeTensorMode():
        i = torch.empty(T, dtype=torch.int32, device="cuda")
        table, x, f = (torch.empty(*s, dtype=d, device="cuda") for s, d in (((V, D), BF), ((T, V), BF), ((T,), F)))
        e = OPS.embed(i, table, 2.0, F)
        assert e.shape == (T, D) and e.dtype == F
        g = OPS.embed_grad(i, e, V, 2.0, F)
        assert g.shape == (V, D) and g.dtype == F
        lp, st = OPS.token_logp(x, i)
        assert lp.shape == (T,) and st.shape == (T, 2) and lp.dtype == st.dtype == F
        assert OPS.logit_grad(x, i, st, f).shape == (T, V)
        off, ref = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
        loss, seq, coef = OPS.pref_loss(lp, off, ref, 0.1, 0.0)
        assert loss.shape == () and seq.shape == (4,) and coef.shape == (T,)
        loss, coef = OPS.policy_loss(lp, i, V, f, f, f, 0.2, 0.2, None, 0.0)
        assert loss.shape == () and coef.shape == (T,)
        # the table's gradient in its own type, whatever the rows' type
        for out in (BF, F):
            ctx = types.SimpleNamespace(saved_tensors=(i,), rows=V, dtype=BF, scale=2.0)
            grads = torch_ops._embed_backward(ctx, torch.empty(T, D, dtype=out, device="cuda"))
            assert grads[1].shape == (V, D) and grads[1].dtype == BF and grads[0] is grads[2] is grads[3] is None


def test_gradients_that_do_not_exist_are_refused():
    g = torch.ones(3)
    with pytest.raises(RuntimeError, match="stats"):
        torch_ops._logp_backward(types.SimpleNamespace(saved_tensors=(g, g, g)), g, g)
    with pytest.raises(RuntimeError, match="beside the loss"):
        torch_ops._loss_backward(types.SimpleNamespace(saved_tensors=(g,), inputs=5), g, g, None)
    ctx = types.SimpleNamespace(saved_tensors=(g,), inputs=5)
    assert torch_ops._loss_backward(ctx, None, None, None) == (None,) * 5
    assert torch_ops._logp_backward(types.SimpleNamespace(saved_tensors=(g, g, g)), None, None) == (None, None)


@pytest.mark.parametrize("t", [torch.ones(()).expand(4, 6), torch.ones(6, 4).t(), torch.ones(4, 1).expand(4, 6)])
def test_gradients_of_broadcasts_are_laid_out(t):
    r = torch_ops._rows(t)
    assert r.stride() == (6, 1) and torch.equal(r, t)
    whole = torch.ones(4, 9)[:, :6]
    assert torch_ops._rows(whole) is whole


def test_cpu_tensors_are_refused():
    i, f, x = torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(4, 6)
    for call in (lambda: OPS.embed(i, x, 1.0, F), lambda: OPS.embed_grad(i, x, 6, 1.0, F),
                 lambda: OPS.token_logp(x, i), lambda: OPS.logit_grad(x, i, torch.zeros(4, 2), f),
                 lambda: OPS.pref_loss(f, i[:3], f[:2], 0.1, 0.0),
                 lambda: OPS.policy_loss(f, i, 6, f, f, f, 0.2, 0.2, None, 0.0)):
        with pytest.raises(NotImplementedError):
            call()
