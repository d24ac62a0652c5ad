"""CPU checks of the custom ops of alternatives and distillation: shapes on fake
tensors, gradients that do not exist, refusals."""
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from lora_rank_adapter_amd import torch_ops, train

OPS = torch.ops.lora_amd
BF, F, I = torch.bfloat16, torch.float32, torch.int32
T, V, K = 12, 50, 7


def test_fake_shapes():
    with FakeTensorMode():
        x, y, f = (torch.empty(*s, dtype=d, device="cuda") for s, d in (((T, V), BF), ((T,), I), ((T,), F)))
        for targets in (y, None):
            logp, entropy, ids, top, stats = OPS.token_top(x, targets, K, 0.7)
            assert logp.shape == ((0,) if targets is None else (T,)) and entropy.shape == (T,)
            assert ids.shape == top.shape == (T, K) and stats.shape == (T, 3)
            assert ids.dtype is I and {t.dtype for t in (logp, entropy, top, stats)} == {F}
            dx = OPS.token_top_grad(x, targets, stats, None, f, 0.7)
            assert dx.shape == (T, V) and dx.dtype is BF
        kl, state = OPS.distill_kl(x, ids, top, 2.0, True)
        assert kl.shape == (T,) and state.shape == (T, K + 2) and kl.dtype is state.dtype is F
        assert OPS.distill_grad(x, ids, state, f, 2.0).shape == (T, V)


def test_gradients_that_do_not_exist_are_refused():
    g = torch.ones(3)
    ctx = types.SimpleNamespace(saved_tensors=(g, None, g), temperature=1.0, needs_input_grad=(True,) + (False,) * 4)
    for others in ((None, g, None), (None, None, g)):
        with pytest.raises(RuntimeError, match="beside logp and entropy"):
            torch_ops._top_backward(ctx, None, g, *others)
    assert torch_ops._top_backward(ctx, g, None, None, None, None) == (None,) * 4
    with pytest.raises(RuntimeError, match="state"):
        torch_ops._distill_backward(ctx, g, g)
    assert torch_ops._distill_backward(ctx, None, None) == (None,) * 5
    ctx.needs_input_grad = (True, False, True, False, False)
    with pytest.raises(RuntimeError, match="top_logp"):
        torch_ops._distill_backward(ctx, g, None)


def test_cpu_tensors_are_refused():
    x, i, f, k = torch.zeros(4, 6), torch.zeros(4, dtype=I), torch.zeros(4), torch.zeros(4, 2, dtype=I)
    for call in (lambda: OPS.token_top(x, i, 2, 1.0), lambda: OPS.token_top_grad(x, i, torch.zeros(4, 3), f, f, 1.0),
                 lambda: OPS.distill_kl(x, k, torch.zeros(4, 2), 1.0, True),
                 lambda: OPS.distill_grad(x, k, torch.zeros(4, 4), f, 1.0)):
        with pytest.raises(NotImplementedError):
            call()


def test_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(train, "_queue", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert train._here(torch.device("cuda:0")) == 0
    with pytest.raises(ValueError, match="current device"):
        train._here(torch.device("cuda:1"))
