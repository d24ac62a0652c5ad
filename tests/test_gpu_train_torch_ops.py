"""The training operators as torch custom ops: opcheck, and gradients through
autograd against the float64 formulas (bounds: every output's own rounding,
and 2^-14 of the largest term for the float32 sums of a row of 1003)."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
import lora_rank_adapter_amd.torch_ops  # noqa: F401, registers the ops
from oracle import train_oracle as O
from tests.gpu_util import DEV, note
from tests.test_gpu_loss import BF, F, f64, make

pytestmark = pytest.mark.gpu
OPS = torch.ops.lora_amd
T, V, D = 37, 1003, 24


def data(dtype):
    torch.manual_seed(2)
    x, y = make(T, V, dtype, 6)
    off = torch.tensor([0, 9, 20, 20, 33], dtype=torch.int32, device=DEV)
    f = [torch.randn(T, device=DEV) * 0.3 - 4 for _ in range(2)]
    return x, y, off, torch.randn(4, device=DEV) * 3 - 30, f, torch.randn(T, device=DEV), torch.rand(T, device=DEV)


def test_opcheck():
    x, y, off, ref, f, adv, w = data(BF)
    table = torch.randn(V, D, device=DEV).to(BF)
    lp, st = OPS.token_logp(x, y)
    cases = [
        (OPS.embed, (y, table.clone().requires_grad_(), 2.0, F)),
        (OPS.embed_grad, (y, torch.randn(T, D, device=DEV), V, 2.0, F)),
        (OPS.logit_grad, (x, y, st, lp)),
        (OPS.token_logp, (x, y)),
        (OPS.pref_loss, (lp, off, ref, 0.1, 0.05)),
        (OPS.policy_loss, (lp, y, V, *f, adv, 0.2, 0.2, w, 0.1)),
    ]
    for op, args in cases:
        note(f"opcheck {op}")
        torch.library.opcheck(op, args)


@pytest.mark.parametrize("dtype,out", [(F, F), (BF, F), (BF, BF)])
def test_embed_gradient(dtype, out):
    note(f"embed autograd {dtype} {out}")
    _, ids, *_ = data(F)
    table = torch.randn(V, D, device=DEV).to(dtype).requires_grad_()
    e = OPS.embed(ids, table, 1.5, out)
    g = torch.randn(T, D, device=DEV).to(out)
    e.backward(g)
    want = O.embed_grad(ids.cpu().numpy(), f64(g), V, 1.5)
    assert table.grad.dtype is dtype
    tol = (2.0 ** -16 + (torch.finfo(BF).eps if dtype is BF else 0)) * np.abs(want) + T * 2.0 ** -24
    assert (np.abs(f64(table.grad) - want) <= tol).all()
    # a sum's gradient comes expanded
    table.grad = None
    OPS.embed(ids, table, 1.0, out).float().sum().backward()
    assert np.array_equal(f64(table.grad), O.embed_grad(ids.cpu().numpy(), np.ones((T, D)), V, 1.0))


@pytest.mark.parametrize("dtype", [F, BF])
def test_pref_gradient(dtype):
    note(f"pref autograd {dtype}")
    x, y, off, ref, *_ = data(dtype)
    yn, x64 = y.cpu().numpy(), f64(x)
    leaf = x.clone().requires_grad_()
    logp, _ = OPS.token_logp(leaf, y)
    (3 * OPS.pref_loss(logp, off, ref, 0.1, 0.05)[0]).backward()
    coef = O.pref_loss(O.token_logp(x64, yn), off.cpu().numpy(), f64(ref), 0.1, 0.05)[2]
    want = O.logit_grad(x64, yn, 3 * coef)
    most = np.abs(3 * coef)[:, None] * np.maximum(O.softmax(x64), np.abs(O.logit_grad(x64, yn, np.ones(T))))
    tol = 2.0 ** -14 * most + torch.finfo(dtype).eps / 2 * 1.01 * np.abs(want) + 1e-37
    assert (np.abs(f64(leaf.grad) - want) <= tol).all()


@pytest.mark.parametrize("dtype", [F, BF])
def test_policy_gradient_is_the_direct_calls(dtype):
    """The same bits as the library's calls one after the other (their bounds
    against float64 are in the loss tests: a policy coefficient is a difference
    of two terms, so no bound relative to itself holds)."""
    note(f"policy autograd {dtype}")
    x, y, _, _, (old, refs), adv, w = data(dtype)
    leaf = x.clone().requires_grad_()
    logp, _ = OPS.token_logp(leaf, y)
    loss, _ = OPS.policy_loss(logp, y, V, old, adv, w, 0.2, 0.3, refs, 0.1)
    (3 * loss).backward()
    lp, stats = L.lora_token_logp(x, y)
    loss2, coef = L.lora_policy_loss(lp, y, V, old, adv, w, 0.2, 0.3, refs, 0.1)
    assert torch.equal(logp.detach(), lp) and torch.equal(loss.detach(), loss2)
    assert torch.equal(leaf.grad, L.lora_logit_grad(x, y, stats, 3 * coef))


def test_outputs_without_gradient_say_so():
    x, y, off, ref, *_ = data(F)
    note("no gradient")
    logp, stats = OPS.token_logp(x.requires_grad_(), y)
    with pytest.raises(RuntimeError, match="stats"):
        stats.sum().backward()
    lp = logp.detach().requires_grad_()
    with pytest.raises(RuntimeError, match="beside the loss"):
        OPS.pref_loss(lp, off, ref, 0.1, 0.0)[1].sum().backward()
