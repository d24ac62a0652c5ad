"""Alternatives and distillation as torch custom ops: opcheck, autograd against
the library's own gradients bit for bit, and both run together in one loss, also
compiled and as a captured and replayed training step."""
import pytest
import torch

import lora_rank_adapter_amd as L
import lora_rank_adapter_amd.torch_ops  # noqa: F401, registers the ops
from tests.gpu_util import DEV, note
from tests.test_gpu_distill import make
from tests.test_gpu_top import BF, F, check_grad, f64

pytestmark = pytest.mark.gpu
OPS = torch.ops.lora_amd
T, V, K = 37, 1003, 9


def data(dtype, T=T, V=V):
    x, ids, logp = make(T, V, K, dtype, 1.5, seed=4)
    logp[2] = -1.0
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    y = torch.randint(0, V, (T,), device=DEV, dtype=torch.int32, generator=g)
    y[::7] = -100
    return x, y, ids, logp, torch.randn(T, device=DEV, generator=g), torch.randn(T, device=DEV, generator=g)


def test_opcheck():
    x, y, ids, logp, g, h = data(BF)
    _, _, _, _, stats = OPS.token_top(x, y, K, 1.5)
    _, state = OPS.distill_kl(x, ids, logp, 1.5, True)
    for op, args in [(OPS.token_top, (x, y, K, 1.5)), (OPS.token_top, (x, None, 0, 1.5)),
                     (OPS.token_top_grad, (x, y, stats, g, h, 1.5)), (OPS.token_top_grad, (x, None, stats, None, h, 1.5)),
                     (OPS.distill_kl, (x, ids, logp, 1.5, True)), (OPS.distill_grad, (x, ids, state, g, 1.5))]:
        note(f"opcheck {op}")
        torch.library.opcheck(op, args)
    for op, args in [(OPS.token_top, (x.clone().requires_grad_(), y, K, 1.5)),
                     (OPS.distill_kl, (x.clone().requires_grad_(), ids, logp, 1.5, True))]:
        note(f"opcheck {op} with gradients")
        torch.library.opcheck(op, args, test_utils=("test_schema", "test_autograd_registration", "test_faketensor"))


@pytest.mark.parametrize("dtype", [F, BF])
def test_autograd(dtype):
    note(f"alternatives autograd {dtype}")
    x, y, ids, teacher, g, h = data(dtype)
    leaf = x.clone().requires_grad_()
    logp, entropy, _, _, stats = OPS.token_top(leaf, y, K, 1.5)
    ((logp * g).sum() + (entropy * h).sum()).backward()
    assert torch.equal(leaf.grad, L.lora_token_top_grad(x, y, stats, g, h, 1.5))
    check_grad(leaf.grad, f64(x), y.cpu().numpy(), f64(g), f64(h), 1.5, dtype)
    # one of the two alone, gradients of a mean (expanded), no targets
    for take, name in ((0, "dlogp"), (1, "dentropy")):
        leaf.grad = None
        OPS.token_top(leaf, y, 0, 1.5)[take].mean().backward()
        want = L.lora_token_top_grad(x, y, stats, temperature=1.5, **{name: torch.full((T,), 1 / T, device=DEV)})
        assert torch.equal(leaf.grad, want)
    leaf.grad = None
    none, entropy, _, _, every = OPS.token_top(leaf, None, 0, 1.5)
    assert none.numel() == 0
    (entropy * h).sum().backward()
    assert torch.equal(leaf.grad, L.lora_token_top_grad(x, None, every, dentropy=h, temperature=1.5))
    with pytest.raises(RuntimeError, match="beside logp and entropy"):
        OPS.token_top(leaf, y, K, 1.5)[3].sum().backward()
    # distillation: autograd through the divergences, and the step of its own
    leaf.grad = None
    kl, state = OPS.distill_kl(leaf, ids, teacher, 1.5, True)
    (kl * g).sum().backward()
    assert torch.equal(leaf.grad, L.lora_distill_grad(x, ids, state, g, 1.5))
    with pytest.raises(RuntimeError, match="top_logp"):
        OPS.distill_kl(leaf, ids, teacher.clone().requires_grad_(), 1.5, True)[0].sum().backward()


def losses(x, y, ids, teacher, old, adv, w):
    """A policy update with an entropy term and a teacher beside it."""
    logp, entropy, *_ = OPS.token_top(x, y, 0, 1.0)
    policy = OPS.policy_loss(logp, y, x.shape[1], old, adv, w, 0.2, 0.2, None, 0.0)[0]
    return policy - 0.01 * (entropy * w).sum() + 0.1 * (OPS.distill_kl(x, ids, teacher, 2.0, True)[0] * w).sum()


@pytest.mark.parametrize("dtype", [F, BF])
def test_traced_step_is_the_eager_one(dtype):
    note(f"traced alternatives {dtype}")
    x, y, ids, teacher, g, h = data(dtype)
    old, w = torch.full((T,), -5.0, device=DEV), 1 / (T + torch.arange(T, device=DEV))
    grads = []
    for call in (losses, torch.compile(losses, backend="aot_eager", fullgraph=True)):
        leaf = x.clone().requires_grad_()
        loss = call(leaf, y, ids, teacher, old, h, w)
        loss.backward()
        grads.append((loss.detach(), leaf.grad))
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])
    # The loss changes along its gradient as that says: over a step of 2 |g| to each side, of which the third order is
    # below |2 g|^2 = 2 % (|g| is 0.04 here), and the float32 losses' rounding counts 64 half steps of 1 + |loss| over 4.
    x, g = x.float(), grads[0][1].float()
    a, b = (losses(x + s * g, y, ids, teacher, old, h, w) for s in (2, -2))
    slope = float((g.double() ** 2).sum())
    assert slope < 0.05 ** 2
    assert abs(float(a - b) / 4 - slope) <= 0.02 * slope + 2.0 ** -20 * (1 + abs(float(a)))


def test_captured_step():
    note("captured alternatives and distillation")
    x, y, ids, teacher, g, h = data(BF, 40, 60001)
    n = x.shape[0]
    old, w = torch.full((n,), -5.0, device=DEV), torch.rand(n, device=DEV)
    leaf = x.clone().requires_grad_()

    def step():
        leaf.grad = None
        loss = losses(leaf, y, ids, teacher, old, h, w)
        loss.backward()
        return loss.detach()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    leaf.grad = None
    with torch.cuda.graph(graph):
        loss = step()
        grad = leaf.grad
    for seed in range(3):
        with torch.no_grad():
            leaf.copy_(torch.randn(x.shape, device=DEV) * (1 + seed))
        graph.replay()
        torch.cuda.synchronize()
        other = leaf.detach().clone().requires_grad_()
        want = losses(other, y, ids, teacher, old, h, w)
        want.backward()
        assert torch.equal(loss, want.detach()) and torch.equal(grad, other.grad), seed
