"""Targets that hold nearly all of the probability: what is left to the others,
q = 1 - p, is the size of the log probability and of the gradient at the
target, and both keep it to a relative bound however small it is.

With t the sum of the others' exp(x_j - x_y), q = t / (1 + t) and logp =
-log(1 + t): relative errors of t pass to both at most once. A term of t is off
by 3 H |d_j| + 2^-23 (H = 2^-24: its difference and exponent rounded, the
exponential off by one step), a lane's additions and those of the joined lanes
by 2 (V / 64 + 64) H, expm1 by 2^-22, and four products and roundings follow.
But for the policy step, rows whose sum is not near 1 take the gradient at the
target from the rounded sum, which loses 4 H of the coefficient: q is at least
1/5 there (float32), or 2^-8.5 (bfloat16)."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
import lora_rank_adapter_amd.torch_ops  # noqa: F401, registers the ops
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
H = 2.0 ** -24
SHAPES = [(26, 128256), (300, 20011), (2100, 515), (130, 60001), (9, 1023), (1100, 9000), (9, 2), (3, 300007)]


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, V, dtype):
    """Rows whose targets leave 0.5 to 1e-13 to the others: to all of them alike, or (every second row) to one
    neighbour of the target."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T + V)
    x = torch.randn(T, V, device=DEV, generator=g)
    y = torch.randint(0, V, (T,), device=DEV, generator=g)
    rows = torch.arange(T, device=DEV)
    q = 10.0 ** -(torch.arange(T, device=DEV).double() * 13 / max(T - 1, 1) + 0.3)
    x[1::2] -= 60.0
    x[rows, y] = -float("inf")
    near = torch.where(y % 8 == 7, y - 1, (y + 1).clamp_max(V - 1))
    near = torch.where(near == y, y - 1, near)
    x[rows[1::2], near[1::2]] = 0.0
    x = x.to(dtype)
    top = torch.logsumexp(x.double(), 1) + torch.log((1 - q) / q)
    x[rows, y] = top.to(dtype)
    return x, y.to(torch.int32)


def left(x, y):
    """(q, log(1 + t), the bound of t's relative error) of each row"""
    T, V = x.shape
    q, lp, err = np.zeros(T), np.zeros(T), np.zeros(T)
    for r in range(T):
        row = f64(x[r])
        d = row - row[y[r]]
        m = row.max()
        e = np.exp(d)
        e[y[r]] = 0.0
        t = e.sum()
        q[r], lp[r] = t / (1 + t), np.log1p(t)
        share = e / t
        err[r] = 3 * H * (share * np.abs(row - m)).sum() + 2.0 ** -23 + 2 * (V / 64 + 64) * H
    return q, lp, err


def close(got, want, rel, what):
    err = np.abs(f64(got) - want)
    tol = rel * np.abs(want) + 1e-37
    assert (err <= tol).all(), (what, int((err / tol).argmax()), float((err / tol).max()))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V", SHAPES)
def test_what_the_others_hold(dtype, T, V):
    note(f"likely targets {dtype} {T} {V}")
    x, y = make(T, V, dtype)
    yn = y.cpu().numpy()
    q, lp, err = left(x, yn)
    logp, stats = L.lora_token_logp(x, y)
    close(logp, -lp, err + 4 * H, "logp")
    at = torch.arange(T, device=DEV), y.long()
    out = torch.finfo(dtype).eps / 2
    grad = err + 2.0 ** -22 + 8 * H + out
    alone = grad + 4 * H / (0.2 if dtype is F else 2.0 ** -8.5)

    # from the statistics: with a factor on the device, over the logits, and through autograd
    coef, two = torch.randn(T, device=DEV), torch.full((), 2.0, device=DEV)
    dx = L.lora_logit_grad(x, y, stats, coef, grad_out=two, scale=0.25)
    close(dx[at], 0.5 * f64(coef) * q, alone, "logit_grad")
    held = L.lora_logit_grad(x, y, stats, coef, grad_out=two, scale=0.25, logp=logp)
    close(held[at], 0.5 * f64(coef) * q, alone, "logit_grad, logp")
    held[at] = dx[at]
    assert torch.equal(held, dx)  # beside the targets the same bits
    over = x.clone()
    L.lora_logit_grad(over, y, stats, coef, grad_out=two, scale=0.25, dlogits=over)
    assert torch.equal(over, dx)
    leaf = x.clone().requires_grad_()
    graph = torch.ops.lora_amd.token_logp(leaf, y)[0]
    graph.add_(1)  # the backward keeps its own
    graph.backward(coef)
    close(leaf.grad[at], f64(coef) * q, alone, "autograd")

    # a policy step: ratios near 1, and the coefficient that these log probabilities give
    one = torch.ones(T, device=DEV)
    args = (logp, coef, one, 0.2, 0.2)
    _, got, dx = L.lora_policy_step(x, y, *args, grad_scale=0.5)
    close(got, -lp, err + 4 * H, "policy logp")
    _, c = L.lora_policy_loss(got, y, V, *args)
    close(dx[at], 0.5 * f64(c) * q, grad, "policy_step")
    over = x.clone()
    L.lora_policy_step(over, y, *args, grad_scale=0.5, dlogits=over)
    assert torch.equal(over, dx)

    # a preference step
    off = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    ref = torch.tensor([-1.0, 2.0], device=DEV)
    _, _, got, dx = L.lora_pref_step(x, y, off, ref, 0.1, grad_scale=3.0)
    assert torch.equal(got, logp)
    _, _, c = L.lora_pref_loss(logp, off, ref, 0.1)
    close(dx[at], 3 * f64(c) * q, alone, "pref_step")
    assert torch.equal(dx, L.lora_logit_grad(x, y, stats, c, scale=3.0, logp=logp))
    over = x.clone()
    L.lora_pref_step(over, y, off, ref, 0.1, grad_scale=3.0, dlogits=over)
    assert torch.equal(over, dx)


@pytest.mark.parametrize("T,V", [(26, 128256), (1100, 9000)])
def test_rows_sum_to_nothing(T, V):
    """The entries of a row cancel: the target's is what the others are together. Each of the others is off by the
    bound above relative to itself, and so is the target's."""
    note(f"likely targets, sums {T} {V}")
    x, y = make(T, V, F)
    q, _, err = left(x, y.cpu().numpy())
    logp, stats = L.lora_token_logp(x, y)
    for lp in (None, logp):
        dx = f64(L.lora_logit_grad(x, y, stats, torch.ones(T, device=DEV), logp=lp))
        assert (np.abs(dx.sum(1)) <= (3 * err + 2.0 ** -21 + 4 * H / 0.2) * q + V * 1e-37).all()


@pytest.mark.parametrize("given", [False, True])
def test_captured_gradient_replays(given):
    note(f"likely targets, graph {given}")
    x, y = make(40, 9001, BF)
    coef = torch.randn(40, device=DEV)
    out = torch.empty_like(x)

    def call(x, out):
        logp, stats = L.lora_token_logp(x, y)
        return L.lora_logit_grad(x, y, stats, coef, dlogits=out, logp=logp if given else None)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(x, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, out)
    for i in range(4):
        x.mul_(0.9)  # some rows cease to be likely
        coef.neg_()
        want = call(x, torch.empty_like(x))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
