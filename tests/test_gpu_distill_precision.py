"""Distillation keeps its precision wherever in a row the likely tokens lie, and
however little the tokens outside the teacher's hold.

Bounds (H = 2^-24), none of them absolute but for underflow. The others'
exponentials are float32, relative to a reference that no logit of the lane so
far exceeds and that lies three binary orders above the largest of them or of the
row's beginning, in trees of eight terms (3 H); a lane that meets a larger logit
moves its reference and scales what it has, and all are scaled to the largest
reference at the end. u is an other logit's distance (over tau) below the largest
of the others:
    one term: exponents of 2 H by what they bridge, in all from the logit up to that reference: 2 H (u + 2.1); 2 H for
    each exponential: its own, the steps' (u / ln(8) + 1), the last; the tree's 3 H:
    e_j = 9 H u_j + 18 H                            (relative)
    e_o = sum of their shares' e_j                  (relative, of the others' sum)
The gradient's exponents are relative to that reference too: 2 H (u + 2.1), 2 H for the exponential and 5 H for the
factors. What is made of the sum is float64, within 2^-45 of its own terms; q_r = 1 - sum q,
where it is above 0, is off by 2^-46 besides. With t = p / p_r, F = Q p_r - q_r:
    err(kl) <= p_r e_o sum q + (1 - p_r) e_o q_r + H |kl| + 2^-45 (sum q (|log q| + |log p|) + q_r (|log q_r| + |log p_r|))
               + 2^-46 (1 + |log q_r| + |log p_r|) [q_r > 0]
    tau err(dx_j) <= t_j (|F| (3 H u_j + 12 H) + max(Q p_r^2, q_r) e_o + 2^-45 (Q p_r + q_r) + 2^-46 [q_r > 0])  elsewhere
                     Q p_k p_r e_o + 4 H |b_k| + 2^-45 (Q p_k + q_k)                at the teacher's tokens
times |coef|, half a step of the output's type, and 2^-126 (|coef| / tau + 1) for what is below that."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from oracle import train_oracle as O
from tests.gpu_util import DEV, note
from tests.test_gpu_distill import make
from tests.test_gpu_top import BF, F, H, close, f64

pytestmark = pytest.mark.gpu


def tight(x64, ids, logp, tau, rest, coef, dtype):
    """(kl, err(kl), dlogits, err(dlogits)); every row has a token and probabilities"""
    T, V = x64.shape
    kl, dx = O.distill(x64, ids, logp, tau, rest)
    e_kl, e_dx = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        on = (ids[t] >= 0) & (ids[t] < V)
        i, lq = ids[t][on], logp[t][on].astype(np.float64)
        z = x64[t] / tau
        p = np.exp(z - z.max())
        p /= p.sum()
        other = np.ones(V, bool)
        other[i] = False
        if not rest:
            lq = lq - (lq.max() + np.log(np.exp(lq - lq.max()).sum()))
        q = np.exp(lq)
        named = np.zeros(V)
        np.add.at(named, i, q)
        assert not rest or abs(1 - q.sum()) > 2.0 ** -40  # whether there is a rest is not a matter of rounding
        p_r = p[other].sum()
        q_r = max(0.0, 1 - q.sum()) if rest and other.any() else 0.0
        Q = q.sum() + q_r
        with np.errstate(invalid="ignore"):  # -inf less -inf
            u = np.where(other, (z[other].max() if other.any() else 0.0) - z, 0.0)
        u = np.where(np.isfinite(u), u, 0.0)
        share = np.where(other & (p_r > 0), p / (p_r or 1.0), 0.0)
        e_o = (share * (9 * H * u + 18 * H)).sum()
        with np.errstate(all="ignore"):
            size = np.where(q > 0, q * (np.abs(lq) + np.abs(np.log(p[i]))), 0.0).sum()
        e_kl[t] = p_r * e_o * q.sum() + H * abs(kl[t])
        if q_r > 0:
            logs = abs(np.log(q_r)) + abs(np.log(p_r))
            size += q_r * logs
            e_kl[t] += (1 - p_r) * e_o * q_r + 2.0 ** -46 * (1 + logs)
        e_kl[t] += 2.0 ** -45 * size
        slack = 2.0 ** -45 * (Q * p_r + q_r) + (2.0 ** -46 if q_r > 0 else 0.0)
        e_dx[t] = np.where(other, share * (abs(Q * p_r - q_r) * (3 * H * u + 12 * H) + max(Q * p_r ** 2, q_r) * e_o + slack),
                           Q * p * p_r * e_o + 4 * H * np.abs(dx[t] * tau) + 2.0 ** -45 * (Q * p + named)) / tau
    c = np.abs(coef)[:, None]
    dx, e_dx = dx * coef[:, None], e_dx * c
    e_dx = np.where(np.isfinite(x64), e_dx + 2.0 ** -126 * (c / tau + 1), 0.0)
    return kl, e_kl, dx, e_dx + torch.finfo(dtype).eps / 2 * (np.abs(dx) + e_dx)


def check(x, ids, logp, tau, rest, coef, rows):
    """Divergence, gradient from its state and step of these rows of the call."""
    T = len(x)
    want, e_kl, dx, e_dx = tight(f64(x[rows]), ids[rows].cpu().numpy(), f64(logp[rows]), tau, rest, f64(coef[rows]), x.dtype)
    kl, state = L.lora_distill_kl(x, ids, logp, tau, rest)
    close(f64(kl[rows]), want, e_kl, "kl")
    close(f64(L.lora_distill_grad(x, ids, state, coef, tau)[rows]), dx, e_dx, "dx")
    loss, kl, got = L.lora_distill_step(x, ids, logp, coef, tau, rest)
    close(f64(kl[rows]), want, e_kl, "kl of the step")
    close(f64(got[rows]), dx, e_dx, "dx of the step")
    total = f64(coef) * f64(kl)
    close(f64(loss), total.sum(), H * abs(total.sum()) + T * 2.0 ** -50 * np.abs(total).sum(), "loss")
    _, _, again = L.lora_distill_step(x, ids, logp, coef, tau, rest, dlogits=x)
    assert again is x and torch.equal(x, got)
    return want, dx, e_dx


# rows by 4 and 8 waves (the gradient's by 16 as well), in pieces of 18000 and of 4000 logits
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("T,V", [(64, 20001), (64, 40000), (120, 130003), (260, 130003), (50, 128256), (3, 128256)])
@pytest.mark.parametrize("above", [25.0, 40.0])
@pytest.mark.parametrize("dtype", [BF, F])
def test_likely_tokens_late_in_a_row(dtype, above, T, V, rest):
    """The likely tokens, the teacher's and one of the others, lie in the last third of a row, far above the rest."""
    note(f"distill late peaks {dtype} {above} {T} {V} {rest}")
    tau, k = (1.0, 0.7)[V % 3 == 0], 6
    g = torch.Generator(device=DEV)
    g.manual_seed(V + T + int(above))
    x = torch.randn(T, V, device=DEV, generator=g) * 0.5
    at = torch.rand(T, V // 3, device=DEV, generator=g).topk(k + 1, 1).indices + (V - V // 3)
    x.scatter_(1, at, (above + torch.rand(T, k + 1, device=DEV, generator=g)) * tau)
    x.scatter_add_(1, at[:, k:], torch.full((T, 1), tau, device=DEV))  # the other one holds about half
    x = x.to(dtype)
    ids = at[:, :k].int().contiguous()
    logp = torch.log_softmax(torch.randn(T, k + 1, device=DEV, generator=g), 1)[:, :k].contiguous()
    coef = 0.5 + torch.rand(T, device=DEV, generator=g)
    check(x, ids, logp, tau, rest, coef, list(range(0, T, max(1, T // 24))))


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("T,V", [(12, 70), (12, 9001), (12, 128256), (260, 80001)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_little_outside_the_teachers_tokens(dtype, T, V, rest):
    """The teacher's tokens hold all but 1e-5 to 1e-22 of the probability; in half of the rows its probabilities sum to
    more than 1, which leaves it no rest."""
    note(f"distill little {dtype} {T} {V} {rest}")
    k = 16
    x, ids, logp = make(T, V, k, dtype, seed=V, std=1.0, noise=0.1)
    ids[2], ids[4] = ids[3], ids[3]
    lead = torch.tensor([22.0, 30.0, 45.0, 60.0], device=DEV).repeat(T // 4)[:, None]
    x.scatter_add_(1, ids.long(), lead.expand(T, k).to(dtype))
    teacher = torch.log_softmax(x.double().gather(1, ids.long()) + 0.01 * torch.randn(T, k, device=DEV), 1)
    more = torch.where(torch.arange(T, device=DEV) // 4 % 2 == 0, 2.0 ** -18, -2.0 ** -18)
    logp = (teacher + torch.log1p(more.double())[:, None]).float()
    total = logp.double().exp().sum(1)
    assert torch.equal(total > 1, more > 0)
    rows = list(range(12))
    want, dx, e_dx = check(x, ids, logp, 1.0, rest, torch.ones(T, device=DEV), rows)
    off = np.ones(dx.shape, bool)
    np.put_along_axis(off, ids[rows].cpu().numpy().astype(np.int64), False, 1)
    # zeros in place of the gradient elsewhere would not pass in any row
    assert ((np.abs(dx) > e_dx) & off).any(1).all()
