"""Distillation from a teacher's top tokens against the float64 definitions.

Error bounds (H = 2^-24, half a step of float32). The others' exponentials are
float32, relative to the largest of them or to the largest of a run of at least
4096 of the row's columns (of all, in a shorter row), which lies reach below at
most, and never more than 64 binary orders; u is an other logit's distance (over tau) below the largest of the others:
    e_j = 3 H (u_j + reach) + 2^-23 + 16 H     (relative, of one exponential)
    e_o = sum of their shares' e_j             (relative, of the others' sum)
Everything of the teacher's tokens is float64 (2^-50 of the terms' magnitudes):
    err(kl) <= p_r e_o sum q + (1 - p_r) e_o q_r + H |kl| + 2^-45 (1 + sum q (|log q| + |log p|))
    tau err(dx_j) <= t_j (|F| (e_j + 8 H) + Q p_r e_o)   elsewhere, F = Q p_r - q_r, t = p / p_r
                     Q p_k p_r e_o + 4 H |b_k|            at the teacher's tokens
times |coef|, and half a step of the output's type. An exponential below 2^-126 may
be 0, which counts |coef F| / tau times at most, and so may an output below it."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from oracle import train_oracle as O
from tests.gpu_util import DEV, note
from tests.test_gpu_top import BF, F, H, close, f64

pytestmark = pytest.mark.gpu


def make(T, V, k, dtype, tau=1.0, seed=0, pad=0, shift=0, std=2.0, noise=0.7):
    """Logits, and the top k tokens of a teacher that mostly agrees; entries and whole rows without a token."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    buf = torch.randn(T * (V + pad) + shift + 1, device=DEV, generator=g).mul_(std).to(dtype)
    x = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    x[torch.arange(T, device=DEV), torch.randint(0, V, (T,), device=DEV, generator=g)] += 6.0
    teacher = (x.double() + torch.randn(T, V, device=DEV, generator=g) * noise) / tau
    lq, at = torch.log_softmax(teacher, 1).topk(min(k, V), 1)
    ids = torch.full((T, k), -1, device=DEV, dtype=torch.int32)
    logp = torch.full((T, k), -float("inf"), device=DEV)
    ids[:, :at.shape[1]], logp[:, :at.shape[1]] = at.int(), lq.float()
    if T > 2:
        ids[2] = torch.tensor([-1, V, -100, 2 ** 31 - 1], dtype=torch.int32, device=DEV).repeat(k)[:k]
        logp[2] = float("nan")  # not used
    if T > 4:
        ids[4, 1::2] = V + 3
    return x, ids, logp


def bounds(x64, ids, logp, tau, rest, coef, dtype):
    """(kl, err(kl), dlogits, err(dlogits))"""
    T, V = x64.shape
    kl, dx = O.distill(x64, ids, logp, tau, rest)
    e_kl, e_dx = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        on = (ids[t] >= 0) & (ids[t] < V)
        if not on.any():
            continue
        i, lq = ids[t][on], logp[t][on].astype(np.float64)
        z = x64[t] / tau
        p = np.exp(z - z.max())
        p /= p.sum()
        other = np.ones(V, bool)
        other[i] = False
        if not rest:
            lq = lq - (lq.max() + np.log(np.exp(lq - lq.max()).sum()))
        q = np.exp(lq)
        p_r = p[other].sum()
        q_r = max(0.0, 1 - q.sum()) if rest and other.any() else 0.0
        Q = q.sum() + q_r
        far = 0.0
        if V > 4096 and other.any():
            hidden = np.where(other, z, -np.inf)
            low = hidden[:V // 2048 * 2048].reshape(-1, 2048).max(1).min()
            far = min(hidden.max() - low, 64 * np.log(2)) if np.isfinite(low) else 64 * np.log(2)
        u = np.where(other, (z[other].max() if other.any() else 0.0) - z, 0.0)
        u = np.where(np.isfinite(u), u, 0.0)
        e = 3 * H * (u + far) + 2.0 ** -23 + 16 * H
        share = np.where(other & (p_r > 0), p / (p_r or 1.0), 0.0)
        e_o = (share * e).sum()
        with np.errstate(all="ignore"):
            size = np.where(q > 0, q * (np.abs(lq) + np.abs(np.log(p[i]))), 0.0).sum()
            size += q_r * (abs(np.log(q_r)) + abs(np.log(p_r))) if q_r > 0 else 0.0
            e_kl[t] = p_r * e_o * q.sum() + (1 - p_r) * e_o * q_r + H * abs(kl[t]) + 2.0 ** -45 * (1 + size)
        e_dx[t] = np.where(other, share * (abs(Q * p_r - q_r) * (e + 8 * H) + Q * p_r * e_o),
                           Q * p * p_r * e_o + 4 * H * np.abs(dx[t] * tau)) / tau
        e_dx[t] = np.where((e_dx[t] > 0) | ~other, e_dx[t] + 2.0 ** -45 / tau, 0.0)
    live = ((ids >= 0) & (ids < V)).any(1)
    dx, e_dx = dx * coef[:, None], e_dx * np.abs(coef)[:, None]
    some = ((e_dx > 0) | np.isfinite(x64)) & live[:, None]
    e_dx = np.where(some, e_dx + 2.0 ** -126 * (np.abs(coef)[:, None] / tau + 1), 0.0)
    return kl, e_kl, dx, e_dx + torch.finfo(dtype).eps / 2 * (np.abs(dx) + e_dx)


SHAPES = [(1, 1, 1, 0, 0), (1, 2, 1, 0, 0), (5, 7, 3, 0, 1), (3, 64, 64, 0, 0), (9, 1023, 20, 1, 1), (40, 1024, 5, 0, 0),
          (3, 32003, 256, 0, 0), (6, 40000, 64, 5, 3), (1, 128256, 32, 0, 0), (700, 515, 8, 0, 0), (70, 8209, 33, 0, 0),
          (60, 20011, 16, 0, 1), (7, 131, 200, 0, 0), (5, 131071, 100, 0, 0), (4, 200003, 64, 0, 0)]


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V,k,pad,shift", SHAPES)
def test_divergence_and_gradient(dtype, rest, T, V, k, pad, shift):
    note(f"distill {dtype} {rest} {T} {V} {k} {pad} {shift}")
    tau = (1.0, 0.7, 2.0)[V % 3]
    x, ids, logp = make(T, V, k, dtype, tau, T + V, pad, shift)
    before = x.clone()
    coef = torch.randn(T, device=DEV)
    live = ((ids >= 0) & (ids < V)).any(1)
    coef[~live] = float("nan")  # a masked token's is not used
    x64, i64, l64 = f64(x), ids.cpu().numpy(), f64(logp)
    c64 = np.nan_to_num(f64(coef))
    want, e_kl, dx, e_dx = bounds(x64, i64, l64, tau, rest, c64, dtype)
    kl, state = L.lora_distill_kl(x, ids, logp, tau, rest)
    close(f64(kl), want, e_kl, "kl")
    assert torch.equal(x, before) and state.shape == (T, k + 2)
    buf = torch.full((T * (V + pad) + shift + 1,), 9.0, device=DEV, dtype=dtype)
    out = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    assert L.lora_distill_grad(x, ids, state, coef, tau, dlogits=out) is out
    close(f64(out), dx, e_dx, "dx")
    left = torch.ones_like(buf, dtype=torch.bool)
    left[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V] = False
    assert bool((buf[left] == 9.0).all())
    # the factor on the device, rows that start elsewhere
    other = torch.empty(T * V + 3, device=DEV, dtype=dtype)[3:].view(T, V)
    L.lora_distill_grad(x, ids, state, coef, tau, grad_out=torch.full((), -2.0, device=DEV), scale=0.5, dlogits=other)
    close(f64(other), -dx, e_dx, "scaled")
    # the step, whose masked tokens' weights are not used either
    weights = torch.where(live, coef, 0.5)
    loss, kl2, dx2 = L.lora_distill_step(x, ids, logp, weights, tau, rest, grad_scale=1.0)
    close(f64(kl2), want, e_kl, "kl of the step")
    close(f64(dx2), dx, e_dx, "dx of the step")
    total = (c64 * want).sum()
    close(f64(loss), total, (np.abs(c64) * e_kl).sum() + H * (abs(total) + np.abs(c64 * want).sum()), "loss")
    loss3, kl3, dx3 = L.lora_distill_step(x, ids, logp, weights, tau, rest)
    assert torch.equal(loss, loss3) and torch.equal(kl2, kl3) and torch.equal(dx2, dx3)
    _, _, dx4 = L.lora_distill_step(x, ids, logp, weights, tau, rest, dlogits=x)
    assert dx4 is x and torch.equal(x, dx2)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("V", [60, 9001, 140000])
def test_masked_vocabularies_and_undefined_rows(dtype, V):
    note(f"distill undefined {dtype} {V}")
    x, ids, logp = make(10, V, 6, dtype, seed=3)
    ids[2], logp[2] = ids[3], logp[3]
    ids[4], logp[4] = ids[3], logp[3]
    low = torch.finfo(dtype).min
    named = torch.zeros(10, V, dtype=torch.bool, device=DEV).scatter_(1, ids.clamp(0, V - 1).long(), True)
    x[0] = -float("inf")                                    # nothing left: NaN
    x[1, V - 1 if not named[1, V - 1] else 0] = float("inf")
    x[2, ids[2, 1].long()] = float("nan")
    x[3, V // 3 if not named[3, V // 3] else V // 3 + 7] = float("nan")
    x[4] = float("nan")
    ids[4] = -1                                             # masked: not read
    x[5] = torch.where(named[5], x[5], -float("inf"))       # only the teacher's tokens left: the rest is infinitely off
    x[6] = torch.where(named[6], x[6], low)                 # the same with the lowest value: finitely off
    x[7, ids[7, 0].long()] = -float("inf")                  # a token of the teacher without probability
    x[8] = torch.where(named[8], -float("inf"), x[8])       # all of them
    x[9, V // 2:] = torch.where(named[9, V // 2:], x[9, V // 2:], -float("inf"))  # half a vocabulary
    one = torch.ones(10, device=DEV)
    kl, state = L.lora_distill_kl(x, ids, logp, 1.0, True)
    dx = L.lora_distill_grad(x, ids, state, one, 1.0)
    assert torch.isnan(kl[:4]).all() and torch.isnan(dx[:4]).all()
    assert kl[4] == 0 and not dx[4].any()
    assert torch.isposinf(kl[[5, 7, 8]]).all()
    x64, i64, l64 = f64(x), ids.cpu().numpy(), f64(logp)
    want, e_kl, wx, ex = bounds(x64[[6, 9]], i64[[6, 9]], l64[[6, 9]], 1.0, True, np.ones(2), dtype)
    close(f64(kl)[[6, 9]], want, e_kl)
    close(f64(dx)[9:], wx[1:], ex[1:])
    assert torch.isfinite(dx[5:]).all()
    assert not dx[5][~named[5]].any() and not dx[9, V // 2:][~named[9, V // 2:]].any()
    # without the rest the others do not count
    kl, state = L.lora_distill_kl(x, ids, logp, 1.0, False)
    dx = L.lora_distill_grad(x, ids, state, one, 1.0)
    assert torch.isnan(kl[:4]).all() and torch.isnan(dx[:4]).all()
    assert torch.isposinf(kl[7:9]).all()
    rows = [5, 6, 9]
    want, e_kl, wx, ex = bounds(x64[rows], i64[rows], l64[rows], 1.0, False, np.ones(3), dtype)
    close(f64(kl)[rows], want, e_kl)
    close(f64(dx)[rows], wx, ex)
    # a weight of zero drops what is infinite or undefined
    weights = torch.zeros(10, device=DEV)
    weights[9] = 2.0
    loss, kl, dx = L.lora_distill_step(x, ids, logp, weights, 1.0, False)
    assert float(loss) == 2 * float(kl[9]) and not dx[:9].any()


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("V", [40, 5000, 128256])
def test_tokens_named_twice_and_in_any_order(dtype, rest, V):
    note(f"distill twice {dtype} {rest} {V}")
    x, ids, logp = make(3, V, 24, dtype, seed=V)
    ids[2], logp[2] = ids[1], logp[1]
    ids[0, 5], ids[0, 9], ids[0, 23] = ids[0, 1], ids[0, 1], ids[0, 2]
    ids[1] = ids[1].flip(0)
    logp[1] = logp[1].flip(0)
    ids[2, 1:] = ids[2, 0]  # one token, again and again
    logp[2] = -4.0
    x64, i64, l64 = f64(x), ids.cpu().numpy(), f64(logp)
    coef = torch.tensor([1.0, -2.0, 0.5], device=DEV)
    want, e_kl, dx, e_dx = bounds(x64, i64, l64, 1.0, rest, f64(coef), dtype)
    loss, kl, got = L.lora_distill_step(x, ids, logp, coef, 1.0, rest)
    close(f64(kl), want, e_kl)
    close(f64(got), dx, e_dx)
    kl, state = L.lora_distill_kl(x, ids, logp, 1.0, rest)
    close(f64(kl), want, e_kl)
    close(f64(L.lora_distill_grad(x, ids, state, coef)), dx, e_dx)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("V", [70, 128256])
def test_little_outside_the_teachers_tokens(dtype, V):
    """The teacher's tokens hold all but 1e-4 to 1e-20 of the probability: what is left keeps its precision."""
    note(f"distill little {dtype} {V}")
    T, k = 4, 16
    x, ids, logp = make(T, V, k, dtype, seed=V, std=1.0, noise=0.1)
    ids[2], logp[2] = ids[3], logp[3]
    lead = torch.tensor([22.0, 30.0, 45.0, 60.0], device=DEV)
    x.scatter_add_(1, ids.clamp(0, V - 1).long(), lead[:, None].expand(T, k).to(dtype))
    teacher = torch.log_softmax(x.double() + 0.01 * torch.randn(T, V, device=DEV), 1)
    logp = teacher.gather(1, ids.clamp(0, V - 1).long()).float()
    x64, i64, l64 = f64(x), ids.cpu().numpy(), f64(logp)
    want, e_kl, dx, e_dx = bounds(x64, i64, l64, 1.0, True, np.ones(T), dtype)
    _, kl, got = L.lora_distill_step(x, ids, logp, torch.ones(T, device=DEV), 1.0, True)
    close(f64(kl), want, e_kl)
    close(f64(got), dx, e_dx)


@pytest.mark.parametrize("rest", [True, False])
def test_gradient_against_differences(rest):
    note("distill gradient by differences")
    T, V, tau, eps = 6, 400, 0.8, 2.0 ** -6
    x, ids, logp = make(T, V, 12, F, tau, 5)
    one = torch.ones(T, device=DEV)
    dx = f64(L.lora_distill_step(x, ids, logp, one, tau, rest)[2])
    u = torch.randn(T, V, device=DEV)
    diff = (f64(L.lora_distill_kl(x + eps * u, ids, logp, tau, rest)[0])
            - f64(L.lora_distill_kl(x - eps * u, ids, logp, tau, rest)[0])) / (2 * eps)
    # third derivatives of two log sums: eps^2 / 6 |u / tau|^3 each, |u| below 5; the values' 2^-20 over eps
    tol = 2 * eps ** 2 * (5 / tau) ** 3 / 6 + 2.0 ** -18 / eps
    assert (np.abs((dx * f64(u)).sum(1) - diff) <= tol).all()


def test_a_teachers_own_tokens():
    """A teacher's pass and the distillation from it, as they are used: the same logits have no divergence."""
    note("distill from alternatives")
    T, V, k, tau = 50, 32003, 40, 2.0
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    teacher = (torch.randn(T, V, device=DEV, generator=g) * 3).to(BF)
    y = torch.randint(0, V, (T,), device=DEV, dtype=torch.int32, generator=g)
    y[:7] = -100
    _, _, ids, logp, _ = L.lora_token_top(teacher, y, k, tau)
    student = (teacher.float() + torch.randn(T, V, device=DEV, generator=g)).to(BF)
    w = torch.full((T,), tau * tau / 43, device=DEV)
    c64 = np.where(np.arange(T) < 7, 0, f64(w))
    for x in (student, teacher):
        want, e_kl, dx, e_dx = bounds(f64(x), ids.cpu().numpy(), f64(logp), tau, True, c64, BF)
        loss, kl, got = L.lora_distill_step(x, ids, logp, w, tau)
        close(f64(kl), want, e_kl)
        close(f64(got), dx, e_dx)
        close(f64(loss), (c64 * want).sum(), (c64 * e_kl).sum() + 2 * H * (c64 * np.abs(want)).sum())
        assert not kl[:7].any() and not got[:7].any()


def test_rows_beyond_32_bit_offsets():
    note("distill beyond 2^31 elements")
    T, V, k = 40_000, 65_000, 3  # 2.6e9 elements
    x = torch.zeros(T, V, dtype=BF, device=DEV)
    ids = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    logp = torch.full((T, k), -1.5, device=DEV)
    rows = [0, 36_000, T - 1]
    for r in rows:
        x[r].normal_()
        ids[r] = torch.tensor([V - 1, 5, 40_000], device=DEV)
    at = torch.tensor(rows, device=DEV)
    want, e_kl, dx, e_dx = bounds(f64(x[at]), ids[at].cpu().numpy(), f64(logp[at]), 1.0, True, np.ones(3), BF)
    loss, kl, got = L.lora_distill_step(x, ids, logp, torch.ones(T, device=DEV), 1.0, True, dlogits=x)
    close(f64(kl[at]), want, e_kl)
    close(f64(got[at]), dx, e_dx)
    assert not kl[1:36_000].any() and not got[1].any() and not got[T - 2].any()


def test_replayed_graph_and_other_stream():
    note("distill in a graph")
    T, V, k = 33, 20011, 12
    x, ids, logp = make(T, V, k, BF, seed=5)
    w = torch.rand(T, device=DEV)
    ws = torch.empty(L.load_library().lora_distill_workspace_bytes(T, V, k), dtype=torch.uint8, device=DEV)

    def step():
        kl, state = L.lora_distill_kl(x, ids, logp, workspace=ws)
        return *L.lora_distill_step(x, ids, logp, w, workspace=ws), kl, L.lora_distill_grad(x, ids, state, w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(4):
        for t, new in zip((x, ids, logp), make(T, V, k, BF, seed=20 + seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        ws.fill_(255)
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), seed
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))


def test_empty_inputs():
    note("distill of nothing")
    i, f = torch.int32, torch.float32
    x = torch.empty(0, 50, device=DEV)
    loss, kl, dx = L.lora_distill_step(x, torch.empty(0, 3, dtype=i, device=DEV), torch.empty(0, 3, device=DEV),
                                       torch.empty(0, device=DEV))
    assert float(loss) == 0 and kl.shape == (0,) and dx.shape == (0, 50)
    x = torch.empty(4, 0, device=DEV)
    loss, kl, dx = L.lora_distill_step(x, torch.zeros(4, 3, dtype=i, device=DEV), torch.zeros(4, 3, device=DEV),
                                       torch.ones(4, device=DEV))
    assert float(loss) == 0 and not kl.any() and dx.shape == (4, 0)
