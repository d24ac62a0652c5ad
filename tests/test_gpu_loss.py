"""Token log probabilities, the losses and the gradient of their logits
against the float64 definitions.

Error bounds (H = 2^-24, half a step of float32; d = x - m for a row's largest
logit m). Each exponential: the difference d and the product d * log2(e) (its
constant too) are rounded, which moves the exponent by at most 3 H |d| in
natural units, and the exponential itself by at most 2^-23 (one step). A sum s
of n of them: the terms' own errors, weighted by their shares p, and n / 64 +
64 additions in a row at most (the row is spread over 64 lanes or more), each
within H, with the same again for the running maximum's rescalings:
    err(s) / s <= 3 H sum(p |d|) + 2^-23 + 2 (n / 64 + 64) H  =: S
    err(logp)  <= S + H (|d_y| + 4 |log s| + |logp|)
    err(dx_j)  <= |c| (p_j (3 H |d_j| + 2^-22 + S + 4 H) + 4 H [j = y])
plus half a step of the output's type, and 1e-37 for flushed denormals."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from oracle import train_oracle as O
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
H = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, V, dtype, seed=0, pad=0, shift=0, std=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    buf = torch.randn(T * (V + pad) + shift + 1, device=DEV, generator=g).mul_(std).to(dtype)
    x = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    y = torch.randint(0, V, (T,), device=DEV, dtype=torch.int32, generator=g)
    x[torch.arange(T, device=DEV), y.long()] += 4.0
    y[::5] = torch.tensor([-100, V, -1, 2 ** 31 - 1], device=DEV, dtype=torch.int32).repeat(T)[:len(y[::5])]
    if T == 1:
        y[0] = V // 2
    return x, y


def row_bounds(x64, y):
    """(S, err(logp), the softmax, |d|) by row"""
    V = x64.shape[1]
    d = np.abs(x64 - x64.max(1, keepdims=True))
    p = O.softmax(x64)
    S = 3 * H * (p * d).sum(1) + 2.0 ** -23 + 2 * (V / 64 + 64) * H
    logp = O.token_logp(x64, y)
    dy = d[np.arange(len(y)), np.where(O.masked(y, V), 0, y)]
    return S, S + H * (dy + 4 * np.log(1 / p.max(1)) + np.abs(logp)), p, d


def grad_bounds(x64, y, coef, dtype):
    S, _, p, d = row_bounds(x64, y)
    hit = np.zeros_like(p)
    live = np.flatnonzero(~O.masked(y, x64.shape[1]))
    hit[live, y[live]] = 1
    want = O.logit_grad(x64, y, coef)
    tol = np.abs(coef)[:, None] * (p * (3 * H * d + 2.0 ** -22 + S[:, None] + 4 * H) + 4 * H * hit) + 1e-37
    return want, tol + torch.finfo(dtype).eps / 2 * (np.abs(want) + tol)


def close(got, want, tol, what=""):
    err = np.abs(np.asarray(got, np.float64) - want)
    assert (err <= tol).all(), (what, float((err / np.maximum(tol, 1e-300)).max()))


SHAPES = [(1, 1, 0, 0), (1, 2, 0, 0), (5, 7, 0, 1), (3, 64, 0, 0), (9, 1023, 1, 1), (40, 1024, 0, 0), (2, 32003, 0, 0),
          (6, 40000, 5, 3), (1, 128256, 0, 0), (2100, 515, 0, 0), (70, 8209, 0, 0), (300, 20011, 0, 1)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V,pad,shift", SHAPES)
def test_logp_and_gradient(dtype, T, V, pad, shift):
    note(f"logp {dtype} {T} {V} {pad} {shift}")
    x, y = make(T, V, dtype, T + V, pad, shift)
    x64, yn = f64(x), y.cpu().numpy()
    logp, stats = L.lora_token_logp(x, y)
    S, tol, p, _ = row_bounds(x64, yn)
    off = O.masked(yn, V)
    assert (f64(logp)[off] == 0).all()
    close(f64(logp), O.token_logp(x64, yn), tol, "logp")
    close(f64(stats)[:, 0], np.where(off, 0, x64.max(1)), 0, "m")
    close(f64(stats)[:, 1], np.where(off, 1, 1 / p.max(1)), S / p.max(1), "s")

    coef = torch.randn(T, device=DEV)
    coef[off] = float("nan")  # a masked token's is not used
    c64 = np.where(off, 0, f64(coef))
    want, tol = grad_bounds(x64, yn, c64, dtype)
    buf = torch.full((T * (V + pad) + shift + 1,), 9.0, device=DEV, dtype=dtype)
    dx = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    assert L.lora_logit_grad(x, y, stats, coef, dlogits=dx) is dx
    close(f64(dx), want, tol, "dx")
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V] = False
    assert bool((buf[rest] == 9.0).all())
    # rows that start elsewhere than the logits', the factor on the device, and in place
    out = torch.empty(T * V + 3, device=DEV, dtype=dtype)[3:].view(T, V)
    two = torch.full((), 2.0, device=DEV)
    L.lora_logit_grad(x, y, stats, coef, grad_out=two, scale=0.25, dlogits=out)
    want, tol = grad_bounds(x64, yn, 0.5 * c64, dtype)
    close(f64(out), want, tol, "scaled dx")
    L.lora_logit_grad(x, y, stats, coef, dlogits=x)
    assert torch.equal(x, dx)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("V", [40, 9001])
def test_infinities_and_masked_vocabulary(dtype, V):
    note(f"infinities {dtype} {V}")
    x, _ = make(8, V, dtype, 3)
    low = torch.finfo(dtype).min
    y = torch.tensor([2, 2, 2, 2, 2, -1, 2, 3], dtype=torch.int32, device=DEV)
    x[0, 5:] = -float("inf")          # most of the vocabulary masked
    x[1, 5:] = low                    # the same with the type's lowest value
    x[2] = -float("inf")              # a row with nothing left: NaN
    x[3] = low                        # every value the lowest: uniform
    x[4, 7] = float("inf")            # NaN, as the formula gives
    x[5] = float("nan")               # masked by its target: not read
    x[6, V - 1] = float("nan")
    x[7] = -float("inf")
    x[7, 3] = low                     # one finite value: probability 1
    logp, stats = L.lora_token_logp(x, y)
    dx = L.lora_logit_grad(x, y, stats, torch.ones(8, device=DEV))
    a = f64(x)[:2, :5]
    S, tol, _, _ = row_bounds(a, np.array([2, 2]))
    extra = 2 * (V / 64 + 64) * H
    close(f64(logp)[:2], O.token_logp(a, [2, 2]), tol + extra)
    want, tol = grad_bounds(a, np.array([2, 2]), np.ones(2), dtype)
    close(f64(dx)[:2, :5], want, tol + extra)
    assert not dx[:2, 5:].any()
    close(f64(logp)[3], -np.log(V), (2 * (V / 64 + 64) + 8 * np.log(V)) * H)
    close(f64(dx)[3], np.where(np.arange(V) == 2, 1, 0) - 1 / V,
          (extra + 8 * H) / V + 4 * H + torch.finfo(dtype).eps / 2)
    for r in (2, 4, 6):
        assert np.isnan(f64(logp)[r]) and torch.isnan(dx[r]).all()
    assert logp[5] == 0 and not dx[5].any()
    assert logp[7] == 0 and not dx[7].any()


def test_rows_beyond_32_bit_offsets():
    note("logits beyond 2^31 elements")
    T, V = 40_000, 65_000  # 2.6e9 elements
    x = torch.zeros(T, V, dtype=BF, device=DEV)
    y = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    rows = [0, 36_000, T - 1]
    for r in rows:
        x[r] = torch.randn(V, device=DEV).to(BF)
        y[r] = V - 1 - r % 7
    logp, stats = L.lora_token_logp(x, y)
    x64, yn = f64(x[rows]), y[rows].cpu().numpy()
    close(f64(logp[rows]), O.token_logp(x64, yn), row_bounds(x64, yn)[1])
    L.lora_logit_grad(x, y, stats, torch.ones(T, device=DEV), dlogits=x)
    want, tol = grad_bounds(x64, yn, np.ones(3), BF)
    close(f64(x[rows]), want, tol)
    assert not x[35_000:36_000].any()


def offsets(T, pairs, rng):
    cuts = np.sort(rng.integers(0, T + 1, 2 * pairs - 1))
    return np.concatenate([[0], cuts, [T]]).astype(np.int32)


@pytest.mark.parametrize("T,pairs,eps", [(0, 1, 0.0), (1, 1, 0.1), (64, 3, 0.0), (1000, 40, 0.2), (5000, 1, 0.05)])
def test_preference_loss(T, pairs, eps):
    note(f"pref_loss {T} {pairs} {eps}")
    rng = np.random.default_rng(T + pairs)
    logp = torch.from_numpy(np.float32(-rng.exponential(2.0, T))).to(DEV)
    off = offsets(T, pairs, rng)
    if pairs == 3:
        off[0], off[-1] = 3, T - 4  # tokens outside every sequence
    seq = np.array([f64(logp)[a:b].sum() for a, b in zip(off[:-1], off[1:])])
    ref = torch.from_numpy(np.float32(seq + rng.normal(size=2 * pairs) * 5)).to(DEV)
    loss, s, coef = L.lora_pref_loss(logp, torch.from_numpy(off).to(DEV), ref, 0.1, eps)
    e32 = np.float64(np.float32(eps))
    want = O.pref_loss(f64(logp), off, f64(ref), np.float64(np.float32(0.1)), e32)
    for got, w in zip((loss, s, coef), want):  # float64 inside, rounded once
        close(f64(got), w, np.abs(w) * 1.01 * H + 1e-13)


def test_preference_loss_extremes():
    note("pref_loss extremes")
    off = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device=DEV)
    lp = torch.tensor([0.0, -1e6, -float("inf"), 0.0], device=DEV)
    zero = torch.zeros(4, device=DEV)
    loss, _, coef = L.lora_pref_loss(lp[:2], off[:3], zero[:2], 1.0)
    assert loss == 0 and not coef.any()
    loss, _, coef = L.lora_pref_loss(lp[2:], off[:3], zero[:2], 1.0)
    assert loss == float("inf") and coef.tolist() == [-1.0, 1.0]
    loss, _, coef = L.lora_pref_loss(lp[:2], off[:3], torch.tensor([-float("inf"), 0.0], device=DEV), 1.0)
    assert loss == 0 and not coef.any()  # z = +inf, no smoothing
    assert torch.isnan(L.lora_pref_loss(lp * float("nan"), off, zero, 1.0)[0])
    # offsets outside [0, T] are clamped to it
    wild = torch.tensor([-5, 1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    loss, s, coef = L.lora_pref_loss(torch.tensor([-1.0, -2.0], device=DEV), wild, zero[:2], 1.0)
    assert s.tolist() == [-1.0, -2.0] and coef[0] < 0 < coef[1]


@pytest.mark.parametrize("T,kl", [(0, 0.0), (1, 0.1), (77, 0.0), (3000, 0.05)])
def test_policy_loss(T, kl):
    note(f"policy_loss {T} {kl}")
    rng = np.random.default_rng(T)
    lp = -rng.exponential(2.0, T)
    lp, old, ref, adv, w = (torch.from_numpy(np.float32(a)).to(DEV) for a in (
        lp, lp + rng.normal(size=T) * 0.3, lp + rng.normal(size=T), rng.normal(size=T),
        rng.uniform(0, 2 / max(T, 1), T)))
    y = torch.from_numpy(np.where(rng.random(T) < 0.2, -100, 5).astype(np.int32)).to(DEV)
    off = O.masked(y.cpu().numpy(), 10)
    for t in (old, ref, adv, w):
        t[torch.from_numpy(off).to(DEV)] = float("nan")  # a masked token's inputs are not used
    low, high, klf = (np.float64(np.float32(v)) for v in (0.2, 0.3, kl))
    loss, coef = L.lora_policy_loss(lp, y, 10, old, adv, w, 0.2, 0.3, ref if kl else None, kl)
    want_loss, want = O.policy_loss(f64(lp), y.cpu().numpy(), 10, f64(old), f64(adv), f64(w), low, high, f64(ref), klf)
    # per token: differences, exponentials of one step (2^-23), products: 12 roundings of the terms' magnitudes
    live = ~off
    r = np.exp(f64(lp) - f64(old))
    k = f64(ref) - f64(lp)
    mag = np.where(live, f64(w) * (np.abs(r * f64(adv)) * (1 + np.abs(f64(lp))) + kl * (np.exp(k) + 2 * np.abs(k) + 2)
                                   * (1 + np.abs(f64(lp)))), 0)
    # a token within rounding of the clip's border may fall to either side
    border = live & (np.minimum(np.abs(r - (1 - low)), np.abs(r - (1 + high))) < 1e-5)
    close(f64(coef)[~border], want[~border], 12 * H * mag[~border])
    close(f64(loss), want_loss, 12 * H * mag.sum() + H * abs(want_loss))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V,pairs", [(0, 50, 1), (5, 50, 1), (33, 1000, 2), (150, 5003, 4), (20, 128256, 1),
                                       (2500, 300, 3), (1100, 9000, 2)])
def test_preference_step(dtype, T, V, pairs):
    note(f"pref_step {dtype} {T} {V} {pairs}")
    rng = np.random.default_rng(T + V)
    x, y = make(T, V, dtype, T + V)
    if T > 40:
        y[10:30] = -100
    off = offsets(T, pairs, rng)
    x64, yn = f64(x), y.cpu().numpy()
    logp64 = O.token_logp(x64, yn)
    seq = np.array([logp64[a:b].sum() for a, b in zip(off[:-1], off[1:])])
    ref = torch.from_numpy(np.float32(seq + rng.normal(size=2 * pairs) * 5)).to(DEV)
    off_d = torch.from_numpy(off).to(DEV)
    loss, s, logp, dx = L.lora_pref_step(x, y, off_d, ref, 0.1, 0.1, grad_scale=2.0)
    # the separate calls give the same values (the log probabilities bit for bit)
    lp2, stats = L.lora_token_logp(x, y)
    loss2, s2, coef = L.lora_pref_loss(lp2, off_d, ref, 0.1, 0.1)
    assert torch.equal(logp, lp2) and torch.equal(loss, loss2) and torch.equal(s, s2)
    b, e = np.float64(np.float32(0.1)), np.float64(np.float32(0.1))
    want_loss, want_seq, want_coef = O.pref_loss(logp64, off, f64(ref), b, e)
    err_lp = row_bounds(x64, yn)[1] if T else np.zeros(0)
    err_seq = np.array([err_lp[a:c].sum() for a, c in zip(off[:-1], off[1:])]) + np.abs(want_seq) * 1.01 * H
    close(f64(s), want_seq, err_seq)
    # the loss moves by at most beta per unit of a sequence's log probability, its slope by a quarter of that
    dz = b * err_seq.sum()
    close(f64(loss), want_loss, dz + H * abs(want_loss) + 1e-12)
    if T == 0:
        return
    moved = np.abs(want_coef) * 1.01 * H + b / pairs * dz / 4 * (want_coef != 0)
    close(f64(coef), want_coef, moved)
    want, tol = grad_bounds(x64, yn, 2 * want_coef, dtype)
    p = O.softmax(x64)
    hit = np.abs(O.logit_grad(x64, yn, np.ones(T)))
    close(f64(dx), want, tol + 2 * moved[:, None] * np.maximum(hit, p) * 1.01)
    assert not dx[torch.from_numpy(O.masked(yn, V)).to(DEV)].any()
    L.lora_pref_step(x, y, off_d, ref, 0.1, 0.1, grad_scale=2.0, dlogits=x)  # in place
    assert torch.equal(x, dx)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V,kl,pad,shift", [(0, 50, 0.0, 0, 0), (1, 1, 0.1, 0, 0), (7, 50, 0.0, 0, 0),
                                              (33, 1001, 0.1, 2, 1), (20, 128256, 0.04, 0, 0), (3, 131071, 0.1, 0, 0),
                                              (1100, 9000, 0.1, 0, 0), (2500, 301, 0.0, 0, 0), (1030, 40003, 0.1, 0, 0)])
def test_policy_step(dtype, T, V, kl, pad, shift):
    note(f"policy_step {dtype} {T} {V} {kl} {pad} {shift}")
    rng = np.random.default_rng(T + V)
    x, y = make(T, V, dtype, T + V, pad, shift)
    lp, stats = L.lora_token_logp(x, y)
    old, ref = lp + torch.randn(T, device=DEV) * 0.3, lp + torch.randn(T, device=DEV) * 0.5
    adv, w = torch.randn(T, device=DEV), torch.rand(T, device=DEV)
    masked = torch.from_numpy(O.masked(y.cpu().numpy(), V)).to(DEV)
    for t in (old, ref, adv, w):
        t[masked] = float("nan")
    args = (old, adv, w, 0.2, 0.3, ref if kl else None, kl)
    loss, logp, dx = L.lora_policy_step(x, y, *args, grad_scale=0.5)
    if T == 0:
        assert loss == 0 and dx.shape == (0, V)
        return
    # log probabilities and loss within the rounding of either's sums
    x64, yn = f64(x), y.cpu().numpy()
    close(f64(logp), O.token_logp(x64, yn), row_bounds(x64, yn)[1])
    loss2, coef = L.lora_policy_loss(logp, y, V, *args)
    assert torch.equal(loss, loss2)
    # a coefficient is that of the log probability returned (within its own rounding)
    c64 = f64(coef)
    want, tol = grad_bounds(x64, yn, 0.5 * c64, dtype)
    close(f64(dx), want, tol + 8 * H * np.abs(want))
    assert not dx[masked].any()
    # the same bits again, then in place
    loss3, logp3, dx3 = L.lora_policy_step(x, y, *args, grad_scale=0.5)
    assert torch.equal(dx, dx3) and torch.equal(logp, logp3) and torch.equal(loss, loss3)
    L.lora_policy_step(x, y, *args, grad_scale=0.5, dlogits=x)
    assert torch.equal(x, dx)


def test_policy_step_gradient_is_the_derivative():
    """Central differences of the float64 loss along random directions at the
    kernel's logits (float32, away from the clip's borders)."""
    note("policy_step differences")
    T, V = 24, 300
    x, y = make(T, V, F, 8)
    lp, _ = L.lora_token_logp(x, y)
    old = lp + torch.where(torch.arange(T, device=DEV) % 2 == 0, 0.05, 0.6)  # inside, and clipped for A > 0... or not
    ref, adv, w = lp + 0.3, torch.randn(T, device=DEV), torch.rand(T, device=DEV) / T
    _, _, dx = L.lora_policy_step(x, y, old, adv, w, 0.2, 0.3, ref, 0.1)
    x64, yn = f64(x), y.cpu().numpy()
    rng = np.random.default_rng(0)

    def f(z):
        return O.policy_loss(O.token_logp(z, yn), yn, V, f64(old), f64(adv), f64(w), 0.2, 0.3, f64(ref), 0.1)[0]

    for _ in range(5):
        e = rng.normal(size=x64.shape)
        d = (f(x64 + 1e-5 * e) - f(x64 - 1e-5 * e)) / 2e-5
        # the gradient's own roundings (about 2^-20 of it) and the differences' (1e-16 / 1e-5, and their second order)
        assert abs(d - (f64(dx) * e).sum()) <= 2.0 ** -20 * np.abs(f64(dx) * e).sum() + 1e-8
