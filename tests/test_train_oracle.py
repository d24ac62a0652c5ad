"""Pins of the float64 definitions in oracle/train_oracle.py: derivatives
against central differences, closed forms, and torch's own float64 functions."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as O


def _case(T=9, V=13, seed=0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, V)) * 2
    y = rng.integers(0, V, T)
    y[[1, 4]] = (-100, V)
    return rng, x, y


def _differences(f, x, step=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + step
        up = f(x)
        x[i] = old - step
        g[i] = (up - f(x)) / (2 * step)
        x[i] = old
    return g


def test_token_logp_is_torch_log_softmax():
    _, x, y = _case()
    want = torch.log_softmax(torch.from_numpy(x), 1).numpy()
    got = O.token_logp(x, y)
    for t, v in enumerate(y):
        assert got[t] == (0.0 if v in (-100, 13) else pytest.approx(want[t, v], abs=1e-13))


@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_preference_gradient_is_the_derivative(eps):
    rng, x, y = _case()
    off, ref = [0, 2, 5, 5, 8], rng.normal(size=4) * 3

    def loss(x):
        return O.pref_loss(O.token_logp(x, y), off, ref, 0.3, eps)[0]

    coef = O.pref_loss(O.token_logp(x, y), off, ref, 0.3, eps)[2]
    assert coef[8] == 0.0  # past the last sequence
    assert np.allclose(O.logit_grad(x, y, coef), _differences(loss, x), atol=1e-9)


@pytest.mark.parametrize("kl", [0.0, 0.2])
def test_policy_gradient_is_the_derivative(kl):
    rng, x, y = _case(seed=3)
    lp = O.token_logp(x, y)
    old, ref = lp + rng.normal(size=9) * 0.3, lp + rng.normal(size=9)
    adv, w = rng.normal(size=9), rng.uniform(0.5, 1, 9)
    args = (y, 13, old, adv, w, 0.2, 0.3, ref, kl)

    def loss(x):
        return O.policy_loss(O.token_logp(x, y), *args)[0]

    coef = O.policy_loss(lp, *args)[1]
    assert (coef[[1, 4]] == 0).all() and (kl > 0 or (coef == 0).sum() > 2)  # masked, and some clipped
    assert np.allclose(O.logit_grad(x, y, coef), _differences(loss, x), atol=1e-8)


def test_preference_loss_closed_forms():
    loss, seq, coef = O.pref_loss(np.zeros(4), [0, 2, 4], np.zeros(2), 0.5, 0.0)
    assert loss == pytest.approx(np.log(2)) and (seq == 0).all()
    assert np.allclose(coef, [-0.25, -0.25, 0.25, 0.25])
    assert O.pref_loss([0.0, -1000.0], [0, 1, 2], np.zeros(2), 1.0, 0.0)[0] == 0.0


def test_embedding_gradient_is_the_transpose_of_the_lookup():
    rng = np.random.default_rng(1)
    ids = rng.integers(-2, 12, 40)  # some outside [0, 10)
    table, dy = rng.normal(size=(10, 6)), rng.normal(size=(40, 6))
    left = (O.embed(ids, table, 1.5) * dy).sum()
    assert left == pytest.approx((O.embed_grad(ids, dy, 10, 1.5) * table).sum(), abs=1e-12)
    assert (O.embed(ids, table, 1.5)[(ids < 0) | (ids >= 10)] == 0).all()


def test_adamw_is_torch_adamw():
    rng = np.random.default_rng(2)
    p = rng.normal(size=50)
    w = torch.nn.Parameter(torch.from_numpy(p.copy()))
    opt = torch.optim.AdamW([w], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    m = v = np.zeros(50)
    for t in range(1, 5):
        g = rng.normal(size=50)
        w.grad = torch.from_numpy(g)
        opt.step()
        p, m, v = O.adamw(p, g, m, v, t, 1e-2, 0.8, 0.95, 1e-6, 0.1)
        assert np.allclose(p, w.detach().numpy(), atol=1e-14)


def test_quantise_is_torch_e4m3():
    rng = np.random.default_rng(3)
    x = np.float32(rng.normal(size=4 * 256) * np.exp(rng.normal(size=1024) * 3))
    x[256:512] = 0
    x[512:768] *= 1e-36
    code, scale = O.quantise(x, False)
    assert scale[1] == 0 and scale[2] == 0 and (code[256:768] == 0).all()
    for b in (0, 3):
        q = np.float64(x[b * 256:(b + 1) * 256]) / scale[b]
        # float32 holds q to 24 bits: torch's rounding of it can differ from the float64's at a tie only
        want = torch.from_numpy(np.float32(q)).to(torch.float8_e4m3fn).double().numpy()
        assert (code[b * 256:(b + 1) * 256] != want).mean() < 0.01
        assert np.abs(code[b * 256:(b + 1) * 256]).max() == 448
    assert (O.quantise(np.abs(x), True)[0][x > 1e-25] > 0).all()
