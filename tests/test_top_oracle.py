"""The float64 definitions of entropy, alternatives and distillation against
differences and identities that hold without them."""
import numpy as np
import pytest

from oracle import train_oracle as O


def rows(T=5, V=23, seed=0):
    return np.random.default_rng(seed).normal(0, 2, (T, V))


@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_entropy_and_alternatives(tau):
    x = rows()
    y = np.array([3, -1, 22, 23, 0])
    logp, entropy, ids, top, stats = O.token_top(x, y, 30, tau)
    p = O.softmax(x / tau)
    for t in (0, 2, 4):
        assert logp[t] == pytest.approx(np.log(p[t, y[t]]), rel=1e-12)
        assert entropy[t] == pytest.approx(-(p[t] * np.log(p[t])).sum(), rel=1e-12)
        assert (np.diff(x[t, ids[t, :23]]) <= 0).all() and sorted(ids[t, :23]) == list(range(23))
        assert np.exp(top[t]).sum() == pytest.approx(1.0, rel=1e-12)
        assert stats[t, 0] == x[t].max() and 1 / (1 + stats[t, 1]) == pytest.approx(p[t].max(), rel=1e-12)
        assert (ids[t, 23:] == -1).all() and np.isneginf(top[t, 23:]).all()
    for t in (1, 3):
        assert logp[t] == entropy[t] == 0 and (ids[t] == -1).all() and np.isneginf(top[t]).all()


def test_ties_go_to_the_lowest_column():
    x = np.array([[1.0, 5.0, 5.0, -0.0, 0.0, 5.0]])
    assert O.token_top(x, None, 6, 1.0)[2].tolist() == [[1, 2, 5, 0, 3, 4]]


@pytest.mark.parametrize("tau", [0.5, 2.0])
def test_gradient_of_log_probability_and_entropy(tau):
    x, y = rows(), np.array([3, 7, 22, -1, 0])
    rng = np.random.default_rng(1)
    g, h = rng.normal(size=5), rng.normal(size=5)

    def loss(v):
        logp, entropy, *_ = O.token_top(v, y, 0, tau)
        return (g * logp + h * entropy).sum()

    dx = O.token_top_grad(x, y, g, h, tau)
    for _ in range(6):
        u = rng.normal(size=x.shape)
        diff = (loss(x + 1e-5 * u) - loss(x - 1e-5 * u)) / 2e-5
        assert (dx * u).sum() == pytest.approx(diff, rel=1e-7, abs=1e-9)


@pytest.mark.parametrize("tau", [0.5, 2.0])
@pytest.mark.parametrize("rest", [True, False])
def test_distillation(tau, rest):
    x, teacher = rows(), rows(seed=7)
    lq = teacher / tau - np.log(np.exp(teacher / tau).sum(1, keepdims=True))
    ids = np.argsort(-teacher, 1)[:, :6].copy()
    logp = np.take_along_axis(lq, ids, 1)
    ids[1, 2:] = -1               # fewer entries
    ids[2] = 23                   # none: masked
    ids[3, 4] = ids[3, 1]         # one token twice
    kl, dx = O.distill(x, ids, logp, tau, rest)
    assert kl[2] == 0 and not dx[2].any()
    assert (kl[[0, 1, 4]] > 0).all()
    rng = np.random.default_rng(2)
    w = rng.normal(size=5)
    for _ in range(6):
        u = rng.normal(size=x.shape)
        diff = (w * (O.distill(x + 1e-5 * u, ids, logp, tau, rest)[0]
                     - O.distill(x - 1e-5 * u, ids, logp, tau, rest)[0])).sum() / 2e-5
        assert (w[:, None] * dx * u).sum() == pytest.approx(diff, rel=1e-7, abs=1e-9)
    # the teacher's own logits: no divergence, no gradient
    keep = [0, 1, 4]
    if rest:
        kl, dx = O.distill(teacher[keep], ids[keep], logp[keep], tau, True)
        assert np.abs(kl).max() < 1e-12 and np.abs(dx).max() < 1e-12
    # the whole vocabulary named: the divergence of two distributions
    full = np.tile(np.arange(23), (5, 1))
    p = O.softmax(x / tau)
    want = (np.exp(lq) * (lq - np.log(p))).sum(1)
    assert O.distill(x, full, lq, tau, rest)[0] == pytest.approx(want, rel=1e-9)
