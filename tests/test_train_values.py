"""Scalars outside their ranges, on the host: refused by the library before any
launch (fake device pointers), and what is inside reaches the launch."""
import math

import pytest
import torch

import lora_rank_adapter_amd as L
from lora_rank_adapter_amd._lib import LoraAdamwHyper, LoraAdamwState, LoraPolicy
from tests.test_train_host import FAKE, by, m, tensors

LAUNCH, VALUE = -7, -9
INF, NAN = math.inf, math.nan
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks (fake device pointers)")


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


def test_status_has_a_name(lib):
    assert b"range" in lib.lora_status_string(VALUE)
    assert "LORA_ERR_VALUE" in str(L.LoraError("call", VALUE))


def test_preference_scalars(lib):
    x = m(8, 1000)

    def loss(beta=0.1, eps=0.0):
        return lib.lora_pref_loss(FAKE, 8, FAKE, 2, FAKE, beta, eps, FAKE, None, None, None)

    def step(beta=0.1, eps=0.0):
        return lib.lora_pref_step(by(x), FAKE, FAKE, 2, FAKE, beta, eps, 1.0, FAKE, None, FAKE, by(x), FAKE, 1 << 40,
                                  None)

    for f in (loss, step):
        for eps in (-0.1, 1.0001, NAN, INF):
            assert f(eps=eps) == VALUE, eps
        for beta in (NAN, INF, -INF):
            assert f(beta=beta) == VALUE, beta
        for beta, eps in ((0.1, 0.0), (0.0, 1.0), (-1.0, 0.5)):
            assert f(beta, eps) == LAUNCH


def test_policy_scalars(lib):
    x = m(8, 1000)

    def scalars(low, high, kl):
        return LoraPolicy(FAKE, FAKE, FAKE, FAKE, FAKE, low, high, kl)

    def loss(*a):
        return lib.lora_policy_loss(FAKE, 8, 1000, by(scalars(*a)), FAKE, None, None)

    def step(*a):
        return lib.lora_policy_step(by(x), by(scalars(*a)), 1.0, FAKE, FAKE, by(x), FAKE, 1 << 40, None)

    for f in (loss, step):
        for a in ((NAN, 0.2, 0.0), (0.2, NAN, 0.0), (-0.2, 0.1, 0.0), (0.1, -INF, 0.0), (0.2, 0.2, NAN),
                  (0.2, 0.2, INF)):
            assert f(*a) == VALUE, a
        for a in ((0.2, 0.2, 0.0), (0.0, 0.0, 0.1), (0.2, INF, 0.0), (INF, INF, -0.1)):
            assert f(*a) == LAUNCH, a


def test_adamw_scalars(lib):
    t = tensors(1000)

    def step(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, decay=0.0):
        st = LoraAdamwState(32, 0, FAKE, FAKE, None, None, FAKE)
        h = LoraAdamwHyper(lr, beta1, beta2, eps, decay, None, None)
        return lib.lora_adamw_step(t, 1, FAKE, 1 << 40, by(st), by(h), None)

    for bad in (dict(lr=NAN), dict(lr=INF), dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=NAN), dict(beta2=1.0),
                dict(beta2=1.5), dict(beta2=NAN), dict(eps=-1e-8), dict(eps=NAN), dict(decay=NAN), dict(decay=INF)):
        assert step(**bad) == VALUE, bad
    for good in (dict(), dict(lr=0.0), dict(beta1=0.0, beta2=0.0), dict(eps=0.0), dict(lr=-1e-3)):
        assert step(**good) == LAUNCH, good
