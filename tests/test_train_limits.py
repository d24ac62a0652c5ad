"""The sizes that one launch can hold, on the host: a grid counts work items in
32 bits, so 2^24 - 1 workgroups of 256. Sizes beyond are refused before
anything is launched (fake device pointers); the largest ones pass the checks
and end where there is no GPU to launch on."""
import ctypes

import pytest
import torch

import lora_rank_adapter_amd as L
from lora_rank_adapter_amd._lib import LoraAdamwHyper, LoraAdamwState, LoraMat, LoraPolicy
from tests.test_train_host import tensors

FAKE = 0x10000
LAUNCH, LIMIT = -7, -8
MOST = 2 ** 24 - 1
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks (fake device pointers)")
by = ctypes.byref
BF, F = 1, 0


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


def m(rows, cols, dtype=BF):
    return LoraMat(FAKE, dtype, 0, rows, cols, cols, 1)


def test_logits(lib):
    def logp(T, V, dtype=BF):
        return lib.lora_token_logp(by(m(T, V, dtype)), FAKE, FAKE, FAKE, FAKE, 1 << 60, None)

    assert logp(MOST, 8) == LAUNCH and logp(MOST + 1, 8) == LIMIT
    assert lib.lora_loss_workspace_bytes(MOST, 8) > 0 and lib.lora_loss_workspace_bytes(MOST + 1, 8) == 0

    def grad(T, V, dtype=BF):
        a = by(m(T, V, dtype))
        return lib.lora_logit_grad(a, FAKE, FAKE, FAKE, None, 1.0, a, None)

    def pref(T, V, dtype=BF):
        a = by(m(T, V, dtype))
        return lib.lora_pref_step(a, FAKE, FAKE, 1, FAKE, 0.1, 0.0, 1.0, FAKE, None, FAKE, a, FAKE, 1 << 60, None)

    def policy(T, V, dtype=BF):
        a = by(m(T, V, dtype))
        p = LoraPolicy(FAKE, FAKE, FAKE, FAKE, FAKE, 0.2, 0.2, 0.1)
        return lib.lora_policy_step(a, by(p), 1.0, FAKE, FAKE, a, FAKE, 1 << 60, None)

    for f in (grad, pref, policy):
        # 2048 bfloat16 or 1024 float32 of a row to a workgroup, and one workgroup for the loss
        assert f(MOST - 1, 2048) == LAUNCH and f(MOST + 1, 1) == LIMIT, f
        assert f(2 ** 23 - 1, 2049) == LAUNCH and f(2 ** 23, 2049) == LIMIT, f
        assert f(2 ** 23 - 1, 1025, F) == LAUNCH and f(2 ** 23, 1025, F) == LIMIT, f
        assert f(8, 0x7FFFFFFF - 2048) == LAUNCH and f(17, 0x7FFFFFFF - 2048) == LIMIT, f
    # rows of 8 and of 16 waves
    assert policy(2 ** 22, 1537 * 8) == LIMIT and policy(2 ** 21 - 1, 1537 * 8) == LAUNCH
    assert policy(2 ** 22, 6145) == LIMIT and policy(2 ** 22 - 1, 6145) == LAUNCH


def test_losses_on_log_probabilities_have_no_grid(lib):
    p = LoraPolicy(FAKE, FAKE, FAKE, FAKE, FAKE, 0.2, 0.2, 0.1)
    assert lib.lora_pref_loss(FAKE, 2 ** 25 - 1, FAKE, 1, FAKE, 0.1, 0.0, FAKE, None, None, None) == LAUNCH
    assert lib.lora_policy_loss(FAKE, 2 ** 25 - 1, 10, by(p), FAKE, None, None) == LAUNCH


def test_embedding(lib):
    def embed(T, D, dtype=F):
        return lib.lora_embed(FAKE, by(m(100, D, dtype)), 1.0, by(m(T, D, dtype)), None)

    # a row of 1024 float32 to a workgroup; 4 vectors per lane of longer ones; 256 rows of one element
    assert embed(MOST, 1024) == LAUNCH and embed(MOST + 1, 1024) == LIMIT
    assert embed(MOST, 4096) == LAUNCH and embed(MOST + 1, 4096) == LIMIT
    assert embed(MOST, 4097) == LIMIT and embed(2 ** 31 - 5000, 1) == LAUNCH

    def grad(T, V, D, add=0, dtype=F):
        return lib.lora_embed_grad(FAKE, by(m(T, D, dtype)), 1.0, by(m(V, D, dtype)), add, FAKE, 1 << 60, None)

    # zeros of the rows without tokens, beside one workgroup for every 8 tokens of 1024 columns
    for T, items in ((64, 64), (65, 9), (8000, 1000)):
        assert grad(T, MOST - items, 1024) == LAUNCH and grad(T, MOST - items + 1, 1024) == LIMIT
        assert grad(T, MOST - items + 1, 1024, add=1) == LAUNCH
    # the sums alone; their merge (512 columns to a workgroup of each run) is the larger grid
    assert grad(8 * (2 ** 23 - 1), 10, 1024, add=1) == LAUNCH and grad(8 * 2 ** 23, 10, 1024, add=1) == LIMIT
    # the grouping: 2^21 workgroups of 1024, 512 rows to each
    assert grad(65, 2 ** 30, 1, add=1) == LAUNCH and grad(65, 2 ** 30 + 4, 1, add=1) == LIMIT
    assert grad(64, 2 ** 30 + 4, 1, add=1) == LAUNCH


def test_adamw(lib):
    for n, status in ((1024 * MOST, LAUNCH), (1024 * MOST + 1, LIMIT)):
        t = tensors(n)
        st = LoraAdamwState(32, 0, FAKE, FAKE, None, None, FAKE)
        h = LoraAdamwHyper(1e-3, 0.9, 0.99, 1e-8, 0.0, None, None)
        assert lib.lora_adamw_table(t, 1, FAKE, 1 << 60, None) == status
        assert lib.lora_adamw_step(t, 1, FAKE, 1 << 60, by(st), by(h), None) == status
        assert (lib.lora_adamw_table_bytes(t, 1) > 0) == (status == LAUNCH)
