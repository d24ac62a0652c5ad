"""A gradient that overlaps its logits otherwise than as a whole, on the host:
refused before any launch (fake device pointers)."""
import pytest
import torch

import lora_rank_adapter_amd as L
from lora_rank_adapter_amd._lib import LoraMat, LoraPolicy
from tests.test_train_host import FAKE, by

LAUNCH, STRIDE = -7, -4
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks (fake device pointers)")


@pytest.fixture(scope="module")
def calls():
    lib = L.load_library()
    p = LoraPolicy(FAKE, FAKE, FAKE, FAKE, FAKE, 0.2, 0.2, 0.0)
    return [
        lambda x, d: lib.lora_logit_grad(by(x), FAKE, FAKE, FAKE, None, 1.0, by(d), None),
        lambda x, d: lib.lora_logit_grad_logp(by(x), FAKE, FAKE, FAKE, FAKE, None, 1.0, by(d), None),
        lambda x, d: lib.lora_pref_step(by(x), FAKE, FAKE, 2, FAKE, 0.1, 0.0, 1.0, FAKE, None, FAKE, by(d), FAKE,
                                        1 << 40, None),
        lambda x, d: lib.lora_policy_step(by(x), by(p), 1.0, FAKE, FAKE, by(d), FAKE, 1 << 40, None),
    ]


def m(rows, cols, at=0, stride=None, dtype=1):
    es = 2 if dtype else 4
    return LoraMat(FAKE + 0x1000000 + at * es, dtype, 0, rows, cols, stride or cols, 1)


@pytest.mark.parametrize("dtype", [0, 1])
def test_overlaps(calls, dtype):
    def at(offset, stride, rows=8, cols=1000):
        return m(rows, cols, offset, stride, dtype)

    x = at(0, 2500)
    for call in calls:
        # the logits themselves, memory before and after them, the columns beside them in the same rows
        for good in (at(0, 2500), at(-8 * 2500, 2500), at(7 * 2500 + 1000, 2500), at(1000, 2500), at(1500, 2500),
                     at(-1000, 2500), at(-1500, 2500), at(2500 + 1000, 2500), at(-7 * 1000 - 1000, 1000)):
            assert call(x, good) == LAUNCH
        # other rows of theirs, columns that begin inside them or end there, other pitches over the same memory
        for bad in (at(2500, 2500), at(-2500, 2500), at(7 * 2500, 2500), at(1, 2500), at(-1, 2500), at(999, 2500),
                    at(1501, 2500), at(-999, 2500), at(-1501, 2500), at(0, 2501), at(0, 1000), at(3000, 1000),
                    at(-7 * 1000 - 999, 1000)):
            assert call(x, bad) == STRIDE
        # one row has no pitch
        assert call(at(0, 2500, rows=1), at(0, 1000, rows=1)) == LAUNCH
        assert call(at(0, 2500, rows=1), at(999, 1000, rows=1)) == STRIDE
        assert call(at(0, 2500, rows=1), at(1000, 1000, rows=1)) == LAUNCH


def test_overlap_in_bytes(calls):
    """Half an element's shift cannot be (alignment), and empty operands overlap nothing."""
    x = m(4, 10)
    for call in calls[:2]:
        assert call(m(0, 10), m(0, 10)) == 0
        assert call(x, LoraMat(x.ptr + 1, 1, 0, 4, 10, 10, 1)) == STRIDE
