"""Entropy, alternatives and distillation on the host: refusals with the
documented status before anything is launched (fake device pointers), and the
binding's own."""
import ctypes

import pytest
import torch

import lora_rank_adapter_amd as L
from lora_rank_adapter_amd import _lib
from lora_rank_adapter_amd._lib import LoraMat, LoraTeacher

FAKE = 0x10000
NULL, SHAPE, DTYPE, STRIDE, WORKSPACE, LAUNCH, LIMIT, VALUE = -1, -2, -3, -4, -6, -7, -8, -9
MOST = 2 ** 24 - 1
HUGE = 1 << 60
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks (fake device pointers)")
by = ctypes.byref
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


def m(rows, cols, dtype=1, sr=None, sc=1, ptr=FAKE):
    return LoraMat(ptr, dtype, 0, rows, cols, cols if sr is None else sr, sc)


def bad_logits():
    return [(None, NULL), (m(4, 9, dtype=5), DTYPE), (m(-1, 9), SHAPE), (m(4, 9, sc=2), STRIDE), (m(4, 9, sr=8), STRIDE),
            (m(4, 9, ptr=FAKE + 1), STRIDE), (m(MOST + 1, 1), LIMIT), (m(4, 9, ptr=None), NULL)]


def test_top(lib):
    need = lib.lora_token_top_workspace_bytes
    assert need(8, 1000, 0) > 0 and need(8, 1000, 128) > 0 and need(0, 0, 5) > 0
    for sizes in ((-1, 9, 1), (9, -1, 1), (9, 9, -1), (9, 9, 129), (MOST + 1, 9, 1), (9, 2 ** 31 - 2048, 1)):
        assert need(*sizes) == 0, sizes

    def top(x, y=FAKE, k=5, tau=1.0, logp=FAKE, entropy=FAKE, ids=FAKE, top=FAKE, stats=FAKE, ws=FAKE, nbytes=HUGE):
        return lib.lora_token_top(x and by(x), y, k, tau, logp, entropy, ids, top, stats, ws, nbytes, None)

    x = m(4, 9)
    for v, status in bad_logits():
        assert top(v) == status
    assert top(m(0, 9)) == 0 and top(x) == LAUNCH and top(m(MOST, 8)) == LAUNCH
    assert top(x, k=0, ids=None, top=None) == LAUNCH
    assert top(x, k=-1) == SHAPE and top(x, k=129) == LIMIT and top(x, k=128) == LAUNCH
    for tau in (0.0, -1.0, NAN, INF, 1e-7, 2e6):
        assert top(x, tau=tau) == VALUE
    assert top(x, tau=1e-6) == LAUNCH and top(x, tau=1e6) == LAUNCH
    assert top(x, y=None) == NULL and top(x, y=None, logp=None) == LAUNCH and top(x, logp=None) == NULL
    for name in ("entropy", "ids", "top", "stats"):
        assert top(x, **{name: None}) == NULL, name
    assert top(x, ws=None) == WORKSPACE and top(x, nbytes=need(4, 9, 5) - 1) == WORKSPACE
    assert top(x, nbytes=need(4, 9, 5)) == LAUNCH and top(x, ws=FAKE + 16) == WORKSPACE


def test_largest_sizes(lib):
    def top(T, V, k, dtype=1):
        assert (lib.lora_token_top_workspace_bytes(T, V, k) > 0) == (T <= MOST)
        return lib.lora_token_top(by(m(T, V, dtype)), FAKE, k, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, HUGE, None)

    assert top(3, 2 ** 22, 128) == LAUNCH
    assert lib.lora_token_top_workspace_bytes(3, 2 ** 22 + 1, 1) == 0
    assert lib.lora_token_top(by(m(3, 2 ** 22 + 1)), FAKE, 1, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, HUGE, None) == LIMIT
    assert top(MOST, 1000, 5) == LAUNCH
    # eight waves to a row, two pieces of a row
    assert top(2 ** 23 - 1, 70001, 20) == LAUNCH
    for T, V, k in ((2 ** 23, 70001, 20), (2 ** 22, 128256, 128)):
        assert lib.lora_token_top_workspace_bytes(T, V, k) == 0
        assert lib.lora_token_top(by(m(T, V)), FAKE, k, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, HUGE, None) == LIMIT

    def kl(T, V, dtype=1):
        t = LoraTeacher(FAKE, FAKE, 64, 1.0, 1)
        return lib.lora_distill_kl(by(m(T, V, dtype)), by(t), FAKE, None, FAKE, HUGE, None)

    assert kl(3, 2 ** 23) == LAUNCH and kl(3, 2 ** 23 + 1) == LIMIT
    assert lib.lora_distill_workspace_bytes(3, 2 ** 23, 1) > 0 and lib.lora_distill_workspace_bytes(3, 2 ** 23 + 1, 1) == 0
    assert kl(MOST, 2560 * 8) == LAUNCH and kl(2 ** 23 - 1, 2561 * 8) == LAUNCH and kl(2 ** 23, 2561 * 8) == LIMIT
    # rows longer than one workgroup takes: three pieces of 131072
    assert kl(MOST // 3, 3 * 131072) == LAUNCH and kl(MOST // 3 + 1, 3 * 131072) == LIMIT


def check_gradients(grad):
    """What every gradient of logits refuses."""
    for v, status in bad_logits():
        assert grad(v, m(4, 9)) == status
    x = m(4, 9)
    assert grad(x, None) == NULL and grad(x, m(4, 9, ptr=None)) == NULL
    assert grad(x, m(4, 8)) == SHAPE and grad(x, m(5, 9)) == SHAPE and grad(x, m(4, 9, dtype=0)) == DTYPE
    assert grad(x, m(4, 9, sc=2)) == STRIDE
    assert grad(x, m(4, 9, ptr=FAKE + 2)) == STRIDE         # they overlap in part
    assert grad(x, x) == LAUNCH and grad(x, m(4, 9, ptr=FAKE + 72)) == LAUNCH
    a = m(2 ** 23 - 1, 2049)
    assert grad(a, a) == LAUNCH and grad(m(2 ** 23, 2049), m(2 ** 23, 2049)) == LIMIT


def test_top_grad(lib):
    def grad(x, dx, y=FAKE, stats=FAKE, g=FAKE, h=FAKE, tau=1.0):
        return lib.lora_token_top_grad(x and by(x), y, stats, g, h, tau, dx and by(dx), None)

    check_gradients(grad)
    x = m(4, 9)
    assert grad(m(0, 9), m(0, 9)) == 0 and grad(m(4, 0), m(4, 0)) == 0
    assert grad(x, x, stats=None) == NULL and grad(x, x, y=None) == NULL
    assert grad(x, x, y=None, g=None) == LAUNCH and grad(x, x, g=None, h=None) == LAUNCH
    for tau in (0.0, -1.0, NAN, INF, 1e-7, 2e6):
        assert grad(x, x, tau=tau) == VALUE


def test_distill(lib):
    need = lib.lora_distill_workspace_bytes
    assert need(8, 1000, 1) > 0 and need(8, 1000, 256) > 0 and need(0, 0, 5) > 0
    for sizes in ((-1, 9, 1), (9, -1, 1), (9, 9, 0), (9, 9, -1), (9, 9, 257), (MOST + 1, 9, 1), (9, 2 ** 31 - 2048, 1)):
        assert need(*sizes) == 0, sizes

    def teacher(ids=FAKE, logp=FAKE, k=5, rest=1, tau=1.0):
        return LoraTeacher(ids, logp, k, tau, rest)

    def kl(x, t=teacher(), out=FAKE, state=FAKE, ws=FAKE, nbytes=HUGE):
        return lib.lora_distill_kl(x and by(x), t and by(t), out, state, ws, nbytes, None)

    def step(x, dx, t=teacher(), weights=FAKE, loss=FAKE, out=FAKE, ws=FAKE, nbytes=HUGE):
        return lib.lora_distill_step(x and by(x), t and by(t), weights, 1.0, loss, out, dx and by(dx), ws, nbytes, None)

    x = m(4, 9)
    for v, status in bad_logits():
        assert kl(v) == status
    check_gradients(step)
    assert kl(x) == LAUNCH and kl(x, state=None) == LAUNCH and kl(m(0, 9)) == 0 and step(m(0, 9), m(0, 9)) == LAUNCH
    both = (lambda t: kl(x, t), lambda t: step(x, x, t))
    for f in both:
        assert f(None) == NULL and f(teacher(ids=None)) == NULL and f(teacher(logp=None)) == NULL
        assert f(teacher(k=0)) == SHAPE and f(teacher(k=257)) == LIMIT and f(teacher(k=256)) == LAUNCH
        for tau in (0.0, -1.0, NAN, INF, 1e-7, 2e6):
            assert f(teacher(tau=tau)) == VALUE
    assert kl(x, out=None) == NULL
    for name in ("weights", "loss", "out"):
        assert step(x, x, **{name: None}) == NULL, name
    size = need(4, 9, 5)
    for f in (lambda **a: kl(x, **a), lambda **a: step(x, x, **a)):
        assert f(ws=None) == WORKSPACE and f(nbytes=size - 1) == WORKSPACE and f(nbytes=size) == LAUNCH
        assert f(ws=FAKE + 16) == WORKSPACE


def test_distill_grad(lib):
    def grad(x, dx, ids=FAKE, k=5, state=FAKE, coef=FAKE, out=None, tau=1.0):
        return lib.lora_distill_grad(x and by(x), ids, k, state, coef, out, 1.0, tau, dx and by(dx), None)

    check_gradients(grad)
    x = m(4, 9)
    assert grad(m(0, 9), m(0, 9)) == 0 and grad(m(4, 0), m(4, 0)) == 0
    for name in ("ids", "state", "coef"):
        assert grad(x, x, **{name: None}) == NULL, name
    assert grad(x, x, k=0) == SHAPE and grad(x, x, k=257) == LIMIT
    for tau in (0.0, -1.0, NAN, INF, 1e-7, 2e6):
        assert grad(x, x, tau=tau) == VALUE


def test_packed_teacher():
    t = LoraTeacher(0x1122334455667788, 0x99AABBCCDDEEFF, 7, 1.5, 1)
    assert _lib.pack_teacher(t.ids, t.logp, 7, 1.5, 1) == bytes(t)


def test_binding_refuses():
    x, i, f = torch.zeros(4, 9), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    y, w = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    for call in (lambda: L.lora_token_top(x, y.long()), lambda: L.lora_token_top(x, y[:3]), lambda: L.lora_token_top(x[0], y),
                 lambda: L.lora_token_top(x, y), lambda: L.lora_token_top_grad(x, y, torch.zeros(4, 2), w),
                 lambda: L.lora_token_top_grad(x, y, torch.zeros(4, 3), w[:2]),
                 lambda: L.lora_token_top_grad(x, y, torch.zeros(4, 3), w),
                 lambda: L.lora_distill_kl(x, i, f[:, :1]), lambda: L.lora_distill_kl(x, i.long(), f),
                 lambda: L.lora_distill_kl(x, i[:3], f[:3]), lambda: L.lora_distill_kl(x, i.t(), f.t()),
                 lambda: L.lora_distill_kl(x, i, f), lambda: L.lora_distill_step(x, i, f, w.double()),
                 lambda: L.lora_distill_step(x, i, f, w[:3]), lambda: L.lora_distill_step(x, i, f, w),
                 lambda: L.lora_distill_grad(x, i, torch.zeros(4, 3), w),
                 lambda: L.lora_distill_grad(x, i, torch.zeros(4, 4), w)):
        with pytest.raises(ValueError):
            call()
