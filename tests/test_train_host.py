"""Refusals of the training-step operators, on the host: the C entry points
with fake device pointers (each call is rejected, or an empty no-op, before
any launch) and the binding's own checks on CPU tensors."""
import ctypes

import pytest
import torch

import lora_rank_adapter_amd as L
from lora_rank_adapter_amd._lib import (LoraAdamwHyper, LoraAdamwState, LoraAdamwTensor, LoraMat, LoraPolicy)

FAKE = 0x10000
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks (fake device pointers)")
by = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


def m(rows, cols, dtype=1, sr=None, sc=1, ptr=FAKE):
    return LoraMat(ptr, dtype, 0, rows, cols, cols if sr is None else sr, sc)


def test_embed(lib):
    def f(ids=FAKE, table=m(100, 16), out=m(8, 16)):
        return lib.lora_embed(ids, table and by(table), 1.0, out and by(out), None)

    assert f(table=None) == -1 and f(out=None) == -1 and f(ids=None) == -1
    assert f(out=m(8, 16, ptr=None)) == -1 and f(table=m(100, 16, ptr=None)) == -1
    assert f(out=m(8, 24)) == -2 and f(table=m(1 << 46, 16)) == -2 and f(table=m(100, 16, sr=-16)) == -2
    assert f(table=m(100, 16, dtype=0)) == -3 and f(table=m(100, 16, dtype=5)) == -3 and f(out=m(8, 16, 5)) == -3
    assert f(table=m(100, 16, sr=15)) == -4 and f(out=m(8, 16, sr=1, sc=8)) == -4
    assert f(table=m(100, 16, ptr=FAKE + 1)) == -4 and f(out=m(8, 16, 0, ptr=FAKE + 2)) == -4
    assert f(table=m(0x7FFFFFFF, 16)) == -8 and f(out=m(0x7FFFFFFF, 16)) == -8
    assert f(out=m(0, 16)) == 0 and f(table=m(100, 0), out=m(8, 0)) == 0


def test_embed_grad(lib):
    need = lib.lora_embed_grad_workspace_bytes(8, 100, 16)
    assert need > 0 and lib.lora_embed_grad_workspace_bytes(0, 100, 16) > 0
    for sizes in ((-1, 100, 16), (8, -1, 16), (8, 100, -1), (0x7FFFFFFF, 100, 16), (8, 1 << 40, 16),
                  (1 << 30, 100, 1 << 46), (1 << 62, 1 << 62, 1 << 62), (8, 0, 16)):
        assert lib.lora_embed_grad_workspace_bytes(*sizes) == 0, sizes

    def f(ids=FAKE, dy=m(8, 16), out=m(100, 16), add=0, ws=FAKE, nbytes=need):
        return lib.lora_embed_grad(ids, dy and by(dy), 1.0, out and by(out), add, ws, nbytes, None)

    assert f(dy=None) == -1 and f(out=None) == -1 and f(ids=None) == -1 and f(dy=m(8, 16, ptr=None)) == -1
    assert f(dy=m(8, 24)) == -2 and f(dy=m(8, 16, 0)) == -3 and f(out=m(100, 16, 9)) == -3
    assert f(dy=m(8, 16, sr=8)) == -4 and f(out=m(100, 16, ptr=FAKE + 1)) == -4
    assert f(ws=None) == -6 and f(ws=FAKE + 128) == -6 and f(nbytes=need - 1) == -6
    assert f(out=m(0x7FFFFFFF, 16)) == -8
    assert f(out=m(0, 16)) == 0 and f(dy=m(8, 0), out=m(100, 0)) == 0 and f(dy=m(0, 16), add=1) == 0


def test_logp_and_logit_grad(lib):
    need = lib.lora_loss_workspace_bytes(8, 1000)
    assert need > 0
    for sizes in ((-1, 8), (8, -1), (1 << 25, 8), (8, 0x7FFFFFFF), (1 << 62, 1 << 62)):
        assert lib.lora_loss_workspace_bytes(*sizes) == 0, sizes

    def f(x=m(8, 1000), y=FAKE, logp=FAKE, stats=FAKE, ws=FAKE, nbytes=need):
        return lib.lora_token_logp(x and by(x), y, logp, stats, ws, nbytes, None)

    assert f(x=None) == -1 and f(y=None) == -1 and f(logp=None) == -1 and f(stats=None) == -1
    assert f(x=m(8, 1000, ptr=None)) == -1 and f(x=m(1 << 46, 1000)) == -2 and f(x=m(8, 1000, 7)) == -3
    assert f(x=m(8, 1000, sr=999)) == -4 and f(x=m(8, 1000, sr=1, sc=8)) == -4 and f(x=m(8, 1000, ptr=FAKE + 1)) == -4
    assert f(ws=None) == -6 and f(ws=FAKE + 8) == -6 and f(nbytes=need - 1) == -6
    assert f(x=m(1 << 25, 8)) == -8 and f(x=m(8, 0x7FFFFFFF)) == -8
    assert f(x=m(0, 1000)) == 0

    def g(x=m(8, 1000), y=FAKE, stats=FAKE, coef=FAKE, dx=m(8, 1000)):
        return lib.lora_logit_grad(x and by(x), y, stats, coef, None, 1.0, dx and by(dx), None)

    assert g(x=None) == -1 and g(dx=None) == -1 and g(y=None) == -1 and g(stats=None) == -1 and g(coef=None) == -1
    assert g(dx=m(8, 999)) == -2 and g(dx=m(8, 1000, 0)) == -3 and g(dx=m(8, 1000, sr=998)) == -4
    assert g(x=m(0, 1000), dx=m(0, 1000)) == 0 and g(x=m(8, 0), dx=m(8, 0)) == 0


def test_losses(lib):
    def pref(logp=FAKE, T=8, off=FAKE, pairs=2, ref=FAKE, loss=FAKE):
        return lib.lora_pref_loss(logp, T, off, pairs, ref, 0.1, 0.0, loss, None, None, None)

    assert pref(logp=None) == -1 and pref(off=None) == -1 and pref(ref=None) == -1 and pref(loss=None) == -1
    assert pref(T=-1) == -2 and pref(pairs=0) == -2 and pref(pairs=-3) == -2 and pref(T=1 << 25) == -8

    def policy(T=8, V=1000, loss=FAKE, logp=FAKE, kl=0.0, **kw):
        a = dict(targets=FAKE, old_logp=FAKE, ref_logp=FAKE, advantages=FAKE, weights=FAKE)
        p = LoraPolicy(*dict(a, **kw).values(), 0.2, 0.2, kl)
        return lib.lora_policy_loss(logp, T, V, by(p), loss, None, None)

    for name in ("targets", "old_logp", "advantages", "weights"):
        assert policy(**{name: None}) == -1, name
    assert policy(ref_logp=None, kl=0.1) == -1 and policy(loss=None) == -1 and policy(logp=None) == -1
    assert lib.lora_policy_loss(FAKE, 8, 10, None, FAKE, None, None) == -1
    assert policy(T=-1) == -2 and policy(V=-1) == -2 and policy(T=1 << 25) == -8

    need = lib.lora_loss_workspace_bytes(8, 1000)

    def step(x=m(8, 1000), dx=m(8, 1000), logp=FAKE, pairs=2, ws=FAKE, nbytes=need, y=FAKE):
        return lib.lora_pref_step(x and by(x), y, FAKE, pairs, FAKE, 0.1, 0.0, 1.0, FAKE, None, logp, dx and by(dx),
                                  ws, nbytes, None)

    assert step(x=None) == -1 and step(dx=None) == -1 and step(logp=None) == -1 and step(y=None) == -1
    assert step(pairs=0) == -2 and step(dx=m(8, 1001)) == -2 and step(dx=m(8, 1000, 0)) == -3
    assert step(ws=None) == -6 and step(nbytes=need - 1) == -6 and step(x=m(8, 1000, sc=2)) == -4

    p = LoraPolicy(FAKE, FAKE, FAKE, FAKE, FAKE, 0.2, 0.2, 0.1)

    def pstep(x=m(8, 1000), dx=m(8, 1000), p=p, logp=FAKE, ws=FAKE, nbytes=need, loss=FAKE):
        return lib.lora_policy_step(x and by(x), p and by(p), 1.0, loss, logp, dx and by(dx), ws, nbytes, None)

    assert pstep(x=None) == -1 and pstep(dx=None) == -1 and pstep(p=None) == -1 and pstep(logp=None) == -1
    assert pstep(loss=None) == -1 and pstep(dx=m(9, 1000)) == -2 and pstep(dx=m(8, 1000, 0)) == -3
    assert pstep(ws=None) == -6 and pstep(ws=FAKE + 1) == -6 and pstep(nbytes=need - 1) == -6


def tensors(*numels, param=FAKE, grad=FAKE, shadow=None, pd=0, gd=0):
    return (LoraAdamwTensor * len(numels))(*[LoraAdamwTensor(param, grad, shadow, n, pd, gd) for n in numels])


def test_adamw(lib):
    t = tensors(1, 256, 257, 0, 5000)
    assert lib.lora_adamw_state_elems(t, 5) == 256 * (1 + 1 + 2 + 0 + 20)
    need = lib.lora_adamw_table_bytes(t, 5)
    assert need >= 256 + 5 * 48 + 4 * (1 + 1 + 1 + 0 + 3)
    assert lib.lora_adamw_table_bytes(t, -1) == 0 and lib.lora_adamw_state_elems(None, 1) == 0
    for bad in (-1, 1 << 46, (1 << 63) - 1):
        assert lib.lora_adamw_table_bytes(tensors(bad), 1) == 0
    assert lib.lora_adamw_table_bytes(tensors(*[1 << 44] * 9), 9) == 0  # too many elements together

    def table(t=t, n=5, table=FAKE, nbytes=need):
        return lib.lora_adamw_table(t, n, table, nbytes, None)

    assert table(t=None) == -1 and table(t=tensors(4, param=None), n=1) == -1
    assert table(t=tensors(4, grad=None), n=1) == -1
    assert table(n=-1) == -2 and table(t=tensors(-5), n=1) == -2
    assert table(t=tensors(4, pd=3), n=1) == -3 and table(t=tensors(4, gd=-1), n=1) == -3
    assert table(t=tensors(4, pd=1, shadow=FAKE), n=1) == -3  # a copy of a bfloat16 param
    assert table(t=tensors(4, param=FAKE + 2), n=1) == -4 and table(t=tensors(4, grad=FAKE + 1, gd=1), n=1) == -4
    assert table(t=tensors(4, shadow=FAKE + 1), n=1) == -4
    assert table(table=None) == -6 and table(table=FAKE + 64) == -6 and table(nbytes=need - 1) == -6
    assert table(n=1 << 23) == -8
    assert table(t=None, n=0) == 0 and table(t=tensors(0, 0, param=None, grad=None), n=2) == 0

    def step(t=t, n=5, bits=32, m=FAKE, v=FAKE, ms=FAKE, vs=FAKE, count=FAKE, nbytes=need, table=FAKE):
        st = LoraAdamwState(bits, 0, m, v, ms, vs, count)
        h = LoraAdamwHyper(1e-3, 0.9, 0.99, 1e-8, 0.0, None, None)
        return lib.lora_adamw_step(t, n, table, nbytes, by(st), by(h), None)

    assert step(m=None) == -1 and step(v=None) == -1 and step(count=None) == -1
    assert step(bits=8, ms=None) == -1 and step(bits=8, vs=None) == -1 and step(bits=4) == -3
    assert step(m=FAKE + 4) == -4 and step(v=FAKE + 8) == -4
    assert step(table=None) == -6 and step(nbytes=need - 1) == -6
    assert step(t=tensors(0), n=1, table=None) == 0
    assert lib.lora_adamw_step(t, 5, FAKE, need, None, None, None) == -1


def test_binding_checks():
    i32, f32 = torch.int32, torch.float32
    x, y = torch.zeros(4, 10), torch.zeros(4, dtype=i32)
    f = torch.zeros(4)
    off, ref = torch.tensor([0, 2, 4], dtype=i32), torch.zeros(2)
    with pytest.raises(ValueError, match="ids"):
        L.lora_embed(torch.zeros(4, dtype=torch.int64), x)
    with pytest.raises(ValueError, match="ids"):
        L.lora_embed_grad(torch.zeros(5, dtype=i32), x, 7)
    with pytest.raises(ValueError, match="rows"):
        L.lora_embed(y, x, out=torch.zeros(3, 10))
    with pytest.raises(ValueError, match="rows"):
        L.lora_embed_grad(y, x, 7, dtable=torch.zeros(6, 10))
    with pytest.raises(ValueError, match="accumulate"):
        L.lora_embed_grad(y, x, 7, accumulate=True)
    with pytest.raises(ValueError, match="targets"):
        L.lora_token_logp(x, y.long())
    with pytest.raises(ValueError, match="targets"):
        L.lora_token_logp(x, torch.zeros(8, dtype=i32)[::2])
    with pytest.raises(ValueError, match="seq_offsets"):
        L.lora_pref_loss(f, torch.zeros(4, dtype=i32), ref, 0.1)
    with pytest.raises(ValueError, match="ref_logp"):
        L.lora_pref_step(x, y, off, torch.zeros(3), 0.1)
    with pytest.raises(ValueError, match="kl_coef"):
        L.lora_policy_loss(f, y, 10, f, f, f, 0.2, 0.2, kl_coef=0.1)
    with pytest.raises(ValueError, match="advantages"):
        L.lora_policy_step(x, y, f, f.double(), f, 0.2, 0.2)
    with pytest.raises(ValueError, match="stats"):
        L.lora_logit_grad(x, y, torch.zeros(4), f)
    with pytest.raises(ValueError, match="grad_out"):
        L.lora_logit_grad(x, y, torch.zeros(4, 2), f, grad_out=torch.zeros((), dtype=torch.float64))
    with pytest.raises(ValueError, match="expected cpu"):
        L.lora_token_logp(x, torch.zeros(4, dtype=i32, device="meta"))
    with pytest.raises(ValueError, match="parameter"):
        L.AdamW([], [], 1e-3)
    with pytest.raises(ValueError, match="state_bits"):
        L.AdamW([f], [f], 1e-3, state_bits=16)
    with pytest.raises(ValueError, match="grads"):
        L.AdamW([f], [f, f], 1e-3)
    with pytest.raises(ValueError, match="grad 0"):
        L.AdamW([f], [torch.zeros(3)], 1e-3)
    with pytest.raises(ValueError, match="param 0"):
        L.AdamW([torch.zeros(8)[::2]], [f], 1e-3)
    with pytest.raises(ValueError, match="shadow 0"):
        L.AdamW([f], [f], 1e-3, shadows=[torch.zeros(4)])
    # CPU tensors never reach the library
    for call in (lambda: L.lora_embed(y, x), lambda: L.lora_embed_grad(y, x, 7), lambda: L.lora_token_logp(x, y),
                 lambda: L.lora_pref_loss(f, off, ref, 0.1), lambda: L.lora_pref_step(x, y, off, ref, 0.1),
                 lambda: L.lora_policy_loss(f, y, 10, f, f, f, 0.2, 0.2),
                 lambda: L.lora_policy_step(x, y, f, f, f, 0.2, 0.2),
                 lambda: L.lora_logit_grad(x, y, torch.zeros(4, 2), f), lambda: L.AdamW([f], [f], 1e-3)):
        with pytest.raises(ValueError, match="GPU"):
            call()
