"""Embedding lookup and its gradient against the float64 definitions.

Tolerances, counted from the roundings (a rounding to t is off by at most
finfo(t).eps / 2 of the value): the lookup rounds the product to float32 and,
for bfloat16, once more; a sum of n float32 terms is off by at most n roundings
of the sum of their magnitudes."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from oracle import train_oracle as O
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
H32 = 2.0 ** -24


def half(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def make_ids(T, V, kind, rng):
    if kind == "same":
        ids = np.full(T, V // 2)
    elif kind == "distinct":
        ids = rng.permutation(np.arange(T) % V)
    elif kind == "outside":
        ids = np.resize([-1, V, -2 ** 31, 2 ** 31 - 1], T)
    else:  # frequent low ids, one in twenty outside the table
        ids = np.floor(np.exp(rng.uniform(0, np.log(V + 1), T)) - 1).clip(0, V - 1)
        ids[rng.random(T) < 0.05] = rng.choice([-1, V, V + 7])
    return torch.from_numpy(ids.astype(np.int32)).to(DEV)


def strided(rows, cols, dtype, pad, shift, std=1.0):
    """rows x cols with a row pitch of cols + pad that starts `shift` elements into its buffer."""
    buf = torch.randn(rows * (cols + pad) + shift + 1, device=DEV).mul_(std).to(dtype)
    return buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


PAIRS = [(F, F), (BF, F), (BF, BF)]


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("T,V,D,pad,shift", [(1, 5, 1, 0, 0), (1, 100, 8192, 0, 0), (3, 7, 7, 0, 1), (70, 50, 129, 3, 1),
                                              (257, 1000, 64, 0, 0), (33, 9, 8, 8, 8), (600, 300, 9000, 0, 0),
                                              (1000, 4, 20, 1, 3)])
def test_lookup(types, T, V, D, pad, shift):
    note(f"embed {types} {T} {V} {D} {pad} {shift}")
    torch.manual_seed(T + D)
    rng = np.random.default_rng(T * 7 + D)
    table = strided(V, D, types[0], pad, shift)
    ids = make_ids(T, V, "zipf", rng)
    out = strided(T, D, types[1], pad, shift)
    whole = out._base.clone()
    got = L.lora_embed(ids, table, 1.7, out=out)
    assert got is out
    want = O.embed(ids.cpu().numpy(), f64(table), np.float64(np.float32(1.7)))
    tol = (H32 + (half(BF) if types[1] is BF else 0)) * 1.01 * np.abs(want)
    assert (np.abs(f64(got) - want) <= tol).all()
    # nothing beside the rows is written
    rest = torch.ones_like(whole, dtype=torch.bool)
    rest[shift:shift + T * (D + pad)].view(T, D + pad)[:, :D] = False
    assert torch.equal(out._base[rest], whole[rest])


def check_grad(got, ids, dy, V, scale, old=None):
    ids, dy64 = ids.cpu().numpy(), f64(dy)
    s = np.float64(np.float32(scale))
    want = O.embed_grad(ids, dy64, V, s, old)
    mag = O.embed_grad(ids, np.abs(dy64), V, abs(s), None if old is None else np.abs(old))
    count = np.bincount(ids[(ids >= 0) & (ids < V)], minlength=V)[:, None] + 3
    tol = count * H32 * mag + (half(BF) * 1.01 * np.abs(want) if got.dtype is BF else 0)
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("T,V,D,kind,pad,shift", [
    (1, 1, 1, "same", 0, 0), (1, 1000, 64, "zipf", 0, 0), (16, 40, 33, "zipf", 3, 1), (17, 3, 8, "zipf", 0, 0),
    (64, 64, 16, "distinct", 0, 0), (500, 700, 100, "same", 0, 0), (1000, 50, 64, "outside", 8, 8),
    (1111, 5000, 257, "zipf", 1, 1), (4097, 513, 24, "zipf", 0, 0), (2000, 140000, 12, "zipf", 0, 0),
    (300, 20, 2500, "zipf", 0, 0), (2048, 2, 4100, "zipf", 4, 0)])
def test_gradient(types, T, V, D, kind, pad, shift):
    note(f"embed_grad {types} {T} {V} {D} {kind} {pad} {shift}")
    torch.manual_seed(T + D)
    rng = np.random.default_rng(T * 7 + D)
    ids = make_ids(T, V, kind, rng)
    dy = strided(T, D, types[0], pad, shift)
    out = strided(V, D, types[1], pad, shift)
    whole = out._base.clone()
    got = L.lora_embed_grad(ids, dy, V, 0.7, dtable=out)
    assert got is out
    check_grad(got, ids, dy, V, 0.7)
    rest = torch.ones_like(whole, dtype=torch.bool)
    rest[shift:shift + V * (D + pad)].view(V, D + pad)[:, :D] = False
    assert torch.equal(out._base[rest], whole[rest])
    # the same bits again, whatever the workspace held
    ws = torch.full((L.load_library().lora_embed_grad_workspace_bytes(T, V, D),), 255, dtype=torch.uint8, device=DEV)
    again = L.lora_embed_grad(ids, dy, V, 0.7, workspace=ws, dtype=types[1])
    assert torch.equal(got, again)
    # added to what is there; rows without tokens are left alone, bit for bit
    old = torch.randn(V, D, device=DEV).to(types[1])
    old[:, 0] = float("nan")
    base = old.clone()
    L.lora_embed_grad(ids, dy, V, 0.7, dtable=old, accumulate=True)
    named = torch.zeros(V, dtype=torch.bool, device=DEV)
    ok = (ids >= 0) & (ids < V)
    named[ids[ok].long()] = True
    view = torch.int16 if types[1] is BF else torch.int32
    assert torch.equal(old[~named].view(view), base[~named].view(view))
    if D > 1:
        check_grad(old[:, 1:], ids, dy[:, 1:], V, 0.7, f64(base[:, 1:]))


def test_gradient_without_tokens_and_large_batches():
    note("embed_grad no tokens")
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    got = L.lora_embed_grad(empty, torch.empty(0, 5, device=DEV), 9)
    assert got.shape == (9, 5) and not got.any()
    assert L.lora_embed(empty, torch.ones(3, 5, device=DEV)).shape == (0, 5)
    note("embed_grad 200000 tokens")
    # integers: every order of the additions gives the same float32
    T, V, D = 200_000, 333, 16
    torch.manual_seed(1)
    ids = torch.randint(-3, V + 3, (T,), dtype=torch.int32, device=DEV)
    dy = torch.randint(-2, 3, (T, D), device=DEV).to(BF)
    want = torch.zeros(V, D, dtype=torch.int64, device=DEV)
    ok = (ids >= 0) & (ids < V)
    want.index_add_(0, ids[ok].long(), dy[ok].long())
    assert torch.equal(L.lora_embed_grad(ids, dy, V).long(), want)


def test_table_beyond_32_bit_offsets():
    note("embed beyond 2^31 elements")
    V, D = 600_000, 4096  # 2.4e9 elements, 4.9 GB
    table = torch.empty(V, D, dtype=BF, device=DEV)
    ids = torch.tensor([0, V - 1, 550_000, V], dtype=torch.int32, device=DEV)
    for v in (0, V - 1, 550_000):
        table[v] = torch.randn(D, device=DEV).to(BF)
    got = L.lora_embed(ids, table)
    assert torch.equal(got[:3], table[ids[:3].long()]) and not got[3].any()
    dy = torch.randn(4, D, device=DEV).to(BF)
    L.lora_embed_grad(ids, dy, V, dtable=table)
    assert torch.equal(table[ids[:3].long()], dy[:3])
    assert int(torch.count_nonzero(table[1:1000])) == 0 and int(torch.count_nonzero(table[599_000:V - 1])) == 0


def test_gradient_is_the_transpose_of_the_lookup():
    """<lookup(table), dy> = <table, gradient(dy)>, and central differences of
    it (the lookup is linear, so any step is exact up to rounding)."""
    note("embed transpose")
    torch.manual_seed(4)
    T, V, D = 700, 90, 48
    ids = torch.randint(-2, V + 2, (T,), dtype=torch.int32, device=DEV)
    table, dy = torch.randn(V, D, device=DEV), torch.randn(T, D, device=DEV)
    grad = L.lora_embed_grad(ids, dy, V, 1.5)
    E = torch.randn(V, D, device=DEV)
    up, down = L.lora_embed(ids, table + E, 1.5), L.lora_embed(ids, table - E, 1.5)
    diff = ((up - down).double() / 2 * dy.double()).sum()
    want = (grad.double() * E.double()).sum()
    mag = (grad.double().abs() * E.double().abs()).sum() + (up.abs() * dy.abs()).sum().double()
    assert abs(float(diff - want)) <= float(mag) * 40 * H32
