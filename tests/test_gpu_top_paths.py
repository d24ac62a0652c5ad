"""Alternatives and distillation at the sizes where the library takes another
path: rows whole or in pieces, the shapes of the workgroups, lists that
overflow, rows that registers hold in part; what lies around the rows; two
calls at once. Bounds as in test_gpu_top and test_gpu_distill."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note
from tests.test_gpu_distill import bounds
from tests.test_gpu_distill import make as make_teacher
from tests.test_gpu_top import BF, F, check, check_grad, close, f64, make, ranked

pytestmark = pytest.mark.gpu
NAN = float("nan")


def framed(x, pad=9, shift=3):
    """x with NaN before, between and behind its rows (which start at any address)."""
    T, V = x.shape
    buf = torch.full((T * (V + pad) + shift + pad,), NAN, device=DEV, dtype=x.dtype)
    out = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    out.copy_(x)
    return out


# rows, columns, k: one piece with 4 waves and short or long lists, with 8, pieces because the list has no room for
# more, few rows in pieces, a long vocabulary, very few rows with 16 waves and what lies beside that
TOPS = [(192, 49153, 1), (192, 49153, 20), (200, 32003, 64), (195, 70001, 20), (193, 128256, 100), (192, 128256, 128),
        (190, 60000, 20), (3, 300007, 64), (2, 49152, 128), (1, 2 ** 20 + 3, 5), (600, 3001, 128),
        (1, 49153, 1), (4, 128256, 64), (3, 131071, 20), (5, 128256, 64), (2, 131073, 20), (1, 131072, 65),
        (5, 2047, 128), (5, 1023, 128), (300, 2041, 127)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V,k", TOPS)
def test_alternatives(dtype, T, V, k):
    note(f"top paths {dtype} {T} {V} {k}")
    x, y = make(T, V, dtype, T + V + k)
    x = framed(x)
    out = L.lora_token_top(x, y, k, 0.9)
    live = ((y >= 0) & (y < V))[:, None]
    assert torch.equal(out[2], torch.where(live, ranked(x, k), -1))
    at = torch.tensor(sorted({0, 1, T // 2, T - 2, T - 1} & set(range(T))), device=DEV)
    check(x[at], y[at], k, 0.9, tuple(t[at] for t in out))
    again = L.lora_token_top(x, y, k, 0.9)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("V,k", [(49153, 1), (50000, 20), (128256, 20), (128256, 64), (128256, 128)])
def test_lists_that_overflow(dtype, V, k):
    """Many rows, so that one workgroup takes a long one: logits that rise along the row, in steps, behind a masked
    beginning, with all of the largest at one lane's places, equal throughout, or masked down to a few."""
    note(f"top overflow {dtype} {V} {k}")
    g = torch.Generator(device=DEV)
    g.manual_seed(V + k)
    n = torch.arange(V, device=DEV, dtype=torch.float32)
    rows = [n / V * 30 - 15, torch.floor(n / 5000), -n / V * 30, torch.zeros(V, device=DEV), (n // 8 % 512 == 5) * 3.0,
            torch.where(n < V // 2, -float("inf"), torch.randn(V, device=DEV, generator=g)),
            torch.where(n < V // 2, torch.finfo(dtype).min, torch.randn(V, device=DEV, generator=g)),
            torch.where(n % 997 == 3, torch.randn(V, device=DEV, generator=g), -float("inf")),
            torch.where(n == V - 2, 2.0, -float("inf")), torch.where(n > V - 40, n, torch.finfo(dtype).min),
            torch.randn(V, device=DEV, generator=g) * 1e-4, n / V * 2e5]
    x = torch.stack(rows).to(dtype)
    x = x.repeat(17, 1)[:200].contiguous()
    out = L.lora_token_top(x, None, k, 1.0)
    assert torch.equal(out[2], ranked(x, k))
    d = x[:12].double() - x[:12].double().amax(1, keepdim=True)
    lse = torch.logsumexp(d, 1, keepdim=True)
    p = torch.exp(d - lse)
    gap = torch.where(p > 0, -p * d, 0.0).sum(1, keepdim=True)
    # terms relative to a logit up to 64 binary orders below the largest: 3 H (u + 45) + 2^-23 + 16 H each
    H = 2.0 ** -24
    step = 3 * H * (torch.where(p > 0, -d, 0.0) + 45) + 2.0 ** -23 + 16 * H
    e = (p * step).sum(1, keepdim=True) + H
    want = d.gather(1, out[2][:12].long()) - lse
    close(f64(out[3][:12]), f64(want), f64(e) + 2 * H * np.abs(f64(want)), "top")
    e_gap = torch.where(p > 0, p * (-d * step + 3 * H * (45 - d)), 0.0).sum(1, keepdim=True) + gap * e + H * gap
    close(f64(out[1][:12]), f64(lse + gap)[:, 0], f64(e + e_gap + H * (lse + gap))[:, 0], "entropy")
    for t in out[1:]:
        assert all(torch.equal(t[:12], t[i:i + 12]) for i in range(12, 192, 12))
    # very few rows at a time
    for i in range(0, 12, 3):
        few = L.lora_token_top(x[i:i + 3], None, k, 1.0)
        assert torch.equal(few[2], out[2][i:i + 3])
        close(f64(few[3]), f64(want[i:i + 3]), (f64(e) + 2 * H * np.abs(f64(want)))[i:i + 3], "top of few")
        close(f64(few[1]), f64(lse + gap)[i:i + 3, 0], f64(e + e_gap + H * (lse + gap))[i:i + 3, 0], "entropy of few")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 9, 198])
@pytest.mark.parametrize("V,k", [(3001, 5), (128256, 20)])
def test_logits_far_from_zero(dtype, T, V, k):
    """Logits around 3e7, 1e10, -1e10 and 1e20, and a few far below zero behind a masked beginning."""
    note(f"top far from zero {dtype} {T} {V} {k}")
    g = torch.Generator(device=DEV)
    g.manual_seed(V + k)
    n = torch.arange(V, device=DEV)
    r = torch.randn(V, device=DEV, generator=g)
    few = (n > V // 2) & (n % (V // 250) == 1)
    rows = [3e7 + 8 * r, 1e10 + 4096 * r, -1e10 + 4096 * r, 1e20 + 1e14 * r, 3e5 + r] + [
        torch.where(few, c + r, -float("inf")) for c in (-60.0, -100.0, -2000.0, 1e9)]
    x = torch.stack(rows).to(dtype).repeat(max(1, T // 9), 1).contiguous()
    y = x.argmax(1).to(torch.int32)
    y[3::9] = int(few.nonzero()[1])
    if T == 1:  # a call for each row
        parts = [L.lora_token_top(x[i:i + 1], y[i:i + 1], k, 0.7) for i in range(9)]
        out = tuple(torch.cat(p) for p in zip(*parts))
    else:
        out = L.lora_token_top(x, y, k, 0.7)
    assert torch.equal(out[2], ranked(x, k))
    check(x[:9], y[:9], k, 0.7, tuple(t[:9] for t in out))
    for t in out:
        assert all(torch.equal(t[:9], t[i:i + 9]) for i in range(9, T, 9))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("k", [0, 5, 100])
@pytest.mark.parametrize("T", [2, 8, 200])
def test_undefined_rows(dtype, T, k):
    """NaN and infinities in rows of 16 waves, in rows of pieces (some of a piece whole) and in rows of one."""
    note(f"top undefined {dtype} {T} {k}")
    V = 128256
    x, _ = make(8, V, dtype, 5)
    x[0] = -float("inf")
    x[1, V // 3] = float("inf")
    x[2, V - 1] = NAN
    x[3] = NAN
    x[4, 50000:70000] = float("inf")
    x[5, 50000:70000] = NAN
    x[6, :V - 3] = -float("inf")
    y = torch.full((8,), V - 2, device=DEV, dtype=torch.int32)
    if T < 8:
        parts = [L.lora_token_top(x[i:i + T], y[i:i + T], k, 1.5) for i in range(0, 8, T)]
        out = tuple(torch.cat(p) for p in zip(*parts))
    else:
        out = L.lora_token_top(x.repeat(T // 8, 1), y.repeat(T // 8), k, 1.5)
    for t in out:
        for i in range(0, len(t), 8):
            assert ((t[i:i + 6] == -1).all() if t.dtype == torch.int32 else torch.isnan(t[i:i + 6]).all())
            assert torch.equal(t[i + 6:i + 8], t[6:8])
    check(x[6:], y[6:], k, 1.5, tuple(t[6:8] for t in out))


# rows that registers hold in part or whole, the same in pieces, rows longer than one workgroup takes
DISTILLS = [(112, 70003, 64), (130, 128256, 33), (64, 40009, 100), (70, 128259, 8), (111, 128256, 16), (63, 50001, 256),
            (3, 262144, 5), (2, 300007, 64), (120, 20481, 3), (1, 49152, 1), (5, 8, 3), (256, 128256, 64),
             (257, 70001, 5), (113, 114696, 7), (112, 131100, 256), (64, 130001, 3)]


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V,k", DISTILLS)
def test_distillation(dtype, rest, T, V, k):
    note(f"distill paths {dtype} {rest} {T} {V} {k}")
    x, ids, logp = make_teacher(T, V, k, dtype, 1.3, T + V + k)
    x = framed(x)
    w = torch.rand(T, device=DEV) + 0.1
    at = torch.tensor(sorted({0, 1, 2, T // 2, T - 1} & set(range(T))), device=DEV)
    c64 = f64(w[at])
    want, e_kl, dx, e_dx = bounds(f64(x[at]), ids[at].cpu().numpy(), f64(logp[at]), 1.3, rest, c64, dtype)
    out = framed(torch.zeros_like(x))
    loss, kl, got = L.lora_distill_step(x, ids, logp, w, 1.3, rest, dlogits=out)
    close(f64(kl[at]), want, e_kl, "kl")
    close(f64(got[at]), dx, e_dx, "dx")
    assert torch.isfinite(got).all() and abs(float(loss) - float((w.double() * kl.double()).sum())) <= (
        2.0 ** -24 * float((w * kl).abs().sum()))
    alone, state = L.lora_distill_kl(x, ids, logp, 1.3, rest)
    close(f64(alone[at]), want, e_kl, "kl alone")
    close(f64(L.lora_distill_grad(x, ids, state, w, 1.3)[at]), dx, e_dx, "dx of the state")
    # in place, and what lies around the rows
    frame = x._base if x._base is not None else x
    edge = torch.isnan(frame)
    L.lora_distill_step(x, ids, logp, w, 1.3, rest, dlogits=x)
    assert torch.equal(x, got) and torch.equal(torch.isnan(frame), edge)


@pytest.mark.parametrize("dtype", [BF, F])
def test_far_logits(dtype):
    """Others far below the teacher's tokens, a largest one far behind a row's beginning, and a masked beginning."""
    note(f"distill far {dtype}")
    T, V, k = 115, 70003, 6
    x, ids, logp = make_teacher(T, V, k, dtype, 1.0, 8)
    ids[2:5], logp[2:5] = ids[5], logp[5]
    x[2] = 0.0
    x[2, V - 3] = 100.0
    x[3, :V // 2] = -float("inf")
    x[4, :V // 2] = torch.finfo(dtype).min
    x[:, ids[5, 0].long()] = 3.0
    x.scatter_add_(1, ids.clamp(0, V - 1).long(), torch.full(ids.shape, 40.0, device=DEV, dtype=dtype))
    at = [1, 2, 3, 4, 7]
    w = torch.ones(T, device=DEV)
    want, e_kl, dx, e_dx = bounds(f64(x)[at], ids.cpu().numpy()[at], f64(logp)[at], 1.0, True, np.ones(5), dtype)
    for rows in (slice(None), slice(0, 9)):  # by rows, in pieces
        _, kl, got = L.lora_distill_step(x[rows], ids[rows], logp[rows], w[rows])
        close(f64(kl)[at], want, e_kl)
        close(f64(got)[at], dx, e_dx)


def test_two_calls_at_once():
    note("two streams at once")
    T, V, k = 40, 128256, 20
    x, y = make(T, V, BF, 1)
    t, ids, logp = make_teacher(T, V, k, BF, seed=2)
    w = torch.rand(T, device=DEV)
    want = L.lora_token_top(x, y, k), L.lora_distill_step(t, ids, logp, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            got[0].append(L.lora_token_top(x, y, k))
        with torch.cuda.stream(streams[1]):
            got[1].append(L.lora_distill_step(t, ids, logp, w))
    torch.cuda.synchronize()
    for one, all_ in zip(want, got):
        for other in all_:
            assert all(torch.equal(a, b) for a, b in zip(one, other))


def test_gradients_of_shared_rows():
    """One row of logits broadcast to all (a stride of zero is refused), and one target and id for all."""
    note("broadcast rows")
    x, y = make(1, 5000, F, 3)
    wide = x.expand(6, 5000)
    y = y.expand(6).contiguous()
    with pytest.raises(L.LoraError) as e:
        L.lora_token_top(wide, y, 3)
    assert e.value.status == -4
    out = L.lora_token_top(wide.contiguous(), y, 3, 1.0)
    g = torch.randn(6, device=DEV)
    dx = L.lora_token_top_grad(wide.contiguous(), y, out[4], g, g, 1.0)
    check_grad(dx, f64(wide), y.cpu().numpy(), f64(g), f64(g), 1.0, F)


@pytest.mark.parametrize("tau", [1e-6, 0.01, 60.0, 1e6])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V", [(6, 3000), (5, 50001), (195, 70001)])
def test_temperatures(dtype, T, V, tau):
    note(f"temperatures {dtype} {T} {V} {tau}")
    k = 12
    x, y = make(T, V, dtype, 7)
    out = L.lora_token_top(x, y, k, tau)
    at = torch.tensor([0, 1, 2, T - 1], device=DEV)
    check(x[at], y[at], k, tau, tuple(t[at] for t in out))
    g = torch.randn(T, device=DEV)
    dx = L.lora_token_top_grad(x, y, out[4], g, g, tau)
    check_grad(dx[at], f64(x[at]), y[at].cpu().numpy(), f64(g[at]), f64(g[at]), tau, dtype)
    x, ids, logp = make_teacher(T, V, k, dtype, tau, 9)
    for rest in (True, False):
        want, e_kl, wx, ex = bounds(f64(x[at]), ids[at].cpu().numpy(), f64(logp[at]), tau, rest, f64(g[at]), dtype)
        _, kl, dx = L.lora_distill_step(x, ids, logp, g, tau, rest)
        close(f64(kl[at]), want, e_kl, "kl")
        close(f64(dx[at]), wx, ex, "dx")
