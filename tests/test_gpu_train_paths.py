"""The training operators where their kernels change over: rows taken whole,
in halves or in pieces; few chunks and many; lists that overflow; rows beyond
32-bit offsets; other streams; captured steps replayed. Bounds as derived in
the tests of each operator."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from oracle import train_oracle as O
from tests.gpu_util import DEV, note
from tests.test_gpu_embed import check_grad, make_ids
from tests.test_gpu_loss import BF, F, H, close, f64, grad_bounds, make, row_bounds

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# policy step: 4, 8 or 16 waves to a row, or pieces of few long rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,T,V", [(BF, 6, 12288), (BF, 6, 12295), (F, 6, 6144), (F, 6, 6151), (BF, 5, 49152),
                                       (BF, 5, 49159), (BF, 127, 49160), (BF, 128, 49160), (F, 9, 24576),
                                       (F, 9, 24581), (F, 127, 49153), (BF, 130, 60001), (BF, 3, 300007)])
def test_policy_step_changes_over(dtype, T, V):
    note(f"policy changes over {dtype} {T} {V}")
    torch.manual_seed(T + V)
    x, y = make(T, V, dtype, T + V, pad=1, shift=1)
    masked = torch.from_numpy(O.masked(y.cpu().numpy(), V)).to(DEV)
    lp, _ = L.lora_token_logp(x, y)
    old, ref = lp + torch.randn(T, device=DEV) * 0.3, lp + torch.randn(T, device=DEV) * 0.5
    adv, w = torch.randn(T, device=DEV), torch.rand(T, device=DEV)
    for t in (old, ref, adv, w):
        t[masked] = float("nan")
    args = (old, adv, w, 0.2, 0.3, ref, 0.1)
    loss, logp, dx = L.lora_policy_step(x, y, *args, grad_scale=0.5)
    x64, yn = f64(x), y.cpu().numpy()
    close(f64(logp), O.token_logp(x64, yn), row_bounds(x64, yn)[1], "logp")
    # the coefficient of a log probability is the same bits in every kernel
    loss2, coef = L.lora_policy_loss(logp, y, V, *args)
    # each token's loss is rounded a few times in either kernel, their sum is float64
    terms = np.abs(f64(w)) * (3 * np.abs(f64(adv)) + 1)
    assert abs(float(loss) - float(loss2)) <= 32 * H * np.nansum(terms)
    want, tol = grad_bounds(x64, yn, 0.5 * f64(coef), dtype)
    close(f64(dx), want, tol + 16 * H * np.abs(want), "dx")
    assert not dx[masked].any()
    L.lora_policy_step(x, y, *args, grad_scale=0.5, dlogits=x)
    assert torch.equal(x, dx)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("V", [40, 9001, 50001])
def test_policy_step_infinities_and_masked_vocabulary(dtype, V):
    """The rows that token_logp's test has; the step gives NaN where it does, and its values elsewhere."""
    note(f"policy infinities {dtype} {V}")
    x, _ = make(8, V, dtype, 3)
    low = torch.finfo(dtype).min
    y = torch.tensor([2, 2, 2, 2, 2, -1, 2, 3], dtype=torch.int32, device=DEV)
    x[0, 5:] = -float("inf")
    x[1, 5:] = low
    x[2] = -float("inf")
    x[3] = low
    x[4, 7] = float("inf")
    x[5] = float("nan")
    x[6, V - 1] = float("nan")
    x[7] = -float("inf")
    x[7, 3] = low
    zero, one = torch.zeros(8, device=DEV), torch.ones(8, device=DEV)
    lp, stats = L.lora_token_logp(x, y)
    # advantage 0 and a KL term with ref = logp - 1: the coefficient is -kl * expm1(-1) = 1 for every token
    kl = float(-1 / np.expm1(-1))
    loss, logp, dx = L.lora_policy_step(x, y, lp, zero, one, 0.2, 0.2, lp - 1, kl)
    want = L.lora_logit_grad(x, y, stats, one)
    nan = [2, 4, 6]
    rest = [0, 1, 3, 5, 7]
    assert torch.isnan(logp[nan]).all() and torch.isnan(dx[nan]).all() and torch.isnan(loss)
    S = 2 * (V / 64 + 64) * H
    close(f64(logp[rest]), f64(lp[rest]), 2 * S + 8 * H * np.abs(f64(lp[rest])))
    close(f64(dx[rest]), f64(want[rest]), (4 * S + 64 * H + torch.finfo(dtype).eps) * np.abs(f64(want[rest])) + 1e-37)
    assert not dx[5].any() and logp[5] == 0
    # with the rows that give NaN masked, the loss is a number
    y[nan] = -100
    loss, _, _ = L.lora_policy_step(x, y, lp, zero, one, 0.2, 0.2, lp - 1, kl)
    assert torch.isfinite(loss)


def test_policy_rows_beyond_32_bit_offsets():
    note("policy rows beyond 2^31 elements")
    T, V = 40_000, 65_000  # 2.6e9 elements
    x = torch.zeros(T, V, dtype=BF, device=DEV)
    y = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    rows = [0, 36_000, T - 1]
    for r in rows:
        x[r] = torch.randn(V, device=DEV).to(BF)
        y[r] = V - 1 - r % 7
    x64, yn = f64(x[rows]), y[rows].cpu().numpy()
    one, old = torch.ones(T, device=DEV), torch.zeros(T, device=DEV)
    lp = O.token_logp(x64, yn)
    old[rows] = torch.from_numpy(np.float32(lp)).to(DEV)  # the ratio is 1 up to rounding: coefficient -1
    _, logp, _ = L.lora_policy_step(x, y, old, one, one, 0.2, 0.2, dlogits=x)
    err = row_bounds(x64, yn)[1]
    close(f64(logp[rows]), lp, err)
    want, tol = grad_bounds(x64, yn, -np.ones(3), BF)
    drift = (err + H * np.abs(lp))[:, None] * 1.01 + 8 * H
    close(f64(x[rows]), want, tol + drift * np.abs(want) * 1.01)
    assert not x[35_000:36_000].any()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V", [(6, 128256), (130, 128256), (2100, 20000), (3, 40000)])
def test_confident_tokens_keep_the_rest_of_the_vocabulary(dtype, T, V):
    """A target far above the others: the sum is 1 and V terms of about 1e-7, each
    below half a step of 1. A batch of 32 meets the 1 in at most five additions of
    its tree, everything else is added in float64 or among its like (2^-21 of the
    tail, at most), and the logarithm is rounded once."""
    note(f"confident {dtype} {T} {V}")
    torch.manual_seed(T)
    x = torch.randn(T, V, device=DEV).mul_(2.0).to(dtype)
    y = torch.randint(0, V, (T,), device=DEV, dtype=torch.int32)
    x[torch.arange(T, device=DEV), y.long()] = 18.0
    rows = list(range(min(T, 40)))
    want = O.token_logp(f64(x[rows]), y[rows].cpu().numpy())
    zero, one = torch.zeros(T, device=DEV), torch.ones(T, device=DEV)
    tol = 6 * H + 2.0 ** -19 * np.abs(want) + H * np.abs(want)
    close(f64(L.lora_token_logp(x, y)[0][rows]), want, tol, "token_logp")
    close(f64(L.lora_policy_step(x, y, zero, one, one, 0.2, 0.2)[1][rows]), want, tol, "policy_step")
    off = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    close(f64(L.lora_pref_step(x, y, off, torch.zeros(2, device=DEV), 0.1)[2][rows]), want, tol, "pref_step")


# ---------------------------------------------------------------------------
# preference step: rows whole or in pieces, joined with the loss or before it
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,V,pairs", [(255, 9000, 3), (256, 9000, 1), (257, 9000, 2), (682, 8200, 4),
                                       (683, 8200, 4), (1365, 8200, 4), (1, 128256, 1), (12, 270000, 2)])
def test_pref_step_changes_over(T, V, pairs):
    note(f"pref changes over {T} {V} {pairs}")
    rng = np.random.default_rng(T + V)
    x, y = make(T, V, BF, T + V)
    off = np.sort(rng.integers(0, T + 1, 2 * pairs + 1)).astype(np.int32)
    x64, yn = f64(x), y.cpu().numpy()
    logp64 = O.token_logp(x64, yn)
    seq = np.array([logp64[a:b].sum() for a, b in zip(off[:-1], off[1:])])
    ref = torch.from_numpy(np.float32(seq + rng.normal(size=2 * pairs) * 5)).to(DEV)
    loss, s, logp, dx = L.lora_pref_step(x, y, torch.from_numpy(off).to(DEV), ref, 0.1, 0.1)
    err = row_bounds(x64, yn)[1]
    close(f64(logp), logp64, err, "logp")
    err_seq = np.array([err[a:b].sum() for a, b in zip(off[:-1], off[1:])]) + np.abs(seq) * 1.01 * H
    close(f64(s), seq, err_seq, "seq")
    b = np.float64(np.float32(0.1))
    want_loss, _, coef = O.pref_loss(logp64, off, f64(ref), b, b)
    close(f64(loss), want_loss, b * err_seq.sum() + H * abs(want_loss) + 1e-12, "loss")
    moved = np.abs(coef) * 1.01 * H + b / pairs * (b * err_seq.sum()) / 4 * (coef != 0)
    want, tol = grad_bounds(x64, yn, coef, BF)
    most = np.maximum(np.abs(O.logit_grad(x64, yn, np.ones(T))), O.softmax(x64))
    close(f64(dx), want, tol + 2 * moved[:, None] * most * 1.01, "dx")
    L.lora_pref_step(x, y, torch.from_numpy(off).to(DEV), ref, 0.1, 0.1, dlogits=x)
    assert torch.equal(x, dx)


# ---------------------------------------------------------------------------
# table gradient: lists in shared memory and beyond them, many ids
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,V,kind", [(40_000, 1000, "same"), (40_000, 5, "zipf"), (16_384, 128_256, "zipf"),
                                      (16_385, 131_072, "zipf"), (20_000, 131_073, "distinct"), (9, 1, "zipf"),
                                      (7, 4, "distinct"), (8, 2, "same"), (3000, 700_001, "zipf")])
def test_gradient_lists(T, V, kind):
    note(f"embed_grad lists {T} {V} {kind}")
    torch.manual_seed(T)
    ids = make_ids(T, V, kind, np.random.default_rng(T + V))
    D = 4
    # integers: every order of the additions gives the same float32
    dy = torch.randint(-2, 3, (T, D), device=DEV).to(BF)
    want = torch.zeros(V, D, dtype=torch.int64, device=DEV)
    ok = (ids >= 0) & (ids < V)
    want.index_add_(0, ids[ok].long(), dy[ok].long())
    assert torch.equal(L.lora_embed_grad(ids, dy, V).long(), want)
    if V <= 5000:
        real = torch.randn(T, D, device=DEV)
        check_grad(L.lora_embed_grad(ids, real, V, 0.7), ids, real, V, 0.7)


@pytest.mark.parametrize("types", [(F, F), (BF, F), (BF, BF)])
@pytest.mark.parametrize("T", [1, 8, 63, 64, 65, 257])
@pytest.mark.parametrize("V,D,kind", [(700, 37, "zipf"), (3, 2100, "zipf"), (5000, 64, "same"), (90, 9, "outside")])
def test_gradient_of_few_tokens(types, T, V, D, kind):
    note(f"embed_grad few {types} {T} {V} {D} {kind}")
    torch.manual_seed(T + V)
    ids = make_ids(T, V, kind, np.random.default_rng(T + V))
    dy = torch.randn(T, D + 3, device=DEV).to(types[0])[:, :D]
    out = torch.full((V, D + 1), 7.0, device=DEV, dtype=types[1])[:, :D]
    got = L.lora_embed_grad(ids, dy, V, 0.7, dtable=out)
    check_grad(got, ids, dy, V, 0.7)
    assert bool((out._base[:, D] == 7.0).all())
    assert torch.equal(got, L.lora_embed_grad(ids, dy, V, 0.7, dtype=types[1]))
    old = torch.randn(V, D, device=DEV).to(types[1])
    base = old.clone()
    L.lora_embed_grad(ids, dy, V, 0.7, dtable=old, accumulate=True)
    check_grad(old, ids, dy, V, 0.7, f64(base))


# ---------------------------------------------------------------------------
# AdamW: few chunks in one workgroup, more in the grid; tiny moments
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [32, 8])
def test_few_and_many_chunks_take_the_same_steps(bits):
    note(f"adamw few and many {bits}")
    sizes = [16 * 1024 - 300, 200]  # 16 and 1 chunks of 1024: alone within the one-workgroup form, together beyond
    torch.manual_seed(3)
    p, g = [torch.randn(n, device=DEV) for n in sizes], [torch.randn(n, device=DEV) for n in sizes]
    alone = p[0].clone()
    both = L.AdamW(p, g, 1e-2, state_bits=bits)
    one = L.AdamW([alone], [g[0]], 1e-2, state_bits=bits)
    for _ in range(3):
        both.step()
        one.step()
    n = one.state["m"].numel()
    assert torch.equal(p[0], alone)
    for k in ("m", "v"):
        assert torch.equal(both.state[k][:n].view(torch.uint8), one.state[k].view(torch.uint8))


def test_tiny_moments_keep_their_ratio():
    """v down to denormal floats: m / sqrt(v) is 1 before and after a step without gradient, up to the roundings
    (v itself is held to half of its last place, 2^-149)."""
    note("adamw tiny moments")
    v = torch.tensor([1e-44, 3e-42, 1e-39, 1e-37, 1e-30, 1e-10], device=DEV)
    n = 256
    state = dict(step=torch.full((1,), 5, device=DEV, dtype=torch.int32), v=torch.zeros(n, device=DEV),
                 m=torch.zeros(n, device=DEV))
    state["v"][:6], state["m"][:6] = v, v.double().sqrt().float()
    m0, v0 = f64(state["m"]), f64(state["v"])
    p, g = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    L.AdamW([p], [g], 1.0, (0.9, 0.99), 1e-30, 0.0, state=state).step()
    want, _, wv = O.adamw(np.zeros(n), np.zeros(n), m0, v0, 6, 1.0, 0.9, 0.99, 1e-30, 0.0)
    held = 2.0 ** -150 / np.maximum(wv, 1e-45)  # of v, half of it in its root
    assert (np.abs(f64(p) - want) <= (40 * H + held) * np.abs(want) + 1e-37).all()


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------

class Step:
    """Every operator once, on buffers that stay."""

    def __init__(self, T=90, V=9001, D=64, bits=32, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.x, self.y = make(T, V, BF, seed)
        self.ids = torch.randint(-1, 500, (T,), device=DEV, dtype=torch.int32, generator=g)
        self.table = torch.randn(500, D, device=DEV, generator=g)
        self.off = torch.tensor([0, 20, 45, 70, 90], device=DEV, dtype=torch.int32)
        self.ref = torch.randn(4, device=DEV, generator=g)
        self.f = [torch.randn(T, device=DEV, generator=g) * 0.1 - 4 for _ in range(2)]
        self.adv, self.w = torch.randn(T, device=DEV, generator=g), torch.rand(T, device=DEV, generator=g)
        self.grads = [torch.empty(500, D, device=DEV)]
        self.shadow = torch.empty(500, D, device=DEV, dtype=BF)
        self.opt = L.AdamW([self.table], self.grads, 1e-2, state_bits=bits, shadows=[self.shadow])

    def run(self):
        e = L.lora_embed(self.ids, self.table, 0.5)
        a = L.lora_pref_step(self.x, self.y, self.off, self.ref, 0.1)
        b = L.lora_policy_step(self.x, self.y, self.f[0], self.adv, self.w, 0.2, 0.2, self.f[1], 0.1)
        L.lora_embed_grad(self.ids, e, 500, dtable=self.grads[0])
        self.opt.step()
        return [e, *a, *b, self.grads[0], self.table, self.shadow, *self.opt.state.values()]


def same(a, b):
    return all(torch.equal(x.reshape(-1).view(torch.uint8), y.reshape(-1).view(torch.uint8))
               for x, y in zip(a, b, strict=True))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_replays(bits):
    note(f"captured step {bits}")
    eager, held = Step(bits=bits), Step(bits=bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        held.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = held.run()
    eager.run()
    for i in range(4):
        # new inputs between the replays, eager work of the library and a synchronisation
        for s in (eager, held):
            s.x.mul_(0.9)
            s.adv.neg_()
        want = [t.clone() for t in eager.run()]
        graph.replay()
        torch.cuda.synchronize()
        assert same(outs, want), i


def test_other_streams():
    """Work queued on the stream that is current when a call is made, in order with torch's own work there."""
    note("side stream")
    want = [t.clone() for t in Step().run()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = Step()
    keep = s.x.clone()
    s.x.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(10):
            big = big @ big * 1e-2  # holds the stream up
        s.x.copy_(keep)
        got = s.run()
        got = [t.clone() for t in got]
    side.synchronize()
    assert same(got, want)
