"""AdamW over many tensors against the float64 definition, one step from a
given state (so that roundings do not compound) and over several steps.

Bounds (H = 2^-24): m and v are sums of two float32 products (at most four
roundings of the terms' magnitudes); the update alpha m / (sqrt(v) inv_root +
eps) takes m's error and at most 12 roundings, those of approximate square
roots and reciprocals counted as two; the constants are rounded once."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from oracle import train_oracle as O
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
H = 2.0 ** -24
LR, B1, B2, EPS, WD = 3e-3, 0.9, 0.99, 1e-8, 0.1
SIZES = [1, 3, 255, 256, 257, 2048, 2049, 5000, 64 * 1000, 0, 12]


def f64(t):
    return t.detach().double().cpu().numpy()


def starts(sizes):
    return np.concatenate([[0], np.cumsum([-(-n // 256) * 256 for n in sizes])]).astype(int)


def build(sizes, pt, gt, shadow, bits, seed=0, shift=0, step=7):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def rnd(n, std, dtype=F):
        return torch.randn(n + shift, device=DEV, generator=g).mul_(std).to(dtype)[shift:]

    params, grads = [rnd(n, 0.5, pt) for n in sizes], [rnd(n, 0.1, gt) for n in sizes]
    shadows = [torch.zeros(n + shift, device=DEV, dtype=BF)[shift:] if shadow else None for n in sizes]
    o = starts(sizes)
    m, v = torch.zeros(o[-1], device=DEV), torch.zeros(o[-1], device=DEV)
    for a, n in zip(o, sizes):
        m[a:a + n] = rnd(n, 0.05)
        v[a:a + n] = rnd(n, 0.1) ** 2
        # some elements and a whole block that were never touched
        m[a:a + n:7], v[a:a + n:7] = 0, 0
    m[:256], v[:256] = 0, 0
    state = dict(step=torch.full((1,), step, device=DEV, dtype=torch.int32))
    if bits == 32:
        state.update(m=m, v=v)
    else:
        for name, x in (("m", f64(m)), ("v", np.sqrt(f64(v)))):
            code, scale = O.quantise(x, name == "v")
            state[name] = torch.from_numpy(np.float32(code)).to(DEV).to(torch.float8_e4m3fn)
            state[name + "_scale"] = torch.from_numpy(np.float32(scale)).to(DEV)
    return params, grads, (shadows if shadow else None), state


def moments(state):
    """m and v that the state stands for, float64"""
    if "m_scale" not in state:
        return f64(state["m"]), f64(state["v"])
    sm, sv = (np.repeat(f64(state[k]), 256) for k in ("m_scale", "v_scale"))
    return f64(state["m"].float()) * sm, (f64(state["v"].float()) * sv) ** 2


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,gt,shadow", [(F, F, True), (F, BF, False), (BF, F, False), (BF, BF, False)])
@pytest.mark.parametrize("shift", [0, 1])
def test_one_step(bits, pt, gt, shadow, shift):
    note(f"adamw {bits} {pt} {gt} {shadow} {shift}")
    params, grads, shadows, state = build(SIZES, pt, gt, shadow, bits, shift=shift)
    if shift:  # sizes whose tensors do not start 16-byte aligned; the states do
        assert params[0].data_ptr() % 16
    before = [p.clone() for p in params]
    m0, v0 = moments(state)
    gs, ls = torch.full((), 0.5, device=DEV), torch.full((), 0.25, device=DEV)
    opt = L.AdamW(params, grads, LR, (B1, B2), EPS, WD, bits, state, shadows)
    opt.step(lr_scale=ls, grad_scale=gs)
    assert int(state["step"]) == 8 and opt.state["m"] is state["m"]
    m1, v1 = moments(state)
    lr = LR * 0.25
    for i, (a, n) in enumerate(zip(starts(SIZES), SIZES)):
        s = slice(a, a + n)
        pad = slice(a + n, starts(SIZES)[i + 1])
        assert not m1[pad].any() and not v1[pad].any()
        if n == 0:
            continue
        g, p = 0.5 * f64(grads[i]), f64(before[i])
        wp, wm, wv = O.adamw(p, g, m0[s], v0[s], 8, lr, B1, B2, EPS, WD)
        em = 4 * H * (B1 * np.abs(m0[s]) + (1 - B1) * np.abs(g))
        ev = 5 * H * wv + 1e-45
        den = np.sqrt(wv / (1 - B2 ** 8)) + EPS
        alpha = lr / (1 - B1 ** 8)
        # 8-bit moments are decoded first: a product (and a square) more, in m and v alike
        ep = alpha * (em * 2 / den + 18 * H * np.abs(wm) / den) + 3 * H * np.abs(p)
        got = f64(params[i])
        tol = ep + torch.finfo(pt).eps / 2 * np.abs(wp) * 1.01
        assert (np.abs(got - wp) <= tol).all(), (i, float((np.abs(got - wp) / tol).max()))
        if shadow:
            assert torch.equal(shadows[i], params[i].to(BF))
        if bits == 32:
            assert (np.abs(m1[s] - wm) <= em).all() and (np.abs(v1[s] - wv) <= ev).all()
            continue
        for name, got, x, ex in (("m", m1[s], wm, em * 2), ("v", np.sqrt(v1[s]), np.sqrt(wv), 8 * H * np.sqrt(wv))):
            scale = np.repeat(f64(state[name + "_scale"]), 256)[s]
            full = np.zeros(-(-n // 256) * 256)
            full[:n] = np.abs(x)
            want_scale = np.repeat(full.reshape(-1, 256).max(1) / 448, 256)[:n]
            want_scale[want_scale < 1e-30 / 448] = 0
            assert (np.abs(scale - want_scale) <= 16 * H * want_scale).all(), (name, i)
            q = np.divide(x, scale, out=np.zeros(n), where=scale > 0)
            near = np.abs(got - x) <= scale * O.e4m3_step(q * (1 + 2.0 ** -18)) / 2 + ex + 16 * H * np.abs(x)
            if name == "v":  # kept above zero
                near |= (got == scale * 2.0 ** -9) & (x > 0) & (x < scale * 2.0 ** -9)
                assert (got[x > 0] > 0).all()
            assert near.all(), (name, i)


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_are_reproducible_and_tensors_independent(bits):
    note(f"adamw reproducible {bits}")
    a = build(SIZES, F, F, True, bits, seed=5, shift=0)
    b = build(SIZES, F, F, True, bits, seed=5, shift=1)  # the same values at other addresses
    b[3].update({k: a[3][k].clone() for k in a[3]})
    for p, q, g, h in zip(a[0], b[0], a[1], b[1]):
        q.copy_(p)
        h.copy_(g)
    for params, grads, shadows, state in (a, b):
        opt = L.AdamW(params, grads, LR, (B1, B2), EPS, WD, bits, state, shadows)
        for _ in range(3):
            opt.step()
    for x, y in zip(a[0] + a[2] + list(a[3].values()), b[0] + b[2] + list(b[3].values())):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # alone, a tensor takes the same steps as among the others
    i = 7
    c = build(SIZES, F, F, True, bits, seed=5)
    o = starts(SIZES)
    one = {"step": c[3]["step"]}
    for k in c[3]:
        if k != "step":
            d = 256 if k.endswith("scale") else 1
            one[k] = c[3][k][o[i] // d:o[i + 1] // d].clone()
    opt = L.AdamW([c[0][i]], [c[1][i]], LR, (B1, B2), EPS, WD, bits, one, [c[2][i]])
    for _ in range(3):
        opt.step()
    assert torch.equal(c[0][i], a[0][i])


def test_many_tensors_from_zero_follow_float64():
    """130 tensors (several batches of the table) over 12 steps, against the
    float64 recursion: each step adds at most the one-step bound, and 0.9 and
    0.99 damp what the moments carry on (a factor of ten covers it)."""
    note("adamw 130 tensors")
    sizes = [(37 * i) % 600 + 1 for i in range(130)]
    params, grads, _, _ = build(sizes, F, F, False, 32, seed=9)
    opt = L.AdamW(params, grads, LR, (B1, B2), EPS, WD)
    p = [f64(x) for x in params]
    m, v = [np.zeros(n) for n in sizes], [np.zeros(n) for n in sizes]
    for t in range(1, 13):
        for i, g in enumerate(grads):
            g.copy_(torch.from_numpy(np.float32(np.cos(np.arange(sizes[i]) * (i + 1) + t))))
            p[i], m[i], v[i] = O.adamw(p[i], f64(g), m[i], v[i], t, LR, B1, B2, EPS, WD)
        opt.step()
    for i in range(130):
        den = np.sqrt(v[i] / (1 - B2 ** 12)) + EPS
        tol = 12 * (3 * H * (np.abs(p[i]) + 1e-2) + LR * 10 * 24 * H / den * (1 + np.abs(m[i])))
        assert (np.abs(f64(params[i]) - p[i]) <= tol).all(), i


def test_eight_bit_states_train_like_32_bit_ones():
    """A quadratic with gradients over five orders of magnitude: 8-bit moments
    (codes within 2^-4) keep each step's size within about 2^-3 of the 32-bit
    one's, so 200 steps end within a fifth of the way travelled."""
    note("adamw 8-bit training")
    torch.manual_seed(0)
    n = 5000
    target = torch.randn(n, device=DEV)
    curve = torch.logspace(-3, 2, n, device=DEV)[torch.randperm(n, device=DEV)]
    ends = []
    for bits in (32, 8):
        p, g = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
        opt = L.AdamW([p], [g], 2e-2, (0.9, 0.99), 1e-8, 0.0, bits)
        for _ in range(200):
            torch.mul(curve, p - target, out=g)
            opt.step()
        ends.append(p)
        assert torch.isfinite(p).all()
    assert float((ends[0] - ends[1]).norm() / ends[0].norm()) <= 0.2
    assert float((ends[1] - target).norm() / target.norm()) <= 0.2


def test_refusals_on_moved_and_mismatched_tensors():
    note("adamw refusals")
    p, g = torch.zeros(100, device=DEV), torch.ones(100, device=DEV)
    opt = L.AdamW([p], [g], 1e-2)
    with pytest.raises(ValueError, match="lr_scale"):
        opt.step(lr_scale=torch.ones(2, device=DEV))
    with pytest.raises(ValueError, match="grad_scale"):
        opt.step(grad_scale=torch.ones(()))
    opt.state["m"] = opt.state["m"].clone()
    with pytest.raises(ValueError, match="state"):
        opt.step()
    opt = L.AdamW([p], [g], 1e-2)
    g.data = torch.full((100,), 2.0, device=DEV)
    with pytest.raises(ValueError, match="moved"):
        opt.step()
    opt.bind([g])
    opt.step()
    assert int(opt.state["step"]) == 1 and bool((p < 0).all())
    with pytest.raises(ValueError, match="state"):
        L.AdamW([p], [g], 1e-2, state=dict(m=opt.state["m"]))
    with pytest.raises(ValueError, match="m must be"):
        L.AdamW([p], [g], 1e-2, state_bits=8, state=dict(opt.state, m_scale=p[:1], v_scale=p[:1]))
    with pytest.raises(L.LoraError):
        L.AdamW([p.half()], [g], 1e-2)
    with pytest.raises(L.LoraError):
        L.AdamW([p.to(BF)], [g], 1e-2, shadows=[p.to(BF)])


def test_table_of_other_tensors_changes_nothing_but_the_count():
    note("adamw foreign table")
    p, g = torch.zeros(1000, device=DEV), torch.ones(1000, device=DEV)
    a, b = L.AdamW([p], [g], 1e-2), L.AdamW([p[:100], p[100:200]], [g[:100], g[100:200]], 1e-2)
    table = torch.cat([b._table, torch.zeros(4096, dtype=torch.uint8, device=DEV)])
    a._table, a._table_bytes = table, table.numel()
    a.step()
    assert int(a.state["step"]) == 1 and not p.any() and not a.state["m"].any()


def test_empty_tensors_are_skipped():
    note("adamw empty")
    e = torch.zeros(0, device=DEV)
    L.AdamW([e], [e.clone()], 1e-2).step()
