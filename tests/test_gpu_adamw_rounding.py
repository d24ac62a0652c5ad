"""AdamW's roots, quotients and 8-bit codes are those of correctly rounded
float32 operations, bit for bit. With beta1 = 0, beta2 = 1/2, a step count that
leaves no bias correction, no decay and parameters of 0 every operation of the
update but these is exact or one that numpy rounds alike:
    m = g,  v = (v + g g) / 2,  p = -(lr m / (sqrt(v) + eps))
An 8-bit moment's block has the scale max / 448 and the codes of
x * (448 / max)."""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu
F = np.float32


def moments(n, rng):
    """Gradients and second moments over many binades; blocks of one size of magnitude, ties of the codes (the
    largest is 448 / 1024: 1024 x falls between two codes), zeros, and values whose squares are denormal."""
    g = (rng.normal(size=n) * np.exp(rng.uniform(-30, 4, n))).astype(F)
    v = (rng.normal(size=n) ** 2 * np.exp(rng.uniform(-40, 5, n))).astype(F)
    g[:256] = (np.arange(256) % 64 + 64 + 0.5 * (np.arange(256) % 2)) * F(2.0) ** rng.integers(-10, -4, 256) / 1024
    g[0] = 448 / 1024
    g[256:512] = 0
    g[512:768] *= F(1e-22)
    g[768:1024] = rng.normal(size=256)
    return g, v


def update(g, v, lr, eps):
    v = (v + g * g) * F(0.5)
    root = np.sqrt(v)
    return -(F(lr) * g / (root + F(eps))), v, root


@pytest.mark.parametrize("n", [16_000, 3_000_000])  # in one workgroup, and in the grid
def test_quotient_and_root(n):
    note(f"adamw rounding {n}")
    g, v = moments(n, np.random.default_rng(n))
    v[512:768] = np.abs(v[512:768]) * F(1e-38)
    lr, eps = 0.3, 1e-3
    for eps in (1e-3, 1e-20):
        state = dict(step=torch.full((1,), 200, dtype=torch.int32, device=DEV), m=torch.zeros(-(-n // 256) * 256, device=DEV))
        state["v"] = torch.zeros_like(state["m"])
        state["v"][:n] = torch.from_numpy(v).to(DEV)
        p = torch.zeros(n, device=DEV)
        L.AdamW([p], [torch.from_numpy(g).to(DEV)], lr, (0.0, 0.5), eps, 0.0, state=state).step()
        want, second, _ = update(g, v, lr, eps)
        assert np.array_equal(state["m"][:n].cpu().numpy(), g)
        got = state["v"][:n].cpu().numpy()
        normal = (second >= 2.0 ** -126) & (g * g >= 2.0 ** -126)  # a denormal square or half is rounded otherwise
        assert np.array_equal(got[normal], second[normal])
        want, _, _ = -(F(lr) * g / (np.sqrt(got) + F(eps))), None, None
        got = p.cpu().numpy()
        normal = (np.abs(want) >= 2.0 ** -126) | (want == 0)
        assert normal.mean() > 0.9 and np.array_equal(got[normal], want[normal])
        assert (np.abs(got - want) <= 2.0 ** -149).all()


@pytest.mark.parametrize("n", [16_000, 3_000_000])
def test_codes_and_scales(n):
    note(f"adamw codes {n}")
    rng = np.random.default_rng(n + 1)
    g, _ = moments(n, rng)
    p = torch.zeros(n, device=DEV)
    opt = L.AdamW([p], [torch.from_numpy(g).to(DEV)], 0.3, (0.0, 0.5), 1e-3, 0.0, state_bits=8)
    opt.state["step"].fill_(200)
    opt.step()
    square = g * g
    root = np.sqrt(square * F(0.5))
    blocks = -(-n // 256)
    for name, x in (("m", g), ("v", root)):
        b = np.zeros(blocks * 256, F)
        b[:n] = x
        b = b.reshape(-1, 256)
        amax = np.abs(b).max(1)
        some = amax >= F(1e-30)
        safe = np.where(some, amax, F(1))
        scale = np.where(some, safe / F(448), F(0))
        assert np.array_equal(opt.state[name + "_scale"].cpu().numpy(), scale), name
        q = b * np.where(some, F(448) / safe, F(0))[:, None]
        if name == "v":
            q = np.where(q > 0, np.maximum(q, F(2.0 ** -9)), q)
        want = torch.from_numpy(q.reshape(-1)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        got = opt.state[name].view(torch.uint8).cpu().numpy()
        # the squares of tiny gradients are denormal: their halves may be rounded otherwise
        sure = np.ones(blocks * 256, bool)
        if name == "v":
            sure[:n] = (square >= 2.0 ** -125) | (square == 0)
        assert sure.mean() > 0.9 and np.array_equal(got[sure], want[sure]), name
