"""Alternatives and entropy keep their precision wherever in a row the likely
tokens lie: a few comparable ones far above everything the row begins with.

Bounds (H = 2^-24; u = (m - x) / tau for a row's largest logit m). No exponent
depends on where a logit lies. A likely token's is a difference from the
largest logit of its part of the row, rounded, and its products with log2(e) /
tau (3 H u), the exponential (2 H), a tree of eight terms (3 H) and the factor
that joins the parts, whose own exponent 3 H u covers as well (2 H): 7 H + 3 H u.
The others are summed as everywhere, 18 H + 3 H u:
    err(r) <= sum over the others of e^-u_j e_j + H r
    err(log1p(r)) <= err(r) / (1 + r)
    err(gap) <= sum p_j (u_j e_j + 3 H u_j) + gap err(r) / (1 + r) + H gap
    err(logp) <= err(log1p(r)) + 2 H |logp|
    err(entropy) <= err(log1p(r)) + err(gap) + H entropy"""
import numpy as np
import pytest
import torch

import lora_rank_adapter_amd as L
from oracle import train_oracle as O
from tests.gpu_util import DEV, note
from tests.test_gpu_top import BF, F, H, close, f64

pytestmark = pytest.mark.gpu


def peaked(T, V, dtype, above, tau, seed, peaks=4):
    """(logits, columns of the peaks): noise, and in the row's last third a few tokens `above` it over tau."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(T, V, device=DEV, generator=g) * 0.5
    at = torch.rand(T, V // 3, device=DEV, generator=g).topk(peaks, 1).indices + (V - V // 3)
    high = (above + torch.rand(T, peaks, device=DEV, generator=g)) * tau
    return x.scatter_(1, at, high).to(dtype), at


# one piece by 4, by 8 and by 16 waves, pieces of 18000 logits
@pytest.mark.parametrize("T,V,k", [(64, 40000, 8), (200, 40000, 0), (200, 128256, 20), (2, 128256, 5), (150, 128256, 20)])
@pytest.mark.parametrize("above", [25.0, 40.0])
@pytest.mark.parametrize("dtype", [BF, F])
def test_likely_tokens_late_in_a_row(dtype, above, T, V, k):
    note(f"late peaks {dtype} {above} {T} {V} {k}")
    tau = (1.0, 0.7)[V % 3 == 0]
    x, at = peaked(T, V, dtype, above, tau, V + T + int(above))
    rows = min(T, 48)
    out = [t[:rows] for t in L.lora_token_top(x, at[:, 0].int().contiguous(), k, tau)]
    x64, y = f64(x[:rows]), at[:rows, 0].cpu().numpy()
    logp, entropy, ids, top, stats = O.token_top(x64, y, k, tau)
    r, gap = stats[:, 1], stats[:, 2]
    u = (stats[:, :1] - x64) / tau
    w = np.exp(-u)
    e = 18 * H + 3 * H * u
    np.put_along_axis(e, at[:rows].cpu().numpy(), 7 * H + 3 * H * np.take_along_axis(u, at[:rows].cpu().numpy(), 1), 1)
    others = w.copy()
    others[np.arange(rows), x64.argmax(1)] = 0.0
    e_r = (others * e).sum(1) + H * r
    e_l = e_r / (1 + r)
    e_gap = (w * u * (e + 3 * H)).sum(1) / (1 + r) + gap * e_l + H * gap
    assert np.array_equal(out[2].cpu().numpy(), ids)
    close(f64(out[4])[:, 1], r, e_r, "r")
    close(f64(out[4])[:, 2], gap, e_gap, "gap")
    close(f64(out[0]), logp, e_l + 2 * H * np.abs(logp), "logp")
    close(f64(out[1]), entropy, e_l + e_gap + H * entropy, "entropy")
    close(f64(out[3]), top, e_l[:, None] + 2 * H * np.abs(top), "top")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("above", [70.0, 500.0, 30000.0])
@pytest.mark.parametrize("T,V", [(200, 128256), (3, 128256), (70, 20011)])
def test_one_token_far_above(dtype, above, T, V):
    """What little the others hold, and nothing where that is below float32."""
    note(f"far above {dtype} {above} {T} {V}")
    x, at = peaked(T, V, dtype, above, 1.0, V + T, peaks=1)
    rows = min(T, 16)
    logp, entropy, ids, _, stats = (t[:rows] for t in L.lora_token_top(x, at[:, 0].int().contiguous(), 1, 1.0))
    x64 = f64(x[:rows])
    want = O.token_top(x64, at[:rows, 0].cpu().numpy(), 1, 1.0)
    u = want[4][:, :1] - x64
    w = np.exp(-u)
    w[np.arange(rows), x64.argmax(1)] = 0.0
    e = 18 * H + 3 * H * u
    e_r = (w * e).sum(1) + H * want[4][:, 1] + V * 2.0 ** -126
    e_gap = (w * u * (e + 3 * H)).sum(1) + want[4][:, 2] * (e_r + H) + V * 2.0 ** -118
    assert np.array_equal(ids.cpu().numpy(), want[2])
    close(f64(stats)[:, 1], want[4][:, 1], e_r)
    close(f64(stats)[:, 2], want[4][:, 2], e_gap)
    close(f64(logp), want[0], e_r + 2 * H * np.abs(want[0]))
    close(f64(entropy), want[1], e_r + e_gap + H * want[1])


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,V,k", [(200, 128256, 20), (70, 40000, 0), (3, 128256, 5), (5, 3001, 5)])
def test_far_below_zero_behind_a_masked_beginning(dtype, T, V, k):
    """Nothing at first, then values of which some share the largest, down to the type's lowest."""
    note(f"far below {dtype} {T} {V} {k}")
    n = torch.arange(V, device=DEV)
    late = n > V // 2
    rows = [torch.where(late, c * (2.0 - (n % many == 1).float()), -float("inf"))
            for c, many in ((-1e31, 1000), (-1.5e38, 3), (-5e29, 1000), (-2e30, V), (-1e4, 1000))]
    rows.append(torch.where(late, torch.finfo(dtype).min, -float("inf")))
    x = torch.stack(rows).to(dtype)
    x = x[torch.arange(T, device=DEV) % 6]
    rows = min(T, 6)
    _, entropy, ids, top, stats = (t if t is None else t[:rows] for t in L.lora_token_top(x, None, k, 1.0))
    x64 = f64(x[:rows])
    want = O.token_top(x64, None, k, 1.0)
    # the largest count alike and nothing else does: exact but for the roundings of the outputs and of the float32
    # trees of ones
    assert np.array_equal(ids.cpu().numpy(), want[2])
    close(f64(stats)[:, 1], want[4][:, 1], H * want[4][:, 1])
    close(f64(stats)[:, 2], want[4][:, 2], 0)
    close(f64(entropy), want[1], 2 * H * want[1])
    close(f64(top), want[3], 3 * H * np.abs(want[3]))
