"""AdamW's table of addresses when gradients are bound anew: under a captured
step, and between streams. The states of both sides take the same steps, so
everything is compared bit for bit."""
import pytest
import torch

import lora_rank_adapter_amd as L
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu
SIZES = [[300, 4096], [300, 40_000]]  # the form of few chunks, and the grid


def twins(sizes, bits):
    """Two optimizers on equal tensors, and two sets of gradients for each."""
    torch.manual_seed(1)
    params = [torch.randn(n, device=DEV) for n in sizes]
    grads = [[torch.randn(n, device=DEV) for n in sizes] for _ in range(2)]
    made = []
    for _ in range(2):
        p, g = [t.clone() for t in params], [[t.clone() for t in each] for each in grads]
        made.append((p, g, L.AdamW(p, g[0], 1e-2, state_bits=bits)))
    return made


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
               for x, y in zip(a[0] + list(a[2].state.values()), b[0] + list(b[2].state.values()), strict=True))


def litter(n):
    """Takes memory that was let go, of about n bytes a piece, and fills it."""
    return [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(32)]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_go_on_with_what_they_bound(sizes, bits):
    note(f"adamw bind under a graph {sizes} {bits}")
    a, b = twins(sizes, bits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a[2].step()
    old = a[2]._table_bytes
    for i in range(3):
        a[2].bind(a[1][1])
        kept = litter(old)
        graph.replay()          # the first gradients
        torch.cuda.synchronize()
        a[2].step()             # the second
        for k in (0, 1):
            b[2].bind(b[1][k])
            b[2].step()
        assert same(a, b), i
        del kept


@pytest.mark.parametrize("sizes", SIZES)
def test_steps_wait_for_a_table_of_another_stream(sizes):
    note(f"adamw bind and step on two streams {sizes}")
    a, b = twins(sizes, 32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.randn(4096, 4096, device=DEV)
    for i in range(3):
        with torch.cuda.stream(side):
            for _ in range(10):
                busy = busy @ busy * 1e-2  # holds the stream up
            a[2].bind(a[1][i % 2])
        a[2].step()  # on the default stream, without a wait of the caller's
        # let go here, while the side stream still has work: the table before it must not be given away
        kept = litter(a[2]._table_bytes)
        b[2].bind(b[1][i % 2])
        b[2].step()
        torch.cuda.synchronize()
        assert same(a, b), i
        with torch.cuda.stream(side):
            for _ in range(10):
                busy = busy @ busy * 1e-2
            a[2].step()
        a[2].bind(a[1][i % 2])  # while the step before it has not begun
        kept += litter(a[2]._table_bytes)
        torch.cuda.synchronize()
        b[2].step()
        assert same(a, b), i
        del kept
