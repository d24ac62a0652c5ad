"""Inputs of the losses that have no gradient: asking for one is refused, not
answered with none. On the CPU, by the backward itself."""
import types

import pytest
import torch

from lora_rank_adapter_amd import torch_ops

G = torch.ones(3)


def ctx(n, *wanted):
    return types.SimpleNamespace(saved_tensors=(G,), inputs=n, needs_input_grad=tuple(i in wanted for i in range(n)))


@pytest.mark.parametrize("backward,n,names", [
    ("_pref_backward", 5, {2: "ref_logp"}),
    ("_policy_backward", 10, {3: "old_logp", 4: "advantages", 5: "weights", 8: "ref_logp"}),
])
def test_constants_say_so(backward, n, names):
    f = getattr(torch_ops, backward)
    for at, name in names.items():
        with pytest.raises(RuntimeError, match=name):
            f(ctx(n, 0, at), G, None, None)
    got = f(ctx(n, 0), 2 * G, None, None)
    assert torch.equal(got[0], 2 * G) and got[1:] == (None,) * (n - 1)
    assert f(ctx(n, 0), None, None, None) == (None,) * n
    with pytest.raises(RuntimeError, match="beside the loss"):
        f(ctx(n, 0), G, G, None)
