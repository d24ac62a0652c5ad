"""What AdamW's binding holds and refuses, on the CPU: the library's launches
are replaced by calls that do nothing, its sizes are its own."""
import pytest
import torch

import lora_rank_adapter_amd as L
from lora_rank_adapter_amd import train


class Library:
    """The library without its launches; counts them."""

    def __init__(self):
        self.tables = self.steps = 0

    def __getattr__(self, name):
        return getattr(L.load_library(), name)

    def lora_adamw_table(self, *_):
        self.tables += 1
        return 0

    def lora_adamw_step(self, *_):
        self.steps += 1
        return 0


@pytest.fixture
def lib(monkeypatch):
    held = Library()
    monkeypatch.setattr(train._lib, "load", lambda: held)
    monkeypatch.setattr(train, "_queue", lambda device: None)
    return held


def test_bind_refuses_sizes_that_the_states_do_not_have(lib):
    p, q = torch.zeros(300), torch.zeros(300, 4)
    opt = L.AdamW([p, q], [p.clone(), q.clone()], 1e-3)
    opt.step()
    before = opt.grads, opt._tensors, opt._table
    # a table that grew: its states would be written past their ends
    q.data = torch.zeros(400, 4)
    with pytest.raises(ValueError, match="param 1"):
        opt.bind([p.clone(), torch.zeros(400, 4)])
    # as many elements in all, but others' states
    p.data, q.data = torch.zeros(1200), torch.zeros(75, 4)
    with pytest.raises(ValueError, match="param 0"):
        opt.bind([p.clone(), q.clone()])
    assert all(a is b for a, b in zip((opt.grads, opt._tensors, opt._table), before)) and lib.tables == 1
    with pytest.raises(ValueError, match="moved"):
        opt.step()
    # the old sizes elsewhere in memory are taken
    p.data, q.data = torch.zeros(300), torch.zeros(300, 4)
    opt.bind([p.clone(), q.clone()])
    opt.step()
    assert lib.tables == lib.steps == 2
