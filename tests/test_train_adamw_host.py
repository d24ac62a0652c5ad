"""What AdamW's binding holds, orders and refuses, on the CPU: the library's
launches are replaced by calls that do nothing (its sizes are its own), and
the streams by what records their use."""
import ctypes
import gc
import weakref

import pytest
import torch

import lora_rank_adapter_amd as L
from lora_rank_adapter_amd import train


class Library:
    """The library without its launches, and the machine's streams: counts and notes what is done."""

    def __init__(self):
        self.tables = self.steps = 0
        self.stream, self.capturing, self.log = 0, False, []

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

    class Stream:
        def wait_event(self, event):
            held.log.append(("wait", held.stream, event.at))

    class Event:
        def record(self, stream):
            assert not held.capturing
            self.at = held.stream

    monkeypatch.setattr(train._lib, "load", lambda: held)
    monkeypatch.setattr(train, "_queue", lambda device: ctypes.c_void_p(held.stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: held.capturing)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream())
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, _: held.log.append(("used", held.stream, t.data_ptr())))
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


def test_what_a_captured_step_uses_is_kept(lib):
    p = torch.zeros(300)
    opt = L.AdamW([p], [p.clone()], 1e-3)
    opt.step()
    seen = [weakref.ref(t) for t in (opt._table, opt.grads[0])]
    opt.bind([p.clone()])
    gc.collect()
    assert not any(r() is not None for r in seen)  # no graph: let go
    seen = [weakref.ref(t) for t in (opt._table, opt.grads[0])]
    lib.stream, lib.capturing = 7, True
    opt.step()
    lib.stream, lib.capturing = 0, False
    for _ in range(2):
        opt.bind([p.clone()])
        opt.step()
    gc.collect()
    assert all(r() is not None for r in seen) and len(opt._kept) == 1
    assert lib.log == []  # a capture waits for nothing and marks nothing


def test_a_step_on_another_stream_waits_for_the_table(lib):
    p = torch.zeros(300)
    lib.stream = 3
    opt = L.AdamW([p], [p.clone()], 1e-3)
    opt.step()
    assert lib.log == []
    for stream in (0, 5):
        lib.stream, lib.log = stream, []
        opt.step()
        opt.step()
        assert lib.log[0] == ("wait", stream, 3)
        assert set(lib.log[1:]) == {("used", stream, t.data_ptr()) for t in (opt._table, *opt.state.values())}
        assert len(lib.log) == 1 + 4
    opt.bind([p.clone()])  # now on stream 5
    lib.stream, lib.log = 3, []
    opt.step()
    assert lib.log[0] == ("wait", 3, 5)


def test_a_table_written_in_a_capture_is_not_waited_for(lib):
    p = torch.zeros(300)
    opt = L.AdamW([p], [p.clone()], 1e-3)
    lib.stream, lib.capturing = 7, True
    opt.bind([p.clone()])
    opt.step()
    lib.stream, lib.capturing, lib.log = 0, False, []
    opt.step()
    assert lib.log and all(kind == "used" for kind, *_ in lib.log)


@pytest.mark.parametrize("shapes", [((8, 24), (24, 8)), ((8, 24), (192,)), ((6,), (6, 1)), ((1, 8), (8,))])
def test_operands_of_another_shape_are_refused(lib, shapes):
    """Elements are paired by their place in memory: a gradient of the transposed weight has as many."""
    p, t = torch.zeros(shapes[0]), torch.zeros(shapes[1])
    with pytest.raises(ValueError, match="grad 0"):
        L.AdamW([p], [t], 1e-3)
    with pytest.raises(ValueError, match="shadow 0"):
        L.AdamW([p], [p.clone()], 1e-3, shadows=[t.to(torch.bfloat16)])
    L.AdamW([p], [p.clone()], 1e-3, shadows=[p.to(torch.bfloat16)])
    L.AdamW([p.view(-1)], [t.view(-1)], 1e-3)  # flat views pair as their owner says
    assert lib.tables == 2


def test_memory_given_twice_is_refused(lib):
    """Two entries over the same elements would be updated by two workgroups at once."""
    p, q = torch.zeros(300), torch.zeros(900)
    g = torch.zeros(300)
    half = torch.zeros(600, dtype=torch.bfloat16)
    for params, shadows in (([p, p], None), ([q[:300], q[299:599]], None), ([q[300:600], q[:600]], None),
                            ([p, q[:300]], [half[:300], half[200:500]]), ([p, q[:300]], [half[:300], half[:300]]),
                            ([p], [p.view(torch.bfloat16)[:300]])):
        grads = [torch.zeros(t.numel()) for t in params]
        with pytest.raises(ValueError, match="share memory"):
            L.AdamW(params, grads, 1e-3, shadows=shadows)
    # neighbours in one buffer, empty tensors, and gradients that are one tensor
    L.AdamW([q[:300], q[300:600], q[200:200]], [g, g, g[:0]], 1e-3, shadows=[half[:300], half[300:], half[9:9]])
