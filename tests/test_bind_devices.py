"""A bound call runs on the device it was bound on, whichever is current when it
is called (no GPU needed: the devices and the library are stand-ins)."""
import pytest
import torch

from indexer_top_sparse_c4_b200 import qsa


class Library:
    def __init__(self, log, now):
        self.log, self.now = log, now

    def qsa_chunk_plan(self, *args):
        self.log.append(("plan", self.now[0], args))
        return 0

    def qsa_topk_groups(self, *args):
        self.log.append(("topk", self.now[0], args))
        return 0


@pytest.fixture
def machine(monkeypatch):
    """(log of library calls, the current device) of a machine of three devices."""
    log, now = [], [0]

    class On:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.was, now[0] = now[0], self.dev

        def __exit__(self, *exc):
            now[0] = self.was

    monkeypatch.setattr(qsa, "_lib", Library(log, now))
    monkeypatch.setattr(qsa, "_current_device", lambda: now[0])
    monkeypatch.setattr(qsa, "_raw_stream", lambda dev: 1000 + dev)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "device", On)
    return log, now


def test_bound_calls_keep_their_device(machine):
    log, now = machine
    go = qsa.bind(lambda: qsa._call(qsa.lib().qsa_chunk_plan, 2, None, 7))
    assert not log and now == [0]
    for current in (0, 2, 1):
        now[0] = current
        go()
        assert log.pop() == ("plan", 2, (7, 1002)) and now == [current]


def test_calls_bound_on_several_devices(machine):
    """Calls of the current device (which name none) and of their tensors' device,
    in their order."""
    log, now = machine
    now[0] = 1

    def step():
        qsa.lib().qsa_topk_groups(1)
        qsa._call(qsa.lib().qsa_chunk_plan, 2, None, 2)
        qsa._call(qsa.lib().qsa_chunk_plan, 1, None, 3)
    go = qsa.bind(step)
    now[0] = 0
    go()
    assert [(n, d, a[0]) for n, d, a in log] == [("topk", 1, 1), ("plan", 2, 2), ("plan", 1, 3)] and now == [0]


def test_a_refused_call_leaves_the_device_as_it_was(machine):
    log, now = machine
    qsa._lib.qsa_last_error_string = lambda: b"no"
    qsa._lib.qsa_status_name = lambda s: b"QSA_ERR_INVALID"
    qsa._lib.qsa_chunk_plan = lambda *a: 1
    go = qsa.bind(lambda: qsa._call(qsa.lib().qsa_chunk_plan, 2, None))
    with pytest.raises(qsa.QSAError, match="no"):
        go()
    assert now == [0]
