"""Workspaces that the binding keeps, without a GPU: whose calls may share one."""
import threading
import types

import pytest
import torch

from combine_get_dispatch_03_gb300 import ep


@pytest.fixture
def streams(monkeypatch):
    """The current stream by name, nothing captured."""
    current = types.SimpleNamespace(stream=1)
    monkeypatch.setattr(ep, "_stream", lambda stream, device: current.stream)
    monkeypatch.setattr(ep, "_capturing", lambda: False)
    return current


def bare_handle():
    h = object.__new__(ep.Handle)
    h.device, h._scratch, h._ptr = torch.device("cpu"), {}, None
    return h


def test_calls_on_a_stream_share_and_streams_do_not(streams):
    h = bare_handle()
    first, _ = ep._scratch(h, 1000, None)
    assert ep._scratch(h, 500, None)[0] == first
    streams.stream = 2
    assert ep._scratch(h, 500, None)[0] != first
    streams.stream = 1
    assert ep._scratch(h, 1000, None)[0] == first
    grown, t = ep._scratch(h, 5000, None)
    assert t.numel() >= 5000 and ep._scratch(h, 1000, None)[0] == grown


def test_threads_do_not_share(streams):
    """A call enqueues more than one kernel: another thread's on the same stream can come between them."""
    h = bare_handle()
    got = {}
    together = threading.Barrier(3)

    def call(name):
        got[name] = ep._scratch(h, 1000, None)
        together.wait()  # all alive at once
        assert ep._scratch(h, 900, None)[0] == got[name][0]
        together.wait()

    threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    call(2)
    for t in threads:
        t.join()
    assert len({address for address, _ in got.values()}) == 3
