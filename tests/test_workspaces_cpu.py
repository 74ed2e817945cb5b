"""The workspaces that the Python binding keeps, with calls of several host threads (no GPU)."""
import threading

import torch

import paged_kv_attention_pa_gb300 as pa
from test_edges_cpu import FakeStream, host_workspaces  # noqa: F401 (a fixture)


def test_threads_that_call_first_share_one_workspace(host_workspaces, monkeypatch):  # noqa: F811
    # both find none and make one, the second while the first is still at it: with two of them the error
    # bits in the one that is not kept would be lost
    zeros, inside, made = torch.zeros, threading.Event(), []

    def slow(*args, **kw):
        inside.set()
        made.append(1)
        waiting.wait(0.5)                           # the other thread comes as far as it can
        return zeros(*args, **kw)

    monkeypatch.setattr(torch, "zeros", slow)
    waiting, got = threading.Event(), [None, None]

    def work(i):
        if i:
            inside.wait(10)
        got[i] = host_workspaces(1 << 16)
        waiting.set()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and got[0] is got[1]
    got[0][0] = pa.PA_DEVERR_SEQ_LEN
    assert pa.read_device_errors(host_workspaces(1 << 16), FakeStream) == pa.PA_DEVERR_SEQ_LEN


def test_a_call_amid_the_making_of_a_workspace(host_workspaces, monkeypatch):  # noqa: F811
    # a finalizer that an allocation sets off calls on the same thread
    zeros, amid, calls = torch.zeros, [], []

    def again(*args, **kw):
        if not amid:
            amid.append(1)
            calls.append(host_workspaces(pa.PA_WORKSPACE_HEADER_BYTES))
        return zeros(*args, **kw)

    monkeypatch.setattr(torch, "zeros", again)
    got = []
    t = threading.Thread(target=lambda: got.append(host_workspaces(1 << 17)), daemon=True)
    t.start()
    t.join(20)
    assert got and got[0].numel() >= 1 << 17 and calls[0] is not got[0]
