"""Host threads that call on one stream, and so on one workspace (GB300 only): the kernels of a call, of
which the second joins what the first leaves in the workspace, stay together."""
import threading

import pytest
import torch

import attend_harness as ah

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_threads_on_one_stream(cuda_lib):
    pa = cuda_lib
    lens = [900, 800, 1500, 77]
    pool = ah.Pool(lens, 2, 128, 16, "bf16", seed=21, prefixes=[(0, 3, 700)])
    kc, vc, bt, sl = pool.cuda()
    groups, prefix = i32([0, 3]), i32([700])
    one, few, many = (ah.queries((4, n, 8, 128), "bf16", n).cuda() for n in (1, 6, 150))
    small = pa.cross(few[:2], kc, vc, bt[:2], sl[:2], 0.09)                  # fewer rows than others' items name
    calls = [lambda: pa.cross(few[:2], kc, vc, bt[:2], sl[:2], 0.09),
             lambda: pa.cross(many, kc, vc, bt, sl, 0.09),
             lambda: pa.decode_shared(few, kc, vc, bt, sl, 0.09, groups, prefix),
             lambda: pa.decode(one[:, 0], kc, vc, bt, sl, 0.09, max_seq_len=1500, splits=9, deterministic=True),
             lambda: pa.decode_plain(one[:, 0].contiguous(), kc, vc, bt, sl, 0.09, max_seq_len=1500)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    assert torch.equal(want[0], small)
    got, start, failed = [[] for _ in calls], threading.Barrier(len(calls)), []

    def work(i):
        try:
            start.wait()
            for _ in range(200):
                got[i].append(calls[i]())
        except Exception as e:                                               # seen by the test, not by its thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and pa.read_device_errors(pa.default_workspace()) == 0
    for i, (outs, w) in enumerate(zip(got, want)):
        assert len(outs) == 200 and all(torch.equal(o, w) for o in outs), f"call {i}"
