"""Cross attention and decode behind shared prefixes with tensors that begin at any 16 bytes and calls on a
given stream (GB300 only)."""
import pytest
import torch

import attend_harness as ah

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def moved(t):
    """A copy that begins 16 bytes behind a 32-byte border, other data before and behind it."""
    n = t.numel() * t.element_size()
    room = torch.full((n + 48,), 0xff, dtype=torch.uint8, device="cuda")     # NaN in every type
    at = 16 if room.data_ptr() % 32 == 0 else 0
    raw = room[at:at + n]
    raw.copy_(t.contiguous().view(torch.uint8).flatten())
    out = raw.view(t.dtype).view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out


@pytest.mark.parametrize("rows", [1, 6, 50])
@pytest.mark.parametrize("D,cache,bs", [(128, "same", 16), (256, "same", 784), (128, "same", 33), (128, "fp8", 16), (256, "fp8", 7)])
def test_tensors_at_any_16_bytes(cuda_lib, D, cache, bs, rows):
    lens = [700, 650, 1200, 30]
    pool = ah.Pool(lens, 2, D, bs, "bf16", cache, seed=rows, prefixes=[(0, 3, 600)])
    kc, vc, bt, sl = pool.cuda()
    q = ah.queries((4, rows, 8, D), "bf16", rows).cuda()
    groups, prefix, kw = i32([0, 3]), i32([600]), dict(k_scale=pool.scale, v_scale=pool.scale)
    want = (cuda_lib.cross(q, kc, vc, bt, sl, 0.09, **kw), cuda_lib.decode_shared(q, kc, vc, bt, sl, 0.09, groups, prefix, **kw))
    q, kc, vc = moved(q), moved(kc), moved(vc)
    for out in (moved(torch.zeros_like(q)), None):
        got = (cuda_lib.cross(q, kc, vc, bt, sl, 0.09, out=out, **kw).clone(),
               cuda_lib.decode_shared(q, kc, vc, bt, sl, 0.09, groups, prefix, out=out, **kw))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_given_streams(cuda_lib):
    # made on a stream of its own, the output used on the current one behind it
    lens = [700, 650, 1200, 30]
    pool = ah.Pool(lens, 2, 128, 16, "f16", seed=1, prefixes=[(0, 3, 600)])
    kc, vc, bt, sl = pool.cuda()
    q = ah.queries((4, 8, 128), "f16", 1).cuda()
    groups, prefix = i32([0, 3]), i32([600])
    calls = [lambda **kw: cuda_lib.cross(q, kc, vc, bt, sl, 0.09, **kw),
             lambda **kw: cuda_lib.decode_shared(q, kc, vc, bt, sl, 0.09, groups, prefix, **kw)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [f(stream=s) for f in calls for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(g, want[i // 3]) for i, g in enumerate(got))
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace(stream=s), stream=s) == 0
