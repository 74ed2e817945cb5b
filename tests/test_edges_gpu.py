"""Calls at the edges of what append, gather and decode take (GB300 only)."""
import numpy as np
import pytest
import torch

import rows_harness as rh
from oracle import int4 as o4

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B", [1, 3])
def test_a_step_without_new_tokens(cuda_lib, B):
    # [B, 0, heads, D]: nothing written, nothing rotated, nothing read
    kc = torch.full((4, 16, 2, 128), 3.0, dtype=torch.float16, device="cuda")
    k, q = (torch.zeros(B, 0, h, 128, dtype=torch.float16, device="cuda") for h in (2, 4))
    bt, sl = i32([[b] for b in range(B)]), i32([5] * B)
    out = cuda_lib.append(k, k, kc, kc, bt, sl, q=q)
    assert out.shape == q.shape and torch.all(kc == 3.0)
    ko, vo = cuda_lib.gather(kc, kc, bt, sl, 0)
    assert ko.shape == vo.shape == k.shape


def test_an_allocation_that_fails_is_out_of_memory(cuda_lib):
    # 2^30 rows of two heads of 128 in 16 bits, 550 GB: the output cannot be made, nothing is launched
    kc = torch.zeros((4, 16, 2, 128), dtype=torch.float16, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        cuda_lib.gather(kc, kc, i32([[0]]), i32([5]), 1 << 30)
    assert cuda_lib.gather(kc, kc, i32([[0]]), i32([5]), 5)[0].shape == (1, 5, 2, 128)


def test_errors_of_append_survive_a_decode_that_grows_the_workspace(cuda_lib):
    s = torch.cuda.Stream()
    kc = torch.zeros((64, 16, 8, 128), dtype=torch.float16, device="cuda")
    k = torch.zeros((1, 8, 128), dtype=torch.float16, device="cuda")
    bt = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    sl = i32([1024])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        cuda_lib.append(k, k, kc, kc, torch.full_like(bt, 99), sl)
        first = cuda_lib.default_workspace(stream=s)
        cuda_lib.decode(k, kc, kc, bt, sl, 0.1, max_seq_len=1024, splits=16)
        assert cuda_lib.default_workspace(stream=s) is not first
        assert cuda_lib.read_device_errors(cuda_lib.default_workspace(stream=s)) == cuda_lib.PA_DEVERR_BLOCK_INDEX
        assert cuda_lib.read_device_errors(cuda_lib.default_workspace(stream=s)) == 0


def test_captured_calls_share_one_workspace_of_their_graph(cuda_lib, monkeypatch):
    # two graphs captured on one stream that has a workspace of its own: each makes one, once;
    # replayed beside each other and beside eager calls of that stream, whose splits share
    # tails through counters in the workspace, all agree
    B, Hkv, L, nb = 2, 2, 8192, 1024
    gen = torch.Generator(device="cuda").manual_seed(1)
    kc, vc = (torch.randn((nb, 16, Hkv, 128), generator=gen, device="cuda").half() for _ in range(2))
    bt = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32).view(B, -1)
    sl = i32([L, L - 777])
    q = torch.randn((B, 8, 128), generator=gen, device="cuda").half()
    S, P = cuda_lib.plan(B, 8, Hkv, 128, 16, L, splits=6)
    assert S > 1 and P * 512 >= 512 << 10     # a shared tail
    call = lambda **kw: cuda_lib.decode(q, kc, vc, bt, sl, 0.088, max_seq_len=L, splits=6, **kw)
    want = call(deterministic=True).float()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()
        eager = cuda_lib.default_workspace()
    torch.cuda.synchronize()
    made = []
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: made.append(1) or zeros(*a, **kw))
    graphs = []
    for _ in range(2):
        g, before = torch.cuda.CUDAGraph(), len(made)
        with torch.cuda.graph(g, stream=s):
            assert cuda_lib.default_workspace() is None
            outs = [call() for _ in range(16)]
            rows = cuda_lib.gather(kc, vc, bt, sl, 3)
            ws = cuda_lib.default_workspace()
        assert len(made) == before + 1 and ws is not eager
        graphs.append((g, outs, rows, ws, torch.cuda.Stream()))
    assert graphs[0][3] is not graphs[1][3]
    with torch.cuda.stream(s):
        assert cuda_lib.default_workspace() is eager
    tol = 2.0 ** -10 * want.abs() + 2.0 ** -14      # a rounding of the output, the order of fp32 sums
    for _ in range(3):
        for g, _, _, _, t in graphs:
            with torch.cuda.stream(t):
                g.replay()
        with torch.cuda.stream(s):
            beside = [call() for _ in range(16)]
        torch.cuda.synchronize()
        for out in graphs[0][1] + graphs[1][1] + beside:
            assert torch.all((out.float() - want).abs() <= tol)
    for _, _, rows, ws, _ in graphs:
        assert torch.equal(rows[0][0], kc[bt[0, -1].long(), 13:16]) and cuda_lib.read_device_errors(ws) == 0
    sl[0] = L + 1                                    # the error of a replay, in its graph's workspace
    graphs[1][0].replay()
    torch.cuda.synchronize()
    assert cuda_lib.read_device_errors(graphs[0][3]) == 0
    assert cuda_lib.read_device_errors(graphs[1][3]) == cuda_lib.PA_DEVERR_SEQ_LEN


class Handle:
    """Another library's stream: a handle and nothing else."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.mark.parametrize("given", [lambda s: s, lambda s: torch.cuda.ExternalStream(s.cuda_stream), Handle])
def test_calls_on_a_given_stream_leave_the_current_one(cuda_lib, given):
    s = torch.cuda.Stream()
    gen = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = (torch.randn((64, 16, 2, 128), generator=gen, device="cuda").half() for _ in range(2))
    k, q = (torch.randn((1, h, 128), generator=gen, device="cuda").half() for h in (2, 4))
    bt, sl = torch.arange(64, dtype=torch.int32, device="cuda")[None], i32([1000])
    want = [cuda_lib.append(k, k, kc, vc, bt, sl, q=q), *cuda_lib.gather(kc, vc, bt, sl, 5),
            cuda_lib.decode(q, kc, vc, bt, sl, 0.088, max_seq_len=1000, deterministic=True)]
    torch.cuda.synchronize()
    here = torch.cuda.current_stream()
    got = [cuda_lib.append(k, k, kc, vc, bt, sl, q=q, stream=given(s)),
           *cuda_lib.gather(kc, vc, bt, sl, 5, stream=given(s)),
           cuda_lib.decode(q, kc, vc, bt, sl, 0.088, max_seq_len=1000, deterministic=True, stream=given(s))]
    assert torch.cuda.current_stream() == here
    s.synchronize()
    assert all(torch.equal(rh.bits(a), rh.bits(b)) for a, b in zip(got, want))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_by_angles_near_the_axes(cuda_lib, interleaved):
    # (2^14, 0) turned by angles all around and close to the multiples of a quarter turn, where
    # the sine or cosine is small and its relative error shows. The angle keeps 32 bits of a turn
    # (2 pi 2^-32 = 1.5e-9) and is rounded to fp32 relative to the nearest quarter (2^-25), sine,
    # cosine (2 units) and their product round relatively as well: 2^-21 in all; the output once
    rng = np.random.default_rng(3)
    T = 4096
    turns = rng.integers(0, 2 ** 64, (T, 64), dtype=np.uint64)
    near = np.exp(rng.uniform(np.log(2.0 ** 34), np.log(2.0 ** 61), (T // 2, 64))).astype(np.uint64)
    sign = rng.integers(0, 2, near.shape).astype(bool)
    turns[:T // 2] = (turns[:T // 2] >> np.uint64(62) << np.uint64(62)) + np.where(sign, near, ~near + np.uint64(1))
    a = turns.astype(np.longdouble) / np.longdouble(2.0 ** 64) * 2
    a = np.where(a >= 1, a - 2, a)                    # half turns in [-1, 1)
    k = np.rint(a * 2)                                # quarters, taken off before the sine is
    r = ((a - k / 2) * np.longdouble(np.pi)).astype(np.float64)
    k = k.astype(np.int64) % 4
    c, s = np.cos(r), np.sin(r)
    cos, sin = np.choose(k, [c, -s, -c, s]), np.choose(k, [s, c, -s, -c])
    q = torch.zeros((1, 1, 128), dtype=torch.float16, device="cuda")
    at = slice(0, 128, 2) if interleaved else slice(0, 64)
    other = slice(1, 128, 2) if interleaved else slice(64, 128)
    q[..., at] = 2.0 ** 14
    kc = torch.zeros((1, 16, 1, 128), dtype=torch.float16, device="cuda")
    bt, sl = i32([[0]]), i32([2])                     # one token, at position 1
    tt = torch.from_numpy(turns.view(np.int64)).cuda()
    got = torch.cat([cuda_lib.append(q, q, kc, kc, bt, sl, q=q, rope=cuda_lib.Rope(tt[i], interleaved))
                     for i in range(T)]).cpu().double().numpy()[:, 0]
    for y, ref in ((got[:, at], cos), (got[:, other], sin)):
        ref = ref * 2.0 ** 14
        tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -21 * np.abs(ref) + 2.0 ** 14 * 1.6e-9 + 2.0 ** -25
        assert np.all(np.abs(y - ref) <= tol)


@pytest.mark.parametrize("scale", [7.0, 0.7, 5.0 / 448, 11.0, 3e38, 1e-38, 0.125])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantised_rows_hold_the_quotient(cuda_lib, dtype, scale):
    # value / scale, the correctly rounded fp32 quotient, and then the nearest code: products
    # with a rounded 1 / scale fall off the ties between codes (1.4375, say, from 10.0625 / 7)
    s32 = np.float32(scale)
    rng = np.random.default_rng(7)
    L, D = 4096, 128
    ties = (2 * rng.integers(8, 16, (L, 2, D)) + 1) / 16 * 2.0 ** rng.integers(-4, 5, (L, 2, D))
    x = np.where(rng.random((L, 2, D)) < 0.5, ties * float(s32), rng.standard_normal((L, 2, D)) * float(s32))
    if scale in (3e38, 1e-38):
        x = rng.standard_normal((L, 2, D)) * (1e38 if scale > 1 and dtype == "bf16" else 1.0)
    with np.errstate(over="ignore", under="ignore"):
        v = torch.from_numpy(x.astype(np.float32)).to(rh.DT[dtype])
        y = (v.float().numpy() / s32).astype(np.float32)
    nb = L // 16
    bt, sl = torch.arange(nb, dtype=torch.int32, device="cuda")[None], i32([L])
    for kind in ("fp8", "int4"):
        if kind == "fp8":
            kc, vc = (torch.zeros((nb, 16, 2, D), device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
        else:
            kc, vc = (torch.zeros((nb, 2, 16, o4.row_bytes(D)), dtype=torch.uint8, device="cuda") for _ in range(2))
        cuda_lib.append(v[None].cuda(), v[None].cuda(), kc, vc, bt, sl, k_scale=scale, v_scale=scale)
        if kind == "fp8":
            want = torch.from_numpy(np.clip(y, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
            got = [c.view(torch.uint8).cpu().reshape(L, 2, D) for c in (kc, vc)]
        else:
            want = torch.from_numpy(o4.quantise(y.astype(np.float64)))
            got = [c.cpu().transpose(1, 2).reshape(L, 2, -1) for c in (kc, vc)]
        assert all(torch.equal(g, want) for g in got), kind
