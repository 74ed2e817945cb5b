"""Cross attention and decode behind shared prefixes at the edges of what they take (GB300 only)."""
import numpy as np
import pytest
import torch

import attend_harness as ah

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def bits(t):
    return t.detach().cpu().contiguous().view(torch.uint8)


def errors(pa):
    torch.cuda.synchronize()
    return pa.read_device_errors(pa.default_workspace())


def check_cross(pool, q, out, scale):
    rows = q.double().cpu().numpy()
    for b in range(len(pool.lens)):
        ref, mag, size = ah.attend(rows[b], pool.K[b], pool.V[b], scale)
        ah.check(out[b], ref, mag, size, pool, scale, f"sequence {b}")


@pytest.mark.parametrize("D,cache,bs", [(128, "same", 16), (256, "same", 16), (128, "fp8", 16), (128, "same", 33)])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-30, 0.5])
def test_scales(cuda_lib, D, cache, bs, scale):
    pool = ah.Pool([300, 77], 2, D, bs, "bf16", cache, seed=1)
    q = ah.queries((2, 70, 4, D), "bf16", 1)
    kc, vc, bt, sl = pool.cuda()
    out = cuda_lib.cross(q.cuda(), kc, vc, bt, sl, scale, k_scale=pool.scale, v_scale=pool.scale)
    assert errors(cuda_lib) == 0
    check_cross(pool, q, out, float(np.float32(scale)))


@pytest.mark.parametrize("D,cache", [(128, "same"), (256, "same"), (128, "fp8")])
@pytest.mark.parametrize("shape", ["climbing", "jump", "falling"])
@pytest.mark.parametrize("rows", [3, 40])
def test_references_that_are_raised(cuda_lib, D, cache, shape, rows):
    # scores that rise slowly past the slack of 8 (in log2), jump far beyond it, or fall: the
    # accumulators, one row tile or two, are rescaled at the right places
    L, g = 900, torch.Generator().manual_seed(4)
    pool = ah.Pool([L], 2, D, 16, "bf16", cache, seed=4)
    u = torch.randn(2, D, generator=g)
    u /= u.norm(dim=-1, keepdim=True)
    height = {"climbing": np.linspace(-4, 4, L), "falling": np.linspace(4, -4, L),
              "jump": np.where(np.arange(L) < 500, 0.0, 4.0)}[shape]
    K = torch.from_numpy(height)[:, None, None] * u[None].double() + 0.05 * torch.randn(L, 2, D, generator=g)
    store = (K / pool.scale).clamp(-448, 448).to(torch.float8_e4m3fn) if cache == "fp8" else K.to(torch.bfloat16)
    raw = pool.caches[0].view(torch.uint8 if cache == "fp8" else torch.int16)
    pos = torch.arange(L)
    raw[pool.bt[0, pos // 16].long(), pos % 16] = store.view(raw.dtype)
    pool.K[0] = store.float().double().numpy() * float(np.float32(pool.scale))
    q = (12.0 * u.repeat_interleave(2, 0)[None, None] + 0.3 * torch.randn(1, rows, 4, D, generator=g)).to(torch.bfloat16)
    kc, vc, bt, sl = pool.cuda()
    out = cuda_lib.cross(q.cuda(), kc, vc, bt, sl, 1.0, k_scale=pool.scale, v_scale=pool.scale)
    assert errors(cuda_lib) == 0
    check_cross(pool, q, out, 1.0)


def test_queries_that_are_slices_and_outputs_at_odd_places(cuda_lib):
    pool = ah.Pool([200, 333], 4, 128, 16, "f16", seed=2)
    kc, vc, bt, sl = pool.cuda()
    wide = ah.queries((2, 9, 20, 128), "f16", 2).cuda()      # heads 2 .. 9 of a projection's 20
    want = cuda_lib.cross(wide[:, :, 2:10].contiguous(), kc, vc, bt, sl, 0.09)
    assert torch.equal(cuda_lib.cross(wide[:, :, 2:10], kc, vc, bt, sl, 0.09), want)
    room = torch.zeros(want.numel() + 16, dtype=torch.float16, device="cuda")
    odd = room[8:8 + want.numel()].view(want.shape)          # 16-byte aligned, not 32
    assert odd.data_ptr() % 32 == 16
    assert cuda_lib.cross(wide[:, :, 2:10], kc, vc, bt, sl, 0.09, out=odd) is odd and torch.equal(odd, want)
    assert torch.all(room[:8] == 0) and torch.all(room[-8:] == 0)
    for refused in (wide.expand(2, 9, 20, 128)[:1].expand(2, 9, 20, 128)[:, :, 2:10], wide[..., ::2, :]):
        with pytest.raises((ValueError, cuda_lib.PAError)):
            cuda_lib.cross(refused, kc, vc, bt, sl, 0.09)
    q = wide[:, :, 2:10].contiguous()
    with pytest.raises(cuda_lib.PAError):
        cuda_lib.cross(q, kc, vc, bt, sl, 0.09, out=q)
    with pytest.raises(cuda_lib.PAError):
        cuda_lib.cross(q, kc, vc, bt, sl, 0.09, workspace=torch.zeros(1 << 14, dtype=torch.uint8, device="cuda"))
    with pytest.raises(cuda_lib.PAError):
        cuda_lib.decode_shared(q, kc, vc, bt, sl, 0.09, i32([0, 2]), i32([9]), out=q)


def test_a_nan_stays_in_its_row(cuda_lib):
    # in the queries: that row alone; in K or V at a live token: the rows that see it
    pool = ah.Pool([300, 90], 2, 128, 16, "bf16", seed=6)
    kc, vc, bt, sl = pool.cuda()
    q = ah.queries((2, 50, 4, 128), "bf16", 6).cuda()
    q[0, 7, 3] = float("nan")
    out = cuda_lib.cross(q, kc, vc, bt, sl, 0.09)
    bad = torch.isnan(out).any(-1)
    assert bad[0, 7, 3] and int(bad.sum()) == 1
    q[0, 7, 3] = 0
    vc[bt[1, 2].long(), 5, 1] = float("nan")
    out = torch.isnan(cuda_lib.cross(q, kc, vc, bt, sl, 0.09)).all(-1)
    assert out[1, :, 2:].all() and not out[0].any() and not out[1, :, :2].any()


@pytest.mark.parametrize("op", ["cross", "shared"])
def test_bad_lengths_tables_and_rows_are_reported(cuda_lib, op):
    # clamped and reported; what is computed is not meaningful, and finite
    lens = [60, 100, 130]
    pool = ah.Pool(lens, 2, 128, 16, "bf16", seed=7)
    kc, vc, bt, sl = pool.cuda()
    kc, vc = torch.nan_to_num(kc), torch.nan_to_num(vc)
    q = ah.queries((3, 4, 128), "bf16", 7).cuda()

    def call(sl=sl, bt=bt, rows=None, prefix=[40]):
        if op == "cross":
            return cuda_lib.cross(q, kc, vc, bt, sl, 0.09, starts=None if rows is None else i32(rows), max_seq_len=130)
        return cuda_lib.decode_shared(q, kc, vc, bt, sl, 0.09, i32([0, 3] if rows is None else rows), i32(prefix),
                                      max_seq_len=130)

    call()
    assert errors(cuda_lib) == 0
    for value in (-3, 131, 2 ** 31 - 1):
        s = sl.clone()
        s[1] = value
        assert torch.isfinite(call(sl=s)).all()
        found = errors(cuda_lib)                            # clamped to 130, its table may end before
        assert found & cuda_lib.PA_DEVERR_SEQ_LEN and not found & ~(cuda_lib.PA_DEVERR_SEQ_LEN | cuda_lib.PA_DEVERR_BLOCK_INDEX)
    for value in (-1, pool.caches[0].shape[0], 2 ** 31 - 1):
        b = bt.clone()
        b[2, 8] = value                                     # holds tokens 128 and 129
        assert torch.isfinite(call(bt=b)).all()
        assert errors(cuda_lib) == cuda_lib.PA_DEVERR_BLOCK_INDEX
    if op == "cross":
        for rows in ([0, 2, 1, 3], [-1, 1, 2, 3], [0, 1, 2, 4], [2 ** 31 - 1, 0, 0, 3]):
            call(rows=rows)
            assert errors(cuda_lib) == cuda_lib.PA_DEVERR_ROWS
    else:
        for rows in ([0, 4], [-1, 3], [2, 1], [3, 2 ** 31 - 1]):
            call(rows=rows)
            assert errors(cuda_lib) & cuda_lib.PA_DEVERR_ROWS
        call(rows=[0, 2, 1, 3], prefix=[40, 9, 30])
        assert errors(cuda_lib) == cuda_lib.PA_DEVERR_ROWS
        for prefix in (-1, 131):
            assert torch.isfinite(call(prefix=[prefix])).all()
            assert errors(cuda_lib) == cuda_lib.PA_DEVERR_SEQ_LEN
    call()
    assert errors(cuda_lib) == 0


def calls(pa, pool, q, groups, prefix):
    kc, vc, bt, sl = pool.cuda()
    g, p = i32(groups), i32(prefix)
    return [lambda: pa.cross(q, kc, vc, bt, sl, 0.09, k_scale=pool.scale, v_scale=pool.scale),
            lambda: pa.decode_shared(q, kc, vc, bt, sl, 0.09, g, p, k_scale=pool.scale, v_scale=pool.scale)], (kc, vc, bt, sl)


@pytest.mark.parametrize("cache", ["same", "fp8"])
def test_calls_repeat_bit_for_bit_beside_others(cuda_lib, cache):
    # two streams and their workspaces, many calls in flight, each equal to the first
    lens = [900, 800, 1500, 77]
    pool = ah.Pool(lens, 2, 128, 16, "bf16", cache, seed=8, prefixes=[(0, 3, 700)])
    q = ah.queries((4, 6, 8, 128), "bf16", 8).cuda()
    fns, _ = calls(cuda_lib, pool, q, [0, 3], [700])
    want = [f() for f in fns]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 3]):
            got.append([f() for f in fns])
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(pair, want))


def test_replays_follow_their_inputs(cuda_lib):
    # captured once, replayed over other lengths, groups and queries: the division of the work is made
    # anew on the device every time
    lens = [900, 800, 1500, 77]
    pool = ah.Pool(lens, 2, 128, 16, "bf16", seed=9, prefixes=[(0, 3, 700)])
    q = ah.queries((4, 8, 128), "bf16", 9).cuda()
    kc, vc, bt, sl = pool.cuda()
    groups, prefix = i32([0, 3]), i32([700])
    run = lambda: (cuda_lib.cross(q, kc, vc, bt, sl, 0.09, max_seq_len=1504),
                   cuda_lib.decode_shared(q, kc, vc, bt, sl, 0.09, groups, prefix, max_seq_len=1504))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = run()
        ws = cuda_lib.default_workspace()
    for new_lens, new_groups, new_prefix in ((lens, [0, 3], 700), ([1, 2, 3, 0], [0, 3], 1), ([0, 0, 0, 0], [1, 2], 5),
                                             ([850, 800, 1499, 77], [0, 2], 650)):
        sl.copy_(i32(new_lens))
        groups.copy_(i32(new_groups))
        prefix.copy_(i32([new_prefix]))
        q.copy_(torch.randn_like(q))
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, run()))
        assert cuda_lib.read_device_errors(ws) == 0


def test_shared_decode_agrees_with_decode(cuda_lib):
    # the same batch with and without its groups, and through decode(): 9000 sequences, more groups than
    # fit the kernel's table, each of two sequences or one
    B, nb = 9000, 2000
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn((nb, 16, 2, 128), generator=gen, device="cuda").bfloat16() for _ in range(2))
    bt = torch.randint(0, nb, (B, 3), generator=gen, device="cuda").to(torch.int32)
    sl = torch.randint(0, 49, (B,), generator=gen, device="cuda").to(torch.int32)
    q = torch.randn((B, 4, 128), generator=gen, device="cuda").bfloat16()
    pairs = torch.arange(0, 500, 2, device="cuda")
    bt[pairs + 1, :2] = bt[pairs, :2]
    groups = torch.cat([pairs, torch.arange(500, B + 1, device="cuda")]).to(torch.int32)
    assert groups.numel() > 8193
    want = cuda_lib.decode(q, kc, vc, bt, sl, 0.09, max_seq_len=48, deterministic=True).float()
    got = cuda_lib.decode_shared(q, kc, vc, bt, sl, 0.09, groups, torch.full_like(groups[1:], 32), max_seq_len=48).float()
    assert errors(cuda_lib) == 0
    # two results, each with weights and output rounded to bf16 (2^-8), over values of a few units
    near = 2 * 2.0 ** -8 * (want.abs() + vc.float().abs().max() * (want != 0))
    assert torch.all((got - want).abs() <= near) and torch.all(got[sl == 0] == 0)
    assert (got - want).norm() <= 2.0 ** -7 * want.norm()


@pytest.mark.parametrize("cache,bs", [("same", 16), ("same", 33), ("fp8", 16)])
def test_caches_beyond_32_bit_offsets(cuda_lib, cache, bs):
    # blocks at both ends of caches of 4.6 GB each: the same rows as in a small one
    Hkv, D, L = 8, 128, 300
    pool = ah.Pool([L], Hkv, D, bs, "bf16", cache, seed=11)
    kc, vc, bt, sl = pool.cuda()
    q = ah.queries((1, 5, 16, D), "bf16", 11).cuda()
    want = cuda_lib.cross(q, kc, vc, bt, sl, 0.09, k_scale=pool.scale, v_scale=pool.scale)
    nb = int(4.6e9 // (bs * Hkv * D * kc.element_size()))
    n = kc.shape[0]
    far = torch.where(torch.arange(n) % 2 == 0, torch.arange(n), nb - 1 - torch.arange(n)).cuda()
    big = []
    for c in (kc, vc):
        x = torch.empty((nb, *c.shape[1:]), dtype=c.dtype, device="cuda")
        raw, src = (t.view(torch.uint8 if cache == "fp8" else torch.int16) for t in (x, c))
        raw[far] = src
        big.append(x)
    bt = torch.where(bt >= 0, far[bt.clamp(min=0).long()].to(torch.int32), bt)
    got = cuda_lib.cross(q, *big, bt, sl, 0.09, k_scale=pool.scale, v_scale=pool.scale)
    assert errors(cuda_lib) == 0 and torch.equal(got, want)
    got = cuda_lib.decode_shared(q, *big, bt, sl, 0.09, i32([0, 1]), i32([20]), k_scale=pool.scale, v_scale=pool.scale)
    want = cuda_lib.decode_shared(q, kc, vc, pool.bt.cuda(), sl, 0.09, i32([0, 1]), i32([20]), k_scale=pool.scale,
                                  v_scale=pool.scale)
    assert torch.equal(got, want)


@pytest.mark.parametrize("cache", ["same", "fp8"])
def test_a_decoder_layer_of_beams(cuda_lib, cache):
    # a step of a decoder layer: five beams of two prompts write their token into the cache, attend to
    # their prompt once for all and to their own tokens, then to the prompt's source; eager and captured
    Hkv, Hq, D, bs, beams, prompts = 2, 8, 128, 16, 5, 2
    B = beams * prompts
    lens = [70 + 3 * b for b in range(beams)] + [210 + 5 * b for b in range(beams)]     # with the new token
    pool = ah.Pool(lens, Hkv, D, bs, "bf16", cache, seed=12, prefixes=[(0, 5, 64), (5, 10, 205)], own_prefix=True)
    source = ah.Pool([500, 333], Hkv, D, bs, "bf16", cache, seed=13)
    kc, vc, bt, sl = pool.cuda()
    skc, svc, sbt, ssl = source.cuda()
    rope = cuda_lib.rope(D)
    x = ah.queries((B, (Hq + 2 * Hkv) * D), "bf16", 12).cuda()
    cross_q = ah.queries((prompts, beams, Hq, D), "bf16", 14).cuda()
    groups, prefix = i32([0, 5, 10]), i32([64, 205])
    scale, s8 = float(np.float32(D ** -0.5)), pool.scale
    step = x.view(B, Hq + 2 * Hkv, D)
    # Every sequence's new token lies in a block of its own (none shares its last block)
    own = bt.clone()

    def layer():
        q = cuda_lib.append(step[:, Hq:Hq + Hkv], step[:, Hq + Hkv:], kc, vc, own, sl, q=step[:, :Hq], rope=rope,
                            k_scale=s8, v_scale=s8)
        a = cuda_lib.decode_shared(q, kc, vc, own, sl, scale, groups, prefix, max_seq_len=max(lens), k_scale=s8, v_scale=s8)
        c = cuda_lib.cross(cross_q, skc, svc, sbt, ssl, scale, max_seq_len=500, k_scale=s8, v_scale=s8)
        return q, a, c

    q, a, c = layer()
    assert errors(cuda_lib) == 0
    # what decode() makes of the same cache, and the definition over the source
    plain = cuda_lib.decode(q, kc, vc, own, sl, scale, max_seq_len=max(lens), k_scale=s8, v_scale=s8,
                            deterministic=True).float()
    assert (a.float() - plain).norm() <= 2.0 ** -7 * plain.norm()
    check_cross(source, cross_q, c, scale)
    # the definition over what the cache holds now
    kn, vn = cuda_lib.gather(kc, vc, own, sl, max(lens), dtype=torch.float16 if cache == "fp8" else torch.bfloat16,
                             k_scale=s8, v_scale=s8)
    for b, L in enumerate(lens):
        K, V = (t[b, max(lens) - L:].double().cpu().numpy() for t in (kn, vn))
        ref, mag, size = ah.attend(q[b].double().cpu().numpy()[None], K, V, scale)
        y = a[b].double().cpu().numpy()
        # fp8 rows are rounded to fp16 as they are gathered (2^-11 of a value, and of a score's terms)
        tol = 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -11 * scale * size + 2.0 ** -14) * mag[0] + 1e-6
        assert np.all(np.abs(y - ref[0]) <= tol)
    before = [bits(t) for t in (q, a, c)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = layer()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(bits(t), w) for t, w in zip(outs, before))


@pytest.mark.parametrize("D,cache", [(128, "same"), (256, "same"), (128, "fp8"), (256, "fp8")])
def test_workspaces_that_hold_anything(cuda_lib, D, cache):
    # only the header has to be zero before a call, and is after it
    lens = [1500, 1100, 2300, 0, 17, 900]
    pool = ah.Pool(lens, 4, D, 16, "f16", cache, seed=6, prefixes=[(0, 3, 1000)])
    kc, vc, bt, sl = pool.cuda()
    scales = dict(k_scale=pool.scale, v_scale=pool.scale)
    many, few = (ah.queries((6, n, 16, D), "f16", n).cuda() for n in (37, 2))
    groups, prefix = i32([0, 3]), i32([1000])
    calls = [lambda ws: cuda_lib.cross(many, kc, vc, bt, sl, 0.08, workspace=ws, **scales),
             lambda ws: cuda_lib.cross(few, kc, vc, bt, sl, 0.08, workspace=ws, **scales),
             lambda ws: cuda_lib.decode_shared(few, kc, vc, bt, sl, 0.08, groups, prefix, workspace=ws, **scales)]
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    want = [call(ws) for call in calls]
    for byte in (0xff, 0x7f, 0x01):
        for call, w in zip(calls, want):
            ws[cuda_lib.PA_WORKSPACE_HEADER_BYTES:] = byte
            assert torch.equal(bits(call(ws)), bits(w))
    assert not ws[:cuda_lib.PA_WORKSPACE_HEADER_BYTES].any()
