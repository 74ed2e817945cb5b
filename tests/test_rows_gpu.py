"""pa.append and pa.gather against the float64 oracle (GB300 only)."""
import numpy as np
import pytest
import torch

import rows_harness as rh
from oracle import int4 as o4
from oracle import rope as orope
from oracle import e4m3_to_float64

pytestmark = pytest.mark.gpu

DT = rh.DT
SCALES = {"same": (1.0, 1.0), "fp8": (0.0625, 5.0 / 448), "int4": (1.0, 0.75)}


def make(lens, new, R, Hq, Hkv, D, bs, dtype, cache, seed, pad=(0, 0)):
    """Device inputs of one append: a projection [T, (Hq + 2 Hkv) D] whose slices are q, k, v;
    pad: rows before the first and behind the last sequence (packed calls)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    starts = None
    if new is not None:
        starts = [pad[0]]
        for n in new:
            starts.append(starts[-1] + n)
        T = starts[-1] + pad[1]
    else:
        T = B * R
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).to(DT[dtype])
    bt, pool = rh.tables_for(lens, bs, seed)
    kc = rh.empty_pool(cache, pool, bs, Hkv, D, dtype, seed + 1, nan=False)
    vc = rh.empty_pool(cache, pool, bs, Hkv, D, dtype, seed + 2, nan=False)
    return dict(qkv=qkv, T=T, bt=bt, kc=kc, vc=vc, starts=starts, lens=list(lens), B=B, R=R, Hq=Hq,
                Hkv=Hkv, D=D, bs=bs, dtype=dtype, cache=cache)


def views(x, qkv):
    lead = (x["T"],) if x["starts"] is not None else (x["B"], x["R"])
    y = qkv.view(*lead, x["Hq"] + 2 * x["Hkv"], x["D"])
    return (y[..., :x["Hq"], :], y[..., x["Hq"]:x["Hq"] + x["Hkv"], :],
            y[..., x["Hq"] + x["Hkv"]:, :])


def i32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def append(pa, x, rope, with_q=True, **kw):
    """Run it: (q_out or None, k_cache, v_cache) on the device."""
    qkv, kc, vc = x["qkv"].cuda(), x["kc"].cuda(), x["vc"].cuda()
    q, k, v = views(x, qkv)
    ks, vs = SCALES[x["cache"]]
    qo = pa.append(k, v, kc, vc, x["bt"].cuda(), i32(x["lens"]), q=q if with_q else None,
                   starts=i32(x["starts"]), rope=rope, k_scale=ks, v_scale=vs, **kw)
    return qo, kc, vc


def check_append(x, freq, amp, il, qo, kc, vc):
    """Every output against the oracle, every other slot of the caches unchanged."""
    D, Hq, Hkv, bs, cache, dtype = (x[n] for n in ("D", "Hq", "Hkv", "bs", "cache", "dtype"))
    xs = rh.f64(x["qkv"]).reshape(x["T"], Hq + 2 * Hkv, D)
    at = rh.positions(x["lens"], x["starts"], x["R"], x["B"])
    live = [(r, b, p) for r, b, p in at if p >= 0]
    half = rh.HALF_STEP[dtype]
    # fp32 rotation: two products and a sum (3 * 2^-24 of |x1| + |x2|), the angle rounded to
    # fp32 (2^-25 half turns = 1e-7 rad) and its sine and cosine (2 units, 1.2e-7): within 5e-7
    rot_err = 5e-7 * abs(amp) if len(freq) else 0.0
    pair = 2 * np.abs(xs).max()

    if qo is not None:
        got = rh.f64(qo).reshape(x["T"], Hq, D)
        rows = [r for r, _, _ in live]
        ref = orope.rotate(xs[rows][:, :Hq], np.array([p for _, _, p in live]), freq, il, amp)
        assert np.all(np.abs(got[rows] - ref) <= half * np.abs(ref) + 2 * rot_err * pair + 2.0 ** -25)
        for r, _, p in at:
            if p < 0:
                assert np.all(got[r] == 0)

    ks, vs = (float(np.float32(s)) for s in SCALES[cache])
    touched = np.zeros(x["kc"].shape[:1] + (bs,), dtype=bool)
    for b in range(x["B"]):
        mine = [(r, p) for r, bb, p in live if bb == b]
        if not mine:
            continue
        pos = np.array([p for _, p in mine])
        touched[x["bt"][b].numpy()[pos // bs], pos % bs] = True
        rows = [r for r, _ in mine]
        k = orope.rotate(xs[rows][:, Hq:Hq + Hkv], pos, freq, il, amp)
        v = xs[rows][:, Hq + Hkv:]
        for y, c, s, err in ((k, kc, ks, 2 * rot_err * pair), (v, vc, vs, 0.0)):
            raw = rh.cache_rows(c, cache, x["bt"], b, pos, bs)
            if cache == "same":
                assert np.all(np.abs(rh.f64(raw) - y) <= half * np.abs(y) + err + 2.0 ** -25)
                if err == 0.0:
                    assert np.array_equal(rh.f64(raw), y)
                continue
            y, err = y / s, err / s + 2.0 ** -22 * np.abs(y / s)   # the inverse scale, the product
            if cache == "fp8":
                w, y = e4m3_to_float64(raw.numpy()), np.clip(y, -448, 448)
                assert np.all(np.abs(w - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + err)
            else:
                w = o4.dequant(raw.numpy())
                _, st, _ = o4.unpack(raw.numpy())
                lim = np.repeat(st, 32, axis=-1) * (0.5 + 2.0 ** -20)
                assert np.all(np.abs(w - y) <= lim + err)
                # the step is no larger than a fifteenth of the range needs: fp16 rounding of
                # the minimum (2^-10 of it, or 2^-24) and of the step itself (2^-10)
                g = y.reshape(*y.shape[:-1], -1, 32)
                low = np.abs(g.min(-1)) * 2.0 ** -10 + 2.0 ** -24
                room = ((g.max(-1) - g.min(-1) + low) / 15) * (1 + 2.0 ** -10) + 2.0 ** -24
                assert np.all(st <= room * (1 + 1e-6) + np.max(err))
    # nothing else changed
    for c, c0 in ((kc, x["kc"]), (vc, x["vc"])):
        a, b = c.cpu().view(torch.uint8), c0.view(torch.uint8)
        if cache == "int4":
            a, b = a.transpose(1, 2), b.transpose(1, 2)
        keep = torch.from_numpy(~touched)
        assert torch.equal(a[keep], b[keep])


def rope_of(pa, rot, il=False, **kw):
    if rot == 0:
        return None, np.zeros(0), 1.0
    r = pa.rope(rot, interleaved=il, scaling=kw.get("kind"), device="cuda",
                **{k: v for k, v in kw.items() if k != "kind"})
    f, amp = orope.frequencies(rot, **kw)
    return r, f, amp


@pytest.mark.parametrize("cache", ["same", "fp8", "int4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,bs,R,lens", [
    (8, 8, 128, 16, 1, [1]),                        # the first token of a sequence
    (32, 8, 128, 16, 1, [17, 16, 1, 0, 33]),        # an empty sequence has no row to write
    (6, 2, 128, 5, 4, [4, 3, 100, 2, 0]),           # rows without a token
    (24, 4, 256, 784, 3, [785, 1569, 3]),
    (3, 3, 128, 1, 2, [2, 40]),                     # heads that do not fill a warp
    (5, 1, 256, 33, 7, [7, 66]),
])
def test_append_rows(cuda_lib, cache, dtype, Hq, Hkv, D, bs, R, lens):
    x = make(lens, None, R, Hq, Hkv, D, bs, dtype, cache, seed=1)
    for rot, il in ((D, False), (D, True), (D // 2, False), (32, True), (16, False), (48, False), (0, False)):
        rope, f, amp = rope_of(cuda_lib, rot, il)
        check_append(x, f, amp, il, *append(cuda_lib, x, rope))
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace()) == 0


@pytest.mark.parametrize("cache", ["same", "fp8", "int4"])
@pytest.mark.parametrize("new,lens,pad", [
    ([5, 0, 1, 300, 0], [5, 7, 1, 4000, 0], (0, 0)),        # sequences without new tokens
    ([0, 0, 2], [0, 3, 50], (3, 9)),                        # padding on both sides
    ([1], [1], (0, 130)),
    ([2] * 70, list(range(2, 72)), (1, 1)),                 # more than one round of the search
    ([0] * 40 + [3] + [0] * 30, [9] * 71, (0, 2)),
    ([1] * 1030, [1 + i % 5 for i in range(1030)], (0, 0)),  # three rounds
])
def test_append_packed(cuda_lib, cache, new, lens, pad):
    x = make(lens, new, 0, 4, 2, 128, 16, "bf16", cache, seed=2, pad=pad)
    rope, f, amp = rope_of(cuda_lib, 64, True, kind="yarn", factor=4.0, original_max=512)
    q, k, v = views(x, x["qkv"])
    q_out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    qo, kc, vc = append(cuda_lib, x, rope, q_out=q_out)
    assert qo is q_out
    check_append(x, f, amp, True, qo, kc, vc)
    s = x["starts"]
    assert torch.all(qo[:s[0]] == 7.0) and torch.all(qo[s[-1]:] == 7.0)   # padding left alone


def test_append_far_positions(cuda_lib):
    # positions where an fp32 angle would be off by whole radians
    lens = [1_000_003, 16_777_217]
    for kw in (dict(), dict(kind="linear", factor=16.0), dict(kind="ntk", factor=4.0)):
        x = dict(make([1, 1], None, 1, 2, 1, 128, 1 << 16, "f16", "same", seed=3))
        bt = torch.full((2, 257), -1, dtype=torch.int32)
        bt[0, 15], bt[1, 256] = 1, 2
        x.update(lens=lens, bt=bt, kc=torch.zeros((3, 1 << 16, 1, 128), dtype=torch.float16),
                 vc=torch.zeros((3, 1 << 16, 1, 128), dtype=torch.float16))
        rope, f, amp = rope_of(cuda_lib, 128, False, **kw)
        check_append(x, f, amp, False, *append(cuda_lib, x, rope))


def test_append_large_prompt_and_strides(cuda_lib):
    # k and v with strides of their own, q in place, a long packed prompt
    Hq, Hkv, D, T = 8, 2, 128, 3001
    x = make([5000], [T], 0, Hq, Hkv, D, 16, "bf16", "int4", seed=4)
    rope, f, amp = rope_of(cuda_lib, 128)
    q, k, v = (t.contiguous().cuda() for t in views(x, x["qkv"]))
    wide = torch.zeros((T, Hkv + 3, D), dtype=k.dtype, device="cuda")
    wide[:, :Hkv] = k
    kc, vc = x["kc"].cuda(), x["vc"].cuda()
    ks, vs = SCALES["int4"]
    qo = cuda_lib.append(wide[:, :Hkv], v, kc, vc, x["bt"].cuda(), i32(x["lens"]), q=q, q_out=q,
                         starts=i32(x["starts"]), rope=rope, k_scale=ks, v_scale=vs)
    assert qo is q
    check_append(x, f, amp, False, qo, kc, vc)


def test_append_without_queries(cuda_lib):
    x = make([40, 3], None, 2, 4, 2, 256, 16, "f16", "fp8", seed=5)
    rope, f, amp = rope_of(cuda_lib, 256)
    qo, kc, vc = append(cuda_lib, x, rope, with_q=False)
    assert qo is None
    check_append(x, f, amp, False, None, kc, vc)


def test_int4_rows_equal_the_quantiser(cuda_lib):
    # unrotated 16-bit rows have exact ties: the bytes equal the oracle's, in both types, for
    # ranges from fp16 subnormals to its top, rows of one value and rows with zeros
    for dtype in ("bf16", "f16"):
        for scale in (1e-6, 1e-3, 1.0, 100.0, 2e4):
            x = make([64], None, 64, 1, 4, 128, 16, dtype, "int4", seed=6)
            x["qkv"] = (x["qkv"].float() * scale).to(DT[dtype])
            x["qkv"][0] = 3.0
            x["qkv"][1] = 0.0
            x["qkv"][2, ::2] = 0.0
            qkv, kc, vc = x["qkv"].cuda(), x["kc"].cuda(), x["vc"].cuda()
            q, k, v = views(x, qkv)
            cuda_lib.append(k, v, kc, vc, x["bt"].cuda(), i32(x["lens"]))
            pos = np.arange(64)
            for t, c in ((k, kc), (v, vc)):
                raw = rh.cache_rows(c, "int4", x["bt"], 0, pos, 16).numpy()
                assert np.array_equal(raw, o4.quantise(rh.f64(t)[0])), (dtype, scale)


def test_non_finite_inputs(cuda_lib):
    # a NaN or infinity poisons its own group of a 4-bit row (and only that), stays NaN in fp8
    # (infinities saturate) and passes through 16-bit rows
    x = make([4], None, 4, 1, 1, 128, 16, "bf16", "int4", seed=7)
    _, k, v = views(x, x["qkv"])
    v[0, 1, 0, 40] = float("nan")
    v[0, 2, 0, 100] = float("inf")
    v[0, 3, 0, 0] = -float("inf")
    bt, lens = x["bt"].cuda(), i32([4])
    for cache in ("int4", "fp8", "same"):
        kc = rh.empty_pool(cache, x["kc"].shape[0], 16, 1, 128, "bf16", 8, nan=False).cuda()
        vc = kc.clone()
        cuda_lib.append(k.cuda(), v.cuda(), kc, vc, bt, lens)
        _, got = cuda_lib.gather(kc, vc, bt, lens, 4, dtype=torch.bfloat16)
        bad = torch.isnan(got).cpu()[0, :, 0]
        want = torch.zeros_like(bad)
        if cache == "int4":
            want[1, 32:64] = want[2, 96:] = want[3, :32] = True
        else:
            want[1, 40] = True
        assert torch.equal(bad, want), cache
        if cache == "same":
            assert torch.equal(rh.bits(got), rh.bits(v.contiguous()))


@pytest.mark.parametrize("cache", ["same", "fp8", "int4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hkv,D,bs,lens,R,new", [
    (8, 128, 16, [500, 17, 1, 0], 20, None),        # shorter than the rows: zeros in front
    (3, 128, 1, [30], 30, None),
    (4, 256, 784, [1600, 785], 900, None),
    (1, 256, 33, [66, 5], None, [66, 0]),
    (8, 128, 16, [33, 0, 100, 7], None, [33, 0, 64, 7]),
])
def test_gather(cuda_lib, cache, dtype, Hkv, D, bs, lens, R, new):
    rng = np.random.default_rng(9)
    bt, pool = rh.tables_for(lens, bs, 10)
    ks, vs = SCALES[cache]
    caches = []
    for i in range(2):
        if cache == "int4":
            c = torch.from_numpy(o4.quantise(rng.standard_normal((pool, Hkv, bs, D))))
        else:
            c = torch.from_numpy(rng.standard_normal((pool, bs, Hkv, D))).to(
                torch.float8_e4m3fn if cache == "fp8" else DT[dtype])
        caches.append(c)
    starts = None if new is None else [2] + [2 + int(n) for n in np.cumsum(new)]
    rows = R if new is None else starts[-1] + 3
    shape = (len(lens), R, Hkv, D) if new is None else (rows, Hkv, D)
    outs = [torch.full(shape, 5.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    k, v = cuda_lib.gather(caches[0].cuda(), caches[1].cuda(), bt.cuda(), i32(lens), rows,
                           starts=i32(starts), dtype=DT[dtype], k_out=outs[0], v_out=outs[1],
                           k_scale=ks, v_scale=vs)
    for got, c, s in ((k, caches[0], ks), (v, caches[1], vs)):
        got = got.cpu().reshape(-1, Hkv, D)
        want = torch.full_like(got, 5.0)
        for r, b, p in rh.positions(lens, starts, R, len(lens)):
            if p < 0:
                want[r] = 0
                continue
            raw = rh.cache_rows(c, cache, bt, b, np.array([p]), bs)
            if cache == "same":
                want[r] = raw[0]
            else:
                # the value is exact in fp32, its product with the scale rounded there, then
                # once to the type: the same two roundings here
                x = torch.from_numpy(rh.values(raw, cache)[0]).float()
                want[r] = (x * torch.tensor(s, dtype=torch.float32)).to(DT[dtype])
        assert torch.equal(rh.bits(got), rh.bits(want))
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace()) == 0


def test_gather_defaults(cuda_lib):
    x = make([20, 9], None, 4, 2, 2, 128, 16, "bf16", "same", seed=11)
    _, kc, vc = append(cuda_lib, x, None)
    k, v = cuda_lib.gather(kc, vc, x["bt"].cuda(), i32(x["lens"]), 4)
    assert k.dtype == torch.bfloat16 and k.shape == (2, 4, 2, 128)
    assert torch.equal(rh.bits(v), rh.bits(views(x, x["qkv"])[2].contiguous()))
    k, v = cuda_lib.gather(kc, vc, x["bt"].cuda(), i32(x["lens"]), 0)
    assert k.shape == (2, 0, 2, 128)


@pytest.mark.parametrize("cache", ["same", "int4"])
def test_bad_tables_and_lengths_are_reported(cuda_lib, cache):
    # a table entry outside the pool, a length past the table and a negative one: the rows are
    # not written, the rest is; the error word tells
    lens = [20, 20, 200, -4]
    x = make([20, 20, 20, 20], None, 2, 2, 1, 128, 16, "bf16", cache, seed=12)
    x["bt"][1, 1] = 99
    clean = dict(x, lens=lens)
    rope, f, amp = rope_of(cuda_lib, 128)
    ws = torch.zeros(cuda_lib.PA_WORKSPACE_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    qo, kc, vc = append(cuda_lib, clean, rope, workspace=ws)
    assert cuda_lib.read_device_errors(ws) == \
        cuda_lib.PA_DEVERR_BLOCK_INDEX | cuda_lib.PA_DEVERR_SEQ_LEN
    assert cuda_lib.read_device_errors(ws) == 0
    assert torch.all(qo[2:] == 0) and torch.isfinite(qo).all()
    # only sequence 0's slots changed
    for c, c0 in ((kc, x["kc"]), (vc, x["vc"])):
        a, b = (t.cpu().view(torch.uint8) for t in (c, c0))
        diff = (a != b).reshape(a.shape[0], -1).any(1)
        assert diff.nonzero().flatten().tolist() == [int(x["bt"][0, 1])]
    k, v = cuda_lib.gather(kc, vc, x["bt"].cuda(), i32(lens), 2, dtype=torch.bfloat16, workspace=ws)
    assert torch.all(k[1:] == 0) and torch.all(v[1:] == 0) and torch.any(k[0] != 0)
    assert cuda_lib.read_device_errors(ws) == \
        cuda_lib.PA_DEVERR_BLOCK_INDEX | cuda_lib.PA_DEVERR_SEQ_LEN


def test_starts_that_do_not_ascend_stay_in_bounds(cuda_lib):
    x = make([20, 20, 20], [2, 2, 2], 0, 2, 1, 128, 16, "bf16", "same", seed=13)
    for starts in ([0, 5, 1, 6], [6, 4, 2, 0], [0, 0, 0, 0], [-3, -2, 9, 3]):
        bad = dict(x, starts=starts)
        append(cuda_lib, bad, None)
    torch.cuda.synchronize()


def test_streams_and_graphs(cuda_lib):
    # two streams with buffers and workspaces of their own, and a captured append + gather
    # replayed on new lengths and new rows
    x = make([33, 50], None, 2, 8, 4, 128, 16, "bf16", "int4", seed=14)
    rope, f, amp = rope_of(cuda_lib, 128)
    ks, vs = SCALES["int4"]
    runs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            runs.append(append(cuda_lib, x, rope))
    torch.cuda.synchronize()
    for r in runs:
        check_append(x, f, amp, False, *r)

    qkv, kc, vc, bt = x["qkv"].cuda(), x["kc"].cuda(), x["vc"].cuda(), x["bt"].cuda()
    lens = i32(x["lens"])
    q, k, v = views(x, qkv)
    ws = torch.zeros(1 << 14, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    cuda_lib.load()
    with torch.cuda.graph(g):
        qo = cuda_lib.append(k, v, kc, vc, bt, lens, q=q, rope=rope, k_scale=ks, v_scale=vs,
                             workspace=ws)
        ko, vo = cuda_lib.gather(kc, vc, bt, lens, 2, dtype=torch.bfloat16, k_scale=ks, v_scale=vs,
                                 workspace=ws)
    for step in range(3):
        y = make([33, 50], None, 2, 8, 4, 128, 16, "bf16", "int4", seed=20 + step)
        y.update(bt=x["bt"], kc=kc.cpu().clone(), vc=vc.cpu().clone(), lens=[30 + step, 45 - step])
        qkv.copy_(y["qkv"])
        lens.copy_(i32(y["lens"]))
        g.replay()
        torch.cuda.synchronize()
        check_append(y, f, amp, False, qo, kc, vc)
        for b in range(2):
            pos = np.arange(y["lens"][b] - 2, y["lens"][b])
            for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
                raw = rh.cache_rows(c, "int4", x["bt"], b, pos, 16)
                want = torch.from_numpy(rh.values(raw, "int4")).float() * np.float32(s)
                assert torch.equal(rh.bits(got[b]), rh.bits(want.to(torch.bfloat16)))


def test_append_then_decode_reads_the_new_tokens(cuda_lib):
    # kernels chained by dependent launches: twenty decode steps, each appending one token and
    # attending to it at once, equal the same steps with a synchronisation after every call
    B, Hq, Hkv, D, bs = 3, 8, 2, 128, 16
    rope, _, _ = rope_of(cuda_lib, 128)
    for cache in ("same", "fp8", "int4"):
        outs = []
        for sync in (False, True):
            torch.manual_seed(15)
            bt = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
            kc = rh.empty_pool(cache, B * 4, bs, Hkv, D, "bf16", 16, nan=False).cuda()
            vc = kc.clone()
            qkv = torch.randn((20, B, (Hq + 2 * Hkv) * D), device="cuda").bfloat16()
            lens = torch.tensor([1, 14, 30], dtype=torch.int32, device="cuda")
            if cache == "int4":
                kc.zero_()
                vc.zero_()
            got = []
            for step in range(20):
                y = qkv[step].view(B, Hq + 2 * Hkv, D)
                q = cuda_lib.append(y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], kc, vc, bt, lens, q=y[:, :Hq],
                                    rope=rope, k_scale=0.05, v_scale=0.05)
                if sync:
                    torch.cuda.synchronize()
                got.append(cuda_lib.decode(q, kc, vc, bt, lens, 0.088, max_seq_len=64, k_scale=0.05,
                                           v_scale=0.05, deterministic=True))
                if sync:
                    torch.cuda.synchronize()
                lens += 1
            outs.append(torch.stack(got).cpu())
        assert torch.isfinite(outs[0]).all()
        assert torch.equal(rh.bits(outs[0]), rh.bits(outs[1])), cache


def test_python_refusals(cuda_lib):
    x = make([20, 20], None, 2, 4, 2, 128, 16, "bf16", "same", seed=17)
    qkv, kc, vc, bt, lens = x["qkv"].cuda(), x["kc"].cuda(), x["vc"].cuda(), x["bt"].cuda(), i32([20, 20])
    q, k, v = views(x, qkv)
    rope = cuda_lib.rope(128)
    with pytest.raises(ValueError):
        cuda_lib.append(k, v[:, :1], kc, vc, bt, lens)
    with pytest.raises(ValueError):
        cuda_lib.append(k.transpose(2, 3).contiguous().transpose(2, 3), v, kc, vc, bt, lens)
    with pytest.raises(ValueError):
        cuda_lib.append(k, v, kc, vc, bt, lens, q=q[:1])
    with pytest.raises(ValueError):
        cuda_lib.append(k, v, kc, vc, bt, lens, q_out=torch.empty_like(q))
    with pytest.raises(ValueError):
        cuda_lib.append(k, v, kc, vc, bt, lens, q=q, q_out=q)           # not contiguous
    with pytest.raises(ValueError):
        cuda_lib.append(k, v, kc, vc, bt, lens, rope=cuda_lib.Rope(rope.turns.cpu()))
    with pytest.raises(TypeError):
        cuda_lib.append(k, v, kc, vc, bt, lens, rope=cuda_lib.Rope(rope.turns.int()))
    with pytest.raises(cuda_lib.PAError):
        cuda_lib.append(k, v, kc, vc, bt, lens, rope=cuda_lib.Rope(rope.turns[:12]))
    with pytest.raises(cuda_lib.PAError):
        cuda_lib.append(k, v, kc.view(torch.uint8).view(torch.float8_e4m3fn)[..., :128].contiguous(),
                        vc.view(torch.uint8).view(torch.float8_e4m3fn)[..., :128].contiguous(),
                        bt, lens, k_scale=0.0)
    with pytest.raises(ValueError):
        cuda_lib.gather(kc, vc, bt, lens, -1)
    with pytest.raises(ValueError):
        cuda_lib.gather(kc, vc, bt, lens, 2, k_out=torch.empty(2, 3, 2, 128, device="cuda").bfloat16())


def test_first_call_in_a_capture_and_given_streams(cuda_lib):
    # a stream whose first call is captured: the workspace made there stays the graph's, and a
    # later call outside it starts from one of its own; and calls on a given stream
    x = make([33, 50], None, 2, 4, 2, 128, 16, "bf16", "int4", seed=30)
    rope, f, amp = rope_of(cuda_lib, 128)
    ks, vs = SCALES["int4"]
    s = torch.cuda.Stream()
    qkv, kc, vc, bt, lens = x["qkv"].cuda(), x["kc"].cuda(), x["vc"].cuda(), x["bt"].cuda(), i32(x["lens"])
    q, k, v = views(x, qkv)
    dq = torch.randn((2, 4, 128), device="cuda").bfloat16()
    long_bt = bt.repeat(1, 40)     # 2560 tokens of repeated blocks: several splits
    long_lens = torch.tensor([2500, 1900], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        qo = cuda_lib.append(k, v, kc, vc, bt, lens, q=q, rope=rope, k_scale=ks, v_scale=vs)
        out = cuda_lib.decode(dq, kc, vc, long_bt, long_lens, 0.088, max_seq_len=2560, deterministic=True,
                              k_scale=ks, v_scale=vs)
    assert cuda_lib.default_workspace(stream=s) is None
    want_cache = append(cuda_lib, x, rope)
    want = cuda_lib.decode(dq, want_cache[1], want_cache[2], long_bt, long_lens, 0.088, max_seq_len=2560,
                           deterministic=True, k_scale=ks, v_scale=vs)
    for _ in range(2):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check_append(x, f, amp, False, qo, kc, vc)
        assert torch.equal(rh.bits(out), rh.bits(want))
    # on the given stream, from another current one
    got = cuda_lib.decode(dq, kc, vc, long_bt, long_lens, 0.088, max_seq_len=2560, deterministic=True,
                          k_scale=ks, v_scale=vs, stream=s)
    gk, gv = cuda_lib.gather(kc, vc, bt, lens, 2, dtype=torch.bfloat16, k_scale=ks, v_scale=vs, stream=s)
    s.synchronize()
    assert torch.equal(rh.bits(got), rh.bits(want)) and torch.isfinite(gk).all() and torch.isfinite(gv).all()
    # (the repeated table holds -1 entries of the shorter sequence: the decode calls report them)
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace(stream=s), stream=s) == \
        cuda_lib.PA_DEVERR_BLOCK_INDEX
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace()) == cuda_lib.PA_DEVERR_BLOCK_INDEX
