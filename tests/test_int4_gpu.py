"""Decode attention over 4-bit caches against the float64 oracle (GB300 only)."""
import math

import numpy as np
import pytest
import torch

import rows_harness as rh
from oracle import decode_ref, decode_ref_rows
from oracle import int4 as o4

pytestmark = pytest.mark.gpu


def tolerance(out_dtype, K, V, step_max, ref, L):
    """Absolute bound of an output element's error. Scores: the query's fp16 form is exact for
    bf16 and for normal fp16 elements, the products with codes are exact, sums are fp32. A
    weight p <= 1 (with the largest >= 2^-4) is rounded to fp16 (2^-11 of it, or 2^-25), and
    so is its product with the token's step; the output once to its type.
      sum p (2^-11 |v| + 2^-11 step n) / sum p <= 2^-11 (Vmax + 15 step_max)
      L 2^-25 (Vmax + 15 step_max) / 2^-4 for weights below fp16's normal range
      2^-16 Vmax for scores off by up to 2^-17 (fp32 sums of up to 256 products of size < 16)"""
    vmax = max(float(np.abs(v).max()) if v.size else 0.0 for v in V)
    spread = vmax + 15 * step_max
    return (rh.HALF_STEP[out_dtype] * np.abs(ref) + 2.0 ** -11 * spread +
            min(2.0 ** -11, L * 2.0 ** -21) * spread + 2.0 ** -16 * vmax)


def run_case(pa, lens, Hq, Hkv, D, bs, dtype="bf16", rows=1, seed=0, scale=None, step=0.3, spread=1.0,
             qmul=1.0, k_scale=1.0, v_scale=1.0, **kw):
    kc, vc, bt, K, V = rh.random_int4_pool(lens, bs, Hkv, D, seed, step, spread)
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    shape = (B, Hq, D) if rows == 1 else (B, rows, Hq, D)
    q = (torch.randn(shape, generator=g) * qmul).to(rh.DT[dtype])
    scale = float(np.float32(scale if scale is not None else 1 / math.sqrt(D)))
    ks, vs = float(np.float32(k_scale)), float(np.float32(v_scale))
    Ks, Vs = [k * ks for k in K], [v * vs for v in V]
    ref = decode_ref(rh.f64(q), Ks, Vs, scale, window=kw.get("window", 0)) if rows == 1 else \
        decode_ref_rows(rh.f64(q), Ks, Vs, scale)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    out = pa.decode(q.cuda(), kc.cuda(), vc.cuda(), bt.cuda(),
                    torch.tensor(lens, dtype=torch.int32, device="cuda"), scale,
                    max_seq_len=max(lens + [1]), k_scale=k_scale, v_scale=v_scale, workspace=ws, **kw)
    got = rh.f64(out)
    assert pa.read_device_errors(ws) == 0
    assert np.all(np.isfinite(got))
    tol = tolerance(dtype, Ks, Vs, vs * step * math.exp(2.5 * spread), ref, max(lens))
    err = np.abs(got - ref)
    assert np.all(err <= tol), (float((err / tol).max()), float(err.max()))
    return float(err.max() / max(np.abs(ref).max(), 1e-30))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,bs,lens", [
    (8, 8, 128, 16, [512]),
    (8, 8, 128, 16, [0, 1, 15, 16, 17, 31, 32, 33]),
    (32, 8, 128, 16, [1000, 37, 4097]),
    (6, 2, 128, 1, [130]),
    (24, 4, 256, 784, [500, 785, 3000]),
    (2, 2, 256, 33, [0, 1, 16, 17, 100]),
    (16, 1, 128, 48, [700]),              # 16 heads per KV head
    (16, 1, 256, 16, [700, 5]),
    (12, 1, 128, 7, [63, 64, 65]),
])
def test_decode_int4(cuda_lib, dtype, Hq, Hkv, D, bs, lens):
    run_case(cuda_lib, lens, Hq, Hkv, D, bs, dtype, seed=1)


@pytest.mark.parametrize("S", [1, 2, 3, 5, 8, 9, 40])
@pytest.mark.parametrize("D,bs", [(128, 16), (256, 100)])
def test_decode_int4_splits(cuda_lib, S, D, bs):
    # one split, splits merging in their cluster, and a merge grid; with and without shared tails
    for det in (False, True):
        run_case(cuda_lib, [2500, 1, 0, 777], 8, 2, D, bs, seed=2, splits=S, deterministic=det)


@pytest.mark.parametrize("rows,Hq,Hkv,D", [(2, 8, 8, 128), (4, 32, 8, 128), (8, 8, 2, 128),
                                           (2, 16, 2, 256), (3, 5, 1, 256)])
def test_decode_int4_query_rows(cuda_lib, rows, Hq, Hkv, D):
    for S in (0, 1, 3):
        run_case(cuda_lib, [600, rows, 1, 0, 33], Hq, Hkv, D, 16, rows=rows, seed=3, splits=S)


@pytest.mark.parametrize("B,Hq,Hkv,D,bs,rows", [
    (32, 16, 8, 128, 16, 1), (50, 8, 4, 128, 16, 2), (200, 4, 2, 128, 16, 1), (256, 6, 2, 256, 48, 1),
    (41, 16, 4, 256, 784, 1), (24, 64, 8, 128, 16, 4), (20, 8, 8, 128, 16, 1),
])
def test_decode_int4_mixed_batches_run_by_length(cuda_lib, B, Hq, Hkv, D, bs, rows):
    # more (sequence, KV head) pairs than SMs (152; the last case has about as many) and the
    # total given: CTAs start by length, in an order of their own, with the same results as in
    # the batch's order
    r = np.random.default_rng(B)
    lens = [int(x) for x in r.integers(0, 200, B)]
    lens[B // 3], lens[B // 2], lens[-1] = 4000, 0, 4000
    run_case(cuda_lib, lens, Hq, Hkv, D, bs, rows=rows, seed=14, total_tokens=sum(lens))
    kc, vc, bt, _, _ = rh.random_int4_pool(lens, bs, Hkv, D, 15)
    q = torch.randn((B, Hq, D) if rows == 1 else (B, rows, Hq, D)).bfloat16().cuda()
    for bad in (False, True):   # lengths that the call reports are clamped in either order
        if bad:
            lens[1], lens[2] = -5, 2 ** 31 - 1
            bt = torch.where(bt < 0, torch.zeros_like(bt), bt)
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        outs, flags = [], []
        for total in (0, 4000 + 100 * B):
            ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
            outs.append(cuda_lib.decode(q, kc.cuda(), vc.cuda(), bt.cuda(), sl, 0.088, max_seq_len=4000,
                                        splits=1, total_tokens=total, workspace=ws))
            flags.append(cuda_lib.read_device_errors(ws))
        assert flags == [cuda_lib.PA_DEVERR_SEQ_LEN if bad else 0] * 2
        assert torch.equal(rh.bits(outs[0].cpu()), rh.bits(outs[1].cpu()))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,Hq,Hkv,D,bs,longest", [
    (40, 8, 4, 128, 16, 300), (160, 1, 1, 128, 7, 2000), (30, 24, 6, 256, 33, 500),
    (300, 8, 8, 128, 16, 70), (20, 64, 8, 128, 16, 1000), (90, 4, 2, 256, 784, 1900),
])
def test_decode_int4_many_short_contexts(cuda_lib, dtype, B, Hq, Hkv, D, bs, longest):
    # more (sequence, KV head) pairs than SMs, unsplit: CTAs of four warps
    r = np.random.default_rng(B)
    lens = [int(x) for x in r.integers(0, longest + 1, B)]
    lens[0], lens[1], lens[2], lens[-1] = longest, 0, 1, longest
    run_case(cuda_lib, lens, Hq, Hkv, D, bs, dtype, seed=16)
    run_case(cuda_lib, lens, Hq, Hkv, D, bs, dtype, seed=17, total_tokens=sum(lens), deterministic=True)
    kc, vc, bt, _, _ = rh.random_int4_pool(lens, bs, Hkv, D, 18)
    lens[3], lens[4] = -1, longest + 1
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    out = cuda_lib.decode(torch.randn((B, Hq, D)).to(rh.DT[dtype]).cuda(), kc.cuda(), vc.cuda(),
                          bt.clamp(min=0).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.088,
                          max_seq_len=longest, workspace=ws)
    assert cuda_lib.read_device_errors(ws) == cuda_lib.PA_DEVERR_SEQ_LEN
    assert torch.isfinite(out[5:]).all() and not out[3].any()


@pytest.mark.parametrize("W", [1, 17, 1000])
def test_decode_int4_window(cuda_lib, W):
    run_case(cuda_lib, [1500, 999, 16, 1], 8, 4, 128, 16, seed=4, window=W)
    run_case(cuda_lib, [1500, 999, 16, 1], 6, 2, 256, 784, "f16", seed=4, window=W)


@pytest.mark.parametrize("qmul", [1e-6, 1e-3, 30.0, 1e4])
def test_decode_int4_query_range(cuda_lib, qmul):
    # queries far from 1 (the scale brings the scores back): the fp16 form follows their range
    run_case(cuda_lib, [300], 8, 2, 128, 16, "bf16", seed=5, qmul=qmul, scale=0.088 / qmul)
    if qmul >= 1e-3:   # fp16 queries lose bits of their own below its normal range
        run_case(cuda_lib, [300], 8, 2, 256, 16, "f16", seed=5, qmul=qmul, scale=0.0625 / qmul)


@pytest.mark.parametrize("step", [1e-2, 1.0, 50.0])
def test_decode_int4_value_range(cuda_lib, step):
    run_case(cuda_lib, [400, 33], 8, 2, 128, 16, seed=6, step=step, scale=0.02 / step)


def test_decode_int4_scales(cuda_lib):
    run_case(cuda_lib, [400, 33], 8, 2, 128, 16, seed=7, k_scale=0.125, v_scale=300.0)
    run_case(cuda_lib, [400, 33], 8, 2, 256, 784, seed=7, k_scale=3.0, v_scale=1e-3)


def test_decode_int4_sharp_scores(cuda_lib):
    # scores far apart: the running maximum climbs through many tiles, weights underflow
    for scale in (1.0, 4.0):
        run_case(cuda_lib, [3000], 4, 1, 128, 16, "f16", seed=8, scale=scale)
        run_case(cuda_lib, [3000], 4, 1, 256, 16, "f16", seed=8, scale=scale, splits=1)


def test_decode_int4_long_context_offsets(cuda_lib):
    # a table whose live blocks lie at the far end of a pool past 4 GB per cache
    Hkv, D, bs, L = 8, 128, 16, 200
    kc4, vc4, bt, K, V = rh.random_int4_pool([L], bs, Hkv, D, 9)
    nb = (5 << 30) // (Hkv * bs * 80)
    pool = [torch.zeros((nb, Hkv, bs, 80), dtype=torch.uint8, device="cuda") for _ in range(2)]
    used = kc4.shape[0]
    for p, c in zip(pool, (kc4, vc4)):
        p[nb - used:] = c.cuda()
    q = torch.randn((1, 8, D), generator=torch.Generator().manual_seed(9)).bfloat16()
    out = cuda_lib.decode(q.cuda(), pool[0], pool[1], (bt + (nb - used)).cuda(),
                          torch.tensor([L], dtype=torch.int32, device="cuda"), 0.088, max_seq_len=L)
    ref = decode_ref(rh.f64(q), K, V, float(np.float32(0.088)))
    tol = tolerance("bf16", K, V, 0.3 * math.exp(2.5), ref, L)
    assert np.all(np.abs(rh.f64(out) - ref) <= tol)
    # append and gather there too
    k = torch.randn((1, Hkv, D)).bfloat16().cuda()
    btc, lens = (bt + (nb - used)).cuda(), torch.tensor([L], dtype=torch.int32, device="cuda")
    cuda_lib.append(k, k, pool[0], pool[1], btc, lens)
    ko, vo = cuda_lib.gather(pool[0], pool[1], btc, lens, 1, dtype=torch.bfloat16)
    assert torch.equal(ko, vo) and (ko[0].float() - k.float()).abs().max() < 0.4


def test_decode_int4_unused_slots_do_not_matter(cuda_lib):
    # NaN steps and minima, then arbitrary finite ones, in every slot without a token
    for lens in ([33], [1, 47, 1000]):
        kc, vc, bt, K, V = rh.random_int4_pool(lens, 16, 2, 128, 10)
        q = torch.randn((len(lens), 8, 128), generator=torch.Generator().manual_seed(1)).half().cuda()
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        outs = []
        for fill in (None, 0x00, 0x7b, 0xfc):   # NaN as made; zero; large; minus infinity
            c = [kc.clone(), vc.clone()]
            if fill is not None:
                live = torch.zeros(kc.shape[0], 16, dtype=torch.bool)
                for b, L in enumerate(lens):
                    p = torch.arange(L)
                    live[bt[b, p // 16].long(), p % 16] = True
                for t in c:
                    y = t.transpose(1, 2)
                    y[~live] = fill
            outs.append(cuda_lib.decode(q, c[0].cuda(), c[1].cuda(), bt.cuda(), sl, 0.088,
                                        max_seq_len=max(lens), deterministic=True).cpu())
        for o in outs[1:]:
            assert torch.equal(rh.bits(o), rh.bits(outs[0]))


def test_decode_int4_nan_group_stays_in_its_elements(cuda_lib):
    # a poisoned group of a live V row makes its own 32 output elements NaN, and no others
    kc, vc, bt, K, V = rh.random_int4_pool([40], 16, 1, 128, 11)
    vc[bt[0, 1], 0, 3, 64 + 2 * 2:64 + 2 * 2 + 2] = 0xFF     # the step of group 2 of token 19
    q = torch.randn((1, 4, 128)).half().cuda()
    out = cuda_lib.decode(q, kc.cuda(), vc.cuda(), bt.cuda(),
                          torch.tensor([40], dtype=torch.int32, device="cuda"), 0.088, max_seq_len=40)
    bad = torch.isnan(out[0]).cpu()
    assert bad[:, 64:96].all() and not bad[:, :64].any() and not bad[:, 96:].any()


def test_decode_int4_graph_and_streams(cuda_lib):
    lens = [700, 33]
    kc, vc, bt, K, V = rh.random_int4_pool(lens, 16, 2, 128, 12)
    dev = [t.cuda() for t in (kc, vc, bt)]
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((2, 8, 128), device="cuda").bfloat16()
    want = cuda_lib.decode(q, *dev, sl, 0.088, max_seq_len=700, deterministic=True).cpu()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):   # each graph with its own workspace and output
        ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cuda_lib.decode(q, *dev, sl, 0.088, out=out, max_seq_len=700, deterministic=True, workspace=ws)
        graphs.append((g, out, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, out, _, s in graphs:
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
        torch.cuda.synchronize()
        for _, out, _, _ in graphs:
            assert torch.equal(rh.bits(out), rh.bits(want))


def test_decode_int4_refusals(cuda_lib):
    c = torch.zeros((4, 2, 16, 80), dtype=torch.uint8, device="cuda")
    bt = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    sl = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    cuda_lib.decode(q, c, c, bt, sl, 0.1)
    with pytest.raises(ValueError):
        cuda_lib.decode(torch.zeros((1, 2, 256), dtype=torch.bfloat16, device="cuda"), c, c, bt, sl, 0.1)
    with pytest.raises(ValueError):
        cuda_lib.decode(q, c[..., :79].contiguous(), c[..., :79].contiguous(), bt, sl, 0.1)
    with pytest.raises(TypeError):
        cuda_lib.decode(q, c, c.view(torch.int8), bt, sl, 0.1)
    with pytest.raises(cuda_lib.PAError):
        cuda_lib.decode(q, c, c, bt, sl, 0.1, k_scale=0.0)


def test_outgrown_workspaces_stay_allocated(cuda_lib):
    # a graph captured with the default workspace keeps writing to it after the workspace of
    # its stream has been replaced by a larger one
    s = torch.cuda.Stream()
    dev = torch.device("cuda", torch.cuda.current_device())
    a = cuda_lib._workspace(1 << 16, dev, s.cuda_stream)
    b = cuda_lib._workspace(a.numel() + 1, dev, s.cuda_stream)
    assert b.numel() >= 2 * a.numel() and any(t is a for t in cuda_lib._outgrown)


@pytest.mark.parametrize("D", [128, 256])
def test_saturated_rows_decode_to_finite_outputs(cuda_lib, D):
    # values past what a row holds: the bytes are the oracle's, and decode (whose sums run from
    # both ends of the codes) agrees with the values they stand for
    Hkv, L, bs = 2, 70, 16
    g = torch.Generator().manual_seed(13)
    v = torch.randn((1, L, Hkv, D), generator=g) * torch.exp(torch.rand((1, L, Hkv, 1), generator=g) * 70 + 8)
    v[0, :20] = torch.sign(v[0, :20]) * 65280.0
    v = v.bfloat16()
    k = torch.randn((1, L, Hkv, D), generator=g).bfloat16()
    nb = -(-L // bs)
    kc, vc = (torch.zeros((nb, Hkv, bs, D // 8 * 5), dtype=torch.uint8, device="cuda") for _ in range(2))
    bt, lens = torch.arange(nb, dtype=torch.int32, device="cuda")[None], torch.tensor([L], dtype=torch.int32, device="cuda")
    cuda_lib.append(k.cuda(), v.cuda(), kc, vc, bt, lens)
    K, V = (c.cpu().transpose(1, 2).reshape(-1, Hkv, D // 8 * 5)[:L].numpy() for c in (kc, vc))
    assert np.array_equal(V, o4.quantise(rh.f64(v[0])))
    q = torch.randn((1, 4, D), generator=g).bfloat16()
    scale = float(np.float32(0.088))
    out = cuda_lib.decode(q.cuda(), kc, vc, bt, lens, scale, max_seq_len=L)
    K, V = [o4.dequant(K)], [o4.dequant(V)]
    ref = decode_ref(rh.f64(q), K, V, scale)
    got = rh.f64(out)
    # (the sixteenth value of a group, rounded to fp16 where the sums start from it: 2^-11)
    tol = tolerance("bf16", K, V, 8704.0, ref, L) + 2.0 ** -11 * 65520
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - ref) <= tol)


def test_workspaces_and_flags_are_checked(cuda_lib):
    c = torch.zeros((4, 2, 16, 80), dtype=torch.uint8, device="cuda")
    bt = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    sl = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    for ws in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            cuda_lib.decode(q, c, c, bt, sl, 0.1, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            cuda_lib.append(q, q, c, c, bt, sl, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            cuda_lib.gather(c, c, bt, sl, 1, dtype=torch.bfloat16, workspace=ws)
    with pytest.raises(RuntimeError):   # no truth value
        cuda_lib.decode(q, c, c, bt, sl, 0.1, deterministic=torch.zeros(2))
    cuda_lib.decode(q, c, c, bt, sl, 0.1)


def test_outputs_of_a_given_stream_are_allocated_in_its_order(cuda_lib):
    # not from memory that the current stream's pending kernels may still use
    nb, s = 64, torch.cuda.Stream()
    c = torch.zeros((nb, 2, 16, 80), dtype=torch.uint8, device="cuda")
    bt = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    sl = torch.tensor([1024], dtype=torch.int32, device="cuda")
    rows = torch.zeros((1, 1024, 2, 128), dtype=torch.bfloat16, device="cuda")
    one = rows[:, 0].contiguous()
    torch.cuda.synchronize()
    for call in (lambda: cuda_lib.gather(c, c, bt, sl, 1024, dtype=torch.bfloat16, stream=s),
                 lambda: [cuda_lib.append(rows, rows, c, c, bt, sl, q=rows, stream=s)],
                 lambda: [cuda_lib.decode(one, c, c, bt, sl, 0.1, stream=s)]):
        torch.cuda.empty_cache()
        freed = [torch.empty_like(rows) for _ in range(4)] + [torch.empty(512, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
        at = {t.data_ptr() for t in freed}
        del freed
        outs = call()
        assert not at & {t.data_ptr() for t in outs}
        s.synchronize()
