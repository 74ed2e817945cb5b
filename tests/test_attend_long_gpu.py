"""Cross attention and decode behind prefixes where every CTA holds pieces of many token tiles, with scores
that raise the rows' references along the context (GB300 only): accumulators rescaled amid a piece, of one row
tile and of two, the ring of tiles around several times within an item, items of both kinds in one run."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import attend_harness as ah

pytestmark = pytest.mark.gpu

LENS = [3900, 2100, 3333, 2900, 4000, 2047, 3100, 2500] * 3 + [3800, 2222, 2999, 3501]
HKV, G = 8, 4
TILE = {128: 128, 256: 64}


def piece_tiles(D, rows, lens):
    """Token tiles of the longest piece that a CTA is sure to hold: the division of the work by units (5 an item, 3
    or 2 a tile with two row tiles or one), a run per SM."""
    tiles = [-(-L // TILE[D]) for L in lens]
    per_item = (2 if D == 128 else 1) * (128 // G)
    items = -(-rows // per_item)
    last = rows - (items - 1) * per_item
    w = [3 if D == 128 else 2] * (items - 1) + [3 if D == 128 and last > 128 // G else 2]
    total = sum(HKV * sum(5 + x * t for x in w) for t in tiles)
    run = -(-total // torch.cuda.get_device_properties(0).multi_processor_count)
    # the part of a run before or after an item's border is at least half of it
    return min(min(tiles), (run - 5) // 2 // max(w))


def cached(shape, D, cache, dtype, seed):
    """K, V [L, HKV, D] of one long context as stored, in 64 bits, and the scores' direction."""
    L, g = max(LENS), torch.Generator(device="cuda").manual_seed(seed)
    u = torch.randn((HKV, D), generator=g, device="cuda", dtype=torch.float64)
    u /= u.norm(dim=-1, keepdim=True)
    t = torch.arange(L, device="cuda", dtype=torch.float64)
    height = {"climbing": t / L * 16 - 8,
              "steps": torch.div(t, 700, rounding_mode="floor") * 2.0 - 6}[shape]
    K = height[:, None, None] * u + 0.05 * torch.randn((L, HKV, D), generator=g, device="cuda")
    V = torch.randn((L, HKV, D), generator=g, device="cuda")
    scale = ah.SCALE8 if cache == "fp8" else 1.0
    store = (lambda x: (x / scale).float().clamp(-448, 448).to(torch.float8_e4m3fn)) if cache == "fp8" else \
        (lambda x: x.to(ah.DT[dtype]))
    stored = [store(x) for x in (K, V)]
    factor = float(np.float32(scale))
    return stored, [x.float().double() * factor for x in stored], u, scale


def paged(stored, bs, seed):
    """The context in blocks at random places, slots behind it NaN; every sequence's table names them."""
    L = stored[0].shape[0]
    n = -(-L // bs)
    perm = torch.randperm(n + 3, generator=torch.Generator().manual_seed(seed))[:n].cuda()
    out = []
    for x in stored:
        c = torch.full((n + 3, bs, HKV, x.shape[-1]), float("nan"), device="cuda").to(x.dtype)
        raw = torch.uint8 if x.dtype == torch.float8_e4m3fn else torch.int16
        t = torch.arange(L, device="cuda")
        c.view(raw)[perm[t // bs], t % bs] = x.view(raw)
        out.append(c)
    return (*out, perm.to(torch.int32)[None].repeat(len(LENS), 1))


def attend(q, K, V, lim):
    """As attend_harness.attend with scale 1, on the GPU. q [n, Hq, D]; row i sees tokens before lim[i]."""
    n = q.shape[0]
    out, mag, size = torch.zeros_like(q), torch.zeros_like(q), 0.0
    masked = torch.arange(K.shape[0], device="cuda")[None, :] >= lim[:, None]
    for h in range(q.shape[1]):
        k, v = K[:, h // G], V[:, h // G]
        s = (q[:, h] @ k.T).masked_fill(masked, -torch.inf)
        w = torch.softmax(s, -1)
        out[:, h], mag[:, h] = w @ v, w @ v.abs()
        size = max(size, float((q[:, h].abs() @ k.abs().T).max()))
    return out.cpu().numpy(), mag.cpu().numpy(), size


def check(got, q, wide, lens, rows, D, cache, dtype, causal):
    K, V = wide
    pool = SimpleNamespace(lens=lens, cache=cache, dtype=dtype, D=D, V=[V.cpu().numpy()])
    for b, L in enumerate(lens):
        lim = torch.full((rows,), L, device="cuda")
        if causal:
            lim = L - rows + 1 + torch.arange(rows, device="cuda")
        ref, mag, size = attend(q[b].double(), K[:L], V[:L], lim)
        ah.check(got[b], ref, mag, size, pool, 1.0, f"sequence {b}")


def queries(rows, u, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = 6.0 * u.repeat_interleave(G, 0) + 0.3 * torch.randn((len(LENS), rows, HKV * G, D), generator=g, device="cuda")
    return q.to(ah.DT[dtype])


@pytest.mark.parametrize("shape", ["climbing", "steps"])
@pytest.mark.parametrize("rows", [3, 24, 40, 70])                     # 12, 96, 160 and 280 rows of a KV head
@pytest.mark.parametrize("D,cache,dtype,bs", [(128, "same", "bf16", 16), (256, "same", "f16", 16), (128, "fp8", "bf16", 16),
                                              (256, "fp8", "f16", 33), (128, "same", "f16", 33)])
def test_cross(cuda_lib, D, cache, dtype, bs, rows, shape):
    assert piece_tiles(D, rows, LENS) >= 6
    stored, wide, u, scale = cached(shape, D, cache, dtype, 7)
    kc, vc, bt = paged(stored, bs, 7)
    q = queries(rows, u, D, dtype, rows)
    sl = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    out = cuda_lib.cross(q, kc, vc, bt, sl, 1.0, k_scale=scale, v_scale=scale)
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace()) == 0
    check(out, q, wide, LENS, rows, D, cache, dtype, False)


@pytest.mark.parametrize("shape", ["climbing", "steps"])
@pytest.mark.parametrize("rows", [1, 5, 40])
@pytest.mark.parametrize("D,cache,dtype", [(128, "same", "bf16"), (256, "same", "f16"), (128, "fp8", "f16")])
def test_decode_shared(cuda_lib, D, cache, dtype, rows, shape):
    # prefixes of 1900 and 2040 tokens and the rest of every sequence behind them, all of one text
    assert piece_tiles(D, rows, [L - 1900 for L in LENS if L > 2600]) >= 3
    stored, wide, u, scale = cached(shape, D, cache, dtype, 8)
    kc, vc, bt = paged(stored, 16, 8)
    q = queries(rows, u, D, dtype, rows)
    sl = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    groups, prefix = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 11, 25], [1900, 2040]))
    out = cuda_lib.decode_shared(q, kc, vc, bt, sl, 1.0, groups, prefix, k_scale=scale, v_scale=scale)
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace()) == 0
    check(out, q, wide, LENS, rows, D, cache, dtype, True)
