"""Cases of the operators around the paged KV cache: appending rotated keys and values,
reading rows back out, and decode attention over a cache held in 4 bits.

`run` computes an operator either in its plain form (elementary torch operations, fp32,
fp64 for the angles of the rotation) or, with `own` set, through the framework's public
calls. `exact` gives the same outputs from the definitions in 64 bits.

Shapes follow the repository's own workloads: 8/8, 32/8 and 32/16 heads with head_dim 128
and 16-token blocks, and the hybrid layer's 24/4 heads with head_dim 256 and 784-token
blocks.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
GROUP = 32  # elements that share a scale and a minimum in a 4-bit cache


# ------------------------------------------------------------------------------- cases
def listed():
    common = dict(rows=1, window=0, rot=128, interleaved=False, scaling="none")
    cases = [
        # the first decode step of one user: one new token, latency only
        dict(name="append 1 token", op="append", dtype="bf16", cache="same", B=1, Hq=8, Hkv=8,
             D=128, bs=16, lo=512, hi=512, ragged=0),
        # a decode step of a serving batch with an fp8 cache and a stretched context
        dict(name="append 64 tokens fp8", op="append", dtype="bf16", cache="fp8", B=64, Hq=32,
             Hkv=8, D=128, bs=16, lo=1024, hi=4096, ragged=0, scaling="yarn"),
        # prompts of odd lengths packed together, half of each head rotated, pairs interleaved
        dict(name="append packed prompts", op="append", dtype="f16", cache="same", B=5, Hq=32,
             Hkv=16, D=128, bs=16, lo=2048, hi=2600, ragged=8191, rot=64, interleaved=True),
        # one chunk of a long prompt into the hybrid layer's cache, a quarter rotated
        dict(name="append hybrid chunk fp8", op="append", dtype="bf16", cache="fp8", B=1, Hq=24,
             Hkv=4, D=256, bs=784, lo=20480, hi=20480, ragged=0, rows=2048, rot=64,
             scaling="linear"),
        # speculative decode into 4 bits: four new rows per sequence, written and read back
        dict(name="append and read rows int4", op="append_gather", dtype="bf16", cache="int4",
             B=8, Hq=32, Hkv=8, D=128, bs=16, lo=777, hi=4097, ragged=0, rows=4),
        # a prompt chunk into 4 bits, then the chunk read back for the prompt's attention
        dict(name="append and read chunk int4", op="append_gather", dtype="f16", cache="int4",
             B=3, Hq=24, Hkv=4, D=256, bs=784, lo=3001, hi=9000, ragged=4095, rot=256,
             scaling="yarn"),
        # a cached prefix of short prompts read back for the next chunk's attention
        dict(name="gather prefixes", op="gather", dtype="bf16", cache="same", B=7, Hq=32, Hkv=8,
             D=128, bs=16, lo=33, hi=1500, ragged=-1),
        # a long cached prefix of the hybrid layer, held in 4 bits
        dict(name="gather 32K int4", op="gather", dtype="bf16", cache="int4", B=1, Hq=24, Hkv=4,
             D=256, bs=784, lo=32768, hi=32768, ragged=0, rows=32768),
        # the smallest decode: one short context
        dict(name="decode int4 512", op="decode", dtype="bf16", cache="int4", B=1, Hq=8, Hkv=8,
             D=128, bs=16, lo=512, hi=512, ragged=0),
        # the hybrid layer at its longest context, one sequence
        dict(name="decode int4 hybrid 32K", op="decode", dtype="bf16", cache="int4", B=1, Hq=24,
             Hkv=4, D=256, bs=784, lo=32768, hi=32768, ragged=0),
        # speculative decode: four rows of four heads per KV head
        dict(name="decode int4 rows 16K", op="decode", dtype="f16", cache="int4", B=8, Hq=32,
             Hkv=8, D=128, bs=16, lo=16384, hi=16384, ragged=0, rows=4),
        # a serving batch of mixed lengths
        dict(name="decode int4 mixed batch", op="decode", dtype="bf16", cache="int4", B=32, Hq=32,
             Hkv=8, D=128, bs=16, lo=1024, hi=32768, ragged=0),
    ]
    return [{**common, **c} for c in cases]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "append_gather", "gather", "decode", "decode", "decode"])
    D, bs = rng.choice([(128, 16), (128, 16), (128, 33), (256, 784), (256, 16)])
    Hkv = rng.choice([4, 8, 16] if D == 128 else [2, 4])
    G = rng.choice([1, 2, 3, 4, 6, 8])
    cache = "int4" if op in ("decode", "append_gather") else rng.choice(["same", "fp8", "int4"])
    if op == "append" and cache == "int4":
        op = "append_gather"
    B = _log(rng, 1, 32)
    hi = _log(rng, 64, min(32768, 4194304 * 128 // (B * Hkv * D)))
    lo = max(1, int(hi * rng.choice([0.05, 0.5, 1.0])))
    most = min(8192, 2 ** 28 // (Hkv * (G + 2) * D))  # rows of a call
    rows, ragged, window = 1, 0, 0
    if op == "decode":
        rows = rng.choice([1, 1, 1, 2, 4]) if G <= 4 else 1
        window = rng.choice([0, 0, 1000]) if rows == 1 else 0
    elif rng.random() < 0.5:
        rows = max(1, min(_log(rng, 1, 4096), lo, most // B))
    elif op == "gather" or rng.random() < 0.3:
        ragged = -1 if B * hi <= most else min(4097, most)
    else:
        ragged = max(B, min(_log(rng, B, most), B * lo))
    return dict(op=op, dtype=rng.choice(["bf16", "f16"]), cache=cache, B=B, Hq=G * Hkv, Hkv=Hkv,
                D=D, bs=bs, lo=lo, hi=hi, ragged=ragged, rows=rows, window=window,
                rot=rng.choice([D, D, D // 2, 32]), interleaved=rng.random() < 0.4,
                scaling=rng.choice(["none", "linear", "yarn"]))


def _lengths(case):
    """(context lengths, new rows per sequence) on the host, fixed by the case."""
    B = case["B"]
    g = torch.Generator().manual_seed(B + case["hi"])
    lens = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=g).tolist()
    if case["ragged"] == -1:           # every token of every sequence
        return lens, list(lens)
    if case["ragged"]:                 # that many rows in all, shared out unevenly
        share = torch.rand(B, generator=g) + 0.2
        cut = (torch.cumsum(share, 0) / share.sum() * case["ragged"]).round().long().tolist()
        rows = [b - a for a, b in zip([0] + cut[:-1], cut)]
        return lens, [min(n, L) for n, L in zip(rows, lens)]
    return lens, [case["rows"]] * B


def _row_bytes(case):
    D = case["D"]
    return {"same": 2 * D, "fp8": D, "int4": D // 2 + 4 * D // GROUP}[case["cache"]]


def work(case):
    lens, new = _lengths(case)
    B, Hq, Hkv, D, T = case["B"], case["Hq"], case["Hkv"], case["D"], sum(new)
    cached = 2 * Hkv * _row_bytes(case)
    if case["op"] == "decode":
        R = case["rows"]
        seen = [min(L, case["window"]) if case["window"] else L for L in lens]
        tables = 4 * sum(-(-L // case["bs"]) for L in seen) + 4 * B
        return {"bytes": sum(seen) * cached + 4 * B * R * Hq * D + tables,
                "flops": 4 * R * Hq * D * sum(seen)}
    tables = 4 * sum(-(-n // case["bs"]) for n in new) + 8 * B
    nbytes, flops = tables, 0
    if case["op"] != "gather":         # q, k, v read; q and the cache rows written
        nbytes += T * ((2 * Hq + 2 * Hkv) * D * 2 + cached)
        flops += T * (Hq + Hkv) * case["rot"] * 3
    if case["op"] != "append":         # cache rows read, 16-bit rows written
        nbytes += T * (cached + 2 * Hkv * D * 2)
    return {"bytes": nbytes, "flops": flops + T * Hkv * D * 4}


# ------------------------------------------------------------------------------- inputs
def _frequencies(case):
    """Angle per token of each pair (radians, fp64) and the amplitude of cos and sin."""
    n = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    if case["scaling"] == "linear":
        return freq / 4.0, 1.0
    if case["scaling"] == "yarn":      # factor 8 over 4096 tokens, 32 to 1 turns kept to blended
        turn = lambda beta: n * math.log(4096 / (beta * 2 * math.pi)) / math.log(10000.0)
        low, high = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), 2 * n - 1)
        ramp = ((torch.arange(n, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
        return freq / 8.0 * ramp + freq * (1 - ramp), 0.1 * math.log(8.0) + 1.0
    return freq, 1.0


def prepare(case, seed):
    lens, new = _lengths(case)
    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device=DEVICE)

    # a pool somewhat larger than the batch needs, its blocks handed out at random
    blocks = [-(-L // bs) for L in lens]
    pool = sum(blocks) + sum(blocks) // 8 + 1
    perm = torch.randperm(pool, generator=gen, device=DEVICE).to(torch.int32)
    tables = torch.full((B, max(blocks)), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(blocks):
        tables[b, :n] = perm[at:at + n]
        at += n
    s = dict(case=case, max_len=max(lens), total=sum(lens), tables=tables,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE), starts=None)
    s["T"] = sum(new)
    if case["ragged"]:
        s["starts"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32,
                                   device=DEVICE)

    # the cache as earlier steps left it (fp8: values up to about 5 sigma at this scale)
    s["scale"] = 5.0 / 448.0 if case["cache"] == "fp8" else 1.0
    caches = []
    for _ in range(2):
        if case["cache"] == "same":
            c = randn(pool, bs, Hkv, D).to(dt)
        elif case["cache"] == "fp8":
            c = (randn(pool, bs, Hkv, D) / s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            c = _pack(randn(pool * Hkv, bs, D)).view(pool, Hkv, bs, -1)
        caches.append(c)
    s["k_cache"], s["v_cache"] = caches

    if case["op"] == "decode":
        shape = (B, Hq, D) if case["rows"] == 1 else (B, case["rows"], Hq, D)
        s["q"] = randn(*shape).to(dt)
    else:
        # one token's queries, keys and values, as a fused projection leaves them
        s["qkv"] = randn(s["T"], (Hq + 2 * Hkv) * D).to(dt)
        freq, s["amplitude"] = _frequencies(case)
        s["freq"] = freq.to(DEVICE)
        # the same angles as 64-bit fractions of a turn, the framework's form of them
        turns = [int(f * 2.0 ** 64 / (2 * math.pi)) for f in freq.tolist()]
        s["turns"] = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns],
                                  dtype=torch.int64, device=DEVICE)
    return s


# ------------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _split(s):
    """Views of the projection's rows: q, k, v as [rows, heads, D] or [B, R, heads, D]."""
    c = s["case"]
    lead = (s["T"],) if s["starts"] is not None else (c["B"], c["rows"])
    x = s["qkv"].view(*lead, c["Hq"] + 2 * c["Hkv"], c["D"])
    return x[..., :c["Hq"], :], x[..., c["Hq"]:c["Hq"] + c["Hkv"], :], x[..., c["Hq"] + c["Hkv"]:, :]


def _run_own(s):
    import paged_kv_attention_pa_gb300 as pa
    c = s["case"]
    kc, vc = s["k_cache"], s["v_cache"]
    if c["op"] == "decode":
        return pa.decode(s["q"], kc, vc, s["tables"], s["lens"], c["D"] ** -0.5,
                         max_seq_len=s["max_len"], window=c["window"], total_tokens=s["total"])
    out = {}
    if c["op"] != "gather":
        q, k, v = _split(s)
        rope = pa.Rope(s["turns"], interleaved=c["interleaved"], amplitude=s["amplitude"])
        out["q"] = pa.append(k, v, kc, vc, s["tables"], s["lens"], q=q, starts=s["starts"],
                             rope=rope, k_scale=s["scale"], v_scale=s["scale"])
        if c["op"] == "append":
            out["k_cache"], out["v_cache"] = kc, vc
    if c["op"] != "append":
        rows = s["T"] if s["starts"] is not None else c["rows"]
        out["k"], out["v"] = pa.gather(kc, vc, s["tables"], s["lens"], rows, starts=s["starts"],
                                       dtype=DTYPES[c["dtype"]], k_scale=s["scale"],
                                       v_scale=s["scale"])
    return out


def _places(s):
    """Position, physical block and slot of every row of the call."""
    c = s["case"]
    r = torch.arange(s["T"], device=DEVICE)
    if s["starts"] is None:
        b = torch.div(r, c["rows"], rounding_mode="floor")
        pos = s["lens"][b].long() - c["rows"] + r % c["rows"]
    else:
        st = s["starts"].long()
        b = (r[:, None] >= st[None, 1:]).sum(1)
        pos = s["lens"][b].long() - (st[b + 1] - r)
    blk = torch.div(pos, c["bs"], rounding_mode="floor")
    return pos, s["tables"][b, blk].long(), pos - blk * c["bs"]


def _run_plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "decode":
        return _decode_plain(s)
    pos, phys, slot = _places(s)
    out, lead = {}, (s["T"],) if s["starts"] is not None else (c["B"], c["rows"])
    if c["op"] != "gather":
        q, k, v = (x.reshape(s["T"], -1, c["D"]).float() for x in _split(s))
        angle = pos.double()[:, None] * s["freq"][None, :]
        cos = (angle.cos() * s["amplitude"]).float()[:, None, :]
        sin = (angle.sin() * s["amplitude"]).float()[:, None, :]
        out["q"] = _rotate(q, cos, sin, c["interleaved"]).to(dt).view(*lead, c["Hq"], c["D"])
        k = _rotate(k, cos, sin, c["interleaved"])
        for cache, x in ((s["k_cache"], k), (s["v_cache"], v)):
            if c["cache"] == "fp8":
                codes = (x / s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
                cache.view(torch.uint8)[phys, slot] = codes.view(torch.uint8)
            elif c["cache"] == "int4":
                cache[phys, :, slot] = _pack(x)
            else:
                cache[phys, slot] = x.to(dt)
        if c["op"] == "append":
            out["k_cache"], out["v_cache"] = s["k_cache"], s["v_cache"]
    if c["op"] != "append":
        for name in ("k", "v"):
            cache = s[name + "_cache"]
            if c["cache"] == "fp8":
                x = cache.view(torch.uint8)[phys, slot].view(torch.float8_e4m3fn).float() * s["scale"]
            elif c["cache"] == "int4":
                x = _unpack(cache[phys, :, slot])
            else:
                x = cache[phys, slot]
            out[name] = x.to(dt).view(*lead, c["Hkv"], c["D"])
    return out


def _rotate(x, cos, sin, interleaved):
    n = cos.shape[-1]
    y = x.clone()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _half(x, up):
    """fp32 x rounded up (down) to an fp16 value, within fp16's range; as fp16."""
    h = x.clamp(-65504.0, 65504.0).half()
    off = (h.float() < x) if up else (h.float() > x)
    away = (h > 0) | ((h == 0) & (x > 0)) if up else (h <= 0)  # one more unit of magnitude
    bits = h.view(torch.int16)
    return torch.where(off & (h.abs() < 65504), torch.where(away, bits + 1, bits - 1), bits).view(torch.float16)


def _pack(x):
    """[rows, H, D] fp32 -> [rows, H, bytes]: codes, fp16 steps, fp16 minima."""
    T, H, D = x.shape
    G = D // GROUP
    x = x.reshape(T, H, G, GROUP)
    low16 = _half(x.amin(-1, keepdim=True), up=False)
    low = low16.float()
    span = x.amax(-1, keepdim=True) - low
    # (divided by a tensor: a Python number would be turned into a multiplication)
    step16 = _half(span / torch.full_like(span, 15.0), up=True)
    step = step16.float()
    n = torch.where(step > 0, (x - low) / step, torch.zeros_like(x)).round().clamp(0, 15)
    n = n.to(torch.uint8)
    n = n.view(T, H, G, 4, 4, 2).transpose(2, 3)          # octets of eight codes, groups inside
    codes = (n[..., 0] | (n[..., 1] << 4)).reshape(T, H, D // 2)
    as_bytes = lambda t: t.view(T, H, G).view(torch.uint8)
    return torch.cat([codes, as_bytes(step16), as_bytes(low16)], dim=-1)


def _unpack(rows):
    """[..., bytes] -> [..., D] fp32."""
    D = rows.shape[-1] * 8 // 5
    G, lead = D // GROUP, rows.shape[:-1]
    code = rows[..., :D // 2].reshape(*lead, 4, G, 4)
    n = torch.stack([code & 15, code >> 4], dim=-1).transpose(-4, -3).reshape(*lead, G, GROUP)
    step, low = (rows[..., a:a + 2 * G].contiguous().view(torch.float16).float().unsqueeze(-1)
                 for a in (D // 2, D // 2 + 2 * G))
    return (n.float() * step + low).reshape(*lead, D)


def _decode_plain(s):
    c = s["case"]
    B, Hkv, D, R = c["B"], c["Hkv"], c["D"], c["rows"]
    G = c["Hq"] // Hkv
    t = torch.arange(s["max_len"], device=DEVICE)
    blk = torch.div(t, c["bs"], rounding_mode="floor")
    phys, slot = s["tables"][:, blk].long().clamp(min=0), (t - blk * c["bs"]).expand(B, -1)
    live = t[None, :] < s["lens"][:, None]                                   # [B, L]
    q = s["q"].float().view(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    k = _unpack(s["k_cache"][phys, :, slot]).permute(0, 2, 3, 1)                # [B, Hkv, D, L]
    score = torch.matmul(q, k) * D ** -0.5
    del k
    last = s["lens"][:, None] - R + torch.arange(R, device=DEVICE)[None, :]  # [B, R]
    seen = t[None, None, :] <= last[:, :, None]
    if c["window"]:
        seen &= t[None, None, :] >= (s["lens"][:, None, None] - c["window"])
    seen = seen[:, None, :, None, :].expand(B, Hkv, R, G, -1).reshape(B, Hkv, R * G, -1)
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    p = torch.where(seen, (score - score.amax(-1, keepdim=True)).exp(), torch.zeros_like(score))
    v = _unpack(s["v_cache"][phys, :, slot])
    v = torch.where(live[:, :, None, None], v, torch.zeros_like(v)).transpose(1, 2)
    den = p.sum(-1, keepdim=True)  # 0 for a row that sees no token: its output is zero
    out = torch.matmul(p, v) / torch.where(den > 0, den, torch.ones_like(den))
    out = out.view(B, Hkv, R, G, D).permute(0, 2, 1, 3, 4).reshape(s["q"].shape)
    return out.to(DTYPES[c["dtype"]])


# ---------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lengths(case)
    if case["op"] == "decode":
        return _exact_decode(s, lens)
    B, bs, D, Hq, Hkv = case["B"], case["bs"], case["D"], case["Hq"], case["Hkv"]
    tables = s["tables"].long()
    place, pos = [], []
    for b in range(B):
        p = torch.arange(lens[b] - new[b], lens[b], device=DEVICE)
        pos.append(p)
        place.append(tables[b, p // bs] * bs + p % bs)
    pos, place = torch.cat(pos), torch.cat(place)
    flat = {n: _by_token(s, n) for n in ("k", "v")}
    out, lead = {}, (s["T"],) if case["ragged"] else (B, case["rows"])
    if case["op"] != "gather":
        x = s["qkv"].double().view(s["T"], Hq + 2 * Hkv, D)
        turn = torch.polar(torch.full_like(s["freq"], s["amplitude"]).expand(s["T"], -1),
                           pos.double()[:, None] * s["freq"])[:, None, :]
        n = case["rot"] // 2
        head = x[:, :Hq + Hkv, :2 * n]
        pairs = head.reshape(*head.shape[:2], n, 2) if case["interleaved"] else \
            head.reshape(*head.shape[:2], 2, n).transpose(-1, -2)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        pairs = pairs if case["interleaved"] else pairs.transpose(-1, -2)
        x = torch.cat([torch.cat([pairs.reshape(head.shape), x[:, :Hq + Hkv, 2 * n:]], -1),
                       x[:, Hq + Hkv:]], 1)
        out["q"] = x[:, :Hq].reshape(*lead, Hq, D)
        written = {"k": x[:, Hq:Hq + Hkv], "v": x[:, Hq + Hkv:]}
        if case["op"] == "append":
            for name, y in written.items():
                c = flat[name].double()
                c[place] = y / s["scale"]
                out[name + "_cache"] = c.view(s[name + "_cache"].shape)
        else:
            for name, y in written.items():
                out[name] = _exact_4bit(y).reshape(*lead, Hkv, D)
    else:
        for name in ("k", "v"):
            rows = flat[name].view(torch.uint8)[place] if case["cache"] == "fp8" else flat[name][place]
            if case["cache"] == "fp8":
                rows = rows.view(torch.float8_e4m3fn).double() * s["scale"]
            elif case["cache"] == "int4":
                rows = _exact_values(rows)
            out[name] = rows.double().reshape(*lead, Hkv, D)
    return out


def _by_token(s, name):
    """The cache as [slots, Hkv, row]; the pages of a 4-bit cache hold head after head."""
    c = s[name + "_cache"]
    c = c.transpose(1, 2) if s["case"]["cache"] == "int4" else c
    return c.reshape(-1, *c.shape[2:])


def _exact_4bit(x):
    """The values a 4-bit cache holds for x [rows, H, D]: per group of 32, the minimum rounded
    down and a fifteenth of the range rounded up (to eleven significant bits, no finer than
    2^-24), and the nearest of the sixteen values between."""
    g = x.unflatten(-1, (-1, GROUP))
    def eleven_bits(x, towards):
        m = torch.frexp(x)[0]
        power = torch.where(m != 0, x / m, torch.zeros_like(x))  # of two, exactly
        unit = (power / torch.full_like(x, 2048)).clamp(min=2.0 ** -24)
        return towards(x / unit) * unit
    low = eleven_bits(g.amin(-1, keepdim=True), torch.floor)
    span = g.amax(-1, keepdim=True) - low
    step = eleven_bits(span / torch.full_like(span, 15), torch.ceil)
    n = torch.where(step > 0, (g - low) / step, torch.zeros_like(g)).round().clamp(0, 15)
    return (low + n * step).flatten(-2)


def _exact_values(rows):
    """Element d of a row, by its place: 32-bit word (d % 32 // 8) * G + d // 32, bits 4 (d % 8)."""
    D = rows.shape[-1] * 8 // 5
    G = D // GROUP
    d = torch.arange(D, device=rows.device)
    at = 4 * ((d % 32) // 8 * G + d // 32) + (d % 8) // 2
    n = (rows[..., at].int() >> (4 * (d % 2)).int()) & 15
    def half(first):  # sign, 5-bit exponent, 10-bit fraction
        i = first + 2 * (d // 32)
        bits = rows[..., i].int() | (rows[..., i + 1].int() << 8)
        e, f = (bits >> 10) & 31, (bits & 1023).double()
        power = torch.tensor([2.0 ** (max(i, 1) - 25) for i in range(32)], dtype=torch.float64,
                             device=rows.device)[e.long()]
        v = torch.where(e > 0, f + 1024, f) * power
        return torch.where(bits >= 32768, -v, v)
    return n.double() * half(D // 2) + half(D // 2 + 2 * G)


def _exact_decode(s, lens):
    c = s["case"]
    B, R, Hkv, D, bs = c["B"], c["rows"], c["Hkv"], c["D"], c["bs"]
    G = c["Hq"] // Hkv
    out = torch.zeros((B, R, Hkv, G, D), dtype=torch.float64, device=DEVICE)
    q = s["q"].double().view(B, R, Hkv, G, D)
    kf, vf = _by_token(s, "k"), _by_token(s, "v")
    for b, L in enumerate(lens):
        t = torch.arange(L, device=DEVICE)
        place = s["tables"][b, t // bs].long() * bs + t % bs
        k, v = _exact_values(kf[place]), _exact_values(vf[place])
        for i in range(R):
            hi = L - R + i + 1
            lo = max(0, L - c["window"]) if c["window"] else 0
            if hi <= lo:
                continue
            w = torch.softmax(torch.einsum("hgd,lhd->hgl", q[b, i], k[lo:hi]) / math.sqrt(D), -1)
            out[b, i] = torch.einsum("hgl,lhd->hgd", w, v[lo:hi])
    return out.reshape(s["q"].shape)
