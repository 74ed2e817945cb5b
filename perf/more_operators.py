"""Cases of attention by many query rows over one paged context: cross attention to an
encoder's states of another length, and decode for batches whose sequences share a prefix.

`run` computes an operator either in its plain form (elementary torch operations, fp32) or,
with `own` set, through the framework's public calls. `exact` gives the same outputs from the
definitions in 64 bits.

Shapes follow the repository's own workloads: 8/8, 32/8 and 32/16 heads with head_dim 128 and
16-token blocks, and the hybrid layer's 24/4 heads with head_dim 256 and 784-token blocks.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
MOST = 2 ** 39                     # flops of a drawn case


# ------------------------------------------------------------------------------- cases
# cross:  B sequences with `rows` query rows each (or `packed` rows in all, shared out
#         unevenly) over contexts of lo..hi states
# shared: B sequences in `groups` groups, each with a shared prefix of plo..phi tokens and
#         lo..hi tokens of its own, `rows` causal query rows per sequence
def listed():
    common = dict(cache="same", rows=1, packed=0, groups=0, plo=0, phi=0)
    cases = [
        # one step of one user over the states of a short recording: latency only
        dict(name="cross 1 row", op="cross", dtype="bf16", B=1, Hq=8, Hkv=8, D=128, bs=16,
             lo=1500, hi=1500),
        # a step of beam search, five beams of every recording over its states
        dict(name="cross beams", op="cross", dtype="f16", B=16, Hq=32, Hkv=8, D=128, bs=16,
             lo=200, hi=1500, rows=5),
        # decoder prompts of odd lengths packed together, each over its own source
        dict(name="cross packed prompts", op="cross", dtype="bf16", B=6, Hq=32, Hkv=8, D=128,
             bs=16, lo=700, hi=4097, packed=2047),
        # a long prompt over a long source, 32/16 heads
        dict(name="cross 4K over 8K", op="cross", dtype="bf16", B=1, Hq=32, Hkv=16, D=128,
             bs=16, lo=8192, hi=8192, rows=4096),
        # a chunk of a prompt over a source held in the hybrid layer's cache
        dict(name="cross hybrid chunk", op="cross", dtype="bf16", B=2, Hq=24, Hkv=4, D=256,
             bs=784, lo=3000, hi=6500, rows=500),
        # the same step as the beams', the source's states held in fp8, blocks of 33 tokens
        dict(name="cross rows fp8", op="cross", dtype="f16", cache="fp8", B=24, Hq=32, Hkv=16,
             D=128, bs=33, lo=1000, hi=6000, rows=7),
        # four answers to one short prompt
        dict(name="shared 4 answers", op="shared", dtype="bf16", B=4, Hq=8, Hkv=8, D=128, bs=16,
             lo=1, hi=64, groups=1, plo=512, phi=512),
        # a serving batch behind one system prompt
        dict(name="shared 64 users", op="shared", dtype="bf16", B=64, Hq=32, Hkv=8, D=128, bs=16,
             lo=128, hi=2048, groups=1, plo=8192, phi=8192),
        # several groups, prefixes that end inside a block, some sequences alone
        dict(name="shared groups", op="shared", dtype="f16", B=48, Hq=32, Hkv=16, D=128, bs=16,
             lo=1, hi=3000, groups=5, plo=700, phi=9000),
        # many questions about one long document held in fp8
        dict(name="shared document fp8", op="shared", dtype="bf16", cache="fp8", B=128, Hq=32,
             Hkv=8, D=128, bs=16, lo=16, hi=700, groups=1, plo=32768, phi=32768),
        # the hybrid layer's decode step behind a shared prefix
        dict(name="shared hybrid", op="shared", dtype="bf16", B=16, Hq=24, Hkv=4, D=256, bs=784,
             lo=100, hi=4000, groups=2, plo=16000, phi=16000),
        # speculative decode: four new rows of every sequence
        dict(name="shared rows", op="shared", dtype="f16", B=32, Hq=32, Hkv=8, D=128, bs=16,
             lo=4, hi=1000, groups=2, plo=4095, phi=4095, rows=4),
    ]
    return [{**common, **c} for c in cases]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross", "shared"])
    D, bs = rng.choice([(128, 16), (128, 16), (128, 64), (128, 33), (256, 784), (256, 16)])
    Hkv = rng.choice([4, 8, 16] if D == 128 else [2, 4])
    G = rng.choice([1, 2, 3, 4, 6, 8])
    B = _log(rng, 1, 128 if op == "shared" else 32)
    case = dict(op=op, dtype=rng.choice(["bf16", "f16"]), B=B, Hq=G * Hkv, Hkv=Hkv, D=D, bs=bs,
                cache=rng.choice(["same", "same", "fp8"]), rows=1, packed=0, groups=0, plo=0, phi=0)
    room = 150_000_000 // (Hkv * D)    # tokens of the caches
    if op == "cross":
        hi = _log(rng, 16, min(16384, max(16, room // B)))
        lo = max(1, int(hi * rng.choice([0.05, 0.5, 1.0])))
        most = max(1, min(16384, MOST // (4 * hi * G * Hkv * D)))   # query rows in all
        if rng.random() < 0.4:
            case["packed"] = max(B, _log(rng, 1, most))
        else:
            case["rows"] = max(1, min(_log(rng, 1, 4096), most // B))
        return dict(case, lo=lo, hi=hi)
    groups = min(B, rng.choice([1, 1, 2, 5]))
    rows = rng.choice([1, 1, 1, 2, 4]) if G <= 4 else 1
    phi = _log(rng, 16, min(32768, room // (2 * groups), MOST // (8 * B * rows * G * Hkv * D)))
    hi = max(rows, _log(rng, 4, min(4096, max(4, room // (2 * B)))))
    return dict(case, rows=rows, groups=groups, plo=int(phi * rng.choice([0.1, 1.0])), phi=phi,
                lo=max(rows, int(hi * rng.choice([0.01, 0.5, 1.0]))), hi=hi)


def _cut(total, parts, g):
    """`total` shared out unevenly: [0, ..., total], ascending, parts + 1 numbers."""
    share = torch.rand(parts, generator=g) + 0.2
    at = (torch.cumsum(share, 0) / share.sum() * total).round().long().tolist()
    return [0] + at[:-1] + [total]


def _layout(case):
    """What the host knows, fixed by the case: context lengths, query rows per sequence, and for
    shared prefixes the groups' first sequences (the last sequence or two belong to none when
    there are several groups) and prefixes."""
    B = case["B"]
    g = torch.Generator().manual_seed(B + case["hi"])
    draw_in = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=g).tolist()
    own_len = draw_in(case["lo"], case["hi"], B)
    if case["op"] == "cross":
        if case["packed"]:
            cut = _cut(case["packed"], B, g)
            return own_len, [b - a for a, b in zip(cut, cut[1:])], None, None
        return own_len, [case["rows"]] * B, None, None
    N = case["groups"]
    grouped = B - 2 if N > 1 and B - 2 >= N else B
    groups = _cut(grouped, N, g)
    prefix = draw_in(case["plo"], case["phi"], N)
    lens = list(own_len)
    for n in range(N):
        for b in range(groups[n], groups[n + 1]):
            lens[b] += prefix[n]
    return lens, [case["rows"]] * B, groups, prefix


def _row_bytes(case):
    return case["D"] * (1 if case["cache"] == "fp8" else 2)


def work(case):
    lens, rows, groups, prefix = _layout(case)
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    seen = sum(L * n for L, n in zip(lens, rows))
    held = sum(lens)                       # tokens in the caches, a shared one once
    if groups is not None:
        seen -= len(lens) * sum(range(case["rows"]))      # causal among the new rows
        held -= sum(p * max(0, b - a - 1) for p, a, b in zip(prefix, groups, groups[1:]))
    nbytes = held * 2 * Hkv * _row_bytes(case) + 4 * sum(rows) * Hq * D + 4 * (held // bs) + 8 * len(lens)
    return {"bytes": nbytes, "flops": 4 * seen * Hq * D}


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    lens, rows, groups, prefix = _layout(case)
    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device=DEVICE)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEVICE)

    # blocks handed out at random from a pool; the whole blocks of a shared prefix are held
    # once, and a block that it ends in is copied for every sequence of the group
    kept = [0] * B                          # leading blocks of b that its group's first holds
    first = list(range(B))
    for n in range(len(prefix or [])):
        for b in range(groups[n] + 1, groups[n + 1]):
            kept[b], first[b] = prefix[n] // bs, groups[n]
    blocks = [-(-L // bs) for L in lens]
    pool = sum(blocks) - sum(kept)
    pool += pool // 8 + 1
    perm = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((B, max(blocks)), -1, dtype=torch.int32)
    at, copies = 0, []
    for b in range(B):
        n = blocks[b] - kept[b]
        table[b, :kept[b]] = table[first[b], :kept[b]]
        table[b, kept[b]:blocks[b]] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    s = dict(case=case, max_len=max(lens), tables=table.to(DEVICE), lens=i32(lens), starts=None,
             longest=lens, counts=rows)
    s["scale"] = 5.0 / 448.0 if case["cache"] == "fp8" else 1.0   # fp8: values up to 5 sigma
    for name in ("k_cache", "v_cache"):
        c = randn(pool, bs, Hkv, D)
        c = (c / s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn) if case["cache"] == "fp8" else c.to(dt)
        raw = c.view(torch.uint8 if case["cache"] == "fp8" else torch.int16)
        for n in range(len(prefix or [])):
            tail = prefix[n] % bs
            later = table[groups[n] + 1:groups[n + 1], prefix[n] // bs] if tail else []
            if len(later):
                raw[later.long().to(DEVICE), :tail] = raw[int(table[groups[n], prefix[n] // bs]), :tail].clone()
        s[name] = c
    lead = (sum(rows),) if case["packed"] else (B,) if case["rows"] == 1 else (B, case["rows"])
    s["q"] = randn(*lead, Hq, D).to(dt)
    if case["packed"]:
        s["starts"] = i32([sum(rows[:b]) for b in range(B + 1)])
    if groups is not None:
        s["groups"], s["prefix"] = i32(groups), i32(prefix)
        s["spans"] = list(zip(groups, groups[1:], prefix))
    return s


# ------------------------------------------------------------------------ one pass
def run(s):
    if own:
        import paged_kv_attention_pa_gb300 as pa
        c = s["case"]
        args = (s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], c["D"] ** -0.5)
        rest = dict(max_seq_len=s["max_len"], k_scale=s["scale"], v_scale=s["scale"])
        if c["op"] == "cross":
            return pa.cross(*args, starts=s["starts"], **rest)
        return pa.decode_shared(*args, s["groups"], s["prefix"], **rest)
    return _cross_plain(s) if s["case"]["op"] == "cross" else _shared_plain(s)


def _cached(s, name, tables, lo, hi):
    """Tokens [lo, hi) of the sequences of `tables` [n, blocks], as [n, Hkv, tokens, D] fp32;
    what lies in no block is whatever block 0 holds."""
    bs = s["case"]["bs"]
    t = torch.arange(lo, hi, device=DEVICE)
    phys, slot = tables[:, t // bs].long().clamp(min=0), (t % bs).expand(tables.shape[0], -1)
    c = s[name]
    if c.dtype == torch.float8_e4m3fn:
        x = c.view(torch.uint8)[phys, slot].view(torch.float8_e4m3fn).float() * s["scale"]
    else:
        x = c[phys, slot].float()
    return x.transpose(1, 2)


def _softmax(score, seen):
    """Weights over the last axis of the scores where `seen`; zeros for a row that sees nothing."""
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top > -math.inf, top, torch.zeros_like(top))).exp()
    den = p.sum(-1, keepdim=True)
    return p / torch.where(den > 0, den, torch.ones_like(den))


def _cross_plain(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    q = s["q"].float().view(-1, Hkv, G, D)
    out, at = [], 0
    for b, n in enumerate(s["counts"]):
        rows = q[at:at + n].permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
        at += n
        k = _cached(s, "k_cache", s["tables"][b:b + 1], 0, s["longest"][b])[0]
        v = _cached(s, "v_cache", s["tables"][b:b + 1], 0, s["longest"][b])[0]
        score = torch.matmul(rows, k.transpose(-1, -2)) * D ** -0.5
        p = (score - score.amax(-1, keepdim=True)).exp()
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        out.append(o.view(Hkv, G, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D))
    return torch.cat(out).to(DTYPES[c["dtype"]]).view(s["q"].shape)


def _shared_plain(s):
    """Every sequence over its whole context, as a user without the operator computes it: in
    chunks of the batch that keep the gathered cache within a few GB."""
    c = s["case"]
    B, Hq, Hkv, D, R = c["B"], c["Hq"], c["Hkv"], c["D"], c["rows"]
    G, L = Hq // Hkv, s["max_len"]
    q = s["q"].float().view(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    t = torch.arange(L, device=DEVICE)
    limit = s["lens"][:, None] - R + 1 + torch.arange(R, device=DEVICE)[None, :]       # [B, R]
    step = max(1, 2 ** 30 // (L * Hkv * D))
    out = []
    for b in range(0, B, step):
        k = _cached(s, "k_cache", s["tables"][b:b + step], 0, L)
        score = torch.matmul(q[b:b + step], k.transpose(-1, -2)) * D ** -0.5
        del k
        n = score.shape[0]
        seen = t[None, None, :] < limit[b:b + step, :, None]
        seen = seen[:, None, :, None, :].expand(n, Hkv, R, G, L).reshape(n, Hkv, R * G, L)
        v = _cached(s, "v_cache", s["tables"][b:b + step], 0, L)
        v = torch.where((t[None, :] < s["lens"][b:b + step, None])[:, None, :, None], v, torch.zeros_like(v))
        out.append(torch.matmul(_softmax(score, seen), v))
    out = torch.cat(out).view(B, Hkv, R, G, D).permute(0, 2, 1, 3, 4)
    return out.reshape(s["q"].shape).to(DTYPES[c["dtype"]])


# ---------------------------------------------------------------------- 64 bits
def exact(case, seed):
    if work(case)["flops"] > 2 ** 42:
        return None
    s = prepare(case, seed)
    lens, rows, _, _ = _layout(case)
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    G, causal = Hq // Hkv, case["op"] == "shared"
    flat = {}
    for name in ("k_cache", "v_cache"):
        flat[name] = s[name].view(-1, Hkv, D)
    q = s["q"].view(-1, Hq, D).double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEVICE)
    at = 0
    for b, (L, n) in enumerate(zip(lens, rows)):
        t = torch.arange(L, device=DEVICE)
        place = s["tables"][b].long()[torch.div(t, bs, rounding_mode="floor")] * bs + t % bs
        for h in range(Hkv):
            k, v = (_wide(flat[x][:, h], place) * s["scale"] for x in ("k_cache", "v_cache"))
            for r in range(at, at + n, 2048):
                x = q[r:min(r + 2048, at + n), h * G:(h + 1) * G]
                w = torch.einsum("rgd,td->rgt", x, k) / math.sqrt(D)
                if causal:
                    i = torch.arange(r - at, r - at + x.shape[0], device=DEVICE)
                    w.masked_fill_((t[None, :] > L - n + i[:, None])[:, None, :], -math.inf)
                out[r:r + x.shape[0], h * G:(h + 1) * G] = torch.einsum("rgt,td->rgd", torch.softmax(w, -1), v)
        at += n
    return out.view(s["q"].shape)


def _wide(x, place):
    if x.dtype == torch.float8_e4m3fn:
        return x.view(torch.uint8)[place].view(torch.float8_e4m3fn).double()
    return x[place].double()
