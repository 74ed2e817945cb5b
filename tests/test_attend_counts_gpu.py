"""Every token that a row sees counts once, in cross attention and decode behind shared prefixes, however
long the context, wherever it is cut into tiles and pieces (GB300 only).

Queries of zero give equal weights, which no rounding touches: 1 (or a power of two) each, their sum a
whole number below 2^24. With V[t, d] = 1 where a mixture of t is d, else 0, out[d] is how many of the
tokens seen have d, over all seen: whole sums below 2^24, then a quotient and a product in fp32 (2^-23
together), and the output's rounding, half a step. With n tokens about n / D have each d, so that one that is
lost, doubled or seen by the wrong row moves an output by D / n of it, beyond that for n < 2^7 D at least."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32, device="cuda")


def column(t, D):
    """Which d a token has: every D in a row have all of them, in changing order."""
    return (t + (t // D) * 37) % D


class Counting:
    """Caches of B sequences of those lengths, each in blocks of its own but for the whole blocks of its
    group's prefix; V of slots that hold no token is NaN, K too."""

    def __init__(self, lens, Hkv, D, bs, dtype, cache, groups=(), prefix=(), seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.Hkv, self.D, self.dt = lens, Hkv, D, DT[dtype]
        need = [-(-L // bs) for L in lens]
        nb = sum(need) + 2
        perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.bt = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
        store = torch.float8_e4m3fn if cache == "fp8" else self.dt
        raw = torch.uint8 if cache == "fp8" else torch.int16
        self.kc, self.vc = (torch.full((nb, bs, Hkv, D), float("nan"), device="cuda").to(store) for _ in range(2))
        at = 0
        for b, (L, n) in enumerate(zip(lens, need)):
            self.bt[b, :n] = perm[at:at + n]
            at += n
            t = torch.arange(L, device="cuda")
            place = self.bt[b].cuda()[t // bs].long(), t % bs
            k = torch.randn((L, Hkv, D), generator=g, device="cuda")
            v = torch.zeros((L, Hkv, D), device="cuda")
            v[t, :, column(t, D)] = 1.0
            for c, x in ((self.kc, k), (self.vc, v)):
                c.view(raw)[place] = x.to(store).view(raw)
        for a, e, P in zip(groups, groups[1:], prefix):
            for b in range(a + 1, e):
                n = min(P, lens[a]) // bs
                self.bt[b, :n] = self.bt[a, :n]

    def args(self):
        return self.kc, self.vc, self.bt.cuda(), i32(self.lens)

    def expected(self, b, rows, causal):
        """[rows, D]: the share of the tokens that each row sees."""
        L = self.lens[b]
        seen = torch.clamp(L - rows + 1 + torch.arange(rows), min=0) if causal else torch.full((rows,), L)
        t = torch.arange(L)
        counts = torch.zeros((L + 1, self.D), dtype=torch.float64)
        counts[t + 1, column(t, self.D)] = 1.0
        counts = counts.cumsum(0)[seen]
        return counts / seen.clamp(min=1)[:, None]

    def check(self, got, rows, causal):
        assert torch.isfinite(got).all()
        at = 0
        for b, n in enumerate(rows):
            want = self.expected(b, n, causal).cuda()[:, None, :]
            y = got[at:at + n].double()
            off = (y - want).abs() > (HALF_STEP[self.dt] + 2.0 ** -23) * want + 2.0 ** -25 * (want > 0)
            assert not off.any(), f"sequence {b} of {self.lens[b]} tokens: {int(off.sum())} of {off.numel()}"
            at += n


LONG = [9000, 1, 4097, 12801, 0, 6399, 127, 10240, 3333, 8191]


@pytest.mark.parametrize("rows", [1, 3, 20, 75, 300])
@pytest.mark.parametrize("D,cache,bs", [(128, "same", 16), (256, "same", 16), (128, "fp8", 16), (256, "fp8", 16),
                                        (128, "same", 33), (256, "same", 784)])
def test_cross(cuda_lib, rows, D, cache, bs):
    # runs of many tiles of one row tile and two, with pieces that begin and end anywhere
    dtype = "f16" if rows in (3, 75) else "bf16"
    pool = Counting(LONG, 4, D, bs, dtype, cache, seed=rows)
    q = torch.zeros((len(LONG), rows, 16, D), dtype=DT[dtype], device="cuda")
    out = cuda_lib.cross(q, *pool.args(), 0.1)
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace()) == 0
    pool.check(out.view(-1, 16, D), [rows] * len(LONG), False)


@pytest.mark.parametrize("D,cache", [(128, "same"), (256, "same"), (128, "fp8")])
def test_packed(cuda_lib, D, cache):
    counts = [1, 0, 500, 33, 7, 129, 64, 65, 0, 2]
    pool = Counting(LONG, 2, D, 16, "bf16", cache, seed=5)
    q = torch.zeros((sum(counts), 6, D), dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([0] + counts).cumsum(0)
    pool.check(cuda_lib.cross(q, *pool.args(), -0.1, starts=i32(starts)), counts, False)


@pytest.mark.parametrize("R", [1, 4, 33, 300, 1100])
@pytest.mark.parametrize("D,cache,bs", [(128, "same", 16), (256, "same", 16), (128, "fp8", 16), (256, "fp8", 33),
                                        (128, "same", 64)])
def test_decode_shared(cuda_lib, R, D, cache, bs):
    # prompts behind prefixes among them: causal limits that cross many tiles, sequences of fewer tokens than
    # rows, prefixes that end inside tiles, one that reaches into the first sequence's own rows
    lens = [5000, 4100, 6000, 7777, 300, 3000, 1, 0, 9000, 9100, 4000]
    groups, prefix = [0, 3, 3, 4, 8, 10], [4099, 77, 100, 250, 8995]
    pool = Counting(lens, 2, D, bs, "bf16" if R != 33 else "f16", cache, groups, prefix, seed=R)
    q = torch.zeros((len(lens), R, 8, D), dtype=pool.dt, device="cuda")
    out = cuda_lib.decode_shared(q, *pool.args(), 0.1, i32(groups), i32(prefix))
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace()) == 0
    pool.check(out.view(-1, 8, D), [R] * len(lens), True)


def test_many_short_sequences(cuda_lib):
    # 700 sequences of 1 to 300 tokens and 5 rows, groups of 1 to 60
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 300, (700,), generator=g).tolist()
    cuts = sorted(set(torch.randint(0, 701, (30,), generator=g).tolist()))
    prefix = [max(0, min(lens[a:e]) - 1) if e > a else 0 for a, e in zip(cuts, cuts[1:])]
    pool = Counting(lens, 1, 128, 16, "bf16", "same", cuts, prefix, seed=4)
    q = torch.zeros((700, 5, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = cuda_lib.decode_shared(q, *pool.args(), 0.1, i32(cuts), i32(prefix))
    pool.check(out.view(-1, 8, 128), [5] * 700, True)
