"""Shared prefixes of so many groups that the table in which the kernel keeps them fills the memory
that tiles of K and V are copied into afterwards (GB300 only)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [8192, 4097])
@pytest.mark.parametrize("D", [128, 256])
def test_tables_that_the_tiles_are_copied_over(cuda_lib, groups, D):
    # groups of two sequences, each sharing a block, by tensor copies; the same batch through decode()
    B, nb, most = 2 * groups, 3000, 44
    gen = torch.Generator(device="cuda").manual_seed(groups + D)
    kc, vc = (torch.randn((nb, 16, 1, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    bt = torch.randint(0, nb, (B, 3), generator=gen, device="cuda").to(torch.int32)
    bt[1::2, 0] = bt[0::2, 0]
    sl = torch.randint(17, most + 1, (B,), generator=gen, device="cuda").to(torch.int32)
    q = torch.randn((B, 2, D), generator=gen, device="cuda").bfloat16()
    bounds = torch.arange(0, B + 1, 2, device="cuda").to(torch.int32)
    prefix = torch.full((groups,), 16, dtype=torch.int32, device="cuda")
    want = cuda_lib.decode(q, kc, vc, bt, sl, 0.09, max_seq_len=most, deterministic=True).float()
    # Two results, each off by half a step of its output and of every weight (2^-8 of bf16), the latter of
    # sum_t w_t |v_t|, which a call over |V| gives. 15% for what is small against that: that call's own error
    # (0.8%), second orders (0.8%), and a score's (D + 3) 2^-24 scale log2(e) sum_d |q_d k_d|, at D = 256 and sums
    # of 200 4e-4 of a weight in each result (10%).
    mag = cuda_lib.decode(q, kc, vc.abs(), bt, sl, 0.09, max_seq_len=most, deterministic=True).float()
    near = 1.15 * 2 * 2.0 ** -8 * (want.abs() + mag)
    first = None
    for _ in range(8):
        got = cuda_lib.decode_shared(q, kc, vc, bt, sl, 0.09, bounds, prefix, max_seq_len=most)
        first = got if first is None else first
        assert torch.equal(got, first)
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace()) == 0
    assert torch.all((first.float() - want).abs() <= near)
