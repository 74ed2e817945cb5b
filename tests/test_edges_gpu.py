"""Calls at the edges of what append, gather and decode take (GB300 only)."""
import numpy as np
import pytest
import torch

import rows_harness as rh

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
