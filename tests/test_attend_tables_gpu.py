"""Tables of sequences whose context ends within the prefix of their group (GB300 only): no entry of theirs
is used, and so none has to name a block."""
import pytest

import attend_harness as ah
from test_decode_shared_gpu import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [16, 64, 784, 33])
@pytest.mark.parametrize("D,cache", [(128, "same"), (256, "same"), (128, "fp8")])
@pytest.mark.parametrize("R", [1, 3])
def test_sequences_that_end_with_the_prefix(cuda_lib, bs, D, cache, R):
    # a prefix that ends inside a block; members that end with it, in its last block, and before that
    P = 1000
    lens = [P, P, P - 3, P // bs * bs + 1, 300, 0, P + 40]
    pool = ah.Pool(lens, 2, D, bs, "bf16", cache, seed=bs, prefixes=[(0, 7, P)], own_prefix=False)
    pool.bt[1:6] = -7
    q = ah.queries((7, R, 8, D), "bf16", R)
    run(cuda_lib, pool, q if R > 1 else q[:, 0], [0, 7], [P], max_seq_len=P + 40)
