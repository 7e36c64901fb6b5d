"""The row bound of the paged attention tests: what it takes and what it refuses."""
import numpy as np
import pytest
import torch

from paged_norm import check_rows
from paged_util import Case

F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("kv,new,d,bits,dtype", [
    ([300, 70], [4, 1], 128, 4, F16), ([40, 60], [30, 16], 64, 2, BF16),
    ([64, 90], [3, 3], 128, 8, BF16), ([500], [2], 64, 2, F16)])
def test_the_bound_refuses_wrong_rows(kv, new, d, bits, dtype):
    c = Case(kv, new, 8, 2, d, bits, 16, dtype)
    exact = torch.from_numpy(c.attention()[0])
    assert check_rows(c, exact.to(dtype)) < 0.5
    shifted = exact.roll(1, 0)      # every row one further
    heads = exact.roll(4, 1)        # the other KV head
    last = exact.clone()
    last[-1, -1] = 0                # a single row of a single head
    for wrong in (exact * 0, exact * 1.05, -exact, exact + exact.abs().mean() / 4, shifted, heads,
                  last):
        with pytest.raises(AssertionError):
            check_rows(c, wrong.to(dtype))


def test_tokens_that_are_left_out_are_not_the_same():
    c = Case([300], [2], 8, 2, 128, 4, 32, F16)
    out = torch.from_numpy(c.attention()[0]).half()
    with pytest.raises(AssertionError):
        check_rows(c, out, gone={0: range(32, 64)})
    c.K[0], c.V[0] = (np.delete(x[0], slice(32, 64), 0) for x in (c.K, c.V))
    c.kv = [268]
    kept = torch.from_numpy(c.attention()[0]).half()
    check_rows(Case([300], [2], 8, 2, 128, 4, 32, F16), kept, gone={0: range(32, 64)})
