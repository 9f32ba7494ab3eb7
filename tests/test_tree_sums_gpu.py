"""attn_decode_tree's sums of weighted values: where they would leave fp32, and in rows of many tiles."""
import math

import pytest
import torch

from test_tree_gpu import _lib, call, problem  # noqa: F401 (_lib is a fixture)
from tree_reference import attention, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,d,Hq,T,old", [
    (2, 64, 2, 9, 3000), (2, 64, 8, 20, 3000), (2, 128, 8, 4, 3000), (2, 128, 4, 20, 3000), (2, 128, 4, 60, 3000), (2, 256, 2, 9, 3000), (2, 256, 4, 30, 3000),
    (2, 512, 2, 5, 3000), (2, 512, 1, 60, 3000), (160, 64, 1, 9, 700), (160, 64, 8, 20, 700), (160, 128, 1, 4, 700), (160, 128, 1, 40, 700), (160, 256, 1, 4, 700)])
@pytest.mark.parametrize("least,most", [(1e38, 3.3e38), (1e-20, 3e-20)])
def test_values_of_one_sign(B, d, Hq, T, old, least, most):
    """bf16 values whose sums do not cancel: the result lies within the type, and so has every sum on the way to within fp32."""
    q, store, view, table, lengths, counts, m, seen = problem(B, Hq, 1, T, d, 16, "heads", torch.bfloat16, "own", old, full=True)
    v = view(store)[1]
    v.copy_((torch.rand(v.shape, generator=torch.Generator().manual_seed(9)).double() * (most - least) + least).to(torch.bfloat16))
    got = call(q.cuda(), store.cuda(), view, table, lengths, counts, m)
    check_attention(got, attention(q, *view(store), table, lengths, counts, seen, 1 / math.sqrt(d)), max(lengths), d, "values of one sign", Hq * T)
