"""Attention of many rows at its limits: what lies in shared memory where a call begins, rows of a tile that are nobody's."""
import pytest
import torch

from test_gpu_wide_attention import BF16, F16, Setup, w4  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, F16)])
def test_queries_and_keys_come_where_the_plan_has_been(w4, dim, dtype):  # noqa: F811
    # The plan of many requests lies where the first boxes of queries and keys are brought, in every call.
    n = 3000
    s = Setup(w4, [2] * n, [2 + 11 * i % 40 for i in range(n)], heads=2, kv=1, dim=dim, dtype=dtype, page=16)
    s.prompt()
    s.check(only=range(0, n, 41))
    first = s.out.clone(), s.lse.clone()
    for _ in range(30):
        s.prompt()
        assert torch.equal(s.out, first[0]) and torch.equal(s.lse, first[1])
