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


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, F16)])
@pytest.mark.parametrize("new,pad", [(3, 40), (49, 0)])
def test_rows_that_are_nobody_s_change_nothing(w4, dim, dtype, new, pad):  # noqa: F811
    # 5 heads to a kv head: a box of queries does not fill a tile, and holds rows of other requests and of none behind a
    # request's last one. So many keys that every CTA has several units of them.
    s = Setup(w4, [new, 20], [50000, 300], heads=10, kv=2, dim=dim, dtype=dtype, q_scale=0.4, pad=pad, page=64)
    loud = Setup(w4, [300], [300], heads=8, kv=2, dim=dim, dtype=dtype, q_scale=1.0)
    for x in (loud.q, loud.k, loud.v):
        x.fill_(200.0)
    mine = slice(0, new)
    s.prompt()
    first = s.out[mine].clone(), s.lse[mine].clone()
    for level in (0.0, 1.0, 30.0, -30.0):
        loud.q.fill_(200.0 + level)
        loud.prompt()  # leaves its numbers in shared memory
        s.q[new:] = level * torch.sign(torch.randn(s.q[new:].shape, device="cuda"))
        s.prompt()
        same = torch.equal(s.out[mine], first[0]), torch.equal(s.lse[mine], first[1])
        assert same == (True, True), level
