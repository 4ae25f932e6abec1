"""GPU tests of the operators between the projections at the limits of what they take: infinities beside finite
values, heads of very different size, weights far below the largest, values on a rounding border, strides beyond
31 bits, streams of the caller's."""
import math

import numpy as np
import pytest
import torch

from test_gpu_decode_ops import (BF16, E, E4M3, F16, U, attention_expect, build, check_attention, f64, i32, make_cache,
                                 normal, w4, within)  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ paged_attention: strides
@pytest.mark.parametrize("page,stride", [(16, 2**29), (4, 2**31 - 16)])
@pytest.mark.parametrize("window", [0, 21])
def test_attention_token_strides_beyond_32_bits(w4, page, stride, window):
    # Tokens outermost: those of a page `stride` elements apart, so that a page's last one begins beyond 2^32 elements.
    # The window begins inside a group of 16 tokens.
    pages, kv, D = 20, 2, 16
    flat = torch.empty((page - 1) * stride + 2 * pages * kv * D, dtype=torch.uint8, device="cuda").view(E4M3)
    pools = [flat[x * pages * kv * D:].as_strided((pages, page, kv, D), (kv * D, stride, D, 1)) for x in (0, 1)]
    for seed, pool in enumerate(pools):
        new = normal((pages, page, kv, D), F16, seed, 40.0).to(E4M3)
        for t in range(page):
            pool[:, t].copy_(new[:, t])
    scales = [torch.full((kv,), 0.02, device="cuda") for _ in (0, 1)]
    lens = [8 * page - 3, 37, 1] if page == 16 else [17 * page - 3, 38, 1]
    width = -(-lens[0] // page)
    table = np.random.default_rng(page).permutation(pages * 3).reshape(3, -1)[:, :width] % pages
    q = normal((3, 4, D), F16, 7, 2.5)
    cache = w4.KVCache(*pools, *scales)
    assert cache.k_token == cache.v_token == stride
    check_attention(w4, q, cache, pools, scales, table, lens, page, window=window)
    del flat, pools, cache
    torch.cuda.empty_cache()
