"""Tokens before the first sequence, behind the last one and between bounds: neither stored nor attended, and their outputs
keep what they held."""
import numpy as np
import pytest
import torch

import heads_util as U
from test_gpu_heads_append import append, check, new_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before,behind", [(0, 5), (70, 0), (3, 200)])
@pytest.mark.parametrize("n", [[1, 1, 1], [40, 0, 9], [130, 64, 1]])
def test_tokens_of_no_sequence(n, before, behind):
    G, H, D = 2, 16, 128
    ctx = U.Context()
    try:
        lens = [k + 50 for k in n]
        cache = U.HeadsCache(sum(-(-x // 64) for x in lens) + 1, G, D, replicas=2)
        # the loose tokens are those of two sequences that the call is not told of
        all_ = U.Seqs([0] + lens + [0], [before] + n + [behind], cache.pages, max_q=max(n), table=None)
        told = U.Seqs(lens, n, cache.pages, table=all_.table[1:-1])
        told.start = all_.start[1:-1]
        told.d_start, told.T = U.i32(told.start), all_.T
        told.struct.q_start = told.d_start.data_ptr()
        kv = new_rows(told.T, G, D, "bf16")
        held = [b.clone() for b in cache.bufs]
        append(ctx, cache, kv, told, "bf16")
        assert check(cache, held, kv, told) == 0 and ctx.invalid() == 0
        q = U.Query(told.T, H, D)
        U.attend(ctx, cache, q, told)
        U.check_all(cache, q, told)              # and that every other row holds its sentinels
    finally:
        ctx.free()
