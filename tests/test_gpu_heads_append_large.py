"""kvpub_heads_append where one launch cannot hold the call's blocks."""
import numpy as np
import pytest

import heads_util as U
from test_gpu_heads_append import append, check, new_rows

pytestmark = pytest.mark.gpu


def test_more_blocks_of_threads_than_a_launch_holds():
    """16,400 sequences, of which three have new tokens: places for 32,801 blocks of positions, 128 heads each, are
    4,198,528 blocks of 1024 threads, beyond 2^32 of them."""
    B, G, D = 16400, 128, 256
    ctx = U.Context()
    try:
        n, lens = np.zeros(B, np.int64), np.zeros(B, np.int64)
        for b, tokens, kv in ((0, 5, 5), (B // 2, 66, 70), (B - 1, 6, 9)):
            n[b], lens[b] = tokens, kv
        assert (n.sum() // 64 + 2 * B) * G * 1024 > 2 ** 32
        cache = U.HeadsCache(4, G, D, 1)
        seqs = U.Seqs(lens, n, cache.pages)
        kv = new_rows(seqs.T, G, D, "bf16")
        before = [b.clone() for b in cache.bufs]
        append(ctx, cache, kv, seqs, "bf16")
        assert check(cache, before, kv, seqs) == 0 and ctx.invalid() == 0
    finally:
        ctx.free()
