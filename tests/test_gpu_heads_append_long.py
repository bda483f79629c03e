"""kvpub_heads_append of more bytes than half of the L2s: codes stored past them."""
import numpy as np
import pytest

import heads_util as U
from test_gpu_heads_append import append, check, new_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("G,D,replicas,n", [(8, 128, 2, [2100, 1, 1999, 70]), (8, 64, 4, [4099, 64]), (4, 256, 3, [2000, 800])])
def test_stored_past_the_l2s(G, D, replicas, n, kind):
    assert sum(n) * G * D * 2 * replicas > 16 << 20
    ctx = U.Context()
    try:
        lens = [k + [100, 0, 37, 63][b] for b, k in enumerate(n)]
        cache = U.HeadsCache(sum(-(-x // 64) for x in lens) + 1, G, D, replicas, pad=16)
        seqs = U.Seqs(lens, n, cache.pages)
        kv, rot = new_rows(seqs.T, G, D, kind), U.Rotation(D // 2, 8, True, 1.1)
        before = [b.clone() for b in cache.bufs]
        append(ctx, cache, kv, seqs, kind, rot)
        assert check(cache, before, kv, seqs, rot) == 0 and ctx.invalid() == 0
    finally:
        ctx.free()
