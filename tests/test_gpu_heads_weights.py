"""kvpub_heads_attend where the softmax weights are the sum of two bf16: calls of at most 16 rows a sequence and key-value
head, and fp16."""
import pytest
import torch

import heads_util as U
from weights_bound import bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,H,lens,n", [(2, 32, [60, 8], [1, 1]), (2, 16, [700, 33], [2, 1]), (1, 4, [5000, 130], [4, 3]), (4, 12, [20, 300], [5, 5]),
                                        (1, 16, [20000], [1])])
def test_outputs_are_as_near_as_two_parts_leave_them(G, H, lens, n, D):
    assert max(n) * H // G <= 16
    ctx = U.Context()
    try:
        cache = U.HeadsCache(sum(-(-x // 64) for x in lens), G, D, replicas=1)
        seqs = U.Seqs(lens, n, cache.pages)
        q = U.Query(seqs.T, H, D)
        U.attend(ctx, cache, q, seqs)
        for b, kv in enumerate(lens):
            a, z = int(seqs.start[b]), int(seqs.start[b + 1])
            vals, _ = cache.values(0, seqs.table[b, :-(-kv // 64)], kv)
            o, l, size, mass = U.reference(q.q[a:z], vals, torch.as_tensor(seqs.seen(b), device="cuda"), q.scale)
            # a score: D + 24 roundings of the sum of its terms' magnitudes; the sums' own within 2^-20
            score = ((D + 24) * 2.0 ** -24 * size + 2.0 ** -20 * (1 + l.abs()))[..., None]
            worst = ((q.out[a:z].double() - o).abs() / bound(o, mass, score, U.half_step(q.dtype))).max().item()
            assert worst <= 1, f"sequence {b}: off by {worst} of its bound"
    finally:
        ctx.free()
