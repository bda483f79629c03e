"""kvpub_heads_attend over values as large as the header allows, and over the least that the cache holds."""
import pytest
import torch

import heads_util as U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 9])
@pytest.mark.parametrize("kv,byte", [(700, 206), (20000, 206), (700, 1), (60, 2), (3000, 3)])
def test_the_ends_of_the_scales(kv, byte, n):
    """448 * 2^79 stays below 2^88.  At the other end a value is a multiple of 2^-135 and bf16 holds multiples of 2^-133:
    half a step, 2^-134, for the values, as much for the output, and 2^-149 for each of the sums."""
    ctx = U.Context()
    try:
        cache = U.HeadsCache(-(-kv // 64), 2, 64, replicas=1)
        cache.scales(0)[:, :, 1] = byte
        seqs = U.Seqs([kv], [n], cache.pages)
        for mag in (1.0, 0.0):                                   # mag 0: equal scores, every weight 1
            q = U.Query(n, 16, 64, mag=mag)
            U.attend(ctx, cache, q, seqs)
            vals, _ = cache.values(0, seqs.table[0], kv)
            assert vals[1].abs().max().item() < 2.0 ** 88
            o, l, size, mass = U.reference(q.q, vals, torch.as_tensor(seqs.seen(0), device="cuda"), q.scale)
            score = ((64 + 24) * 2.0 ** -24 * size + 2.0 ** -20 * (1 + l.abs()))[..., None]
            tol = U.half_step(q.dtype) * o.abs() + (2.0 ** -8 + 2 * score) * mass * 1.01 + 2.0 ** -133 + kv * 2.0 ** -149
            worst = ((q.out.double() - o).abs() / tol).max().item()
            assert worst <= 1, f"off by {worst} of its bound"
    finally:
        ctx.free()
