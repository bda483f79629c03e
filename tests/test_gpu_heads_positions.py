"""Every token turned by its own position, on its way into the cache and as a query: a prompt in chunks, single tokens and a
drafted tree, value by value against the rotation in 64 bits, and the attention over them against its formula."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import heads_util as U
from positions_bound import key_bound, query_bound
from test_gpu_heads_append import append, new_rows
from test_gpu_heads_together import rotated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("halves,scaling", [(True, kvpub.SCALING_NONE), (False, kvpub.SCALING_RAMP)])
def test_prompt_tokens_tree(halves, scaling):
    G, H, D, B = 2, 8, 128, 3
    ctx, rot = U.Context(), U.Rotation(D, 0, halves, 1.1, scaling=scaling, factor=4.0, original=64.0, low=1.0, high=8.0)
    cache = U.HeadsCache(24, G, D, 2, fill=0)
    table = np.arange(24).reshape(B, 8).astype(np.int32)
    full = [[] for _ in range(B)]                 # rotated keys in 64 bits, their bounds, and the values
    try:
        lens = np.zeros(B, np.int64)
        depth, parents = np.array([0, 1, 1, 2, 2, 3]), [None, 0, 0, 1, 2, 3]
        bits = np.zeros((6, 1), np.uint64)
        for i, p in enumerate(parents):
            bits[i, 0] = (bits[p, 0] if p is not None else 0) | np.uint64(1 << i)
        for step, counts in enumerate([[100, 37, 1], [64, 2, 130], [1, 1, 1], [1, 1, 1], [6, 6, 6]]):
            counts, is_tree = np.array(counts), step == 4
            base = lens.copy()
            lens = lens + counts
            seqs = U.Seqs(lens, counts, 24, max_kv=512, table=table, tree=np.concatenate([bits] * B) if is_tree else None)
            at = np.concatenate([b + (depth if is_tree else np.arange(c)) for b, c in zip(base, counts)])
            pos, kv = U.i32(at), new_rows(seqs.T, G, D, "bf16", seed=step)
            append(ctx, cache, kv, seqs, "bf16", rot, pos if is_tree else None)
            q = U.Query(seqs.T, H, D, seed=step)
            raw = q.q.clone()
            q.q.copy_(rotated(ctx, raw, pos, rot))
            want, slack = rot.apply(raw, at)
            assert bool(((q.q.double().cpu() - want).abs() <= query_bound(want, slack)).all()), f"step {step}: queries"
            U.attend(ctx, cache, q, seqs, replica=1)
            U.check_all(cache, q, seqs, 1, f"step {step}")
            keys, slack = rot.apply(kv[:, 0], at)
            for b in range(B):
                a, z, n = int(seqs.start[b]), int(seqs.start[b + 1]), int(lens[b])
                full[b].append([x[a:z].transpose(0, 1).cpu() for x in (keys, slack, kv[:, 1].double())])
                want, off, value = (torch.cat(x, 1) for x in zip(*full[b]))
                got = cache.values(1, table[b], n)[0].cpu()
                # a scale for each block and head, keys and values apart; it may have grown at every call so far
                scale = U.power(cache.scales(1)[table[b]].long().cpu()).permute(2, 1, 0).repeat_interleave(64, 2)[:, :, :n, None]
                assert bool(((got[0] - want).abs() <= key_bound(want, scale[0], off, step)).all()), f"step {step}: keys of sequence {b}"
                assert bool(((got[1] - value).abs() <= key_bound(value, scale[1], 0.0, step)).all()), f"step {step}: values of sequence {b}"
        assert ctx.invalid() == 0
        assert all(torch.equal(cache.bufs[0], b) for b in cache.bufs)
    finally:
        ctx.free()
