"""The operators as a model's step uses them: keys rotated on their way into the cache, queries rotated, attention over it;
prompt in chunks, then single tokens, then a drafted tree whose nodes share positions."""
import math

import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import heads_util as U
from test_gpu_heads_append import append, new_rows

pytestmark = pytest.mark.gpu


def rotated(ctx, x, pos, rot):
    y = torch.zeros_like(x)
    T, H, D = x.shape
    kvpub.check(kvpub.kvpub_rotate(ctx.ctx, kvpub.rotate_io(x.data_ptr(), y.data_ptr(), pos.data_ptr(), rot.struct, T, H, D, kvpub.BF16), U.stream()))
    return y


@pytest.mark.parametrize("halves,scaling", [(True, kvpub.SCALING_NONE), (False, kvpub.SCALING_RAMP)])
def test_prompt_tokens_tree(halves, scaling):
    G, H, D, B = 2, 8, 128, 3
    ctx, rot = U.Context(), U.Rotation(D, 0, halves, 1.1, scaling=scaling, factor=4.0, original=64.0, low=1.0, high=8.0)
    cache = U.HeadsCache(24, G, D, 2, fill=0)
    table = np.arange(24).reshape(B, 8).astype(np.int32)
    full = [[] for _ in range(B)]                 # rotated keys and values in 64 bits, before their codes
    try:
        lens = np.zeros(B, np.int64)
        depth = np.array([0, 1, 1, 2, 2, 3])      # of the tree's nodes
        parents = [None, 0, 0, 1, 2, 3]
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
            U.attend(ctx, cache, q, seqs, replica=1)
            U.check_all(cache, q, seqs, 1, f"step {step}")           # against the cache's own values
            # and against unrounded keys: their codes are off by 2^-4 at most, a scale's growth may round once more, so a
            # score by 2^-3 of its terms' magnitudes; the outputs' spread is wide, their lse is bounded by the scores'
            keys, _ = rot.apply(kv[:, 0], at)
            want, _ = rot.apply(raw, at)
            for b in range(B):
                a, z = int(seqs.start[b]), int(seqs.start[b + 1])
                full[b].append(torch.stack([keys[a:z].cuda(), kv[a:z, 1].double()]))
                vals = torch.cat(full[b], 1).transpose(1, 2)
                ref = U.reference(want[a:z].cuda(), vals, torch.as_tensor(seqs.seen(b)), q.scale)
                assert bool(((q.lse[a:z].double() - ref[1]).abs() <= 2.0 ** -3 * ref[2] + 1e-3).all())
        assert ctx.invalid() == 0
        assert all(torch.equal(cache.bufs[0], b) for b in cache.bufs)
    finally:
        ctx.free()
