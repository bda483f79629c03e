"""kvpub_store_rotated while its context is poisoned: a fence that times out on another stream sets the status at some
moment of a run of stores.  Whenever that is, every token's two rows are stored whole or left as they were."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub, workloads as W
from replicated_fp8_sparse_amd.workloads import CacheLayout

import gpu_util as G
import heads_util as U
from test_gpu_store_rotated import rows_of

pytestmark = pytest.mark.gpu

CALLS, TRIALS = 60, 8


@pytest.mark.parametrize("T", [2048, 2600])
def test_a_token_is_stored_whole_or_left(T):
    """2048 tokens: a wave a piece of a row; 2600: a wave a group of rows."""
    layout = CacheLayout(replicas=1, layers=1, num_pages=-(-CALLS * T // 64))
    rng = np.random.default_rng(T)
    bits = lambda w: W.bf16_bits(rng.standard_normal((T, w), dtype=np.float32))
    slots = rng.permutation(layout.capacity)[:CALLS * T].reshape(CALLS, T)
    d = G.DeviceInputs(W.LayerInputs(bits(512), bits(64), bits(128), slots[0]))
    pos, every = U.i32(rng.integers(0, 2 ** 20, T)), G.to_dev_i64(slots)
    rope, indexer = U.Rotation(64), U.Rotation(64, halves=True)

    def store(dev, k):
        kvpub.check(kvpub.kvpub_store_rotated(dev.ctx, 0, T, d.latent.data_ptr(), 512, d.rope.data_ptr(), 64, d.indexer.data_ptr(), 128,
                                              every[k].data_ptr(), pos.data_ptr(), rope.struct, indexer.struct, U.stream()))

    parts = lambda dev: [x.view(torch.uint8).reshape(CALLS, T, -1) for x in rows_of(dev, layout, 0, 0, slots.reshape(-1))]
    clean = G.DeviceCache(layout)
    try:
        old = [x.clone() for x in parts(clean)]
        for k in range(CALLS):
            store(clean, k)
        torch.cuda.synchronize()
        new = parts(clean)
    finally:
        clean.free()
    for trial in range(TRIALS):
        dev = G.DeviceCache(layout, participants=2, timeout_ns=200_000)        # no peer comes: the fence times out
        try:
            side = torch.cuda.Stream()
            torch.cuda.synchronize()
            kvpub.check(dev.fence(0, side))
            for k in range(CALLS - 1):
                store(dev, k)
            torch.cuda.synchronize()
            st, invalid, flags = dev.errors()
            assert st == kvpub.KVPUB_ERR_FENCE_TIMEOUT and flags & kvpub.KVPUB_FLAG_POISONED and invalid == 0
            store(dev, CALLS - 1)                                              # behind the poison
            torch.cuda.synchronize()
            got = parts(dev)
            stored = [(g == n).all(2) for g, n in zip(got, new)]
            left = [(g == o).all(2) for g, o in zip(got, old)]
            count = int(stored[0].sum())
            G.log(f"trial {trial}: {count} of {CALLS * T} tokens, {int((stored[0].any(1) & ~stored[0].all(1)).sum())} calls in part")
            assert not stored[0][-1].any()
            for s, l in zip(stored, left):
                assert bool((s | l).all()), f"{int((~(s | l)).sum())} rows in part"
                assert torch.equal(s, stored[0]), "one row of a token without the other"
        finally:
            dev.free()
