"""kvpub_store_rotated by groups of four tokens a wave: rows that turn, a last group in part, stores past the L2s."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub
from replicated_fp8_sparse_amd.workloads import CacheLayout

import gpu_util as G
import heads_util as U
import test_gpu_store_rotated as S

pytestmark = pytest.mark.gpu

BOTH = (dict(dim=64), dict(dim=64, halves=True))


def store_turned(T, mag, rope, indexer):
    """One call, and every row of it against kvpub_store, kvpub_rotate and the rotation in 64 bits."""
    layout = CacheLayout(replicas=2, layers=1, num_pages=-(-T // 64) + 1, guard=64)
    x, pos = S.inputs(T, layout.capacity, T + 1, 0, 2, mag)
    dev, plain = G.DeviceCache(layout), G.DeviceCache(layout)
    try:
        d, p = G.DeviceInputs(x), U.i32(pos)
        rope, indexer = rope and U.Rotation(**rope), indexer and U.Rotation(**indexer)
        S.store(dev, 0, d, p, rope, indexer)
        kvpub.check(plain.store(0, d))
        torch.cuda.synchronize()
        live = np.flatnonzero(x.slots >= 0)
        main, codes, scales = S.rows_of(dev, layout, 0, 0, x.slots[live])
        want_main, want_codes, want_scales = S.rows_of(plain, layout, 0, 0, x.slots[live])
        assert torch.equal(main[:, :528], want_main[:, :528])                          # the latent row as the store's
        r = d.rope.view(torch.bfloat16).view(T, 1, 64)
        if rope:
            y = torch.zeros_like(r)
            io = kvpub.rotate_io(r.data_ptr(), y.data_ptr(), p.data_ptr(), rope.struct, T, 1, 64, kvpub.BF16)
            kvpub.check(kvpub.kvpub_rotate(dev.ctx, io, U.stream()))
            r = y
        assert torch.equal(main[:, 528:].contiguous().view(torch.bfloat16), r[live, 0])
        if indexer:
            want, bound = indexer.apply(d.indexer.view(torch.bfloat16).view(T, 1, 128), pos)
            want, bound = want[live, 0], bound[live, 0]
            s = scales.double().cpu()
            amax = want.abs().amax(1)
            # the largest magnitude is off by at most the values' bound, the division rounds once
            assert bool(((s - amax / 448).abs() <= bound.amax(1) / 448 + 2.0 ** -24 * amax / 448).all())
            got = codes.view(torch.float8_e4m3fn).double().cpu() * s[:, None]
            # with y the value (its bound from `want`) and q = RN32(y / s): the code is half a step of e4m3 from q, 2^-4 |q|
            # or 2^-10, and |q s - y| <= 2^-24 |y|, which moves a value across a tie.  In all
            # max(2^-4 |want|, 2^-10 s) + (1 + 2^-4) (2^-24 |want| + bound)
            tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s[:, None]) + 1.07 * (2.0 ** -24 * want.abs() + bound)
            assert bool(((got - want).abs() <= tol).all())
        else:
            assert torch.equal(codes, want_codes) and torch.equal(scales, want_scales)
        for b, c in ((dev.main, plain.main), (dev.idx, plain.idx)):
            assert torch.equal(b[0], b[1])
        rest = np.setdiff1d(np.arange(layout.capacity), x.slots[live])                  # rows of no slot: as before
        for got, want in zip(S.rows_of(dev, layout, 1, 0, rest), S.rows_of(plain, layout, 1, 0, rest)):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    finally:
        dev.free()
        plain.free()


@pytest.mark.parametrize("rope,indexer", [
    BOTH, (dict(dim=40, start=16, halves=True, magnitude=1.2), dict(dim=128)), (dict(dim=8, start=56), dict(dim=24, start=96, halves=True, magnitude=-0.7)),
    (None, dict(dim=120, start=8, halves=True)), (dict(dim=64, halves=True), None)])
@pytest.mark.parametrize("T,mag", [(2049, 1.0), (4099, 30.0), (2050, 1e-3)])
def test_turned_rows(T, mag, rope, indexer):
    store_turned(T, mag, rope, indexer)


def test_turned_rows_past_the_l2s():
    """22,001 tokens of 788 bytes into 2 replicas: more than 32 MiB."""
    assert 22001 * 788 * 2 > 32 << 20
    store_turned(22001, 1.0, *BOTH)


@pytest.mark.parametrize("T,replicas", [(2049, 3), (11003, 4)])
def test_groups_store_the_bytes_of_pieces(T, replicas):
    """The same tokens in calls of up to 2048, a wave a piece, and in one call: padded and invalid slots among them."""
    layout = CacheLayout(replicas=replicas, layers=1, num_pages=-(-T // 64) + 2, guard=64)
    x, pos = S.inputs(T, layout.capacity, T, 9, 40)
    one, many = G.DeviceCache(layout), G.DeviceCache(layout)
    try:
        d, p, rope, indexer = G.DeviceInputs(x), U.i32(pos), U.Rotation(64), U.Rotation(64, 32, True)
        S.store(one, 0, d, p, rope, indexer)
        for t in range(0, T, 2048):
            kvpub.check(kvpub.kvpub_store_rotated(many.ctx, 0, min(2048, T - t), d.latent[t:].data_ptr(), 512, d.rope[t:].data_ptr(), 64,
                                                  d.indexer[t:].data_ptr(), 128, d.slots[t:].data_ptr(), p[t:].data_ptr(), rope.struct,
                                                  indexer.struct, U.stream()))
        torch.cuda.synchronize()
        assert S.same_caches(one, many)
        assert one.errors(False)[1] == many.errors(False)[1] == 9
    finally:
        one.free()
        many.free()
