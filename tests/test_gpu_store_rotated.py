"""kvpub_store_rotated: the bytes of kvpub_store where nothing turns, the bits of kvpub_rotate in the RoPE values, the
Indexer-K codes against 64 bits, and everything kvpub_store promises about slots."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub, workloads as W
from replicated_fp8_sparse_amd.workloads import CacheLayout

import gpu_util as G
import heads_util as U

pytestmark = pytest.mark.gpu


def inputs(T, capacity, seed=0, invalid=0, pads=0, mag=1.0):
    rng = np.random.default_rng(seed)
    slots = rng.choice(capacity, size=T, replace=False).astype(np.int64) if T <= capacity else np.full(T, -1, np.int64)
    order = rng.permutation(T)
    slots[order[:pads]] = -1
    slots[order[pads:pads + invalid]] = np.resize([capacity, -2, 2 ** 40, -2 ** 63], invalid)
    bits = lambda w: W.bf16_bits(mag * rng.standard_normal((T, w), dtype=np.float32))
    return W.LayerInputs(bits(512), bits(64), bits(128), slots), rng.integers(0, 2 ** 20, T)


def store(dev, layer, d, pos, rope, indexer, T=None):
    kvpub.check(kvpub.kvpub_store_rotated(dev.ctx, layer, d.T if T is None else T, d.latent.data_ptr(), 512, d.rope.data_ptr(), 64,
                                          d.indexer.data_ptr(), 128, d.slots.data_ptr(), pos.data_ptr(),
                                          rope and rope.struct, indexer and indexer.struct, U.stream()), "kvpub_store_rotated")
    torch.cuda.synchronize()


def rows_of(dev, layout, replica, layer, slots):
    m = dev.main[replica][layer * layout.main_layer_stride:][:layout.num_pages * layout.main_page_stride].view(layout.num_pages, -1)
    i = dev.idx[replica][layer * layout.idx_layer_stride:][:layout.num_pages * layout.idx_page_stride].view(layout.num_pages, -1)
    s = torch.as_tensor(slots, device="cuda")
    main = m[:, :64 * 656].reshape(-1, 656)[s]
    codes, scales = i[:, :8192].reshape(-1, 128)[s], i[:, 8192:8448].reshape(-1, 4)[s].contiguous().view(torch.float32)[:, 0]
    return main, codes, scales


def same_caches(a, b):
    return all(torch.equal(x, y) for x, y in zip(a.main + a.idx, b.main + b.idx))


@pytest.mark.parametrize("T,replicas,pads,invalid", [(1, 1, 0, 0), (3, 2, 1, 0), (64, 2, 3, 2), (1001, 3, 50, 7), (2500, 8, 100, 0), (4096, 4, 0, 0)])
def test_nothing_turns_gives_the_stores_bytes(T, replicas, pads, invalid):
    layout = CacheLayout(replicas=replicas, layers=2, num_pages=-(-T // 64) + 3, guard=64)
    x, _ = inputs(T, layout.capacity, T, invalid, pads)
    plain, turned = G.DeviceCache(layout), G.DeviceCache(layout)
    try:
        d, zero = G.DeviceInputs(x), torch.zeros(T, dtype=torch.int32, device="cuda")
        kvpub.check(plain.store(1, d))
        for rope, indexer in ((U.Rotation(64), U.Rotation(64, 64, True)), (None, U.Rotation(128)), (U.Rotation(16, 8, True), None), (None, None)):
            store(turned, 1, d, zero, rope, indexer)
            assert same_caches(plain, turned)
            for b in turned.main:
                turned.layout.fill_device(b, "main")
            for b in turned.idx:
                turned.layout.fill_device(b, "idx")
        assert plain.errors(False)[1] == invalid and turned.errors(False)[1] == 4 * invalid
    finally:
        plain.free()
        turned.free()


@pytest.mark.parametrize("rope,indexer", [
    (dict(dim=64), dict(dim=64, halves=True)), (dict(dim=40, start=16, halves=True, magnitude=1.2), dict(dim=128)),
    (dict(dim=8, start=56), dict(dim=24, start=96, halves=True, magnitude=-0.7)), (None, dict(dim=120, start=8, halves=True)),
    (dict(dim=64, halves=True), None)])
@pytest.mark.parametrize("T,mag", [(5, 1.0), (700, 30.0), (1500, 1e-3)])
def test_turned_rows(T, mag, rope, indexer):
    layout = CacheLayout(replicas=2, layers=1, num_pages=-(-T // 64) + 1, guard=64)
    x, pos = inputs(T, layout.capacity, T + 1, 0, 2, mag)
    dev, plain = G.DeviceCache(layout), G.DeviceCache(layout)
    try:
        d, p = G.DeviceInputs(x), U.i32(pos)
        rope, indexer = rope and U.Rotation(**rope), indexer and U.Rotation(**indexer)
        store(dev, 0, d, p, rope, indexer)
        kvpub.check(plain.store(0, d))
        torch.cuda.synchronize()
        live = np.flatnonzero(x.slots >= 0)
        main, codes, scales = rows_of(dev, layout, 0, 0, x.slots[live])
        want_main, want_codes, want_scales = rows_of(plain, layout, 0, 0, x.slots[live])
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
            amax, slack = want.abs().amax(1), bound.amax(1)
            s = scales.double().cpu()
            # the largest magnitude is off by at most the values' bound, the division rounds once
            assert bool(((s - amax / 448).abs() <= slack / 448 + 2.0 ** -24 * amax / 448).all())
            got = codes.view(torch.float8_e4m3fn).double().cpu() * s[:, None]
            # half a step of e4m3 (2^-4 of the value, 2^-10 scales where it is subnormal), at the value's bound away;
            # the quotient's rounding moves it by 2^-24
            tol = 2.0 ** -4 * (1 + 2.0 ** -20) * want.abs() + 2 * bound
            assert bool(((got - want).abs() <= torch.maximum(tol, 2.0 ** -10 * s[:, None] + 2 * bound)).all())
        else:
            assert torch.equal(codes, want_codes) and torch.equal(scales, want_scales)
        for b, c in ((dev.main, plain.main), (dev.idx, plain.idx)):
            assert torch.equal(b[0], b[1])
        # rows of no slot, and everything between: as before
        rest = np.setdiff1d(np.arange(layout.capacity), x.slots[live])
        for got, want in zip(rows_of(dev, layout, 1, 0, rest), rows_of(plain, layout, 1, 0, rest)):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    finally:
        dev.free()
        plain.free()


def test_a_row_of_zeros_and_strides_beyond_the_width():
    layout = CacheLayout(replicas=1, layers=1, num_pages=2, guard=64)
    dev = G.DeviceCache(layout)
    try:
        x, pos = inputs(6, layout.capacity, 3)
        lat, rope, ind = (torch.zeros(6, w, dtype=torch.bfloat16, device="cuda") for w in (520, 640, 136))
        d, p, s = G.DeviceInputs(x), U.i32(pos), torch.arange(6, device="cuda")
        lat[:, :512], rope[:, :64] = d.latent.view(torch.bfloat16), d.rope.view(torch.bfloat16)
        rot = U.Rotation(64)
        kvpub.check(kvpub.kvpub_store_rotated(dev.ctx, 0, 6, lat.data_ptr(), 520, rope.data_ptr(), 640, ind.data_ptr(), 136, s.data_ptr(),
                                              p.data_ptr(), rot.struct, rot.struct, U.stream()))
        torch.cuda.synchronize()
        main, codes, scales = rows_of(dev, layout, 0, 0, np.arange(6))
        assert bool((codes == 0).all()) and bool((scales == 0).all())
        want, bound = rot.apply(rope[:, None, :64], pos)
        got = main[:, 528:].contiguous().view(torch.bfloat16).double().cpu()
        assert bool(((got - want[:, 0]).abs() <= bound[:, 0] + 2.0 ** -8 * want[:, 0].abs() + 1e-30).all())
    finally:
        dev.free()


def test_a_poisoned_context_stores_nothing():
    layout = CacheLayout(replicas=2, layers=1, num_pages=2, guard=64)
    dev, clean = G.DeviceCache(layout, participants=2, timeout_ns=1000000), G.DeviceCache(layout)
    try:
        x, pos = inputs(20, layout.capacity, 4, invalid=2)
        kvpub.check(dev.fence(0))                 # the peer never signals: times out
        torch.cuda.synchronize()
        store(dev, 0, G.DeviceInputs(x), U.i32(pos), U.Rotation(64), U.Rotation(64))
        assert same_caches(dev, clean)
        st, n, flags = dev.errors(False)
        assert st == kvpub.KVPUB_ERR_FENCE_TIMEOUT and flags & kvpub.KVPUB_FLAG_POISONED and n == 0
    finally:
        dev.free()
        clean.free()


def test_graph_replays():
    layout = CacheLayout(replicas=2, layers=1, num_pages=4, guard=64)
    dev, eager = G.DeviceCache(layout), G.DeviceCache(layout)
    try:
        x, pos = inputs(100, layout.capacity, 5)
        d, p, rot = G.DeviceInputs(x), U.i32(pos), U.Rotation(64, halves=True)
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            kvpub.check(kvpub.kvpub_store_rotated(dev.ctx, 0, 100, d.latent.data_ptr(), 512, d.rope.data_ptr(), 64, d.indexer.data_ptr(), 128,
                                                  d.slots.data_ptr(), p.data_ptr(), rot.struct, rot.struct, s.cuda_stream))
        for k in range(3):
            p += 777 * k
            d.rope.copy_(torch.randn(100, 64, device="cuda").bfloat16().view(torch.int16).view_as(d.rope))
            graph.replay()
            torch.cuda.synchronize()
            store(eager, 0, d, p, rot, rot)
            assert same_caches(dev, eager)
    finally:
        dev.free()
        eager.free()
