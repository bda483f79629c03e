"""kvpub_heads_append: scales, codes and untouched bytes against 64 bits."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub, workloads as W
from replicated_fp8_sparse_amd.workloads import CacheLayout

import gpu_util as G
import heads_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = U.Context()
    yield c
    c.free()


def new_rows(T, G, D, kind, seed=0, pad=0, mag=1.0):
    """Keys and values of a token side by side: [T, 2, G, D + pad]."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 11)
    x = torch.randn((max(T, 1), 2, G, D + pad), generator=g, device="cuda") * torch.exp(0.5 * torch.randn((max(T, 1), 2, G, 1), generator=g, device="cuda"))
    return (mag * x).to(U.TYPES[kind][0])


def append(ctx, cache, kv, seqs, kind, rot=None, positions=None, D=None):
    D = D or cache.D
    size, G = kv.element_size(), cache.G
    r = kvpub.heads_rows(kv.data_ptr(), kv.data_ptr() + kv.stride(1) * size, seqs.T, U.TYPES[kind][1], kv.stride(0), kv.stride(2),
                         kv.stride(0), kv.stride(2))
    kvpub.check(kvpub.kvpub_heads_append(ctx.ctx, cache.struct, cache.layer, r, seqs.struct, rot and rot.struct,
                                         None if positions is None else positions.data_ptr(), U.stream()), "kvpub_heads_append")
    torch.cuda.synchronize()


def check(cache, before, kv, seqs, rot=None, positions=None, what=""):
    """`before`: the replicas' buffers as they were.  Blocks one by one; what no block writes is as before, bit for bit."""
    D, G = cache.D, cache.G
    expect = [b.clone() for b in before]
    old = type(cache).__new__(type(cache))
    old.__dict__.update(cache.__dict__)
    old.bufs = expect
    bad = 0
    for b in range(len(seqs.lens)):
        kv_len, n, q0 = seqs.kv(b), int(seqs.n[b]), int(seqs.start[b])
        base = kv_len - n
        begin, end = max(base, 0), base + min(n, seqs.max_q)
        if end <= begin:
            continue
        t0 = q0 + begin - base
        x = kv[t0:t0 + end - begin, :, :, :D].double()                           # [m, 2, G, D]
        slack = torch.zeros_like(x)
        if rot:
            at = np.arange(begin, end) if positions is None else positions.cpu().numpy()[t0:t0 + end - begin]
            y, bound = rot.apply(x[:, 0], at)
            x[:, 0], slack[:, 0] = y.cuda(), bound.cuda()
        for block in range(begin // 64, (end - 1) // 64 + 1):
            page = int(seqs.table[b, block])
            if not 0 <= page < cache.pages:
                bad += 1
                continue
            lo, hi = max(begin, block * 64), min(end, block * 64 + 64)
            r0 = lo - block * 64
            new, err = x[lo - begin:hi - begin].permute(2, 1, 0, 3), slack[lo - begin:hi - begin].permute(2, 1, 0, 3)   # [G, 2, rows, D]
            finite = torch.where(torch.isfinite(new), new.abs(), 0.0)
            byte = U.byte_of(finite.amax((2, 3)))
            had = old.scales(0)[page].long().clamp(1, 245)
            if r0:
                byte = torch.maximum(byte, had)
            for r in range(len(before)):
                got_byte, got = cache.scales(r)[page].long(), cache.codes(r)[page].view(torch.float8_e4m3fn).double()
                # the largest magnitude is off by the values' bound: next to a power of two the scale may be either
                low, high = U.byte_of((finite - err).clamp(min=0).amax((2, 3))), U.byte_of((finite + err).amax((2, 3)))
                if r0:
                    low, high = torch.maximum(low, had), torch.maximum(high, had)
                assert bool(((got_byte >= low) & (got_byte <= high)).all()), f"{what}: scale of sequence {b} block {block}"
                s = U.power(got_byte)[..., None, None]
                values = got[:, :, r0:r0 + hi - lo] * s
                exact = U.e4m3(new / s) * s
                # rotated values: half a step of e4m3 around them, moved by their bound
                half = torch.maximum(2.0 ** -4 * new.abs(), 2.0 ** -10 * s) * (1 + 2.0 ** -20) + 2 * err
                near = ((values - new).abs() <= half) | (new.abs() > 448 * s) & (values == exact)
                same = (values == exact) | torch.isnan(values) & torch.isnan(exact)
                assert bool(torch.where(err > 0, near, same).all()), f"{what}: codes of sequence {b} block {block}"
                page_codes = old.codes(r)[page]
                page_codes[:, :, r0:r0 + hi - lo] = cache.codes(r)[page][:, :, r0:r0 + hi - lo]
                if r0:
                    was = before[0][cache.layer * cache.layer_stride:][page * cache.page_stride:][:G * 128 * D].view(G, 2, 64, D)[:, :, :r0]
                    value = was.view(torch.float8_e4m3fn).double()
                    again = U.e4m3(value * torch.exp2((had - got_byte).double())[..., None, None])
                    now = got[:, :, :r0]
                    grown = (got_byte > had)[..., None, None]
                    assert bool((~grown | (now == again) | torch.isnan(now) & torch.isnan(again)).all()), f"{what}: older rows, sequence {b}"
                    keep = cache.codes(r)[page][:, :, :r0]
                    page_codes[:, :, :r0] = torch.where(grown, keep, page_codes[:, :, :r0])
                old.scales(r)[page] = cache.scales(r)[page]
    for r, e in enumerate(expect):
        assert torch.equal(cache.bufs[r], e), f"{what}: bytes that the call does not own, replica {r}"
    return bad


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,n,G,pad,replicas", [
    ([1], [1], 1, 0, 1), ([64, 65, 63, 128], [1, 1, 1, 1], 3, 8, 2), ([200, 70, 1, 300], [130, 3, 1, 300], 2, 0, 3),
    ([100, 0, 130, 5, 64], [36, 0, 66, 5, 64], 8, 16, 2), ([10, 3, 77], [12, 9, 77], 1, 0, 8)])
def test_append(ctx, lens, n, G, pad, replicas, D, kind):
    """Blocks partly filled before, whole, ended inside; more new tokens than positions (the first ones are negative)."""
    cache = U.HeadsCache(sum(-(-max(x, 1) // 64) for x in lens) + 2, G, D, replicas, pad=32)
    seqs = U.Seqs(lens, n, cache.pages)
    kv = new_rows(seqs.T, G, D, kind, pad=pad)
    before = [b.clone() for b in cache.bufs]
    append(ctx, cache, kv, seqs, kind)
    assert check(cache, before, kv, seqs) == 0
    assert ctx.invalid() == 0


@pytest.mark.parametrize("dim,start,halves,magnitude,given", [(128, 0, True, 1.0, False), (40, 8, True, 1.3, True), (8, 120, False, 1.0, False),
                                                              (128, 0, False, 0.5, True), (24, 64, True, 1.0, False)])
def test_rotated(ctx, dim, start, halves, magnitude, given):
    cache = U.HeadsCache(12, 3, 128, 2)
    seqs = U.Seqs([190, 66, 200], [150, 2, 1], cache.pages)
    kv = new_rows(seqs.T, 3, 128, "bf16", seed=dim)
    rot = U.Rotation(dim, start, halves, magnitude)
    pos = U.i32(np.random.default_rng(dim).integers(0, 2 ** 20, seqs.T)) if given else None
    before = [b.clone() for b in cache.bufs]
    append(ctx, cache, kv, seqs, "bf16", rot, pos)
    check(cache, before, kv, seqs, rot, pos)


@pytest.mark.parametrize("mag", [1e-3, 1.0, 40.0, 2.0 ** 60, 2.0 ** -60, 2.0 ** 100])
def test_growth_token_by_token(ctx, mag):
    """A block filled one token at a time, each 2^k times the last: older rows follow the scale, into subnormals."""
    cache = U.HeadsCache(3, 2, 64, 2, fill=0)
    lens = 0
    for i in range(70):
        seqs = U.Seqs([lens + 1], [1], cache.pages, max_kv=128)
        kv = new_rows(1, 2, 64, "bf16", seed=i, mag=mag * 2.0 ** (i // 3 if mag < 2 ** 90 else 0))
        before = [b.clone() for b in cache.bufs]
        append(ctx, cache, kv, seqs, "bf16")
        check(cache, before, kv, seqs, what=f"token {i}")
        lens += 1


def test_no_new_token_rounds_what_keeps_its_scale(ctx):
    cache = U.HeadsCache(1, 1, 128, 1, fill=0)
    kv = new_rows(64, 1, 128, "bf16")
    one = U.Seqs([64], [64], 1)
    append(ctx, cache, kv, one, "bf16")
    whole = cache.bufs[0].clone()
    # the token with the largest magnitudes first: the scale never grows again, and the codes are the same
    first = int(kv[:, 0].abs().amax((1, 2)).argmax())
    order = torch.cat([torch.tensor([first]), torch.tensor([i for i in range(64) if i != first])]).cuda()
    stepped = U.HeadsCache(1, 1, 128, 1, fill=0)
    for i in range(64):
        append(ctx, stepped, kv[order[i:i + 1]], U.Seqs([i + 1], [1], 1, max_kv=64), "bf16")
    a, b = cache.codes(0)[0, 0, 0], stepped.codes(0)[0, 0, 0]
    assert torch.equal(a[order.long()], b) and int(cache.scales(0)[0, 0, 0]) == int(stepped.scales(0)[0, 0, 0])
    assert torch.equal(whole, cache.bufs[0])


def test_what_is_not_finite(ctx):
    cache = U.HeadsCache(2, 1, 64, 1)
    kv = new_rows(70, 1, 64, "bf16")
    kv[3, 0, 0, 5], kv[4, 1, 0, 6], kv[5, 0, 0, 7] = float("inf"), float("-inf"), float("nan")
    kv[66, 0, 0, 0], kv[66, 1, 0, 1] = 3e38, -3e38                              # beyond 448 * 2^118
    kv[67, 0, 0, 0] = 2.0 ** -133                                               # subnormal
    seqs = U.Seqs([70], [70], 2)
    before = [b.clone() for b in cache.bufs]
    append(ctx, cache, kv, seqs, "bf16")
    check(cache, before, kv, seqs)
    first = cache.codes(0)[int(seqs.table[0, 0]), 0].view(torch.float8_e4m3fn).float()
    assert first[0, 3, 5] == 448 and first[1, 4, 6] == -448 and bool(torch.isnan(first[0, 5, 7]))
    assert int(cache.scales(0)[int(seqs.table[0, 1]), 0, 0]) == 245


def test_a_block_of_zeros_and_the_least_scale(ctx):
    cache = U.HeadsCache(2, 2, 64, 1, fill=0xFF)
    kv = torch.zeros(40, 2, 2, 64, dtype=torch.float16, device="cuda")
    kv[7, 1, 1] = 2.0 ** -24
    seqs = U.Seqs([40], [40], 2)
    before = [b.clone() for b in cache.bufs]
    append(ctx, cache, kv, seqs, "fp16")
    check(cache, before, kv, seqs)
    assert cache.scales(0)[int(seqs.table[0, 0])].flatten().tolist()[:3] == [1, 1, 1]


def test_old_scale_bytes_outside_the_range(ctx):
    for byte in (0, 255):
        cache = U.HeadsCache(1, 1, 64, 2)
        for b in cache.bufs:
            cache.page_view(b)[:, 128 * 64:128 * 64 + 2] = byte
        kv = new_rows(1, 1, 64, "bf16")
        seqs = U.Seqs([11], [1], 1)
        before = [b.clone() for b in cache.bufs]
        append(ctx, cache, kv, seqs, "bf16")
        check(cache, before, kv, seqs)


def test_bad_pages_drop_their_rows_and_are_counted(ctx):
    cache = U.HeadsCache(10, 3, 64, 2)
    table = np.array([[0, -1, 2], [10, 3, 4], [5, 6, 2 ** 31 - 1]], np.int32)
    seqs = U.Seqs([190, 130, 140], [150, 1, 100], 10, max_kv=192, table=table)
    kv = new_rows(seqs.T, 3, 64, "bf16")
    before = [b.clone() for b in cache.bufs]
    append(ctx, cache, kv, seqs, "bf16")
    assert check(cache, before, kv, seqs) == 2          # sequence 1 appends to its third page only
    assert ctx.invalid() == 2


def test_bounds_cut_lengths_and_tokens(ctx):
    cache = U.HeadsCache(20, 1, 64, 1)
    seqs = U.Seqs([1000, -5, 130, 64], [30, 4, 100, 10], 20, max_kv=192, max_q=20, seed=3)
    kv = new_rows(seqs.T, 1, 64, "bf16")
    before = [b.clone() for b in cache.bufs]
    append(ctx, cache, kv, seqs, "bf16")
    check(cache, before, kv, seqs)


@pytest.mark.parametrize("B,one_each", [(1, True), (63, True), (64, False), (65, False), (300, True), (5000, False)])
def test_many_sequences(ctx, B, one_each):
    """Places by the sequences' bound and by tokens: 64 sequences a search step."""
    rng = np.random.default_rng(B)
    n = np.ones(B, np.int64) if one_each else rng.integers(0, 4, B)
    if not one_each:
        n[B // 2] = 500
    lens = n + rng.integers(0, 100, B)
    cache = U.HeadsCache(int((-(-np.maximum(lens, 1) // 64)).sum()), 2, 64, 1)
    seqs = U.Seqs(lens, n, cache.pages, one_each=one_each, seed=B)
    kv = new_rows(seqs.T, 2, 64, "bf16", seed=B)
    before = [b.clone() for b in cache.bufs]
    append(ctx, cache, kv, seqs, "bf16")
    if B <= 300:
        check(cache, before, kv, seqs)
        return
    # the codes of every new row, all at once
    b = np.repeat(np.arange(B), n)
    pos = torch.from_numpy(np.concatenate([np.arange(l - k, l) for l, k in zip(lens, n)])).cuda()
    page = torch.from_numpy(seqs.table[b, pos.cpu().numpy() // 64].astype(np.int64)).cuda()
    s = U.power(cache.scales(0)[page].long())[..., None]                                          # [T, G, 2, 1]
    got = cache.codes(0)[page, :, :, pos % 64].view(torch.float8_e4m3fn).double() * s
    assert torch.equal(got, (U.e4m3(kv.double().transpose(1, 2) / s) * s))


def test_a_poisoned_context_appends_nothing():
    layout = CacheLayout(replicas=1, layers=1, num_pages=1, guard=64)
    dev = G.DeviceCache(layout, participants=2, timeout_ns=1000000)
    try:
        kvpub.check(dev.fence(0))                 # the peer never signals: times out
        torch.cuda.synchronize()
        cache = U.HeadsCache(3, 2, 128, 2)
        before = [b.clone() for b in cache.bufs]
        append(dev, cache, new_rows(100, 2, 128, "bf16"), U.Seqs([100], [100], 3), "bf16")
        assert all(torch.equal(a, b) for a, b in zip(before, cache.bufs))
    finally:
        dev.free()


def test_beyond_4_gib(ctx):
    pages = 2 ** 32 // kvpub.heads_page_bytes(8, 256) + 40
    cache = U.HeadsCache(pages, 8, 256, 1, layers=1, layer=0, fill=0)
    seqs = U.Seqs([200], [150], pages, table=np.array([[pages - 1, 3, pages - 20, pages - 7]], np.int32))
    kv = new_rows(150, 8, 256, "bf16")
    rot = U.Rotation(256, halves=True)
    append(ctx, cache, kv, seqs, "bf16", rot)
    want, bound = rot.apply(kv[:, 0], np.arange(50, 200))
    vals, _ = cache.values(0, seqs.table[0], 200)
    s = U.power(cache.scales(0)[torch.from_numpy(seqs.table[0].astype(np.int64)).cuda()].long()).permute(2, 1, 0)      # [2, G, page]
    step = s.repeat_interleave(64, 2)[:, :, 50:200, None]
    new = torch.stack([want.cuda(), kv[:, 1].double()]).transpose(1, 2)
    err = torch.stack([bound.cuda(), torch.zeros_like(bound.cuda())]).transpose(1, 2)
    tol = torch.maximum(2.0 ** -4 * new.abs(), 2.0 ** -10 * step) * (1 + 2.0 ** -20) + 2 * err
    assert bool(((vals[:, :, 50:200] - new).abs() <= tol).all())
    assert int(torch.count_nonzero(cache.page_view(cache.bufs[0])[:pages - 20])) == int(torch.count_nonzero(cache.page_view(cache.bufs[0])[3]))


def test_graph_replays(ctx):
    cache, eager = U.HeadsCache(8, 2, 128, 2), U.HeadsCache(8, 2, 128, 2)
    seqs = U.Seqs([70, 130], [30, 1], 8, max_kv=256)
    kv, rot = new_rows(31, 2, 128, "bf16"), U.Rotation(128)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    r = kvpub.heads_rows(kv.data_ptr(), kv.data_ptr() + kv.stride(1) * 2, 31, kvpub.BF16, kv.stride(0), 128, kv.stride(0), 128)
    with torch.cuda.graph(graph, stream=s):
        kvpub.check(kvpub.kvpub_heads_append(ctx.ctx, cache.struct, cache.layer, r, seqs.struct, rot.struct, None, s.cuda_stream))
    for k in range(4):
        kv.copy_(new_rows(31, 2, 128, "bf16", seed=k, mag=2.0 ** k))
        graph.replay()
        torch.cuda.synchronize()
        append(ctx, eager, kv, seqs, "bf16", rot)
        assert all(torch.equal(a, b) for a, b in zip(cache.bufs, eager.bufs))
        seqs.d_len += torch.tensor([30, 1], device="cuda", dtype=torch.int32)
        torch.cuda.synchronize()
