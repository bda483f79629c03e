"""kvpub_attend and kvpub_attend_slots where a call's bounds promise long runs of
tiles for many query rows (64 and more a sequence, at least 16 tiles a block):
another kernel takes these than the short calls of the other attention tests.
The sequences themselves may be short: the bounds decide."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import attend_util as A
import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    kvpub.load()
    yield
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def cache(_gpu):
    c = A.Cache(160, seed=13)
    yield c
    c.free()


def long_pages(cache, lens, n, heads, seed=0, tree_words=0):
    """Pages of a call whose max_kv_len makes at least 2^12 tiles (16 for each of 256 blocks) of its units of 64 rows."""
    pg = A.Paged(cache, lens, n, seed=seed, tree_words=tree_words)
    units = sum(-(-int(max(n)) * heads // 64) for _ in lens)
    by_tokens = pg.T * heads // 64 + len(lens)
    tiles = -(-4096 // min(units, by_tokens))
    held = pg.table.shape[1]
    width = max(held, tiles)
    table = np.full((len(lens), width), -1, np.int32)        # behind kv_len: never read
    table[:, :held] = pg.table
    pg.table, pg.d_table, pg.max_kv = table, A.dev_i32(table), width * 64
    pg.struct.page_table, pg.struct.page_table_stride, pg.struct.max_kv_len = pg.d_table.data_ptr(), width, width * 64
    return pg


CASES = [
    # heads, lengths, tokens of each sequence
    (128, [1], [1]),
    (128, [64, 65], [1, 1]),
    (128, [2500], [1]),
    (128, [900, 333, 0, 1000], [1, 1, 1, 1]),
    (64, [777, 64, 2, 1999], [1, 1, 1, 1]),
    (100, [200, 450], [2, 1]),                  # 56 rows in a unit behind the first
    (33, [300, 129, 130], [1, 2, 1]),
    (16, [1500, 700], [40, 9]),
    (16, [200], [130]),                         # the first unit's rows see less than the last's
    (128, [70], [75]),                          # more tokens than positions: the first see nothing
    (5, [3000, 40], [33, 12]),
]


@pytest.mark.parametrize("heads,lens,n", CASES)
def test_causal(cache, heads, lens, n):
    G.log(f"attend long H={heads} lens={lens} n={n}")
    pg = long_pages(cache, lens, n, heads, seed=heads)
    q, o = A.Queries(pg.T, heads, seed=heads, pad=8), A.Outputs(pg.T, heads, pad=8)
    cache.invalid()
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)
    o.untouched(range(pg.T))
    assert cache.invalid() == 0


@pytest.mark.parametrize("heads,lens,n,words", [
    (32, [500, 130], [24, 9], 1), (16, [300], [100], 2), (128, [90, 200], [64, 3], 1), (8, [1000], [64], 1),
    (64, [40], [70], 1),                        # nodes beyond the words, and negative positions
])
def test_tree(cache, heads, lens, n, words):
    G.log(f"attend long tree H={heads} lens={lens} n={n} words={words}")
    pg = long_pages(cache, lens, n, heads, seed=heads, tree_words=words)
    q, o = A.Queries(pg.T, heads, seed=heads), A.Outputs(pg.T, heads)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)


@pytest.mark.parametrize("order", ["rising", "falling", "late"])
def test_maxima_that_move(cache, order):
    """Scores that grow from tile to tile (every tile outgrows the last maximum by more than 2^8), fall, or
    jump in one row only: a query along one position's own vector, scaled."""
    heads, kv = 128, 900
    pg = long_pages(cache, [kv], [1], heads)
    q, o = A.Queries(1, heads), A.Outputs(1, heads)
    c, r = cache.values(1, pg.slots(0))
    # queries along the difference of late and early rows; row h follows its own direction
    k = torch.cat([c, r], 1)
    t = torch.linspace(-1, 1, kv, dtype=torch.float64, device="cuda")
    along = (k * (t if order != "falling" else -t)[:, None]).sum(0)
    along = 12 * along / along.norm()
    gen = torch.Generator(device="cuda").manual_seed(1)
    mix = torch.randn(heads, generator=gen, device="cuda", dtype=torch.float64).abs() * 3 + 1
    if order == "late":
        mix = torch.zeros_like(mix)
        mix[77] = 4
    rows = (mix[:, None] * along[None]).bfloat16()
    q.latent.copy_(q.latent + rows[None, :, :512])
    q.rope.copy_(q.rope + rows[None, :, 512:])
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)


@pytest.mark.parametrize("scale,mag", [(0.0, 1.0), (-0.5, 1.0), (3.0, 1.0), (0.07, 1e-30), (0.07, 30.0)])
def test_scales_and_sizes(cache, scale, mag):
    pg = long_pages(cache, [700, 90], [1, 1], 128)
    q, o = A.Queries(pg.T, 128, scale=scale, mag=mag), A.Outputs(pg.T, 128)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)


def test_hidden_rows_may_hold_anything():
    """NaN codes, scales and RoPE values behind the last position; the newest position NaN: only the last token's rows."""
    c = A.Cache(6, seed=5, written=[])
    pg = long_pages(c, [330], [3], 128)
    slots = pg.slots(0)
    c.free()
    c = A.Cache(6, seed=5, written=slots[:-1])
    try:
        q, o = A.Queries(3, 128), A.Outputs(3, 128)
        A.attend(c, q, pg, o)
        v, r = c.values(1, slots)
        want = A.reference(q.latent[:2], q.rope[:2], q.scale, v, r, pg.seen(0)[:2])
        A.check_rows(o.out[:2], o.lse[:2], want)
        assert bool(torch.isnan(o.out[2]).all()) and bool(torch.isnan(o.lse[2]).all())
    finally:
        c.free()


@pytest.mark.parametrize("long", [False, True])
def test_bad_pages_are_hidden_and_counted_once(cache, long):
    """Among them pages that only the last tokens' rows see."""
    lens, n, heads = [200, 640], [130, 2], 16
    pg = long_pages(cache, lens, n, heads) if long else A.Paged(cache, lens, n)
    pg.table[0, 0], pg.table[0, 3], pg.table[1, 9] = cache.pages, -1, np.iinfo(np.int32).min
    pg.d_table.copy_(A.dev_i32(pg.table))
    q, o = A.Queries(pg.T, heads), A.Outputs(pg.T, heads)
    cache.invalid()
    A.attend(cache, q, pg, o)
    assert cache.invalid() == 3
    for b in range(2):
        p = np.arange(lens[b])
        ok = (pg.table[b, p // 64] >= 0) & (pg.table[b, p // 64] < cache.pages)
        c, r = cache.values(1, np.where(ok, pg.table[b, p // 64].astype(np.int64) * 64 + p % 64, 0))
        a, z = int(pg.start[b]), int(pg.start[b + 1])
        seen = pg.seen(b) & torch.from_numpy(ok).cuda()
        A.check_rows(o.out[a:z], o.lse[a:z], A.reference(q.latent[a:z], q.rope[a:z], q.scale, c, r, seen))


@pytest.mark.parametrize("heads,lists,width", [(128, [2048] * 3 + [5, 0, 64, 65, 1000], 32768), (64, [700, 1, 130], 1 << 17)])
def test_slots(cache, heads, lists, width):
    """Padding all over a long list."""
    G.log(f"slots long H={heads} lists={lists} width={width}")
    rng = np.random.default_rng(heads)
    T = len(lists)
    slots = np.full((T, width), -1, np.int64)
    for t, k in enumerate(lists):
        slots[t, rng.choice(width, size=k, replace=False)] = rng.choice(cache.layout.capacity, size=k, replace=False)
    slots[0, :3] = [cache.layout.capacity, -2, 2 ** 62]
    d = torch.from_numpy(slots).cuda()
    q, o = A.Queries(T, heads, pad=8), A.Outputs(T, heads, pad=8)
    size = kvpub.kvpub_attend_slots_workspace(q.struct, width)
    buf, ws = A.workspace(size)
    cache.invalid()
    kvpub.check(kvpub.kvpub_attend_slots(cache.ctx, 1, cache.layer, q.struct, d.data_ptr(), width, width, *o.args(), ws, size,
                                         torch.cuda.current_stream().cuda_stream), "kvpub_attend_slots")
    torch.cuda.synchronize()
    A.guards_whole(buf)
    assert cache.invalid() == 3
    for t in range(T):
        pick = slots[t][(slots[t] >= 0) & (slots[t] < cache.layout.capacity)]
        c, r = cache.values(1, pick)
        want = A.reference(q.latent[t:t + 1], q.rope[t:t + 1], q.scale, c, r, torch.ones(1, len(pick), dtype=torch.bool, device="cuda"))
        A.check_rows(o.out[t:t + 1], o.lse[t:t + 1], want, f"token {t}")
    o.untouched(range(T))


def test_captured_replayed_and_the_same_bits(cache):
    """A captured call gives the eager call's bits on every replay, with its inputs changed and other work between."""
    pg = long_pages(cache, [900, 333, 65], [1, 3, 1], 128)
    q, o = A.Queries(pg.T, 128), A.Outputs(pg.T, 128)
    size = kvpub.kvpub_attend_workspace(q.struct, pg.struct)
    buf, ws = A.workspace(size)
    call = lambda s: kvpub.check(kvpub.kvpub_attend(cache.ctx, 1, cache.layer, q.struct, pg.struct, *o.args(), ws, size, s.cuda_stream))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call(side)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            call(torch.cuda.current_stream())
    for k in range(4):
        q.latent.mul_(0.75)
        pg.d_len.copy_(A.dev_i32([900 - 70 * k, 333 - k, 65]))
        o.buf.fill_(A.SENTINEL)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        first, lse = o.out.clone(), o.lse.clone()
        o.buf.fill_(A.SENTINEL)
        other = A.Outputs(pg.T, 128)
        A.attend(cache, q, pg, other)
        assert torch.equal(first, other.out) and torch.equal(lse, other.lse), k
        pg.lens = np.array([900 - 70 * k, 333 - k, 65])
        A.check_paged(cache, q, pg, other)
    A.guards_whole(buf)


def weigh(cache, q, pg, o):
    from test_gpu_attend import check_weights
    A.attend(cache, q, pg, o)
    g = torch.Generator(device="cuda").manual_seed(3)
    w_in = torch.rand((len(pg.lens), pg.max_kv + 7), generator=g, device="cuda")
    for source in (w_in, None):
        w_out = torch.full_like(w_in, A.SENTINEL)
        kvpub.check(kvpub.kvpub_attend_weights(cache.ctx, 1, cache.layer, q.struct, pg.struct, *o.args()[3:],
                                               None if source is None else source.data_ptr(), w_out.data_ptr(), w_in.shape[1],
                                               torch.cuda.current_stream().cuda_stream), "kvpub_attend_weights")
        torch.cuda.synchronize()
        check_weights(cache, q, pg, o.lse, source, w_out)
        assert bool((w_out[:, pg.max_kv:] == A.SENTINEL).all())


def test_weights_of_ragged_sequences(cache):
    """Empty sequences and one without tokens between, a bound far behind the lengths."""
    lens, n, heads = [1600, 0, 1, 64, 1300, 129], [1, 1, 1, 0, 2, 5], 128
    pg = long_pages(cache, lens, n, heads)
    weigh(cache, A.Queries(pg.T, heads), pg, A.Outputs(pg.T, heads))


@pytest.mark.parametrize("seqs", [64, 65, 80])
def test_weights_of_many_sequences(cache, seqs):
    rng = np.random.default_rng(seqs)
    lens, n = rng.integers(0, 129, seqs), rng.integers(0, 3, seqs)
    pg = A.Paged(cache, lens, n, max_kv=128)
    weigh(cache, A.Queries(pg.T, 16), pg, A.Outputs(pg.T, 16))


def test_weights_of_a_very_long_sequence(cache):
    """More tiles a block than it sums at once (pages stand in the table many times)."""
    lens, heads = [270037, 5000], 4
    pg = A.Paged(cache, [64, 64], [1, 1])
    rng = np.random.default_rng(2)
    width = 4300
    pg.lens, pg.max_kv = np.array(lens), width * 64
    pg.table = rng.integers(0, cache.pages, (2, width)).astype(np.int32)
    pg.d_len, pg.d_table = A.dev_i32(lens), A.dev_i32(pg.table)
    pg.struct = kvpub.pages(pg.d_len.data_ptr(), pg.d_table.data_ptr(), width, 2, width * 64, q_start=pg.d_start.data_ptr())
    q, o = A.Queries(2, heads), A.Outputs(2, heads)
    weigh(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)


def test_weights_without_queries_are_copied(cache):
    pg = long_pages(cache, [130, 64], [1, 1], 64)
    q = A.Queries(0, 64)
    w_in = torch.rand((2, pg.max_kv), device="cuda")
    w_out = torch.full_like(w_in, A.SENTINEL)
    pg.struct.q_start = pg.d_start.data_ptr()
    kvpub.check(kvpub.kvpub_attend_weights(cache.ctx, 1, cache.layer, q.struct, pg.struct, None, 0, w_in.data_ptr(),
                                           w_out.data_ptr(), pg.max_kv, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(w_in, w_out)


def test_a_poisoned_context_attends_but_does_not_evict():
    c = A.Cache(6, seed=4)
    dev = G.DeviceCache(c.layout, participants=2, timeout_ns=2_000_000)     # a second context that poisons itself
    try:
        for a, b in zip(dev.main + dev.idx, c.dev.main + c.dev.idx):
            a.copy_(b)
        kvpub.check(dev.fence(0))
        st, _, flags = dev.errors()
        assert st == kvpub.KVPUB_ERR_FENCE_TIMEOUT and flags & kvpub.KVPUB_FLAG_POISONED
        pg = A.Paged(c, [300], [1])
        q, good, o = A.Queries(1, 64), A.Outputs(1, 64), A.Outputs(1, 64)
        A.attend(c, q, pg, good)
        own, c.ctx = c.ctx, dev.ctx
        try:
            A.attend(c, q, pg, o)
        finally:
            c.ctx = own
        assert torch.equal(o.out, good.out) and torch.equal(o.lse, good.lse)
        w = torch.rand((1, 300), device="cuda")
        kept, new, out = (torch.full((1, k), 77, dtype=torch.int32, device="cuda") for k in (100, 1, 1))
        w_out = torch.full_like(w, A.SENTINEL)
        io = kvpub.evict_io(w.data_ptr(), w_out.data_ptr(), 300, pg.d_len.data_ptr(), pg.d_table.data_ptr(), pg.table.shape[1],
                            pg.d_table.data_ptr(), pg.table.shape[1], kept.data_ptr(), 100, new.data_ptr(), 1, 300, 100)
        before = dev.host()
        buf, ws = A.workspace(kvpub.kvpub_evict_workspace(io))
        kvpub.check(kvpub.kvpub_evict(dev.ctx, c.layer, io, ws, kvpub.kvpub_evict_workspace(io),
                                      torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        after = dev.host()
        for a, b in zip(before[0] + before[1], after[0] + after[1]):
            assert np.array_equal(a, b)
        assert bool((kept == 77).all()) and bool((new == 77).all()) and bool((w_out == A.SENTINEL).all())
    finally:
        dev.free()
        c.free()
