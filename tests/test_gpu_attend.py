"""Latent attention over the published cache, absorbed form: kvpub_attend
(pages; causal and drafted trees), kvpub_attend_slots and kvpub_attend_weights,
against plain forms in 64 bits computed from the cache's bytes."""
import math

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
    c = A.Cache(160, seed=3)
    yield c
    c.free()


PAGED = [
    # heads, lengths, tokens of each sequence
    (1, [1], [1]),
    (16, [700], [1]),
    (16, [64], [1]),
    (5, [63, 65, 1, 128], [1, 1, 1, 1]),
    (16, [1000, 0, 130], [2, 1, 0]),            # an empty sequence, one without tokens
    (32, [500, 129], [1, 1]),
    (24, [300, 40], [1, 3]),
    (64, [777, 64, 2], [1, 1, 1]),
    (128, [900, 333], [1, 1]),
    (100, [200, 450], [2, 1]),
    (128, [320], [7]),
    (3, [10], [25]),                            # more tokens than positions: the first see nothing
    (16, [400, 257], [40, 9]),
    (7, [2500], [1]),
    (128, [2500], [1]),
]


@pytest.mark.parametrize("heads,lens,n", PAGED)
def test_paged_causal(cache, heads, lens, n):
    G.log(f"attend H={heads} lens={lens} n={n}")
    pg = A.Paged(cache, lens, n, seed=heads)
    q, o = A.Queries(pg.T, heads, seed=heads, pad=8), A.Outputs(pg.T, heads, pad=8)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)
    o.untouched(range(pg.T))
    assert cache.invalid() == 0


@pytest.mark.parametrize("heads,lens,n,words", [
    (16, [24], [24], 1),                        # nothing but the tree
    (16, [1000], [24], 1),
    (32, [200, 90], [64, 13], 1),
    (8, [300, 128], [130, 70], 3),
    (4, [150], [70], 1),                        # nodes from 64 on have no bit: not seen, not even by themselves
    (128, [100], [5], 2),
    (2, [20], [33], 1),                         # negative first positions
])
def test_paged_tree(cache, heads, lens, n, words):
    G.log(f"attend tree H={heads} lens={lens} n={n} words={words}")
    pg = A.Paged(cache, lens, n, seed=heads + words, tree_words=words)
    q, o = A.Queries(pg.T, heads, seed=heads), A.Outputs(pg.T, heads)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)
    o.untouched(range(pg.T))


def test_empty_masks_give_zeros():
    """A tree of all-clear words with nothing behind it: every row is empty."""
    c = A.Cache(2, seed=1)
    try:
        pg = A.Paged(c, [10], [10], tree_words=1)
        pg.d_tree.zero_()
        q, o = A.Queries(10, 16), A.Outputs(10, 16)
        A.attend(c, q, pg, o)
        assert bool((o.out == 0).all()) and bool(torch.isneginf(o.lse).all())
    finally:
        c.free()


@pytest.mark.parametrize("heads", [16, 128])
def test_one_token_a_sequence_without_q_start(cache, heads):
    pg = A.Paged(cache, [65, 300, 0, 7], [1, 1, 1, 1], one_each=True)
    q, o = A.Queries(pg.T, heads), A.Outputs(pg.T, heads)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)


@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0])
def test_scales(cache, scale):
    pg = A.Paged(cache, [200, 30], [1, 4])
    q, o = A.Queries(pg.T, 16, scale=scale), A.Outputs(pg.T, 16)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)


@pytest.mark.parametrize("mag", [1e-30, 30.0])
def test_small_and_large_queries(cache, mag):
    """Flat weights, and weights of one position."""
    pg = A.Paged(cache, [500], [2])
    q, o = A.Queries(pg.T, 16, mag=mag), A.Outputs(pg.T, 16)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)


@pytest.mark.parametrize("tree", [0, 1])
def test_hidden_rows_may_hold_anything(tree):
    """NaN codes, scales and RoPE values behind the last position, and in a drafted row that no token sees."""
    n, kv = 6, 70
    pg_slots = None
    for heads in (4, 128):
        c = A.Cache(4, seed=5, written=[])
        try:
            pg = A.Paged(c, [kv], [n], tree_words=tree)
            hidden = kv - 2                       # node 4
            if tree:
                pg.tree[:, 0] &= ~(np.uint64(1) << np.uint64(4))
                pg.d_tree.copy_(torch.from_numpy(pg.tree.view(np.int64)))
            pg_slots = pg.slots(0)
            keep = [s for i, s in enumerate(pg_slots) if not (tree and i == hidden)]
            c.free()
            c = A.Cache(4, seed=5, written=keep)
            q, o = A.Queries(n, heads), A.Outputs(n, heads)
            A.attend(c, q, pg, o)
            A.check_paged(c, q, pg, o)
        finally:
            c.free()


def test_a_nan_row_reaches_only_those_that_see_it():
    """The newest position's row is NaN: the last token's rows are NaN, the others are not touched."""
    c = A.Cache(4, seed=5, written=[])
    pg = A.Paged(c, [100], [3])
    slots = pg.slots(0)
    c.free()
    c = A.Cache(4, seed=5, written=slots[:-1])
    try:
        q, o = A.Queries(3, 16), A.Outputs(3, 16)
        A.attend(c, q, pg, o)
        v, r = c.values(1, slots)
        seen = pg.seen(0)
        want = A.reference(q.latent[:2], q.rope[:2], q.scale, v, r, seen[:2])
        A.check_rows(o.out[:2], o.lse[:2], want)
        assert bool(torch.isnan(o.out[2]).all()) and bool(torch.isnan(o.lse[2]).all())
    finally:
        c.free()


def test_bad_pages_are_hidden_and_counted(cache):
    pg = A.Paged(cache, [300, 200], [2, 1])
    pg.table[0, 1], pg.table[0, 3], pg.table[1, 0] = -1, cache.pages, np.iinfo(np.int32).max
    pg.d_table.copy_(A.dev_i32(pg.table))
    for heads in (16, 128):
        q, o = A.Queries(pg.T, heads), A.Outputs(pg.T, heads)
        cache.invalid()
        A.attend(cache, q, pg, o)
        assert cache.invalid() == 3
        for b in range(2):
            p = np.arange(int(pg.lens[b]))
            ok = (pg.table[b, p // 64] >= 0) & (pg.table[b, p // 64] < cache.pages)
            c, r = cache.values(1, np.where(ok, pg.table[b, p // 64].astype(np.int64) * 64 + p % 64, 0))
            a, z = int(pg.start[b]), int(pg.start[b + 1])
            seen = pg.seen(b) & torch.from_numpy(ok).cuda()
            A.check_rows(o.out[a:z], o.lse[a:z], A.reference(q.latent[a:z], q.rope[a:z], q.scale, c, r, seen))


def test_lengths_are_clamped_and_padding_tokens_left(cache):
    """kv_len beyond max_kv_len and below 0, more tokens than max_q_len, tokens behind the last sequence."""
    pg = A.Paged(cache, [128, 128], [3, 2], max_kv=128, max_q=2)
    pg.d_len.copy_(A.dev_i32([10 ** 9, -5]))
    q, o = A.Queries(pg.T + 2, 16), A.Outputs(pg.T + 2, 16)
    A.attend(cache, q, pg, o)
    c, r = cache.values(1, pg.slots(0))
    want = A.reference(q.latent[:2], q.rope[:2], q.scale, c, r, A.visible(3, 128)[:2])
    A.check_rows(o.out[:2], o.lse[:2], want)
    assert bool((o.out[3:5] == 0).all()) and bool(torch.isneginf(o.lse[3:5]).all())
    o.untouched([0, 1, 3, 4])


def test_many_sequences_and_no_lse(cache):
    lens = [int(x) for x in np.random.default_rng(0).integers(0, 65, 150)]
    pg = A.Paged(cache, lens, [1] * 150)
    q, o = A.Queries(pg.T, 8), A.Outputs(pg.T, 8)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)
    first = o.out.clone()
    size = kvpub.kvpub_attend_workspace(q.struct, pg.struct)
    buf, ws = A.workspace(size)
    o.buf.fill_(A.SENTINEL)
    kvpub.check(kvpub.kvpub_attend(cache.ctx, 1, cache.layer, q.struct, pg.struct, o.buf.data_ptr(), o.token, o.head, None, 0,
                                   ws, size, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(o.out, first)


def test_600_sequences():
    """More sequences than a block has threads."""
    c = A.Cache(600, seed=9, replicas=1)
    try:
        lens = [int(x) for x in np.random.default_rng(0).integers(1, 65, 600)]
        pg = A.Paged(c, lens, [1] * 600)
        q, o = A.Queries(600, 16), A.Outputs(600, 16)
        A.attend(c, q, pg, o, replica=0)
        A.check_paged(c, q, pg, o, replica=0)
    finally:
        c.free()


@pytest.mark.parametrize("heads,lists", [
    (1, [1]), (16, [64, 3]), (64, [256, 0, 65, 128]), (128, [300, 1]), (128, [2048]), (40, [63, 129]), (16, [2500]),
])
def test_slots(cache, heads, lists):
    G.log(f"slots H={heads} lists={lists}")
    rng = np.random.default_rng(heads)
    T, K = len(lists), max(lists)
    slots = np.full((T, K + 3), -1, np.int64)
    for t, k in enumerate(lists):
        slots[t, :k] = rng.choice(cache.layout.capacity, size=k, replace=False)
        rng.shuffle(slots[t, :K])              # padding among the valid ones
    slots[:, K:] = 5                           # behind the list
    d = torch.from_numpy(slots).cuda()
    q, o = A.Queries(T, heads, pad=8), A.Outputs(T, heads, pad=8)
    size = kvpub.kvpub_attend_slots_workspace(q.struct, K)
    buf, ws = A.workspace(size)
    cache.invalid()
    kvpub.check(kvpub.kvpub_attend_slots(cache.ctx, 1, cache.layer, q.struct, d.data_ptr(), K + 3, K, *o.args(), ws, size,
                                         torch.cuda.current_stream().cuda_stream), "kvpub_attend_slots")
    torch.cuda.synchronize()
    A.guards_whole(buf)
    for t in range(T):
        pick = slots[t, :K][slots[t, :K] >= 0]
        c, r = cache.values(1, pick)
        want = A.reference(q.latent[t:t + 1], q.rope[t:t + 1], q.scale, c, r, torch.ones(1, len(pick), dtype=torch.bool, device="cuda"))
        A.check_rows(o.out[t:t + 1], o.lse[t:t + 1], want, f"token {t}")
    o.untouched(range(T))
    assert cache.invalid() == 0


def test_bad_and_repeated_slots(cache):
    cap = cache.layout.capacity
    slots = torch.tensor([[3, 3, cap, -2, 2 ** 62, -1, 9], [-1] * 7, [cap, cap, cap, -7, -1, -1, cap]], device="cuda")
    for heads in (16, 128):
        q, o = A.Queries(3, heads), A.Outputs(3, heads)
        size = kvpub.kvpub_attend_slots_workspace(q.struct, 7)
        buf, ws = A.workspace(size)
        cache.invalid()
        kvpub.check(kvpub.kvpub_attend_slots(cache.ctx, 1, cache.layer, q.struct, slots.data_ptr(), 7, 7, *o.args(), ws, size,
                                             torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert cache.invalid() == 3 + 5
        c, r = cache.values(1, [3, 3, 9])
        want = A.reference(q.latent[:1], q.rope[:1], q.scale, c, r, torch.ones(1, 3, dtype=torch.bool, device="cuda"))
        A.check_rows(o.out[:1], o.lse[:1], want)
        assert bool((o.out[1:] == 0).all()) and bool(torch.isneginf(o.lse[1:]).all())


def test_no_slots_give_zeros(cache):
    q, o = A.Queries(2, 16), A.Outputs(2, 16)
    size = kvpub.kvpub_attend_slots_workspace(q.struct, 0)
    buf, ws = A.workspace(size)
    kvpub.check(kvpub.kvpub_attend_slots(cache.ctx, 0, 0, q.struct, None, 0, 0, *o.args(), ws, size,
                                         torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert bool((o.out == 0).all()) and bool(torch.isneginf(o.lse).all())


# ---- weights -------------------------------------------------------------------

def check_weights(cache, q, pg, lse, w_in, w_out, replica=1):
    """Each sum of exp(s - lse) is within the scores' error, relative (see attend_util.check_rows), plus
    binary32 sums of the rows' weights; what is beyond kv_len keeps its weight."""
    for b in range(len(pg.lens)):
        a, z, kv = int(pg.start[b]), int(pg.start[b + 1]), int(pg.lens[b])
        got = w_out[b].double()
        base = w_in[b].double() if w_in is not None else torch.zeros_like(got)
        if a == z or kv == 0:
            assert torch.equal(got[:pg.max_kv], base[:pg.max_kv])
            continue
        c, r = cache.values(replica, pg.slots(b))
        _, l, w, size, _ = A.reference(q.latent[a:z], q.rope[a:z], q.scale, c, r, pg.seen(b))
        moved = torch.where(torch.isinf(l), 0.0, torch.exp(torch.where(torch.isinf(l), 0.0, l - lse[a:z].double())))
        want = base.clone()
        total = (w * moved[..., None]).sum((0, 1))
        want[:kv] += total
        rel = 600 * 2.0 ** -24 * size.max().item() + 2.0 ** -20 * (4 + l[~torch.isinf(l)].abs().max().item())
        tol = rel * 1.1 * total + (w.shape[0] * w.shape[1] + 16) * 2.0 ** -24 * total + 2.0 ** -23 * want[:kv].abs() + 1e-37
        worst = ((got[:kv] - want[:kv]).abs() / tol).max().item()
        assert worst <= 1, f"sequence {b}: off by {worst} of its bound"
        assert torch.equal(got[kv:pg.max_kv], base[kv:pg.max_kv])


@pytest.mark.parametrize("heads,lens,n,words", [
    (16, [700], [1], 0), (128, [500, 65, 0, 64], [1, 1, 1, 1], 0), (128, [130], [3], 0), (5, [40, 2000], [9, 1], 0),
    (16, [300, 70], [40, 24], 1), (1, [1], [1], 0), (3, [10], [25], 0),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_weights(cache, heads, lens, n, words, in_place):
    G.log(f"weights H={heads} lens={lens} n={n} words={words} in_place={in_place}")
    pg = A.Paged(cache, lens, n, seed=heads, tree_words=words, max_kv=max(lens) + 7)
    q, o = A.Queries(pg.T, heads), A.Outputs(pg.T, heads)
    A.attend(cache, q, pg, o)
    stride = pg.max_kv + 5
    w_in = torch.rand(len(lens), stride, device="cuda")
    w_out = w_in.clone() if in_place else torch.full_like(w_in, A.SENTINEL)
    src = w_out if in_place else w_in
    for _ in range(1):
        kvpub.check(kvpub.kvpub_attend_weights(cache.ctx, 1, cache.layer, q.struct, pg.struct, o.lse_buf.data_ptr(), heads + 1,
                                               src.data_ptr(), w_out.data_ptr(), stride, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    check_weights(cache, q, pg, o.lse, w_in, w_out)
    edge = w_in[:, pg.max_kv:] if in_place else torch.full_like(w_in[:, pg.max_kv:], A.SENTINEL)
    assert torch.equal(w_out[:, pg.max_kv:], edge)


def test_weights_from_nothing(cache):
    pg = A.Paged(cache, [300], [1])
    q, o = A.Queries(1, 64), A.Outputs(1, 64)
    A.attend(cache, q, pg, o)
    w = torch.full((1, 300), math.nan, device="cuda")
    kvpub.check(kvpub.kvpub_attend_weights(cache.ctx, 1, cache.layer, q.struct, pg.struct, o.lse_buf.data_ptr(), 65, None,
                                           w.data_ptr(), 300, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    check_weights(cache, q, pg, o.lse, None, w)
    assert abs(w.double().sum().item() - 64) < 1e-3      # every head's weights sum to 1


def test_weights_ignore_hidden_rows_and_bad_pages():
    c = A.Cache(4, seed=5, written=[])
    pg = A.Paged(c, [70], [4])
    c.free()
    c = A.Cache(4, seed=5, written=pg.slots(0)[:69])      # the newest row is NaN
    try:
        q, o = A.Queries(4, 16), A.Outputs(4, 16)
        A.attend(c, q, pg, o)
        o.lse[3] = -math.inf                              # whose token is left out
        w = torch.zeros(1, 128, device="cuda")
        kvpub.check(kvpub.kvpub_attend_weights(c.ctx, 1, c.layer, q.struct, pg.struct, o.lse_buf.data_ptr(), 17, None,
                                               w.data_ptr(), 128, torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert bool(torch.isfinite(w).all()) and abs(w.double().sum().item() - 48) < 1e-3 and w[0, 69] == 0
    finally:
        c.free()


# ---- streams, graphs, two calls at once ----------------------------------------

def test_two_streams_with_workspaces_of_their_own(cache):
    sets = []
    for i, heads in enumerate((16, 128)):
        pg = A.Paged(cache, [900 + i, 333], [1, 1], seed=i)
        q, o = A.Queries(pg.T, heads, seed=i), A.Outputs(pg.T, heads)
        size = kvpub.kvpub_attend_workspace(q.struct, pg.struct)
        sets.append((pg, q, o, A.workspace(size), size, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        for pg, q, o, (buf, ws), size, s in sets:
            kvpub.check(kvpub.kvpub_attend(cache.ctx, 1, cache.layer, q.struct, pg.struct, *o.args(), ws, size, s.cuda_stream))
    torch.cuda.synchronize()
    for pg, q, o, _, _, _ in sets:
        A.check_paged(cache, q, pg, o)


def test_captured_calls_follow_their_inputs(cache):
    """attend + weights captured once; queries, lengths and tables change between replays."""
    pg = A.Paged(cache, [500, 200], [2, 1], max_kv=640)
    q, o = A.Queries(pg.T, 32), A.Outputs(pg.T, 32)
    size = kvpub.kvpub_attend_workspace(q.struct, pg.struct)
    buf, ws = A.workspace(size)
    w = torch.zeros(2, 640, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = torch.cuda.current_stream().cuda_stream
        kvpub.check(kvpub.kvpub_attend(cache.ctx, 1, cache.layer, q.struct, pg.struct, *o.args(), ws, size, s))
        kvpub.check(kvpub.kvpub_attend_weights(cache.ctx, 1, cache.layer, q.struct, pg.struct, o.lse_buf.data_ptr(), 33, None,
                                               w.data_ptr(), 640, s))
    for k, lens in enumerate([[500, 200], [640, 1], [3, 0], [64, 65]]):
        other = A.Paged(cache, lens, [2, 1], seed=k + 50, max_kv=640)
        pg.lens, pg.table = other.lens, other.table
        pg.d_len.copy_(other.d_len)
        pg.d_table.copy_(other.d_table)
        fresh = A.Queries(pg.T, 32, seed=k + 9)
        q._l.copy_(fresh._l)
        q._r.copy_(fresh._r)
        g.replay()
        torch.cuda.synchronize()
        A.check_paged(cache, q, pg, o)
        check_weights(cache, q, pg, o.lse, None, w)


def test_the_same_bits_again(cache):
    pg = A.Paged(cache, [2500, 700, 64], [1, 3, 1])
    q, o = A.Queries(pg.T, 128), A.Outputs(pg.T, 128)
    A.attend(cache, q, pg, o)
    first, lse = o.out.clone(), o.lse.clone()
    for _ in range(5):
        A.attend(cache, q, pg, o)
        assert torch.equal(o.out, first) and torch.equal(o.lse, lse)
