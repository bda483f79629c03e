"""kvpub_heads_attend against its formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import heads_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = U.Context()
    yield c
    c.free()


def cache_for(lens, G, D, **kw):
    return U.HeadsCache(int(sum(-(-max(int(x), 1) // 64) for x in lens)) + 1, G, D, **kw)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,H", [(1, 1), (2, 16), (3, 15), (2, 64)])
@pytest.mark.parametrize("lens,n", [([1], [1]), ([33, 0, 64, 700], [1, 1, 1, 1]), ([5, 130, 65], [5, 2, 65])])
def test_causal(ctx, lens, n, G, H, D, kind):
    cache = cache_for(lens, G, D, replicas=2, pad=16)
    seqs = U.Seqs(lens, n, cache.pages)
    q = U.Query(seqs.T, H, D, kind, pad=8)
    U.attend(ctx, cache, q, seqs, replica=1)
    U.check_all(cache, q, seqs, 1)
    assert ctx.invalid() == 0


@pytest.mark.parametrize("D,G,H,kv,n", [(128, 1, 8, 20000, 1), (64, 2, 2, 40000, 3), (128, 2, 32, 9000, 40), (256, 1, 16, 5000, 5), (128, 1, 128, 3001, 7)])
def test_long_contexts_cut_into_chunks(ctx, D, G, H, kv, n):
    lens = [kv, kv // 3, 40]
    cache = cache_for(lens, G, D, replicas=1)
    seqs = U.Seqs(lens, [n, 1, min(n, 40)], cache.pages)
    q = U.Query(seqs.T, H, D)
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)
    first = q._out.clone(), q._lse.clone()
    U.attend(ctx, cache, q, seqs)
    assert torch.equal(first[0], q._out) and torch.equal(first[1], q._lse)       # the same call gives the same bits


@pytest.mark.parametrize("n,kv,words,G,H,D", [(24, 1000, 1, 2, 16, 128), (64, 64, 1, 1, 4, 64), (130, 400, 3, 2, 2, 128), (100, 130, 1, 1, 5, 256),
                                              (7, 39, 2, 3, 12, 64)])
def test_trees(ctx, n, kv, words, G, H, D):
    """Trees at every offset within a tile; nodes beyond 64 * words are seen by none."""
    lens, counts = [kv, kv - 1, n + 33, n], [n, n - 1, n, n]
    tree = U.random_tree(counts, words, n)
    tree[3] = 0                                                                     # sees only what lies before the tree
    tree[sum(counts[:3]) + 1] = 0                                                   # and this one nothing at all
    cache = cache_for(lens, G, D, replicas=1)
    seqs = U.Seqs(lens, counts, cache.pages, tree=tree)
    q = U.Query(seqs.T, H, D)
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)


def test_more_tokens_than_positions_and_bounds(ctx):
    """The first tokens are before the sequence and see nothing; lengths and tokens beyond the call's bounds."""
    lens, n = [10, 300, -3, 40, 64], [25, 1, 3, 50, 64]
    cache = U.HeadsCache(30, 2, 64, replicas=1)
    for tree in (None, U.random_tree(n, 1, 5)):
        seqs = U.Seqs(lens, n, 30, max_kv=200, max_q=30, tree=tree)
        q = U.Query(seqs.T, 6, 64)
        U.attend(ctx, cache, q, seqs)
        U.check_all(cache, q, seqs)


@pytest.mark.parametrize("fill", [0xFF, 0x7F])
def test_what_is_not_seen_has_no_effect(ctx, fill):
    """Rows behind the end, rows hidden by causality or by a tree, hold NaN codes; scale bytes are what they are."""
    n, kv = 20, 50
    for tree in (None, U.random_tree([n], 1, 3)):
        cache = U.HeadsCache(2, 2, 128, replicas=1)
        seqs = U.Seqs([kv], [n], 2, tree=tree)
        page = int(seqs.table[0, 0])
        cache.codes(0)[page, :, :, kv:] = fill
        hidden = 44                                                                 # some tokens do not see it
        cache.codes(0)[page, :, :, hidden] = fill
        q = U.Query(n, 8, 128)
        U.attend(ctx, cache, q, seqs)
        seen = seqs.seen(0)
        vals, _ = cache.values(0, seqs.table[0, :1], kv)
        clean = np.flatnonzero(~seen[:, hidden])
        assert 0 < len(clean) < n
        want = U.reference(q.q, vals, torch.as_tensor(seen), q.scale)
        for i in clean:
            U.check_rows(q, i, i + 1, [x[i:i + 1] for x in want], f"token {i}")
        for i in np.flatnonzero(seen[:, hidden]):
            assert bool(torch.isnan(q.out[i]).all()) and bool(torch.isnan(q.lse[i]).all())


def test_values_alone_that_are_nan_reach_only_who_sees_them(ctx):
    cache = U.HeadsCache(2, 1, 64, replicas=1)
    seqs = U.Seqs([100], [60], 2)
    cache.codes(0)[int(seqs.table[0, 1]), 0, 1, 10, 3] = 0x7F                        # position 74, value 3
    q = U.Query(60, 4, 64)
    U.attend(ctx, cache, q, seqs)
    vals, _ = cache.values(0, seqs.table[0], 100)
    want = U.reference(q.q, vals, torch.as_tensor(seqs.seen(0)), q.scale)
    for i in range(60):
        if 40 + i < 74:
            U.check_rows(q, i, i + 1, [x[i:i + 1] for x in want], f"token {i}")
        else:
            assert bool(torch.isnan(q.out[i, :, 3]).all())


def test_queries_that_are_not_finite_keep_to_their_row(ctx):
    cache = U.HeadsCache(4, 2, 64, replicas=1)
    seqs = U.Seqs([200], [9], 4)
    q = U.Query(9, 8, 64)
    q.q[4, 3, 7] = float("nan")
    q.q[5, 6, 1] = float("inf")
    U.attend(ctx, cache, q, seqs)
    vals, _ = cache.values(0, seqs.table[0], 200)
    want = U.reference(torch.nan_to_num(q.q, nan=0.0, posinf=0.0), vals, torch.as_tensor(seqs.seen(0)), q.scale)
    for t in range(9):
        for h in range(8):
            if (t, h) in ((4, 3), (5, 6)):
                continue
            one = U.Query.__new__(U.Query)
            one.__dict__.update(q.__dict__)
            one.out, one.lse = q.out[:, h:h + 1], q.lse[:, h:h + 1]
            U.check_rows(one, t, t + 1, [x[t:t + 1, h:h + 1] for x in want], f"token {t} head {h}")
    assert bool(torch.isnan(q.out[4, 3]).all())


def test_bad_pages_hide_their_positions_and_are_counted_once(ctx):
    cache = U.HeadsCache(20, 4, 64, replicas=1)
    table = np.array([[0, -1, 2, 20], [4, 5, 6, 7], [-7, 8, 9, 10], [11, 12, 2 ** 31 - 1, 13]], np.int32)
    seqs = U.Seqs([256, 200, 60, 130], [100, 3, 1, 50], 20, max_kv=256, table=table)
    q = U.Query(seqs.T, 16, 64)
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)
    assert ctx.invalid() == 4
    q = U.Query(seqs.T, 16, 64, lse=False)
    U.attend(ctx, cache, q, seqs)
    assert ctx.invalid() == 4 and bool((q.lse == U.SENTINEL).all())
    # a drafted page that no node sees is not counted: 70 nodes behind 64 positions, the last 6 on a bad page
    for sees, count in ((0, 0), (1, 1)):
        tree = np.zeros((70, 2), np.uint64)
        tree[:, 0] = 1
        tree[5, 1] = sees << 3
        seqs = U.Seqs([134], [70], 20, table=np.array([[0, 1, 99]], np.int32), tree=tree)
        q = U.Query(70, 16, 64)
        U.attend(ctx, cache, q, seqs)
        U.check_all(cache, q, seqs)
        assert ctx.invalid() == count


def test_scores_of_all_sizes(ctx):
    """Large scores (weights of one position), equal ones, negative scales; zero scale averages."""
    cache = U.HeadsCache(12, 2, 64, replicas=1, spread=2.0)
    seqs = U.Seqs([700], [2], 12)
    for scale, mag in ((1.0, 8.0), (-0.125, 1.0), (0.0, 1.0), (1e-30, 1.0)):
        q = U.Query(2, 8, 64, scale=scale, mag=mag)
        U.attend(ctx, cache, q, seqs)
        U.check_all(cache, q, seqs, what=f"scale {scale}")


@pytest.mark.parametrize("H", [8, 40])
def test_scores_of_many_powers_of_two_a_step(ctx, H):
    """Scores of some 2^27, below the documented 2^30: the largest is some 2^25 above the others, so its value comes out alone."""
    cache = U.HeadsCache(4, 1, 64, replicas=1)
    seqs = U.Seqs([200], [1], 4)
    q = U.Query(1, H, 64, scale=1.0, mag=2.0 ** 24)
    U.attend(ctx, cache, q, seqs)
    kv, _ = cache.values(0, seqs.table[0], 200)
    x = q.q[0, :, :64].double() @ kv[0, 0].T
    two = x.topk(2, 1)
    assert bool((two.values[:, 0] < 2.0 ** 30).all()) and bool((two.values[:, 0] - two.values[:, 1] > 2.0 ** 16).all())
    want = kv[1, 0][two.indices[:, 0]]
    # the one weight, 2^x, is rounded to bf16 beside a sum that is not: half a step, 2^-8, and the output's own half
    tol = (U.half_step(q.dtype) + 2.0 ** -8) * (1 + 2.0 ** -8) * want.abs()
    assert bool(((q.out[0].double() - want).abs() <= tol).all())
    # a score: D + 24 roundings of the sum of its terms' magnitudes
    tol = (64 + 24) * 2.0 ** -24 * (q.q[0, :, :64].double().abs() @ kv[0, 0].abs().T).amax(1)
    assert bool(((q.lse[0].double() - two.values[:, 0]).abs() <= tol).all())


def test_scales_far_apart(ctx):
    """Blocks of 2^-40 and of 2^30 beside each other: the weights decide, not the order."""
    cache = U.HeadsCache(6, 1, 128, replicas=1)
    seqs = U.Seqs([384], [1], 6)
    for at, power in ((0, -40), (1, 30), (2, 0), (3, -100), (4, 5), (5, -3)):
        cache.scales(0)[int(seqs.table[0, at]), 0, 1] = 127 + power
    for kind in ("bf16", "fp16"):
        q = U.Query(1, 16, 128, kind)
        if kind == "fp16":
            cache.scales(0)[int(seqs.table[0, 1]), 0, 1] = 127 + 2
        U.attend(ctx, cache, q, seqs)
        U.check_all(cache, q, seqs)


@pytest.mark.parametrize("B,n", [(64, 1), (65, 1), (200, 3), (4500, 1)])
def test_many_sequences(ctx, B, n):
    rng = np.random.default_rng(B)
    counts = np.full(B, n) if n == 1 else rng.integers(0, n + 1, B)
    lens = counts + rng.integers(0, 90, B)
    if n > 1:
        counts[B // 3] = lens[B // 3] = 300
    cache = cache_for(lens, 2, 64, replicas=1)
    seqs = U.Seqs(lens, counts, cache.pages, one_each=n == 1)
    q = U.Query(seqs.T, 4, 64)
    U.attend(ctx, cache, q, seqs)
    if B <= 200:
        U.check_all(cache, q, seqs)
    else:
        for b in rng.choice(B, 100, replace=False):
            vals, _ = cache.values(0, seqs.table[b], int(lens[b]))
            U.check_rows(q, int(b), int(b) + 1, U.reference(q.q[b:b + 1], vals, torch.as_tensor(seqs.seen(b)), q.scale), f"sequence {b}")
        q.untouched(range(B))


def test_rows_of_128_query_heads(ctx):
    cache = cache_for([100, 2000], 2, 128, replicas=1)
    seqs = U.Seqs([100, 2000], [3, 1], cache.pages)
    q = U.Query(seqs.T, 256, 128)
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)


def test_beyond_4_gib(ctx):
    pages = 2 ** 32 // kvpub.heads_page_bytes(8, 256) + 40
    cache = U.HeadsCache(pages, 8, 256, 1, layers=1, layer=0, fill=0)
    table = np.array([[pages - 1, 3, pages - 20, pages - 7]], np.int32)
    small = U.HeadsCache(4, 8, 256, 1, layers=1, layer=0)
    cache.page_view(cache.bufs[0])[torch.from_numpy(table[0].astype(np.int64)).cuda()] = small.page_view(small.bufs[0])
    seqs = U.Seqs([250], [3], pages, table=table)
    q = U.Query(3, 16, 256)
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)


def test_graph_replays_and_two_streams(ctx):
    """A captured call beside an eager one on another stream, each with its workspace."""
    cache = cache_for([3000, 500], 2, 128, replicas=1)
    seqs = U.Seqs([3000, 500], [1, 1], cache.pages)
    q, other = U.Query(2, 16, 128), U.Query(2, 16, 128, seed=4)
    size = kvpub.kvpub_heads_attend_workspace(cache.struct, q.struct, seqs.struct)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s, graph, side = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    call = lambda query, w, on: kvpub.check(kvpub.kvpub_heads_attend(ctx.ctx, cache.struct, 0, cache.layer, query.struct, seqs.struct,
                                                                    w.data_ptr(), size, on.cuda_stream))
    with torch.cuda.graph(graph, stream=s):
        call(q, ws[0], s)
    for k in range(4):
        q.q.copy_(torch.randn_like(q.q))
        torch.cuda.synchronize()
        graph.replay()
        call(other, ws[1], side)
        torch.cuda.synchronize()
        U.check_all(cache, q, seqs, what=f"replay {k}")
        U.check_all(cache, other, seqs)


def test_no_positions_at_all(ctx):
    """max_kv_len 0: every token sees nothing, and the tables are not looked at."""
    cache = U.HeadsCache(1, 2, 64, replicas=1)
    for lens in ([0, 0], [5, 300]):
        seqs = U.Seqs(lens, [3, 1], 10, max_kv=0, table=np.full((2, 1), 2 ** 31 - 1))
        q = U.Query(4, 4, 64)
        U.attend(ctx, cache, q, seqs)
        assert bool((q.out == 0).all()) and bool((q.lse == -math.inf).all())
        q.untouched(range(4))
    assert ctx.invalid() == 0


@pytest.mark.parametrize("kv", [511, 512, 513, 767, 768, 769, 1024, 1025, 65536 + 7])
def test_lengths_around_the_cuts(ctx, kv):
    cache = cache_for([kv, 600], 1, 64, replicas=1)
    seqs = U.Seqs([kv, 600], [2, 1], cache.pages)
    q = U.Query(3, 4, 64)
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)


@pytest.mark.parametrize("B,n,kv", [(40, 24, 300), (3, 500, 900), (200, 9, 40)])
def test_units_of_32_and_64_rows_in_one_call(ctx, B, n, kv):
    """Ragged chunks: sequences of one token beside those of many, places by tokens and by the bound."""
    rng = np.random.default_rng(B)
    counts = rng.integers(1, n + 1, B)
    counts[0], counts[-1] = n, 1
    lens = counts + rng.integers(0, kv, B)
    cache = cache_for(lens, 2, 128, replicas=1)
    seqs = U.Seqs(lens, counts, cache.pages)
    q = U.Query(seqs.T, 14, 128)
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)


@pytest.mark.parametrize("kv,n,G,H,D", [(66000, 1, 1, 3, 256), (20000, 3, 1, 8, 128), (9000, 2, 2, 6, 64), (40000, 20, 1, 4, 256)])
def test_more_cuts_than_one_group_of_lanes_joins(ctx, kv, n, G, H, D):
    cache = cache_for([kv, kv // 2], G, D, replicas=1)
    seqs = U.Seqs([kv, kv // 2], [n, n], cache.pages)
    q = U.Query(seqs.T, H, D)
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("kv,n,G,H,D", [(513, 40, 1, 8, 256), (769, 33, 2, 8, 128), (1024, 26, 1, 16, 256), (3000, 90, 1, 16, 64), (6215, 26, 1, 16, 256)])
def test_few_units_of_many_rows_are_cut_finely(ctx, kv, n, G, H, D, kind):
    """A prompt and a tree of the same lengths: rows whose positions end in a cut before the last."""
    lens, counts = [kv, n + 3], [n, n]
    cache = cache_for(lens, G, D, replicas=1)
    tree = U.random_tree(counts, 2, kv)
    for mask in (None, tree):
        seqs = U.Seqs(lens, counts, cache.pages, tree=mask)
        q = U.Query(seqs.T, H, D, kind)
        U.attend(ctx, cache, q, seqs)
        U.check_all(cache, q, seqs)


def test_prompts_that_fill_the_card(ctx):
    """More than 1024 blocks of 64 rows, and queries of both types."""
    for kind in ("bf16", "fp16"):
        cache = cache_for([1100, 900], 16, 64, replicas=1)
        seqs = U.Seqs([1100, 900], [1100, 900], cache.pages)
        q = U.Query(2000, 64, 64, kind)
        U.attend(ctx, cache, q, seqs)
        U.check_all(cache, q, seqs)
