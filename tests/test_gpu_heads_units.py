"""kvpub_heads_attend in units of 16, 32 and 64 rows, whole and cut: every kernel that a launch can choose, with causal
sequences, drafted trees, bad pages and hidden rows of NaN codes.  The sizes come with the plan that they are meant for."""
import numpy as np
import pytest
import torch

import heads_util as U
from heads_plan import plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = U.Context()
    yield c
    c.free()


def cache_for(lens, G, D, **kw):
    return U.HeadsCache(int(sum(-(-max(int(x), 1) // 64) for x in lens)) + 1, G, D, replicas=1, **kw)


# rows of a unit, cuts: (key-value heads, query heads, values a head, tokens of each sequence, positions of each)
SIZES = [
    ((64, 1), (8, 32, 128, [1100, 1083], [1100, 1500])),
    ((64, 1), (8, 24, 128, [700, 650, 1], [700, 900, 65])),
    ((64, 1), (8, 32, 128, [256] * 4, [5000, 256, 4100, 2500])),
    ((64, 1), (16, 64, 64, [1200, 1100], [1200, 1163])),
    ((32, 1), (8, 32, 128, [256, 200], [300, 260])),
    ((32, 5), (8, 32, 128, [70, 3], [6000, 3100])),
    ((32, 1), (2, 14, 64, [24, 9], [70, 300])),
    ((32, 11), (1, 16, 64, [26, 5], [4000, 2000])),
    ((32, 1), (4, 16, 256, [130, 77], [400, 77])),
    ((32, 9), (2, 16, 256, [40, 1], [2300, 1100])),
    ((32, 24), (1, 16, 256, [16], [9000])),
    ((16, 1), (8, 32, 64, [4, 1, 2], [700, 64, 65])),
    ((16, 1), (8, 32, 128, [4, 1, 2], [700, 64, 65])),
    ((16, 1), (8, 32, 256, [4, 1, 2], [700, 64, 65])),
    ((16, 16), (2, 16, 64, [2, 1], [4000, 1100])),
    ((16, 16), (2, 16, 128, [2, 1], [4000, 1100])),
    ((16, 16), (2, 16, 256, [2, 1], [4000, 1100])),
    ((16, 66), (1, 16, 64, [1], [16700])),
    ((16, 66), (1, 16, 128, [1], [16700])),
    ((16, 66), (1, 16, 256, [1], [16700])),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("want,size", SIZES)
def test_causal(ctx, want, size, kind):
    G, H, D, n, lens = size
    cache = cache_for(lens, G, D, pad=16)
    seqs = U.Seqs(lens, n, cache.pages)
    q = U.Query(seqs.T, H, D, kind, pad=8)
    assert plan(G, H, D, n, seqs.max_kv)[:2] == want
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)
    first = q._out.clone(), q._lse.clone()
    U.attend(ctx, cache, q, seqs)
    assert torch.equal(first[0], q._out) and torch.equal(first[1], q._lse)
    assert ctx.invalid() == 0


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("want,G,H,D,n,lens", [
    ((64, 1), 8, 32, 128, [64] * 15 + [61], [3000, 64, 100, 700] * 4), ((64, 1), 8, 32, 128, [256] * 4, [4900, 256, 300, 2500]),
    ((64, 1), 16, 64, 64, [64] * 15 + [61], [1000, 64, 100, 700] * 4), ((32, 2), 8, 32, 128, [24] * 7 + [21], [2500, 24, 100, 700] * 2),
    ((32, 4), 4, 16, 256, [70, 33], [2500, 90])])
def test_trees(ctx, want, G, H, D, n, lens, kind):
    """Nodes that see what lies before the tree alone, one that sees nothing, nodes beyond the mask's words."""
    tree = U.random_tree(n, -(-max(n) // 64), sum(n))
    tree[3], tree[n[0] + 1] = 0, 0
    cache = cache_for(lens, G, D)
    seqs = U.Seqs(lens, n, cache.pages, tree=tree)
    q = U.Query(seqs.T, H, D, kind)
    assert plan(G, H, D, n, seqs.max_kv)[:2] == want
    U.attend(ctx, cache, q, seqs)
    U.check_all(cache, q, seqs)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("want,G,H,D,n,lens", [
    ((64, 1), 8, 32, 128, [600, 520], [600, 1000]), ((64, 1), 8, 32, 128, [256] * 4, [4500, 256, 300, 2500]),
    ((64, 1), 16, 64, 64, [1200, 1100], [1200, 1163]), ((32, 1), 8, 32, 128, [130, 120], [200, 400]), ((32, 4), 4, 16, 256, [70, 33], [2500, 90])])
def test_bad_pages_and_hidden_nan_codes(ctx, want, G, H, D, n, lens, kind):
    """A page that is not there in the middle and at the end of a sequence, and a position whose codes are NaN among the
    new ones: who does not see it has the formula's result."""
    for tree in (None, U.random_tree(n, -(-max(n) // 64), 3) if max(n) <= 4096 else None):
        cache = cache_for(lens, G, D)
        seqs = U.Seqs(lens, n, cache.pages, tree=tree)
        table = seqs.table.copy()
        table[0, 1], table[1, -(-lens[1] // 64) - 1] = cache.pages, -1
        seqs = U.Seqs(lens, n, cache.pages, table=table, tree=tree)
        # a position of the last sequence's new tokens, which the earlier ones do not see
        b = len(n) - 1
        hidden = lens[b] - n[b] // 2
        if table[b, hidden // 64] < 0:
            hidden = lens[b] // 64 * 64 - 5
        for i in (0, 1):
            cache.codes(0)[int(table[b, hidden // 64]), :, i, hidden % 64] = (0x7F, 0xFF)[i]
        q = U.Query(seqs.T, H, D, kind)
        assert plan(G, H, D, n, seqs.max_kv)[:2] == want
        U.attend(ctx, cache, q, seqs)
        assert ctx.invalid() == 2
        for k in range(len(n)):
            a, m, kv = int(seqs.start[k]), n[k], lens[k]
            vals, ok = cache.values(0, table[k, :-(-kv // 64)], kv)
            seen = torch.as_tensor(seqs.seen(k), device="cuda") & ok[None]
            ref = U.reference(q.q[a:a + m], vals, seen, q.scale)
            clean = np.ones(m, bool) if k != b else ~seqs.seen(k)[:, hidden]
            assert clean.any() and (k != b or not clean.all())
            for lo, hi in runs(clean):
                U.check_rows(q, a + lo, a + hi, [x[lo:hi] for x in ref], f"sequence {k} tokens {lo} to {hi}")
            assert bool(torch.isnan(q.out[a:a + m][torch.as_tensor(~clean, device="cuda")]).all())
        q.untouched(range(seqs.T))


def runs(mask):
    """[first, end) of the runs of true values."""
    edges = np.flatnonzero(np.diff(np.r_[0, mask.astype(np.int8), 0]))
    return list(zip(edges[::2].tolist(), edges[1::2].tolist()))


def test_units_of_64_rows_stay_whole(ctx):
    """512 blocks of them give the bits that the same tokens have in a call of more blocks."""
    G, H, D, n, lens = 8, 32, 128, [256] * 4, [5000, 256, 4100, 2500]
    cache = cache_for(lens + [64], G, D)
    few = U.Seqs(lens, n, cache.pages, seed=1)
    table = np.concatenate([few.table, np.full((1, few.table.shape[1]), cache.pages - 1, np.int32)])
    more = U.Seqs(lens + [64], n + [64], cache.pages, table=table)
    assert plan(G, H, D, few.n, few.max_kv) == (64, 1, 512) and plan(G, H, D, more.n, more.max_kv)[0] == 64
    a, b = U.Query(few.T, H, D), U.Query(more.T, H, D)
    b.q[:few.T] = a.q
    U.attend(ctx, cache, a, few)
    U.attend(ctx, cache, b, more)
    assert torch.equal(a.out, b.out[:few.T]) and torch.equal(a.lse, b.lse[:few.T])
