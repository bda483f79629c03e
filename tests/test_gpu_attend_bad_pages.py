"""Bad page numbers in the reading calls: kvpub_attend and kvpub_attend_weights hide
their positions and count each once a call, if some token of the call would have
seen a position of it."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import attend_util as A
import gpu_util as G
from test_gpu_attend_bounds import pages_shared
from test_gpu_attend_long import long_pages

pytestmark = pytest.mark.gpu

I32 = np.iinfo(np.int32)


@pytest.fixture(scope="module")
def cache():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    kvpub.load()
    c = A.Cache(160, seed=31)
    yield c
    c.free()
    torch.cuda.empty_cache()


def good(cache, pg, b):
    """Which positions of sequence b lie on a page of the context."""
    page = pg.table[b, np.arange(int(pg.lens[b])) // 64]
    return (page >= 0) & (page < cache.pages)


def expected_count(cache, pg, max_q):
    """Bad tiles of which some computed token sees a position."""
    count = 0
    for b in range(len(pg.lens)):
        m = min(int(pg.n[b]), max_q)
        if m == 0 or pg.lens[b] == 0:
            continue
        hidden = pg.seen(b)[:m].cpu().numpy().any(0) & ~good(cache, pg, b)
        count += len(set(np.flatnonzero(hidden) // 64))
    return count


def check(cache, q, pg, max_q):
    """attend and weights: outputs, sums and both counts."""
    o = A.Outputs(pg.T, q.H)
    cache.invalid()
    A.attend(cache, q, pg, o)
    want = expected_count(cache, pg, max_q)
    assert cache.invalid() == want
    g = torch.Generator(device="cuda").manual_seed(3)
    w_in = torch.rand((len(pg.lens), pg.max_kv), generator=g, device="cuda")
    w_out = torch.full_like(w_in, A.SENTINEL)
    kvpub.check(kvpub.kvpub_attend_weights(cache.ctx, 1, cache.layer, q.struct, pg.struct, *o.args()[3:], w_in.data_ptr(),
                                           w_out.data_ptr(), pg.max_kv, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert cache.invalid() == want
    for b in range(len(pg.lens)):
        a, kv, m = int(pg.start[b]), int(pg.lens[b]), min(int(pg.n[b]), max_q)
        if m == 0 or kv == 0:
            assert torch.equal(w_out[b], w_in[b])
            continue
        ok = good(cache, pg, b)
        p = np.arange(kv)
        c, r = cache.values(1, np.where(ok, pg.table[b, p // 64].astype(np.int64) * 64 + p % 64, 0))
        seen = pg.seen(b)[:m] & torch.from_numpy(ok).cuda()
        ref = A.reference(q.latent[a:a + m], q.rope[a:a + m], q.scale, c, r, seen)
        A.check_rows(o.out[a:a + m], o.lse[a:a + m], ref, f"sequence {b}")
        # sums: a score is off by at most 600 roundings, and so is the lse (attend_util.check_rows); m * H terms
        _, l, w, size, _ = ref
        total = w.sum((0, 1))
        alive = l[~torch.isinf(l)]
        rel = 2 * (600 * 2.0 ** -24 * size.max().item() + 2.0 ** -20 * (4 + (alive.abs().max().item() if alive.numel() else 0)))
        tol = (rel * 1.1 + (m * q.H + 16) * 2.0 ** -24) * total + 2.0 ** -23 * (total + 1)
        assert bool(((w_out[b, :kv].double() - w_in[b, :kv].double() - total).abs() <= tol).all()), f"sequence {b}: weights"
        gone = torch.from_numpy(np.concatenate([~ok, np.ones(pg.max_kv - kv, bool)])).cuda()
        assert torch.equal(w_out[b][gone], w_in[b][gone]), f"sequence {b}: weights of positions that are not there"


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("heads,lens,n", [
    (16, [300, 640], [10, 3]),
    (128, [300, 640], [3, 1]),                  # weights: several passes of 128 rows over a tile
    (5, [64, 200, 0], [64, 1, 1]),
])
def test_inside_the_lengths(cache, heads, lens, n, long):
    G.log(f"bad pages H={heads} lens={lens} n={n} long={long}")
    pg = long_pages(cache, lens, n, heads) if long else A.Paged(cache, lens, n)
    pg.table[0, 0], pg.table[1, 1], pg.table[1, -(-lens[1] // 64) - 1] = -1, cache.pages, I32.min
    pg.d_table.copy_(A.dev_i32(pg.table))
    check(cache, A.Queries(pg.T, heads), pg, max(n))


@pytest.mark.parametrize("seqs", [64, 65, 200])
@pytest.mark.parametrize("heads", [16, 128])
def test_of_many_sequences(cache, seqs, heads):
    G.log(f"bad pages of {seqs} sequences H={heads}")
    rng = np.random.default_rng(seqs)
    lens, n = rng.integers(0, 200, seqs), rng.integers(0, 3, seqs)
    lens[3], n[3], lens[-1], n[-1] = 199, 2, 130, 1
    pg = pages_shared(cache, lens, n)
    rng = np.random.default_rng(1)
    for b in range(0, seqs, 3):
        pg.table[b, rng.integers(0, pg.table.shape[1])] = [-1, cache.pages, I32.min, I32.max][b % 4]
    pg.table[-1, :3] = -1                       # a sequence with no page at all
    pg.d_table.copy_(A.dev_i32(pg.table))
    check(cache, A.Queries(pg.T, heads), pg, int(max(n)))


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("heads,max_q", [(16, 80), (16, 20), (3, 1)])
def test_drafted_positions(cache, heads, max_q, long):
    """200 positions, 80 of them drafted: a bad tile of drafted nodes counts if some node that is computed sees one of them."""
    G.log(f"bad pages of drafted positions H={heads} max_q={max_q} long={long}")
    lens, n = [200, 200, 64], [80, 80, 10]
    pg = long_pages(cache, lens, n, heads, tree_words=2) if long else A.Paged(cache, lens, n, tree_words=2)
    pg.struct.max_q_len = max_q
    pg.tree[:80, 0] &= np.uint64(0xFF)          # of the first sequence only nodes 0..7 (positions 120..127) are seen
    pg.tree[:80, 1] = 0
    pg.tree[160:170] = 0                        # of the third nothing but the context
    pg.d_tree.copy_(torch.from_numpy(pg.tree.view(np.int64)))
    pg.table[0, 2:4] = -1                       # positions 128..199: nobody sees one
    pg.table[1, 2:4] = cache.pages              # the same, seen by their nodes
    pg.table[2, 0] = -5
    pg.d_table.copy_(A.dev_i32(pg.table))
    check(cache, A.Queries(pg.T, heads), pg, max_q)


@pytest.mark.parametrize("heads", [16, 128])
def test_chunks_beyond_max_q_len(cache, heads):
    """Of a chunk of 100 tokens 30 are computed: the last positions are seen by none of them."""
    pg = A.Paged(cache, [250, 250], [100, 30], max_q=30)
    pg.table[0, 3], pg.table[1, 3] = -1, -1     # positions 192..249; the 30th token of the first sees 0..179
    pg.d_table.copy_(A.dev_i32(pg.table))
    check(cache, A.Queries(pg.T, heads), pg, 30)
