"""kvpub_attend and kvpub_attend_slots at sizes between the thresholds of their plan:
units of 16, 32 and 64 rows, slot lists and pages, up to and beyond 64 sequences (whose
prefix sums a block forms together).  Each case says which unit it is there for, and the
workspace's size shows that the library takes it."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import attend_util as A
import gpu_util as G
from test_gpu_attend_bounds import pages_shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cache():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    kvpub.load()
    c = A.Cache(160, seed=41)
    yield c
    c.free()
    torch.cuda.empty_cache()


def takes(size, rows):
    """256 blocks, each with a note of 20 bytes and two parts of `rows` rows: 512 values and their sum."""
    return size == 256 * (20 + 2 * rows * (512 + 1) * 4)


@pytest.mark.parametrize("heads,tokens,width,rows", [
    (16, 130, 200, 16),
    (128, 16, 2048, 32),
    (128, 5, 2048, 32),
    (100, 9, 1500, 32),
    (64, 12, 700, 32),
    (17, 64, 250, 32),
    (128, 40, 2048, 64),
    (128, 130, 640, 64),
    (33, 160, 2048, 64),
])
def test_slots(cache, heads, tokens, width, rows):
    """Full, short, empty and padded lists; bad and repeated slots."""
    G.log(f"slots H={heads} tokens={tokens} width={width} rows={rows}")
    rng = np.random.default_rng(heads + tokens)
    lists = rng.integers(0, width + 1, tokens)
    lists[:4] = [width, 0, 1, width - 1]
    cap = cache.layout.capacity
    slots = np.full((tokens, width + 1), -1, np.int64)
    for t, k in enumerate(lists):
        slots[t, rng.choice(width, size=k, replace=False)] = rng.integers(0, cap, k)      # some of them twice
    slots[:, width] = 3                                                                   # behind the list
    for t, i, bad in ((0, 0, cap), (0, 64, -2), (2, width - 1, 2 ** 62), (tokens - 1, 5, -2 ** 63)):
        slots[t, i] = bad
    d = torch.from_numpy(slots).cuda()
    q, o = A.Queries(tokens, heads, pad=8), A.Outputs(tokens, heads, pad=8)
    size = kvpub.kvpub_attend_slots_workspace(q.struct, width)
    assert takes(size, rows)
    buf, ws = A.workspace(size)
    cache.invalid()
    kvpub.check(kvpub.kvpub_attend_slots(cache.ctx, 1, cache.layer, q.struct, d.data_ptr(), width + 1, width, *o.args(), ws, size,
                                         torch.cuda.current_stream().cuda_stream), "kvpub_attend_slots")
    torch.cuda.synchronize()
    A.guards_whole(buf)
    assert cache.invalid() == 4
    for t in range(tokens):
        pick = slots[t, :width][(slots[t, :width] >= 0) & (slots[t, :width] < cap)]
        c, r = cache.values(1, pick)
        want = A.reference(q.latent[t:t + 1], q.rope[t:t + 1], q.scale, c, r, torch.ones(1, len(pick), dtype=torch.bool, device="cuda"))
        A.check_rows(o.out[t:t + 1], o.lse[t:t + 1], want, f"token {t}")
    o.untouched(range(tokens))


@pytest.mark.parametrize("heads,seqs,kv,most,rows", [
    (16, 65, 512, 1, 16),
    (64, 65, 130, 1, 32),
    (128, 80, 200, 1, 32),
    (64, 600, 64, 1, 32),
    (32, 100, 150, 3, 32),
    (128, 600, 320, 1, 64),
    (128, 65, 2000, 1, 64),
    (128, 80, 640, 2, 32),                      # 87 tokens: 2540 tiles of 64 rows, below ten a block
    (128, 80, 900, 2, 64),
    (40, 300, 500, 5, 64),
])
def test_many_sequences(cache, heads, seqs, kv, most, rows):
    """Ragged lengths and tokens, empty sequences and sequences without tokens among them."""
    G.log(f"attend H={heads} seqs={seqs} kv={kv} tokens up to {most} rows={rows}")
    rng = np.random.default_rng(heads + seqs)
    lens = rng.integers(0, kv + 1, seqs)
    n = np.ones(seqs, np.int64) if most == 1 else rng.integers(0, most + 1, seqs)
    lens[:3], n[:3] = [kv, 0, 1], [most, 1, 1]
    lens[-2:], n[-1] = [kv, 64], most
    pg = pages_shared(cache, lens, n)
    q, o = A.Queries(pg.T, heads, seed=heads), A.Outputs(pg.T, heads)
    assert takes(kvpub.kvpub_attend_workspace(q.struct, pg.struct), rows)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)
    o.untouched(range(pg.T))


@pytest.mark.parametrize("heads,seqs,kv,nodes,rows", [(16, 70, 100, 20, 32), (64, 66, 300, 10, 32), (64, 66, 600, 10, 64)])
def test_trees_of_many_sequences(cache, heads, seqs, kv, nodes, rows):
    G.log(f"tree H={heads} seqs={seqs} kv={kv} nodes={nodes} rows={rows}")
    rng = np.random.default_rng(seqs)
    lens, n = rng.integers(nodes, kv + 1, seqs), rng.integers(1, nodes + 1, seqs)
    lens[0], n[0] = kv, nodes
    pg = pages_shared(cache, lens, n)
    pg.tree = np.concatenate([A.random_tree(int(k), 1, b) for b, k in enumerate(pg.n)])
    pg.d_tree = torch.from_numpy(pg.tree.view(np.int64)).cuda()
    pg.struct.tree_mask, pg.struct.tree_words = pg.d_tree.data_ptr(), 1
    q, o = A.Queries(pg.T, heads, seed=heads), A.Outputs(pg.T, heads)
    assert takes(kvpub.kvpub_attend_workspace(q.struct, pg.struct), rows)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)
