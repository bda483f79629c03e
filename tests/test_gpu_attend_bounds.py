"""kvpub_attend where the call's bounds are far above what is there: one long chunk
among single tokens, and a max_q_len that no sequence reaches.  The bounds choose
kernels and sizes; the work goes by the sequences."""
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
    c = A.Cache(160, seed=23)
    yield c
    c.free()


@pytest.mark.parametrize("max_q", [None, 2 ** 32 - 1])
@pytest.mark.parametrize("heads", [5, 128])
def test_one_chunk_among_single_tokens(cache, heads, max_q):
    G.log(f"attend a chunk among single tokens H={heads} max_q={max_q}")
    lens, n = [100, 700, 0, 64] + [65, 30] * 16, [1, 230, 1, 0] + [1] * 32
    pg = pages_shared(cache, lens, n, max_q)
    q, o = A.Queries(pg.T + 1, heads, seed=heads), A.Outputs(pg.T + 1, heads)
    A.attend(cache, q, pg, o)
    A.check_paged(cache, q, pg, o)
    o.untouched(range(pg.T))


def pages_shared(cache, lens, n, max_q=None):
    """A.Paged with pages that several sequences share (they are only read)."""
    width = -(-max(lens) // 64)
    pg = A.Paged(cache, [1], [1])
    rng = np.random.default_rng(len(lens))
    pg.lens, pg.n, pg.max_kv = np.asarray(lens, np.int64), np.asarray(n, np.int64), width * 64
    pg.table = rng.integers(0, cache.pages, (len(lens), width)).astype(np.int32)
    pg.start = np.concatenate([[0], np.cumsum(pg.n)])
    pg.T = int(pg.start[-1])
    pg.d_len, pg.d_table, pg.d_start = A.dev_i32(pg.lens), A.dev_i32(pg.table), A.dev_i32(pg.start)
    pg.struct = kvpub.pages(pg.d_len.data_ptr(), pg.d_table.data_ptr(), width, len(lens), pg.max_kv,
                            q_start=pg.d_start.data_ptr(), max_q_len=int(max_q if max_q is not None else pg.n.max()))
    return pg


def test_the_time_goes_by_the_tokens_not_by_the_bounds(cache):
    """65536 sequences of one token and a bound that would allow each of them all tokens: 7e10 padded rows,
    seconds if anything walked them; what is there is 65536 tokens of 16 heads over one page each."""
    seqs, heads = 65536, 16
    G.log(f"attend {seqs} sequences, loose max_q_len")
    lens = np.random.default_rng(1).integers(0, 65, seqs)
    lens[-1] = 64
    pg = pages_shared(cache, lens, np.ones(seqs, np.int64), 2 ** 32 - 1)
    q, o = A.Queries(pg.T, heads, seed=3), A.Outputs(pg.T, heads)
    size = kvpub.kvpub_attend_workspace(q.struct, pg.struct)
    buf, ws = A.workspace(size)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    s = torch.cuda.current_stream().cuda_stream
    begin.record()
    kvpub.check(kvpub.kvpub_attend(cache.ctx, 1, cache.layer, q.struct, pg.struct, *o.args(), ws, size, s), "kvpub_attend")
    end.record()
    torch.cuda.synchronize()
    A.guards_whole(buf)
    ms = begin.elapsed_time(end)
    G.log(f"{ms:.2f} ms")
    assert ms < 1000
    for b in [0, 1, 2, 63, 64, 255, 256, 257, 40000, seqs - 2, seqs - 1]:
        c, r = cache.values(1, pg.slots(b))
        want = A.reference(q.latent[b:b + 1], q.rope[b:b + 1], q.scale, c, r, pg.seen(b))
        A.check_rows(o.out[b:b + 1], o.lse[b:b + 1], want, f"sequence {b}")
    empty = torch.from_numpy(lens == 0).cuda()
    assert bool((o.out[empty] == 0).all()) and bool(torch.isneginf(o.lse[empty]).all())
    assert bool(torch.isfinite(o.lse[~empty]).all())
