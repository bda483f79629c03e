"""The calls that read a published cache, and the eviction, in a layer that lies
beyond 2^32 bytes and spans more than that itself: rows of its first and last pages."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub, workloads as W

import attend_util as A
import gpu_util as G
from test_gpu_attend import check_weights
from test_gpu_evict import plain_kept

pytestmark = pytest.mark.gpu

PAGES = 103_000
USED = np.concatenate([np.arange(0, 30), np.arange(PAGES - 50, PAGES)])      # page numbers with stored rows
assert (PAGES - 50) * W.MAIN_PAGE > 1 << 32


@pytest.fixture(scope="module")
def cache():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    kvpub.load()
    G.log("caches of two layers of 103,000 pages")
    slots = (USED[:, None] * 64 + np.arange(64)).reshape(-1)
    c = A.Cache(PAGES, seed=51, replicas=1, written=slots, guard=64)
    yield c
    c.free()
    torch.cuda.empty_cache()


def paged(cache, lens, n, seed):
    """Sequences over disjoint used pages, most of them from the end."""
    width = -(-max(lens) // 64)
    pg = A.Paged(cache, [1], [1])
    order = np.random.default_rng(seed).permutation(USED)
    pg.lens, pg.n, pg.max_kv = np.asarray(lens, np.int64), np.asarray(n, np.int64), max(lens)
    pg.table = order[:len(lens) * width].reshape(len(lens), width).astype(np.int32)
    pg.start = np.concatenate([[0], np.cumsum(pg.n)])
    pg.T = int(pg.start[-1])
    pg.d_len, pg.d_table, pg.d_start = A.dev_i32(pg.lens), A.dev_i32(pg.table), A.dev_i32(pg.start)
    pg.struct = kvpub.pages(pg.d_len.data_ptr(), pg.d_table.data_ptr(), width, len(lens), pg.max_kv,
                            q_start=pg.d_start.data_ptr(), max_q_len=int(pg.n.max()))
    pg.left = order[len(lens) * width:]
    return pg


@pytest.mark.parametrize("heads,lens,n", [(16, [700], [1]), (64, [900, 333, 64], [1, 3, 1]), (128, [2500, 1000], [20, 9])])
def test_attend_and_weights(cache, heads, lens, n):
    pg = paged(cache, lens, n, heads)
    q, o = A.Queries(pg.T, heads, seed=heads), A.Outputs(pg.T, heads)
    A.attend(cache, q, pg, o, replica=0)
    A.check_paged(cache, q, pg, o, replica=0)
    w = torch.full((len(lens), pg.max_kv), A.SENTINEL, device="cuda")
    kvpub.check(kvpub.kvpub_attend_weights(cache.ctx, 0, cache.layer, q.struct, pg.struct, *o.args()[3:], None, w.data_ptr(),
                                           pg.max_kv, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    check_weights(cache, q, pg, o.lse, None, w, replica=0)
    assert cache.invalid() == 0


@pytest.mark.parametrize("heads,tokens,width", [(16, 3, 700), (128, 16, 2048), (128, 60, 2048)])
def test_slots(cache, heads, tokens, width):
    slots = np.random.default_rng(heads + tokens).choice(USED, (tokens, width)).astype(np.int64) * 64
    slots += np.random.default_rng(1).integers(0, 64, slots.shape)
    d = torch.from_numpy(slots).cuda()
    q, o = A.Queries(tokens, heads), A.Outputs(tokens, heads)
    size = kvpub.kvpub_attend_slots_workspace(q.struct, width)
    buf, ws = A.workspace(size)
    kvpub.check(kvpub.kvpub_attend_slots(cache.ctx, 0, cache.layer, q.struct, d.data_ptr(), width, width, *o.args(), ws, size,
                                         torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    A.guards_whole(buf)
    assert cache.invalid() == 0
    for t in range(tokens):
        c, r = cache.values(0, slots[t])
        want = A.reference(q.latent[t:t + 1], q.rope[t:t + 1], q.scale, c, r, torch.ones(1, width, dtype=torch.bool, device="cuda"))
        A.check_rows(o.out[t:t + 1], o.lse[t:t + 1], want, f"token {t}")


@pytest.mark.parametrize("in_place", [False, True])
def test_evict(cache, in_place):
    lens, budget, first, last = [1000, 700], 300, 4, 30
    pg = paged(cache, lens, [1, 1], 7)
    L, layer, main, idx = cache.layout, cache.layer, cache.dev.main[0], cache.dev.idx[0]
    dst = pg.table if in_place else pg.left[:10].reshape(2, 5).astype(np.int32)
    d_dst = pg.d_table if in_place else A.dev_i32(dst)
    host = np.random.default_rng(3).random((2, 1000)).astype(np.float32)
    w = torch.from_numpy(host).cuda()
    w_out = w if in_place else torch.empty_like(w)
    kept, new = torch.zeros(2, budget, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    io = kvpub.evict_io(w.data_ptr(), w_out.data_ptr(), 1000, pg.d_len.data_ptr(), pg.d_table.data_ptr(), pg.table.shape[1],
                        d_dst.data_ptr(), dst.shape[1], kept.data_ptr(), budget, new.data_ptr(), 2, 1000, budget, first, last)
    m0, i0 = main.clone(), idx.clone()
    want_m, want_i = main.clone(), idx.clone()
    for b, n in enumerate(lens):
        ks = plain_kept(host[b], n, budget, first, last)
        for i, p in enumerate(ks):
            s = layer * L.main_layer_stride + int(pg.table[b, p // 64]) * L.main_page_stride + int(p % 64) * 656
            d = layer * L.main_layer_stride + int(dst[b, i // 64]) * L.main_page_stride + (i % 64) * 656
            want_m[d:d + 656] = m0[s:s + 656]
            s = layer * L.idx_layer_stride + int(pg.table[b, p // 64]) * L.idx_page_stride
            d = layer * L.idx_layer_stride + int(dst[b, i // 64]) * L.idx_page_stride
            a, z = int(p % 64), i % 64
            want_i[d + z * 128:d + z * 128 + 128] = i0[s + a * 128:s + a * 128 + 128]
            want_i[d + 8192 + z * 4:d + 8196 + z * 4] = i0[s + 8192 + a * 4:s + 8196 + a * 4]
    size = kvpub.kvpub_evict_workspace(io)
    buf, ws = A.workspace(size)
    kvpub.check(kvpub.kvpub_evict(cache.ctx, layer, io, ws, size, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    A.guards_whole(buf)
    try:
        for b, n in enumerate(lens):
            ks = plain_kept(host[b], n, budget, first, last)
            assert np.array_equal(kept[b].cpu().numpy(), ks) and int(new[b]) == budget
            assert np.array_equal(w_out[b, :budget].cpu().numpy(), host[b, ks]) and bool((w_out[b, budget:] == 0).all())
        assert torch.equal(main, want_m) and torch.equal(idx, want_i)
        assert cache.invalid() == 0
    finally:
        main.copy_(m0)
        idx.copy_(i0)
