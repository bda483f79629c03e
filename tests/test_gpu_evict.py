"""kvpub_evict against a plain form: which positions stay, and every byte of
every replica (Main-KV, Indexer-K, guards), in place and into other pages."""
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


def plain_kept(w, n, budget, first, last):
    """The kept positions of one sequence, ascending."""
    if n <= budget:
        return np.arange(n)
    z = n - last
    v = np.where(np.isnan(w[first:z]), -np.inf, w[first:z]).astype(np.float64)
    nan = np.isnan(w[first:z])
    mid = np.lexsort((np.arange(len(v)), nan, -v))[:budget - first - last]     # a NaN behind -inf
    return np.sort(np.concatenate([np.arange(first), mid + first, np.arange(z, n)]))


def expected(cache, table, dst, kept):
    """Every buffer of the device cache after the moves, on the host."""
    L, layer = cache.layout, cache.layer
    mains, idxs = cache.dev.host()
    m0, i0 = mains[0].copy(), idxs[0].copy()
    for b, ks in enumerate(kept):
        for i, p in enumerate(ks):
            ps, pd = int(table[b, p // 64]), int(dst[b, i // 64])
            if not (0 <= ps < L.num_pages and 0 <= pd < L.num_pages):
                continue
            s = layer * L.main_layer_stride + ps * L.main_page_stride + (p % 64) * 656
            d = layer * L.main_layer_stride + pd * L.main_page_stride + (i % 64) * 656
            for m in mains:
                m[d:d + 656] = m0[s:s + 656]
            s = layer * L.idx_layer_stride + ps * L.idx_page_stride
            d = layer * L.idx_layer_stride + pd * L.idx_page_stride
            a, z = p % 64, i % 64
            for x in idxs:
                x[d + z * 128:d + z * 128 + 128] = i0[s + a * 128:s + a * 128 + 128]
                x[d + 8192 + z * 4:d + 8192 + z * 4 + 4] = i0[s + 8192 + a * 4:s + 8192 + a * 4 + 4]
    return mains, idxs


class Eviction:
    def __init__(self, cache, lens, budget, first, last, in_place, weights, seed=0, weights_in_place=None, max_kv=None):
        B = len(lens)
        self.max_kv = max_kv or max(1, max(lens))
        ws, wd = -(-self.max_kv // 64), -(-min(budget, self.max_kv) // 64)
        rng = np.random.default_rng(seed)
        pages = rng.permutation(cache.pages)
        self.table = pages[:B * ws].reshape(B, ws).astype(np.int32)
        self.dst = self.table if in_place else pages[B * ws:B * (ws + wd)].reshape(B, wd).astype(np.int32)
        self.lens, self.budget, self.first, self.last = lens, budget, first, last
        self.w = weights
        stride = weights.shape[1]
        self.d_w = torch.from_numpy(weights).cuda()
        own = in_place if weights_in_place is None else weights_in_place
        self.d_out = self.d_w if own else torch.full_like(self.d_w, A.SENTINEL)
        self.d_len, self.d_table = A.dev_i32(lens), A.dev_i32(self.table)
        self.d_dst = self.d_table if in_place else A.dev_i32(self.dst)
        self.d_kept = torch.full((B, budget + 3), 77, dtype=torch.int32, device="cuda")
        self.d_new = torch.full((B,), 77, dtype=torch.int32, device="cuda")
        self.io = kvpub.evict_io(self.d_w.data_ptr(), self.d_out.data_ptr(), stride, self.d_len.data_ptr(),
                                 self.d_table.data_ptr(), ws, self.d_dst.data_ptr(), ws if in_place else wd,
                                 self.d_kept.data_ptr(), budget + 3, self.d_new.data_ptr(), B, self.max_kv, budget, first, last)

    def run(self, cache, stream=None):
        size = kvpub.kvpub_evict_workspace(self.io)
        buf, ws = A.workspace(size)
        s = (stream or torch.cuda.current_stream()).cuda_stream
        kvpub.check(kvpub.kvpub_evict(cache.ctx, cache.layer, self.io, ws, size, s), "kvpub_evict")
        torch.cuda.synchronize()
        A.guards_whole(buf)

    def check(self, want_kept):
        kept, new, out = self.d_kept.cpu().numpy(), self.d_new.cpu().numpy(), self.d_out.cpu().numpy()
        for b, ks in enumerate(want_kept):
            assert new[b] == len(ks)
            assert np.array_equal(kept[b, :len(ks)], ks), f"sequence {b}"
            assert (kept[b, len(ks):self.budget] == -1).all() and (kept[b, self.budget:] == 77).all()
            assert np.array_equal(out[b, :len(ks)].view(np.uint32), self.w[b, ks].view(np.uint32))
            assert (out[b, len(ks):self.max_kv].view(np.uint32) == 0).all()
            edge = self.w[b, self.max_kv:] if self.d_out is self.d_w else np.full(self.w.shape[1] - self.max_kv, A.SENTINEL)
            assert np.array_equal(out[b, self.max_kv:], edge)


def run_case(pages, lens, budget, first, last, in_place, weights=None, seed=0, replicas=2, **kw):
    G.log(f"evict lens={lens} budget={budget} first={first} last={last} in_place={in_place}")
    c = A.Cache(pages, seed=seed, replicas=replicas)
    try:
        if weights is None:
            weights = np.exp(2 * np.random.default_rng(seed).standard_normal((len(lens), max(max(lens), 1) + 5))).astype(np.float32)
        e = Eviction(c, lens, budget, first, last, in_place, weights, seed=seed, **kw)
        kept = [plain_kept(weights[b], n, budget, first, last) for b, n in enumerate(lens)]
        mains, idxs = expected(c, e.table, e.dst, kept)
        e.run(c)
        e.check(kept)
        got_m, got_i = c.dev.host()
        for r in range(replicas):
            assert np.array_equal(got_m[r], mains[r]), G.describe_diff(got_m[r], mains[r], c.layout, "main")
            assert np.array_equal(got_i[r], idxs[r]), G.describe_diff(got_i[r], idxs[r], c.layout, "idx")
        assert c.invalid() == 0
    finally:
        c.free()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,budget,first,last", [
    ([1], 1, 0, 0),
    ([2], 1, 0, 0),
    ([2], 1, 0, 1),
    ([1000, 300], 256, 4, 64),
    ([500, 64, 65, 0, 256, 257], 64, 0, 0),
    ([700], 699, 3, 3),
    ([700], 64, 32, 32),                        # nothing of the middle stays
    ([640, 1000], 999, 0, 999),
    ([130], 500, 10, 10),                       # a budget above every length
])
def test_evict(lens, budget, first, last, in_place):
    run_case(64, lens, budget, first, last, in_place, seed=len(lens) + budget)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["ties", "zeros", "special", "negative", "rising", "falling"])
def test_weights_of_all_kinds(kind, in_place):
    n, rng = 900, np.random.default_rng(4)
    w = {"ties": rng.integers(0, 4, (1, n)), "zeros": np.where(rng.random((1, n)) < 0.5, 0.0, -0.0),
         "special": rng.choice([np.inf, -np.inf, np.nan, -np.nan, 0.0, -0.0, 1e-45, -1e-45, 3e38, 1.0], (1, n)),
         "negative": -np.exp(rng.standard_normal((1, n))), "rising": np.arange(n)[None], "falling": -np.arange(n)[None]}[kind]
    run_case(32, [n], 333, 5, 40, in_place, weights=w.astype(np.float32), replicas=1)


@pytest.mark.parametrize("in_place", [False, True])
def test_beyond_the_lds_copy(in_place):
    """33000 positions: the weights are read again for each digit."""
    run_case(1100, [33000], 20000, 16, 256, in_place, seed=2, replicas=1)


def test_weights_in_place_with_other_pages():
    run_case(48, [1000, 300], 256, 4, 64, False, seed=8, weights_in_place=True)


@pytest.mark.parametrize("lens,budget", [([20000, 6000], 15000), ([8000] * 6, 64)])
def test_weights_in_place_of_long_sequences_with_other_pages(lens, budget):
    """Weights that move down within their array while the rows go elsewhere: many blocks read what others overwrite."""
    most = max(lens)
    rising = np.linspace(0, 1, most + 5, dtype=np.float32)                    # the last ones stay: every weight moves far
    weights = np.stack([np.random.default_rng(b).permutation(rising) if b % 2 else rising for b in range(len(lens))])
    width = -(-most // 64) + -(-min(budget, most) // 64)
    run_case(width * len(lens), lens, budget, 0, 1, False, weights=weights, seed=4, replicas=1, weights_in_place=True)


def test_bad_pages_are_skipped_and_counted():
    c = A.Cache(32, seed=1, replicas=1)
    try:
        w = np.ones((1, 300), np.float32)
        e = Eviction(c, [300], 128, 0, 128, False, w)
        e.table[0, 4], e.dst[0, 0] = 99, -3      # positions 256..299 and destinations 0..63
        e.d_table.copy_(A.dev_i32(e.table))
        e.d_dst.copy_(A.dev_i32(e.dst))
        kept = [np.arange(172, 300)]
        mains, idxs = expected(c, e.table, e.dst, kept)
        e.run(c)
        e.check(kept)
        got_m, got_i = c.dev.host()
        assert np.array_equal(got_m[0], mains[0]) and np.array_equal(got_i[0], idxs[0])
        bad = sum(1 for i, p in enumerate(kept[0]) if p >= 256 or i < 64)
        assert c.invalid() == bad
    finally:
        c.free()


def test_lengths_are_clamped():
    c = A.Cache(32, seed=1, replicas=1)
    try:
        w = np.random.default_rng(0).random((2, 200)).astype(np.float32)
        e = Eviction(c, [200, 200], 100, 1, 1, False, w)
        e.d_len.copy_(A.dev_i32([10 ** 9, -4]))
        e.run(c)
        e.check([plain_kept(w[0], 200, 100, 1, 1), np.arange(0)])
    finally:
        c.free()


def test_a_captured_eviction_in_place_replayed():
    """Each replay evicts what the last one left, after the lengths and weights are set anew."""
    c = A.Cache(40, seed=6, replicas=2)
    try:
        lens, budget = [1000, 700], 300
        rng = np.random.default_rng(1)
        w = rng.random((2, 1000)).astype(np.float32)
        e = Eviction(c, lens, budget, 2, 30, True, w)
        size = kvpub.kvpub_evict_workspace(e.io)
        buf, ws = A.workspace(size)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvpub.check(kvpub.kvpub_evict(c.ctx, c.layer, e.io, ws, size, torch.cuda.current_stream().cuda_stream))
        for k in range(4):
            e.w = rng.random((2, 1000)).astype(np.float32)
            e.d_w.copy_(torch.from_numpy(e.w))
            e.d_len.copy_(A.dev_i32(lens))
            kept = [plain_kept(e.w[b], n, budget, 2, 30) for b, n in enumerate(lens)]
            mains, idxs = expected(c, e.table, e.dst, kept)
            g.replay()
            torch.cuda.synchronize()
            e.check(kept)
            got_m, got_i = c.dev.host()
            for r in range(2):
                assert np.array_equal(got_m[r], mains[r]) and np.array_equal(got_i[r], idxs[r])
            lens = [1000 - 100 * k, 301 + k]
    finally:
        c.free()


def test_store_attend_weigh_evict_attend():
    """The operators as they are used together: a sequence is attended, its weights
    accumulated over two steps, evicted to a budget in place, and attended again;
    what the kept positions held is what is attended then."""
    c = A.Cache(32, seed=12)
    try:
        pg = A.Paged(c, [900, 500], [1, 1], max_kv=900)
        w = torch.zeros(2, 900, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        for step in range(2):
            q, o = A.Queries(2, 16, seed=step), A.Outputs(2, 16)
            A.attend(c, q, pg, o)
            A.check_paged(c, q, pg, o)
            kvpub.check(kvpub.kvpub_attend_weights(c.ctx, 1, c.layer, q.struct, pg.struct, o.lse_buf.data_ptr(), 17,
                                                   w.data_ptr(), w.data_ptr(), 900, s))
        torch.cuda.synchronize()
        assert abs(w[0].double().sum().item() - 32) < 1e-3
        host = w.cpu().numpy()
        kept = [plain_kept(host[b], n, 256, 4, 32) for b, n in enumerate([900, 500])]
        before = [c.values(1, pg.slots(b)[kept[b]]) for b in range(2)]
        d_kept, d_new = torch.zeros(2, 256, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
        io = kvpub.evict_io(w.data_ptr(), w.data_ptr(), 900, pg.d_len.data_ptr(), pg.d_table.data_ptr(), pg.table.shape[1],
                            pg.d_table.data_ptr(), pg.table.shape[1], d_kept.data_ptr(), 256, d_new.data_ptr(), 2, 900, 256, 4, 32)
        buf, ws = A.workspace(kvpub.kvpub_evict_workspace(io))
        kvpub.check(kvpub.kvpub_evict(c.ctx, c.layer, io, ws, kvpub.kvpub_evict_workspace(io), s))
        pg.d_len.copy_(d_new)
        torch.cuda.synchronize()
        pg.lens = np.array([256, 256])
        for b in range(2):
            assert np.array_equal(d_kept[b].cpu().numpy(), kept[b])
            lat, rope = c.values(1, pg.slots(b))
            assert torch.equal(lat, before[b][0]) and torch.equal(rope, before[b][1])
        q, o = A.Queries(2, 16, seed=5), A.Outputs(2, 16)
        A.attend(c, q, pg, o)
        A.check_paged(c, q, pg, o)
    finally:
        c.free()
