"""kvpub_evict while its context is poisoned: a fence that times out on another
stream sets the status at some moment of a run of evictions.  Whenever that is,
every sequence of every call is evicted whole or left as it was."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub, workloads as W
from replicated_fp8_sparse_amd.workloads import CacheLayout

import attend_util as A
import gpu_util as G
from test_gpu_evict import plain_kept

pytestmark = pytest.mark.gpu

CALLS, SEQS, LEN, BUDGET = 40, 64, 200, 100
SRC, DST = -(-LEN // 64), -(-BUDGET // 64)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    kvpub.load()
    yield
    torch.cuda.empty_cache()


def index_views(b, pages):
    a = b[:pages * W.IDX_PAGE].view(pages, W.IDX_PAGE)
    return a[:, :8192].view(pages, 64, 128), a[:, 8192:].view(torch.int32).view(pages, 64)


@pytest.mark.parametrize("in_place", [False, True])
def test_a_sequence_is_evicted_whole_or_left(in_place):
    pages = CALLS * SEQS * (SRC if in_place else SRC + DST)
    G.log(f"evict while the context is poisoned, in_place={in_place}, {pages} pages")
    layout = CacheLayout(replicas=1, layers=1, num_pages=pages)
    dev = G.DeviceCache(layout, participants=2, timeout_ns=200_000)        # no peer comes: the fence times out
    try:
        g = torch.Generator(device="cuda").manual_seed(5)
        main, idx = dev.main[0], dev.idx[0]
        for b in (main, idx):
            b.copy_(torch.randint(0, 256, b.shape, generator=g, device="cuda", dtype=torch.uint8))
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = order[:CALLS * SEQS * SRC].view(CALLS, SEQS, SRC)
        dst = table if in_place else order[CALLS * SEQS * SRC:].view(CALLS, SEQS, DST)
        w = torch.rand((CALLS, SEQS, LEN), generator=g, device="cuda")
        w_in, w_out = w.clone(), torch.full_like(w, A.SENTINEL)
        if in_place:
            w_out = w_in
        lens = torch.full((SEQS,), LEN, dtype=torch.int32, device="cuda")
        kept = torch.full((CALLS, SEQS, BUDGET), 77, dtype=torch.int32, device="cuda")
        new = torch.full((CALLS, SEQS), 77, dtype=torch.int32, device="cuda")
        ios = [kvpub.evict_io(w_in[k].data_ptr(), w_out[k].data_ptr(), LEN, lens.data_ptr(), table[k].data_ptr(), SRC,
                              dst[k].data_ptr(), dst.shape[2], kept[k].data_ptr(), BUDGET, new[k].data_ptr(), SEQS, LEN, BUDGET, 3, 5)
               for k in range(CALLS)]
        size = kvpub.kvpub_evict_workspace(ios[0])
        buf, ws = A.workspace(size)
        before = (main.clone(), idx.clone())
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        kvpub.check(dev.fence(0, side))
        s = torch.cuda.current_stream().cuda_stream
        for io in ios[:-1]:
            kvpub.check(kvpub.kvpub_evict(dev.ctx, 0, io, ws, size, s), "kvpub_evict")
        torch.cuda.synchronize()
        st, invalid, flags = dev.errors()
        assert st == kvpub.KVPUB_ERR_FENCE_TIMEOUT and flags & kvpub.KVPUB_FLAG_POISONED and invalid == 0
        kvpub.check(kvpub.kvpub_evict(dev.ctx, 0, ios[-1], ws, size, s), "kvpub_evict")       # behind the poison
        torch.cuda.synchronize()
        A.guards_whole(buf)

        done = (new == BUDGET).cpu().numpy()
        G.log(f"evicted {int(done.sum())} of {done.size} sequences, {int((done.any(1) & ~done.all(1)).sum())} calls in part")
        assert not done[-1].any()
        assert bool(((new == BUDGET) | (new == 77)).all())
        host = w.cpu().numpy()
        want_kept = np.full(kept.shape, 77, np.int32)
        want_w = w_in.new_full(w.shape, A.SENTINEL).cpu().numpy() if not in_place else host.copy()
        rows, codes, scales = main[:pages * W.MAIN_PAGE].view(-1, 656), *index_views(idx, pages)
        old_rows, old_codes, old_scales = before[0][:pages * W.MAIN_PAGE].view(-1, 656), *index_views(before[1], pages)
        want_rows, want_codes, want_scales = old_rows.clone(), old_codes.clone(), old_scales.clone()
        i = np.arange(BUDGET)
        for k, b in zip(*np.nonzero(done)):
            ks = plain_kept(host[k, b], LEN, BUDGET, 3, 5)
            want_kept[k, b] = ks
            want_w[k, b] = 0
            want_w[k, b, :BUDGET] = host[k, b, ks]
            at, to = torch.from_numpy(ks).cuda(), torch.from_numpy(i).cuda()
            ps, pd = table[k, b, at // 64].long(), dst[k, b, to // 64].long()
            want_rows[pd * 64 + to % 64] = old_rows[ps * 64 + at % 64]
            want_codes[pd, to % 64] = old_codes[ps, at % 64]
            want_scales[pd, to % 64] = old_scales[ps, at % 64]
        assert np.array_equal(kept.cpu().numpy(), want_kept)
        assert np.array_equal(w_out.cpu().numpy().view(np.uint32), want_w.view(np.uint32))
        assert torch.equal(rows, want_rows) and torch.equal(codes, want_codes) and torch.equal(scales, want_scales)
    finally:
        dev.free()
