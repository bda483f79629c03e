"""kvpub_evict in place with pages outside the context's: every kept position whose
source or destination lies on one is left and counted, also one that does not move."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import attend_util as A
from test_gpu_evict import Eviction, expected, plain_kept

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    kvpub.load()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bad", [
    {(0, 0): -1},                               # positions 0..63 stay where they are
    {(0, 0): 99, (0, 3): np.iinfo(np.int32).min, (1, 1): np.iinfo(np.int32).max},
    {(1, 0): 32},                               # the first page behind the context's
])
def test_positions_on_bad_pages_are_counted(bad):
    lens, budget, first, last = [300, 100], 128, 100, 10      # the second sequence keeps all of its positions
    c = A.Cache(32, seed=1, replicas=2)
    try:
        w = np.random.default_rng(2).random((2, 305)).astype(np.float32)
        e = Eviction(c, lens, budget, first, last, True, w)
        for at, page in bad.items():
            e.table[at] = page
        e.d_table.copy_(A.dev_i32(e.table))
        kept = [plain_kept(w[b], n, budget, first, last) for b, n in enumerate(lens)]
        mains, idxs = expected(c, e.table, e.table, kept)
        e.run(c)
        e.check(kept)
        got_m, got_i = c.dev.host()
        for r in range(2):
            assert np.array_equal(got_m[r], mains[r]) and np.array_equal(got_i[r], idxs[r])
        wrong = lambda b, p: not 0 <= int(e.table[b, p // 64]) < c.pages
        assert c.invalid() == sum(wrong(b, p) or wrong(b, i) for b, ks in enumerate(kept) for i, p in enumerate(ks)) > 0
    finally:
        c.free()
