"""kvpub_attend_expanded where max_q_len is far above most sequences' tokens: one long
prompt among single tokens, and bounds that no sequence reaches.  Past twice the
tokens' own tiles the grid goes by tokens; these calls take that form unless they say so."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import attend_util as A
import gpu_util as G
from test_gpu_expanded import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    kvpub.load()
    c = A.Cache(1, replicas=1, layers=1, layer=0)
    yield c.ctx
    c.free()
    torch.cuda.empty_cache()


def by_tokens(c):
    """The rule of the launch: padded tiles against the places that the tokens need."""
    tiles = -(-min(c.io.max_q_len, c.io.num_tokens) // 128)
    return c.io.num_seqs * tiles > 2 * (c.io.num_tokens // 128 + c.io.num_seqs)


CASES = [
    # tokens and keys of each sequence, heads
    ([1] * 5 + [1000] + [1] * 60, [3] * 5 + [1100] + [70] * 60, 3),
    ([0] * 70 + [513] + [1, 0, 127, 128, 129] * 10, [5] * 70 + [513] + [1, 2, 127, 300, 129] * 10, 2),
    ([700] + [1] * 64, [700] + [65] * 64, 16),
    ([1] * 300 + [1300], [1] * 300 + [1300], 1),            # the longest one last, more than 256 sequences
    ([0] * 200 + [40], [0] * 200 + [50], 5),
]


@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("n,m,H", CASES)
def test_one_long_prompt_among_short_ones(ctx, n, m, H, causal):
    G.log(f"expanded by tokens: {len(n)} sequences, {sum(n)} tokens, H={H} causal={causal}")
    c = Case(n, m, H, causal, seed=sum(n), max_q=2 ** 32 - 1)
    assert by_tokens(c) or sum(n) < 128
    c.run(ctx)
    c.check()
    c.o.untouched(range(sum(n)))


def test_tokens_before_the_first_sequence_and_beyond_max_q_len_are_left(ctx):
    """The call's sequences begin at token 300; of 400 tokens 260 are computed."""
    n, m = [300, 400] + [1] * 40, [10, 450] + [3] * 40
    c = Case(n, m, 2, seed=8, max_q=260)
    c.io.q_start += 4
    c.io.k_start += 4
    c.io.num_seqs -= 1
    assert by_tokens(c)
    c.run(ctx)
    whole = Case(n, m, 2, seed=8)
    whole.run(ctx)
    whole.check()
    for a, z in ((300, 560), (700, 740)):
        assert torch.equal(c.o.out[a:z], whole.o.out[a:z]) and torch.equal(c.o.lse[a:z], whole.o.lse[a:z])
    c.o.untouched(list(range(300, 560)) + list(range(700, 740)))


def test_the_time_goes_by_the_tokens_not_by_the_bounds(ctx):
    """65535 sequences of one token, any of which might hold all by the bound: 5e8 blocks of the padded form,
    seconds; what is there is 65535 tokens of 16 heads over three keys each."""
    seqs, H = 65535, 16
    G.log(f"expanded {seqs} sequences, loose max_q_len")
    c = Case([1] * seqs, [3] * seqs, H, seed=1, max_q=2 ** 32 - 1)
    assert by_tokens(c)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    kvpub.check(kvpub.kvpub_attend_expanded(ctx, c.io, torch.cuda.current_stream().cuda_stream))
    end.record()
    torch.cuda.synchronize()
    ms = begin.elapsed_time(end)
    G.log(f"{ms:.2f} ms")
    assert ms < 1000
    k = torch.cat([c.kn.double(), c.kr.double()[:, None].expand(-1, H, -1)], 2).view(seqs, 3, H, 192)
    q = torch.cat([c.qn.double(), c.qr.double()], 2)[:, None]
    x = (q * k).sum(-1) * c.scale                                                  # [sequence, key, head]
    size = ((q * k).abs().sum(-1) * c.scale).amax(1)
    lse = torch.logsumexp(x, 1)
    w = torch.exp(x - lse[:, None])[..., None]
    v = c.v.double().view(seqs, 3, H, 128)
    out, mass = (w * v).sum(1), (w * v.abs()).sum(1)
    # the bounds of Case.check
    tol_l = 220 * 2.0 ** -24 * size + 2.0 ** -20 * (1 + lse.abs())
    assert bool(((c.o.lse.double() - lse).abs() <= tol_l).all())
    tol_o = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * tol_l[..., None]) * mass * 1.01 + 1e-30
    assert bool(((c.o.out.double() - out).abs() <= tol_o).all())
    c.o.untouched(range(seqs))


def test_one_sequence_with_all_tokens_by_its_bound(ctx):
    """2^24 tokens by the bound, 130 there, 128 heads: 2^24 blocks of the padded form, two launches."""
    c = Case([130], [200], 128, seed=2)
    c.io.num_tokens = c.io.max_q_len = 1 << 24       # no row behind the sequence's is touched
    assert not by_tokens(c)
    c.run(ctx)
    c.check()
    c.o.untouched(range(130))
