"""kvpub_attend_expanded against a plain form in 64 bits."""
import math

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
def ctx(_gpu):
    c = A.Cache(1, replicas=1, layers=1, layer=0)
    yield c.ctx
    c.free()


class Case:
    def __init__(self, n, m, H, causal=1, interleaved=True, pad=0, seed=0, scale=1 / math.sqrt(192), mag=1.0, max_q=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.n, self.m, self.H, self.causal, self.scale = n, m, H, causal, scale
        self.qs, self.ks = np.concatenate([[0], np.cumsum(n)]), np.concatenate([[0], np.cumsum(m)])
        T, U = int(self.qs[-1]), int(self.ks[-1])
        rnd = lambda *s: (mag * torch.randn(s, generator=g, device="cuda")).bfloat16()
        self._qn, self._qr = rnd(max(T, 1), H, 128 + pad), rnd(max(T, 1), H, 64 + pad)
        self._kr = rnd(max(U, 1), 64 + pad)
        if interleaved:
            self._kv = rnd(max(U, 1), H, 256 + pad)
            self.kn, self.v = self._kv[..., :128], self._kv[..., 128:256]
        else:
            self._kn, self._v = rnd(max(U, 1), H, 128 + pad), rnd(max(U, 1), H, 128 + pad)
            self.kn, self.v = self._kn[..., :128], self._v[..., :128]
        self.qn, self.qr, self.kr = self._qn[..., :128], self._qr[..., :64], self._kr[:, :64]
        self.o = A.Outputs(T, H, width=128, pad=pad)
        self.d_qs, self.d_ks = A.dev_i32(self.qs), A.dev_i32(self.ks)
        io = kvpub.expanded_io(0, 0, 0, 0, 0, 0, 0, self.d_qs.data_ptr(), self.d_ks.data_ptr(), len(n), H, T, U,
                               max(1, max(n)) if max_q is None else max_q, scale, causal=causal)
        io.q_nope, io.q_rope, io.k_nope = self._qn.data_ptr(), self._qr.data_ptr(), self.kn.data_ptr()
        io.k_rope, io.v = self._kr.data_ptr(), self.v.data_ptr()
        io.q_nope_token_stride, io.q_nope_head_stride = H * (128 + pad), 128 + pad
        io.q_rope_token_stride, io.q_rope_head_stride = H * (64 + pad), 64 + pad
        io.k_nope_token_stride, io.k_nope_head_stride = self.kn.stride(0), self.kn.stride(1)
        io.v_token_stride, io.v_head_stride = self.v.stride(0), self.v.stride(1)
        io.k_rope_token_stride = 64 + pad
        io.out, io.out_token_stride, io.out_head_stride, io.lse, io.lse_token_stride = self.o.args()
        self.io = io

    def run(self, ctx, stream=None):
        kvpub.check(kvpub.kvpub_attend_expanded(ctx, self.io, (stream or torch.cuda.current_stream()).cuda_stream),
                    "kvpub_attend_expanded")
        torch.cuda.synchronize()

    def seen(self, b):
        n, m = int(self.n[b]), int(self.m[b])
        p, i = np.arange(m), np.arange(n)[:, None]
        s = p[None] <= m - n + i if self.causal else np.ones((n, m), bool)
        return torch.from_numpy(s).cuda()

    def check(self, rows=None):
        """Bounds as in attend_util.check_rows, with 192 terms in a score and bf16 weights."""
        for b in range(len(self.n)):
            a, z, k0, k1 = int(self.qs[b]), int(self.qs[b + 1]), int(self.ks[b]), int(self.ks[b + 1])
            if a == z:
                continue
            seen = self.seen(b)
            for h in range(self.H):
                q = torch.cat([self.qn[a:z, h], self.qr[a:z, h]], 1).double()
                k = torch.cat([self.kn[k0:k1, h], self.kr[k0:k1]], 1).double()
                v = self.v[k0:k1, h].double()
                x = torch.where(seen, q @ k.T * self.scale, -math.inf)
                size = torch.where(seen, q.abs() @ k.abs().T * abs(self.scale), 0.0)
                lse = torch.logsumexp(x, 1) if k1 > k0 else torch.full((z - a,), -math.inf, dtype=torch.float64, device="cuda")
                dead = torch.isinf(lse)
                w = torch.where(seen & ~dead[:, None], torch.exp(x - torch.where(dead, 0.0, lse)[:, None]), 0.0)
                live = torch.where(seen.any(0)[:, None], v, 0.0)
                out, mass = w @ live, w @ live.abs()
                pick = slice(None) if rows is None else rows
                g_o, g_l = self.o.out[a:z, h].double()[pick], self.o.lse[a:z, h].double()[pick]
                out, mass, lse, dead = out[pick], mass[pick], lse[pick], dead[pick]
                tol_l = 220 * 2.0 ** -24 * (size[pick].amax(1) if k1 > k0 else 0) + 2.0 ** -20 * (1 + torch.where(dead, 0.0, lse).abs())
                assert torch.equal(torch.isinf(g_l), dead)
                err = torch.where(dead, 0.0, g_l - torch.where(dead, 0.0, lse)).abs()
                assert bool((err <= tol_l).all()), f"sequence {b} head {h}: lse off by {(err / tol_l).max().item()} of its bound"
                tol_o = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * tol_l[:, None]) * mass * 1.01 + 1e-30
                worst = ((g_o - out).abs() / tol_o).max().item()
                assert worst <= 1, f"sequence {b} head {h}: out off by {worst} of its bound"


@pytest.mark.parametrize("n,m,H,causal", [
    ([1], [1], 1, 1), ([100], [100], 16, 1), ([64], [64], 3, 1), ([128], [128], 2, 0), ([129], [300], 4, 1),
    ([257, 1, 64], [257, 65, 500], 5, 1), ([10, 0, 3], [0, 5, 3], 2, 1), ([50], [20], 2, 1), ([50], [20], 2, 0),
    ([1000], [1500], 2, 1), ([1], [1000], 8, 1), ([300, 300], [300, 700], 1, 0),
])
@pytest.mark.parametrize("interleaved,pad", [(True, 0), (False, 8)])
def test_expanded(ctx, n, m, H, causal, interleaved, pad):
    G.log(f"expanded n={n} m={m} H={H} causal={causal} interleaved={interleaved} pad={pad}")
    c = Case(n, m, H, causal, interleaved, pad, seed=sum(n))
    c.run(ctx)
    c.check()
    c.o.untouched(range(sum(n)))


@pytest.mark.parametrize("scale,mag", [(0.0, 1.0), (-0.2, 1.0), (1.0, 4.0), (0.07, 1e-20)])
def test_scales(ctx, scale, mag):
    c = Case([130], [200], 2, scale=scale, mag=mag)
    c.run(ctx)
    c.check()


def test_hidden_keys_may_hold_anything(ctx):
    """NaN and infinite keys and values after a token's own position leave it as it is."""
    c = Case([100], [150], 2, seed=3)
    for at, x in ((149, math.nan), (148, math.inf), (140, -math.inf)):
        c.v[at] = x
    c.kn[147], c.kr[146] = math.nan, math.inf
    c.run(ctx)
    clean = Case([100], [150], 2, seed=3)
    clean.run(ctx)
    assert torch.equal(c.o.out[:90], clean.o.out[:90]) and torch.equal(c.o.lse[:90], clean.o.lse[:90])
    clean.check()
    assert not bool(torch.isfinite(c.o.out[99]).any())


def test_tokens_beyond_max_q_len_are_left(ctx):
    c = Case([200, 5], [200, 50], 2, max_q=130)
    c.run(ctx)
    c.check(rows=slice(0, 5))
    c.o.untouched(list(range(130)) + list(range(200, 205)))


def test_captured_and_replayed(ctx):
    c = Case([150, 70], [200, 70], 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvpub.check(kvpub.kvpub_attend_expanded(ctx, c.io, torch.cuda.current_stream().cuda_stream))
    for k in range(3):
        fresh = Case([150, 70], [200, 70], 4, seed=k + 20)
        c._qn.copy_(fresh._qn)
        c._kv.copy_(fresh._kv)
        g.replay()
        torch.cuda.synchronize()
        c.check()


def test_the_two_forms_agree():
    """The absorbed form over the cache's rows and the expanded form over their
    projections are one operator: same lse, same outputs once projected."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    n, kv, H = 40, 200, 4
    c = A.Cache(4, seed=2)
    try:
        pg = A.Paged(c, [kv], [n])
        lat, rope = c.values(1, pg.slots(0))
        wk = torch.randn(H, 512, 128, generator=g, device="cuda", dtype=torch.float64) / 24
        wv = torch.randn(H, 512, 128, generator=g, device="cuda", dtype=torch.float64) / 24
        e = Case([n], [kv], H, interleaved=False)
        for h in range(H):
            e.kn[:, h], e.v[:, h] = (lat @ wk[h]).bfloat16(), (lat @ wv[h]).bfloat16()
        e.kr.copy_(rope.bfloat16())
        e.run(c.ctx)
        e.check()
        q, o = A.Queries(n, H), A.Outputs(n, H)
        for h in range(H):
            q.latent[:, h] = (e.qn[:, h].double() @ wk[h].T).bfloat16()
        q.rope.copy_(e.qr)
        A.attend(c, q, pg, o)
        # keys, absorbed queries and values are each rounded to bf16 once: a score is off by at
        # most 2^-8 of its terms' magnitudes twice, in the mean far less; 512 random terms of it
        # leave 2^-8 * sqrt(2) * |s| spread, well under 0.05 here
        assert (o.lse - e.o.lse).abs().max().item() < 0.05
        for h in range(H):
            a, b = o.out[:, h].double() @ wv[h], e.o.out[:, h].double()
            assert ((a - b).norm() / b.norm()).item() < 0.03
    finally:
        c.free()


def test_bounds_far_beyond_the_lengths(ctx):
    """2^17 tokens of which the sequences hold few, any of them by its bound in one of 1024 sequences: 2^24 blocks."""
    n, m = [3, 0, 130, 1] + [1] * 20 + [0] * 1000, [70, 5, 200, 1] + [2] * 1020
    c = Case(n, m, 16, seed=6)
    c.io.num_tokens = c.io.max_q_len = 1 << 17       # no row behind the sequences' is touched
    c.run(ctx)
    c.check()
    c.o.untouched(range(sum(n)))
