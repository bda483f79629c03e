"""Helpers of the attention and eviction tests: caches written by kvpub_store,
calls through the C ABI, and plain forms in 64 bits computed from the bytes."""
import math

import numpy as np
import torch

from replicated_fp8_sparse_amd import kvpub, workloads as W
from replicated_fp8_sparse_amd.workloads import CacheLayout

import gpu_util as G

SENTINEL = 7.0


class Cache:
    """Replicas of a guarded layout; every slot of `layer` holds a stored row (or,
    with fill="nan", what was there: NaN codes, infinite scales and NaN RoPE values,
    except for the slots in `written`)."""

    def __init__(self, pages, seed=0, replicas=2, layers=2, layer=1, guard=64, written=None, spread=0.5):
        self.layout = CacheLayout(replicas=replicas, layers=layers, num_pages=pages, guard=guard)
        self.dev = G.DeviceCache(self.layout)
        self.ctx, self.layer, self.pages = self.dev.ctx, layer, pages
        rng = np.random.default_rng(seed)
        slots = np.arange(self.layout.capacity) if written is None else np.asarray(written)
        T = len(slots)
        if written is not None:
            for b in self.dev.main:     # 0xFF bytes: NaN codes, NaN scales, NaN RoPE values
                end = layers * self.layout.main_layer_stride
                b[:end].view(-1, self.layout.main_page_stride)[:, :W.MAIN_PAGE] = 0xFF
        mag = np.exp(spread * rng.standard_normal((T, 1))).astype(np.float32)
        x = W.LayerInputs(W.bf16_bits(rng.standard_normal((T, 512), dtype=np.float32) * mag),
                          W.bf16_bits(rng.standard_normal((T, 64), dtype=np.float32)),
                          W.bf16_bits(rng.standard_normal((T, 128), dtype=np.float32)), slots.astype(np.int64))
        kvpub.check(self.dev.store(layer, G.DeviceInputs(x)), "kvpub_store")
        torch.cuda.synchronize()

    def rows(self, replica):
        """Raw rows [slots, 656] of the layer."""
        L = self.layout
        a = self.dev.main[replica][self.layer * L.main_layer_stride:(self.layer + 1) * L.main_layer_stride]
        return a.view(L.num_pages, L.main_page_stride)[:, :W.MAIN_PAGE].reshape(-1, 656)

    def index_rows(self, replica):
        """(codes [slots, 128], scales [slots]) of the Indexer-K cache, raw."""
        L = self.layout
        a = self.dev.idx[replica][self.layer * L.idx_layer_stride:(self.layer + 1) * L.idx_layer_stride]
        a = a.view(L.num_pages, L.idx_page_stride)
        return a[:, :8192].reshape(-1, 128), a[:, 8192:8448].reshape(-1, 4).contiguous().view(torch.int32)[:, 0]

    def values(self, replica, slots):
        """Latent and RoPE values of slots, in 64 bits."""
        raw = self.rows(replica)[torch.as_tensor(slots, dtype=torch.int64, device="cuda")]
        codes = raw[:, :512].contiguous().view(torch.float8_e4m3fn).double().view(-1, 4, 128)
        scale = raw[:, 512:528].contiguous().view(torch.float32).double()
        return (codes * scale[:, :, None]).view(-1, 512), raw[:, 528:].contiguous().view(torch.bfloat16).double()

    def invalid(self, clear=True):
        st, n, _ = self.dev.errors(clear)
        kvpub.check(st)
        return n

    def free(self):
        self.dev.free()


def tables(seqs, width, pages, seed):
    """Disjoint random pages for each sequence."""
    assert seqs * width <= pages
    rng = np.random.default_rng(seed + 100)
    return rng.permutation(pages)[:seqs * width].reshape(seqs, width).astype(np.int32)


class Queries:
    """bf16 queries, `pad` extra values between rows and heads."""

    def __init__(self, T, H, seed=0, pad=0, scale=1 / math.sqrt(192), mag=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 17)
        self.T, self.H, self.scale = T, H, scale
        full = lambda w: (mag * torch.randn((max(T, 1), H, w + pad), generator=g, device="cuda")).bfloat16()
        self._l, self._r = full(512), full(64)
        self.latent, self.rope = self._l[:, :, :512], self._r[:, :, :64]
        self.struct = kvpub.queries(self._l.data_ptr(), self._r.data_ptr(), T, H, scale, H * (512 + pad), 512 + pad,
                                    H * (64 + pad), 64 + pad)


def dev_i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def reference(ql, qr, scale, c, r, seen):
    """One sequence: (out [n, H, 512], lse [n, H], w [n, H, P], bound of sum |terms| of a score [n, H])."""
    n, H, P = ql.shape[0], ql.shape[1], c.shape[0]
    q = torch.cat([ql.double(), qr.double()], 2).reshape(n * H, 576)
    k = torch.cat([c, r], 1)
    x = (q @ k.T * scale).view(n, H, P)
    size = (q.abs() @ k.abs().T * abs(scale)).view(n, H, P)
    # what is hidden may hold anything
    x = torch.where(seen[:, None], x, -math.inf)
    size = torch.where(seen[:, None], size, 0.0)
    top = x.amax(-1, keepdim=True) if P else torch.full((n, H, 1), -math.inf, dtype=torch.float64, device="cuda")
    ref = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(x - ref)
    total = e.sum(-1)
    lse = ref[..., 0] + torch.log(total)
    w = e / total.clamp(min=1e-300)[..., None]
    live = torch.where(seen.any(0)[:, None], c, 0.0) if P else c
    out = (w.reshape(n * H, P) @ live).view(n, H, 512)
    mass = (w.reshape(n * H, P) @ live.abs()).view(n, H, 512)
    return out, lse, w, (size.amax(-1) if P else torch.zeros(n, H, dtype=torch.float64, device="cuda")), mass


def check_rows(out, lse, want, what=""):
    """out and lse against `reference`.

    lse: a score is a binary32 sum of 576 exact products (and 4 products with a
    tile scale, one with the scale): at most 600 roundings of 2^-24 of the sum of
    the terms' magnitudes; the sum's and logarithm's own are within 2^-20.
    out: half a bf16 step of the result (2^-8), and of each weight times its
    tile scale (2^-8 of the sum of |w v|); a score's error e moves a weight by e."""
    o, l, _, size, mass = want
    tol_l = 600 * 2.0 ** -24 * size + 2.0 ** -20 * (1 + torch.where(torch.isinf(l), 0.0, l).abs())
    dead = torch.isinf(l)
    assert torch.equal(torch.isinf(lse), dead) and bool((lse[dead] < 0).all()), what
    worst = (torch.where(dead, 0.0, lse.double() - torch.where(dead, 0.0, l)).abs() / tol_l).max().item() if l.numel() else 0
    assert worst <= 1, f"{what}: lse off by {worst} of its bound"
    tol_o = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * tol_l[..., None]) * mass * 1.01 + 1e-30
    got = out.double()
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    worst = ((got - o).abs() / tol_o).max().item() if o.numel() else 0
    assert worst <= 1, f"{what}: out off by {worst} of its bound"


def visible(n, kv, tree=None):
    """[n, kv] of what the n newest positions see; tree: [n, words] uint64 or None."""
    base = kv - n
    p = np.arange(kv)
    if tree is None:
        return torch.from_numpy(p[None] <= base + np.arange(n)[:, None]).cuda()
    seen = np.zeros((n, kv), bool)
    for i in range(n):
        for x in range(kv):
            j = x - base
            seen[i, x] = j < 0 or (j < 64 * tree.shape[1] and bool((int(tree[i, j // 64]) >> (j % 64)) & 1))
    return torch.from_numpy(seen).cuda()


def random_tree(n, words, seed):
    rng = np.random.default_rng(seed)
    m = np.zeros((n, words), np.uint64)
    for i in range(n):
        if i:
            m[i] = m[rng.integers(max(0, i - 4), i)]
        if i < 64 * words:
            m[i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return m


class Outputs:
    def __init__(self, T, H, width=512, pad=0, extra=2):
        self.buf = torch.full((T + extra, H, width + pad), SENTINEL, dtype=torch.bfloat16, device="cuda")
        self.out = self.buf[:T, :, :width]
        self.lse_buf = torch.full((T + extra, H + 1), SENTINEL, device="cuda")
        self.lse = self.lse_buf[:T, :H]
        self.token, self.head, self.T, self.H, self.width = H * (width + pad), width + pad, T, H, width

    def args(self):
        return self.buf.data_ptr(), self.token, self.head, self.lse_buf.data_ptr(), self.H + 1

    def untouched(self, tokens):
        """Nothing but the rows of `tokens` was written."""
        rest = torch.ones(self.buf.shape[0], dtype=torch.bool, device="cuda")
        rest[torch.as_tensor(sorted(tokens), dtype=torch.int64, device="cuda")] = False
        assert bool((self.buf[rest] == SENTINEL).all()) and bool((self.lse_buf[rest] == SENTINEL).all())
        assert bool((self.buf[:, :, self.width:] == SENTINEL).all()) and bool((self.lse_buf[:, self.H:] == SENTINEL).all())


def workspace(size, guard=256):
    """A workspace of exactly `size` bytes between guard bytes."""
    buf = torch.full((size + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf, buf.data_ptr() + guard


def guards_whole(buf, guard=256):
    assert bool((buf[:guard] == 0xA5).all()) and bool((buf[-guard:] == 0xA5).all())


class Paged:
    """One call's pages: lengths, tokens and tables of the sequences."""

    def __init__(self, cache, lens, n, seed=0, tree_words=0, max_kv=None, max_q=None, one_each=False):
        self.lens, self.n = np.asarray(lens, np.int64), np.asarray(n, np.int64)
        B = len(lens)
        self.max_kv = int(max_kv if max_kv is not None else max(1, self.lens.max(initial=0)))
        width = max(1, -(-self.max_kv // 64))
        self.table = tables(B, width, cache.pages, seed)
        self.start = np.concatenate([[0], np.cumsum(self.n)])
        self.T = int(self.start[-1])
        self.tree = (np.concatenate([random_tree(int(k), tree_words, seed + b) for b, k in enumerate(self.n)])
                     if tree_words else None)
        self.d_len, self.d_table = dev_i32(self.lens), dev_i32(self.table)
        self.d_start = None if one_each else dev_i32(self.start)
        self.d_tree = torch.from_numpy(self.tree.view(np.int64)).cuda() if tree_words else None
        self.struct = kvpub.pages(self.d_len.data_ptr(), self.d_table.data_ptr(), width, B, self.max_kv,
                                  q_start=0 if one_each else self.d_start.data_ptr(),
                                  max_q_len=int(max_q if max_q is not None else max(1, self.n.max(initial=0))),
                                  tree_mask=0 if self.tree is None else self.d_tree.data_ptr(), tree_words=tree_words)

    def slots(self, b):
        p = np.arange(int(self.lens[b]))
        return self.table[b, p // 64].astype(np.int64) * 64 + p % 64

    def seen(self, b):
        tree = None if self.tree is None else self.tree[self.start[b]:self.start[b + 1]]
        return visible(int(self.n[b]), int(self.lens[b]), tree)


def attend(cache, q, pg, o, replica=1, stream=None):
    size = kvpub.kvpub_attend_workspace(q.struct, pg.struct)
    buf, ws = workspace(size)
    s = (stream or torch.cuda.current_stream()).cuda_stream
    kvpub.check(kvpub.kvpub_attend(cache.ctx, replica, cache.layer, q.struct, pg.struct, *o.args(), ws, size, s), "kvpub_attend")
    torch.cuda.synchronize()
    guards_whole(buf)


def check_paged(cache, q, pg, o, replica=1, what=""):
    for b in range(len(pg.lens)):
        a, z = int(pg.start[b]), int(pg.start[b + 1])
        if a == z:
            continue
        c, r = cache.values(replica, pg.slots(b))
        want = reference(q.latent[a:z], q.rope[a:z], q.scale, c, r, pg.seen(b))
        check_rows(o.out[a:z], o.lse[a:z], want, f"{what} sequence {b}")
