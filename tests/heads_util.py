"""Helpers of the tests of rotations and of the cache of heads: plain forms in 64 bits."""
import math

import numpy as np
import torch

from replicated_fp8_sparse_amd import kvpub

TYPES = {"bf16": (torch.bfloat16, kvpub.BF16), "fp16": (torch.float16, kvpub.FP16), "fp32": (torch.float32, kvpub.FP32)}
SENTINEL = 7.0


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Context:
    """A context over one page of a latent cache: gives the device, the fail-closed state and the counter."""

    def __init__(self):
        self.main = torch.zeros(64 * 656, dtype=torch.uint8, device="cuda")
        self.idx = torch.zeros(64 * 132, dtype=torch.uint8, device="cuda")
        st, self.ctx = kvpub.kvpub_create(kvpub.kvpub_config_init(1, 1, 1), [self.main.data_ptr()], [self.idx.data_ptr()])
        kvpub.check(st, "kvpub_create")

    def invalid(self):
        st, n, _ = kvpub.kvpub_error_read(self.ctx, True)
        kvpub.check(st)
        return n

    def free(self):
        torch.cuda.synchronize()
        kvpub.check(kvpub.kvpub_destroy(self.ctx))


def stream():
    return torch.cuda.current_stream().cuda_stream


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Rotation:
    """A table of frequencies on the device, and the rotation in 64 bits by it."""

    def __init__(self, dim, start=0, halves=False, magnitude=1.0, base=10000.0, **config):
        st, self.turns = kvpub.kvpub_rotation_turns(kvpub.rotation_config(dim, base, **config))
        kvpub.check(st)
        self.table = torch.from_numpy(self.turns.view(np.int64)).cuda()
        self.dim, self.start, self.halves, self.magnitude = dim, start, halves, magnitude
        self.struct = kvpub.rotation(self.table.data_ptr(), dim, start, kvpub.ROTATE_HALVES if halves else kvpub.ROTATE_PAIRS, magnitude)

    def angles(self, positions):
        """Radians [token, pair] from whole numbers: position * turns modulo 2^64."""
        rows = [[(int(p) * int(t)) % 2 ** 64 for t in self.turns] for p in positions]
        turns = np.array([[(v - 2 ** 64 if v >= 2 ** 63 else v) / 2 ** 64 for v in r] for r in rows]).reshape(len(rows), -1)
        return torch.from_numpy(turns * 2 * math.pi)

    def parts(self):
        i = torch.arange(self.dim // 2)
        return (self.start + i, self.start + self.dim // 2 + i) if self.halves else (self.start + 2 * i, self.start + 2 * i + 1)

    def apply(self, x, positions, transpose=False):
        """(rotated x [token, head, width] in 64 bits on the host, bound of the error before the last rounding).

        Sine and cosine: 2^-32 turns of angle (2^-29.3 in the value), 2^-29 of polynomial, a rest below 0.8 rounded
        once (2^-25) and an evaluation within 2 roundings of 2^-24, the magnitude's product one more: 4 * 2^-24.
        A value is two products and a sum: at most 3 roundings of the terms' magnitudes.  7 in all, taken as 8."""
        x = x.double().cpu()
        a = self.angles(positions)[:, None]
        c, s = torch.cos(a) * self.magnitude, torch.sin(a) * (-self.magnitude if transpose else self.magnitude)
        j, k = self.parts()
        y, bound = x.clone(), torch.zeros_like(x)
        y[..., j] = x[..., j] * c - x[..., k] * s
        y[..., k] = x[..., j] * s + x[..., k] * c
        size = 8 * 2.0 ** -24 * abs(self.magnitude) * (x[..., j].abs() + x[..., k].abs())
        bound[..., j], bound[..., k] = size, size
        return y, bound


# ---- the cache of heads --------------------------------------------------------

def byte_of(amax):
    """Exponent byte of the least 2^e with amax <= 448 2^e, for amax in 64 bits."""
    a = amax.double()
    e = torch.ceil(torch.log2(torch.where(a > 0, a, 1.0) / 448.0))
    return torch.where(a > 0, (e + 127).clamp(1, 245), 1.0).to(torch.int64)


def power(byte):
    return torch.exp2(byte.clamp(1, 245).double() - 127)


def e4m3(x):
    """x in 64 bits, rounded to the nearest e4m3 value, ties to even; beyond 448: 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    y = (torch.round(x / step) * step).clamp(-448, 448)
    return torch.where(torch.isnan(x), x, y)


class HeadsCache:
    """Replicas of a layer among others, its bytes filled with `fill` or with random codes and scales of N(0, 1) values."""

    def __init__(self, pages, G, D, replicas=2, layers=2, layer=1, pad=0, fill=None, seed=0, spread=0.3):
        self.pages, self.G, self.D, self.layer = pages, G, D, layer
        self.bytes = kvpub.heads_page_bytes(G, D)
        self.page_stride, self.layer_stride = self.bytes + pad, pages * (self.bytes + pad) + 2 * pad
        self.bufs = [torch.full((layers * self.layer_stride,), 0xA5 if fill is None else fill, dtype=torch.uint8, device="cuda")
                     for _ in range(replicas)]
        if fill is None:
            g = torch.Generator(device="cuda")
            g.manual_seed(seed + 5)
            x = torch.randn((pages, G, 2, 64, D), generator=g, device="cuda") * torch.exp(
                spread * torch.randn((pages, G, 2, 1, 1), generator=g, device="cuda"))
            byte = byte_of(x.abs().amax((3, 4)))
            codes = e4m3(x.double() / power(byte)[..., None, None]).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
            for b in self.bufs:
                p = self.page_view(b)
                p[:, :G * 128 * D] = codes.reshape(pages, -1)
                p[:, G * 128 * D:G * 128 * D + 2 * G] = byte.to(torch.uint8).reshape(pages, -1)
        self.struct = kvpub.heads([b.data_ptr() for b in self.bufs], pages, G, D, num_layers=layers, page_stride=self.page_stride,
                                  layer_stride=self.layer_stride)

    def page_view(self, buf):
        a = buf[self.layer * self.layer_stride:][:self.pages * self.page_stride]
        return a.view(self.pages, self.page_stride)

    def codes(self, replica):
        """Raw bytes [page, head, key or value, row, D] of the layer."""
        return self.page_view(self.bufs[replica])[:, :self.G * 128 * self.D].reshape(self.pages, self.G, 2, 64, self.D)

    def scales(self, replica):
        at = self.G * 128 * self.D
        return self.page_view(self.bufs[replica])[:, at:at + 2 * self.G].reshape(self.pages, self.G, 2)

    def values(self, replica, table, kv):
        """[key or value, head, position, D] in 64 bits of a sequence's first kv positions."""
        t = torch.as_tensor(np.asarray(table, np.int64), device="cuda")
        ok = (t >= 0) & (t < self.pages)
        t = torch.where(ok, t, 0)
        x = self.codes(replica)[t].view(torch.float8_e4m3fn).double() * power(self.scales(replica)[t].long())[..., None, None]
        return x.permute(2, 1, 0, 3, 4).reshape(2, self.G, -1, self.D)[:, :, :kv], ok.repeat_interleave(64)[:kv]


class Seqs:
    """Lengths, tokens and tables of a call's sequences; pages of one sequence are its own."""

    def __init__(self, lens, n, pages, seed=0, max_kv=None, max_q=None, one_each=False, tree=None, table=None):
        self.lens, self.n = np.asarray(lens, np.int64), np.asarray(n, np.int64)
        self.max_kv = int(max_kv if max_kv is not None else max(1, self.lens.max(initial=0)))
        self.max_q = int(max_q if max_q is not None else max(1, self.n.max(initial=0)))
        B, width = len(self.lens), max(1, -(-self.max_kv // 64))
        if table is None:
            # pages beyond a sequence's length are not looked at: numbers that would fault
            table = np.full((B, width), 2 ** 31 - 1, np.int32)
            order, at = np.random.default_rng(seed + 100).permutation(pages), 0
            for b in range(B):
                k = -(-min(max(int(self.lens[b]), 0), self.max_kv) // 64)
                table[b, :k] = order[at:at + k]
                at += k
            assert at <= pages
        self.table = np.asarray(table, np.int32)
        self.start = np.concatenate([[0], np.cumsum(self.n)])
        self.T = int(self.start[-1])
        self.tree = tree
        self.d_len, self.d_table, self.d_start = i32(self.lens), i32(self.table), i32(self.start)
        self.d_tree = None if tree is None else torch.from_numpy(np.ascontiguousarray(tree).view(np.int64)).cuda()
        self.struct = kvpub.pages(self.d_len.data_ptr(), self.d_table.data_ptr(), width, B, self.max_kv,
                                  q_start=0 if one_each else self.d_start.data_ptr(), max_q_len=self.max_q,
                                  tree_mask=0 if tree is None else self.d_tree.data_ptr(), tree_words=0 if tree is None else tree.shape[1])

    def kv(self, b):
        return int(min(max(self.lens[b], 0), self.max_kv))

    def seen(self, b):
        """[tokens the call takes, kv] of what they see."""
        kv, n = self.kv(b), int(self.n[b])
        m, base = min(n, self.max_q), kv - n
        p, i = np.arange(kv), np.arange(m)[:, None]
        if self.tree is None:
            return p[None] <= base + i
        j = p - base
        word = np.clip(j // 64, 0, self.tree.shape[1] - 1)
        rows = self.tree[self.start[b]:self.start[b] + m]
        bit = (rows[:, word] >> (j % 64).astype(np.uint64)) & np.uint64(1)
        return (j[None] < 0) | ((bit != 0) & (j < 64 * self.tree.shape[1])[None])


def random_tree(counts, words, seed):
    """Ancestor bits of random trees, one row a token."""
    rng, rows = np.random.default_rng(seed), []
    for n in counts:
        m = np.zeros((int(n), words), np.uint64)
        for i in range(int(n)):
            if i:
                m[i] = m[rng.integers(max(0, i - 4), i)]
            if i < 64 * words:
                m[i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
        rows.append(m)
    return np.concatenate(rows)


class Query:
    """Queries [T, H, D] with `pad` values between rows, and outputs between sentinels."""

    def __init__(self, T, H, D, kind="bf16", seed=0, pad=0, scale=None, mag=1.0, extra=2, lse=True):
        dtype, code = TYPES[kind]
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 17)
        self.T, self.H, self.D, self.dtype, self.kind = T, H, D, dtype, kind
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        self._q = (mag * torch.randn((max(T, 1), H, D + pad), generator=g, device="cuda")).to(dtype)
        self.q = self._q[:T, :, :D]
        self._out = torch.full((T + extra, H, D + pad), SENTINEL, dtype=dtype, device="cuda")
        self._lse = torch.full((T + extra, H + 1), SENTINEL, device="cuda")
        self.out, self.lse = self._out[:T, :, :D], self._lse[:T, :H]
        self.struct = kvpub.heads_queries(self._q.data_ptr(), self._out.data_ptr(), self._lse.data_ptr() if lse else None, T, H, D,
                                          self.scale, code, q_token_stride=H * (D + pad), q_head_stride=D + pad,
                                          out_token_stride=H * (D + pad), out_head_stride=D + pad, lse_token_stride=H + 1)

    def untouched(self, tokens):
        rest = torch.ones(self._out.shape[0], dtype=torch.bool, device="cuda")
        rest[torch.as_tensor(sorted(tokens), dtype=torch.int64, device="cuda")] = False
        assert bool((self._out[rest] == SENTINEL).all()) and bool((self._lse[rest] == SENTINEL).all())
        assert bool((self._out[:, :, self.D:] == SENTINEL).all()) and bool((self._lse[:, self.H:] == SENTINEL).all())


def workspace(size, guard=256):
    buf = torch.full((size + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf, buf.data_ptr() + guard


def attend(ctx, cache, q, seqs, replica=0, on=None):
    size = kvpub.kvpub_heads_attend_workspace(cache.struct, q.struct, seqs.struct)
    buf, ws = workspace(size)
    kvpub.check(kvpub.kvpub_heads_attend(ctx.ctx, cache.struct, replica, cache.layer, q.struct, seqs.struct, ws, size,
                                         on.cuda_stream if on else stream()), "kvpub_heads_attend")
    torch.cuda.synchronize()
    assert bool((buf[:256] == 0xA5).all()) and bool((buf[-256:] == 0xA5).all())


def reference(q, kv, seen, scale):
    """One sequence: q [n, H, D], kv [2, G, P, D], seen [n, P] -> out, lse, bound of |score terms|, mass [n, H, D]."""
    n, H, D = q.shape
    G, P = kv.shape[1], kv.shape[2]
    qq = q.double().view(n, G, H // G, D).permute(1, 0, 2, 3).reshape(G, -1, D)
    look = lambda a: torch.nan_to_num(a, nan=0.0, posinf=0.0, neginf=0.0)     # what is hidden may hold anything
    k, v = look(kv[0]), look(kv[1])
    x = (torch.matmul(qq, k.transpose(1, 2)) * scale).view(G, n, H // G, P)
    size = (torch.matmul(qq.abs(), k.abs().transpose(1, 2)) * abs(scale)).view(G, n, H // G, P)
    hide = ~torch.as_tensor(seen, device="cuda")[None, :, None]
    x, size = x.masked_fill(hide, -math.inf), size.masked_fill(hide, 0.0)
    if P == 0:
        zero = torch.zeros(n, H, D, dtype=torch.float64, device="cuda")
        return zero, torch.full((n, H), -math.inf, dtype=torch.float64, device="cuda"), zero[..., 0], zero
    top = x.amax(-1, keepdim=True)
    ref = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(x - ref)
    total = e.sum(-1)
    lse = ref[..., 0] + torch.log(total)
    w = (e / total.clamp(min=1e-300)[..., None]).reshape(G, -1, P)
    heads = lambda a: a.view(G, n, H // G, -1).permute(1, 0, 2, 3).reshape(n, H, -1)
    return heads(torch.matmul(w, v)), heads(lse)[..., 0], heads(size.amax(-1))[..., 0], heads(torch.matmul(w, v.abs()))


def check_rows(q, a, z, want, what=""):
    """Rows a..z of q's outputs against `reference`.

    lse: a score is a binary32 sum of D exact products, two products with scales and the running maximum's difference: at
    most D + 24 roundings of 2^-24 of the sum of the terms' magnitudes; the sum's and the logarithm's own stay within 2^-20.
    out: half a step of the result; of each weight half a step of bf16 (2^-8; fp16: of its low part, 2^-16) of the sum of
    |w v|; a score's error e moves a weight by e."""
    o, l, size, mass = want
    dead = torch.isinf(l)
    got_l, got = q.lse[a:z].double(), q.out[a:z].double()
    assert torch.equal(torch.isinf(got_l), dead) and bool((got_l[dead] < 0).all()), what
    tol_l = (q.D + 24) * 2.0 ** -24 * size + 2.0 ** -20 * (1 + torch.where(dead, 0.0, l).abs())
    off = (torch.where(dead, 0.0, got_l) - torch.where(dead, 0.0, l)).abs()
    worst = (off / tol_l).max().item() if l.numel() else 0
    assert worst <= 1, f"{what}: lse off by {worst} of its bound"
    weight = 2.0 ** -8 if q.kind == "bf16" else 2.0 ** -16
    tiny = 2.0 ** -25 if q.kind == "fp16" else 1e-30
    tol = half_step(q.dtype) * o.abs() + (weight + 2 * tol_l[..., None]) * mass * 1.01 + tiny
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    worst = ((got - o).abs() / tol).max().item() if o.numel() else 0
    assert worst <= 1, f"{what}: out off by {worst} of its bound"


def check_all(cache, q, seqs, replica=0, what=""):
    """Every sequence's rows, and nothing else written."""
    done = set()
    for b in range(len(seqs.lens)):
        m, kv = min(int(seqs.n[b]), seqs.max_q), seqs.kv(b)
        a = int(seqs.start[b])
        if not m:
            continue
        done |= set(range(a, a + m))
        vals, ok = cache.values(replica, seqs.table[b, :max(1, -(-kv // 64))], kv)
        seen = torch.as_tensor(seqs.seen(b), device="cuda") & ok[None]
        check_rows(q, a, a + m, reference(q.q[a:a + m], vals, seen, q.scale), f"{what} sequence {b}")
    q.untouched(done)
