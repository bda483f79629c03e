"""Workloads of the operators around positions and of the cache of key and value heads.

  rotate   rotary positions applied to rows of heads (or, transposed, to their gradients)
  store    the latent cache's store with the position rotation on the way
  append   new keys (rotated) and values appended to a paged e4m3 cache of heads, one
           power-of-two scale for each block of 64 tokens and head
  attend   attention over that cache: grouped heads, causal or a drafted tree

A page of the cache of heads holds 64 positions: for each key-value head [64, D]
codes of the keys, then of the values, and behind all heads a scale byte (2^(b-127))
for the keys and one for the values of each head.

``own`` false: elementary torch operations in 32 bits (angles in 64).  ``own``
true: the library's kernels.  ``exact`` computes each result in 64 bits.
"""
import math
import weakref

import numpy as np
import torch

own = False

PAGE = 64
ROW = 656
MAIN_PAGE = PAGE * ROW
IDX_PAGE = PAGE * 132
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the RoPE part of one decode token's queries, 8 heads of 192: latency counts
        dict(name="rotate-1x8-of-192", op="rotate", tokens=1, heads=8, width=64, row=192, start=0, dim=64, layout="pairs",
             scaling="none", type="bf16", far=4096, transpose=False),
        # a prefill chunk's queries, 128 heads, their RoPE part cut out of rows of 192, frequencies stretched for a long context
        dict(name="rotate-8192x128-of-192-ramp", op="rotate", tokens=8192, heads=128, width=64, row=192, start=0, dim=64,
             layout="pairs", scaling="ramp", type="bf16", far=131072, transpose=False),
        # the gradient of a rotation of 48 of a head's 128 values, halves, 32 bits
        dict(name="rotate-3000x32-48-of-128-gradient", op="rotate", tokens=3000, heads=32, width=128, row=128, start=16, dim=48,
             layout="halves", scaling="blend", type="fp32", far=131072, transpose=True),
        # a decode batch's rows, two replicas
        dict(name="store-64-r2", op="store", tokens=64, replicas=2, pages=64, scaling="none", far=32768),
        # a prefill chunk, four replicas, a few padded tokens
        dict(name="store-8192-r4", op="store", tokens=8192, replicas=4, pages=256, scaling="ramp", far=131072),
        # one token each of 64 sequences, 8 heads of 128, two replicas: most blocks are partly filled
        dict(name="append-64x1-8x128-r2", op="append", seqs=64, q_len=1, kv=8192, groups=8, dim=128, replicas=2, ragged=True,
             type="bf16", layout="halves", rotated=128),
        # prefill chunks of four prompts
        dict(name="append-4x2048-8x128-r2", op="append", seqs=4, q_len=2048, kv=4096, groups=8, dim=128, replicas=2, ragged=True,
             type="bf16", layout="halves", rotated=128),
        # one sequence's next token on a rank that holds 16 heads over 2
        dict(name="attend-1x700-16over2x128", op="attend", seqs=1, q_len=1, kv=700, heads=16, groups=2, dim=128, ragged=False,
             tree=False, type="bf16"),
        # a decode batch of 64 sequences of ragged lengths
        dict(name="attend-64x8192-32over8x128", op="attend", seqs=64, q_len=1, kv=8192, heads=32, groups=8, dim=128, ragged=True,
             tree=False, type="bf16"),
        # 16 sequences verify trees of up to 24 drafted tokens
        dict(name="attend-tree-16x24-8192-32over8x128", op="attend", seqs=16, q_len=24, kv=8192, heads=32, groups=8, dim=128,
             ragged=True, tree=True, type="bf16"),
        # prefill chunks behind as much context
        dict(name="attend-2x4096-8192-16over4x128", op="attend", seqs=2, q_len=4096, kv=8192, heads=16, groups=4, dim=128,
             ragged=True, tree=False, type="bf16"),
        # short prompts of a model with small heads, each with keys of its own, 16-bit floats
        dict(name="attend-5x333-333-12over12x64-fp16", op="attend", seqs=5, q_len=333, kv=333, heads=12, groups=12, dim=64,
             ragged=True, tree=False, type="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "store", "append", "attend", "attend"])
    if op == "rotate":
        width = rng.choice([64, 64, 80, 96, 128, 256])
        dim = rng.choice([d for d in (8, 16, 32, 48, 64, 80, 96, 128, 256) if d <= width])
        start = 8 * rng.randint(0, (width - dim) // 8)
        heads = rng.choice([1, 5, 8, 16, 24, 32, 64, 100, 128])
        tokens = max(1, min(_log(rng, 1, 16384), 2 ** 25 // (heads * width)))
        return dict(op=op, tokens=tokens, heads=heads, width=width, row=width + rng.choice([0, 0, 8, 128]), start=start, dim=dim,
                    layout=rng.choice(["pairs", "halves"]), scaling=rng.choice(["none", "linear", "grown", "ramp", "blend"]),
                    type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), far=_log(rng, 1, 2 ** 20), transpose=rng.random() < 0.3)
    if op == "store":
        tokens = _log(rng, 1, 8192)
        return dict(op=op, tokens=tokens, replicas=rng.choice([1, 2, 4]), pages=-(-tokens // 64) + rng.randint(1, 40),
                    scaling=rng.choice(["none", "linear", "ramp"]), far=_log(rng, 1, 2 ** 20))
    groups, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128, 256])
    ragged, kind = rng.random() < 0.7, rng.choice(["bf16", "bf16", "fp16"])
    if op == "append":
        kv = _log(rng, 1, 32768)
        q_len = min(kv, rng.choice([1, 1, 2, 5, 24, _log(rng, 1, 4096)]))
        seqs = max(1, min(_log(rng, 1, 64), 8192 // q_len))
        return dict(op=op, seqs=seqs, q_len=q_len, kv=kv, groups=groups, dim=dim, replicas=rng.choice([1, 2]), ragged=ragged,
                    type=kind, layout=rng.choice(["pairs", "halves"]), rotated=rng.choice([0, 16, dim // 2, dim]))
    heads = groups * rng.choice([1, 2, 4, 5, 7, 8, 16])
    mode = rng.choice(["decode", "decode", "tree", "chunk"])
    if mode == "chunk":
        q_len = _log(rng, 2, 2048)
        kv = q_len + (0 if rng.random() < 0.5 else _log(rng, 1, 4096))
        seqs = max(1, min(_log(rng, 1, 8), 2 ** 28 // (q_len * kv * heads)))
    else:
        kv = _log(rng, 1, 65536) if mode == "decode" else _log(rng, 64, 16384)
        q_len = 1 if mode == "decode" else min(kv, _log(rng, 2, 130))
        seqs = max(1, min(_log(rng, 1, 64), 262144 // kv, 2 ** 27 // (kv * heads * q_len)))
    return dict(op=op, seqs=seqs, q_len=q_len, kv=kv, heads=heads, groups=groups, dim=dim, ragged=ragged, tree=mode == "tree",
                type=kind, empty=mode == "decode" and seqs > 1 and rng.random() < 0.3)


# ---- inputs ------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _spec(case, dim):
    """The frequencies' description: base, scaling and what it goes by."""
    return dict(dim=dim, scaling=case.get("scaling", "none"), base=10000.0, factor=8.0, original=4096.0, low=1.0, high=32.0)


def _magnitude(case):
    return 0.1 * math.log(8.0) + 1.0 if case.get("scaling") == "ramp" else 1.0


def _counts(case):
    """Tokens of each sequence; the same for every seed, as the outputs' shape goes by them."""
    B, q = case["seqs"], case["q_len"]
    n = np.random.default_rng(3).integers(1, q + 1, B) if case["ragged"] else np.full(B, q)
    n[0] = q
    return n.astype(np.int32)


def _lengths(case, n, rng):
    """Positions of each sequence, its new tokens included: all the same, or spread below the largest."""
    B, kv = case["seqs"], case["kv"]
    lens = rng.integers(min(case["q_len"], kv), kv + 1, B) if case["ragged"] else np.full(B, kv)
    lens[0] = kv
    if case.get("empty"):
        lens[-1] = 0
    return lens.astype(np.int32)


def _bytes_of_scale(amax):
    """Exponent bytes of the least powers of two s with amax <= 448 s."""
    m, e = torch.frexp(amax)                     # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    byte = (e - 9 + (m > 0.875)).clamp(-126, 118) + 127
    return torch.where(amax > 0, byte, 1)


def _scale(byte):
    return torch.exp2(byte.float() - 127.0)


def _encode(x, byte):
    return (x * torch.exp2(127.0 - byte.float())).to(torch.float8_e4m3fn)


def _heads_pages(case, g, pages):
    """`pages` full pages of N(0, 1) keys and values: [pages, stride] bytes."""
    G, D = case["groups"], case["dim"]
    stride = -(-(G * 128 * D + 2 * G) // 16) * 16
    cache = torch.zeros(pages, stride, dtype=torch.uint8, device="cuda")
    step = max(1, 2 ** 28 // (G * 128 * D))
    for a in range(0, pages, step):
        z = min(pages, a + step)
        x = _randn(g, z - a, G, 2, 64 * D) * torch.exp(0.3 * _randn(g, z - a, G, 2, 1))
        byte = _bytes_of_scale(x.abs().amax(-1))
        cache[a:z, :G * 128 * D] = _encode(x, byte[..., None]).view(torch.uint8).view(z - a, -1)
        cache[a:z, G * 128 * D:G * 128 * D + 2 * G] = byte.to(torch.uint8).view(z - a, -1)
    return cache


def _ancestors(rng, n):
    """Visibility in a random tree of n nodes: bit j of word j/64 of row i set if i descends from j (or is j)."""
    m = np.zeros((n, -(-n // 64)), np.uint64)
    for i in range(n):
        if i:
            m[i] = m[rng.integers(max(0, i - 8), i)]
        m[i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return m


def prepare(case, seed):
    s = dict(case=case, op=case["op"])
    {"rotate": _prepare_rotate, "store": _prepare_store, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](s, case, seed)
    if own:
        _plan(s)
    return s


def _prepare_rotate(s, case, seed):
    g, T, H = _gen(seed), case["tokens"], case["heads"]
    s["rows"] = _randn(g, T, H, case["row"]).to(TYPES[case["type"]])
    s["x"] = s["rows"][..., case["row"] - case["width"]:]         # behind what is not rotated at all
    s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda").to(torch.int32)
    s["y"] = torch.zeros(T, H, case["width"], dtype=TYPES[case["type"]], device="cuda")


def _prepare_store(s, case, seed):
    g, T = _gen(seed), case["tokens"]
    s["latent"] = (_randn(g, T, 512) * torch.exp(0.3 * _randn(g, T, 1))).bfloat16()
    s["rope"], s["indexer"] = _randn(g, T, 64).bfloat16(), _randn(g, T, 128).bfloat16()
    slots = torch.randperm(case["pages"] * PAGE, generator=g, device="cuda")[:T].sort()[0]
    s["slots"] = torch.where(torch.rand(T, generator=g, device="cuda") < (0.03 if T > 100 else 0.0), -1, slots)
    s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda").to(torch.int32)
    s["main"] = [torch.zeros(case["pages"] * PAGE, ROW, dtype=torch.uint8, device="cuda") for _ in range(case["replicas"])]
    s["idx"] = [torch.zeros(case["pages"], IDX_PAGE, dtype=torch.uint8, device="cuda") for _ in range(case["replicas"])]


def _prepare_append(s, case, seed):
    g, rng, G, D = _gen(seed), np.random.default_rng([seed, 1]), case["groups"], case["dim"]
    n = _counts(case)
    lens = _lengths(case, n, rng)
    first, last = np.maximum(lens - n, 0) // PAGE, (lens - 1) // PAGE
    # the pages that get new rows are the pool, in random order; the table's others are never touched.  The
    # pool has the size that any seed may need, as the outputs' shape goes by it.
    pool = int((n // PAGE + 2).sum())
    order, at = rng.permutation(pool), 0
    table = np.zeros((case["seqs"], -(-case["kv"] // PAGE)), np.int32)
    for b in range(case["seqs"]):
        k = last[b] - first[b] + 1
        table[b, first[b]:last[b] + 1] = order[at:at + k]
        at += k
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = s["tokens"] = int(start[-1])
    cache = _heads_pages(case, g, pool)
    s.update(pages=pool, stride=cache.shape[1], cache=[cache] + [cache.clone() for _ in range(case["replicas"] - 1)],
             n=torch.from_numpy(n).cuda(), kv_len=torch.from_numpy(lens).cuda(), start=torch.from_numpy(start).cuda(),
             table=torch.from_numpy(table).cuda())
    # what a projection gives: keys and values of a token side by side
    s["kv"] = (_randn(g, T, 2, G, D) * torch.exp(0.5 * _randn(g, T, 2, G, 1))).to(TYPES[case["type"]])


def _prepare_attend(s, case, seed):
    g, rng, B = _gen(seed), np.random.default_rng([seed, 2]), case["seqs"]
    n = _counts(case)
    lens = _lengths(case, n, rng)
    per = -(-case["kv"] // PAGE)
    cache = _heads_pages(case, g, B * per)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = s["tokens"] = int(start[-1])
    s.update(pages=B * per, stride=cache.shape[1], cache=[cache], n=torch.from_numpy(n).cuda(),
             kv_len=torch.from_numpy(lens).cuda(), start=torch.from_numpy(start).cuda(),
             table=torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per))
    s["q"] = _randn(g, T, case["heads"], case["dim"]).to(TYPES[case["type"]])
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(T, case["heads"], device="cuda")
    if case["tree"]:
        s["tree"] = torch.from_numpy(np.concatenate([_ancestors(rng, case["q_len"])[:k] for k in n]).view(np.int64)).cuda()


# ---- the library's calls -----------------------------------------------------

class _Context:
    """The program's handle: over its latent cache, or over one page where only the device counts."""

    def __init__(self, s):
        from replicated_fp8_sparse_amd import kvpub
        self.k = kvpub
        self.main = s.get("main") or [torch.zeros(MAIN_PAGE, dtype=torch.uint8, device="cuda")]
        self.idx = s.get("idx") or [torch.zeros(IDX_PAGE, dtype=torch.uint8, device="cuda")]
        cfg = kvpub.kvpub_config_init(len(self.main), 1, s["case"].get("pages", 1))
        st, self.ctx = kvpub.kvpub_create(cfg, [b.data_ptr() for b in self.main], [b.data_ptr() for b in self.idx])
        kvpub.check(st, "kvpub_create")
        weakref.finalize(self, kvpub.kvpub_destroy, self.ctx)         # at the latest before the interpreter takes modules down


def _rotation(s, name, dim, start, layout):
    """The frequencies' table, laid out once, and the descriptor that names it."""
    k, case = s["handle"].k, s["case"]
    spec = _spec(case, dim)
    scaling = dict(none=k.SCALING_NONE, linear=k.SCALING_LINEAR, grown=k.SCALING_GROWN, ramp=k.SCALING_RAMP, blend=k.SCALING_BLEND)
    st, turns = k.kvpub_rotation_turns(k.rotation_config(dim, spec["base"], scaling[spec["scaling"]], spec["factor"], spec["original"],
                                                         spec["low"], spec["high"]))
    k.check(st, "kvpub_rotation_turns")
    s["turns_" + name] = torch.from_numpy(turns.view(np.int64)).cuda()
    s["rotation_" + name] = k.rotation(s["turns_" + name].data_ptr(), dim, start=start,
                                       layout=k.ROTATE_PAIRS if layout == "pairs" else k.ROTATE_HALVES, magnitude=_magnitude(case))


def _plan(s):
    """The descriptors and workspace that a program keeps beside its buffers."""
    s["handle"] = _Context(s)
    k, case, op = s["handle"].k, s["case"], s["op"]
    kind = dict(bf16=k.BF16, fp16=k.FP16, fp32=k.FP32).get(case.get("type"))
    if op == "rotate":
        H, w, row = case["heads"], case["width"], case["row"]
        _rotation(s, "x", case["dim"], case["start"], case["layout"])
        s["io"] = k.rotate_io(s["x"].data_ptr(), s["y"].data_ptr(), s["positions"].data_ptr(), s["rotation_x"], case["tokens"], H, w,
                              kind, x_token_stride=H * row, x_head_stride=row, transpose=int(case["transpose"]))
        return
    if op == "store":
        _rotation(s, "rope", 64, 0, "pairs")
        _rotation(s, "indexer", 64, 0, "halves")
        return
    G, D, B = case["groups"], case["dim"], case["seqs"]
    s["heads"] = k.heads([c.data_ptr() for c in s["cache"]], s["pages"], G, D)
    tree = s.get("tree")
    s["desc"] = k.pages(s["kv_len"].data_ptr(), s["table"].data_ptr(), s["table"].shape[1], B, case["kv"], q_start=s["start"].data_ptr(),
                        max_q_len=case["q_len"], tree_mask=0 if tree is None else tree.data_ptr(),
                        tree_words=0 if tree is None else tree.shape[1])
    if op == "append":
        s["rows"] = k.heads_rows(s["kv"].data_ptr(), s["kv"].data_ptr() + G * D * s["kv"].element_size(), s["tokens"], kind,
                                 k_token_stride=2 * G * D, k_head_stride=D, v_token_stride=2 * G * D, v_head_stride=D)
        s["rotation_k"] = None
        if case["rotated"]:
            _rotation(s, "k", case["rotated"], 0, case["layout"])
        return
    s["queries"] = k.heads_queries(s["q"].data_ptr(), s["out"].data_ptr(), s["lse"].data_ptr(), s["tokens"], case["heads"], D,
                                   1.0 / math.sqrt(D), kind)
    size = k.kvpub_heads_attend_workspace(s["heads"], s["queries"], s["desc"])
    s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")


def _own_run(s):
    h, op, case = s["handle"], s["op"], s["case"]
    k, ctx, stream = h.k, h.ctx, torch.cuda.current_stream().cuda_stream
    if op == "rotate":
        k.check(k.kvpub_rotate(ctx, s["io"], stream), "kvpub_rotate")
        return s["y"]
    if op == "store":
        k.check(k.kvpub_store_rotated(ctx, 0, case["tokens"], s["latent"].data_ptr(), 512, s["rope"].data_ptr(), 64,
                                      s["indexer"].data_ptr(), 128, s["slots"].data_ptr(), s["positions"].data_ptr(),
                                      s["rotation_rope"], s["rotation_indexer"], stream), "kvpub_store_rotated")
        return _stored(s)
    if op == "append":
        k.check(k.kvpub_heads_append(ctx, s["heads"], 0, s["rows"], s["desc"], s["rotation_k"], None, stream), "kvpub_heads_append")
        return _appended(s)
    k.check(k.kvpub_heads_attend(ctx, s["heads"], 0, 0, s["queries"], s["desc"], s["workspace"].data_ptr(), s["workspace"].numel(),
                                 stream), "kvpub_heads_attend")
    return s["out"], s["lse"]


# ---- plain forms -------------------------------------------------------------

def _frequencies(spec):
    """Radians a position of each pair, in 64 bits."""
    dim, base, factor = spec["dim"], spec["base"], spec["factor"]
    i = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    if spec["scaling"] == "grown":
        base = base * factor ** (dim / (dim - 2))
    f = base ** (-2.0 * i / dim)
    if spec["scaling"] == "linear":
        return f / factor
    if spec["scaling"] == "ramp":       # by the pair's index, between those that turn `high` and `low` times over the original length
        at = lambda turns: dim * math.log(spec["original"] / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(spec["high"])), 0), min(math.ceil(at(spec["low"])), dim - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    elif spec["scaling"] == "blend":    # by the turns themselves
        keep = ((spec["original"] * f / (2 * math.pi) - spec["low"]) / (spec["high"] - spec["low"])).clamp(0, 1)
    else:
        return f
    return f * keep + f / factor * (1 - keep)


def _turned(x, positions, spec, start, layout, magnitude, transpose=False):
    """Rows x [token, ..., width] in 32 bits with [start, start + dim) rotated."""
    dim = spec["dim"]
    angle = positions.double()[:, None] * _frequencies(spec)
    shape = (len(positions),) + (1,) * (x.dim() - 2) + (dim // 2,)
    cos, sin = torch.cos(angle).float().view(shape) * magnitude, torch.sin(angle).float().view(shape) * magnitude
    if transpose:
        sin = -sin
    part = x[..., start:start + dim]
    if layout == "pairs":
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = part[..., :dim // 2], part[..., dim // 2:]
        part = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([x[..., :start], part, x[..., start + dim:]], -1)


def _plain_rotate(s):
    case = s["case"]
    y = _turned(s["x"].float(), s["positions"], _spec(case, case["dim"]), case["start"], case["layout"], _magnitude(case), case["transpose"])
    return y.to(TYPES[case["type"]])


def _stored(s):
    got = []
    for m, i in zip(s["main"], s["idx"]):
        got += [m[:, :512].view(torch.float8_e4m3fn), m.view(torch.float32)[:, 128:132], m.view(torch.bfloat16)[:, 264:],
                i[:, :8192].view(torch.float8_e4m3fn), i[:, 8192:].view(torch.float32)]
    return got


def _tiles(x):
    """(e4m3 codes, scales) of rows [n, k * 128]."""
    t = x.view(len(x), -1, 128)
    scale = t.abs().amax(-1) / 448.0
    code = torch.where(scale[..., None] > 0, t / scale[..., None], 0.0).to(torch.float8_e4m3fn)
    return code.view(torch.uint8).view(len(x), -1), scale


def _plain_store(s):
    case = s["case"]
    live = s["slots"] >= 0
    slot = s["slots"][live]
    rope = _turned(s["rope"].float(), s["positions"], _spec(case, 64), 0, "pairs", _magnitude(case)).bfloat16()[live]
    indexer = _turned(s["indexer"].float(), s["positions"], _spec(case, 64), 0, "halves", _magnitude(case))[live]
    codes, scale = _tiles(s["latent"].float()[live])
    icodes, iscale = _tiles(indexer)
    row = torch.cat([codes, scale.contiguous().view(torch.uint8), rope.contiguous().view(torch.uint8)], 1)
    for r in range(case["replicas"]):
        s["main"][r][slot] = row
        s["idx"][r][:, :8192].unflatten(1, (PAGE, 128))[slot // PAGE, slot % PAGE] = icodes
        s["idx"][r].view(torch.float32)[slot // PAGE, 2048 + slot % PAGE] = iscale[:, 0]
    return _stored(s)


def _appended(s):
    G, D = s["case"]["groups"], s["case"]["dim"]
    got = []
    for c in s["cache"]:
        got += [c[:, :G * 128 * D].view(torch.float8_e4m3fn), c[:, G * 128 * D:G * 128 * D + 2 * G].view(torch.float8_e8m0fnu)]
    return got


def _plain_append(s):
    case, G, D, B = s["case"], s["case"]["groups"], s["case"]["dim"], s["case"]["seqs"]
    token = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["start"][1:].long(), token, right=True)
    base = (s["kv_len"] - s["n"]).long()
    position = base[seq] + token - s["start"].long()[seq]
    x = s["kv"].float()
    if case["rotated"]:
        k = _turned(x[:, 0], position, _spec(case, case["rotated"]), 0, case["layout"], _magnitude(case))
        x = torch.cat([k[:, None], x[:, 1:]], 1)
    page = s["table"].long()[seq, position // PAGE]
    # the pool's pages: older rows are those below the first new one where the block began before it
    amax = torch.zeros(s["pages"], 2, G, device="cuda").scatter_reduce(0, page[:, None, None].expand(-1, 2, G), x.abs().amax(-1), "amax")
    byte = _bytes_of_scale(amax)
    older = torch.zeros(s["pages"], dtype=torch.long, device="cuda")
    first = s["table"].long()[torch.arange(B, device="cuda"), base // PAGE]
    older[first] = base % PAGE
    touched = torch.zeros(s["pages"], dtype=torch.bool, device="cuda")
    touched[page] = True
    cache = s["cache"][0]
    had = cache[:, G * 128 * D:G * 128 * D + 2 * G].view(-1, G, 2).transpose(1, 2).int()
    byte = torch.where((older > 0)[:, None, None], torch.maximum(byte, had), byte)
    byte = torch.where(touched[:, None, None], byte, had)
    rows = cache[:, :G * 128 * D].view(torch.float8_e4m3fn).unflatten(1, (G, 2, PAGE, D))
    again = (rows.float() * torch.exp2((had - byte).float()).transpose(1, 2)[..., None, None]).to(torch.float8_e4m3fn)
    is_older = (torch.arange(PAGE, device="cuda") < older[:, None])[:, None, None, :, None]
    rows = torch.where(is_older, again.view(torch.uint8), rows.view(torch.uint8))
    rows[page, :, :, position % PAGE] = _encode(x, byte[page][..., None]).view(torch.uint8).transpose(1, 2)
    for c in s["cache"]:
        c[:, :G * 128 * D] = rows.flatten(1)
        c[:, G * 128 * D:G * 128 * D + 2 * G] = byte.transpose(1, 2).to(torch.uint8).flatten(1)
    return _appended(s)


def _visible(s, width):
    """[B, query, position]: what query i of each sequence sees."""
    n, kv = s["n"].long(), s["kv_len"].long()
    p, i = torch.arange(width, device="cuda"), torch.arange(s["case"]["q_len"], device="cuda")
    base = (kv - n)[:, None, None]
    inside = (p < kv[:, None, None]) & (i[:, None] < n[:, None, None])
    if not s["case"]["tree"]:
        return inside & (p <= base + i[:, None])
    token = (s["start"][:-1].long()[:, None] + i).clamp(max=s["tokens"] - 1)
    bits = (s["tree"][token][:, :, i // 64] >> (i % 64)) & 1            # [B, query, node]
    node = (p - base[:, :, 0]).clamp(0, len(i) - 1)
    drafted = bits.gather(2, node[:, None].expand(-1, len(i), -1)) != 0
    return inside & ((p < base) | drafted)


def _plain_attend(s):
    case, G, D, B, N = s["case"], s["case"]["groups"], s["case"]["dim"], s["case"]["seqs"], s["case"]["q_len"]
    H = case["heads"]
    page = s["cache"][0][s["table"].long()]                                                    # [B, pages, stride]
    scale = _scale(page[..., G * 128 * D:G * 128 * D + 2 * G]).unflatten(2, (G, 2))
    kv = page[..., :G * 128 * D].view(torch.float8_e4m3fn).unflatten(2, (G, 2, PAGE, D)).float() * scale[..., None, None]
    k, v = (kv[:, :, :, j].permute(0, 2, 1, 3, 4).reshape(B, G, -1, D) for j in (0, 1))
    i = torch.arange(N, device="cuda")
    token = (s["start"][:-1].long()[:, None] + i).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[token].view(B, N, G, H // G, D).permute(0, 2, 1, 3, 4).reshape(B, G, -1, D)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, G, N, H // G, -1)
    x *= 1.0 / math.sqrt(D)
    x.masked_fill_(~_visible(s, k.shape[2])[:, None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    x -= top
    x.exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, G, -1, x.shape[-1]), v).view(B, G, N, H // G, D) / total.clamp(min=1e-38)
    lse = (top + torch.log(total))[..., 0]
    real = i < s["n"][:, None]
    return (out.permute(0, 2, 1, 3, 4).reshape(B, N, H, D)[real].to(TYPES[case["type"]]),
            lse.permute(0, 2, 1, 3).reshape(B, N, H)[real])


def run(state):
    if own:
        return _own_run(state)
    op = state["op"]
    if op == "rotate":
        return _plain_rotate(state)
    if op == "store":
        return _plain_store(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attend(state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op == "rotate":
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": case["tokens"] * (case["heads"] * case["width"] * 2 * size + 4),
                "flops": 3.0 * case["tokens"] * case["heads"] * case["dim"]}
    if op == "store":
        return {"bytes": case["tokens"] * (1408 + 12 + 788 * case["replicas"]), "flops": 0}
    G, D, n = case["groups"], case["dim"], _counts(case)
    if op == "append":
        return {"bytes": int(n.sum()) * G * D * 2 * (2 + case["replicas"]), "flops": 0}
    kv = np.full(case["seqs"], case["kv"], float)
    if case["ragged"]:
        kv[1:] = (case["kv"] + min(case["q_len"], case["kv"])) / 2
    if case.get("empty"):
        kv[-1] = 0
    H = case["heads"]
    seen = np.maximum(kv - (n / 2 if case["tree"] else (n - 1) / 2), 0)
    return {"bytes": float((kv * (G * D * 2 + G / 32) + n * H * (4 * D + 4)).sum()), "flops": float((4.0 * n * H * D * seen).sum())}


# ---- 64 bits -----------------------------------------------------------------

def _angles64(positions, spec):
    """cos and sin on the host, [token, pair]: the frequencies one by one from their definition."""
    dim, base, f = spec["dim"], spec["base"], []
    where = lambda turns: dim * math.log(spec["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(where(spec["high"])), 0), min(math.ceil(where(spec["low"])), dim - 1)
    for i in range(dim // 2):
        w = base ** (-2 * i / dim)
        if spec["scaling"] == "grown":
            w = (base * spec["factor"] ** (dim / (dim - 2))) ** (-2 * i / dim)
        elif spec["scaling"] == "linear":
            w /= spec["factor"]
        elif spec["scaling"] in ("ramp", "blend"):
            turns = spec["original"] * w / (2 * math.pi)
            keep = (turns - spec["low"]) / (spec["high"] - spec["low"]) if spec["scaling"] == "blend" else 1 - (i - lo) / max(hi - lo, 0.001)
            keep = min(max(keep, 0.0), 1.0)
            w *= keep + (1 - keep) / spec["factor"]
        f.append(w)
    a = positions.cpu().numpy().astype(np.float64)[:, None] * np.array(f)
    return torch.from_numpy(np.exp(1j * a)).cuda()


def _turned64(x, positions, spec, start, layout, magnitude, transpose=False):
    """The rotation as a product of complex numbers; x [token, head, width] in 64 bits."""
    y, dim = x.clone(), spec["dim"]
    turn = _angles64(positions, spec)[:, None] * magnitude
    if transpose:
        turn = turn.conj()
    part = x[..., start:start + dim]
    if layout == "pairs":
        z = torch.view_as_complex(part.reshape(*part.shape[:-1], dim // 2, 2).contiguous()) * turn
        y[..., start:start + dim] = torch.view_as_real(z).reshape(part.shape)
    else:
        z = torch.complex(part[..., :dim // 2], part[..., dim // 2:]) * turn
        y[..., start:start + dim] = torch.cat([z.real, z.imag], -1)
    return y


def _e4m3(x):
    """x in 64 bits rounded to the nearest e4m3 value, ties to even."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        return _turned64(s["x"].double(), s["positions"], _spec(case, case["dim"]), case["start"], case["layout"], _magnitude(case),
                         case["transpose"])
    return {"store": _exact_store, "append": _exact_append, "attend": _exact_attend}[op](s, case)


def _exact_store(s, case):
    pages = case["pages"]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")
    codes, scales, ropes = new(pages * PAGE, 512), new(pages * PAGE, 4), new(pages * PAGE, 64)
    icodes, iscales = new(pages * PAGE, 128), new(pages * PAGE)
    keep = torch.nonzero(s["slots"] >= 0)[:, 0]
    at, m = s["slots"][keep], _magnitude(case)
    lat = s["latent"].double()[keep].view(-1, 4, 128)
    scale = (lat.abs().amax(-1) / 448).float().double()
    codes[at] = _e4m3((lat / scale[..., None]).float().double()).view(-1, 512)
    scales[at] = scale
    ropes[at] = _turned64(s["rope"].double()[:, None], s["positions"], _spec(case, 64), 0, "pairs", m)[keep, 0].bfloat16().double()
    ix = _turned64(s["indexer"].double()[:, None], s["positions"], _spec(case, 64), 0, "halves", m)[keep, 0]
    iscale = (ix.abs().amax(-1) / 448).float().double()
    icodes[at] = _e4m3(ix / iscale[:, None])
    iscales[at] = iscale
    return [codes, scales, ropes, icodes.view(pages, -1), iscales.view(pages, -1)] * case["replicas"]


def _exact_append(s, case):
    """Sequence by sequence and block by block, on the host's lists."""
    G, D = case["groups"], case["dim"]
    if s["tokens"] > 20000 or case["seqs"] * (case["q_len"] // PAGE + 2) > 2000:
        return None
    cache = s["cache"][0].clone()
    had = cache[:, G * 128 * D:G * 128 * D + 2 * G].view(-1, G, 2).cpu().double()
    rows = cache[:, :G * 128 * D].view(torch.float8_e4m3fn).unflatten(1, (G, 2, PAGE, D)).double()
    scales = torch.exp2(had - 127).cuda()
    start, lens, table = s["start"].tolist(), s["kv_len"].tolist(), s["table"].tolist()
    for b in range(case["seqs"]):
        n = start[b + 1] - start[b]
        first = lens[b] - n
        x = s["kv"][start[b]:start[b + 1]].double().transpose(0, 1)               # [2, n, G, D]
        k = x[0]
        if case["rotated"]:
            k = _turned64(k, torch.arange(first, lens[b]), _spec(case, case["rotated"]), 0, case["layout"], _magnitude(case))
        x = torch.stack([k, x[1]]).permute(2, 0, 1, 3)                            # [G, 2, n, D]
        for block in range(first // PAGE, (lens[b] - 1) // PAGE + 1):
            lo, hi = max(first, block * PAGE), min(lens[b], block * PAGE + PAGE)
            new = x[:, :, lo - first:hi - first]
            top = new.abs().amax((2, 3)) / 448
            scale = torch.exp2(torch.ceil(torch.log2(top)).clamp(min=-126, max=118))
            page, at = table[b][block], lo - block * PAGE
            if at:
                scale = torch.maximum(scale, scales[page])
                rows[page, :, :, :at] = _e4m3(rows[page, :, :, :at] * (scales[page] / scale)[..., None, None])
            scales[page] = scale
            rows[page, :, :, at:at + hi - lo] = _e4m3(new / scale[..., None, None])
    return [rows.flatten(1), scales.flatten(1)] * case["replicas"]


def _exact_attend(s, case):
    G, D, H = case["groups"], case["dim"], case["heads"]
    start, lens = s["start"].tolist(), s["kv_len"].tolist()
    if sum((z - a) * l for a, z, l in zip(start, start[1:], lens)) * H * D > 2e13:
        return None
    outs, lses = [], []
    for b in range(case["seqs"]):
        a, z, kv = start[b], start[b + 1], lens[b]
        n = z - a
        if kv == 0:
            outs.append(torch.zeros(n, H, D, dtype=torch.float64, device="cuda"))
            lses.append(torch.full((n, H), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        pages = s["cache"][0][s["table"][b].long()]
        power = pages[:, G * 128 * D:G * 128 * D + 2 * G].double().view(-1, G, 2, 1, 1) - 127
        val = pages[:, :G * 128 * D].contiguous().view(torch.float8_e4m3fn).double().view(-1, G, 2, PAGE, D) * 2.0 ** power
        val = val.permute(2, 1, 0, 3, 4).reshape(2, G, -1, D)[:, :, :kv]
        seen = torch.ones(n, kv, dtype=torch.bool, device="cuda")
        if case["tree"]:
            w = s["tree"][a:z].cpu().numpy().view(np.uint64)
            bits = np.stack([(w[:, j // 64] >> np.uint64(j % 64)) & np.uint64(1) for j in range(n)], 1).astype(bool)
            seen[:, kv - n:] = torch.from_numpy(bits).cuda()
        else:
            seen = seen.tril(kv - n)
        step = max(1, 2 ** 28 // (kv * H))
        for t in range(0, n, step):
            q = s["q"][a + t:min(a + t + step, z)].double().view(-1, G, H // G, D)
            x = torch.einsum("nghd,gpd->nghp", q, val[0]) / math.sqrt(D)
            x = torch.where(seen[t:t + step, None, None], x, -math.inf)
            outs.append(torch.einsum("nghp,gpd->nghd", torch.softmax(x, -1), val[1]).reshape(-1, H, D))
            lses.append(torch.logsumexp(x, -1).reshape(-1, H))
    return torch.cat(outs), torch.cat(lses)
