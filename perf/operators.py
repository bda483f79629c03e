"""Workloads of the operators that read a published latent cache.

A cache row holds 512 e4m3 latent codes with one fp32 scale per 128, and 64
bf16 RoPE values (656 bytes, 64 rows a page).  The operators:

  attend    latent attention, absorbed form, over a paged cache: every head of
            a query shares the position's latent vector as key and value
  slots     the same over a list of slots for each token (a selection)
  tree      the same where the last positions are a tree of drafted tokens
  weights   softmax weights accumulated for each cached position
  evict     the positions of largest weight kept, their rows copied together
  expanded  latent attention, expanded form: keys and values for each head

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the
library's kernels.  ``exact`` computes each result in 64 bits.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
ROW = 656
MAIN_PAGE = PAGE * ROW
IDX_PAGE = PAGE * 132
SCALE = 1.0 / math.sqrt(192.0)


def listed():
    return [
        # one sequence's next token on a rank that holds 16 heads: latency counts
        dict(name="attend-decode-1x700-h16", op="attend", seqs=1, heads=16, q_len=1, kv=700, ragged=False),
        # a decode batch of 64 sequences of ragged lengths, all heads on one GPU
        dict(name="attend-decode-64x8192-h128", op="attend", seqs=64, heads=128, q_len=1, kv=8192, ragged=True),
        # a few tokens' selections, short lists
        dict(name="slots-4x256-h64", op="slots", seqs=4, heads=64, k=256, kv=1000),
        # the top-k pattern: 16 requests that each select 2048 of their slots
        dict(name="slots-16x2048-h128", op="slots", seqs=16, heads=128, k=2048, kv=32768),
        # a small tree of drafts over a short context
        dict(name="tree-1x24-1000-h16", op="tree", seqs=1, heads=16, q_len=24, kv=1000, ragged=False),
        # 16 sequences verify 64 drafted tokens each
        dict(name="tree-16x64-8192-h32", op="tree", seqs=16, heads=32, q_len=64, kv=8192, ragged=True),
        # the weights of one decode step of one sequence
        dict(name="weights-1x700-h16", op="weights", seqs=1, heads=16, q_len=1, kv=700, ragged=False),
        # the weights of a decode step of 16 long sequences
        dict(name="weights-16x16384-h128", op="weights", seqs=16, heads=128, q_len=1, kv=16384, ragged=True),
        # 4 short sequences brought back to a small budget
        dict(name="evict-4x1000-256", op="evict", seqs=4, kv=1000, budget=256, first=4, last=64, replicas=1, ragged=False),
        # 32 long sequences halved, into pages of their own, two replicas
        dict(name="evict-32x16384-8192", op="evict", seqs=32, kv=16384, budget=8192, first=16, last=256, replicas=2, ragged=True),
        # prefill of one short prompt
        dict(name="expanded-1x100-h16", op="expanded", seqs=1, heads=16, q_len=100, kv=100, ragged=False),
        # prefill chunks of 4096 tokens behind as much context
        dict(name="expanded-2x4096-8192-h16", op="expanded", seqs=2, heads=16, q_len=4096, kv=8192, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "slots", "tree", "weights", "evict", "expanded"])
    ragged = rng.random() < 0.7
    heads = rng.choice([1, 5, 8, 16, 24, 32, 64, 100, 128])
    if op == "attend":
        kv = _log(rng, 1, 65536)
        q_len = rng.choice([1, 1, 1, 2, 4, 7, 100])
        seqs = max(1, min(_log(rng, 1, 64), 262144 // kv, 2 ** 27 // (kv * heads * q_len)))
        return dict(op=op, seqs=seqs, heads=heads, q_len=q_len, kv=kv, ragged=ragged, empty=seqs > 1 and rng.random() < 0.3)
    if op == "slots":
        return dict(op=op, seqs=_log(rng, 1, 32), heads=heads, k=_log(rng, 1, 2048), kv=_log(rng, 2048, 16384))
    if op == "tree":
        kv = _log(rng, 64, 16384)
        q_len = min(kv, _log(rng, 2, 130))
        seqs = max(1, min(_log(rng, 1, 16), 2 ** 27 // (kv * heads * q_len)))
        return dict(op=op, seqs=seqs, heads=heads, q_len=q_len, kv=kv, ragged=ragged)
    if op == "weights":
        kv = _log(rng, 1, 65536)
        q_len = rng.choice([1, 1, 2, 5])
        seqs = max(1, min(_log(rng, 1, 64), 262144 // kv, 2 ** 26 // (kv * heads * q_len)))
        return dict(op=op, seqs=seqs, heads=heads, q_len=q_len, kv=kv, ragged=ragged)
    if op == "evict":
        kv = _log(rng, 100, 65536)
        seqs = max(1, min(_log(rng, 1, 32), 262144 // kv))
        return dict(op=op, seqs=seqs, kv=kv, budget=max(80, int(kv * rng.uniform(0.1, 0.95))), first=rng.randint(0, 16),
                    last=rng.randint(0, 64), replicas=rng.choice([1, 2]), ragged=ragged)
    q_len = _log(rng, 1, 4096)
    kv = q_len + (0 if rng.random() < 0.5 else _log(rng, 1, 4096))
    seqs = max(1, min(_log(rng, 1, 8), 2 ** 29 // (q_len * kv * min(heads, 32))))
    return dict(op=op, seqs=seqs, heads=min(heads, 32), q_len=q_len, kv=kv, ragged=ragged)


# ---- inputs ------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _lengths(case, seed):
    """Cached positions of each sequence: all the same, or spread below the largest."""
    rng = np.random.default_rng([seed, 1])
    B, kv, low = case["seqs"], case["kv"], case.get("q_len", 1)
    n = rng.integers(min(low, kv), kv + 1, B).astype(np.int32) if case.get("ragged") else np.full(B, kv, np.int32)
    n[0] = kv
    if case.get("empty"):
        n[-1] = 0
    return n


def _counts(case):
    """Query tokens of each sequence; the same for every seed, as the outputs' shape goes by them."""
    B, q = case["seqs"], case.get("q_len", 1)
    n = np.random.default_rng(3).integers(1, q + 1, B) if case.get("ragged") else np.full(B, q)
    n[0] = q
    return n


def _rows(g, n):
    """n published Main-KV rows of N(0, 1) values under a spread of token magnitudes."""
    x = _randn(g, n, 512) * torch.exp(0.3 * _randn(g, n, 1))
    x = x.bfloat16().float().view(n, 4, 128)
    s = x.abs().amax(-1, keepdim=True) / 448.0
    codes = (x / s).to(torch.float8_e4m3fn).view(torch.uint8).view(n, 512)
    rope = _randn(g, n, 64).bfloat16().view(torch.uint8).view(n, 128)
    return torch.cat([codes, s.view(n, 4).view(torch.uint8).view(n, 16), rope], 1)


def _cache(case, seed, g, replicas=1, extra=0):
    """A cache of just the sequences' pages (and `extra` more), in random order."""
    per = -(-case["kv"] // PAGE)
    used = case["seqs"] * per
    n = used + extra
    row = _rows(g, used * PAGE)
    main = torch.empty(n * PAGE, ROW, dtype=torch.uint8, device="cuda")
    main[:used * PAGE] = row
    main[used * PAGE:] = 0
    idx = torch.zeros(n, IDX_PAGE, dtype=torch.uint8, device="cuda")
    table = torch.randperm(used, generator=g, device="cuda").to(torch.int32).view(case["seqs"], per)
    return dict(main=[main] + [main.clone() for _ in range(replicas - 1)],
                idx=[idx] + [idx.clone() for _ in range(replicas - 1)], num_pages=n, table=table)


def _ancestors(rng, n):
    """Visibility in a random tree of n nodes: bit j of word j/64 of row i set if i descends from j (or is j)."""
    words = -(-n // 64)
    m = np.zeros((n, words), np.uint64)
    for i in range(n):
        if i:
            m[i] = m[rng.integers(max(0, i - 8), i)]
        m[i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return m


def prepare(case, seed):
    op, g, B = case["op"], _gen(seed), case["seqs"]
    s = dict(case=case, op=op)
    if op == "expanded":
        _prepare_expanded(s, case, seed, g)
    elif op == "evict":
        per = -(-min(case["budget"], case["kv"]) // PAGE)
        s.update(_cache(case, seed, g, case["replicas"], B * per))
        for i in s["idx"]:
            i.copy_(torch.randint(0, 256, i.shape, generator=_gen(seed + 1), device="cuda", dtype=torch.uint8))
        # the fresh pages, behind those in use
        s["used"] = s["num_pages"] - B * per
        s["dst"] = (s["used"] + torch.arange(B * per, device="cuda", dtype=torch.int32)).view(B, per)
        s["kv_len"] = torch.from_numpy(_lengths(case, seed)).cuda()
        # accumulated weights: few large ones, a long tail
        s["weights"] = torch.exp(2.0 * _randn(g, B, case["kv"]))
        s["weights_out"] = torch.zeros(B, case["kv"], device="cuda")
        s["kept"] = torch.zeros(B, min(case["budget"], case["kv"]), dtype=torch.int32, device="cuda")
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    else:
        H = case["heads"]
        s.update(_cache(case, seed, g))
        rng = np.random.default_rng([seed, 2])
        n, lens = _counts(case), _lengths(case, seed)
        start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        T = int(start[-1])
        s["tokens"], s["n"] = T, torch.from_numpy(n.astype(np.int32)).cuda()
        s["start"] = torch.from_numpy(start).cuda()
        s["q_latent"] = _randn(g, T, H, 512).bfloat16()
        s["q_rope"] = _randn(g, T, H, 64).bfloat16()
        s["kv_len"] = torch.from_numpy(lens).cuda()
        s["out"] = torch.zeros(T, H, 512, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(T, H, device="cuda")
        if op == "tree":
            s["tree"] = torch.from_numpy(np.concatenate([_ancestors(rng, case["q_len"])[:k] for k in n]).view(np.int64)).cuda()
        if op == "slots":
            # each token's selection of its own sequence's slots, in random order; the short ones end in padding
            pick = torch.rand(B, s["table"].shape[1] * PAGE, generator=g, device="cuda").argsort(1)[:, :case["k"]]
            slot = s["table"].long().gather(1, pick // PAGE) * PAGE + pick % PAGE
            count = torch.randint(max(1, case["k"] // 2), case["k"] + 1, (B, 1), generator=g, device="cuda")
            count[0] = case["k"]
            s["slots"] = torch.where(torch.arange(slot.shape[1], device="cuda") < count, slot, -1)
        if op == "weights":
            s["lse"] = _plain_attend(s)[1]
            s["weights"] = torch.rand(B, case["kv"], generator=g, device="cuda")
            s["weights_out"] = torch.zeros(B, case["kv"], device="cuda")
    if own:
        _plan(s)
    return s


def _prepare_expanded(s, case, seed, g):
    B, H = case["seqs"], case["heads"]
    n = _counts(case)
    m = n + (case["kv"] - case["q_len"])
    q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    k_start = np.concatenate([[0], np.cumsum(m)]).astype(np.int32)
    T, S = int(q_start[-1]), int(k_start[-1])
    s.update(tokens=T, keys=S, q_start=torch.from_numpy(q_start).cuda(), k_start=torch.from_numpy(k_start).cuda())
    s["q_nope"] = _randn(g, T, H, 128).bfloat16()
    s["q_rope"] = _randn(g, T, H, 64).bfloat16()
    s["kv"] = _randn(g, S, H, 256).bfloat16()        # what the up-projection gives: key part, value
    s["k_rope"] = _randn(g, S, 64).bfloat16()
    s["out"] = torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(T, H, device="cuda")


# ---- the library's calls -----------------------------------------------------

class _Context:
    """The program's handle on its cache."""

    def __init__(self, s):
        from replicated_fp8_sparse_amd import kvpub
        self.k = kvpub
        if s["op"] == "expanded":      # reads no cache: a context over one page gives the device
            s["main"] = [torch.zeros(MAIN_PAGE, dtype=torch.uint8, device="cuda")]
            s["idx"] = [torch.zeros(IDX_PAGE, dtype=torch.uint8, device="cuda")]
            s["num_pages"] = 1
        cfg = kvpub.kvpub_config_init(len(s["main"]), 1, s["num_pages"])
        st, self.ctx = kvpub.kvpub_create(cfg, [b.data_ptr() for b in s["main"]], [b.data_ptr() for b in s["idx"]])
        kvpub.check(st, "kvpub_create")

    def __del__(self):
        self.k.kvpub_destroy(self.ctx)


def _plan(s):
    """The descriptors and workspace that a program keeps beside its buffers."""
    s["handle"] = _Context(s)
    k, case, op = s["handle"].k, s["case"], s["op"]
    if op == "expanded":
        s["io"] = k.expanded_io(s["q_nope"].data_ptr(), s["q_rope"].data_ptr(), s["kv"].data_ptr(), s["k_rope"].data_ptr(),
                                s["kv"].data_ptr() + 256, s["out"].data_ptr(), s["lse"].data_ptr(), s["q_start"].data_ptr(),
                                s["k_start"].data_ptr(), case["seqs"], case["heads"], s["tokens"], s["keys"], case["q_len"], SCALE,
                                k_head_stride=256, v_head_stride=256, causal=1)
        return
    if op == "evict":
        s["io"] = k.evict_io(s["weights"].data_ptr(), s["weights_out"].data_ptr(), case["kv"], s["kv_len"].data_ptr(),
                             s["table"].data_ptr(), s["table"].shape[1], s["dst"].data_ptr(), s["dst"].shape[1],
                             s["kept"].data_ptr(), s["kept"].shape[1], s["new_len"].data_ptr(), case["seqs"], case["kv"],
                             s["kept"].shape[1], case["first"], case["last"])
        size = k.kvpub_evict_workspace(s["io"])
    else:
        s["queries"] = k.queries(s["q_latent"].data_ptr(), s["q_rope"].data_ptr(), s["tokens"], case["heads"], SCALE)
        if op == "slots":
            size = k.kvpub_attend_slots_workspace(s["queries"], s["slots"].shape[1])
        else:
            tree = s.get("tree")
            s["pages"] = k.pages(s["kv_len"].data_ptr(), s["table"].data_ptr(), s["table"].shape[1], case["seqs"], case["kv"],
                                 q_start=s["start"].data_ptr(), max_q_len=case["q_len"],
                                 tree_mask=0 if tree is None else tree.data_ptr(), tree_words=0 if tree is None else tree.shape[1])
            size = 0 if op == "weights" else k.kvpub_attend_workspace(s["queries"], s["pages"])
    s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")


def _own_run(s):
    h, op, H = s["handle"], s["op"], s["case"].get("heads")
    k, ctx, stream = h.k, h.ctx, torch.cuda.current_stream().cuda_stream
    if op == "expanded":
        k.check(k.kvpub_attend_expanded(ctx, s["io"], stream), "kvpub_attend_expanded")
        return s["out"], s["lse"]
    ws, size = s["workspace"].data_ptr(), s["workspace"].numel()
    if op == "evict":
        k.check(k.kvpub_evict(ctx, 0, s["io"], ws, size, stream), "kvpub_evict")
        return _evicted(s)
    if op == "slots":
        k.check(k.kvpub_attend_slots(ctx, 0, 0, s["queries"], s["slots"].data_ptr(), s["slots"].shape[1], s["slots"].shape[1],
                                     s["out"].data_ptr(), H * 512, 512, s["lse"].data_ptr(), H, ws, size, stream),
                "kvpub_attend_slots")
        return s["out"], s["lse"]
    if op == "weights":
        k.check(k.kvpub_attend_weights(ctx, 0, 0, s["queries"], s["pages"], s["lse"].data_ptr(), H, s["weights"].data_ptr(),
                                       s["weights_out"].data_ptr(), s["case"]["kv"], stream), "kvpub_attend_weights")
        return s["weights_out"]
    k.check(k.kvpub_attend(ctx, 0, 0, s["queries"], s["pages"], s["out"].data_ptr(), H * 512, 512, s["lse"].data_ptr(), H,
                           ws, size, stream), "kvpub_attend")
    return s["out"], s["lse"]


# ---- plain forms -------------------------------------------------------------

def _values(rows):
    """Latent and RoPE values of raw rows [..., 656], in 32 bits."""
    lead = rows.shape[:-1]
    codes = rows[..., :512].contiguous().view(torch.float8_e4m3fn).float().view(*lead, 4, 128)
    scale = rows[..., 512:528].contiguous().view(torch.float32)
    rope = rows[..., 528:].contiguous().view(torch.bfloat16).float()
    return (codes * scale[..., None]).view(*lead, 512), rope


def _visible(s, width):
    """[B, query, position]: what query i of each sequence sees."""
    n, kv = s["n"].long(), s["kv_len"].long()
    p = torch.arange(width, device="cuda")
    i = torch.arange(s["case"].get("q_len", 1), device="cuda")
    base = (kv - n)[:, None, None]
    inside = (p < kv[:, None, None]) & (i[:, None] < n[:, None, None])
    if s["op"] != "tree":
        return inside & (p <= base + i[:, None])
    token = (s["start"][:-1].long()[:, None] + i).clamp(max=s["tokens"] - 1)
    j = torch.arange(s["case"]["q_len"], device="cuda")
    bits = (s["tree"][token][:, :, j // 64] >> (j % 64)) & 1            # [B, query, node]
    node = (p - base[:, :, 0]).clamp(0, len(j) - 1)
    drafted = bits.gather(2, node[:, None].expand(-1, len(i), -1)) != 0
    return inside & ((p < base) | drafted)


def _padded_queries(s):
    """Queries as [B, query, head, 576] in 32 bits."""
    i = torch.arange(s["case"].get("q_len", 1), device="cuda")
    token = (s["start"][:-1].long()[:, None] + i).clamp(max=s["tokens"] - 1)
    return torch.cat([s["q_latent"].float(), s["q_rope"].float()], 2)[token]


def _scores(s):
    """(scores [B, query, head, position], -inf where hidden; latent values)."""
    rows = s["main"][0].view(-1, PAGE, ROW)[s["table"].long()].view(s["case"]["seqs"], -1, ROW)
    c, r = _values(rows)
    q = _padded_queries(s)
    B, N, H, _ = q.shape
    x = torch.matmul(q.view(B, N * H, 576), torch.cat([c, r], 2).transpose(1, 2)).view(B, N, H, -1) * SCALE
    return x.masked_fill_(~_visible(s, c.shape[1])[:, :, None], float("-inf")), c


def _softmax_values(x, c):
    """(normalised weights times values, log of the sum); zero and -inf where nothing is seen."""
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.view(e.shape[0], -1, e.shape[-1]), c).view(*e.shape[:-1], c.shape[-1])
    return out / total.clamp(min=1e-38), (top + torch.log(total))[..., 0]


def _flat(s, x):
    """[B, query, ...] back to [token, ...]."""
    i = torch.arange(x.shape[1], device="cuda")
    return x[i < s["n"][:, None]]


def _plain_attend(s):
    x, c = _scores(s)
    out, lse = _softmax_values(x, c)
    return _flat(s, out).bfloat16(), _flat(s, lse)


def _plain_slots(s):
    ok = s["slots"] >= 0
    c, r = _values(s["main"][0][s["slots"].clamp(min=0)])
    q = torch.cat([s["q_latent"].float(), s["q_rope"].float()], 2)
    x = torch.matmul(q, torch.cat([c, r], 2).transpose(1, 2)) * SCALE
    out, lse = _softmax_values(x.masked_fill(~ok[:, None], float("-inf")), c)
    return out.bfloat16(), lse


def _plain_weights(s):
    x, _ = _scores(s)
    i = torch.arange(x.shape[1], device="cuda")
    token = (s["start"][:-1].long()[:, None] + i).clamp(max=s["tokens"] - 1)
    lse = s["lse"][token].clamp(min=torch.finfo(torch.float32).min)
    total = torch.exp(x - lse[..., None]).sum((1, 2))[:, :s["case"]["kv"]]
    return s["weights"] + total


def _evicted(s):
    """What eviction leaves: the kept positions, lengths, weights, and the fresh pages' contents of every replica."""
    got = [s["kept"], s["new_len"], s["weights_out"]]
    rows = [m[s["used"] * PAGE:] for m in s["main"]]
    pages = [i[s["used"]:] for i in s["idx"]]
    got += [r[:, :512].view(torch.float8_e4m3fn) for r in rows]
    got += [r.view(torch.float32)[:, 128:132] for r in rows] + [r.view(torch.bfloat16)[:, 264:] for r in rows]
    return got + [p[:, :8192] for p in pages] + [p[:, 8192:].view(torch.int32) for p in pages]


def _plain_evict(s):
    case, B = s["case"], s["case"]["seqs"]
    kv, keep = s["kv_len"].long()[:, None], s["kept"].shape[1]
    p = torch.arange(case["kv"], device="cuda")
    w = s["weights"].masked_fill((p < case["first"]) | (p >= kv - case["last"]), float("inf"))
    w = w.masked_fill(p >= kv, float("-inf"))
    order = torch.sort(w, dim=1, descending=True, stable=True)[1][:, :keep]
    i = torch.arange(keep, device="cuda")
    live = i < kv
    kept = torch.where(live, order, case["kv"]).sort(1)[0]
    at = kept.clamp(max=case["kv"] - 1)
    src = (s["table"].long().gather(1, at // PAGE) * PAGE + at % PAGE)[live]
    dst = (s["dst"].long()[:, i // PAGE] * PAGE + i % PAGE)[live]
    main = s["main"][0][src]
    codes = s["idx"][0][:, :8192].unflatten(1, (PAGE, 128))[src // PAGE, src % PAGE]
    scales = s["idx"][0].view(torch.int32)[src // PAGE, 2048 + src % PAGE]
    s["kept"].copy_(torch.where(live, kept, -1))
    s["new_len"].copy_(kv[:, 0].clamp(max=keep))
    s["weights_out"].zero_()
    s["weights_out"][:, :keep] = torch.where(live, s["weights"].gather(1, at), 0.0)
    for r in range(case["replicas"]):
        s["main"][r][dst] = main
        s["idx"][r][:, :8192].unflatten(1, (PAGE, 128))[dst // PAGE, dst % PAGE] = codes
        s["idx"][r].view(torch.int32)[dst // PAGE, 2048 + dst % PAGE] = scales
    return _evicted(s)


def _plain_expanded(s):
    case = s["case"]
    qs, ks = s["q_start"].long(), s["k_start"].long()
    n, m = (qs[1:] - qs[:-1])[:, None], (ks[1:] - ks[:-1])[:, None]
    i, p = torch.arange(case["q_len"], device="cuda"), torch.arange(case["kv"], device="cuda")
    qt = (qs[:-1, None] + i).clamp(max=s["tokens"] - 1)
    kt = (ks[:-1, None] + p).clamp(max=s["keys"] - 1)
    q = torch.cat([s["q_nope"].float(), s["q_rope"].float()], 2)[qt].transpose(1, 2)           # [B, H, query, 192]
    kv = s["kv"][kt].float().transpose(1, 2)                                                    # [B, H, key, 256]
    kr = s["k_rope"][kt].float()[:, None]
    x = torch.matmul(q[..., :128], kv[..., :128].transpose(2, 3))
    x += torch.matmul(q[..., 128:], kr.transpose(2, 3))
    x *= SCALE
    sees = (p < m[..., None]) & (p <= (m - n)[..., None] + i[:, None])
    x.masked_fill_(~sees[:, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    x -= top
    x.exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, kv[..., 128:]) / total
    lse = (top + torch.log(total))[..., 0]
    real = i < n
    return out.transpose(1, 2)[real].bfloat16(), lse.transpose(1, 2)[real]


def run(state):
    if own:
        return _own_run(state)
    op = state["op"]
    if op == "expanded":
        return _plain_expanded(state)
    if op == "evict":
        return _plain_evict(state)
    if op == "slots":
        return _plain_slots(state)
    if op == "weights":
        return _plain_weights(state)
    return _plain_attend(state)


# ---- what a pass cannot do without ------------------------------------------

def _mean_len(case):
    return case["kv"] if not case.get("ragged") or case["seqs"] == 1 else (case["kv"] + (case["seqs"] - 1) * case["kv"] / 2) / case["seqs"]


def _mean_q(case):
    q = case.get("q_len", 1)
    return q if not case.get("ragged") or case["seqs"] == 1 else (q + (case["seqs"] - 1) * (q + 1) / 2) / case["seqs"]


def work(case):
    op, B, H = case["op"], case["seqs"], case.get("heads", 0)
    kv, n = _mean_len(case), _mean_q(case)
    if op == "slots":
        k = case["k"] if B == 1 else case["k"] * (1 + 0.75 * (B - 1)) / B
        return {"bytes": B * (k * (ROW + 8) + H * (1152 + 1028)), "flops": 2.0 * B * H * k * (576 + 512)}
    if op in ("attend", "tree"):
        seen = kv - (n - 1) / 2 if op == "attend" else kv - n / 2
        return {"bytes": B * (kv * ROW + n * H * (1152 + 1028)), "flops": 2.0 * B * n * H * max(seen, 1) * (576 + 512)}
    if op == "weights":
        return {"bytes": B * (kv * (ROW + 4) + case["kv"] * 4 + n * H * 1156), "flops": 2.0 * B * n * H * max(kv - (n - 1) / 2, 1) * 576}
    if op == "evict":
        keep = min(case["budget"], kv)
        return {"bytes": B * (kv * 4 + case["kv"] * 4 + keep * (4 + (ROW + 132) * (1 + case["replicas"]))), "flops": 0}
    before = case["kv"] - case["q_len"]
    return {"bytes": B * (n * H * (384 + 260) + (n + before) * (H * 512 + 128)),
            "flops": 2.0 * B * H * n * (before + (n + 1) / 2) * (192 + 128)}


# ---- 64 bits -----------------------------------------------------------------

def _row64(raw):
    """One sequence's rows [n, 656] as (latent, RoPE) in 64 bits."""
    codes = raw[:, :512].contiguous().view(torch.float8_e4m3fn).double()
    tile = raw[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
    return codes * tile, raw[:, 528:].contiguous().view(torch.bfloat16).double()


def _one64(ql, qr, c, r, seen):
    """softmax attention of queries [n, H, .] over one sequence's rows; seen [n, position]."""
    x = (torch.einsum("nhd,pd->nhp", ql.double(), c) + torch.einsum("nhd,pd->nhp", qr.double(), r)) * SCALE
    x = torch.where(seen[:, None], x, float("-inf"))
    lse = torch.logsumexp(x, -1)
    w = torch.where(seen[:, None], torch.exp(x - lse[..., None]), 0.0)
    return torch.einsum("nhp,pd->nhd", w, c), lse, w


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "evict":
        return _exact_evict(s, case)
    if op == "expanded":
        return _exact_expanded(s, case)
    outs, lses, sums = [], [], []
    if op == "slots":
        for t in range(case["seqs"]):
            pick = s["slots"][t][s["slots"][t] >= 0]
            c, r = _row64(s["main"][0][pick])
            o, l, _ = _one64(s["q_latent"][t:t + 1], s["q_rope"][t:t + 1], c, r,
                             torch.ones(1, len(pick), dtype=torch.bool, device="cuda"))
            outs.append(o)
            lses.append(l)
        return torch.cat(outs), torch.cat(lses)
    start, lens = s["start"].tolist(), s["kv_len"].tolist()
    for b in range(case["seqs"]):
        a, z, kv = start[b], start[b + 1], lens[b]
        n = z - a
        c, r = _row64(s["main"][0].view(-1, PAGE, ROW)[s["table"][b].long()].view(-1, ROW)[:kv])
        seen = torch.ones(n, kv, dtype=torch.bool, device="cuda")
        if op == "tree":
            w = s["tree"][a:z].cpu().numpy().view(np.uint64)
            bits = np.stack([(w[:, j // 64] >> np.uint64(j % 64)) & np.uint64(1) for j in range(n)], 1).astype(bool)
            seen[:, kv - n:] = torch.from_numpy(bits).cuda()
        else:
            seen = seen.tril(kv - n)
        step = max(1, 2 ** 28 // (max(kv, 1) * case["heads"]))
        total = torch.zeros(case["kv"], dtype=torch.float64, device="cuda")
        for t in range(0, n, step):
            o, l, w = _one64(s["q_latent"][a + t:min(a + t + step, z)], s["q_rope"][a + t:min(a + t + step, z)], c, r, seen[t:t + step])
            outs.append(o)
            lses.append(l)
            if op == "weights":
                given = s["lse"][a + t:min(a + t + step, z)].double()
                total[:kv] += (w * torch.exp(l - given)[..., None]).sum((0, 1))
        sums.append(s["weights"][b].double() + total if op == "weights" else None)
    return torch.stack(sums) if op == "weights" else (torch.cat(outs), torch.cat(lses))


def _exact_evict(s, case):
    """The kept positions by a sort of (weight, position) on the host; the rest moves bytes and has no rounding."""
    keep = s["kept"].shape[1]
    kept = np.full((case["seqs"], keep), -1, np.int32)
    lens = s["kv_len"].cpu().numpy()
    weights = s["weights"].cpu().numpy()
    moved = np.zeros_like(weights, dtype=np.float64)
    for b, n in enumerate(lens):
        if n <= keep:
            pos = np.arange(n)
        else:
            a, z = case["first"], n - case["last"]
            mid = a + np.lexsort((np.arange(a, z), -weights[b, a:z].astype(np.float64)))[:keep - case["first"] - case["last"]]
            pos = np.sort(np.concatenate([np.arange(a), mid, np.arange(z, n)]))
        kept[b, :len(pos)] = pos
        moved[b, :len(pos)] = weights[b, pos]
    return [torch.from_numpy(kept), torch.from_numpy(np.minimum(lens, keep).astype(np.int32)), torch.from_numpy(moved)]


def _exact_expanded(s, case):
    qs, ks = s["q_start"].tolist(), s["k_start"].tolist()
    outs, lses = [], []
    for b in range(case["seqs"]):
        k = s["kv"][ks[b]:ks[b + 1]].double()
        r = s["k_rope"][ks[b]:ks[b + 1]].double()
        m, n = len(k), qs[b + 1] - qs[b]
        for t in range(0, n, 512):
            a, z = qs[b] + t, min(qs[b] + t + 512, qs[b + 1])
            x = torch.einsum("nhd,mhd->hnm", s["q_nope"][a:z].double(), k[..., :128])
            x = (x + torch.einsum("nhd,md->hnm", s["q_rope"][a:z].double(), r)) * SCALE
            seen = torch.ones(z - a, m, dtype=torch.bool, device="cuda").tril(m - n + t)
            x = torch.where(seen, x, float("-inf"))
            outs.append(torch.einsum("hnm,mhd->nhd", torch.softmax(x, -1), k[..., 128:]))
            lses.append(torch.logsumexp(x, -1).T)
    return torch.cat(outs), torch.cat(lses)
