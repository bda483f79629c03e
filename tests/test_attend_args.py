"""Argument checks of the attention and eviction entry points, on the host.

The context is a block of memory that holds a configuration whose device does
not exist: a call that passes every check stops where it would select the device
(KVPUB_ERR_HIP), before anything is launched; a refused one returns
KVPUB_ERR_INVALID_ARG before that."""
import ctypes
import math
import os
import random
import subprocess

import pytest

from replicated_fp8_sparse_amd import kvpub

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20                     # an aligned address that is never read
BAD, PASSED, OK = kvpub.KVPUB_ERR_INVALID_ARG, kvpub.KVPUB_ERR_HIP, kvpub.KVPUB_OK


class Context:
    def __init__(self, **kw):
        cfg = kvpub.kvpub_config_init(2, 3, 100)
        cfg.device = 1 << 20
        for k, v in kw.items():
            setattr(cfg, k, v)
        self.buf = ctypes.create_string_buffer(1 << 16)
        ctypes.memmove(self.buf, ctypes.byref(cfg), ctypes.sizeof(cfg))
        self.ptr = ctypes.addressof(self.buf)


class Lazy:
    """Built by the first call: collecting these tests loads no library."""
    made = None

    @property
    def ptr(self):
        self.made = self.made or Context()
        return self.made.ptr


CTX = Lazy()
LIMIT = 2 ** 31


def queries(**kw):
    q = kvpub.queries(P, P, 6, 16, 0.07)
    return change(q, kw)


def pages(**kw):
    return change(kvpub.pages(P, P, 20, 3, 1200, q_start=P, max_q_len=4), kw)


def change(s, kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def attend(q=None, g=None, ctx=None, replica=1, layer=2, out=P, token=16 * 512, head=512, lse=P, lse_token=16, ws=P, size=1 << 40):
    return kvpub.kvpub_attend((ctx or CTX).ptr, replica, layer, q or queries(), g or pages(), out, token, head, lse, lse_token, ws, size)


def slots(q=None, ctx=None, replica=1, layer=2, slots=P, stride=70, n=70, out=P, token=16 * 512, head=512, lse=P, lse_token=16,
          ws=P, size=1 << 40):
    return kvpub.kvpub_attend_slots((ctx or CTX).ptr, replica, layer, q or queries(), slots, stride, n, out, token, head, lse,
                                    lse_token, ws, size)


def weights(q=None, g=None, ctx=None, replica=1, layer=2, lse=P, lse_token=16, w_in=P, w_out=P, stride=1200):
    return kvpub.kvpub_attend_weights((ctx or CTX).ptr, replica, layer, q or queries(), g or pages(), lse, lse_token, w_in, w_out,
                                      stride)


def evict_io(**kw):
    return change(kvpub.evict_io(P, P, 1200, P, P, 20, 2 * P, 5, P, 300, 2 * P, 3, 1200, 300, 4, 64), kw)


def evict(io=None, ctx=None, layer=2, ws=P, size=1 << 40):
    return kvpub.kvpub_evict((ctx or CTX).ptr, layer, io or evict_io(), ws, size)


def expanded_io(**kw):
    return change(kvpub.expanded_io(P, P, P, P, P, P, P, P, P, 3, 16, 40, 90, 20, 0.07, k_head_stride=256, v_head_stride=256), kw)


def expanded(io=None, ctx=None):
    return kvpub.kvpub_attend_expanded((ctx or CTX).ptr, io or expanded_io())


def test_struct_sizes_and_offsets_match_the_header(tmp_path):
    names = ["kvpub_queries", "kvpub_pages", "kvpub_evict_io", "kvpub_expanded_io"]
    src = ["#include <stddef.h>", "#include <stdio.h>", '#include "kvpub.h"', "int main(void) {"]
    for n in names:
        src.append(f'printf("%zu\\n", sizeof({n}));')
        src += [f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in getattr(kvpub, n)._fields_]
    (tmp_path / "sizes.c").write_text("\n".join(src + ["return 0; }", ""]))
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "sizes.c"), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for n in names:
        s = getattr(kvpub, n)
        want += [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


def test_calls_that_pass_every_check():
    assert attend() == slots() == weights() == evict() == expanded() == PASSED
    assert attend(lse=None, lse_token=0) == slots(lse=None, lse_token=0) == PASSED
    assert attend(g=pages(q_start=0)) == PASSED
    assert attend(g=pages(tree_mask=P, tree_words=64)) == PASSED
    assert attend(queries(q_latent_token_stride=0, q_rope_token_stride=0)) == PASSED          # one row for all tokens
    assert attend(queries(num_heads=1, q_latent_head_stride=0, q_rope_head_stride=0), head=0, token=512) == PASSED
    assert slots(slots=None, stride=0, n=0) == PASSED
    assert weights(w_in=None) == PASSED
    assert weights(queries(num_tokens=0, q_latent=0), pages(q_start=0), lse=None) == PASSED   # the weights are still copied
    assert evict(evict_io(dst_table=P, dst_table_stride=20)) == PASSED                        # in place
    assert expanded(expanded_io(lse=0, causal=0)) == PASSED
    assert expanded(expanded_io(num_keys=0, k_nope=0, k_rope=0, v=0)) == PASSED
    assert expanded(expanded_io(k_rope_token_stride=0)) == PASSED                             # rows that are read may share memory


def test_calls_with_nothing_to_do():
    assert attend(queries(num_tokens=0, q_latent=0, q_rope=0), out=None, ws=None, size=0) == OK
    assert attend(g=pages(num_seqs=0, kv_len=0, page_table=0), out=None, ws=None, size=0) == OK
    assert slots(queries(num_tokens=0), slots=None, out=None, ws=None, size=0) == OK
    assert weights(g=pages(num_seqs=0)) == weights(g=pages(max_kv_len=0)) == OK
    assert evict(evict_io(num_seqs=0, kv_len=0)) == OK
    assert expanded(expanded_io(num_tokens=0, q_nope=0)) == expanded(expanded_io(num_seqs=0)) == OK


@pytest.mark.parametrize("call", [attend, slots, weights])
def test_contexts_replicas_and_layers(call):
    assert call(replica=2) == call(layer=3) == BAD
    assert call(ctx=Context(num_pages=0)) == BAD              # nothing is backed


def test_null_contexts_and_descriptors():
    assert kvpub.kvpub_attend(None, 0, 0, queries(), pages(), P, 8192, 512, P, 16, P, 1 << 40) == BAD
    assert kvpub.kvpub_attend(CTX.ptr, 0, 0, None, pages(), P, 8192, 512, P, 16, P, 1 << 40) == BAD
    assert kvpub.kvpub_attend(CTX.ptr, 0, 0, queries(), None, P, 8192, 512, P, 16, P, 1 << 40) == BAD
    assert kvpub.kvpub_attend_slots(None, 0, 0, queries(), P, 70, 70, P, 8192, 512, P, 16, P, 1 << 40) == BAD
    assert kvpub.kvpub_attend_slots(CTX.ptr, 0, 0, None, P, 70, 70, P, 8192, 512, P, 16, P, 1 << 40) == BAD
    assert kvpub.kvpub_attend_weights(None, 0, 0, queries(), pages(), P, 16, P, P, 1200) == BAD
    assert kvpub.kvpub_attend_weights(CTX.ptr, 0, 0, None, pages(), P, 16, P, P, 1200) == BAD
    assert kvpub.kvpub_attend_weights(CTX.ptr, 0, 0, queries(), None, P, 16, P, P, 1200) == BAD
    assert kvpub.kvpub_evict(None, 0, evict_io(), P, 1 << 40) == kvpub.kvpub_evict(CTX.ptr, 0, None, P, 1 << 40) == BAD
    assert kvpub.kvpub_attend_expanded(None, expanded_io()) == kvpub.kvpub_attend_expanded(CTX.ptr, None) == BAD
    assert evict(layer=3) == evict(ctx=Context(num_pages=0)) == BAD


@pytest.mark.parametrize("call", [attend, slots, weights])
@pytest.mark.parametrize("field,value", [
    ("q_latent", 0), ("q_latent", P + 8), ("q_rope", 0), ("q_rope", P + 2),
    ("q_latent_token_stride", -512), ("q_latent_token_stride", 8196), ("q_latent_token_stride", LIMIT),
    ("q_latent_head_stride", 504), ("q_latent_head_stride", 516), ("q_latent_head_stride", LIMIT),
    ("q_rope_token_stride", -8), ("q_rope_token_stride", 1028), ("q_rope_head_stride", 56), ("q_rope_head_stride", 68),
    ("num_tokens", -1), ("num_tokens", (1 << 24) + 1), ("num_heads", 0), ("num_heads", 129),
    ("scale", math.nan), ("scale", math.inf), ("scale", 3e38),
])
def test_refused_queries(call, field, value):
    assert call(queries(**{field: value})) == BAD


@pytest.mark.parametrize("call", [attend, weights])
@pytest.mark.parametrize("change", [
    dict(kv_len=0), dict(kv_len=P + 2), dict(page_table=0), dict(page_table=P + 1), dict(q_start=P + 2),
    dict(page_table_stride=18), dict(page_table_stride=LIMIT), dict(page_table_stride=-20),
    dict(num_seqs=65537), dict(max_q_len=0), dict(max_kv_len=(1 << 30) + 1),
    dict(tree_mask=P), dict(tree_words=1), dict(tree_mask=P, tree_words=65), dict(tree_mask=P + 4, tree_words=1),
    dict(q_start=0, num_seqs=7),                                   # one token a sequence: 6 tokens
    dict(num_seqs=65536, max_kv_len=1 << 30, page_table_stride=1 << 24, max_q_len=1),   # 2^40 tiles
])
def test_refused_pages(call, change):
    kw = dict(stride=1 << 30) if call is weights else {}
    assert call(g=pages(**change), **kw) == BAD


@pytest.mark.parametrize("call", [attend, slots])
@pytest.mark.parametrize("change", [
    dict(out=None), dict(out=P + 8), dict(token=504), dict(token=8196), dict(token=0), dict(head=504), dict(head=516),
    dict(token=LIMIT), dict(head=LIMIT), dict(lse=P + 2), dict(lse_token=15), dict(lse_token=-16), dict(lse_token=LIMIT),
    dict(ws=None), dict(ws=P + 8), dict(size=0),
])
def test_refused_outputs_and_workspaces(call, change):
    assert call(**change) == BAD


def test_a_workspace_of_exactly_the_size_is_taken():
    q, g = queries(), pages()
    size = kvpub.kvpub_attend_workspace(q, g)
    assert attend(q, g, size=size) == PASSED and attend(q, g, size=size - 1) == BAD
    size = kvpub.kvpub_attend_slots_workspace(q, 70)
    assert slots(q, size=size) == PASSED and slots(q, size=size - 1) == BAD
    size = kvpub.kvpub_evict_workspace(evict_io())
    assert evict(size=size) == PASSED and evict(size=size - 1) == BAD


@pytest.mark.parametrize("change", [
    dict(slots=None), dict(slots=P + 4), dict(stride=69), dict(stride=LIMIT), dict(n=(1 << 24) + 1, stride=1 << 25),
    dict(n=1 << 24, stride=1 << 24, q=kvpub.queries(P, P, 1 << 24, 16, 0.07)),            # 2^42 tiles
])
def test_refused_slots(change):
    assert slots(**change) == BAD


@pytest.mark.parametrize("change", [
    dict(lse=None), dict(lse=P + 2), dict(lse_token=15), dict(lse_token=LIMIT), dict(w_out=None), dict(w_out=P + 2),
    dict(w_in=P + 1), dict(stride=1199), dict(stride=LIMIT),
])
def test_refused_weights(change):
    assert weights(**change) == BAD


@pytest.mark.parametrize("change", [
    *[{f: v} for f in ("weights_in", "weights_out", "kv_len", "page_table", "dst_table", "kept", "new_len") for v in (0, P + 2)],
    dict(weights_stride=1199), dict(weights_stride=LIMIT), dict(kept_stride=299), dict(kept_stride=LIMIT),
    dict(page_table_stride=18), dict(page_table_stride=LIMIT), dict(dst_table_stride=4), dict(dst_table_stride=LIMIT),
    dict(dst_table=P, dst_table_stride=21),                        # in place with strides that differ
    dict(new_len=P),                                               # kv_len itself
    dict(num_seqs=65537), dict(max_kv_len=0), dict(max_kv_len=(1 << 30) + 1), dict(budget=0), dict(budget=(1 << 30) + 1),
    dict(first=237, last=64), dict(first=0xFFFFFFFF, last=2), dict(reserved=1),
])
def test_refused_evictions(change):
    assert evict(evict_io(**change)) == BAD


@pytest.mark.parametrize("change", [
    *[{f: v} for f in ("q_nope", "q_rope", "k_nope", "k_rope", "v", "out") for v in (0, P + 8)],
    *[{f: v} for f in ("q_start", "k_start") for v in (0, P + 2)],
    *[{f + "_token_stride": v} for f in ("q_nope", "q_rope", "k_nope", "k_rope", "v", "out") for v in (-8, 2052, LIMIT)],
    dict(q_nope_head_stride=120), dict(q_rope_head_stride=56), dict(k_nope_head_stride=124), dict(v_head_stride=120),
    dict(out_head_stride=120), dict(out_token_stride=120),
    dict(lse=P + 2), dict(lse_token_stride=15), dict(num_tokens=-1), dict(num_tokens=(1 << 24) + 1), dict(num_keys=-1),
    dict(num_keys=(1 << 24) + 1), dict(num_seqs=65536), dict(num_heads=0), dict(num_heads=129), dict(max_q_len=0),
    dict(causal=2), dict(scale=math.nan), dict(scale=-math.inf), dict(reserved=1),
])
def test_refused_expanded(change):
    assert expanded(expanded_io(**change)) == BAD


def test_workspaces_of_invalid_descriptors_are_empty():
    assert kvpub.kvpub_attend_workspace(None, pages()) == kvpub.kvpub_attend_workspace(queries(), None) == 0
    assert kvpub.kvpub_attend_workspace(queries(num_heads=129), pages()) == 0
    assert kvpub.kvpub_attend_workspace(queries(), pages(max_q_len=0)) == 0
    assert kvpub.kvpub_attend_slots_workspace(None, 5) == kvpub.kvpub_attend_slots_workspace(queries(num_heads=0), 5) == 0
    assert kvpub.kvpub_evict_workspace(None) == kvpub.kvpub_evict_workspace(evict_io(budget=0)) == 0


def test_workspaces_grow_with_every_size():
    """A workspace sized for the largest call serves every smaller one."""
    rng = random.Random(5)
    pick = lambda top: min(top, int(2 ** rng.uniform(0, math.log2(top) + 1)))

    def paged(v):
        return kvpub.kvpub_attend_workspace(kvpub.queries(P, P, v["t"], v["h"], 1.0),
                                            kvpub.pages(P, P, 1 << 24, v["s"], v["kv"], q_start=P, max_q_len=v["q"]))

    def listed(v):
        return kvpub.kvpub_attend_slots_workspace(kvpub.queries(P, P, v["t"], v["h"], 1.0), v["kv"])

    def evicted(v):
        return kvpub.kvpub_evict_workspace(evict_io(num_seqs=v["s"], max_kv_len=v["kv"]))

    for _ in range(3000):
        v = dict(t=pick(5000), h=pick(128), s=pick(700), kv=pick(200000), q=pick(600))
        k = rng.choice(list(v))
        w = dict(v, **{k: min(v[k] + pick(2 * v[k]), 128 if k == "h" else 1 << 24)})
        for f in (paged, listed, evicted):
            assert 0 < f(v) <= f(w), (f.__name__, v, w)
