"""Argument checks of the rotations and of the cache of heads, on the host.

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
LIMIT = 2 ** 31


class Lazy:
    """Built by the first call: collecting these tests loads no library."""
    buf = None

    @property
    def ptr(self):
        if self.buf is None:
            cfg = kvpub.kvpub_config_init(2, 3, 100)
            cfg.device = 1 << 20
            self.buf = ctypes.create_string_buffer(1 << 16)
            ctypes.memmove(self.buf, ctypes.byref(cfg), ctypes.sizeof(cfg))
        return ctypes.addressof(self.buf)


CTX = Lazy()


def change(s, kw):
    for k, v in kw.items():
        o = s
        *path, k = k.split("__")
        for x in path:
            o = getattr(o, x)
        if isinstance(k, str) and k.startswith("bases") and k != "bases":
            o.bases[int(k[5:])] = v
        else:
            setattr(o, k, v)
    return s


def rotation(**kw):
    return change(kvpub.rotation(P, 64, 0, 0, 1.0), kw)


def rotate_io(**kw):
    return change(kvpub.rotate_io(P, 2 * P, P, rotation(), 6, 16, 192, kvpub.BF16), kw)


def rotate(io=None):
    return kvpub.kvpub_rotate(CTX.ptr, io or rotate_io())


def store(layer=2, T=6, lat=P, ls=512, rp=P, rs=64, ix=P, xs=128, slots=P, pos=P, rr=True, ri=True):
    make = lambda r: rotation() if r is True else r
    return kvpub.kvpub_store_rotated(CTX.ptr, layer, T, lat, ls, rp, rs, ix, xs, slots, pos, make(rr), make(ri))


def heads(**kw):
    return change(kvpub.heads([P, 2 * P], 100, 8, 128, num_layers=3), kw)


def rows(**kw):
    return change(kvpub.heads_rows(P, P, 6, kvpub.BF16, 2048, 128, 2048, 128), kw)


def pages(**kw):
    return change(kvpub.pages(P, P, 20, 3, 1200, q_start=P, max_q_len=4), kw)


def append(c=None, r=None, g=None, rot=True, pos=P, layer=2):
    return kvpub.kvpub_heads_append(CTX.ptr, c or heads(), layer, r or rows(), g or pages(), rotation() if rot is True else rot, pos)


def queries(**kw):
    return change(kvpub.heads_queries(P, 2 * P, P, 6, 32, 128, 0.1, kvpub.BF16), kw)


def attend(c=None, q=None, g=None, replica=1, layer=2, ws=P, size=1 << 40):
    return kvpub.kvpub_heads_attend(CTX.ptr, c or heads(), replica, layer, q or queries(), g or pages(), ws, size)


def workspace(c=None, q=None, g=None):
    return kvpub.kvpub_heads_attend_workspace(c or heads(), q or queries(), g or pages())


def test_struct_sizes_and_offsets_match_the_header(tmp_path):
    names = ["kvpub_rotation", "kvpub_rotation_config", "kvpub_rotate_io", "kvpub_heads", "kvpub_heads_rows", "kvpub_heads_queries"]
    src = ["#include <stddef.h>", "#include <stdio.h>", '#include "kvpub.h"', "int main(void) {"]
    for n in names:
        src.append(f'printf("%zu\\n", sizeof({n}));')
        src += [f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in getattr(kvpub, n)._fields_]
    for g, d in ((1, 64), (3, 128), (8, 256), (128, 256), (7, 64)):
        src.append(f'printf("%zu\\n", (size_t)KVPUB_HEADS_PAGE_BYTES({g}, {d}));')
    (tmp_path / "sizes.c").write_text("\n".join(src + ["return 0; }", ""]))
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "sizes.c"), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for n in names:
        s = getattr(kvpub, n)
        want += [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    want += [kvpub.heads_page_bytes(g, d) for g, d in ((1, 64), (3, 128), (8, 256), (128, 256), (7, 64))]
    assert got == want


def test_calls_that_pass_every_check():
    assert rotate() == store() == append() == attend() == PASSED
    assert rotate(rotate_io(y=P)) == PASSED                                              # in place
    assert rotate(rotate_io(x_token_stride=0)) == PASSED                                 # one row for all tokens
    assert rotate(rotate_io(num_heads=1, x_head_stride=0, y_head_stride=0)) == PASSED
    assert rotate(rotate_io(rotation__start=128, type=kvpub.FP32, transpose=1)) == PASSED
    assert rotate(rotate_io(num_tokens=1, y_token_stride=0)) == PASSED
    assert store(rr=None) == store(ri=None) == PASSED
    assert store(rr=None, ri=None, pos=None) == PASSED                                   # kvpub_store
    assert store(ri=rotation(dim=128)) == PASSED
    assert append(rot=None, pos=None) == append(pos=None) == append(g=pages(q_start=0)) == PASSED
    assert append(rot=None, pos=3) == PASSED                                             # not read
    assert append(heads(num_layers=1, layer_stride=0), layer=0) == PASSED
    assert attend(q=queries(lse=None, lse_token_stride=0)) == PASSED
    assert attend(g=pages(tree_mask=P, tree_words=64)) == attend(g=pages(q_start=0)) == PASSED
    assert attend(q=queries(type=kvpub.FP16, num_heads=1024, lse_token_stride=1024)) == PASSED


def test_nothing_to_do_is_no_error():
    assert rotate(rotate_io(num_tokens=0, x=0, y=0, positions=0)) == OK
    assert store(T=0, lat=None, rp=None, ix=None, slots=None, pos=None) == OK
    assert append(r=rows(num_tokens=0, k=0, v=0)) == append(g=pages(num_seqs=0, kv_len=0, page_table=0)) == OK
    assert attend(q=queries(num_tokens=0, q=0, out=0), ws=None, size=0) == attend(g=pages(num_seqs=0), ws=None, size=0) == OK
    assert workspace(q=queries(num_tokens=0)) == workspace(g=pages(num_seqs=0)) == 0


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(y=0), dict(x=P + 8), dict(y=P + 8), dict(positions=0), dict(positions=P + 2),
    dict(x_token_stride=12), dict(x_head_stride=184), dict(x_head_stride=196), dict(y_token_stride=184), dict(y_token_stride=0),
    dict(y_head_stride=184), dict(x_token_stride=LIMIT), dict(y_head_stride=LIMIT), dict(x_token_stride=-8),
    dict(y=P, y_token_stride=32 * 192), dict(y=P, y_head_stride=200),
    dict(num_tokens=-1), dict(num_tokens=2 ** 24 + 1), dict(num_heads=0), dict(num_heads=1025), dict(head_dim=0), dict(head_dim=1032),
    dict(head_dim=60), dict(type=3), dict(transpose=2),
    dict(rotation__turns=0), dict(rotation__turns=P + 4), dict(rotation__dim=0), dict(rotation__dim=4), dict(rotation__dim=60),
    dict(rotation__dim=200), dict(rotation__start=4), dict(rotation__start=136), dict(rotation__start=2 ** 32 - 8), dict(rotation__layout=2),
    dict(rotation__magnitude=math.inf), dict(rotation__magnitude=math.nan)])
def test_rotate_refuses(kw):
    assert rotate(rotate_io(**kw)) == BAD


@pytest.mark.parametrize("kw", [
    dict(layer=3), dict(T=-1), dict(lat=None), dict(rp=P + 8), dict(ix=None), dict(slots=None), dict(slots=P + 4), dict(ls=504),
    dict(rs=60), dict(xs=LIMIT), dict(pos=None), dict(pos=P + 2),
    dict(rr=(72, 0)), dict(rr=(64, 8)), dict(ri=(128, 8)), dict(ri=(136, 0)), dict(ri=(12, 0))])
def test_store_rotated_refuses(kw):
    kw = {k: rotation(dim=v[0], start=v[1]) if isinstance(v, tuple) else v for k, v in kw.items()}
    assert store(**kw) == BAD


HEADS_BAD = [dict(num_replicas=0), dict(num_replicas=9), dict(num_layers=0), dict(num_kv_heads=0), dict(num_kv_heads=129), dict(head_dim=32),
             dict(head_dim=96), dict(head_dim=512), dict(num_pages=0), dict(num_pages=LIMIT), dict(page_stride=8 * 16384),
             dict(page_stride=8 * 16384 + 24), dict(layer_stride=99 * (8 * 16384 + 16)), dict(layer_stride=200 * 8 * 16384 + 8),
             dict(bases0=0), dict(bases1=P + 8)]
PAGES_BAD = [dict(kv_len=0), dict(page_table=0), dict(kv_len=P + 2), dict(page_table=P + 1), dict(q_start=P + 2), dict(page_table_stride=18),
             dict(page_table_stride=LIMIT), dict(num_seqs=65537), dict(max_q_len=0), dict(max_kv_len=2 ** 30 + 1),
             dict(tree_words=1), dict(tree_mask=P), dict(tree_mask=P, tree_words=65), dict(tree_mask=P + 4, tree_words=1),
             dict(q_start=0, num_seqs=7)]


@pytest.mark.parametrize("kw", HEADS_BAD)
def test_bad_caches_are_refused(kw):
    assert append(heads(**kw)) == BAD and attend(heads(**kw)) == BAD and workspace(heads(**kw)) == 0


@pytest.mark.parametrize("kw", PAGES_BAD)
def test_bad_pages_are_refused(kw):
    assert append(g=pages(**kw)) == BAD and attend(g=pages(**kw)) == BAD


@pytest.mark.parametrize("kw", [
    dict(k=0), dict(v=0), dict(k=P + 8), dict(v=P + 2), dict(k_token_stride=12), dict(k_head_stride=120), dict(v_head_stride=64),
    dict(v_token_stride=LIMIT), dict(num_tokens=-1), dict(num_tokens=2 ** 24 + 1), dict(type=kvpub.FP32), dict(reserved=1)])
def test_append_refuses(kw):
    assert append(r=rows(**kw)) == BAD


def test_append_refuses_the_rest():
    assert append(layer=3) == append(pos=P + 2) == append(rot=rotation(dim=136)) == append(rot=rotation(start=72)) == BAD
    assert kvpub.kvpub_heads_append(None, heads(), 0, rows(), pages()) == BAD
    assert kvpub.kvpub_heads_append(CTX.ptr, None, 0, rows(), pages()) == BAD
    assert kvpub.kvpub_heads_append(CTX.ptr, heads(), 0, None, pages()) == BAD
    assert kvpub.kvpub_heads_append(CTX.ptr, heads(), 0, rows(), None) == BAD
    assert kvpub.kvpub_rotate(None, rotate_io()) == kvpub.kvpub_rotate(CTX.ptr, None) == BAD
    assert kvpub.kvpub_store_rotated(None, 0, 1, P, 512, P, 64, P, 128, P, P, rotation(), None) == BAD


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(out=0), dict(q=P + 8), dict(out=P + 8), dict(lse=P + 2), dict(q_token_stride=4), dict(q_head_stride=120),
    dict(out_token_stride=120), dict(out_head_stride=64), dict(out_head_stride=132), dict(lse_token_stride=31), dict(lse_token_stride=LIMIT),
    dict(num_tokens=-1), dict(num_tokens=2 ** 24 + 1), dict(num_heads=0), dict(num_heads=12), dict(num_heads=1032), dict(type=2),
    dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38), dict(reserved=1)])
def test_attend_refuses(kw):
    assert attend(q=queries(**kw)) == BAD


def test_attend_refuses_the_rest():
    assert attend(replica=2) == attend(layer=3) == BAD
    assert attend(heads(num_kv_heads=1), queries(num_heads=129)) == BAD                       # 128 query heads to a key-value head at most
    size = workspace()
    assert size > 0 and attend(size=size) == PASSED
    assert attend(size=size - 1) == attend(ws=None) == attend(ws=P + 8) == BAD
    assert kvpub.kvpub_heads_attend(None, heads(), 0, 0, queries(), pages(), P, 1 << 40) == BAD
    assert kvpub.kvpub_heads_attend(CTX.ptr, None, 0, 0, queries(), pages(), P, 1 << 40) == BAD
    assert kvpub.kvpub_heads_attend(CTX.ptr, heads(), 0, 0, None, pages(), P, 1 << 40) == BAD
    assert kvpub.kvpub_heads_attend(CTX.ptr, heads(), 0, 0, queries(), None, P, 1 << 40) == BAD
    assert kvpub.kvpub_heads_attend_workspace(None, queries(), pages()) == kvpub.kvpub_heads_attend_workspace(heads(), None, pages()) == 0


def test_workspace_grows_with_every_bound():
    rng = random.Random(5)
    pick = lambda hi: int(round(math.exp(rng.uniform(0, math.log(hi)))))
    for _ in range(3000):
        G, group = pick(128), pick(128)
        if G * group > 1024:
            continue
        a = dict(T=pick(2 ** 24), seqs=pick(65536), q=pick(2 ** 24), kv=pick(2 ** 30), D=rng.choice([64, 128, 256]))

        def size(T, seqs, q, kv, D, G=G, group=group):
            return workspace(heads(num_kv_heads=G, head_dim=D, page_stride=kvpub.heads_page_bytes(128, 256), layer_stride=1 << 40),
                             queries(num_tokens=T, num_heads=G * group), pages(num_seqs=seqs, max_q_len=q, max_kv_len=kv))
        base = size(**a)
        assert base > 0
        for k, top in (("T", 2 ** 24), ("seqs", 65536), ("q", 2 ** 24), ("kv", 2 ** 30)):
            more = dict(a)
            more[k] = min(top, a[k] + pick(top))
            assert size(**more) >= base, (a, more, G, group)
        if a["D"] < 256:
            assert size(**dict(a, D=2 * a["D"])) >= base
        if (G + 1) * group <= 1024 and G < 128:
            assert size(**a, G=G + 1) >= base
        if G * (group + 1) <= 1024 and group < 128:
            assert size(**a, group=group + 1) >= base
