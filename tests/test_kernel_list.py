"""Kernels of the rotations and of the cache of heads in the built library: those that a launch can choose, and no other
(no GPU)."""
import itertools
import re

from replicated_fp8_sparse_amd import kvpub

TYPE = {"DF16b": "bf16", "DF16_": "fp16", "f": "fp32"}


def built(kernel):
    """Template arguments of every instantiation: the names by which the host code registers its kernels."""
    with open(kvpub.LIB_PATH, "rb") as f:
        names = set(re.findall(rb"_ZN5kvpub12_GLOBAL__N_1\d+" + kernel.encode() + rb"I(\w+?)EEvNS", f.read()))
    out = set()
    for n in names:
        args = re.findall(r"DF16b|DF16_|^f|L[bij]\d+E?", n.decode())
        out.add(tuple(TYPE[a] if a in TYPE else int(re.sub(r"\D", "", a)) for a in args))
    return out


def test_rotate():
    want = set(itertools.product(("bf16", "fp16"), (0, 1), (1, 4))) | {("fp32", 0, 1), ("fp32", 1, 1)}
    assert built("rotate_kernel") == want


def test_store_rotated():
    assert built("store_rotated_kernel") == {(1, 0), (0, 0), (0, 1)}


def test_append():
    want = {(t, d, n, r) for t in ("bf16", "fp16") for d, n, r in ((64, 128, 2), (64, 512, 2), (128, 128, 2), (128, 512, 4), (256, 128, 2), (256, 1024, 4))}
    assert built("heads_append_kernel") == want


def test_attend():
    want = {(t, d, rt) for t in ("bf16", "fp16") for d in (64, 128, 256) for rt in (1, 2, 4) if d * rt < 1024}
    assert built("heads_attend_kernel") == want


def test_join():
    assert built("join_kernel") == set(itertools.product(("bf16", "fp16"), (64, 128, 256), (0, 1)))
