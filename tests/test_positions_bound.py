"""The bounds of test_gpu_heads_positions.py hold for keys and queries turned by their own positions, and break where they
are turned by the next one, by none, or without the magnitude (no GPU)."""
import pytest
import torch

import heads_util as U
from positions_bound import key_bound, query_bound
from replicated_fp8_sparse_amd import kvpub


def rotation(dim, halves, magnitude):
    r = U.Rotation.__new__(U.Rotation)
    _, r.turns = kvpub.kvpub_rotation_turns(kvpub.rotation_config(dim))
    r.dim, r.start, r.halves, r.magnitude = dim, 0, halves, magnitude
    return r


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("P", [1, 3, 40, 200])
def test_a_planted_mistake_breaks_them(P, halves):
    g = torch.Generator().manual_seed(P)
    x = torch.randn((P, 2, 128), generator=g).bfloat16().double()
    pos = torch.arange(1, P + 1).numpy()                             # position 0 turns nothing
    rot, plain = rotation(128, halves, 1.1), rotation(128, halves, 1.0)
    want, slack = rot.apply(x, pos)

    def key(y):
        scale = U.power(U.byte_of(y.abs().amax()))
        return bool(((U.e4m3(y / scale) * scale - want).abs() <= key_bound(want, scale, slack, 4)).all())

    def query(y):
        return bool(((y.bfloat16().double() - want).abs() <= query_bound(want, slack)).all())

    assert key(want) and query(want)
    for y in (rot.apply(x, pos + 1)[0], rot.apply(x, pos - 1)[0], plain.apply(x, pos)[0], x):
        assert not key(y) and not query(y)
