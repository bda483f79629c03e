"""kvpub_rotate's angles: what a rotation of (1, 0) gives, cosine and sine, over angles of every size."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import heads_util as U

pytestmark = pytest.mark.gpu


def along_the_circle():
    """(error along the circle, rest of the angle beside the nearest quarter turn, radians) of 2^22 rotations of (1, 0)."""
    T, D = 8192, 1024
    rng = np.random.default_rng(8)
    turns = rng.integers(0, 2 ** 63, D // 2, dtype=np.uint64)
    pos = rng.integers(1, 2 ** 20, T)
    pos[::2] *= -1
    ctx = U.Context()
    try:
        table = torch.from_numpy(turns.view(np.int64)).cuda()
        rot = kvpub.rotation(table.data_ptr(), D)
        x = torch.zeros(T, 1, D, device="cuda")
        x[..., 0::2] = 1.0
        y, d_pos = torch.empty_like(x), U.i32(pos)
        io = kvpub.rotate_io(x.data_ptr(), y.data_ptr(), d_pos.data_ptr(), rot, T, 1, D, kvpub.FP32)
        kvpub.check(kvpub.kvpub_rotate(ctx.ctx, io, U.stream()), "kvpub_rotate")
        got = y.view(T, D // 2, 2).cpu().numpy().astype(np.longdouble)
    finally:
        ctx.free()
    tau = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))
    angle = (pos[:, None].astype(np.int64).view(np.uint64) * turns[None]).view(np.int64).astype(np.longdouble) / 2.0 ** 64
    a, rest = angle * tau, (angle - np.round(angle * 4) / 4) * tau
    return np.cos(a) * (got[..., 1] - np.sin(a)) - np.sin(a) * (got[..., 0] - np.cos(a)), rest


def test_angles_are_rounded_and_not_cut_off():
    """To a multiple of 2^-32 turns: cut off they would be 2^-33 turns, 7.3e-10, low in the mean; roundings of some 2^-25 over
    2^22 angles leave 2^-25 / 2^11 = 1.5e-11 of one step in the mean."""
    along, _ = along_the_circle()
    assert abs(float(along.mean())) <= 8 * 2.0 ** -36, float(along.mean())


def test_the_angle_has_no_error_of_its_own():
    """Sine and cosine are taken at a rest x of at most an eighth of a turn beside the nearest quarter.  Their error along the
    circle is rounding, which averages out, and x times the relative error of the factor that makes radians of x, which
    does not: a binary32 number, so half a step of 2 pi 2^-34, 2^-56 / (2 pi 2^-34) = 3.8e-8 of it, at most.  Over 2^22
    angles roundings of some 2^-25 leave less than 2^-25 / 2^11 / 0.45 (x's own spread), and what is cut off each angle,
    2^-32 turns, does not go with x: 1e-10 is allowed for both."""
    along, rest = along_the_circle()
    factor = float((along * rest).sum() / (rest * rest).sum())
    assert abs(factor) <= 2.0 ** -56 / (2 * np.pi * 2.0 ** -34) + 1e-10, factor
    assert float(np.abs(along).max()) <= 4 * 2.0 ** -24
