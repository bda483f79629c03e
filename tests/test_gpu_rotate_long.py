"""kvpub_rotate with more tokens than a launch has rows of blocks: a block takes a second token."""
import numpy as np
import pytest
import torch

import heads_util as U
from test_gpu_rotate import check, rows, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,T,H,tokens", [("fp32", 65600, 2, 1), ("bf16", 131200, 4, 2), ("fp16", 131200, 4, 2)])
@pytest.mark.parametrize("halves", [False, True])
def test_blocks_that_take_two_tokens(kind, T, H, tokens, halves):
    """Heads of 1024 values are 128 threads, so a block of 256 holds two heads of a token (binary32), or, with four heads
    a thread, two tokens: 65,535 such rows of blocks are a launch's most."""
    assert T > 65535 * tokens
    ctx = U.Context()
    try:
        rot = U.Rotation(1000, 16, halves, 0.75)
        _, x = rows(T, H, 1024, kind, seed=H)
        y = torch.full_like(x, U.SENTINEL)
        pos = np.random.default_rng(T).integers(0, 2 ** 20, T)
        run(ctx, x, y, U.i32(pos), rot, kind)
        edge = 65535 * tokens
        pick = np.r_[0:20, edge - 20:edge + 20, T - 20:T]
        want, bound = rot.apply(x[pick], pos[pick])
        check(y[pick], want, bound, x.dtype)
        assert torch.equal(y[..., :16], x[..., :16]) and torch.equal(y[..., 1016:], x[..., 1016:])      # copied, in every token
    finally:
        ctx.free()
