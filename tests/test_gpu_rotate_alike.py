"""kvpub_rotate gives a value the same bits wherever it stands: in any head, in place or not, alone or in a large call."""
import numpy as np
import pytest
import torch

import heads_util as U
from test_gpu_rotate import rows, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("T,H,width,dim,start", [(19, 1000, 208, 112, 32), (300, 61, 128, 128, 0), (5000, 7, 64, 32, 16)])
def test_same_bits_everywhere(T, H, width, dim, start, halves, kind):
    ctx = U.Context()
    try:
        rot, pos = U.Rotation(dim, start, halves, 1.25), np.random.default_rng(T).integers(0, 2 ** 20, T)
        _, x = rows(T, H, width, kind, seed=T)
        x = x.contiguous()
        d_pos, y, z = U.i32(pos), torch.zeros_like(x), torch.zeros_like(x)
        run(ctx, x, y, d_pos, rot, kind)
        run(ctx, x.roll(1, 1), z, d_pos, rot, kind)
        assert torch.equal(z.roll(-1, 1), y), "another head"
        for t in range(0, T, max(1, T // 50)):
            run(ctx, x[t:t + 1], z[t:t + 1], d_pos[t:t + 1], rot, kind)
            assert torch.equal(z[t], y[t]), f"token {t} alone"
        run(ctx, x, x, d_pos, rot, kind)
        assert torch.equal(x, y), "in place"
    finally:
        ctx.free()
