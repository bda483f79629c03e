"""kvpub_rotate against the rotation in 64 bits, at the sizes, strides and positions where it can go wrong."""
import numpy as np
import pytest
import torch

from replicated_fp8_sparse_amd import kvpub

import heads_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = U.Context()
    yield c
    c.free()


def rows(T, H, width, kind, seed=0, pad=0, head_pad=0):
    """[T, H, width] inside a larger buffer of sentinels."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 3)
    buf = torch.full((T + 1, H, width + head_pad), U.SENTINEL, dtype=U.TYPES[kind][0], device="cuda")
    if pad:
        buf = torch.cat([buf.view(T + 1, -1), torch.full((T + 1, pad), U.SENTINEL, dtype=buf.dtype, device="cuda")], 1)
    else:
        buf = buf.view(T + 1, -1)
    view = buf[:T].as_strided((T, H, width), (buf.shape[1], width + head_pad, 1))
    view.copy_(torch.randn((T, H, width), generator=g, device="cuda"))
    return buf, view


def check(got, want, bound, dtype, what=""):
    tol = bound + U.half_step(dtype) * want.abs() + torch.finfo(dtype).smallest_normal * U.half_step(dtype) * 2
    worst = ((got.double().cpu() - want).abs() / tol).max().item()
    assert worst <= 1, f"{what}: off by {worst} of its bound"


def run(ctx, x, y, pos, rot, kind, transpose=0):
    T, H, w = x.shape
    io = kvpub.rotate_io(x.data_ptr(), y.data_ptr(), pos.data_ptr(), rot.struct, T, H, w, U.TYPES[kind][1], x_token_stride=x.stride(0),
                         x_head_stride=x.stride(1), y_token_stride=y.stride(0), y_head_stride=y.stride(1), transpose=transpose)
    kvpub.check(kvpub.kvpub_rotate(ctx.ctx, io, U.stream()), "kvpub_rotate")


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("T,H,width,dim,start,pad,head_pad", [
    (1, 1, 8, 8, 0, 0, 0), (1, 16, 64, 64, 0, 0, 128), (5, 3, 80, 24, 16, 8, 0), (7, 128, 128, 48, 72, 0, 8), (3, 1, 1024, 1024, 0, 0, 0),
    (300, 100, 96, 40, 56, 16, 0), (6000, 5, 64, 32, 8, 0, 0), (9000, 3, 64, 64, 0, 8, 0), (9, 1000, 64, 64, 0, 0, 0), (2, 7, 1000, 8, 992, 0, 0), (700, 33, 256, 256, 0, 0, 0)])
def test_rotation(ctx, T, H, width, dim, start, pad, head_pad, halves, kind):
    rng = np.random.default_rng(T + H)
    pos = rng.integers(0, 2 ** 20, T)
    pos[:1] = 2 ** 31 - 1
    pos[-1:] = -12345
    rot = U.Rotation(dim, start, halves, 1.25)
    xb, x = rows(T, H, width, kind, pad=pad, head_pad=head_pad)
    yb, y = rows(T, H, width, kind, seed=1, pad=pad, head_pad=head_pad)
    before = xb.clone()
    d_pos = U.i32(pos)
    run(ctx, x, y, d_pos, rot, kind)
    want, bound = rot.apply(x, pos)
    check(y, want, bound, x.dtype)
    assert torch.equal(xb, before)
    rest = [k for k in range(width) if not start <= k < start + dim]
    assert torch.equal(y[..., rest], x[..., rest])
    y.copy_(torch.full_like(y, U.SENTINEL))
    assert bool((yb == U.SENTINEL).all())                      # nothing between or behind the rows
    # in place, transposed: what the kernel writes elsewhere, in the same bits
    run(ctx, x, y, d_pos, rot, kind, transpose=1)
    want, bound = rot.apply(x, pos, transpose=True)
    check(y, want, bound, x.dtype, "transposed")
    run(ctx, x, x, d_pos, rot, kind, transpose=1)
    assert torch.equal(x, y)
    x.copy_(torch.full_like(x, U.SENTINEL))
    assert bool((xb == U.SENTINEL).all())


def test_no_tokens_and_more_tokens_than_a_grid_has_rows(ctx):
    rot = U.Rotation(8)
    x = torch.ones(4, 1, 8, dtype=torch.bfloat16, device="cuda")
    io = kvpub.rotate_io(x.data_ptr(), x.data_ptr(), U.i32([0] * 4).data_ptr(), rot.struct, 0, 1, 8, kvpub.BF16)
    kvpub.check(kvpub.kvpub_rotate(ctx.ctx, io, U.stream()))
    assert bool((x == 1).all())
    T = 150001
    _, x = rows(T, 1, 16, "fp32")
    pos = np.arange(T)
    y = torch.zeros(T, 1, 16, device="cuda")
    run(ctx, x, y, U.i32(pos), rot, "fp32")
    pick = np.r_[0:100, 65500:65600, 131000:131100, T - 100:T]
    want, bound = rot.apply(x[pick], pos[pick])
    check(y[pick], want, bound, torch.float32)


def test_wide_rows_of_many_heads(ctx):
    """1024 heads of 1024 values: 512 blocks a token, so several launches' worth of tokens share a grid row."""
    rot = U.Rotation(1024, halves=True)
    _, x = rows(40, 1024, 1024, "bf16")
    y = torch.zeros_like(x)
    pos = np.arange(40) * 1000
    run(ctx, x, y, U.i32(pos), rot, "bf16")
    want, bound = rot.apply(x[:, ::97], pos)
    check(y[:, ::97], want, bound, torch.bfloat16)


def test_one_row_for_all_tokens(ctx):
    rot = U.Rotation(32, 8, True)
    _, x = rows(1, 4, 64, "bf16")
    pos = np.array([0, 5, 100000])
    y = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    run(ctx, x.expand(3, 4, 64), y, U.i32(pos), rot, "bf16")
    want, bound = rot.apply(x.expand(3, 4, 64), pos)
    check(y, want, bound, torch.bfloat16)


def test_a_value_that_is_not_finite_reaches_its_own_pair_only(ctx):
    for halves in (False, True):
        rot = U.Rotation(64, 0, halves)
        _, x = rows(2, 2, 72, "bf16")
        want, bound = rot.apply(x, [3, 4])
        j, k = rot.parts()
        x[0, 0, j[5]], x[1, 1, k[9]], x[1, 0, 70] = float("nan"), float("inf"), float("nan")
        y = torch.zeros_like(x)
        run(ctx, x, y, U.i32([3, 4]), rot, "bf16")
        bad = torch.zeros(2, 2, 72, dtype=torch.bool)
        bad[0, 0, [j[5], k[5]]] = bad[1, 1, [j[9], k[9]]] = bad[1, 0, 70] = True
        assert torch.equal(~torch.isfinite(y).cpu(), bad)
        assert bool(((y.double().cpu() - want).abs() <= bound + 2.0 ** -8 * want.abs() + 1e-30)[~bad].all())


def test_position_zero_and_no_turn_change_nothing(ctx):
    rot = U.Rotation(64)
    _, x = rows(3, 5, 64, "bf16")
    y = torch.zeros_like(x)
    run(ctx, x, y, U.i32([0, 0, 0]), rot, "bf16")
    assert torch.equal(x, y)


def test_the_transpose_is_the_gradient(ctx):
    """<R x, g> = <x, R^T g>, and R^T g against differences of <R x, g> in 32 bits (R is linear: a step of 1 has no
    truncation error, only the roundings of two sums of 2 * 48 terms)."""
    rot = U.Rotation(48, 8, True, 1.5)
    _, x = rows(4, 3, 64, "fp32")
    _, g = rows(4, 3, 64, "fp32", seed=9)
    pos = U.i32([1, 70, 5000, 131071])
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    run(ctx, x, y, pos, rot, "fp32")
    run(ctx, g, dx, pos, rot, "fp32", transpose=1)
    left, right = (y.double() * g.double()).sum().item(), (x.double() * dx.double()).sum().item()
    size = 1.5 * 2 * (x.double().abs() * g.double().abs()).sum().item() + (y.double().abs() * g.double().abs()).sum().item()
    assert abs(left - right) <= 16 * 2.0 ** -24 * size
    for t, h, k in ((0, 0, 8), (1, 2, 31), (2, 1, 40), (3, 0, 55), (3, 2, 60)):
        more, ym = x.clone(), torch.zeros_like(x)
        more[t, h, k] += 1.0
        run(ctx, more, ym, pos, rot, "fp32")
        slope = ((ym.double() - y.double()) * g.double()).sum().item()
        around = x[t, h].double().abs().max().item() + 1
        assert abs(slope - dx[t, h, k].item()) <= 32 * 2.0 ** -24 * 1.5 * 2 * around * g[t, h].double().abs().sum().item()


def test_graph_and_another_stream(ctx):
    rot = U.Rotation(64, halves=True)
    _, x = rows(33, 8, 64, "bf16")
    pos, y = U.i32(np.arange(33)), torch.zeros(33, 8, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(ctx, x, y, pos, rot, "bf16")
    for k in range(3):
        x.copy_(torch.randn_like(x))
        pos += 1000 * k
        graph.replay()
        torch.cuda.synchronize()
        want, bound = rot.apply(x, pos.cpu().numpy())
        check(y, want, bound, torch.bfloat16, f"replay {k}")
