"""The sizes of test_gpu_heads_units.py go to every kernel of kvpub_heads_attend (no GPU)."""
from heads_plan import plan
from test_gpu_heads_units import SIZES


def test_each_kernel_is_among_the_sizes():
    """Units of 64 rows stay whole; the others meet both joins, of up to 16 cuts and of more."""
    got = {(D, rows, 0 if cuts == 1 else 1 if cuts <= 16 else 2) for (rows, cuts), (_, _, D, _, _) in SIZES}
    assert {(D, R) for D, R, _ in got} == {(D, R) for D in (64, 128, 256) for R in (16, 32, 64) if D * R < 256 * 64}
    assert {(D, c) for D, _, c in got} == {(D, c) for D in (64, 128, 256) for c in (0, 1, 2)}
    for want, (G, H, D, n, lens) in SIZES:
        assert plan(G, H, D, n, max(lens))[:2] == want, (G, H, D, n, lens)
