"""What the source of the store with rotations has to keep, where a run shows it by chance only (no GPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "replicated_fp8_sparse_amd", "csrc")


def test_one_thread_reads_the_status_for_waves_that_share_a_token():
    """The status may change while a block runs: waves that read it for themselves could store a part of a token's rows.
    (The window is some 100 ns once in a context's life, which test_gpu_store_rotated_poison.py seldom meets.)"""
    with open(os.path.join(CSRC, "store_rotated_kernel.hip")) as f:
        reads = [line for line in f if re.search(r"p\.s\.head\b", line)]
    assert reads and all("if (!Split || threadIdx.x == 0)" in line for line in reads), reads
