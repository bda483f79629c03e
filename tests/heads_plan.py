"""How kvpub_heads_attend cuts a call (plan_heads_attend), from the constants in the kernel's source: what the tests of its
kernels expect beside their sizes, so that a changed constant cannot quietly send them elsewhere."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "replicated_fp8_sparse_amd", "csrc",
                      "heads_attend_kernel.hip")


def constants():
    with open(SOURCE) as f:
        found = dict(re.findall(r"\b(k[A-Z]\w*) = (\d+)\b", " ".join(re.findall(r"^constexpr uint32_t ([^;]*);", f.read(), re.M))))
    return {k: int(v) for k, v in found.items()}


def unit_places(rows, group, seqs, tokens, max_q):
    return min((tokens * group >> (rows.bit_length() - 1)) + seqs, seqs * -(-max_q * group // rows))


def plan(G, H, D, n, max_kv, seqs=None, tokens=None, max_q=None):
    """(rows of a unit, cuts, blocks of one cut) of a call with n[b] tokens a sequence."""
    k, group = constants(), H // G
    seqs, tokens, max_q = seqs or len(n), tokens or int(sum(n)), max_q or int(max(n))
    rows = max_q * group
    R = 16 if rows <= 16 else 32 if rows <= 32 or D == 256 else 64
    if R == 64 and unit_places(64, group, seqs, tokens, max_q) * G < k["kFull"] * (2 if D == 64 else 1):
        R = 32
    blocks = max(1, unit_places(R, group, seqs, tokens, max_q) * G)
    cuts = lambda most, wanted: min(most, k["kMostChunks"], wanted // blocks)
    each, cut = max(k["kChunk"], min(rows, R) * k["kChunkRows"]), 1
    if max_kv > k["kWhole"] and R < 64:
        cut = max(cut, cuts(-(-max_kv // each), k["kWanted"] if R == 16 else k["kWantedWide"]))
        cut = max(cut, cuts(-(-max_kv // k["kLeastChunk"]), k["kFill"]))
        cut = max(cut, cuts(max_kv // (2 * k["kChunk"]), 2 * k["kFill"]))
    chunk = max(k["kLeastChunk"], -(-(-(-max_kv // cut)) // 128) * 128)
    return R, max(1, -(-max_kv // chunk)), blocks
